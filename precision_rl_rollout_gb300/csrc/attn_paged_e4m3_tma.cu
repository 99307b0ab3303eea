// attn_paged_e4m3_tma.cu -- paged attention over E4M3 caches, pages loaded by the copy engine
// (attn_paged.cuh).
#include "attn_paged.cuh"

namespace fp8rl {

cudaError_t launch_attn_e4m3_tma(const AttnParams& p, cudaStream_t st) {
    return attn::pick<true, true>(p.D, (int64_t)p.Hq / p.Hkv * p.Lq,
                                   [&](auto c) { return attn::launch<decltype(c)>(p, st); });
}

}  // namespace fp8rl
