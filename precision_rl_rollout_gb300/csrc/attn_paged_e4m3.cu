// attn_paged_e4m3.cu -- paged attention over E4M3 caches, pages of any size, loaded 16 bytes a thread
// (attn_paged.cuh).
#include "attn_paged.cuh"

namespace fp8rl {

cudaError_t launch_attn_e4m3(const AttnParams& p, cudaStream_t st) {
    return attn::pick<true, false>(p.D, (int64_t)p.Hq / p.Hkv * p.Lq,
                                   [&](auto c) { return attn::launch<decltype(c)>(p, st); });
}

}  // namespace fp8rl
