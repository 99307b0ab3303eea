// attn_paged_bf16_tma.cu -- paged attention over bf16 caches, pages loaded by the copy engine
// (attn_paged.cuh).
#include "attn_paged.cuh"

namespace fp8rl {

cudaError_t launch_attn_bf16_tma(const AttnParams& p, cudaStream_t st) {
    return attn::pick<false, true>(p.D, (int64_t)p.Hq / p.Hkv * p.Lq,
                                   [&](auto c) { return attn::launch<decltype(c)>(p, st); });
}

}  // namespace fp8rl
