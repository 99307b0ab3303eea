// attn_paged_bf16.cu -- paged attention over bf16 caches, pages of any size, loaded 16 bytes a thread
// (attn_paged.cuh).
#include "attn_paged.cuh"

namespace fp8rl {

cudaError_t launch_attn_bf16(const AttnParams& p, cudaStream_t st) {
    return attn::pick<false, false>(p.D, (int64_t)p.Hq / p.Hkv * p.Lq,
                                   [&](auto c) { return attn::launch<decltype(c)>(p, st); });
}

}  // namespace fp8rl
