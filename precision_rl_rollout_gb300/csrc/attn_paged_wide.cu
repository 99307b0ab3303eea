// attn_paged_wide.cu -- paged attention over bf16 caches for more than 32 query rows a kv
// head (attn_paged_wide.cuh).
#include "attn_paged_wide.cuh"

namespace fp8rl {

cudaError_t launch_attn_wide(const AttnParams& p, cudaStream_t st) {
    return attn::pick_wide(p.D, (int64_t)p.Hq / p.Hkv * p.Lq,
                           [&](auto c) { return attn::launch_wide<decltype(c)>(p, st); });
}

}  // namespace fp8rl
