// attn_paged_e4m3.cu -- paged attention over E4M3 caches (attn_paged.cuh).
#include "attn_paged.cuh"

namespace fp8rl {

cudaError_t launch_attn_paged_e4m3(const AttnParams& p, cudaStream_t st) {
    return attn::pick<true>(p.D, (int64_t)p.Hq / p.Hkv * p.Lq, [&](auto c) { return attn::launch<decltype(c)>(p, st); });
}
attn::Plan plan_attn_paged_e4m3(int64_t D, int64_t rows, int64_t max_len) {
    return attn::pick<true>(D, rows, [&](auto c) { return attn::plan<decltype(c)>(max_len); });
}

}  // namespace fp8rl
