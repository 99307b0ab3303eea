// attn_paged.cu -- the paged attention call: its sizes and its two cache types
// (attn_paged.cuh has the kernels).
#include "attn_paged.cuh"

namespace fp8rl {

size_t attn_paged_workspace_bytes(int64_t B, int64_t Lq, int64_t Hq, int64_t Hkv, int64_t D, int64_t max_len) {
    (void)B;                                   // two slots a CTA, whatever the batch
    const size_t a = plan_attn_paged_bf16(D, Hq / Hkv * Lq, max_len).ws, b = plan_attn_paged_e4m3(D, Hq / Hkv * Lq, max_len).ws;
    return a > b ? a : b;
}

int attn_paged_kernel_count(int64_t B, int64_t Lq, int64_t Hq, int64_t Hkv, int64_t D, int64_t max_len, bool e4m3) {
    (void)B;
    return (e4m3 ? plan_attn_paged_e4m3 : plan_attn_paged_bf16)(D, Hq / Hkv * Lq, max_len).kernels;
}

cudaError_t launch_attn_paged(const AttnParams& a, bool e4m3, cudaStream_t st) {
    AttnParams p = a;
    p.err = device_error_word();
    if (!p.err) return cudaErrorUnknown;
    return e4m3 ? launch_attn_paged_e4m3(p, st) : launch_attn_paged_bf16(p, st);
}

}  // namespace fp8rl
