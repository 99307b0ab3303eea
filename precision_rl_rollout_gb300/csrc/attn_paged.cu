// attn_paged.cu -- the paged attention call: its sizes, and which loader and kernel a
// cache takes (attn_paged.cuh and attn_paged_wide.cuh have the kernels).
#include "attn_paged_wide.cuh"

namespace fp8rl {

namespace {

attn::Plan plan_of(int64_t B, int64_t Lq, int64_t Hq, int64_t Hkv, int64_t D, int64_t max_len, bool e4m3) {
    const int64_t rows = Hq / Hkv * Lq;
    auto f = [&](auto c) { return attn::plan<decltype(c)>(B, Hkv, rows, max_len); };
    if (e4m3) return attn::pick<true, true>(D, rows, f);
    // what either of the kernels for a bf16 cache takes: the pages tell which
    const attn::Plan a = attn::pick<false, false>(D, rows, f);
    if (!attn::is_wide(D, rows)) return a;
    const attn::Plan b = attn::pick_wide(D, rows, [&](auto c) { return attn::plan_wide<decltype(c)>(max_len); });
    return attn::Plan{a.ws > b.ws ? a.ws : b.ws, a.kernels > b.kernels ? a.kernels : b.kernels};
}

// The copy engine loads boxes of 8 tokens or more of one page, by the strides of
// a tensor map; other pages go 16 bytes a thread.
bool copy_engine(const AttnParams& p, bool e4m3) {
    const int64_t es = e4m3 ? 1 : 2, most = (int64_t)1 << 40;
    return p.page_size % 8 == 0 && p.c_token > 0 && (p.c_head > 0 || p.Hkv == 1) && (p.c_page > 0 || p.num_pages == 1) &&
           p.c_token * es < most && p.c_head * es < most && p.c_page * es < most && p.c_token * p.page_size * es < most;
}

}  // namespace

size_t attn_paged_workspace_bytes(int64_t B, int64_t Lq, int64_t Hq, int64_t Hkv, int64_t D, int64_t max_len) {
    const size_t a = plan_of(B, Lq, Hq, Hkv, D, max_len, false).ws, b = plan_of(B, Lq, Hq, Hkv, D, max_len, true).ws;
    return a > b ? a : b;
}

int attn_paged_kernel_count(int64_t B, int64_t Lq, int64_t Hq, int64_t Hkv, int64_t D, int64_t max_len, bool e4m3) {
    return plan_of(B, Lq, Hq, Hkv, D, max_len, e4m3).kernels;
}

cudaError_t launch_attn_paged(const AttnParams& a, bool e4m3, cudaStream_t st) {
    AttnParams p = a;
    p.err = device_error_word();
    if (!p.err) return cudaErrorUnknown;
    const bool engine = copy_engine(p, e4m3);
    // many rows over bf16 by tcgen05, whose operands are as the copy engine lays them
    if (engine && !e4m3 && attn::is_wide(p.D, (int64_t)p.Hq / p.Hkv * p.Lq)) return launch_attn_wide(p, st);
    if (engine) return e4m3 ? launch_attn_e4m3_tma(p, st) : launch_attn_bf16_tma(p, st);
    return e4m3 ? launch_attn_e4m3(p, st) : launch_attn_bf16(p, st);
}

}  // namespace fp8rl
