// attn_paged.cu -- attention of a sequence's new tokens over a paged key-value
// cache.  Query i of Lq stands at position p = len - Lq + i and sees the cached
// tokens j with max(0, p - window + 1) <= j <= p (window 0: from 0 on):
//   o = sum_j exp(x_j - m) v_j / sum_j exp(x_j - m),  x_j = scale q.k_j,
// one pass over the cache with the running maximum m and sum; a query that sees
// nothing gets zeros and a log-sum of -inf.
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace fp8rl {

namespace {

constexpr uint32_t kKernelAttn = 10;
constexpr int kAThreads = 128;
constexpr int kMaxD = 256;

template <bool kE4m3>
__device__ __forceinline__ float cache_value(const void* pool, int64_t at) {
    if constexpr (kE4m3) {
        const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<const uint8_t*>(pool)[at], __NV_E4M3);
        return __half2float(*reinterpret_cast<const __half*>(&h));
    } else {
        return __uint_as_float((uint32_t)static_cast<const uint16_t*>(pool)[at] << 16);
    }
}

// One CTA per (sequence, query, head); each warp takes every fourth token.
template <bool kE4m3>
__global__ void __launch_bounds__(kAThreads)
attn_simple_kernel(const __grid_constant__ AttnParams p) {
    __shared__ float sm[4], sl[4], so[4][kMaxD];
    pdl_wait_then_release();
    const int hq = blockIdx.x % p.Hq, i = (blockIdx.x / p.Hq) % p.Lq, b = blockIdx.x / p.Hq / p.Lq;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, h = hq / (p.Hq / p.Hkv);
    int len = p.lens[b];
    if (len < 0 || len > p.max_len) {
        if (threadIdx.x == 0) atomicCAS(p.err, 0u, (kKernelAttn << 24) | (1u << 16) | 2u);
        len = len < 0 ? 0 : p.max_len;
    }
    const int last = len - p.Lq + i;                                   // this query's position
    const int first = p.window && last >= p.window ? last - p.window + 1 : 0;
    const uint16_t* q = p.q + b * p.q_seq + i * p.q_token + hq * p.q_head;
    const float ks = kE4m3 ? *p.k_scale : 1.f, vs = kE4m3 ? *p.v_scale : 1.f;
    float qv[kMaxD / 32], o[kMaxD / 32] = {}, m = -INFINITY, l = 0.f;
    for (int d = lane, n = 0; d < p.D; d += 32, ++n) qv[n] = __uint_as_float((uint32_t)q[d] << 16) * ks * p.scale;
    for (int j = first + warp; j <= last; j += 4) {
        int page = p.pages[b * p.pages_seq + j / p.page_size];
        if (page < 0 || page >= p.num_pages) {
            if (lane == 0) atomicCAS(p.err, 0u, (kKernelAttn << 24) | (2u << 16) | 2u);
            page = 0;
        }
        const int64_t at = page * p.c_page + (j % p.page_size) * p.c_token + h * p.c_head;
        float x = 0.f;
        for (int d = lane, n = 0; d < p.D; d += 32, ++n) x += qv[n] * cache_value<kE4m3>(p.kpool, at + d);
        for (int off = 16; off; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
        const float mn = fmaxf(m, x), base = mn == -INFINITY ? 0.f : mn;
        const float keep = expf(m - base), w = expf(x - base);
        l = l * keep + w;
        for (int d = lane, n = 0; d < p.D; d += 32, ++n) o[n] = o[n] * keep + w * cache_value<kE4m3>(p.vpool, at + d);
        m = mn;
    }
    if (lane == 0) sm[warp] = m, sl[warp] = l;
    for (int d = lane, n = 0; d < p.D; d += 32, ++n) so[warp][d] = o[n];
    __syncthreads();
    const float mx = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3])), base = mx == -INFINITY ? 0.f : mx;
    float wt[4], total = 0.f;
    for (int w = 0; w < 4; ++w) wt[w] = expf(sm[w] - base), total += wt[w] * sl[w];
    const int64_t row = (int64_t)blockIdx.x;
    for (int d = threadIdx.x; d < p.D; d += kAThreads) {
        float v = 0.f;
        for (int w = 0; w < 4; ++w) v += wt[w] * so[w][d];
        p.o[row * p.D + d] = (uint16_t)f32_to_bf16_bits(total == 0.f ? 0.f : v * vs / total);
    }
    if (p.lse && threadIdx.x == 0) p.lse[row] = total == 0.f ? -INFINITY : logf(total) + base;
}

}  // namespace

size_t attn_paged_workspace_bytes(int64_t, int64_t, int64_t, int64_t, int64_t, int64_t) { return 0; }
int attn_paged_kernel_count(int64_t, int64_t, int64_t, int64_t, int64_t, int64_t) { return 1; }

cudaError_t launch_attn_paged(const AttnParams& a, bool e4m3, cudaStream_t st) {
    AttnParams p = a;
    p.err = device_error_word();
    if (!p.err) return cudaErrorUnknown;
    const dim3 grid((unsigned)((int64_t)p.B * p.Lq * p.Hq));
    return launch_pdl(e4m3 ? attn_simple_kernel<true> : attn_simple_kernel<false>, grid, dim3(kAThreads), 0, st, p);
}

}  // namespace fp8rl
