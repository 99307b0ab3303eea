// linear_logp.cu -- log-probabilities of chosen tokens straight from the hidden states H
// and the output matrix W, without keeping the logits, and their gradient.
//
//   x_mv = scale h_m . w_v,   lse_m = log sum_v exp x_mv,   p = exp(x - lse),
//   logp_m = x_mt - lse_m,    entropy_m = - sum_v p_v log p_v,
//   D_mv = g_m (d_vt - p_mv) - e_m p_mv (log p_mv + entropy_m),
//   dH = scale D W,   dW = scale D^T H.
//
// Forward: tiles of logits, of which each row leaves its maximum, its sum of exponentials
// and sum of weighted differences; a second launch joins a row's tiles.  Backward: the
// vocabulary in pieces; a piece's D as bf16 (each D rounded once, relative to the call's
// largest g or e, to 2^-9 of itself), then its part of dH, summed in fp32 over the pieces, and its rows of dW.
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace fp8rl {

namespace {

constexpr int kTile = 64, kDepth = 16, kThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;

struct Tile {
    float a[kDepth][kTile + 4], b[kDepth][kTile + 4];
};

__device__ __forceinline__ float bf(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }

// c[i][j] += sum_k A(row0 + 16 i + ty, k) B(col0 + 16 j + tx, k), values past the edges zero.
template <typename FA, typename FB>
__device__ __forceinline__ void multiply(Tile& s, int64_t K, FA A, FB B, float (&c)[4][4]) {
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int64_t k0 = 0; k0 < K; k0 += kDepth) {
        __syncthreads();
        for (int e = threadIdx.x; e < kTile * kDepth; e += kThreads) {
            const int r = e / kDepth, d = e % kDepth;
            s.a[d][r] = k0 + d < K ? A(r, k0 + d) : 0.f;
            s.b[d][r] = k0 + d < K ? B(r, k0 + d) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int d = 0; d < kDepth; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) c[i][j] = fmaf(s.a[d][16 * i + ty], s.b[d][16 * j + tx], c[i][j]);
    }
}

__device__ __forceinline__ bool counts(const LogpParams& p, int64_t m) {
    return m < p.M && p.targets[m] >= 0 && p.targets[m] < p.V;
}

// A tile's logits, rows that do not count as zeros.
__device__ __forceinline__ void logits(const LogpParams& p, Tile& s, int64_t m0, int64_t v0, float (&c)[4][4]) {
    multiply(s, p.K, [&](int r, int64_t k) { return counts(p, m0 + r) ? bf(p.H[(m0 + r) * p.ldh + k]) : 0.f; },
             [&](int r, int64_t k) { return v0 + r < p.V ? bf(p.W[(v0 + r) * p.ldw + k]) : 0.f; }, c);
}

__global__ void __launch_bounds__(kThreads)
logp_tile_kernel(const __grid_constant__ LogpParams p) {
    __shared__ Tile s;
    __shared__ float x[kTile][kTile + 1];
    pdl_wait_then_release();
    const int64_t v0 = (int64_t)blockIdx.x * kTile, m0 = (int64_t)blockIdx.y * kTile;
    float c[4][4] = {};
    logits(p, s, m0, v0, c);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) x[16 * i + ty][16 * j + tx] = c[i][j] * p.scale;
    __syncthreads();
    const int64_t m = m0 + threadIdx.x;
    if (threadIdx.x >= kTile || m >= p.M) return;
    const int cols = (int)min((int64_t)kTile, p.V - v0);
    float top = -INFINITY, sum = 0.f, dev = 0.f;
    for (int j = 0; j < cols; ++j) top = fmaxf(top, x[threadIdx.x][j]);
    for (int j = 0; j < cols; ++j) {
        const float d = x[threadIdx.x][j] - top, e = expf(d);
        sum += e, dev = fmaf(e, d, dev);
    }
    const int64_t at = blockIdx.x * p.M + m, size = (int64_t)gridDim.x * p.M;
    p.part[at] = top, p.part[size + at] = sum, p.part[2 * size + at] = dev;
    const int64_t t = p.targets[m] - v0;
    if (t >= 0 && t < cols) p.picked[m] = x[threadIdx.x][t];
}

__global__ void __launch_bounds__(kThreads)
logp_join_kernel(const __grid_constant__ LogpParams p, int64_t tiles) {
    pdl_wait_then_release();
    const int64_t m = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (m >= p.M) return;
    float logp = 0.f, lse = 0.f, entropy = 0.f;
    if (counts(p, m)) {
        float top = -INFINITY;
        for (int64_t t = 0; t < tiles; ++t) top = fmaxf(top, p.part[t * p.M + m]);
        float sum = 0.f, dev = 0.f;
        const int64_t size = tiles * p.M;
        for (int64_t t = 0; t < tiles; ++t) {
            const float d = p.part[t * p.M + m] - top, e = expf(d), s = p.part[size + t * p.M + m];
            sum = fmaf(e, s, sum);
            dev = fmaf(e, fmaf(d, s, p.part[2 * size + t * p.M + m]), dev);
        }
        lse = top + logf(sum), logp = p.picked[m] - lse, entropy = logf(sum) - dev / sum;
    }
    p.logp[m] = logp, p.lse[m] = lse;
    if (p.entropy) p.entropy[m] = entropy;
}

// The largest |g| and |e| of the rows that count.
__global__ void __launch_bounds__(1024)
grad_scale_kernel(const __grid_constant__ LogpParams p) {
    __shared__ float w[32];
    pdl_wait_then_release();
    float a = 0.f;
    for (int64_t m = threadIdx.x; m < p.M; m += 1024)
        if (counts(p, m)) a = fmaxf(a, fmaxf(fabsf(p.g[m]), p.ge ? fabsf(p.ge[m]) : 0.f));
    for (int o = 16; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    if ((threadIdx.x & 31) == 0) w[threadIdx.x >> 5] = a;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < 32; ++i) a = fmaxf(a, w[i]);
        *p.largest = a > 0.f ? a : 1.f;
    }
}

// D of vocabulary rows [first, first + count), as bf16 [M][count].
__global__ void __launch_bounds__(kThreads)
grad_tile_kernel(const __grid_constant__ LogpParams p, int64_t first, int64_t count) {
    __shared__ Tile s;
    pdl_wait_then_release();
    const int64_t v0 = first + (int64_t)blockIdx.x * kTile, m0 = (int64_t)blockIdx.y * kTile;
    float c[4][4] = {};
    logits(p, s, m0, v0, c);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const float largest = *p.largest;
    for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + 16 * i + ty;
        if (m >= p.M) continue;
        const bool live = counts(p, m);
        const float g = live ? p.g[m] / largest : 0.f, ge = live && p.ge ? p.ge[m] / largest : 0.f;
        const float lse = live ? p.lse[m] : 0.f, ent = live && p.ge ? p.entropy[m] : 0.f;
        for (int j = 0; j < 4; ++j) {
            const int64_t v = v0 + 16 * j + tx;
            if (v >= first + count) continue;
            const float lp = c[i][j] * p.scale - lse, pr = expf(lp);
            float d = g * ((p.targets[m] == v ? 1.f : 0.f) - pr);
            if (p.ge) d -= ge * pr * (lp + ent);
            p.D[m * p.piece + v - first] = live ? (uint16_t)f32_to_bf16_bits(d) : 0;
        }
    }
}

// acc [M][K] (+)= D W
__global__ void __launch_bounds__(kThreads)
grad_h_kernel(const __grid_constant__ LogpParams p, int64_t first, int64_t count) {
    __shared__ Tile s;
    pdl_wait_then_release();
    const int64_t k0 = (int64_t)blockIdx.x * kTile, m0 = (int64_t)blockIdx.y * kTile;
    float c[4][4] = {};
    multiply(s, count, [&](int r, int64_t v) { return m0 + r < p.M ? bf(p.D[(m0 + r) * p.piece + v]) : 0.f; },
             [&](int r, int64_t v) { return k0 + r < p.K ? bf(p.W[(first + v) * p.ldw + k0 + r]) : 0.f; }, c);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + 16 * i + ty, k = k0 + 16 * j + tx;
            if (m < p.M && k < p.K) p.acc[m * p.K + k] = (first ? p.acc[m * p.K + k] : 0.f) + c[i][j];
        }
}

__global__ void __launch_bounds__(kThreads)
grad_w_kernel(const __grid_constant__ LogpParams p, int64_t first, int64_t count) {
    __shared__ Tile s;
    pdl_wait_then_release();
    const int64_t k0 = (int64_t)blockIdx.x * kTile, v0 = (int64_t)blockIdx.y * kTile;
    float c[4][4] = {};
    multiply(s, p.M, [&](int r, int64_t m) { return v0 + r < count ? bf(p.D[m * p.piece + v0 + r]) : 0.f; },
             [&](int r, int64_t m) { return k0 + r < p.K && counts(p, m) ? bf(p.H[m * p.ldh + k0 + r]) : 0.f; }, c);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const float f = *p.largest * p.scale;
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t v = v0 + 16 * i + ty, k = k0 + 16 * j + tx;
            if (v < count && k < p.K) p.dW[(first + v) * p.K + k] = (uint16_t)f32_to_bf16_bits(c[i][j] * f);
        }
}

__global__ void __launch_bounds__(kThreads)
grad_h_round_kernel(const __grid_constant__ LogpParams p) {
    pdl_wait_then_release();
    const float f = *p.largest * p.scale;
    const int64_t step = (int64_t)gridDim.x * kThreads;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < p.M * p.K; i += step)
        p.dH[i] = (uint16_t)f32_to_bf16_bits(counts(p, i / p.K) ? p.acc[i] * f : 0.f);
}

constexpr int64_t up16(int64_t n) { return (n + 15) / 16 * 16; }
int64_t piece_of(int64_t M, int64_t V) {
    int64_t n = (64ll << 20) / (2 * M) / kTile * kTile;
    n = n < kTile ? kTile : n;
    return n < V ? n : V;
}

}  // namespace

size_t linear_logp_workspace_bytes(int64_t M, int64_t V, int64_t K) {
    if (M <= 0 || V <= 0 || K <= 0) return 0;
    return (size_t)up16(4 * (3 * ((V + kTile - 1) / kTile) * M + M));
}

size_t linear_logp_backward_workspace_bytes(int64_t M, int64_t V, int64_t K) {
    if (M <= 0 || V <= 0 || K <= 0) return 0;
    return (size_t)(16 + up16(M * K * 4) + up16(M * piece_of(M, V) * 2));
}

cudaError_t launch_linear_logp(LogpParams p, void* ws, cudaStream_t st) {
    const int64_t tiles = (p.V + kTile - 1) / kTile, mt = (p.M + kTile - 1) / kTile;
    p.part = static_cast<float*>(ws);
    p.picked = p.part + 3 * tiles * p.M;
    cudaError_t e = launch_pdl(logp_tile_kernel, dim3((unsigned)tiles, (unsigned)mt), dim3(kThreads), 0, st, p);
    if (e != cudaSuccess) return e;
    return launch_pdl(logp_join_kernel, dim3((unsigned)((p.M + kThreads - 1) / kThreads)), dim3(kThreads), 0, st, p, tiles);
}

cudaError_t launch_linear_logp_backward(LogpParams p, void* ws, cudaStream_t st) {
    if (p.M == 0) return p.dW ? cudaMemsetAsync(p.dW, 0, (size_t)(p.V * p.K) * 2, st) : cudaSuccess;
    uint8_t* b = static_cast<uint8_t*>(ws);
    p.largest = reinterpret_cast<float*>(b);
    p.acc = reinterpret_cast<float*>(b + 16);
    p.D = reinterpret_cast<uint16_t*>(b + 16 + up16(p.M * p.K * 4));
    p.piece = piece_of(p.M, p.V);
    auto blocks = [](int64_t n) { return (unsigned)((n + kTile - 1) / kTile); };
    cudaError_t e = launch_pdl(grad_scale_kernel, dim3(1), dim3(1024), 0, st, p);
    for (int64_t v = 0; v < p.V && e == cudaSuccess; v += p.piece) {
        const int64_t n = p.V - v < p.piece ? p.V - v : p.piece;
        e = launch_pdl(grad_tile_kernel, dim3(blocks(n), blocks(p.M)), dim3(kThreads), 0, st, p, v, n);
        if (p.dH && e == cudaSuccess)
            e = launch_pdl(grad_h_kernel, dim3(blocks(p.K), blocks(p.M)), dim3(kThreads), 0, st, p, v, n);
        if (p.dW && e == cudaSuccess)
            e = launch_pdl(grad_w_kernel, dim3(blocks(p.K), blocks(n)), dim3(kThreads), 0, st, p, v, n);
    }
    if (!p.dH || e != cudaSuccess) return e;
    return launch_pdl(grad_h_round_kernel, dim3((unsigned)(4 * num_sms())), dim3(kThreads), 0, st, p);
}

}  // namespace fp8rl
