// distill_topk.cu -- distillation from a teacher's top logits, and its gradient.
//
// Row m has the student's logits x_v (scaled: y_v = scale x_v), and k entries of the
// teacher: a token i and its logit t_i.  The teacher's probabilities q_i are the softmax
// of scale t_i over the entries or, with the teacher's own log-sum, exp(scale t_i - lse_t),
// and then what they leave, q_r = 1 - sum q_i, may stand as one more class, the tokens
// outside the entries.  With p = softmax(y) and Q = sum q_i (+ q_r),
//   loss = sum_i q_i (log q_i - log p_i)  (+ q_r (log q_r - log p_r)),
//   d loss / d y_v = Q p_v - q_v  inside,   Q p_v - q_r exp(y_v - lse_r)  outside
// (no q_r without the rest), lse_r the log-sum outside.
//
// The loss is a difference of near terms once the student is close, so the logarithms
// meet in 64 bits; the sums of exponentials are fp32 relative to a maximum.  With the rest
// the pass over the logits sums the tokens outside, relative to their own maximum, and the
// entries are added to that: a difference, or one maximum for both, would lose a small rest.
// The gradient outside is exp(y_v - lse_r) (Q exp(lse_r - lse) - q_r), no factor above 1.
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace fp8rl {

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr float kLog2e = 1.4426950408889634f;
constexpr double kLn2 = 0.6931471805599453;

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// log of a positive fp32 sum to some 1e-8 absolute: the exponent apart, the rest as log1p.
__device__ __forceinline__ double log_sum(float s) {
    int e;
    float f = frexpf(s, &e);                          // [0.5, 1)
    if (f < 0.70710678f) f *= 2.f, --e;
    return (double)e * kLn2 + (double)log1pf(f - 1.f);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
template <typename T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// Over the CTA, the same for every thread; fixed order.
template <typename T>
__device__ __forceinline__ T block_sum(T v, T* buf) {
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    T r = buf[0];
    for (int w = 1; w < kWarps; ++w) r += buf[w];
    return r;
}
__device__ __forceinline__ float block_max(float v, float* buf) {
    v = warp_max(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    float r = buf[0];
    for (int w = 1; w < kWarps; ++w) r = fmaxf(r, buf[w]);
    return r;
}

__device__ __forceinline__ float value(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float value(const uint16_t* p, int64_t i) { return __uint_as_float((uint32_t)p[i] << 16); }
__device__ __forceinline__ void put(float* p, int64_t i, float v) { p[i] = v; }
__device__ __forceinline__ void put(uint16_t* p, int64_t i, float v) { p[i] = (uint16_t)f32_to_bf16_bits(v); }

// The teacher's entries of a row in shared memory, and the tokens they name as bits.
// Shared by both kernels; every thread of the CTA takes part.
struct Entries {
    int32_t* id;       // [k], -1 where the entry names no token
    float* q;          // [k], the teacher's probability
    float* x;          // [k], the student's logit
    uint32_t* bits;    // [ceil(V / 32)]
    float* fbuf;       // [kWarps]
    double* dbuf;      // [kWarps]
    int count, distinct;
    double total;      // sum of q
    double shift;      // log q_i = scale t_i - shift
};

template <typename T>
__device__ __forceinline__ void load_entries(Entries& n, const DistillParams& p, int64_t m, const T* X) {
    const int words = (int)((p.V + 31) / 32);
    for (int w = threadIdx.x; w < words; w += kThreads) n.bits[w] = 0;
    __syncthreads();
    int count = 0, distinct = 0;
    float top = -INFINITY;
    for (int i = threadIdx.x; i < p.k; i += kThreads) {
        int32_t id = p.ids[m * p.k + i];
        if (id < 0 || id >= p.V) id = -1;
        n.id[i] = id;
        float t = p.t[m * p.k + i];
        if (id >= 0) {
            ++count;
            distinct += (atomicOr(&n.bits[id >> 5], 1u << (id & 31)) >> (id & 31) & 1) == 0;
            n.x[i] = value(X, id);
            top = fmaxf(top, t);
        }
    }
    const int both = block_sum(count | distinct << 16, reinterpret_cast<int*>(n.fbuf));
    n.count = both & 0xffff, n.distinct = both >> 16;
    const double scale = (double)p.scale;
    if (p.teacher_lse) {
        n.shift = (double)p.teacher_lse[m];
    } else {
        top = block_max(top, n.fbuf);
        float s = 0.f;
        for (int i = threadIdx.x; i < p.k; i += kThreads)
            if (n.id[i] >= 0) s += expf((p.t[m * p.k + i] - top) * p.scale);
        s = block_sum(s, n.fbuf);
        n.shift = (double)top * scale + log_sum(s);
    }
    double total = 0.0;
    for (int i = threadIdx.x; i < p.k; i += kThreads) {
        const float q = n.id[i] >= 0 ? expf((float)((double)p.t[m * p.k + i] * scale - n.shift)) : 0.f;
        n.q[i] = q;
        total += (double)q;
    }
    n.total = block_sum(total, n.dbuf);
}

__device__ __forceinline__ Entries entries(uint8_t* smem, int k) {
    Entries n;
    n.dbuf = reinterpret_cast<double*>(smem);
    n.fbuf = reinterpret_cast<float*>(n.dbuf + kWarps);
    n.id = reinterpret_cast<int32_t*>(n.fbuf + kWarps);
    n.q = reinterpret_cast<float*>(n.id + k);
    n.x = n.q + k;
    n.bits = reinterpret_cast<uint32_t*>(n.x + k);
    return n;
}
size_t smem_bytes(int64_t k, int64_t V) { return kWarps * 12 + (size_t)k * 12 + (size_t)((V + 31) / 32) * 4; }

// Whether entry i is the first that names its token.
__device__ __forceinline__ bool first_of(const Entries& n, int i) {
    if (n.distinct < n.count)
        for (int j = 0; j < i; ++j)
            if (n.id[j] == n.id[i]) return false;
    return true;
}

// What the tokens outside the entries are worth: 1 - sum q, none where every token is an entry.
__device__ __forceinline__ double rest_of(const Entries& n, const DistillParams& p) {
    return p.rest_lse && n.distinct < p.V ? fmax(1.0 - n.total, 0.0) : 0.0;
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
distill_kernel(const __grid_constant__ DistillParams p) {
    extern __shared__ __align__(16) uint8_t smem[];
    pdl_wait_then_release();
    Entries n = entries(smem, p.k);
    for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x) {
        __syncthreads();
        const T* X = static_cast<const T*>(p.X) + m * p.ldx;
        load_entries(n, p, m, X);
        if (n.count == 0) {                          // nobody's row: whatever it holds
            if (threadIdx.x == 0) {
                p.loss[m] = 0.f, p.lse[m] = 0.f;
                if (p.rest_lse) p.rest_lse[m] = 0.f;
            }
            continue;
        }
        const float c = p.scale * kLog2e;
        const bool apart = p.rest_lse != nullptr;
        auto skip = [&](int64_t v) { return apart && (n.bits[v >> 5] >> (v & 31) & 1); };
        float top = -3.4e38f, sum = 0.f;
        for (int64_t v = threadIdx.x; v < p.V; v += kThreads)
            if (!skip(v)) top = fmaxf(top, value(X, v));
        top = block_max(top, n.fbuf);
        for (int64_t v = threadIdx.x; v < p.V; v += kThreads)
            if (!skip(v)) sum += ex2((value(X, v) - top) * c);
        sum = block_sum(sum, n.fbuf);
        const double scale = (double)p.scale;
        double lse = sum > 0.f ? (double)top * scale + log_sum(sum) : -INFINITY;
        const double rest = lse;
        if (apart) {                                 // the entries, each token once
            float most = -3.4e38f, in = 0.f;
            for (int i = threadIdx.x; i < p.k; i += kThreads)
                if (n.id[i] >= 0) most = fmaxf(most, n.x[i]);
            most = block_max(most, n.fbuf);
            for (int i = threadIdx.x; i < p.k; i += kThreads)
                if (n.id[i] >= 0 && first_of(n, i)) in += ex2((n.x[i] - most) * c);
            in = block_sum(in, n.fbuf);
            if (in > 0.f) {
                const double inside = (double)most * scale + log_sum(in), far = fmin(inside, rest) - fmax(inside, rest);
                lse = fmax(inside, rest) + (far < -100.0 ? 0.0 : (double)log1pf(expf((float)far)));
            }
        }
        double loss = 0.0;
        for (int i = threadIdx.x; i < p.k; i += kThreads)
            if (n.q[i] > 0.f)
                loss += (double)n.q[i] * (((double)p.t[m * p.k + i] * scale - n.shift) - ((double)n.x[i] * scale - lse));
        loss = block_sum(loss, n.dbuf);
        if (threadIdx.x == 0) {
            const double qr = rest_of(n, p);
            if (qr > 0.0) loss += qr * ((double)logf((float)qr) - (rest - lse));
            p.loss[m] = (float)loss, p.lse[m] = (float)lse;
            if (p.rest_lse) p.rest_lse[m] = (float)rest;
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
distill_grad_kernel(const __grid_constant__ DistillParams p) {
    extern __shared__ __align__(16) uint8_t smem[];
    pdl_wait_then_release();
    Entries n = entries(smem, p.k);
    for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x) {
        __syncthreads();
        const T* X = static_cast<const T*>(p.X) + m * p.ldx;
        T* D = static_cast<T*>(p.dX) + m * p.lddx;
        load_entries(n, p, m, X);                     // reads the entries' logits before any is overwritten
        if (n.count == 0) {
            for (int64_t v = threadIdx.x; v < p.V; v += kThreads) put(D, v, 0.f);
            continue;
        }
        const float qr = (float)rest_of(n, p);
        const float lse = p.lse[m], g = p.g[m] * p.scale, Q = (float)n.total + qr, c = p.scale * kLog2e;
        const float l2 = lse * kLog2e;
        float a = g * Q, r2 = l2;
        if (qr > 0.f && p.rest_lse[m] > -INFINITY) {
            const float rest = p.rest_lse[m];
            a = g * (Q * expf(rest - lse) - qr), r2 = rest * kLog2e;
        }
        for (int64_t v = threadIdx.x; v < p.V; v += kThreads) put(D, v, a * ex2(fmaf(value(X, v), c, -r2)));
        __syncthreads();
        for (int i = threadIdx.x; i < p.k; i += kThreads) {
            if (n.id[i] < 0) continue;
            float q = n.q[i];
            if (n.distinct < n.count) {                // a token named twice has both entries' weight
                q = 0.f;
                for (int j = 0; j < p.k; ++j) q += n.id[j] == n.id[i] ? n.q[j] : 0.f;
            }
            put(D, n.id[i], g * (Q * ex2(fmaf(n.x[i], c, -l2)) - q));
        }
    }
}

template <typename F>
cudaError_t launch(F* f, const DistillParams& p, cudaStream_t st) {
    const size_t smem = smem_bytes(p.k, p.V);
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    const int64_t most = 8 * (int64_t)num_sms();
    return launch_pdl(f, dim3((unsigned)(p.M < most ? p.M : most)), dim3(kThreads), smem, st, p);
}

}  // namespace

cudaError_t launch_distill_topk(const DistillParams& p, bool bf16, bool backward, cudaStream_t st) {
    if (backward) return bf16 ? launch(distill_grad_kernel<uint16_t>, p, st) : launch(distill_grad_kernel<float>, p, st);
    return bf16 ? launch(distill_kernel<uint16_t>, p, st) : launch(distill_kernel<float>, p, st);
}

}  // namespace fp8rl
