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
//
// Both are bound by HBM: the logits are read once (and the gradient written once), 16 bytes
// a load, four loads a thread in flight while the four before are worked on.  A CTA has a
// row, or with few rows a part of one; in the forward the parts are a cluster, whose first
// CTA gets the others' maxima and sums through shared memory.  Tokens that the teacher names
// are bits in shared memory, a byte for the eight bf16 of a load.
#include <math.h>

#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "sm100_ptx.cuh"

namespace fp8rl {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32, kMostRanks = 16, kFlight = 4;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLog2eRest = 1.9259629911266175e-8f;   // log2(e) - kLog2e
constexpr double kLn2 = 0.6931471805599453;
constexpr float kLowest = -3.3895314e38f;              // the lowest finite bf16

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// exp(scale d) for d <= 0: the constant scale log2(e) in two parts, since its rounding alone
// would be a change of temperature, some 1e-6 of the sum.
struct Scale {
    float c, rest;
    __device__ __forceinline__ explicit Scale(float scale)
        : c(scale * kLog2e), rest(fmaf(scale, kLog2e, -(scale * kLog2e)) + scale * kLog2eRest) {}
    __device__ __forceinline__ float exp(float d) const { return ex2(fmaf(d, c, d * rest)); }
};

// log of a positive fp32 sum to some 1e-8 absolute: the exponent apart, the rest as log1p.
__device__ __forceinline__ double log_sum(float s) {
    int e;
    float f = frexpf(s, &e);                          // [0.5, 1)
    if (f < 0.70710678f) f *= 2.f, --e;
    return (double)e * kLn2 + (double)log1pf(f - 1.f);
}
// exp of a 64-bit argument as fp32: what its rounding to 32 bits loses, to first order
__device__ __forceinline__ float exp64(double a) {
    const float hi = (float)a;
    return hi < -104.f ? 0.f : expf(hi) * (1.f + (float)(a - (double)hi));
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
#pragma unroll
    for (int w = 1; w < kWarps; ++w) r += buf[w];
    return r;
}
__device__ __forceinline__ float block_max(float v, float* buf) {
    v = warp_max(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    float r = buf[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) r = fmaxf(r, buf[w]);
    return r;
}

__device__ __forceinline__ float value(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float value(const uint16_t* p, int64_t i) { return __uint_as_float((uint32_t)p[i] << 16); }
__device__ __forceinline__ void put(float* p, int64_t i, float v) { p[i] = v; }
__device__ __forceinline__ void put(uint16_t* p, int64_t i, float v) { p[i] = (uint16_t)f32_to_bf16_bits(v); }

// The logits of one 16-byte load.
template <typename T>
struct Chunk;
template <>
struct Chunk<uint16_t> {
    static constexpr int N = 8;
    static constexpr uint32_t kPad = 0xFF7FFF7Fu;              // kLowest twice
    uint32_t w[4];
    __device__ __forceinline__ void drop(uint32_t those) {     // as if they were not there
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (those >> e & 1) w[e >> 1] = e & 1 ? (w[e >> 1] & 0xFFFFu) | 0xFF7F0000u : (w[e >> 1] & 0xFFFF0000u) | 0xFF7Fu;
    }
    __device__ __forceinline__ void clamp() {                  // -inf to kLowest, NaN kept
#pragma unroll
        for (int i = 0; i < 4; ++i) asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(w[i]) : "r"(kPad));
    }
    __device__ __forceinline__ float most() const {
        uint32_t a, b;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(w[0]), "r"(w[1]));
        asm("max.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(w[2]), "r"(w[3]));
        asm("max.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
        return fmaxf(bf16_lo(a), bf16_hi(a));
    }
    __device__ __forceinline__ float at(int e) const { return e & 1 ? bf16_hi(w[e >> 1]) : bf16_lo(w[e >> 1]); }
    template <typename F>
    __device__ __forceinline__ uint4 map(F f) const {
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2(f(bf16_lo(w[i])), f(bf16_hi(w[i])));
        return make_uint4(o[0], o[1], o[2], o[3]);
    }
};
template <>
struct Chunk<float> {
    static constexpr int N = 4;
    static constexpr uint32_t kPad = 0xFF7F0000u;              // kLowest
    uint32_t w[4];
    __device__ __forceinline__ void drop(uint32_t those) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (those >> e & 1) w[e] = kPad;
    }
    __device__ __forceinline__ void clamp() {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float v = __uint_as_float(w[i]);
            asm("max.NaN.f32 %0, %0, %1;" : "+f"(v) : "f"(kLowest));
            w[i] = __float_as_uint(v);
        }
    }
    __device__ __forceinline__ float most() const { return fmaxf(fmaxf(at(0), at(1)), fmaxf(at(2), at(3))); }
    __device__ __forceinline__ float at(int e) const { return __uint_as_float(w[e]); }
    template <typename F>
    __device__ __forceinline__ uint4 map(F f) const {
        return make_uint4(__float_as_uint(f(at(0))), __float_as_uint(f(at(1))), __float_as_uint(f(at(2))),
                          __float_as_uint(f(at(3))));
    }
};

// Not by the read-only path: the gradient may overwrite the logits.
__device__ __forceinline__ uint4 load16(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
// kFlight loads of a thread, those past the end kLowest
template <typename T>
__device__ __forceinline__ void fetch(Chunk<T> (&b)[kFlight], const T* X, int at, int end) {
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
        const int g = at + u * kThreads;
        const uint4 v = g < end ? load16(X + (int64_t)g * Chunk<T>::N)
                                : make_uint4(Chunk<T>::kPad, Chunk<T>::kPad, Chunk<T>::kPad, Chunk<T>::kPad);
        b[u].w[0] = v.x, b[u].w[1] = v.y, b[u].w[2] = v.z, b[u].w[3] = v.w;
    }
}

// The teacher's entries of a row in shared memory, and the tokens they name as bits.
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

    __device__ __forceinline__ Entries(uint8_t* smem, int k) {
        dbuf = reinterpret_cast<double*>(smem);
        fbuf = reinterpret_cast<float*>(dbuf + kWarps);
        id = reinterpret_cast<int32_t*>(fbuf + kWarps);
        q = reinterpret_cast<float*>(id + k);
        x = q + k;
        bits = reinterpret_cast<uint32_t*>(x + k);
    }
    // Tokens, and their logits; every thread of the CTA takes part in this and the next.
    template <typename T>
    __device__ __forceinline__ void load(const DistillParams& p, int64_t m, const T* X) {
        const int words = (int)((p.V + 31) / 32);
        for (int w = threadIdx.x; w < words; w += kThreads) bits[w] = 0;
        __syncthreads();
        int both = 0;
        for (int i = threadIdx.x; i < p.k; i += kThreads) {
            int32_t t = p.ids[m * p.k + i];
            if (t < 0 || t >= p.V) t = -1;
            id[i] = t;
            if (t >= 0) {
                both += 1 | ((atomicOr(&bits[t >> 5], 1u << (t & 31)) >> (t & 31) & 1) ? 0 : 1 << 16);
                x[i] = value(X, t);
            }
        }
        both = block_sum(both, reinterpret_cast<int*>(fbuf));
        count = both & 0xffff, distinct = both >> 16;
    }
    __device__ __forceinline__ void weigh(const DistillParams& p, int64_t m) {
        const float* t = p.t + m * p.k;
        const double scale = (double)p.scale;
        if (p.teacher_lse) {
            shift = (double)p.teacher_lse[m];
        } else {
            float top = -INFINITY, s = 0.f;
            for (int i = threadIdx.x; i < p.k; i += kThreads)
                if (id[i] >= 0) top = fmaxf(top, t[i]);
            top = block_max(top, fbuf);
            for (int i = threadIdx.x; i < p.k; i += kThreads)
                if (id[i] >= 0) s += exp64(((double)t[i] - (double)top) * scale);
            s = block_sum(s, fbuf);
            shift = top > -INFINITY ? (double)top * scale + log_sum(s) : 0.0;   // no entry with any weight: all q 0
        }
        double sum = 0.0;
        for (int i = threadIdx.x; i < p.k; i += kThreads) {
            const float v = id[i] >= 0 ? exp64((double)t[i] * scale - shift) : 0.f;
            q[i] = v;
            sum += (double)v;
        }
        total = block_sum(sum, dbuf);
    }
    // What the tokens outside the entries are worth: 1 - sum q, none where every token is an entry.
    __device__ __forceinline__ double rest(const DistillParams& p) const {
        return p.rest_lse && distinct < p.V ? fmax(1.0 - total, 0.0) : 0.0;
    }
    // Whether entry i is the first that names its token.
    __device__ __forceinline__ bool first(int i) const {
        if (distinct < count)
            for (int j = 0; j < i; ++j)
                if (id[j] == id[i]) return false;
        return true;
    }
};
size_t smem_bytes(int64_t k, int64_t V) { return kWarps * 12 + (size_t)k * 12 + (size_t)((V + 31) / 32) * 4; }

struct Sum {
    float top, sum;
    __device__ __forceinline__ void add(float t, float s, const Scale& f) {
        const float most = fmaxf(top, t);
        sum = sum * f.exp(top - most) + s * f.exp(t - most);
        top = most;
    }
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 4)
distill_kernel(const __grid_constant__ DistillParams p, int ranks) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ uint64_t parts[kMostRanks];              // of the cluster's CTAs, in its first one's
    __shared__ Sum warps[kWarps];
    constexpr int N = Chunk<T>::N;
    if (ranks > 1) sm100::cluster_arrive();              // all have started (waited for below)
    pdl_wait_then_release();
    const int rank = (int)(blockIdx.x % (unsigned)ranks), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t m = blockIdx.x / (unsigned)ranks;
    const T* X = static_cast<const T*>(p.X) + m * p.ldx;
    const int chunks = (int)(p.V / N);
    int at = (int)((int64_t)chunks * rank / ranks);
    const int end = (int)((int64_t)chunks * (rank + 1) / ranks);
    at += threadIdx.x;
    Chunk<T> now[kFlight];
    fetch(now, X, at, end);
    Entries n(smem, p.k);
    n.load(p, m, X);
    const bool apart = p.rest_lse != nullptr, nobody = n.count == 0;
    const Scale f(p.scale);
    Sum s{kLowest, 0.f};
    const uint8_t* named = reinterpret_cast<const uint8_t*>(n.bits);
    for (; at < end && !nobody; at += kFlight * kThreads) {
        Chunk<T> next[kFlight];
        fetch(next, X, at + kFlight * kThreads, end);
        float most = s.top;
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            const int g = at + u * kThreads;
            if (apart && g < end) {
                const uint32_t those = N == 8 ? named[g] : named[g >> 1] >> (g & 1) * 4 & 15u;
                if (those) now[u].drop(those);
            }
            now[u].clamp();
            most = fmaxf(most, now[u].most());
        }
        if (most > s.top) s.sum *= f.exp(s.top - most), s.top = most;
        float part[kFlight];
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            part[u] = 0.f;
#pragma unroll
            for (int e = 0; e < N; ++e) part[u] += f.exp(now[u].at(e) - s.top);
            now[u] = next[u];
        }
        // kLowest stands for what is not there: where nothing else is, its terms are not either
        const float more = (part[0] + part[1]) + (part[2] + part[3]);
        if (s.top > kLowest || isnan(more)) s.sum += more;
    }
    const int last = chunks * N + (int)threadIdx.x;      // logits past the last whole 16 bytes
    if (rank == ranks - 1 && last < p.V && !nobody && !(apart && (n.bits[last >> 5] >> (last & 31) & 1))) {
        const float x = value(X, last);
        if (x != -INFINITY) s.add(x, 1.f, f);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float t = __shfl_xor_sync(0xffffffffu, s.top, o), v = __shfl_xor_sync(0xffffffffu, s.sum, o);
        s.add(t, v, f);
    }
    __syncthreads();
    if (lane == 0) warps[warp] = s;
    __syncthreads();
    s = warps[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) s.add(warps[w].top, warps[w].sum, f);
    if (ranks > 1) {
        sm100::cluster_wait();                           // the first CTA's shared memory is there
        if (threadIdx.x == 0)
            sm100::st_cluster_u64(sm100::map_to_rank(sm100::smem_u32(&parts[rank]), 0),
                                  sm100::f32x2_pack(__float_as_uint(s.top), __float_as_uint(s.sum)));
        sm100::cluster_arrive();
        sm100::cluster_wait();
        if (rank > 0) return;
        s = Sum{kLowest, 0.f};
        for (int r = 0; r < ranks; ++r) {
            const float2 v = sm100::f32x2_unpack(parts[r]);
            s.add(v.x, v.y, f);
        }
    }
    if (nobody) {                                        // whatever the row holds
        if (threadIdx.x == 0) {
            p.loss[m] = 0.f, p.lse[m] = 0.f;
            if (p.rest_lse) p.rest_lse[m] = 0.f;
        }
        return;
    }
    n.weigh(p, m);
    const double scale = (double)p.scale;
    double lse = s.sum == 0.f ? -INFINITY : (double)s.top * scale + log_sum(s.sum);
    const double rest = lse;
    if (apart) {                                         // the entries, each token once
        Sum in{kLowest, 0.f};
        for (int i = threadIdx.x; i < p.k; i += kThreads)
            if (n.id[i] >= 0 && n.x[i] != -INFINITY && n.first(i)) in.add(n.x[i], 1.f, f);
        const float most = block_max(in.top, n.fbuf), sum = block_sum(in.sum * f.exp(in.top - most), n.fbuf);
        if (sum != 0.f) {
            const double inside = (double)most * scale + log_sum(sum), far = fmin(inside, rest) - fmax(inside, rest);
            lse = fmax(inside, rest) + (far < -100.0 ? 0.0 : (double)log1pf(expf((float)far)));
            if (isnan(sum) || isnan(s.sum)) lse = NAN;
        }
    }
    double loss = 0.0;
    for (int i = threadIdx.x; i < p.k; i += kThreads)
        if (n.q[i] > 0.f)
            loss += (double)n.q[i] * (((double)p.t[m * p.k + i] * scale - n.shift) - ((double)n.x[i] * scale - lse));
    loss = block_sum(loss, n.dbuf);
    if (threadIdx.x == 0) {
        const double qr = n.rest(p);
        if (qr > 0.0) loss += qr * ((double)logf((float)qr) - (rest - lse));
        p.loss[m] = (float)loss, p.lse[m] = (float)lse;
        if (p.rest_lse) p.rest_lse[m] = (float)rest;
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4)
distill_grad_kernel(const __grid_constant__ DistillParams p, int ranks) {
    extern __shared__ __align__(16) uint8_t smem[];
    constexpr int N = Chunk<T>::N;
    pdl_wait_then_release();
    const int rank = (int)(blockIdx.x % (unsigned)ranks);
    const int64_t m = blockIdx.x / (unsigned)ranks;
    const T* X = static_cast<const T*>(p.X) + m * p.ldx;
    T* D = static_cast<T*>(p.dX) + m * p.lddx;
    const int chunks = (int)(p.V / N);
    const int from = (int)((int64_t)chunks * rank / ranks), end = (int)((int64_t)chunks * (rank + 1) / ranks);
    // this CTA's logits, the last one's with what is past the last whole 16 bytes
    const int64_t lo = (int64_t)from * N, hi = rank == ranks - 1 ? p.V : (int64_t)end * N;
    int at = from + (int)threadIdx.x;
    Chunk<T> now[kFlight];
    fetch(now, X, at, end);
    Entries n(smem, p.k);
    n.load(p, m, X);                                     // before any of this CTA's logits is overwritten
    n.weigh(p, m);
    const float c = p.scale * kLog2e;
    float a = 0.f, r2 = 0.f, g = 0.f, Q = 0.f, l2 = 0.f;
    if (n.count > 0) {
        const float qr = (float)n.rest(p), lse = p.lse[m];
        g = p.g[m] * p.scale, Q = (float)n.total + qr, l2 = lse * kLog2e;
        a = g * Q, r2 = l2;
        if (qr > 0.f && p.rest_lse[m] > -INFINITY) {
            const float rest = p.rest_lse[m];
            a = g * (Q * expf(rest - lse) - qr), r2 = rest * kLog2e;
        }
    }
    const bool nobody = n.count == 0;                    // zeros, whatever the row holds
    auto grad = [&](float x) { return nobody ? 0.f : a * ex2(fmaf(x, c, -r2)); };
    for (; at < end; at += kFlight * kThreads) {
        Chunk<T> next[kFlight];
        fetch(next, X, at + kFlight * kThreads, end);
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            const int g4 = at + u * kThreads;
            if (g4 < end) __stcs(reinterpret_cast<uint4*>(D + (int64_t)g4 * N), now[u].map(grad));
            now[u] = next[u];
        }
    }
    if (chunks * (int64_t)N + threadIdx.x < hi && rank == ranks - 1) {
        const int64_t v = chunks * (int64_t)N + threadIdx.x;
        put(D, v, grad(value(X, v)));
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.k; i += kThreads) {
        const int64_t t = n.id[i];
        if (t < lo || t >= hi) continue;                 // -1 is below every CTA's
        float q = n.q[i];
        if (n.distinct < n.count) {                      // a token named twice has both entries' weight
            q = 0.f;
            for (int j = 0; j < p.k; ++j) q += n.id[j] == t ? n.q[j] : 0.f;
        }
        put(D, t, g * (Q * ex2(fmaf(n.x[i], c, -l2)) - q));
    }
}

using Kernel = void(const DistillParams, int);
Kernel* const kKernels[4] = {distill_kernel<float>, distill_kernel<uint16_t>, distill_grad_kernel<float>,
                             distill_grad_kernel<uint16_t>};

// Clusters of 16 and more than 48 KB of shared memory have to be asked for, once a device.
cudaError_t ask() {
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && ready.load(std::memory_order_relaxed) >> dev & 1)) return e;
    for (Kernel* k : kKernels) {
        e = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
        if (e != cudaSuccess) return e;
    }
    if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
    return e;
}

cudaError_t launch(Kernel* f, const DistillParams& p, int per_load, bool cluster, cudaStream_t st) {
    const cudaError_t e = ask();
    if (e != cudaSuccess) return e;
    // CTAs a row: while all of them find a place at once (four an SM; clusters of 16 only
    // with an SM a CTA) and each thread keeps two loads
    const int64_t sms = num_sms();
    int ranks = 1;
    while (2 * ranks <= kMostRanks && 2 * ranks * p.M <= (ranks == 8 ? sms : 4 * sms) && p.V / per_load >= 2 * ranks * kThreads)
        ranks *= 2;
    const size_t smem = smem_bytes(p.k, p.V);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.M * ranks));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim = {(unsigned)ranks, 1, 1};
    cfg.attrs = at;
    cfg.numAttrs = cluster && ranks > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, f, p, ranks);
}

}  // namespace

cudaError_t launch_distill_topk(const DistillParams& p, bool bf16, bool backward, cudaStream_t st) {
    return launch(kKernels[2 * backward + bf16], p, bf16 ? 8 : 4, !backward, st);
}

}  // namespace fp8rl
