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
// are taken to 1e-9 and meet in 64 bits; the sums of exponentials are fp32 relative to a maximum.
// Logits enter it relative to the sums' references alone, so neither logits that share a large
// part nor rows of nothing but a mask's value lose anything to them.  With the rest
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

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "internal.h"
#include "sm100_ptx.cuh"

namespace fp8rl {

namespace {

constexpr int kMostRanks = 16, kFlight = 4;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLog2eRest = 1.9259629911266175e-8f;   // log2(e) - kLog2e
constexpr double kLn2 = 0.6931471805599453;
constexpr float kLowest = -3.40282347e38f;             // the lowest of fp32: nothing seen yet

// Two fp32 to bf16, rounded to nearest even, in one instruction (one by one they are slow).
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint64_t pk2(float lo, float hi) {
    return sm100::f32x2_pack(__float_as_uint(lo), __float_as_uint(hi));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
// exp(scale d) for d <= 0: the constant scale log2(e) in two parts, since its rounding alone
// would be a change of temperature, some 1e-6 of the sum.  Both parts are positive, so that
// both products of d = -inf (a lowest logit under one of 1e37) are -inf.
struct Scale {
    float c, rest;
    __device__ __forceinline__ explicit Scale(float scale) : c(scale * kLog2e), rest(left(scale)) {
        if (rest < 0.f) c = __uint_as_float(__float_as_uint(c) - 1), rest = left(scale);
        rest = fmaxf(rest, 1e-45f);
    }
    __device__ __forceinline__ float left(float scale) const { return fmaf(scale, kLog2e, -c) + scale * kLog2eRest; }
    __device__ __forceinline__ float exp(float d) const { return ex2(fmaf(d, c, d * rest)); }
    // of two logits relative to a maximum, given as pairs with -top
    __device__ __forceinline__ uint64_t exp(uint64_t x, uint64_t low) const {
        const uint64_t d = add2(x, low), a = fma2(d, pk2(c, c), mul2(d, pk2(rest, rest)));
        const float2 v = sm100::f32x2_unpack(a);
        return pk2(ex2(v.x), ex2(v.y));
    }
};

// A natural logarithm good to some 1e-9 in mostly 32-bit steps, since 64-bit arithmetic is
// slow here (three of the library's cost a row 3 us): v = 2^e f, f c = 1 + r with c near
// 1 / f of ten bits, one of 32, so that r < 1/50 is all but exact; log v = e log 2 - log c +
// log1p(r), the last by its series, and what v loses as fp32 to first order.
struct Near {
    float c;
    double log;                                        // -log c
};
__constant__ Near kNear[32] = {
    {0.984375, 0.015748356968139168}, {0.955078125, 0.045962135564635756},
    {0.927734375, 0.07500982100486657}, {0.90234375, 0.10275973395776894},
    {0.876953125, 0.1313017372972535}, {0.853515625, 0.15839142994391764},
    {0.83203125, 0.18388527877013736}, {0.810546875, 0.21004610480880948},
    {0.791015625, 0.23443755793296864}, {0.771484375, 0.2594388601383859},
    {0.75390625, 0.2824872555746769}, {0.736328125, 0.30607943759149703},
    {0.71875, 0.33024168687057687}, {0.703125, 0.3522205935893521},
    {0.6875, 0.3746934494414107}, {0.673828125, 0.394780208008148},
    {0.66015625, 0.415278729556489}, {0.646484375, 0.43620624966244487},
    {0.6328125, 0.4575811092471784}, {0.62109375, 0.47627324225933093},
    {0.609375, 0.4953214372300254}, {0.59765625, 0.514739523087127},
    {0.587890625, 0.5312143602906321}, {0.576171875, 0.5513492686996879},
    {0.56640625, 0.5684437020589881}, {0.556640625, 0.5858354447708572},
    {0.546875, 0.6035350218702582}, {0.537109375, 0.6215535273729365},
    {0.529296875, 0.6362058041598069}, {0.51953125, 0.6548283162578087},
    {0.51171875, 0.6699801212784109}, {0.50390625, 0.6853650401178903}};
__device__ __forceinline__ double log64(double v) {
    const float s = (float)v, lost = (float)(v - (double)s);
    if (!(s > 1e-37f && s < 3e38f)) return v > 0.0 ? log(v) : v == 0.0 ? -INFINITY : NAN;
    const uint32_t b = __float_as_uint(s);
    const Near& n = kNear[b >> 18 & 31];
    const float r = fmaf(__uint_as_float((b & 0x007FFFFFu) | 0x3F800000u), n.c, -1.f);
    const float series = r * r * fmaf(r, fmaf(r, fmaf(r, 0.2f, -0.25f), 1.f / 3.f), -0.5f);
    return (double)((int)(b >> 23) - 127) * kLn2 + n.log + (double)(r + (series + lost / s));
}

// (a - b) - (c - d), off by a rounding of the result and some 2^-46 of either difference
__device__ __forceinline__ float apart_of(float a, float b, float c, float d) {
    const float s = a - b, u = c - d;
    if (!(fabsf(s) < INFINITY)) return s - u;
    const float sb = s - a, ub = u - c;
    const float se = (a - (s - sb)) + (-b - sb), ue = (c - (u - ub)) + (-d - ub);
    return (s - u) + (se - ue);
}

// exp(scale t - shift) as fp32, shift in two parts: what the argument's roundings lose, to
// first order
__device__ __forceinline__ float exp_less(float t, float scale, float shift, float shift_rest) {
    const float y = t * scale, rest = fmaf(t, scale, -y), hi = y - shift, back = hi - y;
    const float lo = (y - (hi - back)) + (-shift - back) + (rest - shift_rest), arg = hi + lo;
    return hi < -104.f ? 0.f : expf(arg) * (1.f + (lo - (arg - hi)));
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
    static constexpr uint32_t kPad = 0xFF80FF80u;              // -inf twice
    uint32_t w[4];
    __device__ __forceinline__ void drop(uint32_t those) {     // as if they were not there
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (those >> e & 1) w[e >> 1] = e & 1 ? (w[e >> 1] & 0xFFFFu) | 0xFF800000u : (w[e >> 1] & 0xFFFF0000u) | 0xFF80u;
    }
    __device__ __forceinline__ float most() const {
        uint32_t a, b;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(w[0]), "r"(w[1]));
        asm("max.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(w[2]), "r"(w[3]));
        asm("max.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
        return fmaxf(bf16_lo(a), bf16_hi(a));
    }
    __device__ __forceinline__ uint64_t pair(int i) const { return pk2(bf16_lo(w[i]), bf16_hi(w[i])); }
    template <typename F>
    __device__ __forceinline__ uint4 map(F f) const {
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = pack2(f(bf16_lo(w[i])), f(bf16_hi(w[i])));
        return make_uint4(o[0], o[1], o[2], o[3]);
    }
};
template <>
struct Chunk<float> {
    static constexpr int N = 4;
    static constexpr uint32_t kPad = 0xFF800000u;              // -inf
    uint32_t w[4];
    __device__ __forceinline__ void drop(uint32_t those) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (those >> e & 1) w[e] = kPad;
    }
    __device__ __forceinline__ float most() const { return fmaxf(fmaxf(at(0), at(1)), fmaxf(at(2), at(3))); }
    __device__ __forceinline__ float at(int e) const { return __uint_as_float(w[e]); }
    __device__ __forceinline__ uint64_t pair(int i) const { return sm100::f32x2_pack(w[2 * i], w[2 * i + 1]); }
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
// kFlight loads of a thread, those past the end -inf
template <int kThreads, typename T>
__device__ __forceinline__ void fetch(Chunk<T> (&b)[kFlight], const T* X, int at, int end) {
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
        const int g = at + u * kThreads;
        const uint4 v = g < end ? load16(X + (int64_t)g * Chunk<T>::N)
                                : make_uint4(Chunk<T>::kPad, Chunk<T>::kPad, Chunk<T>::kPad, Chunk<T>::kPad);
        b[u].w[0] = v.x, b[u].w[1] = v.y, b[u].w[2] = v.z, b[u].w[3] = v.w;
    }
}

// The teacher's entries of a row in shared memory, and the tokens they name as bits.  A
// thread's first entry waits in registers until it is used: its token, the teacher's
// logit and the student's are under way while the row's first logits are.  What is left
// to do with them then is one warp's: this GPU's 64-bit arithmetic is slow, and eight warps
// each with the same few steps of it took a CTA 2 us.
template <int kThreads>
struct Entries {
    int32_t* id;       // [k], -1 where the entry names no token
    float* q;          // [k], the teacher's logit, then its probability
    float* x;          // [k], the student's logit
    uint32_t* bits;    // [ceil(V / 32)]
    int32_t mine = -1;
    float my_t = 0.f, my_x = 0.f;
    bool any, twice = false;       // the row names a token; it names one twice (where there are bits)
    bool every = false;            // every token is named
    double total;      // sum of q
    float shift, shift_rest;       // log q_i = scale t_i - shift
    float center;                  // some t_i for which that is near 0

    __device__ __forceinline__ Entries(uint8_t* smem, const DistillParams& p, int64_t m) {
        id = reinterpret_cast<int32_t*>(smem);
        q = reinterpret_cast<float*>(id + p.k);
        x = q + p.k;
        bits = reinterpret_cast<uint32_t*>(x + p.k);
        const int64_t at = m * p.k;
        if ((int)threadIdx.x < p.k) mine = p.ids[at + threadIdx.x], my_t = p.t[at + threadIdx.x];
        for (int i = threadIdx.x + kThreads; i < p.k; i += kThreads) id[i] = p.ids[at + i], q[i] = p.t[at + i];
    }
    // Tokens, as bits where wanted, and their logits under way.  Every thread takes part.
    template <typename T>
    __device__ __forceinline__ void load(const DistillParams& p, const T* X, bool as_bits) {
        if (as_bits) {
            const int words = (int)((p.V + 31) / 32);
            for (int w = threadIdx.x; w < words; w += kThreads) bits[w] = 0;
            __syncthreads();
        }
        int named = 0, fresh = 0;
        for (int i = threadIdx.x; i < p.k; i += kThreads) {
            int32_t v = i < kThreads ? mine : id[i];
            if (v < 0 || v >= p.V) v = -1;
            id[i] = v;
            if (v < 0) continue;
            ++named;
            if (as_bits) fresh += (atomicOr(&bits[v >> 5], 1u << (v & 31)) >> (v & 31) & 1) == 0;
            if (i < kThreads) my_x = value(X, v);
            else x[i] = value(X, v);
        }
        any = __syncthreads_or(named);
        if (!as_bits) return;
        twice = __syncthreads_or(named != fresh);
        if (p.k >= p.V) {                                  // few tokens: are all of them named?
            int left = 0;
            for (int64_t v = threadIdx.x; v < p.V; v += kThreads) left |= !(bits[v >> 5] >> (v & 31) & 1);
            every = !__syncthreads_or(left);
        }
    }
    __device__ __forceinline__ void settle(const DistillParams& p) {
        if ((int)threadIdx.x < p.k) q[threadIdx.x] = my_t, x[threadIdx.x] = my_x;
    }
    // One warp, after settle() and a barrier: the teacher's probabilities; each lane has its
    // own of `each`, which is called with every entry, its logit and its probability.
    template <typename F>
    __device__ __forceinline__ void weigh(const DistillParams& p, int64_t m, F each) {
        const int lane = threadIdx.x & 31;
        if (p.teacher_lse) {
            shift = p.teacher_lse[m], shift_rest = 0.f;
        } else {
            float top = -INFINITY, s = 0.f;
            for (int i = lane; i < p.k; i += 32)
                if (id[i] >= 0) top = fmaxf(top, q[i]);
            top = warp_max(top);
            if (fabsf(top) > 16777216.f && fabsf(top) < INFINITY) {   // past what shift and its rest can hold
                for (int i = lane; i < p.k; i += 32) q[i] -= top;
                top = 0.f;
            }
            const float y = top * p.scale, rest = fmaf(top, p.scale, -y);
            for (int i = lane; i < p.k; i += 32)
                if (id[i] >= 0) s += exp_less(q[i], p.scale, y, rest);
            s = warp_sum(s);
            // no entry with any weight: all q 0
            const double all = top > -INFINITY ? (double)top * (double)p.scale + log64((double)s) : 0.0;
            shift = (float)all, shift_rest = (float)(all - (double)shift);
        }
        center = shift / p.scale;
        if (!(fabsf(center) < INFINITY)) center = 0.f;
        double sum = 0.0;
        for (int i = lane; i < p.k; i += 32) {
            const float t = q[i], v = id[i] >= 0 ? exp_less(t, p.scale, shift, shift_rest) : 0.f;
            q[i] = v;
            sum += (double)v;
            each(i, t, v);
        }
        total = warp_sum(sum);
        __syncwarp();
    }
    // What the tokens outside the entries are worth: 1 - sum q, none where every token is an entry.
    __device__ __forceinline__ double rest(const DistillParams& p) const {
        return p.rest_lse && !every ? fmax(1.0 - total, 0.0) : 0.0;
    }
    // Whether entry i is the first that names its token.
    __device__ __forceinline__ bool first(int i) const {
        if (twice)
            for (int j = 0; j < i; ++j)
                if (id[j] == id[i]) return false;
        return true;
    }
};
size_t smem_bytes(int64_t k, int64_t V, bool bits) { return (size_t)k * 12 + (bits ? (size_t)((V + 31) / 32) * 4 : 0); }

struct Sum {
    float top, sum;
    __device__ __forceinline__ void add(float t, float s, const Scale& f) {
        const float most = fmaxf(top, t);
        sum = sum * f.exp(top - most) + s * f.exp(t - most);
        top = most;
    }
};

template <typename T, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads)
distill_kernel(const __grid_constant__ DistillParams p, int ranks) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ uint64_t parts[kMostRanks];              // of the cluster's CTAs, in its first one's
    constexpr int N = Chunk<T>::N, kWarps = kThreads / 32;
    __shared__ Sum warps[kWarps];
    if (ranks > 1) sm100::cluster_arrive();              // all have started (waited for below)
    pdl_wait_then_release();
    const int rank = (int)(blockIdx.x % (unsigned)ranks), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t m = blockIdx.x / (unsigned)ranks;
    const T* X = static_cast<const T*>(p.X) + m * p.ldx;
    const int chunks = (int)(p.V / N);
    int at = (int)((int64_t)chunks * rank / ranks);
    const int end = (int)((int64_t)chunks * (rank + 1) / ranks);
    at += threadIdx.x;
    Entries<kThreads> n(smem, p, m);
    Chunk<T> now[kFlight];
    fetch<kThreads>(now, X, at, end);
    const bool apart = p.rest_lse != nullptr;
    n.load(p, X, apart);
    const bool nobody = !n.any;
    const Scale f(p.scale);
    Sum s{kLowest, 0.f};
    const uint8_t* named = reinterpret_cast<const uint8_t*>(n.bits);
    for (; at < end && !nobody; at += kFlight * kThreads) {
        Chunk<T> next[kFlight];
        fetch<kThreads>(next, X, at + kFlight * kThreads, end);
        float most = s.top;
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            const int g = at + u * kThreads;
            if (apart && g < end) {
                const uint32_t those = N == 8 ? named[g] : named[g >> 1] >> (g & 1) * 4 & 15u;
                if (those) now[u].drop(those);
            }
            most = fmaxf(most, now[u].most());
        }
        if (most > s.top) s.sum *= f.exp(s.top - most), s.top = most;
        uint64_t part[2] = {0, 0};
        const uint64_t low = pk2(-s.top, -s.top);
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
#pragma unroll
            for (int e = 0; e < N / 2; ++e) part[u & 1] = add2(part[u & 1], f.exp(now[u].pair(e), low));
            now[u] = next[u];
        }
        const float2 sums = sm100::f32x2_unpack(add2(part[0], part[1]));
        s.sum += sums.x + sums.y;                        // (terms of -inf are 0: the reference is finite)
    }
    const int last = chunks * N + (int)threadIdx.x;      // logits past the last whole 16 bytes
    if (rank == ranks - 1 && last < p.V && !nobody && !(apart && (n.bits[last >> 5] >> (last & 31) & 1))) {
        const float x = value(X, last);
        s.add(x, 1.f, f);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float t = __shfl_xor_sync(0xffffffffu, s.top, o), v = __shfl_xor_sync(0xffffffffu, s.sum, o);
        s.add(t, v, f);
    }
    if (lane == 0) warps[warp] = s;
    n.settle(p);
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
        s = Sum{kLowest, 0.f};
        if (rank == 0)
            for (int r = 0; r < ranks; ++r) {
                const float2 v = sm100::f32x2_unpack(parts[r]);
                s.add(v.x, v.y, f);
            }
    }
    if (rank > 0 || warp > 0) return;
    if (nobody) {                                        // whatever the row holds
        if (lane == 0) {
            p.loss[m] = 0.f, p.lse[m] = 0.f;
            if (p.rest_lse) p.rest_lse[m] = 0.f;
        }
        return;
    }
    // In the rest's reading the log-sum is relative to the outside's reference, so that the
    // whole's sum is that of the two: where the student is near, what the log-sums
    // share cancels in the loss, and what they do not would stay.  Entries so far
    // above that it would overflow: relative to their own maximum, and the outside
    // adds nothing.
    float top = s.top, sum = 0.f;
    bool above = false;
    if (apart) {
        float most = kLowest;
        for (int i = lane; i < p.k; i += 32)
            if (n.id[i] >= 0) most = fmaxf(most, n.x[i]);
        most = warp_max(most);
        above = s.sum == 0.f || (most - s.top) * p.scale > 60.f;
        if (above) top = most;
    }
    // loss = scale sum_i q_i ((t_i - center) - (x_i - top)) + sum_i q_i (lse - (shift - scale center))
    //        + q_r (log q_r - (lse_r - lse)),
    // lse relative to top where it stands behind q_i: the differences in fp32, their weighted sums and the log-sums in 64 bits
    double far = 0.0;
    n.weigh(p, m, [&](int i, float t, float q) {
        if (q > 0.f) far += (double)(q * apart_of(t, n.x[i], n.center, top));
    });
    far = warp_sum(far);
    const double scale = (double)p.scale, qr = n.rest(p);
    if (apart) {
        for (int i = lane; i < p.k; i += 32)             // the entries, each token once
            if (n.id[i] >= 0 && n.x[i] != -INFINITY && n.first(i)) sum += f.exp(n.x[i] - top);
        sum = warp_sum(sum);
    }
    // three logarithms by three lanes: of the sums outside and of all, of the rest
    const double all = isnan(s.sum) ? NAN : (double)sum + (above ? 0.0 : (double)s.sum);
    const double l = log64(lane == 0 ? (double)s.sum : lane == 1 ? all : qr);
    const double whole = __shfl_sync(0xffffffffu, l, 1), log_qr = __shfl_sync(0xffffffffu, l, 2);
    const double v = l + (double)(lane == 0 ? s.top : top) * scale, lse = __shfl_sync(0xffffffffu, v, 1);
    if (lane == 0) {
        double loss = far * scale;
        if (n.total != 0.0) loss += n.total * (whole - (((double)n.shift - scale * (double)n.center) + (double)n.shift_rest));
        // (above, the outside's reference is another one)
        if (qr > 0.0) loss += qr * (log_qr - (above ? v - lse : l - whole));
        p.loss[m] = (float)loss, p.lse[m] = (float)lse;
        if (p.rest_lse) p.rest_lse[m] = (float)v;
    }
}

// A row whose log-sums are too far from 0 for fp32 to tell its probabilities by them (masks
// alone, or logits that share a large part): one CTA takes its maxima and sums again, of all tokens
// and of those outside the entries, in passes of its own.  Rare, and written to be short.
constexpr float kFarLse = 65536.f;                       // 2^-8 of a probability, bf16's own rounding

template <typename T, int kThreads>
__device__ __noinline__ void far_row(const T* X, T* D, int64_t V, float scale, const uint32_t* bits, const int32_t* id,
                                     const float* q, int k, float g, float Q, float qr) {
    __shared__ float all[kThreads / 32], out[kThreads / 32];
    const int warp = threadIdx.x >> 5;
    auto named = [&](int64_t v) { return bits[v >> 5] >> (v & 31) & 1; };
    float top = kLowest, top_out = kLowest, sum = 0.f, sum_out = 0.f;
    for (int64_t v = threadIdx.x; v < V; v += kThreads) {
        const float x = value(X, v);
        top = fmaxf(top, x);
        if (!named(v)) top_out = fmaxf(top_out, x);
    }
    all[warp] = warp_max(top), out[warp] = warp_max(top_out);
    __syncthreads();
    for (int w = 0; w < kThreads / 32; ++w) top = fmaxf(top, all[w]), top_out = fmaxf(top_out, out[w]);
    __syncthreads();
    for (int64_t v = threadIdx.x; v < V; v += kThreads) {
        const float x = value(X, v);
        sum += expf((x - top) * scale);
        if (!named(v)) sum_out += expf((x - top_out) * scale);
    }
    all[warp] = warp_sum(sum), out[warp] = warp_sum(sum_out);
    __syncthreads();
    sum = sum_out = 0.f;
    for (int w = 0; w < kThreads / 32; ++w) sum += all[w], sum_out += out[w];
    const float a = Q / sum, b = qr > 0.f && sum_out > 0.f ? qr / sum_out : 0.f;
    for (int64_t v = threadIdx.x; v < V; v += kThreads) {  // a thread's own logits, which D may overwrite
        const float x = value(X, v);
        float less = 0.f;
        if (named(v)) {
            for (int j = 0; j < k; ++j) less += id[j] == v ? q[j] : 0.f;
        } else if (b != 0.f) {
            less = b * expf((x - top_out) * scale);
        }
        put(D, v, g * (a * expf((x - top) * scale) - less));
    }
}

template <typename T, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads)
distill_grad_kernel(const __grid_constant__ DistillParams p, int ranks) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float factors[6];                         // outside: a exp(y - r); inside: g (Q exp(y - l) - q); q_r
    __shared__ bool far;
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
    Entries<kThreads> n(smem, p, m);
    Chunk<T> now[kFlight];
    fetch<kThreads>(now, X, at, end);
    n.load(p, X, true);
    n.settle(p);                                         // the entries' logits are read before any of this CTA's is overwritten
    __syncthreads();
    if (threadIdx.x < 32 && n.any) {
        n.weigh(p, m, [](int, float, float) {});
        if (threadIdx.x == 0) {
            const float qr = (float)n.rest(p), lse = p.lse[m], g = p.g[m] * p.scale, Q = (float)n.total + qr;
            float a = g * Q, r2 = lse * kLog2e;
            far = fabsf(lse) > kFarLse;
            if (qr > 0.f && p.rest_lse[m] > -INFINITY) {
                const float rest = p.rest_lse[m];
                far |= fabsf(rest) > kFarLse;
                a = g * (Q * expf(rest - lse) - qr), r2 = rest * kLog2e;
            }
            factors[0] = a, factors[1] = r2, factors[2] = g, factors[3] = Q, factors[4] = lse * kLog2e, factors[5] = qr;
        }
    }
    __syncthreads();
    const float c = p.scale * kLog2e, a = factors[0], r2 = factors[1], g = factors[2], Q = factors[3], l2 = factors[4];
    if (!n.any || Q == 0.f) {                            // no entries, or none of any weight: zeros, whatever the row holds
        for (; at < end; at += kThreads) __stcs(reinterpret_cast<uint4*>(D + (int64_t)at * N), make_uint4(0, 0, 0, 0));
        for (int64_t v = (int64_t)end * N + threadIdx.x; v < hi; v += kThreads) put(D, v, 0.f);
        return;
    }
    if (far) {                                           // one CTA's, since D may be X
        if (rank == 0) far_row<T, kThreads>(X, D, p.V, p.scale, n.bits, n.id, n.q, p.k, g, Q, factors[5]);
        return;
    }
    auto grad = [&](float x) { return a * ex2(fmaf(x, c, -r2)); };
    for (; at < end; at += kFlight * kThreads) {
        Chunk<T> next[kFlight];
        fetch<kThreads>(next, X, at + kFlight * kThreads, end);
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            const int g4 = at + u * kThreads;
            if (g4 < end) __stcs(reinterpret_cast<uint4*>(D + (int64_t)g4 * N), now[u].map(grad));
            now[u] = next[u];
        }
    }
    for (int64_t v = (int64_t)end * N + threadIdx.x; v < hi; v += kThreads) put(D, v, grad(value(X, v)));
    __syncthreads();
    for (int i = threadIdx.x; i < p.k; i += kThreads) {
        const int64_t t = n.id[i];
        if (t < lo || t >= hi) continue;                 // -1 is below every CTA's
        float q = n.q[i];
        if (n.twice) {                                   // a token named twice has both entries' weight
            q = 0.f;
            for (int j = 0; j < p.k; ++j) q += n.id[j] == t ? n.q[j] : 0.f;
        }
        put(D, t, g * (Q * ex2(fmaf(n.x[i], c, -l2)) - q));
    }
}

using Kernel = void(const DistillParams, int);
// [gradient][bf16][128 threads]
Kernel* const kKernels[2][2][2] = {
    {{distill_kernel<float, 256>, distill_kernel<float, 128>}, {distill_kernel<uint16_t, 256>, distill_kernel<uint16_t, 128>}},
    {{distill_grad_kernel<float, 256>, distill_grad_kernel<float, 128>},
     {distill_grad_kernel<uint16_t, 256>, distill_grad_kernel<uint16_t, 128>}}};

// Clusters of 16 and more than 48 KB of shared memory have to be asked for, once a device.
cudaError_t ask() {
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && ready.load(std::memory_order_relaxed) >> dev & 1)) return e;
    for (auto& some : kKernels)
        for (auto& pair : some)
            for (Kernel* k : pair) {
                e = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
                if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
                if (e != cudaSuccess) return e;
            }
    if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
    return e;
}

// Threads and CTAs a row.  Measured (us by events, one state, every row counted: with 0.1 of the rows not
// counted 4096 of 152064 take 187 and 365):
// - loss, more rows than find a place at 256 threads (four CTAs an SM): 128 threads, a CTA a
//   row, 777 rows of 50257 fp32 34 (256 threads 40), 1500 of 32000 bf16 29 (31), 4096 of 152064
//   bf16 199 (205); two CTAs a row 41, 34, 213;
// - gradient, more rows than SMs: 128 threads, two CTAs a row and up to 80 KB of logits each,
//   4096 of 152064 bf16 383 (a CTA a row 405, 256 threads 401 and 391 with two), 2000 of them
//   fp32 368 (389; 384, 376), 300 bf16 31.5 (43; 34, 32), 1500 of 32000 33.8 (37.9; 34.6, 39.6);
// - otherwise 256 threads and as many CTAs as make the least of the waves (half a wave more
//   where there is more than one) times a CTA's time: its bytes at its share of HBM's rate or
//   at what its own loads in flight allow, and what comes before and after, some 2 us, with a
//   cluster to join 4.5, in the gradient 1.5.  64 rows of 152064: loss 20, 14, 13, 12 with 1, 2, 4
//   and 8 CTAs a row.  Clusters of 16 only with an SM a CTA; each thread keeps two loads.
struct Shape {
    int small, ranks;                                     // 128 threads; CTAs a row
};
Shape shape_of(bool backward, bool bf16, const DistillParams& p) {
    const int64_t sms = num_sms(), row = p.V / (bf16 ? 8 : 4) * 16;
    if (!backward && p.M > 4 * sms) return {1, 1};
    int ranks = 1;
    if (backward && p.M > sms) {
        while (ranks < kMostRanks && (row / ranks > 80 * 1024 || (ranks == 1 && row >= 2 * 32 * 128))) ranks *= 2;
        return {1, ranks};
    }
    const double bytes = (double)(backward ? 2 * row : row);
    double least = 1e30;
    for (int r = 1; r <= kMostRanks; r *= 2) {
        if (r > 1 && (row < (int64_t)r * 32 * 256 || (r > 8 && r * p.M > sms))) break;
        const int64_t ctas = r * p.M, slots = 4 * sms;
        const double rate = std::min(backward ? 36e3 : 20e3, 6.7e6 / (double)std::min(ctas, slots));   // bytes a us
        const double waves = ctas <= slots ? 1.0 : (double)ctas / slots + 0.5;
        const double cost = waves * (bytes / r / rate + (backward ? 1.5 : r > 1 ? 4.5 : 2.0));
        if (cost < least) least = cost, ranks = r;
    }
    return {0, ranks};
}

cudaError_t launch(bool backward, bool bf16, const DistillParams& p, cudaStream_t st) {
    const cudaError_t e = ask();
    if (e != cudaSuccess) return e;
    const Shape shape = shape_of(backward, bf16, p);
    const int small = shape.small, ranks = shape.ranks;
    const bool cluster = !backward;
    Kernel* const f = kKernels[backward][bf16][small];
    const size_t smem = smem_bytes(p.k, p.V, !cluster || p.rest_lse);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.M * ranks));
    cfg.blockDim = dim3(256 >> small);
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
    return launch(backward, bf16, p, st);
}

}  // namespace fp8rl
