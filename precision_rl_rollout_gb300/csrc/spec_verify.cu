// spec_verify.cu -- verification of drafted tokens against the target model's
// probabilities, with every random number given.
//
// Draft i of a sequence (token t_i, drawn from q_i) is kept while
// u_i q_i(t_i) < p_i(t_i); both factors are fp32 or bf16, so the product is
// exact in fp64 and the decision is exact.  At the first refusal n the sequence
// gets one token from the residual max(p_n - q_n, 0), after len accepted drafts
// one from p_len: as an exponential race, argmax_v w_v / e_v with e_v ~ Exp(1)
// given.  Each score is one IEEE division, so the winner does not depend on how
// the vocabulary is split; equal scores go to the lowest index.
//
// Only row n of p and q and the sequence's e are read: 12 bytes a vocabulary
// entry, bound by HBM in a batch and by latency for one sequence.  A cluster of
// CTAs shares a row; each finds n for itself and takes part of the row, the
// parts' winners meet in the CTAs' shared memory.
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "sm100_ptx.cuh"

namespace fp8rl {

namespace {

constexpr uint32_t kKernelVerify = 9;
constexpr int kVThreads = 512;
constexpr int kVWarps = kVThreads / 32;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }

// Four entries of a row that starts on their boundary, past L1 (each is read once).
template <typename T>
struct Quad;
template <>
struct Quad<float> {
    uint4 x;
    __device__ __forceinline__ void load(const float* p) { x = ld_stream_v4(p); }
    __device__ __forceinline__ float at(int k) const {
        return __uint_as_float(k == 0 ? x.x : k == 1 ? x.y : k == 2 ? x.z : x.w);
    }
};
template <>
struct Quad<uint16_t> {
    uint2 x;
    __device__ __forceinline__ void load(const uint16_t* p) {
        asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(x.x), "=r"(x.y) : "l"(p));
    }
    __device__ __forceinline__ uint16_t at(int k) const { return (uint16_t)((k < 2 ? x.x : x.y) >> (k & 1 ? 16 : 0)); }
};

// The race so far: score bits and one (scores are >= 0, so they order as integers) and
// the complement of the index, as one 64-bit key; larger wins.  Without an entry that
// takes part (score -1) the upper half is 0 and the index 0: an entry of positive weight
// takes part even where its score rounds to 0.
__device__ __forceinline__ uint64_t race_key(float score, uint32_t idx) {
    return ((uint64_t)(score < 0.f ? 0u : __float_as_uint(score) + 1u) << 32) | (uint32_t)~idx;
}
__device__ __forceinline__ uint64_t warp_max_key(uint64_t k) {
    const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32));
    const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
    return ((uint64_t)hi << 32) | lo;
}

template <typename T>
__global__ void __launch_bounds__(kVThreads, 2)
spec_verify_kernel(const __grid_constant__ VerifyParams p) {
    __shared__ uint64_t wkey[kVWarps];
    __shared__ uint64_t part[2][16];           // [round][cluster rank], written by every CTA of the cluster
    __shared__ int s_n, s_len;
    sm100::cluster_arrive();                    // every CTA of the cluster has started (waited for below)
    pdl_wait_then_release();
    const uint32_t rank = sm100::cluster_ctarank(), ranks = gridDim.x;
    const int64_t b = blockIdx.y;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const T* P = static_cast<const T*>(p.P) + b * p.p_seq;
    const T* Q = p.Q ? static_cast<const T*>(p.Q) + b * p.q_seq : nullptr;
    if (warp == 0) {
        int len = p.lens ? p.lens[b] : p.K;
        if (len < 0 || len > p.K) {
            if (lane == 0) atomicCAS(p.err, 0u, (kKernelVerify << 24) | (1u << 16) | 2u);
            len = len < 0 ? 0 : p.K;
        }
        bool keep = false;
        if (lane < len) {
            const int32_t tok = p.drafts[b * p.K + lane];
            if (tok >= 0 && tok < p.V) {
                const double u = (double)p.u[b * p.K + lane];
                const double pt = (double)to_f32(P[lane * p.p_step + tok]);
                const double qt = Q ? (double)to_f32(Q[lane * p.q_step + tok]) : 1.0;
                keep = u * qt < pt;
            } else {
                atomicCAS(p.err, 0u, (kKernelVerify << 24) | (2u << 16) | 2u);
            }
        }
        const uint32_t refused = ~__ballot_sync(0xffffffffu, keep);   // lanes from len on count as refused
        if (lane == 0) {
            s_len = len;
            s_n = refused ? __ffs((int)refused) - 1 : 32;
        }
    }
    __syncthreads();
    const int n = s_n, len = s_len;
    bool residual = n < len;
    const T* pr = P + n * p.p_step;
    const T* qr = residual && Q ? Q + n * p.q_step : nullptr;
    const int32_t drop = residual && !Q ? p.drafts[b * p.K + n] : -1;   // a drafter without probabilities: q is 1 there
    const float* e = p.noise + b * p.e_seq;
    const int32_t V = (int32_t)p.V, step = (int32_t)(ranks * kVThreads), v_first = (int32_t)(rank * kVThreads + threadIdx.x);
    // This thread's part of the race, several entries a turn with their loads in
    // flight together.  A quotient that rounds to more than top is more than top, so
    // w > top * e, and all the more w > top * e rounded down (subnormal numbers too):
    // one product settles nearly every entry without dividing.
    float top = -1.f;
    uint32_t at = 0;
    auto entry = [&](int32_t v, float w, float d) {
        if (w > __fmul_rd(top, d) && w > 0.f) {
            const float s = __fdiv_rn(w, d);
            if (s > top) top = s, at = (uint32_t)v;
        }
    };
    auto race = [&](auto minus_q) {
        constexpr bool kQ = decltype(minus_q)::value;
        const int32_t skip = kQ || !residual ? -1 : drop;
        auto weight = [&](int32_t v, T w, T q) {
            const float x = kQ ? __fsub_rn(to_f32(w), to_f32(q)) : to_f32(w);
            return !kQ && v == skip ? 0.f : x;
        };
        auto aligned = [](const void* x, uintptr_t n) { return (reinterpret_cast<uintptr_t>(x) & (n - 1)) == 0; };
        int32_t v, turn;
        if (aligned(pr, 4 * sizeof(T)) && aligned(e, 16) && (!kQ || aligned(qr, 4 * sizeof(T)))) {
            // rows that start on the boundary of four entries: 59 us for 256 rows of
            // 152064 in fp32, against 72 us an entry at a time
            constexpr int U = 3;
            for (v = 4 * v_first, turn = 4 * step; v + 3 < V - (U - 1) * turn; v += U * turn) {
                Quad<T> w[U], q[U];
                Quad<float> d[U];
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    w[i].load(pr + v + i * turn);
                    if constexpr (kQ) q[i].load(qr + v + i * turn);
                    d[i].load(e + v + i * turn);
                }
#pragma unroll
                for (int i = 0; i < U; ++i)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int32_t x = v + i * turn + k;
                        entry(x, weight(x, w[i].at(k), kQ ? q[i].at(k) : T{}), d[i].at(k));
                    }
            }
            for (; v < V; v += turn)
                for (int32_t x = v; x < v + 4 && x < V; ++x) entry(x, weight(x, pr[x], kQ ? qr[x] : T{}), e[x]);
            return;
        }
        constexpr int U = 8;
        for (v = v_first; v < V - (U - 1) * step; v += U * step) {
            T w[U], q[U];
            float d[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                w[i] = pr[v + i * step];
                if constexpr (kQ) q[i] = qr[v + i * step];
                d[i] = e[v + i * step];
            }
#pragma unroll
            for (int i = 0; i < U; ++i) entry(v + i * step, weight(v + i * step, w[i], kQ ? q[i] : T{}), d[i]);
        }
        for (; v < V; v += step) entry(v, weight(v, pr[v], kQ ? qr[v] : T{}), e[v]);
    };
    uint64_t best = 0;
    for (int round = 0;; ++round) {
        top = -1.f, at = 0;
        if (residual && qr)
            race(std::true_type{});
        else
            race(std::false_type{});
        uint64_t key = warp_max_key(race_key(top, at));
        if (lane == 0) wkey[warp] = key;
        __syncthreads();
        if (round == 0) sm100::cluster_wait();
        if (warp == 0) {
            key = warp_max_key(lane < kVWarps ? wkey[lane] : 0ull);
            if (lane < ranks) sm100::st_cluster_u64(sm100::map_to_rank(sm100::smem_u32(&part[round][rank]), lane), key);
        }
        __syncwarp();
        sm100::cluster_arrive();
        sm100::cluster_wait();
        best = part[round][0];
        for (uint32_t r = 1; r < ranks; ++r) best = part[round][r] > best ? part[round][r] : best;
        // a residual with nothing in it (p <= q everywhere, by rounding): draw from p
        if (!residual || (best >> 32)) break;
        residual = false;
        __syncthreads();
    }
    if (rank == 0) {
        const int32_t token = (int32_t)~(uint32_t)best;
        for (int i = threadIdx.x; i <= p.K; i += kVThreads)
            p.out[b * (p.K + 1) + i] = i < n ? p.drafts[b * p.K + i] : i == n ? token : -1;
        if (threadIdx.x == 0) p.accepted[b] = n;
    }
}

}  // namespace

cudaError_t launch_spec_verify(const VerifyParams& a, bool bf16, cudaStream_t st) {
    VerifyParams p = a;
    p.err = device_error_word();
    if (!p.err) return cudaErrorUnknown;
    cudaLaunchConfig_t cfg = {};
    // As many CTAs a row as one wave of two CTAs an SM holds for the whole batch, up to
    // eight; 16 (for which a kernel has to ask) while they leave each CTA an SM of its
    // own: one row of 152064 takes 6.9 us so and 7.5 with eight, but 19 rows 14.2 and
    // 10.3, their clusters not all finding a place at once.
    static std::atomic<uint64_t> ready{0};                    // devices on which it has
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
        for (auto k : {spec_verify_kernel<uint16_t>, spec_verify_kernel<float>}) {
            e = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e != cudaSuccess) return e;
        }
        if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    unsigned c = 16 * p.B <= num_sms() ? 16 : 8;
    while (c > 1 && (int64_t)c * p.B > 2 * (int64_t)num_sms()) c /= 2;
    cfg.gridDim = dim3(c, (unsigned)p.B);
    cfg.blockDim = dim3(kVThreads);
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim = {c, 1, 1};
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, bf16 ? spec_verify_kernel<uint16_t> : spec_verify_kernel<float>, p);
}

}  // namespace fp8rl
