// attn_paged.cuh -- attention of a sequence's new tokens over a paged key-value
// cache, as one pass over the cache with a running maximum and sum.  Query i of
// Lq stands at position p = len - Lq + i and sees the cached tokens j with
// max(0, p - window + 1) <= j <= p (window 0: from 0 on):
//   x_j = scale q.k_j,  o = sum_j e^(x_j - m) v_j / sum_j e^(x_j - m);
// a query that sees nothing gets zeros and a log-sum of -inf.
//
// What bounds it.  Every cached key and value is read once and meets the group's
// query rows (query heads of the kv head x Lq): rows flop a bf16 byte, 2 rows an E4M3
// byte.  With the 5-8 rows of one new token that is far below the tensor
// cores' rate at HBM speed, and the kernel is a stream: 128 sequences of 40/8 heads
// of 128 over bf16, 4.3 GB, in 658 us (6.6 TB/s, 97% of a plain copy), one sequence
// of 131072 tokens in 84 us (6.4 TB/s); 64 ragged sequences of 28/4 heads over E4M3,
// 270 MB, in 52 us (5.2 TB/s; the start, the last tiles and the join are 11 of it).
// Five new tokens over E4M3 (25 rows, 32 in the product) take 140 us for 555 MB:
// m16n8k16 runs at 8.3 cycles a scheduler here, 61 us of it, and the conversions,
// exponentials and matrix loads around it do not all hide behind one another.
//
// Why mma.sync.  tcgen05 wants 128 rows an instruction on the M side, 16-bit
// operands on both sides or 8-bit ones on both.  Tokens or head values can be that
// side, but E4M3 values would have to go through registers and shared memory again
// as fp16 (queries and probabilities do not fit 8 bits: the tail of a long row is
// more than 2^18 below its maximum), and the probabilities through tensor memory
// and back, for a product that mostly waits for HBM.  mma.sync.m16n8k32 on E4M3 with
// the queries as two E4M3 parts was tried for the scores: exact enough, but it
// costs 10-15 cycles with fresh operands, more than fp16 with one conversion
// shared by all rows (verification 285 us against 149).  More than 32 rows over
// bf16 are worth tcgen05, with tokens as that side: attn_paged_wide.cuh.
//
// The CTA.  Four warps compute, a fifth loads: it keeps a ring of tiles (K and V of
// CT tokens) full, by the copy engine where pages hold a multiple of 8 tokens, else
// 16 bytes a lane.  A tile's work in each warp: S^T = K Q^T for its own tokens
// (tokens the M side, 8 query rows the N side: a group of 5-8 heads fills it); the
// probabilities of its tokens into shared memory; then O^T += V^T P^T for its own
// quarter of the head over all tokens of the tile.  So a warp holds 1/4 of the sums
// (the same rows summed by four warps over their own tokens took the registers of
// two CTAs, and a reduction of all sums at every item's end), and the sums need no
// joining inside the CTA.  The loads were first issued between the products by the
// warps themselves; that was 500 cycles on every tile's way (63 -> 54 us, 64
// sequences over E4M3).
//
// Operands.  K comes through ldmatrix, V and the probabilities through its and
// stmatrix's transposing forms.  E4M3 is converted to fp16 in registers (exact);
// the key's values are taken in an order of the head dimension that makes each
// 4-byte piece of a row two operand words, Q follows the same order, and transposed
// V comes out as even and odd head values.  For E4M3 caches the bf16 queries are
// held as fp16, scaled by a power of two that puts the row's largest value at 2^14
// (exact down to 2^-28 of it).  Probabilities are rounded to the product's type
// relative to the running reference (fp16: times 2^6, so that 2^-20 of the maximum
// is still a normal number); their sum is of the unrounded fp32 values.
//
// Running reference.  A row's reference is the CTA's and moves only when some score
// passes it by 2^8: exact arithmetic does not change, and fp32 sums, bf16 and fp16
// probabilities all have the room.
//
// Work split.  The unit is a tile of one item (sequence, kv head, chunk of query
// rows).  All tiles of the batch, in item order, with a few places more for each
// item's start and end, are cut into equal ranges, one a CTA, one wave of CTAs:
// ragged lengths need no plan on the host, and one long sequence spreads over the
// GPU.  The lengths are read on the device.  A CTA writes an item that lies wholly
// in its range; of items that do not it has at most two, whose unnormalised sums go
// to its two slots of the workspace, joined in a second launch in CTA order.  A
// short batch is one launch: each item has a cluster of CTAs, which join their sums
// through each other's shared memory, a part of the rows each (1 x 777 tokens: 10.3 ->
// 7.1 us).  "Short" goes by the host's bound max_len: under a loose one the same batch
// takes the two launches.
#pragma once

#include <math.h>

#include <atomic>

#include "common.cuh"
#include "internal.h"
#include "sm100_ptx.cuh"

namespace fp8rl {
namespace attn {
namespace {      // each translation unit its own configurations

constexpr uint32_t kKernelAttn = 10;
constexpr int kWarps = 4, kConsumers = kWarps * 32, kThreads = kConsumers + 32;   // and a warp that loads
constexpr float kLazy = 8.f;                  // log2 by which a score may pass the reference before a rescale
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kNone = -3.402823466e38f;     // reference of a row that has seen nothing: any score passes it
constexpr uint64_t kWaitLimitNs = 2000000000ull;   // 2 s: far above any legitimate wait

template <bool kE4m3_, bool kTma_, int DP_, int RT_>
struct Config {
    static constexpr bool kE4m3 = kE4m3_, kTma = kTma_;
    static constexpr int DP = DP_;                           // padded head width
    static constexpr int RT = RT_, NT = RT / 8;              // query rows of a CTA, in tiles of eight
    static constexpr int ES = kE4m3 ? 1 : 2, RB = DP * ES;   // bytes of a value, of a cached head
    static constexpr int PB = RB < 128 ? RB : 128;           // row bytes of a piece of a tile
    static constexpr int CPR = RB / 16;                      // 16-byte chunks of a cached head
    static constexpr int MT = RT <= 16 && RB <= 128 ? 2 : 1;   // 16-token tiles a warp
    static constexpr int TT = 16 * MT, CT = kWarps * TT;     // tokens of a warp, of a CTA's tile
    static constexpr int MW = DP / 64;                       // 16-value tiles of the head a warp sums
    static constexpr int kTile = CT * RB, kStage = 2 * kTile;
    // Probabilities, 16 bits; bf16 ones as the sum of two where a few rows leave the
    // tensor cores idle: one rounding of 2^-8 beside the result's own makes the
    // output's error 1.3 times a single rounding's (2.1e-3 and 1.65e-3 of its norm).
    // With 17 to 32 rows the second part costs 25 rows of 32 sequences to 16384 184 ->
    // 194 us, with heads of 64 128 -> 152: one there.
    static constexpr int kParts = !kE4m3 && RT <= 16 ? 2 : 1, kPart = RT * CT * 2, kP = kParts * kPart;
    static constexpr int kQ = NT * (DP / 32) * 512;          // query operands
    static constexpr int kSmall = RT * 4 * (kWarps + 3) + 12 * 8 + 16;
    // CTAs an SM.  Two for heads of 256 over E4M3, of 64 tokens a tile, rather than one
    // of 128: 120 sequences to 57, 16/16 heads: 63 -> 30 us; 64 of 8191, 28/4: 171 -> 169
    // (three: 25 and 176).
    static constexpr int kCtas = DP > 128 ? (kE4m3 ? 2 : 1) : kE4m3 ? 3 : 2;
    static constexpr int kBudget = 233472 / kCtas - 1024;    // 228 KB an SM, 1 KB of it kept for each CTA
    static constexpr int kRest = kP + kQ + kSmall;
    static constexpr int kFit = (kBudget - kRest) / kStage;
    // 128 KB in flight on an SM keep HBM busy.  More is slower: three tiles a CTA
    // instead of two took 703 us where these take 654 (128 sequences, bf16).
    static constexpr int kWant = 131072 / (kCtas * kStage) > 2 ? 131072 / (kCtas * kStage) : 2;
    static constexpr int kStages = kFit < kWant ? kFit : kWant < 6 ? kWant : 6;
    static constexpr int kSmem = kStages * kStage + kRest;
    // what an item costs a CTA beside its tiles (queries, result), in tiles, as the
    // time of 64 KB (with many rows 96 KB) of the cache
    static constexpr int kCost = RT > 16 ? 98304 : 65536, kItem = kCost / kStage > 1 ? kCost / kStage : 1;
    static_assert(kStages >= 2, "too little shared memory for two stages");
};

// The tokens [lo, len) a sequence's queries see at all, and the item's tiles from
// `start` on (lo rounded down to a box of the cache's pages); one tile at least,
// so that every item has a writer.
struct Span {
    int start, lo, len, tiles;
};
template <bool kL2 = false>
__device__ __forceinline__ Span span_of(const AttnParams& p, int b, int ct) {
    Span s;
    s.len = min(max(kL2 ? __ldcg(p.lens + b) : p.lens[b], 0), p.max_len);
    s.lo = p.window ? max(0, s.len - p.Lq + 1 - p.window) : 0;
    s.start = s.lo & -p.box;
    s.tiles = max(1, (s.len - s.start + ct - 1) / ct);
    return s;
}

// Places in the order of all work: an item takes kItem places, then one a tile.
// The whole warp: places of sequences [0, b_end), and of all; hr items a sequence.
template <class C, bool kL2 = false>
__device__ __forceinline__ void count_places(const AttnParams& p, int hr, int b_end, int64_t* before, int64_t* total) {
    const int lane = threadIdx.x & 31;
    int64_t x = 0, y = 0;
#pragma unroll 4
    for (int b = lane; b < p.B; b += 32) {
        const int n = span_of<kL2>(p, b, C::CT).tiles + C::kItem;
        y += n;
        if (b < b_end) x += n;
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) {
        if (b_end) x += __shfl_xor_sync(0xffffffffu, x, off);
        y += __shfl_xor_sync(0xffffffffu, y, off);
    }
    *before = x * hr;
    *total = y * hr;
}

__device__ __forceinline__ int64_t div_ceil(int64_t a, int b) {
    return (a + b - 1) >> 32 ? (a + b - 1) / b : (uint32_t)(a + b - 1) / (uint32_t)b;
}

// ---------------------------------------------------------------- PTX

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// The thread's copies so far count as its arrival on the barrier when they are done.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm2_t(uint32_t (&r)[2], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr));
}
template <bool kF16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (kF16)
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The low and high two of four E4M3 codes as fp16 pairs (exact; NaN stays NaN).
__device__ __forceinline__ void e4m3x4_f16(uint32_t v, uint32_t& lo, uint32_t& hi) {
    asm("{\n.reg .b16 l, h;\nmov.b32 {l, h}, %2;\ncvt.rn.f16x2.e4m3x2 %0, l;\ncvt.rn.f16x2.e4m3x2 %1, h;\n}"
        : "=r"(lo), "=r"(hi)
        : "r"(v));
}
__device__ __forceinline__ uint32_t pack2_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Shared-memory offset of chunk c of row r of a tile: pieces of 128 bytes a row,
// 16-byte chunks exchanged as the copy engine's 128-byte (for rows of 64 bytes:
// 64-byte) swizzle does, so that the eight rows of a matrix load lie in different
// banks.
template <class C>
__device__ __forceinline__ uint32_t swz(int r, int c) {
    if constexpr (C::RB >= 128)
        return (uint32_t)((c >> 3) * (C::CT * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
    else
        return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}
// The same for the probabilities: row of a query, chunk of eight tokens.
template <class C>
__device__ __forceinline__ uint32_t swz_p(int r, int c) {
    return (uint32_t)((c >> 3) * (C::RT * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}
__device__ __forceinline__ void ldsm2(uint32_t (&r)[2], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr));
}
__device__ __forceinline__ void stsm4_t(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b),
                 "r"(c), "r"(d)
                 : "memory");
}
__device__ __forceinline__ void stsm2_t(uint32_t addr, uint32_t a, uint32_t b) {
    asm volatile("stmatrix.sync.aligned.m8n8.x2.trans.shared.b16 [%0], {%1,%2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}

// Brings an address's sector to L1 (the value is not used).
__device__ __forceinline__ void touch_l1(const void* p) {
    uint32_t v;
    asm volatile("ld.global.u32 %0, [%1];" : "=r"(v) : "l"(p));
    (void)v;
}
__device__ __forceinline__ void st_zero16(uint32_t addr) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(addr), "r"(0) : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* tmap, uint32_t bar, int32_t c0, int32_t c1,
                                            int32_t c2, int32_t c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
        : "memory");
}

// One cached value in shared memory.
template <bool kE4m3>
__device__ __forceinline__ float ld_value(uint32_t addr) {
    uint32_t raw;
    if constexpr (kE4m3) {
        uint32_t f16, unused;
        asm volatile("ld.shared.u8 %0, [%1];" : "=r"(raw) : "r"(addr) : "memory");
        e4m3x4_f16(raw, f16, unused);
        return __half2float(__ushort_as_half((unsigned short)f16));
    } else {
        asm volatile("ld.shared.u16 %0, [%1];" : "=r"(raw) : "r"(addr) : "memory");
        return __uint_as_float(raw << 16);
    }
}
template <bool kE4m3>
__device__ __forceinline__ void st_zero(uint32_t addr) {
    if constexpr (kE4m3)
        asm volatile("st.shared.u8 [%0], %1;" ::"r"(addr), "r"(0) : "memory");
    else
        asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"((uint16_t)0) : "memory");
}

// ---------------------------------------------------------------- the kernel

// A tile of the CTA's range; `place` counts from the range's first.
struct Cursor {
    Span s;
    int b, hr, tile, place;
    template <class C>
    __device__ __forceinline__ void next(const AttnParams& p, int hr_n) {
        ++place;
        if (++tile < s.tiles) return;
        tile = 0;
        place += C::kItem;
        if (++hr < hr_n) return;
        hr = 0;
        if (++b < p.B) s = span_of(p, b, C::CT);
    }
};

// The CTA's range of places: its length (or 0), and its first tile in `at`.
template <class C>
__device__ __forceinline__ int first_tile(const AttnParams& p, int hr_n, Cursor& at) {
    const int lane = threadIdx.x & 31;
    at.place = 0;
    int64_t before, total;
    count_places<C>(p, hr_n, 0, &before, &total);
    const int64_t chunk = div_ceil(total, gridDim.x), u0 = (int64_t)blockIdx.x * chunk;
    const int size = (int)(total - u0 < chunk ? total - u0 : chunk);
    if (size <= 0) return 0;
    int64_t base = 0;                                         // first place of the sequence the range begins in
    for (int b0 = 0;; b0 += 32) {
        const int n = b0 + lane < p.B ? span_of(p, b0 + lane, C::CT).tiles + C::kItem : 0;
        int64_t inc = n;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t o = __shfl_up_sync(0xffffffffu, inc, off);
            if (lane >= off) inc += o;
        }
        const uint32_t in = __ballot_sync(0xffffffffu, base + inc * hr_n > u0);
        const int l = in ? __ffs((int)in) - 1 : 31;
        base += __shfl_sync(0xffffffffu, (in ? inc - n : inc) * hr_n, l);
        at.b = b0 + l;
        if (in) break;
    }
    at.s = span_of(p, at.b, C::CT);
    const int64_t in = u0 - base;                             // below 2^31 items of a sequence
    const int each = at.s.tiles + C::kItem;
    at.hr = (int)(in >> 32 ? in / each : (uint32_t)in / (uint32_t)each);
    at.tile = max(0, (int)(in - (int64_t)at.hr * each) - C::kItem);
    at.place = (int)((int64_t)at.hr * each + C::kItem + at.tile - in);
    return size;
}

// kCluster: an item a cluster (p.cluster CTAs); else the tiles are cut into ranges.
template <class C, bool kCluster>
__global__ void __launch_bounds__(kThreads, C::kCtas)
attn_paged_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap) {
    extern __shared__ __align__(1024) uint8_t smem[];          // the ring first: the swizzle wants 1 KB
    constexpr bool kE = C::kE4m3, kTma = C::kTma;
    constexpr int NT = C::NT, RT = C::RT, TT = C::TT, MT = C::MT, CT = C::CT, ES = C::ES, MW = C::MW;
    constexpr int KS = C::DP / 16, S = C::kStages;
    constexpr float kBias = kE ? 6.f : 0.f;
    uint8_t* const smem_p = smem + S * C::kStage;
    uint4* const sq = reinterpret_cast<uint4*>(smem_p + C::kP);               // [row tile][KS / 2][lane]
    float* const s_fac = reinterpret_cast<float*>(smem_p + C::kP + C::kQ);    // [RT] log2 units of a unit of the product
    int* const s_hi = reinterpret_cast<int*>(s_fac + RT);                     // [RT] tokens lo .. hi - 1 are seen
    int* const s_lo = s_hi + RT;
    float* const s_w = reinterpret_cast<float*>(s_lo + RT);                   // [warp][RT] maxima, sums
    const uint32_t full = sm100::smem_u32(s_w + kWarps * RT), empty = full + 48;   // [S] each
    volatile int* const abort = reinterpret_cast<int*>(s_w + kWarps * RT) + 24;

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int group = p.Hq / p.Hkv, rows = group * p.Lq, chunks = (rows + RT - 1) / RT, hr_n = p.Hkv * chunks;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            sm100::mbar_init(full + 8 * i, kTma ? 1 : 32);     // one arrival and its bytes, or each lane's copies
            sm100::mbar_init(empty + 8 * i, kWarps);
        }
        *abort = 0;
        sm100::fence_mbar_init();
        if constexpr (kTma) {
            sm100::prefetch_tmap(&kmap);
            sm100::prefetch_tmap(&vmap);
        }
    }
    __syncthreads();
    pdl_wait_then_release();

    if (sm100::smem_u32(smem) & 1023u) {                       // as the runtime places it; nothing below would fit
        if (threadIdx.x == 0) atomicCAS(p.err, 0u, (kKernelAttn << 24) | (4u << 16) | 2u);
        return;
    }
    if (blockIdx.x == 0 && warp == 0)
        for (int b = lane; b < p.B; b += 32)
            if (p.lens[b] < 0 || p.lens[b] > p.max_len) atomicCAS(p.err, 0u, (kKernelAttn << 24) | (1u << 16) | 2u);
    Cursor at;
    int size;
    if constexpr (kCluster) {                                 // this CTA's share of the cluster's item
        const int item = blockIdx.x / p.cluster, rank = blockIdx.x - item * p.cluster;
        at.b = item / hr_n, at.hr = item - at.b * hr_n;
        at.s = span_of(p, at.b, C::CT);
        const int each = (at.s.tiles + p.cluster - 1) / p.cluster;
        at.tile = rank * each;
        at.place = 0;
        size = min(each, at.s.tiles - at.tile);               // none or less: nothing of it
    } else {
        size = first_tile<C>(p, hr_n, at);
        if (at.place >= size) return;                         // no work, or the range ends before its first tile
    }

    const uint32_t ring = sm100::smem_u32(smem);              // a tile a slot
    auto head_of = [&](const Cursor& c) { return chunks == 1 ? c.hr : c.hr / chunks; };
    bool dead = false;                                        // a wait ran out: nothing more is loaded or waited for
    auto wait = [&](uint32_t bar, uint32_t parity, uint32_t site) {
        if (!dead && !sm100::mbar_wait_bounded(bar, parity, abort, kWaitLimitNs)) {
            if (lane == 0) atomicCAS(p.err, 0u, (kKernelAttn << 24) | (site << 16) | 1u);
            *abort = 1;
            dead = true;
        }
        dead = __any_sync(0xffffffffu, dead);
    };

    // The loading warp keeps every slot full; nothing it does is on the other warps'
    // way (loads issued between their products cost 500 cycles a tile).  By the copy
    // engine a lane takes a box of one page, else each lane copies 16 bytes a turn.
    if (warp == kWarps) {
        auto page_of = [&](int j) { return p.page_shift >= 0 ? j >> p.page_shift : j / p.page_size; };
        auto page_at = [&](int pg) {
            int page = p.pages[at.b * p.pages_seq + pg];
            if ((uint32_t)page >= (uint64_t)p.num_pages) {
                atomicCAS(p.err, 0u, (kKernelAttn << 24) | (2u << 16) | 2u);
                page = 0;
            }
            return page;
        };
        int n = 0;
#pragma unroll 1
        for (bool first = true; at.place < size; at.next<C>(p, hr_n), ++n, first = false) {
            const int c0 = at.s.start + at.tile * CT, h = head_of(at);
            if (first || (at.tile & 15) == 0) {               // page numbers to L1 ahead of their use, a tile a lane
                const int64_t j = c0 + (int64_t)lane * CT;
                if (j < at.s.len) touch_l1(p.pages + at.b * p.pages_seq + page_of((int)j));
            }
            const uint32_t slot = n % S, bar = full + 8 * slot, dst = ring + slot * C::kStage;
            if constexpr (kTma) {
                const int i = lane * p.box, j = c0 + i;
                const bool load = i < CT && j < at.s.len;
                const int pg = load ? page_of(j) : 0, page = load ? page_at(pg) : 0, row = j - pg * p.page_size;
                const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, load));
                if (n >= S) wait(empty + 8 * slot, (n / S - 1) & 1, 5);
                if (dead) break;
                if (lane == 0) sm100::mbar_arrive_expect_tx(bar, boxes * 2 * p.box * C::RB);
                __syncwarp();
                if (load)
#pragma unroll
                    for (int x = 0; x < C::RB / C::PB; ++x) {
                        const uint32_t d = dst + x * (CT * C::PB) + i * C::PB;
                        tma_load_4d(d, &kmap, bar, x * (C::PB / ES), p.order ? row : h, p.order ? h : row, page);
                        tma_load_4d(d + C::kTile, &vmap, bar, x * (C::PB / ES), p.order ? row : h, p.order ? h : row, page);
                    }
            } else {
                int64_t off[CT / 32];                          // this lane's tokens' offsets in bytes, -1: no such token
#pragma unroll
                for (int i = 0; i < CT / 32; ++i) {
                    const int j = c0 + i * 32 + lane;
                    off[i] = -1;
                    if (j < at.s.len) {
                        const int pg = page_of(j);
                        off[i] = (page_at(pg) * p.c_page + (int64_t)(j - pg * p.page_size) * p.c_token + h * p.c_head) * ES;
                    }
                }
                if (n >= S) wait(empty + 8 * slot, (n / S - 1) & 1, 5);
                if (dead) break;
                const int cpr = p.D * ES / 16;                // chunks the cache has of a head
                constexpr int RPI = 32 / C::CPR;              // rows a turn
#pragma unroll
                for (int i = 0; i < CT / 32; ++i)
#pragma unroll 4
                    for (int k = 0; k < 32; k += RPI) {
                        const int r = k + lane / C::CPR, c = lane % C::CPR;
                        const int64_t o = __shfl_sync(0xffffffffu, off[i], r);
                        const uint32_t bytes = o >= 0 && c < cpr ? 16u : 0u;
                        const int64_t src = bytes ? o + c * 16 : 0;
                        cp_async16(dst + swz<C>(i * 32 + r, c), static_cast<const uint8_t*>(p.kpool) + src, bytes);
                        cp_async16(dst + C::kTile + swz<C>(i * 32 + r, c), static_cast<const uint8_t*>(p.vpool) + src, bytes);
                    }
                cp_async_arrive(bar);
            }
        }
        if (dead)                                              // copies still in flight write to this CTA's memory
            for (int k = n > S ? n - S : 0; k < n; ++k) sm100::mbar_drain(full + 8 * (k % S), (k / S) & 1, kWaitLimitNs);
        return;
    }
    auto consumers_sync = [&]() { sm100::named_bar_sync(2, kConsumers); };

    // a segment's running reference and sums; columns 2t and 2t + 1 of each row tile
    float o[NT][MW][4] = {}, ref[NT][2], sum[NT][2] = {};
#pragma unroll
    for (int n = 0; n < NT; ++n) ref[n][0] = ref[n][1] = kNone;

    // A segment's queries into shared memory as operands, a row tile a warp, and the
    // rows' factors and bounds.
    auto begin = [&]() {
        const int h = head_of(at), r0 = (at.hr - h * chunks) * RT;
        const float xs = p.scale * kLog2e * (kE ? *p.k_scale : 1.f);
#pragma unroll 1
        for (int n = warp; n < NT; n += kWarps) {
            const int r = r0 + n * 8 + g, i = r / group;
            const uint16_t* src = p.q + at.b * p.q_seq + i * p.q_token + (h * group + r - i * group) * p.q_head;
            uint32_t w[KS][2];
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                w[k][0] = w[k][1] = 0;
                if (r < rows && 16 * k < p.D) {
                    if constexpr (kE) {
                        const uint2 v = *reinterpret_cast<const uint2*>(src + 16 * k + 4 * t);
                        w[k][0] = v.x, w[k][1] = v.y;
                    } else {
                        w[k][0] = *reinterpret_cast<const uint32_t*>(src + 16 * k + 2 * t);
                        w[k][1] = *reinterpret_cast<const uint32_t*>(src + 16 * k + 8 + 2 * t);
                    }
                }
            }
            float fac = xs;
            if constexpr (kE) {
                float top = 0.f;
#pragma unroll
                for (int k = 0; k < KS; ++k)
                    top = fmaxf(top, fmaxf(fmaxf(fabsf(bf16_lo(w[k][0])), fabsf(bf16_hi(w[k][0]))),
                                           fmaxf(fabsf(bf16_lo(w[k][1])), fabsf(bf16_hi(w[k][1])))));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int e = (int)(__float_as_uint(top) >> 23);            // biased exponent
                // 2^(141 - e) puts the largest in [2^14, 2^15); its reciprocal goes into the factor
                const int up = e == 0 || e == 255 ? 0 : min(141 - e, 100);
                const float x = __int_as_float((127 + up) << 23);
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int c = 0; c < 2; ++c) w[k][c] = pack_f16x2(bf16_lo(w[k][c]) * x, bf16_hi(w[k][c]) * x);
                fac *= __int_as_float((127 - up) << 23);
            }
#pragma unroll
            for (int k = 0; k < KS; k += 2)
                sq[(n * (KS / 2) + k / 2) * 32 + lane] = make_uint4(w[k][0], w[k][1], w[k + 1][0], w[k + 1][1]);
            if (t == 0) {
                const int hi = r < rows ? at.s.len - p.Lq + i + 1 : 0;
                s_fac[n * 8 + g] = fac;
                s_hi[n * 8 + g] = hi;
                s_lo[n * 8 + g] = p.window ? max(0, hi - p.window) : 0;
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            ref[n][0] = ref[n][1] = kNone;
            sum[n][0] = sum[n][1] = 0.f;
#pragma unroll
            for (int k = 0; k < MW; ++k) o[n][k][0] = o[n][k][1] = o[n][k][2] = o[n][k][3] = 0.f;
        }
        consumers_sync();
    };

    // A lane's row of a matrix load, as an offset in a tile; chunk c (even) is at
    // (tile + offset) ^ (c & 7) * 16, plus whole pieces.
    const int lane_vr = kE ? lane & 15 : (lane & 7) + (lane >> 4) * 8, lane_vc = kE ? lane >> 4 : lane >> 3 & 1;
    const uint32_t lane_k = swz<C>(warp * TT + (lane & 15), lane >> 4), lane_v = swz<C>(lane_vr, lane_vc);
    auto piece = [](uint32_t at, int c) -> uint32_t { return (at ^ (uint32_t)((c & 7) << 4)) + (c >> 3) * (CT * 128); };
    const uint32_t sp = sm100::smem_u32(smem_p);
    // probabilities, stored and loaded by pairs of row tiles, or both parts of one
    const uint32_t p_lane = sp + swz_p<C>((NT > 1 ? lane >> 4 : 0) * 8 + (lane & 7), lane >> 3 & 1) +
                            (NT == 1 && C::kParts == 2 ? (lane >> 4) * C::kPart : 0);
    auto p_at = [](uint32_t at, int n, int c) -> uint32_t {   // row tile n, chunk c, both even
        return (at ^ (uint32_t)((c & 7) << 4)) + (c >> 3) * (RT * 128) + n * 1024;
    };

    // The tile's values that are not finite and that only some of the queries see:
    // added where they are seen, then taken out of the warp's part of the tile, which
    // no other warp reads.
    auto settle = [&](uint32_t vb, int ct0) {
        for (int j = 0; j < CT; ++j)
#pragma unroll
            for (int k = 0; k < MW; ++k)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int d = (warp * MW + k) * 16 + (kE ? 2 * g + e : g + 8 * e);
                    const uint32_t a = vb + swz<C>(j, d * ES / 16) + d * ES % 16;
                    const float v = ld_value<kE>(a);
                    if (isfinite(v)) continue;
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const int r = n * 8 + 2 * t + c;
                            const uint32_t w = *reinterpret_cast<const uint16_t*>(smem_p + swz_p<C>(r, j / 8) + (j & 7) * 2);
                            const float pr = kE ? __half2float(__ushort_as_half((unsigned short)w)) : __uint_as_float(w << 16);
                            if (ct0 + j < s_hi[r] && ct0 + j >= s_lo[r]) o[n][k][2 * e + c] += pr * v;
                        }
                }
        __syncwarp();
        for (int i = lane; i < CT * 16 * MW; i += 32) {
            const int j = i / (16 * MW), d = warp * MW * 16 + i - j * (16 * MW);
            const uint32_t a = vb + swz<C>(j, d * ES / 16) + d * ES % 16;
            if (!isfinite(ld_value<kE>(a))) st_zero<kE>(a);
        }
        if constexpr (kTma) sm100::fence_proxy_async_smem();
        __syncwarp();
    };

    auto compute = [&](uint32_t kb, int ct0) {
        const uint32_t vb = kb + C::kTile, ka = kb + lane_k, va = vb + lane_v;
        const int t0 = ct0 + warp * TT;                       // this warp's first token
        // S^T = K Q^T over the warp's tokens
        float s[NT][MT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int m = 0; m < MT; ++m) s[n][m][0] = s[n][m][1] = s[n][m][2] = s[n][m][3] = 0.f;
#pragma unroll
        for (int k = 0; k < KS; k += 2) {
            uint32_t a0[MT][4], a1[MT][4];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                if constexpr (kE) {
                    uint32_t w[4];
                    ldsm4(w, piece(ka, k) + m * 16 * C::PB);
                    e4m3x4_f16(w[0], a0[m][0], a0[m][2]);
                    e4m3x4_f16(w[1], a0[m][1], a0[m][3]);
                    e4m3x4_f16(w[2], a1[m][0], a1[m][2]);
                    e4m3x4_f16(w[3], a1[m][1], a1[m][3]);
                } else {
                    ldsm4(a0[m], piece(ka, 2 * k) + m * 16 * C::PB);
                    ldsm4(a1[m], piece(ka, 2 * k + 2) + m * 16 * C::PB);
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint4 v = sq[(n * (KS / 2) + k / 2) * 32 + lane];          // steps k and k + 1
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    mma16816<kE>(s[n][m], a0[m], v.x, v.y);
                    mma16816<kE>(s[n][m], a1[m], v.z, v.w);
                }
            }
        }
        // log2 scores above the running reference; tokens that a query does not see at -inf
        const bool edge = ct0 + CT > at.s.len - p.Lq + 1 || (p.window && ct0 < at.s.len - p.window);
        float x[NT][MT][4];
        auto relative = [&]() {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float2 f = *reinterpret_cast<const float2*>(s_fac + n * 8 + 2 * t);
                int2 hi = make_int2(0, 0), lo = make_int2(0, 0);
                if (edge) {
                    hi = *reinterpret_cast<const int2*>(s_hi + n * 8 + 2 * t);
                    lo = *reinterpret_cast<const int2*>(s_lo + n * 8 + 2 * t);
                }
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x[n][m][e] = fmaf(s[n][m][e], e & 1 ? f.y : f.x, -ref[n][e & 1]);
                        const int j = t0 + m * 16 + g + 8 * (e >> 1);
                        if (edge && (j >= (e & 1 ? hi.y : hi.x) || j < (e & 1 ? lo.y : lo.x))) x[n][m][e] = -INFINITY;
                    }
            }
        };
        relative();
        float top = -INFINITY;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int m = 0; m < MT; ++m)
                top = fmaxf(top, fmaxf(fmaxf(x[n][m][0], x[n][m][1]), fmaxf(x[n][m][2], x[n][m][3])));
        // The reference is the CTA's; maxima are only taken when some score passes the
        // room.  This barrier also says that every warp is done with the tile before.
        if (sm100::bar_red_or(1, kConsumers, top > kLazy + kBias)) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float2 f = *reinterpret_cast<const float2*>(s_fac + n * 8 + 2 * t);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float r = kNone;
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int e = c; e < 4; e += 2)
                            if (x[n][m][e] != -INFINITY) r = fmaxf(r, s[n][m][e] * (c ? f.y : f.x) - kBias);
                    r = fmaxf(r, __shfl_xor_sync(0xffffffffu, r, 4));
                    r = fmaxf(r, __shfl_xor_sync(0xffffffffu, r, 8));
                    r = fmaxf(r, __shfl_xor_sync(0xffffffffu, r, 16));
                    if (g == 0) s_w[warp * RT + n * 8 + 2 * t + c] = r;
                }
            }
            consumers_sync();
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float f[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float r = ref[n][c];
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) r = fmaxf(r, s_w[w * RT + n * 8 + 2 * t + c]);
                    f[c] = ex2(ref[n][c] - r);
                    ref[n][c] = r;
                    sum[n][c] *= f[c];
                }
#pragma unroll
                for (int k = 0; k < MW; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[n][k][e] *= f[e & 1];
            }
            relative();
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int m = 0; m < MT; ++m) {
#pragma unroll
                for (int e = 0; e < 4; ++e) x[n][m][e] = ex2(x[n][m][e]);
                sum[n][0] += x[n][m][0] + x[n][m][2];
                sum[n][1] += x[n][m][1] + x[n][m][3];
            }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int c = (warp * MT + m) * 2;
            auto pack = [&](int n, int e) {
                return kE ? pack_f16x2(x[n][m][e], x[n][m][e + 1]) : pack2_bf16(x[n][m][e], x[n][m][e + 1]);
            };
            auto rest = [&](int n, int e, uint32_t of) {      // what the rounding to `of` leaves
                return pack2_bf16(x[n][m][e] - bf16_lo(of), x[n][m][e + 1] - bf16_hi(of));
            };
            if constexpr (NT == 1 && C::kParts == 1) {
                stsm2_t(p_at(p_lane, 0, c), pack(0, 0), pack(0, 2));
            } else if constexpr (NT == 1) {
                const uint32_t u = pack(0, 0), v = pack(0, 2);
                stsm4_t(p_at(p_lane, 0, c), u, v, rest(0, 0, u), rest(0, 2, v));
            } else {
#pragma unroll
                for (int n = 0; n < NT; n += 2) {
                    const uint32_t u[4] = {pack(n, 0), pack(n, 2), pack(n + 1, 0), pack(n + 1, 2)};
                    stsm4_t(p_at(p_lane, n, c), u[0], u[1], u[2], u[3]);
                    if constexpr (C::kParts == 2)
                        stsm4_t(p_at(p_lane, n, c) + C::kPart, rest(n, 0, u[0]), rest(n, 2, u[1]), rest(n + 1, 0, u[2]),
                                rest(n + 1, 2, u[3]));
                }
            }
        }
        // What the product must not meet.  Rows of no visible token (a whole box is
        // loaded) become zero.  A value that only some of the queries see must not
        // reach the others as 0 x NaN: looked for here, settled below.
        bool bad = false;
        if (edge) {
            const int both_lo = p.window ? at.s.len - p.window : 0, both_hi = at.s.len - p.Lq + 1;   // seen by every query
            for (int i = 0; i < TT; ++i) {
                const int j = t0 + i, r = warp * TT + i;
                const bool none = j < at.s.lo || j >= at.s.len;
                if (none && kTma) {
                    if (lane < C::CPR) st_zero16(vb + swz<C>(r, lane));
                } else if (!none && (j < both_lo || j >= both_hi)) {
                    for (int d = lane; d < p.D; d += 32)
                        bad |= !isfinite(ld_value<kE>(vb + swz<C>(r, d * ES / 16) + d * ES % 16));
                }
            }
            if constexpr (kTma) sm100::fence_proxy_async_smem();      // the copy engine writes these rows next
        }
        if (sm100::bar_red_or(1, kConsumers, bad)) settle(vb, ct0);
        // O^T += V^T P^T: the warp's part of the head over the CTA's tokens
#pragma unroll
        for (int kt = 0; kt < CT / 16; ++kt) {
            uint32_t b[C::kParts][NT][2];
            if constexpr (NT == 1 && C::kParts == 1) {
                ldsm2(b[0][0], p_at(p_lane, 0, 2 * kt));
            } else {
#pragma unroll
                for (int i = 0; i < (NT == 1 ? 1 : C::kParts); ++i)
#pragma unroll
                    for (int n = 0; n < NT; n += 2) {
                        uint32_t v[4];
                        ldsm4(v, p_at(p_lane, n, 2 * kt) + i * C::kPart);
                        const int i1 = NT == 1 ? 1 : i, n1 = NT == 1 ? 0 : n + 1;
                        b[i][n][0] = v[0], b[i][n][1] = v[1], b[i1][n1][0] = v[2], b[i1][n1][1] = v[3];
                    }
            }
            const uint32_t row = kt * 16 * C::PB;
            uint32_t a[MW][4];
            if constexpr (kE && MW == 1) {                    // one chunk of the head: 16 tokens of it
                uint32_t w[2];
                ldsm2_t(w, vb + swz<C>(kt * 16 + (lane & 15), warp));
                e4m3x4_f16(__byte_perm(w[0], 0, 0x3120), a[0][0], a[0][1]);
                e4m3x4_f16(__byte_perm(w[1], 0, 0x3120), a[0][2], a[0][3]);
            } else if constexpr (kE) {
#pragma unroll
                for (int k = 0; k < MW; k += 2) {
                    uint32_t w[4];
                    ldsm4_t(w, piece(va, warp * MW + k) + row);
                    e4m3x4_f16(__byte_perm(w[0], 0, 0x3120), a[k][0], a[k][1]);
                    e4m3x4_f16(__byte_perm(w[1], 0, 0x3120), a[k][2], a[k][3]);
                    e4m3x4_f16(__byte_perm(w[2], 0, 0x3120), a[k + 1][0], a[k + 1][1]);
                    e4m3x4_f16(__byte_perm(w[3], 0, 0x3120), a[k + 1][2], a[k + 1][3]);
                }
            } else {
#pragma unroll
                for (int k = 0; k < MW; ++k) ldsm4_t(a[k], piece(va, (warp * MW + k) * 2) + row);
            }
#pragma unroll
            for (int k = 0; k < MW; ++k)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < C::kParts; ++i) mma16816<kE>(o[n][k], a[k], b[i][n][0], b[i][n][1]);
        }
    };

    // A segment's sums made one and written: the result if the item lies wholly in
    // this CTA's range, else one of the CTA's two slots.  Each warp has its part of
    // the head for every row.
    auto finish = [&]() {
        const int first = at.place - at.tile;                 // the item's tiles: first .. first + tiles - 1
        const bool whole = first >= 0 && first + at.s.tiles <= size;
        const int h = head_of(at), r0 = (at.hr - h * chunks) * RT;
        float* const slot = p.ws + ((int64_t)blockIdx.x * 2 + (first <= 0 ? 0 : 1)) * (RT * (C::DP + 2));
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float x = sum[n][c];
                x += __shfl_xor_sync(0xffffffffu, x, 4);
                x += __shfl_xor_sync(0xffffffffu, x, 8);
                x += __shfl_xor_sync(0xffffffffu, x, 16);
                if (g == 0) s_w[warp * RT + n * 8 + 2 * t + c] = x;
            }
        consumers_sync();
        const float vs = kE ? *p.v_scale : 1.f;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int r = n * 8 + 2 * t + c, rr = r0 + r;
                float l = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) l += s_w[w * RT + r];
                const bool mine = warp == 0 && g == 0;
                if (whole) {
                    if (rr >= rows) continue;
                    const int qi = rr / group;
                    const int64_t row = ((int64_t)at.b * p.Lq + qi) * p.Hq + h * group + rr - qi * group;
                    const float f = l == 0.f ? 0.f : vs / l;
#pragma unroll
                    for (int k = 0; k < MW; ++k) {
                        const int d = (warp * MW + k) * 16 + (kE ? 2 * g : g);
                        const float v0 = l == 0.f ? 0.f : o[n][k][c] * f, v1 = l == 0.f ? 0.f : o[n][k][c + 2] * f;
                        uint16_t* to = p.o + row * p.D + d;
                        if constexpr (kE) {
                            if (d < p.D) *reinterpret_cast<uint32_t*>(to) = pack2_bf16(v0, v1);
                        } else if (d < p.D) {
                            const uint32_t v = pack2_bf16(v0, v1);
                            to[0] = (uint16_t)v, to[8] = (uint16_t)(v >> 16);
                        }
                    }
                    if (p.lse && mine) p.lse[row] = l == 0.f ? -INFINITY : (ref[n][c] + log2f(l)) * kLn2;
                } else {
#pragma unroll
                    for (int k = 0; k < MW; ++k) {
                        float* to = slot + r * C::DP + (warp * MW + k) * 16 + (kE ? 2 * g : g);
                        if constexpr (kE)
                            *reinterpret_cast<float2*>(to) = make_float2(o[n][k][c], o[n][k][c + 2]);
                        else
                            to[0] = o[n][k][c], to[8] = o[n][k][c + 2];
                    }
                    if (mine) slot[RT * C::DP + r] = ref[n][c], slot[RT * C::DP + RT + r] = l;
                }
            }
    };

    // A cluster's item: every CTA lays its sums into its ring (all its tiles are done),
    // and takes a part of the rows' values from all of them.
    auto finish_cluster = [&]() {
        float* const part = reinterpret_cast<float*>(smem);       // [RT][DP], then the references, the sums
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float x = sum[n][c];
                x += __shfl_xor_sync(0xffffffffu, x, 4);
                x += __shfl_xor_sync(0xffffffffu, x, 8);
                x += __shfl_xor_sync(0xffffffffu, x, 16);
                if (g == 0) s_w[warp * RT + n * 8 + 2 * t + c] = x;
            }
        consumers_sync();                                     // (and the last tile's products are done)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int r = n * 8 + 2 * t + c;
#pragma unroll
                for (int k = 0; k < MW; ++k) {
                    float* to = part + r * C::DP + (warp * MW + k) * 16 + (kE ? 2 * g : g);
                    to[0] = o[n][k][c], to[kE ? 1 : 8] = o[n][k][c + 2];
                }
                if (warp == 0 && g == 0) {
                    float l = 0.f;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) l += s_w[w * RT + r];
                    part[RT * C::DP + r] = ref[n][c], part[RT * C::DP + RT + r] = l;
                }
            }
        __syncwarp();
        sm100::cluster_arrive();
        sm100::cluster_wait();
        const int h = head_of(at), r0 = (at.hr - h * chunks) * RT;
        const uint32_t rank = sm100::cluster_ctarank(), base = sm100::smem_u32(part);
        const float vs = kE ? *p.v_scale : 1.f;
        for (int i = rank * kConsumers + threadIdx.x; i < RT * (C::DP / 4); i += p.cluster * kConsumers) {
            const int r = i / (C::DP / 4), d = (i - r * (C::DP / 4)) * 4, rr = r0 + r;
            if (rr >= rows || d >= p.D) continue;
            float m = kNone, l = 0.f;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int w = 0; w < p.cluster; ++w)
                m = fmaxf(m, sm100::ld_cluster_f32(sm100::map_to_rank(base + (RT * C::DP + r) * 4, w)));
#pragma unroll 4
            for (int w = 0; w < p.cluster; ++w) {
                const float f = ex2(sm100::ld_cluster_f32(sm100::map_to_rank(base + (RT * C::DP + r) * 4, w)) - m);
                const float4 y = sm100::ld_cluster_v4(sm100::map_to_rank(base + (r * C::DP + d) * 4, w));
                l += f * sm100::ld_cluster_f32(sm100::map_to_rank(base + (RT * C::DP + RT + r) * 4, w));
                v.x += y.x * f, v.y += y.y * f, v.z += y.z * f, v.w += y.w * f;
            }
            const int qi = rr / group;
            const int64_t row = ((int64_t)at.b * p.Lq + qi) * p.Hq + h * group + rr - qi * group;
            const float f = vs / l;
            *reinterpret_cast<uint2*>(p.o + row * p.D + d) =
                l == 0.f ? make_uint2(0, 0) : make_uint2(pack2_bf16(v.x * f, v.y * f), pack2_bf16(v.z * f, v.w * f));
            if (p.lse && d == 0) p.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
        }
        __syncwarp();
        sm100::cluster_arrive();                              // nobody leaves while its sums are read
        sm100::cluster_wait();
    };

    // The next segment's queries are brought to L1 while this one finishes.
    auto touch = [&](const Cursor& c) {
        const int h = head_of(c), r0 = (c.hr - h * chunks) * RT;
        for (int n = warp; n < NT; n += kWarps) {
            const int r = r0 + n * 8 + g, i = r / group;
            const uint16_t* src = p.q + c.b * p.q_seq + i * p.q_token + (h * group + r - i * group) * p.q_head;
            for (int d = t * 16; d < p.D; d += 64)            // a 32-byte sector a lane
                if (r < rows) touch_l1(src + d);
        }
    };

    bool fresh = true;
#pragma unroll 1
    for (int n = 0; at.place < size; ++n) {
        if (fresh) begin();
        wait(full + 8 * (n % S), (n / S) & 1, 3);
        compute(ring + (n % S) * C::kStage, at.s.start + at.tile * CT);
        __syncwarp();
        if (lane == 0) sm100::mbar_arrive(empty + 8 * (n % S));
        Cursor then = at;
        then.next<C>(p, hr_n);
        fresh = then.tile == 0 || then.place >= size;
        if constexpr (kCluster) {
            if (fresh) break;                                 // `at` stays in the item
        } else if (fresh) {
            if (then.place < size) touch(then);
            finish();
        }
        at = then;
    }
    if constexpr (kCluster) finish_cluster();
}

// Joins the slots of the items that lie in several CTAs' ranges, in CTA order.
// One warp a row; `spread`: a CTA a row, its warps over the slots (few items,
// many slots each).
template <class C>
__global__ void __launch_bounds__(256)
attn_join_kernel(const __grid_constant__ AttnParams p, int ctas, int spread) {
    constexpr int RT = C::RT, DP = C::DP, kW = 8, V4 = DP / 128 > 0 ? DP / 128 : 1;
    __shared__ float4 so[kW][DP / 4];
    __shared__ float sm[kW], sl[kW];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int group = p.Hq / p.Hkv, rows = group * p.Lq, chunks = (rows + RT - 1) / RT, hr_n = p.Hkv * chunks;
    const int b = blockIdx.x / hr_n, hr = blockIdx.x - b * hr_n;
    // The lengths were there before the kernel this one follows: it started after
    // that one had passed its own wait.  Read from L2, where they are.
    int64_t before, total;
    count_places<C, true>(p, hr_n, b, &before, &total);
    const Span s = span_of<true>(p, b, C::CT);
    const int64_t chunk = div_ceil(total, ctas), first = before + (int64_t)hr * (s.tiles + C::kItem) + C::kItem;
    const int c0 = (int)(first / chunk), c1 = (int)((first + s.tiles - 1) / chunk);
    pdl_wait_then_release();
    if (c0 == c1) return;
    const int h = hr / chunks, r0 = (hr - h * chunks) * RT;
    auto slot = [&](int c) {
        return p.ws + ((int64_t)c * 2 + (first <= (int64_t)c * chunk ? 0 : 1)) * (RT * (DP + 2));
    };
    const float vs = C::kE4m3 ? *p.v_scale : 1.f;
    for (int r = spread ? blockIdx.y : warp; r < RT && r0 + r < rows; r += spread ? gridDim.y : kW) {
        float m = kNone, l = 0.f;
        float4 o[V4];
#pragma unroll
        for (int k = 0; k < V4; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        const int begin = c0 + (spread ? warp : 0), step = spread ? kW : 1;
        constexpr int kBatch = 4;                             // slots whose loads are in flight together
        for (int c = begin; c <= c1; c += kBatch * step) {
            float xm[kBatch], xl[kBatch];
            float4 v[kBatch][V4];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const bool in = c + i * step <= c1;
                const float* x = slot(in ? c + i * step : c);
                xm[i] = in ? x[RT * DP + r] : kNone;
                xl[i] = in ? x[RT * DP + RT + r] : 0.f;
#pragma unroll
                for (int k = 0; k < V4; ++k)
                    v[i][k] = in && (k * 32 + lane) * 4 < DP
                                  ? *reinterpret_cast<const float4*>(x + r * DP + (k * 32 + lane) * 4)
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            float top = m;
#pragma unroll
            for (int i = 0; i < kBatch; ++i) top = fmaxf(top, xm[i]);
            const float f0 = ex2(m - top);
            m = top, l *= f0;
#pragma unroll
            for (int k = 0; k < V4; ++k) o[k].x *= f0, o[k].y *= f0, o[k].z *= f0, o[k].w *= f0;
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const float f = ex2(xm[i] - m);
                l += xl[i] * f;
#pragma unroll
                for (int k = 0; k < V4; ++k)
                    o[k].x += f * v[i][k].x, o[k].y += f * v[i][k].y, o[k].z += f * v[i][k].z, o[k].w += f * v[i][k].w;
            }
        }
        if (spread) {
            if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
            for (int k = 0; k < V4; ++k)
                if ((k * 32 + lane) * 4 < DP) so[warp][k * 32 + lane] = o[k];
            __syncthreads();
            m = kNone, l = 0.f;
            for (int w = 0; w < kW; ++w) m = fmaxf(m, sm[w]);
#pragma unroll
            for (int k = 0; k < V4; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (warp == 0)
                for (int w = 0; w < kW; ++w) {
                    const float f = ex2(sm[w] - m);
                    l += sl[w] * f;
#pragma unroll
                    for (int k = 0; k < V4; ++k)
                        if ((k * 32 + lane) * 4 < DP) {
                            const float4 v = so[w][k * 32 + lane];
                            o[k].x += f * v.x, o[k].y += f * v.y, o[k].z += f * v.z, o[k].w += f * v.w;
                        }
                }
            __syncthreads();
            if (warp != 0) continue;
        }
        const int qi = (r0 + r) / group;
        const int64_t row = ((int64_t)b * p.Lq + qi) * p.Hq + h * group + r0 + r - qi * group;
        const float f = vs / l;
#pragma unroll
        for (int k = 0; k < V4; ++k) {
            const int d = (k * 32 + lane) * 4;
            if (d < p.D)
                *reinterpret_cast<uint2*>(p.o + row * p.D + d) =
                    l == 0.f ? make_uint2(0, 0)
                             : make_uint2(pack_bf16x2(o[k].x * f, o[k].y * f), pack_bf16x2(o[k].z * f, o[k].w * f));
        }
        if (p.lse && lane == 0) p.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    }
}

// CTAs a cluster where an item goes to one cluster, in one launch: short bounds on
// the lengths, whose items fill at most one wave and leave a CTA a few tiles.  0:
// the tiles are cut into ranges, and joined in a second launch.  One sequence of
// 777 tokens, 28/4 heads over bf16: 10.3 us in two launches, 7.0 in one; 4000
// tokens: 10.4 and 12.2.
template <class C>
int cluster_of(int64_t items, int64_t max_len) {
    const int64_t tiles = (max_len + C::CT - 1) / C::CT, wave = (int64_t)num_sms() * C::kCtas;
    int c = 8;
    while (c > 1 && (c > tiles || items * c > wave)) c /= 2;
    const int64_t most = items * c * 2 >= wave ? 8 : 4;       // tiles a CTA
    return tiles <= most * c && items * c <= wave ? c : 0;
}
// What a configuration takes for these sizes.
struct Plan {
    size_t ws;
    int kernels;
};
template <class C>
Plan plan(int64_t B, int64_t Hkv, int64_t rows, int64_t max_len) {
    if (max_len <= C::CT || cluster_of<C>(B * Hkv * ((rows + C::RT - 1) / C::RT), max_len)) return Plan{0, 1};
    return Plan{(size_t)num_sms() * C::kCtas * 2 * C::RT * (C::DP + 2) * sizeof(float), 2};
}

// The copy engine's view of a pool: [page][token][head][value] (the two in the
// middle in the order of their strides), boxes of `box` tokens of one head.
template <class C>
bool make_map(CUtensorMap* m, const void* pool, const AttnParams& p) {
    const bool by_head = p.order == 0;                        // heads inside tokens
    const uint64_t head = p.Hkv == 1 ? p.D : p.c_head, page = p.num_pages == 1 ? p.c_token * p.page_size : p.c_page;
    const uint64_t dims[4] = {(uint64_t)p.D, by_head ? (uint64_t)p.Hkv : (uint64_t)p.page_size,
                              by_head ? (uint64_t)p.page_size : (uint64_t)p.Hkv, (uint64_t)p.num_pages};
    const uint64_t strides[3] = {(by_head ? head : p.c_token) * C::ES, (by_head ? p.c_token : head) * C::ES, page * C::ES};
    const uint32_t box[4] = {C::PB / C::ES, by_head ? 1u : (uint32_t)p.box, by_head ? (uint32_t)p.box : 1u, 1u};
    return make_tmap_4d(m, pool, C::kE4m3, dims, strides, box, C::PB);
}

template <class C>
cudaError_t launch(const AttnParams& a, cudaStream_t st) {
    AttnParams p = a;
    CUtensorMap km = {}, vm = {};
    p.box = 1;
    p.page_shift = p.page_size & (p.page_size - 1) ? -1 : __builtin_ctz((unsigned)p.page_size);
    if constexpr (C::kTma) {
        p.box = C::CT;
        while (p.page_size % p.box) p.box /= 2;
        p.order = p.c_token < p.c_head && p.Hkv > 1;
        if (!make_map<C>(&km, p.kpool, p) || !make_map<C>(&vm, p.vpool, p)) return cudaErrorInvalidValue;
    }
    const int rows = p.Hq / p.Hkv * p.Lq, chunks = (rows + C::RT - 1) / C::RT;
    const int64_t items = (int64_t)p.B * p.Hkv * chunks, tiles = (p.max_len + C::CT - 1) / C::CT;
    const int64_t most = items * ((tiles > 1 ? tiles : 1) + C::kItem), wave = (int64_t)num_sms() * C::kCtas;
    static std::atomic<uint64_t> ready{0};                    // devices whose kernel has its shared memory
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
        for (auto k : {attn_paged_kernel<C, false>, attn_paged_kernel<C, true>}) {
            e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
            if (e != cudaSuccess) return e;
        }
        if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    p.cluster = cluster_of<C>(items, p.max_len);
    if (p.cluster) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(items * p.cluster));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = C::kSmem;
        cfg.stream = st;
        cudaLaunchAttribute at[2];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim = {(unsigned)p.cluster, 1, 1};
        at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = at;
        cfg.numAttrs = 2;
        return cudaLaunchKernelEx(&cfg, attn_paged_kernel<C, true>, p, km, vm);
    }
    const int ctas = (int)(most < wave ? most : wave);
    e = launch_pdl(attn_paged_kernel<C, false>, dim3((unsigned)ctas), dim3(kThreads), C::kSmem, st, p, km, vm);
    if (e != cudaSuccess || tiles <= 1) return e;             // items of one tile: nothing to join
    const bool spread = items * 2 < num_sms();
    return launch_pdl(attn_join_kernel<C>, dim3((unsigned)items, spread ? (unsigned)(rows < C::RT ? rows : C::RT) : 1u),
                      dim3(256), 0, st, p, ctas, (int)spread);
}

// The configuration for a head width and a number of query rows (query heads of
// a kv head x Lq): as few row tiles as hold them, so that no product is spent on
// rows that are not there; above the largest the rows go in chunks, each reading
// the cache again.
template <bool kE4m3, bool kTma, int DP, class F>
auto pick_rows(int64_t rows, F f) {
    if (rows <= 8) return f(Config<kE4m3, kTma, DP, 8>{});
    if (rows <= 16) return f(Config<kE4m3, kTma, DP, 16>{});
    // 64 rows at once only where their sums and scores leave room for the operands:
    // 40 rows over E4M3 took 299 us so and 267 us in two chunks, over bf16 325 and 358
    // (there only without the copy engine: attn_paged_wide.cuh has the rest)
    if constexpr (!kE4m3 && !kTma && DP <= 128)
        if (rows > 32) return f(Config<kE4m3, kTma, DP, 64>{});
    return f(Config<kE4m3, kTma, DP, 32>{});
}
template <bool kE4m3, bool kTma, class F>
auto pick(int64_t D, int64_t rows, F f) {
    if (D <= 64) return pick_rows<kE4m3, kTma, 64>(rows, f);
    if (D <= 128) return pick_rows<kE4m3, kTma, 128>(rows, f);
    return pick_rows<kE4m3, kTma, 256>(rows, f);
}

}  // namespace
}  // namespace attn

// One translation unit a cache type and loader (they compile side by side).
cudaError_t launch_attn_bf16_tma(const AttnParams& p, cudaStream_t st);
cudaError_t launch_attn_wide(const AttnParams& p, cudaStream_t st);
cudaError_t launch_attn_bf16(const AttnParams& p, cudaStream_t st);
cudaError_t launch_attn_e4m3_tma(const AttnParams& p, cudaStream_t st);
cudaError_t launch_attn_e4m3(const AttnParams& p, cudaStream_t st);

}  // namespace fp8rl
