// attn_paged.cuh -- attention of a sequence's new tokens over a paged key-value
// cache, as one pass over the cache with a running maximum and sum.  Query i of
// Lq stands at position p = len - Lq + i and sees the cached tokens j with
// max(0, p - window + 1) <= j <= p (window 0: from 0 on):
//   x_j = scale q.k_j,  o = sum_j e^(x_j - m) v_j / sum_j e^(x_j - m);
// a query that sees nothing gets zeros and a log-sum of -inf.
//
// What bounds it.  Every cached key and value is read once and meets the group's
// query rows (query heads of the kv head x Lq): 2 rows flop a bf16 byte, 4 rows
// an E4M3 byte.  With 5-8 rows that is far below the tensor cores' rate at HBM
// speed even for mma.sync, so the kernel is a stream from HBM, and the design
// keeps about 128 KB of loads in flight on every SM.  The tcgen05 form would
// want 128 query or cache rows an instruction, its scores in tensor memory, and
// E4M3 operands on both sides (which the queries and probabilities are not).
//
// Products.  A warp takes 16 (E4M3: 32) tokens at a time: S^T = K Q^T with the
// tokens as the M side and 8 query rows as the N side of m16n8k16, so a group of
// 5-8 heads fills the tile; O^T += V^T P^T with 16 head values as the M side.
// K comes through ldmatrix, V through its transposing form, P^T from the scores'
// registers through an 8x8 register transpose.  E4M3 is converted to fp16 in
// registers (exact); the key's values are taken in an order of the head
// dimension that makes each 4-byte piece of a row two operand words, Q follows
// the same order, and transposed V comes out as even and odd head values.  For
// E4M3 caches the bf16 queries are held as fp16, scaled by a power of two that
// puts the row's largest value at 2^14 (exact down to 2^-28 of it).
// Probabilities are rounded to the product's type relative to the running
// maximum (fp16: times 2^6, so that 2^-20 of the maximum is still a normal
// number); their sum is of the unrounded fp32 values.
//
// Running maximum.  Products are rescaled only when a tile's maximum passes the
// reference by 2^8: exact arithmetic does not change, and fp32 sums, bf16 and
// fp16 probabilities all have the room.
//
// Work split.  The unit is a tile of the CTA (its token groups side by side) of
// one item (sequence, kv head, chunk of query rows).  All units of the batch, in
// item order, are cut into equal ranges, one a CTA, one wave of CTAs: ragged
// lengths need no plan on the host, and one long sequence spreads over the GPU.
// The lengths are read on the device.  A CTA writes an item that lies wholly in
// its range; of items that do not it has at most two, whose unnormalised sums go
// to its two slots of the workspace, joined in a second launch in CTA order.
#pragma once

#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "sm100_ptx.cuh"

namespace fp8rl {
namespace attn {

constexpr uint32_t kKernelAttn = 10;
constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr float kLazy = 8.f;                  // log2 by which a score may pass the reference before a rescale
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kNone = -3.402823466e38f;     // reference of a row that has seen nothing: any score passes it
constexpr uint64_t kWaitLimitNs = 2000000000ull;   // 2 s: far above any legitimate wait

template <bool kE4m3_, bool kTma_, int DP_, int NT_, int WR_>
struct Config {
    static constexpr bool kE4m3 = kE4m3_, kTma = kTma_;
    static constexpr int DP = DP_;             // padded head width
    static constexpr int NT = NT_, WR = WR_;   // 8-row tiles a warp, warps over the rows
    static constexpr int RT = 8 * NT * WR;     // query rows of a CTA
    static constexpr int WT = kWarps / WR;     // token groups
    static constexpr int ES = kE4m3 ? 1 : 2, RB = DP * ES;   // bytes of a value, of a cached head
    static constexpr int PB = RB < 128 ? RB : 128;           // row bytes of a piece of a tile
    static constexpr int CPR = RB / 16;                      // 16-byte chunks of a cached head
    static constexpr int TT = kE4m3 && NT <= 2 ? 32 : 16, MT = TT / 16;   // tokens of a warp's tile
    static constexpr int CT = TT * WT;                       // tokens of a CTA's tile
    static constexpr int kStage = 2 * TT * RB;               // K and V of one group's tile
    static constexpr int kQ = NT * DP > 256 ? NT * WR * (DP / 32) * 512 : 0;   // queries, where registers do not hold them
    static constexpr int kPass = NT > 2 ? 2 : 1;             // parts in which the groups' sums are added
    static constexpr int kJoin = (WT / 2) * RT * DP * 4 / kPass, kOut = RT * DP * 4;
    static constexpr int kMerge = kJoin > kOut ? kJoin : kOut;
    static constexpr int kCtas = DP > 128 ? 1 : 2;           // CTAs an SM
    static constexpr int kBudget = 233472 / kCtas - 1024;    // 228 KB an SM, 1 KB of it kept for each CTA
    static constexpr int kRest = kMerge + kQ + WT * RT * 8 + 6 * WT * 8 + 16;
    static constexpr int kFit = (kBudget - kRest - 1024) / (WT * kStage);   // 1 KB to align the ring
    static constexpr int kStages = kFit > 6 ? 6 : kFit;
    static constexpr int kSmem = kStages * WT * kStage + kRest + 1024;
    static_assert(kStages >= 2, "too little shared memory for two stages");
};

// The tokens [lo, len) a sequence's queries see at all, and the item's tiles from
// `start` on (lo rounded down to a box of the cache's pages); one tile at least,
// so that every item has a writer.
struct Span {
    int start, lo, len, tiles;
};
__device__ __forceinline__ Span span_of(const AttnParams& p, int b, int ct) {
    Span s;
    s.len = min(max(p.lens[b], 0), p.max_len);
    s.lo = p.window ? max(0, s.len - p.Lq + 1 - p.window) : 0;
    s.start = s.lo & -p.box;
    s.tiles = max(1, (s.len - s.start + ct - 1) / ct);
    return s;
}

// The whole warp: units of sequences [0, b_end), and of all; hr items a sequence.
__device__ __forceinline__ void count_units(const AttnParams& p, int ct, int hr, int b_end, int64_t* before,
                                            int64_t* total) {
    const int lane = threadIdx.x & 31;
    int64_t x = 0, y = 0;
    for (int b = lane; b < p.B; b += 32) {
        const int n = span_of(p, b, ct).tiles;
        y += n;
        if (b < b_end) x += n;
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) {
        x += __shfl_xor_sync(0xffffffffu, x, off);
        y += __shfl_xor_sync(0xffffffffu, y, off);
    }
    *before = x * hr;
    *total = y * hr;
}

__device__ __forceinline__ int64_t chunk_of(int64_t total, int ctas) { return (total + ctas - 1) / ctas; }

// ---------------------------------------------------------------- PTX

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
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
        return (uint32_t)((c >> 3) * (C::TT * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
    else
        return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
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

// A position in the CTA's range of units.
struct Cursor {
    Span s;
    int b, hr, tile;
    __device__ __forceinline__ void next(const AttnParams& p, int ct, int hr_n) {
        if (++tile < s.tiles) return;
        tile = 0;
        if (++hr < hr_n) return;
        hr = 0;
        if (++b < p.B) s = span_of(p, b, ct);
    }
};

template <class C>
__global__ void __launch_bounds__(kThreads, C::kCtas)
attn_paged_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap) {
    extern __shared__ uint8_t smem_raw[];
    constexpr bool kE = C::kE4m3, kTma = C::kTma;
    constexpr int NT = C::NT, WR = C::WR, RT = C::RT, WT = C::WT, TT = C::TT, MT = C::MT, CT = C::CT, ES = C::ES;
    constexpr int KS = C::DP / 16, S = C::kStages, kTile = TT * C::RB;
    constexpr float kBias = kE ? 6.f : 0.f;
    uint8_t* const smem = smem_raw + ((1024u - (sm100::smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* at_smem = smem + S * WT * C::kStage;
    float* const merge = reinterpret_cast<float*>(at_smem);
    uint4* const sq = reinterpret_cast<uint4*>(at_smem + C::kMerge);          // [row tile][KS / 2][lane]
    float* const sm_m = reinterpret_cast<float*>(at_smem + C::kMerge + C::kQ);   // [WT][RT]
    float* const sm_l = sm_m + WT * RT;
    const uint32_t bars = sm100::smem_u32(sm_l + WT * RT);                    // [S][WT], TMA only
    volatile int* const abort = reinterpret_cast<int*>(sm_l + WT * RT) + 2 * 6 * WT;

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int tg = warp / WR, wr = warp % WR;                // token group, row group
    const int group = p.Hq / p.Hkv, rows = group * p.Lq, chunks = (rows + RT - 1) / RT, hr_n = p.Hkv * chunks;
    if constexpr (kTma) {
        if (threadIdx.x == 0) {
            for (int i = 0; i < S * WT; ++i) sm100::mbar_init(bars + 8 * i, 1);
            *abort = 0;
            sm100::fence_mbar_init();
            sm100::prefetch_tmap(&kmap);
            sm100::prefetch_tmap(&vmap);
        }
        __syncthreads();
    }
    pdl_wait_then_release();

    // the CTA's range of units, and where it begins
    int64_t before, total;
    count_units(p, CT, hr_n, 0, &before, &total);
    const int64_t chunk = chunk_of(total, gridDim.x), u0 = (int64_t)blockIdx.x * chunk;
    if (u0 >= total) return;
    const int count = (int)(total - u0 < chunk ? total - u0 : chunk);
    Cursor ld;
    int64_t item0 = 0;                                        // first unit of the sequence the range begins in
    for (int base = 0;; base += 32) {
        const int b = base + lane;
        const int n = b < p.B ? span_of(p, b, CT).tiles : 0;
        if (blockIdx.x == 0 && warp == 0 && b < p.B && (p.lens[b] < 0 || p.lens[b] > p.max_len))
            atomicCAS(p.err, 0u, (kKernelAttn << 24) | (1u << 16) | 2u);
        int64_t inc = n;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t o = __shfl_up_sync(0xffffffffu, inc, off);
            if (lane >= off) inc += o;
        }
        const uint32_t in = __ballot_sync(0xffffffffu, item0 + inc * hr_n > u0);
        if (in && blockIdx.x != 0) {
            const int l = __ffs((int)in) - 1;
            item0 += __shfl_sync(0xffffffffu, (inc - n) * hr_n, l);
            ld.b = base + l;
            break;
        }
        if (blockIdx.x == 0 && base + 32 >= p.B) {            // this one has looked at every length
            item0 = 0, ld.b = 0;
            break;
        }
        if (blockIdx.x != 0) item0 += __shfl_sync(0xffffffffu, inc * hr_n, 31);
    }
    ld.s = span_of(p, ld.b, CT);
    ld.hr = (int)((u0 - item0) / ld.s.tiles);
    ld.tile = (int)((u0 - item0) - (int64_t)ld.hr * ld.s.tiles);
    Cursor at = ld;

    // The loader fills the group's ring, a tile a stage, S - 1 tiles ahead.  Pages
    // are looked up one tile before they are used, by one lane a box (copy engine)
    // or a lane a token.
    const uint32_t ring = sm100::smem_u32(smem) + tg * C::kStage;      // stage s: + s * WT * kStage
    const int unit = kTma ? p.box : 1;                                  // tokens a lane looks up
    auto lookup = [&](const Cursor& c) -> int64_t {           // -1: nothing to load
        const int i = kTma ? lane * unit : lane % TT;
        const int j = c.s.start + c.tile * CT + tg * TT + i;
        if (i >= TT || j >= c.s.len) return -1;
        const int pg = j / p.page_size;
        int page = p.pages[c.b * p.pages_seq + pg];
        if ((uint32_t)page >= (uint64_t)p.num_pages) {
            atomicCAS(p.err, 0u, (kKernelAttn << 24) | (2u << 16) | 2u);
            page = 0;
        }
        if constexpr (kTma) return ((int64_t)page << 32) | (uint32_t)(j - pg * p.page_size);
        return (page * p.c_page + (int64_t)(j - pg * p.page_size) * p.c_token + (c.hr / chunks) * p.c_head) * ES;
    };
    const bool loads = !kTma || wr == 0;
    int issued = 0, armed = 0;
    bool dead = false;                                        // a wait ran out: nothing more is loaded or computed
    int64_t off = loads ? lookup(ld) : 0;
    auto issue = [&]() {
        if (issued < count && loads && !dead) {
            const uint32_t slot = issued % S, dst = ring + slot * (WT * C::kStage);
            if constexpr (kTma) {
                const uint32_t bar = bars + 8 * (slot * WT + tg);
                const uint32_t n = __popc(__ballot_sync(0xffffffffu, off >= 0));
                ++armed;
                if (lane == 0) sm100::mbar_arrive_expect_tx(bar, n * 2 * unit * C::RB);
                __syncwarp();
                if (off >= 0) {
                    const int h = ld.hr / chunks, page = (int)(off >> 32), row = (int)(uint32_t)off;
#pragma unroll
                    for (int x = 0; x < C::RB / C::PB; ++x) {
                        const uint32_t d = dst + x * (TT * C::PB) + lane * unit * C::PB;
                        tma_load_4d(d, &kmap, bar, x * (C::PB / ES), p.order ? row : h, p.order ? h : row, page);
                        tma_load_4d(d + kTile, &vmap, bar, x * (C::PB / ES), p.order ? row : h, p.order ? h : row, page);
                    }
                }
            } else {
                const int cpr = p.D * ES / 16;                // chunks the cache has of a head
                constexpr int RPI = 32 / C::CPR > 0 ? 32 / C::CPR : 1;      // rows a warp covers at once
                constexpr int kTurns = TT / RPI / WR;
#pragma unroll
                for (int i = 0; i < kTurns; ++i) {
                    const int r = (wr * kTurns + i) * RPI + (C::CPR < 32 ? lane / C::CPR : 0), c = lane % C::CPR;
                    const int64_t o = __shfl_sync(0xffffffffu, off, r);
                    const uint32_t n = o >= 0 && c < cpr ? 16u : 0u;
                    const int64_t src = n ? o + c * 16 : 0;
                    cp_async16(dst + swz<C>(r, c), static_cast<const uint8_t*>(p.kpool) + src, n);
                    cp_async16(dst + kTile + swz<C>(r, c), static_cast<const uint8_t*>(p.vpool) + src, n);
                }
            }
            ld.next(p, CT, hr_n);
            if (issued + 1 < count) off = lookup(ld);
        }
        ++issued;
        if constexpr (!kTma) cp_async_commit();
    };
    auto group_sync = [&]() {
        if constexpr (WR == 1)
            __syncwarp();
        else
            sm100::named_bar_sync(1 + tg, WR * 32);
    };
    // Tile n has landed for the whole group, whose warps are all past tile n - 1.
    auto arrived = [&](int n) {
        if constexpr (kTma) {
            if (!dead && !sm100::mbar_wait_bounded(bars + 8 * (n % S * WT + tg), (n / S) & 1, abort, kWaitLimitNs)) {
                if (lane == 0) atomicCAS(p.err, 0u, (kKernelAttn << 24) | (3u << 16) | 1u);
                *abort = 1;
                dead = true;
            }
            if constexpr (WR == 1)
                dead = __any_sync(0xffffffffu, dead);
            else
                dead = sm100::bar_red_or(1 + tg, WR * 32, dead);
        } else {
            cp_async_wait<S - 2>();
            group_sync();
        }
    };

    // a segment's queries, bounds and sums; columns 2t and 2t + 1 of each row tile
    uint32_t q[C::kQ ? 1 : NT][KS][2];
    float fac[NT][2];                          // log2 units of a unit of the product
    int hi[NT][2], lo[NT][2];                  // tokens the columns' queries see
    float o[NT][KS][4], ref[NT][2], sum[NT][2];
    const float xs = p.scale * kLog2e * (kE ? *p.k_scale : 1.f);

    auto begin = [&]() {
        const int h = at.hr / chunks, r0 = (at.hr - h * chunks) * RT + wr * 8 * NT;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
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
            fac[n][0] = fac[n][1] = xs;
            if constexpr (kE) {
                float top = 0.f;
#pragma unroll
                for (int k = 0; k < KS; ++k)
                    top = fmaxf(top, fmaxf(fmaxf(fabsf(bf16_lo(w[k][0])), fabsf(bf16_hi(w[k][0]))),
                                           fmaxf(fabsf(bf16_lo(w[k][1])), fabsf(bf16_hi(w[k][1])))));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int e = (int)(__float_as_uint(top) >> 23);            // biased exponent
                // 2^(141 - e) puts the largest at 2^14; its reciprocal goes into the factor
                const int up = e == 0 || e == 255 ? 0 : min(141 - e, 100);
                const float x = __int_as_float((127 + up) << 23), down = __int_as_float((127 - up) << 23);
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int c = 0; c < 2; ++c) w[k][c] = pack_f16x2(bf16_lo(w[k][c]) * x, bf16_hi(w[k][c]) * x);
                fac[n][0] *= __shfl_sync(0xffffffffu, down, 8 * t);         // row 2t is held by lanes 8t .. 8t + 3
                fac[n][1] *= __shfl_sync(0xffffffffu, down, 8 * t + 4);
            }
            if constexpr (C::kQ) {
                if (tg == n % WT)
#pragma unroll
                    for (int k = 0; k < KS; k += 2)
                        sq[((wr * NT + n) * (KS / 2) + k / 2) * 32 + lane] =
                            make_uint4(w[k][0], w[k][1], w[k + 1][0], w[k + 1][1]);
            } else {
#pragma unroll
                for (int k = 0; k < KS; ++k) q[n][k][0] = w[k][0], q[n][k][1] = w[k][1];
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int rc = r0 + n * 8 + 2 * t + c;
                hi[n][c] = rc < rows ? at.s.len - p.Lq + rc / group + 1 : 0;
                lo[n][c] = p.window ? max(0, hi[n][c] - p.window) : 0;
                ref[n][c] = kNone;
                sum[n][c] = 0.f;
            }
#pragma unroll
            for (int k = 0; k < KS; ++k) o[n][k][0] = o[n][k][1] = o[n][k][2] = o[n][k][3] = 0.f;
        }
        if constexpr (C::kQ) __syncthreads();
    };

    // What the product must not meet in an edge tile.  Rows of no visible token
    // (a whole box is loaded) become zero.  A value that only some of the queries
    // see must not reach the others as 0 x NaN: what is not finite is added where
    // it is seen, and taken out of the tile.  x: the tile's probabilities.
    auto hide = [&](uint32_t vb, int t0, const float (&x)[NT][MT][4]) {
        const int both_lo = p.window ? at.s.len - p.window : 0, both_hi = at.s.len - p.Lq + 1;   // seen by every query
        bool bad = false;
        for (int j = 0; j < TT; ++j) {
            const bool none = t0 + j < at.s.lo || t0 + j >= at.s.len;
            if (none && kTma) {
                if (lane < C::CPR) st_zero16(vb + swz<C>(j, lane));
            } else if (!none && (t0 + j < both_lo || t0 + j >= both_hi)) {
                for (int d = lane; d < p.D; d += 32)
                    bad |= !isfinite(ld_value<kE>(vb + swz<C>(j, d * ES / 16) + d * ES % 16));
            }
        }
        bad = __any_sync(0xffffffffu, bad);
        group_sync();                                         // the group's warps have all looked
        if (bad) {
            for (int j = 0; j < TT; ++j)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float w0 = 0.f, w1 = 0.f;                  // the token's probabilities in columns 2t, 2t + 1
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        const float y0 = __shfl_sync(0xffffffffu, j & 8 ? x[n][m][2] : x[n][m][0], (j & 7) * 4 + t);
                        const float y1 = __shfl_sync(0xffffffffu, j & 8 ? x[n][m][3] : x[n][m][1], (j & 7) * 4 + t);
                        if (m == j >> 4) w0 = y0, w1 = y1;
                    }
                    const bool see0 = t0 + j < hi[n][0] && t0 + j >= lo[n][0];
                    const bool see1 = t0 + j < hi[n][1] && t0 + j >= lo[n][1];
#pragma unroll
                    for (int k = 0; k < KS; ++k)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int d = kE ? 16 * k + 2 * g + e : 16 * k + g + 8 * e;
                            const float v = ld_value<kE>(vb + swz<C>(j, d * ES / 16) + d * ES % 16);
                            if (!isfinite(v) && see0) o[n][k][2 * e] += w0 * v;
                            if (!isfinite(v) && see1) o[n][k][2 * e + 1] += w1 * v;
                        }
                }
            group_sync();                                     // and added
            for (int i = lane; i < TT * p.D; i += 32) {
                const int j = i / p.D, d = i - j * p.D;
                const uint32_t a = vb + swz<C>(j, d * ES / 16) + d * ES % 16;
                if (!isfinite(ld_value<kE>(a))) st_zero<kE>(a);
            }
            group_sync();
        }
        if constexpr (kTma) sm100::fence_proxy_async_smem();  // the copy engine writes these rows next
    };

    auto compute = [&](uint32_t kb, int t0) {
        const uint32_t vb = kb + kTile;
        // S^T = K Q^T
        float s[NT][MT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int m = 0; m < MT; ++m) s[n][m][0] = s[n][m][1] = s[n][m][2] = s[n][m][3] = 0.f;
#pragma unroll
        for (int k = 0; k < KS; k += 2) {
            uint32_t b[NT][4];                                // queries of steps k and k + 1
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if constexpr (C::kQ) {
                    const uint4 v = sq[((wr * NT + n) * (KS / 2) + k / 2) * 32 + lane];
                    b[n][0] = v.x, b[n][1] = v.y, b[n][2] = v.z, b[n][3] = v.w;
                } else {
                    b[n][0] = q[n][k][0], b[n][1] = q[n][k][1], b[n][2] = q[n][k + 1][0], b[n][3] = q[n][k + 1][1];
                }
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const int r = m * 16 + (lane & 15);
                uint32_t a0[4], a1[4];
                if constexpr (kE) {
                    uint32_t w[4];
                    ldsm4(w, kb + swz<C>(r, k + (lane >> 4)));
                    e4m3x4_f16(w[0], a0[0], a0[2]);
                    e4m3x4_f16(w[1], a0[1], a0[3]);
                    e4m3x4_f16(w[2], a1[0], a1[2]);
                    e4m3x4_f16(w[3], a1[1], a1[3]);
                } else {
                    ldsm4(a0, kb + swz<C>(r, 2 * k + (lane >> 4)));
                    ldsm4(a1, kb + swz<C>(r, 2 * k + 2 + (lane >> 4)));
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) mma16816<kE>(s[n][m], a0, b[n][0], b[n][1]);
#pragma unroll
                for (int n = 0; n < NT; ++n) mma16816<kE>(s[n][m], a1, b[n][2], b[n][3]);
            }
        }
        // log2 scores above the running reference; tokens that a query does not see at -inf
        const bool edge = t0 + TT > at.s.len - p.Lq + 1 || (p.window && t0 < at.s.len - p.window);
        float x[NT][MT][4];
        uint32_t seen = 0xffffffffu;
        if (edge) {
            seen = 0;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = t0 + m * 16 + g + 8 * (e >> 1);
                        seen |= (uint32_t)(j < hi[n][e & 1] && j >= lo[n][e & 1]) << ((n * MT + m) * 4 + e);
                    }
        }
        auto relative = [&]() {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[n][m][e] = fmaf(s[n][m][e], fac[n][e & 1], -ref[n][e & 1]);
            if (edge)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (!(seen >> ((n * MT + m) * 4 + e) & 1)) x[n][m][e] = -INFINITY;
        };
        relative();
        float top = -INFINITY;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int m = 0; m < MT; ++m)
                top = fmaxf(top, fmaxf(fmaxf(x[n][m][0], x[n][m][1]), fmaxf(x[n][m][2], x[n][m][3])));
        // the maximum is only reduced over the lanes when some score passes the room
        if (__any_sync(0xffffffffu, top > kLazy + kBias)) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float f[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float r = ref[n][c];
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int e = c; e < 4; e += 2)
                            if (seen >> ((n * MT + m) * 4 + e) & 1) r = fmaxf(r, s[n][m][e] * fac[n][c] - kBias);
                    r = fmaxf(r, __shfl_xor_sync(0xffffffffu, r, 4));
                    r = fmaxf(r, __shfl_xor_sync(0xffffffffu, r, 8));
                    r = fmaxf(r, __shfl_xor_sync(0xffffffffu, r, 16));
                    f[c] = ex2(ref[n][c] - r);
                    ref[n][c] = r;
                    sum[n][c] *= f[c];
                }
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[n][k][e] *= f[e & 1];
            }
            relative();
        }
        uint32_t pt[NT][MT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int m = 0; m < MT; ++m) {
#pragma unroll
                for (int e = 0; e < 4; ++e) x[n][m][e] = ex2(x[n][m][e]);
                sum[n][0] += x[n][m][0] + x[n][m][2];
                sum[n][1] += x[n][m][1] + x[n][m][3];
                pt[n][m][0] = transpose8x8(kE ? pack_f16x2(x[n][m][0], x[n][m][1]) : pack_bf16x2(x[n][m][0], x[n][m][1]));
                pt[n][m][1] = transpose8x8(kE ? pack_f16x2(x[n][m][2], x[n][m][3]) : pack_bf16x2(x[n][m][2], x[n][m][3]));
            }
        if (edge) hide(vb, t0, x);
        // O^T += V^T P^T
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int k = 0; k < KS; k += 2) {
                uint32_t a0[4], a1[4];
                if constexpr (kE) {
                    uint32_t w[4];
                    ldsm4_t(w, vb + swz<C>(m * 16 + (lane & 15), k + (lane >> 4)));
                    e4m3x4_f16(__byte_perm(w[0], 0, 0x3120), a0[0], a0[1]);
                    e4m3x4_f16(__byte_perm(w[1], 0, 0x3120), a0[2], a0[3]);
                    e4m3x4_f16(__byte_perm(w[2], 0, 0x3120), a1[0], a1[1]);
                    e4m3x4_f16(__byte_perm(w[3], 0, 0x3120), a1[2], a1[3]);
                } else {
                    const int r = m * 16 + (lane & 7) + (lane >> 4) * 8;
                    ldsm4_t(a0, vb + swz<C>(r, 2 * k + ((lane >> 3) & 1)));
                    ldsm4_t(a1, vb + swz<C>(r, 2 * k + 2 + ((lane >> 3) & 1)));
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    mma16816<kE>(o[n][k], a0, pt[n][m][0], pt[n][m][1]);
                    mma16816<kE>(o[n][k + 1], a1, pt[n][m][0], pt[n][m][1]);
                }
            }
    };

    // The groups' sums of a segment made one and written: the result if the item
    // lies wholly in this CTA's range, else one of the CTA's two slots.
    auto finish = [&](int64_t u) {                            // u: the segment's last unit
        float L[NT][2], M[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float x = sum[n][c];
                x += __shfl_xor_sync(0xffffffffu, x, 4);
                x += __shfl_xor_sync(0xffffffffu, x, 8);
                x += __shfl_xor_sync(0xffffffffu, x, 16);
                const int r = wr * 8 * NT + n * 8 + 2 * t + c;
                if (g == 0) sm_m[tg * RT + r] = ref[n][c], sm_l[tg * RT + r] = x;
            }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int r = wr * 8 * NT + n * 8 + 2 * t + c;
                float m = kNone, l = 0.f;
#pragma unroll
                for (int w = 0; w < WT; ++w) m = fmaxf(m, sm_m[w * RT + r]);
#pragma unroll
                for (int w = 0; w < WT; ++w) l += sm_l[w * RT + r] * ex2(sm_m[w * RT + r] - m);
                const float f = ex2(ref[n][c] - m);
#pragma unroll
                for (int k = 0; k < KS; ++k) o[n][k][c] *= f, o[n][k][c + 2] *= f;
                M[n][c] = m, L[n][c] = l;
            }
        // the groups' sums, halved in number at each step, kPass parts of the head a step
        constexpr int KP = KS / C::kPass;
        auto place = [&](int n, int k, int e, int width) {     // [row][value] of a sum
            const int d = kE ? 16 * k + 2 * g + (e >> 1) : 16 * k + g + 8 * (e >> 1);
            return (wr * 8 * NT + n * 8 + 2 * t + (e & 1)) * width + d;
        };
#pragma unroll
        for (int half = WT / 2; half >= 1; half /= 2)
#pragma unroll
            for (int part = 0; part < C::kPass; ++part) {
                constexpr int W = 16 * KP;
                if (tg >= half && tg < 2 * half)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int k = 0; k < KP; ++k)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                merge[(tg - half) * RT * W + place(n, k, e, W)] = o[n][part * KP + k][e];
                __syncthreads();
                if (tg < half)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int k = 0; k < KP; ++k)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                o[n][part * KP + k][e] += merge[tg * RT * W + place(n, k, e, W)];
                __syncthreads();
            }
        if (tg == 0) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) merge[place(n, k, e, C::DP)] = o[n][k][e];
                if (g == 0)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int r = wr * 8 * NT + n * 8 + 2 * t + c;
                        sm_m[r] = M[n][c], sm_l[r] = L[n][c];
                    }
            }
        }
        __syncthreads();
        const int64_t first = u - at.tile;                    // the item's units: first .. first + tiles - 1
        const bool whole = first >= u0 && first + at.s.tiles <= u0 + count;
        const int h = at.hr / chunks, r0 = (at.hr - h * chunks) * RT;
        if (whole) {
            const float vs = kE ? *p.v_scale : 1.f;
            for (int i = threadIdx.x; i < RT * (C::DP / 4); i += kThreads) {
                const int r = i / (C::DP / 4), d = (i - r * (C::DP / 4)) * 4, rr = r0 + r;
                if (rr >= rows || d >= p.D) continue;
                const float l = sm_l[r], f = l == 0.f ? 0.f : vs / l;
                const float4 v = *reinterpret_cast<const float4*>(merge + r * C::DP + d);
                const int qi = rr / group;
                const int64_t row = ((int64_t)at.b * p.Lq + qi) * p.Hq + h * group + rr - qi * group;
                *reinterpret_cast<uint2*>(p.o + row * p.D + d) =
                    l == 0.f ? make_uint2(0, 0)
                             : make_uint2(pack_bf16x2(v.x * f, v.y * f), pack_bf16x2(v.z * f, v.w * f));
                if (p.lse && d == 0) p.lse[row] = l == 0.f ? -INFINITY : (sm_m[r] + log2f(l)) * kLn2;
            }
        } else {
            float* slot = p.ws + ((int64_t)blockIdx.x * 2 + (first <= u0 ? 0 : 1)) * (RT * (C::DP + 2));
            for (int i = threadIdx.x; i < RT * (C::DP / 4); i += kThreads)
                *reinterpret_cast<float4*>(slot + i * 4) = *reinterpret_cast<const float4*>(merge + i * 4);
            for (int r = threadIdx.x; r < RT; r += kThreads) {
                slot[RT * C::DP + r] = sm_m[r];
                slot[RT * C::DP + RT + r] = sm_l[r];
            }
        }
        __syncthreads();
    };

#pragma unroll 1
    for (int i = 0; i < S - 1; ++i) issue();
    begin();
#pragma unroll 1
    for (int n = 0; n < count; ++n) {
        arrived(n);
        issue();
        const int t0 = at.s.start + at.tile * CT + tg * TT;
        if (t0 < at.s.len && !dead) compute(ring + (n % S) * (WT * C::kStage), t0);
        const bool end = at.tile + 1 == at.s.tiles || n + 1 == count;
        if (end) finish(u0 + n);
        at.next(p, CT, hr_n);
        if (end && n + 1 < count) begin();
    }
    if (kTma && dead && lane == 0)                             // the copies still in flight write to this CTA's memory
        for (int n = armed > S ? armed - S : 0; n < armed; ++n)
            sm100::mbar_drain(bars + 8 * (n % S * WT + tg), (n / S) & 1, kWaitLimitNs);
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
    pdl_wait_then_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int group = p.Hq / p.Hkv, rows = group * p.Lq, chunks = (rows + RT - 1) / RT, hr_n = p.Hkv * chunks;
    const int b = blockIdx.x / hr_n, hr = blockIdx.x - b * hr_n;
    int64_t before, total;
    count_units(p, C::CT, hr_n, b, &before, &total);
    const Span s = span_of(p, b, C::CT);
    const int64_t chunk = chunk_of(total, ctas), first = before + (int64_t)hr * s.tiles;
    const int c0 = (int)(first / chunk), c1 = (int)((first + s.tiles - 1) / chunk);
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
        for (int c = begin + lane * step; c <= c1; c += 32 * step) m = fmaxf(m, slot(c)[RT * DP + r]);
#pragma unroll
        for (int off = 16; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
#pragma unroll 4
        for (int c = begin; c <= c1; c += step) {
            const float* x = slot(c);
            const float f = ex2(x[RT * DP + r] - m);
            l += x[RT * DP + RT + r] * f;
#pragma unroll
            for (int k = 0; k < V4; ++k) {
                const int d = (k * 32 + lane) * 4;
                if (d < DP) {
                    const float4 v = *reinterpret_cast<const float4*>(x + r * DP + d);
                    o[k].x += f * v.x, o[k].y += f * v.y, o[k].z += f * v.z, o[k].w += f * v.w;
                }
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

// What a configuration takes for these sizes.
struct Plan {
    size_t ws;
    int kernels;
};
template <class C>
Plan plan(int64_t max_len) {
    if (max_len <= C::CT) return Plan{0, 1};                  // one tile covers every item: nothing is split
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
    if constexpr (C::kTma) {
        p.box = C::TT;
        while (p.page_size % p.box) p.box /= 2;
        p.order = p.c_token < p.c_head && p.Hkv > 1;
        if (!make_map<C>(&km, p.kpool, p) || !make_map<C>(&vm, p.vpool, p)) return cudaErrorInvalidValue;
    }
    const int rows = p.Hq / p.Hkv * p.Lq, chunks = (rows + C::RT - 1) / C::RT;
    const int64_t items = (int64_t)p.B * p.Hkv * chunks, tiles = (p.max_len + C::CT - 1) / C::CT;
    const int64_t most = items * (tiles > 1 ? tiles : 1), wave = (int64_t)num_sms() * C::kCtas;
    cudaError_t e = cudaFuncSetAttribute(attn_paged_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    const int ctas = (int)(most < wave ? most : wave);
    e = launch_pdl(attn_paged_kernel<C>, dim3((unsigned)ctas), dim3(kThreads), C::kSmem, st, p, km, vm);
    if (e != cudaSuccess || tiles <= 1) return e;
    const bool spread = items * 2 < num_sms();
    return launch_pdl(attn_join_kernel<C>, dim3((unsigned)items, spread ? (unsigned)(rows < C::RT ? rows : C::RT) : 1u),
                      dim3(256), 0, st, p, ctas, (int)spread);
}

// The configuration for a head width and a number of query rows (query heads of
// a kv head x Lq): as few row tiles as hold them, so that no product is spent on
// rows that are not there; above the largest the rows go in chunks, each reading
// the cache again.
template <bool kE4m3, bool kTma, class F>
auto pick(int64_t D, int64_t rows, F f) {
    if (D <= 64) {
        if (rows <= 8) return f(Config<kE4m3, kTma, 64, 1, 1>{});
        if (rows <= 16) return f(Config<kE4m3, kTma, 64, 2, 1>{});
        if (rows <= 32) return f(Config<kE4m3, kTma, 64, 4, 1>{});
        return f(Config<kE4m3, kTma, 64, 4, 2>{});
    }
    if (D <= 128) {
        if (rows <= 8) return f(Config<kE4m3, kTma, 128, 1, 1>{});
        if (rows <= 16) return f(Config<kE4m3, kTma, 128, 2, 1>{});
        if (rows <= 32) return f(Config<kE4m3, kTma, 128, 4, 1>{});
        return f(Config<kE4m3, kTma, 128, 4, 2>{});
    }
    if (rows <= 8) return f(Config<kE4m3, kTma, 256, 1, 1>{});
    if (rows <= 16) return f(Config<kE4m3, kTma, 256, 2, 1>{});
    return f(Config<kE4m3, kTma, 256, 2, 2>{});
}

}  // namespace attn

// One translation unit a cache type and loader (they compile side by side).
cudaError_t launch_attn_bf16_tma(const AttnParams& p, cudaStream_t st);
cudaError_t launch_attn_bf16(const AttnParams& p, cudaStream_t st);
cudaError_t launch_attn_e4m3_tma(const AttnParams& p, cudaStream_t st);
cudaError_t launch_attn_e4m3(const AttnParams& p, cudaStream_t st);

}  // namespace fp8rl
