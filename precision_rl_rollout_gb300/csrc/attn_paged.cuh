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
constexpr float kLog2e = 1.4426950408889634f;

template <bool kE4m3_, int DP_, int NT_, int WR_>
struct Config {
    static constexpr bool kE4m3 = kE4m3_;
    static constexpr int DP = DP_;             // padded head width
    static constexpr int NT = NT_, WR = WR_;   // 8-row tiles a warp, warps over the rows
    static constexpr int RT = 8 * NT * WR;     // query rows of a CTA
    static constexpr int WT = kWarps / WR;     // token groups
    static constexpr int RB = DP * (kE4m3 ? 1 : 2);      // bytes of a cached head
    static constexpr int CPR = RB / 16;                  // its 16-byte chunks
    static constexpr int TT = kE4m3 ? 32 : 16, MT = TT / 16;   // tokens of a warp's tile
    static constexpr int CT = TT * WT;                   // tokens of a CTA's tile
    static constexpr int kStage = 2 * TT * RB;           // K and V of one group's tile
    static constexpr int kMerge = (WT > 1 ? WT / 2 : 1) * RT * DP * 4;
    static constexpr int kCtas = DP > 128 ? 1 : 2;       // CTAs an SM
    static constexpr int kBudget = 233472 / kCtas - 1024;     // 228 KB an SM, 1 KB of it kept for each CTA
    static constexpr int kFit = (kBudget - kMerge - WT * RT * 8) / (WT * kStage);
    static constexpr int kStages = kFit > 6 ? 6 : kFit;
    static constexpr int kSmem = kStages * WT * kStage + kMerge + WT * RT * 8;
    static_assert(kStages >= 2, "too little shared memory for two stages");
};

// Tokens the sequence's queries see at all, and the item's tiles over them (one
// at least, so that every item has a writer).
struct Span {
    int lo, len, tiles;
};
__device__ __forceinline__ Span span_of(const AttnParams& p, int b, int ct) {
    Span s;
    s.len = min(max(p.lens[b], 0), p.max_len);
    s.lo = p.window ? max(0, s.len - p.Lq + 1 - p.window) : 0;
    s.tiles = max(1, (s.len - s.lo + ct - 1) / ct);
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
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
template <bool kF16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (kF16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
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

// Shared-memory offset of chunk c of row r: 16-byte chunks exchanged so that the
// eight rows of a matrix load lie in different banks.
template <int RB>
__device__ __forceinline__ uint32_t swz(int r, int c) {
    if constexpr (RB >= 128)
        return (uint32_t)(r * RB + ((c ^ (r & 7)) << 4));
    else
        return (uint32_t)(r * RB + ((c ^ ((r >> 1) & 3)) << 4));
}

// Two packed 16-bit floats with infinities and NaN replaced by zero.
template <bool kF16>
__device__ __forceinline__ uint32_t finite2(uint32_t v, bool& bad) {
    constexpr uint32_t e = kF16 ? 0x7C00u : 0x7F80u;
    const bool l = (v & e) == e, h = (v & (e << 16)) == (e << 16);
    bad |= l | h;
    return (l ? 0u : v & 0xFFFFu) | (h ? 0u : v & 0xFFFF0000u);
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
attn_paged_kernel(const __grid_constant__ AttnParams p) {
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr bool kE = C::kE4m3;
    constexpr int NT = C::NT, WR = C::WR, RT = C::RT, WT = C::WT, RB = C::RB, TT = C::TT, MT = C::MT, CT = C::CT;
    constexpr int KS = C::DP / 16, S = C::kStages;
    constexpr float kBias = kE ? 6.f : 0.f;
    float* const merge = reinterpret_cast<float*>(smem + S * WT * C::kStage);
    float* const sm_m = merge + C::kMerge / 4;               // [WT][RT]
    float* const sm_l = sm_m + WT * RT;

    pdl_wait_then_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int tg = warp / WR, wr = warp % WR;                // token group, row group
    const int group = p.Hq / p.Hkv, rows = group * p.Lq, chunks = (rows + RT - 1) / RT, hr_n = p.Hkv * chunks;

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

    // loader: this lane's token offsets of the next tile, looked up a tile ahead
    const uint32_t ring = sm100::smem_u32(smem) + tg * C::kStage;      // stage s: + s * WT * kStage
    const int cpr = p.D * (kE ? 1 : 2) / 16;                            // chunks the cache has of a head
    const uint8_t* const kp = static_cast<const uint8_t*>(p.kpool);
    const uint8_t* const vp = static_cast<const uint8_t*>(p.vpool);
    constexpr int ES = kE ? 1 : 2;
    auto lookup = [&](const Cursor& c) -> int64_t {                     // -1: no such token
        const int j = c.s.lo + c.tile * CT + tg * TT + (lane % TT);
        if (j >= c.s.len) return -1;
        const int pg = j / p.page_size;
        int page = p.pages[c.b * p.pages_seq + pg];
        if ((uint32_t)page >= (uint64_t)p.num_pages) {
            atomicCAS(p.err, 0u, (kKernelAttn << 24) | (2u << 16) | 2u);
            page = 0;
        }
        return (page * p.c_page + (int64_t)(j - pg * p.page_size) * p.c_token + (c.hr / chunks) * p.c_head) * ES;
    };
    int issued = 0;
    int64_t off = lookup(ld);
    auto issue = [&]() {
        if (issued < count) {
            const uint32_t dst = ring + (issued % S) * (WT * C::kStage);
            constexpr int RPI = 32 / C::CPR > 0 ? 32 / C::CPR : 1;      // rows a warp covers at once
            constexpr int CPI = C::CPR > 32 ? C::CPR / 32 : 1;          // turns a row takes
            constexpr int kTurns = TT / RPI / WR;
#pragma unroll
            for (int i = 0; i < kTurns; ++i) {
                const int r = (wr * kTurns + i) * RPI + (C::CPR < 32 ? lane / C::CPR : 0);
                const int64_t o = __shfl_sync(0xffffffffu, off, r);
#pragma unroll
                for (int k = 0; k < CPI; ++k) {
                    const int c = C::CPR < 32 ? lane % C::CPR : lane + 32 * k;
                    const uint32_t n = o >= 0 && c < cpr ? 16u : 0u;
                    const int64_t src = n ? o + c * 16 : 0;
                    cp_async16(dst + swz<RB>(r, c), kp + src, n);
                    cp_async16(dst + TT * RB + swz<RB>(r, c), vp + src, n);
                }
            }
            ld.next(p, CT, hr_n);
            ++issued;
            if (issued < count) off = lookup(ld);
        }
        cp_async_commit();
    };
    auto group_sync = [&]() {
        if constexpr (WR == 1)
            __syncwarp();
        else
            sm100::named_bar_sync(1 + tg, WR * 32);
    };

    // a segment's queries and bounds
    uint32_t q[NT][KS][2];
    float fac[NT][2];                          // log2 units a unit of the product, columns 2t and 2t + 1
    int hi[NT][2], lo[NT][2];                  // tokens the columns' queries see
    float o[NT][KS][4], ref[NT][2], sum[NT][2];
    const float xs = p.scale * kLog2e * (kE ? *p.k_scale : 1.f);

    auto begin = [&]() {
        const int h = at.hr / chunks, r0 = (at.hr - h * chunks) * RT + wr * 8 * NT;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = r0 + n * 8 + g, i = r / group;
            const uint16_t* src = p.q + at.b * p.q_seq + i * p.q_token + (h * group + r - i * group) * p.q_head;
            float f0 = xs, f1 = xs;
            if constexpr (kE) {
                float top = 0.f;
                uint2 w[KS];
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    w[k] = make_uint2(0, 0);
                    if (r < rows && 16 * k < p.D) w[k] = *reinterpret_cast<const uint2*>(src + 16 * k + 4 * t);
                    top = fmaxf(top, fmaxf(fmaxf(fabsf(bf16_lo(w[k].x)), fabsf(bf16_hi(w[k].x))),
                                           fmaxf(fabsf(bf16_lo(w[k].y)), fabsf(bf16_hi(w[k].y)))));
                }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int e = (int)(__float_as_uint(top) >> 23);            // biased exponent
                // 2^(141 - e) puts the largest at 2^14; its reciprocal goes into the factor
                const bool plain = e == 0 || e == 255;
                const float up = plain ? 1.f : exp2f((float)(141 - e)), down = plain ? 1.f : exp2f((float)(e - 141));
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    q[n][k][0] = pack_f16x2(bf16_lo(w[k].x) * up, bf16_hi(w[k].x) * up);
                    q[n][k][1] = pack_f16x2(bf16_lo(w[k].y) * up, bf16_hi(w[k].y) * up);
                }
                f0 *= __shfl_sync(0xffffffffu, down, 8 * t);                // row 2t is held by lanes 8t .. 8t + 3
                f1 *= __shfl_sync(0xffffffffu, down, 8 * t + 4);
            } else {
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    q[n][k][0] = q[n][k][1] = 0;
                    if (r < rows && 16 * k < p.D) {
                        q[n][k][0] = *reinterpret_cast<const uint32_t*>(src + 16 * k + 2 * t);
                        q[n][k][1] = *reinterpret_cast<const uint32_t*>(src + 16 * k + 8 + 2 * t);
                    }
                }
            }
            fac[n][0] = f0, fac[n][1] = f1;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int rc = r0 + n * 8 + 2 * t + c;
                hi[n][c] = rc < rows ? at.s.len - p.Lq + rc / group + 1 : 0;
                lo[n][c] = p.window ? max(0, hi[n][c] - p.window) : 0;
                ref[n][c] = -INFINITY;
                sum[n][c] = 0.f;
            }
#pragma unroll
            for (int k = 0; k < KS; ++k) o[n][k][0] = o[n][k][1] = o[n][k][2] = o[n][k][3] = 0.f;
        }
    };

    auto compute = [&](uint32_t kb, int t0) {
        const uint32_t vb = kb + TT * RB;
        // S^T: two chains of products, added at the end
        float s[NT][MT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            float s2[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[n][m][e] = s2[n][e] = 0.f;
            const int r = m * 16 + (lane & 15);
            if constexpr (kE) {
#pragma unroll
                for (int k = 0; k < KS; k += 2) {
                    uint32_t w[4], a[4], b[4];
                    ldsm4(w, kb + swz<RB>(r, k + (lane >> 4)));
                    e4m3x4_f16(w[0], a[0], a[2]);
                    e4m3x4_f16(w[1], a[1], a[3]);
                    e4m3x4_f16(w[2], b[0], b[2]);
                    e4m3x4_f16(w[3], b[1], b[3]);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma16816<true>(s[n][m], a, q[n][k][0], q[n][k][1]);
                        mma16816<true>(s2[n], b, q[n][k + 1][0], q[n][k + 1][1]);
                    }
                }
            } else {
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    uint32_t a[4];
                    ldsm4(a, kb + swz<RB>(r, 2 * k + (lane >> 4)));
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma16816<false>(k & 1 ? s2[n] : s[n][m], a, q[n][k][0], q[n][k][1]);
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[n][m][e] = (s[n][m][e] + s2[n][e]) * fac[n][e & 1];
        }
        // tokens that some of the queries do not see
        const bool edge = t0 + TT > at.s.len - p.Lq + 1 || (p.window && t0 < at.s.len - p.window);
        if (edge) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = t0 + m * 16 + g + 8 * (e >> 1);
                        if (j >= hi[n][e & 1] || j < lo[n][e & 1]) s[n][m][e] = -INFINITY;
                    }
        }
        // running reference
        bool grow = false;
        float top[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float x = -INFINITY;
#pragma unroll
                for (int m = 0; m < MT; ++m) x = fmaxf(x, fmaxf(s[n][m][c], s[n][m][c + 2]));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                top[n][c] = x - kBias;
                grow |= top[n][c] > ref[n][c] + kLazy;
            }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float f[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float r = fmaxf(ref[n][c], top[n][c]);
                    f[c] = r == -INFINITY ? 1.f : ex2(ref[n][c] - r);
                    ref[n][c] = r;
                    sum[n][c] *= f[c];
                }
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[n][k][e] *= f[e & 1];
            }
        }
        uint32_t pt[NT][MT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float r0 = ref[n][0] == -INFINITY ? 0.f : ref[n][0], r1 = ref[n][1] == -INFINITY ? 0.f : ref[n][1];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
#pragma unroll
                for (int e = 0; e < 4; ++e) s[n][m][e] = ex2(s[n][m][e] - (e & 1 ? r1 : r0));
                sum[n][0] += s[n][m][0] + s[n][m][2];
                sum[n][1] += s[n][m][1] + s[n][m][3];
                const uint32_t x = kE ? pack_f16x2(s[n][m][0], s[n][m][1]) : pack_bf16x2(s[n][m][0], s[n][m][1]);
                const uint32_t y = kE ? pack_f16x2(s[n][m][2], s[n][m][3]) : pack_bf16x2(s[n][m][2], s[n][m][3]);
                pt[n][m][0] = transpose8x8(x);
                pt[n][m][1] = transpose8x8(y);
            }
        }
        // O^T += V^T P^T.  A value that only some of the queries see must not reach
        // the others as 0 x NaN: in an edge tile of several queries what is not
        // finite is left out of the product, and added where it is seen below.
        const bool guard = edge && p.Lq > 1;
        bool bad = false;
        auto product = [&](int m, int k, uint32_t (&a)[4]) {
            if (guard)
#pragma unroll
                for (int e = 0; e < 4; ++e) a[e] = finite2<kE>(a[e], bad);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816<kE>(o[n][k], a, pt[n][m][0], pt[n][m][1]);
        };
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            if constexpr (kE) {
#pragma unroll
                for (int k = 0; k < KS; k += 2) {
                    uint32_t w[4], a[4], b[4];
                    ldsm4_t(w, vb + swz<RB>(m * 16 + (lane & 15), k + (lane >> 4)));
                    e4m3x4_f16(__byte_perm(w[0], 0, 0x3120), a[0], a[1]);
                    e4m3x4_f16(__byte_perm(w[1], 0, 0x3120), a[2], a[3]);
                    e4m3x4_f16(__byte_perm(w[2], 0, 0x3120), b[0], b[1]);
                    e4m3x4_f16(__byte_perm(w[3], 0, 0x3120), b[2], b[3]);
                    product(m, k, a);
                    product(m, k + 1, b);
                }
            } else {
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    uint32_t a[4];
                    ldsm4_t(a, vb + swz<RB>(m * 16 + (lane & 7) + (lane >> 4) * 8, 2 * k + ((lane >> 3) & 1)));
                    product(m, k, a);
                }
            }
        }
        if (guard && __any_sync(0xffffffffu, bad)) {
            for (int j = 0; j < TT; ++j)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float w0 = 0.f, w1 = 0.f;              // the token's probabilities in columns 2t, 2t + 1
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        const float x0 = j & 8 ? s[n][m][2] : s[n][m][0], x1 = j & 8 ? s[n][m][3] : s[n][m][1];
                        const float y0 = __shfl_sync(0xffffffffu, x0, (j & 7) * 4 + t);
                        const float y1 = __shfl_sync(0xffffffffu, x1, (j & 7) * 4 + t);
                        if (m == j >> 4) w0 = y0, w1 = y1;
                    }
                    const bool see0 = t0 + j < hi[n][0] && t0 + j >= lo[n][0];
                    const bool see1 = t0 + j < hi[n][1] && t0 + j >= lo[n][1];
#pragma unroll
                    for (int k = 0; k < KS; ++k)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int d = kE ? 16 * k + 2 * g + e : 16 * k + g + 8 * e;
                            float v;
                            const uint32_t a = vb + swz<RB>(j, d * ES / 16) + (d * ES) % 16;
                            uint32_t raw;
                            if constexpr (kE) {
                                uint32_t f16, unused;
                                asm volatile("ld.shared.u8 %0, [%1];" : "=r"(raw) : "r"(a) : "memory");
                                e4m3x4_f16(raw, f16, unused);
                                v = __half2float(__ushort_as_half((unsigned short)f16));
                            } else {
                                asm volatile("ld.shared.u16 %0, [%1];" : "=r"(raw) : "r"(a) : "memory");
                                v = __uint_as_float(raw << 16);
                            }
                            if (isfinite(v)) continue;
                            if (see0) o[n][k][2 * e] += w0 * v;
                            if (see1) o[n][k][2 * e + 1] += w1 * v;
                        }
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
                float m = -INFINITY, l = 0.f;
#pragma unroll
                for (int w = 0; w < WT; ++w) m = fmaxf(m, sm_m[w * RT + r]);
                const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
                for (int w = 0; w < WT; ++w) l += sm_l[w * RT + r] * ex2(sm_m[w * RT + r] - base);
                const float f = ex2(ref[n][c] - base);
#pragma unroll
                for (int k = 0; k < KS; ++k) o[n][k][c] *= f, o[n][k][c + 2] *= f;
                M[n][c] = m, L[n][c] = l;
            }
        auto place = [&](int n, int k, int e) {                // [row][value] of a sum
            const int d = kE ? 16 * k + 2 * g + (e >> 1) : 16 * k + g + 8 * (e >> 1);
            return (wr * 8 * NT + n * 8 + 2 * t + (e & 1)) * C::DP + d;
        };
#pragma unroll
        for (int half = WT / 2; half >= 1; half /= 2) {
            if (tg >= half && tg < 2 * half)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int k = 0; k < KS; ++k)
#pragma unroll
                        for (int e = 0; e < 4; ++e) merge[(tg - half) * RT * C::DP + place(n, k, e)] = o[n][k][e];
            __syncthreads();
            if (tg < half)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int k = 0; k < KS; ++k)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[n][k][e] += merge[tg * RT * C::DP + place(n, k, e)];
            __syncthreads();
        }
        if (tg == 0) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) merge[place(n, k, e)] = o[n][k][e];
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
                if (p.lse && d == 0) p.lse[row] = l == 0.f ? -INFINITY : (sm_m[r] + log2f(l)) * 0.6931471805599453f;
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

#pragma unroll
    for (int s = 0; s < S - 1; ++s) issue();
    begin();
    for (int n = 0; n < count; ++n) {
        cp_async_wait<S - 2>();
        group_sync();
        issue();
        const int t0 = at.s.lo + at.tile * CT + tg * TT;
        if (t0 < at.s.len) compute(ring + (n % S) * (WT * C::kStage), t0);
        const bool end = at.tile + 1 == at.s.tiles || n + 1 == count;
        if (end) finish(u0 + n);
        at.next(p, CT, hr_n);
        if (end && n + 1 < count) begin();
    }
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
        float m = -INFINITY, l = 0.f;
        float4 o[V4];
#pragma unroll
        for (int k = 0; k < V4; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        const int begin = c0 + (spread ? warp : 0), step = spread ? kW : 1;
        for (int c = begin + lane * step; c <= c1; c += 32 * step) m = fmaxf(m, slot(c)[RT * DP + r]);
#pragma unroll
        for (int off = 16; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        const float base = m == -INFINITY ? 0.f : m;
#pragma unroll 4
        for (int c = begin; c <= c1; c += step) {
            const float* x = slot(c);
            const float f = ex2(x[RT * DP + r] - base);
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
            m = -INFINITY, l = 0.f;
            for (int w = 0; w < kW; ++w) m = fmaxf(m, sm[w]);
            const float top = m == -INFINITY ? 0.f : m;
#pragma unroll
            for (int k = 0; k < V4; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (warp == 0)
                for (int w = 0; w < kW; ++w) {
                    const float f = ex2(sm[w] - top);
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
        if (p.lse && lane == 0) p.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
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

template <class C>
cudaError_t launch(const AttnParams& p, cudaStream_t st) {
    const int rows = p.Hq / p.Hkv * p.Lq, chunks = (rows + C::RT - 1) / C::RT;
    const int64_t items = (int64_t)p.B * p.Hkv * chunks, tiles = (p.max_len + C::CT - 1) / C::CT;
    const int64_t most = items * (tiles > 1 ? tiles : 1), wave = (int64_t)num_sms() * C::kCtas;
    cudaError_t e = cudaFuncSetAttribute(attn_paged_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    const int ctas = (int)(most < wave ? most : wave);
    e = launch_pdl(attn_paged_kernel<C>, dim3((unsigned)ctas), dim3(kThreads), C::kSmem, st, p);
    if (e != cudaSuccess || tiles <= 1) return e;
    const bool spread = items * 2 < num_sms();
    return launch_pdl(attn_join_kernel<C>, dim3((unsigned)items, spread ? (unsigned)(rows < C::RT ? rows : C::RT) : 1u),
                      dim3(256), 0, st, p, ctas, (int)spread);
}

// The configuration for a head width and a number of query rows (query heads of
// a kv head x Lq): as few row tiles as hold them, so that no product is spent on
// rows that are not there; above the largest the rows go in chunks, each reading
// the cache again (from L2, where the chunks of an item stand side by side).
template <bool kE4m3, class F>
auto pick(int64_t D, int64_t rows, F f) {
    if (D <= 64) {
        if (rows <= 8) return f(Config<kE4m3, 64, 1, 1>{});
        if (rows <= 16) return f(Config<kE4m3, 64, 2, 1>{});
        if (rows <= 32) return f(Config<kE4m3, 64, 2, 2>{});
        return f(Config<kE4m3, 64, 2, 4>{});
    }
    if (D <= 128) {
        if (rows <= 8) return f(Config<kE4m3, 128, 1, 1>{});
        if (rows <= 16) return f(Config<kE4m3, 128, 2, 1>{});
        if (rows <= 32) return f(Config<kE4m3, 128, 2, 2>{});
        return f(Config<kE4m3, 128, 2, 4>{});
    }
    if (rows <= 8) return f(Config<kE4m3, 256, 1, 1>{});
    if (rows <= 16) return f(Config<kE4m3, 256, 1, 2>{});
    return f(Config<kE4m3, 256, 1, 4>{});
}

}  // namespace attn

// One translation unit a cache type (they compile side by side).
cudaError_t launch_attn_paged_bf16(const AttnParams& p, cudaStream_t st);
cudaError_t launch_attn_paged_e4m3(const AttnParams& p, cudaStream_t st);
attn::Plan plan_attn_paged_bf16(int64_t D, int64_t rows, int64_t max_len);
attn::Plan plan_attn_paged_e4m3(int64_t D, int64_t rows, int64_t max_len);

}  // namespace fp8rl
