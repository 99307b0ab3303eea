// linear_logp.cu -- log-probabilities of chosen tokens straight from the hidden states H
// and the output matrix W, without keeping the logits, and their gradient.
//
//   x_mv = scale h_m . w_v,   lse_m = log sum_v exp x_mv,   p = exp(x - lse),
//   logp_m = x_mt - lse_m,    entropy_m = - sum_v p_v log p_v,
//   D_mv = g_m (d_vt - p_mv) - e_m p_mv (log p_mv + entropy_m),
//   dH = scale D W,   dW = scale D^T H.
//
// Rows that count are brought together first (rows_kernel): prompts and padding take no
// part in the products, and what they hold reaches nothing.
//
// All products are tiles of 256 x 256 by a pair of CTAs (tcgen05.mma.cta_group::2, bf16,
// sums in tensor memory, fp32): each CTA stages 128 rows of either operand, 64 of the
// reduction a stage, and has 128 of the tile's rows in its tensor memory, two tiles of them,
// so that one tile's threads' part runs under the next one's products.  Up to 128 rows the
// forward is a pass over W, and the roles change (logp_few_kernel).
//
// Forward (kLogp): tile by tile each row leaves a maximum, its sum of exponentials and
// of weighted differences (12 bytes for 128 logits); logp_join_kernel joins a row's tiles.
// Backward: the vocabulary in pieces, two launches each.  kGrad writes a piece's D as bf16
// (rounded once, relative to the call's largest |g| and |e|: a mean's gradient, 1/n
// everywhere, is then exact); kBack multiplies it with W's rows (D as it lies, W with the
// reduction outside: MN-major) into fp32 sums of dH that the pieces add to, and its
// transpose with H (both MN-major) into the piece's rows of dW.  Nothing is transposed in
// memory, and each sum of dH is added to once a launch, so results do not depend on order.
//
// What bounds it: the tensor cores, and for long calls the power they draw.  4096 rows of
// 152064 words x 3584: 2.30 ms alone, 1.94 PFLOP/s (the measured peak is 1.92), 2.6 in a loop, where
// the clocks fall to 1.55 GHz and a library's product of this size makes 1.8; 8192 rows, 5734 of
// them counted, 3.9.  Both gradients of 4096 rows 7.8 to 8.0 ms (1.67 to 1.72 PFLOP/s), of 2731 among 4096
// 5.5, 4.86 alone.  Profiled on 2048 rows of 65536: kLogp 0.50 ms, kGrad 0.52, kBack 1.01, the tensor pipe
// 84 to 89% active.  One row 161 to 164 us, 48 rows x 5120 228 to 233: the copy rate.  With few rows
// the gradient is bound by writing dW (a stream of writes alone makes 4 TB/s): one row 0.55 ms.
#include <math.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "internal.h"
#include "sm100_ptx.cuh"

namespace fp8rl {

using namespace sm100;

namespace {

constexpr uint32_t kKernelLogp = 10;
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr float kLog2e = 1.4426950408889634f;
constexpr double kLn2 = 0.6931471805599453;

constexpr int kTile = 256, kHalf = 128, kStep = 64;     // a pair's tile, a CTA's share, the reduction a stage
constexpr int kPiece = 64 * 128;                        // 64 rows of 64 values, as the copy engine lays them
constexpr int kOutBytes = 32 * 128;                     // a warp's staging

enum Mode { kLogp, kGrad, kBack };

// Eight warps have the threads' part, half of a row a thread.  kLogp and kGrad keep it in registers,
// which the other warps let go of.  kLogp stages nothing; the others stage what they write, a box
// a warp.  Six stages: with five, and two boxes, the gradients take 1 to 9% longer (500 rows of
// 32000 x 1024 99 us for 91), with seven the forward up to 3%.
template <Mode kMode>
struct Config {
    static constexpr bool kForward = kMode == kLogp;
    static constexpr int kStages = 6, kStageBytes = 4 * kPiece;   // two pieces of either operand
    static constexpr int kEpiWarps = 8, kThreads = 32 * (4 + kEpiWarps);
    static constexpr int kOuts = kForward ? 0 : 1;           // boxes a warp stages at once
    static constexpr int kOutOffset = kStages * kStageBytes;
    static constexpr int kBarOffset = kOutOffset + kEpiWarps * kOuts * kOutBytes;
    static constexpr int kSmemBytes = kBarOffset + 256 + 1024;
    static_assert(kSmemBytes <= 232448, "shared memory per CTA");
};
constexpr int kLaunchRegs = 168, kOtherRegs = 40, kEpiRegs = 232;   // kLogp, kGrad: registers a thread, at launch and after
static_assert(128 * kOtherRegs + 256 * kEpiRegs <= 384 * kLaunchRegs, "the split must fit the launch's registers");

// The tensor cores' fp32 sums lose more at each step than rounding to nearest would, and the
// loss grows with the steps: 3.1e-6 of the log-probabilities over 3584 products (against 64 bits;
// 32-bit torch 4.5e-7).  The forward takes the sums out of tensor memory every 896 products
// at most and adds in registers: 6.9e-7.  Every 512 it is 3.6e-7, but 8% slower, since tensor
// memory serves these reads at the products' expense.  Few rows, bound by HBM, every 256:
// 1.1e-7, and 0 to 3% slower than every 512 with 2.1e-7.  The gradient's logits are summed in the
// same steps, so that they have the bits of those that lse came from: a target's D is g (1 - p), and
// an error that its logit has and lse has not is not relative to 1 - p.  Left in tensor memory for
// all of 3584 products it was 6e-5 g, and dH of a row whose policy is sure to 1e-4 off by 1.5 times itself
// (32-bit torch: 6e-3); now 5e-7 g and 1.5e-2.  Both gradients of 4096 rows take 1.7% longer (7.64 -> 7.77
// ms), of one row 1%, dH alone 2 to 5%.
constexpr int kSegment = 896 / kStep, kFewSegment = 256 / kStep;
// kBack's sums run over rows (dW) or words (dH), and leave tensor memory once: 16 bits are
// kept of them.  Past this many products a unit's sums are put together from parts of as many (see
// the products): dW of 2^20 rows whose terms have one sign was off by 6.1e-3, its own rounding being 1.6e-3.
constexpr int kBackSegment = 65536 / kStep;

// ------------------------------------------------------------------ pairs of CTAs

// A box into this CTA's shared memory, counted on the barrier of the pair's first CTA.
__device__ __forceinline__ void pair_load(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, uint64_t pol) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2.L2::cache_hint"
        " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "l"(pol)
        : "memory");
}
__device__ __forceinline__ void pair_load_mn(uint32_t dst, const CUtensorMap* map, uint32_t bar, int piece, int row,
                                             uint64_t pol) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(piece), "r"(bar), "l"(pol)
        : "memory");
}
__device__ __forceinline__ uint64_t policy_evict_normal() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n.reg .pred p;\n"
        "setp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// One arrival on the barrier at this offset in both CTAs, once the products so far are done.
__device__ __forceinline__ void pair_commit(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}
// What it hands over is tensor memory, which the tcgen05 fence before it orders; no other
// memory, so no release at cluster scope (that waits for this thread's stores to global memory).
__device__ __forceinline__ void pair_arrive(uint32_t cluster_bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}
__device__ __forceinline__ void tma_add_2d(const CUtensorMap* map, uint32_t src, int x, int y) {
    asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(src)
                 : "memory");
}

// An operand of two pieces with the reduction outside (MN-major): 16 of the reduction are
// 2048 bytes on, the next 64 values a piece.
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr) {
    return (uint64_t)((addr >> 4) & 0x3FFFu) | (uint64_t)(kPiece >> 4) << 16 | (uint64_t)(1024u >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// bf16 x bf16 -> fp32, 256 x 256; bits 15 and 16: A, B are MN-major
constexpr uint32_t kIdesc = 1u << 4 | 1u << 7 | 1u << 10 | (kTile >> 3) << 17 | (uint32_t)(kTile >> 4) << 24;

// Two fp32 to bf16, rounded to nearest even, in one instruction: converted one by one, a
// tile of dW's 64 values a thread take its CTA 1000 cycles.
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

// A ring's stage and the phase of its barriers, and whether the barrier that is waited for
// next was seen complete already.  One thread issues the products and one or two the
// loads; a wait that finds its barrier complete still takes 200 cycles before anything after
// it is issued, and so each looks one stage ahead before it issues what it has.
template <int kStages>
struct Ring {
    uint32_t s = 0, phase = 0;
    bool ready = false;
    __device__ __forceinline__ void next() {
        if (++s == kStages) s = 0, phase ^= 1;
    }
    // bars: the barriers; flip: 0 for what is filled, 1 for what is emptied (free at first)
    __device__ __forceinline__ void look(uint32_t bars, uint32_t flip) { ready = mbar_test(bars + 8 * s, phase ^ flip); }
    __device__ __forceinline__ bool wait(uint32_t bars, uint32_t flip, const volatile int* abort) {
        return ready || mbar_wait_bounded(bars + 8 * s, phase ^ flip, abort, kWaitLimitNs);
    }
};

// Loads with the reduction inside are boxes of 64 values of 128 rows, or of 64 where no more
// rows count; with the reduction outside 64 rows of two pieces of 64 values (*_mn; of one
// where a row of W does not end with a piece).
struct Maps {
    CUtensorMap h, h64, h_mn, w, w_mn, d, d64, d_mn, d_out, acc, dw;
};

// ------------------------------------------------------------------ the work

// A tile: rows a of the first operand, rows b of the second, steps [k, k + n) of 64 of
// the reduction.
struct Unit {
    int kind;           // 0: logits, 1: dH, 2: dW
    int a, b, k, n, slot;
};

// Tile order of the logits: groups of row tiles whose H stays in L2; in a group the row
// tile runs fastest, so that a tile of W is read by all of them while it is there.
__device__ __forceinline__ void tile_of(int u, int rows, int cols, int group, int& r, int& c) {
    const int g = u / (group * cols), left = u - g * group * cols, here = min(group, rows - g * group);
    c = left / here;
    r = g * group + left % here;
}

constexpr int kLeastSteps = 6;   // steps' time that writing a tile of dW takes all the same

template <Mode kMode>
struct Work {
    const LogpParams& p;
    int rows, live, pair, pairs, i = 0;
    // kLogp, kGrad: row tiles a group.  kBack: units of dH and of dW, dH's a row of parts, steps
    // of dW, units of dW taken first by pairs from `from` on, in all, which comes first, phase
    int group = 1, nh = 0, nw = 0, part = 1, wsteps = 0, extra = 0, from = 0, head = 0, flip = 0, phase = 0;

    __device__ __forceinline__ Work(const LogpParams& p_) : p(p_) {
        live = *p.live;
        rows = (live + kTile - 1) / kTile;
        pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
        if constexpr (kMode != kBack) {
            const int groups = max(1, (rows + p.group - 1) / p.group);
            group = (rows + groups - 1) / groups;
        } else {
            // dH's units and dW's in turn: pairs that have one unit of dH less take as many of
            // dW as last as long, the others follow in turn.  With few rows and a W not much larger
            // than L2 every other pair takes dW's first, so that writing goes on beside reading and
            // products (one after the other, then beside each other, us: 500 rows of 32000 x 1024 92 and
            // 90, 200 of 32000 x 2048 105 and 101, 20 of it 92.7 and 91.1); else each is better off with L2
            // and HBM to itself (20 rows of 50257 x 2048 129.6 and 131.6, of 152064 x 5120 754 and
            // 797, one of 152064 x 3584 549 and 557, 1000 of 50257 x 896 198 and 210; 200 rows of 50257 to
            // 100000 x 2048 would gain 1%).
            part = max(1, rows * p.ktiles);
            nh = p.dH ? rows * p.ktiles * p.split : 0, nw = p.dW ? p.tiles * p.ktiles : 0;
            wsteps = (live + kStep - 1) / kStep, from = nh % pairs;
            const int cost = max(wsteps, kLeastSteps);
            extra = from && wsteps ? (p.steps / p.split + cost / 2) / cost : 0, head = extra * (pairs - from);
            flip = wsteps < 10 && p.V * p.K <= 80ll << 20 ? pair & 1 : 0;
        }
    }
    __device__ __forceinline__ bool next(Unit& u) {
        if constexpr (kMode != kBack) {
            const int at = pair + i++ * pairs;
            if (at >= rows * p.tiles) return false;
            int r, c;
            tile_of(at, rows, p.tiles, group, r, c);
            u = Unit{0, r * kTile, c * kTile, 0, p.ksteps, c};
            return true;
        } else {
            for (; phase < 2; ++phase, i = 0) {
                if (phase ^ flip) {
                    int at = head + pair + i * pairs;
                    if (pair >= from && extra)
                        at = i < extra ? pair - from + i * (pairs - from) : head + pair + (i - extra) * pairs;
                    if (at >= nw) continue;
                    ++i;
                    const int v = (int)((uint32_t)at / (uint32_t)p.ktiles);
                    u = Unit{2, v * kTile, (at - v * p.ktiles) * kTile, 0, wsteps, 0};
                    return true;
                }
                const int at = pair + i * pairs;
                if (at >= nh) continue;
                ++i;
                const int s = at / part, t = at - s * part, r = t / p.ktiles;
                const int k = s * p.steps / p.split, end = (s + 1) * p.steps / p.split;
                u = Unit{1, r * kTile, (t - r * p.ktiles) * kTile, k, end - k, s};
                return true;
            }
            return false;
        }
    }
};

// ------------------------------------------------------------------ a tile's threads' part

// Of a row's logits y = scale log2(e) x: a reference, the sum of 2^(y - top) and that of
// 2^(y - top) (y - top).
struct Sums {
    float top = -3.0e38f, sum = 0.f, dev = 0.f;
    __device__ __forceinline__ void add(float t, float s, float d) {
        const float most = fmaxf(top, t), d0 = top - most, d1 = t - most, f0 = ex2(d0), f1 = ex2(d1);
        dev = (sum > 0.f ? f0 * fmaf(d0, sum, dev) : 0.f) + (s > 0.f ? f1 * fmaf(d1, s, d) : 0.f);
        sum = fmaf(f0, sum, f1 * s);
        if (isnan(t)) sum = t;
        top = most;
    }
};

__device__ __forceinline__ uint64_t pk2(float lo, float hi) { return f32x2_pack(__float_as_uint(lo), __float_as_uint(hi)); }
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
__device__ __forceinline__ uint64_t ex2_2(uint64_t v) {
    const float2 f = f32x2_unpack(v);
    return pk2(ex2(f.x), ex2(f.y));
}

// kCols logits of a row, of which the first n are there, two at a time
template <int kCols, bool kDev>
__device__ __forceinline__ void sums_of(Sums& s, const uint64_t (&x)[kCols / 2], int n, float c) {
    float most = -3.0e38f;
    if (n >= kCols) {
#pragma unroll
        for (int j = 0; j < kCols / 2; ++j) {
            const float2 v = f32x2_unpack(x[j]);
            most = fmaxf(most, fmaxf(v.x, v.y));
        }
    } else {
#pragma unroll
        for (int j = 0; j < kCols / 2; ++j) {
            const float2 v = f32x2_unpack(x[j]);
            if (2 * j < n) most = fmaxf(most, v.x);
            if (2 * j + 1 < n) most = fmaxf(most, v.y);
        }
    }
    s.top = fmaxf(most * c, -3.0e38f);                  // finite where every logit is -inf
    const uint64_t cc = pk2(c, c), low = pk2(-s.top, -s.top);
    uint64_t sum = 0, dev = 0;
    bool careful = n < kCols;
    if (!careful) {
#pragma unroll
        for (int j = 0; j < kCols / 2; ++j) {
            const uint64_t a = fma2(x[j], cc, low), e = ex2_2(a);
            sum = add2(sum, e);
            if (kDev) dev = fma2(e, a, dev);
        }
        if (kDev) {                                     // 0 times a logit of -inf
            const float2 d = f32x2_unpack(dev);
            careful = isnan(d.x + d.y);
        }
    }
    if (careful) {
        sum = dev = 0;
#pragma unroll
        for (int j = 0; j < kCols / 2; ++j) {
            const uint64_t a = fma2(x[j], cc, low);
            float2 e = f32x2_unpack(ex2_2(a));
            e.x = 2 * j < n ? e.x : 0.f, e.y = 2 * j + 1 < n ? e.y : 0.f;
            sum = add2(sum, pk2(e.x, e.y));
            const float2 d = f32x2_unpack(a);
            if (kDev) dev = add2(dev, pk2(e.x > 0.f ? e.x * d.x : 0.f, e.y > 0.f ? e.y * d.y : 0.f));
        }
    }
    const float2 t = f32x2_unpack(sum), d = f32x2_unpack(dev);
    s.sum = t.x + t.y, s.dev = d.x + d.y;
}

// x[i] by masks: an index would put the values in memory
template <int kCols>
__device__ __forceinline__ float pick(const uint64_t (&x)[kCols / 2], int i) {
    uint32_t r = 0;
#pragma unroll
    for (int e = 0; e < kCols; ++e) {
        uint32_t same;
        asm("{\n.reg .pred p;\nsetp.eq.s32 p, %1, %2;\nselp.b32 %0, 0xFFFFFFFF, 0, p;\n}\n" : "=r"(same) : "r"(e), "r"(i));
        const float2 v = f32x2_unpack(x[e / 2]);
        r |= __float_as_uint(e & 1 ? v.y : v.x) & same;
    }
    return __uint_as_float(r);
}
__device__ __forceinline__ float pick32(const float (&x)[32], int i) {
    uint32_t r = 0;
#pragma unroll
    for (int e = 0; e < 32; ++e) {
        uint32_t same;
        asm("{\n.reg .pred p;\nsetp.eq.s32 p, %1, %2;\nselp.b32 %0, 0xFFFFFFFF, 0, p;\n}\n" : "=r"(same) : "r"(e), "r"(i));
        r |= __float_as_uint(x[e]) & same;
    }
    return __uint_as_float(r);
}
__device__ __forceinline__ float mask01(int e, int i) {
    float f;
    asm("{\n.reg .pred p;\nsetp.eq.s32 p, %1, %2;\nselp.f32 %0, 0f3F800000, 0f00000000, p;\n}\n" : "=f"(f) : "r"(e), "r"(i));
    return f;
}

// 64 columns of this thread's row
__device__ __forceinline__ void tmem_ld_64(uint32_t taddr, uint32_t (&r)[64]) {
    tmem_ld_32x32b_x32(taddr, *reinterpret_cast<uint32_t(*)[32]>(r));
    tmem_ld_32x32b_x32(taddr + 32, *reinterpret_cast<uint32_t(*)[32]>(r + 32));
    tmem_wait_ld();
}
// A box of 32 rows of 128 bytes of a warp's own, one row a lane, staged under the 128-byte swizzle.
__device__ __forceinline__ void stage16(uint8_t* out, int lane, int chunk, uint4 v) {
    *reinterpret_cast<uint4*>(out + lane * 128 + ((chunk ^ (lane & 7)) << 4)) = v;
}

// The logits of half of this thread's row: a tile's sums as they come out of tensor memory, `segment` of
// its n steps at once, added up.  Where `wanted` is not set they are waited for and let go of
// all the same.  False: a wait has run out.
__device__ __forceinline__ bool take_logits(uint64_t (&x)[kHalf / 2], int n, int segment, bool wanted, uint32_t& tile,
                                            uint32_t taddr, uint32_t tfull0, uint32_t empty_bar, const volatile int* abort) {
    for (int k0 = 0; k0 < n; k0 += segment, ++tile) {
        const uint32_t buf = tile & 1, use = (tile >> 1) & 1;
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(tfull0 + 8 * buf, use, abort, kWaitLimitNs))) return false;
        tc_fence_after();
        // 32 columns at a time: tensor memory serves these loads at the expense of
        // the products' sums, and four at once cost 4096 rows 2% (2544 -> 2614 us)
        if (wanted) {
#pragma unroll
            for (int j = 0; j < kHalf; j += 32) {
                uint32_t r[32];
                tmem_ld_32x32b_x32(taddr + buf * kTile + j, r);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const uint64_t v = f32x2_pack(r[2 * e], r[2 * e + 1]);
                    x[j / 2 + e] = k0 == 0 ? v : add2(x[j / 2 + e], v);
                }
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane_id() == 0) pair_arrive(empty_bar + 8 * buf);
    }
    return true;
}

template <Mode kMode>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Config<kMode>::kThreads, 1)
logp_pair_kernel(const __grid_constant__ Maps maps, const __grid_constant__ LogpParams p) {
    using C = Config<kMode>;
    constexpr int kStages = C::kStages;
    constexpr bool kForward = C::kForward;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBarOffset);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kStages + 4);
    volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + kStages);
    const uint32_t tfull0 = smem_u32(bars + 2 * kStages), tempty0 = smem_u32(bars + 2 * kStages + 2);
    const uint32_t warp = warp_id(), lane = lane_id(), rank = cluster_ctarank();
    auto gave_up = [&](uint32_t site) {
        atomicCAS(p.err, 0u, kKernelLogp << 24 | site << 16 | 1u);
        *abort = 1;
    };

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull0 + 8 * b, 1);
            mbar_init(tempty0 + 8 * b, 2 * C::kEpiWarps);
        }
        *abort = 0;
        fence_mbar_init();
        if (kMode != kBack) {
            prefetch_tmap(&maps.h);
            prefetch_tmap(&maps.h64);
            prefetch_tmap(&maps.w);
            if (kMode == kGrad) prefetch_tmap(&maps.d_out);
        } else {
            prefetch_tmap(&maps.d);
            prefetch_tmap(&maps.d64);
            prefetch_tmap(&maps.w_mn);
            prefetch_tmap(&maps.acc);
            prefetch_tmap(&maps.d_mn);
            prefetch_tmap(&maps.h_mn);
            prefetch_tmap(&maps.dw);
        }
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(2 * kTile)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();                                  // both CTAs' barriers are there
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // W's part of the first tile into L2 while the kernel before ends, by where it is if
    // enough rows count (elsewhere nobody is harmed)
    if (kMode != kBack && warp == 3 && lane == 0) {
        const int rows = (int)((p.M + kTile - 1) / kTile), pair = blockIdx.x >> 1;
        if (pair < rows * p.tiles) {
            int r, c;
            const int groups = (rows + p.group - 1) / p.group;
            tile_of(pair, rows, p.tiles, (rows + groups - 1) / groups, r, c);
            for (int k = 0; k < min(p.ksteps, 16); ++k)
                tma_prefetch_l2_2d(&maps.w, k * kStep, p.first + c * kTile + (int)rank * kHalf);
        }
    }
    grid_dependency_wait();
    grid_launch_dependents();

    Work<kMode> work(p);
    Unit u;
    if (kMode != kBack && warp < 4) regs_dec<kOtherRegs>();
    if ((warp == 0 || warp == 3) && lane == 0) {
        // ---------------- loads: this CTA's rows of the first operand, and by another warp
        // of the second (an issued copy takes its thread some 100 cycles and the wait before
        // it 200; one thread with four copies a stage took 600 where the products take 512)
        const bool first = warp == 0;
        // W is read by a group's row tiles at about the same time and may go then, except that
        // kGrad's drift apart (2048 rows of 65536 x 3584 read 0.73 to 1.2 GB where W has 0.47;
        // 0.48 without the hint, and the gradients of 1531 rows and more 0.2 to 0.5% faster; the
        // forward reads 0.48 with it and is 1% faster, two row tiles in kGrad up to 4%)
        const uint64_t policy = first || kMode == kBack ? policy_evict_last()
                                : kMode == kGrad && work.rows > 2 ? policy_evict_normal() : policy_evict_first();
        const uint32_t bar0 = map_to_rank(full0, 0);
        Ring<kStages> ring;
        uint32_t it = 0;
        while (!*abort && work.next(u)) {
            const int a = u.a + (int)rank * kHalf, b = u.b + (int)rank * kHalf;
            // Rows past those that count: 64 of them at once are left as they are in shared
            // memory; whatever that makes of their products reaches no other row, and nobody
            // reads theirs.
            const bool by_row = kMode != kBack || u.kind == 1;
            const int pieces = by_row ? min(2, max(0, (work.live - a + 63) / 64)) : 2;
            const int other = by_row ? min(2, max(0, (work.live - a - kHalf + 63) / 64)) : 2;
            const uint32_t bytes = (uint32_t)(4 + pieces + other) * kPiece;
            for (int k = 0; k < u.n; ++k, ++it) {
                if (!ring.wait(empty0, 1, abort)) {
                    gave_up(1);
                    break;
                }
                const uint32_t s = ring.s, dst = smem_u32(smem + s * C::kStageBytes), bar = bar0 + 8 * s;
                const int at = (u.k + k) * kStep;
                ring.next();
                ring.look(empty0, 1);
                if (first) {
                    if (rank == 0) mbar_arrive_expect_tx(full0 + 8 * s, bytes);
                    if (!by_row) pair_load_mn(dst, &maps.d_mn, bar, a / 64, at, policy);
                    else if (pieces == 2) pair_load(dst, kMode != kBack ? &maps.h : &maps.d, bar, at, a, policy);
                    else if (pieces == 1) pair_load(dst, kMode != kBack ? &maps.h64 : &maps.d64, bar, at, a, policy);
                } else if (kMode != kBack) {
                    pair_load(dst + 2 * kPiece, &maps.w, bar, at, p.first + b, policy);
                } else if (u.kind == 2) {
                    pair_load_mn(dst + 2 * kPiece, &maps.h_mn, bar, b / 64, at, policy);
                } else if (p.whole) {
                    pair_load_mn(dst + 2 * kPiece, &maps.w_mn, bar, b / 64, p.first + at, policy);
                } else {
                    pair_load(dst + 2 * kPiece, &maps.w_mn, bar, b, p.first + at, policy);
                    pair_load(dst + 3 * kPiece, &maps.w_mn, bar, b + 64, p.first + at, policy);
                }
            }
        }
        if (*abort && first && rank == 0)                // both CTAs' copies in flight land before either ends
            for (uint32_t j = it > (uint32_t)kStages ? it - kStages : 0; j < it; ++j)
                mbar_drain(full0 + 8 * (j % kStages), (j / kStages) & 1, kWaitLimitNs);
    } else if (warp == 1 && lane == 0 && rank == 0) {
        // ---------------- products, for both CTAs
        // Tiles, or with kLogp and kGrad parts of one, take the two halves of tensor memory in turn.  With
        // kBack a tile's first part stays in its half, and the others come into the other one,
        // from where the threads add them to it.
        Ring<kStages> ring;
        uint32_t tile = 0, used = 0;                     // used: of either half, the phase of its barriers
        const uint32_t stages = smem_u32(smem);
        while (!*abort && work.next(u)) {
            const bool a_mn = kMode == kBack && u.kind == 2, b_mn = kMode == kBack;
            const uint32_t idesc = kIdesc | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u);
            const uint32_t a_step = a_mn ? 2048 >> 4 : 32 >> 4, b_step = b_mn ? 2048 >> 4 : 32 >> 4;
            const uint64_t a0 = a_mn ? desc_mn(stages) : umma_desc_k128_sw128(stages);
            const uint64_t b0 = b_mn ? desc_mn(stages + 2 * kPiece) : umma_desc_k128_sw128(stages + 2 * kPiece);
            const int segment = kMode != kBack ? p.segment : kBackSegment;
            for (int k0 = 0; k0 < u.n && !*abort; k0 += segment) {
                const uint32_t buf = (tile ^ (kMode == kBack && k0 > 0)) & 1, use = used >> buf & 1;
                used ^= 1u << buf;
                if (kMode != kBack) ++tile;
                if (!mbar_wait_bounded(tempty0 + 8 * buf, use ^ 1, abort, kWaitLimitNs)) {
                    gave_up(3);
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem + buf * kTile;
                const int end = min(u.n, k0 + segment);
                for (int k = k0; k < end; ++k) {
                    if (!ring.wait(full0, 0, abort)) {
                        gave_up(2);
                        break;
                    }
                    tc_fence_after();
                    const uint32_t s = ring.s;
                    const uint64_t ad = a0 + s * (C::kStageBytes >> 4), bd = b0 + s * (C::kStageBytes >> 4);
                    ring.next();
                    ring.look(full0, 0);
                    pair_mma(d, ad, bd, idesc, k > k0);
#pragma unroll
                    for (int j = 1; j < 4; ++j) pair_mma(d, ad + j * a_step, bd + j * b_step, idesc, 1);
                    pair_commit(empty0 + 8 * s);
                }
                pair_commit(tfull0 + 8 * buf);
            }
            if (kMode == kBack && u.n > 0) ++tile;
        }
    } else if (kForward && warp >= 4) {
        // ---------------- the tile's threads' part: half of a row a thread
        if constexpr (kForward) {
            regs_inc<kEpiRegs>();
            const int q = warp & 3, half = (int)(warp - 4) >> 2, row = 32 * q + (int)lane;
            const uint32_t empty_bar = map_to_rank(tempty0, 0);
            const float c = p.scale * kLog2e;
            const int64_t size = (int64_t)p.parts * p.rows_pad;
            const uint32_t taddr = tmem + ((uint32_t)(32 * q) << 16) + half * kHalf;
            uint32_t tile = 0;
            while (work.next(u)) {
                const int m = u.a + (int)rank * kHalf + row;             // the row among those that count
                const int t = p.row_target[m] - u.b - half * kHalf, cols = (int)p.V - u.b - half * kHalf;
                uint64_t x[kHalf / 2];
                if (!take_logits(x, u.n, p.segment, true, tile, taddr, tfull0, empty_bar, abort)) {
                    if (lane == 0) gave_up(4);
                    break;
                }
                Sums s;
                if (cols > 0) {
                    if (p.entropy) sums_of<kHalf, true>(s, x, cols, c);
                    else sums_of<kHalf, false>(s, x, cols, c);
                    if (t >= 0 && t < kHalf) p.picked[m] = pick<kHalf>(x, t);
                }
                float* part = p.part + (int64_t)(2 * u.slot + half) * p.rows_pad + m;
                part[0] = s.top, part[size] = s.sum;
                if (p.entropy) part[2 * size] = s.dev;
            }
        }
    } else if (kMode == kGrad && warp >= 4) {
        // ---------------- the tile's threads' part: half of a row a thread
        if constexpr (kMode == kGrad) {
            regs_inc<kEpiRegs>();
            const int q = warp & 3, half = (int)(warp - 4) >> 2, row = 32 * q + (int)lane;
            uint8_t* const out = smem + C::kOutOffset + (warp - 4) * C::kOuts * kOutBytes;
            const uint32_t empty_bar = map_to_rank(tempty0, 0), taddr = tmem + ((uint32_t)(32 * q) << 16) + half * kHalf;
            const float c = p.scale * kLog2e;
            const bool entropy = p.ge != nullptr;
            uint32_t tile = 0;
            while (work.next(u)) {
                const int y = u.a + (int)rank * kHalf + 32 * q, x0 = u.b + half * kHalf;   // the warp's first row and column
                const int m = y + (int)lane;                             // the row among those that count
                const int t = p.row_target[m] - p.first - x0;
                const float g = p.row_g[m], ge = p.row_ge[m], l2 = p.row_lse[m] * kLog2e, plus = p.row_entropy[m];
                // words of this half; none for a row past those that count (0 times what its
                // logits come to would be NaN where W holds infinities)
                const int cols = m >= work.live ? 0 : (int)min((int64_t)kTile, p.V - p.first - u.b) - half * kHalf;
                // rows that nobody reads: past the last 64 of those that count
                const bool wanted = y < (work.live + 63) / 64 * 64;
                uint64_t x[kHalf / 2];
                if (!take_logits(x, u.n, p.segment, wanted, tile, taddr, tfull0, empty_bar, abort)) {
                    if (lane == 0) gave_up(4);
                    break;
                }
                if (!wanted) continue;
                const uint64_t cc = pk2(c, c), low = pk2(-l2, -l2), ng = pk2(-g, -g), ng2 = pk2(-ge, -ge);
                const uint64_t ln2 = pk2(0.69314718f, 0.69314718f), pl = pk2(plus, plus);
#pragma unroll
                for (int j = 0; j < kHalf; j += 64) {
                    float v[64];
                    uint32_t packed[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const uint64_t a = fma2(x[j / 2 + e], cc, low), pr = ex2_2(a);
                        uint64_t d = mul2(ng, pr);
                        if (entropy) {
                            // log p times a p of 0 is 0 where the logit is -inf too (a NaN is in d already)
                            const float2 l = f32x2_unpack(a);
                            d = fma2(mul2(ng2, pr), fma2(pk2(fmaxf(l.x, -1e30f), fmaxf(l.y, -1e30f)), ln2, pl), d);
                        }
                        const float2 two = f32x2_unpack(d);
                        v[2 * e] = two.x, v[2 * e + 1] = two.y;
                    }
                    if (t >= j && t < j + 64) {
#pragma unroll
                        for (int e = 0; e < 64; ++e) v[e] = fmaf(g, mask01(e, t - j), v[e]);
                    }
                    if (cols < j + 64) {
#pragma unroll
                        for (int e = 0; e < 64; ++e)
                            if (j + e >= cols) v[e] = 0.f;
                    }
#pragma unroll
                    for (int e = 0; e < 32; ++e) packed[e] = pack2(v[2 * e], v[2 * e + 1]);
                    // the staging box, once the copy engine has read what was in it
                    if (lane == 0) bulk_wait_read_all();
                    __syncwarp();
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        stage16(out, lane, e, make_uint4(packed[4 * e], packed[4 * e + 1], packed[4 * e + 2], packed[4 * e + 3]));
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_2d(&maps.d_out, smem_u32(out), x0 + j, y);
                        bulk_commit();
                    }
                }
            }
            if (lane == 0) bulk_wait_all();
            __syncwarp();
        }
    } else if (kMode == kBack && warp >= 4) {
        // ---------------- the tile's threads' part: half of a row a thread
        const int q = warp & 3, half = (int)(warp - 4) >> 2;
        uint8_t* const out = smem + C::kOutOffset + (warp - 4) * C::kOuts * kOutBytes;
        const uint32_t empty_bar = map_to_rank(tempty0, 0);
        const float f = kMode == kBack ? *p.largest * p.scale : 0.f;
        uint32_t tile = 0, used = 0;
        bool ok = true;
        while (work.next(u)) {
            const uint32_t buf = tile & 1;
            const uint32_t taddr = tmem + ((uint32_t)(32 * q) << 16) + buf * kTile + half * kHalf;
            if (u.n > 0) ++tile;
            else if (u.kind == 1) continue;
            auto release = [&](uint32_t b) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) pair_arrive(empty_bar + 8 * b);
            };
            for (int k0 = 0; k0 < u.n; k0 += kBackSegment) {
                const uint32_t b = (buf ^ (k0 > 0)) & 1, use = used >> b & 1;
                used ^= 1u << b;
                ok = __all_sync(0xffffffffu, mbar_wait_bounded(tfull0 + 8 * b, use, abort, kWaitLimitNs));
                if (!ok) break;
                tc_fence_after();
                if (k0 == 0) continue;
#pragma unroll 1
                for (int j = 0; j < kHalf; j += 32) {
                    uint32_t sum[32], more[32];
                    tmem_ld_32x32b_x32(taddr + j, sum);
                    tmem_ld_32x32b_x32(tmem + ((uint32_t)(32 * q) << 16) + b * kTile + half * kHalf + j, more);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e) sum[e] = __float_as_uint(__uint_as_float(sum[e]) + __uint_as_float(more[e]));
                    tmem_st_32x32b_x32(taddr + j, sum);
                }
                tmem_wait_st();
                release(b);
            }
            if (!ok) {
                if (lane == 0) gave_up(4);
                break;
            }
            // the staging box, once the copy engine has read what was in it
            auto clear = [&]() {
                if (lane == 0) bulk_wait_read_all();
                __syncwarp();
            };
            const int y = u.a + (int)rank * kHalf + 32 * q, x = u.b + half * kHalf;   // the warp's first row and column
            if (u.kind == 1 && y >= work.live) {             // rows that nobody reads: past those that count
                release(buf);
                continue;
            }
            // 64 columns from tensor memory, which is let go of after the last of them
            auto take = [&](int j, uint32_t (&r)[64]) {
                if (u.n > 0) {
                    tmem_ld_64(taddr + j, r);
                    if (j + 64 == kHalf) release(buf);
                } else {
#pragma unroll
                    for (int e = 0; e < 64; ++e) r[e] = 0;
                }
            };
            if (u.kind == 1) {
#pragma unroll 1
                for (int j = 0; j < kHalf; j += 64) {
                    uint32_t r[64];
                    take(j, r);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        clear();
#pragma unroll
                        for (int e = 8 * h; e < 8 * h + 8; ++e)
                            stage16(out, lane, e & 7, make_uint4(r[4 * e], r[4 * e + 1], r[4 * e + 2], r[4 * e + 3]));
                        fence_proxy_async_smem();
                        __syncwarp();
                        const int at = x + j + 32 * h, to = u.slot * p.rows_pad + y;
                        if (lane == 0 && at < p.K) {
                            if (p.first == 0) tma_store_2d(&maps.acc, smem_u32(out), at, to);
                            else tma_add_2d(&maps.acc, smem_u32(out), at, to);
                            bulk_commit();
                        }
                    }
                }
                continue;
            }
#pragma unroll 1
            for (int j = 0; j < kHalf; j += 64) {
                uint32_t r[64], packed[32];
                take(j, r);
#pragma unroll
                for (int e = 0; e < 32; ++e) packed[e] = pack2(__uint_as_float(r[2 * e]) * f, __uint_as_float(r[2 * e + 1]) * f);
                clear();
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    stage16(out, lane, e, make_uint4(packed[4 * e], packed[4 * e + 1], packed[4 * e + 2], packed[4 * e + 3]));
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if (x + j < p.K && p.first + y < p.V) tma_store_2d(&maps.dw, smem_u32(out), x + j, p.first + y);
                    bulk_commit();
                }
            }
        }
        if (lane == 0) bulk_wait_all();
        __syncwarp();
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();                                  // neither CTA's memory is in use any more
    if (warp == 2) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * kTile) : "memory");
    }
}

// ------------------------------------------------------------------ few rows

// Up to 128 rows: a pass over W that HBM bounds, so the roles change: W's rows are the
// products' 256, 128 a CTA, the rows that count their 64 or 128 columns, and nearly all of
// shared memory holds W on its way (11 stages of 16 KB of it, 9 with 128 columns; with rows
// on the other side it was 6, every product was made for 256 rows, and 48 rows of
// 152064 x 5120 took 272 us, 228 here).  A thread has a word of the vocabulary and 32 columns at a time; a
// column's maximum and sums over a warp's 32 words meet by exchanges that halve the
// columns at each step, so that lane l ends up with column l, whose sums it keeps over
// all of its warp's tiles.  Columns do not meet, so H is read as it lies, rows that do not
// count (and what they hold) among the others: nothing is brought together first.
template <int kN>
struct FewConfig {
    static constexpr int kRows = kN / 2;                                  // of H, a CTA's
    static constexpr int kStageBytes = kHalf * 128 + kRows * 128, kStages = kN == 64 ? 11 : 9;
    static constexpr int kGroups = kN / 64;                               // of 32 columns, a warp's
    static constexpr int kThreads = 32 * 12, kBarOffset = kStages * kStageBytes, kSmemBytes = kBarOffset + 256 + 1024;
    static constexpr uint32_t kIdesc = 1u << 4 | 1u << 7 | 1u << 10 | (uint32_t)(kN >> 3) << 17 | (uint32_t)(kTile >> 4) << 24;
    static constexpr uint32_t kCols = 2 * kN;
    static_assert(kSmemBytes <= 232448 && kStageBytes % 1024 == 0, "shared memory per CTA");
};

// r[j] of every lane to op over the lanes of r[l] in lane l
template <typename F>
__device__ __forceinline__ float across(float (&r)[32], int lane, F op) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const bool upper = lane & o;
#pragma unroll
        for (int j = 0; j < o; ++j) {
            const float keep = upper ? r[j + o] : r[j], send = upper ? r[j] : r[j + o];
            r[j] = op(keep, __shfl_xor_sync(0xffffffffu, send, o));
        }
    }
    return r[0];
}

template <int kN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(FewConfig<kN>::kThreads, 1)
logp_few_kernel(const __grid_constant__ Maps maps, const __grid_constant__ LogpParams p) {
    using C = FewConfig<kN>;
    constexpr int kStages = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBarOffset);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kStages + 4);
    volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + kStages);
    const uint32_t tfull0 = smem_u32(bars + 2 * kStages), tempty0 = smem_u32(bars + 2 * kStages + 2);
    const uint32_t warp = warp_id(), lane = lane_id(), rank = cluster_ctarank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    auto gave_up = [&](uint32_t site) {
        atomicCAS(p.err, 0u, kKernelLogp << 24 | site << 16 | 1u);
        *abort = 1;
    };
    if (warp == 0 && lane == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull0 + 8 * b, 1);
            mbar_init(tempty0 + 8 * b, 2 * 8);
        }
        *abort = 0;
        fence_mbar_init();
        prefetch_tmap(&maps.h);
        prefetch_tmap(&maps.w);
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(C::kCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    grid_dependency_wait();
    grid_launch_dependents();
    if (warp == 0 && lane == 0) {
        // ---------------- loads
        const uint64_t keep = policy_evict_last(), once = policy_evict_first();
        const uint32_t bar0 = map_to_rank(full0, 0);
        const uint32_t total = pair < p.tiles ? (uint32_t)((p.tiles - pair + pairs - 1) / pairs) * p.ksteps : 0;
        // (H in boxes of few_box rows; where there are none shared memory is left as it is)
        const uint32_t bytes = 4 * kPiece + (uint32_t)(p.few_box * 128) * (p.M > C::kRows ? 2 : 1);
        int step = 0, tile = pair;
        uint32_t it = 0;
        Ring<kStages> ring;
        for (; it < total && !*abort; ++it) {
            if (!ring.wait(empty0, 1, abort)) {
                gave_up(1);
                break;
            }
            const uint32_t s = ring.s, dst = smem_u32(smem + s * C::kStageBytes), bar = bar0 + 8 * s;
            ring.next();
            ring.look(empty0, 1);
            if (rank == 0) mbar_arrive_expect_tx(full0 + 8 * s, bytes);
            pair_load(dst, &maps.w, bar, step * kStep, tile * kTile + (int)rank * kHalf, once);
            if ((int)rank * C::kRows < p.M) pair_load(dst + 2 * kPiece, &maps.h, bar, step * kStep, (int)rank * C::kRows, keep);
            if (++step == p.ksteps) step = 0, tile += pairs;
        }
        if (*abort && rank == 0)
            for (uint32_t j = it > (uint32_t)kStages ? it - kStages : 0; j < it; ++j)
                mbar_drain(full0 + 8 * (j % kStages), (j / kStages) & 1, kWaitLimitNs);
    } else if (warp == 1 && lane == 0 && rank == 0) {
        Ring<kStages> ring;
        uint32_t tile = 0;
        const uint64_t a0 = umma_desc_k128_sw128(smem_u32(smem)), b0 = umma_desc_k128_sw128(smem_u32(smem) + 2 * kPiece);
        for (int v = pair; v < p.tiles && !*abort; v += pairs)
            for (int k0 = 0; k0 < p.ksteps && !*abort; k0 += p.segment, ++tile) {
                const uint32_t buf = tile & 1, use = (tile >> 1) & 1;
                if (!mbar_wait_bounded(tempty0 + 8 * buf, use ^ 1, abort, kWaitLimitNs)) {
                    gave_up(3);
                    break;
                }
                tc_fence_after();
                const int end = min(p.ksteps, k0 + p.segment);
                for (int k = k0; k < end; ++k) {
                    if (!ring.wait(full0, 0, abort)) {
                        gave_up(2);
                        break;
                    }
                    tc_fence_after();
                    const uint32_t s = ring.s;
                    const uint64_t a = a0 + s * (C::kStageBytes >> 4), b = b0 + s * (C::kStageBytes >> 4);
                    ring.next();
                    ring.look(full0, 0);
                    pair_mma(tmem + buf * kN, a, b, C::kIdesc, k > k0);
#pragma unroll
                    for (int j = 1; j < 4; ++j) pair_mma(tmem + buf * kN, a + 2 * j, b + 2 * j, C::kIdesc, 1);
                    pair_commit(empty0 + 8 * s);
                }
                pair_commit(tfull0 + 8 * buf);
            }
    } else if (warp >= 4) {
        const int q = warp & 3, half = (int)(warp - 4) >> 2;
        const uint32_t empty_bar = map_to_rank(tempty0, 0);
        const float c = p.scale * kLog2e;
        const bool dev = p.entropy != nullptr;
        constexpr float kNone = -3.0e38f;
        Sums s[C::kGroups];
        int target[C::kGroups];
#pragma unroll
        for (int g = 0; g < C::kGroups; ++g) {
            const int m = half * (kN / 2) + g * 32 + (int)lane;
            target[g] = m < p.M ? p.targets[m] : -1;
        }
        uint32_t tile = 0;
        bool ok = true;
        for (int v = pair; v < p.tiles && ok; v += pairs) {
            const int word0 = v * kTile + (int)rank * kHalf + 32 * q;
            const bool there = word0 + (int)lane < p.V;
            float x[C::kGroups][32];
            for (int k0 = 0; k0 < p.ksteps; k0 += p.segment, ++tile) {
                const uint32_t buf = tile & 1, use = (tile >> 1) & 1;
                if (!__all_sync(0xffffffffu, mbar_wait_bounded(tfull0 + 8 * buf, use, abort, kWaitLimitNs))) {
                    if (lane == 0) gave_up(4);
                    ok = false;
                    break;
                }
                tc_fence_after();
#pragma unroll
                for (int g = 0; g < C::kGroups; ++g) {
                    uint32_t r[32];
                    tmem_ld_32x32b_x32(tmem + ((uint32_t)(32 * q) << 16) + buf * kN + half * (kN / 2) + g * 32, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[g][e] = k0 == 0 ? __uint_as_float(r[e]) : x[g][e] + __uint_as_float(r[e]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) pair_arrive(empty_bar + 8 * buf);
            }
            if (!ok) break;
#pragma unroll
            for (int g = 0; g < C::kGroups; ++g) {
                float w[32];
                // a target among this warp's words: its logit to its row
                uint32_t hits = __ballot_sync(0xffffffffu, target[g] >= word0 && target[g] < word0 + 32);
                while (hits) {
                    const int j = __ffs((int)hits) - 1;
                    hits &= hits - 1;
                    const int owner = __shfl_sync(0xffffffffu, target[g], j) - word0;
                    if ((int)lane == owner) p.picked[half * (kN / 2) + g * 32 + j] = pick32(x[g], j);
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) w[e] = there ? x[g][e] : kNone;
                const float top = fmaxf(across(w, lane, [](float a, float b) { return fmaxf(a, b); }) * c, kNone);
                float d[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const float a = fmaf(x[g][e], c, -__shfl_sync(0xffffffffu, top, e));
                    w[e] = there ? ex2(a) : 0.f;
                    d[e] = w[e] > 0.f ? w[e] * a : 0.f;
                }
                const auto plus = [](float a, float b) { return a + b; };
                const float sum = across(w, lane, plus), weighted = dev ? across(d, lane, plus) : 0.f;
                if (word0 < p.V) s[g].add(top, sum, weighted);
            }
        }
        // this warp's part of its columns: one of 8 a pair
        const int64_t size = (int64_t)8 * pairs * p.rows_pad, at = (int64_t)(8 * pair + 4 * (int)rank + q) * p.rows_pad;
#pragma unroll
        for (int g = 0; g < C::kGroups; ++g) {
            float* part = p.part + at + half * (kN / 2) + g * 32 + lane;
            part[0] = s[g].top, part[size] = s[g].sum;
            if (dev) part[2 * size] = s[g].dev;
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    if (warp == 2) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kCols) : "memory");
    }
}

// ------------------------------------------------------------------ before and after the products

__device__ __forceinline__ bool counts(const LogpParams& p, int64_t m) { return p.targets[m] >= 0 && p.targets[m] < p.V; }

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// The rows that count, brought together: their hidden states, targets and gradients; zeros
// for the results of the others.  Every CTA goes over all targets (they are in L2) to find
// where its own rows go, so nothing is waited for.
static_assert(kLogpRows <= 1024 * 2048, "rows a CTA");
constexpr int kRowThreads = 256, kMostRows = 2048;

template <bool kBackward>
__global__ void __launch_bounds__(kRowThreads)
rows_kernel(const __grid_constant__ LogpParams p, int rows) {
    __shared__ int place[kMostRows], before_w[8], all_w[8];
    __shared__ float largest_w[8];
    pdl_wait_then_release();
    const int M = (int)p.M, m0 = blockIdx.x * rows, mine = min(rows, M - m0);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int before = 0, all = 0;
    float largest = 0.f;
    for (int r = warp; r < mine; r += kRowThreads / 32)      // this CTA's rows on their way to L2
        for (int i = lane * 64; i < p.K; i += 32 * 64) prefetch_l2(p.H + (m0 + r) * p.ldh + i);
    for (int m = threadIdx.x; m < M; m += kRowThreads) {
        const int t = p.targets[m];
        const float g = kBackward ? fabsf(p.g[m]) : 0.f, e = kBackward && p.ge ? fabsf(p.ge[m]) : 0.f;
        if (t >= 0 && t < p.V) {
            before += m < m0, ++all;
            if (fmaxf(g, e) < INFINITY) largest = fmaxf(largest, fmaxf(g, e));   // an infinite one is its row's alone
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        before += __shfl_xor_sync(0xffffffffu, before, o);
        all += __shfl_xor_sync(0xffffffffu, all, o);
        largest = fmaxf(largest, __shfl_xor_sync(0xffffffffu, largest, o));
    }
    if (lane == 0) before_w[warp] = before, all_w[warp] = all, largest_w[warp] = largest;
    __syncthreads();
    before = all = 0, largest = 0.f;
    for (int w = 0; w < 8; ++w) before += before_w[w], all += all_w[w], largest = fmaxf(largest, largest_w[w]);
    if (largest == 0.f) largest = 1.f;
    if (warp == 0)
        for (int r = 0; r < mine; r += 32) {
            const bool yes = r + lane < mine && counts(p, m0 + r + lane);
            const uint32_t those = __ballot_sync(0xffffffffu, yes);
            if (r + lane < mine) place[r + lane] = yes ? before + __popc(those & ((1u << lane) - 1)) : -1;
            before += __popc(those);
        }
    __syncthreads();
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        *p.live = all;
        if (kBackward) *p.largest = largest;
    }
    const int chunks = (int)(p.K / 8);
    for (int r = warp; r < mine; r += 8) {
        const int m = m0 + r, at = place[r];
        if (at < 0) {
            if (!kBackward) {
                if (lane == 0) {
                    p.logp[m] = 0.f, p.lse[m] = 0.f;
                    if (p.entropy) p.entropy[m] = 0.f;
                }
            } else if (p.dH) {
                uint4* d = reinterpret_cast<uint4*>(p.dH + (int64_t)m * p.K);
                for (int i = lane; i < chunks; i += 32) d[i] = make_uint4(0, 0, 0, 0);
            }
            continue;
        }
        if (lane == 0) {
            p.row_of[at] = m, p.row_target[at] = p.targets[m];
            if (kBackward) {
                p.row_g[at] = p.g[m] / largest, p.row_ge[at] = p.ge ? p.ge[m] / largest : 0.f;
                p.row_lse[at] = p.lse[m], p.row_entropy[at] = p.ge ? p.entropy[m] : 0.f;
            }
        }
        const uint4* src = reinterpret_cast<const uint4*>(p.H + m * p.ldh);
        uint4* dst = reinterpret_cast<uint4*>(p.rows_h + (int64_t)at * p.pitch);
        for (int i = lane; i < chunks; i += 32) dst[i] = ld_stream_v4(src + i);
        for (int i = chunks + lane; i < p.pitch / 8; i += 32) dst[i] = make_uint4(0, 0, 0, 0);
    }
    // up to the last tile's edge no target and no gradient; hidden states of zeros up to the
    // last 64 rows' end (past M the copy engine fills them in; further ones are not loaded)
    const int edge = (all + kTile - 1) / kTile * kTile, zeros = min(M, (all + 63) / 64 * 64);
    if (blockIdx.x == 0 && all + (int)threadIdx.x < edge) {
        const int at = all + threadIdx.x;
        p.row_target[at] = -1;
        if (kBackward) p.row_g[at] = 0.f, p.row_ge[at] = 0.f, p.row_lse[at] = 0.f, p.row_entropy[at] = 0.f;
    }
    for (int at = all + blockIdx.x; at < zeros; at += gridDim.x) {
        uint4* dst = reinterpret_cast<uint4*>(p.rows_h + (int64_t)at * p.pitch);
        for (int i = threadIdx.x; i < p.pitch / 8; i += kRowThreads) dst[i] = make_uint4(0, 0, 0, 0);
    }
}

// Joins a row's tiles: eight rows a CTA (a sector of each array), a 64th of the tiles a thread.
constexpr int kJoinThreads = 512, kJoinRows = 8;

template <bool kFew>
__global__ void __launch_bounds__(kJoinThreads)
logp_join_kernel(const __grid_constant__ LogpParams p) {
    __shared__ Sums part[kJoinThreads / 32][kJoinRows];
    pdl_wait_then_release();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = threadIdx.x % kJoinRows;
    const int live = kFew ? (int)p.M : *p.live, m = blockIdx.x * kJoinRows + r;
    if ((int)blockIdx.x * kJoinRows >= live) return;
    const int64_t size = (int64_t)p.parts * p.rows_pad;
    const bool dev = p.entropy != nullptr;
    Sums s;
    if (m < live) {
        constexpr int kStride = kJoinThreads / kJoinRows;
        for (int t = threadIdx.x / kJoinRows; t < p.parts; t += 4 * kStride) {
            float v[4][3];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const bool there = t + u * kStride < p.parts;
                const float* at = p.part + (int64_t)(t + u * kStride) * p.rows_pad + m;
                v[u][0] = there ? at[0] : -3.0e38f, v[u][1] = there ? at[size] : 0.f, v[u][2] = there && dev ? at[2 * size] : 0.f;
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) s.add(v[u][0], v[u][1], v[u][2]);
        }
    }
#pragma unroll
    for (int o = kJoinRows; o < 32; o *= 2)
        s.add(__shfl_xor_sync(0xffffffffu, s.top, o), __shfl_xor_sync(0xffffffffu, s.sum, o),
              __shfl_xor_sync(0xffffffffu, s.dev, o));
    if (lane < kJoinRows) part[warp][lane] = s;
    __syncthreads();
    if (threadIdx.x >= kJoinRows || m >= live) return;
    for (int w = 1; w < kJoinThreads / 32; ++w) s.add(part[w][r].top, part[w][r].sum, part[w][r].dev);
    const float ls = logf(s.sum);
    const double lse = (double)s.top * kLn2 + (double)ls;
    const int row = kFew ? m : p.row_of[m];
    if (kFew && !counts(p, m)) {
        p.logp[row] = 0.f, p.lse[row] = 0.f;
        if (dev) p.entropy[row] = 0.f;
        return;
    }
    p.logp[row] = (float)((double)p.scale * (double)p.picked[m] - lse);
    p.lse[row] = (float)lse;
    if (dev) p.entropy[row] = ls - (float)kLn2 * s.dev / s.sum;
}

// dH from its fp32 sums, a row a CTA
__global__ void __launch_bounds__(256)
grad_h_kernel(const __grid_constant__ LogpParams p) {
    pdl_wait_then_release();
    const int live = *p.live;
    const float f = *p.largest * p.scale;
    for (int m = blockIdx.x; m < live; m += gridDim.x) {
        uint2* dst = reinterpret_cast<uint2*>(p.dH + (int64_t)p.row_of[m] * p.K);
        for (int i = threadIdx.x; i < (int)(p.K / 4); i += 256) {
            const float* at = p.acc + (int64_t)m * p.K + 4 * i;
            const int64_t part = (int64_t)p.rows_pad * p.K;
            float4 v = *reinterpret_cast<const float4*>(at);
            for (int s = 1; s < p.split; s += 4) {           // four parts' loads in flight, added in their order
                float4 w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (s + j < p.split) w[j] = *reinterpret_cast<const float4*>(at + (s + j) * part);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (s + j < p.split) v.x += w[j].x, v.y += w[j].y, v.z += w[j].z, v.w += w[j].w;
            }
            dst[i] = make_uint2(pack2(v.x * f, v.y * f), pack2(v.z * f, v.w * f));
        }
    }
}

// ------------------------------------------------------------------ host

constexpr int64_t kFewRows = 128;

constexpr int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// A workspace's parts, 256 bytes apart.
struct Arena {
    uint8_t* base;
    size_t used = 0;
    template <typename T>
    T* take(int64_t n) {
        T* at = base ? reinterpret_cast<T*>(base + used) : nullptr;
        used += (size_t)up(n * (int64_t)sizeof(T), 256);
        return at;
    }
};

void lay_rows(Arena& a, LogpParams& p) {
    p.rows_pad = (int)up(p.M, kTile);
    p.live = a.take<int>(1), p.largest = a.take<float>(1);
    p.row_of = a.take<int>(p.rows_pad), p.row_target = a.take<int>(p.rows_pad);
    p.pitch = (int)up(p.K, kStep);
    p.rows_h = a.take<uint16_t>(p.M * p.pitch);
}
void lay_forward(Arena& a, LogpParams& p, int pairs) {
    p.tiles = (int)((p.V + kTile - 1) / kTile);
    if (p.M <= kFewRows) {
        p.rows_pad = kFewRows;
        p.parts = 8 * std::min(pairs, p.tiles);
    } else {
        lay_rows(a, p);
        p.parts = 2 * p.tiles;
    }
    p.picked = a.take<float>(p.rows_pad);
    p.part = a.take<float>(3 * (int64_t)p.parts * p.rows_pad);
}

// The backward's pieces of the vocabulary, and the parts of a piece that dH's tiles are cut
// into (summed apart).  Taken by what the pairs' longest share comes to, in steps: kGrad's
// tiles in waves, then dH's, alone (once) and with dW's (twice), which fill the gaps; 8 steps' time
// at a tile's ends, 40 a launch, a part's sums a fortieth.  The same whichever gradients are wanted, so
// that dH has the same bits.  D of a piece is at most kMostD bytes, a fifth of what 4096 rows
// of 152064 have: with 64 MB both gradients of those take 8.4 ms, with 128 8.2, 256 8.0, 512 7.9.
constexpr int64_t kMostD = 256ll << 20;

void plan(int64_t M, int64_t V, int64_t K, int pairs, int64_t& piece, int& split) {
    const int64_t rows = (M + kTile - 1) / kTile, kt = (K + kTile - 1) / kTile, words = (V + kTile - 1) / kTile;
    const int64_t most = std::max<int64_t>(kMostD / (2 * rows * kTile * kTile), 4), least = (words + most - 1) / most;
    const double ksteps = (double)((K + kStep - 1) / kStep), wsteps = std::max<double>(rows * kTile / kStep, kLeastSteps);
    double best = 1e30;
    for (int64_t n = least; n <= std::min(words, least + 8); ++n) {
        const int64_t w = (words + n - 1) / n, steps = w * kTile / kStep;
        const int64_t launches = (words + w - 1) / w;
        const double grad = (double)((rows * w + pairs - 1) / pairs) * (ksteps + 8);
        for (int s = 1; s <= 16 && s * 8 <= steps; ++s) {
            const double each = (double)steps / s + 8, turns = (double)((rows * kt * s + pairs - 1) / pairs);
            const double alone = turns * each;
            const double both = std::max(alone, ((double)(rows * kt * s) * each + (double)(w * kt) * (wsteps + 2)) / pairs + wsteps / 2);
            const double cost = (double)launches * (3 * grad + (alone + 2 * both) * (1 + 0.025 * s) + 240);
            if (cost < best) best = cost, piece = w * kTile, split = s;
        }
        if (steps < 8) {                                // a piece that is hardly one
            const double cost = (double)launches * 3 * (grad + (double)((rows * kt + pairs - 1) / pairs) * (steps + 8) + 80);
            if (cost < best) best = cost, piece = w * kTile, split = 1;
        }
    }
}
void lay_backward(Arena& a, LogpParams& p, int pairs) {
    lay_rows(a, p);
    p.row_g = a.take<float>(p.rows_pad), p.row_ge = a.take<float>(p.rows_pad);
    p.row_lse = a.take<float>(p.rows_pad), p.row_entropy = a.take<float>(p.rows_pad);
    plan(p.M, p.V, p.K, pairs, p.piece, p.split);
    p.D = a.take<uint16_t>((int64_t)p.rows_pad * p.piece);
    p.acc = a.take<float>((int64_t)p.split * p.rows_pad * p.K);
}

cudaError_t launch_clusters(void (*kernel)(Maps, LogpParams), int pairs, int threads, int smem, cudaStream_t st,
                            const Maps& maps, const LogpParams& p) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * pairs);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, maps, p);
}
template <Mode kMode>
cudaError_t launch_pairs(int pairs, cudaStream_t st, const Maps& maps, const LogpParams& p) {
    return launch_clusters(logp_pair_kernel<kMode>, pairs, Config<kMode>::kThreads, Config<kMode>::kSmemBytes, st, maps, p);
}
template <int kN>
cudaError_t launch_few(int pairs, cudaStream_t st, const Maps& maps, const LogpParams& p) {
    using C = FewConfig<kN>;
    return launch_clusters(logp_few_kernel<kN>, std::min(pairs, p.tiles), C::kThreads, C::kSmemBytes, st, maps, p);
}

int pairs_of(void (*kernel)(Maps, LogpParams), int threads, int smem, int regs) {
    cudaFuncAttributes fa;
    // a split of registers (regs > 0) is made for just that many a thread at launch: with
    // others the threads' part could wait for registers for ever
    if (cudaFuncGetAttributes(&fa, kernel) != cudaSuccess || (regs && up(fa.numRegs, 8) != regs) ||
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * 512);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2, at[0].val.clusterDim.y = 1, at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int n = 0;
    return cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess ? n : 0;
}
template <Mode kMode>
int pairs_of_tiles() {
    return pairs_of(logp_pair_kernel<kMode>, Config<kMode>::kThreads, Config<kMode>::kSmemBytes, kMode == kBack ? 0 : kLaunchRegs);
}
template <int kN>
int pairs_of_few() {
    return pairs_of(logp_few_kernel<kN>, FewConfig<kN>::kThreads, FewConfig<kN>::kSmemBytes, 0);
}
// Pairs of CTAs of one kind of call that run at once on the current device; 0: its kernels do
// not run there (which says nothing of the others').
enum Call { kFewCall, kForwardCall, kBackwardCall };
int pairs_here(Call call) {
    static std::atomic<int> known[3][64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    int n = known[call][dev].load(std::memory_order_relaxed);
    if (!n) {
        n = call == kFewCall ? std::min(pairs_of_few<64>(), pairs_of_few<128>())
            : call == kForwardCall ? pairs_of_tiles<kLogp>() : std::min(pairs_of_tiles<kGrad>(), pairs_of_tiles<kBack>());
        n = std::min(n, num_sms() / 2);
        known[call][dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

// 64 rows of two pieces of 64 values of a row-major bf16 matrix whose rows are whole pieces
bool load_map_mn(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int64_t pitch) {
    return make_tmap_bf16_pieces(m, base, (uint64_t)rows, (uint64_t)cols / 64, (uint64_t)pitch, 64, 2);
}
bool load_map(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int64_t pitch, uint32_t box_rows) {
    return make_tmap_bf16_load(m, base, (uint64_t)rows, (uint64_t)cols, (uint64_t)pitch, box_rows);
}

cudaError_t launch_rows(const LogpParams& p, bool backward, cudaStream_t st) {
    // rows a CTA: four up to a CTA an SM, then to sixteen; every CTA goes over all targets,
    // so not more than 1024 CTAs
    const int64_t even = (p.M + num_sms() - 1) / num_sms();
    const int rows = (int)std::max<int64_t>(std::min<int64_t>(std::max<int64_t>(even, 4), 16), (p.M + 1023) / 1024);
    const dim3 grid((unsigned)((p.M + rows - 1) / rows));
    return backward ? launch_pdl(rows_kernel<true>, grid, dim3(kRowThreads), 0, st, p, rows)
                    : launch_pdl(rows_kernel<false>, grid, dim3(kRowThreads), 0, st, p, rows);
}

// Row tiles whose hidden states take some 40 MB, a third of L2.
int group_of(int64_t K) { return (int)std::max<int64_t>(1, (40ll << 20) / (kTile * K * 2)); }

// Steps of the logits' products that are summed in tensor memory: the same in both directions,
// so that the backward's logits have the bits of those that lse came from.
int segment_of(const LogpParams& p) {
    const int most = p.M <= kFewRows ? kFewSegment : kSegment, segments = (p.ksteps + most - 1) / most;
    return (p.ksteps + segments - 1) / segments;
}

int pairs_or_default() {
    const int n = num_sms() / 2;
    return n > 0 ? n : 76;
}

}  // namespace

size_t linear_logp_workspace_bytes(int64_t M, int64_t V, int64_t K) {
    if (M <= 0 || V <= 0 || K <= 0 || M > kLogpRows || V > kLogpRows || K > kLogpK) return 0;
    LogpParams p{};
    p.M = M, p.V = V, p.K = K;
    Arena a{nullptr};
    lay_forward(a, p, pairs_or_default());
    return a.used;
}

size_t linear_logp_backward_workspace_bytes(int64_t M, int64_t V, int64_t K) {
    if (M <= 0 || V <= 0 || K <= 0 || M > kLogpRows || V > kLogpRows || K > kLogpK) return 0;
    LogpParams p{};
    p.M = M, p.V = V, p.K = K;
    Arena a{nullptr};
    lay_backward(a, p, pairs_or_default());
    return a.used;
}

cudaError_t launch_linear_logp(LogpParams p, void* ws, cudaStream_t st) {
    const bool few = p.M <= kFewRows;
    const int pairs = pairs_here(few ? kFewCall : kForwardCall);
    if (!pairs || pairs > pairs_or_default()) return cudaErrorInvalidDeviceFunction;
    Arena a{static_cast<uint8_t*>(ws)};
    lay_forward(a, p, pairs_or_default());
    p.err = device_error_word();
    p.ksteps = (int)((p.K + kStep - 1) / kStep), p.group = group_of(p.K);
    p.segment = segment_of(p);
    Maps maps{};
    if (!p.err || !load_map(&maps.w, p.W, p.V, p.K, p.ldw, kHalf)) return cudaErrorInvalidValue;
    if (few) {
        // (as many pairs as the parts are laid out for)
        const bool least = p.M <= 64;
        p.few_box = (int)std::min<int64_t>(least ? 32 : 64, up(p.M, 8));
        if (!load_map(&maps.h, p.H, p.M, p.K, p.ldh, (uint32_t)p.few_box)) return cudaErrorInvalidValue;
        p.parts = 8 * std::min(pairs, p.tiles);
        const cudaError_t e = least ? launch_few<64>(pairs, st, maps, p) : launch_few<128>(pairs, st, maps, p);
        if (e != cudaSuccess) return e;
        return launch_pdl(logp_join_kernel<true>, dim3((unsigned)((p.M + kJoinRows - 1) / kJoinRows)), dim3(kJoinThreads), 0, st, p);
    }
    if (!load_map(&maps.h, p.rows_h, p.M, p.pitch, p.pitch, kHalf) || !load_map(&maps.h64, p.rows_h, p.M, p.pitch, p.pitch, 64))
        return cudaErrorInvalidValue;
    cudaError_t e = launch_rows(p, false, st);
    if (e == cudaSuccess) e = launch_pairs<kLogp>(pairs, st, maps, p);
    if (e != cudaSuccess) return e;
    return launch_pdl(logp_join_kernel<false>, dim3((unsigned)((p.M + kJoinRows - 1) / kJoinRows)), dim3(kJoinThreads), 0, st, p);
}

cudaError_t launch_linear_logp_backward(LogpParams p, void* ws, cudaStream_t st) {
    if (p.M == 0) return p.dW ? cudaMemsetAsync(p.dW, 0, (size_t)(p.V * p.K) * 2, st) : cudaSuccess;
    const int pairs = pairs_here(kBackwardCall);
    if (!pairs) return cudaErrorInvalidDeviceFunction;
    Arena a{static_cast<uint8_t*>(ws)};
    lay_backward(a, p, pairs_or_default());
    p.err = device_error_word();
    p.ksteps = (int)((p.K + kStep - 1) / kStep), p.group = group_of(p.K);
    p.ktiles = (int)((p.K + kTile - 1) / kTile), p.segment = segment_of(p);
    Maps maps{};
    p.whole = p.K % 64 == 0;
    if (!p.err || !load_map(&maps.h, p.rows_h, p.M, p.pitch, p.pitch, kHalf) ||
        !load_map(&maps.h64, p.rows_h, p.M, p.pitch, p.pitch, 64) || !load_map_mn(&maps.h_mn, p.rows_h, p.M, p.pitch, p.pitch) ||
        !load_map(&maps.w, p.W, p.V, p.K, p.ldw, kHalf) ||
        !(p.whole ? load_map_mn(&maps.w_mn, p.W, p.V, p.K, p.ldw) : load_map(&maps.w_mn, p.W, p.V, p.K, p.ldw, 64)) ||
        !load_map(&maps.d, p.D, p.rows_pad, p.piece, p.piece, kHalf) || !load_map(&maps.d64, p.D, p.rows_pad, p.piece, p.piece, 64) ||
        !load_map_mn(&maps.d_mn, p.D, p.rows_pad, p.piece, p.piece) ||
        !make_tmap_bf16_store(&maps.d_out, p.D, (uint64_t)p.rows_pad, (uint64_t)p.piece, (uint64_t)p.piece, 64, 32) ||
        !make_tmap_f32_store(&maps.acc, p.acc, (uint64_t)p.split * p.rows_pad, (uint64_t)p.K, (uint64_t)p.K, 32, 32) ||
        (p.dW && !make_tmap_bf16_store(&maps.dw, p.dW, (uint64_t)p.V, (uint64_t)p.K, (uint64_t)p.K, 64, 32)))
        return cudaErrorInvalidValue;
    cudaError_t e = launch_rows(p, true, st);
    for (int64_t v = 0; v < p.V && e == cudaSuccess; v += p.piece) {
        const int64_t n = std::min(p.piece, p.V - v);
        p.first = (int)v, p.tiles = (int)((n + kTile - 1) / kTile), p.steps = (int)((n + kStep - 1) / kStep);
        e = launch_pairs<kGrad>(pairs, st, maps, p);
        if (e == cudaSuccess) e = launch_pairs<kBack>(pairs, st, maps, p);
    }
    if (!p.dH || e != cudaSuccess) return e;
    return launch_pdl(grad_h_kernel, dim3((unsigned)std::min<int64_t>(p.M, 8 * num_sms())), dim3(256), 0, st, p);
}

}  // namespace fp8rl
