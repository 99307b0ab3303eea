// attn_paged_wide.cuh -- attention over a paged bf16 cache for more query rows than
// mma.sync carries well: 33 and more a kv head (long drafts, trees of them, chunks of
// a prompt behind a cached prefix).  Mathematics, work split and workspace are those
// of attn_paged.cuh.
//
// What bounds it.  Each cached byte meets rows flop; 40 rows at HBM's speed are 0.3
// PFLOP/s, more than mma.sync makes here beside its matrix loads (64 rows at once, their
// sums spilled: 0.14).  tcgen05 has the rate, so the work is a stream again, and beyond
// that the threads' part: a tile of 128 tokens takes them 1.4 us with 40 rows, 2.0 with
// 80, where HBM takes 1.5.  32 sequences to 16384, 8 kv heads of 128, pages of 64, 1.1 GB:
// 40 rows in 186 us (5.9 TB/s; by mma.sync in chunks of 32 335), 80 in 211 (530), 120 in
// 294 (707).  Prompt chunks of 512 behind up to 3488 tokens, 8 sequences, 28/4 heads: 420
// us, 0.29 PFLOP/s (1534), every chunk of rows over all of its sequence's tiles.  Pages of
// 16 tokens are eight boxes a tile instead of two: 40 rows 238 us, 80 rows 260.
//
// Products.  Tokens, then head values are the M side, the rows the N side:
//   S^T [128 tokens x rows] = K Q^T      K and Q with the head inside (K-major),
//   O^T [head x rows] += V^T P^T         V and P with the head and rows inside (MN-major),
// so K and V are operands as the copy engine lays them, 64 values of 128 tokens a piece
// under the 128-byte swizzle, and nothing is transposed.  Scores and sums are in tensor
// memory, fp32.  Two threads share a token's scores, every other eight rows
// each: exponentials, their token's part of the rows' sums, and 16-byte pieces of P
// (bf16, one rounding: the reference is the running one of attn_paged.cuh,
// moved rarely, and then the sums in tensor memory are scaled).
//
// A warp loads, one issues the products: a tile's scores while the tile before is in
// the exponentials, and where two buffers of probabilities fit, the exponentials while
// the product before sums.  The last tile of an item lets go of the queries' buffer, so the
// next item's first scores are under way while this one's result is written.
#pragma once

#include "attn_paged.cuh"

namespace fp8rl {
namespace attn {
namespace {

template <int DP_, int RT_>
struct WideConfig {
    static constexpr bool kE4m3 = false, kTma = true;
    static constexpr int DP = DP_, RT = RT_, ES = 2, RB = DP * ES, PB = 128, CT = 128;
    static constexpr int kTile = CT * RB, kCtas = 1;
    static constexpr int kPiece = CT * 128;                  // 64 values of a tile's tokens
    static constexpr int kPart = (RT + 63) / 64 * kPiece, kBufs = DP == 128 && RT == 128 ? 1 : 2, kP = kBufs * kPart;   // probabilities
    static constexpr int kQ = DP / 64 * RT * 128;
    static constexpr int kSmall = RT * 4 * 9 + 28 * 8 + 16;
    // a tile of keys or of values a slot, let go of by its own product
    static constexpr int kFit = (232448 - kP - kQ - kSmall) / kTile, kSlots = kFit < 8 ? kFit : 8;
    static constexpr int kSmem = kSlots * kTile + kP + kQ + kSmall;
    // An item's start and end, in tiles: 100 sequences to 1500, 40 rows, heads of 128:
    // 105 us with two, 92 with four, 96 with six; prompt chunks of 512: 528, 466, 420.
    static constexpr int kItem = 6;
    static constexpr int kUnits = RT / 16;                   // eights of rows a thread, kept or taken four at a time
    static constexpr int kGroup = kUnits <= 6 ? kUnits : 4;
    static constexpr uint32_t kSlice = RT <= 64 ? 64 : 128, kCols = 4 * kSlice;   // two tiles' scores, the sums, what is set apart
    static_assert(kSlots >= 4 && RT % 16 == 0 && RT <= 128 && kUnits % kGroup == 0 && (DP == 64 || DP == 128), "");
};

constexpr int kWideWarps = 8, kWideThreads = kWideWarps * 32 + 64;   // and one that loads, one that multiplies

// An MN-major operand of pieces of 64 values (rows of the K side 128 bytes apart, in
// eights; the next 64 values a piece on).
__device__ __forceinline__ uint64_t wide_desc_mn(uint32_t addr, uint32_t piece) {
    return (uint64_t)((addr >> 4) & 0x3FFFu) | (uint64_t)(piece >> 4) << 16 | (uint64_t)(1024u >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void st_shared16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ void tmem_ld_x8(uint32_t taddr, float* r) {
    uint32_t v[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = __uint_as_float(v[i]);
}
__device__ __forceinline__ void tmem_st_x8(uint32_t taddr, const float* r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
                 "r"(__float_as_uint(r[0])), "r"(__float_as_uint(r[1])), "r"(__float_as_uint(r[2])),
                 "r"(__float_as_uint(r[3])), "r"(__float_as_uint(r[4])), "r"(__float_as_uint(r[5])),
                 "r"(__float_as_uint(r[6])), "r"(__float_as_uint(r[7]))
                 : "memory");
}
// Eight values of each lane joined over the warp: lane l gets value (l >> 2)'s.
template <class Op>
__device__ __forceinline__ float join8(const float* x, Op op) {
    const int lane = threadIdx.x & 31;
    float a[4], b[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool up = lane & 16;
        a[i] = op(up ? x[i + 4] : x[i], __shfl_xor_sync(0xffffffffu, up ? x[i] : x[i + 4], 16));
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const bool up = lane & 8;
        b[i] = op(up ? a[i + 2] : a[i], __shfl_xor_sync(0xffffffffu, up ? a[i] : a[i + 2], 8));
    }
    const bool up = lane & 4;
    float c = op(up ? b[1] : b[0], __shfl_xor_sync(0xffffffffu, up ? b[0] : b[1], 4));
    c = op(c, __shfl_xor_sync(0xffffffffu, c, 2));
    return op(c, __shfl_xor_sync(0xffffffffu, c, 1));
}

template <class C>
__global__ void __launch_bounds__(kWideThreads, 1)
attn_paged_wide_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap) {
    extern __shared__ __align__(1024) uint8_t smem[];
    constexpr int RT = C::RT, CT = C::CT, S = C::kSlots, DP = C::DP, U = C::kUnits, kN = kWideWarps * 32;
    const uint32_t ring = sm100::smem_u32(smem), sp = ring + S * C::kTile, sq = sp + C::kP;
    int* const s_hi = reinterpret_cast<int*>(smem + S * C::kTile + C::kP + C::kQ);   // [RT] tokens lo .. hi - 1 are seen
    int* const s_lo = s_hi + RT;
    int* const s_row = s_lo + RT;                             // [RT] the row's place in its sequence's output
    float* const s_ref = reinterpret_cast<float*>(s_row + RT);   // [RT] running reference
    float* const s_fac = s_ref + RT;                          // [RT] a rescale's or the result's factor
    float* const s_w = s_fac + RT;                            // [quarter of the tokens][RT] maxima, sums
    const uint32_t bars = sm100::smem_u32(s_w + 4 * RT);
    const uint32_t full = bars, empty = full + 8 * S, s_full = empty + 8 * S, s_free = s_full + 16, p_full = s_free + 16,
                   pv = p_full + 16, q_full = pv + 16, drained = q_full + 8;
    volatile int* const abort = reinterpret_cast<int*>(s_w + 4 * RT) + 56;
    volatile uint32_t* const s_tmem = reinterpret_cast<uint32_t*>(s_w + 4 * RT) + 57;

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int group = p.Hq / p.Hkv, rows = group * p.Lq, chunks = (rows + RT - 1) / RT, hr_n = p.Hkv * chunks;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            sm100::mbar_init(full + 8 * i, 1);
            sm100::mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            sm100::mbar_init(s_full + 8 * i, 1);
            sm100::mbar_init(s_free + 8 * i, kWideWarps);
            sm100::mbar_init(p_full + 8 * i, kWideWarps);
            sm100::mbar_init(pv + 8 * i, 1);
        }
        sm100::mbar_init(q_full, kWideWarps);
        sm100::mbar_init(drained, 1);
        *abort = 0;
        sm100::fence_mbar_init();
        sm100::prefetch_tmap(&kmap);
        sm100::prefetch_tmap(&vmap);
    }
    if (threadIdx.x < RT) s_ref[threadIdx.x] = kNone;
    __syncthreads();
    sm100::grid_dependency_wait();
    if (ring & 1023u) {                                       // as the runtime places it; nothing below would fit
        if (threadIdx.x == 0) atomicCAS(p.err, 0u, (kKernelAttn << 24) | (4u << 16) | 2u);
        return;
    }
    if (blockIdx.x == 0 && warp == 0)
        for (int b = lane; b < p.B; b += 32)
            if (p.lens[b] < 0 || p.lens[b] > p.max_len) atomicCAS(p.err, 0u, (kKernelAttn << 24) | (1u << 16) | 2u);
    Cursor at;
    const int size = first_tile<C>(p, hr_n, at);
    if (at.place >= size) return;                             // the same for every warp
    if (warp == kWideWarps + 1) {
        sm100::tmem_alloc(sm100::smem_u32(const_cast<uint32_t*>(s_tmem)), C::kCols);
        sm100::tc_fence_before();
    }
    __syncthreads();
    sm100::tc_fence_after();
    // The next kernel may be scheduled only now: one that takes tensor memory before it
    // waits for this kernel, on an SM that has room for both, would keep it from this one.
    sm100::grid_launch_dependents();
    const uint32_t tmem = *s_tmem, t_o = tmem + 2 * C::kSlice, t_x = tmem + 3 * C::kSlice;

    auto head_of = [&](const Cursor& c) { return chunks == 1 ? c.hr : c.hr / chunks; };
    bool dead = false;                                        // a wait ran out: nothing more is issued or waited for
    auto wait = [&](uint32_t bar, uint32_t parity, uint32_t site) {
        if (!dead && !sm100::mbar_wait_bounded(bar, parity, abort, kWaitLimitNs)) {
            if (lane == 0) atomicCAS(p.err, 0u, (kKernelAttn << 24) | (site << 16) | 1u);
            *abort = 1;
            dead = true;
        }
        dead = __any_sync(0xffffffffu, dead);
    };

    if (warp == kWideWarps) {                                 // loads: a box of one page a lane
        auto page_of = [&](int j) { return p.page_shift >= 0 ? j >> p.page_shift : j / p.page_size; };
        int m = 0;                                            // tile n: 2n its keys, 2n + 1 its values
#pragma unroll 1
        for (bool first = true; at.place < size; at.next<C>(p, hr_n), first = false) {
            const int c0 = at.s.start + at.tile * CT, h = head_of(at);
            if (first || (at.tile & 15) == 0) {               // page numbers to L1 ahead of their use, a tile a lane
                const int64_t j = c0 + (int64_t)lane * CT;
                if (j < at.s.len) touch_l1(p.pages + at.b * p.pages_seq + page_of((int)j));
            }
            const int i = lane * p.box, j = c0 + i;
            const bool load = i < CT && j < at.s.len;
            const int pg = load ? page_of(j) : 0;
            int page = load ? p.pages[at.b * p.pages_seq + pg] : 0;
            if ((uint32_t)page >= (uint64_t)p.num_pages) {
                atomicCAS(p.err, 0u, (kKernelAttn << 24) | (2u << 16) | 2u);
                page = 0;
            }
            const int row = j - pg * p.page_size;
            const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, load));
#pragma unroll 1
            for (int kv = 0; kv < 2 && !dead; ++kv, ++m) {
                const uint32_t bar = full + 8 * (m % S), dst = ring + m % S * C::kTile + i * 128;
                if (m >= S) wait(empty + 8 * (m % S), (m / S - 1) & 1, 5);
                if (dead) break;
                if (lane == 0) sm100::mbar_arrive_expect_tx(bar, boxes * p.box * C::RB);
                __syncwarp();
                if (load)
#pragma unroll
                    for (int x = 0; x < DP / 64; ++x)
                        tma_load_4d(dst + x * C::kPiece, kv ? &vmap : &kmap, bar, x * 64, p.order ? row : h, p.order ? h : row, page);
            }
            if (dead) break;
        }
        if (dead)                                              // copies still in flight write to this CTA's memory
            for (int k = m > S ? m - S : 0; k < m; ++k) sm100::mbar_drain(full + 8 * (k % S), (k / S) & 1, kWaitLimitNs);
    } else if (warp == kWideWarps + 1) {                      // multiplies
        // fp32 sums of bf16 products, 128 x RT; for O^T both operands MN-major
        constexpr uint32_t kS = 1u << 4 | 1u << 7 | 1u << 10 | (uint32_t)(RT >> 3) << 17 | (128u >> 4) << 24;
        constexpr uint32_t kO = kS | 1u << 15 | 1u << 16;
        auto scores = [&](int n, bool first, int item) {
            const int m = 2 * n;
            wait(full + 8 * (m % S), (m / S) & 1, 3);
            if (first) wait(q_full, item & 1, 6);
            if (n >= 2) wait(s_free + 8 * (n & 1), ((n >> 1) - 1) & 1, 7);
            if (dead) return;
            sm100::tc_fence_after();
            if (lane == 0) {
                const uint64_t a = sm100::umma_desc_k128_sw128(ring + m % S * C::kTile), b = sm100::umma_desc_k128_sw128(sq);
#pragma unroll
                for (int k = 0; k < DP / 16; ++k)
                    sm100::mma_f16(tmem + (n & 1) * C::kSlice, a + (k >> 2) * (C::kPiece >> 4) + (k & 3) * 2,
                                   b + (k >> 2) * (RT * 128 >> 4) + (k & 3) * 2, kS, k > 0);
                sm100::tc_commit(empty + 8 * (m % S));
                sm100::tc_commit(s_full + 8 * (n & 1));
            }
            __syncwarp();
        };
        int item = 0;
        bool first = true;
        scores(0, true, 0);
#pragma unroll 1
        for (int n = 0; at.place < size && !dead; ++n) {
            Cursor then = at;
            then.next<C>(p, hr_n);
            const bool more = then.place < size, fresh = then.tile == 0;
            if (more && !fresh) scores(n + 1, false, item);
            const int m = 2 * n + 1;
            wait(full + 8 * (m % S), (m / S) & 1, 3);
            wait(p_full + 8 * (n & 1), (n >> 1) & 1, 8);
            if (dead) break;
            sm100::tc_fence_after();
            if (lane == 0) {
                // M is 128; a head of 64 has its second half beyond the tile: any
                // values, on lanes that nobody reads
                const uint64_t a = wide_desc_mn(ring + m % S * C::kTile, C::kPiece);
                const uint64_t b = wide_desc_mn(sp + n % C::kBufs * C::kPart, C::kPiece);
#pragma unroll
                for (int k = 0; k < CT / 16; ++k)
                    sm100::mma_f16(t_o, a + k * (16 * 128 >> 4), b + k * (16 * 128 >> 4), kO, !first || k > 0);
                sm100::tc_commit(empty + 8 * (m % S));
                sm100::tc_commit(pv + 8 * (n & 1));
            }
            __syncwarp();
            if (more && fresh) scores(n + 1, true, ++item);
            first = fresh;
            at = then;
        }
        if (dead) {                                           // products in flight end before tensor memory is freed
            if (lane == 0) {
                sm100::tc_commit(drained);
                sm100::mbar_drain(drained, 0, kWaitLimitNs);
            }
            __syncwarp();
        }
    } else {
        // eights of rows 2u + half are this thread's, of its token
        const int quad = warp & 3, half = warp >> 2, c0 = half * 8, tok = quad * 32 + lane;
        const uint32_t t_lane = (uint32_t)(quad * 32) << 16;
        const float xs = p.scale * kLog2e;
        auto sync = [&]() { sm100::named_bar_sync(2, kN); };
        auto summed = [&](int n) {                            // tile n's product is in the sums
            wait(pv + 8 * (n & 1), (n >> 1) & 1, 10);
            sm100::tc_fence_after();
        };
        float sum[8 * U];
        int live = 0;                                         // rows of the item that are there
        int both_lo = 0, both_hi = 0;
        auto on = [&](int u) { return (2 * u + half) * 8 < live; };
        bool set_apart = false;                               // products with values that are not finite, in t_x

        // An item's queries as the N operand, and its rows' bounds.
        auto begin = [&](const Cursor& c) {
            const int h = head_of(c), r0 = (c.hr - h * chunks) * RT;
            sync();                                           // nobody is at the bounds of the item before
            constexpr int kEach = (RT * (DP / 8) + kN - 1) / kN;
            uint4 v[kEach];
#pragma unroll
            for (int i = 0; i < kEach; ++i) {                 // in flight together
                const int r = (i * kN + threadIdx.x) / (DP / 8), k = threadIdx.x % (DP / 8), rr = r0 + r, qi = rr / group;
                v[i] = make_uint4(0, 0, 0, 0);
                if (r < RT && rr < rows && k * 8 < p.D)
                    v[i] = *reinterpret_cast<const uint4*>(p.q + c.b * p.q_seq + qi * p.q_token +
                                                           (h * group + rr - qi * group) * p.q_head + k * 8);
            }
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const int r = (i * kN + threadIdx.x) / (DP / 8), k = threadIdx.x % (DP / 8);
                if (r < RT) st_shared16(sq + (k >> 3) * (RT * 128) + r * 128 + (((k & 7) ^ (r & 7)) << 4), v[i].x, v[i].y, v[i].z, v[i].w);
            }
            if (threadIdx.x < RT) {
                const int r = threadIdx.x, hi = r0 + r < rows ? c.s.len - p.Lq + (r0 + r) / group + 1 : 0;
                s_hi[r] = hi;
                s_lo[r] = p.window ? max(0, hi - p.window) : 0;
            }
            sm100::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) sm100::mbar_arrive(q_full);
            sync();
        };

        auto compute = [&](int n, bool first) {
            const int t0 = at.s.start + at.tile * CT, j = t0 + tok;
            const uint32_t t_s = tmem + (n & 1) * C::kSlice + c0 + t_lane, vb = ring + (2 * n + 1) % S * C::kTile;
            // tokens both_lo .. both_hi - 1 are seen by every row of the item
            const bool edge = t0 + CT > both_hi || t0 < both_lo;
            wait(s_full + 8 * (n & 1), (n >> 1) & 1, 9);
            sm100::tc_fence_after();
            // a group's log2 scores, above the running reference or as they are; tokens
            // that a query does not see at -inf
            constexpr int G = C::kGroup;
            float x[8 * G];
            auto load = [&](int u0, bool above) {
#pragma unroll
                for (int u = 0; u < G; ++u) tmem_ld_x8(t_s + (u0 + u) * 16, x + 8 * u);
                sm100::tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 8 * G; e += 4) {
                    const float4 r = above ? *reinterpret_cast<const float4*>(s_ref + c0 + (u0 + e / 8) * 16 + e % 8)
                                           : make_float4(0.f, 0.f, 0.f, 0.f);
                    x[e] = fmaf(x[e], xs, -r.x), x[e + 1] = fmaf(x[e + 1], xs, -r.y);
                    x[e + 2] = fmaf(x[e + 2], xs, -r.z), x[e + 3] = fmaf(x[e + 3], xs, -r.w);
                }
                if (edge) {
#pragma unroll
                    for (int e = 0; e < 8 * G; e += 4) {
                        const int c = c0 + (u0 + e / 8) * 16 + e % 8;
                        const int4 hi = *reinterpret_cast<const int4*>(s_hi + c), lo = *reinterpret_cast<const int4*>(s_lo + c);
                        x[e] = j >= hi.x || j < lo.x ? -INFINITY : x[e];
                        x[e + 1] = j >= hi.y || j < lo.y ? -INFINITY : x[e + 1];
                        x[e + 2] = j >= hi.z || j < lo.z ? -INFINITY : x[e + 2];
                        x[e + 3] = j >= hi.w || j < lo.w ? -INFINITY : x[e + 3];
                    }
                }
            };
            float top = -INFINITY;
#pragma unroll
            for (int u0 = 0; u0 < U; u0 += G) {
                load(u0, true);
#pragma unroll
                for (int e = 0; e < 8 * G; ++e) top = fmaxf(top, x[e]);
            }
            const bool moved = sm100::bar_red_or(1, kN, top > kLazy);
            if (moved) {                                      // the rows' references move
#pragma unroll 1
                for (int u0 = 0; u0 < U; u0 += G) {
                    load(u0, false);
#pragma unroll
                    for (int u = 0; u < G; ++u) {
                        const float r = join8(x + 8 * u, [](float a, float b) { return fmaxf(a, b); });
                        if ((lane & 3) == 0) s_w[quad * RT + c0 + (u0 + u) * 16 + (lane >> 2)] = fmaxf(r, kNone);
                    }
                }
                sync();
                if (threadIdx.x < RT) {
                    const int r = threadIdx.x;
                    const float was = s_ref[r], now = fmaxf(was, fmaxf(fmaxf(s_w[r], s_w[RT + r]),
                                                                       fmaxf(s_w[2 * RT + r], s_w[3 * RT + r])));
                    s_fac[r] = ex2(was - now);
                    s_ref[r] = now;
                }
                sync();
#pragma unroll
                for (int i = 0; i < 8 * U; ++i) sum[i] *= s_fac[c0 + (i >> 3) * 16 + (i & 7)];
                if (!first) {
                    summed(n - 1);
#pragma unroll 1
                    for (int u = 0; u < U; ++u) {
                        float o[8];
                        tmem_ld_x8(t_o + t_lane + c0 + u * 16, o);
                        sm100::tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 8; ++e) o[e] *= s_fac[c0 + u * 16 + e];
                        tmem_st_x8(t_o + t_lane + c0 + u * 16, o);
                    }
                    sm100::tmem_wait_st();
                }
            }
            // the probabilities of the tile that had this buffer are read
            if (n >= C::kBufs) summed(n - C::kBufs);
            // row of the token, eight eights a piece
            const uint32_t sp_n = sp + n % C::kBufs * C::kPart, pr = sp_n + tok * 128;
#pragma unroll
            for (int u0 = 0; u0 < U; u0 += G) {
                if (U > G || moved) load(u0, true);           // (more than a group is not kept)
#pragma unroll
                for (int u = 0; u < G; ++u) {
                    float* const y = x + 8 * u;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        y[e] = ex2(y[e]);
                        sum[8 * (u0 + u) + e] += y[e];
                    }
                    const int cu = 2 * (u0 + u) + half;
                    st_shared16(pr + (cu >> 3) * C::kPiece + (((cu & 7) ^ (tok & 7)) << 4), pack2_bf16(y[0], y[1]),
                                pack2_bf16(y[2], y[3]), pack2_bf16(y[4], y[5]), pack2_bf16(y[6], y[7]));
                }
            }
            sm100::tc_fence_before();
            __syncwarp();
            if (lane == 0) sm100::mbar_arrive(s_free + 8 * (n & 1));
            // What the product must not meet: rows of no visible token become zero, and
            // values that are not finite and that only some queries see are set apart.
            if (edge) {
                wait(full + 8 * ((2 * n + 1) % S), ((2 * n + 1) / S) & 1, 3);
                auto some = [&](int i) { return i >= at.s.lo && i < at.s.len && (i < both_lo || i >= both_hi); };
                auto value = [&](int i, int d) {
                    return vb + (d >> 6) * C::kPiece + i * 128 + (((d >> 3 & 7) ^ (i & 7)) << 4) + (d & 7) * 2;
                };
                bool bad = false;
                if (j < at.s.lo || j >= at.s.len) {
                    for (int d = half * (DP / 2); d < (half + 1) * (DP / 2); d += 8) st_zero16(value(tok, d));
                } else if (some(j)) {
                    for (int d = half * (DP / 2); d < (half + 1) * (DP / 2); d += 8) {
                        const uint4 v = ld_shared16(value(tok, d));
                        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) bad |= !isfinite(bf16_lo(w[e])) || !isfinite(bf16_hi(w[e]));
                    }
                }
                if (sm100::bar_red_or(1, kN, bad)) {
                    const int d = quad * 32 + lane;
#pragma unroll 1
                    for (int u = 0; u < U && on(u); ++u) {
                        const int cu = 2 * u + half;
                        float y[8] = {};
                        if (set_apart) {
                            tmem_ld_x8(t_x + t_lane + c0 + u * 16, y);
                            sm100::tmem_wait_ld();
                        }
#pragma unroll 1
                        for (int i = 0; i < CT; ++i) {
                            if (!some(t0 + i)) continue;
                            const float v = d < DP ? ld_value<false>(value(i, d)) : 0.f;
                            if (isfinite(v)) continue;
                            const uint32_t pi = sp_n + (cu >> 3) * C::kPiece + i * 128 + (((cu & 7) ^ (i & 7)) << 4);
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                if (t0 + i < s_hi[cu * 8 + e] && t0 + i >= s_lo[cu * 8 + e])
                                    y[e] += ld_value<false>(pi + 2 * e) * v;
                        }
                        __syncwarp();
                        tmem_st_x8(t_x + t_lane + c0 + u * 16, y);
                    }
                    sm100::tmem_wait_st();
                    set_apart = true;
                    sync();
                    if (half == 0 && d < DP)
                        for (int i = 0; i < CT; ++i)
                            if (some(t0 + i) && !isfinite(ld_value<false>(value(i, d)))) st_zero<false>(value(i, d));
                }
            }
            sm100::tc_fence_before();
            sm100::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) sm100::mbar_arrive(p_full + 8 * (n & 1));
        };

        // An item's sums written: the result if it lies wholly in this CTA's range,
        // else one of the CTA's two slots.  Tensor memory's lanes are the head's values.
        auto finish = [&](int n, const Cursor& c) {
            const int begun = c.place - c.tile;               // the item's tiles: begun .. begun + tiles - 1
            const bool whole = begun >= 0 && begun + c.s.tiles <= size;
            const int h = head_of(c), r0 = (c.hr - h * chunks) * RT;
            float* const slot = p.ws + ((int64_t)blockIdx.x * 2 + (begun <= 0 ? 0 : 1)) * (RT * (DP + 2));
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float y = join8(sum + 8 * u, [](float a, float b) { return a + b; });
                if ((lane & 3) == 0) s_w[quad * RT + c0 + u * 16 + (lane >> 2)] = y;
            }
            sync();
            if (threadIdx.x < RT) {
                const int r = threadIdx.x, rr = r0 + r, qi = rr / group;
                const float l = (s_w[r] + s_w[RT + r]) + (s_w[2 * RT + r] + s_w[3 * RT + r]);
                s_row[r] = qi * p.Hq + h * group + rr - qi * group;
                s_fac[r] = l == 0.f ? 0.f : 1.f / l;
                if (!whole)
                    slot[RT * DP + r] = s_ref[r], slot[RT * DP + RT + r] = l;
                else if (p.lse && r < live)
                    p.lse[(int64_t)c.b * p.Lq * p.Hq + s_row[r]] = l == 0.f ? -INFINITY : (s_ref[r] + log2f(l)) * kLn2;
                s_ref[r] = kNone;
            }
            summed(n);
            sync();
            const int d = quad * 32 + lane;
            uint16_t* const out = p.o + (int64_t)c.b * p.Lq * p.Hq * p.D + d;
#pragma unroll 1
            for (int u = 0; u < U && on(u); ++u) {
                float o[8], y[8];
                tmem_ld_x8(t_o + t_lane + c0 + u * 16, o);
                if (set_apart) tmem_ld_x8(t_x + t_lane + c0 + u * 16, y);
                sm100::tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int r = c0 + u * 16 + e;
                    if (set_apart) o[e] += y[e];
                    if (!whole) {
                        if (d < DP) slot[r * DP + d] = o[e];
                    } else if (r < live && d < p.D) {
                        const float f = s_fac[r];
                        out[(int64_t)s_row[r] * p.D] = (uint16_t)pack2_bf16(f == 0.f ? 0.f : o[e] * f, 0.f);
                    }
                }
            }
            set_apart = false;
        };

        begin(at);
        bool first = true;
#pragma unroll 1
        for (int n = 0; at.place < size; ++n) {
            if (first) {
                const int r0 = (at.hr - head_of(at) * chunks) * RT, p0 = at.s.len - p.Lq + 1;
                live = min(RT, rows - r0);
                both_hi = p0 + r0 / group;
                both_lo = p.window ? p0 + (r0 + live - 1) / group - p.window : 0;
#pragma unroll
                for (int i = 0; i < 8 * U; ++i) sum[i] = 0.f;
            }
            compute(n, first);
            Cursor then = at;
            then.next<C>(p, hr_n);
            first = then.tile == 0 || then.place >= size;
            if (first) {
                const Cursor done = at;
                if (then.place < size) begin(then);
                finish(n, done);
            }
            at = then;
        }
        sm100::tc_fence_before();
    }
    __syncthreads();
    if (warp == kWideWarps + 1) {
        sm100::tc_fence_after();
        sm100::tmem_dealloc(tmem, C::kCols);
    }
}

template <class C>
cudaError_t launch_wide(const AttnParams& a, cudaStream_t st) {
    AttnParams p = a;
    CUtensorMap km = {}, vm = {};
    p.page_shift = p.page_size & (p.page_size - 1) ? -1 : __builtin_ctz((unsigned)p.page_size);
    p.box = C::CT;
    while (p.page_size % p.box) p.box /= 2;
    p.order = p.c_token < p.c_head && p.Hkv > 1;
    p.cluster = 0;
    if (!make_map<C>(&km, p.kpool, p) || !make_map<C>(&vm, p.vpool, p)) return cudaErrorInvalidValue;
    const int rows = p.Hq / p.Hkv * p.Lq, chunks = (rows + C::RT - 1) / C::RT;
    const int64_t items = (int64_t)p.B * p.Hkv * chunks, tiles = (p.max_len + C::CT - 1) / C::CT;
    const int64_t most = items * ((tiles > 1 ? tiles : 1) + C::kItem), wave = num_sms();
    static std::atomic<uint64_t> ready{0};                    // devices whose kernel has its shared memory
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
        e = cudaFuncSetAttribute(attn_paged_wide_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        if (e != cudaSuccess) return e;
        if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    const int ctas = (int)(most < wave ? most : wave);
    e = launch_pdl(attn_paged_wide_kernel<C>, dim3((unsigned)ctas), dim3(kWideThreads), C::kSmem, st, p, km, vm);
    if (e != cudaSuccess || tiles <= 1) return e;             // items of one tile: nothing to join
    const bool spread = items * 2 < num_sms();
    return launch_pdl(attn_join_kernel<C>, dim3((unsigned)items, spread ? (unsigned)(rows < C::RT ? rows : C::RT) : 1u),
                      dim3(256), 0, st, p, ctas, (int)spread);
}

template <class C>
Plan plan_wide(int64_t max_len) {
    if (max_len <= C::CT) return Plan{0, 1};
    return Plan{(size_t)num_sms() * 2 * C::RT * (C::DP + 2) * sizeof(float), 2};
}

// Where it is taken, and its configuration: as few rows as hold them, in chunks of up
// to 96, each reading the cache again; up to 128 in one, whose scores a thread cannot
// keep, so that it reads them twice.  120 rows, 32 sequences to 16384: 294 us in one,
// 353 in two chunks; 320 rows, 16 sequences: 438 us in chunks of 128, 403 in ones of 80;
// prompt chunks of 512 behind up to 3488 tokens, 7 heads a kv head: 483 and 420.
inline bool is_wide(int64_t D, int64_t rows) { return rows > 32 && D <= 128; }
template <int DP, class F>
auto pick_wide_rows(int64_t rows, F f) {
    if (rows > 96 && rows <= 128) return f(WideConfig<DP, 128>{});
    const int64_t chunks = (rows + 95) / 96, each = (rows + chunks - 1) / chunks;
    if (each <= 48) return f(WideConfig<DP, 48>{});
    if (each <= 64) return f(WideConfig<DP, 64>{});
    if (each <= 80) return f(WideConfig<DP, 80>{});
    return f(WideConfig<DP, 96>{});
}
template <class F>
auto pick_wide(int64_t D, int64_t rows, F f) {
    return D <= 64 ? pick_wide_rows<64>(rows, f) : pick_wide_rows<128>(rows, f);
}

}  // namespace
}  // namespace attn
}  // namespace fp8rl
