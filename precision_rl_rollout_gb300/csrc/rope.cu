// rope.cu -- rotary positions (forward and gradient), and the append that
// rotates a step's queries and keys and stores keys and values in a paged cache.
//
// The first R of a head's D values are R/2 pairs (x1, x2): (i, i + R/2) in the
// half layout, (2i, 2i + 1) in the interleaved one.  With c, s the cosine and
// sine of the token's position times the pair's frequency (table row: R/2
// cosines, then R/2 sines),
//   y1 = c x1 - s x2,  y2 = s x1 + c x2;   gradient: the same with s -> -s.
// Products and their difference are rounded one by one (no FMA), so that the
// fp32 result, and with it every stored E4M3 code, is a function of the inputs
// alone; then one rounding to the output's type.  A cached key is rounded once,
// from the fp32 rotation, not through bf16.
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace fp8rl {

namespace {

constexpr uint32_t kKernelRope = 8;
constexpr int kRopeThreads = 256;

__device__ __forceinline__ void record_data_error(uint32_t* err, uint32_t site) {
    atomicCAS(err, 0u, (kKernelRope << 24) | (site << 16) | 2u);
}

struct Row {              // one token's position and cache slot
    const float* cs;      // its table row
    int64_t slot;         // offset of its cache slot in elements, < 0: not stored
};

__device__ __forceinline__ Row token_row(const RopeParams& p, int64_t t, bool first) {
    Row r{nullptr, -1};
    if (p.R) {
        int64_t pos = p.pos[t];
        if (pos < 0 || pos >= p.max_pos) {
            if (first) record_data_error(p.err, 1);
            pos = pos < 0 ? 0 : p.max_pos - 1;
        }
        r.cs = p.table + pos * p.R;
    }
    if (p.Hkv) {
        const int64_t slot = p.slots[t];
        if (slot >= 0) {
            // a 64-bit division costs a hundred instructions; most pools need none
            const int64_t page = slot >> 32 ? slot / p.page_size : (uint32_t)slot / (uint32_t)p.page_size;
            if (page < p.num_pages)
                r.slot = page * p.c_page + (slot - page * p.page_size) * p.c_token;
            else if (first)
                record_data_error(p.err, 2);
        }
    }
    return r;
}

// W bf16 values moved as one access: 8 (16 bytes) or 4 (8 bytes).
template <int W>
struct Chunk {
    uint32_t w[W / 2];
    __device__ __forceinline__ void unpack(float* f) const {
#pragma unroll
        for (int e = 0; e < W / 2; ++e) f[2 * e] = bf16_lo(w[e]), f[2 * e + 1] = bf16_hi(w[e]);
    }
    __device__ __forceinline__ void pack(const float* f) {
#pragma unroll
        for (int e = 0; e < W / 2; ++e) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[e]) : "f"(f[2 * e + 1]), "f"(f[2 * e]));
    }
    // Read once, past L1; not the read-only path, the rotation may be in place.
    __device__ __forceinline__ void load(const uint16_t* p) {
        if constexpr (W == 8)
            asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                         : "l"(p)
                         : "memory");
        else
            asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p) : "memory");
    }
    __device__ __forceinline__ void store(uint16_t* p) const {
        if constexpr (W == 8)
            __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
        else
            __stcs(reinterpret_cast<uint2*>(p), make_uint2(w[0], w[1]));
    }
};
// (The packed fp32 forms were tried: a packed product and a packed sum that
// follow one another came out as one fused rounding in places.)
__device__ __forceinline__ void rotate(float& a, float& b, float c, float s) {
    const float ya = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    const float yb = __fadd_rn(__fmul_rn(a, s), __fmul_rn(b, c));
    a = ya, b = yb;
}

// The E4M3 code of f / scale, the quotient the IEEE one.  Keys are no longer bf16
// values here, so the divisor of common.cuh, checked over the bf16 domain, does not
// apply.  f times the rounded reciprocal is within three units in the last place of
// the quotient (three roundings of 2^-24), and has its code unless a boundary
// between two codes lies between them: a number of at most five significant bits,
// its 19 low mantissa bits zero.  So only a product within four units of such a
// number is divided.  Where the scale is a power of two the product is the quotient;
// a scale outside [2^-100, 2^100], 0 and NaN included, always divides.
struct Quant {
    float s, r;
    bool divide, exact;
    __device__ __forceinline__ explicit Quant(float scale) {
        s = scale, r = __frcp_rn(scale);
        divide = !(scale >= 0x1p-100f && scale <= 0x1p100f);
        exact = (__float_as_uint(scale) & 0x7FFFFFu) == 0;
    }
    template <int W>
    __device__ __forceinline__ void store(uint8_t* to, const float* f) const {
        float q[W];
        uint32_t near = 0x7FFFFu;
#pragma unroll
        for (int e = 0; e < W; ++e) {
            q[e] = __fmul_rn(f[e], r);
            near = min(near, (__float_as_uint(q[e]) + 4u) & 0x7FFFFu);
        }
        if (divide || (near <= 8u && !exact)) {
#pragma unroll
            for (int e = 0; e < W; ++e) q[e] = __fdiv_rn(f[e], s);
        }
        uint32_t o[W / 4];
#pragma unroll
        for (int e = 0; e < W / 4; ++e)
            o[e] = e4m3x2(q[4 * e], q[4 * e + 1]) | (e4m3x2(q[4 * e + 2], q[4 * e + 3]) << 16);
        if constexpr (W == 8)
            *reinterpret_cast<uint2*>(to) = make_uint2(o[0], o[1]);
        else
            *reinterpret_cast<uint32_t*>(to) = o[0];
    }
};

// A head is cut into columns, one a thread, of chunks of W values (16 bytes; 8 where
// alignment or a half of R that is no multiple of 8 wants it): in the half layout
// column j < R / 2W is the chunks j and j + R / 2W, whose values pair up, and what lies
// past R is two chunks a column as well, its first half and its second; interleaved, a
// chunk holds its own pairs and is a column.  Threads that rotate and that do not share
// their loads and stores, so a warp that holds both takes the longer way once (append
// of 8192 tokens, 28 + 2 x 4 heads, 64 of 128 values, over bf16: 42 us with a way each
// and one chunk a column past R, 28 so).
// A thread keeps its column's cosines and sines in registers and goes over the
// token's heads (queries, keys, values) p.lanes apart, kBatch at a time with their
// loads in flight together; the first batch is in flight while the position and
// its row come.  Two at a time where codes are stored: the quotients take the
// registers of the others (the append above over E4M3: 57 us with a division a
// value, 42 with the products and four at a time, 36 so).  Loads pass L1 and stores go out evict-first: nothing is read
// twice (49 -> 45 us for the gradient below).
// Bound by HBM: 2 bytes in, 2 (E4M3: 1) out a value.  8192 tokens, 40 + 8 heads of
// 128: 32 us, 6.3 TB/s; gradient of 16411 tokens, 28 + 4 heads, 64 of 128 values
// interleaved: 42 us, 6.5 TB/s; append of 8192 tokens, 40 + 2 x 8 heads, bf16
// pages: 38 us, 6.3 TB/s; in 8-byte chunks (11041 tokens, 28 + 4 heads, 56 of 80
// values) 22 us, 5.2 TB/s, a value at a time 82.  What is left there is the start and the
// last wave.  Over E4M3 the append is not HBM's: 8192 tokens of 28 + 2 x 4 heads take 33 us
// for 147 MB, 4.4 TB/s, with codes leaving 8 bytes at a time and two heads' loads in flight.
__host__ __device__ inline int rope_columns(int D, int R, bool inter, int W) {
    return inter ? D / W : R / (2 * W) + ((D - R) / W + 1) / 2;
}

template <bool kInter, bool kE4m3, int W>
__global__ void __launch_bounds__(kRopeThreads, 3)
rope_kernel(const __grid_constant__ RopeParams p) {
    pdl_wait_then_release();
    const int pairs = p.R / (kInter ? W : 2 * W), cols = rope_columns(p.D, p.R, kInter, W);
    const int j = threadIdx.x % cols, hl = threadIdx.x / cols % p.lanes, tok = threadIdx.x / (cols * p.lanes);
    const int64_t t = (int64_t)blockIdx.x * p.cta_tokens + tok;
    if (tok >= p.cta_tokens || t >= p.T) return;
    const bool turn = j < pairs;                              // a column that rotates
    const int apart = kInter ? 0 : turn ? p.R / 2 : (cols - pairs) * W;
    const int d = turn ? j * W : p.R + (j - pairs) * W;
    const bool two = !kInter && d + apart < p.D;
    constexpr int NC = kInter ? W / 2 : W;
    float c[NC], s[NC];
    const uint16_t* const q = p.q + t * p.q_token + d;
    const uint16_t* const k = p.k + t * p.k_token + d;
    const uint16_t* const v = p.v + t * p.v_token + d;
    uint16_t* const y = p.y + t * p.y_token + d;
    const int heads = p.Hq + 2 * p.Hkv;
    // queries rotated in place: their columns past R stay as they are
    int h0 = hl;
    if (p.in_place && !turn)
        while (h0 < p.Hq) h0 += p.lanes;
    constexpr int kBatch = kE4m3 ? 2 : 4;
    Chunk<W> x0[kBatch], x1[kBatch];
    auto load = [&]() {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int h = h0 + u * p.lanes;
            if (h >= heads) break;
            const uint16_t* src = h < p.Hq ? q + h * p.q_head
                                           : h < p.Hq + p.Hkv ? k + (h - p.Hq) * p.k_head : v + (h - p.Hq - p.Hkv) * p.v_head;
            x0[u].load(src);
            if (two) x1[u].load(src + apart);
        }
    };
    load();                                                   // in flight while the position and its row come
    const Row row = token_row(p, t, threadIdx.x == tok * cols * p.lanes);
    const Quant kq(kE4m3 ? *p.k_scale : 1.f), vq(kE4m3 ? *p.v_scale : 1.f);
    if (turn) {
        if constexpr (NC >= 4) {
#pragma unroll
            for (int e = 0; e < NC; e += 4) {
                const float4 a = *reinterpret_cast<const float4*>(row.cs + j * NC + e);
                const float4 b = *reinterpret_cast<const float4*>(row.cs + p.R / 2 + j * NC + e);
                c[e] = a.x, c[e + 1] = a.y, c[e + 2] = a.z, c[e + 3] = a.w;
                s[e] = p.sign * b.x, s[e + 1] = p.sign * b.y, s[e + 2] = p.sign * b.z, s[e + 3] = p.sign * b.w;
            }
        } else {
            const float2 a = *reinterpret_cast<const float2*>(row.cs + j * NC);
            const float2 b = *reinterpret_cast<const float2*>(row.cs + p.R / 2 + j * NC);
            c[0] = a.x, c[1] = a.y, s[0] = p.sign * b.x, s[1] = p.sign * b.y;
        }
    }
    // the chunks' values, rotated where the column and the head are
    auto values = [&](int u, bool is_v, float* a, float* b) {
        x0[u].unpack(a);
        if constexpr (kInter) {
            if (turn && !is_v) {
#pragma unroll
                for (int e = 0; e < W / 2; ++e) rotate(a[2 * e], a[2 * e + 1], c[e], s[e]);
            }
        } else {
            x1[u].unpack(b);
            if (turn && !is_v) {
#pragma unroll
                for (int e = 0; e < W; ++e) rotate(a[e], b[e], c[e], s[e]);
            }
        }
    };
    const int stored = row.slot < 0 ? p.Hq : heads;
    for (;;) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int h = h0 + u * p.lanes;
            if (h >= stored) break;
            const bool is_q = h < p.Hq, is_v = h >= p.Hq + p.Hkv;
            float a[W], b[W];
            const int64_t at = row.slot + d + (h - p.Hq - (is_v ? p.Hkv : 0)) * p.c_head;
            void* const pool = is_v ? p.vpool : p.kpool;
            if (kE4m3 && !is_q) {
                values(u, is_v, a, b);
                const Quant& z = is_v ? vq : kq;
                z.template store<W>(static_cast<uint8_t*>(pool) + at, a);
                if (two) z.template store<W>(static_cast<uint8_t*>(pool) + at + apart, b);
            } else {
                if (turn && !is_v) {
                    values(u, is_v, a, b);
                    x0[u].pack(a);
                    if (!kInter) x1[u].pack(b);
                }
                uint16_t* to = is_q ? y + h * p.y_head : static_cast<uint16_t*>(pool) + at;
                x0[u].store(to);
                if (two) x1[u].store(to + apart);
            }
        }
        h0 += kBatch * p.lanes;
        if (h0 >= stored) return;
        load();
    }
}

// The same one pair (or one value past R, or of v) at a time, for widths and
// strides that 8-byte chunks do not divide.
template <bool kInter, bool kE4m3>
__global__ void __launch_bounds__(kRopeThreads)
rope_narrow_kernel(const __grid_constant__ RopeParams p) {
    pdl_wait_then_release();
    const int64_t t = blockIdx.x;
    const Row row = token_row(p, t, threadIdx.x == 0);
    const int half = p.R / 2, rest = p.D - p.R;
    const int per_q = half + (p.in_place ? 0 : rest), per_k = half + rest, per_v = p.D;
    const int nq = p.Hq * per_q, nk = nq + p.Hkv * per_k, n = nk + p.Hkv * per_v;
    auto bf = [](uint16_t h) { return __uint_as_float((uint32_t)h << 16); };
    auto cache = [&](void* pool, int64_t at, float f, const float* scale) {
        if (kE4m3)
            static_cast<uint8_t*>(pool)[at] = (uint8_t)e4m3x2(__fdiv_rn(f, *scale), 0.f);
        else
            static_cast<uint16_t*>(pool)[at] = (uint16_t)f32_to_bf16_bits(f);
    };
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        if (i >= nq && row.slot < 0) break;
        if (i >= nk) {
            const int h = (i - nk) / per_v, d = i - nk - h * per_v;
            cache(p.vpool, row.slot + h * p.c_head + d, bf(p.v[t * p.v_token + h * p.v_head + d]), p.v_scale);
            continue;
        }
        const bool is_k = i >= nq;
        const int ii = is_k ? i - nq : i, per = is_k ? per_k : per_q;
        const int h = ii / per, j = ii - h * per;
        const uint16_t* src = is_k ? p.k + t * p.k_token + h * p.k_head : p.q + t * p.q_token + h * p.q_head;
        const int64_t dst = is_k ? row.slot + h * p.c_head : t * p.y_token + h * p.y_head;
        auto put = [&](int d, float f) {
            if (is_k)
                cache(p.kpool, dst + d, f, p.k_scale);
            else
                p.y[dst + d] = (uint16_t)f32_to_bf16_bits(f);
        };
        if (j >= half) {
            const int d = p.R + (j - half);
            put(d, bf(src[d]));
        } else {
            const int da = kInter ? 2 * j : j, db = kInter ? 2 * j + 1 : j + half;
            float a = bf(src[da]), b = bf(src[db]);
            rotate(a, b, row.cs[j], p.sign * row.cs[half + j]);
            put(da, a);
            put(db, b);
        }
    }
}

// cos | sin of position x frequency, in fp64 and rounded once: at position
// 131071 an fp32 angle is off by up to 4e-3 radians, a bf16 ulp of the result.
// Made once per model; fp64 rate bounds it (a few ms at 131072 x 128).
__global__ void __launch_bounds__(256)
rope_table_kernel(const double* __restrict__ freq, int64_t max_pos, int half, double mag,
                  float* __restrict__ table) {
    pdl_wait_then_release();
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= max_pos * half) return;
    const int64_t pos = i / half;
    const int j = (int)(i - pos * half);
    double s, c;
    sincos((double)pos * freq[j], &s, &c);
    table[pos * 2 * half + j] = (float)(mag * c);
    table[pos * 2 * half + half + j] = (float)(mag * s);
}

template <bool kInter, bool kE4m3>
cudaError_t launch_t(RopeParams& p, int width, cudaStream_t st) {
    const int heads = p.Hq + 2 * p.Hkv;
    if (!width) return launch_pdl(rope_narrow_kernel<kInter, kE4m3>, dim3((unsigned)p.T), dim3(kRopeThreads), 0, st, p);
    // A thread goes over up to eight heads, fewer where that leaves SMs without two
    // CTAs: its own work (the token's row, its column's cosines) is then spread over
    // more bytes.  us with up to one, four, eight and sixteen heads a thread: 8192 tokens
    // of 48 heads of 128 41, 32.0, 32.4, 33.3; the gradient above 59, 45, 42, 43; the append
    // of 40 + 2 x 8 heads 48, 40, 38, 40, but the one of 28 + 2 x 4 heads 42, 27, 26, 22.
    // Four where codes are stored: that append over E4M3 57, 33, 35, 29.
    const int cols = rope_columns(p.D, p.R, kInter, width), most = kRopeThreads / cols;
    const int64_t room = p.T * heads * cols / (2 * (int64_t)num_sms() * kRopeThreads);
    constexpr int kMost = kE4m3 ? 4 : 8;
    const int each = room < 1 ? 1 : room > kMost ? kMost : (int)room;
    p.lanes = (heads + each - 1) / each;
    if (p.lanes > most) p.lanes = most;
    p.cta_tokens = each == 1 ? 1 : most / p.lanes;
    const dim3 grid((unsigned)((p.T + p.cta_tokens - 1) / p.cta_tokens));
    const dim3 block((unsigned)((cols * p.lanes * p.cta_tokens + 31) / 32 * 32));
    return launch_pdl(width == 8 ? rope_kernel<kInter, kE4m3, 8> : rope_kernel<kInter, kE4m3, 4>, grid, block, 0, st, p);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& a, bool interleaved, bool e4m3, cudaStream_t st) {
    RopeParams p = a;
    p.err = device_error_word();
    if (!p.err) return cudaErrorUnknown;
    if (p.Hkv == 0 && (p.Hq == 0 || (p.in_place && p.R == 0))) return cudaSuccess;
    // the widest chunks that widths, strides and addresses allow; 0: one value at a time
    const uintptr_t at = reinterpret_cast<uintptr_t>(p.q) | reinterpret_cast<uintptr_t>(p.k) |
                         reinterpret_cast<uintptr_t>(p.v) | reinterpret_cast<uintptr_t>(p.y);
    const int64_t strides = p.q_token | p.q_head | p.y_token | p.y_head | p.k_token | p.k_head | p.v_token | p.v_head;
    auto fits = [&](int w) {
        return p.D % w == 0 && p.R % (interleaved ? w : 2 * w) == 0 && p.D / w <= kRopeThreads && strides % w == 0 &&
               (at & (2 * w - 1)) == 0 && (reinterpret_cast<uintptr_t>(p.table) & 15u) == 0;
    };
    const int width = fits(8) ? 8 : fits(4) ? 4 : 0;
    if (interleaved) return e4m3 ? launch_t<true, true>(p, width, st) : launch_t<true, false>(p, width, st);
    return e4m3 ? launch_t<false, true>(p, width, st) : launch_t<false, false>(p, width, st);
}

cudaError_t launch_rope_table(const double* freq, int64_t max_pos, int64_t R, double mag, float* table,
                              cudaStream_t st) {
    const int64_t n = max_pos * (R / 2);
    return launch_pdl(rope_table_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, freq, max_pos,
                      (int)(R / 2), mag, table);
}

}  // namespace fp8rl
