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
        const int64_t page = slot / p.page_size;
        if (slot >= 0 && page < p.num_pages)
            r.slot = page * p.c_page + (slot - page * p.page_size) * p.c_token;
        else if (slot >= 0 && first)
            record_data_error(p.err, 2);
    }
    return r;
}

__device__ __forceinline__ void unpack8(uint4 v, float* f) {
    f[0] = bf16_lo(v.x), f[1] = bf16_hi(v.x), f[2] = bf16_lo(v.y), f[3] = bf16_hi(v.y);
    f[4] = bf16_lo(v.z), f[5] = bf16_hi(v.z), f[6] = bf16_lo(v.w), f[7] = bf16_hi(v.w);
}
__device__ __forceinline__ uint4 pack8(const float* f) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ void rotate(float& a, float& b, float c, float s) {
    const float ya = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    const float yb = __fadd_rn(__fmul_rn(a, s), __fmul_rn(b, c));
    a = ya, b = yb;
}

// Eight fp32 values to the cache at element offset `at`.  The quotient by the
// scale is the IEEE one: keys are no longer bf16 values here, so the divisor of
// common.cuh, checked over the bf16 domain, does not apply.
template <bool kE4m3>
__device__ __forceinline__ void store_cache8(void* pool, int64_t at, const float* f, float scale) {
    if constexpr (kE4m3) {
        uint2 o;
        o.x = e4m3x2(__fdiv_rn(f[0], scale), __fdiv_rn(f[1], scale)) |
              (e4m3x2(__fdiv_rn(f[2], scale), __fdiv_rn(f[3], scale)) << 16);
        o.y = e4m3x2(__fdiv_rn(f[4], scale), __fdiv_rn(f[5], scale)) |
              (e4m3x2(__fdiv_rn(f[6], scale), __fdiv_rn(f[7], scale)) << 16);
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(pool) + at) = o;
    } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(pool) + at) = pack8(f);
    }
}

// Work items of a token, 16-byte chunks of 8 values:
//   per q head: pairs (half layout: chunk j and chunk j + R/16; interleaved:
//   chunk j alone), then the chunks past R (only when not in place);
//   per k head: the same, always stored; per v head: D / 8 chunks.
// threadIdx.y: token of the CTA.
template <bool kInter, bool kE4m3>
__global__ void __launch_bounds__(kRopeThreads)
rope_kernel(const __grid_constant__ RopeParams p) {
    pdl_wait_then_release();
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    if (t >= p.T) return;
    const Row row = token_row(p, t, threadIdx.x == 0);
    const int pairs = p.R / (kInter ? 8 : 16);              // pair items per head
    const int rest = (p.D - p.R) / 8;                       // chunks past R per head
    const int per_q = pairs + (p.in_place ? 0 : rest), per_k = pairs + rest, per_v = p.D / 8;
    const int nq = p.Hq * per_q, nk = nq + p.Hkv * per_k, n = nk + p.Hkv * per_v;
    const int half = p.R / 2;
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        if (i >= nk) {                                      // v: stored as it is
            if (row.slot < 0) break;
            const int h = (i - nk) / per_v, d = (i - nk - h * per_v) * 8;
            float f[8];
            unpack8(*reinterpret_cast<const uint4*>(p.v + t * p.v_token + h * p.v_head + d), f);
            store_cache8<kE4m3>(p.vpool, row.slot + h * p.c_head + d, f, kE4m3 ? *p.v_scale : 1.f);
            continue;
        }
        const bool is_k = i >= nq;
        if (is_k && row.slot < 0) break;
        const int ii = is_k ? i - nq : i, per = is_k ? per_k : per_q;
        const int h = ii / per, j = ii - h * per;
        const uint16_t* src = is_k ? p.k + t * p.k_token + h * p.k_head : p.q + t * p.q_token + h * p.q_head;
        const int64_t dst = is_k ? row.slot + h * p.c_head : t * p.y_token + h * p.y_head;
        auto put = [&](int d, const float* f) {
            if (is_k)
                store_cache8<kE4m3>(p.kpool, dst + d, f, kE4m3 ? *p.k_scale : 1.f);
            else
                *reinterpret_cast<uint4*>(p.y + dst + d) = pack8(f);
        };
        if (j >= pairs) {
            const int d = p.R + (j - pairs) * 8;
            float f[8];
            unpack8(*reinterpret_cast<const uint4*>(src + d), f);
            put(d, f);
        } else if (kInter) {
            float f[8];
            unpack8(*reinterpret_cast<const uint4*>(src + j * 8), f);
            const float4 c = *reinterpret_cast<const float4*>(row.cs + j * 4);
            const float4 s = *reinterpret_cast<const float4*>(row.cs + half + j * 4);
            rotate(f[0], f[1], c.x, p.sign * s.x);
            rotate(f[2], f[3], c.y, p.sign * s.y);
            rotate(f[4], f[5], c.z, p.sign * s.z);
            rotate(f[6], f[7], c.w, p.sign * s.w);
            put(j * 8, f);
        } else {
            float a[8], b[8];
            unpack8(*reinterpret_cast<const uint4*>(src + j * 8), a);
            unpack8(*reinterpret_cast<const uint4*>(src + half + j * 8), b);
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
                const float4 c = *reinterpret_cast<const float4*>(row.cs + j * 8 + e);
                const float4 s = *reinterpret_cast<const float4*>(row.cs + half + j * 8 + e);
                rotate(a[e], b[e], c.x, p.sign * s.x);
                rotate(a[e + 1], b[e + 1], c.y, p.sign * s.y);
                rotate(a[e + 2], b[e + 2], c.z, p.sign * s.z);
                rotate(a[e + 3], b[e + 3], c.w, p.sign * s.w);
            }
            put(j * 8, a);
            put(half + j * 8, b);
        }
    }
}

// The same one pair (or one value past R, or of v) at a time, for widths and
// strides that 16-byte chunks do not divide.
template <bool kInter, bool kE4m3>
__global__ void __launch_bounds__(kRopeThreads)
rope_narrow_kernel(const __grid_constant__ RopeParams p) {
    pdl_wait_then_release();
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    if (t >= p.T) return;
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
        if (i >= nk) {
            if (row.slot < 0) break;
            const int h = (i - nk) / per_v, d = i - nk - h * per_v;
            cache(p.vpool, row.slot + h * p.c_head + d, bf(p.v[t * p.v_token + h * p.v_head + d]), p.v_scale);
            continue;
        }
        const bool is_k = i >= nq;
        if (is_k && row.slot < 0) break;
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
cudaError_t launch_t(const RopeParams& p, bool narrow, int items, cudaStream_t st) {
    // items over x in whole warps, several tokens in a CTA where one has few
    const int passes = (items + kRopeThreads - 1) / kRopeThreads;
    const int tx = ((items + passes - 1) / passes + 31) / 32 * 32;
    const int ty = kRopeThreads / tx > 1 ? kRopeThreads / tx : 1;
    const dim3 grid((unsigned)((p.T + ty - 1) / ty)), block((unsigned)tx, (unsigned)ty);
    return launch_pdl(narrow ? rope_narrow_kernel<kInter, kE4m3> : rope_kernel<kInter, kE4m3>, grid, block, 0, st,
                      p);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& a, bool interleaved, bool e4m3, cudaStream_t st) {
    RopeParams p = a;
    p.err = device_error_word();
    if (!p.err) return cudaErrorUnknown;
    auto aligned = [](const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15u) == 0; };
    const int unit = interleaved ? 8 : 16;
    bool wide = p.D % 8 == 0 && p.R % unit == 0;
    wide = wide && aligned(p.q) && aligned(p.y) && aligned(p.table) &&
           (p.q_token | p.q_head | p.y_token | p.y_head) % 8 == 0;
    wide = wide && aligned(p.k) && aligned(p.v) && (p.k_token | p.k_head | p.v_token | p.v_head) % 8 == 0;
    const int64_t pairs = wide ? p.R / (interleaved ? 8 : 16) : p.R / 2;
    const int64_t rest = wide ? (p.D - p.R) / 8 : p.D - p.R, vs = wide ? p.D / 8 : p.D;
    const int64_t items = p.Hq * (pairs + (p.in_place ? 0 : rest)) + p.Hkv * (pairs + rest + vs);
    if (items == 0) return cudaSuccess;
    if (interleaved)
        return e4m3 ? launch_t<true, true>(p, !wide, (int)items, st) : launch_t<true, false>(p, !wide, (int)items, st);
    return e4m3 ? launch_t<false, true>(p, !wide, (int)items, st) : launch_t<false, false>(p, !wide, (int)items, st);
}

cudaError_t launch_rope_table(const double* freq, int64_t max_pos, int64_t R, double mag, float* table,
                              cudaStream_t st) {
    const int64_t n = max_pos * (R / 2);
    return launch_pdl(rope_table_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, freq, max_pos,
                      (int)(R / 2), mag, table);
}

}  // namespace fp8rl
