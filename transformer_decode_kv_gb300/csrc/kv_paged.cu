// Rows of K and V between dense buffers and the cells of a paged cache: the store casts or quantises
// a row as it is written, the load reads it back.
//
// F8_E4M3 rows carry one power-of-two scale s = 2^e, the least with max|x| / s <= 448 over the row's finite
// values: x / s is then exact, and the value is rounded once, by the conversion to E4M3 (nearest, ties
// to even, saturating). The read back, s * q, is exact in float32, and in f16/bf16 whenever it is in
// range (E4M3 has 4 significant bits). A free scale (max|x| / 448) would use at most one more of the format's
// 18 binades and would add a rounding in each direction.
//
// F4_E2M1 rows carry such a scale too, the least with max|x| / s <= 2688 = 6 * 448, and an E4M3 scale b per 16 values: the
// nearest to max|x / s| / 6 of the block. A code is the E2M1 value nearest to x / (s b). Two quotients round before the
// conversion does, and neither moves a value over a border: a border is 6 m or m b, m a midpoint, of a few significant bits, so a
// float32 number that is not on it is a whole step of float32 away, and at the quotient's size that is more than half of one.
// The quotients by b are correctly rounded with r = 1 / b (rounded once per block) and an exact remainder: q0 = y r,
// q = q0 + (y - q0 b) r (P. Markstein's theorem, IBM J. Res. Dev. 34, 1990).
//
// F4_E2M1 has kernels of its own, whose threads hold a block of K and one of V: 8192 rows of K and V as below, stored and read
// back, take 19.5 us for 87 MB (4.4 TB/s; 12.8 us at the card's copy rate). Where the same rows come again and again, L2 holds
// them: 16.2 us, of which launches that do not overlap would make 20.8, and one row a thread, K and V apart, 27.2. Store 13.7 and
// load 9.4 under the profiler; the store issues instructions 56% of the time: seven per value, of which the quotient takes four.
//
// Both kernels of the other types move every byte once. 8192 rows of K and V (8 heads of 128, bf16 values, E4M3 cache), stored and read back,
// take 23.8 us for 101 MB (4.3 TB/s; 15.0 us at the card's copy rate): a step's few rows are bound by the launch,
// large calls by what a row costs beside its bytes (its place: two quotients and 64-bit addresses). So a thread
// holds 16 values of a row, HD / 16 neighbours the row, whose maximum they reduce with shuffles; with 8 values each the
// same took 35 us; two rows of 16 values a thread were 2 us slower, four 8 us. Heads follow each other, so a warp's
// accesses run over contiguous memory in the usual token-major layouts.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>
#include <cstdint>

#include "paged.h"

namespace llm {

namespace {

constexpr int kThr = 256;
constexpr int kVals = 16;                                   // values of a row per thread

template <int T>
__device__ __forceinline__ void load8(const void* base, int64_t elem, float* x) {
    if constexpr (T == W_F32) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + elem);
        const float4 a = p[0], b = p[1];
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
        const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + elem);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (T == W_F16) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                x[2 * i] = f.x; x[2 * i + 1] = f.y;
            } else {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
    }
}

template <int T>
__device__ __forceinline__ void store8(void* base, int64_t elem, const float* x) {
    if constexpr (T == W_F32) {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + elem);
        p[0] = make_float4(x[0], x[1], x[2], x[3]);
        p[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (T == W_F16) {
                const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + elem) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

template <int T>
__device__ __forceinline__ void load_vals(const void* base, int64_t elem, float* x) {
#pragma unroll
    for (int i = 0; i < kVals; i += 8) load8<T>(base, elem + i, x + i);
}
template <int T>
__device__ __forceinline__ void store_vals(void* base, int64_t elem, const float* x) {
#pragma unroll
    for (int i = 0; i < kVals; i += 8) store8<T>(base, elem + i, x + i);
}

// (lo, hi) -> two E4M3 bytes, nearest even, saturating to +-448 (NaN stays NaN)
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// four pairs of E2M1 codes (nearest even, saturating to +-6) and back
__device__ __forceinline__ uint32_t to_e2m1x8(const float* x) {
    uint32_t r;
    asm("{\n .reg .b8 b0, b1, b2, b3;\n cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n mov.b32 %0, {b0, b1, b2, b3};\n}\n"
        : "=r"(r) : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return r;
}
__device__ __forceinline__ void from_e2m1x8(uint32_t w, float s, float* x) {
    uint32_t h[4];
    asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n cvt.rn.f16x2.e2m1x2 %0, b0;\n cvt.rn.f16x2.e2m1x2 %1, b1;\n"
        " cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}\n" : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
        x[2 * i] = f.x * s;
        x[2 * i + 1] = f.y * s;
    }
}

// A thread's part of a row, and where the row goes; rows in the order token, K or V, head. cell -1: nothing to do.
struct RowAt {
    int64_t dense;                                          // first value of the thread's part in the buffers
    int32_t page, at, g, cell, part;
    bool v;
};

template <int HD>
__device__ __forceinline__ RowAt row_at(const KvRowsArgs& a) {
    constexpr uint32_t P = HD / kVals;
    const uint32_t cols = 2u * (uint32_t)a.kv.Hkv;
    const uint64_t row = (uint64_t)blockIdx.x * (kThr / P) + threadIdx.x / P;
    const uint64_t q = row >> 32 ? row / cols : (uint32_t)row / cols;   // (a 64-bit quotient costs as much as the rest)
    const uint32_t col = (uint32_t)(row - q * cols);
    const int64_t i = (int64_t)q;
    RowAt r;
    r.part = threadIdx.x % P;
    r.v = col >= (uint32_t)a.kv.Hkv;
    r.g = (int32_t)(r.v ? col - a.kv.Hkv : col);
    r.cell = i < a.n ? a.cell[i] : -1;
    r.dense = i * a.s_tok + r.g * a.s_head + r.part * kVals;
    const uint32_t ps = (uint32_t)a.kv.page_size, cell = (uint32_t)max(r.cell, 0);
    const uint32_t page = (ps & (ps - 1)) == 0 ? cell >> (__ffs(ps) - 1) : cell / ps;
    r.page = (int32_t)page;
    r.at = (int32_t)(cell - page * ps);
    if (page >= (uint32_t)a.kv.n_pages) {
        if (r.part == 0 && r.cell >= 0 && a.err) atomicOr(a.err, ERR_SLOT_RANGE);
        r.cell = -1;
    }
    return r;
}
__device__ __forceinline__ uint8_t* row_ptr(const PagedKv& kv, const RowAt& r) {
    return (r.v ? kv.v : kv.k) + (int64_t)r.page * kv.sb_page + r.at * kv.sb_cell + r.g * kv.sb_head;
}
__device__ __forceinline__ float* scale_ptr(const PagedKv& kv, const RowAt& r) {
    return (r.v ? kv.vs : kv.ks) + (int64_t)r.page * kv.ss_page + r.at * kv.ss_cell + r.g * kv.ss_head;
}

template <int HD, int CT, int T>
__global__ void __launch_bounds__(kThr) kv_store_kernel(KvRowsArgs a) {
    const RowAt r = row_at<HD>(a);
    float x[kVals] = {};
    if (r.cell >= 0) load_vals<T>(r.v ? a.v : a.k, r.dense, x);
    if constexpr (CT == W_F8) {
        auto row_max = [&](bool finite) {
            float m = 0.f;                                  // (fmaxf passes over NaN)
#pragma unroll
            for (int e = 0; e < kVals; ++e) {
                const float f = fabsf(x[e]);
                if (!finite || f <= FLT_MAX) m = fmaxf(m, f);
            }
#pragma unroll
            for (int o = HD / kVals / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            return m;
        };
        float amax = row_max(false);
        if (__any_sync(0xffffffffu, amax > FLT_MAX)) amax = row_max(true);
        if (r.cell < 0) return;
        // 448 = 1.75 * 2^8: e = exponent(amax) - 8, one more above a mantissa of 1.75
        const uint32_t b = __float_as_uint(amax);
        int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u);
        e = amax == 0.f ? 0 : max(e, -126);
        const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
        uint32_t w[kVals / 4];
#pragma unroll
        for (int i = 0; i < kVals / 4; ++i)
            w[i] = to_e4m3x2(x[4 * i] * inv, x[4 * i + 1] * inv) | to_e4m3x2(x[4 * i + 2] * inv, x[4 * i + 3] * inv) << 16;
        *reinterpret_cast<uint4*>(row_ptr(a.kv, r) + r.part * kVals) = make_uint4(w[0], w[1], w[2], w[3]);
        if (r.part == 0) *scale_ptr(a.kv, r) = __uint_as_float((uint32_t)(e + 127) << 23);
    } else {
        if (r.cell >= 0) store_vals<CT>(row_ptr(a.kv, r), r.part * kVals, x);
    }
}

template <int HD, int CT, int T>
__global__ void __launch_bounds__(kThr) kv_load_kernel(KvRowsArgs a) {
    const RowAt r = row_at<HD>(a);
    if (r.cell < 0) return;
    float x[kVals];
    if constexpr (CT == W_F8) {
        const uint4 u = *reinterpret_cast<const uint4*>(row_ptr(a.kv, r) + r.part * kVals);
        const float s = *scale_ptr(a.kv, r);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f0 = from_e4m3x2(w[i] & 0xffffu), f1 = from_e4m3x2(w[i] >> 16);
            x[4 * i] = f0.x * s;
            x[4 * i + 1] = f0.y * s;
            x[4 * i + 2] = f1.x * s;
            x[4 * i + 3] = f1.y * s;
        }
    } else {
        load_vals<CT>(row_ptr(a.kv, r), r.part * kVals, x);
    }
    store_vals<T>(r.v ? a.v : a.k, r.dense, x);
}

// ---- F4_E2M1: a thread holds 16 values of K and the same of V, a block each; where they go is worked out once for both.
struct At4 { int64_t dense, row, blk, scale; int part; bool there; };

template <int HD>
__device__ __forceinline__ At4 at4(const KvRowsArgs& a) {
    constexpr uint32_t P = HD / kVals;
    const uint32_t Hkv = (uint32_t)a.kv.Hkv, ps = (uint32_t)a.kv.page_size;
    const uint64_t row = (uint64_t)blockIdx.x * (kThr / P) + threadIdx.x / P;   // (token, head)
    const uint64_t i = (Hkv & (Hkv - 1)) == 0 ? row >> (__ffs(Hkv) - 1) : row >> 32 ? row / Hkv : (uint32_t)row / Hkv;
    const uint32_t g = (uint32_t)(row - i * Hkv);
    At4 r;
    r.part = threadIdx.x % P;
    const int cell = i < (uint64_t)a.n ? a.cell[i] : -1;
    const uint32_t c = (uint32_t)max(cell, 0), page = (ps & (ps - 1)) == 0 ? c >> (__ffs(ps) - 1) : c / ps, at = c - page * ps;
    r.there = cell >= 0 && page < (uint32_t)a.kv.n_pages;
    if (r.part == 0 && cell >= 0 && !r.there && a.err) atomicOr(a.err, ERR_SLOT_RANGE);
    r.dense = (int64_t)i * a.s_tok + g * a.s_head + r.part * kVals;
    r.row = page * a.kv.sb_page + at * a.kv.sb_cell + g * a.kv.sb_head + r.part * (kVals / 2);
    r.blk = page * a.kv.sk_page + at * a.kv.sk_cell + g * a.kv.sk_head + r.part;
    r.scale = page * a.kv.ss_page + at * a.kv.ss_cell + g * a.kv.ss_head;
    return r;
}
// A thread's 16 values of the dense rows: whole 32-byte sectors at once where rows lie on their boundaries (two half
// sectors 16 bytes apart in two instructions cost the load 2 us of 13 for 8192 rows of 8 heads of 128).
template <int T>
__device__ __forceinline__ void load_dense(const void* base, int64_t elem, bool wide, float* x) {
    if (!wide) {
        load_vals<T>(base, elem, x);
        return;
    }
#pragma unroll
    for (int i = 0; i < (T == W_F32 ? 2 : 1); ++i) {
        uint32_t w[8];
        const uint8_t* p = static_cast<const uint8_t*>(base) + elem * (T == W_F32 ? 4 : 2) + 32 * i;
        asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7]) : "l"(p));
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if constexpr (T == W_F32) {
                x[8 * i + j] = __uint_as_float(w[j]);
            } else if constexpr (T == W_F16) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
                x[2 * j] = f.x; x[2 * j + 1] = f.y;
            } else {
                x[2 * j] = __uint_as_float(w[j] << 16);
                x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
            }
        }
    }
}
template <int T>
__device__ __forceinline__ void store_dense(void* base, int64_t elem, bool wide, const float* x) {
    if (!wide) {
        store_vals<T>(base, elem, x);
        return;
    }
#pragma unroll
    for (int i = 0; i < (T == W_F32 ? 2 : 1); ++i) {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if constexpr (T == W_F32) {
                w[j] = __float_as_uint(x[8 * i + j]);
            } else if constexpr (T == W_F16) {
                const __half2 h = __floats2half2_rn(x[2 * j], x[2 * j + 1]);
                w[j] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
                w[j] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
        uint8_t* p = static_cast<uint8_t*>(base) + elem * (T == W_F32 ? 4 : 2) + 32 * i;
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                     "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]) : "memory");
    }
}
// the largest of three magnitudes, NaN if one is
__device__ __forceinline__ float max3_abs(float x, float y, float z) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
    return r;
}

template <int HD, int T>
__global__ void __launch_bounds__(kThr) kv_store4_kernel(KvRowsArgs a) {
    // (launched early: nothing is read or written before the kernel in front has ended)
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const At4 r = at4<HD>(a);
    float x[2][kVals] = {};
    if (r.there) {
        load_dense<T>(a.k, r.dense, a.wide, x[0]);
        load_dense<T>(a.v, r.dense, a.wide, x[1]);
    }
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        float bmax = 0.f;                                   // of the block
#pragma unroll
        for (int e = 0; e < kVals; e += 2) bmax = max3_abs(bmax, x[v][e], x[v][e + 1]);
        bool nan = false;
        const bool odd = __any_sync(0xffffffffu, !(bmax <= FLT_MAX));
        if (odd) {                                          // NaN or infinities: the largest of the others
            bmax = 0.f;
#pragma unroll
            for (int e = 0; e < kVals; ++e) {
                const float f = fabsf(x[v][e]);
                nan = nan || f != f;
                if (f <= FLT_MAX) bmax = fmaxf(bmax, f);
            }
        }
        float amax = bmax;
#pragma unroll
        for (int o = HD / kVals / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        // 2688 = 1.3125 * 2^11: e = exponent(amax) - 11, one more above that mantissa
        const uint32_t bits = __float_as_uint(amax);
        int e = (int)(bits >> 23) - 127 - 11 + ((bits & 0x7fffffu) > 0x280000u);
        e = amax == 0.f ? 0 : max(e, -126);
        const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
        uint32_t bc = to_e4m3x2(fmaxf(__fdiv_rn(bmax * inv, 6.f), 0x1p-9f), 0.f);
        const float b = from_e4m3x2(bc).x, rb = __frcp_rn(b);
        if (odd) {                                          // infinities: a number that is above 6 b
            const float top = e + 12 > 127 ? FLT_MAX : __uint_as_float((uint32_t)(e + 12 + 127) << 23);
#pragma unroll
            for (int i = 0; i < kVals; ++i) x[v][i] = fminf(fmaxf(x[v][i], -top), top);
        }
        // The remainder is exact whatever its rounding mode; downwards, that of -0 is -0, and so the quotient keeps its sign.
#pragma unroll
        for (int i = 0; i < kVals; ++i) {
            const float y = x[v][i] * inv, q0 = y * rb;
            x[v][i] = fmaf(__fmaf_rd(-q0, b, y), rb, q0);
        }
        if (nan) bc = 0x7fu;                                // there is no code for NaN: the block is
        if (r.there) {
            *reinterpret_cast<uint2*>((v ? a.kv.v : a.kv.k) + r.row) = make_uint2(to_e2m1x8(x[v]), to_e2m1x8(x[v] + 8));
            (v ? a.kv.vb : a.kv.kb)[r.blk] = (uint8_t)bc;
            if (r.part == 0) (v ? a.kv.vs : a.kv.ks)[r.scale] = __uint_as_float((uint32_t)(e + 127) << 23);
        }
    }
}

template <int HD, int T>
__global__ void __launch_bounds__(kThr) kv_load4_kernel(KvRowsArgs a) {
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const At4 r = at4<HD>(a);
    if (!r.there) return;
    uint2 u[2];
    uint32_t b[2];
    float s[2];
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        u[v] = *reinterpret_cast<const uint2*>((v ? a.kv.v : a.kv.k) + r.row);
        b[v] = (v ? a.kv.vb : a.kv.kb)[r.blk];
        s[v] = (v ? a.kv.vs : a.kv.ks)[r.scale];
    }
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        // (Both products are exact: code and block scale make a multiple of 2^-10 of six significant bits at most, and s, a power of two of
        // 2^-126 or more, leaves a multiple of 2^-136, which float32 holds below its normal range too. The one rounding is that to
        // the rows' type.)
        float x[kVals];
        const float bs = from_e4m3x2(b[v]).x;
        from_e2m1x8(u[v].x, bs, x);
        from_e2m1x8(u[v].y, bs, x + 8);
#pragma unroll
        for (int i = 0; i < kVals; ++i) x[i] *= s[v];
        store_dense<T>(v ? a.v : a.k, r.dense, a.wide, x);
    }
}

template <int HD>
bool go4(KvRowsArgs a, bool store, cudaStream_t st) {
    const int64_t es = a.type == W_F32 ? 4 : 2;
    a.wide = ((reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v)) & 31) == 0 && ((a.s_tok | a.s_head) * es) % 32 == 0;
    constexpr int64_t per = kThr * kVals / HD;
    const int64_t blocks = ((int64_t)a.n * a.kv.Hkv + per - 1) / per;
    if (blocks > 0x7fffffff) return false;
    auto launch = [&](void (*kernel)(KvRowsArgs)) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)blocks);
        cfg.blockDim = dim3(kThr);
        cfg.stream = st;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess;
    };
    switch (a.type) {
        case W_F32: return launch(store ? kv_store4_kernel<HD, W_F32> : kv_load4_kernel<HD, W_F32>);
        case W_F16: return launch(store ? kv_store4_kernel<HD, W_F16> : kv_load4_kernel<HD, W_F16>);
        case W_BF16: return launch(store ? kv_store4_kernel<HD, W_BF16> : kv_load4_kernel<HD, W_BF16>);
    }
    return false;
}

template <int HD, int CT, int T>
bool go(const KvRowsArgs& a, bool store, cudaStream_t st) {
    constexpr int64_t per = kThr * kVals / HD;
    const int64_t blocks = ((int64_t)a.n * a.kv.Hkv * 2 + per - 1) / per;
    if (blocks > 0x7fffffff) return false;
    if (store) kv_store_kernel<HD, CT, T><<<(unsigned)blocks, kThr, 0, st>>>(a);
    else kv_load_kernel<HD, CT, T><<<(unsigned)blocks, kThr, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess;
}
template <int HD, int CT>
bool go_t(const KvRowsArgs& a, bool store, cudaStream_t st) {
    switch (a.type) {
        case W_F32: return go<HD, CT, W_F32>(a, store, st);
        case W_F16: return go<HD, CT, W_F16>(a, store, st);
        case W_BF16: return go<HD, CT, W_BF16>(a, store, st);
    }
    return false;
}
template <int HD>
bool go_ct(const KvRowsArgs& a, bool store, cudaStream_t st) {
    switch (a.kv.type) {
        case W_F16: return go_t<HD, W_F16>(a, store, st);
        case W_BF16: return go_t<HD, W_BF16>(a, store, st);
        case W_F8: return go_t<HD, W_F8>(a, store, st);
        case W_F4: return go4<HD>(a, store, st);
    }
    return false;
}
bool go_hd(const KvRowsArgs& a, bool store, cudaStream_t st) {
    if (a.n == 0) return true;
    switch (a.kv.hd) {
        case 32: return go_ct<32>(a, store, st);
        case 64: return go_ct<64>(a, store, st);
        case 128: return go_ct<128>(a, store, st);
    }
    return false;
}

}  // namespace

bool launch_kv_rows_store(const KvRowsArgs& a, cudaStream_t st) { return go_hd(a, true, st); }
bool launch_kv_rows_load(const KvRowsArgs& a, cudaStream_t st) { return go_hd(a, false, st); }

}  // namespace llm
