// Rows of K and V between dense buffers and the cells of a paged cache: the store casts or quantises
// a row as it is written, the load reads it back.
//
// F8_E4M3 rows carry one power-of-two scale s = 2^e, the least with max|x| / s <= 448 over the row's finite
// values: x / s is then exact, and the value is rounded once, by the conversion to E4M3 (nearest, ties
// to even, saturating). The read back, s * q, is exact in float32, and in f16/bf16 whenever it is in
// range (E4M3 has 4 significant bits). A free scale (max|x| / 448) would use at most one more of the format's
// 18 binades and would add a rounding in each direction.
//
// Both kernels move every byte once. 8192 rows of K and V (8 heads of 128, bf16 values, E4M3 cache), stored and read back,
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
