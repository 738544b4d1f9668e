// Rows of K and V between dense buffers and the cells of a paged cache: the store casts or quantises
// a row as it is written, the load reads it back.
//
// F8_E4M3 rows carry one power-of-two scale s = 2^e, the least with max|x| / s <= 448 over the row's finite
// values: x / s is then exact, and the value is rounded once, by the conversion to E4M3 (nearest, ties
// to even, saturating). The read back, s * q, is exact in float32, and in f16/bf16 whenever it is in
// range (E4M3 has 4 significant bits). A free scale (max|x| / 448) would use at most one more of the format's
// 18 binades and would add a rounding in each direction.
//
// Both kernels move every byte once and are bound by HBM (by the launch at a few rows). A thread holds 8
// consecutive values of a row (one 16-byte access of a 2-byte type), HD / 8 neighbouring threads hold
// the row and reduce its maximum with shuffles, and heads follow each other, so a warp's accesses
// run over contiguous memory in the usual token-major layouts.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>
#include <cstdint>

#include "paged.h"

namespace llm {

namespace {

constexpr int kThr = 256;
constexpr int kRows = 4;                                    // rows a thread has in flight

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

// Rows in the order token, K or V, head: a block's threads take kRows times kThr * 8 / HD consecutive ones. A row's
// place, found once per row; cell -1 where there is nothing to do.
struct RowAt {
    int64_t dense;                                          // first value of the row in the buffers
    int64_t page;
    int32_t at, g, cell;
    bool v;
};

template <int HD>
__device__ __forceinline__ void rows_at(const KvRowsArgs& a, RowAt* r) {
    constexpr int N = kThr * 8 / HD;                        // rows of a block at a time
    const uint32_t cols = 2u * (uint32_t)a.kv.Hkv, part = threadIdx.x % (HD / 8);
    const uint64_t first = (uint64_t)blockIdx.x * (N * kRows);
    const uint64_t i0 = first / cols;
    const uint32_t c0 = (uint32_t)(first - i0 * cols) + threadIdx.x / (HD / 8);
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
        const uint32_t c = c0 + j * N, di = c / cols, col = c - di * cols;
        const int64_t i = (int64_t)i0 + di;
        r[j].v = col >= (uint32_t)a.kv.Hkv;
        r[j].g = (int32_t)(r[j].v ? col - a.kv.Hkv : col);
        r[j].cell = i < a.n ? a.cell[i] : -1;
        r[j].dense = i * a.s_tok + r[j].g * a.s_head + part * 8;
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
        const uint32_t page = (uint32_t)max(r[j].cell, 0) / (uint32_t)a.kv.page_size;
        r[j].page = page;
        r[j].at = (int32_t)((uint32_t)max(r[j].cell, 0) - page * (uint32_t)a.kv.page_size);
        if (page >= (uint32_t)a.kv.n_pages) {
            if (part == 0 && r[j].cell >= 0 && a.err) atomicOr(a.err, ERR_SLOT_RANGE);
            r[j].cell = -1;
        }
    }
}
__device__ __forceinline__ uint8_t* row_ptr(const PagedKv& kv, const RowAt& r) {
    return (r.v ? kv.v : kv.k) + r.page * kv.sb_page + r.at * kv.sb_cell + r.g * kv.sb_head;
}
__device__ __forceinline__ float* scale_ptr(const PagedKv& kv, const RowAt& r) {
    return (r.v ? kv.vs : kv.ks) + r.page * kv.ss_page + r.at * kv.ss_cell + r.g * kv.ss_head;
}

template <int HD, int CT, int T>
__global__ void __launch_bounds__(kThr) kv_store_kernel(KvRowsArgs a) {
    constexpr int P = HD / 8;
    const int part = threadIdx.x % P;
    RowAt r[kRows];
    rows_at<HD>(a, r);
    float x[kRows][8];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
        if (r[j].cell >= 0) {
            load8<T>(r[j].v ? a.v : a.k, r[j].dense, x[j]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[j][e] = 0.f;
        }
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
        if constexpr (CT == W_F8) {
            float amax = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float f = fabsf(x[j][e]);
                if (f <= FLT_MAX) amax = fmaxf(amax, f);
            }
#pragma unroll
            for (int o = P / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            if (r[j].cell < 0) continue;
            // 448 = 1.75 * 2^8: e = exponent(amax) - 8, one more above a mantissa of 1.75
            const uint32_t b = __float_as_uint(amax);
            int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u);
            e = amax == 0.f ? 0 : max(e, -126);
            const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = to_e4m3x2(x[j][2 * i] * inv, x[j][2 * i + 1] * inv);
            *reinterpret_cast<uint2*>(row_ptr(a.kv, r[j]) + part * 8) = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
            if (part == 0) *scale_ptr(a.kv, r[j]) = __uint_as_float((uint32_t)(e + 127) << 23);
        } else {
            if (r[j].cell >= 0) store8<CT>(row_ptr(a.kv, r[j]), part * 8, x[j]);
        }
    }
}

template <int HD, int CT, int T>
__global__ void __launch_bounds__(kThr) kv_load_kernel(KvRowsArgs a) {
    const int part = threadIdx.x % (HD / 8);
    RowAt r[kRows];
    rows_at<HD>(a, r);
    float x[kRows][8];
    if constexpr (CT == W_F8) {
        uint2 u[kRows];
        float s[kRows];
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
            if (r[j].cell < 0) continue;
            u[j] = *reinterpret_cast<const uint2*>(row_ptr(a.kv, r[j]) + part * 8);
            s[j] = *scale_ptr(a.kv, r[j]);
        }
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
            if (r[j].cell < 0) continue;
            const uint32_t w[4] = {u[j].x & 0xffffu, u[j].x >> 16, u[j].y & 0xffffu, u[j].y >> 16};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = from_e4m3x2(w[i]);
                x[j][2 * i] = f.x * s[j];
                x[j][2 * i + 1] = f.y * s[j];
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < kRows; ++j)
            if (r[j].cell >= 0) load8<CT>(row_ptr(a.kv, r[j]), part * 8, x[j]);
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j)
        if (r[j].cell >= 0) store8<T>(r[j].v ? a.v : a.k, r[j].dense, x[j]);
}

template <int HD, int CT, int T>
bool go(const KvRowsArgs& a, bool store, cudaStream_t st) {
    constexpr int64_t per = kThr * 8 / HD * kRows;
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
