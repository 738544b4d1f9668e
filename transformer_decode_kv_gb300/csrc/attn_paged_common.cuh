// Device pieces of the attention over a paged cache that both tile forms share: where a key's row
// lies, which keys a row may see, the output store, the careful recomputation of a unit whose
// operands are not finite, and the merge of a tile's partial results.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "paged.h"

namespace llm {
namespace pattn {

// 2^x by the hardware approximation (a few ulp of float32; -inf gives 0)
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t e4m3x2_to_h2(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    return h;
}

__device__ __forceinline__ AttnUnit load_unit(const AttnUnit* u) {
    AttnUnit r;
    const int4* s = reinterpret_cast<const int4*>(u);
    int4* d = reinterpret_cast<int4*>(&r);
    d[0] = s[0]; d[1] = s[1]; d[2] = s[2]; d[3] = s[3];
    return r;
}

// four E4M3 codes to two f16 pairs (exact)
__device__ __forceinline__ void e4m3x4_to_h2(uint32_t four, uint32_t& lo, uint32_t& hi) {
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}\n"
        : "=r"(lo), "=r"(hi) : "r"(four));
}

// A key of a unit: its cell as byte and scale offsets (without the head) and number, its position. off < 0: a cell
// outside the cache.
struct KeyAt { int64_t off, soff; int pos, cell; };

__device__ __forceinline__ KeyAt key_at(const AttnPagedArgs& a, const AttnUnit& u, int v) {
    const int j = v < u.n_sink_keys ? v : v - u.n_sink_keys + u.key_lo;
    const int ps = a.kv.page_size;
    int pg = j, at = 0;
    if (ps != 1) {
        pg = (ps & (ps - 1)) == 0 ? j >> (__ffs(ps) - 1) : j / ps;
        at = j - pg * ps;
    }
    const int page = a.table[u.table + pg];
    KeyAt k;
    k.pos = a.key_pos ? a.key_pos[u.table + j] : j;
    k.cell = page * ps + at;
    if ((unsigned)page >= (unsigned)a.kv.n_pages) {
        if (a.err) atomicOr(a.err, ERR_SLOT_RANGE);
        k.off = k.soff = -1;
        k.pos = INT_MAX;
    } else {
        k.off = (int64_t)page * a.kv.sb_page + (int64_t)at * a.kv.sb_cell;
        k.soff = (int64_t)page * a.kv.ss_page + (int64_t)at * a.kv.ss_cell;
    }
    return k;
}

// The token of a sequence's row (token * G + head) and its position.
__device__ __forceinline__ int row_token(const AttnPagedArgs& a, const AttnUnit& u, int row) {
    const int t = u.tok0 + row / a.G;
    return a.perm ? a.perm[t] : t;
}
__device__ __forceinline__ int row_pos(const AttnPagedArgs& a, const AttnUnit& u, int row, int token) {
    return a.tok_pos ? a.tok_pos[token] : u.p0 + row / a.G;
}
// The last position the window hides from a row at position p (INT_MIN: none).
__device__ __forceinline__ int hidden_below(const AttnPagedArgs& a, int p) {
    if (a.window == 0) return INT_MIN;
    const int64_t h = (int64_t)p - a.window;
    return h < INT_MIN ? INT_MIN : (int)h;
}
__device__ __forceinline__ bool sees(int kp, int p, int hidden, int n_sink) {
    return kp <= p && (kp > hidden || kp < n_sink);
}

// What a row without any weight gives: zeros where it sees no key (its position is negative: new tokens that have no
// cached row; any other sees itself), else 0 / 0, its scores being -inf alone.
__device__ __forceinline__ float weightless(const AttnPagedArgs& a, const AttnUnit& u, int row, int token) {
    return row_pos(a, u, row, token) < 0 ? 0.f : NAN;
}

__device__ __forceinline__ float load_q(const AttnPagedArgs& a, int64_t i) {
    if (a.q_type == W_F32) return static_cast<const float*>(a.q)[i];
    if (a.q_type == W_F16) return __half2float(static_cast<const __half*>(a.q)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[i]);
}

__device__ __forceinline__ void store_out1(const AttnPagedArgs& a, int64_t i, float v) {
    if (a.out_kind == AO_F32) {
        static_cast<float*>(a.out)[i] = v;
    } else if (a.out_kind == AO_F16) {
        static_cast<__half*>(a.out)[i] = __float2half_rn(v);
    } else {
        const __nv_bfloat16 hi = __float2bfloat16_rn(v);
        static_cast<__nv_bfloat16*>(a.out)[i] = hi;
        if (a.out_kind == AO_BF16_PAIR)
            static_cast<__nv_bfloat16*>(a.out_lo)[i] = __float2bfloat16_rn(v - __bfloat162float(hi));
    }
}
// Four consecutive values (element i a multiple of 4, rows aligned to 16 bytes).
__device__ __forceinline__ void store_out4(const AttnPagedArgs& a, int64_t i, const float* v) {
    if (a.out_kind == AO_F32) {
        *reinterpret_cast<float4*>(static_cast<float*>(a.out) + i) = make_float4(v[0], v[1], v[2], v[3]);
    } else if (a.out_kind == AO_F16) {
        const __half2 x = __floats2half2_rn(v[0], v[1]), y = __floats2half2_rn(v[2], v[3]);
        *reinterpret_cast<uint2*>(static_cast<__half*>(a.out) + i) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
    } else if (a.out_kind == AO_BF16) {
        const __nv_bfloat162 x = __floats2bfloat162_rn(v[0], v[1]), y = __floats2bfloat162_rn(v[2], v[3]);
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + i) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) store_out1(a, i + j, v[j]);
    }
}

// 32 bytes at once (a whole sector per lane), 32-byte aligned
__device__ __forceinline__ void store32b(void* p, const uint32_t* w) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]) : "memory");
}
// 32 consecutive values; whole sectors where the output's rows allow it (a.out32)
__device__ __forceinline__ void store_out32(const AttnPagedArgs& a, int64_t i, const float* v) {
    if (a.out32 && (a.out_kind == AO_F16 || a.out_kind == AO_BF16)) {
        uint32_t w[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            if (a.out_kind == AO_F16) {
                const __half2 h = __floats2half2_rn(v[2 * j], v[2 * j + 1]);
                w[j] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
                w[j] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
        store32b(static_cast<uint16_t*>(a.out) + i, w);
        store32b(static_cast<uint16_t*>(a.out) + i + 16, w + 8);
    } else {
#pragma unroll
        for (int j = 0; j < 32; j += 4) store_out4(a, i + j, v + j);
    }
}

// One value of a cached row as float32.
__device__ __forceinline__ float kv_value(const AttnPagedArgs& a, const uint8_t* row, float s, int d) {
    if (a.kv.type == W_F16) return __half2float(reinterpret_cast<const __half*>(row)[d]);
    if (a.kv.type == W_BF16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(row)[d]);
    const uint32_t h = e4m3x2_to_h2(row[d]);
    return s * __half2float(__ushort_as_half((unsigned short)(h & 0xffffu)));
}

// One row of a unit in float32, a warp per row, key by key: a key the row does not see is left out
// altogether, so what it holds cannot reach the row. The tile kernels multiply hidden keys by zero,
// which is right for finite values only (0 * NaN is NaN); a unit whose result is not finite is
// redone this way. o: HD / 32 values per lane, dims lane * HD / 32 ..
template <int HD>
__device__ __noinline__ void careful_row(const AttnPagedArgs& a, const AttnUnit& u, int kvh, int row, float* o,
                                         float& m, float& l) {
    constexpr int D = HD / 32;
    const int lane = threadIdx.x & 31;
    const int tok = row_token(a, u, row), p = row_pos(a, u, row, tok), hid = hidden_below(a, p);
    float q[D];
#pragma unroll
    for (int d = 0; d < D; ++d) {
        q[d] = load_q(a, (int64_t)tok * a.q_tok + (int64_t)(kvh * a.G + row % a.G) * a.q_head + lane * D + d);
        o[d] = 0.f;
    }
    m = -INFINITY;
    l = 0.f;
    for (int v = u.v0; v < u.v1; ++v) {
        const KeyAt k = key_at(a, u, v);
        if (k.off < 0 || !sees(k.pos, p, hid, a.n_sink)) continue;
        const uint8_t* kr = a.kv.k + k.off + kvh * a.kv.sb_head;
        const uint8_t* vr = a.kv.v + k.off + kvh * a.kv.sb_head;
        float ks = 1.f, vs = 1.f;
        if (a.kv.type == W_F8) {
            ks = a.kv.ks[k.soff + kvh * a.kv.ss_head];
            vs = a.kv.vs[k.soff + kvh * a.kv.ss_head];
        }
        float s = 0.f;
#pragma unroll
        for (int d = 0; d < D; ++d) s = fmaf(q[d], kv_value(a, kr, ks, lane * D + d), s);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        s *= a.scale_log2;
        const float mn = fmaxf(m, s);
        // (a score of -inf has no weight, whatever has been seen; one of NaN passes into the sum)
        const float f = m == mn ? 1.f : exp2f(m - mn), e = s == -INFINITY ? 0.f : exp2f(s - mn);
        l = l * f + e;
#pragma unroll
        for (int d = 0; d < D; ++d) o[d] = o[d] * f + e * kv_value(a, vr, vs, lane * D + d);
        m = mn;
    }
}

// What a part with (reference, sum) x counts under the reference M. A part without a visible key has nothing to add
// (its reference is -inf); NaN sums pass.
__device__ __forceinline__ float part_factor(float2 x, float M) {
    if (x.x == -INFINITY && x.y == 0.f) return 0.f;
    return x.x == M ? 1.f : exp2f(x.x - M);
}

// Merge the partial results of rows r0 .. r0 + NR - 1 (those below u.n_row) of a cut tile into the output, by one warp;
// in the units' order, so the result does not depend on which of them was last. rows: the tile form's rows. A
// lane weighs up to one unit in 32 at a time (weight exp2(m - M) against the largest reference M), then the warp
// adds the units' rows, HD / 32 neighbouring values per lane; NR rows keep NR times as many loads under way.
template <int HD, int NR>
__device__ void merge_rows(const AttnPagedArgs& a, const float* part_o, const float2* part_ml, const AttnUnit& u, int rows,
                           int r0) {
    constexpr int D = HD / 32;
    const int lane = threadIdx.x & 31;
    float M[NR], L[NR], o[NR][D];
    const float2* ml = part_ml + (int64_t)u.part * rows + r0;
#pragma unroll
    for (int k = 0; k < NR; ++k) {
        M[k] = -INFINITY;
        L[k] = 0.f;
#pragma unroll
        for (int d = 0; d < D; ++d) o[k][d] = 0.f;
        for (int c = lane; c < u.n_chunk; c += 32)
            if (r0 + k < u.n_row) M[k] = fmaxf(M[k], __ldcg(&ml[(int64_t)c * rows + k]).x);
    }
#pragma unroll
    for (int k = 0; k < NR; ++k)
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) M[k] = fmaxf(M[k], __shfl_xor_sync(0xffffffffu, M[k], s));
    for (int c0 = 0; c0 < u.n_chunk; c0 += 32) {
        float f[NR];
#pragma unroll
        for (int k = 0; k < NR; ++k) {
            f[k] = 0.f;
            if (c0 + lane < u.n_chunk && r0 + k < u.n_row) {
                const float2 x = __ldcg(&ml[(int64_t)(c0 + lane) * rows + k]);
                f[k] = part_factor(x, M[k]);
                L[k] += f[k] * x.y;
            }
        }
        const int n = min(32, u.n_chunk - c0);
        const float* p = part_o + ((int64_t)(u.part + c0) * rows + r0) * HD + lane * D;
#pragma unroll 2
        for (int c = 0; c < n; ++c)
#pragma unroll
            for (int k = 0; k < NR; ++k) {
                const float fc = __shfl_sync(0xffffffffu, f[k], c);
                const float* q = p + ((int64_t)c * rows + k) * HD;
                if (fc == 0.f) continue;                    // (also rows that are not the tile's)
                if constexpr (D == 4) {
                    const float4 w = __ldcg(reinterpret_cast<const float4*>(q));
                    o[k][0] += fc * w.x; o[k][1] += fc * w.y; o[k][2] += fc * w.z; o[k][3] += fc * w.w;
                } else if constexpr (D == 2) {
                    const float2 w = __ldcg(reinterpret_cast<const float2*>(q));
                    o[k][0] += fc * w.x; o[k][1] += fc * w.y;
                } else {
                    o[k][0] += fc * __ldcg(q);
                }
            }
    }
#pragma unroll
    for (int k = 0; k < NR; ++k) {
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) L[k] += __shfl_xor_sync(0xffffffffu, L[k], s);
        if (r0 + k >= u.n_row) continue;
        const int row = u.row0 + r0 + k, tok = row_token(a, u, row);
        const float inv = 1.f / L[k], none = L[k] == 0.f ? weightless(a, u, row, tok) : 0.f;
        const int64_t at = (int64_t)tok * a.o_tok + (int64_t)(u.head * a.G + row % a.G) * a.o_head + lane * D;
#pragma unroll
        for (int d = 0; d < D; ++d) o[k][d] = L[k] == 0.f ? none : o[k][d] * inv;
        if constexpr (D == 4) store_out4(a, at, o[k]);
        else
#pragma unroll
            for (int d = 0; d < D; ++d) store_out1(a, at + d, o[k][d]);
    }
}

// Count a unit of a cut tile as finished, by one thread after a barrier behind the writes of its partial results
// (each writer's followed by a __threadfence); true for the last one, whose threads may read all of them after
// another barrier.
__device__ __forceinline__ bool count_unit(const AttnPagedArgs& a, const AttnUnit& u) {
    __threadfence();
    int* t = a.tickets + u.ticket;
    const bool last = atomicAdd(t, 1) + 1 == u.n_chunk;
    if (last) *t = 0;
    __threadfence();
    return last;
}

// The plan was made for other forms than this launch runs: nothing is computed, the caller learns of it.
__device__ __forceinline__ bool form_missing(const AttnPagedArgs& a) {
    if ((a.hdr[PH_FORM] & ~a.form) == 0) return false;
    if (blockIdx.x == 0 && threadIdx.x == 0 && a.err) atomicOr(a.err, ERR_PLAN_FORM);
    return true;
}

}  // namespace pattn
}  // namespace llm
