// Attention of new tokens over a paged cache, 16-row tiles: out = softmax(scale q K^T, masked) V for the
// (token, query head) pairs that share a KV head, an optional sliding window and sink keys.
//
// A warp owns 16 rows and walks blocks of 16 keys; the four warps of a CTA take every fourth block
// of the unit's keys and merge their (maximum, sum, output) at the end, the units of a tile
// through partial results in global memory (the last to finish merges). Per block and warp:
//   S = Q K^T    mma.sync m16n8k16, two 8-key column tiles, float32 sums
//   softmax      p = 2^(s - m) with a reference m and the sum l per row in float32, in the log2 domain. m is 6
//                below a row maximum and raised lazily, when p would pass 2^14: O is rarely rescaled, the
//                largest p is between 2^6 and 2^14, and f16's subnormal steps start 2^20 below it
//   O += P V     mma.sync, the score fragments are the A operand as they stand
// This form is for few rows per KV head (single tokens, short chunks), where reading K and V once is the
// bound. A contraction may be taken in any order, so a thread's 16 bytes of a key row simply are the dims its
// B fragments hold (Q is loaded in the same order), and a thread's values of four keys become fragments
// by byte permutes (f16/bf16: pairs of keys; E4M3: 4 x 4 bytes, then the conversion to f16, which is
// exact). Every thread copies just the bytes it will use, asynchronously, into its own places of a ring in shared
// memory (no bank conflicts, no barrier), as many blocks ahead as two CTAs per SM have room for: 3 blocks
// of 8 KB per warp of an f16 cache with head_dim 128, 6 of an E4M3 one.
//
// Precision: products of f16 (bf16) terms with float32 sums. F16 activations and caches enter as they
// are. BF16 or F32 activations over an f16-typed product are scaled per row by a power of two (taken out of the
// scores again), so that no value leaves f16's range; F32 ones enter as two f16 terms (22 bits). P is
// rounded to f16 (relative 2^-11 / 2) where activations are f16; for F32 activations and for bf16 products
// it enters as two terms, so its rounding (2^-9 / 2 for bf16) does not show. An E4M3 row's scale multiplies
// the score (K) or p (V, relative to the largest scale seen so far by the warp, a power of two, so exact
// down to f16's subnormals).
#include "attn_paged_common.cuh"

#include <algorithm>

namespace llm {

namespace {

using namespace pattn;

constexpr int kWarps = 4;
constexpr int kThr = 32 * kWarps;

template <bool BF>
__device__ __forceinline__ void mma(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
    if constexpr (BF)
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// (lo, hi) as two f16 or bf16; with `rest` the rounding errors as a second pair
template <bool BF>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
    if constexpr (BF) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __half2 h = __floats2half2_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}
template <bool BF>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if constexpr (BF) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    else return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <bool BF>
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
    hi = pack2<BF>(x, y);
    const float2 f = unpack2<BF>(hi);
    lo = pack2<BF>(x - f.x, y - f.y);
}

// N words (N = 1, 2, 4) from global memory to this thread's place in shared memory, asynchronously; zeros
// where the key is not read
template <int N>
__device__ __forceinline__ void fetch(uint32_t dst, const uint8_t* src, bool ok) {
    if constexpr (N == 4)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
    else if constexpr (N == 2)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(ok ? 8 : 0) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(ok ? 4 : 0) : "memory");
}
template <int N>
__device__ __forceinline__ void take(uint32_t* d, const uint8_t* p) {
    if constexpr (N == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        d[0] = v.x; d[1] = v.y; d[2] = v.z; d[3] = v.w;
    } else if constexpr (N == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        d[0] = v.x; d[1] = v.y;
    } else {
        d[0] = *reinterpret_cast<const uint32_t*>(p);
    }
}

// Where lane L finds key L % 16 of a block (off < 0: not read) and its position.
struct Info { int64_t off, soff; int pos; };

template <int HD, int CT, int QT>
struct Cfg {
    static constexpr bool F8 = CT == W_F8, BF = CT == W_BF16;
    static constexpr bool SPLIT_Q = QT == W_F32;
    static constexpr bool SPLIT_P = QT == W_F32 || BF;
    static constexpr bool ROW_SCALE = !BF && QT != W_F16;
    static constexpr int KS = HD / 16;                          // k-steps of Q K^T
    static constexpr int KW = F8 ? HD / 16 : HD / 8;            // words of a key a thread holds
    static constexpr int KC = KW < 4 ? KW : 4;                  // ... loaded KC at a time
    static constexpr int NT = HD / 8;                           // 8-dim column tiles of O
    static constexpr int VP = F8 ? HD / 8 : (HD / 8 < 8 ? HD / 8 : 8);   // contiguous dims of a value per thread
    static constexpr int VH = HD / 8 / VP;                      // ... in VH places 8 * VP dims apart
    static constexpr int VWP = F8 ? VP / 4 : VP / 2;            // words of one place
    // a stage: 16 keys of K and V as the lanes will read them (piece by piece, a lane's words side by
    // side), then the keys' positions and, for E4M3, scales
    static constexpr int KB = 2 * KW * 128, VB = 4 * VH * VWP * 128;
    static constexpr int STAGE = KB + VB + 64 + (F8 ? 128 : 0);
    static constexpr int OUT = kWarps * 16 * (HD + 4) * 4;       // the warps' results, over the stages
    static constexpr int FIT = (112 * 1024 - 1024) / (kWarps * STAGE);
    static constexpr int S = FIT < 8 ? FIT : 8;                 // two CTAs per SM
    static constexpr int RING = kWarps * S * STAGE;
    static constexpr int BYTES = (RING > OUT ? RING : OUT) + 2 * kWarps * 16 * 4 + 16;
};

template <int HD, int CT, int QT>
__global__ void __launch_bounds__(kThr, 2) attn_rows_kernel(AttnPagedArgs a) {
    using C = Cfg<HD, CT, QT>;
    constexpr bool F8 = C::F8, BF = C::BF;
    extern __shared__ __align__(16) uint8_t sm[];
    float (*s_o)[16][HD + 4] = reinterpret_cast<float (*)[16][HD + 4]>(sm);
    constexpr int kEnd = C::RING > C::OUT ? C::RING : C::OUT;
    float (*s_m)[16] = reinterpret_cast<float (*)[16]>(sm + kEnd);
    float (*s_l)[16] = s_m + kWarps;
    int& s_flag = *reinterpret_cast<int*>(sm + kEnd + 2 * kWarps * 16 * 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    if (a.pdl) asm volatile("griddepcontrol.wait;" ::: "memory");
    if (form_missing(a)) return;
    const int n_units = a.hdr[PH_UNITS1] * a.kv.Hkv;

    for (int ui = blockIdx.x; ui < n_units; ui += gridDim.x) {
        const AttnUnit u = load_unit(a.units1 + ui / a.kv.Hkv);
        const int kvh = ui % a.kv.Hkv;
        const uint8_t* kbase = a.kv.k + (int64_t)kvh * a.kv.sb_head;
        const uint8_t* vbase = a.kv.v + (int64_t)kvh * a.kv.sb_head;
        const float* ksb = F8 ? a.kv.ks + (int64_t)kvh * a.kv.ss_head : nullptr;
        const float* vsb = F8 ? a.kv.vs + (int64_t)kvh * a.kv.ss_head : nullptr;

        // rows g and g + 8 of the tile: position, first hidden position, Q fragments
        int rp[2], rh[2];
        float rs[2] = {a.scale_log2, a.scale_log2};
        uint32_t qf[C::KS][4], ql[C::SPLIT_Q ? C::KS : 1][4];
        int pmin = INT_MAX, pmax = INT_MIN;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = g + 8 * h;
            rp[h] = INT_MIN;
            rh[h] = INT_MIN;
            float x[C::KS][4];
#pragma unroll
            for (int s = 0; s < C::KS; ++s)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[s][e] = 0.f;
            if (r < u.n_row) {
                const int row = u.row0 + r, tok = row_token(a, u, row);
                rp[h] = row_pos(a, u, row, tok);
                rh[h] = hidden_below(a, rp[h]);
                pmin = min(pmin, rp[h]);
                pmax = max(pmax, rp[h]);
                const int64_t qo = (int64_t)tok * a.q_tok + (int64_t)(kvh * a.G + row % a.G) * a.q_head;
#pragma unroll
                for (int s = 0; s < C::KS; ++s) {
                    // the four dims of k-step s this thread's key words hold
                    const int d = !F8 ? 32 * (s / 2) + 8 * c + 4 * (s % 2)
                                : HD >= 64 ? 64 * (s / 4) + 16 * c + 4 * (s % 4) : 8 * c + 4 * s;
                    if constexpr (QT == W_F32) {
                        const float4 f = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + qo + d);
                        x[s][0] = f.x; x[s][1] = f.y; x[s][2] = f.z; x[s][3] = f.w;
                    } else {
                        const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.q) + qo + d);
                        const float2 f0 = unpack2<QT == W_BF16>(w.x), f1 = unpack2<QT == W_BF16>(w.y);
                        x[s][0] = f0.x; x[s][1] = f0.y; x[s][2] = f1.x; x[s][3] = f1.y;
                    }
                }
            }
            if constexpr (C::ROW_SCALE) {
                // bring the row's largest value to [1, 2) (exactly; not finite or zero: as it is)
                float mx = 0.f;
#pragma unroll
                for (int s = 0; s < C::KS; ++s)
#pragma unroll
                    for (int e = 0; e < 4; ++e) mx = fmaxf(mx, fabsf(x[s][e]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const uint32_t ex = __float_as_uint(mx) >> 23;
                if (ex > 0u && ex < 254u) {
                    const float dn = __uint_as_float((254u - ex) << 23), up = __uint_as_float(ex << 23);
#pragma unroll
                    for (int s = 0; s < C::KS; ++s)
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[s][e] *= dn;
                    rs[h] *= up;
                }
            }
#pragma unroll
            for (int s = 0; s < C::KS; ++s) {
                if constexpr (C::SPLIT_Q) {
                    split2<BF>(x[s][0], x[s][1], qf[s][h], ql[s][h]);
                    split2<BF>(x[s][2], x[s][3], qf[s][h + 2], ql[s][h + 2]);
                } else {
                    qf[s][h] = pack2<BF>(x[s][0], x[s][1]);
                    qf[s][h + 2] = pack2<BF>(x[s][2], x[s][3]);
                }
            }
        }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            pmin = min(pmin, __shfl_xor_sync(0xffffffffu, pmin, o));
            pmax = max(pmax, __shfl_xor_sync(0xffffffffu, pmax, o));
        }
        // a key no row sees is not read: its cell may hold anything
        const int hid_all = hidden_below(a, pmin);

        const int nb = (u.v1 - u.v0 + 15) / 16;
        auto lookup = [&](int b) {
            Info f{-1, 0, INT_MAX};
            const int v = u.v0 + 16 * b + (lane & 15);
            if (b < nb && v < u.v1) {
                const KeyAt k = key_at(a, u, v);
                if (k.off >= 0 && sees(k.pos, pmax, hid_all, a.n_sink)) {
                    f.off = k.off;
                    f.soff = k.soff;
                    f.pos = k.pos;
                }
            }
            return f;
        };
        uint8_t* const ring = sm + warp * C::S * C::STAGE;
        // the copies of block b into stage s; a group of copies is counted even where there is no block
        auto issue = [&](int b, int s, const Info& f) {
            uint8_t* const st = ring + s * C::STAGE;
            if (b < nb) {
                const uint32_t ka = static_cast<uint32_t>(__cvta_generic_to_shared(st));
                const uint32_t va = ka + C::KB;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const int64_t off = __shfl_sync(0xffffffffu, f.off, 8 * t + g);
                    const uint8_t* src = kbase + (off >= 0 ? off : 0) + 4 * C::KC * c;
#pragma unroll
                    for (int i = 0; i < C::KW / C::KC; ++i)
                        fetch<C::KC>(ka + (t * C::KW / C::KC + i) * 128 * C::KC + lane * 4 * C::KC, src + 16 * C::KC * i,
                                     off >= 0);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int64_t off = __shfl_sync(0xffffffffu, f.off, 2 * c + (e & 1) + 8 * (e >> 1));
                    const uint8_t* src = vbase + (off >= 0 ? off : 0) + 4 * C::VWP * g;
#pragma unroll
                    for (int i = 0; i < C::VH; ++i)
                        fetch<C::VWP>(va + (e * C::VH + i) * 128 * C::VWP + lane * 4 * C::VWP, src + 32 * C::VWP * i, off >= 0);
                }
                const uint32_t ma = va + C::VB;
                if (lane < 16) *reinterpret_cast<int*>(st + C::KB + C::VB + 4 * lane) = f.pos;
                if constexpr (F8)
                    fetch<1>(ma + 64 + 4 * lane,
                             reinterpret_cast<const uint8_t*>((lane < 16 ? ksb : vsb) + (f.off >= 0 ? f.soff : 0)), f.off >= 0);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };

        float O[C::NT][4];
#pragma unroll
        for (int n = 0; n < C::NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) O[n][e] = 0.f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        float E = 0.f;                                      // O is in units of E (E4M3 values only)

        Info nxt;
        {
            Info f[C::S - 1];
#pragma unroll
            for (int s = 0; s < C::S - 1; ++s) f[s] = lookup(warp + s * kWarps);
#pragma unroll
            for (int s = 0; s < C::S - 1; ++s) issue(warp + s * kWarps, s, f[s]);
            nxt = lookup(warp + (C::S - 1) * kWarps);
        }
        int stage = 0, free_stage = C::S - 1;
        for (int b = warp; b < nb; b += kWarps) {
            asm volatile("cp.async.wait_group %0;" ::"n"(C::S - 2) : "memory");
            __syncwarp();
            // the stage read in the last round takes the block S - 1 rounds ahead
            issue(b + (C::S - 1) * kWarps, free_stage, nxt);
            nxt = lookup(b + C::S * kWarps);
            const uint8_t* const st = ring + stage * C::STAGE;
            free_stage = stage;
            if (++stage == C::S) stage = 0;
            float S[2][4] = {};
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                uint32_t kr[C::KW];
#pragma unroll
                for (int i = 0; i < C::KW / C::KC; ++i)
                    take<C::KC>(&kr[C::KC * i], st + (t * C::KW / C::KC + i) * 128 * C::KC + lane * 4 * C::KC);
#pragma unroll
                for (int s = 0; s < C::KS; ++s) {
                    uint32_t b0, b1;
                    if constexpr (F8) {
                        b0 = e4m3x2_to_h2(kr[s] & 0xffffu);
                        b1 = e4m3x2_to_h2(kr[s] >> 16);
                    } else {
                        b0 = kr[2 * s];
                        b1 = kr[2 * s + 1];
                    }
                    mma<BF>(S[t], qf[s], b0, b1);
                    if constexpr (C::SPLIT_Q) mma<BF>(S[t], ql[s], b0, b1);
                }
            }
            const uint8_t* const meta = st + C::KB + C::VB;
            // scores in the log2 domain, masked; the rows' maxima
            float mx[2] = {-INFINITY, -INFINITY};
            float kvs[2][2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int2 kp2 = *reinterpret_cast<const int2*>(meta + 4 * (8 * t + 2 * c));
                float2 ks2 = make_float2(1.f, 1.f);
                if constexpr (F8) {
                    ks2 = *reinterpret_cast<const float2*>(meta + 64 + 4 * (8 * t + 2 * c));
                    const float2 v2 = *reinterpret_cast<const float2*>(meta + 128 + 4 * (8 * t + 2 * c));
                    kvs[t][0] = v2.x;
                    kvs[t][1] = v2.y;
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int kp = e ? kp2.y : kp2.x;
                    const float ksc = e ? ks2.y : ks2.x;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float& s = S[t][2 * h + e];
                        s = sees(kp, rp[h], rh[h], a.n_sink) ? s * (F8 ? rs[h] * ksc : rs[h]) : -INFINITY;
                        mx[h] = fmaxf(mx[h], s);
                    }
                }
            }
            bool up = false;
            float f[2] = {1.f, 1.f};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
                mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
                if (mx[h] > m[h] + 14.f) {                  // true from nothing too
                    f[h] = ex2(m[h] - (mx[h] - 6.f));       // 0 from nothing
                    m[h] = mx[h] - 6.f;
                    l[h] *= f[h];
                    up = true;
                }
            }
            if constexpr (F8) {
                // the values' scales relative to the largest seen
                float e = fmaxf(fmaxf(kvs[0][0], kvs[0][1]), fmaxf(kvs[1][0], kvs[1][1]));
                e = fmaxf(e, __shfl_xor_sync(0xffffffffu, e, 1));
                e = fmaxf(e, __shfl_xor_sync(0xffffffffu, e, 2));
                if (e > E) {
                    f[0] *= E / e;
                    f[1] *= E / e;
                    E = e;
                    up = true;
                }
            }
            if (__any_sync(0xffffffffu, up)) {
#pragma unroll
                for (int n = 0; n < C::NT; ++n) {
                    O[n][0] *= f[0]; O[n][1] *= f[0];
                    O[n][2] *= f[1]; O[n][3] *= f[1];
                }
            }
            uint32_t pf[4], pl[C::SPLIT_P ? 4 : 1];
            const float inv = E > 0.f ? 1.f / E : 0.f;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float p0 = m[h] == -INFINITY ? 0.f : ex2(S[t][2 * h] - m[h]);
                    float p1 = m[h] == -INFINITY ? 0.f : ex2(S[t][2 * h + 1] - m[h]);
                    l[h] += p0 + p1;
                    if constexpr (F8) { p0 *= kvs[t][0] * inv; p1 *= kvs[t][1] * inv; }
                    if constexpr (C::SPLIT_P) split2<BF>(p0, p1, pf[2 * t + h], pl[2 * t + h]);
                    else pf[2 * t + h] = pack2<BF>(p0, p1);
                }
            auto pv = [&](int n, uint32_t b0, uint32_t b1) {
                mma<BF>(O[n], pf, b0, b1);
                if constexpr (C::SPLIT_P) mma<BF>(O[n], pl, b0, b1);
            };
#pragma unroll
            for (int p = 0; p < C::VH; ++p) {
                uint32_t vr[4][C::VWP];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    take<C::VWP>(vr[e], st + C::KB + (e * C::VH + p) * 128 * C::VWP + lane * 4 * C::VWP);
#pragma unroll
                for (int w = 0; w < C::VWP; ++w) {
                    const int i = p * C::VWP + w;
                    const uint32_t w0 = vr[0][w], w1 = vr[1][w], w2 = vr[2][w], w3 = vr[3][w];
                    if constexpr (F8) {
                        const uint32_t x0 = __byte_perm(w0, w1, 0x5140), x1 = __byte_perm(w0, w1, 0x7362);
                        const uint32_t y0 = __byte_perm(w2, w3, 0x5140), y1 = __byte_perm(w2, w3, 0x7362);
                        pv(4 * i, e4m3x2_to_h2(x0 & 0xffffu), e4m3x2_to_h2(y0 & 0xffffu));
                        pv(4 * i + 1, e4m3x2_to_h2(x0 >> 16), e4m3x2_to_h2(y0 >> 16));
                        pv(4 * i + 2, e4m3x2_to_h2(x1 & 0xffffu), e4m3x2_to_h2(y1 & 0xffffu));
                        pv(4 * i + 3, e4m3x2_to_h2(x1 >> 16), e4m3x2_to_h2(y1 >> 16));
                    } else {
                        pv(2 * i, __byte_perm(w0, w1, 0x5410), __byte_perm(w2, w3, 0x5410));
                        pv(2 * i + 1, __byte_perm(w0, w1, 0x7632), __byte_perm(w2, w3, 0x7632));
                    }
                }
            }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();                                    // the results go where the stages were
        // this warp's state to shared memory: row sums over the four threads of a row
        bool finite = true;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
            if (c == 0) { s_m[warp][g + 8 * h] = m[h]; s_l[warp][g + 8 * h] = l[h]; }
            finite = finite && l[h] <= 3.0e38f && m[h] <= 3.0e38f;
#pragma unroll
            for (int n = 0; n < C::NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float o = F8 ? O[n][2 * h + e] * E : O[n][2 * h + e];
                    finite = finite && fabsf(o) <= 3.0e38f;
                    s_o[warp][g + 8 * h][(n / C::VP) * 8 * C::VP + C::VP * (2 * c + e) + n % C::VP] = o;
                }
        }
        const bool redo = __syncthreads_or(!finite);
        if (redo) {
            // not every operand was finite: the rows again, key by key; warp 0's state takes the result
            for (int r = warp; r < u.n_row; r += kWarps) {
                float o[HD / 32], rm, rl;
                careful_row<HD>(a, u, kvh, u.row0 + r, o, rm, rl);
#pragma unroll
                for (int d = 0; d < HD / 32; ++d) s_o[0][r][lane * (HD / 32) + d] = o[d];
                if (lane == 0) {
                    s_m[0][r] = rm;
                    s_l[0][r] = rl;
                    for (int w = 1; w < kWarps; ++w) { s_m[w][r] = -INFINITY; s_l[w][r] = 0.f; }
                }
            }
            __syncthreads();
        }
        // merge the warps; one unit alone writes the output, several their partial results
        for (int x = threadIdx.x; x < u.n_row * (HD / 4); x += kThr) {
            const int r = x / (HD / 4), d = (x % (HD / 4)) * 4;
            float M = -INFINITY, L = 0.f, v[4] = {};
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][r]);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                if (s_m[w][r] == -INFINITY && s_l[w][r] == 0.f) continue;
                const float f = s_m[w][r] == M ? 1.f : ex2(s_m[w][r] - M);
                L += f * s_l[w][r];
                const float4 o = *reinterpret_cast<const float4*>(&s_o[w][r][d]);
                v[0] += f * o.x; v[1] += f * o.y; v[2] += f * o.z; v[3] += f * o.w;
            }
            if (u.n_chunk == 1) {
                const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = L == 0.f ? 0.f : v[j] * inv;
                const int row = u.row0 + r, tok = row_token(a, u, row);
                store_out4(a, (int64_t)tok * a.o_tok + (int64_t)(kvh * a.G + row % a.G) * a.o_head + d, v);
            } else {
                const int64_t at = ((int64_t)(u.part + u.chunk) * a.kv.Hkv + kvh) * kUnitRows1 + r;
                *reinterpret_cast<float4*>(a.part_o + at * HD + d) = make_float4(v[0], v[1], v[2], v[3]);
                if (d == 0) a.part_ml[at] = make_float2(M, L);
            }
        }
        if (u.n_chunk > 1 && last_of_tile(a, u, kvh, &s_flag)) merge_parts<HD>(a, u, kvh, kUnitRows1);
        __syncthreads();                                    // shared memory is free for the next unit
    }
}

template <int HD, int CT, int QT>
bool go(const AttnPagedArgs& a, cudaStream_t st) {
    using C = Cfg<HD, CT, QT>;
    if (cudaFuncSetAttribute(attn_rows_kernel<HD, CT, QT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::BYTES) !=
        cudaSuccess)
        return false;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * a.n_sm);                         // two CTAs per SM, each walking its units
    cfg.blockDim = dim3(kThr);
    cfg.dynamicSmemBytes = C::BYTES;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = a.pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, attn_rows_kernel<HD, CT, QT>, a) == cudaSuccess;
}
template <int HD>
bool go_hd(const AttnPagedArgs& a, cudaStream_t st) {
    if (a.kv.type == W_F16) return a.q_type == W_F16 ? go<HD, W_F16, W_F16>(a, st) : go<HD, W_F16, W_F32>(a, st);
    if (a.kv.type == W_BF16) return go<HD, W_BF16, W_BF16>(a, st);
    if (a.q_type == W_F16) return go<HD, W_F8, W_F16>(a, st);
    return a.q_type == W_BF16 ? go<HD, W_F8, W_BF16>(a, st) : go<HD, W_F8, W_F32>(a, st);
}

}  // namespace

bool attn_paged_types_ok(int32_t q, int32_t kv) {
    if (kv == W_F16) return q == W_F16 || q == W_F32;
    if (kv == W_BF16) return q == W_BF16;
    return kv == W_F8 && (q == W_F16 || q == W_BF16 || q == W_F32);
}

bool launch_attn_paged(const AttnPagedArgs& a, cudaStream_t st) {
    if (!attn_paged_types_ok(a.q_type, a.kv.type)) return false;
    if (a.form & ATTN_FORM_TC) {
        if (!launch_attn_paged_tc(a, st)) return false;
    }
    if (!(a.form & ATTN_FORM_ROWS)) return true;
    switch (a.kv.hd) {
        case 32: return go_hd<32>(a, st);
        case 64: return go_hd<64>(a, st);
        case 128: return go_hd<128>(a, st);
    }
    return false;
}

}  // namespace llm
