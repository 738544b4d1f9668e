// Attention of new tokens over a paged cache, 8- and 16-row tiles: out = softmax(scale q K^T, masked) V for
// the (token, query head) pairs that share a KV head, an optional sliding window and sink keys.
//
// A CTA walks its share of the plan's units. Its warps take every so many'th 32 keys of a unit and
// merge their (reference, sum, output) at the end; the units of a cut tile merge through partial results in
// global memory (the last to finish does it). Per 32 keys and warp, with the keys and dims as the rows of the MMA
// and the tile's 8 (or 2 x 8) rows as its columns, so that few rows waste little:
//   S^T = K Q^T      mma.sync m16n8k16, 16 keys x 8 rows, float32 sums
//   softmax          p = 2^(s - m) with a reference m per row in float32, in the log2 domain. m is 6 below a
//                    row maximum and raised lazily, when some p would pass 2^14: no maximum is reduced
//                    otherwise, O is rarely rescaled, the largest p is between 2^6 and 2^14, and f16's
//                    subnormal steps start 2^20 below it
//   O^T += V^T P^T   mma.sync, 16 dims x 8 rows; P^T from S^T by an 8x8 transpose between the lanes
// This form is for few rows per KV head (single tokens, short chunks), where reading K and V once is the
// bound. A contraction may be taken in any order, so a lane's 16 bytes of a key row simply are the dims its
// A fragments hold (Q is loaded in the same order), and a lane's values of four keys become fragments
// by byte permutes (f16/bf16: pairs of keys; E4M3: 4 x 4 bytes, then the conversion to f16, which is
// exact). Rows come by asynchronous 16-byte copies, a row by neighbouring lanes, into a warp's own ring in
// shared memory: 32 keys are used while the next are under way, and a ring's 16-byte chunks are permuted so that
// both ways of reading them are free of bank conflicts. (Lanes copying just the bytes they use would need no
// permutation, but touch K rows in 64-byte pieces: 5.3 TB/s at most for E4M3 rows of 128 bytes, against
// 7.0 TB/s for whole rows.)
//
// Measured, 32 / 8 heads of 128: 32 single f16 tokens over 1 .. 2304 keys 39 us (156 MB, 4.0 TB/s), 16 over 9k .. 33k
// E4M3 keys 145 us (709 MB, 4.9 TB/s of the 6.8 that the card copies at), one over 513 keys 12 us, which is
// latency: the plan, the page table, the rows and the parts' join follow from each other.
//
// Precision: products of f16 (bf16) terms with float32 sums. F16 activations and caches enter as they
// are. BF16 or F32 activations over an f16-typed product are scaled per row by a power of two (taken out of the
// scores again), so that no value leaves f16's range; F32 ones enter as two f16 terms (22 bits). P is
// rounded to f16 (half a step: 2^-11) where activations are f16; for F32 activations and for bf16 products
// it enters as two terms, so its rounding (2^-8 for bf16) does not show. An E4M3 row's scale multiplies
// the score (K) or p (V, relative to E, the largest scale of the values that the query row has seen so far, a power
// of two, so exact down to f16's subnormals). Each query row has an E of its own: a value that only later tokens see
// does not push a row's own values out of f16's range. Rows of zeros, whose scale is 1 whatever the others are, do not
// count. 1 / E is part of the exponent: 2^(s - m - log2 E) is summed and times the scale is the operand; m is a whole
// number here, so that the sum m + log2 E is exact. (Eight sequences of 4 tokens over 8192 keys: 45.5 us with one E for
// the tile, 48.2 with a product with 1 / E for each weight, 47.3 so.)
#include "attn_paged_common.cuh"

#include <algorithm>
#include <type_traits>

namespace llm {

namespace {

using namespace pattn;

template <bool BF>
__device__ __forceinline__ void mma(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
    if constexpr (BF)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// the 8x8 matrix of 16-bit values whose row lane / 4 this lane holds two of, transposed
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
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
// (x, y) as two terms: rounded, and the rounding errors
template <bool BF>
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
    hi = pack2<BF>(x, y);
    const float2 f = unpack2<BF>(hi);
    lo = pack2<BF>(x - f.x, y - f.y);
}

// 16 or 4 bytes from global to shared memory, asynchronously; zeros where the key is not read
__device__ __forceinline__ void fetch16(uint32_t dst, const uint8_t* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void fetch16z(uint32_t dst, const uint8_t* src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void fetch4z(uint32_t dst, const float* src, bool ok) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(ok ? 4 : 0) : "memory");
}
// Byte offset of 16-byte chunk `ch` of row `row` in a tile of rows of ROWB bytes. The chunks of a 128-byte line are
// permuted so that neither a K fragment's read (rows g, 16-byte chunks c) nor a V fragment's (rows 2 c, chunks g or
// parts of them) meets a bank twice.
template <int ROWB>
__device__ __forceinline__ uint32_t at16(int row, int ch) {
    if constexpr (ROWB >= 128) return (uint32_t)(row * ROWB + ((ch ^ (((row >> 1) & 3) << 1) ^ ((row & 1) << 2)) << 4));
    else if constexpr (ROWB == 64)
        return (uint32_t)((row >> 1) * 128 + (((((row & 1) << 2) | ch) ^ (((row >> 1) & 3) << 1)) << 4));
    else return (uint32_t)((row >> 2) * 128 + (((((row & 3) << 1) | ch) ^ (((row >> 2) & 1) << 1)) << 4));
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

constexpr int kMaxSm = 160;

// Where this lane's key of 32 lies (off < 0: not read) and its position.
struct Info { int64_t off, soff; int pos; };

template <int HD, int CT, int QT, int ROWS>
struct Cfg {
    static constexpr bool F8 = CT == W_F8, BF = CT == W_BF16;
    static constexpr bool SPLIT_Q = QT == W_F32;
    static constexpr bool SPLIT_P = QT == W_F32 || BF;
    static constexpr bool ROW_SCALE = !BF && QT != W_F16;
    static constexpr int W = attn_rows_warps(HD, CT, ROWS);     // warps
    static constexpr int R = ROWS / 8;                          // 8-row column tiles
    static constexpr int KS = HD / 16;                          // k-steps of K Q^T
    static constexpr int KW = F8 ? HD / 16 : HD / 8;            // words of a key a lane holds
    static constexpr int KC = KW < 4 ? KW : 4;                  // ... copied KC at a time
    static constexpr int KP = KW / KC;
    static constexpr int MT = HD / 16;                          // 16-dim row tiles of O^T
    static constexpr int VP = F8 ? HD / 8 : (HD / 8 < 8 ? HD / 8 : 8);   // contiguous dims of a value per lane
    static constexpr int VH = HD / 8 / VP;                      // ... in VH places 8 * VP dims apart
    static constexpr int VW = F8 ? VP / 4 : VP / 2;             // words of one place
    // a stage: 32 rows of K and of V, then the keys' positions, which of them are read, and, for E4M3, scales
    static constexpr int ROWB = F8 ? HD : 2 * HD;
    static constexpr int META = 64 * ROWB;
    static constexpr int STAGE = META + 128 + 16 + (F8 ? 256 : 0);
    static constexpr int OUT = W * ROWS * (HD + 4) * 4;          // the warps' results, over the stages
    static constexpr int FIT = (227 * 1024 / kAttnRowsCtas - 4096) / (W * STAGE);
    static constexpr int S = FIT < 6 ? FIT : 6;
    static constexpr int RING = W * S * STAGE;
    static constexpr int END = RING > OUT ? RING : OUT;
    static constexpr int BYTES = END + W * 256 + 2 * W * ROWS * 4 + 16;
    static_assert(S >= 2, "a stage to read and one to fill");
    // the join of a cut tile: (reference, sum) of its rows from every CTA, and a part at least
    static_assert(END >= 8 * ROWS * kAttnRowsCtas * kMaxSm + ROWS * HD * 4, "parts of a cut tile");
};

template <int HD, int CT, int QT, int ROWS>
__global__ void __launch_bounds__(32 * attn_rows_warps(HD, CT, ROWS), kAttnRowsCtas)
attn_rows_kernel(AttnPagedArgs a) {
    using C = Cfg<HD, CT, QT, ROWS>;
    constexpr int kWarps = C::W, kThr = 32 * kWarps;
    constexpr bool F8 = C::F8, BF = C::BF;
    constexpr int R = C::R;
    extern __shared__ __align__(16) uint8_t sm[];
    float (*s_o)[ROWS][HD + 4] = reinterpret_cast<float (*)[ROWS][HD + 4]>(sm);
    int64_t (*s_off)[32] = reinterpret_cast<int64_t (*)[32]>(sm + C::END);
    float (*s_m)[ROWS] = reinterpret_cast<float (*)[ROWS]>(sm + C::END + kWarps * 256);
    float (*s_l)[ROWS] = s_m + kWarps;
    int& s_flag = *reinterpret_cast<int*>(s_l + kWarps);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    asm volatile("griddepcontrol.launch_dependents;");      // the 256-row tiles of a mixed plan may start
    const int ui0 = a.first1[blockIdx.x], ui1 = a.first1[blockIdx.x + 1];   // (on their way with the header)
    if (form_missing(a) || (a.hdr[PH_FORM] & (ROWS == 8 ? ATTN_FORM_ROWS8 : ATTN_FORM_ROWS16)) == 0) return;

    for (int ui = ui0; ui < ui1; ++ui) {
        const AttnUnit u = load_unit(a.units1 + ui);
        const int kvh = u.head;
        const uint8_t* kbase = a.kv.k + (int64_t)kvh * a.kv.sb_head;
        const uint8_t* vbase = a.kv.v + (int64_t)kvh * a.kv.sb_head;
        const float* ksb = F8 ? a.kv.ks + (int64_t)kvh * a.kv.ss_head : nullptr;
        const float* vsb = F8 ? a.kv.vs + (int64_t)kvh * a.kv.ss_head : nullptr;

        // positions of the tile's rows: a row per lane, then what every lane needs of them
        int rpos = INT_MIN, pmin = INT_MAX, pmax = INT_MIN, rtok = 0;
        if (lane < u.n_row) {
            rtok = row_token(a, u, u.row0 + lane);
            rpos = row_pos(a, u, u.row0 + lane, rtok);
            pmin = pmax = rpos;
        }
        pmin = __reduce_min_sync(0xffffffffu, pmin);
        pmax = __reduce_max_sync(0xffffffffu, pmax);
        const int hid_min = hidden_below(a, pmin), hid_max = hidden_below(a, pmax);

        const int n_keys = u.v1 - u.v0;
        // this warp's groups of 32 keys: 32 (warp + kWarps i)
        const int n_st = max(0, (n_keys - 32 * warp + 32 * kWarps - 1) / (32 * kWarps));
        auto lookup = [&](int i) {
            Info f{-1, 0, INT_MAX};
            const int v = 32 * (warp + kWarps * i) + lane;
            if (v < n_keys) {
                const KeyAt k = key_at(a, u, u.v0 + v);
                // a key no row sees is not read: its cell may hold anything
                if (k.off >= 0 && sees(k.pos, pmax, hid_min, a.n_sink)) {
                    f.off = k.off;
                    f.soff = k.soff;
                    f.pos = k.pos;
                }
            }
            return f;
        };
        uint8_t* const ring = sm + warp * C::S * C::STAGE;
        Info fnext = lookup(0);
        int in = 0, in_stage = 0;
        // the copies of the next 32 keys; a group of copies is counted even where there are none
        auto issue = [&]() {
            if (in < n_st) {
                const Info f = fnext;
                uint8_t* const st = ring + in_stage * C::STAGE;
                const uint32_t sa = static_cast<uint32_t>(__cvta_generic_to_shared(st));
                const unsigned read = __ballot_sync(0xffffffffu, f.off >= 0);
                __syncwarp();                               // the last offsets have been read
                s_off[warp][lane] = f.off >= 0 ? f.off : 0;
                reinterpret_cast<int*>(st + C::META)[lane] = f.pos;
                if (lane == 0) *reinterpret_cast<unsigned*>(st + C::META + 128) = read;
                if constexpr (F8) {
                    const int64_t so = f.off >= 0 ? f.soff : 0;
                    fetch4z(sa + C::META + 144 + 4 * lane, ksb + so, f.off >= 0);
                    fetch4z(sa + C::META + 272 + 4 * lane, vsb + so, f.off >= 0);
                }
                __syncwarp();
                constexpr int LPR = C::ROWB / 16, RPI = 32 / LPR;   // lanes per row, rows per copy
                // (all offsets before the first copy: the copies do not wait for one another's)
                int64_t off[LPR];
#pragma unroll
                for (int x = 0; x < LPR; ++x) off[x] = s_off[warp][x * RPI + lane / LPR] + 16 * (lane % LPR);
                if (read == 0xffffffffu) {
#pragma unroll
                    for (int x = 0; x < LPR; ++x) {
                        const uint32_t d = sa + at16<C::ROWB>(x * RPI + lane / LPR, lane % LPR);
                        fetch16(d, kbase + off[x]);
                        fetch16(d + 32 * C::ROWB, vbase + off[x]);
                    }
                } else {
#pragma unroll
                    for (int x = 0; x < LPR; ++x) {
                        const int k = x * RPI + lane / LPR;
                        const uint32_t d = sa + at16<C::ROWB>(k, lane % LPR);
                        fetch16z(d, kbase + off[x], read >> k & 1u);
                        fetch16z(d + 32 * C::ROWB, vbase + off[x], read >> k & 1u);
                    }
                }
                fnext = lookup(++in);
                if (++in_stage == C::S) in_stage = 0;
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
#pragma unroll
        for (int s = 0; s < C::S - 1; ++s) issue();

        // Q fragments: column g of column tile r is row 8 r + g; a lane's dims as its key words hold them
        uint32_t qf[R][C::KS][2], ql[C::SPLIT_Q ? R : 1][C::KS][2];
        float rsc[R];                                       // scale of row 8 r + g
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float x[C::KS][4];
#pragma unroll
            for (int s = 0; s < C::KS; ++s)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[s][e] = 0.f;
            const int tok = __shfl_sync(0xffffffffu, rtok, 8 * r + g);
            if (8 * r + g < u.n_row) {
                const int row = u.row0 + 8 * r + g;
                const int64_t qo = (int64_t)tok * a.q_tok + (int64_t)(kvh * a.G + row % a.G) * a.q_head;
#pragma unroll
                for (int s = 0; s < C::KS; ++s) {
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
            rsc[r] = a.scale_log2;
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
                    const float dn = __uint_as_float((254u - ex) << 23);
#pragma unroll
                    for (int s = 0; s < C::KS; ++s)
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[s][e] *= dn;
                    rsc[r] *= __uint_as_float(ex << 23);
                }
            }
#pragma unroll
            for (int s = 0; s < C::KS; ++s) {
                if constexpr (C::SPLIT_Q) {
                    split2<BF>(x[s][0], x[s][1], qf[r][s][0], ql[r][s][0]);
                    split2<BF>(x[s][2], x[s][3], qf[r][s][1], ql[r][s][1]);
                } else {
                    qf[r][s][0] = pack2<BF>(x[s][0], x[s][1]);
                    qf[r][s][1] = pack2<BF>(x[s][2], x[s][3]);
                }
            }
        }
        // the score fragment's columns are rows 8 r + 2 c + e: their positions and scales
        int rp[R][2], rh[R][2];
        float rs[R][2];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                rp[r][e] = __shfl_sync(0xffffffffu, rpos, 8 * r + 2 * c + e);
                rh[r][e] = hidden_below(a, rp[r][e]);
                rs[r][e] = __shfl_sync(0xffffffffu, rsc[r], 4 * (2 * c + e));
            }

        float O[R][C::MT][4];
        float m[R][2], l[R][2];
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int t = 0; t < C::MT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) O[r][t][e] = 0.f;
            m[r][0] = m[r][1] = -INFINITY;
            l[r][0] = l[r][1] = 0.f;
        }
        // E4M3 values: l and O are in units of E, the largest scale seen by a row (0: none yet, the unit is 1); mE is
        // m + log2 E. E stays within 2^-80 .. 2^80, so that weights in its units neither pass float32 nor vanish: below, the
        // unit is done key by key, above, values that f16 does not hold send it there.
        constexpr float kMinE = 0x1p-80f, kMaxE = 0x1p80f;
        float E[F8 ? R : 1][2] = {}, mE[F8 ? R : 1][2] = {};
        float least = 0.f;                                  // the least E of the lane's rows
        bool lost = false;                                  // E too small, or mE not exact (scores past 2^24)

        int stage = 0;
        for (int n = 0; n < n_st; ++n) {
            asm volatile("cp.async.wait_group %0;" ::"n"(C::S - 2) : "memory");
            __syncwarp();                                   // every lane's part of the stage, and of the last is done with
            const uint8_t* const st = ring + stage * C::STAGE;
            if (++stage == C::S) stage = 0;
            const uint8_t* const meta = st + C::META;
            const unsigned read = *reinterpret_cast<const unsigned*>(meta + 128);
            // keys 16 b + g and 16 b + g + 8, read ahead of the next copies in the memory pipe's queue
            uint32_t k[2][2][C::KW];
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < C::KP; ++i) {
                        const int at = 4 * C::KC * (4 * i + c);   // byte of the row
                        take<C::KC>(&k[b][t][C::KC * i], st + at16<C::ROWB>(16 * b + 8 * t + g, at >> 4) + (at & 15));
                    }
            issue();
            if (read == 0u) continue;
            // S[b][r][2 h + e] is key 16 b + 8 h + g, row 8 r + 2 c + e
            float S[2][R][4];
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int r = 0; r < R; ++r) S[b][r][0] = S[b][r][1] = S[b][r][2] = S[b][r][3] = 0.f;
#pragma unroll
            for (int i = 0; i < C::KP; ++i) {
                constexpr int PER = F8 ? C::KC : C::KC / 2;  // k-steps of a piece
#pragma unroll
                for (int j = 0; j < PER; ++j)
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        uint32_t ka[4];
                        if constexpr (F8) {
                            e4m3x4_to_h2(k[b][0][C::KC * i + j], ka[0], ka[2]);
                            e4m3x4_to_h2(k[b][1][C::KC * i + j], ka[1], ka[3]);
                        } else {
                            ka[0] = k[b][0][C::KC * i + 2 * j]; ka[1] = k[b][1][C::KC * i + 2 * j];
                            ka[2] = k[b][0][C::KC * i + 2 * j + 1]; ka[3] = k[b][1][C::KC * i + 2 * j + 1];
                        }
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            mma<BF>(S[b][r], ka, qf[r][i * PER + j][0], qf[r][i * PER + j][1]);
                            if constexpr (C::SPLIT_Q) mma<BF>(S[b][r], ka, ql[r][i * PER + j][0], ql[r][i * PER + j][1]);
                        }
                    }
            }
            // scores in the log2 domain
            const int* kpos = reinterpret_cast<const int*>(meta);
            const float* sc = reinterpret_cast<const float*>(meta + 144);
            float vs[2][2];
            const int k_lo = kpos[0], k_hi = kpos[31];
            // every row sees every key (positions ascend)
            const bool open = read == 0xffffffffu && k_hi <= pmin && (k_lo > hid_max || k_hi < a.n_sink);
            bool raise = false;
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float ks = F8 ? sc[16 * b + 8 * h + g] : 1.f;
                    vs[b][h] = F8 ? sc[32 + 16 * b + 8 * h + g] : 1.f;
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int e = 0; e < 2; ++e) S[b][r][2 * h + e] *= F8 ? rs[r][e] * ks : rs[r][e];
                    if (!open) {
                        const int kp = kpos[16 * b + 8 * h + g];
#pragma unroll
                        for (int r = 0; r < R; ++r)
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                if (!sees(kp, rp[r][e], rh[r][e], a.n_sink)) S[b][r][2 * h + e] = -INFINITY;
                    }
                }
            float mx[R][2];
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    mx[r][e] = fmaxf(fmaxf(S[0][r][e], S[0][r][2 + e]), fmaxf(S[1][r][e], S[1][r][2 + e]));
                    raise = raise || mx[r][e] > m[r][e] + 14.f;
                }
            // (scales above that of some row: whether it sees them, and whether they are of zeros, is looked into below)
            if constexpr (F8) raise = raise || fmaxf(fmaxf(vs[0][0], vs[0][1]), fmaxf(vs[1][0], vs[1][1])) > least;
            if (__any_sync(0xffffffffu, raise)) {
                if constexpr (F8) {
                    if (__any_sync(0xffffffffu, vs[0][0] == 1.f || vs[0][1] == 1.f || vs[1][0] == 1.f || vs[1][1] == 1.f)) {
                        // rows of zeros? (key `lane` of the stage)
                        uint32_t bits = 0u;
#pragma unroll
                        for (int ch = 0; ch < C::ROWB / 16; ++ch) {
                            const uint4 x = *reinterpret_cast<const uint4*>(st + 32 * C::ROWB + at16<C::ROWB>(lane, ch));
                            bits |= x.x | x.y | x.z | x.w;
                        }
                        const unsigned zero = __ballot_sync(0xffffffffu, (bits & 0x7f7f7f7fu) == 0u);
#pragma unroll
                        for (int b = 0; b < 2; ++b)
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                if (zero >> (16 * b + 8 * h + g) & 1u) vs[b][h] = 0.f;
                    }
                    least = INFINITY;
                }
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    float f[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1)
                            mx[r][e] = fmaxf(mx[r][e], __shfl_xor_sync(0xffffffffu, mx[r][e], o));
                        f[e] = 1.f;
                        if (mx[r][e] > m[r][e] + 14.f) {    // true from nothing too
                            const float to = F8 ? floorf(mx[r][e] - 6.f) : mx[r][e] - 6.f;
                            f[e] = ex2(m[r][e] - to);       // 0 from nothing
                            m[r][e] = to;
                        }
                        if constexpr (F8) {
                            float em = 0.f;                 // the largest scale that the row sees here
#pragma unroll
                            for (int b = 0; b < 2; ++b)
#pragma unroll
                                for (int h = 0; h < 2; ++h)
                                    if (S[b][r][2 * h + e] != -INFINITY) em = fmaxf(em, vs[b][h]);
#pragma unroll
                            for (int o = 4; o < 32; o <<= 1) em = fmaxf(em, __shfl_xor_sync(0xffffffffu, em, o));
                            if (em > E[r][e]) {
                                // (the next power of two where a caller's scale is none)
                                const uint32_t up = (__float_as_uint(em) + 0x7fffffu) & 0x7f800000u;
                                const float to = fminf(fmaxf(__uint_as_float(up), kMinE), kMaxE);
                                f[e] *= (E[r][e] > 0.f ? E[r][e] : 1.f) / to;
                                E[r][e] = to;
                            }
                            const float le = E[r][e] > 0.f ? (float)((int)(__float_as_uint(E[r][e]) >> 23) - 127) : 0.f;
                            mE[r][e] = m[r][e] + le;
                            if (rp[r][e] != INT_MIN) least = fminf(least, E[r][e]);   // (places past the tile's rows do not count)
                            lost = lost || (m[r][e] > -INFINITY && mE[r][e] - m[r][e] != le) || E[r][e] == kMinE;
                        }
                        l[r][e] *= f[e];
                    }
#pragma unroll
                    for (int t = 0; t < C::MT; ++t) {
                        O[r][t][0] *= f[0]; O[r][t][1] *= f[1];
                        O[r][t][2] *= f[0]; O[r][t][3] *= f[1];
                    }
                }
            }
            // P^T fragments: pf[b][r][h] holds keys 16 b + 8 h + 2 c, + 1 of row 8 r + g
            uint32_t pf[2][R][2], pl[2][C::SPLIT_P ? R : 1][2];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                // (nothing seen yet: scores of -inf, or NaN, which has to show)
                const float m0 = m[r][0] == -INFINITY ? 0.f : F8 ? mE[F8 ? r : 0][0] : m[r][0];
                const float m1 = m[r][1] == -INFINITY ? 0.f : F8 ? mE[F8 ? r : 0][1] : m[r][1];
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float p0 = ex2(S[b][r][2 * h] - m0), p1 = ex2(S[b][r][2 * h + 1] - m1);
                        l[r][0] += p0;
                        l[r][1] += p1;
                        if constexpr (F8) { p0 *= vs[b][h]; p1 *= vs[b][h]; }
                        if constexpr (C::SPLIT_P) {
                            uint32_t hi, lo;
                            split2<BF>(p0, p1, hi, lo);
                            pf[b][r][h] = transpose8(hi);
                            pl[b][r][h] = transpose8(lo);
                        } else {
                            pf[b][r][h] = transpose8(pack2<BF>(p0, p1));
                        }
                    }
            }
            // V^T fragments: rows g and g + 8 of a 16-dim tile are two neighbouring dims of the lane's
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                auto pv = [&](int t, const uint32_t* va) {
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        mma<BF>(O[r][t], va, pf[b][r][0], pf[b][r][1]);
                        if constexpr (C::SPLIT_P) mma<BF>(O[r][t], va, pl[b][r][0], pl[b][r][1]);
                    }
                };
#pragma unroll
                for (int p = 0; p < C::VH; ++p) {
                    uint32_t vr[4][C::VW];                  // keys 16 b + 2c, 2c + 1, 2c + 8, 2c + 9
                    const int at = 4 * C::VW * (8 * p + g);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        take<C::VW>(vr[e], st + 32 * C::ROWB + (at & 15) +
                                               at16<C::ROWB>(16 * b + 2 * c + (e & 1) + 8 * (e >> 1), at >> 4));
#pragma unroll
                    for (int w = 0; w < C::VW; ++w) {
                        const uint32_t w0 = vr[0][w], w1 = vr[1][w], w2 = vr[2][w], w3 = vr[3][w];
                        if constexpr (F8) {
                            uint32_t a0[4], a1[4];
                            e4m3x4_to_h2(__byte_perm(w0, w1, 0x5140), a0[0], a0[1]);
                            e4m3x4_to_h2(__byte_perm(w2, w3, 0x5140), a0[2], a0[3]);
                            e4m3x4_to_h2(__byte_perm(w0, w1, 0x7362), a1[0], a1[1]);
                            e4m3x4_to_h2(__byte_perm(w2, w3, 0x7362), a1[2], a1[3]);
                            pv(2 * (p * C::VW + w), a0);
                            pv(2 * (p * C::VW + w) + 1, a1);
                        } else {
                            const uint32_t a0[4] = {__byte_perm(w0, w1, 0x5410), __byte_perm(w0, w1, 0x7632),
                                                    __byte_perm(w2, w3, 0x5410), __byte_perm(w2, w3, 0x7632)};
                            pv(p * C::VW + w, a0);
                        }
                    }
                }
            }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();                                    // the results go where the stages were
        // this warp's state to shared memory: row sums over the lanes that share a row
        bool finite = !lost;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float unit = F8 && E[F8 ? r : 0][e] > 0.f ? E[F8 ? r : 0][e] : 1.f;
                if constexpr (F8) l[r][e] *= unit;
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l[r][e] += __shfl_xor_sync(0xffffffffu, l[r][e], o);
                const int row = 8 * r + 2 * c + e;
                if (g == 0) { s_m[warp][row] = m[r][e]; s_l[warp][row] = l[r][e]; }
                finite = finite && l[r][e] <= 3.0e38f && m[r][e] <= 3.0e38f;
#pragma unroll
                for (int t = 0; t < C::MT; ++t)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float o = F8 ? O[r][t][2 * h + e] * unit : O[r][t][2 * h + e];
                        finite = finite && fabsf(o) <= 3.0e38f;
                        const int i = 2 * t + h;            // the lane's i-th dim
                        s_o[warp][row][(i / C::VP) * 8 * C::VP + C::VP * g + i % C::VP] = o;
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
                const int row = u.row0 + r, tok = row_token(a, u, row);
                const float inv = 1.f / L, none = L == 0.f ? weightless(a, u, row, tok) : 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = L == 0.f ? none : v[j] * inv;
                store_out4(a, (int64_t)tok * a.o_tok + (int64_t)(kvh * a.G + row % a.G) * a.o_head + d, v);
            } else {
                const int64_t at = (int64_t)(u.part + u.chunk) * ROWS + r;
                *reinterpret_cast<float4*>(a.part_o + at * HD + d) = make_float4(v[0], v[1], v[2], v[3]);
                if (d == 0) a.part_ml[at] = make_float2(M, L);
            }
        }
        if (u.n_chunk > 1) {
            __threadfence();
            __syncthreads();
            if (threadIdx.x == 0) s_flag = count_unit(a, u);
            __syncthreads();
            if (s_flag) {
                // The last unit of a cut tile joins the partial results, as many at a time as the stages' place
                // holds: asynchronous copies keep them all under way. (Row by row through registers, four tokens
                // after 8192 keys took 47 us, 32 / 8 heads of 128, f16; so they take 29 us.)
                constexpr int NP = (ROWS * (HD / 4) + kThr - 1) / kThr;   // 4 dims of a row: a thread has so many
                const int n_ml = u.n_chunk * u.n_row, row_n = u.n_row * (HD / 4);
                const int fit = (C::END - 8 * n_ml) / (u.n_row * HD * 4);
                float2* s_ml = reinterpret_cast<float2*>(sm + C::END - 8 * n_ml);
                auto bring = [&](int i0) {
                    const float* src = a.part_o + (int64_t)(u.part + i0) * ROWS * HD;
                    const int n = min(fit, u.n_chunk - i0);
                    for (int i = warp; i < n; i += kWarps) {
                        const float* from = src + (int64_t)i * ROWS * HD + 4 * lane;
                        const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(sm)) + 16 * (i * row_n + lane);
#pragma unroll 4
                        for (int y = 0; y < row_n - lane; y += 32)
                            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + 16 * y), "l"(from + 4 * y) : "memory");
                    }
                    asm volatile("cp.async.commit_group;" ::: "memory");
                };
                bring(0);
                const float2* ml = a.part_ml + (int64_t)u.part * ROWS;
                const int r_ml = threadIdx.x % ROWS;
                if (r_ml < u.n_row)
#pragma unroll 8
                    for (int i = threadIdx.x / ROWS; i < u.n_chunk; i += kThr / ROWS)
                        s_ml[i * u.n_row + r_ml] = __ldcg(&ml[i * ROWS + r_ml]);
                __syncthreads();
                for (int r = warp; r < u.n_row; r += kWarps) {   // a part's reference becomes its factor
                    float M = -INFINITY, L = 0.f;
                    for (int i = lane; i < u.n_chunk; i += 32) M = fmaxf(M, s_ml[i * u.n_row + r].x);
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
                    for (int i = lane; i < u.n_chunk; i += 32) {
                        const float2 x = s_ml[i * u.n_row + r];
                        const float f = part_factor(x, M);
                        s_ml[i * u.n_row + r].x = f;
                        L += f * x.y;
                    }
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
                    if (lane == 0) s_l[0][r] = L;
                }
                float v[NP][4] = {};
                for (int i0 = 0; i0 < u.n_chunk; i0 += fit) {
                    if (i0) bring(i0);
                    const int n = min(fit, u.n_chunk - i0);
                    asm volatile("cp.async.wait_group 0;" ::: "memory");
                    __syncthreads();
#pragma unroll
                    for (int y = 0; y < NP; ++y) {
                        const int x = threadIdx.x + y * kThr;
                        if (x >= row_n) break;
                        const float2* fr = s_ml + i0 * u.n_row + x / (HD / 4);
#pragma unroll 4
                        for (int i = 0; i < n; ++i) {
                            const float f = fr[i * u.n_row].x;
                            const float4 o = *reinterpret_cast<const float4*>(sm + 16 * (i * row_n + x));
                            if (f != 0.f) {                  // (a part without a visible key may hold anything)
                                v[y][0] += f * o.x; v[y][1] += f * o.y; v[y][2] += f * o.z; v[y][3] += f * o.w;
                            }
                        }
                    }
                    __syncthreads();
                }
#pragma unroll
                for (int y = 0; y < NP; ++y) {
                    const int x = threadIdx.x + y * kThr, r = x / (HD / 4);
                    if (x >= row_n) break;
                    const int row = u.row0 + r, tok = row_token(a, u, row);
                    const float L = s_l[0][r], inv = 1.f / L, none = L == 0.f ? weightless(a, u, row, tok) : 0.f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[y][e] = L == 0.f ? none : v[y][e] * inv;
                    store_out4(a, (int64_t)tok * a.o_tok + (int64_t)(kvh * a.G + row % a.G) * a.o_head + x % (HD / 4) * 4, v[y]);
                }
            }
        }
        __syncthreads();                                    // shared memory is free for the next unit
    }
}

template <int HD, int CT, int QT, int ROWS>
bool go(const AttnPagedArgs& a, cudaStream_t st) {
    using C = Cfg<HD, CT, QT, ROWS>;
    if (a.n_sm > kMaxSm) return false;
    static std::atomic<uint64_t> done{0};
    if (!allow_smem(reinterpret_cast<const void*>(attn_rows_kernel<HD, CT, QT, ROWS>), C::BYTES, done)) return false;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kAttnRowsCtas * a.n_sm);             // the plan's CTAs
    cfg.blockDim = dim3(32 * C::W);
    cfg.dynamicSmemBytes = C::BYTES;
    cfg.stream = st;
    return cudaLaunchKernelEx(&cfg, attn_rows_kernel<HD, CT, QT, ROWS>, a) == cudaSuccess;
}
template <int HD, int ROWS>
bool go_types(const AttnPagedArgs& a, cudaStream_t st) {
    if (a.kv.type == W_F16)
        return a.q_type == W_F16 ? go<HD, W_F16, W_F16, ROWS>(a, st) : go<HD, W_F16, W_F32, ROWS>(a, st);
    if (a.kv.type == W_BF16) return go<HD, W_BF16, W_BF16, ROWS>(a, st);
    if (a.q_type == W_F16) return go<HD, W_F8, W_F16, ROWS>(a, st);
    return a.q_type == W_BF16 ? go<HD, W_F8, W_BF16, ROWS>(a, st) : go<HD, W_F8, W_F32, ROWS>(a, st);
}
template <int ROWS>
bool go_rows(const AttnPagedArgs& a, cudaStream_t st) {
    switch (a.kv.hd) {
        case 32: return go_types<32, ROWS>(a, st);
        case 64: return go_types<64, ROWS>(a, st);
        case 128: return go_types<128, ROWS>(a, st);
    }
    return false;
}

}  // namespace

bool attn_paged_types_ok(int32_t q, int32_t kv) {
    if (kv == W_F16) return q == W_F16 || q == W_F32;
    if (kv == W_BF16) return q == W_BF16;
    return kv == W_F8 && (q == W_F16 || q == W_BF16 || q == W_F32);
}

bool launch_attn_paged(const AttnPagedArgs& a, cudaStream_t st) {
    if (!attn_paged_types_ok(a.q_type, a.kv.type)) return false;
    if ((a.form & ATTN_FORM_ROWS8) && !go_rows<8>(a, st)) return false;
    if ((a.form & ATTN_FORM_ROWS16) && !go_rows<16>(a, st)) return false;
    return (a.form & ATTN_FORM_TC) == 0 || launch_attn_paged_tc(a, st);
}

}  // namespace llm
