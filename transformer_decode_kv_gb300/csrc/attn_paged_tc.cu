// Attention of new tokens over a paged cache, 256-row tiles on the fifth-generation tensor cores
// (tcgen05, accumulators in TMEM): chunks of new tokens, where the products are the bound. F16, BF16 and
// E4M3 caches, head_dim 64 and 128, F16 or BF16 activations (F32 ones rounded to f16 where the caller's precision is
// that: see attn_paged_tc_ok).
//
// A CTA takes a unit: up to 256 rows of (token, query head) pairs of one KV head, as two halves of 128
// MMA rows, against a range of keys in blocks of 128. Per block and half:
//   S = Q K^T     tcgen05.mma M 128 x N 128, into the half's TMEM columns
//   softmax       a thread per row: p = 2^(s - m) in float32, written back to TMEM as f16 (bf16) over the
//                 second half of S's columns
//   O += P V      tcgen05.mma M 128 x N head_dim, P the A operand from TMEM, V as stored ([keys][dims], an
//                 MN-major B operand)
// While one half's rows are in the softmax, the tensor cores work on the other half. K and V tiles are
// shared by both halves, so each byte from L2 feeds 256 rows. The MMAs of a CTA are issued by one
// thread and run in issue order, so O += P V of block j may be followed at once by S of block j + 1 over
// the same columns, and a completed S means that every product before it is complete too.
//
// Roles (12 warps; warps 0-3 give registers to warps 4-11, whose threads hold a row of scores each): warps
// 0 and 1 (E4M3: 3 too) bring K and V rows into a ring of 128-byte-swizzled tiles, with the keys' positions: a block whose keys are
// all read in bulk tensor copies of the runs of neighbouring cells that pages are, others in 16-byte
// asynchronous copies row by row, and E4M3 rows as raw bytes, converted to f16 from there;
// warp 2 issues the MMAs; warps 4-7 and 8-11 are the two halves' softmax and epilogue (a thread owns a
// TMEM lane: warp w reads lanes 32 (w % 4) on). m is 6 below a row maximum and raised lazily, when p would
// pass 2^14: O, in TMEM, is rarely rescaled, and never more than it must. P is rounded to f16 (half a step 2^-11)
// or, for bf16 products, to bf16 (2^-8 of p: the sums run over the rounded values' float32 originals, and
// the output is rounded to bf16 itself).
//
// E4M3 rows enter as f16 numbers q * s / s0 with s0 the largest scale of the unit's first block (a power
// of two like s; rows of zeros, whose scale is 1, do not count): exact from s0 2^-15 to s0 2^7. A unit with a row out of
// this range is done key by key, after the CTA's other units, as is one with values that are not finite.
//
// Measured, 32 / 8 heads of 128: 2048 bf16 tokens at the end of 32768 keys 769 us (1.4 PFLOP/s, 0.72 of the rate of a
// large bf16 matrix product), bound by what stands between a half's two products (scores out of TMEM, exponentials, P
// back into TMEM): at the end of 8192 keys the tensor pipe is active for 56% of the time, issue slots are used for 38%, the
// exponential unit for 29%. 512 f16 tokens at the end of 8192 take 80 us, where cut tiles weigh; over E4M3 1203 and 113
// us, where the rows' conversion shares issue slots and shared memory with the softmax (tensor pipe 30%, issue slots 37%).
//
// Every wait is bounded by a wall-clock limit; a timeout sets ERR_TIMEOUT, ends every role's loop, and
// the CTA leaves after its copies and with its TMEM freed.
#include "attn_paged_common.cuh"

#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>

namespace llm {

namespace {

using namespace pattn;

constexpr int kProdWarps = 2;
constexpr int kMmaWarp = 2;
constexpr int kSoft0 = 4;                                  // first softmax warp
constexpr int kThr = 12 * 32;
constexpr int kKeys = 128;                                 // keys per block
constexpr int kStages = 5;                                 // K or V tiles in flight (E4M3: one less, its place holds raw rows)
constexpr int kMeta = 3;                                   // blocks whose positions are kept (see meta_full)
constexpr uint32_t kBlk = 128 * 128;                       // [128 rows][64 16-bit values], swizzled
constexpr uint64_t kWaitNs = 2000000000ull;
static_assert(kUnitRows2 == 256, "two halves of 128 MMA rows");

template <int HD>
struct Smem {
    static constexpr uint32_t tile = HD / 64 * kBlk;
    static constexpr uint32_t q = 0;                        // [2] tiles
    static constexpr uint32_t kv = q + 2 * tile;            // [kStages] tiles
    static constexpr uint32_t kpos = kv + kStages * tile;   // int [kMeta][kKeys]
    static constexpr uint32_t full = kpos + kMeta * kKeys * 4;   // uint32 [kMeta]: every key is read
    static constexpr uint32_t rs = full + 16;               // float [256]: scale of a row's scores, where they differ
    static constexpr uint32_t bars = rs + 256 * 4;
    static constexpr uint32_t misc = bars + 24 * 8;
    static constexpr uint32_t bytes = misc + 28 * 4;
};
static_assert(Smem<128>::bytes <= 227 * 1024, "shared memory of one CTA");

__device__ __forceinline__ uint32_t sa(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ uint64_t now_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
__device__ __forceinline__ void bar_init(uint64_t* b, uint32_t n) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(sa(b)), "r"(n));
}
__device__ __forceinline__ void bar_arrive(uint64_t* b) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(sa(b)) : "memory");
}
__device__ __forceinline__ bool bar_try(uint64_t* b, uint32_t par) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok) : "r"(sa(b)), "r"(par) : "memory");
    return ok != 0;
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void to_async_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// a barrier of n threads that tells each of them whether any passed true
__device__ __forceinline__ bool any_of(int id, int n, bool x) {
    uint32_t r;
    asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %3, 0;\n bar.red.or.pred q, %1, %2, p;\n selp.u32 %0, 1, 0, q;\n}\n"
                 : "=r"(r) : "r"(id), "r"(n), "r"((uint32_t)x) : "memory");
    return r != 0;
}

// Shared-memory matrix descriptors of a swizzled tile (8-row groups 1024 bytes apart), low words; the high word is
// the same for all. K-major: rows are M or N. MN-major: rows are the contracted dimension, blocks of 64
// columns kBlk apart.
constexpr uint32_t kDescHi = (1024 >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_k(uint32_t s) { return ((s & 0x3FFFFu) >> 4) | 1u << 16; }
__device__ __forceinline__ uint32_t desc_mn(uint32_t s) { return ((s & 0x3FFFFu) >> 4) | (kBlk >> 4) << 16; }
// kind::f16 with f16 or bf16 A and B, float32 D
__host__ __device__ constexpr uint32_t idesc(bool bf, int m, int n, bool b_mn) {
    return (1u << 4) | (bf ? (1u << 7) | (1u << 10) : 0u) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(m >> 4) << 24);
}
// One k-step of 16 (ACC 0: the product replaces D; 1: it is added; 2: as `acc` says). The whole warp computes the
// operands, so that they stay in uniform registers, and one thread issues.
template <int AO, int BO, int ACC>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t id) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b32 x, y;\n .reg .b64 da, db;\n add.u32 x, %1, %4;\n add.u32 y, %2, %5;\n"
        " mov.b64 da, {x, %6};\n mov.b64 db, {y, %6};\n setp.ne.b32 p, %7, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n}\n" ::"r"(d), "r"(a), "r"(b), "r"(id), "n"(AO),
        "n"(BO), "r"(kDescHi), "n"(ACC));
}
template <int AO, int BO, int ACC>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t acc) {
    if constexpr (ACC == 2)
        asm volatile(
            "{\n .reg .pred p;\n .reg .b32 x, y;\n .reg .b64 db;\n add.u32 x, %1, %4;\n add.u32 y, %2, %5;\n"
            " mov.b64 db, {y, %6};\n setp.ne.b32 p, %7, 0;\n"
            " tcgen05.mma.cta_group::1.kind::f16 [%0], [x], db, %3, p;\n}\n" ::"r"(d), "r"(a), "r"(b), "r"(id), "n"(AO),
            "n"(BO), "r"(kDescHi), "r"(acc));
    else
        asm volatile(
            "{\n .reg .pred p;\n .reg .b32 x, y;\n .reg .b64 db;\n add.u32 x, %1, %4;\n add.u32 y, %2, %5;\n"
            " mov.b64 db, {y, %6};\n setp.ne.b32 p, %7, 0;\n"
            " tcgen05.mma.cta_group::1.kind::f16 [%0], [x], db, %3, p;\n}\n" ::"r"(d), "r"(a), "r"(b), "r"(id), "n"(AO),
            "n"(BO), "r"(kDescHi), "n"(ACC));
}
// S = Q K^T: HD / 16 k-steps, four to a 64-column block
template <int HD, int KK = 0>
__device__ __forceinline__ void mma_scores(uint32_t d, uint32_t q, uint32_t k, uint32_t id) {
    if constexpr (KK < HD / 16) {
        constexpr int o = (KK >> 2) * (kBlk >> 4) + 2 * (KK & 3);
        mma_ss<o, o, (KK > 0)>(d, q, k, id);
        mma_scores<HD, KK + 1>(d, q, k, id);
    }
}
// O (+)= P V: 8 k-steps of 16 keys, P's words 8 TMEM columns apart, V's rows 2048 bytes
template <int KK = 0>
__device__ __forceinline__ void mma_outputs(uint32_t d, uint32_t p, uint32_t v, uint32_t id, uint32_t acc) {
    if constexpr (KK < kKeys / 16) {
        mma_ts<8 * KK, KK * (2048 >> 4), (KK > 0) ? 1 : 2>(d, p, v, id, acc);
        mma_outputs<KK + 1>(d, p, v, id, acc);
    }
}
__device__ __forceinline__ bool elect_one() {
    uint32_t x;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(x));
    return x != 0;
}
__device__ __forceinline__ void commit(uint64_t* b) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(sa(b)) : "memory");
}

#define R8(r, o) "=r"(r[o]), "=r"(r[o + 1]), "=r"(r[o + 2]), "=r"(r[o + 3]), "=r"(r[o + 4]), "=r"(r[o + 5]), "=r"(r[o + 6]), "=r"(r[o + 7])
#define W8(r, o) "r"(r[o]), "r"(r[o + 1]), "r"(r[o + 2]), "r"(r[o + 3]), "r"(r[o + 4]), "r"(r[o + 5]), "r"(r[o + 6]), "r"(r[o + 7])
// this thread's lane, 32 columns from taddr; warp-wide, and waited for by ld_wait
__device__ __forceinline__ void tld32(uint32_t taddr, uint32_t* r) {
    __syncwarp();
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : R8(r, 0), R8(r, 8), R8(r, 16), R8(r, 24) : "r"(taddr));
}
__device__ __forceinline__ void ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tst32(uint32_t taddr, const uint32_t* r) {
    __syncwarp();
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr), W8(r, 0), W8(r, 8), W8(r, 16), W8(r, 24)
        : "memory");
}
__device__ __forceinline__ void st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
#undef R8
#undef W8

// two float32 numbers in a register pair, for the instructions that work on both
__device__ __forceinline__ uint64_t pair(float x, float y) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(x), "f"(y));
    return d;
}
__device__ __forceinline__ void unpair(uint64_t d, float& x, float& y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(d)); }
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t s, uint64_t b) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(x), "l"(s), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
    return d;
}

template <bool BF>
__device__ __forceinline__ uint32_t pack(float x, float y) {
    if constexpr (BF) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __half2 h = __floats2half2_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}

// byte offset of 16-byte chunk ch of row r in a swizzled tile
__device__ __forceinline__ uint32_t swz(int r, int ch) {
    return (uint32_t)((ch >> 3) * kBlk + r * 128 + ((((uint32_t)ch & 7u) ^ ((uint32_t)r & 7u)) << 4));
}

// How bulk tensor copies find a cell: maps of K and V as [page][head][cell][dim] (one page of all cells where
// the pages follow each other evenly), in boxes of `rows` cells x 64 dims (rows = 0: none).
// even: the maps have one page. aligned: the plan's blocks of keys are whole runs.
struct TmaRuns { int rows; bool even, aligned; };

template <int N>
struct Ring {                                              // position in the ring of K and V tiles
    uint32_t s = 0, ph = 0;
    __device__ __forceinline__ void next() { if (++s == N) { s = 0; ph ^= 1u; } }
};
struct MetaAt {
    uint32_t s = 0, ph = 0;
    __device__ __forceinline__ void next() { if (++s == kMeta) { s = 0; ph ^= 1u; } }
};

// The least and the largest position of a unit's rows.
__device__ __forceinline__ void unit_positions(const AttnPagedArgs& a, const AttnUnit& u, int& pmin, int& pmax) {
    const int r1 = u.row0 + u.n_row - 1;
    pmin = row_pos(a, u, u.row0, row_token(a, u, u.row0));
    pmax = row_pos(a, u, r1, row_token(a, u, r1));
    if (a.tok_pos)                                          // any order: over all of the unit's tokens
        for (int r = u.row0; r <= r1; r += a.G) {
            const int p = row_pos(a, u, r, row_token(a, u, r));
            pmin = min(pmin, p);
            pmax = max(pmax, p);
        }
}

// A key that a producer lane brings: byte offset of its row (-1: not read), position, cell, scale.
struct Key { int64_t off; int pos, cell; float s; };

// Keys 32 i + lane of a unit's block j. First every load of a kind, then what follows from them (one key after the
// other, each would wait for memory by itself).
template <bool F8>
__device__ __forceinline__ void look_up(const AttnPagedArgs& a, const AttnUnit& u, int j, int pmax, int hid_all,
                                        const float* scales, Key* k) {
    const int v = u.v0 + j * kKeys + (threadIdx.x & 31), ps = a.kv.page_size;
    const int sh = (ps & (ps - 1)) == 0 ? __ffs(ps) - 1 : -1;
    int page[4], at[4];
    bool past = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int w = min(v + 32 * i, u.v1 - 1);
        const int x = w < u.n_sink_keys ? w : w - u.n_sink_keys + u.key_lo;
        const int pg = sh >= 0 ? x >> sh : x / ps;
        at[i] = x - pg * ps;
        k[i].pos = x;
        page[i] = a.table[u.table + pg];
    }
    if (a.key_pos)
#pragma unroll
        for (int i = 0; i < 4; ++i) k[i].pos = a.key_pos[u.table + k[i].pos];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool there = v + 32 * i < u.v1, bad = (unsigned)page[i] >= (unsigned)a.kv.n_pages;
        const bool seen = there && !bad && sees(k[i].pos, pmax, hid_all, a.n_sink);
        past = past || (there && bad);
        k[i].cell = page[i] * ps + at[i];
        k[i].off = seen ? (int64_t)page[i] * a.kv.sb_page + (int64_t)at[i] * a.kv.sb_cell : -1;
        if (!seen) k[i].pos = INT_MAX;
        k[i].s = 0.f;
        if constexpr (F8)
            if (seen) k[i].s = scales[(int64_t)page[i] * a.kv.ss_page + (int64_t)at[i] * a.kv.ss_cell];
    }
    if (past && a.err) atomicOr(a.err, ERR_SLOT_RANGE);
}

// s / s0 between which q * s / s0 is exact in f16: the least E4M3 number is 2^-9, the largest 448
constexpr float kRatioMin = 0x1p-15f, kRatioMax = 0x1p7f;

// whether an E4M3 row of n bytes is zeros (rarely asked: few instructions, and no call, which would cost its caller's
// registers)
__device__ __forceinline__ bool row_is_zero(const uint8_t* row, int n) {
    uint32_t bits = 0u;
#pragma unroll 1
    for (int i = 0; i < n; i += 16) {
        const uint4 x = *reinterpret_cast<const uint4*>(row + i);
        bits |= x.x | x.y | x.z | x.w;
    }
    return (bits & 0x7f7f7f7fu) == 0u;
}

template <int HD, int CT, int QT>
__global__ void __launch_bounds__(kThr, 1) attn_tc_rows_kernel(AttnPagedArgs a, TmaRuns runs, int beside,
                                                               const __grid_constant__ CUtensorMap map_k,
                                                               const __grid_constant__ CUtensorMap map_v) {
    using M = Smem<HD>;
    constexpr bool F8 = CT == W_F8, BF = CT == W_BF16;
    constexpr int CH = HD / 8;                              // 16-byte chunks of a 16-bit row
    constexpr int NS = F8 ? kStages - 1 : kStages;
    extern __shared__ __align__(1024) uint8_t sm[];
    int* kpos = reinterpret_cast<int*>(sm + M::kpos);
    volatile uint32_t* full = reinterpret_cast<volatile uint32_t*>(sm + M::full);
    float* rs_s = reinterpret_cast<float*>(sm + M::rs);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + M::bars);
    uint64_t* kv_full = bars;                               // [kStages] 1: the producing warp (and its bulk copies' bytes)
    uint64_t* kv_empty = bars + kStages;                    // [kStages] 1: MMA commit
    uint64_t* s_full = bars + 2 * kStages;                  // [2] 1: MMA commit
    uint64_t* p_full = s_full + 2;                          // [2] 128: the softmax threads
    uint64_t* o_done = p_full + 2;                          // [2] 1: MMA commit after the unit's last product
    uint64_t* q_full = o_done + 2;                          // 1: the loading warp, or 256: the softmax threads
    // [kMeta] a block's positions. Slot j % 3 is written again for block j + 3, whose K tile needs the
    // ring place of V tile j (five stages) or K tile j + 1 (four), freed after both halves' softmax of block j.
    uint64_t* meta_full = q_full + 1;
    uint64_t* q_empty = meta_full + kMeta;                  // 1: MMA commit after the unit's last scores
    uint64_t* drained = q_empty + 1;                        // 1: MMA commit after a wait that gave up
    static_assert(2 * kStages + 7 + kMeta + 2 <= 24, "places of the barriers");
    int* misc = reinterpret_cast<int*>(sm + M::misc);
    volatile int* abort_f = misc;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc + 2);
    // of the units with keys a producer may look at the fourth ahead (a unit has two tiles at least): by unit % 8
    volatile int* redo_f = misc + 4;                        // [8] the unit has to be done again
    float* s0 = reinterpret_cast<float*>(misc + 12);        // [8][2] E4M3: scale of the K and V tiles

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // beside: the small tiles of the same plan run just before; nothing here depends on them, so this kernel
    // starts where they leave SMs free, and waits for them at its end
    asm volatile("griddepcontrol.launch_dependents;");
    if (form_missing(a)) return;
    if (sa(sm) & 1023u) {                                   // the swizzle patterns repeat every 1024 bytes
        if (tid == 0 && a.err) atomicOr(a.err, ERR_TIMEOUT);
        return;
    }
    const int ui0 = a.first2[blockIdx.x], ui1 = a.first2[blockIdx.x + 1];
    if ((a.hdr[PH_FORM] & ATTN_FORM_TC) == 0 || ui0 >= ui1) {
        if (beside) asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }

    // Q rows that are changed on their way (scaled to f16's range, rounded to f16, negated for a negative scale) are
    // loaded by the softmax threads; others by warp 3, while the unit before is still in its last block and its epilogue
    constexpr bool SCALED = !BF && QT != W_F16;
    const bool own_q = F8 || SCALED || a.scale_log2 < 0.f;   // (E4M3: warp 3 is a producer)
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) { bar_init(&kv_full[i], 1); bar_init(&kv_empty[i], 1); }
        for (int i = 0; i < 2; ++i) { bar_init(&s_full[i], 1); bar_init(&p_full[i], 128); bar_init(&o_done[i], 1); }
        bar_init(q_full, own_q ? 256 : 1);
        bar_init(q_empty, 1);
        bar_init(drained, 1);
        for (int i = 0; i < kMeta; ++i) bar_init(&meta_full[i], 1);
        *abort_f = 0;
        for (int i = 0; i < 8; ++i) redo_f[i] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sa(tmem_slot)), "r"(512u));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = *tmem_slot;

    auto wait = [&](uint64_t* b, uint32_t par) -> bool {
        if (bar_try(b, par)) return true;
        const uint64_t t0 = now_ns();
        while (!bar_try(b, par)) {
            if (*abort_f) return false;
            if (now_ns() - t0 > kWaitNs) {
                if (a.err) atomicOr(a.err, ERR_TIMEOUT);
                *abort_f = 1;
                return false;
            }
        }
        return true;
    };

    // Each role walks the CTA's units by itself; the barriers above keep them in step. Registers: three warpgroups
    // of 168 a thread at launch, 504 >= kRegsLow + 2 kRegsHigh. What is spilled comes back from L2 (shared memory
    // leaves L1 little), so both parts count: 2048 new tokens at the end of 32768 E4M3 keys (32 / 8 heads of 128) took
    // 5360 us with 120 + 192 and 3720 us with 152 + 176 while producers held raw rows in registers; with the raw rows in
    // shared memory 1240 us with 104 + 200 and 1190 us as here.
    constexpr int kRegsLow = F8 ? 120 : 88, kRegsHigh = F8 ? 192 : 208;
    static_assert(kRegsLow + 2 * kRegsHigh <= 3 * 168, "registers of the launch");
    Ring<NS> ring;
    MetaAt meta;
    if (warp < kSoft0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLow));
        if (F8 && warp != kMmaWarp) {
            // ---- E4M3: three producers take the tiles K, V, K, V ... in turn (two, one for K and one for V: 1300 us
            // instead of 1190). Raw rows travel by asynchronous
            // copies into a producer's part of the ring's last place, a tile in eight pieces of 16 rows, the fifth
            // piece to come brought as soon as one is converted: three or four are under way all the time, and none in
            // registers. A lane converts the bytes that it copied. Lanes of a quarter warp hold two rows' chunks of
            // one 64-column block, so that their stores' banks differ (eight chunks of one row, all even, would
            // meet in pairs); the raw rows' halves are swapped in odd rows for the same reason.
            constexpr int LR = HD / 16;                     // lanes per row, 16 values each
            constexpr int RI = 32 / LR;                     // rows at a time
            constexpr int BX = 16 / RI;                     // ... times in a piece
            constexpr int PR = 3;
            static_assert(PR * 64 * HD <= (int)M::tile, "raw rows in the ring's last place");
            const int pr = warp == 3 ? 2 : warp;
            const int lr = LR == 8 ? ((lane >> 2) & 1) | ((lane >> 4) << 1) : lane / LR;
            const int lc = LR == 8 ? (lane & 3) | ((lane >> 1) & 4) : lane % LR;
            const uint8_t* const raw = sm + M::kv + NS * M::tile + pr * 64 * HD + lr * HD +
                                       16 * (LR == 8 ? lc ^ ((lr & 1) << 2) : lc);
            const uint32_t raw_s = sa(raw);
            uint32_t before = 0;                            // tiles of the units before
            int with_keys = 0;                              // units with keys
            bool ok = true;
            for (int ui = ui0; ui < ui1 && ok; ++ui) {
                const AttnUnit u = load_unit(a.units2 + ui);
                const int n_tile = 2 * ((u.v1 - u.v0 + kKeys - 1) / kKeys);
                if (n_tile == 0) continue;
                const int slot = with_keys++ & 7;
                int pmin, pmax;
                unit_positions(a, u, pmin, pmax);
                const int hid_all = hidden_below(a, pmin);
                auto scales = [&](int x) { return ((x & 1) ? a.kv.vs : a.kv.ks) + (int64_t)u.head * a.kv.ss_head; };
                auto rows_of = [&](int x) { return ((x & 1) ? a.kv.v : a.kv.k) + (int64_t)u.head * a.kv.sb_head; };
                Key cur[4], nxt[4];
                auto bring = [&](int64_t row_off, int x, int q) {   // piece q of tile x, its rows' offsets in the lanes
                    const uint8_t* base = rows_of(x) + 16 * lc;
#pragma unroll
                    for (int y = 0; y < BX; ++y) {
                        const int64_t off = __shfl_sync(0xffffffffu, row_off, 16 * (q & 1) + y * RI + lr);
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(raw_s + (16 * (q & 3) + y * RI) * HD),
                                     "l"(base + (off >= 0 ? off : 0)), "r"(off >= 0 ? 16 : 0) : "memory");
                    }
                };
                float inv[2];                               // s0 of this unit: the largest scale of its first block
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    look_up<true>(a, u, 0, pmax, hid_all, scales(v), cur);
                    if (__any_sync(0xffffffffu, cur[0].s == 1.f || cur[1].s == 1.f || cur[2].s == 1.f || cur[3].s == 1.f))
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (cur[i].s == 1.f && row_is_zero(rows_of(v) + cur[i].off, HD)) cur[i].s = 0.f;
                    float mx = fmaxf(fmaxf(cur[0].s, cur[1].s), fmaxf(cur[2].s, cur[3].s));
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                    if (!(mx > 0.f)) mx = 1.f;
                    if (lane == 0) s0[2 * slot + v] = mx;   // (the same from each producer)
                    inv[v] = 1.f / mx;
                }
                int x = (int)((pr + 2 * before) % PR);      // the first tile of this producer: (before + x) % PR = pr
                if (x < n_tile) {
                    look_up<true>(a, u, x >> 1, pmax, hid_all, scales(x), cur);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        bring(cur[q >> 1].off, x, q);
                        asm volatile("cp.async.commit_group;" ::: "memory");
                    }
                }
                for (; x < n_tile; x += PR) {
                    const uint32_t it = before + x, stage = it % NS, ph = (it / NS) & 1u;
                    uint8_t* const dst = sm + M::kv + stage * M::tile;
                    const bool is_v = x & 1, more = x + PR < n_tile;
                    if (more) look_up<true>(a, u, (x + PR) >> 1, pmax, hid_all, scales(x + PR), nxt);
                    bool all = true, fits = true;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        cur[i].s *= is_v ? inv[1] : inv[0];
                        all = all && cur[i].off >= 0;
                        fits = fits && (cur[i].off < 0 || (cur[i].s >= kRatioMin && cur[i].s <= kRatioMax));
                    }
                    all = __all_sync(0xffffffffu, all);
                    if (!__all_sync(0xffffffffu, fits))
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (cur[i].off >= 0 && !(cur[i].s >= kRatioMin && cur[i].s <= kRatioMax)) {
                                // f16 would not hold it, unless it is zeros
                                if (cur[i].s != cur[i].s || !row_is_zero(rows_of(x) + cur[i].off, HD)) redo_f[slot] = 1;
                                cur[i].s = 0.f;
                            }
                    ok = it < NS || wait(&kv_empty[stage], ph ^ 1u);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
#pragma unroll 1
                    for (int q = 0; q < 8; ++q) {
                        asm volatile("cp.async.wait_group 3;" ::: "memory");
                        float sq = cur[0].s;
#pragma unroll
                        for (int i = 1; i < 4; ++i) if (q >> 1 == i) sq = cur[i].s;
                        uint4 in[BX];                       // (all read before the first store: the two might alias)
                        __half2 fh[BX];
#pragma unroll
                        for (int y = 0; y < BX; ++y) {
                            in[y] = *reinterpret_cast<const uint4*>(raw + (16 * (q & 3) + y * RI) * HD);
                            fh[y] = __float2half2_rn(__shfl_sync(0xffffffffu, sq, 16 * (q & 1) + y * RI + lr));
                        }
#pragma unroll
                        for (int y = 0; y < BX; ++y) {
                            const uint32_t w[4] = {in[y].x, in[y].y, in[y].z, in[y].w};
                            uint32_t h[8];
#pragma unroll
                            for (int i = 0; i < 4; ++i) e4m3x4_to_h2(w[i], h[2 * i], h[2 * i + 1]);
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const __half2 z = __hmul2(*reinterpret_cast<const __half2*>(&h[i]), fh[y]);
                                h[i] = *reinterpret_cast<const uint32_t*>(&z);
                            }
                            const int row = 16 * q + y * RI + lr;
                            *reinterpret_cast<uint4*>(dst + swz(row, 2 * lc)) = make_uint4(h[0], h[1], h[2], h[3]);
                            *reinterpret_cast<uint4*>(dst + swz(row, 2 * lc + 1)) = make_uint4(h[4], h[5], h[6], h[7]);
                        }
                        if (q < 4) bring(q < 2 ? cur[2].off : cur[3].off, x, q + 4);
                        else if (more) bring(q < 6 ? nxt[0].off : nxt[1].off, x + PR, q - 4);
                        asm volatile("cp.async.commit_group;" ::: "memory");
                    }
                    const int m = (int)((it >> 1) % kMeta);
                    if (!is_v) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) kpos[m * kKeys + 32 * i + lane] = cur[i].pos;
                        if (lane == 0) full[m] = all;
                    }
                    to_async_proxy();
                    __syncwarp();
                    if (lane == 0) {
                        bar_arrive(&kv_full[stage]);
                        if (!is_v) bar_arrive(&meta_full[m]);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) cur[i] = nxt[i];
                }
                before += n_tile;
            }
            if (!ok) asm volatile("cp.async.wait_group 0;" ::: "memory");
        } else if (!F8 && warp < kProdWarps) {
            // ---- K (warp 0) and V (warp 1) tiles, the even and odd ones of the ring
            const bool is_v = warp == 1;
            uint32_t it = is_v ? 1 : 0;                     // tile number, over all units
            bool ok = true;
            int bulk_at[kStages];                           // phase of a stage's last bulk copies, -1: none
#pragma unroll
            for (int i = 0; i < kStages; ++i) bulk_at[i] = -1;
            const uint64_t map = reinterpret_cast<uint64_t>(is_v ? &map_v : &map_k);
            for (int ui = ui0; ui < ui1 && ok; ++ui) {
                const AttnUnit u = load_unit(a.units2 + ui);
                const int kvh = u.head;
                const int nt = (u.v1 - u.v0 + kKeys - 1) / kKeys;
                if (nt == 0) continue;
                const uint8_t* base = (is_v ? a.kv.v : a.kv.k) + (int64_t)kvh * a.kv.sb_head;
                int pmin, pmax;
                unit_positions(a, u, pmin, pmax);
                const int hid_all = hidden_below(a, pmin);
                // Blocks that need no look at single keys: positions are indices, the block's pages hold whole runs, and
                // some row sees each key. A lane brings one box of 64 dims x runs.rows cells.
                constexpr int HB = HD / 64;
                const int n_box = runs.rows > 0 ? kKeys / runs.rows * HB : 0;
                const bool paged = runs.rows > 0 && runs.aligned && !a.key_pos;
                auto plain = [&](int j) {
                    const int v = u.v0 + j * kKeys;
                    if (!paged || v + kKeys > u.v1) return false;
                    if (v < u.n_sink_keys) return v + kKeys <= u.n_sink_keys && v + kKeys <= min(a.n_sink, pmax + 1);
                    const int k = v - u.n_sink_keys + u.key_lo;
                    return k + kKeys - 1 <= pmax && (k > hid_all || k + kKeys <= a.n_sink);
                };
                auto box_page = [&](int j, int& at) {       // this lane's page, its first cell there
                    const int v = u.v0 + j * kKeys + (lane < n_box ? lane / HB : 0) * runs.rows;
                    const int k = v < u.n_sink_keys ? v : v - u.n_sink_keys + u.key_lo;
                    const int ps = a.kv.page_size, pg = (ps & (ps - 1)) == 0 ? k >> (__ffs(ps) - 1) : k / ps;
                    at = k - pg * ps;
                    return a.table[u.table + pg];
                };
                int page_nxt = 0, at_nxt = 0;
                bool plain_nxt = plain(0);
                if (plain_nxt) page_nxt = box_page(0, at_nxt);
                // row copies are announced one tile of this warp's later, when they have landed (not two: K tile
                // j + 2 needs the place of V tile j - 1, which is not free before the scores of block j)
                int pend = -1;                              // stage
                auto announce = [&](uint32_t s) {
                    to_async_proxy();
                    __syncwarp();
                    if (lane == 0) bar_arrive(&kv_full[s]);
                };
                auto flush = [&]() {
                    if (pend < 0) return;
                    asm volatile("cp.async.wait_group 0;" ::: "memory");
                    announce(pend);
                    pend = -1;
                };
                for (int j = 0; j < nt; ++j, it += 2) {
                    const uint32_t stage = it % NS, ph = (it / NS) & 1u;
                    uint8_t* const dst = sm + M::kv + stage * M::tile;
                    const uint32_t fb = sa(&kv_full[stage]);
                    auto claim = [&]() {
                        ok = it < NS || wait(&kv_empty[stage], ph ^ 1u);
                        ok = __all_sync(0xffffffffu, ok);
                        return ok;
                    };
                    auto box = [&](uint32_t d, int h, int cell, int page) {
                        asm volatile(
                            "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
                            " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(d), "l"(map), "r"(fb), "r"(64 * h), "r"(cell),
                            "r"(kvh), "r"(page) : "memory");
                    };
                    auto expect = [&]() {
                        if (lane == 0)
                            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(fb),
                                         "r"(kKeys * HD * 2) : "memory");
                        __syncwarp();
                        bulk_at[stage] = (int)ph;
                    };
                    const int page = page_nxt, at = at_nxt;
                    bool now = plain_nxt;
                    plain_nxt = j + 1 < nt && plain(j + 1);
                    if (plain_nxt) page_nxt = box_page(j + 1, at_nxt);
                    if (now && __any_sync(0xffffffffu, (unsigned)page >= (unsigned)a.kv.n_pages)) now = false;
                    if (now) {
                        flush();
                        if (!claim()) break;
                        expect();
                        if (lane < n_box) {
                            const int k = lane / HB * runs.rows, h = lane % HB;
                            box(sa(dst) + h * kBlk + k * 128, h, runs.even ? page * a.kv.page_size + at : at, runs.even ? 0 : page);
                        }
                        if (!is_v) {
                            const int v = u.v0 + j * kKeys, p0 = v < u.n_sink_keys ? v : v - u.n_sink_keys + u.key_lo;
                            reinterpret_cast<int4*>(kpos + meta.s * kKeys)[lane] =
                                make_int4(p0 + 4 * lane, p0 + 4 * lane + 1, p0 + 4 * lane + 2, p0 + 4 * lane + 3);
                            if (lane == 0) full[meta.s] = 1u;
                        }
                    } else {
                        Key cur[4];
                        look_up<false>(a, u, j, pmax, hid_all, nullptr, cur);
                        bool all = true;
#pragma unroll
                        for (int i = 0; i < 4; ++i) all = all && cur[i].off >= 0;
                        all = __all_sync(0xffffffffu, all);
                        {
                            // runs of neighbouring cells among single cells
                            bool run = runs.rows > 0 && all;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int prev = __shfl_up_sync(0xffffffffu, cur[i].cell, 1);
                                const int last = __shfl_sync(0xffffffffu, cur[i > 0 ? i - 1 : 0].cell, 31);
                                const bool starts = ((32 * i + lane) & (runs.rows - 1)) == 0;
                                run = run && (starts ? runs.even || cur[i].cell % a.kv.page_size + runs.rows <= a.kv.page_size
                                                     : cur[i].cell == (lane > 0 ? prev : last) + 1);
                            }
                            run = __all_sync(0xffffffffu, run);
                            if (run) flush();
                            if (!claim()) break;
                            if (run) {
                                expect();
                                const int k = lane < n_box ? lane / HB * runs.rows : 0, h = lane % HB;
                                int c = 0;
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const int ci = __shfl_sync(0xffffffffu, cur[i].cell, k & 31);
                                    if (k >> 5 == i) c = ci;
                                }
                                if (lane < n_box) {
                                    const int pg = runs.even ? 0 : c / a.kv.page_size;
                                    box(sa(dst) + h * kBlk + k * 128, h, c - pg * a.kv.page_size, pg);
                                }
                            } else {
                                constexpr int RI = 32 / CH; // rows per instruction
                                const int ch = lane % CH, r0 = lane / CH;
#pragma unroll
                                for (int i = 0; i < 4; ++i)
#pragma unroll 4
                                    for (int x = 0; x < 32 / RI; ++x) {
                                        const int r = r0 + x * RI;
                                        const int64_t off = __shfl_sync(0xffffffffu, cur[i].off, r);
                                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sa(dst) + swz(32 * i + r, ch)),
                                                     "l"(base + (off >= 0 ? off : 0) + 16 * ch), "r"(off >= 0 ? 16 : 0) : "memory");
                                    }
                                asm volatile("cp.async.commit_group;" ::: "memory");
                                if (pend >= 0) {
                                    asm volatile("cp.async.wait_group 1;" ::: "memory");
                                    announce(pend);
                                }
                                pend = (int)stage;
                            }
                        }
                        if (!is_v) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) kpos[meta.s * kKeys + 32 * i + lane] = cur[i].pos;
                            if (lane == 0) full[meta.s] = all;
                        }
                    }
                    if (!is_v) {
                        __syncwarp();
                        if (lane == 0) bar_arrive(&meta_full[meta.s]);
                        meta.next();
                    }
                }
                flush();
            }
            // after a wait that gave up nobody may wait for the copies under way: they land before the CTA leaves
            if (!ok) {
                asm volatile("cp.async.wait_group 0;" ::: "memory");
                for (int i = 0; i < kStages; ++i) {
                    const uint64_t t0 = now_ns();
                    while (bulk_at[i] >= 0 && !bar_try(&kv_full[i], (uint32_t)bulk_at[i]) && now_ns() - t0 < kWaitNs) {}
                }
            }
        } else if (warp == kMmaWarp) {
            // ---- MMA issuer
            constexpr uint32_t ids = idesc(BF, 128, kKeys, false), ido = idesc(BF, 128, HD, true);
            uint32_t q_ph = 0, p_ph[2] = {0u, 0u};
            const bool leader = elect_one();
            const uint32_t qd = desc_k(sa(sm + M::q)), kd = desc_k(sa(sm + M::kv)), vd = desc_mn(sa(sm + M::kv));
            bool ok = true;
            // the warp goes on, or gives up, as one: it meets at warp barriers between the waits
            auto wait_all = [&](uint64_t* b, uint32_t par) -> bool { return __all_sync(0xffffffffu, wait(b, par)); };
            for (int ui = ui0; ui < ui1 && ok; ++ui) {
                const AttnUnit u = load_unit(a.units2 + ui);
                const int nt = (u.v1 - u.v0 + kKeys - 1) / kKeys, halves = u.n_row > 128 ? 2 : 1;
                if (nt == 0) continue;
                ok = wait_all(q_full, q_ph);
                q_ph ^= 1u;
                auto scores = [&](int t, uint32_t stage) {
                    const uint32_t q = qd + t * (M::tile >> 4), k = kd + stage * (M::tile >> 4), d = tmem + 128 * t;
                    if (leader) {
                        mma_scores<HD>(d, q, k, ids);
                        commit(&s_full[t]);
                    }
                    __syncwarp();                           // (the others do not spin on a barrier before it has issued)
                };
                ok = ok && wait_all(&kv_full[ring.s], ring.ph);
                if (ok) {
                    tc_after();
                    for (int t = 0; t < halves; ++t) scores(t, ring.s);
                    if (leader) commit(&kv_empty[ring.s]);
                    if (leader && nt == 1) commit(q_empty);
                    __syncwarp();
                    ring.next();
                }
                for (int j = 0; j < nt && ok; ++j) {
                    const Ring<NS> rv = ring;
                    ring.next();
                    const Ring<NS> rk = ring;
                    const bool more = j + 1 < nt;
                    if (!(ok = wait_all(&kv_full[rv.s], rv.ph))) break;
                    const uint32_t v = vd + rv.s * (M::tile >> 4);
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (t >= halves) break;
                        if (!(ok = wait_all(&p_full[t], p_ph[t]))) break;
                        p_ph[t] ^= 1u;
                        tc_after();
                        if (leader) {
                            mma_outputs(tmem + 256 + 128 * t, tmem + 128 * t + 64, v, ido, j > 0);
                            if (t == halves - 1) commit(&kv_empty[rv.s]);
                        }
                        __syncwarp();
                        if (more) {
                            if (t == 0 && !(ok = wait_all(&kv_full[rk.s], rk.ph))) break;
                            tc_after();
                            scores(t, rk.s);
                        } else if (leader) {
                            commit(&o_done[t]);
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                    if (more) {
                        if (leader) commit(&kv_empty[rk.s]);
                        if (leader && j + 2 == nt) commit(q_empty);
                        __syncwarp();
                        ring.next();
                    }
                }
            }
            // after a wait that gave up, products under way end before shared memory and TMEM are given back
            if (!ok) {
                if (leader) commit(drained);
                __syncwarp();
                const uint64_t t0 = now_ns();
                while (!bar_try(drained, 0) && now_ns() - t0 < kWaitNs) {}
            }
        } else if (!F8 && warp == 3 && !own_q) {
            // ---- Q tiles: a lane copies 16 bytes, CH lanes a row
            constexpr int RI = 32 / CH;                     // rows per copy
            uint32_t e_ph = 1;                              // (the first unit waits for nothing)
            bool ok = true;
            for (int ui = ui0; ui < ui1 && ok; ++ui) {
                const AttnUnit u = load_unit(a.units2 + ui);
                if (u.v1 <= u.v0) continue;
                int64_t at[8];                              // where rows 8 lane .. 8 lane + 7 lie, -1: past the unit
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int r = 8 * lane + i, row = u.row0 + r;
                    at[i] = -1;
                    if (r < u.n_row) {
                        const int tok = row_token(a, u, row);
                        at[i] = ((int64_t)tok * a.q_tok + (int64_t)(u.head * a.G + row % a.G) * a.q_head) * 2;
                    }
                }
                ok = __all_sync(0xffffffffu, wait(q_empty, e_ph));
                if (!ok) break;
                e_ph ^= 1u;
#pragma unroll 1
                for (int l = 0; l < 32 / RI; ++l)           // rows 8 (l RI + lane / CH) + i
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int from = l * RI + lane / CH, r = 8 * from + i, ch = lane % CH;
                        const int64_t o = __shfl_sync(0xffffffffu, at[i], from);
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                         sa(sm + M::q + (r >> 7) * M::tile) + swz(r & 127, ch)),
                                     "l"(static_cast<const uint8_t*>(a.q) + (o >= 0 ? o : 0) + 16 * ch), "r"(o >= 0 ? 16 : 0)
                                     : "memory");
                    }
                asm volatile("cp.async.commit_group;" ::: "memory");
                asm volatile("cp.async.wait_group 0;" ::: "memory");
                to_async_proxy();
                __syncwarp();
                if (lane == 0) bar_arrive(q_full);
            }
        }
        __syncwarp();
    } else {
        // ---- the two halves: Q tile, softmax, epilogue
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsHigh));
        const int t = warp >= kSoft0 + 4 ? 1 : 0;
        const int ht = tid - 32 * (kSoft0 + 4 * t);         // thread of the half
        uint32_t s_ph = 0, o_ph = 0;
        int with_keys = 0, done = ui1;                      // units before `done` are written, or marked in redo2
        bool again = false;
        AttnUnit u = load_unit(a.units2 + ui0);
        for (int ui = ui0; ui < ui1; ++ui) {
            const int kvh = u.head;
            const int nt = (u.v1 - u.v0 + kKeys - 1) / kKeys, halves = u.n_row > 128 ? 2 : 1;
            const int slot = with_keys & 7;
            if (nt > 0) ++with_keys;
            if (nt > 0 && own_q) {
                // neighbouring threads hold a row: 8 values each
                uint8_t* qs = sm + M::q + t * M::tile;
                constexpr int RQ = 128 / CH;                // rows the half loads at once
                const int ch = ht % CH;
#pragma unroll 1
                for (int r0 = ht / CH; r0 < 128; r0 += 8 * RQ) {
                uint4 qv[8];                                // eight loads under way (float32: rounded below)
                float rq[8];                                // scale of the row's scores
                float4 fq[QT == W_F32 ? 16 : 1];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int r = r0 + i * RQ, row = u.row0 + 128 * t + r;
                    qv[i] = make_uint4(0u, 0u, 0u, 0u);
                    if constexpr (QT == W_F32) fq[2 * i] = fq[2 * i + 1] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (128 * t + r < u.n_row) {
                        const int tok = row_token(a, u, row);
                        const int64_t at = (int64_t)tok * a.q_tok + (int64_t)(kvh * a.G + row % a.G) * a.q_head + ch * 8;
                        if constexpr (QT == W_F32) {
                            const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + at);
                            const float4 x = p[0], y = p[1];
                            fq[2 * i] = x;
                            fq[2 * i + 1] = y;
                        } else {
                            qv[i] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + at);
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    rq[i] = fabsf(a.scale_log2);
                    if constexpr (SCALED) {
                        // f16 products: the row times a power of two that brings its largest value to [1, 2)
                        float x[8];
                        if constexpr (QT == W_F32) {
                            x[0] = fq[2 * i].x; x[1] = fq[2 * i].y; x[2] = fq[2 * i].z; x[3] = fq[2 * i].w;
                            x[4] = fq[2 * i + 1].x; x[5] = fq[2 * i + 1].y; x[6] = fq[2 * i + 1].z; x[7] = fq[2 * i + 1].w;
                        } else {
                            const uint32_t w[4] = {qv[i].x, qv[i].y, qv[i].z, qv[i].w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                x[2 * e] = __uint_as_float(w[e] << 16);
                                x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
                            }
                        }
                        float mx = 0.f;
#pragma unroll
                        for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(x[e]));
#pragma unroll
                        for (int o = CH / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                        const uint32_t ex = __float_as_uint(mx) >> 23;
                        float dn = 1.f;
                        if (ex > 0u && ex < 254u) {
                            dn = __uint_as_float((254u - ex) << 23);
                            rq[i] *= __uint_as_float(ex << 23);
                        }
                        qv[i] = make_uint4(pack<false>(x[0] * dn, x[1] * dn), pack<false>(x[2] * dn, x[3] * dn),
                                           pack<false>(x[4] * dn, x[5] * dn), pack<false>(x[6] * dn, x[7] * dn));
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int r = r0 + i * RQ;
                    const uint4 w = qv[i];
                    uint32_t v[4] = {w.x, w.y, w.z, w.w};
                    if (a.scale_log2 < 0.f)                 // the scores' scale is positive, the sign is in Q
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[e] ^= 0x80008000u;
                    *reinterpret_cast<uint4*>(qs + swz(r, ch)) = make_uint4(v[0], v[1], v[2], v[3]);
                    if (SCALED && ch == 0) rs_s[128 * t + r] = rq[i];
                }
                }
                to_async_proxy();
                // the rows' scales are read by other threads of the half
                asm volatile("bar.sync %0, 128;" ::"r"(2 + t) : "memory");
                bar_arrive(q_full);
            }
            const int r = 32 * (warp & 3) + lane;           // this thread's row of the half, its TMEM lane
            const uint32_t lane_at = (uint32_t)(32 * (warp & 3)) << 16;
            const uint32_t sb = tmem + 128 * t + lane_at, ob = tmem + 256 + 128 * t + lane_at;
            const bool mine = 128 * t + r < u.n_row;
            const int row = u.row0 + min(128 * t + r, u.n_row - 1);
            const int tok = row_token(a, u, row);
            const int rp = row_pos(a, u, row, tok), rh = hidden_below(a, rp);
            const int wp_min = __reduce_min_sync(0xffffffffu, rp), wh_max = __reduce_max_sync(0xffffffffu, rh);
            float rs = SCALED && nt > 0 ? rs_s[128 * t + r] : fabsf(a.scale_log2);
            float m = -INFINITY, l = 0.f;
            bool live = t < halves;
            for (int j = 0; j < nt && live; ++j) {
                const bool got = wait(&meta_full[meta.s], meta.ph) && wait(&s_full[t], s_ph);
                if (!__all_sync(0xffffffffu, got)) { live = false; break; }
                tc_after();
                s_ph ^= 1u;
                if (F8 && j == 0) rs *= s0[2 * slot];
                const int* kp = kpos + meta.s * kKeys;
                const int4* kp4 = reinterpret_cast<const int4*>(kp);
                const bool open = full[meta.s] != 0u &&
                                  kp[kKeys - 1] <= wp_min && (kp[0] > wh_max || kp[kKeys - 1] < a.n_sink);
                if (!open) {
                    // some row does not see some key: -inf over those scores, in TMEM (few blocks do this; the code
                    // of the others stays short enough for the instruction cache)
#pragma unroll 1
                    for (int c = 0; c < kKeys; c += 32) {
                        uint32_t x[32];
                        tld32(sb + c, x);
                        ld_wait();
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            const int4 k = kp4[(c + i) / 4];
                            if (!sees(k.x, rp, rh, a.n_sink)) x[i] = __float_as_uint(-INFINITY);
                            if (!sees(k.y, rp, rh, a.n_sink)) x[i + 1] = __float_as_uint(-INFINITY);
                            if (!sees(k.z, rp, rh, a.n_sink)) x[i + 2] = __float_as_uint(-INFINITY);
                            if (!sees(k.w, rp, rh, a.n_sink)) x[i + 3] = __float_as_uint(-INFINITY);
                        }
                        tst32(sb + c, x);
                    }
                    st_wait();
                }
                uint32_t v[64], w[64];                      // the row's scores
                tld32(sb, v);
                tld32(sb + 32, v + 32);
                tld32(sb + 64, w);
                tld32(sb + 96, w + 32);
                ld_wait();
                float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
                for (int c = 0; c < 64; c += 2) {
                    t0 = fmaxf(fmaxf(t0, __uint_as_float(v[c])), __uint_as_float(v[c + 1]));
                    t1 = fmaxf(fmaxf(t1, __uint_as_float(w[c])), __uint_as_float(w[c + 1]));
                }
                const float mx = fmaxf(t0, t1) * rs;
                float f = 1.f;
                bool up = false;
                if (mx > m + 14.f) {
                    f = ex2(m - (mx - 6.f));                // 0 from nothing
                    m = mx - 6.f;
                    l *= f;
                    up = true;
                }
                // nothing seen: every score is -inf
                const uint64_t rs2 = pair(rs, rs), bias2 = m == -INFINITY ? 0ull : pair(-m, -m);
                uint64_t sum = 0ull;
                auto powers = [&](uint32_t* x) {            // 64 scores to 32 words of P
#pragma unroll
                    for (int c = 0; c < 64; c += 2) {
                        float p0, p1;
                        unpair(fma2(pair(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), rs2, bias2), p0, p1);
                        p0 = ex2(p0);
                        p1 = ex2(p1);
                        sum = add2(sum, pair(p0, p1));
                        x[c / 2] = pack<BF>(p0, p1);
                    }
                };
                // P over S's second half, which has been read
                powers(v);
                tst32(sb + 64, v);
                powers(w);
                tst32(sb + 96, w);
                float s0f, s1f;
                unpair(sum, s0f, s1f);
                l += s0f + s1f;
                // O is complete up to the block before (its products precede these scores)
                if (j > 0 && __any_sync(0xffffffffu, up)) {
#pragma unroll 1
                    for (int c = 0; c < HD; c += 32) {
                        uint32_t o[32];
                        tld32(ob + c, o);
                        ld_wait();
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                        tst32(ob + c, o);
                    }
                }
                st_wait();
                tc_before();
                bar_arrive(&p_full[t]);
                meta.next();
            }
            if (t >= halves)
                for (int j = 0; j < nt; ++j) meta.next();   // the other half's blocks
            if (live && nt > 0) {
                if (!__all_sync(0xffffffffu, wait(&o_done[t], o_ph))) live = false;
                o_ph ^= 1u;
                tc_after();
            }
            const AttnUnit u_nxt = load_unit(a.units2 + min(ui + 1, ui1 - 1));   // (on its way meanwhile)
            // ---- epilogue: a unit alone writes its rows, one of several its partial result
            if (live) {
                bool finite = l <= 3.0e38f && m <= 3.0e38f;
                const float inv = 1.f / l, none = l == 0.f ? weightless(a, u, row, tok) : 0.f, sv = F8 && nt > 0 ? s0[2 * slot + 1] : 1.f;
                const int64_t at = (int64_t)(u.part + u.chunk) * kUnitRows2 + 128 * t + r;
                const int64_t oi = (int64_t)tok * a.o_tok + (int64_t)(kvh * a.G + row % a.G) * a.o_head;
                if (u.n_chunk > 1 && mine) a.part_ml2[at] = make_float2(m, l);
#pragma unroll 1
                for (int c = 0; c < HD; c += 32) {
                    uint32_t o[32];
                    if (nt > 0) {
                        tld32(ob + c, o);
                        ld_wait();
                    }
                    float x[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        x[i] = nt > 0 ? __uint_as_float(o[i]) * sv : 0.f;
                        finite = finite && fabsf(x[i]) <= 3.0e38f;
                        if (u.n_chunk == 1) x[i] = l == 0.f ? none : x[i] * inv;
                    }
                    if (!mine) continue;
                    if (u.n_chunk == 1) {
                        store_out32(a, oi + c, x);
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; i += 8) store32b(a.part_o2 + at * HD + c + i, reinterpret_cast<const uint32_t*>(x) + i);
                    }
                }
                if (!finite && mine) redo_f[slot] = 1;
            }
            tc_before();
            // the unit is written (all softmax warps agree on whether to go on: a wait that gave up ends every role)
            if (any_of(1, 256, *abort_f != 0)) { done = ui; break; }
            const bool redo = nt > 0 && redo_f[slot];
            if (t == 0 && ht == 0) a.redo2[ui] = redo;
            if (redo) {
                again = true;
                asm volatile("bar.sync 1, 256;" ::: "memory");   // (all have read the slot's word)
                if (t == 0 && ht == 0) redo_f[slot] = 0;
            }
            u = u_nxt;
        }
        // Units with operands that were not finite (or an E4M3 row that f16 did not hold), key by key. That may take long, so it
        // comes last: no other role waits for it with a limit. Rows that a wait that gave up has cost are NaN, here or
        // in the join, and the error word tells.
        if (again || done < ui1) {
            asm volatile("bar.sync 1, 256;" ::: "memory");   // the marks are written
            for (int ui = ui0; ui < ui1; ++ui) {
                if (ui < done && __ldcg(&a.redo2[ui]) == 0) continue;
                const AttnUnit v = load_unit(a.units2 + ui);
                for (int x = warp - kSoft0; x < v.n_row; x += 8) {
                    float o[HD / 32], rm = -INFINITY, rl = NAN;
#pragma unroll
                    for (int d = 0; d < HD / 32; ++d) o[d] = NAN;
                    const int row = v.row0 + x, tok = row_token(a, v, row);
                    if (ui < done) careful_row<HD>(a, v, v.head, row, o, rm, rl);
                    const int64_t at = (int64_t)(v.part + v.chunk) * kUnitRows2 + x;
                    const int64_t oi = (int64_t)tok * a.o_tok + (int64_t)(v.head * a.G + row % a.G) * a.o_head;
                    const float inv = 1.f / rl, none = rl == 0.f ? weightless(a, v, row, tok) : 0.f;
#pragma unroll
                    for (int d = 0; d < HD / 32; ++d) {
                        if (v.n_chunk == 1) store_out1(a, oi + lane * (HD / 32) + d, rl == 0.f ? none : o[d] * inv);
                        else a.part_o2[at * HD + lane * (HD / 32) + d] = o[d];
                    }
                    if (v.n_chunk > 1 && lane == 0) a.part_ml2[at] = make_float2(rm, rl);
                }
            }
        }
    }
    if (beside) asm volatile("griddepcontrol.wait;" ::: "memory");
    __syncthreads();
    if (warp == kMmaWarp) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
}

// The rows of the cut tiles from their units' partial results, four rows a warp. A kernel of its own: the last unit of a
// tile to finish would do 256 rows alone while the other SMs are idle (512 tokens over 8192 keys: 170 us so, against
// 114 us in all with this kernel).
constexpr int kMergeThr = 256;

template <int HD>
__global__ void __launch_bounds__(kMergeThr) attn_tc_merge_kernel(AttnPagedArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if ((a.hdr[PH_FORM] & ~a.form) != 0 || (a.hdr[PH_FORM] & ATTN_FORM_TC) == 0) return;
    constexpr int NR = 4;                                   // rows per warp
    const int n = a.hdr[PH_CUTS2] * (kUnitRows2 / NR);
    for (int x = blockIdx.x * (kMergeThr / 32) + (threadIdx.x >> 5); x < n; x += gridDim.x * (kMergeThr / 32)) {
        const AttnUnit u = load_unit(a.units2 + a.cuts2[x / (kUnitRows2 / NR)]);
        const int r = x % (kUnitRows2 / NR) * NR;
        if (r < u.n_row) merge_rows<HD, NR>(a, a.part_o2, a.part_ml2, u, kUnitRows2, r);
    }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        cudaDriverEntryPointQueryResult q;
        void* p = nullptr;
        const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
                        q == cudaDriverEntryPointSuccess;
        return ok ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p) : nullptr;
    }();
    return fn;
}

// The maps of a 16-bit cache and the runs of cells they copy: up to 64 neighbouring cells of a page (a power of two
// from 8 on that divides the page), any 64 where the pages follow each other evenly. No runs: row copies only.
TmaRuns cell_runs(const PagedKv& kv, CUtensorMap* mk, CUtensorMap* mv) {
    TmaRuns r{0, false, false};
    const bool even = kv.n_pages == 1 || kv.page_size == 1 || kv.sb_page == kv.page_size * kv.sb_cell;
    const int64_t sb_cell = kv.page_size > 1 ? kv.sb_cell : kv.sb_page;
    const int64_t cells = (int64_t)kv.page_size * kv.n_pages;
    int rows = 64;
    if (kv.page_size > 1)                                   // (pages of one cell: whatever neighbours there are)
        while (rows >= 8 && kv.page_size % rows) rows /= 2;
    if (rows < 8 || cells < rows) return r;
    const uint64_t one = 2 * kv.hd;                         // a stride no copy uses
    const cuuint64_t dims[4] = {(cuuint64_t)kv.hd, (cuuint64_t)(even ? cells : kv.page_size), (cuuint64_t)kv.Hkv,
                                (cuuint64_t)(even ? 1 : kv.n_pages)};
    const cuuint64_t strides[3] = {(cuuint64_t)sb_cell, kv.Hkv > 1 ? (cuuint64_t)kv.sb_head : one,
                                   even ? one : (cuuint64_t)kv.sb_page};
    const cuuint32_t box[4] = {64, (cuuint32_t)rows, 1, 1}, es[4] = {1, 1, 1, 1};
    const auto fn = encode_fn();
    for (int i = 0; i < 2; ++i)
        if (!fn || fn(i ? mv : mk, kv.type == W_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                      i ? kv.v : kv.k, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                      CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return r;
    r.rows = rows;
    r.even = even;
    r.aligned = kv.page_size % rows == 0;
    return r;
}

template <int HD, int CT, int QT>
bool go(const AttnPagedArgs& a, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    if (!allow_smem(reinterpret_cast<const void*>(attn_tc_rows_kernel<HD, CT, QT>), Smem<HD>::bytes, done)) return false;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.n_sm);                             // one CTA per SM, each walking its units
    cfg.blockDim = dim3(kThr);
    cfg.dynamicSmemBytes = Smem<HD>::bytes;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    const int beside = (a.form & ~ATTN_FORM_TC) != 0;
    cfg.numAttrs = beside ? 1 : 0;
    CUtensorMap mk{}, mv{};
    TmaRuns runs{0, false, false};
    if (CT != W_F8) runs = cell_runs(a.kv, &mk, &mv);
    if (cudaLaunchKernelEx(&cfg, attn_tc_rows_kernel<HD, CT, QT>, a, runs, beside, mk, mv) != cudaSuccess) return false;
    // (launched early, it waits for the kernel above)
    cfg.gridDim = dim3(4 * a.n_sm);
    cfg.blockDim = dim3(kMergeThr);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_tc_merge_kernel<HD>, a) == cudaSuccess;
}
template <int HD>
bool go_hd(const AttnPagedArgs& a, cudaStream_t st) {
    if (a.kv.type == W_F16) return a.q_type == W_F16 ? go<HD, W_F16, W_F16>(a, st) : go<HD, W_F16, W_F32>(a, st);
    if (a.kv.type == W_BF16) return go<HD, W_BF16, W_BF16>(a, st);
    if (a.q_type == W_F16) return go<HD, W_F8, W_F16>(a, st);
    return a.q_type == W_BF16 ? go<HD, W_F8, W_BF16>(a, st) : go<HD, W_F8, W_F32>(a, st);
}

}  // namespace

// F32 activations stay with the 16-row tiles, which carry Q and P as two terms each, unless the caller's precision is
// that of f16 activations (round_q: the context's f16 forward passes).
bool attn_paged_tc_ok(int32_t hd, int32_t kv_type, int32_t q_type, bool round_q) {
    return (hd == 64 || hd == 128) && (q_type != W_F32 || round_q) && attn_paged_types_ok(q_type, kv_type);
}

bool launch_attn_paged_tc(const AttnPagedArgs& a, cudaStream_t st) {
    if (!attn_paged_tc_ok(a.kv.hd, a.kv.type, a.q_type, true)) return false;
    return a.kv.hd == 64 ? go_hd<64>(a, st) : go_hd<128>(a, st);
}

}  // namespace llm
