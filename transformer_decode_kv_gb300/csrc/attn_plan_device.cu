// The attention plan of a step made on the device: what attn_paged_plan.cpp does on the host, from lengths and a page table
// in device memory, so that a captured step follows lengths that the host never sees.
//
// The host deals tiles out one after the other. Here the tiles of all sequences and heads lie on one line, each as long as
// its blocks of keys and a unit's fixed cost, and CTA c takes [c share, (c + 1) share) of it: where a CTA's end falls
// inside a tile's blocks the tile is cut there. That needs no order of execution: a tile's place is a running sum (over
// the tiles of the sequences, one head's worth; the heads repeat it), its units follow from its place, and their
// numbers from how many cuts lie before it, which a running sum over the CTAs' ends tells. The same bounds hold as
// on the host: a CTA end cuts one tile at most, so there are at most (tiles + CTAs) units, two cut ones per CTA.
//
// One CTA makes the units, the others copy the page table. It is latency: lengths, four running sums, and two rounds of
// independent items, the CTAs' ends (a thread finds the tile that its end falls into, and makes the unit that begins there)
// and the tiles (each its first unit). 32 single tokens with 8 KV heads take 7.8 us (18.5 with the lists in global memory and
// eight lanes a tile, 9.5 with all places in 64 bits), six chunks of 1228 tokens together 9.8. Planned again and again: 512 single
// tokens 16.6 us, 2048 93, a prompt of 8192 f32 tokens (16-row tiles) 42, of f16 ones 7.3. A layer's attention of these steps takes
// 85 us (of 32 .. 256 keys each; 457 of 512 .. 4096), 615, 5866 and 479, and one plan serves all layers: one CTA is enough.
#include "paged.h"

#include <algorithm>

namespace llm {

namespace {

constexpr int kThr = 512;
constexpr int kMaxCtas = 2 * 160;
constexpr int kSeqs = 512, kTiles = 1024;                   // steps up to this size are planned in shared memory
static_assert(kMaxCtas + 1 <= kThr, "one thread per CTA end");

// Running sums of N numbers per thread over the block, without the thread's own; `all` receives the totals.
template <int N, typename I>
__device__ __forceinline__ void block_sums(const I* x, I* s /* [16 N] */, I* before, I* all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int W = kThr / 32;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        I in = x[i];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const I p = __shfl_up_sync(0xffffffffu, in, o);
            if (lane >= o) in += p;
        }
        if (lane == 31) s[W * i + warp] = in;
        before[i] = in - x[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        I w = lane < W ? s[W * i + lane] : 0;
#pragma unroll
        for (int o = 1; o < W; o <<= 1) {
            const I p = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += p;
        }
        all[i] = __shfl_sync(0xffffffffu, w, W - 1);
        const I b = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
        if (warp) before[i] += b;
    }
    __syncthreads();                                        // s may be written again
}
template <typename I>
__device__ __forceinline__ I block_sum(I x, int64_t* s, I& all) {
    I before;
    block_sums<1>(&x, reinterpret_cast<I*>(s), &before, &all);
    return before;
}

// x / y for x >= 0 and a y that is often a power of two (a quotient by another costs some 150 cycles)
__device__ __forceinline__ int by(int x, int y) { return (y & (y - 1)) == 0 ? x >> (__ffs(y) - 1) : x / y; }

struct Keys { int32_t n_sink, lo, n; };

// The virtual key range of rows [row0, row0 + n) of a sequence (as on the host, for positions that are indices).
__device__ __forceinline__ Keys tile_keys(const PlanDeviceArgs& a, int p0, int n_keys, int row0, int n, int align) {
    const int64_t pmin = (int64_t)p0 + by(row0, a.G), pmax = (int64_t)p0 + by(row0 + n - 1, a.G);
    auto first = [&](int64_t p) { return (int)min(max(p, (int64_t)0), (int64_t)n_keys); };
    Keys k{0, 0, 0};
    const int hi = first(pmax + 1);
    if (a.window == 0) {
        k.n = hi;
        return k;
    }
    k.lo = min(hi, first(pmin - a.window + 1)) & -align;    // (a power of two)
    k.n_sink = min(k.lo, (first(a.n_sink) + align - 1) & -align);
    k.n = k.n_sink + hi - k.lo;
    return k;
}

__device__ __forceinline__ int64_t pages_of(const PlanDeviceArgs& a, int n_kv) {
    if (n_kv <= 0) return 0;
    const uint32_t ps = (uint32_t)a.page_size, n = (uint32_t)n_kv + ps - 1u;
    return (ps & (ps - 1u)) == 0u ? n >> (__ffs(ps) - 1) : n / ps;
}

struct Shared {
    int64_t scan[32];
    int32_t cut[kMaxCtas + 1], cut_tile[kMaxCtas + 1];      // CTA ends that cut a tile; of these, a tile's first
    int32_t start[kSeqs + 1], n_kv[kSeqs], off[kSeqs], base[2][kSeqs + 1];
    int64_t pre[kTiles + 1];
};
// The step's lists, in shared memory or, where they are long, in the plan's scratch.
struct Lists { const int32_t *start, *n_kv; int32_t* off; int32_t* base[2]; };

// The last i of a[0 .. n) (ascending, a[0] <= x) with a[i] <= x.
template <typename T>
__device__ __forceinline__ int last_at_most(const T* a, int n, T x) {
    int lo = 0;
    for (int w = n; w > 1;) {
        const int h = w >> 1;
        if (a[lo + h] <= x) { lo += h; w -= h; }
        else w = h;
    }
    return lo;
}

// Tile t of sequence s for one head, its place on the line and its number.
// (The numbers of all tiles and heads fit 32 bits: there are not more of them than rows.)
template <typename I> struct Tile { int s, head, row0, n_row, p0, rank, blocks; Keys keys; I at; };

// I: the type of places on the line, 32 bits where the plan's bounds allow.
template <int F, typename I>
struct Line {
    const PlanDeviceArgs& a;
    const Lists& l;
    const I* pre;                                           // places of a head's tiles [n_tile + 1]
    int n_tile;
    I share;

    __device__ __forceinline__ Tile<I> shape(int s, int t) const {
        Tile<I> x;
        const int n_new = l.start[s + 1] - l.start[s], rows = F ? kUnitRows2 : a.rows1;
        x.s = s;
        x.p0 = l.n_kv[s] - n_new;
        x.row0 = t * rows;
        x.n_row = min(rows, n_new * a.G - x.row0);
        x.keys = tile_keys(a, x.p0, l.n_kv[s], x.row0, x.n_row, F ? a.align : 1);
        x.blocks = (int)(((uint32_t)x.keys.n + (uint32_t)a.bk[F] - 1u) / (uint32_t)a.bk[F]);
        return x;
    }
    __device__ __forceinline__ Tile<I> tile(int s, int head, int t) const {
        Tile<I> x = shape(s, t);
        const int b0 = l.base[F][s], b1 = l.base[F][s + 1];
        x.head = head;
        x.rank = b0 * a.Hkv + head * (b1 - b0) + t;
        x.at = pre[b0] * a.Hkv + head * (pre[b1] - pre[b0]) + pre[b0 + t] - pre[b0];
        return x;
    }
    // number r in the plan's order: sequences, heads, tiles
    __device__ __forceinline__ Tile<I> ranked(int r) const {
        const int32_t* base = l.base[F];
        const int s = last_at_most(base, a.n_seq, by(r, a.Hkv));
        const int T = base[s + 1] - base[s], rem = r - base[s] * a.Hkv, head = by(rem, T);
        return tile(s, head, rem - head * T);
    }
    // the tile at place x of the line
    __device__ __forceinline__ Tile<I> at(I x) const {
        const int32_t* base = l.base[F];
        // tiles of a sequence: the sequence of the last tile whose place, all heads before it counted, is not after x
        int lo = 0;
        for (int w = n_tile; w > 1;) {
            const int h = w >> 1;
            if (pre[lo + h] * a.Hkv <= x) { lo += h; w -= h; }
            else w = h;
        }
        // (lo may be any tile of the sequence: its own head's place comes first in the sequence's stretch)
        const int s = last_at_most(base, a.n_seq, lo);
        const int b0 = base[s], T = base[s + 1] - b0;
        const I one = pre[b0 + T] - pre[b0], in = x - pre[b0] * a.Hkv;
        const int head = (int)quotient(in, one);
        const I y = pre[b0] + in - head * one;
        return tile(s, head, last_at_most(pre + b0, T, y));
    }
    __device__ __forceinline__ static I quotient(I x, I y) {
        if constexpr (sizeof(I) > 4)
            if ((x | y) >> 32) return x / y;
        return (I)((uint32_t)x / (uint32_t)y);
    }
    __device__ __forceinline__ int cta_at(I x) const { return (int)quotient(x, share); }
    // block at which CTA c's part of a tile begins
    __device__ __forceinline__ int cut_at(const Tile<I>& x, int c) const {
        return (int)min(max(c * share - x.at - a.cost[F], (I)0), (I)x.blocks);
    }
    // the CTAs of a tile's first place, first unit (another where only the fixed cost lies in the former) and last unit
    __device__ __forceinline__ void span(const Tile<I>& x, int& c0, int& cf, int& c1) const {
        c0 = cta_at(x.at);
        c1 = cta_at(x.at + x.blocks + a.cost[F] - 1);
        cf = c1 > c0 && (c0 + 1) * share - x.at <= a.cost[F] ? c0 + 1 : c0;
    }
};

// The units of form F; returns its number of cut tiles, -1 without units.
template <int F, typename I>
__device__ int make_units(const PlanDeviceArgs& a, const Lists& l, Shared& sh) {
    const int tid = threadIdx.x, n_tile = l.base[F][a.n_seq];
    if (n_tile == 0) return -1;
    I* pre = reinterpret_cast<I*>(n_tile <= kTiles ? sh.pre : a.tile_pre[F]);
    Line<F, I> line{a, l, pre, n_tile, 1};
    I total = 0;
    for (int t0 = 0; t0 < n_tile; t0 += kThr) {
        const int t = t0 + tid;
        I len = 0, all;
        if (t < n_tile) {
            const int s = last_at_most(l.base[F], a.n_seq, t);
            len = line.shape(s, t - l.base[F][s]).blocks + a.cost[F];
        }
        const I before = block_sum(len, sh.scan, all);
        if (t < n_tile) pre[t] = total + before;
        total += all;
    }
    if (tid == 0) pre[n_tile] = total;
    const int n_cta = a.n_cta[F], cost = a.cost[F], bk = a.bk[F];
    const I length = total * a.Hkv;
    const int n_rank = n_tile * a.Hkv;
    const I share = max(Line<F, I>::quotient(length + n_cta - 1, n_cta), (I)cost + 1);
    line.share = share;
    __syncthreads();
    // a thread per CTA end: the tile that it falls into, and whether it cuts it
    const int c = tid;
    const bool end = c <= n_cta && c * share < length;
    Tile<I> mine;
    int c0 = 0, cf = 0, c1 = 0;
    bool cuts = false;
    int own = 0, all;                                       // (cuts above, tiles' first cuts below: fewer than 2^15 of each)
    if (end) {
        mine = line.at(c * share);
        line.span(mine, c0, cf, c1);
        cuts = c > c0 && c * share - mine.at > cost;
        own = cuts ? 1 << 16 | (c == cf + 1) : 0;
    }
    const int sum = block_sum(own, sh.scan, all) + own;
    if (c <= n_cta) { sh.cut[c] = sum >> 16; sh.cut_tile[c] = sum & 0xffff; }
    __syncthreads();
    // the unit of tile x that belongs to CTA u_c
    auto write = [&](const Tile<I>& x, int t0, int tf, int t1, int u_c) {
        const int u0 = x.rank + sh.cut[t0], n = t1 - tf + 1;
        AttnUnit u{};
        u.tok0 = l.start[x.s];
        u.row0 = x.row0;
        u.n_row = x.n_row;
        u.p0 = x.p0;
        u.table = l.off[x.s];
        u.n_sink_keys = x.keys.n_sink;
        u.key_lo = x.keys.lo;
        u.v0 = u_c == tf ? 0 : line.cut_at(x, u_c) * bk;
        u.v1 = u_c == t1 ? x.keys.n : line.cut_at(x, u_c + 1) * bk;
        u.n_chunk = n;
        u.chunk = u_c - tf;
        u.part = n > 1 ? sh.cut[t0] + sh.cut_tile[t0] : 0;
        u.ticket = n > 1 ? sh.cut_tile[t0] : 0;
        u.head = x.head;
        int4* d = reinterpret_cast<int4*>(a.units[F] + u0 + u.chunk);
        const int4* q = reinterpret_cast<const int4*>(&u);
        d[0] = q[0]; d[1] = q[1]; d[2] = q[2]; d[3] = q[3];
        if (F && n > 1 && u_c == tf) a.cuts[u.ticket] = u0;
    };
    if (cuts) write(mine, c0, cf, c1, c);
    // where each CTA's units begin
    if (c <= n_cta) a.first[F][c] = end ? mine.rank + sh.cut[c0] + max(0, c - cf) : n_rank + sh.cut[n_cta];
    // and each tile's first unit
    for (int r = tid; r < n_rank; r += kThr) {
        const Tile<I> x = line.ranked(r);
        int t0, tf, t1;
        line.span(x, t0, tf, t1);
        write(x, t0, tf, t1, tf);
    }
    return sh.cut_tile[n_cta];
}

template <typename I>
__global__ void __launch_bounds__(kThr) attn_plan_kernel(PlanDeviceArgs a) {
    __shared__ Shared sh;
    const int tid = threadIdx.x;
    // The attention may be launched while this runs (it waits for the end of it), as this may be while the kernel in front runs.
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (blockIdx.x > 0) {
        // the page tables, one behind the other
        int64_t at = 0;
        int done = 0;
        for (int s = blockIdx.x - 1; s < a.n_seq; s += gridDim.x - 1) {
            int64_t mine = 0, all;
            for (int i = done + tid; i < s; i += kThr) mine += pages_of(a, a.n_kv[i]);
            block_sum(mine, sh.scan, all);
            at += all;
            done = s;
            const int64_t n = min(min(pages_of(a, a.n_kv[s]), (int64_t)a.ld_table), a.max_table - at);
            const int32_t* from = a.table + (int64_t)s * a.ld_table;
            for (int64_t i = tid; i < n; i += kThr) a.table_out[at + i] = from[i];
        }
        return;
    }
    // the step's lengths
    const bool small = a.n_seq <= kSeqs;
    const Lists l{small ? sh.start : a.start, small ? sh.n_kv : a.n_kv, small ? sh.off : a.table_off,
                  {small ? sh.base[0] : a.tile_base[0], small ? sh.base[1] : a.tile_base[1]}};
    bool bad = a.n_seq == 0 && a.start[0] != 0;
    int64_t pages = 0;
    int tiles[2] = {0, 0};
    for (int s0 = 0; s0 < a.n_seq; s0 += kThr) {
        const int s = s0 + tid;
        int64_t pg = 0;
        int T[2] = {0, 0};
        if (s < a.n_seq) {
            const int from = a.start[s], to = a.start[s + 1], n_kv = a.n_kv[s];
            const int64_t n_new = (int64_t)to - from;
            if (small) {
                sh.start[s] = from;
                sh.start[s + 1] = to;                       // (the next thread writes the same)
                sh.n_kv[s] = n_kv;
            }
            pg = pages_of(a, n_kv);
            if ((s == 0 && from != 0) || n_new < 0 || n_new > a.max_new || to > a.max_tok || n_kv < 0 || n_kv > a.max_keys || pg > a.ld_table) {
                bad = true;
            } else {
                const int f = a.tc && n_new * a.G >= a.tc_rows ? 1 : 0, step = f ? kUnitRows2 : a.rows1;
                T[f] = (int)(((uint32_t)n_new * (uint32_t)a.G + (uint32_t)step - 1u) / (uint32_t)step);   // (rows are below 2^31)
            }
        }
        const int64_t x[2] = {pg, (int64_t)T[1] << 32 | (uint32_t)T[0]};
        int64_t before[2], all[2];
        block_sums<2>(x, sh.scan, before, all);
        if (s < a.n_seq) {
            l.off[s] = (int)min(pages + before[0], a.max_table);
            l.base[0][s] = tiles[0] + (int)(uint32_t)before[1];
            l.base[1][s] = tiles[1] + (int)(before[1] >> 32);
        }
        // (a bad step may have any sums; nobody looks at them)
        pages += all[0];
        tiles[0] += (int)(uint32_t)all[1];
        tiles[1] += (int)(all[1] >> 32);
    }
    if (tid < 2) l.base[tid][a.n_seq] = tiles[tid];
    bad = __syncthreads_or(bad) || pages > a.max_table;
    int n0 = -1, n1 = -1;
    if (!bad) {
        n0 = make_units<0, I>(a, l, sh);
        if (a.tc) {
            __syncthreads();
            n1 = make_units<1, I>(a, l, sh);
        }
    }
    if (tid == 0) {
        a.hdr[PH_FORM] = (n0 >= 0 ? a.rows1 == 8 ? ATTN_FORM_ROWS8 : ATTN_FORM_ROWS16 : 0) | (n1 >= 0 ? ATTN_FORM_TC : 0);
        a.hdr[PH_CUTS2] = max(n1, 0);
        if (bad && a.err) atomicOr(a.err, ERR_STEP_RANGE);
    }
}

}  // namespace

bool launch_attn_plan_device(const PlanDeviceArgs& a, cudaStream_t st) {
    if (a.n_cta[0] > kMaxCtas || a.n_cta[1] > kMaxCtas) return false;
    const int copies = a.n_seq < kMaxCtas ? a.n_seq : kMaxCtas;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1 + copies);
    cfg.blockDim = dim3(kThr);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    // The line is no longer than the most tiles of the most keys; every multiple of a CTA's share up to its end, and one share more,
    // has to fit.
    const int64_t keys = std::min<int64_t>(std::min<int64_t>(a.max_table, a.ld_table) * a.page_size, a.max_keys);
    bool fits = true;
    for (int f = 0; f < 2; ++f) {
        const double line = (double)a.max_tiles[f] * (double)(keys / a.bk[f] + 2 + a.cost[f]) * a.Hkv;
        fits = fits && line + 2.0 * a.n_cta[f] * (a.cost[f] + 2) + line / a.n_cta[f] < 2147483000.0;
    }
    return cudaLaunchKernelEx(&cfg, fits ? attn_plan_kernel<int32_t> : attn_plan_kernel<int64_t>, a) == cudaSuccess;
}

}  // namespace llm
