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
// One CTA makes the units, the others copy the page table. It is latency: lengths, three running sums, two walks over the
// tiles.
#include "paged.h"

namespace llm {

namespace {

constexpr int kThr = 512;
constexpr int kLanes = 8;                                   // threads that share a tile
constexpr int kMaxCtas = 2 * 160;
static_assert(kMaxCtas + 1 <= kThr, "one thread per CTA end");

// Running sums of a number per thread over the block, without the thread's own; `all` receives the total.
__device__ __forceinline__ int64_t block_sum(int64_t x, int64_t* s /* [32] */, int64_t& all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t in = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t p = __shfl_up_sync(0xffffffffu, in, o);
        if (lane >= o) in += p;
    }
    if (lane == 31) s[warp] = in;
    __syncthreads();
    int64_t w = lane < kThr / 32 ? s[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t p = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += p;
    }
    all = __shfl_sync(0xffffffffu, w, 31);
    const int64_t before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
    __syncthreads();                                        // s may be written again
    return (warp ? before : 0) + in - x;
}

struct Keys { int32_t n_sink, lo, n; };

// The virtual key range of rows [row0, row0 + n) of a sequence (as on the host, for positions that are indices).
__device__ __forceinline__ Keys tile_keys(const PlanDeviceArgs& a, int p0, int n_keys, int row0, int n, int align) {
    const int64_t pmin = (int64_t)p0 + row0 / a.G, pmax = (int64_t)p0 + (row0 + n - 1) / a.G;
    auto first = [&](int64_t p) { return (int)min(max(p, (int64_t)0), (int64_t)n_keys); };
    Keys k{0, 0, 0};
    const int hi = first(pmax + 1);
    if (a.window == 0) {
        k.n = hi;
        return k;
    }
    k.lo = min(hi, first(pmin - a.window + 1)) / align * align;
    k.n_sink = min(k.lo, (first(a.n_sink) + align - 1) / align * align);
    k.n = k.n_sink + hi - k.lo;
    return k;
}

__device__ __forceinline__ int n_new_of(const PlanDeviceArgs& a, int s) { return a.start[s + 1] - a.start[s]; }
__device__ __forceinline__ int64_t pages_of(const PlanDeviceArgs& a, int s) {
    const int n = a.n_kv[s];
    return n <= 0 ? 0 : ((int64_t)n + a.page_size - 1) / a.page_size;
}
__device__ __forceinline__ int form_of(const PlanDeviceArgs& a, int n_new) {
    return a.tc && (int64_t)n_new * a.G >= a.tc_rows ? 1 : 0;
}

// The sequence whose tiles contain tile x: the last with base[s] <= x.
__device__ __forceinline__ int seq_of(const int32_t* base, int n, int x) {
    int lo = 0;
    for (int w = n; w > 1;) {
        const int h = w >> 1;
        if (base[lo + h] <= x) { lo += h; w -= h; }
        else w = h;
    }
    return lo;
}

struct Tile { int s, head, row0, n_row, p0; Keys keys; int64_t at, len, rank; };

template <int F>
__device__ __forceinline__ int tile_rows(const PlanDeviceArgs& a) { return F ? kUnitRows2 : a.rows1; }
template <int F>
__device__ __forceinline__ Tile tile_of(const PlanDeviceArgs& a, int s, int t) {
    Tile x;
    const int n_new = n_new_of(a, s);
    x.s = s;
    x.p0 = a.n_kv[s] - n_new;
    x.row0 = t * tile_rows<F>(a);
    x.n_row = min(tile_rows<F>(a), n_new * a.G - x.row0);
    x.keys = tile_keys(a, x.p0, a.n_kv[s], x.row0, x.n_row, F ? a.align : 1);
    x.len = (x.keys.n + a.bk[F] - 1) / a.bk[F] + a.cost[F];
    return x;
}
// (tile, head) r in the plan's order: sequences, heads, tiles
template <int F>
__device__ __forceinline__ Tile ranked(const PlanDeviceArgs& a, int64_t r, int64_t total) {
    const int32_t* base = a.tile_base[F];
    const int s = seq_of(base, a.n_seq, (int)(r / a.Hkv));
    const int T = base[s + 1] - base[s], rem = (int)(r - (int64_t)base[s] * a.Hkv);
    const int head = rem / T, t = rem - head * T;
    Tile x = tile_of<F>(a, s, t);
    x.head = head;
    x.rank = r;
    const int64_t pre0 = a.tile_pre[F][base[s]], pre = a.tile_pre[F][base[s] + t];
    const int64_t one = (base[s + 1] < base[a.n_seq] ? a.tile_pre[F][base[s + 1]] : total) - pre0;   // a head's tiles
    x.at = pre0 * a.Hkv + head * one + pre - pre0;
    return x;
}

struct Shared {
    int64_t scan[32];
    int32_t cut[kMaxCtas + 1], cut_tile[kMaxCtas + 1];      // CTA ends that cut a tile; of these, a tile's first
};

// The units of form F; returns its number of cut tiles, -1 without units.
template <int F>
__device__ int make_units(const PlanDeviceArgs& a, Shared& sh) {
    const int tid = threadIdx.x, n_tile = a.tile_base[F][a.n_seq];
    if (n_tile == 0) return -1;
    int64_t total = 0;
    for (int t0 = 0; t0 < n_tile; t0 += kThr) {
        const int t = t0 + tid;
        int64_t len = 0, all;
        if (t < n_tile) {
            const int s = seq_of(a.tile_base[F], a.n_seq, t);
            len = tile_of<F>(a, s, t - a.tile_base[F][s]).len;
        }
        const int64_t before = block_sum(len, sh.scan, all);
        if (t < n_tile) a.tile_pre[F][t] = total + before;
        total += all;
    }
    const int n_cta = a.n_cta[F], cost = a.cost[F], bk = a.bk[F];
    const int64_t line = total * a.Hkv, share = max((line + n_cta - 1) / n_cta, (int64_t)cost + 1);
    auto cta_at = [&](int64_t x) { return (int)((x | share) >> 32 ? x / share : (int64_t)((uint32_t)x / (uint32_t)share)); };
    for (int c = tid; c <= n_cta; c += kThr) sh.cut[c] = sh.cut_tile[c] = 0;
    __syncthreads();
    const int64_t n_rank = (int64_t)n_tile * a.Hkv;
    const int lane = tid % kLanes;
    for (int64_t r = tid / kLanes; r < n_rank; r += kThr / kLanes) {
        const Tile x = ranked<F>(a, r, total);
        const int c0 = cta_at(x.at), c1 = cta_at(x.at + x.len - 1);
        for (int c = c0 + 1 + lane; c <= c1; c += kLanes)
            if (c * share - x.at > cost) {
                sh.cut[c] = 1;
                sh.cut_tile[c] = c == c0 + 1 || (c - 1) * share - x.at <= cost;
            }
    }
    __syncthreads();
    {   // (both sums at once)
        int64_t all;
        const int64_t own = tid <= n_cta ? (int64_t)sh.cut[tid] << 32 | sh.cut_tile[tid] : 0;
        const int64_t sum = block_sum(own, sh.scan, all) + own;
        if (tid <= n_cta) { sh.cut[tid] = (int)(sum >> 32); sh.cut_tile[tid] = (int)(sum & 0x7fffffff); }
        __syncthreads();
    }
    for (int64_t r = tid / kLanes; r < n_rank; r += kThr / kLanes) {
        const Tile x = ranked<F>(a, r, total);
        const int c0 = cta_at(x.at), c1 = cta_at(x.at + x.len - 1);
        // the CTA of the first unit: not c0 where only the fixed cost lies there
        const int cf = c1 > c0 && (c0 + 1) * share - x.at <= cost ? c0 + 1 : c0;
        const int u0 = (int)x.rank + sh.cut[c0], n = c1 - cf + 1;
        const int blocks = (int)(x.len - cost);
        auto cut_at = [&](int c) { return (int)min(max(c * share - x.at - cost, (int64_t)0), (int64_t)blocks); };
        for (int c = cf + lane; c <= c1; c += kLanes) {
            AttnUnit u{};
            u.tok0 = a.start[x.s];
            u.row0 = x.row0;
            u.n_row = x.n_row;
            u.p0 = x.p0;
            u.table = a.table_off[x.s];
            u.n_sink_keys = x.keys.n_sink;
            u.key_lo = x.keys.lo;
            u.v0 = c == cf ? 0 : cut_at(c) * bk;
            u.v1 = c == c1 ? x.keys.n : cut_at(c + 1) * bk;
            u.n_chunk = n;
            u.chunk = c - cf;
            u.part = n > 1 ? sh.cut[c0] + sh.cut_tile[c0] : 0;
            u.ticket = n > 1 ? sh.cut_tile[c0] : 0;
            u.head = x.head;
            int4* d = reinterpret_cast<int4*>(a.units[F] + u0 + u.chunk);
            const int4* q = reinterpret_cast<const int4*>(&u);
            d[0] = q[0]; d[1] = q[1]; d[2] = q[2]; d[3] = q[3];
            if (F && n > 1 && c == cf) a.cuts[u.ticket] = u0;
        }
        // CTA ends in this tile: where the CTA's units begin
        for (int c = c0 + (c0 * share < x.at) + lane; c <= c1; c += kLanes) a.first[F][c] = u0 + max(0, c - cf);
    }
    for (int c = cta_at(line - 1) + 1 + tid; c <= n_cta; c += kThr) a.first[F][c] = (int)n_rank + sh.cut[n_cta];
    return sh.cut_tile[n_cta];
}

__global__ void __launch_bounds__(kThr) attn_plan_kernel(PlanDeviceArgs a) {
    __shared__ Shared sh;
    const int tid = threadIdx.x;
    if (blockIdx.x > 0) {
        // the page tables, one behind the other
        int64_t at = 0;
        int done = 0;
        for (int s = blockIdx.x - 1; s < a.n_seq; s += gridDim.x - 1) {
            int64_t mine = 0, all;
            for (int i = done + tid; i < s; i += kThr) mine += pages_of(a, i);
            block_sum(mine, sh.scan, all);
            at += all;
            done = s;
            const int64_t n = min(min(pages_of(a, s), (int64_t)a.ld_table), a.max_table - at);
            const int32_t* from = a.table + (int64_t)s * a.ld_table;
            for (int64_t i = tid; i < n; i += kThr) a.table_out[at + i] = from[i];
        }
        return;
    }
    // the step's lengths
    bool bad = tid == 0 && (a.start[0] != 0 || a.start[a.n_seq] > a.max_tok);
    int64_t pages = 0;
    int tiles[2] = {0, 0};
    for (int s0 = 0; s0 < a.n_seq; s0 += kThr) {
        const int s = s0 + tid;
        int64_t pg = 0, all;
        int T[2] = {0, 0};
        if (s < a.n_seq) {
            const int64_t n_new = (int64_t)a.start[s + 1] - a.start[s];
            const int n_kv = a.n_kv[s];
            pg = pages_of(a, s);
            if (n_new < 0 || n_new > a.max_new || n_new > a.max_tok || n_kv < 0 || n_kv > a.max_keys || pg > a.ld_table) {
                bad = true;
            } else {
                const int f = form_of(a, (int)n_new), step = f ? kUnitRows2 : a.rows1;
                T[f] = ((int)n_new * a.G + step - 1) / step;
            }
        }
        const int64_t p = block_sum(pg, sh.scan, all);
        if (s < a.n_seq) a.table_off[s] = (int)min(pages + p, a.max_table);
        pages += all;
        const int64_t t = block_sum((int64_t)T[1] << 32 | (uint32_t)T[0], sh.scan, all);
        if (s < a.n_seq) {
            a.tile_base[0][s] = tiles[0] + (int)(uint32_t)t;
            a.tile_base[1][s] = tiles[1] + (int)(t >> 32);
        }
        // (a bad step may have any sums; nobody looks at them)
        tiles[0] += (int)(uint32_t)all;
        tiles[1] += (int)(all >> 32);
    }
    if (tid < 2) a.tile_base[tid][a.n_seq] = tiles[tid];
    bad = __syncthreads_or(bad) || pages > a.max_table;
    int n0 = -1, n1 = -1;
    if (!bad) {
        n0 = make_units<0>(a, sh);
        __syncthreads();
        n1 = make_units<1>(a, sh);
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
    attn_plan_kernel<<<1 + copies, kThr, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess;
}

}  // namespace llm
