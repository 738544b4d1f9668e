// Page tables on the device: the pages, cells and positions of a step's new tokens from the sequences' lengths, and
// the way back of pages that are no longer needed.
//
// A sequence of n rows holds ceil(n / page_size) pages, the first entries of its table row. Adding m rows takes
// ceil((n + m) / page_size) - ceil(n / page_size) pages from the top of the stack of free ones, sequence by sequence; a
// token at position p lies in cell table[p / page_size] * page_size + p % page_size. So two running sums over the
// sequences (tokens, pages) say all there is to know, and every token finds its sequence by bisection in the first.
//
// The work is a few hundred bytes to a few hundred kilobytes; what it costs is the launch and the chain lengths -> sums ->
// bisection -> cells. One CTA, or one cluster where there are many tokens, whose CTAs all make the sums for themselves (a
// thousand lengths are a few microseconds' worth of nothing) and share out the tokens; its barrier keeps lengths and
// the stack's size in place until every CTA has read them, so that both may be updated where they are. 64 sequences take
// 5.4 us on the GPU (a launch of nothing: about 2), 512 with 17 thousand new tokens 9.5 with eight CTAs, 11.4 with four,
// 16 with two. Trims, one after the other: 64 sequences of which eight end and give back 1632 pages 3.6 us, 512 of which 32 end,
// 37 thousand pages, 7.1; all 512 at once, 546 thousand pages, 53 (a bisection per page: a server that ends that many in one
// step has no tokens to wait for).
#include "paged.h"

namespace llm {

namespace {

constexpr int kThr = 1024;                                  // sequences at a time
constexpr uint32_t kMany = 0x7fffffffu;                     // sums stop here: more than fits anything

__device__ __forceinline__ uint32_t add_sat(uint32_t a, uint32_t b) { return min(a + b, kMany); }

// Running sums of two numbers per thread over the block, without the thread's own, and the totals.
struct Sums { uint32_t x, y, all_x, all_y; };
__device__ __forceinline__ Sums block_sums(uint32_t x, uint32_t y, uint32_t* s /* [64] */) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t ix = x, iy = y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t px = __shfl_up_sync(0xffffffffu, ix, o), py = __shfl_up_sync(0xffffffffu, iy, o);
        if (lane >= o) { ix = add_sat(ix, px); iy = add_sat(iy, py); }
    }
    if (lane == 31) { s[warp] = ix; s[32 + warp] = iy; }
    // (the exclusive sum by another shuffle: a saturated one has no difference to take)
    uint32_t ex = __shfl_up_sync(0xffffffffu, ix, 1), ey = __shfl_up_sync(0xffffffffu, iy, 1);
    if (lane == 0) ex = ey = 0u;
    __syncthreads();
    const int n_warp = blockDim.x >> 5;
    uint32_t wx = lane < n_warp ? s[lane] : 0u, wy = lane < n_warp ? s[32 + lane] : 0u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t px = __shfl_up_sync(0xffffffffu, wx, o), py = __shfl_up_sync(0xffffffffu, wy, o);
        if (lane >= o) { wx = add_sat(wx, px); wy = add_sat(wy, py); }
    }
    Sums r;
    r.all_x = __shfl_sync(0xffffffffu, wx, 31);
    r.all_y = __shfl_sync(0xffffffffu, wy, 31);
    const uint32_t bx = __shfl_sync(0xffffffffu, wx, max(warp - 1, 0)), by = __shfl_sync(0xffffffffu, wy, max(warp - 1, 0));
    r.x = warp ? add_sat(bx, ex) : ex;
    r.y = warp ? add_sat(by, ey) : ey;
    __syncthreads();                                        // s may be written again
    return r;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n barrier.cluster.wait.acquire;" ::: "memory");
}

// The launch may overlap the end of the kernel in front; nothing is read or written before that has ended.
__device__ __forceinline__ void begin() {
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

__device__ __forceinline__ uint32_t div_up(uint32_t n, uint32_t ps) { return n / ps + (n % ps != 0); }

// The last i of a[0 .. n) (ascending, a[0] <= x) with a[i] <= x.
__device__ __forceinline__ int last_at_most(const uint32_t* a, int n, uint32_t x) {
    int lo = 0;
    for (int w = n; w > 1;) {
        const int h = w >> 1;
        if (a[lo + h] <= x) { lo += h; w -= h; }
        else w = h;
    }
    return lo;
}

struct Seq { uint32_t have, add, held, need; int given; bool bad; };
__device__ __forceinline__ Seq seq_extend(const PageListArgs& a, int i) {
    Seq q{0u, 0u, 0u, 0u, 0, false};
    if (i >= a.n_seq) return q;
    const int have = a.n_kv[i], add = a.n_new[i];
    q.given = have;
    const uint32_t ps = (uint32_t)a.page_size;
    q.bad = have < 0 || add < 0 || add > a.max_tok || (int64_t)have + add > INT32_MAX;
    if (q.bad) return q;
    q.have = (uint32_t)have;
    q.add = (uint32_t)add;
    q.held = div_up(q.have, ps);
    const uint32_t to = div_up(q.have + q.add, ps);
    q.need = to - q.held;
    q.bad = to > (uint32_t)a.ld_table;
    return q;
}

__global__ void __launch_bounds__(kThr) pages_extend_kernel(PageListArgs a, int n_cta) {
    __shared__ uint32_t s_scan[64], s_tok[kThr], s_page[kThr], s_have[kThr];
    const int tid = threadIdx.x, nt = blockDim.x, rank = blockIdx.x;
    begin();
    const uint32_t ps = (uint32_t)a.page_size;
    const int n_free = *a.n_free;
    const int n_chunk = max(1, (a.n_seq + nt - 1) / nt);
    // whether the step fits: sums over all sequences
    uint32_t tok = 0u, page = 0u;
    bool bad = n_free < 0 || n_free > a.max_free;
    int mine = 0;                                           // the new length, where a thread has one sequence
    Sums at{};
    for (int c = 0; c < n_chunk; ++c) {
        const Seq q = seq_extend(a, c * nt + tid);
        mine = q.given + (int)q.add;
        bad = bad || q.bad;
        at = block_sums(q.add, q.need, s_scan);
        tok = add_sat(tok, at.all_x);
        page = add_sat(page, at.all_y);
        s_tok[tid] = at.x; s_page[tid] = at.y; s_have[tid] = q.have;
    }
    bad = __syncthreads_or(bad) || tok > (uint32_t)a.max_tok || page > (uint32_t)n_free || page >= kMany;
    if (bad && n_chunk == 1) mine = tid < a.n_seq ? a.n_kv[tid] : 0;
    if (!bad) {
        uint32_t tok0 = 0u, page0 = 0u;                     // before the sequences at hand
        for (int c = 0; c < n_chunk; ++c) {
            if (n_chunk > 1) {
                const Seq q = seq_extend(a, c * nt + tid);
                at = block_sums(q.add, q.need, s_scan);
                s_tok[tid] = at.x; s_page[tid] = at.y; s_have[tid] = q.have;
                __syncthreads();
            }
            const int i0 = c * nt, n = min(nt, a.n_seq - i0);
            if (rank == 0 && tid < n) a.start[i0 + tid] = (int)(tok0 + at.x);
            for (uint32_t t = rank * nt + tid; t < at.all_x; t += n_cta * nt) {
                const int i = last_at_most(s_tok, n, t);
                const uint32_t p = s_have[i] + t - s_tok[i], k = p / ps, held = div_up(s_have[i], ps);
                int32_t* const entry = a.table + (int64_t)(i0 + i) * a.ld_table + k;
                int pg;
                if (k >= held) {
                    pg = a.free_pages[n_free - 1 - (int)(page0 + s_page[i] + k - held)];
                    if (p == k * ps) *entry = pg;           // the page's first token puts it into the table
                } else {
                    pg = *entry;
                }
                const bool in = (unsigned)pg < (unsigned)a.n_pages;
                if (!in && a.err) atomicOr(a.err, ERR_SLOT_RANGE);
                a.cell[tok0 + t] = in ? (int)(pg * ps + (p - k * ps)) : -1;
                a.pos[tok0 + t] = (int)p;
            }
            tok0 += at.all_x;
            page0 += at.all_y;
            __syncthreads();                                // the sums may be written again
        }
    } else {
        tok = page = 0u;
        if (rank == 0) {
            if (tid == 0 && a.err) atomicOr(a.err, ERR_STEP_RANGE);
            for (int i = tid; i < a.n_seq; i += nt) a.start[i] = 0;
        }
    }
    for (int t = (int)tok + rank * nt + tid; t < a.max_tok; t += n_cta * nt) a.cell[t] = a.pos[t] = -1;
    if (n_cta > 1) cluster_sync();                          // everybody has read the lengths
    else __syncthreads();
    if (rank == 0) {
        if (n_chunk == 1) {
            if (tid < a.n_seq) a.n_kv_out[tid] = mine;
        } else {
            for (int i = tid; i < a.n_seq; i += nt) a.n_kv_out[i] = a.n_kv[i] + (bad ? 0 : a.n_new[i]);
        }
        if (tid == 0) {
            a.start[a.n_seq] = (int)tok;
            *a.n_free_out = n_free - (int)page;
        }
    }
}

// A sequence's pages that go back: entries [from, from + gone) of its table row.
struct Cut { uint32_t from, gone; int left; bool bad; };
__device__ __forceinline__ Cut seq_trim(const PageListArgs& a, int i) {
    Cut q{0u, 0u, 0, false};
    if (i >= a.n_seq) return q;
    const int have = a.n_kv[i], keep = a.n_new[i];
    const uint32_t ps = (uint32_t)a.page_size;
    q.left = have;
    q.bad = have < 0 || keep > have || div_up((uint32_t)max(have, 0), ps) > (uint32_t)a.ld_table;
    if (q.bad || keep < 0) return q;
    q.left = keep;
    q.from = div_up((uint32_t)keep, ps);
    q.gone = div_up((uint32_t)have, ps) - q.from;
    return q;
}

__global__ void __launch_bounds__(kThr) pages_trim_kernel(PageListArgs a, int n_cta) {
    __shared__ uint32_t s_scan[64], s_page[kThr], s_from[kThr];
    const int tid = threadIdx.x, nt = blockDim.x, rank = blockIdx.x;
    begin();
    const int n_free = *a.n_free;
    const int n_chunk = max(1, (a.n_seq + nt - 1) / nt);
    uint32_t page = 0u;
    bool bad = n_free < 0 || n_free > a.max_free;
    Sums at{};
    for (int c = 0; c < n_chunk; ++c) {
        const Cut q = seq_trim(a, c * nt + tid);
        bad = bad || q.bad;
        at = block_sums(q.gone, 0u, s_scan);
        page = add_sat(page, at.all_x);
        s_page[tid] = at.x; s_from[tid] = q.from;
    }
    bad = __syncthreads_or(bad) || (int64_t)n_free + page > a.max_free || page >= kMany;
    if (!bad) {
        uint32_t page0 = 0u;
        for (int c = 0; c < n_chunk; ++c) {
            if (n_chunk > 1) {
                const Cut q = seq_trim(a, c * nt + tid);
                at = block_sums(q.gone, 0u, s_scan);
                s_page[tid] = at.x; s_from[tid] = q.from;
                __syncthreads();
            }
            const int i0 = c * nt, n = min(nt, a.n_seq - i0);
            for (uint32_t j = rank * nt + tid; j < at.all_x; j += n_cta * nt) {
                const int i = last_at_most(s_page, n, j);
                const int pg = a.table[(int64_t)(i0 + i) * a.ld_table + s_from[i] + (j - s_page[i])];
                if ((unsigned)pg >= (unsigned)a.n_pages && a.err) atomicOr(a.err, ERR_SLOT_RANGE);
                a.free_pages[n_free + (int)(page0 + j)] = pg;
            }
            page0 += at.all_x;
            __syncthreads();
        }
    } else {
        page = 0u;
        if (rank == 0 && tid == 0 && a.err) atomicOr(a.err, ERR_STEP_RANGE);
    }
    if (n_cta > 1) cluster_sync();
    else __syncthreads();
    if (rank == 0) {
        for (int i = tid; i < a.n_seq; i += nt) a.n_kv_out[i] = bad ? a.n_kv[i] : seq_trim(a, i).left;
        if (tid == 0) *a.n_free_out = n_free + (int)page;
    }
}

bool go(void (*kernel)(PageListArgs, int), const PageListArgs& a, int64_t work, cudaStream_t st) {
    // more CTAs where there is more than two rounds of work for one
    const int n_cta = (int)(work <= 2 * kThr ? 1 : work <= 8 * kThr ? 4 : 8);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(n_cta);
    // fewer threads meet faster at the barriers
    cfg.blockDim = dim3(a.n_seq <= 256 && work <= 512 ? 256 : kThr);
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = n_cta;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = n_cta > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, a, n_cta) == cudaSuccess;
}

}  // namespace

bool launch_pages_extend(const PageListArgs& a, cudaStream_t st) { return go(pages_extend_kernel, a, a.max_tok, st); }
bool launch_pages_trim(const PageListArgs& a, cudaStream_t st) { return go(pages_trim_kernel, a, a.max_free, st); }

}  // namespace llm
