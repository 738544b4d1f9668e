// The sampler chain (repeat penalty, top-k, top-p, min-p, temperature, pick) for every row of logits of
// a step in one launch, a cluster of CTAs per row ([P1] "llama.cpp AI LLM Engine - Як це працює", the
// sampler chain after Крок 14; the steps are those of sampler.cu).
//
// A row is read once: each CTA of its cluster keeps a contiguous slice in shared memory as
// order-preserving 32-bit keys. The candidates' order is (logit descending, id ascending), so an element is
// the 64-bit number key << 32 | ~id, and every cut-off (top-k, top-p, min-p, and the pick itself) is "the
// elements down to the first one where a running sum reaches a target".
//
// Up to kListMax candidates (top_k): one histogram of 512 bins between the row's largest value and its mean finds an
// upper set of at least k elements that hardly exceeds k (a second histogram of the last bin where the first
// leaves too many); they move into the first CTA, which sorts them and goes on with prefix sums.
// More candidates, or rows where that set stays too large (ties, infinities): every cut-off is found where the
// elements lie, by a radix select over the 64-bit numbers: per digit a histogram of the running sum (a
// count, or weights), summed over the cluster through distributed shared memory, and a scan from the top; it
// stops as soon as the bin found is needed whole, or holds one element.
//
// Sums of probabilities are integers: a weight exp((l - l_max) / t) is rounded to a multiple of 2^-44, so
// sums of up to 2^18 of them are exact in 64 bits whatever their order, and the pick depends on neither
// the launch nor the order of atomics. The weight itself is computed to about 2^-42 relative (a
// two-float argument, a table of 2^(i/64) and a short polynomial, in 64-bit integers): float32 weights
// would move a boundary by 1e-7 and with it one pick in some thousands; FP64 units are slow here.
//
// Measured: one row of 151936 with every step and 64 listed tokens 20.5 us, 32 rows of 128256 (16 MB) with top-k 40 and
// top-p 28.0 us. That is latency: the start of the clusters, the row, the histograms, the sort and the chain on the
// sorted list follow from one another; issue slots are used for a third of the time, and warps wait for barriers most.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <utility>

#include "paged.h"

namespace cg = cooperative_groups;

namespace llm {

namespace {

constexpr int kThr = 512;
constexpr int kWarps = kThr / 32;
constexpr int kListMax = 4096;
constexpr int kBins = 256;
constexpr int kNear = 512;                                   // bins from the largest value to the mean; kThr of them
constexpr int kClusterMax = 8;
constexpr int kSliceMax = 45056;                             // keys of a slice: 176 KB
constexpr int kWeightBits = 44;

// 2^(i/64) in units of 2^-62
__constant__ uint64_t kExp2[64] = {
    0x4000000000000000ull, 0x40b268f9de0183baull, 0x4166c34c5615d0ecull, 0x421d1461d66f2023ull,
    0x42d561b3e6243d8aull, 0x438fb0cb4f468808ull, 0x444c0740496d4294ull, 0x450a6abaa4b77ecdull,
    0x45cae0f1f545eb73ull, 0x468d6fadbf2dd4f3ull, 0x47521cc5a2e6a9e0ull, 0x4818ee218a3358eeull,
    0x48e1e9b9d588e19bull, 0x49ad159789f37496ull, 0x4a7a77d47f7b84b1ull, 0x4b4a169b900c2d00ull,
    0x4c1bf828c6dc54b8ull, 0x4cf022c9905bfd32ull, 0x4dc69cdceaa72a9cull, 0x4e9f6cd3967fdba8ull,
    0x4f7a993048d088d7ull, 0x50582887dcb8a7e1ull, 0x513821818624b40cull, 0x521a8ad704f3404full,
    0x52ff6b54d8a89c75ull, 0x53e6c9da74b29ab5ull, 0x54d0ad5a753e077cull, 0x55bd1cdad49f699cull,
    0x56ac1f752150a563ull, 0x579dbc56b48521baull, 0x5891fac0e95612c8ull, 0x5988e20954889245ull,
    0x5a827999fcef3242ull, 0x5b7ec8f19468bbc9ull, 0x5c7dd7a3b17dcf75ull, 0x5d7fad59099f22feull,
    0x5e8451cfac061b5full, 0x5f8bccdb3d398841ull, 0x6096266533384a2bull, 0x61a3666d124bb204ull,
    0x62b39508aa836d6full, 0x63c6ba6455dcd8aeull, 0x64dcdec3371793d1ull, 0x65f60a7f79393e2eull,
    0x6712460a8fc24072ull, 0x683199ed779592caull, 0x69540ec8f895722dull, 0x6a79ad55e7f6fd10ull,
    0x6ba27e656b4eb57aull, 0x6cce8ae13c57ebdbull, 0x6dfddbcbed791babull, 0x6f307a412f074892ull,
    0x70666f76154a7089ull, 0x719fc4b95f452d29ull, 0x72dc8373be41a454ull, 0x741cb5281e25ee34ull,
    0x75606373ee921c97ull, 0x76a7980f6cca15c2ull, 0x77f25ccdee6d7ae6ull, 0x7940bb9e2cffd89dull,
    0x7a92be8a92436616ull, 0x7be86fb985689ddcull, 0x7d41d96db915019dull, 0x7e9f06067a4360baull,
};

__device__ __forceinline__ uint32_t key_of(float v) {
    if (v != v) return 0u;                                   // NaN orders below everything
    const uint32_t b = __float_as_uint(v + 0.f);             // -0 is +0
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
constexpr uint32_t kKeyNan = 0u, kKeyNegInf = 0x007fffffu;

// The factor log2(e) / t as two floats.
struct Slope { float hi, lo; };
constexpr double kLog2E = 1.4426950408889634074;
constexpr Slope kSlopeOne{(float)kLog2E, (float)(kLog2E - (double)(float)kLog2E)};
__device__ __forceinline__ Slope slope_of(double t) {
    const double c = kLog2E / t;
    Slope s;
    s.hi = (float)c;
    s.lo = isinf(s.hi) ? 0.f : (float)(c - (double)s.hi);
    return s;
}

// round(2^44 exp((l - top) / t)) for l <= top; 0 for -infinity and NaN, 2^44 where l == top.
__device__ __forceinline__ uint64_t weight_of(uint32_t key, float top, const Slope c) {
    if (key <= kKeyNegInf) return 0ull;
    const float l = value_of(key);
    if (l == top) return 1ull << kWeightBits;
    // d = l - top = dh + dl exactly
    const float dh = l - top, t = dh - l;
    const float dl = (l - (dh - t)) + (-top - t);
    // y = d * c = yh + ye to about 2^-47 of |y|
    const float yh = __fmul_rn(dh, c.hi);
    if (!(yh > -64.f)) return 0ull;                          // below half of 2^-44 (or -inf)
    const float ye = fmaf(dh, c.hi, -yh) + fmaf(dh, c.lo, dl * c.hi);
    const float n = rintf(yh);
    // y in units of 2^-46 (yh - n is exact)
    const int64_t y = (int64_t)n * (1ll << 46) + __float2ll_rn((yh - n) * 70368744177664.f) +
                      __float2ll_rn(ye * 70368744177664.f);
    const int e = (int)(y >> 46);                            // floor
    const uint64_t f = (uint64_t)y & ((1ull << 46) - 1);
    const int i = (int)(f >> 40);
    const uint64_t r = (f & ((1ull << 40) - 1)) << 18;       // the rest of the fraction, in 2^-64 (below 2^-6)
    // z = r ln 2 < 0.0109; e^z - 1 = z + z^2 / 2 + z^3 (1/6 + z/24 + z^2/120), in 2^-64
    const uint64_t z = __umul64hi(r, 0xb17217f7d1cf79acull);
    const uint64_t z2 = __umul64hi(z, z);
    const float zf = __ull2float_rn(z) * 5.4210108624275222e-20f;
    const float tail = zf * zf * zf * fmaf(zf, fmaf(zf, 1.f / 120.f, 1.f / 24.f), 1.f / 6.f);
    const uint64_t m1 = z + (z2 >> 1) + (uint64_t)(tail * 1.8446744073709552e19f);
    const uint64_t m = kExp2[i] + __umul64hi(kExp2[i], m1);  // 2^frac in 2^-62
    const int sh = 62 - kWeightBits - e;                     // e <= 0 here
    if (sh > 63) return 0ull;
    return (m >> sh) + ((m >> (sh - 1)) & 1ull);
}

struct Shared {
    uint64_t sum[2][kBins];                                  // histograms, alternating
    union {
        uint32_t cnt[2][kBins];
        uint32_t near[kNear];                                // elements by distance from the largest
    };
    uint64_t best;                                           // the slice's first element
    float total_v[kClusterMax];                              // the slices' sums of finite values, and how many
    uint32_t n_finite[kClusterMax];
    uint64_t bests[kClusterMax];
    float wsumf[kWarps];
    uint32_t near_bin, near_before, near_count;
    // FP64 is slow here: one thread computes what needs it, early
    Slope slope;                                             // of the row's temperature
    double log_min_p;
    uint64_t target;
    uint64_t wsum[kWarps];
    uint32_t wcnt[kWarps];
    uint64_t found_before, total;
    uint32_t found_bin, found_count, n_list;
    int found;
};

constexpr size_t kSharedBytes = (sizeof(Shared) + 15) / 16 * 16;
constexpr int kPer = kListMax / kThr;                        // listed elements per thread
static_assert(kListMax >= 2 * kThr, "places for both orders");
static_assert(kNear == kThr, "a thread per bin");

enum Measure : int { M_COUNT = 0, M_WEIGHT = 1 };

// A CTA's slice of the row.
struct Elems {
    const uint32_t* keys;
    int n, base;
    __device__ __forceinline__ uint64_t at(int i) const { return ((uint64_t)keys[i] << 32) | (uint32_t)~(uint32_t)(base + i); }
};

// The CTAs of a row.
struct Group {
    Shared* sh;
    int size;                                                // CTAs
    int phase;                                               // histogram in use
};

__device__ __forceinline__ void group_sync(const Group&) { cg::this_cluster().sync(); }

// The bin histogram of the elements x >= cut whose digits above `shift` equal prefix's.
__device__ void histogram(const Elems& el, Group& g, Measure what, uint64_t cut, uint64_t prefix, int shift, int bits,
                          float top, const Slope c) {
    Shared& sh = *g.sh;
    uint64_t* sum = sh.sum[g.phase];
    uint32_t* cnt = sh.cnt[g.phase];
    for (int i = threadIdx.x; i < kBins; i += kThr) { sum[i] = 0ull; cnt[i] = 0u; }
    __syncthreads();
    const int lane = threadIdx.x & 31;
    const int up = shift + bits;
    for (int i0 = 0; i0 < el.n; i0 += kThr) {
        const int i = i0 + threadIdx.x;
        uint32_t bin = 0xffffffffu;
        uint64_t w = 0ull;
        if (i < el.n) {
            const uint64_t x = el.at(i);
            if (x >= cut && (up >= 64 || (x >> up) == (prefix >> up))) {
                bin = (uint32_t)(x >> shift) & ((1u << bits) - 1u);
                if (what == M_WEIGHT) w = weight_of((uint32_t)(x >> 32), top, c);
            }
        }
        if (!__any_sync(0xffffffffu, bin != 0xffffffffu)) continue;
        // one update per distinct bin of the warp
        const unsigned same = __match_any_sync(0xffffffffu, bin);
        const bool first = lane == __ffs(same) - 1;
        if (what == M_WEIGHT) {
            // 45-bit weights in two sums of at most 32 x 2^23
            const uint32_t lo = __reduce_add_sync(same, (uint32_t)w & 0x7fffffu);
            const uint32_t hi = __reduce_add_sync(same, (uint32_t)(w >> 23));
            if (bin != 0xffffffffu && first)
                atomicAdd(reinterpret_cast<unsigned long long*>(&sum[bin]), ((unsigned long long)hi << 23) + lo);
        }
        if (bin != 0xffffffffu && first) atomicAdd(&cnt[bin], (uint32_t)__popc(same));
    }
    group_sync(g);
}

// Sum the group's histograms and scan from the top bin: the first bin where before + the running sum
// reaches target (into sh.found_*; found = 0 if none does). Threads 0 .. kBins - 1 hold bin kBins - 1 - t.
__device__ void scan_bins(Group& g, Measure what, uint64_t before, uint64_t target) {
    Shared& sh = *g.sh;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    uint64_t s = 0ull;
    uint32_t n = 0u;
    if (t < kBins) {
        const int b = kBins - 1 - t;
        for (int r = 0; r < g.size; ++r) {
            const Shared* o = cg::this_cluster().map_shared_rank(&sh, r);
            n += o->cnt[g.phase][b];
            if (what == M_WEIGHT) s += o->sum[g.phase][b];
        }
        if (what == M_COUNT) s = n;
    }
    uint64_t inc = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
    }
    if (lane == 31) sh.wsum[warp] = inc;
    if (t == 0) sh.found = 0;
    __syncthreads();
    uint64_t add = before;
    for (int w = 0; w < warp && w < kBins / 32; ++w) add += sh.wsum[w];
    inc += add;
    if (t < kBins && n > 0u && inc - s < target && inc >= target) {
        sh.found = 1;
        sh.found_bin = (uint32_t)(kBins - 1 - t);
        sh.found_before = inc - s;
        sh.found_count = n;
        sh.total = inc;
    }
    __syncthreads();
    g.phase ^= 1;
}

// The least cut' >= cut such that the elements >= cut' hold at least `target` of the measure; cut itself if
// all elements together hold less. `one` asks for the boundary element itself: the digits are followed until
// a single element is left.
__device__ uint64_t select_cut(const Elems& el, Group& g, Measure what, uint64_t cut, uint64_t target, bool one,
                               float top, const Slope c) {
    uint64_t prefix = 0ull, before = 0ull;
    for (int shift = 56; shift >= 0; shift -= 8) {
        histogram(el, g, what, cut, prefix, shift, 8, top, c);
        scan_bins(g, what, before, target);
        const Shared& sh = *g.sh;
        if (!sh.found) return cut;                           // only in the first pass
        prefix |= (uint64_t)sh.found_bin << shift;
        before = sh.found_before;
        const bool whole = sh.total == target && what == M_COUNT, single = sh.found_count == 1u;
        __syncthreads();
        if (single || (whole && !one)) break;
    }
    return max(prefix, cut);
}

// The sum of the weights of the elements >= cut over the group.
__device__ uint64_t total_weight(const Elems& el, Group& g, uint64_t cut, float top, const Slope c) {
    Shared& sh = *g.sh;
    uint64_t w = 0ull;
    for (int i = threadIdx.x; i < el.n; i += kThr) {
        const uint64_t x = el.at(i);
        if (x >= cut) w += weight_of((uint32_t)(x >> 32), top, c);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
    if ((threadIdx.x & 31) == 0) sh.wsum[threadIdx.x >> 5] = w;
    __syncthreads();
    if (threadIdx.x == 0) {
        uint64_t s = 0ull;
        for (int i = 0; i < kWarps; ++i) s += sh.wsum[i];
        sh.sum[g.phase][0] = s;
    }
    group_sync(g);
    uint64_t z = 0ull;
    for (int r = 0; r < g.size; ++r)
        z += cg::this_cluster().map_shared_rank(&sh, r)->sum[g.phase][0];
    g.phase ^= 1;
    __syncthreads();
    return z;
}

// The key of the least float l with l - top >= ln(min_p) in double (the top's own key at most).
__device__ __forceinline__ uint32_t min_p_key(float top, double log_min_p) {
    const double lim = (double)top + log_min_p;
    float f = (float)lim;
    if ((double)f < lim) f = nextafterf(f, INFINITY);
    return min(key_of(f), key_of(top));
}
// The pick is the first candidate whose running weight exceeds u z.
__device__ __forceinline__ uint64_t pick_target(uint64_t z, float u) {
    u = fminf(fmaxf(u, 0.f), 0.99999994f);                   // (NaN: 0)
    return min(z, (uint64_t)floor((double)u * (double)z) + (uint64_t)1);
}
// x * f rounded as a double, up to a whole number, within [1, x] (f in (0, 1))
__device__ __forceinline__ uint64_t share_up(uint64_t x, float f) {
    const double t = ceil((double)f * (double)x);
    return t < 1.0 ? 1ull : min(x, (uint64_t)t);
}

// Inclusive prefix sum over the block; *total the sum of all (kThr threads, sh.wsum free before and after).
__device__ uint64_t block_scan(Shared& sh, uint64_t v, uint64_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += x;
    }
    if (lane == 31) sh.wsum[warp] = v;
    __syncthreads();
    uint64_t add = 0ull, all = 0ull;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const uint64_t x = sh.wsum[w];
        if (w < warp) add += x;
        all += x;
    }
    *total = all;
    __syncthreads();
    return v + add;
}

// The first of the m sorted elements (thread t holds w[] of per t ..) where the running weight reaches the target
// that thread 0 has from make(); m - 1 if none does. `before`: the thread's exclusive prefix.
template <typename F>
__device__ int first_reaching(Shared& sh, const uint64_t* w, uint64_t before, int per, int m, F make) {
    if (threadIdx.x == 0) {
        sh.found = m - 1;
        sh.target = make();
    }
    __syncthreads();
    const uint64_t target = sh.target;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        if (j >= per) break;
        const int i = threadIdx.x * per + j;
        if (i < m && before < target && before + w[j] >= target) sh.found = i;   // one thread's, once
        before += w[j];
    }
    __syncthreads();
    const int f = sh.found;
    __syncthreads();
    return f;
}

// The chain over n listed elements, an upper set of the row with at least min(k, candidates) of them: sorted, then
// cut to k, by top-p and min-p, then the pick. One CTA; list has kListMax places.
__device__ int32_t list_chain(Shared& sh, uint64_t* list, int n, int k, float top_p, float min_p, float u) {
    const int tid = threadIdx.x;
    if (n <= kThr) {
        // few: a thread per element counts those before it; sorted into the list's next places
        uint64_t* spare = list + kThr;
        const uint64_t x = tid < n ? list[tid] : 0ull;
        int r = 0;
        for (int i = 0; i < n; ++i) r += list[i] > x;
        if (tid < n) spare[r] = x;
        __syncthreads();
        list = spare;
    } else {
        int P = 2 * kThr;
        while (P < n) P <<= 1;
        for (int i = n + tid; i < P; i += kThr) list[i] = 0ull;
        __syncthreads();
        for (int size = 2; size <= P; size <<= 1)
            for (int stride = size >> 1; stride > 0; stride >>= 1) {
                for (int p = tid; p < P / 2; p += kThr) {
                    const int i = 2 * p - (p & (stride - 1)), j = i + stride;
                    const uint64_t x = list[i], y = list[j];
                    if ((x < y) == ((i & size) == 0)) { list[i] = y; list[j] = x; }   // descending
                }
                __syncthreads();
            }
    }
    // the sorted elements per t .. per t + per - 1 are thread t's
    const int per = (n + kThr - 1) / kThr;
    uint64_t x[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) x[j] = j < per && tid * per + j < n ? list[tid * per + j] : 0ull;
    const float top = value_of((uint32_t)(list[0] >> 32));
    int m = min(n, k);
    uint64_t w[kPer], z, loc;
    auto weigh = [&](const Slope c) {
        loc = 0ull;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            w[j] = 0ull;
            if (j < per && tid * per + j < m) w[j] = weight_of((uint32_t)(x[j] >> 32), top, c);
            loc += w[j];
        }
        return block_scan(sh, loc, &z) - loc;
    };
    if (top_p < 1.f) {
        const uint64_t before = weigh(kSlopeOne);
        m = first_reaching(sh, w, before, per, m, [&] { return share_up(z, top_p); }) + 1;
    }
    if (min_p > 0.f) {
        if (tid == 0) sh.target = min_p_key(top, sh.log_min_p);
        __syncthreads();
        const uint32_t least = (uint32_t)sh.target;
        int c = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) c += j < per && tid * per + j < m && (uint32_t)(x[j] >> 32) >= least;
        uint64_t all;
        block_scan(sh, (uint64_t)c, &all);
        m = max(1, (int)all);
    }
    const uint64_t before = weigh(sh.slope);
    const int f = first_reaching(sh, w, before, per, m, [&] { return pick_target(z, u); });
    return (int32_t)~(uint32_t)list[f];
}

// Bin of value v by its distance from the largest, 0 the nearest; kNear or more: farther than the mean.
__device__ __forceinline__ uint32_t near_bin(float v, float top, float scale) {
    const float d = (top - v) * scale;                       // (monotone: the elements up to a bin are an upper set)
    return d < (float)kNear ? (uint32_t)d : (uint32_t)kNear; // NaN and -infinity are far
}

// sh.near summed over the cluster, and the bin where the count from the top reaches k: sh.near_*; near_count = 0 if
// none does. The others may still be reading near afterwards: a cluster barrier before it is written again.
__device__ void near_scan(Shared& sh, int CL, uint32_t k) {
    cg::cluster_group cluster = cg::this_cluster();
    if (threadIdx.x == 0) sh.near_count = 0u;
    cluster.sync();
    uint32_t n = 0u;
#pragma unroll
    for (int r = 0; r < kClusterMax; ++r)
        if (r < CL) n += cluster.map_shared_rank(&sh, r)->near[threadIdx.x];
    uint64_t all;
    const uint32_t inc = (uint32_t)block_scan(sh, n, &all);
    if (inc >= k && inc - n < k) {
        sh.near_bin = threadIdx.x;
        sh.near_before = inc - n;
        sh.near_count = n;
    }
    __syncthreads();
}

template <int T>
__device__ __forceinline__ float logit(const void* p, int64_t i) {
    if constexpr (T == W_F32) return static_cast<const float*>(p)[i];
    else if constexpr (T == W_F16) return __half2float(static_cast<const __half*>(p)[i]);
    else return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

// f(key, index) for every key of a slice (16-byte aligned, its length rounded up to 32 keys).
template <typename F>
__device__ __forceinline__ void each_key(const uint32_t* keys, int n, F f) {
#pragma unroll 2
    for (int i = 4 * threadIdx.x; i < n; i += 4 * kThr) {
        const uint4 x = *reinterpret_cast<const uint4*>(keys + i);
        f(x.x, i);
        if (i + 1 < n) f(x.y, i + 1);
        if (i + 2 < n) f(x.z, i + 2);
        if (i + 3 < n) f(x.w, i + 3);
    }
}

template <int T>
__global__ void __launch_bounds__(kThr) sample_rows_kernel(SampleRowsArgs a, int slice, int aligned) {
    extern __shared__ __align__(16) uint8_t raw[];
    Shared& sh = *reinterpret_cast<Shared*>(raw);
    uint64_t* list = reinterpret_cast<uint64_t*>(raw + kSharedBytes);                  // [kListMax], first CTA
    uint32_t* keys = reinterpret_cast<uint32_t*>(list + kListMax);                     // [slice]
    uint32_t* marked = keys + slice;                                                  // a bit per key
    cg::cluster_group cluster = cg::this_cluster();
    const int CL = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int e = blockIdx.x / CL;                                                    // entry
    const int64_t row = a.row ? a.row[e] : e;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b0 = rank * slice, n = max(0, min(slice, a.V - b0));
    const float temp = a.temperature ? a.temperature[e] : 0.f;
    const float top_p = a.top_p ? a.top_p[e] : 1.f;
    const float min_p = a.min_p ? a.min_p[e] : 0.f;
    const float u = a.u ? a.u[e] : 0.f;
    const int k = a.top_k ? a.top_k[e] : 0;
    const float pen = a.penalty ? a.penalty[e] : 1.f;

    // the row's penalty list starts its way before the logits do
    const bool penal = pen != 1.f && a.pen_start && a.pen_tok;
    const int pen0 = penal ? max(a.pen_start[e], 0) : 0, pen1 = penal ? min(a.pen_start[e + 1], a.n_pen) : 0;
    const int pen_first = pen0 + tid < pen1 ? a.pen_tok[pen0 + tid] : -1;
    if (penal)
        for (int i = tid; i < (n + 31) / 32; i += kThr) marked[i] = 0u;
    if (tid == 0) sh.n_list = 0u;
    if (tid == kThr - 1) {
        if (temp > 0.f) sh.slope = slope_of((double)temp);
        if (min_p > 0.f) sh.log_min_p = log((double)fminf(min_p, 1.f));
    }
    auto started = cluster.barrier_arrive();
    // the slice's first element, and the sum and number of its finite values
    uint32_t top = 0u, top_i = 0u, fin = 0u;
    float sum = 0.f;
    auto note = [&](uint32_t x, int i) {
        if (x > top) { top = x; top_i = (uint32_t)i; }
        const float v = value_of(x);
        if (fabsf(v) <= 3.0e38f && x != kKeyNan) { sum += v; ++fin; }
    };
    // the slice: 16 bytes a load, eight under way
    constexpr int ES = T == W_F32 ? 4 : 2, PV = 16 / ES;
    const uint8_t* src = static_cast<const uint8_t*>(a.logits) + (row * a.ld + b0) * ES;
    const int nv = aligned ? n / PV : 0;
    for (int i0 = 0; i0 < nv; i0 += 8 * kThr) {
        uint4 q[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = i0 + j * kThr + tid;
            if (i < nv) q[j] = __ldcs(reinterpret_cast<const uint4*>(src) + i);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = i0 + j * kThr + tid;
            if (i >= nv) continue;
            uint32_t x[PV];
#pragma unroll
            for (int c = 0; c < PV; ++c) {
                x[c] = key_of(logit<T>(&q[j], c));
                note(x[c], i * PV + c);
            }
#pragma unroll
            for (int c = 0; c < PV; c += 4)
                *reinterpret_cast<uint4*>(keys + i * PV + c) = make_uint4(x[c], x[c + 1], x[c + 2], x[c + 3]);
        }
    }
    for (int i = nv * PV + tid; i < n; i += kThr) {
        keys[i] = key_of(logit<T>(src, i));
        note(keys[i], i);
    }
    if (penal) {
        __syncthreads();
        for (int j = pen0 + tid; j < pen1; j += kThr) {
            const int t = (j < pen0 + kThr ? pen_first : a.pen_tok[j]) - b0;
            if (t < 0 || t >= n) continue;
            if (atomicOr(&marked[t >> 5], 1u << (t & 31)) >> (t & 31) & 1u) continue;   // listed before
            const float v = value_of(keys[t]);
            if (keys[t] != kKeyNan) keys[t] = key_of(v > 0.f ? __fdiv_rn(v, pen) : __fmul_rn(v, pen));
        }
        __syncthreads();
        top = top_i = fin = 0u;
        sum = 0.f;
        each_key(keys, n, note);
    }
    uint64_t best = ((uint64_t)top << 32) | (uint32_t)~(uint32_t)(b0 + top_i);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    fin = __reduce_add_sync(0xffffffffu, fin);
    if (lane == 0) { sh.wsum[warp] = best; sh.wsumf[warp] = sum; sh.wcnt[warp] = fin; }
    __syncthreads();
    cluster.barrier_wait(std::move(started));               // every CTA of the row is running
    if (tid < CL) {                                         // to every CTA
        float s = 0.f;
        uint32_t c = 0u;
        uint64_t x = 0ull;
        for (int i = 0; i < kWarps; ++i) { x = max(x, sh.wsum[i]); s += sh.wsumf[i]; c += sh.wcnt[i]; }
        Shared* o = cluster.map_shared_rank(&sh, tid);
        o->bests[rank] = x;
        o->total_v[rank] = s;
        o->n_finite[rank] = c;
    }
    cluster.sync();
    best = 0ull;
    sum = 0.f;
    fin = 0u;
    for (int r = 0; r < CL; ++r) { best = max(best, sh.bests[r]); sum += sh.total_v[r]; fin += sh.n_finite[r]; }
    top = (uint32_t)(best >> 32);
    const float top_v = value_of(top);
    if (!(temp > 0.f) || !(top_p > 0.f) || top <= kKeyNegInf) {   // the first candidate, or none
        if (rank == 0 && tid == 0) a.token[e] = top <= kKeyNegInf ? -1 : (int32_t)~(uint32_t)best;
        return;                                              // (no CTA reads another's memory after the barrier)
    }
    if (k > 0 && k <= kListMax && k < a.V) {
        // an upper set of k elements or slightly more. Of logits spread like a normal distribution the k first are within
        // 0.4 of the way to the mean where they are few (0.2% of the vocabulary), and within two thirds up to
        // some 7%; other rows look as far as the mean
        const float gap = top_v - sum / (float)max(fin, 1u);
        uint32_t bin1 = kNear, bin2 = kNear, count = 0xffffffffu, floor_key = 0u;
        float scale = 0.f, lo = 0.f, fine = 0.f;
        // no element below it is within `bins` bins (rounding errors of top - v and of this included)
        auto key_below = [&](float bins) { return key_of(top_v - bins / scale - fabsf(top_v) * 1e-6f); };
        for (int far = 0; far < 2 && count == 0xffffffffu; ++far) {
            scale = (float)kNear / (far ? gap : gap * (k <= a.V / 512 ? 0.4f : 0.667f));
            if (!(scale > 0.f && scale < 3.0e38f)) break;
            if (far) cluster.sync();
            sh.near[tid] = 0u;
            __syncthreads();
            floor_key = key_below((float)kNear + 1.f);
            each_key(keys, n, [&](uint32_t x, int) {
                if (x < floor_key) return;
                const uint32_t b = near_bin(value_of(x), top_v, scale);
                if (b < kNear) atomicAdd(&sh.near[b], 1u);
            });
            near_scan(sh, CL, (uint32_t)k);
            if (sh.near_count > 0u) {
                bin1 = sh.near_bin;
                count = sh.near_before + sh.near_count;
            }
        }
        if (bin1 < kNear && count > kListMax) {
            // the last bin again, 512 times as fine
            const uint32_t before = sh.near_before;
            lo = (float)bin1;
            fine = (float)kNear;
            cluster.sync();
            sh.near[tid] = 0u;
            __syncthreads();
            each_key(keys, n, [&](uint32_t x, int) {
                const float v = value_of(x);
                if (near_bin(v, top_v, scale) != bin1) return;
                atomicAdd(&sh.near[min((uint32_t)(((top_v - v) * scale - lo) * fine), (uint32_t)kNear - 1u)], 1u);
            });
            near_scan(sh, CL, (uint32_t)k - before);
            bin2 = sh.near_bin;                              // (found: the bin's elements reach k)
            count = before + sh.near_before + sh.near_count;
        }
        if (bin1 < kNear) floor_key = key_below((float)bin1 + 2.f);
        if (count <= kListMax) {
            Shared* s0 = cluster.map_shared_rank(&sh, 0);
            uint64_t* l0 = cluster.map_shared_rank(list, 0);
            auto give = [&](uint32_t x, int i) {            // the whole warp
                bool take = x >= floor_key && i < n;
                if (take) {
                    const float v = value_of(x);
                    const uint32_t b = near_bin(v, top_v, scale);
                    take = b < bin1 || (b == bin1 && (bin2 == kNear ||
                                                      min((uint32_t)(((top_v - v) * scale - lo) * fine), (uint32_t)kNear - 1u) <= bin2));
                }
                const unsigned ball = __ballot_sync(0xffffffffu, take);
                if (!ball) return;
                uint32_t at = 0u;
                if (lane == 0) at = atomicAdd(&s0->n_list, (uint32_t)__popc(ball));
                at = __shfl_sync(0xffffffffu, at, 0) + __popc(ball & ((1u << lane) - 1u));
                if (take && at < (uint32_t)kListMax) l0[at] = ((uint64_t)x << 32) | (uint32_t)~(uint32_t)(b0 + i);
            };
            for (int i0 = 0; i0 < n; i0 += 4 * kThr) {      // (the slice's places past n hold no key: i < n above)
                const int i = i0 + 4 * tid;
                uint4 x = make_uint4(0u, 0u, 0u, 0u);
                if (i < n) x = *reinterpret_cast<const uint4*>(keys + i);
                if (!__any_sync(0xffffffffu, max(max(x.x, x.y), max(x.z, x.w)) >= floor_key)) continue;
                give(x.x, i); give(x.y, i + 1); give(x.z, i + 2); give(x.w, i + 3);
            }
            cluster.sync();
            if (rank != 0) return;                           // nobody reads or writes this CTA any more
            const int32_t tok = list_chain(sh, list, (int)min(sh.n_list, (uint32_t)kListMax), k,
                                           top_p, min_p, u);
            if (tid == 0) a.token[e] = tok;
            return;
        }
    }
    // every candidate where it lies
    cluster.sync();                                          // (the histograms share their memory with the one above)
    Group g{&sh, CL, 0};
    const Elems el{keys, n, b0};
    uint64_t cut = (uint64_t)(kKeyNan + 1u) << 32;           // NaN is no candidate
    if (k > 0 && k < a.V) cut = select_cut(el, g, M_COUNT, cut, (uint64_t)k, false, top_v, Slope{0.f, 0.f});
    if (top_p < 1.f) {
        const uint64_t z = total_weight(el, g, cut, top_v, kSlopeOne);
        cut = select_cut(el, g, M_WEIGHT, cut, share_up(z, top_p), false, top_v, kSlopeOne);
    }
    if (min_p > 0.f) cut = max(cut, (uint64_t)min_p_key(top_v, sh.log_min_p) << 32);
    const Slope slope = sh.slope;
    const uint64_t z = total_weight(el, g, cut, top_v, slope);
    cut = select_cut(el, g, M_WEIGHT, cut, pick_target(z, u), true, top_v, slope);
    // the boundary element is the least one >= its prefix
    best = ~0ull;
    for (int i = tid; i < el.n; i += kThr) {
        const uint64_t x = el.at(i);
        if (x >= cut) best = min(best, x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) best = min(best, __shfl_xor_sync(0xffffffffu, best, o));
    if (lane == 0) sh.wsum[warp] = best;
    __syncthreads();
    if (tid == 0) {
        for (int i = 0; i < kWarps; ++i) best = min(best, sh.wsum[i]);
        sh.best = best;
    }
    cluster.sync();
    if (rank == 0 && tid == 0) {
        for (int r = 0; r < CL; ++r) best = min(best, cluster.map_shared_rank(&sh, r)->best);
        a.token[e] = (int32_t)~(uint32_t)best;
    }
    cluster.sync();                                          // no CTA leaves while another reads it
}

size_t smem_bytes(int slice) {
    return kSharedBytes + sizeof(uint64_t) * kListMax + sizeof(uint32_t) * ((size_t)slice + (slice + 31) / 32);
}

template <int T>
bool go(const SampleRowsArgs& a, cudaStream_t st) {
    // CTAs per row: a slice of about 16384 keys each (64 KB, so that two CTAs fit an SM)
    int cl = 1;
    while (cl < kClusterMax && (int64_t)cl * 16384 < a.V) cl *= 2;
    const int slice = ((a.V + cl - 1) / cl + 31) / 32 * 32;
    if (slice > kSliceMax) return false;
    const size_t bytes = smem_bytes(slice);
    static std::atomic<uint64_t> done{0};
    if (!allow_smem(reinterpret_cast<const void*>(sample_rows_kernel<T>), smem_bytes(kSliceMax), done)) return false;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.n_rows * cl));
    cfg.blockDim = dim3(kThr);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)cl;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const int es = T == W_F32 ? 4 : 2;
    const int aligned = (reinterpret_cast<uintptr_t>(a.logits) % 16 == 0) && a.ld * es % 16 == 0;
    return cudaLaunchKernelEx(&cfg, sample_rows_kernel<T>, a, slice, aligned) == cudaSuccess;
}

}  // namespace

int32_t sample_rows_max_vocab() { return kClusterMax * kSliceMax; }

bool launch_sample_rows(const SampleRowsArgs& a, cudaStream_t st) {
    if (a.n_rows == 0) return true;
    switch (a.type) {
        case W_F32: return go<W_F32>(a, st);
        case W_F16: return go<W_F16>(a, st);
        case W_BF16: return go<W_BF16>(a, st);
    }
    return false;
}

}  // namespace llm
