// Host plan of the attention over a paged cache: tiles of (token, query head) rows per sequence, the
// keys each tile may see, and an even share of all of that for every CTA that runs at once.
#include "paged.h"

#include <algorithm>

namespace llm {

namespace {

// Keys are dealt out in blocks: what the warps of a small-tile CTA take at once (32 keys each), or the 128 keys
// that the 256-row form multiplies at a time.
int64_t block_keys(const PlanShape& s, int f, int rows) { return f ? 128 : 32 * attn_rows_warps(s.hd, s.kv_type, rows); }
// What a unit costs beyond its keys, in blocks: Q in, the warps' (halves') results out and merged. (32 / 8 heads of
// 128. Small tiles: 32 single tokens over 1 .. 2304 keys took 47, 39 and 39 us at 0, 1 and 2, one over 513 11.3, 12.3
// and 14 us. 256 rows: chunks of 20 .. 1000 tokens of five sequences 99, 89 and 87 us at 2, 3 and 4, 16 tokens over
// 8192 keys 40 us at 3 and 46 us at 4. E2M1 caches. Small tiles: the same single tokens 23.8 and 24.8 us at 1 and 2, one over 513
// 9.2 and 8.4. 256 rows at 2, 3, 4 and 6, bf16: five chunks of 20 .. 1000 tokens 155, 131, 128 and 133 us, under a window of
// 1024 72, 69, 68 and 60; 512 tokens over 8192 keys 87, 84, 83 and 91; 16 over 8192 40, 39, 46 and 46: 3 fits them as well, and
// a windowed step of short chunks would gain a seventh at 6.)
constexpr int64_t kUnitCost[2] = {1, 3};
// Sequences with at least this many rows per KV head take 256-row tiles. 32 / 8 heads of 128, small tiles against large
// ones, us: f16, one sequence over 8192 keys: 32 rows 30 : 40, 64 rows 37 : 40, 96 rows 45 : 41, 128 rows 52 : 42;
// sixteen over 2048: 32 rows 58 : 39, 64 rows 96 : 39. E4M3 (whose large tiles convert their rows first): one, 64 rows
// 29 : 46, 128 rows 44 : 47; sixteen, 32 rows 37 : 60, 64 rows 73 : 60. E2M1: one, 32 rows 24 : 39, 64 rows 29 : 40, 96 rows
// 39 : 41, 128 rows 44 : 42; sixteen, 32 rows 37 : 39, 64 rows 75 : 40. One number for all types is a compromise: it fits
// many sequences of E4M3 and E2M1 rows and costs a single one 17 and 11 us at 64 rows, and f16 steps of many sequences would
// gain at 32.
constexpr int64_t kTcRows = 64;

int64_t ctas(const PlanShape& s, int f) { return (int64_t)s.n_sm * (f ? 1 : kAttnRowsCtas); }

// Where the 256-row form's key ranges begin: at multiples of a run of a page's cells.
int64_t block_align(const PlanShape& s) {
    int64_t align = 64;
    while (align > 1 && s.page_size % align) align /= 2;
    return align;
}

int64_t up_to(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// The virtual key range of the rows [row0, row0 + n) of a sequence: sink keys, then [lo, hi).
struct Keys { int32_t n_sink, lo, n; };

// align > 1: both parts begin and end (the sinks) at multiples of it, so that blocks of keys are whole runs of a
// page's cells; the keys that come in by this are hidden from every row.
Keys tile_keys(const PlanShape& s, const PlanSeq& q, int64_t row0, int64_t n, int64_t align) {
    const int64_t t0 = row0 / s.G, t1 = (row0 + n - 1) / s.G;
    int64_t pmin = (int64_t)q.p0 + t0, pmax = (int64_t)q.p0 + t1;
    if (q.tok_pos) {
        pmin = pmax = q.tok_pos[t0];
        for (int64_t t = t0 + 1; t <= t1; ++t) {
            pmin = std::min<int64_t>(pmin, q.tok_pos[t]);
            pmax = std::max<int64_t>(pmax, q.tok_pos[t]);
        }
    }
    // keys in position order: the first with a position >= p
    auto first = [&](int64_t p) -> int64_t {
        if (!q.key_pos) return std::min<int64_t>(std::max<int64_t>(p, 0), q.n_keys);
        if (p > INT32_MAX) return q.n_keys;
        return std::lower_bound(q.key_pos, q.key_pos + q.n_keys, (int32_t)std::max<int64_t>(p, INT32_MIN)) - q.key_pos;
    };
    Keys k{};
    const int64_t hi = first(pmax + 1);
    if (s.window == 0) {
        k.n = (int32_t)hi;
        return k;
    }
    const int64_t lo = std::min(hi, first(pmin - s.window + 1)) / align * align;
    k.n_sink = (int32_t)std::min(lo, up_to(first(s.n_sink), align));
    k.lo = (int32_t)lo;
    k.n = (int32_t)(k.n_sink + hi - lo);
    return k;
}

}  // namespace

void build_paged_plan(const PlanShape& s, const std::vector<PlanSeq>& seqs, PagedPlan& plan) {
    plan = PagedPlan();
    auto tc = [&](const PlanSeq& q) { return s.tc && (int64_t)q.n_new * s.G >= kTcRows; };
    // rows of the small tiles: 8 where every sequence that takes them fits (half the products of 16)
    plan.rows1 = 8;
    for (const PlanSeq& q : seqs)
        if (!tc(q) && (int64_t)q.n_new * s.G > 8) plan.rows1 = 16;
    const int64_t align = block_align(s);
    struct Tile { int32_t seq, row0, n_row; Keys keys; };
    std::vector<Tile> tiles[2];
    int64_t total[2] = {0, 0};
    for (size_t i = 0; i < seqs.size(); ++i) {
        const int64_t rows = (int64_t)seqs[i].n_new * s.G;
        const int f = tc(seqs[i]);
        const int64_t step = f ? kUnitRows2 : plan.rows1;
        for (int64_t r = 0; r < rows; r += step) {
            Tile t{(int32_t)i, (int32_t)r, (int32_t)std::min(step, rows - r), {}};
            t.keys = tile_keys(s, seqs[i], t.row0, t.n_row, f && !seqs[i].key_pos ? align : 1);
            const int64_t bk = block_keys(s, f, plan.rows1);
            total[f] += (t.keys.n + bk - 1) / bk + kUnitCost[f];
            tiles[f].push_back(t);
        }
    }
    for (int f = 0; f < 2; ++f) {
        PlanForm& pf = plan.form_[f];
        if (tiles[f].empty()) continue;
        const int64_t n_cta = ctas(s, f), cost = kUnitCost[f], bk = block_keys(s, f, plan.rows1);
        // a CTA's share: what is there divided evenly, and one more unit for the cut at its end
        const int64_t share = (total[f] * s.Hkv + n_cta - 1) / n_cta + cost;
        int64_t left = share;                           // of the current CTA's share
        pf.first.assign(1, 0);
        auto next_cta = [&]() { pf.first.push_back((int32_t)pf.units.size()); left = share; };
        size_t i0 = 0;
        while (i0 < tiles[f].size()) {
            // the tiles of a sequence head by head, so that neighbouring CTAs read the same keys
            size_t i1 = i0;
            while (i1 < tiles[f].size() && tiles[f][i1].seq == tiles[f][i0].seq) ++i1;
            for (int32_t h = 0; h < s.Hkv; ++h)
                for (size_t i = i0; i < i1; ++i) {
                    const Tile& t = tiles[f][i];
                    const PlanSeq& q = seqs[t.seq];
                    const int64_t blocks = (t.keys.n + bk - 1) / bk;
                    const size_t u0 = pf.units.size();
                    int64_t at = 0;
                    do {
                        const bool last_cta = (int64_t)pf.first.size() >= n_cta;
                        if (left <= cost && !last_cta) next_cta();
                        int64_t take = blocks - at;
                        // past the share: cut (a remainder shorter than a unit's cost is not left over)
                        if ((int64_t)pf.first.size() < n_cta && take > left) take = left - cost;
                        AttnUnit u{};
                        u.tok0 = q.tok0;
                        u.row0 = t.row0;
                        u.n_row = t.n_row;
                        u.p0 = q.p0;
                        u.table = q.table;
                        u.n_sink_keys = t.keys.n_sink;
                        u.key_lo = t.keys.lo;
                        u.v0 = (int32_t)(at * bk);
                        u.v1 = (int32_t)std::min<int64_t>(t.keys.n, (at + take) * bk);
                        u.chunk = (int32_t)(pf.units.size() - u0);
                        u.head = h;
                        pf.units.push_back(u);
                        at += take;
                        left -= take + cost;
                    } while (at < blocks);
                    const int32_t n = (int32_t)(pf.units.size() - u0);
                    for (size_t j = u0; j < pf.units.size(); ++j) {
                        pf.units[j].n_chunk = n;
                        pf.units[j].part = n > 1 ? pf.n_parts : 0;
                        pf.units[j].ticket = n > 1 ? (int32_t)pf.cuts.size() : 0;
                    }
                    if (n > 1) {
                        pf.n_parts += n;
                        pf.cuts.push_back((int32_t)u0);
                    }
                }
            i0 = i1;
        }
        while ((int64_t)pf.first.size() <= n_cta) pf.first.push_back((int32_t)pf.units.size());
    }
}

PagedPlanCaps paged_plan_caps(const PlanShape& s, int32_t max_tok, int32_t max_seq) {
    // Every (tile, head) is one unit, plus one for each cut, and a CTA's share ends in one cut at most. So a
    // CTA has at most two partial units (its first and its last), and fewer tiles than CTAs are cut.
    PagedPlanCaps c{};
    const int64_t rows = (int64_t)max_tok * s.G;
    const int64_t t1 = rows / 8 + std::min<int64_t>(max_seq, max_tok);
    const int64_t t2 = s.tc ? rows / kUnitRows2 + std::min<int64_t>(max_seq, rows / kTcRows) : 0;
    c.ctas1 = ctas(s, 0);
    c.ctas2 = s.tc ? ctas(s, 1) : 0;
    c.units1 = t1 * s.Hkv + c.ctas1;
    c.units2 = t2 * s.Hkv + c.ctas2;
    c.tickets = c.ctas1;
    c.parts1 = 2 * c.ctas1;
    c.parts2 = 2 * c.ctas2;
    c.tiles1 = t1;
    c.tiles2 = t2;
    return c;
}

int32_t plan_numbers(const PlanShape& s, int32_t max_new, PlanDeviceArgs& a) {
    const int64_t rows = (int64_t)max_new * s.G;
    a.G = s.G; a.Hkv = s.Hkv; a.window = s.window; a.n_sink = s.n_sink; a.page_size = s.page_size;
    a.rows1 = rows <= 8 ? 8 : 16;
    a.tc = s.tc && rows >= kTcRows;
    a.tc_rows = (int32_t)kTcRows;
    a.align = (int32_t)block_align(s);
    for (int f = 0; f < 2; ++f) {
        a.bk[f] = (int32_t)block_keys(s, f, a.rows1);
        a.cost[f] = (int32_t)kUnitCost[f];
        a.n_cta[f] = (int32_t)ctas(s, f);
    }
    a.max_new = max_new;
    return (a.rows1 == 8 ? ATTN_FORM_ROWS8 : ATTN_FORM_ROWS16) | (a.tc ? ATTN_FORM_TC : 0);
}

}  // namespace llm
