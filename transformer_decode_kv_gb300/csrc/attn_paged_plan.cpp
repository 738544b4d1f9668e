// Host plan of the attention over a paged cache: tiles of (token, query head) rows per sequence, the
// keys each tile may see, and the split of long key ranges into units so that every SM gets a share.
#include "paged.h"

#include <algorithm>

namespace llm {

namespace {

// CTAs of each form that run at once (attn_paged.cu: two per SM; attn_paged_tc.cu: one).
int64_t slots(const PlanShape& s, bool tc) { return (int64_t)s.n_sm * (tc ? 1 : 2); }
// Shortest key range worth a unit of its own: a unit of the 16-row form gives each of its four warps one
// block of 16 keys, one of the 256-row form one step of 128 keys.
constexpr int64_t kMinKeys1 = 64, kMinKeys2 = 128;
// Sequences with at least this many rows per KV head take 256-row tiles.
constexpr int64_t kTcRows = 64;

int64_t up_to(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// The virtual key range of the rows [row0, row0 + n) of a sequence: sink keys, then [lo, hi).
struct Keys { int32_t n_sink, lo, n; };

Keys tile_keys(const PlanShape& s, const PlanSeq& q, int64_t row0, int64_t n) {
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
    const int64_t lo = std::min(hi, first(pmin - s.window + 1));
    k.n_sink = (int32_t)std::min(lo, first(s.n_sink));
    k.lo = (int32_t)lo;
    k.n = (int32_t)(k.n_sink + hi - lo);
    return k;
}

}  // namespace

void build_paged_plan(const PlanShape& s, const std::vector<PlanSeq>& seqs, PagedPlan& plan) {
    plan = PagedPlan();
    struct Tile { int32_t seq, row0, n_row; Keys keys; };
    std::vector<Tile> tiles[2];
    int64_t total[2] = {0, 0};
    for (size_t i = 0; i < seqs.size(); ++i) {
        const int64_t rows = (int64_t)seqs[i].n_new * s.G;
        const int f = s.tc && rows >= kTcRows ? 1 : 0;
        const int64_t step = f ? kUnitRows2 : kUnitRows1;
        for (int64_t r = 0; r < rows; r += step) {
            Tile t{(int32_t)i, (int32_t)r, (int32_t)std::min(step, rows - r), {}};
            t.keys = tile_keys(s, seqs[i], t.row0, t.n_row);
            total[f] += t.keys.n;
            tiles[f].push_back(t);
        }
    }
    for (int f = 0; f < 2; ++f) {
        std::vector<AttnUnit>& units = f ? plan.units2 : plan.units1;
        int32_t& parts = f ? plan.n_parts2 : plan.n_parts1;
        // an even share of all keys per running CTA is the longest unit
        const int64_t min_keys = f ? kMinKeys2 : kMinKeys1;
        const int64_t share = (total[f] * s.Hkv + slots(s, f) - 1) / slots(s, f);
        const int64_t chunk = std::max(min_keys, up_to(share, min_keys));
        for (const Tile& t : tiles[f]) {
            const PlanSeq& q = seqs[t.seq];
            AttnUnit u{};
            u.tok0 = q.tok0;
            u.row0 = t.row0;
            u.n_row = t.n_row;
            u.p0 = q.p0;
            u.table = q.table;
            u.n_sink_keys = t.keys.n_sink;
            u.key_lo = t.keys.lo;
            u.tile = plan.n_tiles++;
            u.n_chunk = (int32_t)std::max<int64_t>(1, (t.keys.n + chunk - 1) / chunk);
            u.part = u.n_chunk > 1 ? parts : 0;
            if (u.n_chunk > 1) parts += u.n_chunk;
            // equal pieces in whole blocks
            const int64_t piece = up_to((t.keys.n + u.n_chunk - 1) / u.n_chunk, f ? 128 : 16);
            for (int32_t i = 0; i < u.n_chunk; ++i) {
                u.chunk = i;
                u.v0 = (int32_t)std::min<int64_t>(t.keys.n, i * piece);
                u.v1 = (int32_t)std::min<int64_t>(t.keys.n, (i + 1) * piece);
                units.push_back(u);
            }
        }
        // longest first, so that the CTAs' last units are short ones
        std::stable_sort(units.begin(), units.end(),
                         [](const AttnUnit& a, const AttnUnit& b) { return a.v1 - a.v0 > b.v1 - b.v0; });
    }
}

PagedPlanCaps paged_plan_caps(const PlanShape& s, int32_t max_tok, int32_t max_seq) {
    // A tile is cut into ceil(n / chunk) units with chunk >= total * Hkv / slots: the cuts of all tiles
    // add at most slots / Hkv units to one per tile, and the units of the tiles that are cut are at most
    // twice that (such a tile is longer than a chunk).
    PagedPlanCaps c{};
    const int64_t rows = (int64_t)max_tok * s.G;
    const int64_t t1 = rows / kUnitRows1 + std::min<int64_t>(max_seq, max_tok);
    const int64_t t2 = s.tc ? rows / kUnitRows2 + std::min<int64_t>(max_seq, rows / kTcRows) : 0;
    const int64_t x1 = slots(s, false) / s.Hkv + 1, x2 = s.tc ? slots(s, true) / s.Hkv + 1 : 0;
    c.units1 = t1 + x1;
    c.units2 = t2 + x2;
    c.tiles = t1 + t2;
    c.parts1 = 2 * x1;
    c.parts2 = 2 * x2;
    return c;
}

}  // namespace llm
