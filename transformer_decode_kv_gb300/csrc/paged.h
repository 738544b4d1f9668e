// Operators over a paged KV cache (kv_paged.cu, attn_paged.cu) and the batched sampler
// (sample_rows.cu): launch arguments shared by the C entry points (op_api.cu) and the decode loop.
#pragma once

#include <atomic>
#include <cstdint>
#include <string>
#include <vector>

#include <cuda_runtime.h>

#include "kernels.h"

namespace llm {

constexpr int32_t W_F8 = 100;                    // LLM_TYPE_F8_E4M3
enum : uint32_t { ERR_PLAN_FORM = 16u };         // beside the bits of kernels.h

// Allow a kernel its dynamic shared memory, once per device (`done`: a bit per device; the call costs about as much
// as a launch).
inline bool allow_smem(const void* kernel, size_t bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
    if (bit && (done.load(std::memory_order_acquire) & bit)) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess) return false;
    done.fetch_or(bit, std::memory_order_release);
    return true;
}

// A paged cache as the kernels see it; strides in bytes (scales: elements).
struct PagedKv {
    int32_t type = W_F16, Hkv = 0, hd = 0, page_size = 1, n_pages = 0;
    uint8_t *k = nullptr, *v = nullptr;
    int64_t sb_page = 0, sb_cell = 0, sb_head = 0;
    float *ks = nullptr, *vs = nullptr;
    int64_t ss_page = 0, ss_cell = 0, ss_head = 0;
};

// Rows between dense token-major buffers and cache cells (kv_paged.cu); strides in elements.
struct KvRowsArgs {
    PagedKv kv;
    int32_t type = W_F32;                        // of the dense rows
    void *k = nullptr, *v = nullptr;
    int64_t s_tok = 0, s_head = 0;
    const int32_t* cell = nullptr;
    int32_t n = 0;
    uint32_t* err = nullptr;
};
bool launch_kv_rows_store(const KvRowsArgs& a, cudaStream_t st);
bool launch_kv_rows_load(const KvRowsArgs& a, cudaStream_t st);

// One unit of attention work: rows of one tile of a sequence for one KV head against a range of the keys
// those rows may see. A tile's rows are (token, query head) pairs of the KV head's group, row
// token * G + head. Its keys are numbered by a virtual index: sink keys 0 .. n_sink_keys - 1, then the
// keys from key_lo on (the sequence's keys between the sinks and the tile's windows are left out).
struct AttnUnit {
    int32_t tok0, row0, n_row, p0;               // first token of the sequence; the tile's rows; position of tok0
    int32_t table, n_sink_keys, key_lo, v0;      // page-table offset; the virtual key range [v0, v1)
    int32_t v1, n_chunk, chunk, part;            // units of this tile; this one; the first's partial slot
    int32_t ticket, head, pad[2];                // counter of the tile's finished units (small tiles); KV head
};
static_assert(sizeof(AttnUnit) == 64, "read as four int4");

// Forms of the kernels: 8- and 16-row tiles on mma.sync, 256-row tiles on tcgen05.
enum : int32_t { ATTN_FORM_ROWS8 = 1, ATTN_FORM_ROWS16 = 2, ATTN_FORM_TC = 4 };
constexpr int kUnitRows2 = 256;
// The small-tile forms run two CTAs per SM. A warp keeps 32 keys in use and 32 under way, so a 16-bit cache with
// head_dim 128 (33 KB a warp) leaves room for three warps per CTA; the others take six, or four where the
// 16-row form needs the registers.
constexpr int kAttnRowsCtas = 2;
constexpr int attn_rows_warps(int hd, int kv_type, int rows) {
    return hd == 128 && kv_type != W_F8 ? 3 : rows == 8 ? 6 : 4;
}
enum AttnOut : int32_t { AO_F16 = 0, AO_BF16 = 1, AO_F32 = 2, AO_BF16_PAIR = 3 };

// Header words of a plan's device buffer.
enum : int32_t { PH_FORM = 0, PH_CUTS2 = 1, PH_WORDS = 8 };

struct AttnPagedArgs {
    PagedKv kv;
    int32_t q_type = W_F16, G = 1;
    const void* q = nullptr;
    int64_t q_tok = 0, q_head = 0;               // elements
    void* out = nullptr;
    void* out_lo = nullptr;                      // AO_BF16_PAIR: the low terms
    int32_t out_kind = AO_F16;
    int64_t o_tok = 0, o_head = 0;
    bool out32 = false;                          // the rows of out start on 32-byte boundaries
    float scale_log2 = 0.f;                      // scale * log2(e)
    int32_t window = 0, n_sink = 0;
    const int32_t* hdr = nullptr;
    // units of the small-tile and the 256-row form, and where each CTA's begin [CTAs + 1]
    const AttnUnit *units1 = nullptr, *units2 = nullptr;
    const int32_t *first1 = nullptr, *first2 = nullptr;
    const int32_t* cuts2 = nullptr;              // first unit of each cut 256-row tile
    const int32_t* table = nullptr;
    const int32_t* perm = nullptr;               // token order (null: identity)
    const int32_t* tok_pos = nullptr;            // positions of tokens (null: p0 + token)
    const int32_t* key_pos = nullptr;            // positions of the page-table's keys, pages of one cell
    float* part_o = nullptr;                     // [part][rows][hd] unnormalised
    float2* part_ml = nullptr;                   // [part][rows] (running max, sum)
    float* part_o2 = nullptr;                    // the same of the 256-row tiles
    float2* part_ml2 = nullptr;
    int32_t* redo2 = nullptr;                    // per 256-row unit: its rows have to be done key by key
    int32_t* tickets = nullptr;                  // zero between launches
    uint32_t* err = nullptr;
    int32_t form = 0;                            // forms the caller launches
    int32_t n_sm = 148;
};
// Both forms' kernels as the plan's form says; false if a launch failed.
bool launch_attn_paged(const AttnPagedArgs& a, cudaStream_t st);
bool attn_paged_types_ok(int32_t q_type, int32_t kv_type);
// 256-row tiles serve this shape (attn_paged_tc.cu).
bool attn_paged_tc_ok(int32_t hd, int32_t kv_type, int32_t q_type, bool round_q = false);
bool launch_attn_paged_tc(const AttnPagedArgs& a, cudaStream_t st);

// ---- host plan (attn_paged_plan.cpp)
struct PlanSeq {
    int32_t tok0, n_new, p0;                     // its tokens; position of the first
    int32_t table, n_keys;                       // its keys (in position order)
    // positions where they are not the indices: of its tokens (through perm) and of its keys
    const int32_t *tok_pos = nullptr, *key_pos = nullptr;
};
struct PlanShape {
    int32_t G = 1, Hkv = 1, window = 0, n_sink = 0, n_sm = 148;
    int32_t hd = 128, kv_type = W_F16, page_size = 1;
    bool tc = false;                             // 256-row tiles allowed
};
struct PlanForm {
    std::vector<AttnUnit> units;
    std::vector<int32_t> first;                  // where each CTA's units begin [CTAs + 1]
    std::vector<int32_t> cuts;                   // the first unit of each tile that is cut
    int32_t n_parts = 0;
};
struct PagedPlan {
    PlanForm form_[2];                           // small tiles, 256-row tiles
    int32_t rows1 = 8;                           // rows of the small tiles
    int32_t form() const {
        return (form_[0].units.empty() ? 0 : rows1 == 8 ? ATTN_FORM_ROWS8 : ATTN_FORM_ROWS16) |
               (form_[1].units.empty() ? 0 : ATTN_FORM_TC);
    }
};
void build_paged_plan(const PlanShape& s, const std::vector<PlanSeq>& seqs, PagedPlan& plan);
// Upper bounds for buffers over every plan of at most max_tok tokens in max_seq sequences.
struct PagedPlanCaps { int64_t units1, units2, ctas1, ctas2, tickets, parts1, parts2; };
PagedPlanCaps paged_plan_caps(const PlanShape& s, int32_t max_tok, int32_t max_seq);
// Partial results of both forms: rows of head_dim values, the small tiles' first.
inline int64_t plan_part_rows(const PagedPlanCaps& c, bool both) { return c.parts1 * 16 + (both ? c.parts2 * kUnitRows2 : 0); }

// ---- the sampler chain per row (sample_rows.cu)
struct SampleRowsArgs {
    int32_t type = W_F32, n_rows = 0, V = 0;
    const void* logits = nullptr;
    int64_t ld = 0;
    const int32_t* row = nullptr;                // logits row of each entry (null: identity)
    const int32_t* top_k = nullptr;
    const float *top_p = nullptr, *min_p = nullptr, *temperature = nullptr, *u = nullptr, *penalty = nullptr;
    const int32_t *pen_start = nullptr, *pen_tok = nullptr;
    int32_t n_pen = 0;                           // entries of pen_tok
    int32_t* token = nullptr;
};
int32_t sample_rows_max_vocab();
bool launch_sample_rows(const SampleRowsArgs& a, cudaStream_t st);

}  // namespace llm
