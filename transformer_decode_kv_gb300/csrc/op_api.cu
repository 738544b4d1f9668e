// C entry points of the operators on the caller's device buffers (include/llm.h): argument checks, the
// device the buffers live on, the attention plan's host and device state. Nothing here throws past
// the C boundary.
#include "../../include/llm.h"

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <new>
#include <string>
#include <vector>

#include "paged.h"

using namespace llm;

static_assert(W_F8 == LLM_TYPE_F8_E4M3, "type numbers");

namespace {

thread_local char g_op_error[256] = "";

int refuse(const char* why) {
    std::snprintf(g_op_error, sizeof(g_op_error), "%s", why);
    return -1;
}
int failed(const char* what, cudaError_t e) {
    std::snprintf(g_op_error, sizeof(g_op_error), "%s: %s", what, cudaGetErrorString(e));
    return -3;
}

// Makes a device current for a scope, and the previous one again.
class OnDevice {
public:
    explicit OnDevice(int dev) {
        ok_ = cudaGetDevice(&prev_) == cudaSuccess && (prev_ == dev || cudaSetDevice(dev) == cudaSuccess);
        dev_ = dev;
    }
    ~OnDevice() { if (ok_ && prev_ != dev_) cudaSetDevice(prev_); }
    bool ok() const { return ok_; }
private:
    int prev_ = -1, dev_ = -1;
    bool ok_ = false;
};

// The device p lives on: 0 and *dev, -1 for memory that is not device memory, -3 for a CUDA failure.
// dev >= 0 on entry: it has to be that one.
int device_of(const void* p, const char* name, int* dev) {
    cudaPointerAttributes at{};
    const cudaError_t e = cudaPointerGetAttributes(&at, p);
    if (e != cudaSuccess) { cudaGetLastError(); return failed("cudaPointerGetAttributes", e); }
    if (at.type != cudaMemoryTypeDevice && at.type != cudaMemoryTypeManaged) {
        std::snprintf(g_op_error, sizeof(g_op_error), "%s is not device memory", name);
        return -1;
    }
    if (*dev >= 0 && at.device != *dev) {
        std::snprintf(g_op_error, sizeof(g_op_error), "%s is on another device", name);
        return -1;
    }
    *dev = at.device;
    return 0;
}

int32_t esize(int32_t t) { return t == LLM_TYPE_F32 ? 4 : t == LLM_TYPE_F8_E4M3 ? 1 : 2; }
bool act_type(int32_t t) { return t == LLM_TYPE_F32 || t == LLM_TYPE_F16 || t == LLM_TYPE_BF16; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Strides (elements) of dimensions with extents n: not negative, multiples of `mult` where the extent is
// above 1, and no two rows of `row` elements may overlap.
bool strides_ok(const int64_t* stride, const int64_t* n, int dims, int64_t row, int64_t mult, bool distinct) {
    int order[3] = {0, 1, 2};
    for (int i = 0; i < dims; ++i) {
        if (n[i] <= 1) continue;
        if (stride[i] < 0 || stride[i] % mult != 0 || stride[i] > ((int64_t)1 << 44) / n[i]) return false;
    }
    if (!distinct) return true;
    std::sort(order, order + dims, [&](int a, int b) { return stride[a] < stride[b]; });
    int64_t extent = row;
    for (int i = 0; i < dims; ++i) {
        const int d = order[i];
        if (n[d] <= 1) continue;
        if (stride[d] < extent) return false;
        extent += stride[d] * (n[d] - 1);
    }
    return true;
}

const char* kv_shape_fault(const llm_kv_pages* kv) {
    if (!kv) return "NULL cache";
    if (kv->type != LLM_TYPE_F16 && kv->type != LLM_TYPE_BF16 && kv->type != LLM_TYPE_F8_E4M3)
        return "a paged cache is F16, BF16 or F8_E4M3";
    if (kv->head_dim != 32 && kv->head_dim != 64 && kv->head_dim != 128) return "head_dim must be 32, 64 or 128";
    if (kv->n_head_kv < 1 || kv->n_head_kv > 1024) return "n_head_kv out of range";
    if (kv->page_size < 1 || kv->n_pages < 1) return "page_size and n_pages must be positive";
    if ((int64_t)kv->page_size * kv->n_pages > INT32_MAX) return "more than 2^31 - 1 cells";
    return nullptr;
}

const char* kv_fault(const llm_kv_pages* kv) {
    if (const char* w = kv_shape_fault(kv)) return w;
    if (!kv->k || !kv->v) return "NULL cache";
    if (!aligned16(kv->k) || !aligned16(kv->v)) return "cache rows must start on 16-byte boundaries";
    const int64_t n[3] = {kv->n_pages, kv->page_size, kv->n_head_kv};
    const int64_t s[3] = {kv->stride_page, kv->stride_cell, kv->stride_head};
    if (!strides_ok(s, n, 3, kv->head_dim, 16 / esize(kv->type), true))
        return "cache strides must keep rows on 16-byte boundaries and apart";
    if (kv->type == LLM_TYPE_F8_E4M3) {
        if (!kv->k_scale || !kv->v_scale) return "an F8_E4M3 cache needs its scales";
        if ((reinterpret_cast<uintptr_t>(kv->k_scale) | reinterpret_cast<uintptr_t>(kv->v_scale)) & 3)
            return "scales must be 4-byte aligned";
        const int64_t ss[3] = {kv->sstride_page, kv->sstride_cell, kv->sstride_head};
        if (!strides_ok(ss, n, 3, 1, 1, true)) return "scale strides must keep the scales apart";
    }
    return nullptr;
}

// strides of a dimension of extent 1 are never used: zero, so that no unchecked number is multiplied
PagedKv paged_kv(const llm_kv_pages* kv) {
    PagedKv p;
    const int64_t es = esize(kv->type);
    p.type = kv->type; p.Hkv = kv->n_head_kv; p.hd = kv->head_dim;
    p.page_size = kv->page_size; p.n_pages = kv->n_pages;
    p.k = static_cast<uint8_t*>(kv->k); p.v = static_cast<uint8_t*>(kv->v);
    p.sb_page = kv->n_pages > 1 ? kv->stride_page * es : 0;
    p.sb_cell = kv->page_size > 1 ? kv->stride_cell * es : 0;
    p.sb_head = kv->n_head_kv > 1 ? kv->stride_head * es : 0;
    if (kv->type == LLM_TYPE_F8_E4M3) {
        p.ks = kv->k_scale; p.vs = kv->v_scale;
        p.ss_page = kv->n_pages > 1 ? kv->sstride_page : 0;
        p.ss_cell = kv->page_size > 1 ? kv->sstride_cell : 0;
        p.ss_head = kv->n_head_kv > 1 ? kv->sstride_head : 0;
    }
    return p;
}

int kv_devices(const llm_kv_pages* kv, int* dev) {
    int r = device_of(kv->k, "k", dev);
    if (!r) r = device_of(kv->v, "v", dev);
    if (!r && kv->type == LLM_TYPE_F8_E4M3) r = device_of(kv->k_scale, "k_scale", dev);
    if (!r && kv->type == LLM_TYPE_F8_E4M3) r = device_of(kv->v_scale, "v_scale", dev);
    return r;
}

const char* attn_shape_fault(const llm_attn_shape* s, const llm_kv_pages* kv) {
    if (!s) return "NULL shape";
    if (const char* w = kv_shape_fault(kv)) return w;
    if (!act_type(s->type) || !attn_paged_types_ok(s->type, kv->type))
        return "F16 caches take F16 or F32 activations, BF16 caches BF16, F8_E4M3 caches all three";
    if (s->n_head < 1 || s->n_head > 1024 || s->n_head % kv->n_head_kv != 0)
        return "n_head must be a multiple of n_head_kv, at most 1024";
    if (!std::isfinite(s->scale)) return "scale must be finite";
    if (s->window < 0 || s->n_sink < 0) return "window and n_sink must not be negative";
    if (s->max_tok < 1 || s->max_seq < 1 || s->max_table < 1 || s->max_tok > (1 << 24) || s->max_seq > (1 << 20) ||
        s->max_table > (1 << 28))
        return "max_tok, max_seq or max_table out of range";
    // rows (token, query head) and the units made of them are counted in 32 bits
    if ((int64_t)s->max_tok * s->n_head > INT32_MAX) return "max_tok times n_head must be below 2^31";
    return nullptr;
}

PlanShape plan_shape(const llm_attn_shape* s, const llm_kv_pages* kv, int32_t n_sm, bool tc) {
    PlanShape p;
    p.G = s->n_head / kv->n_head_kv;
    p.Hkv = kv->n_head_kv;
    p.window = s->window;
    p.n_sink = s->n_sink;
    p.n_sm = n_sm;
    p.hd = kv->head_dim;
    p.kv_type = kv->type;
    p.page_size = kv->page_size;
    p.tc = tc;
    return p;
}

constexpr int32_t kMaxKeys = INT32_MAX - 512;    // of a sequence
int64_t pages_of(const llm_kv_pages& kv, int32_t n_kv) { return ((int64_t)n_kv + kv.page_size - 1) / kv.page_size; }

// Why a step's lengths do not fit the shape (null: they do).
const char* step_fault(const llm_attn_shape* s, const llm_kv_pages& kv, int32_t n_seq, const int32_t* n_new,
                       const int32_t* n_kv) {
    if (n_seq < 0 || n_seq > s->max_seq) return "more sequences than the plan's max_seq";
    if (n_seq > 0 && (!n_new || !n_kv)) return "NULL lengths";
    int64_t tok = 0, tab = 0;
    for (int32_t i = 0; i < n_seq; ++i) {
        // (the kernels number keys in 32 bits, up to a few blocks past the last one)
        if (n_new[i] < 0 || n_kv[i] < 0 || n_kv[i] > kMaxKeys) return "a length out of range";
        tok += n_new[i];
        tab += pages_of(kv, n_kv[i]);
    }
    if (tok > s->max_tok) return "more tokens than the plan's max_tok";
    if (tab > s->max_table) return "more pages than the plan's max_table";
    return nullptr;
}

std::vector<PlanSeq> plan_seqs(const llm_kv_pages& kv, int32_t n_seq, const int32_t* n_new, const int32_t* n_kv) {
    std::vector<PlanSeq> seqs((size_t)n_seq);
    int32_t t0 = 0, b0 = 0;
    for (int32_t i = 0; i < n_seq; ++i) {
        PlanSeq& q = seqs[i];
        q.tok0 = t0; q.n_new = n_new[i]; q.p0 = n_kv[i] - n_new[i]; q.table = b0; q.n_keys = n_kv[i];
        t0 += n_new[i];
        b0 += (int32_t)pages_of(kv, n_kv[i]);
    }
    return seqs;
}

int kv_rows(const llm_kv_pages* kv, int32_t type, void* k, void* v, int64_t s_tok, int64_t s_head,
            const int32_t* cell, int32_t n, uint32_t* err, void* stream, bool store) {
    if (const char* w = kv_fault(kv)) return refuse(w);
    if (!act_type(type)) return refuse("rows are F32, F16 or BF16");
    if (n < 0) return refuse("n < 0");
    if (n == 0) return 0;
    if (!k || !v || !cell) return refuse("NULL rows or cells");
    if (!aligned16(k) || !aligned16(v)) return refuse("rows must start on 16-byte boundaries");
    if (reinterpret_cast<uintptr_t>(cell) & 3) return refuse("cells must be 4-byte aligned");
    const int64_t ext[2] = {n, kv->n_head_kv}, str[2] = {s_tok, s_head};
    if (!strides_ok(str, ext, 2, kv->head_dim, 16 / esize(type), !store))
        return refuse("row strides must be multiples of 16 bytes, not negative, and keep outputs apart");
    if ((int64_t)n * kv->n_head_kv * kv->head_dim / 4 > ((int64_t)1 << 38)) return refuse("too many rows");
    int dev = -1;
    int r = kv_devices(kv, &dev);
    if (!r) r = device_of(k, "rows of k", &dev);
    if (!r) r = device_of(v, "rows of v", &dev);
    if (!r) r = device_of(cell, "cell", &dev);
    if (!r && err) r = device_of(err, "err", &dev);
    if (r) return r;
    OnDevice on(dev);
    if (!on.ok()) return failed("cudaSetDevice", cudaGetLastError());
    KvRowsArgs a;
    a.kv = paged_kv(kv);
    a.type = type; a.k = k; a.v = v;
    a.s_tok = n > 1 ? s_tok : 0; a.s_head = kv->n_head_kv > 1 ? s_head : 0;
    a.cell = cell; a.n = n; a.err = err;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (store ? !launch_kv_rows_store(a, st) : !launch_kv_rows_load(a, st))
        return failed(store ? "kv_store launch" : "kv_load launch", cudaGetLastError());
    return 0;
}

}  // namespace

struct llm_attn_plan {
    llm_attn_shape shape{};
    llm_kv_pages kv{};                           // type, head count, head_dim, page size, page count
    PlanShape ps;
    PagedPlanCaps caps{};
    int device = 0;
    float scale_log2 = 0.f;
    PagedPlan plan;
    // device buffer: header, both forms' CTA starts, their units, page table; the pinned copy it is uploaded from
    size_t off_first[2] = {0, 0}, off_cuts = 0, off_units[2] = {0, 0}, off_table = 0, bytes = 0;
    uint8_t *d_buf = nullptr, *h_buf = nullptr;
    float* part_o = nullptr;
    float2* part_ml = nullptr;
    int32_t *tickets = nullptr, *redo = nullptr;
    uint32_t* err = nullptr;
    cudaEvent_t uploaded = nullptr;
    bool pending = false;
};

extern "C" {

const char* llm_op_last_error(void) { return g_op_error; }

int llm_kv_store(const llm_kv_pages* kv, int32_t type, const void* k, const void* v, int64_t stride_tok,
                 int64_t stride_head, const int32_t* cell, int32_t n, uint32_t* err, void* stream) {
    return kv_rows(kv, type, const_cast<void*>(k), const_cast<void*>(v), stride_tok, stride_head, cell, n, err,
                   stream, true);
}

int llm_kv_load(const llm_kv_pages* kv, int32_t type, void* k, void* v, int64_t stride_tok, int64_t stride_head,
                const int32_t* cell, int32_t n, uint32_t* err, void* stream) {
    return kv_rows(kv, type, k, v, stride_tok, stride_head, cell, n, err, stream, false);
}

llm_attn_plan* llm_attn_plan_init(const llm_attn_shape* s, const llm_kv_pages* kv) {
    auto no = [](const char* w) -> llm_attn_plan* { refuse(w); return nullptr; };
    if (const char* w = attn_shape_fault(s, kv)) return no(w);
    llm_attn_plan* p = new (std::nothrow) llm_attn_plan();
    if (!p) return no("out of memory");
    auto die = [&](const char* what, cudaError_t e) -> llm_attn_plan* {
        failed(what, e);
        cudaGetLastError();
        llm_attn_plan_free(p);
        return nullptr;
    };
    p->shape = *s;
    p->kv = *kv;
    p->scale_log2 = (float)((s->scale == 0.f ? 1.0 / std::sqrt((double)kv->head_dim) : (double)s->scale) *
                            1.4426950408889634);
    int n_sm = 0;
    cudaError_t e = cudaGetDevice(&p->device);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, p->device);
    if (e != cudaSuccess) return die("device", e);
    p->ps = plan_shape(s, kv, n_sm, attn_paged_tc_ok(kv->head_dim, kv->type, s->type));
    p->caps = paged_plan_caps(p->ps, s->max_tok, s->max_seq);
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    p->off_first[0] = up(PH_WORDS * sizeof(int32_t));
    p->off_first[1] = p->off_first[0] + up((p->caps.ctas1 + 1) * sizeof(int32_t));
    p->off_cuts = p->off_first[1] + up((p->caps.ctas2 + 1) * sizeof(int32_t));
    p->off_units[0] = p->off_cuts + up(p->caps.ctas2 * sizeof(int32_t));
    p->off_units[1] = p->off_units[0] + up(p->caps.units1 * sizeof(AttnUnit));
    p->off_table = p->off_units[1] + up(p->caps.units2 * sizeof(AttnUnit));
    p->bytes = p->off_table + up((size_t)s->max_table * sizeof(int32_t));
    const int64_t rows = plan_part_rows(p->caps, true);
    auto get = [&](auto** q, size_t n) {
        void* v = nullptr;
        if (e == cudaSuccess) e = cudaMalloc(&v, n);
        *q = static_cast<std::remove_reference_t<decltype(**q)>*>(v);
    };
    get(&p->d_buf, p->bytes);
    get(&p->part_o, (size_t)rows * kv->head_dim * sizeof(float));
    get(&p->part_ml, (size_t)rows * sizeof(float2));
    get(&p->tickets, (size_t)p->caps.tickets * sizeof(int32_t));
    get(&p->redo, (size_t)std::max<int64_t>(1, p->caps.units2) * sizeof(int32_t));
    get(&p->err, sizeof(uint32_t));
    if (e == cudaSuccess) {
        void* h = nullptr;
        e = cudaMallocHost(&h, p->bytes);
        p->h_buf = static_cast<uint8_t*>(h);
    }
    if (e == cudaSuccess) e = cudaMemset(p->tickets, 0, (size_t)p->caps.tickets * sizeof(int32_t));
    if (e == cudaSuccess) e = cudaMemset(p->err, 0, sizeof(uint32_t));
    if (e == cudaSuccess) e = cudaMemset(p->d_buf, 0, p->off_units[0]);
    if (e == cudaSuccess) e = cudaEventCreateWithFlags(&p->uploaded, cudaEventDisableTiming);
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return die("llm_attn_plan_init", e);
    return p;
}

void llm_attn_plan_free(llm_attn_plan* p) {
    if (!p) return;
    {
        OnDevice on(p->device);
        if (p->uploaded) {
            cudaEventSynchronize(p->uploaded);
            cudaEventDestroy(p->uploaded);
        }
        cudaFree(p->d_buf);                      // cudaFree waits for the device
        cudaFree(p->part_o);
        cudaFree(p->part_ml);
        cudaFree(p->tickets);
        cudaFree(p->redo);
        cudaFree(p->err);
        if (p->h_buf) cudaFreeHost(p->h_buf);
        cudaGetLastError();
    }
    delete p;
}

int llm_attn_plan_set(llm_attn_plan* p, int32_t n_seq, const int32_t* n_new, const int32_t* n_kv,
                      const int32_t* pages, int32_t ld_pages, void* stream) {
    if (!p) return refuse("NULL plan");
    if (const char* w = step_fault(&p->shape, p->kv, n_seq, n_new, n_kv)) return refuse(w);
    int64_t tab = 0;
    for (int32_t i = 0; i < n_seq; ++i) {
        const int64_t need = pages_of(p->kv, n_kv[i]);
        if (need > 0 && (!pages || need > ld_pages)) return refuse("a page-table row is shorter than its sequence");
        for (int64_t j = 0; j < need; ++j) {
            const int32_t pg = pages[(int64_t)i * ld_pages + j];
            if (pg < 0 || pg >= p->kv.n_pages) return refuse("a page outside the cache");
        }
        tab += need;
    }
    OnDevice on(p->device);
    if (!on.ok()) return failed("cudaSetDevice", cudaGetLastError());
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
    cudaError_t e = cudaStreamIsCapturing(st, &cs);
    if (e != cudaSuccess) { cudaGetLastError(); return failed("stream", e); }
    if (cs != cudaStreamCaptureStatusNone) return refuse("a plan cannot be set in a captured stream");
    PagedPlan plan;
    try {
        build_paged_plan(p->ps, plan_seqs(p->kv, n_seq, n_new, n_kv), plan);
    } catch (const std::exception&) {
        return refuse("out of memory");
    }
    const int64_t max_units[2] = {p->caps.units1, p->caps.units2}, max_cta[2] = {p->caps.ctas1, p->caps.ctas2},
                  max_parts[2] = {p->caps.parts1, p->caps.parts2};
    for (int f = 0; f < 2; ++f)
        if ((int64_t)plan.form_[f].units.size() > max_units[f] || (int64_t)plan.form_[f].first.size() > max_cta[f] + 1 ||
            plan.form_[f].n_parts > max_parts[f] || (int64_t)plan.form_[f].cuts.size() > max_cta[f])
            return refuse("plan exceeds its buffers");
    // the previous upload has read the pinned buffer
    if (p->pending && (e = cudaEventSynchronize(p->uploaded)) != cudaSuccess) return failed("upload", e);
    p->pending = false;
    int32_t* hdr = reinterpret_cast<int32_t*>(p->h_buf);
    std::memset(hdr, 0, PH_WORDS * sizeof(int32_t));
    hdr[PH_FORM] = plan.form();
    for (int f = 0; f < 2; ++f) {
        const PlanForm& pf = plan.form_[f];
        if (pf.units.empty()) continue;
        std::memcpy(p->h_buf + p->off_first[f], pf.first.data(), pf.first.size() * sizeof(int32_t));
        std::memcpy(p->h_buf + p->off_units[f], pf.units.data(), pf.units.size() * sizeof(AttnUnit));
    }
    const std::vector<int32_t>& cuts = plan.form_[1].cuts;
    hdr[PH_CUTS2] = (int32_t)cuts.size();
    if (!cuts.empty()) std::memcpy(p->h_buf + p->off_cuts, cuts.data(), cuts.size() * sizeof(int32_t));
    int32_t* table = reinterpret_cast<int32_t*>(p->h_buf + p->off_table);
    for (int32_t i = 0; i < n_seq; ++i) {
        const int64_t need = pages_of(p->kv, n_kv[i]);
        if (need) std::memcpy(table, pages + (int64_t)i * ld_pages, (size_t)need * sizeof(int32_t));
        table += need;
    }
    auto copy = [&](size_t off, size_t n) {
        if (e == cudaSuccess && n)
            e = cudaMemcpyAsync(p->d_buf + off, p->h_buf + off, n, cudaMemcpyHostToDevice, st);
    };
    copy(0, p->off_units[0] + plan.form_[0].units.size() * sizeof(AttnUnit));
    copy(p->off_units[1], plan.form_[1].units.size() * sizeof(AttnUnit));
    copy(p->off_table, (size_t)tab * sizeof(int32_t));
    if (e == cudaSuccess) e = cudaEventRecord(p->uploaded, st);
    if (e != cudaSuccess) { cudaGetLastError(); return failed("plan upload", e); }
    p->pending = true;
    p->plan = std::move(plan);
    return 0;
}

int llm_attn_run(llm_attn_plan* p, const void* q, int64_t q_stride_tok, int64_t q_stride_head, const llm_kv_pages* kv,
                 void* out, int64_t o_stride_tok, int64_t o_stride_head, void* stream) {
    if (!p) return refuse("NULL plan");
    if (const char* w = kv_fault(kv)) return refuse(w);
    if (kv->type != p->kv.type || kv->n_head_kv != p->kv.n_head_kv || kv->head_dim != p->kv.head_dim ||
        kv->page_size != p->kv.page_size || kv->n_pages != p->kv.n_pages)
        return refuse("the cache is not of the plan's type and shape");
    if (p->plan.form() == 0) {
        // (a graph without the kernels would replay later steps as nothing, and nobody would learn of it)
        cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
        OnDevice on(p->device);
        if (cudaStreamIsCapturing(static_cast<cudaStream_t>(stream), &cs) != cudaSuccess) cudaGetLastError();
        return cs == cudaStreamCaptureStatusNone ? 0 : refuse("an empty step cannot be captured");
    }
    if (!q || !out) return refuse("NULL q or out");
    if (!aligned16(q) || !aligned16(out)) return refuse("rows must start on 16-byte boundaries");
    // checked for max_tok rows: a captured run replays with whatever the plan is set to then
    const int64_t ext[2] = {p->shape.max_tok, p->shape.n_head};
    const int64_t sq[2] = {q_stride_tok, q_stride_head}, so[2] = {o_stride_tok, o_stride_head};
    const int64_t mult = 16 / esize(p->shape.type);
    if (!strides_ok(sq, ext, 2, kv->head_dim, mult, false) || !strides_ok(so, ext, 2, kv->head_dim, mult, true))
        return refuse("row strides must be multiples of 16 bytes, not negative, and keep outputs apart");
    int dev = p->device;
    int r = kv_devices(kv, &dev);
    if (!r) r = device_of(q, "q", &dev);
    if (!r) r = device_of(out, "out", &dev);
    if (r) return r;
    OnDevice on(dev);
    if (!on.ok()) return failed("cudaSetDevice", cudaGetLastError());
    AttnPagedArgs a;
    a.kv = paged_kv(kv);
    a.q_type = p->shape.type;
    a.G = p->ps.G;
    a.q = q; a.q_tok = p->shape.max_tok > 1 ? q_stride_tok : 0; a.q_head = p->shape.n_head > 1 ? q_stride_head : 0;
    a.out = out; a.o_tok = p->shape.max_tok > 1 ? o_stride_tok : 0; a.o_head = p->shape.n_head > 1 ? o_stride_head : 0;
    a.out_kind = p->shape.type == LLM_TYPE_F32 ? AO_F32 : p->shape.type == LLM_TYPE_F16 ? AO_F16 : AO_BF16;
    const int64_t oes = esize(p->shape.type);
    a.out32 = (reinterpret_cast<uintptr_t>(out) & 31) == 0 && a.o_tok * oes % 32 == 0 && a.o_head * oes % 32 == 0;
    a.scale_log2 = p->scale_log2;
    a.window = p->shape.window;
    a.n_sink = p->shape.n_sink;
    a.hdr = reinterpret_cast<const int32_t*>(p->d_buf);
    a.first1 = reinterpret_cast<const int32_t*>(p->d_buf + p->off_first[0]);
    a.first2 = reinterpret_cast<const int32_t*>(p->d_buf + p->off_first[1]);
    a.cuts2 = reinterpret_cast<const int32_t*>(p->d_buf + p->off_cuts);
    a.units1 = reinterpret_cast<const AttnUnit*>(p->d_buf + p->off_units[0]);
    a.units2 = reinterpret_cast<const AttnUnit*>(p->d_buf + p->off_units[1]);
    a.table = reinterpret_cast<const int32_t*>(p->d_buf + p->off_table);
    a.part_o = p->part_o; a.part_ml = p->part_ml;
    a.part_o2 = p->part_o + plan_part_rows(p->caps, false) * kv->head_dim;
    a.part_ml2 = p->part_ml + plan_part_rows(p->caps, false);
    a.tickets = p->tickets; a.redo2 = p->redo; a.err = p->err;
    a.form = p->plan.form();
    a.n_sm = p->ps.n_sm;
    if (!launch_attn_paged(a, static_cast<cudaStream_t>(stream))) return failed("attention launch", cudaGetLastError());
    return 0;
}

int llm_attn_plan_form(const llm_attn_plan* p) { return p ? p->plan.form() : refuse("NULL plan"); }

uint32_t llm_attn_plan_error(llm_attn_plan* p) {
    if (!p) return 0;
    OnDevice on(p->device);
    uint32_t e = 0;
    if (cudaDeviceSynchronize() != cudaSuccess || cudaMemcpy(&e, p->err, sizeof(e), cudaMemcpyDeviceToHost) != cudaSuccess) {
        failed("llm_attn_plan_error", cudaGetLastError());
        return ~0u;
    }
    // (a memset returns before it is done: a run on a stream of its own could set a bit in between, to be lost)
    if (e && (cudaMemset(p->err, 0, sizeof(e)) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess)) {
        failed("llm_attn_plan_error", cudaGetLastError());
        return ~0u;
    }
    return e;
}

int64_t llm_debug_attn_units(const llm_attn_shape* s, const llm_kv_pages* kv, int32_t n_sm, int32_t tc, int32_t n_seq,
                             const int32_t* n_new, const int32_t* n_kv, int32_t* out, int64_t cap,
                             int64_t* n_rows_units, int32_t* first, int64_t caps[7]) {
    if (const char* w = attn_shape_fault(s, kv)) return refuse(w);
    if (n_sm < 1) return refuse("n_sm < 1");
    if (const char* w = step_fault(s, *kv, n_seq, n_new, n_kv)) return refuse(w);
    PagedPlan plan;
    const PlanShape ps = plan_shape(s, kv, n_sm, tc != 0);
    try {
        build_paged_plan(ps, plan_seqs(*kv, n_seq, n_new, n_kv), plan);
    } catch (const std::exception&) {
        return refuse("out of memory");
    }
    const std::vector<AttnUnit>&u1 = plan.form_[0].units, &u2 = plan.form_[1].units;
    const int64_t n1 = (int64_t)u1.size(), n2 = (int64_t)u2.size();
    for (int64_t i = 0; out && i < n1 + n2 && i < cap; ++i)
        std::memcpy(out + 16 * i, i < n1 ? &u1[i] : &u2[i - n1], sizeof(AttnUnit));
    if (first) {
        std::memset(first, 0, sizeof(int32_t) * 2 * (2 * (size_t)n_sm + 1));
        for (int f = 0; f < 2; ++f)
            std::copy(plan.form_[f].first.begin(), plan.form_[f].first.end(), first + f * (2 * n_sm + 1));
    }
    if (n_rows_units) *n_rows_units = n1;
    if (caps) {
        const PagedPlanCaps c = paged_plan_caps(ps, s->max_tok, s->max_seq);
        caps[0] = c.units1; caps[1] = c.units2; caps[2] = c.ctas1; caps[3] = c.ctas2;
        caps[4] = c.tickets; caps[5] = c.parts1; caps[6] = c.parts2;
    }
    return n1 + n2;
}

int llm_sample_rows(const llm_sample_rows_args* s, void* stream) {
    if (!s) return refuse("NULL arguments");
    if (!act_type(s->type)) return refuse("logits are F32, F16 or BF16");
    if (s->n_rows < 0 || s->n_rows > (1 << 24)) return refuse("n_rows out of range");
    if (s->n_vocab < 1 || s->n_vocab > sample_rows_max_vocab()) return refuse("n_vocab out of range");
    if (s->n_rows == 0) return 0;
    if (!s->logits || !s->token) return refuse("NULL logits or token");
    if (s->ld < 0 || (s->n_rows > 1 && s->ld > ((int64_t)1 << 40))) return refuse("ld out of range");
    if (s->temperature && !s->u) return refuse("sampling at a temperature needs u");
    if (s->repeat_penalty && (!s->penalty_start || (!s->penalty_token && s->n_penalty_token > 0) || s->n_penalty_token < 0))
        return refuse("repeat_penalty needs its token lists");
    if (reinterpret_cast<uintptr_t>(s->logits) % esize(s->type)) return refuse("logits are not aligned to their type");
    int dev = -1;
    int r = device_of(s->logits, "logits", &dev);
    if (!r) r = device_of(s->token, "token", &dev);
    const void* opt[] = {s->top_k, s->top_p, s->min_p, s->temperature, s->u, s->repeat_penalty,
                         s->repeat_penalty ? s->penalty_start : nullptr,
                         s->repeat_penalty ? s->penalty_token : nullptr};
    for (const void* q : opt)
        if (!r && q) r = device_of(q, "a parameter array", &dev);
    if (r) return r;
    OnDevice on(dev);
    if (!on.ok()) return failed("cudaSetDevice", cudaGetLastError());
    SampleRowsArgs a;
    a.type = s->type; a.n_rows = s->n_rows; a.V = s->n_vocab;
    a.logits = s->logits; a.ld = s->n_rows > 1 ? s->ld : 0;
    a.top_k = s->top_k; a.top_p = s->top_p; a.min_p = s->min_p; a.temperature = s->temperature; a.u = s->u;
    a.penalty = s->repeat_penalty;
    a.pen_start = s->penalty_start; a.pen_tok = s->penalty_token; a.n_pen = s->n_penalty_token;
    a.token = s->token;
    if (!launch_sample_rows(a, static_cast<cudaStream_t>(stream))) return failed("sampler launch", cudaGetLastError());
    return 0;
}

}  // extern "C"
