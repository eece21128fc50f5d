// C entry points of libdt.so (declared and documented in include/dt.h):
// host-side validation, launch planning and the two kernel launches.
// Nothing here allocates, synchronises or keeps state between calls.
#include <math.h>
#include <string.h>

#include <mutex>

#include "common.h"
#include "pass.h"

namespace dt {

static int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
static int64_t round_up(int64_t a, int64_t m) { return ceil_div(a, m) * m; }

SweepPlan plan_sweep(const dt_params* p) {
    SweepPlan s{};
    s.rows = (int64_t)p->B * p->d;
    const int V = p->V;
    int C;
    int lists = kWaves;
    const int64_t by_merge4 = kMergeKeysPerRow / (p->k * kWaves);     // chunks with one list per wave
    const int64_t by_merge1 = kMergeKeysPerRow / p->k;                // chunks with one list per chunk
    if (p->sweep_chunks > 0) {
        C = p->sweep_chunks;
        if (C > by_merge4) lists = 1;
    } else {
        // at least ~two 256-thread workgroups per CU (256 CUs) and chunks of
        // >= 4096 elements; a row merges at most kMergeKeysPerRow keys, so
        // short chunks (small batches) merge their four wave lists in the
        // workgroup first
        const int64_t target = 512;
        int64_t c = s.rows >= target ? 1 : ceil_div(target, s.rows > 0 ? s.rows : 1);
        const int64_t by_len = V / 4096 > 1 ? V / 4096 : 1;
        if (c > by_len) c = by_len;
        if (c > by_merge4) {
            lists = 1;
            if (c > by_merge1) c = by_merge1;
        }
        C = (int)(c < 1 ? 1 : c);
    }
    if (C > V) C = V;
    s.chunk = (int)round_up(ceil_div(V, C), 8);
    s.C = (int)ceil_div(V, s.chunk);
    s.lists = lists;
    return s;
}

int n_contexts(int kind, int d, int k) {
    if (kind == DT_NGRAM_NONE) return 0;
    if (kind == DT_NGRAM_HASH_TRIGRAM) return d == 1 ? 1 : 1 + k + (d - 2) * k * k;
    return 1 + (d - 1) * k;
}

WorkspacePlan plan_workspace(const dt_params* p, const SweepPlan& s) {
    WorkspacePlan w{};
    const int64_t n = s.rows * s.C * s.lists;    // partial lists
    const int64_t rows = s.rows, k = p->k;
    w.n_ctx_cap = n_contexts(DT_NGRAM_HASH_TRIGRAM, p->d, p->k);   // the largest kind
    int64_t off = 0;
    auto take = [&](int64_t bytes) {
        const int64_t o = round_up(off, 256);
        off = o + bytes;
        return (size_t)o;
    };
    w.off_m = take(n * 4);
    w.off_s = take(n * 8);
    w.off_keys = take(n * k * 8);
    w.off_lse = take(rows * 8);
    w.off_ttok = take(rows * k * 4);
    w.off_tx = take(rows * k * 4);
    w.off_vmask = take((int64_t)p->B * w.n_ctx_cap * 4);
    w.off_g = take(p->mode == DT_MODE_DARTREE ? rows * k * k * 8 : 0);
    const bool full = p->mode == DT_MODE_DARTREE_FULL;
    const int64_t B = p->B, fw = full ? (int64_t)p->B * p->W : 0, nn = full ? fw * p->d : 0;
    // chunks of at least kVocabChunk tokens, about kVocabGroups workgroups
    // per depth over all request groups
    const int64_t ngroups = ceil_div(p->B > 0 ? p->B : 1, kVocabReqPerGroup);
    const int64_t want = kVocabGroups / ngroups > 1 ? kVocabGroups / ngroups : 1;
    const int64_t vc = round_up(ceil_div(p->V, want), 16);
    w.vchunk = (int)(vc > kVocabChunk ? vc : kVocabChunk);
    w.C2 = full ? (int)ceil_div(p->V, w.vchunk) : 0;
    w.off_f_tok = take(fw * 4);
    w.off_f_rk = take(fw * 8);
    w.off_f_s = take(fw * 8);
    w.off_f_node = take(fw * 4);
    w.off_f_n = take(full ? B * 4 : 0);
    w.off_n_tree = take(full ? B * 4 : 0);
    w.off_nd_tok = take(nn * 4);
    w.off_nd_par = take(nn * 4);
    w.off_nd_dep = take(nn * 4);
    w.off_nd_s = take(nn * 8);
    w.off_part = take(fw * w.C2 * (int64_t)sizeof(VocabEntry));
    w.off_fnorm = take(full ? (int64_t)p->V * 4 : 0);
    w.off_fbf = take(full ? (int64_t)p->V * p->R * 2 : 0);
    w.off_seed = take(full ? B * 8 : 0);
    w.off_cmp_n = take(full ? B * 4 : 0);
    w.off_cmp = take(full ? B * kFrontCap * (int64_t)sizeof(VocabEntry) : 0);
    w.total = (size_t)round_up(off, 256);
    return w;
}

TreePlan plan_tree(const dt_params* p, int kind) {
    TreePlan P{};
    const int d = p->d, k = p->k, W = p->W;
    P.n_ctx = n_contexts(kind, d, k);
    P.max_nodes = d * W;
    P.max_cand = W * k;
    int off = 0;
    auto take = [&](int bytes, int align) {
        off = (int)round_up(off, align);
        const int o = off;
        off += bytes;
        return o;
    };
    P.off_lse = take(d * 8, 8);
    P.off_g = take(p->mode == DT_MODE_DARTREE ? d * k * k * 8 : 0, 16);
    P.off_ttok = take(d * k * 4, 4);
    P.off_tx = take(d * k * 4, 4);
    P.off_vmask = take(P.n_ctx * 4, 4);
    P.off_misc = take(kMiscInts * 4, 4);
    P.off_sv_key = take((P.max_cand + 32) * 16, 16);  // + a block of sentinels
    P.off_sv_s = take((P.max_cand + 32) * 16, 16);
    const int nn = P.max_nodes;
    P.off_n_rec = take((nn + 1) * 32, 16);      // + the root's record
    P.off_n_s = take(nn * 8, 8);
    P.off_n_tok = take(nn * 4, 4);
    P.off_n_par = take(nn * 4, 4);
    P.off_n_dep = take(nn * 4, 4);
    P.off_n_new = take(nn * 4, 4);
    P.off_n_out = take(nn * 4, 4);
    P.total = (int)round_up(off, 16);
    return P;
}

// ---------------------------------------------------------------------------
// validation (host only; no HIP call)
// ---------------------------------------------------------------------------
static dt_status check_shape(const dt_params* p) {
    if (!p) return DT_ERR_INVALID_ARG;
    if (p->B < 0 || p->d < 1 || p->k < 1 || p->V < 1 || p->W < 1 || p->budget < 1)
        return DT_ERR_INVALID_ARG;
    if (p->k > p->V) return DT_ERR_INVALID_ARG;
    if (p->dtype != DT_DTYPE_F32 && p->dtype != DT_DTYPE_BF16) return DT_ERR_INVALID_ARG;
    if (p->mode != DT_MODE_DART && p->mode != DT_MODE_DARTREE && p->mode != DT_MODE_DARTREE_FULL)
        return DT_ERR_INVALID_ARG;
    if (p->sweep_chunks < 0) return DT_ERR_INVALID_ARG;
    if (p->d > kMaxD || p->k > kMaxK || p->W > kMaxW || p->budget > kMaxBudget ||
        p->W * p->k > kMaxCandidates || p->V >= kMaxV)
        return DT_ERR_UNSUPPORTED;
    const SweepPlan s = plan_sweep(p);
    if ((int64_t)s.C * s.lists * p->k > kMergeKeysPerRow || (int64_t)s.C * s.lists > 256) return DT_ERR_UNSUPPORTED;
    return DT_OK;
}

static dt_status check_workspace(const dt_params* p) {
    const WorkspacePlan w = plan_workspace(p, plan_sweep(p));
    if (w.total == 0) return DT_OK;
    if (!p->workspace || ((uintptr_t)p->workspace & 15u) || p->workspace_bytes < w.total)
        return DT_ERR_WORKSPACE;
    return DT_OK;
}

static dt_status check_ngram(const dt_ngram_table* g) {
    if (!g) return DT_ERR_INVALID_ARG;
    const bool finite = !(isinf(g->min_logp) && g->min_logp < 0);
    if (isnan(g->min_logp)) return DT_ERR_INVALID_ARG;
    switch (g->kind) {
    case DT_NGRAM_NONE:
        return DT_OK;
    case DT_NGRAM_DENSE_BIGRAM:
        return g->dense_logp ? DT_OK : DT_ERR_INVALID_ARG;
    case DT_NGRAM_CSR_BIGRAM:
        // an empty table (nnz = 0) needs no successor arrays
        if (!g->row_ptr || g->nnz < 0) return DT_ERR_INVALID_ARG;
        if (g->nnz > 0 && (!g->col || (finite && !g->csr_logp))) return DT_ERR_INVALID_ARG;
        return DT_OK;
    case DT_NGRAM_HASH_TRIGRAM:
        if (!g->keys || !g->succ || (finite && !g->hash_logp)) return DT_ERR_INVALID_ARG;
        if (g->cap < 2 || (g->cap & (g->cap - 1)) != 0) return DT_ERR_INVALID_ARG;
        if (g->S < 1 || g->S > 64) return DT_ERR_UNSUPPORTED;
        if (((uintptr_t)g->keys & 15u) != 0) return DT_ERR_INVALID_ARG;
        return DT_OK;
    default:
        return DT_ERR_INVALID_ARG;
    }
}

}  // namespace dt

using namespace dt;

extern "C" const char* dt_status_string(dt_status s) {
    // any int may arrive from C: read the bits without loading an
    // out-of-range enumeration value
    int v;
    memcpy(&v, &s, sizeof v);
    switch (v) {
    case DT_OK: return "DT_OK";
    case DT_ERR_INVALID_ARG: return "DT_ERR_INVALID_ARG: null pointer, value out of range or misaligned buffer";
    case DT_ERR_UNSUPPORTED: return "DT_ERR_UNSUPPORTED: outside the library's limits";
    case DT_ERR_WORKSPACE: return "DT_ERR_WORKSPACE: workspace missing, misaligned or smaller than dt_workspace_size()";
    case DT_ERR_HIP: return "DT_ERR_HIP: the HIP runtime refused a launch";
    default: return "unknown dt_status";
    }
}

extern "C" size_t dt_workspace_size(const dt_params* p) {
    if (check_shape(p) != DT_OK) return 0;
    return plan_workspace(p, plan_sweep(p)).total;
}

static dt_status launch_sweep_for(const void* logits, const dt_params* p, const SweepPlan& s,
                                  const WorkspacePlan& w, bool take_turns) {
    hipStream_t stream = (hipStream_t)p->stream;
    char* ws = (char*)p->workspace;
    SweepArgs sa{};
    sa.logits = logits;
    sa.V = p->V;
    sa.C = s.C;
    sa.chunk = s.chunk;
    sa.lists = s.lists;
    sa.k = p->k;
    sa.part_m = (float*)(ws + w.off_m);
    sa.part_s = (double*)(ws + w.off_s);
    sa.part_keys = (unsigned long long*)(ws + w.off_keys);
    if (p->prof_event_start && hipEventRecord((hipEvent_t)p->prof_event_start, stream) != hipSuccess)
        return DT_ERR_HIP;
    if (launch_sweep(sa, s.rows, p->dtype, take_turns, stream) != hipSuccess) return DT_ERR_HIP;
    if (p->prof_event_stop && hipEventRecord((hipEvent_t)p->prof_event_stop, stream) != hipSuccess)
        return DT_ERR_HIP;
    return DT_OK;
}

// Full-vocabulary DARTree mode: the sweep and the row merge give lse; then
// per depth the vocabulary kernel and the frontier merge; then the budget
// and the outputs.  The profiling events (if given) bracket the depth loop.
static dt_status build_full(const void* logits, const dt_params* p, const SweepPlan& s, const WorkspacePlan& w,
                            const dt_tree_out* out) {
    hipStream_t stream = (hipStream_t)p->stream;
    char* ws = (char*)p->workspace;
    SweepArgs sa{};
    sa.logits = logits;
    sa.V = p->V;
    sa.C = s.C;
    sa.chunk = s.chunk;
    sa.lists = s.lists;
    sa.k = p->k;
    sa.part_m = (float*)(ws + w.off_m);
    sa.part_s = (double*)(ws + w.off_s);
    sa.part_keys = (unsigned long long*)(ws + w.off_keys);
    if (launch_sweep(sa, s.rows, p->dtype, false, stream) != hipSuccess) return DT_ERR_HIP;
    MergeArgs ma{};
    ma.rows = (int)s.rows;
    ma.C = s.C * s.lists;
    ma.k = p->k;
    ma.part_m = sa.part_m;
    ma.part_s = sa.part_s;
    ma.part_keys = sa.part_keys;
    ma.lse = (double*)(ws + w.off_lse);
    ma.tok = (int32_t*)(ws + w.off_ttok);
    ma.val = (float*)(ws + w.off_tx);
    if (launch_merge(ma, stream) != hipSuccess) return DT_ERR_HIP;

    VocabArgs va{};
    va.B = p->B;
    va.V = p->V;
    va.d = p->d;
    va.W = p->W;
    va.R = p->R;
    va.dtype = p->dtype;
    va.vchunk = w.vchunk;
    va.C2 = w.C2;
    va.logits = logits;
    va.E = p->E;
    va.F = p->F;
    va.fnorm = (const float*)(ws + w.off_fnorm);
    va.Fbf = (const uint16_t*)(ws + w.off_fbf);
    va.ctx = p->ctx;
    va.f_tok = (const int32_t*)(ws + w.off_f_tok);
    va.f_rk = (const double*)(ws + w.off_f_rk);
    va.f_n = (const int32_t*)(ws + w.off_f_n);
    va.part = (VocabEntry*)(ws + w.off_part);
    va.seed = (const double*)(ws + w.off_seed);
    va.cmp_n = (int32_t*)(ws + w.off_cmp_n);
    va.cmp = (VocabEntry*)(ws + w.off_cmp);
    FrontierArgs fa{};
    fa.B = p->B;
    fa.d = p->d;
    fa.W = p->W;
    fa.C2 = w.C2;
    fa.part = va.part;
    fa.cmp_n = va.cmp_n;
    fa.cmp = va.cmp;
    fa.lse = ma.lse;
    fa.f_tok = (int32_t*)(ws + w.off_f_tok);
    fa.f_rk = (double*)(ws + w.off_f_rk);
    fa.f_s = (double*)(ws + w.off_f_s);
    fa.f_node = (int32_t*)(ws + w.off_f_node);
    fa.f_n = (int32_t*)(ws + w.off_f_n);
    fa.n_tree = (int32_t*)(ws + w.off_n_tree);
    fa.nd_tok = (int32_t*)(ws + w.off_nd_tok);
    fa.nd_par = (int32_t*)(ws + w.off_nd_par);
    fa.nd_dep = (int32_t*)(ws + w.off_nd_dep);
    fa.nd_s = (double*)(ws + w.off_nd_s);
    fa.V = p->V;
    fa.k = p->k;
    fa.R = p->R;
    fa.ttok = ma.tok;
    fa.tx = ma.val;
    fa.E = p->E;
    fa.F = p->F;
    fa.seed = (double*)(ws + w.off_seed);
    fa.fnorm = va.fnorm;
    if (launch_fnorm(p->F, p->V, p->R, (float*)(ws + w.off_fnorm), (uint16_t*)(ws + w.off_fbf), stream) != hipSuccess)
        return DT_ERR_HIP;
    fa.t = 0;
    if (launch_seed1(fa, p->ctx, stream) != hipSuccess) return DT_ERR_HIP;
    if (p->prof_event_start && hipEventRecord((hipEvent_t)p->prof_event_start, stream) != hipSuccess)
        return DT_ERR_HIP;
    for (int t = 1; t <= p->d; ++t) {
        va.t = t;
        fa.t = t;
        if (launch_vocab(va, stream) != hipSuccess) return DT_ERR_HIP;
        if (launch_frontier(fa, stream) != hipSuccess) return DT_ERR_HIP;
    }
    if (p->prof_event_stop && hipEventRecord((hipEvent_t)p->prof_event_stop, stream) != hipSuccess)
        return DT_ERR_HIP;
    FinishArgs na{};
    na.B = p->B;
    na.d = p->d;
    na.W = p->W;
    na.budget = p->budget;
    na.mask_words = (p->budget + 31) / 32;
    na.n_tree = fa.n_tree;
    na.nd_tok = fa.nd_tok;
    na.nd_par = fa.nd_par;
    na.nd_dep = fa.nd_dep;
    na.nd_s = fa.nd_s;
    na.n_nodes = out->n_nodes;
    na.tokens = out->tokens;
    na.parents = out->parents;
    na.depths = out->depths;
    na.scores = out->scores;
    na.mask = out->mask;
    if (launch_finish(na, stream) != hipSuccess) return DT_ERR_HIP;
    return DT_OK;
}

static dt_status enqueue_build(const void* logits, const dt_ngram_table* ngram, const dt_params* p,
                               const dt_tree_out* out);

// Every argument check of dt_build_tree except the workspace's; host only.
// DT_OK with *nothing = true means a valid call with nothing to enqueue (B = 0).
static dt_status check_build(const void* logits, const dt_ngram_table* ngram, const dt_params* p,
                             const dt_tree_out* out, bool* nothing) {
    *nothing = false;
    dt_status st = check_shape(p);
    if (st != DT_OK) return st;
    if ((st = check_ngram(ngram)) != DT_OK) return st;
    if (!out) return DT_ERR_INVALID_ARG;
    if (p->mode == DT_MODE_DARTREE) {
        if (!p->E || !p->F) return DT_ERR_INVALID_ARG;
        if (p->R < 4 || p->R > 256 || p->R % 4 != 0) return DT_ERR_UNSUPPORTED;
        if (((uintptr_t)p->E & 15u) || ((uintptr_t)p->F & 15u)) return DT_ERR_INVALID_ARG;
    }
    if (p->mode == DT_MODE_DARTREE_FULL) {
        if (!p->E || !p->F) return DT_ERR_INVALID_ARG;
        if (((uintptr_t)p->E & 15u) || ((uintptr_t)p->F & 15u)) return DT_ERR_INVALID_ARG;
        if (p->R != 16 && p->R != 32 && p->R != 64) return DT_ERR_UNSUPPORTED;
        if (p->W > kFullMaxW || ngram->kind != DT_NGRAM_NONE) return DT_ERR_UNSUPPORTED;
    }
    const TreePlan plan = plan_tree(p, ngram->kind);
    if (plan.total > kTreeLdsLimit) return DT_ERR_UNSUPPORTED;
    if (p->B == 0) {
        *nothing = true;
        return DT_OK;
    }
    if (!logits || ((uintptr_t)logits & 15u) || !p->ctx) return DT_ERR_INVALID_ARG;
    if (!out->n_nodes || !out->tokens || !out->parents || !out->depths || !out->scores || !out->mask)
        return DT_ERR_INVALID_ARG;
    return DT_OK;
}

extern "C" dt_status dt_build_tree(const void* logits, const dt_ngram_table* ngram,
                                   const dt_params* p, const dt_tree_out* out) {
    bool nothing;
    dt_status st = check_build(logits, ngram, p, out, &nothing);
    if (st != DT_OK || nothing) return st;
    if ((st = check_workspace(p)) != DT_OK) return st;
    return enqueue_build(logits, ngram, p, out);
}

// The scratch buffer of dt_build_tree_noalloc: a device array of fixed size
// in this library's code object, one copy per GPU, held until the process
// ends.  Host code never passes the array's own name to a kernel (on the
// host it is only a stand-in for the symbol): the device address of each
// GPU's copy comes from hipGetSymbolAddress, looked up once per device on
// the first call there and kept below.
static __device__ __align__(256) unsigned char scratch[DT_NOALLOC_SCRATCH_BYTES];
constexpr int kMaxDevices = 64;
static void* g_scratch_ptr[kMaxDevices];
static std::mutex g_scratch_mu;

static dt_status scratch_of(hipStream_t stream, void** ptr_out) {
    int dev = 0;
    if ((stream ? hipStreamGetDevice(stream, &dev) : hipGetDevice(&dev)) != hipSuccess) return DT_ERR_HIP;
    if (dev < 0 || dev >= kMaxDevices) return DT_ERR_UNSUPPORTED;
    std::lock_guard<std::mutex> lock(g_scratch_mu);
    if (!g_scratch_ptr[dev]) {
        int cur = 0;
        if (hipGetDevice(&cur) != hipSuccess) return DT_ERR_HIP;
        if (cur != dev && hipSetDevice(dev) != hipSuccess) return DT_ERR_HIP;
        void* ptr = nullptr;
        const hipError_t e = hipGetSymbolAddress(&ptr, HIP_SYMBOL(scratch));
        if (cur != dev && hipSetDevice(cur) != hipSuccess) return DT_ERR_HIP;
        if (e != hipSuccess || !ptr) return DT_ERR_HIP;
        g_scratch_ptr[dev] = ptr;
    }
    *ptr_out = g_scratch_ptr[dev];
    return DT_OK;
}

extern "C" dt_status dt_build_tree_noalloc(const void* logits, const dt_ngram_table* ngram,
                                           const dt_params* p, const dt_tree_out* out) {
    bool nothing;
    dt_status st = check_build(logits, ngram, p, out, &nothing);
    if (st != DT_OK || nothing) return st;
    if (plan_workspace(p, plan_sweep(p)).total > (size_t)DT_NOALLOC_SCRATCH_BYTES) return DT_ERR_WORKSPACE;
    dt_params q = *p;
    if ((st = scratch_of((hipStream_t)p->stream, &q.workspace)) != DT_OK) return st;
    q.workspace_bytes = DT_NOALLOC_SCRATCH_BYTES;
    return enqueue_build(logits, ngram, &q, out);
}

// Launches of the whole path for validated arguments and a large enough workspace.
static dt_status enqueue_build(const void* logits, const dt_ngram_table* ngram, const dt_params* p,
                               const dt_tree_out* out) {
    dt_status st;
    const TreePlan plan = plan_tree(p, ngram->kind);
    const SweepPlan s = plan_sweep(p);
    const WorkspacePlan w = plan_workspace(p, s);
    if (p->mode == DT_MODE_DARTREE_FULL) {
        if (w.C2 > kMaxVocabChunks) return DT_ERR_UNSUPPORTED;   // cannot happen: chunks adapt to V
        return build_full(logits, p, s, w, out);
    }
    char* ws = (char*)p->workspace;
    const bool take_turns = s.rows * s.C >= kSweepTurnMinGrid && s.rows * s.C <= kSweepTurnMaxGrid &&
                            plan.total + kPrepLds <= kTreeLdsLimit - 2 * kSweepLdsTurn;
    if ((st = launch_sweep_for(logits, p, s, w, take_turns)) != DT_OK) return st;
    PrepArgs pa{};
    pa.B = p->B;
    pa.d = p->d;
    pa.k = p->k;
    pa.L = s.C * s.lists;                         // partial lists per row
    pa.mode = p->mode;
    pa.R = p->R;
    pa.n_ctx = w.n_ctx_cap;
    pa.ctx = p->ctx;
    pa.part_m = (const float*)(ws + w.off_m);
    pa.part_s = (const double*)(ws + w.off_s);
    pa.part_keys = (const unsigned long long*)(ws + w.off_keys);
    pa.ng.kind = ngram->kind;
    pa.ng.V = p->V;
    pa.ng.min_logp = ngram->min_logp;
    pa.ng.dense = ngram->dense_logp;
    pa.ng.row_ptr = ngram->row_ptr;
    pa.ng.col = ngram->col;
    pa.ng.csr_logp = ngram->csr_logp;
    pa.ng.keys = (const unsigned long long*)ngram->keys;
    pa.ng.succ = ngram->succ;
    pa.ng.hash_logp = ngram->hash_logp;
    pa.ng.cap = ngram->cap;
    pa.ng.S = ngram->S;
    pa.E = p->E;
    pa.F = p->F;
    pa.lse = (double*)(ws + w.off_lse);
    pa.ttok = (int32_t*)(ws + w.off_ttok);
    pa.tx = (float*)(ws + w.off_tx);
    pa.vmask = (uint32_t*)(ws + w.off_vmask);
    pa.g = (double*)(ws + w.off_g);
    // the k^2 trigram contexts of a depth are split over workgroups of
    // kPrepContexts lookups
    pa.nsplit = ngram->kind == DT_NGRAM_HASH_TRIGRAM ? (int)ceil_div((int64_t)p->k * p->k, kPrepContexts) : 1;
    if (launch_prep(pa, (hipStream_t)p->stream) != hipSuccess) return DT_ERR_HIP;

    TreeArgs ta{};
    ta.B = p->B;
    ta.d = p->d;
    ta.k = p->k;
    ta.W = p->W;
    ta.budget = p->budget;
    ta.mode = p->mode;
    ta.mask_words = (p->budget + 31) / 32;
    ta.ng_kind = ngram->kind;
    ta.n_ctx = w.n_ctx_cap;                       // per-request stride of vmask
    ta.lse = pa.lse;
    ta.ttok = pa.ttok;
    ta.tx = pa.tx;
    ta.vmask = pa.vmask;
    ta.g = pa.g;
    ta.n_nodes = out->n_nodes;
    ta.tokens = out->tokens;
    ta.parents = out->parents;
    ta.depths = out->depths;
    ta.scores = out->scores;
    ta.mask = out->mask;
    ta.plan = plan;
    if (launch_tree(ta, (hipStream_t)p->stream) != hipSuccess) return DT_ERR_HIP;
    return DT_OK;
}

extern "C" dt_status dt_position_topk(const void* logits, const dt_params* p, double* lse,
                                      int32_t* topk_tok, float* topk_val) {
    dt_status st = check_shape(p);
    if (st != DT_OK) return st;
    if (p->B == 0) return DT_OK;
    if (!logits || ((uintptr_t)logits & 15u) || !lse || !topk_tok || !topk_val) return DT_ERR_INVALID_ARG;
    if ((st = check_workspace(p)) != DT_OK) return st;
    const SweepPlan s = plan_sweep(p);
    const WorkspacePlan w = plan_workspace(p, s);
    if ((st = launch_sweep_for(logits, p, s, w, false)) != DT_OK) return st;
    char* ws = (char*)p->workspace;
    MergeArgs ma{};
    ma.rows = (int)s.rows;
    ma.C = s.C * s.lists;
    ma.k = p->k;
    ma.part_m = (const float*)(ws + w.off_m);
    ma.part_s = (const double*)(ws + w.off_s);
    ma.part_keys = (const unsigned long long*)(ws + w.off_keys);
    ma.lse = lse;
    ma.tok = topk_tok;
    ma.val = topk_val;
    if (launch_merge(ma, (hipStream_t)p->stream) != hipSuccess) return DT_ERR_HIP;
    return DT_OK;
}

extern "C" dt_status dt_ngram_update(const dt_ngram_table* table, const int32_t* ctx, const int32_t* tokens,
                                     const int32_t* lengths, int32_t B, int32_t L, float new_logp,
                                     int32_t* counts, void* stream) {
    if (!table || table->kind != DT_NGRAM_HASH_TRIGRAM) return DT_ERR_INVALID_ARG;
    if (B < 0 || L < 0 || isnan(new_logp)) return DT_ERR_INVALID_ARG;
    if (!table->keys || !table->succ || table->cap < 2 || (table->cap & (table->cap - 1)) != 0)
        return DT_ERR_INVALID_ARG;
    if (((uintptr_t)table->keys & 7u) != 0 || ((uintptr_t)table->succ & 3u) != 0 ||
        ((uintptr_t)table->hash_logp & 3u) != 0)
        return DT_ERR_INVALID_ARG;
    if (table->S < 1 || table->S > 64) return DT_ERR_UNSUPPORTED;
    if ((int64_t)B * L == 0) return DT_OK;
    if (!ctx || !tokens || !lengths) return DT_ERR_INVALID_ARG;
    NGramUpdateArgs a{};
    a.B = B;
    a.L = L;
    a.S = table->S;
    a.cap = table->cap;
    a.new_logp = new_logp;
    a.ctx = ctx;
    a.tokens = tokens;
    a.lengths = lengths;
    a.keys = (unsigned long long*)table->keys;           // the update writes the table in place
    a.succ = (int32_t*)table->succ;
    a.hash_logp = (float*)table->hash_logp;
    a.counts = counts;
    if (launch_ngram_update(a, (hipStream_t)stream) != hipSuccess) return DT_ERR_HIP;
    return DT_OK;
}

extern "C" dt_status dt_verify_length(const dt_tree_out* tree, int32_t B, int32_t budget, double cost_fixed,
                                      double cost_per_token, int32_t* n_verify, int32_t* rank, void* stream) {
    if (!tree || B < 0 || budget < 1) return DT_ERR_INVALID_ARG;
    if (!(cost_fixed > 0.0) || !isfinite(cost_fixed) || !(cost_per_token >= 0.0) || !isfinite(cost_per_token))
        return DT_ERR_INVALID_ARG;
    if (budget > kMaxBudget) return DT_ERR_UNSUPPORTED;
    if (B == 0) return DT_OK;
    if (!tree->n_nodes || !tree->parents || !tree->depths || !tree->scores || !n_verify || !rank)
        return DT_ERR_INVALID_ARG;
    VerifyArgs a{};
    a.B = B;
    a.budget = budget;
    a.cost_fixed = cost_fixed;
    a.cost_per_token = cost_per_token;
    a.n_nodes = tree->n_nodes;
    a.parents = tree->parents;
    a.depths = tree->depths;
    a.scores = tree->scores;
    a.n_verify = n_verify;
    a.rank = rank;
    if (launch_verify(a, (hipStream_t)stream) != hipSuccess) return DT_ERR_HIP;
    return DT_OK;
}

// ---------------------------------------------------------------------------
// the verification pass (dt.h, second part)
// ---------------------------------------------------------------------------
namespace dt {

// Makes the stream's device current for the launches of one call.
class DeviceScope {
public:
    explicit DeviceScope(hipStream_t stream) {
        int dev = 0;
        if (hipGetDevice(&cur_) != hipSuccess) return;
        if (stream ? hipStreamGetDevice(stream, &dev) != hipSuccess : false) return;
        if (stream && dev != cur_) {
            if (hipSetDevice(dev) != hipSuccess) return;
            moved_ = true;
        }
        ok_ = true;
    }
    ~DeviceScope() {
        if (moved_) (void)hipSetDevice(cur_);
    }
    DeviceScope(const DeviceScope&) = delete;
    DeviceScope& operator=(const DeviceScope&) = delete;
    bool ok() const { return ok_; }

private:
    int cur_ = 0;
    bool moved_ = false, ok_ = false;
};

static bool misaligned(const void* p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) != 0; }
static bool bad_stride(int64_t s) { return s < 0 || (s & 7) != 0; }

// Two layers, pages, slots or heads at less than a head's distance share
// elements: fine to read, but a call that writes them would race with itself.
static bool shares_elements(const dt_kv_cache* kv) {
    return (kv->layers > 1 && kv->layer_stride < kv->D) || (kv->num_pages > 1 && kv->page_stride < kv->D) ||
           (kv->page_size > 1 && kv->slot_stride < kv->D) || (kv->Hkv > 1 && kv->head_stride < kv->D);
}

// A cache's shape; its pointers too where `pointers` is set.
static dt_status check_cache(const dt_kv_cache* kv, bool pointers) {
    if (!kv) return DT_ERR_INVALID_ARG;
    if (kv->layers < 1 || kv->num_pages < 1 || kv->page_size < 1 || kv->max_pages < 1 || kv->Hkv < 1 || kv->D < 1)
        return DT_ERR_INVALID_ARG;
    if (kv->dtype != DT_DTYPE_BF16 && kv->dtype != DT_DTYPE_F16) return DT_ERR_INVALID_ARG;
    if ((kv->layers > 1 && bad_stride(kv->layer_stride)) || (kv->num_pages > 1 && bad_stride(kv->page_stride)) ||
        (kv->page_size > 1 && bad_stride(kv->slot_stride)) || (kv->Hkv > 1 && bad_stride(kv->head_stride)))
        return DT_ERR_INVALID_ARG;
    if (kv->D != 64 && kv->D != 128 && kv->D != 256) return DT_ERR_UNSUPPORTED;
    if (kv->Hkv > kMaxPassHeads || (int64_t)kv->max_pages * kv->page_size > kMaxSlots) return DT_ERR_UNSUPPORTED;
    if (pointers && (!kv->k || !kv->v || !kv->page_table || misaligned(kv->k, 16) || misaligned(kv->v, 16) ||
                     misaligned(kv->page_table, 4)))
        return DT_ERR_INVALID_ARG;
    return DT_OK;
}

static dt_status check_chunk(const dt_chunk* c, bool pointers) {
    if (!c || c->B < 0 || c->lead < 0 || c->n_max < 0) return DT_ERR_INVALID_ARG;
    const int64_t rows = (int64_t)c->lead + c->n_max;
    if (rows < 1) return DT_ERR_INVALID_ARG;
    if (c->B > 65535 || rows > kMaxChunkRows || c->B * rows > kMaxBatchRows) return DT_ERR_UNSUPPORTED;
    if (pointers && c->B > 0 && (!c->ctx_len || misaligned(c->ctx_len, 4) || misaligned(c->n_nodes, 4) ||
                                 misaligned(c->mask, 4) || misaligned(c->depths, 4)))
        return DT_ERR_INVALID_ARG;
    return DT_OK;
}

static ChunkArgs chunk_args(const dt_chunk* c) {
    ChunkArgs a{};
    a.B = c->B;
    a.lead = c->lead;
    a.n_max = c->n_max;
    a.rows = c->lead + c->n_max;
    a.mask_words = (c->n_max + 31) / 32;
    a.ctx_len = c->ctx_len;
    a.n_nodes = c->n_nodes;
    a.mask = c->n_max ? c->mask : nullptr;
    a.depths = c->n_max ? c->depths : nullptr;
    return a;
}

static CacheArgs cache_args(const dt_kv_cache* kv, int layer) {
    CacheArgs a{};
    const int64_t at = kv->layers > 1 ? layer * kv->layer_stride : 0;
    a.k = (uint16_t*)kv->k + at;
    a.v = (uint16_t*)kv->v + at;
    a.page_table = kv->page_table;
    a.page_stride = kv->num_pages > 1 ? kv->page_stride : 0;
    a.slot_stride = kv->page_size > 1 ? kv->slot_stride : 0;
    a.head_stride = kv->Hkv > 1 ? kv->head_stride : 0;
    a.num_pages = kv->num_pages;
    a.page_size = kv->page_size;
    a.max_pages = kv->max_pages;
    a.Hkv = kv->Hkv;
    a.D = kv->D;
    a.cap = (int)((int64_t)kv->max_pages * kv->page_size);
    a.page_shift = (kv->page_size & (kv->page_size - 1)) == 0 ? __builtin_ctz((unsigned)kv->page_size) : -1;
    return a;
}

// Rows of `heads` heads of D elements: aligned, and apart where there are several.
static bool bad_rows(const void* p, int64_t stride, int64_t rows, int64_t heads, int D) {
    return !p || misaligned(p, 16) || (rows > 1 && (bad_stride(stride) || stride < heads * D));
}

static dt_status check_attention_shape(const dt_kv_cache* kv, const dt_chunk* c, int32_t Hq) {
    dt_status st = check_cache(kv, false);
    if (st != DT_OK) return st;
    if ((st = check_chunk(c, false)) != DT_OK) return st;
    if (Hq < 1 || Hq % kv->Hkv != 0) return DT_ERR_INVALID_ARG;
    if (Hq > kMaxPassHeads) return DT_ERR_UNSUPPORTED;
    if ((int64_t)c->B * (c->lead + c->n_max) * Hq > INT32_MAX) return DT_ERR_UNSUPPORTED;
    return DT_OK;
}

}  // namespace dt

extern "C" dt_status dt_rope_frequencies(int32_t kind, int32_t rot_dim, double base, double factor, double low,
                                         double high, double original, double* freqs, float* scale) {
    if (!freqs || !scale || rot_dim < 2 || rot_dim % 2 != 0) return DT_ERR_INVALID_ARG;
    if (kind < DT_ROPE_NONE || kind > DT_ROPE_YARN) return DT_ERR_INVALID_ARG;
    if (!isfinite(base) || !(base > 1.0) || !isfinite(factor) || !(factor > 0.0)) return DT_ERR_INVALID_ARG;
    const bool blend = kind == DT_ROPE_WAVELENGTH || kind == DT_ROPE_YARN;
    if (blend && (!(low > 0.0) || !(high > low) || !isfinite(high) || !(original > 0.0) || !isfinite(original)))
        return DT_ERR_INVALID_ARG;
    const double pi2 = 6.283185307179586476925;
    double i_low = 0, i_high = 0;
    if (kind == DT_ROPE_YARN) {
        const auto pair_of = [&](double turns) { return rot_dim * log(original / (pi2 * turns)) / (2 * log(base)); };
        const auto clamp = [&](double x) { return x < 0 ? 0 : (x > rot_dim - 1 ? rot_dim - 1 : x); };
        i_low = clamp(floor(pair_of(high)));
        i_high = clamp(ceil(pair_of(low)));
        if (i_high == i_low) i_high += 0.001;
    }
    for (int i = 0; i < rot_dim / 2; ++i) {
        const double f = pow(base, -2.0 * i / rot_dim);
        double s = 1;                              // weight of the unscaled frequency
        if (kind == DT_ROPE_LINEAR) s = 0;
        if (kind == DT_ROPE_WAVELENGTH) {
            const double turns = original * f / pi2;   // within the original context
            s = turns < low ? 0 : (turns > high ? 1 : (turns - low) / (high - low));
        }
        if (kind == DT_ROPE_YARN) {
            const double t = (i - i_low) / (i_high - i_low);
            s = 1 - (t < 0 ? 0 : (t > 1 ? 1 : t));
        }
        freqs[i] = (1 - s) * f / factor + s * f;
    }
    *scale = kind == DT_ROPE_YARN && factor > 1 ? (float)(0.1 * log(factor) + 1) : 1.0f;
    return DT_OK;
}

extern "C" dt_status dt_kv_append(const dt_kv_cache* kv, const dt_chunk* chunk, const dt_append_params* p) {
    if (!p) return DT_ERR_INVALID_ARG;
    dt_status st = check_cache(kv, !chunk || chunk->B != 0);
    if (st != DT_OK) return st;
    if (shares_elements(kv)) return DT_ERR_INVALID_ARG;
    if ((st = check_chunk(chunk, true)) != DT_OK) return st;
    if (p->layer < 0 || p->layer >= kv->layers || !isfinite(p->eps) || p->eps < 0 || !isfinite(p->rot_scale))
        return DT_ERR_INVALID_ARG;
    if (p->rot_dim < 0 || p->rot_dim > kv->D) return DT_ERR_INVALID_ARG;
    if (p->rot_dim % 16 != 0) return DT_ERR_UNSUPPORTED;
    if (p->rot_dim > 0 && (!p->freqs || misaligned(p->freqs, 8))) return DT_ERR_INVALID_ARG;
    if ((p->q == nullptr) != (p->q_out == nullptr)) return DT_ERR_INVALID_ARG;
    const int64_t rows = (int64_t)chunk->B * (chunk->lead + chunk->n_max);
    if (p->q) {
        if (p->Hq < 1) return DT_ERR_INVALID_ARG;
        if (p->Hq > kMaxPassHeads) return DT_ERR_UNSUPPORTED;
    }
    if (misaligned(p->q_norm, 16) || misaligned(p->k_norm, 16)) return DT_ERR_INVALID_ARG;
    if (chunk->B == 0) return DT_OK;
    if (bad_rows(p->k, p->k_stride, rows, kv->Hkv, kv->D) || bad_rows(p->v, p->v_stride, rows, kv->Hkv, kv->D))
        return DT_ERR_INVALID_ARG;
    if (p->q && (bad_rows(p->q, p->q_stride, rows, p->Hq, kv->D) ||
                 bad_rows(p->q_out, p->q_out_stride, rows, p->Hq, kv->D) ||
                 (rows > 1 && p->q == p->q_out && p->q_stride != p->q_out_stride)))
        return DT_ERR_INVALID_ARG;
    AppendArgs a{};
    a.c = chunk_args(chunk);
    a.kv = cache_args(kv, p->layer);
    a.q = (const uint16_t*)p->q;
    a.k = (const uint16_t*)p->k;
    a.v = (const uint16_t*)p->v;
    a.q_out = (uint16_t*)p->q_out;
    a.q_stride = p->q_stride;
    a.k_stride = p->k_stride;
    a.v_stride = p->v_stride;
    a.q_out_stride = p->q_out_stride;
    a.Hq = p->q ? p->Hq : 0;
    a.q_norm = (const uint16_t*)p->q_norm;
    a.k_norm = (const uint16_t*)p->k_norm;
    a.eps = p->eps;
    a.rot_scale = p->rot_scale;
    a.freqs = p->freqs;
    a.rot_dim = p->rot_dim;
    a.interleaved = p->interleaved != 0;
    const DeviceScope scope((hipStream_t)p->stream);
    if (!scope.ok() || launch_append(a, kv->dtype, (hipStream_t)p->stream) != hipSuccess) return DT_ERR_HIP;
    return DT_OK;
}

extern "C" size_t dt_attention_workspace(const dt_kv_cache* kv, const dt_chunk* chunk, int32_t Hq) {
    if (check_attention_shape(kv, chunk, Hq) != DT_OK) return 0;
    return attention_workspace(chunk_args(chunk), kv->Hkv, Hq, kv->D);
}

extern "C" dt_status dt_tree_attention(const dt_kv_cache* kv, const dt_chunk* chunk, const dt_attention_params* p) {
    if (!p) return DT_ERR_INVALID_ARG;
    dt_status st = check_attention_shape(kv, chunk, p->Hq);
    if (st != DT_OK) return st;
    if ((st = check_cache(kv, chunk->B != 0)) != DT_OK) return st;
    if ((st = check_chunk(chunk, true)) != DT_OK) return st;
    if (p->layer < 0 || p->layer >= kv->layers || !isfinite(p->scale) || !(p->scale > 0)) return DT_ERR_INVALID_ARG;
    if (misaligned(p->lse, 4)) return DT_ERR_INVALID_ARG;
    if (chunk->B == 0) return DT_OK;
    const int64_t rows = (int64_t)chunk->B * (chunk->lead + chunk->n_max);
    if (bad_rows(p->q, p->q_stride, rows, p->Hq, kv->D) || bad_rows(p->out, p->out_stride, rows, p->Hq, kv->D) ||
        p->q == p->out)
        return DT_ERR_INVALID_ARG;
    AttentionArgs a{};
    a.c = chunk_args(chunk);
    a.kv = cache_args(kv, p->layer);
    const size_t need = attention_workspace(a.c, kv->Hkv, p->Hq, kv->D);
    if (need > 0 && (!p->workspace || misaligned(p->workspace, 16) || p->workspace_bytes < need))
        return DT_ERR_WORKSPACE;
    a.q = (const uint16_t*)p->q;
    a.out = (uint16_t*)p->out;
    a.q_stride = p->q_stride;
    a.out_stride = p->out_stride;
    a.Hq = p->Hq;
    a.G = p->Hq / kv->Hkv;
    a.by8 = kv->page_size % 8 == 0 && a.kv.slot_stride < (1 << 26);
    a.scale_log2 = (float)(p->scale * 1.4426950408889634074);
    a.lse = p->lse;
    const DeviceScope scope((hipStream_t)p->stream);
    if (!scope.ok() || launch_attention(a, kv->dtype, p->workspace, (hipStream_t)p->stream) != hipSuccess)
        return DT_ERR_HIP;
    return DT_OK;
}

extern "C" dt_status dt_process_logits(const dt_logits_params* p) {
    if (!p || p->B < 0 || p->lead < 0 || p->n_max < 0 || p->V < 1) return DT_ERR_INVALID_ARG;
    const int64_t rows = (int64_t)p->lead + p->n_max;
    if (rows < 1 || p->history_max < 0 || p->n_bias < 0) return DT_ERR_INVALID_ARG;
    if (p->dtype != DT_DTYPE_F32 && p->dtype != DT_DTYPE_BF16) return DT_ERR_INVALID_ARG;
    if (p->B > 65535 || rows > kMaxChunkRows || p->V >= kMaxV || p->n_bias > 65534) return DT_ERR_UNSUPPORTED;
    if (p->node_tokens && p->n_max > kMaxCommitNodes) return DT_ERR_UNSUPPORTED;
    if (p->history && !p->history_len) return DT_ERR_INVALID_ARG;
    if (p->node_tokens && !p->node_mask) return DT_ERR_INVALID_ARG;
    if (p->bias_ids && !p->bias) return DT_ERR_INVALID_ARG;
    if (p->allow && p->allow_rows < 1) return DT_ERR_INVALID_ARG;
    if (p->allow && !p->allow_index && p->allow_rows < p->B * rows) return DT_ERR_INVALID_ARG;
    for (const void* q : {(const void*)p->n_nodes, (const void*)p->history, (const void*)p->history_len,
                          (const void*)p->prompt_len, (const void*)p->node_tokens, (const void*)p->node_mask,
                          (const void*)p->repetition, (const void*)p->frequency, (const void*)p->presence,
                          (const void*)p->bias_ids, (const void*)p->bias, (const void*)p->allow,
                          (const void*)p->allow_index})
        if (misaligned(q, 4)) return DT_ERR_INVALID_ARG;
    if (p->B == 0) return DT_OK;
    if (!p->logits || !p->out || misaligned(p->logits, 16) || misaligned(p->out, 16)) return DT_ERR_INVALID_ARG;
    LogitsArgs a{};
    a.logits = p->logits;
    a.out = p->out;
    a.B = p->B;
    a.lead = p->lead;
    a.n_max = p->n_max;
    a.rows = (int)rows;
    a.V = p->V;
    a.mask_words = (p->n_max + 31) / 32;
    a.n_nodes = p->n_nodes;
    a.history = p->history_max > 0 ? p->history : nullptr;
    a.history_max = p->history_max;
    a.history_len = p->history_len;
    a.prompt_len = p->prompt_len;
    a.node_tokens = p->n_max > 0 ? p->node_tokens : nullptr;
    a.node_mask = p->node_mask;
    a.repetition = p->repetition;
    a.frequency = p->frequency;
    a.presence = p->presence;
    a.bias_ids = p->bias_ids;
    a.bias = p->bias;
    a.n_bias = p->bias_ids ? p->n_bias : 0;
    a.allow = p->allow;
    a.allow_index = p->allow_index;
    a.allow_rows = p->allow_rows;
    const DeviceScope scope((hipStream_t)p->stream);
    if (!scope.ok() || launch_logits(a, p->dtype, (hipStream_t)p->stream) != hipSuccess) return DT_ERR_HIP;
    return DT_OK;
}

extern "C" dt_status dt_commit_path(const dt_kv_cache* kv, const dt_chunk* chunk, const dt_commit_params* p) {
    if (!p) return DT_ERR_INVALID_ARG;
    dt_status st;
    if (kv && (st = check_cache(kv, !chunk || chunk->B != 0)) != DT_OK) return st;
    if (kv && shares_elements(kv)) return DT_ERR_INVALID_ARG;
    if ((st = check_chunk(chunk, true)) != DT_OK) return st;
    if (chunk->lead < 1 || p->L < 1) return DT_ERR_INVALID_ARG;
    if (chunk->n_max > kMaxCommitNodes) return DT_ERR_UNSUPPORTED;
    if (chunk->B == 0) return DT_OK;
    if (!p->target || !p->accepted || !p->lengths || (chunk->n_max > 0 && (!p->tokens || !p->parents)))
        return DT_ERR_INVALID_ARG;
    for (const void* q : {(const void*)p->tokens, (const void*)p->parents, (const void*)p->target,
                          (const void*)p->accepted, (const void*)p->lengths, (const void*)p->nodes})
        if (misaligned(q, 4)) return DT_ERR_INVALID_ARG;
    CommitArgs a{};
    a.c = chunk_args(chunk);
    if (kv) {
        a.kv = cache_args(kv, 0);
        a.layer_stride = kv->layers > 1 ? kv->layer_stride : 0;
        a.layers = kv->layers;
    }
    a.tokens = p->tokens;
    a.parents = p->parents;
    a.target = p->target;
    a.L = p->L;
    a.accepted = p->accepted;
    a.lengths = p->lengths;
    a.nodes = p->nodes;
    const DeviceScope scope((hipStream_t)p->stream);
    if (!scope.ok() || launch_commit(a, (hipStream_t)p->stream) != hipSuccess) return DT_ERR_HIP;
    return DT_OK;
}
