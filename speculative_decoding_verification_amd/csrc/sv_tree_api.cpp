// C ABI of the tree-drafting operators: host-side argument checks, workspace
// planning and dispatch.  Every check runs before anything is enqueued.
#include <cmath>
#include <cstdint>

#include "specverify.h"
#include "sv_tree.h"

namespace sv {
namespace {

constexpr size_t kAlign = 256;
constexpr double kLog2E = 1.4426950408889634;

size_t align_up(size_t x) { return (x + kAlign - 1) & ~(kAlign - 1); }

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

bool stride_ok(int64_t s) { return s >= 0 && s % 8 == 0; }

// log2 of a page size, or -1.
int page_shift_of(int32_t size) {
    for (int s = 0; s <= 10; ++s)
        if (size == 1 << s) return s;
    return -1;
}

sv_status plan_attention(const sv_tree_attention_desc* d, AttnPlan* p) {
    if (!d) return SV_ERR_NULL_ARG;
    if (d->B < 0 || d->B > 65535 || d->k < 0 || d->k > SV_MAX_DRAFT) return SV_ERR_BAD_SHAPE;
    if (d->kv_heads < 1 || d->q_heads < 1 || d->q_heads > 256 || d->q_heads % d->kv_heads) return SV_ERR_BAD_SHAPE;
    if (d->head_dim != 64 && d->head_dim != 96 && d->head_dim != 128 && d->head_dim != 256) return SV_ERR_BAD_SHAPE;
    const int shift = page_shift_of(d->page_size);
    if (shift < 0 || d->n_pages < 1 || d->max_pages < 1) return SV_ERR_BAD_SHAPE;
    if ((static_cast<int64_t>(d->max_pages) << shift) > (int64_t{1} << 30)) return SV_ERR_BAD_SHAPE;
    // the kernel numbers the cache's rows in 32 bits (n_pages and kv_heads << shift are each below 2^31)
    if (static_cast<uint64_t>(d->n_pages) * (static_cast<uint64_t>(d->kv_heads) << shift) >= (uint64_t{1} << 32))
        return SV_ERR_BAD_SHAPE;
    if (d->dtype != SV_BF16 && d->dtype != SV_F16) return SV_ERR_BAD_DTYPE;
    if (!(d->scale > 0.f) || !std::isfinite(d->scale)) return SV_ERR_BAD_SCALE;
    if (!stride_ok(d->q_stride_b) || !stride_ok(d->q_stride_r) || !stride_ok(d->q_stride_h)) return SV_ERR_MISALIGNED;
    p->batch = d->B;
    p->k = d->k;
    p->q_heads = d->q_heads;
    p->kv_heads = d->kv_heads;
    p->head_dim = d->head_dim;
    p->group = d->q_heads / d->kv_heads;
    p->rows = (d->k + 1) * p->group;
    // Query rows in as few units as the accumulators allow, the units as even as whole 16-row tiles are.
    const int most = attn_max_row_tiles(d->head_dim);
    const int tiles = (p->rows + 15) / 16;
    const int units = (tiles + most - 1) / most;
    p->row_tiles = (tiles + units - 1) / units;
    p->row_units = (tiles + p->row_tiles - 1) / p->row_tiles;
    // The units of one key head read the same keys: a cluster of workgroups on one die, so that these pass its L2 once.
    constexpr int per_die = kAttnWgs / kAttnDies;
    p->cluster = p->row_units < per_die ? p->row_units : per_die;
    p->clusters = kAttnDies * (per_die / p->cluster);
    p->n_pages = d->n_pages;
    p->page_shift = shift;
    p->max_pages = d->max_pages;
    p->is_f16 = d->dtype == SV_F16;
    p->scale_log2 = static_cast<float>(static_cast<double>(d->scale) * kLog2E);
    p->q_stride_b = d->q_stride_b;
    p->q_stride_r = d->q_stride_r;
    p->q_stride_h = d->q_stride_h;
    return SV_OK;
}

size_t attention_slot_rows(const AttnPlan& p) {
    return static_cast<size_t>(p.clusters) * p.row_units * 2 * p.row_tiles * 16;
}
size_t attention_acc_bytes(const AttnPlan& p) { return align_up(attention_slot_rows(p) * p.head_dim * sizeof(float)); }
size_t attention_ml_bytes(const AttnPlan& p) { return align_up(attention_slot_rows(p) * 2 * sizeof(float)); }

size_t attention_bytes(const AttnPlan& p) {
    return attention_acc_bytes(p) + attention_ml_bytes(p) +
           align_up(static_cast<size_t>(p.clusters) * p.row_units * sizeof(AttnSplit));
}

// As many slices of whole tiles to a row as make up to `wgs` workgroups on `rows` rows.
void tree_slices(int64_t vocab, int64_t rows, int64_t wgs, int64_t* per, int32_t* slices) {
    const int64_t tiles = (vocab + kTreeTile - 1) / kTreeTile;
    int64_t n = (tiles + kTreeMaxSlices - 1) / kTreeMaxSlices;
    while (n < tiles && (tiles + n - 1) / n * rows > wgs) ++n;
    *per = n * kTreeTile;
    *slices = static_cast<int32_t>((tiles + n - 1) / n);
}

uint64_t tree_wait_ticks = kTreeWaitTicks;  // tests set it to 0

sv_status plan_tree(const sv_verify_tree_desc* d, TreePlan* p) {
    if (!d) return SV_ERR_NULL_ARG;
    if (d->B < 0 || d->B > kTreeMaxBatch || d->k < 1 || d->k > SV_MAX_DRAFT || d->V < 1 || d->V > (1 << 24)) return SV_ERR_BAD_SHAPE;
    if (d->dtype != SV_F32 && d->dtype != SV_BF16) return SV_ERR_BAD_DTYPE;
    if (d->draft_kind != SV_DRAFT_LOGITS && d->draft_kind != SV_DRAFT_ONEHOT) return SV_ERR_BAD_DRAFT_KIND;
    const float t = d->temperature;
    if (!(t == 0.f || (std::isfinite(t) && t >= 1e-4f))) return SV_ERR_BAD_TEMPERATURE;
    p->kind = t == 0.f ? kTreeGreedy : d->draft_kind == SV_DRAFT_ONEHOT ? kTreeOneHot : kTreeLogits;
    if (p->kind == kTreeLogits && (d->draft_rows < 1 || d->draft_rows > d->k + 1)) return SV_ERR_BAD_SHAPE;
    p->batch = d->B;
    p->k = d->k;
    p->vocab = d->V;
    p->draft_rows = p->kind == kTreeLogits ? d->draft_rows : 0;
    p->elem_bytes = d->dtype == SV_BF16 ? 2 : 4;
    p->c2 = t == 0.f ? 0.0 : kLog2E / static_cast<double>(t);
    p->per_c2 = t == 0.f ? 0.0 : static_cast<double>(t) / kLog2E;
    tree_slices(p->vocab, p->batch, kTreeWgs, &p->per, &p->slices);
    tree_slices(p->vocab, static_cast<int64_t>(p->batch) * (p->k + 1), kTreeRowWgs, &p->row_per, &p->row_slices);
    p->wait_ticks = tree_wait_ticks;
    return SV_OK;
}

size_t tree_state_bytes(int64_t batch) { return align_up(static_cast<size_t>(batch) * sizeof(TreeState)); }

// What one call leaves to the next (all 0) stands at the same place whatever
// the shape: words of another call's shape never lie there.
constexpr size_t kTreeCountBytes = (static_cast<size_t>(kTreeMaxBatch) * sizeof(uint32_t) + kAlign - 1) & ~(kAlign - 1);
constexpr size_t kTreeExchangeBytes = static_cast<size_t>(kTreeWgs) * 8 * sizeof(uint64_t);
constexpr size_t kTreeZeroBytes = 2 * kTreeCountBytes + kTreeExchangeBytes;

// Whether the statistics of every row are taken at once.
bool all_rows(const TreePlan& p) {
    const int64_t most = p.kind == kTreeGreedy ? kTreeAllRowsGreedy : kTreeAllRows;
    return p.kind != kTreeLogits && p.slices > 1 && static_cast<int64_t>(p.batch) * (p.k + 1) * p.vocab <= most;
}

size_t tree_bytes(const TreePlan& p) {
    size_t n = kTreeZeroBytes + tree_state_bytes(p.batch);
    if (all_rows(p))
        n += align_up(static_cast<size_t>(p.batch) * (p.k + 1) * kTreeMaxSlices * 2 * sizeof(double));
    return n;
}

sv_status plan_cache(const sv_cache_desc* d, CachePlan* p) {
    if (!d) return SV_ERR_NULL_ARG;
    const int shift = page_shift_of(d->page_size);
    if (d->n_seqs < 0 || d->n_seqs > kCacheMaxSeqs || d->n_pages < 1 || shift < 0 || d->max_pages < 1 ||
        d->n_layers < 1 || d->kv_heads < 1 || d->kv_heads > 1024 || d->head_dim < 8 || d->head_dim > 1024 ||
        d->head_dim % 8)
        return SV_ERR_BAD_SHAPE;
    if ((static_cast<int64_t>(d->max_pages) << shift) > (int64_t{1} << 30)) return SV_ERR_BAD_SHAPE;
    // positions in the cache are counted in 16-byte pieces in 63 bits
    if (static_cast<double>(d->n_pages) * d->n_layers * d->kv_heads * d->page_size * d->head_dim >= 4e18)
        return SV_ERR_BAD_SHAPE;
    if (d->dtype != SV_BF16 && d->dtype != SV_F16) return SV_ERR_BAD_DTYPE;
    p->n_seqs = d->n_seqs;
    p->n_pages = d->n_pages;
    p->page_shift = shift;
    p->max_pages = d->max_pages;
    p->n_layers = d->n_layers;
    p->kv_heads = d->kv_heads;
    p->head_dim = d->head_dim;
    return SV_OK;
}

sv_status check_cache_arrays(const void* k_cache, const void* v_cache) {
    if (!k_cache || !v_cache) return SV_ERR_NULL_ARG;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16)) return SV_ERR_MISALIGNED;
    if (k_cache == v_cache) return SV_ERR_ALIASED;
    return SV_OK;
}

sv_status launched(hipError_t e) { return e == hipSuccess ? SV_OK : SV_ERR_HIP; }

}  // namespace
}  // namespace sv

extern "C" {

size_t sv_tree_attention_workspace_bytes(const sv_tree_attention_desc* desc) {
    sv::AttnPlan p{};
    return sv::plan_attention(desc, &p) == SV_OK ? sv::attention_bytes(p) : 0;
}

sv_status sv_tree_attention(const sv_tree_attention_desc* desc, const void* q, const void* k_cache,
                            const void* v_cache, const int32_t* page_table, const int32_t* seq_len,
                            const int32_t* parents, void* out, float* lse_out, void* workspace,
                            size_t workspace_bytes, hipStream_t stream) {
    sv::AttnPlan p{};
    const sv_status st = sv::plan_attention(desc, &p);
    if (st != SV_OK) return st;
    if (p.batch == 0) return SV_OK;
    if (!q || !k_cache || !v_cache || !page_table || !seq_len || !out || !workspace) return SV_ERR_NULL_ARG;
    if (p.k > 0 && !parents) return SV_ERR_NULL_ARG;
    if (!sv::aligned(q, 16) || !sv::aligned(k_cache, 16) || !sv::aligned(v_cache, 16) || !sv::aligned(out, 16) ||
        !sv::aligned(workspace, 16))
        return SV_ERR_MISALIGNED;
    if (workspace_bytes < sv::attention_bytes(p)) return SV_ERR_WORKSPACE_TOO_SMALL;
    if (out == q) return SV_ERR_ALIASED;  // rows are written while workgroups with other keys still read them
    p.q = q;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.page_table = page_table;
    p.seq_len = seq_len;
    p.parents = parents;
    p.out = out;
    p.lse = lse_out;
    char* const base = static_cast<char*>(workspace);
    p.part_acc = reinterpret_cast<float*>(base);
    p.part_ml = reinterpret_cast<float*>(base + sv::attention_acc_bytes(p));
    p.splits = reinterpret_cast<sv::AttnSplit*>(base + sv::attention_acc_bytes(p) + sv::attention_ml_bytes(p));
    return sv::launched(sv::launch_tree_attention(p, stream));
}

// For tests of what follows a wait that ran out: the longest wait, in 10 ns.
void sv_internal_tree_wait(uint64_t ticks) { sv::tree_wait_ticks = ticks; }

size_t sv_verify_tree_workspace_bytes(const sv_verify_tree_desc* desc) {
    sv::TreePlan p{};
    return sv::plan_tree(desc, &p) == SV_OK ? sv::tree_bytes(p) : 0;
}

sv_status sv_verify_tree(const sv_verify_tree_desc* desc, const void* target_logits, const void* draft_logits,
                         const int32_t* draft_tokens, const int32_t* parents, const float* uniforms,
                         int32_t* accepted_len, int32_t* out_tokens, int32_t* path_out, void* workspace,
                         size_t workspace_bytes, hipStream_t stream) {
    sv::TreePlan p{};
    const sv_status st = sv::plan_tree(desc, &p);
    if (st != SV_OK) return st;
    if (p.batch == 0) return SV_OK;
    if (!target_logits || !draft_tokens || !parents || !accepted_len || !out_tokens || !path_out || !workspace)
        return SV_ERR_NULL_ARG;
    if (p.kind != sv::kTreeGreedy && !uniforms) return SV_ERR_NULL_ARG;
    if (p.kind == sv::kTreeLogits && !draft_logits) return SV_ERR_NULL_ARG;
    if (!sv::aligned(workspace, 64)) return SV_ERR_MISALIGNED;
    if (!sv::aligned(target_logits, p.elem_bytes) || (draft_logits && !sv::aligned(draft_logits, p.elem_bytes)))
        return SV_ERR_MISALIGNED;
    if (workspace_bytes < sv::tree_bytes(p)) return SV_ERR_WORKSPACE_TOO_SMALL;
    p.target = target_logits;
    p.draft = p.kind == sv::kTreeLogits ? draft_logits : nullptr;
    p.tokens = draft_tokens;
    p.parents = parents;
    p.uniforms = uniforms;
    p.accepted_len = accepted_len;
    p.out_tokens = out_tokens;
    p.path = path_out;
    char* base = static_cast<char*>(workspace);
    p.arrived = reinterpret_cast<uint32_t*>(base);
    p.finished = reinterpret_cast<uint32_t*>(base + sv::kTreeCountBytes);
    p.exchange = reinterpret_cast<uint64_t*>(base + 2 * sv::kTreeCountBytes);
    base += sv::kTreeZeroBytes;
    p.state = reinterpret_cast<sv::TreeState*>(base);
    p.row_part = sv::all_rows(p) ? reinterpret_cast<double*>(base + sv::tree_state_bytes(p.batch)) : nullptr;
    p.vec = static_cast<int64_t>(p.vocab) * p.elem_bytes % 16 == 0 && sv::aligned(target_logits, 16) &&
            (!p.draft || sv::aligned(p.draft, 16));
    return sv::launched(sv::launch_verify_tree(p, stream));
}

sv_status sv_cache_append(const sv_cache_desc* desc, const sv_cache_rows* rows, const void* k_new, const void* v_new,
                          const int32_t* count, const int32_t* page_table, const int32_t* seq_len, void* k_cache,
                          void* v_cache, hipStream_t stream) {
    if (!rows) return SV_ERR_NULL_ARG;
    sv::AppendPlan p{};
    sv_status st = sv::plan_cache(desc, &p.c);
    if (st != SV_OK) return st;
    if (rows->t < 0) return SV_ERR_BAD_SHAPE;
    if (!sv::stride_ok(rows->k_stride_b) || !sv::stride_ok(rows->k_stride_t) || !sv::stride_ok(rows->k_stride_h) ||
        !sv::stride_ok(rows->v_stride_b) || !sv::stride_ok(rows->v_stride_t) || !sv::stride_ok(rows->v_stride_h))
        return SV_ERR_MISALIGNED;
    if (p.c.n_seqs == 0 || rows->t == 0) return SV_OK;
    if (!k_new || !v_new || !page_table || !seq_len) return SV_ERR_NULL_ARG;
    st = sv::check_cache_arrays(k_cache, v_cache);
    if (st != SV_OK) return st;
    if (!sv::aligned(k_new, 16) || !sv::aligned(v_new, 16)) return SV_ERR_MISALIGNED;
    p.c.k_cache = k_cache;
    p.c.v_cache = v_cache;
    p.c.page_table = const_cast<int32_t*>(page_table);  // read only
    p.c.seq_len = const_cast<int32_t*>(seq_len);        // read only
    p.k_new = k_new;
    p.v_new = v_new;
    p.count = count;
    p.t = rows->t;
    p.k_stride_b = rows->k_stride_b;
    p.k_stride_t = rows->k_stride_t;
    p.k_stride_h = rows->k_stride_h;
    p.v_stride_b = rows->v_stride_b;
    p.v_stride_t = rows->v_stride_t;
    p.v_stride_h = rows->v_stride_h;
    return sv::launched(sv::launch_cache_append(p, stream));
}

sv_status sv_cache_commit(const sv_cache_desc* desc, int32_t k, const int32_t* path, const int32_t* accepted_len,
                          const int32_t* page_table, const int32_t* seq_len, int32_t* new_len, void* k_cache,
                          void* v_cache, hipStream_t stream) {
    sv::CommitPlan p{};
    sv_status st = sv::plan_cache(desc, &p.c);
    if (st != SV_OK) return st;
    if (k < 1 || k > SV_MAX_DRAFT) return SV_ERR_BAD_SHAPE;
    if (p.c.n_seqs == 0) return SV_OK;
    if (!path || !accepted_len || !page_table || !seq_len || !new_len) return SV_ERR_NULL_ARG;
    st = sv::check_cache_arrays(k_cache, v_cache);
    if (st != SV_OK) return st;
    if (new_len == seq_len) return SV_ERR_ALIASED;
    p.c.k_cache = k_cache;
    p.c.v_cache = v_cache;
    p.c.page_table = const_cast<int32_t*>(page_table);  // read only
    p.c.seq_len = const_cast<int32_t*>(seq_len);        // read only
    p.path = path;
    p.accepted_len = accepted_len;
    p.new_len = new_len;
    p.k = k;
    return sv::launched(sv::launch_cache_commit(p, stream));
}

size_t sv_cache_fork_workspace_bytes(const sv_cache_desc* desc, int32_t n) {
    sv::CachePlan c{};
    if (sv::plan_cache(desc, &c) != SV_OK || n < 0 || n > sv::kCacheMaxSeqs) return 0;
    const size_t bytes = 2 * sv::align_up(static_cast<size_t>(n) * sizeof(int32_t));
    return bytes < sv::kAlign ? sv::kAlign : bytes;
}

sv_status sv_cache_fork(const sv_cache_desc* desc, int32_t n, const int32_t* src, const int32_t* dst,
                        int32_t* page_table, int32_t* page_count, int32_t* page_refs, int32_t* seq_len,
                        void* k_cache, void* v_cache, int32_t* status, void* workspace, size_t workspace_bytes,
                        hipStream_t stream) {
    sv::ForkPlan p{};
    sv_status st = sv::plan_cache(desc, &p.c);
    if (st != SV_OK) return st;
    if (n < 0 || n > sv::kCacheMaxSeqs) return SV_ERR_BAD_SHAPE;
    if (n == 0) return SV_OK;
    if (!src || !dst || !page_table || !page_count || !page_refs || !seq_len || !workspace) return SV_ERR_NULL_ARG;
    st = sv::check_cache_arrays(k_cache, v_cache);
    if (st != SV_OK) return st;
    if (!sv::aligned(workspace, 4)) return SV_ERR_MISALIGNED;
    if (workspace_bytes < sv_cache_fork_workspace_bytes(desc, n)) return SV_ERR_WORKSPACE_TOO_SMALL;
    p.c.k_cache = k_cache;
    p.c.v_cache = v_cache;
    p.c.page_table = page_table;
    p.c.page_count = page_count;
    p.c.page_refs = page_refs;
    p.c.seq_len = seq_len;
    p.src = src;
    p.dst = dst;
    p.status = status;
    char* base = static_cast<char*>(workspace);
    p.new_page = reinterpret_cast<int32_t*>(base);
    p.old_page = reinterpret_cast<int32_t*>(base + sv::align_up(static_cast<size_t>(n) * sizeof(int32_t)));
    p.n = n;
    return sv::launched(sv::launch_cache_fork(p, stream));
}

sv_status sv_cache_resize(const sv_cache_desc* desc, const int32_t* want_len, int32_t* page_table,
                          int32_t* page_count, int32_t* page_refs, int32_t* status, hipStream_t stream) {
    sv::CachePlan c{};
    const sv_status st = sv::plan_cache(desc, &c);
    if (st != SV_OK) return st;
    if (c.n_seqs == 0) return SV_OK;
    if (!want_len || !page_table || !page_count || !page_refs) return SV_ERR_NULL_ARG;
    c.page_table = page_table;
    c.page_count = page_count;
    c.page_refs = page_refs;
    return sv::launched(sv::launch_cache_resize(c, want_len, status, stream));
}

}  // extern "C"
