// Internal interface between the C-ABI layer of the tree-drafting operators
// (sv_tree_api.cpp) and their gfx950 kernels (sv_tree_attn.hip,
// sv_tree_verify.hip, sv_cache.hip).  Not installed; not part of the public ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

namespace sv {

// ---- attention of a tree over the paged cache --------------------------------

// Workgroups of the attention kernel: two for each of the 256 compute units,
// so that one's loads go on while the other starts or ends a run of keys.
constexpr int kAttnWgs = 512;
constexpr int kAttnDies = 8;
constexpr int kAttnStep = 32;  // keys one wavefront takes per step

// Wavefronts per workgroup and row tiles of 16 query rows per workgroup: what
// the staging buffers (160 KiB of LDS for two workgroups) and the accumulators
// (512 registers a lane) hold.
constexpr int attn_waves(int head_dim) { return head_dim > 128 ? 1 : head_dim > 64 ? 2 : 4; }
constexpr int attn_max_row_tiles(int head_dim) { return head_dim > 128 ? 2 : 4; }

// A (sequence, key head) whose keys several clusters share, seen from the
// first of them; k_tree_combine joins their partial results.
struct AttnSplit {
    int32_t b;      // -1: none starts here
    int32_t head;   // key head
    int32_t last;   // the last cluster that has part of it
    int32_t slot1;  // the first cluster's part is in its second slot
};

struct AttnPlan {
    const void* q;
    const void* k_cache;
    const void* v_cache;
    const int32_t* page_table;
    const int32_t* seq_len;
    const int32_t* parents;  // NULL when k == 0
    void* out;
    float* lse;              // may be NULL
    float* part_acc;         // [clusters][row_units][2 slots][row_tiles * 16][head_dim]
    float* part_ml;          // the same [..][2]
    AttnSplit* splits;       // [clusters][row_units]
    int64_t q_stride_b, q_stride_r, q_stride_h;
    int32_t batch;
    int32_t k;
    int32_t q_heads, kv_heads, head_dim;
    int32_t group;           // q_heads / kv_heads
    int32_t rows;            // (k + 1) * group: query rows of one key head
    int32_t row_tiles;       // 16-row tiles of one unit, 1 .. attn_max_row_tiles
    int32_t row_units;       // units that share one key head's rows
    int32_t cluster;         // workgroups that take the same keys, a unit (or several, in turn) each
    int32_t clusters;
    int32_t n_pages, page_shift, max_pages;
    int32_t is_f16;
    float scale_log2;        // scale * log2(e)
};

hipError_t launch_tree_attention(const AttnPlan& p, hipStream_t stream);

// ---- verification of a tree ---------------------------------------------------

constexpr int kTreeThreads = 256;
constexpr int kTreeMaxSlices = 64;
constexpr int kTreeMaxBatch = 65535;
constexpr int kTreeWgs = 1024;   // workgroups of a walk's pass: as many as run at once
// Workgroups that read every row at once, about: as many as run at once.  8 x 17
// rows of 151936: 39 us with 1024, 42 with 1536, 44 with 2048.
constexpr int kTreeRowWgs = 1024;
constexpr int kTreeDies = 8;
constexpr uint64_t kTreeWaitTicks = 2000000;  // of 10 ns: how long a workgroup waits for the others of its sequence
constexpr int kTreeTile = kTreeThreads * 8;  // tokens one workgroup takes at a time
// Logits up to which every row is read at once (one-hot children, and greedy
// walks, which read twice as fast): rows of 151936, k = 16, 8 sequences (20 Mi)
// take 35 us at once against 41 row by row, 16 take 62 against 41; greedy walks
// of 16 (39 Mi) 25 against 36, of 32 (79 Mi) 43 against 40.
constexpr int64_t kTreeAllRows = int64_t{24} << 20;
constexpr int64_t kTreeAllRowsGreedy = int64_t{64} << 20;

enum TreeKind : int32_t { kTreeGreedy = 0, kTreeOneHot = 1, kTreeLogits = 2 };

// One sequence's walk between two passes (workspace, 64-byte aligned).
struct TreeState {
    double m_t, z_t;     // target row of `at`: whole power of two m >= max l c2, sum of 2^(l c2 - m)
    double m_q, z_q;     // its draft row
    double t, f;         // residual max(0, p - t q) and its mass F(t)
    int32_t at;          // node whose children are tested, -1 the root
    int32_t stage;       // what the next pass computes (TreeStage)
    uint64_t left;       // children of `at` not yet tested
    int32_t kept;        // nodes accepted so far
    int32_t pad[7];
};

struct TreePlan {
    const void* target;          // [B][k+1][V]
    const void* draft;           // [B][draft_rows][V] or NULL
    const int32_t* tokens;       // [B][k]
    const int32_t* parents;      // [B][k]
    const float* uniforms;       // [B][k+1] or NULL
    int32_t* accepted_len;
    int32_t* out_tokens;
    int32_t* path;
    // Left at 0 by every call, at the same place whatever its shape:
    uint32_t* arrived;           // [kTreeMaxBatch]: workgroups that have handed in a row's partial
    uint32_t* finished;          // [kTreeMaxBatch]: the sequence's outputs are written
    uint64_t* exchange;          // [kTreeWgs][2][4]: partials of a walk's passes, tagged
    // Written by a call before it is read:
    TreeState* state;            // [B]
    double* row_part;            // [B][k+1][kTreeMaxSlices][2]: every row's, or NULL (rows read as the walk comes to them)
    int64_t per, row_per;        // tokens of one slice: of a pass, and where every row is read at once
    int32_t slices, row_slices;  // workgroups on one row
    int32_t batch, k, vocab, draft_rows;
    int32_t kind;                // TreeKind
    int32_t elem_bytes;          // 4 fp32, 2 bf16
    int32_t vec;                 // rows start on 16-byte boundaries
    uint64_t wait_ticks;
    double c2, per_c2;           // log2(e) / T and one over it (0 and 0 for greedy walks)
};

hipError_t launch_verify_tree(const TreePlan& p, hipStream_t stream);

// ---- pages of the cache --------------------------------------------------------

constexpr int kCacheMaxSeqs = 4096;  // what one workgroup's LDS holds in sv_cache_resize and sv_cache_fork

struct CachePlan {
    void* k_cache;
    void* v_cache;
    int32_t* page_table;     // [n_seqs][max_pages]
    int32_t* page_count;     // [n_seqs]
    int32_t* page_refs;      // [n_pages]
    int32_t* seq_len;        // [n_seqs]
    int32_t n_seqs, n_pages, page_shift, max_pages, n_layers, kv_heads, head_dim;
};

struct AppendPlan {
    CachePlan c;             // page_count, page_refs unused; one layer
    const void* k_new;
    const void* v_new;
    const int32_t* count;    // [n_seqs] or NULL
    int64_t k_stride_b, k_stride_t, k_stride_h, v_stride_b, v_stride_t, v_stride_h;
    int32_t t;
};

struct CommitPlan {
    CachePlan c;
    const int32_t* path;
    const int32_t* accepted_len;
    int32_t* new_len;
    int32_t k;
};

struct ForkPlan {
    CachePlan c;
    const int32_t* src;
    const int32_t* dst;
    int32_t* status;
    int32_t* new_page;       // workspace: [n]
    int32_t* old_page;       // workspace: [n]
    int32_t n;
};

hipError_t launch_cache_append(const AppendPlan& p, hipStream_t stream);
hipError_t launch_cache_commit(const CommitPlan& p, hipStream_t stream);
hipError_t launch_cache_fork(const ForkPlan& p, hipStream_t stream);
hipError_t launch_cache_resize(const CachePlan& p, const int32_t* want_len, int32_t* status, hipStream_t stream);

}  // namespace sv
