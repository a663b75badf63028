// gfx950 kernels of the paged key/value cache: rows appended behind a
// sequence, an accepted branch moved to the front of a tree's rows, sequences
// forked, pages allotted and given back.
//
// All of them move bytes or count references; nothing is computed.  Rows are
// moved in 16-byte pieces with consecutive lanes on consecutive pieces.  A
// page is free when nothing refers to it (page_refs 0); pages are given out
// lowest number first, and reference counts are changed with integer atomics,
// so the outcome does not depend on any order of execution.
//
// Measured (bf16 or f16, 8 key heads of 128): appending 16 x 4096 rows moves
// 349 MB in 67 to 72 us, 4.9 to 5.2 TB/s read and written, as fast as a plain
// copy (4.76).  Moving the accepted rows of 128 sequences in 32 layers, 77 MB in
// pieces of 256 bytes, takes 24 us (3.2 TB/s).  Copying the 112 begun pages of
// 16 sequences forked seven times, 32 layers, 1.2 GB, takes 218 to 250 us by the
// card (4.8 to 5.5 TB/s).  The bookkeeping is one workgroup's, a thread to a
// sequence and its ranks and counts in LDS: 5 us a fork of 3 and 4 a resize, 11
// and 10 with 128 sequences (17 and 15 with a wavefront to a sequence from the
// start, and 24 a fork of 3 through memory with fences).  Calls that move less
// are bound by their launch.
#include <hip/hip_runtime.h>

#include <climits>
#include <cstdint>

#include "specverify.h"
#include "sv_tree.h"

namespace sv {
namespace {

constexpr int kCopyThreads = 256;
constexpr int kBookThreads = 1024;  // the page bookkeeping runs in one workgroup
constexpr int kBookWaves = kBookThreads / 64;

// A barrier that the bookkeeping workgroup's stores and counts have passed:
// they have reached the L2 that fresh() reads from.
__device__ __forceinline__ void settle() {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
}

// A value that other threads of the workgroup may have changed, past the
// compute unit's own cache.
__device__ __forceinline__ int fresh(const int32_t* x) {
    return __hip_atomic_load(x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Row of the cache (in units of head_dim) that position pos of sequence b has
// under key head 0, or -1 (no page, or a page number out of range).
__device__ __forceinline__ int64_t cache_row(const CachePlan& c, int b, int64_t pos) {
    const int64_t slot = pos >> c.page_shift;
    if (pos < 0 || slot >= c.max_pages) return -1;
    const int id = c.page_table[static_cast<int64_t>(b) * c.max_pages + slot];
    if (id < 0 || id >= c.n_pages) return -1;
    return ((static_cast<int64_t>(id) * c.kv_heads) << c.page_shift) + (pos & ((1 << c.page_shift) - 1));
}

__global__ __launch_bounds__(kCopyThreads) void k_cache_append(AppendPlan p) {
    const int b = blockIdx.y;
    const int len = p.c.seq_len[b];
    if (len < 0) return;
    int n = p.t;
    if (p.count) n = min(max(p.count[b], 0), p.t);
    const int pieces = p.c.head_dim / 8;
    const int per_row = p.c.kv_heads * pieces;
    const int64_t items = static_cast<int64_t>(n) * per_row;
    const uint4* const ks = static_cast<const uint4*>(p.k_new);
    const uint4* const vs = static_cast<const uint4*>(p.v_new);
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kCopyThreads + threadIdx.x; i < items;
         i += static_cast<int64_t>(gridDim.x) * kCopyThreads) {
        const int j = static_cast<int>(i / per_row);
        const int e = static_cast<int>(i - static_cast<int64_t>(j) * per_row);
        const int h = e / pieces, c = e - h * pieces;
        const int64_t row = cache_row(p.c, b, static_cast<int64_t>(len) + j);
        if (row < 0) continue;
        const int64_t to = (row + (static_cast<int64_t>(h) << p.c.page_shift)) * pieces + c;
        static_cast<uint4*>(p.c.k_cache)[to] = ks[(b * p.k_stride_b + j * p.k_stride_t + h * p.k_stride_h) / 8 + c];
        static_cast<uint4*>(p.c.v_cache)[to] = vs[(b * p.v_stride_b + j * p.v_stride_t + h * p.v_stride_h) / 8 + c];
    }
}

// Rows len + 1 + path[j] become rows len + 1 + j, in place.  path is
// increasing, so path[j] >= j and a row is overwritten only by a later or the
// same node's: a thread that takes one piece of every row in ascending order
// never overwrites what it has yet to read.  Eight rows are read before they
// are written, which keeps eight loads in flight.
__global__ __launch_bounds__(kCopyThreads) void k_cache_commit(CommitPlan p) {
    __shared__ int64_t from[SV_MAX_DRAFT], to[SV_MAX_DRAFT];
    __shared__ int moves;
    const int b = blockIdx.y;
    const int len = p.c.seq_len[b];
    if (threadIdx.x < 64) {
        const int lane = threadIdx.x;
        int acc = p.accepted_len[b];
        const bool in = lane < min(acc, p.k);
        const int node = in ? p.path[static_cast<int64_t>(b) * p.k + lane] : lane;
        const int prev = __shfl_up(node, 1);
        const bool bad = in && (node < lane || node >= p.k || (lane > 0 && node <= prev));
        // an unusable path, a refused sequence: nothing moves, the length stays
        if (__any(bad) || acc > p.k || len < 0) acc = -1;
        int64_t f = -1, t = -1;
        if (in && acc >= 0 && node != lane) {
            f = cache_row(p.c, b, static_cast<int64_t>(len) + 1 + node);
            t = cache_row(p.c, b, static_cast<int64_t>(len) + 1 + lane);
        }
        const bool move = f >= 0 && t >= 0;
        const uint64_t all = __ballot(move);
        if (move) {
            const int at = __popcll(all & ((uint64_t{1} << lane) - 1));
            from[at] = f;
            to[at] = t;
        }
        if (lane == 0) {
            moves = __popcll(all);
            if (blockIdx.x == 0) p.new_len[b] = acc < 0 ? len : len + 1 + acc;
        }
    }
    __syncthreads();
    const int n = moves;
    if (n == 0) return;
    const int pieces = p.c.head_dim / 8;
    const int per_layer = p.c.kv_heads * pieces;
    const int64_t layer = (static_cast<int64_t>(p.c.n_pages) * p.c.kv_heads << p.c.page_shift) * pieces;
    const int64_t items = static_cast<int64_t>(p.c.n_layers) * 2 * per_layer;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kCopyThreads + threadIdx.x; i < items;
         i += static_cast<int64_t>(gridDim.x) * kCopyThreads) {
        const int l = static_cast<int>(i / (2 * per_layer));
        int e = static_cast<int>(i - static_cast<int64_t>(l) * 2 * per_layer);
        uint4* base = static_cast<uint4*>(e < per_layer ? p.c.k_cache : p.c.v_cache) + l * layer;
        if (e >= per_layer) e -= per_layer;
        const int h = e / pieces, c = e - h * pieces;
        base += (static_cast<int64_t>(h) << p.c.page_shift) * pieces + c;
        for (int j = 0; j < n; j += 8) {
            uint4 x[8];
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (j + q < n) x[q] = base[from[j + q] * pieces];
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (j + q < n) base[to[j + q] * pieces] = x[q];
        }
    }
}

// Inclusive sum over the bookkeeping workgroup, and the total.
template <typename N>
__device__ __forceinline__ N book_scan(N v, N* total, N* tmp) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const N o = __shfl_up(v, d);
        if (lane >= d) v += o;
    }
    __syncthreads();
    if (lane == 63) tmp[wave] = v;
    __syncthreads();
    N all = 0;
#pragma unroll
    for (int w = 0; w < kBookWaves; ++w) {
        if (w < wave) v += tmp[w];
        all += tmp[w];
    }
    *total = all;
    return v;
}

// Calls give(rank, page) for the free pages of rank 0 .. need - 1 in ascending
// order of their numbers; returns how many there were.
template <typename Give>
__device__ __forceinline__ int free_pages(const CachePlan& c, int need, int* tmp, const Give& give) {
    constexpr int PER = 4;
    int found = 0;
    for (int64_t base = 0; base < c.n_pages && found < need; base += kBookThreads * PER) {
        const int64_t i = base + threadIdx.x * PER;
        int free_mask = 0;
#pragma unroll
        for (int j = 0; j < PER; ++j)
            if (i + j < c.n_pages && fresh(&c.page_refs[i + j]) == 0) free_mask |= 1 << j;
        const int mine = __popc(free_mask);
        int all;
        int rank = found + book_scan(mine, &all, tmp) - mine;
#pragma unroll
        for (int j = 0; j < PER; ++j)
            if ((free_mask >> j) & 1) {
                if (rank < need) give(rank, static_cast<int>(i + j));
                ++rank;
            }
        found += all;
    }
    return min(found, need);
}

__global__ __launch_bounds__(kBookThreads) void k_cache_resize(CachePlan c, const int32_t* want, int32_t* status) {
    // Pages asked for by the sequences up to and including this one; together
    // they may ask for more than 2^31.
    __shared__ int64_t ends[kCacheMaxSeqs];
    __shared__ int64_t wide[kBookWaves];
    __shared__ int tmp[kBookWaves];
    __shared__ int cut;  // the sequence whose wish the last free page falls into
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t page = int64_t{1} << c.page_shift;
    // A count or a wish that the table cannot hold is refused; the others are
    // the pages a sequence is to have.
    const auto target = [&](int b, int have) -> int64_t {
        const int64_t w = want[b];
        if (have < 0 || have > c.max_pages) return -1;
        const int64_t t = w < 0 ? have : (w + page - 1) >> c.page_shift;
        return t > c.max_pages ? -1 : t;
    };
    // Shorter ones give back the pages behind their new end.  A thread to a
    // sequence for what it has and wants, a wavefront to one that gives back.
    if (threadIdx.x == 0) cut = -1;
    for (int b = threadIdx.x; b < c.n_seqs; b += kBookThreads) {
        const int have = c.page_count[b];
        const int64_t t = target(b, have);
        const bool less = t >= 0 && t < have;
        ends[b] = less ? static_cast<int64_t>(have) << 32 | t : -1;
        if (less) c.page_count[b] = static_cast<int>(t);
    }
    __syncthreads();
    for (int b = wave; b < c.n_seqs; b += kBookWaves) {
        if (ends[b] < 0) continue;
        const int64_t have = ends[b] >> 32, t = ends[b] & 0xFFFFFFFF;
        int32_t* const row = c.page_table + static_cast<int64_t>(b) * c.max_pages;
        for (int64_t i = t + lane; i < have; i += 64) {
            const int id = row[i];
            if (id >= 0 && id < c.n_pages) atomicSub(&c.page_refs[id], 1);
            row[i] = -1;
        }
    }
    settle();
    int64_t need = 0;
    for (int base = 0; base < c.n_seqs; base += kBookThreads) {
        const int b = base + threadIdx.x;
        int64_t more = 0;
        if (b < c.n_seqs) {
            const int have = fresh(&c.page_count[b]);
            const int64_t t = target(b, have);
            more = t > have ? t - have : 0;
            if (status) status[b] = t >= 0;
        }
        int64_t all;
        const int64_t incl = book_scan(more, &all, wide);
        if (b < c.n_seqs) ends[b] = need + incl;
        need += all;
    }
    __syncthreads();
    if (need == 0) return;
    const auto begin_of = [&](int b) -> int64_t { return b ? ends[b - 1] : 0; };
    const int found = free_pages(c, static_cast<int>(min(need, static_cast<int64_t>(c.n_pages))), tmp, [&](int rank, int id) {
        int lo = 0, hi = c.n_seqs - 1;  // the first sequence whose end is past this rank
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (ends[mid] > rank) hi = mid;
            else lo = mid + 1;
        }
        c.page_table[static_cast<int64_t>(lo) * c.max_pages + fresh(&c.page_count[lo]) + rank - begin_of(lo)] = id;
        c.page_refs[id] = 1;
    });
    settle();
    // Served are the sequences whose whole wish lies before the last free
    // page; the one that it falls into gives its part back.
    for (int b = threadIdx.x; b < c.n_seqs; b += kBookThreads) {
        const int64_t lo = begin_of(b), hi = ends[b];
        if (lo == hi) continue;
        if (hi <= found) {
            c.page_count[b] = static_cast<int>(fresh(&c.page_count[b]) + hi - lo);
            continue;
        }
        if (status) status[b] = 0;
        if (lo < found) cut = b;
    }
    __syncthreads();
    if (cut < 0) return;
    int32_t* const row = c.page_table + static_cast<int64_t>(cut) * c.max_pages + fresh(&c.page_count[cut]);
    for (int i = threadIdx.x; i < static_cast<int>(found - begin_of(cut)); i += kBookThreads) {
        c.page_refs[fresh(&row[i])] = 0;
        row[i] = -1;
    }
}

// The pairs' claims, ranks and pages stay in LDS; only the copy list goes to
// memory.  new_page of a pair: first the rank of its copy among all copies,
// then the page (-1: nothing to copy, -2: the pair is refused).
__global__ __launch_bounds__(kBookThreads) void k_cache_fork(ForkPlan p) {
    __shared__ int claim[kCacheMaxSeqs];     // the first pair that names the sequence as its destination
    __shared__ int new_page[kCacheMaxSeqs];
    __shared__ int pair_of[kCacheMaxSeqs];   // the pair of each rank
    __shared__ int tmp[kBookWaves];
    const CachePlan& c = p.c;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int page_mask = (1 << c.page_shift) - 1;
    const auto in_range = [&](int s) { return s >= 0 && s < c.n_seqs; };
    for (int i = threadIdx.x; i < c.n_seqs; i += kBookThreads) claim[i] = INT_MAX;
    __syncthreads();
    for (int i = threadIdx.x; i < p.n; i += kBookThreads)
        if (in_range(p.dst[i])) atomicMin(&claim[p.dst[i]], i);
    __syncthreads();
    int need = 0;
    for (int base = 0; base < p.n; base += kBookThreads) {
        const int i = base + threadIdx.x;
        bool ok = false;
        int len = 0;
        if (i < p.n) {
            const int s = p.src[i], d = p.dst[i];
            // a source that is a destination too would be read while it is written
            if (in_range(s) && in_range(d) && claim[d] == i && claim[s] == INT_MAX) {
                len = c.seq_len[s];
                const int have = c.page_count[s];
                ok = c.page_count[d] == 0 && len >= 0 && have >= 0 && have <= c.max_pages &&
                     ((static_cast<int64_t>(len) + page_mask) >> c.page_shift) <= have;
            }
        }
        const int more = ok && (len & page_mask) != 0;
        int all;
        const int incl = book_scan(more, &all, tmp);
        if (i < p.n) {
            new_page[i] = ok ? (more ? need + incl - 1 : -1) : -2;
            if (more) pair_of[need + incl - 1] = i;
        }
        need += all;
    }
    __syncthreads();
    const int found = free_pages(c, need, tmp, [&](int rank, int id) {
        new_page[pair_of[rank]] = id;
        c.page_refs[id] = 1;
    });
    __syncthreads();
    for (int r = found + threadIdx.x; r < need; r += kBookThreads) new_page[pair_of[r]] = -2;  // none left
    __syncthreads();
    // A thread to a pair for the counts and the begun page, a wavefront for the
    // whole pages: what it needs stays where the claims and ranks were.
    for (int i = threadIdx.x; i < p.n; i += kBookThreads) {
        const int id = new_page[i];
        p.new_page[i] = id;
        if (p.status) p.status[i] = id != -2;
        int old = -1, whole = -1;
        if (id != -2) {
            const int s = p.src[i], d = p.dst[i], len = c.seq_len[s];
            whole = len >> c.page_shift;
            if (id >= 0) {
                old = c.page_table[static_cast<int64_t>(s) * c.max_pages + whole];
                c.page_table[static_cast<int64_t>(d) * c.max_pages + whole] = id;
            }
            c.page_count[d] = whole + (id >= 0);
            c.seq_len[d] = len;
            claim[i] = s;
            pair_of[i] = d;
        }
        p.old_page[i] = old;
        new_page[i] = whole;
    }
    __syncthreads();
    for (int i = wave; i < p.n; i += kBookWaves) {
        const int whole = new_page[i];
        if (whole <= 0) continue;
        const int32_t* const from = c.page_table + static_cast<int64_t>(claim[i]) * c.max_pages;
        int32_t* const to = c.page_table + static_cast<int64_t>(pair_of[i]) * c.max_pages;
        for (int q = lane; q < whole; q += 64) {
            const int x = from[q];
            to[q] = x;
            if (x >= 0 && x < c.n_pages) atomicAdd(&c.page_refs[x], 1);
        }
    }
}

// Begun pages are copied whole, every layer's keys and values.
__global__ __launch_bounds__(kCopyThreads) void k_cache_copy_pages(ForkPlan p) {
    const CachePlan& c = p.c;
    const int i = blockIdx.y;
    const int from = p.old_page[i], to = p.new_page[i];
    if (from < 0 || from >= c.n_pages || to < 0) return;
    const int64_t pieces = (static_cast<int64_t>(c.kv_heads) << c.page_shift) * (c.head_dim / 8);
    const int64_t items = pieces * 2 * c.n_layers;
    for (int64_t e = static_cast<int64_t>(blockIdx.x) * kCopyThreads + threadIdx.x; e < items;
         e += static_cast<int64_t>(gridDim.x) * kCopyThreads) {
        const int64_t half = e / pieces, at = e - half * pieces;
        uint4* const base = static_cast<uint4*>(half & 1 ? c.v_cache : c.k_cache) + (half >> 1) * c.n_pages * pieces;
        base[to * pieces + at] = base[from * pieces + at];
    }
}

uint32_t blocks_for(int64_t items, int64_t most) {
    const int64_t n = (items + kCopyThreads - 1) / kCopyThreads;
    return static_cast<uint32_t>(n < 1 ? 1 : n < most ? n : most);
}

}  // namespace

hipError_t launch_cache_append(const AppendPlan& p, hipStream_t stream) {
    const int64_t items = static_cast<int64_t>(p.t) * p.c.kv_heads * (p.c.head_dim / 8);
    k_cache_append<<<dim3(blocks_for(items, 4096), p.c.n_seqs), kCopyThreads, 0, stream>>>(p);
    return hipGetLastError();
}

hipError_t launch_cache_commit(const CommitPlan& p, hipStream_t stream) {
    const int64_t items = static_cast<int64_t>(p.c.n_layers) * 2 * p.c.kv_heads * (p.c.head_dim / 8);
    k_cache_commit<<<dim3(blocks_for(items, 4096), p.c.n_seqs), kCopyThreads, 0, stream>>>(p);
    return hipGetLastError();
}

hipError_t launch_cache_fork(const ForkPlan& p, hipStream_t stream) {
    k_cache_fork<<<1, kBookThreads, 0, stream>>>(p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t items =
        (static_cast<int64_t>(p.c.kv_heads) << p.c.page_shift) * (p.c.head_dim / 8) * 2 * p.c.n_layers;
    k_cache_copy_pages<<<dim3(blocks_for(items, 1024), p.n), kCopyThreads, 0, stream>>>(p);
    return hipGetLastError();
}

hipError_t launch_cache_resize(const CachePlan& p, const int32_t* want_len, int32_t* status, hipStream_t stream) {
    k_cache_resize<<<1, kBookThreads, 0, stream>>>(p, want_len, status);
    return hipGetLastError();
}

}  // namespace sv
