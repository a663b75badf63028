// gfx950 kernels of sv_verify_tree: the lossless walk down a drafted tree.
//
// Mathematics.  At a node (first the root) let p be the target's distribution
// there and c_1, c_2, ... its children in index order.
//   Greedy (T = 0): the child whose token is p's lowest argmax is kept.
//   One-hot children: c_j is kept iff u_j (1 - sum of p over the distinct
//     earlier siblings' tokens) < p(x_j), a token drafted again is never kept;
//     the draw is from p without the siblings' tokens.
//   Children drawn independently from the draft row's q: the target for child
//     j+1 is the residual r_j ~ max(0, r_{j-1} - q) with r_0 = p.  All of them
//     lie on one line, r_j = max(0, p - t_j q) / F(t_j), F(t) = sum_y max(0,
//     p(y) - t q(y)), t_0 = 0, F(0) = 1, t_{j+1} = t_j + F(t_j): with s =
//     1 / F(t), max(0, s max(0, p - t q) - q) = s max(0, p - (t + F(t)) q).
//     So child j is kept iff u_j F(t) q(x_j) < max(0, p(x_j) - t q(x_j)), and
//     one rejection costs one sum over the row.
//   A kept child is the next node; where none is kept, one token is drawn from
//   what is left (p itself at a leaf) by inverting its cumulative sum with the
//   sequence's last uniform: the smallest y with C(y) > u C(V-1).
//
// Arithmetic is 64-bit: with 10^5 tokens of similar mass a relative error of
// 1e-7 in a cumulative sum moves about one draw in a hundred to another token.
// 2^f is a polynomial of degree 8 (Chebyshev nodes on [-1/2, 1/2], relative
// error 1.1e-12); 64-bit multiply-adds run at the rate of 32-bit ones here.
//
// Only the rows on the walked path are read.
#include <hip/hip_runtime.h>

#include <climits>
#include <cstdint>

#include "specverify.h"
#include "sv_tree.h"

namespace sv {
namespace {

constexpr int NT = kTreeThreads;
constexpr int NWAVES = NT / 64;

enum TreeStage : int32_t {
    kStageRow = 0,   // the statistics of the row of `at`
    kStageMass = 1,  // F(t) on the row of `at`
    kStageDone = 2
};

// 2^y for y <= 0 (0 below 2^-1000, so that a logit of -inf has no mass).
__device__ __forceinline__ double exp2_neg(double y) {
    const double magic = 6755399441055744.0;  // 1.5 * 2^52: the low word holds the rounded y
    const double yc = __builtin_fmax(y, -1000.0);
    const double s = yc + magic;
    const double f = yc - (s - magic);
    double r = 1.3255224884799127e-06;
    r = __builtin_fma(r, f, 1.5310079402383103e-05);
    r = __builtin_fma(r, f, 0.00015403455852419016);
    r = __builtin_fma(r, f, 0.0013333450568000008);
    r = __builtin_fma(r, f, 0.00961812915940262);
    r = __builtin_fma(r, f, 0.05550410941205934);
    r = __builtin_fma(r, f, 0.2402265069581299);
    r = __builtin_fma(r, f, 0.6931471805459335);
    r = __builtin_fma(r, f, 1.0);
    const int n = __double2loint(s);
    const double v = __hiloint2double(__double2hiint(r) + static_cast<int>(static_cast<unsigned>(n) << 20), __double2loint(r));
    return y >= -1000.0 ? v : 0.0;
}

template <typename T>
__device__ __forceinline__ float value(T x);
template <>
__device__ __forceinline__ float value<float>(float x) {
    return x;
}
template <>
__device__ __forceinline__ float value<uint16_t>(uint16_t x) {
    return __int_as_float(static_cast<int>(x) << 16);
}

constexpr int kPer = 8;  // consecutive elements of one thread and tile

// Elements [i, i + kPer) of a row, -inf from `end` on.  Rows that do not start
// on 16-byte boundaries (V not a multiple of 16 bytes) are read one by one.
template <typename T>
__device__ __forceinline__ void load8(const T* row, int64_t i, int64_t end, bool vec, float (&x)[kPer]) {
    if (vec && i + kPer <= end) {
        T raw[kPer];
#pragma unroll
        for (int j = 0; j < static_cast<int>(kPer * sizeof(T) / 16); ++j)
            reinterpret_cast<uint4*>(raw)[j] = reinterpret_cast<const uint4*>(row + i)[j];
#pragma unroll
        for (int j = 0; j < kPer; ++j) x[j] = value<T>(raw[j]);
    } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j) x[j] = i + j < end ? value<T>(row[i + j]) : -__builtin_inff();
    }
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
    return v;
}

struct Shared {
    double wave_a[NWAVES], wave_b[NWAVES];
    float wave_f[NWAVES];
    int wave_i[NWAVES];
    double bcast[8];
    int ibcast[8];
    int gone[SV_MAX_DRAFT];  // one-hot: the rejected siblings' tokens
    int n_gone;
    TreeState st;
};

// Sum over the workgroup, on every thread, in a fixed order.
__device__ __forceinline__ double block_sum(double v, double* tmp) {
    v = wave_sum(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = v;
    __syncthreads();
    double s = 0.0;
#pragma unroll
    for (int w = 0; w < NWAVES; ++w) s += tmp[w];
    return s;
}

__device__ __forceinline__ float block_max(float v, float* tmp) {
    v = wave_max(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = tmp[0];
#pragma unroll
    for (int w = 1; w < NWAVES; ++w) s = fmaxf(s, tmp[w]);
    return s;
}

// (maximum, lowest index) of a slice.
template <typename T>
__device__ void slice_argmax(const T* row, int64_t lo, int64_t hi, bool vec, Shared& sh, float* best, int* where) {
    float m = -__builtin_inff();
    int at = INT_MAX;
    for (int64_t i = lo + threadIdx.x * kPer; i < hi; i += NT * kPer) {
        float x[kPer];
        load8(row, i, hi, vec, x);
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (i + j < hi && (x[j] > m || at == INT_MAX)) {
                m = x[j];
                at = static_cast<int>(i + j);
            }
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        const float om = __shfl_xor(m, d);
        const int oa = __shfl_xor(at, d);
        if (om > m || (om == m && oa < at)) {
            m = om;
            at = oa;
        }
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 0) {
        sh.wave_f[threadIdx.x >> 6] = m;
        sh.wave_i[threadIdx.x >> 6] = at;
    }
    __syncthreads();
    m = sh.wave_f[0];
    at = sh.wave_i[0];
    for (int w = 1; w < NWAVES; ++w)
        if (sh.wave_f[w] > m || (sh.wave_f[w] == m && sh.wave_i[w] < at)) {
            m = sh.wave_f[w];
            at = sh.wave_i[w];
        }
    *best = m;
    *where = at;
}

// (maximum of l c2, sum of 2^(l c2 - maximum)) of a slice.
template <typename T>
__device__ void slice_stats(const T* row, int64_t lo, int64_t hi, bool vec, double c2, Shared& sh, double* m_out,
                            double* z_out) {
    float m = -__builtin_inff();
    for (int64_t i = lo + threadIdx.x * kPer; i < hi; i += NT * kPer) {
        float x[kPer];
        load8(row, i, hi, vec, x);
#pragma unroll
        for (int j = 0; j < kPer; ++j) m = fmaxf(m, x[j]);
    }
    m = block_max(m, sh.wave_f);
    const double mc = static_cast<double>(m) * c2;
    double z = 0.0;
    for (int64_t i = lo + threadIdx.x * kPer; i < hi; i += NT * kPer) {
        float x[kPer];
        load8(row, i, hi, vec, x);
#pragma unroll
        for (int j = 0; j < kPer; ++j) z += exp2_neg(__builtin_fma(static_cast<double>(x[j]), c2, -mc));
    }
    z = block_sum(z, sh.wave_a);
    *m_out = mc;
    *z_out = m == -__builtin_inff() ? 0.0 : z;
}

// Mass of one token: max(0, p - t q), or p where t is 0 (q is not read).
__device__ __forceinline__ double mass_of(double lt, double lq, const TreeState& s, double iz_t, double iz_q, double c2,
                                          bool pair) {
    const double p = exp2_neg(__builtin_fma(lt, c2, -s.m_t)) * iz_t;
    if (!pair) return p;
    const double q = exp2_neg(__builtin_fma(lq, c2, -s.m_q)) * iz_q;
    return __builtin_fmax(0.0, __builtin_fma(-s.t, q, p));
}

// Sum of max(0, p - t q) over a slice.
template <typename T>
__device__ double slice_mass(const T* tr, const T* qr, int64_t lo, int64_t hi, bool vec, double c2, const TreeState& s,
                             Shared& sh) {
    const double iz_t = 1.0 / s.z_t, iz_q = 1.0 / s.z_q;
    double f = 0.0;
    for (int64_t i = lo + threadIdx.x * kPer; i < hi; i += NT * kPer) {
        float x[kPer], y[kPer];
        load8(tr, i, hi, vec, x);
        load8(qr, i, hi, vec, y);
#pragma unroll
        for (int j = 0; j < kPer; ++j) f += mass_of(x[j], y[j], s, iz_t, iz_q, c2, true);
    }
    return block_sum(f, sh.wave_a);
}

// The smallest token of [lo, hi) at which the cumulative mass, `run` before lo,
// passes `goal`; where rounding leaves none, the last one of positive mass (or
// lo).  Tokens of sh.gone have no mass.
template <typename T>
__device__ int slice_draw(const T* tr, const T* qr, int64_t lo, int64_t hi, bool vec, double c2, const TreeState& s,
                          double run, double goal, Shared& sh) {
    const bool pair = qr != nullptr;
    const double iz_t = 1.0 / s.z_t, iz_q = pair ? 1.0 / s.z_q : 0.0;
    int last = static_cast<int>(lo);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int64_t base = lo; base < hi; base += NT * kPer) {
        const int64_t i = base + threadIdx.x * kPer;
        float x[kPer], y[kPer];
        load8(tr, i, hi, vec, x);
        if (pair) load8(qr, i, hi, vec, y);
        double w[kPer], sum = 0.0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) w[j] = mass_of(x[j], pair ? y[j] : 0.f, s, iz_t, iz_q, c2, pair);
        for (int e = 0; e < sh.n_gone; ++e) {
            const int64_t d = sh.gone[e] - i;
#pragma unroll
            for (int j = 0; j < kPer; ++j) w[j] = d == j ? 0.0 : w[j];
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            sum += w[j];
            if (w[j] > 0.0) last = static_cast<int>(i + j);
        }
        double incl = sum;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const double o = __shfl_up(incl, d);
            if (lane >= d) incl += o;
        }
        __syncthreads();
        if (lane == 63) sh.wave_a[wave] = incl;
        if (threadIdx.x == 0) sh.ibcast[0] = INT_MAX;
        __syncthreads();
        double all = 0.0, before = run + (incl - sum);
#pragma unroll
        for (int v = 0; v < NWAVES; ++v) {
            if (v < wave) before += sh.wave_a[v];
            all += sh.wave_a[v];
        }
        int hit = INT_MAX;
        double c = before;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            c += w[j];
            if (hit == INT_MAX && w[j] > 0.0 && c > goal) hit = static_cast<int>(i + j);
        }
        if (hit != INT_MAX) atomicMin(&sh.ibcast[0], hit);  // integers: the same whatever the order
        __syncthreads();
        const int found = sh.ibcast[0];
        __syncthreads();
        if (found != INT_MAX) return found;
        run += all;
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) last = max(last, __shfl_xor(last, d));
    if (lane == 0) sh.wave_i[wave] = last;
    __syncthreads();
    for (int v = 0; v < NWAVES; ++v) last = max(last, sh.wave_i[v]);
    return last;
}

// The walk's next decision, taken by the first wavefront (lane i stands for
// node i).  On entry st holds this pass's result (statistics, or F(t)); on
// return its stage says what is needed next, and the answer is true when a
// token is to be drawn from what is left at st.at.
template <typename T, int KIND>
__device__ bool decide(const TreePlan& p, int b, TreeState& st, int argmax, Shared& sh) {
    const int lane = threadIdx.x & 63;
    const int64_t bk = static_cast<int64_t>(b) * p.k;
    int tok = -1;
    double u = 0.0;
    if (lane < p.k) {
        tok = p.tokens[bk + lane];
        if (KIND != kTreeGreedy) u = static_cast<double>(p.uniforms[bk + b + lane]);
    }
    const bool child = (st.left >> lane) & 1;
    int hit = -1;
    bool more = false;
    if (KIND == kTreeGreedy) {
        const uint64_t eq = __ballot(child && tok == argmax);
        hit = eq ? __builtin_ctzll(eq) : -1;
    } else {
        const int64_t row = static_cast<int64_t>(b) * (p.k + 1) + st.at + 1;
        double px = 0.0, qx = 0.0;
        if (child) {
            const float l = value<T>(static_cast<const T*>(p.target)[row * p.vocab + tok]);
            px = exp2_neg(__builtin_fma(static_cast<double>(l), p.c2, -st.m_t)) / st.z_t;
            if (KIND == kTreeLogits) {
                const int64_t dr = static_cast<int64_t>(b) * p.draft_rows + st.at + 1;
                const float d = value<T>(static_cast<const T*>(p.draft)[dr * p.vocab + tok]);
                qx = exp2_neg(__builtin_fma(static_cast<double>(d), p.c2, -st.m_q)) / st.z_q;
            }
        }
        if (KIND == kTreeOneHot) {
            double gone = 0.0;
            int n = 0;
            for (uint64_t rest = st.left; rest; rest &= rest - 1) {
                const int c = __builtin_ctzll(rest);
                const int x = __shfl(tok, c);
                const double pc = __shfl(px, c), uc = __shfl(u, c);
                const bool again = __ballot(child && lane < c && tok == x) != 0;
                if (!again && uc * (1.0 - gone) < pc) {
                    hit = c;
                    break;
                }
                if (!again) {
                    gone += pc;
                    if (lane == 0) sh.gone[n] = x;
                    ++n;
                }
            }
            if (lane == 0) sh.n_gone = n;
        } else if (st.left) {
            const int c = __builtin_ctzll(st.left);
            const double pc = __shfl(px, c), qc = __shfl(qx, c), uc = __shfl(u, c);
            if (uc * qc * st.f < __builtin_fmax(0.0, pc - st.t * qc)) {
                hit = c;
            } else {
                st.left &= st.left - 1;
                st.t += st.f;
                st.stage = kStageMass;
                more = true;
            }
        }
    }
    if (hit >= 0) {
        const int x = __shfl(tok, hit);
        if (lane == 0) {
            p.path[bk + st.kept] = hit;
            p.out_tokens[bk + b + st.kept] = x;
        }
        st.kept += 1;
        st.at = hit;
        const int up = lane < p.k ? p.parents[bk + lane] : -2;
        st.left = __ballot(up == hit);
        st.stage = kStageRow;
        st.t = 0.0;
        st.f = 1.0;
        return false;
    }
    return !more;
}

// The tree is checked and the walk stands at the root.  A tree that names a
// parent out of order, a child of an absent node, a token out of range or an
// inner node without a draft row is refused: accepted_len -1.
__device__ void begin(const TreePlan& p, int b, TreeState& st, bool draft) {
    const int lane = threadIdx.x & 63;
    const int64_t bk = static_cast<int64_t>(b) * p.k;
    int up = -2, tok = 0;
    if (lane < p.k) {
        up = p.parents[bk + lane];
        tok = p.tokens[bk + lane];
    }
    const uint64_t there = __ballot(up != -2);
    bool bad = up < -2 || up >= lane;
    if (up >= 0 && up < lane) bad = bad || !((there >> up) & 1) || (draft && up + 1 >= p.draft_rows);
    if (up != -2) bad = bad || tok < 0 || tok >= p.vocab;
    const bool refuse = __any(bad);
    st.at = -1;
    st.left = __ballot(up == -1);
    st.kept = 0;
    st.t = 0.0;
    st.f = 1.0;
    st.stage = refuse ? kStageDone : kStageRow;
    if (refuse) {
        if (lane == 0) {
            p.accepted_len[b] = -1;
            p.out_tokens[bk + b + p.k] = -1;
        }
        if (lane < p.k) {
            p.out_tokens[bk + b + lane] = -1;
            p.path[bk + lane] = -1;
        }
    }
}

__device__ void finish(const TreePlan& p, int b, const TreeState& st, int token) {
    const int lane = threadIdx.x & 63;
    const int64_t bk = static_cast<int64_t>(b) * p.k;
    if (lane == 0) {
        p.accepted_len[b] = st.kept;
        p.out_tokens[bk + b + st.kept] = token;
    }
    for (int i = lane; i <= p.k; i += 64) {
        if (i > st.kept) p.out_tokens[bk + b + i] = -1;
        if (i >= st.kept && i < p.k) p.path[bk + i] = -1;
    }
}

// The whole walk of one sequence by one workgroup.
template <typename T, int KIND>
__global__ __launch_bounds__(NT) void k_tree_walk(TreePlan p) {
    __shared__ Shared sh;
    const int b = blockIdx.x;
    const int64_t V = p.vocab;
    const bool vec = p.vec != 0;
    if (threadIdx.x < 64) {
        TreeState st{};
        begin(p, b, st, KIND == kTreeLogits);
        if (threadIdx.x == 0) {
            sh.st = st;
            sh.n_gone = 0;
        }
    }
    __syncthreads();
    while (true) {
        TreeState st = sh.st;
        if (st.stage == kStageDone) return;
        const T* const tr = static_cast<const T*>(p.target) + (static_cast<int64_t>(b) * (p.k + 1) + st.at + 1) * V;
        const bool pair = KIND == kTreeLogits && (st.left != 0 || st.stage == kStageMass);
        const T* const qr = pair ? static_cast<const T*>(p.draft) + (static_cast<int64_t>(b) * p.draft_rows + st.at + 1) * V
                                 : nullptr;
        int best = 0;
        if (KIND == kTreeGreedy) {
            float m;
            slice_argmax(tr, 0, V, vec, sh, &m, &best);
        } else if (st.stage == kStageRow) {
            slice_stats(tr, 0, V, vec, p.c2, sh, &st.m_t, &st.z_t);
            if (pair) slice_stats(qr, 0, V, vec, p.c2, sh, &st.m_q, &st.z_q);
        } else {
            st.f = slice_mass(tr, qr, 0, V, vec, p.c2, st, sh);
        }
        __syncthreads();
        if (threadIdx.x < 64) {
            const bool draw = decide<T, KIND>(p, b, st, best, sh);
            if (threadIdx.x == 0) {
                sh.st = st;
                sh.ibcast[1] = draw;
            }
        }
        __syncthreads();
        if (!sh.ibcast[1]) continue;
        st = sh.st;
        int y = best;
        if (KIND != kTreeGreedy) {
            double all;
            if (st.stage == kStageMass)
                all = st.f;
            else {
                all = 1.0;
                for (int e = 0; e < sh.n_gone; ++e)
                    all -= exp2_neg(__builtin_fma(static_cast<double>(value<T>(tr[sh.gone[e]])), p.c2, -st.m_t)) / st.z_t;
            }
            const double u = p.uniforms[static_cast<int64_t>(b) * (p.k + 1) + p.k];
            y = slice_draw(tr, st.stage == kStageMass ? qr : nullptr, 0, V, vec, p.c2, st, 0.0, u * all, sh);
        }
        if (threadIdx.x < 64) finish(p, b, st, y);
        return;
    }
}

template <typename T>
hipError_t launch_t(const TreePlan& p, hipStream_t stream) {
    const dim3 grid(p.batch), block(NT);
    switch (p.kind) {
        case kTreeGreedy: k_tree_walk<T, kTreeGreedy><<<grid, block, 0, stream>>>(p); break;
        case kTreeOneHot: k_tree_walk<T, kTreeOneHot><<<grid, block, 0, stream>>>(p); break;
        default: k_tree_walk<T, kTreeLogits><<<grid, block, 0, stream>>>(p); break;
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_verify_tree(const TreePlan& p, hipStream_t stream) {
    return p.elem_bytes == 4 ? launch_t<float>(p, stream) : launch_t<uint16_t>(p, stream);
}

}  // namespace sv
