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
// 2^x is good to 4.5e-12 (Power).  64-bit multiply-adds run at about the rate of
// 32-bit ones here (5.3 against 4.7 cycles a wavefront, measured).
// Row maxima are kept as whole powers of two (M >= max l c2), so that sums over
// parts of a row join by exact shifts, and the rounding to the power, the
// exponent's bias and M are one constant: see Power.
//
// Kernels.  k_tree_cluster takes the walks row by row and reads only the rows on
// the walked path, several workgroups to a sequence, on one die, which hand each
// other a pass's partials and all take the same decision.  k_tree_rows reads
// every row of the trees at once instead, where there are few (kTreeAllRows):
// it reads more and waits less.  k_tree_walk is one workgroup a sequence: the
// whole walk of a small vocabulary, and the end of a walk whose workgroups did
// not wait for each other long enough.
//
// What bounds them (V = 151936, bf16, k = 16).  128 sequences with a drafter's
// rows: 151 us, 3.4 passes over two rows on average and up to 6; the 264 MB that
// have to be read take 38 us at 7.0 TB/s and the logits' 2^x, 12 operations
// each, about 65 us.  A pass of all sequences takes about 21 us of that
// arithmetic, 6 of waiting for the slowest workgroup of a sequence, 1.6 of the
// decision; the rest is sequences that walk longer than others.  64 with
// one-hot children 56 us, 64 greedy walks 46 us.  8 with one-hot children, all
// 41 MB of rows at once, 35 us: 6 of reading, 8 of 2^x, then the walk, the draw
// within a slice, and the launch.  4 sequences of 1000 tokens 15 us, one
// workgroup each: four or five trips to memory one after the other.
// Workgroups of 256: 512 took 213 us where 256 take 188 and 128 take 203.
#include <hip/hip_runtime.h>

#include <climits>
#include <cstdint>
#include <type_traits>

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

// 2^(l c2 - M) for logits l.  k1 = 1.5 2^46 + 1023 - M: the sum l c2 + k1 is
// rounded to a multiple of 1/64, whose low word is 64 times the biased exponent
// plus the index i of 2^(i / 64) in the table; what the rounding took off, at
// most 1/128, is the polynomial's argument (degree 3 at Chebyshev nodes,
// relative error 4.5e-12).  The table's high words have i 2^14 taken off, so
// that the low word, shifted by 14, adds the exponent and nothing else.  64
// entries are two to each pair of LDS banks: a read takes two turns at most.
// Against one polynomial of degree 7 (5.5e-11, 14 operations of 64 bits a
// logit) this is 9 of 64 bits and three of 32.  Logits are raised to `low`,
// where the result is 2^-1000: nothing in a sum, and the exponent stays in
// range (a logit of -inf is never drawn, see slice_draw).
constexpr int kPow2 = 64;

__device__ __forceinline__ double pow2_entry(int i) {
    const double t = exp2(static_cast<double>(i) / kPow2);
    return __hiloint2double((__double2hiint(t) & 0xFFFFF) - (i << 14), __double2loint(t));
}

struct Scale {
    double c2, per_c2;  // log2(e) / T and one over it
    __device__ __forceinline__ explicit Scale(const TreePlan& p) : c2(p.c2), per_c2(p.per_c2) {}
};

struct Power {
    const double* table;
    double c2, k1, low;
    __device__ __forceinline__ Power(const double* table_, const Scale& c, double m) : table(table_), c2(c.c2) {
        k1 = 105553116266496.0 + (1023.0 - m);
        low = (m - 1000.0) * c.per_c2;
    }
    __device__ __forceinline__ double operator()(float l) const {
        const double x = __builtin_fmax(static_cast<double>(l), low);
        const double s = __builtin_fma(x, c2, k1);
        const double f = __builtin_fma(x, c2, k1 - s);
        const int n = __double2loint(s);
        const double t = table[n & (kPow2 - 1)];
        double r = 0.055504190037736274;
        r = __builtin_fma(r, f, 0.24022709400357053);
        r = __builtin_fma(r, f, 0.6931471805593249);
        r = __builtin_fma(r, f, 0.9999999999955212);
        return r * __hiloint2double(__double2hiint(t) + static_cast<int>(static_cast<uint32_t>(n) << 14), __double2loint(t));
    }
};

// The whole power of two that bounds a row's largest 2^(l c2).
__device__ __forceinline__ double power_of(float top, double c2) {
    const double y = static_cast<double>(top) * c2;
    // finite rows give finite bounds; an empty part of a row, or a part of -inf alone, gives 0
    return y >= -8e12 && y <= 8e12 ? __builtin_ceil(y) : 0.0;
}

// x 2^(m - top), m <= top whole numbers.
__device__ __forceinline__ double shift_to(double x, double m, double top) {
    return __builtin_ldexp(x, static_cast<int>(__builtin_fmax(m - top, -4000.0)));
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

// Eight elements as they lie in memory.  Loads and conversions are apart, so
// that the loads of several tiles are in flight together.
template <typename T>
struct Raw {
    uint4 v[sizeof(T) / 2];
    __device__ __forceinline__ void get(float (&x)[kPer]) const {
        const uint32_t* const w = reinterpret_cast<const uint32_t*>(v);
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            if constexpr (sizeof(T) == 4) x[j] = __uint_as_float(w[j]);
            else x[j] = __uint_as_float(j & 1 ? w[j >> 1] & 0xFFFF0000u : w[j >> 1] << 16);
        }
    }
};

// Elements [i, i + kPer) of a row, -inf from `end` on.  Rows that do not start
// on 16-byte boundaries (V not a multiple of 16 bytes) are read one by one.
template <typename T>
__device__ __forceinline__ Raw<T> load8(const T* row, int64_t i, int64_t end, bool vec) {
    constexpr int NV = sizeof(T) / 2;
    Raw<T> r;
    constexpr uint32_t none = sizeof(T) == 4 ? 0xFF800000u : 0xFF80FF80u;  // -inf
#pragma unroll
    for (int j = 0; j < NV; ++j) r.v[j] = uint4{none, none, none, none};
    if (vec && i + kPer <= end) {
#pragma unroll
        for (int j = 0; j < NV; ++j) r.v[j] = reinterpret_cast<const uint4*>(row + i)[j];
    } else if (i < end) {
        uint32_t w[4 * NV];
#pragma unroll
        for (int j = 0; j < 4 * NV; ++j) w[j] = none;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            if (i + j >= end) continue;
            if constexpr (sizeof(T) == 4) w[j] = __float_as_uint(row[i + j]);
            else if (j & 1) w[j >> 1] = (w[j >> 1] & 0xFFFFu) | (static_cast<uint32_t>(row[i + j]) << 16);
            else w[j >> 1] = (w[j >> 1] & 0xFFFF0000u) | row[i + j];
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) r.v[j] = uint4{w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]};
    }
    return r;
}

// The value of the lane that is D away, or for 4 and 8 of one in the
// neighbouring group of as many: the same for a reduction, which has made the
// lanes of a group alike by then.  Up to 8 it is an operand's permutation
// (DPP), not a trip through LDS.
template <int D>
__device__ __forceinline__ int from_lane(int v) {
    if constexpr (D == 1) return __builtin_amdgcn_mov_dpp(v, 0xB1, 0xF, 0xF, true);       // 1 0 3 2 in four
    else if constexpr (D == 2) return __builtin_amdgcn_mov_dpp(v, 0x4E, 0xF, 0xF, true);  // 2 3 0 1
    else if constexpr (D == 4) return __builtin_amdgcn_mov_dpp(v, 0x141, 0xF, 0xF, true); // eight mirrored
    else if constexpr (D == 8) return __builtin_amdgcn_mov_dpp(v, 0x140, 0xF, 0xF, true); // sixteen mirrored
    else return __shfl_xor(v, D);
}
template <int D>
__device__ __forceinline__ float from_lane(float v) {
    return __int_as_float(from_lane<D>(__float_as_int(v)));
}
template <int D>
__device__ __forceinline__ double from_lane(double v) {
    return __hiloint2double(from_lane<D>(__double2hiint(v)), from_lane<D>(__double2loint(v)));
}

template <typename F>
__device__ __forceinline__ void reduce_steps(const F& f) {
    f(std::integral_constant<int, 1>{});
    f(std::integral_constant<int, 2>{});
    f(std::integral_constant<int, 4>{});
    f(std::integral_constant<int, 8>{});
    f(std::integral_constant<int, 16>{});
    f(std::integral_constant<int, 32>{});
}

__device__ __forceinline__ double wave_sum(double v) {
    reduce_steps([&](auto d) { v += from_lane<d.value>(v); });
    return v;
}
__device__ __forceinline__ float wave_max(float v) {
    reduce_steps([&](auto d) { v = fmaxf(v, from_lane<d.value>(v)); });
    return v;
}

__device__ __forceinline__ void wave_argmax(float& m, int& at) {
    reduce_steps([&](auto d) {
        const float om = from_lane<d.value>(m);
        const int oa = from_lane<d.value>(at);
        if (om > m || (om == m && oa < at)) {
            m = om;
            at = oa;
        }
    });
}

// Joins the (M, sum) of the slices that the lanes hold; returns this lane's
// sum against the common power.
__device__ __forceinline__ double join(bool mine, double m, double z, double* m_out, double* z_out) {
    const bool some = mine && z > 0.0;
    double top = some ? m : -1e300;
    reduce_steps([&](auto d) { top = __builtin_fmax(top, from_lane<d.value>(top)); });
    if (top == -1e300) top = 0.0;
    const double s = some ? shift_to(z, m, top) : 0.0;
    *m_out = top;
    *z_out = wave_sum(s);
    return s;
}

// What a complete pass leads to.
struct Next {
    bool draw;         // a token is due: from the tokens [from, from + len), `run` the mass before them
    int best;          // greedy: the token
    int64_t from, len;
    double run, goal;
};

constexpr int kGroup = 8;  // tiles whose loads are in flight together, times the size of an element (16 spilled, and was 9% slower)

struct Shared {
    double pow2[kPow2];
    double wave_a[NWAVES], wave_b[NWAVES];
    float wave_f[NWAVES];
    int wave_i[NWAVES];
    double bcast[8];
    int ibcast[8];
    double scan[kGroup][NWAVES];
    int gone[SV_MAX_DRAFT];  // one-hot: the rejected siblings' tokens and their p
    double gone_p[SV_MAX_DRAFT];
    int n_gone;
    double row_m[SV_MAX_DRAFT + 1], row_z[SV_MAX_DRAFT + 1];  // every row's statistics: join_rows
    TreeState st;
    Next nx;
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
    constexpr int GROUP = kGroup / sizeof(T);
    float m = -__builtin_inff();
    int at = INT_MAX;
    for (int64_t base = lo; base < hi; base += GROUP * NT * kPer) {
        Raw<T> raw[GROUP];
#pragma unroll
        for (int t = 0; t < GROUP; ++t) raw[t] = load8(row, base + (t * NT + threadIdx.x) * kPer, hi, vec);
#pragma unroll
        for (int t = 0; t < GROUP; ++t) {
            if (base + t * (NT * kPer) >= hi) continue;  // the whole workgroup at once
            const int64_t i = base + (t * NT + threadIdx.x) * kPer;
            float x[kPer];
            raw[t].get(x);
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                if (i + j < hi && (x[j] > m || at == INT_MAX)) {
                    m = x[j];
                    at = static_cast<int>(i + j);
                }
        }
    }
    wave_argmax(m, at);
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

// (M, sum of 2^(l c2 - M)) of a slice, M the power of its maximum, in one
// sweep: a thread sums against its own power, raised once per group of tiles.
template <typename T>
__device__ void slice_stats(const T* row, int64_t lo, int64_t hi, bool vec, const Scale& scale, Shared& sh, double* m_out,
                            double* z_out) {
    constexpr int GROUP = kGroup / sizeof(T);
    float top = -__builtin_inff();
    double m = 0.0, z = 0.0;
    for (int64_t base = lo; base < hi; base += GROUP * NT * kPer) {
        Raw<T> raw[GROUP];
#pragma unroll
        for (int t = 0; t < GROUP; ++t) raw[t] = load8(row, base + (t * NT + threadIdx.x) * kPer, hi, vec);
        float x[kPer], was = top;
#pragma unroll
        for (int t = 0; t < GROUP; ++t) {
            raw[t].get(x);
#pragma unroll
            for (int j = 0; j < kPer; ++j) top = fmaxf(top, x[j]);
        }
        if (top > was) {
            const double mn = power_of(top, scale.c2);
            z = was == -__builtin_inff() ? 0.0 : shift_to(z, m, mn);
            m = mn;
        }
        const Power power(sh.pow2, scale, m);
#pragma unroll
        for (int t = 0; t < GROUP; ++t) {
            if (base + t * (NT * kPer) >= hi) continue;  // the whole workgroup at once
            raw[t].get(x);
#pragma unroll
            for (int j = 0; j < kPer; ++j) z += power(x[j]);
        }
    }
    const float all = block_max(top, sh.wave_f);
    const double mc = power_of(all, scale.c2);
    z = top == -__builtin_inff() ? 0.0 : shift_to(z, m, mc);
    *z_out = block_sum(z, sh.wave_a);
    *m_out = mc;
}

// max(0, p - t q) of one token, p and q by their rows' statistics.
struct Mass {
    Power p, q;
    double iz, tq;
    __device__ __forceinline__ Mass(const double* pow2, const TreeState& s, const Scale& c)
        : p(pow2, c, s.m_t), q(pow2, c, s.m_q), iz(1.0 / s.z_t), tq(s.t / s.z_q) {}
    __device__ __forceinline__ double operator()(float lt, float lq) const {
        return __builtin_fmax(0.0, __builtin_fma(-tq, q(lq), iz * p(lt)));
    }
};

// Sum of max(0, p - t q) over a slice.
template <typename T>
__device__ double slice_mass(const T* tr, const T* qr, int64_t lo, int64_t hi, bool vec, const Scale& scale, const TreeState& s,
                             Shared& sh) {
    constexpr int GROUP = kGroup / sizeof(T) / 2;
    const Mass mass(sh.pow2, s, scale);
    double f = 0.0;
    for (int64_t base = lo; base < hi; base += GROUP * NT * kPer) {
        Raw<T> a[GROUP], b[GROUP];
#pragma unroll
        for (int t = 0; t < GROUP; ++t) {
            a[t] = load8(tr, base + (t * NT + threadIdx.x) * kPer, hi, vec);
            b[t] = load8(qr, base + (t * NT + threadIdx.x) * kPer, hi, vec);
        }
#pragma unroll
        for (int t = 0; t < GROUP; ++t) {
            if (base + t * (NT * kPer) >= hi) continue;  // the whole workgroup at once
            float x[kPer], y[kPer];
            a[t].get(x);
            b[t].get(y);
#pragma unroll
            for (int j = 0; j < kPer; ++j) f += mass(x[j], y[j]);
        }
    }
    return block_sum(f, sh.wave_a);
}

// The smallest token of [lo, hi) at which the cumulative mass, `run` before lo,
// passes `goal`; where rounding leaves none, the last one of positive mass (or
// lo).  Tokens of sh.gone have no mass.  A group of tiles is loaded and scanned
// at a time; the thread in whose eight tokens the goal lies looks for it there.
template <typename T, bool PAIR>
__device__ int slice_draw(const T* tr, const T* qr, int64_t lo, int64_t hi, bool vec, const Scale& scale, const TreeState& s,
                          double run, double goal, Shared& sh) {
    constexpr int GROUP = PAIR ? 1 : kGroup / sizeof(T) / 2;  // more are spilled
    const Mass mass(sh.pow2, s, scale);
    int last = static_cast<int>(lo);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const auto weights = [&](const Raw<T>& a, const Raw<T>& b, int64_t i, double (&w)[kPer]) {
        float x[kPer], y[kPer];
        a.get(x);
        b.get(y);
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            w[j] = PAIR ? mass(x[j], y[j]) : mass.iz * mass.p(x[j]);
            if (!(x[j] >= mass.p.low)) w[j] = 0.0;  // logits of -inf are never drawn
        }
        for (int e = 0; e < sh.n_gone; ++e) {
            const int64_t d = sh.gone[e] - i;
#pragma unroll
            for (int j = 0; j < kPer; ++j) w[j] = d == j ? 0.0 : w[j];
        }
    };
    for (int64_t base = lo; base < hi; base += GROUP * NT * kPer) {
        Raw<T> a[GROUP], b[GROUP];
#pragma unroll
        for (int t = 0; t < GROUP; ++t) {
            const int64_t i = base + (t * NT + threadIdx.x) * kPer;
            a[t] = load8(tr, i, hi, vec);
            b[t] = PAIR ? load8(qr, i, hi, vec) : a[t];
        }
        double sum[GROUP], incl[GROUP];
#pragma unroll
        for (int t = 0; t < GROUP; ++t) {
            const int64_t i = base + (t * NT + threadIdx.x) * kPer;
            sum[t] = 0.0;
            if (base + t * (NT * kPer) < hi) {  // the whole workgroup at once
                double w[kPer];
                weights(a[t], b[t], i, w);
#pragma unroll
                for (int j = 0; j < kPer; ++j) {
                    sum[t] += w[j];
                    if (w[j] > 0.0) last = static_cast<int>(i + j);
                }
            }
            incl[t] = sum[t];
        }
#pragma unroll
        for (int d = 1; d < 64; d <<= 1)
#pragma unroll
            for (int t = 0; t < GROUP; ++t) {
                const double o = __shfl_up(incl[t], d);
                if (lane >= d) incl[t] += o;
            }
        __syncthreads();
        if (lane == 63)
#pragma unroll
            for (int t = 0; t < GROUP; ++t) sh.scan[t][wave] = incl[t];
        if (threadIdx.x == 0) sh.ibcast[0] = INT_MAX;
        __syncthreads();
        double before[GROUP];
#pragma unroll
        for (int t = 0; t < GROUP; ++t) {
            before[t] = run + (incl[t] - sum[t]);
#pragma unroll
            for (int v = 0; v < NWAVES; ++v) {
                if (v < wave) before[t] += sh.scan[t][v];
                run += sh.scan[t][v];
            }
            const uint64_t past = __ballot(sum[t] > 0.0 && before[t] + sum[t] > goal);
            if (past && lane == __builtin_ctzll(past)) atomicMin(&sh.ibcast[0], t * NT + static_cast<int>(threadIdx.x));  // integers: the same whatever the order
        }
        __syncthreads();
        const int found = sh.ibcast[0];
        if (found != INT_MAX) {
            if (static_cast<int>(threadIdx.x) == found % NT) {
#pragma unroll
                for (int t = 0; t < GROUP; ++t) {
                    if (t != found / NT) continue;
                    const int64_t i = base + (t * NT + threadIdx.x) * kPer;
                    double w[kPer], c = before[t];
                    weights(a[t], b[t], i, w);
                    int hit = 0;
                    bool done = false;
#pragma unroll
                    for (int j = 0; j < kPer; ++j) {
                        c += w[j];
                        if (!done && w[j] > 0.0) hit = j;
                        done = done || (w[j] > 0.0 && c > goal);
                    }
                    sh.ibcast[3] = static_cast<int>(i) + hit;
                }
            }
            __syncthreads();
            return sh.ibcast[3];
        }
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) last = max(last, __shfl_xor(last, d));
    if (lane == 0) sh.wave_i[wave] = last;
    __syncthreads();
    for (int v = 0; v < NWAVES; ++v) last = max(last, sh.wave_i[v]);
    return last;
}

// A token from what is left at the row that `st` stands at.
template <typename T, int KIND>
__device__ __forceinline__ int draw_from(const T* target, const T* draft, int64_t lo, int64_t hi, bool vec, const Scale& scale,
                                         const TreeState& st, double run, double goal, Shared& sh) {
    if (KIND == kTreeLogits && st.stage == kStageMass)
        return slice_draw<T, true>(target, draft, lo, hi, vec, scale, st, run, goal, sh);
    return slice_draw<T, false>(target, target, lo, hi, vec, scale, st, run, goal, sh);
}

// What lane i knows of node i: read once, ahead of the rows, so that no
// decision waits for memory.
struct Node {
    int up, tok;
    double u;
    float l, d;  // the logits of its token in its parent's target and draft row
};

template <typename T, int KIND>
__device__ __forceinline__ Node node_of(const TreePlan& p, int b) {
    const int lane = threadIdx.x & 63;
    const int64_t bk = static_cast<int64_t>(b) * p.k;
    Node n{-2, -1, 0.0, 0.f, 0.f};
    if (lane < p.k) {
        n.up = p.parents[bk + lane];
        n.tok = p.tokens[bk + lane];
        if (KIND != kTreeGreedy) n.u = static_cast<double>(p.uniforms[bk + b + lane]);
        // (a refused tree may name anything: nothing is read for it)
        const bool fine = n.up >= -1 && n.up < lane && n.tok >= 0 && n.tok < p.vocab;
        if (KIND != kTreeGreedy && fine) {
            const int64_t row = static_cast<int64_t>(b) * (p.k + 1) + n.up + 1;
            n.l = value<T>(static_cast<const T*>(p.target)[row * p.vocab + n.tok]);
        }
        if (KIND == kTreeLogits && fine && n.up + 1 < p.draft_rows) {
            const int64_t row = static_cast<int64_t>(b) * p.draft_rows + n.up + 1;
            n.d = value<T>(static_cast<const T*>(p.draft)[row * p.vocab + n.tok]);
        }
    }
    return n;
}

// The walk's next decision, taken by the first wavefront.  On entry st holds
// the row's statistics (or F(t)); on return its stage says what is needed next,
// and the answer is true when a token is to be drawn from what is left at st.at.
// Every workgroup of a sequence may take the decision, one (`lead`) writes it.
template <int KIND>
__device__ __forceinline__ bool decide(const TreePlan& p, int b, const Node& node, TreeState& st, int argmax, bool lead, Shared& sh) {
    const int lane = threadIdx.x & 63;
    const int64_t bk = static_cast<int64_t>(b) * p.k;
    const bool child = (st.left >> lane) & 1;
    int hit = -1;
    bool more = false;
    if (KIND == kTreeGreedy) {
        const uint64_t eq = __ballot(child && node.tok == argmax);
        hit = eq ? __builtin_ctzll(eq) : -1;
    } else {
        double px = 0.0, qx = 0.0;
        if (child) {
            const Power pt(sh.pow2, Scale(p), st.m_t);
            px = node.l < pt.low ? 0.0 : pt(node.l) / st.z_t;
            if (KIND == kTreeLogits) {
                const Power pq(sh.pow2, Scale(p), st.m_q);
                qx = node.d < pq.low ? 0.0 : pq(node.d) / st.z_q;
            }
        }
        if (KIND == kTreeOneHot) {
            double gone = 0.0;
            int n = 0;
            for (uint64_t rest = st.left; rest; rest &= rest - 1) {
                const int c = __builtin_ctzll(rest);
                const int x = __shfl(node.tok, c);
                const double pc = __shfl(px, c), uc = __shfl(node.u, c);
                const bool again = __ballot(child && lane < c && node.tok == x) != 0;
                if (!again && uc * (1.0 - gone) < pc) {
                    hit = c;
                    break;
                }
                if (!again) {
                    gone += pc;
                    if (lane == 0) {
                        sh.gone[n] = x;
                        sh.gone_p[n] = pc;
                    }
                    ++n;
                }
            }
            if (lane == 0) sh.n_gone = n;
        } else if (st.left) {
            const int c = __builtin_ctzll(st.left);
            const double pc = __shfl(px, c), qc = __shfl(qx, c), uc = __shfl(node.u, c);
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
        const int x = __shfl(node.tok, hit);
        if (lead && lane == 0) {
            p.path[bk + st.kept] = hit;
            p.out_tokens[bk + b + st.kept] = x;
        }
        st.kept += 1;
        st.at = hit;
        st.left = __ballot(node.up == hit);
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
template <int KIND>
__device__ void begin(const TreePlan& p, int b, const Node& node, TreeState& st) {
    const int lane = threadIdx.x & 63;
    const uint64_t there = __ballot(node.up != -2);
    bool bad = node.up < -2 || node.up >= lane;
    if (node.up >= 0 && node.up < lane)
        bad = bad || !((there >> node.up) & 1) || (KIND == kTreeLogits && node.up + 1 >= p.draft_rows);
    if (node.up != -2) bad = bad || node.tok < 0 || node.tok >= p.vocab;
    const bool refuse = __any(bad);
    st.at = -1;
    st.left = __ballot(node.up == -1);
    st.kept = 0;
    st.t = 0.0;
    st.f = 1.0;
    st.stage = refuse ? kStageDone : kStageRow;
}

__device__ void refuse(const TreePlan& p, int b) {
    const int lane = threadIdx.x & 63;
    const int64_t bk = static_cast<int64_t>(b) * p.k;
    if (lane == 0) p.accepted_len[b] = -1;
    for (int i = lane; i <= p.k; i += 64) {
        p.out_tokens[bk + b + i] = -1;
        if (i < p.k) p.path[bk + i] = -1;
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

// The rows that a pass over `st` reads: the target row of the node it stands
// at, and the draft row where children or a residual need it.
template <typename T, int KIND>
struct Rows {
    const T* target;
    const T* draft;  // NULL: not read
    __device__ Rows(const TreePlan& p, int b, const TreeState& st) {
        const bool pair = KIND == kTreeLogits && (st.left != 0 || st.stage == kStageMass);
        target = static_cast<const T*>(p.target) + (static_cast<int64_t>(b) * (p.k + 1) + st.at + 1) * p.vocab;
        draft = pair ? static_cast<const T*>(p.draft) + (static_cast<int64_t>(b) * p.draft_rows + st.at + 1) * p.vocab
                     : nullptr;
    }
};

// Mass of the removed tokens (one-hot) that lie in [lo, hi).
__device__ __forceinline__ double gone_mass(const Shared& sh, int64_t lo, int64_t hi) {
    double sum = 0.0;
    for (int e = 0; e < sh.n_gone; ++e)
        if (sh.gone[e] >= lo && sh.gone[e] < hi) sum += sh.gone_p[e];
    return sum;
}

// Hands four words to the workgroup that arrives last: agent-scope stores
// reach memory past this die's L2, the wait sees them arrive, and only then is
// the arrival counted, so no cache is written back or invalidated.  Called
// by one thread; true on the last arrival.
__device__ __forceinline__ bool hand_in(double* part, const double (&r)[4], int n, uint32_t* arrived, uint32_t all) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < n) __hip_atomic_store(part + i, r[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    return __hip_atomic_fetch_add(arrived, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == all - 1;
}

__device__ __forceinline__ double taken(const double* part) {
    return __hip_atomic_load(part, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Whether the state that the pass before left can be read by.  A workspace
// that was not zero-filled leaves anything; what does not fit ends the walk
// (outputs unspecified), so that every access stays in bounds.
template <int KIND>
__device__ __forceinline__ bool in_range(const TreePlan& p, const TreeState& st) {
    const bool pair = KIND == kTreeLogits && (st.left != 0 || st.stage == kStageMass);
    return (st.stage == kStageRow || (KIND == kTreeLogits && st.stage == kStageMass)) && st.at >= -1 && st.at < p.k &&
           st.kept >= 0 && st.kept <= p.k && (st.kept < p.k || st.left == 0) && (!pair || st.at + 1 < p.draft_rows);
}
template <int KIND>
__device__ __forceinline__ bool fits(const TreePlan& p, int b, const Node& node, const TreeState& st) {
    TreeState start{};
    begin<KIND>(p, b, node, start);
    return start.stage != kStageDone && (st.left & ~__ballot(node.up == st.at)) == 0;
}

// Joins the partials of every row, those that were read at once, for the first
// wavefront, by the others: several rows to a wavefront, a lane to a slice.
template <int KIND>
__device__ __forceinline__ void join_rows(const TreePlan& p, int b, Shared& sh) {
    int width = 1;
    while (width < p.row_slices) width <<= 1;
    const int i = threadIdx.x & (width - 1);
    for (int row = (threadIdx.x - 64) / width; row <= p.k; row += (NT - 64) / width) {
        const double* const part = p.row_part + ((static_cast<int64_t>(b) * (p.k + 1) + row) * kTreeMaxSlices + i) * 2;
        double m = 0.0, z = 0.0;
        if (i < p.row_slices) {
            m = taken(part);
            z = taken(part + 1);
        }
        if (KIND == kTreeGreedy) {  // (maximum, lowest index)
            if (i >= p.row_slices) m = -__builtin_inf(), z = INT_MAX;
            for (int d = width >> 1; d; d >>= 1) {
                const double om = __shfl_xor(m, d), oz = __shfl_xor(z, d);
                if (om > m || (om == m && oz < z)) {
                    m = om;
                    z = oz;
                }
            }
            if (i == 0) sh.row_z[row] = z;
            continue;
        }
        double top = z > 0.0 ? m : -1e300;
        for (int d = width >> 1; d; d >>= 1) top = __builtin_fmax(top, __shfl_xor(top, d));
        if (top == -1e300) top = 0.0;
        double sum = z > 0.0 ? shift_to(z, m, top) : 0.0;
        for (int d = width >> 1; d; d >>= 1) sum += __shfl_xor(sum, d);
        if (i == 0) {
            sh.row_m[row] = top;
            sh.row_z[row] = sum;
        }
    }
}

// Where the token lies that is to be drawn, by the mass of each lane's slice
// (the first wavefront).
template <int KIND>
__device__ __forceinline__ void place(const TreePlan& p, int b, double mass, int slices, int64_t per, const Shared& sh,
                                      Next& nx) {
    const int lane = threadIdx.x & 63;
    if (KIND == kTreeOneHot) mass = __builtin_fmax(0.0, mass - gone_mass(sh, lane * per, (lane + 1) * per));
    if (lane >= slices) mass = 0.0;
    double cum = mass;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const double o = __shfl_up(cum, d);
        if (lane >= d) cum += o;
    }
    nx.goal = static_cast<double>(p.uniforms[static_cast<int64_t>(b) * (p.k + 1) + p.k]) * __shfl(cum, 63);
    uint64_t past = __ballot(mass > 0.0 && cum > nx.goal);
    if (!past) {  // rounding left none: the last slice that holds anything
        const uint64_t any = __ballot(mass > 0.0);
        past = any ? uint64_t{1} << (63 - __builtin_clzll(any)) : 1;
    }
    const int at = __builtin_ctzll(past);
    nx.run = __shfl(cum - mass, at);
    nx.from = at * per;
    nx.len = per;
}

// Goes on with a walk whose pass is complete, by one decision (the first
// wavefront).  r: the pass's partials, lane i's of slice i.  st is what the next
// pass works on.
template <int KIND>
__device__ __forceinline__ Next go_on(const TreePlan& p, int b, const Node& node, TreeState& st, const double (&r)[4],
                                      bool lead, Shared& sh) {
    const bool mine = static_cast<int>(threadIdx.x & 63) < p.slices;
    Next nx{false, 0, 0, 0, 0.0, 0.0};
    double mass = 0.0;  // of this lane's slice
    if (KIND == kTreeGreedy) {
        float m = mine ? static_cast<float>(r[0]) : -__builtin_inff();
        nx.best = mine ? static_cast<int>(r[1]) : INT_MAX;
        wave_argmax(m, nx.best);
    } else if (st.stage == kStageRow) {
        mass = join(mine, r[0], r[1], &st.m_t, &st.z_t) / st.z_t;
        if (KIND == kTreeLogits && st.left) join(mine, r[2], r[3], &st.m_q, &st.z_q);
    } else {
        mass = mine ? r[0] : 0.0;
        st.f = wave_sum(mass);
    }
    nx.draw = decide<KIND>(p, b, node, st, nx.best, lead, sh);
    if (nx.draw && KIND != kTreeGreedy) place<KIND>(p, b, mass, p.slices, p.per, sh, nx);
    return nx;
}

// The whole walk, every row's statistics being there (the first wavefront).
template <int KIND>
__device__ __forceinline__ Next walk_rows(const TreePlan& p, int b, const Node& node, TreeState& st, Shared& sh) {
    const int lane = threadIdx.x & 63;
    Next nx{false, 0, 0, 0, 0.0, 0.0};
    while (!nx.draw) {
        if (KIND == kTreeGreedy) {
            nx.best = static_cast<int>(sh.row_z[st.at + 1]);
        } else {
            st.m_t = sh.row_m[st.at + 1];
            st.z_t = sh.row_z[st.at + 1];
        }
        nx.draw = decide<KIND>(p, b, node, st, nx.best, true, sh);
    }
    if (KIND == kTreeOneHot) {
        const int64_t row = static_cast<int64_t>(b) * (p.k + 1) + st.at + 1;
        const double* const part = p.row_part + (row * kTreeMaxSlices + lane) * 2;
        double m = 0.0, z = 0.0;
        if (lane < p.row_slices) {
            m = taken(part);
            z = taken(part + 1);
        }
        place<KIND>(p, b, z > 0.0 ? shift_to(z, m, st.m_t) / st.z_t : 0.0, p.row_slices, p.row_per, sh, nx);
    }
    return nx;
}

// The token that is due, and the sequence's end (the whole workgroup).
template <typename T, int KIND>
__device__ void draw_token(const TreePlan& p, int b, const TreeState& st, const Next& nx, Shared& sh) {
    int y = nx.best;
    if (KIND != kTreeGreedy) {
        const Rows<T, KIND> rows(p, b, st);
        y = draw_from<T, KIND>(rows.target, rows.draft, nx.from, min(static_cast<int64_t>(p.vocab), nx.from + nx.len),
                               p.vec != 0, Scale(p), st, nx.run, nx.goal, sh);
    }
    if (threadIdx.x < 64) finish(p, b, st, y);
}

// The statistics of every row of the tree at once; the last workgroup of a
// sequence then takes the walk.  Not for children from a draft row: there a
// rejection asks for another pass over its rows, and walks of the cluster's
// kind were faster from 1 sequence (53 against 72 us, k = 16, V = 151936) to 64
// (101 against 285).
template <typename T, int KIND>
__global__ __launch_bounds__(NT) void k_tree_rows(TreePlan p) {
    static_assert(KIND != kTreeLogits);
    __shared__ Shared sh;
    const int slice = blockIdx.x, row = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
    const int64_t V = p.vocab, lo = slice * p.row_per, hi = min(V, lo + p.row_per);
    if (tid < 64) {
        // rows of absent nodes are not read
        const int up = tid < p.k ? p.parents[static_cast<int64_t>(b) * p.k + tid] : -2;
        const bool wanted = row == 0 || __shfl(up, max(row - 1, 0)) != -2;
        if (KIND != kTreeGreedy) sh.pow2[tid] = pow2_entry(tid);
        if (tid == 0) {
            sh.ibcast[0] = wanted;
            sh.n_gone = 0;
        }
    }
    __syncthreads();
    double r[4] = {0.0, 0.0, 0.0, 0.0};
    if (sh.ibcast[0]) {
        const T* const x = static_cast<const T*>(p.target) + (static_cast<int64_t>(b) * (p.k + 1) + row) * V;
        if (KIND == kTreeGreedy) {
            float m;
            int where;
            slice_argmax(x, lo, hi, p.vec != 0, sh, &m, &where);
            r[0] = m;
            r[1] = where;
        } else {
            slice_stats(x, lo, hi, p.vec != 0, Scale(p), sh, &r[0], &r[1]);
        }
    }
    if (tid == 0)
        sh.ibcast[2] =
            hand_in(p.row_part + ((static_cast<int64_t>(b) * (p.k + 1) + row) * kTreeMaxSlices + slice) * 2, r, 2,
                    &p.arrived[b], static_cast<uint32_t>(p.row_slices) * (p.k + 1));
    __syncthreads();
    if (!sh.ibcast[2]) return;
    Node node{};
    if (tid < 64) node = node_of<T, KIND>(p, b);
    else join_rows<KIND>(p, b, sh);
    __syncthreads();
    if (tid < 64) {
        TreeState st{};
        begin<KIND>(p, b, node, st);
        Next nx{false, 0, 0, 0, 0.0, 0.0};
        if (st.stage == kStageDone) refuse(p, b);
        else nx = walk_rows<KIND>(p, b, node, st, sh);
        if (tid == 0) {
            sh.st = st;
            sh.nx = nx;
            p.arrived[b] = 0;
        }
    }
    __syncthreads();
    const TreeState st = sh.st;
    const Next nx = sh.nx;
    if (nx.draw) draw_token<T, KIND>(p, b, st, nx, sh);
}

// A value handed to the other workgroups: its low byte (2^-44 of it) is the
// pass's number, so that a word tells by itself whether it is this pass's.
__device__ __forceinline__ uint64_t tagged(double x, uint32_t pass) {
    return (static_cast<uint64_t>(__double_as_longlong(x)) & ~uint64_t{255}) | pass;
}

// The walks, p.slices workgroups to a sequence, each on its part of the
// vocabulary.  After each pass every workgroup reads the others' partials and
// takes the same decision from them, so nothing goes through memory but the
// partials, once; the one in whose part the token lies draws it.
//
// Waiting.  A sequence's workgroups have consecutive places on one die, whose
// dispatch is in order, so they come to run whatever else does.  Nothing
// depends on it: the wait is bounded (p.wait_ticks of 10 ns), a workgroup that
// gives up leaves, the first one leaves the state behind, and k_tree_walk ends
// the walk from there.
template <typename T, int KIND>
__global__ __launch_bounds__(NT, 4) void k_tree_cluster(TreePlan p) {
    __shared__ Shared sh;
    const int tid = threadIdx.x, lane = tid & 63;
    const int die = blockIdx.x % kTreeDies, on_die = blockIdx.x / kTreeDies;
    const int b = on_die / p.slices * kTreeDies + die, slice = on_die % p.slices;
    if (b >= p.batch) return;
    const bool lead = slice == 0;
    TreeState st{};
    Node node{};
    if (tid < 64) {
        if (KIND != kTreeGreedy) sh.pow2[tid] = pow2_entry(tid);
        node = node_of<T, KIND>(p, b);
        begin<KIND>(p, b, node, st);
        if (st.stage == kStageDone && lead) {
            refuse(p, b);
            if (tid == 0) p.finished[b] = 1;
        }
        if (tid == 0) {
            sh.st = st;
            sh.n_gone = 0;
        }
    }
    const int64_t V = p.vocab, lo = slice * p.per, hi = min(V, lo + p.per);
    const bool vec = p.vec != 0;
    uint64_t* const words = p.exchange + (static_cast<int64_t>(b) * p.slices) * 8;
    __syncthreads();
    for (uint32_t pass = 1; pass <= SV_MAX_DRAFT + 1u; ++pass) {
        st = sh.st;
        if (st.stage == kStageDone) return;  // a refused tree
        const Rows<T, KIND> rows(p, b, st);
        double r[4] = {0.0, 0.0, 0.0, 0.0};
        int n = KIND == kTreeGreedy || st.stage == kStageMass ? 1 : rows.draft ? 4 : 2;
        float best_m = 0.f;
        int best_at = 0;
        if (KIND == kTreeGreedy) {
            slice_argmax(rows.target, lo, hi, vec, sh, &best_m, &best_at);
        } else if (st.stage == kStageRow) {
            slice_stats(rows.target, lo, hi, vec, Scale(p), sh, &r[0], &r[1]);
            if (rows.draft) slice_stats(rows.draft, lo, hi, vec, Scale(p), sh, &r[2], &r[3]);
        } else {
            r[0] = slice_mass(rows.target, rows.draft, lo, hi, vec, Scale(p), st, sh);
        }
        if (tid < 64) {
            // Everything else of the sequence waits for this.
            __builtin_amdgcn_s_setprio(3);
            // Two sets of words in turn: a workgroup is at most one pass ahead
            // of the slowest, which still reads the other set.
            uint64_t* const set = words + (pass & 1) * 4;
            if (tid == 0) {
                if (KIND == kTreeGreedy) {
                    // an empty slice's index (all ones) is past every token
                    const uint64_t w = static_cast<uint64_t>(__float_as_uint(best_m)) << 32 |
                                       static_cast<uint64_t>(min(best_at, 0xFFFFFF)) << 8 | pass;
                    __hip_atomic_store(set + slice * 8, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (i < n)
                            __hip_atomic_store(set + slice * 8 + i, tagged(r[i], pass), __ATOMIC_RELAXED,
                                               __HIP_MEMORY_SCOPE_AGENT);
                }
            }
            const uint64_t began = __builtin_amdgcn_s_memrealtime();
            bool here = false;
            uint64_t w[4] = {0, 0, 0, 0};
            while (true) {
                bool ok = true;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i < n && lane < p.slices) {
                        w[i] = __hip_atomic_load(set + lane * 8 + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                        ok = ok && (w[i] & 255) == pass;
                    }
                here = __all(ok);
                if (here || __builtin_amdgcn_s_memrealtime() - began > p.wait_ticks) break;
                __builtin_amdgcn_s_sleep(1);
            }
            Next nx{false, 0, 0, 0, 0.0, 0.0};
            if (here) {
#pragma unroll
                for (int i = 0; i < 4; ++i) r[i] = __longlong_as_double(static_cast<long long>(w[i] & ~uint64_t{255}));
                if (KIND == kTreeGreedy) {
                    r[0] = __uint_as_float(static_cast<uint32_t>(w[0] >> 32));
                    r[1] = static_cast<double>((w[0] >> 8) & 0xFFFFFF);
                }
                nx = go_on<KIND>(p, b, node, st, r, lead, sh);
            }
            if (tid == 0) {
                sh.st = st;
                sh.nx = nx;
                sh.ibcast[1] = here;
                // what the walk goes on from, should this pass or the draw not be ended here
                if (lead && (!here || nx.draw)) p.state[b] = st;
            }
            __builtin_amdgcn_s_setprio(0);
        }
        __syncthreads();
        if (!sh.ibcast[1]) return;
        const Next nx = sh.nx;
        if (nx.draw) {
            const bool mine = KIND == kTreeGreedy ? lead : slice == nx.from / p.per;
            if (mine) {
                st = sh.st;
                draw_token<T, KIND>(p, b, st, nx, sh);
                if (tid == 0) p.finished[b] = 1;
            }
            return;
        }
    }
}

// The rest of a walk (all of it where no pass came before) by one workgroup
// per sequence.
template <typename T, int KIND>
__global__ __launch_bounds__(NT) void k_tree_walk(TreePlan p, int first) {
    __shared__ Shared sh;
    const int b = blockIdx.x;
    const int64_t V = p.vocab;
    const bool vec = p.vec != 0;
    Node node{};
    if (!first) {  // the workspace as the next call expects it
        const bool done = p.finished[b] != 0;
        __syncthreads();
        for (int i = threadIdx.x; i < p.slices * 8; i += NT) p.exchange[static_cast<int64_t>(b) * p.slices * 8 + i] = 0;
        if (threadIdx.x == 0) p.finished[b] = 0;
        if (done) return;
    }
    if (threadIdx.x < 64) {
        if (KIND != kTreeGreedy) sh.pow2[threadIdx.x] = pow2_entry(threadIdx.x);
        TreeState st{};
        if (!first) st = p.state[b];
        const bool ranged = first || in_range<KIND>(p, st);
        if (ranged) node = node_of<T, KIND>(p, b);
        if (first) begin<KIND>(p, b, node, st);
        if (first && st.stage == kStageDone) refuse(p, b);
        if (!first && (!ranged || !fits<KIND>(p, b, node, st))) st.stage = kStageDone;
        if (threadIdx.x == 0) {
            sh.st = st;
            sh.n_gone = 0;
        }
    }
    __syncthreads();
    while (true) {
        TreeState st = sh.st;
        if (st.stage == kStageDone) return;
        const Rows<T, KIND> rows(p, b, st);
        int best = 0;
        if (KIND == kTreeGreedy) {
            float m;
            slice_argmax(rows.target, 0, V, vec, sh, &m, &best);
        } else if (st.stage == kStageRow) {
            slice_stats(rows.target, 0, V, vec, Scale(p), sh, &st.m_t, &st.z_t);
            if (rows.draft) slice_stats(rows.draft, 0, V, vec, Scale(p), sh, &st.m_q, &st.z_q);
        } else {
            st.f = slice_mass(rows.target, rows.draft, 0, V, vec, Scale(p), st, sh);
        }
        __syncthreads();
        if (threadIdx.x < 64) {
            const bool draw = decide<KIND>(p, b, node, st, best, true, sh);
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
            const double all = st.stage == kStageMass ? st.f : 1.0 - gone_mass(sh, 0, V);
            const double u = p.uniforms[static_cast<int64_t>(b) * (p.k + 1) + p.k];
            y = draw_from<T, KIND>(rows.target, rows.draft, 0, V, vec, Scale(p), st, 0.0, u * all, sh);
        }
        if (threadIdx.x < 64) finish(p, b, st, y);
        return;
    }
}

template <typename T, int KIND>
hipError_t launch_kind(const TreePlan& p, hipStream_t stream) {
    if (p.slices == 1) {
        k_tree_walk<T, KIND><<<p.batch, NT, 0, stream>>>(p, 1);
        return hipGetLastError();
    }
    if constexpr (KIND != kTreeLogits) {
        if (p.row_part) {
            k_tree_rows<T, KIND><<<dim3(p.row_slices, p.k + 1, p.batch), NT, 0, stream>>>(p);
            return hipGetLastError();
        }
    }
    const int blocks = (p.batch + kTreeDies - 1) / kTreeDies * kTreeDies * p.slices;
    k_tree_cluster<T, KIND><<<blocks, NT, 0, stream>>>(p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    k_tree_walk<T, KIND><<<p.batch, NT, 0, stream>>>(p, 0);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_t(const TreePlan& p, hipStream_t stream) {
    switch (p.kind) {
        case kTreeGreedy: return launch_kind<T, kTreeGreedy>(p, stream);
        case kTreeOneHot: return launch_kind<T, kTreeOneHot>(p, stream);
        default: return launch_kind<T, kTreeLogits>(p, stream);
    }
}

}  // namespace

hipError_t launch_verify_tree(const TreePlan& p, hipStream_t stream) {
    return p.elem_bytes == 4 ? launch_t<float>(p, stream) : launch_t<uint16_t>(p, stream);
}

}  // namespace sv
