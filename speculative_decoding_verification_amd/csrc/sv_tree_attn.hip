// gfx950 kernels of sv_tree_attention: the rows of a drafted tree (its root
// and k nodes, several query heads to a key head) attend to a paged cache and
// to their own ancestors.
//
// Mathematics.  Row r of key head h sees the committed keys, the root and its
// ancestors: o_r = sum_j e^{s_rj - m_r} v_j / sum_j e^{s_rj - m_r}, s_rj =
// scale q_r . k_j.  One pass over the keys with a running maximum m and sum l
// (base 2: the scale carries log2 e); partial results (m, l, sum) over
// disjoint key ranges join exactly as l = sum_i l_i 2^{m_i - m}.
//
//  k_tree_attn     Work is cut into key tiles of 32 keys per wavefront.  A unit
//                  is one (sequence, key head, block of up to 64 query rows),
//                  the units of one key head a cluster; the tiles of all key
//                  heads stand in one line, and each cluster takes an equal run
//                  of it, whatever the lengths of the sequences are: a single
//                  long sequence is spread over the device and a ragged batch
//                  stays balanced, with no host knowledge of the lengths.  512
//                  workgroups run, two to a compute unit, so that one's loads go
//                  on while the other starts or ends a run; the workgroups of a
//                  cluster read the same keys at the same time on one die, so
//                  that its L2 gives all but the first their keys.  Within a
//                  workgroup the wavefronts take turns at 32-key steps, each
//                  with all of the unit's rows, so a wavefront's keys and values
//                  pass through LDS of its own and the loop holds no barrier.
//                  K and V rows go from memory straight to LDS
//                  (global_load_lds_dwordx4): K of the step after the next and V
//                  of the next are in flight while a step is computed, and page
//                  numbers go the same way (a load of one into a register makes
//                  the compiler wait for every load in flight).  Scores are
//                  formed transposed, S^T = K Q^T (v_mfma_f32_16x16x32), so a
//                  lane holds keys of one query row: maxima and sums need two
//                  lane exchanges, and the weights are in the operand layout of
//                  O^T = V^T P^T as they stand.  V^T comes from row-major V by
//                  the transposing LDS read (ds_read_b64_tr_b16).
//                  The maximum is raised only when a score passes it by 2^8
//                  (weights up to 256 are exact enough in 32-bit sums and in
//                  the 16-bit operand, whose relative rounding is the same), so
//                  most steps neither exchange lanes nor rescale.
//                  Weights are rounded to the cache's 16-bit type for the
//                  matrix product, by at most 2^-8 (bf16) or 2^-11 (f16) of
//                  themselves; sums, maxima and products are 32-bit.
//  k_tree_combine  Joins the partial results of units that several clusters
//                  share, in their order (no atomics: reproducible), and writes
//                  the zeros of absent sequences.
//
// What bounds it.  (k + 1) q_heads / kv_heads rows use each key: up to about 100
// rows memory does, beyond that the matrix cores.  Measured, both kernels
// (bf16 unless said, head size 128, 8 key heads):
//   1 sequence of 1000 keys, 4 rows a key head   9 + 4 us: launches, and two
//     trips to memory (the run, its pages) before the first key
//   64 x 2.9 K keys, 32 rows   142 + 10 us; its 709 MB take 101 us at the
//     7.0 TB/s of a plain read.  6.5 TB/s inside a run; its start (finding the
//     run 2 us, the first loads 2.5 us), its end and the combine are the rest
//   16 x 11 K keys, 520 rows, f16   640 + 16 us, 570 TFLOP/s of the 1330 that a
//     library product of 8192^3 reaches: matrix instructions take 26% of the
//     cycles, vector instructions, most of them the softmax's, 37%, and a SIMD
//     has one wavefront, which waits for the rest.  Units of 64 rows,
//     not fewer: 638 us against 734 with 48 and 1059 with 32, since each unit
//     reads the keys from the L2 again.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "specverify.h"
#include "sv_tree.h"

namespace sv {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef short shortx4_t __attribute__((ext_vector_type(4)));
typedef short shortx8_t __attribute__((ext_vector_type(8)));
typedef float floatx4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) shortx4_t lds_shortx4_t;

constexpr float kRaise = 8.f;  // log2 by which a score may pass the running maximum

template <bool F16>
__device__ __forceinline__ floatx4_t mma(shortx8_t a, shortx8_t b, floatx4_t c) {
    if constexpr (F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b),
                                                      c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                       __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

template <bool F16>
__device__ __forceinline__ short to16(float x) {
    if constexpr (F16)
        return __builtin_bit_cast(short, static_cast<_Float16>(x));
    else
        return __builtin_bit_cast(short, static_cast<__bf16>(x));
}

template <bool F16>
__device__ __forceinline__ float from16(uint16_t x) {
    if constexpr (F16)
        return static_cast<float>(__builtin_bit_cast(_Float16, x));
    else
        return __int_as_float(static_cast<int>(x) << 16);
}

template <bool F16>
__device__ __forceinline__ bool nonfinite16(uint32_t x) {
    constexpr uint32_t e = F16 ? 0x7C00u : 0x7F80u;
    return (x & e) == e;
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// 16-byte piece c of row r of a staged tile sits at piece c ^ swizzle(r), which
// spreads the rows that one LDS read touches over the banks.  K reads take one
// piece of 16 rows, V reads a pair of pieces of four rows; rows of 12 pieces
// (head size 96) start at four different bank groups by themselves, and the
// swizzle stays within groups of four pieces.
template <int D>
__device__ __forceinline__ int swizzle_k(int r) {
    if constexpr (D == 96) return (r >> 2) & 3;
    if constexpr (D == 64) return r & 7;
    return r & 15;
}
template <int D>
__device__ __forceinline__ int swizzle_v(int r) {
    if constexpr (D == 96) return (r >> 1) & 2;
    if constexpr (D == 64) return (2 * r) & 7;
    return (2 * r) & 15;
}

// Byte addresses of a lane's staged operands: piece kk of K's row, and for
// each block of 16 columns four keys of V's column (the transposing read wants
// the address of the piece that the lane brings in, not of its result).  For
// the powers of two the swizzle is an exclusive or of the address; for head
// size 96 it adds `odd` to even column blocks and takes it from odd ones.
template <int D>
struct KAddress {
    uint32_t base;
    __device__ __forceinline__ KAddress(uint32_t lds, int row, int g) {
        base = lds + row * (D * 2) + ((g ^ swizzle_k<D>(row)) << 4);
    }
    __device__ __forceinline__ uint32_t at(int kk) const { return base ^ (kk << 6); }
};

template <int D>
struct VAddress {
    uint32_t base;
    uint32_t odd;
    __device__ __forceinline__ VAddress(uint32_t lds, int lane) {
        const int i = lane & 15, r = (lane >> 4) * 4 + (i >> 2), pair = (i & 3) >> 1, sw = swizzle_v<D>(r);
        odd = D == 96 ? (sw >> 1) * 32 : 0;
        base = lds + r * (D * 2) + (D == 96 ? pair * 16 : (pair ^ sw) << 4) + (i & 1) * 8;
    }
    __device__ __forceinline__ uint32_t at(int db) const { return base ^ (db << 5); }
};

// All of a step's reads in one piece of assembly that waits for them: the
// compiler cannot tell a transposing read from the loads in flight to the other
// buffers and would wait for all of these too.  a[kb][kk]: K, 16 keys kb; lo,
// hi[db]: V, the first and second 16 keys; page: the lane's page number.
template <int D>
__device__ __forceinline__ void read_step(const KAddress<D>& k, const VAddress<D>& v, shortx8_t (&a)[2][D / 32],
                                          shortx4_t (&lo)[D / 16], shortx4_t (&hi)[D / 16],
                                          uint32_t page_at, int& page) {
    if constexpr (D == 64)
        asm volatile(
                     "ds_read_b128 %0, %13 offset:0\n\t"
                     "ds_read_b128 %1, %14 offset:0\n\t"
                     "ds_read_b128 %2, %13 offset:2048\n\t"
                     "ds_read_b128 %3, %14 offset:2048\n\t"
                     "ds_read_b64_tr_b16 %4, %15 offset:0\n\t"
                     "ds_read_b64_tr_b16 %5, %15 offset:2048\n\t"
                     "ds_read_b64_tr_b16 %6, %16 offset:0\n\t"
                     "ds_read_b64_tr_b16 %7, %16 offset:2048\n\t"
                     "ds_read_b64_tr_b16 %8, %17 offset:0\n\t"
                     "ds_read_b64_tr_b16 %9, %17 offset:2048\n\t"
                     "ds_read_b64_tr_b16 %10, %18 offset:0\n\t"
                     "ds_read_b64_tr_b16 %11, %18 offset:2048\n\t"
                     "ds_read_b32 %12, %19\n\t"
                     "s_waitcnt lgkmcnt(0)"
                     : "=&a"(a[0][0]), "=&a"(a[0][1]), "=&a"(a[1][0]), "=&a"(a[1][1]), "=&v"(lo[0]), "=&v"(hi[0]),
                       "=&v"(lo[1]), "=&v"(hi[1]), "=&v"(lo[2]), "=&v"(hi[2]), "=&v"(lo[3]), "=&v"(hi[3]), "=&v"(page)
                     : "v"(k.at(0)), "v"(k.at(1)), "v"(v.at(0)), "v"(v.at(1)), "v"(v.at(2)), "v"(v.at(3)), "v"(page_at)
                     : "memory");
    else if constexpr (D == 96)
        asm volatile(
                     "ds_read_b128 %0, %19 offset:0\n\t"
                     "ds_read_b128 %1, %19 offset:64\n\t"
                     "ds_read_b128 %2, %19 offset:128\n\t"
                     "ds_read_b128 %3, %19 offset:3072\n\t"
                     "ds_read_b128 %4, %19 offset:3136\n\t"
                     "ds_read_b128 %5, %19 offset:3200\n\t"
                     "ds_read_b64_tr_b16 %6, %20 offset:0\n\t"
                     "ds_read_b64_tr_b16 %7, %20 offset:3072\n\t"
                     "ds_read_b64_tr_b16 %8, %21 offset:32\n\t"
                     "ds_read_b64_tr_b16 %9, %21 offset:3104\n\t"
                     "ds_read_b64_tr_b16 %10, %20 offset:64\n\t"
                     "ds_read_b64_tr_b16 %11, %20 offset:3136\n\t"
                     "ds_read_b64_tr_b16 %12, %21 offset:96\n\t"
                     "ds_read_b64_tr_b16 %13, %21 offset:3168\n\t"
                     "ds_read_b64_tr_b16 %14, %20 offset:128\n\t"
                     "ds_read_b64_tr_b16 %15, %20 offset:3200\n\t"
                     "ds_read_b64_tr_b16 %16, %21 offset:160\n\t"
                     "ds_read_b64_tr_b16 %17, %21 offset:3232\n\t"
                     "ds_read_b32 %18, %22\n\t"
                     "s_waitcnt lgkmcnt(0)"
                     : "=&a"(a[0][0]), "=&a"(a[0][1]), "=&a"(a[0][2]), "=&a"(a[1][0]), "=&a"(a[1][1]),
                       "=&a"(a[1][2]), "=&v"(lo[0]), "=&v"(hi[0]), "=&v"(lo[1]), "=&v"(hi[1]), "=&v"(lo[2]),
                       "=&v"(hi[2]), "=&v"(lo[3]), "=&v"(hi[3]), "=&v"(lo[4]), "=&v"(hi[4]), "=&v"(lo[5]),
                       "=&v"(hi[5]), "=&v"(page)
                     : "v"(k.base), "v"(v.base + v.odd), "v"(v.base - v.odd), "v"(page_at)
                     : "memory");
    else if constexpr (D == 128)
        asm volatile(
                     "ds_read_b128 %0, %25 offset:0\n\t"
                     "ds_read_b128 %1, %26 offset:0\n\t"
                     "ds_read_b128 %2, %27 offset:0\n\t"
                     "ds_read_b128 %3, %28 offset:0\n\t"
                     "ds_read_b128 %4, %25 offset:4096\n\t"
                     "ds_read_b128 %5, %26 offset:4096\n\t"
                     "ds_read_b128 %6, %27 offset:4096\n\t"
                     "ds_read_b128 %7, %28 offset:4096\n\t"
                     "ds_read_b64_tr_b16 %8, %29 offset:0\n\t"
                     "ds_read_b64_tr_b16 %9, %29 offset:4096\n\t"
                     "ds_read_b64_tr_b16 %10, %30 offset:0\n\t"
                     "ds_read_b64_tr_b16 %11, %30 offset:4096\n\t"
                     "ds_read_b64_tr_b16 %12, %31 offset:0\n\t"
                     "ds_read_b64_tr_b16 %13, %31 offset:4096\n\t"
                     "ds_read_b64_tr_b16 %14, %32 offset:0\n\t"
                     "ds_read_b64_tr_b16 %15, %32 offset:4096\n\t"
                     "ds_read_b64_tr_b16 %16, %33 offset:0\n\t"
                     "ds_read_b64_tr_b16 %17, %33 offset:4096\n\t"
                     "ds_read_b64_tr_b16 %18, %34 offset:0\n\t"
                     "ds_read_b64_tr_b16 %19, %34 offset:4096\n\t"
                     "ds_read_b64_tr_b16 %20, %35 offset:0\n\t"
                     "ds_read_b64_tr_b16 %21, %35 offset:4096\n\t"
                     "ds_read_b64_tr_b16 %22, %36 offset:0\n\t"
                     "ds_read_b64_tr_b16 %23, %36 offset:4096\n\t"
                     "ds_read_b32 %24, %37\n\t"
                     "s_waitcnt lgkmcnt(0)"
                     : "=&a"(a[0][0]), "=&a"(a[0][1]), "=&a"(a[0][2]), "=&a"(a[0][3]), "=&a"(a[1][0]),
                       "=&a"(a[1][1]), "=&a"(a[1][2]), "=&a"(a[1][3]), "=&v"(lo[0]), "=&v"(hi[0]), "=&v"(lo[1]),
                       "=&v"(hi[1]), "=&v"(lo[2]), "=&v"(hi[2]), "=&v"(lo[3]), "=&v"(hi[3]), "=&v"(lo[4]),
                       "=&v"(hi[4]), "=&v"(lo[5]), "=&v"(hi[5]), "=&v"(lo[6]), "=&v"(hi[6]), "=&v"(lo[7]),
                       "=&v"(hi[7]), "=&v"(page)
                     : "v"(k.at(0)), "v"(k.at(1)), "v"(k.at(2)), "v"(k.at(3)), "v"(v.at(0)), "v"(v.at(1)),
                       "v"(v.at(2)), "v"(v.at(3)), "v"(v.at(4)), "v"(v.at(5)), "v"(v.at(6)), "v"(v.at(7)), "v"(page_at)
                     : "memory");
    else
        asm volatile(
                     "ds_read_b128 %0, %49 offset:0\n\t"
                     "ds_read_b128 %1, %50 offset:0\n\t"
                     "ds_read_b128 %2, %51 offset:0\n\t"
                     "ds_read_b128 %3, %52 offset:0\n\t"
                     "ds_read_b128 %4, %53 offset:0\n\t"
                     "ds_read_b128 %5, %54 offset:0\n\t"
                     "ds_read_b128 %6, %55 offset:0\n\t"
                     "ds_read_b128 %7, %56 offset:0\n\t"
                     "ds_read_b128 %8, %49 offset:8192\n\t"
                     "ds_read_b128 %9, %50 offset:8192\n\t"
                     "ds_read_b128 %10, %51 offset:8192\n\t"
                     "ds_read_b128 %11, %52 offset:8192\n\t"
                     "ds_read_b128 %12, %53 offset:8192\n\t"
                     "ds_read_b128 %13, %54 offset:8192\n\t"
                     "ds_read_b128 %14, %55 offset:8192\n\t"
                     "ds_read_b128 %15, %56 offset:8192\n\t"
                     "ds_read_b64_tr_b16 %16, %57 offset:0\n\t"
                     "ds_read_b64_tr_b16 %17, %57 offset:8192\n\t"
                     "ds_read_b64_tr_b16 %18, %58 offset:0\n\t"
                     "ds_read_b64_tr_b16 %19, %58 offset:8192\n\t"
                     "ds_read_b64_tr_b16 %20, %59 offset:0\n\t"
                     "ds_read_b64_tr_b16 %21, %59 offset:8192\n\t"
                     "ds_read_b64_tr_b16 %22, %60 offset:0\n\t"
                     "ds_read_b64_tr_b16 %23, %60 offset:8192\n\t"
                     "ds_read_b64_tr_b16 %24, %61 offset:0\n\t"
                     "ds_read_b64_tr_b16 %25, %61 offset:8192\n\t"
                     "ds_read_b64_tr_b16 %26, %62 offset:0\n\t"
                     "ds_read_b64_tr_b16 %27, %62 offset:8192\n\t"
                     "ds_read_b64_tr_b16 %28, %63 offset:0\n\t"
                     "ds_read_b64_tr_b16 %29, %63 offset:8192\n\t"
                     "ds_read_b64_tr_b16 %30, %64 offset:0\n\t"
                     "ds_read_b64_tr_b16 %31, %64 offset:8192\n\t"
                     "ds_read_b64_tr_b16 %32, %65 offset:0\n\t"
                     "ds_read_b64_tr_b16 %33, %65 offset:8192\n\t"
                     "ds_read_b64_tr_b16 %34, %66 offset:0\n\t"
                     "ds_read_b64_tr_b16 %35, %66 offset:8192\n\t"
                     "ds_read_b64_tr_b16 %36, %67 offset:0\n\t"
                     "ds_read_b64_tr_b16 %37, %67 offset:8192\n\t"
                     "ds_read_b64_tr_b16 %38, %68 offset:0\n\t"
                     "ds_read_b64_tr_b16 %39, %68 offset:8192\n\t"
                     "ds_read_b64_tr_b16 %40, %69 offset:0\n\t"
                     "ds_read_b64_tr_b16 %41, %69 offset:8192\n\t"
                     "ds_read_b64_tr_b16 %42, %70 offset:0\n\t"
                     "ds_read_b64_tr_b16 %43, %70 offset:8192\n\t"
                     "ds_read_b64_tr_b16 %44, %71 offset:0\n\t"
                     "ds_read_b64_tr_b16 %45, %71 offset:8192\n\t"
                     "ds_read_b64_tr_b16 %46, %72 offset:0\n\t"
                     "ds_read_b64_tr_b16 %47, %72 offset:8192\n\t"
                     "ds_read_b32 %48, %73\n\t"
                     "s_waitcnt lgkmcnt(0)"
                     : "=&a"(a[0][0]), "=&a"(a[0][1]), "=&a"(a[0][2]), "=&a"(a[0][3]), "=&a"(a[0][4]),
                       "=&a"(a[0][5]), "=&a"(a[0][6]), "=&a"(a[0][7]), "=&a"(a[1][0]), "=&a"(a[1][1]),
                       "=&a"(a[1][2]), "=&a"(a[1][3]), "=&a"(a[1][4]), "=&a"(a[1][5]), "=&a"(a[1][6]),
                       "=&a"(a[1][7]), "=&v"(lo[0]), "=&v"(hi[0]), "=&v"(lo[1]), "=&v"(hi[1]), "=&v"(lo[2]),
                       "=&v"(hi[2]), "=&v"(lo[3]), "=&v"(hi[3]), "=&v"(lo[4]), "=&v"(hi[4]), "=&v"(lo[5]),
                       "=&v"(hi[5]), "=&v"(lo[6]), "=&v"(hi[6]), "=&v"(lo[7]), "=&v"(hi[7]), "=&v"(lo[8]),
                       "=&v"(hi[8]), "=&v"(lo[9]), "=&v"(hi[9]), "=&v"(lo[10]), "=&v"(hi[10]), "=&v"(lo[11]),
                       "=&v"(hi[11]), "=&v"(lo[12]), "=&v"(hi[12]), "=&v"(lo[13]), "=&v"(hi[13]), "=&v"(lo[14]),
                       "=&v"(hi[14]), "=&v"(lo[15]), "=&v"(hi[15]), "=&v"(page)
                     : "v"(k.at(0)), "v"(k.at(1)), "v"(k.at(2)), "v"(k.at(3)), "v"(k.at(4)), "v"(k.at(5)),
                       "v"(k.at(6)), "v"(k.at(7)), "v"(v.at(0)), "v"(v.at(1)), "v"(v.at(2)), "v"(v.at(3)),
                       "v"(v.at(4)), "v"(v.at(5)), "v"(v.at(6)), "v"(v.at(7)), "v"(v.at(8)), "v"(v.at(9)),
                       "v"(v.at(10)), "v"(v.at(11)), "v"(v.at(12)), "v"(v.at(13)), "v"(v.at(14)), "v"(v.at(15)), "v"(page_at)
                     : "memory");
}

__device__ __forceinline__ int parent_of(const AttnPlan& p, int b, int lane) {
    return lane < p.k ? p.parents[static_cast<int64_t>(b) * p.k + lane] : -2;
}

// Ancestors of draft node `lane`, of parent `up`, as a bit mask (itself included; 0 for an
// absent node: parent -2, out of range, or absent itself), by doubling.
__device__ __forceinline__ uint64_t ancestors(int up, int lane) {
    if (up >= lane || up < -2) up = -2;
    uint64_t mask = up == -2 ? 0 : (uint64_t{1} << lane);
    bool gone = up == -2;
#pragma unroll
    for (int i = 0; i < 6; ++i) {
        const int from = up < 0 ? lane : up;
        const uint64_t m = __shfl(static_cast<unsigned long long>(mask), from);
        const int u = __shfl(up, from);
        if (up >= 0) {
            mask |= m;
            up = u;
        }
        gone = gone || up == -2;
    }
    return gone ? 0 : mask;
}

// Key tiles of a sequence of n committed keys (0: absent, a negative length
// or one that its page table row cannot hold).
__device__ __forceinline__ int tiles_of(const AttnPlan& p, int n, int tile_keys) {
    const int64_t keys = static_cast<int64_t>(n) + p.k + 1;
    if (n < 0 || keys > (static_cast<int64_t>(p.max_pages) << p.page_shift)) return 0;
    return static_cast<int>((keys + tile_keys - 1) / tile_keys);
}

// Inclusive sum over the workgroup's threads, and the total.  A sequence has
// at most 2^24 tiles, so a wavefront's sums fit 32 bits.
template <int NT>
__device__ __forceinline__ int64_t block_scan(int v, int64_t* total, int64_t* tmp) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(v, d);
        if (lane >= d) v += o;
    }
    if constexpr (NT == 64) {
        *total = __builtin_amdgcn_readlane(v, 63);
        return v;
    }
    __syncthreads();
    if (lane == 63) tmp[wave] = v;
    __syncthreads();
    int64_t all = 0, mine = v;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) {
        if (w < wave) mine += tmp[w];
        all += tmp[w];
    }
    *total = all;
    return mine;
}

// What a workgroup finds of the line of all sequences' key tiles, key head
// by key head: its run, and where the run begins.
struct Line {
    int64_t begin, end, share;
    int b, len;     // the sequence that `begin` lies in, and its committed keys
    int64_t b_off;  // the line's index of that sequence's first tile
};

template <int NT>
__device__ __forceinline__ Line find_run(const AttnPlan& p, int cluster, int tile_keys, int64_t* tmp) {
    __shared__ int64_t found_off;
    __shared__ int found_b, found_len;
    const int heads = p.kv_heads, tid = threadIdx.x;
    Line r;
    int64_t total = 0, before_all = 0, incl = 0, all;
    int n = -1, mine = 0;
    for (int c = 0; c < p.batch; c += NT) {
        n = c + tid < p.batch ? p.seq_len[c + tid] : -1;
        mine = tiles_of(p, n, tile_keys);
        incl = block_scan<NT>(mine, &all, tmp);
        total += all;
    }
    const bool once = p.batch <= NT;  // the one scan has it all
    total *= heads;
    r.share = (total + p.clusters - 1) / p.clusters;
    if (r.share < 1) r.share = 1;
    r.begin = cluster * r.share;
    r.end = min(r.begin + r.share, total);
    if (r.begin >= r.end) return r;
    for (int c = 0; c < p.batch; c += NT) {
        if (!once) {
            n = c + tid < p.batch ? p.seq_len[c + tid] : -1;
            mine = tiles_of(p, n, tile_keys);
            incl = block_scan<NT>(mine, &all, tmp);
        }
        const int64_t before = before_all + incl - mine;
        if (mine > 0 && r.begin >= before * heads && r.begin < (before + mine) * heads) {
            found_b = c + tid;
            found_len = n;
            found_off = before * heads;
        }
        before_all += all;
        if (once || before_all * heads > r.begin) break;
    }
    __syncthreads();
    r.b = found_b;
    r.len = found_len;
    r.b_off = found_off;
    return r;
}

template <bool F16, int D, int MT>
__global__ __launch_bounds__(attn_waves(D) * 64, 1) void k_tree_attn(AttnPlan p) {
    constexpr int NW = attn_waves(D);
    constexpr int NT = NW * 64;
    constexpr int STEP = kAttnStep;
    constexpr int TILE = NW * STEP;           // keys of one tile: a step of each wavefront
    constexpr int CH = D / 8;                 // 16-byte pieces of a row
    constexpr int NL = STEP * CH / 64;        // direct-to-LDS loads of one step and operand
    constexpr int KK = D / 32;                // matrix steps along the head
    constexpr int DB = D / 16;                // output blocks along the head
    static_assert(STEP * CH % 64 == 0 && 2 * NL < 63, "whole loads, countable");
    // Two steps' K and V for each wavefront: [wavefront][K, V][step parity].
    // At the end of a run they hold the wavefronts' sums, a buffer's size for
    // each row tile.
    constexpr int BUF = STEP * D;  // elements of one buffer
    __shared__ __attribute__((aligned(1024))) uint16_t stage[NW * 4 * BUF];
    __shared__ float wave_m[NW][MT * 16], wave_l[NW][MT * 16];
    __shared__ float row_f[MT * 16];      // what a row's sum is multiplied by as it is written
    __shared__ int64_t row_to[MT * 16];   // where: row of the output, or of the partial results; -1 nowhere
    __shared__ int wave_odd[NW];  // whether the wavefront met a tree row's value that is not finite
    __shared__ uint64_t ancs[NW][SV_MAX_DRAFT];  // each wavefront's own copy: it needs no barrier
    __shared__ int32_t pages[NW][2][64];  // page numbers of steps to come, by parity
    __shared__ int64_t scan_tmp[NW];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);  // one value a wavefront: what follows from it stays scalar
    const int q_of = lane & 15, g = lane >> 4;
    const uint16_t* const kc = static_cast<const uint16_t*>(p.k_cache);
    const uint16_t* const vc = static_cast<const uint16_t*>(p.v_cache);
    const int page_mask = (1 << p.page_shift) - 1;
    // Blocks are dealt to the eight dies in turn; a cluster's stand on one die.
    const int on_die = blockIdx.x / kAttnDies, per_die = p.clusters / kAttnDies;
    const int cluster = (blockIdx.x % kAttnDies) * per_die + on_die / p.cluster;
    const bool works = on_die < per_die * p.cluster;
    Line run{0, 0, 1, 0, 0, 0};
    if (works) run = find_run<NT>(p, cluster, TILE, scan_tmp);

    for (int ru = on_die % p.cluster; works && ru < p.row_units; ru += p.cluster) {
    int64_t pos = run.begin;
    int b = run.b, len = run.len;
    int64_t seq_off = run.b_off;  // the line's index of sequence b's first tile
    AttnSplit split{-1, 0, 0, 0};
    int nt = pos < run.end ? tiles_of(p, len, TILE) : 0;
    while (pos < run.end) {
        while (pos >= seq_off + static_cast<int64_t>(nt) * p.kv_heads) {  // the next sequence that has tiles
            seq_off += static_cast<int64_t>(nt) * p.kv_heads;
            ++b;
            len = p.seq_len[b];
            nt = tiles_of(p, len, TILE);
        }
        const int64_t in_seq = pos - seq_off;
        const int h = static_cast<int>(in_seq / nt);
        const int64_t unit_off = seq_off + static_cast<int64_t>(h) * nt;
        const int t0 = static_cast<int>(pos - unit_off);
        const int t1 = static_cast<int>(min<int64_t>(nt, t0 + (run.end - pos)));
        int row0 = ru * (MT * 16);
        asm volatile("" : "+s"(row0));  // what follows from it is worked out in place: hoisted out of the loop over the
                                        // key heads it would hold registers through the steps
        const int keys = len + p.k + 1;
        const int steps = t1 - t0;
        const auto key_of = [&](int s) { return ((t0 + s) * NW + wave) * STEP; };
        const int32_t* const table = p.page_table + static_cast<int64_t>(b) * p.max_pages;
        // Everything that the first steps need is asked for at once; of the
        // pages, those of the keys themselves, and the root's.
        const auto page_of = [&](int s) {
            return table + (min(key_of(min(s, steps - 1)) + (lane & 31), keys - 1) >> p.page_shift);
        };
        const int pa = *page_of(0), pb = *page_of(1), pc = *page_of(2), pd = *page_of(3);
        const int root_page = table[len >> p.page_shift];
        const int up = parent_of(p, b, lane);

        shortx8_t qf[MT][KK];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int r = min(row0 + mt * 16 + q_of, p.rows - 1);
            const int node = r / p.group, head = h * p.group + r - node * p.group;
            const uint16_t* src = static_cast<const uint16_t*>(p.q) + static_cast<int64_t>(b) * p.q_stride_b +
                                  static_cast<int64_t>(node) * p.q_stride_r + static_cast<int64_t>(head) * p.q_stride_h;
#pragma unroll
            for (int kk = 0; kk < KK; ++kk)
                qf[mt][kk] = *reinterpret_cast<const shortx8_t*>(src + (kk * 4 + g) * 8);
        }
        const uint64_t own_mask = p.k > 0 ? ancestors(up, lane) : 0;
        const uint64_t present = __ballot(own_mask != 0);
        uint64_t* const anc = ancs[wave];
        anc[lane] = own_mask;
        // Queries and page numbers are here: without this wait the compiler
        // would wait for the queries inside the loop, and so for all loads.
        __builtin_amdgcn_s_waitcnt(0x0F70);

        floatx4_t acc[MT][DB];
        float m[MT], l[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            m[mt] = -__builtin_inff();
            l[mt] = 0.f;
#pragma unroll
            for (int db = 0; db < DB; ++db) acc[mt][db] = floatx4_t{0.f, 0.f, 0.f, 0.f};
        }

        // Steps whose keys are all committed ones come first.
        const int full = min(steps, max(0, (len - wave * STEP) / STEP + NW - 1) / NW - t0);
        // Steps that hold any key for this wavefront.
        const int mine_n = min(steps, max(0, (keys - wave * STEP + STEP - 1) / STEP + NW - 1) / NW - t0);
        uint16_t* const mine = stage + wave * (4 * BUF);
        const uint32_t lds = static_cast<uint32_t>(
            reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint16_t*)mine));
        const KAddress<D> k_at(lds, q_of, g);
        const VAddress<D> v_at(lds + 2 * BUF * 2, lane);
        // Row of the cache (of head_dim elements) for the position that lane
        // (mod 32) stands for in step s.  Positions past the last key, and slots
        // of absent nodes, may hold anything (a NaN would spoil a product even
        // at weight 0): the root's row is read in their place.  Page numbers out
        // of range are read as page 0: the result is then unspecified, the
        // access in bounds.
        const auto row_at = [&](int page, int pos) {
            const uint32_t id = static_cast<uint32_t>(page) < static_cast<uint32_t>(p.n_pages) ? page : 0;
            return ((id * p.kv_heads + h) << p.page_shift) + (pos & page_mask);
        };
        const uint32_t root_row = row_at(root_page, len);
        const auto row_of = [&](int s, int page) {
            const int key = key_of(min(s, steps - 1)) + (lane & 31);
            const uint32_t row = row_at(page, key);
            if (s < full) return row;
            const int j = key - len - 1;
            const bool there = j < 0 || (j < p.k && ((present >> (j & 63)) & 1));
            return there ? row : root_row;
        };
        // One operand's rows of a step, straight to LDS.  A load takes whole
        // rows for the head sizes that are powers of two, and where these stand
        // together in one page its address is one base for all lanes; otherwise
        // every lane takes its row's.
        const auto dma = [&](const uint16_t* cache, uint16_t* to, int s, uint32_t row, const auto& swizzle) {
            constexpr int RPI = 512 / D;  // rows of one load
            if (D != 96 && s < full && (1 << p.page_shift) >= RPI) {
#pragma unroll
                for (int i = 0; i < NL; ++i) {
                    const int r = i * RPI + lane / CH, c = lane % CH;
                    const uint32_t first = __builtin_amdgcn_readlane(row, i * RPI);
                    const char* const base = reinterpret_cast<const char*>(cache) + static_cast<uint64_t>(first) * (D * 2);
                    const uint32_t off = (lane / CH) * (D * 2) + ((c ^ swizzle(r)) << 4);
                    __builtin_amdgcn_global_load_lds((const void*)(base + off),
                        (__attribute__((address_space(3))) void*)(to + i * 512), 16, 0, 0);
                }
            } else {
                int ln = lane;
                asm volatile("" : "+v"(ln));  // worked out where it is needed: hoisted, these offsets cost 32 registers
#pragma unroll
                for (int i = 0; i < NL; ++i) {
                    const int e = i * 64 + ln;
                    const int r = e / CH, c = e - r * CH;
                    const uint64_t at = static_cast<uint64_t>(static_cast<uint32_t>(__shfl(static_cast<int>(row), r))) * D;
                    __builtin_amdgcn_global_load_lds((const void*)(cache + at + ((c ^ swizzle(r)) << 3)),
                        (__attribute__((address_space(3))) void*)(to + i * 512), 16, 0, 0);
                }
            }
        };
        const auto k_dma = [&](int s, uint32_t row) { dma(kc, mine + (s & 1) * BUF, s, row, swizzle_k<D>); };
        const auto v_dma = [&](int s, uint32_t row) { dma(vc, mine + (2 + (s & 1)) * BUF, s, row, swizzle_v<D>); };
        // Scores of 32 keys, transposed: lane's row q_of, keys 16 kb + 4 g + i.
        const auto scores = [&](const shortx8_t (&a)[2][KK], floatx4_t (&sc)[MT][2]) {
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int kk = 0; kk < KK; ++kk)
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
                        sc[mt][kb] = mma<F16>(a[kb][kk], qf[mt][kk], kk ? sc[mt][kb] : floatx4_t{0.f, 0.f, 0.f, 0.f});
        };
        // The scores that a row's ancestry hides become -inf.
        const auto hide = [&](int s, floatx4_t (&sc)[MT][2]) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const int node = min(row0 + mt * 16 + q_of, p.rows - 1) / p.group;
                const uint64_t see = node == 0 ? 0 : anc[node - 1];  // the draft nodes that the lane's row sees
                uint32_t seen = 0;                                   // which of the lane's 8 keys it does
#pragma unroll
                for (int kb = 0; kb < 2; ++kb) {
                    // of the draft node at the lane's first key; -1 is the root, committed keys are below
                    const int j = key_of(s) + kb * 16 + g * 4 - len - 1;
                    const uint32_t low = j >= 0 ? static_cast<uint32_t>(j < 64 ? see >> j : 0)
                                                : static_cast<uint32_t>(see << min(-j, 4)) | ((1u << min(-j, 4)) - 1);
                    seen |= (low & 15u) << (kb * 4);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    sc[mt][i >> 2][i & 3] = (seen >> i) & 1 ? sc[mt][i >> 2][i & 3] : -__builtin_inff();
            }
        };
        // Whether a score passes its row's maximum by 2^kRaise; raise() then
        // takes the maxima up to it.  The sums are rescaled outside the loop
        // over steps that need it not: a branch over them inside made the
        // compiler copy all accumulators at every step.
        const auto top_of = [&](const floatx4_t (&sc)[MT][2], int mt) {
            float t = sc[mt][0][0];
#pragma unroll
            for (int i = 1; i < 8; ++i) t = fmaxf(t, sc[mt][i >> 2][i & 3]);
            return t * p.scale_log2;
        };
        const auto past = [&](const floatx4_t (&sc)[MT][2]) {
            bool any = false;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) any = any || top_of(sc, mt) > m[mt] + kRaise;
            return __any(any) != 0;
        };
        const auto raise = [&](const floatx4_t (&sc)[MT][2]) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                float t = top_of(sc, mt);
                t = fmaxf(t, __shfl_xor(t, 16));
                t = fmaxf(t, __shfl_xor(t, 32));
                const float mn = fmaxf(m[mt], t);
                const float f = m[mt] == mn ? 1.f : exp2_fast(m[mt] - mn);
                m[mt] = mn;
                l[mt] *= f;
#pragma unroll
                for (int db = 0; db < DB; ++db) {
                    acc[mt][db] *= f;
                    __builtin_amdgcn_sched_barrier(0);  // one after the other: all at once they fill the vector registers
                }
            }
        };
        const auto weights = [&](int mt, const floatx4_t (&sc)[MT][2]) {
            const float ms = m[mt] == -__builtin_inff() ? 0.f : m[mt];
            shortx8_t pf;
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float w = exp2_fast(__builtin_fmaf(sc[mt][i >> 2][i & 3], p.scale_log2, -ms));
                sum += w;
                pf[i] = to16<F16>(w);
            }
            l[mt] += sum;
            return pf;
        };
        // A value that is not finite must reach only the rows that see its
        // node, and the matrix product would multiply it by the other rows'
        // zero weights.  Such values (there are hardly ever any) are cleared
        // here and added where the sums are written.
        bool odd = false;
        const auto clear_odd = [&](int s) {
            uint4* const vs = reinterpret_cast<uint4*>(mine + (2 + (s & 1)) * BUF);
            constexpr uint32_t e = F16 ? 0x7C007C00u : 0x7F807F80u;
            bool here = false;
#pragma unroll
            for (int i = 0; i < BUF / 512; ++i) {
                const uint4 x = vs[i * 64 + lane];
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {  // a half of y is 0 where that value's exponent is all ones
                    const uint32_t y = (w[j] & e) ^ e;
                    here = here || (((y - 0x00010001u) & ~y & 0x80008000u) != 0);
                }
            }
            if (__any(here)) {
                uint16_t* const v = mine + (2 + (s & 1)) * BUF;
#pragma unroll 1
                for (int r = max(0, len - key_of(s)); r < STEP; ++r)  // the tree's rows only: every row sees the others
#pragma unroll 1
                    for (int d = lane; d < D; d += 64)
                        if (nonfinite16<F16>(v[r * D + d])) {
                            v[r * D + d] = 0;
                            odd = true;
                        }
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            }
        };

        // While step s is worked on, the scores of step s + 1 are formed (its K
        // has landed), and K of steps s + 2 and s + 3 and V of steps s + 1 and
        // s + 2 are on their way: a buffer is filled again as soon as it has
        // been read.  Page numbers are asked for a step ahead of the rows.
        // Nothing is loaded past the last step, so the last two steps wait for
        // fewer loads in flight.
        constexpr int kOne = NL, kTwo = 2 * NL;
        const auto landed = [&](auto left) {  // all but the last `left` loads
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_waitcnt(0x0F70 | (decltype(left)::value & 15) | ((decltype(left)::value >> 4) << 14));
            asm volatile("" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
        };
        floatx4_t sc[MT][2], next[MT][2];
        shortx8_t a[2][KK];
        shortx4_t lo[DB], hi[DB];
        // Page numbers go through LDS too: for one loaded to a register the
        // compiler would wait for every load in flight.
        const auto page_dma = [&](int s) {
            __builtin_amdgcn_global_load_lds((const void*)page_of(s),
                (__attribute__((address_space(3))) void*)&pages[wave][s & 1][0], 4, 0, 0);
        };
        const uint32_t pages_at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
            (__attribute__((address_space(3))) int32_t*)&pages[wave][0][lane]));
        int page;
        const auto read = [&](int s) {  // K of step s, V of step s - 1, the pages of step s + 3
            KAddress<D> k = k_at;
            VAddress<D> v = v_at;
            k.base += (s & 1) * (BUF * 2);
            v.base += (~s & 1) * (BUF * 2);
            read_step<D>(k, v, a, lo, hi, pages_at + (~s & 1) * 256, page);
        };
        uint32_t row_v, row_k;  // of steps s + 2 and s + 3
        {
            const uint32_t r0 = row_of(0, pa), r1 = row_of(1, pb);
            row_v = row_of(2, pc);
            row_k = row_of(3, pd);
            if (mine_n > 0) {
                page_dma(4);
                k_dma(0, r0);
                if (mine_n > 1) k_dma(1, r1);
                v_dma(0, r0);
                if (mine_n > 1) landed(std::integral_constant<int, kTwo>{});
                else landed(std::integral_constant<int, kOne>{});
                read(0);  // (nothing of V yet)
                scores(a, sc);
                if (mine_n > 2) k_dma(2, row_v);
                if (mine_n > 1) v_dma(1, r1);
            }
        }
        const auto step = [&](auto hot, int s) {
            constexpr bool HOT = decltype(hot)::value;
            if (HOT || s + 2 < mine_n) landed(std::integral_constant<int, kTwo>{});
            else if (s + 2 == mine_n) landed(std::integral_constant<int, kOne>{});
            else landed(std::integral_constant<int, 0>{});
            if (!HOT && s >= full) clear_odd(s);
            read(s + 1);
            page_dma(s + 5);
            if (HOT || s + 3 < mine_n) k_dma(s + 3, row_k);
            if (HOT || s + 2 < mine_n) v_dma(s + 2, row_v);
            __builtin_amdgcn_sched_barrier(0);
            // One block without branches or memory: the next step's scores and
            // this one's products on the matrix cores, its weights beside them.
            scores(a, next);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                // Key slot j of the product's lane group g is key 4g + j of the
                // first 16 keys, for j >= 4 key 4g + j - 4 of the second: the
                // weights stand so already, and the transposing read gave each
                // lane four keys of one column.
                const shortx8_t pf = weights(mt, sc);
#pragma unroll
                for (int db = 0; db < DB; ++db)
                    acc[mt][db] = mma<F16>(__builtin_shufflevector(lo[db], hi[db], 0, 1, 2, 3, 4, 5, 6, 7), pf, acc[mt][db]);
            }
#pragma unroll
            for (int i = 0; i < MT * (2 * KK + DB); ++i) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // a matrix instruction,
                __builtin_amdgcn_sched_group_barrier(0x002, 2, 0);  // two vector ones
            }
            __builtin_amdgcn_sched_barrier(0);
            row_v = row_k;
            row_k = row_of(s + 4, page);
            if (!HOT && s + 1 >= full) hide(s + 1, next);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                sc[mt][0] = next[mt][0];
                sc[mt][1] = next[mt][1];
            }
        };
        if (full <= 0 && mine_n > 0) hide(0, sc);
        // Steps that are followed by three more and have only committed keys,
        // the next one's too, need none of the conditions (and with a load that
        // may not be there the compiler would wait for all of them at each
        // page number).
        const int hot_n = min(mine_n - 3, full - 1);
        for (int s = 0; s < mine_n;) {
            raise(sc);
            bool again = false;
            while (s < hot_n) {
                step(std::true_type{}, s++);
                if ((again = past(sc))) break;
            }
            if (again) continue;
            while (s < mine_n) {
                step(std::false_type{}, s++);
                if (s < mine_n && past(sc)) break;
            }
        }
        __builtin_amdgcn_s_waitcnt(0x0F70);  // no load may land in a buffer that holds sums
        asm volatile("" ::: "memory");

        // Join the wavefronts.
        int thread = tid;
        asm volatile("" : "+v"(thread), "+s"(row0));  // as above
        const int q_at = thread & 15, g_at = (thread & 63) >> 4;
        odd = __any(odd);
        if (lane == 0) wave_odd[wave] = odd;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            float t = l[mt] + __shfl_xor(l[mt], 16);
            t += __shfl_xor(t, 32);
            if (g_at == 0) {
                wave_m[wave][mt * 16 + q_at] = m[mt];
                wave_l[wave][mt * 16 + q_at] = t;
            }
        }
        __syncthreads();  // and every wavefront has left the buffers
        const bool whole = t0 == 0 && t1 == nt;
        // A cluster's first slot takes the keys that its run begins with, its
        // second those that go on in the next run.
        const int second = pos != run.begin;
        if (t0 == 0 && !whole)
            split = AttnSplit{b, h, static_cast<int>((unit_off + nt - 1) / run.share), second};
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            float mm = wave_m[0][mt * 16 + q_at];
#pragma unroll
            for (int w = 1; w < NW; ++w) mm = fmaxf(mm, wave_m[w][mt * 16 + q_at]);
            const float f = m[mt] == -__builtin_inff() ? 0.f : (m[mt] == mm ? 1.f : exp2_fast(m[mt] - mm));
            float* const buf = reinterpret_cast<float*>(stage) + mt * (NW * 16 * D);
#pragma unroll
            for (int db = 0; db < DB; ++db) {
                const int c = (db * 4 + g_at) ^ (q_at & 7);
                *reinterpret_cast<floatx4_t*>(buf + (wave * 16 + q_at) * D + c * 4) = acc[mt][db] * f;
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        if (thread < MT * 16) {  // a thread settles a row
            const int row = row0 + thread;
            float mm = wave_m[0][thread], ll = 0.f;
#pragma unroll
            for (int w = 1; w < NW; ++w) mm = fmaxf(mm, wave_m[w][thread]);
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float mw = wave_m[w][thread];
                ll += mw == -__builtin_inff() ? 0.f : wave_l[w][thread] * (mw == mm ? 1.f : exp2_fast(mw - mm));
            }
            const int node = min(row, p.rows - 1) / p.group;
            const bool there = row < p.rows && (node == 0 || anc[node - 1] != 0);
            if (whole) {
                const int head = h * p.group + row - node * p.group;
                const int64_t at = (static_cast<int64_t>(b) * (p.k + 1) + node) * p.q_heads + head;
                row_to[thread] = row < p.rows ? at : -1;
                row_f[thread] = there ? 1.f / ll : 0.f;
                if (p.lse && row < p.rows)
                    p.lse[at] = there ? (mm + __log2f(ll)) * 0.69314718055994531f : -__builtin_inff();
            } else {
                // rows of absent nodes are joined as having seen nothing
                const int64_t at =
                    ((static_cast<int64_t>(cluster) * p.row_units + ru) * 2 + second) * (MT * 16) + thread;
                row_to[thread] = row < p.rows ? at : -1;
                row_f[thread] = 1.f;
                reinterpret_cast<float2*>(p.part_ml)[at] = there ? float2{mm, ll} : float2{-__builtin_inff(), 0.f};
            }
        }
        __syncthreads();
        int any_odd = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w) any_odd |= wave_odd[w];
#pragma unroll 4
        for (int e = thread; e < MT * 16 * (D / 4); e += NT) {
            const int lr = e / (D / 4), c4 = e % (D / 4);
            const int64_t to = row_to[lr];
            const float f = row_f[lr];
            const float* const buf = reinterpret_cast<const float*>(stage) + (lr >> 4) * (NW * 16 * D);
            floatx4_t o{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < NW; ++w)
                o += *reinterpret_cast<const floatx4_t*>(buf + (w * 16 + (lr & 15)) * D + ((c4 ^ (lr & 7)) << 2));
            if (to < 0) continue;
            if (any_odd) {
                const int node = (row0 + lr) / p.group;
#pragma unroll 1
                for (int j = 0; j <= p.k; ++j) {
                    if (j > 0 && (node == 0 || !((anc[node - 1] >> (j - 1)) & 1))) continue;
                    const uint64_t at = row_at(table[(len + j) >> p.page_shift], len + j);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint16_t x = vc[at * D + c4 * 4 + i];
                        if (nonfinite16<F16>(x)) o[i] += from16<F16>(x);
                    }
                }
            }
            if (whole) {
                shortx4_t x;
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = f != 0.f ? to16<F16>(o[i] * f) : short{0};
                *reinterpret_cast<shortx4_t*>(static_cast<uint16_t*>(p.out) + to * D + c4 * 4) = x;
            } else {
                *reinterpret_cast<floatx4_t*>(p.part_acc + to * D + c4 * 4) = o;
            }
        }
        __syncthreads();  // the buffers are free again
        pos += steps;
    }
    if (tid == 0) p.splits[static_cast<int64_t>(cluster) * p.row_units + ru] = split;
    }
    // Absent sequences have no tiles; their rows are zeros.
    for (int b = blockIdx.x; b < p.batch; b += kAttnWgs) {
        if (tiles_of(p, p.seq_len[b], TILE) > 0) continue;
        const int64_t n = static_cast<int64_t>(p.k + 1) * p.q_heads;
        for (int64_t e = tid; e < n * (D / 8); e += NT)
            reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + b * n * D)[e] = uint4{0, 0, 0, 0};
        if (p.lse)
            for (int64_t e = tid; e < n; e += NT) p.lse[b * n + e] = -__builtin_inff();
    }
}

// Joins the parts of what several clusters share: a wavefront for each row,
// its lanes in groups of D / 4 that take the parts in turn.
template <bool F16, int D>
__global__ __launch_bounds__(256) void k_tree_combine(AttnPlan p) {
    const int cluster = blockIdx.x / p.row_units, ru = blockIdx.x - cluster * p.row_units;
    const AttnSplit s = p.splits[blockIdx.x];
    if (s.b < 0) return;
    constexpr int LANES = D / 4, GROUPS = 64 / LANES, AHEAD = 4;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int unit_rows = p.row_tiles * 16;
    const int lr = blockIdx.y * 4 + wave;
    const int row = ru * unit_rows + lr;
    if (row >= p.rows) return;
    const int count = s.last - cluster + 1;
    const int group = min(lane / LANES, GROUPS - 1), c = (lane % LANES) * 4;
    float m = -__builtin_inff(), l = 0.f;
    floatx4_t o{0.f, 0.f, 0.f, 0.f};
    for (int base = group; base < count; base += GROUPS * AHEAD) {
        float2 ml[AHEAD];
        floatx4_t x[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int part = min(base + i * GROUPS, count - 1);
            const int64_t slot = (static_cast<int64_t>(cluster + part) * p.row_units + ru) * 2 + (part == 0 ? s.slot1 : 0);
            ml[i] = reinterpret_cast<const float2*>(p.part_ml)[slot * unit_rows + lr];
            x[i] = *reinterpret_cast<const floatx4_t*>(p.part_acc + (slot * unit_rows + lr) * D + c);
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            if (base + i * GROUPS >= count || ml[i].x == -__builtin_inff()) continue;
            const float mn = fmaxf(m, ml[i].x);
            const float a = m == mn ? 1.f : exp2_fast(m - mn), b = ml[i].x == mn ? 1.f : exp2_fast(ml[i].x - mn);
            m = mn;
            l = l * a + ml[i].y * b;
            o = o * a + x[i] * b;
        }
    }
    // The groups' results, in their order.
    const float m0 = m, l0 = l;
    const floatx4_t o0 = o;
#pragma unroll
    for (int q = 1; q < GROUPS; ++q) {
        const int from = (lane + q * LANES) & 63;
        const float mq = __shfl(m0, from), lq = __shfl(l0, from);
        floatx4_t oq;
#pragma unroll
        for (int i = 0; i < 4; ++i) oq[i] = __shfl(o0[i], from);
        if (mq == -__builtin_inff()) continue;
        const float mn = fmaxf(m, mq);
        const float a = m == mn ? 1.f : exp2_fast(m - mn), b = mq == mn ? 1.f : exp2_fast(mq - mn);
        m = mn;
        l = l * a + lq * b;
        o = o * a + oq * b;
    }
    if (lane >= LANES) return;
    const bool there = m != -__builtin_inff();
    const int node = row / p.group, head = s.head * p.group + row - node * p.group;
    const int64_t at = (static_cast<int64_t>(s.b) * (p.k + 1) + node) * p.q_heads + head;
    const float inv = 1.f / l;
    shortx4_t x;
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = there ? to16<F16>(o[i] * inv) : short{0};
    *reinterpret_cast<shortx4_t*>(static_cast<uint16_t*>(p.out) + at * D + c) = x;
    if (p.lse && lane == 0) p.lse[at] = there ? (m + __log2f(l)) * 0.69314718055994531f : -__builtin_inff();
}

template <bool F16, int D>
hipError_t launch_d(const AttnPlan& p, hipStream_t stream) {
    const dim3 grid(kAttnWgs), block(attn_waves(D) * 64);
    switch (p.row_tiles) {
        case 1: k_tree_attn<F16, D, 1><<<grid, block, 0, stream>>>(p); break;
        case 2: k_tree_attn<F16, D, 2><<<grid, block, 0, stream>>>(p); break;
        case 3:
            if constexpr (attn_max_row_tiles(D) >= 3) k_tree_attn<F16, D, 3><<<grid, block, 0, stream>>>(p);
            break;
        default:
            if constexpr (attn_max_row_tiles(D) >= 4) k_tree_attn<F16, D, 4><<<grid, block, 0, stream>>>(p);
            break;
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    k_tree_combine<F16, D><<<dim3(p.clusters * p.row_units, p.row_tiles * 4), dim3(256), 0, stream>>>(p);
    return hipGetLastError();
}

template <bool F16>
hipError_t launch_t(const AttnPlan& p, hipStream_t stream) {
    switch (p.head_dim) {
        case 64: return launch_d<F16, 64>(p, stream);
        case 96: return launch_d<F16, 96>(p, stream);
        case 128: return launch_d<F16, 128>(p, stream);
        default: return launch_d<F16, 256>(p, stream);
    }
}

}  // namespace

hipError_t launch_tree_attention(const AttnPlan& p, hipStream_t stream) {
    return p.is_f16 ? launch_t<true>(p, stream) : launch_t<false>(p, stream);
}

}  // namespace sv
