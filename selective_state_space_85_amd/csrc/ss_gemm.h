// Matrix-product core of the feed-forward and cross-entropy kernels (gfx950).
//
//   C[m, n] = sum_k A(m, k) B(n, k)
//
// One workgroup of WM x WN waves forms a BM x BN tile of C in its registers, fp32, from
// 16x16 MFMA products; A and B tiles of 8 x 16 bytes per row of k pass through LDS, two
// buffers (three of B under the two-group schedule, see mm_loop) in turn, loaded from global
// memory straight to LDS 16 bytes a lane.  Either operand is stored with k contiguous (KC: rows
// of A or B) or with m/n contiguous (MC: the transpose), so products with a transposed operand
// need no transposing pass: bf16 MC fragments are read from LDS with the transposing read.
// All products are bf16 ones; fp32 operands are split into three bf16 parts (see MM<0>) in
// registers on their way to LDS, and transposed there where they are MC; that takes any alignment.
//
// What bounds it at large sizes is the power that the matrix cores may take.  8192 x 8192 outputs
// over 4096, bf16, both operands KC: 434 us, 1266 TFLOP/s (B MC 1254, both MC 1201), the cores 71%
// busy at 1.8 GHz; operands of zeros, which cost little power: 1700.  fp32, 4096 x 4096 over 2048:
// 390 us, 176 TFLOP/s.
//
// LDS swizzle.  The direct load writes lane i's 16 bytes at base + 16 i, so a permutation of
// a row's 16-byte chunks has to be applied to the source address instead:
//   KC tile: rows of 128 bytes = 8 chunks; chunk c of row r sits at position c ^ (r & 7), so
//     the 16 rows that a fragment read touches fall on different banks;
//   MC tile: rows of one k, BM (BN) elements; the 16-element granule g of row k sits at
//     granule g ^ idx(k), where idx differs for the rows that one read touches together.
//
// Internal to the library.
#pragma once

#include <hip/hip_runtime.h>

#include "ss_device.h"
#include "ss_tiles.h"

namespace ssk {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// What rows past the end of k read: loads that must not contribute are pointed here.
__device__ const uint32_t g_zero_chunk[4] __attribute__((aligned(16))) = {0, 0, 0, 0};

typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(1))) const void glb_void;

__device__ __forceinline__ void load_to_lds(const void* src, void* dst)
{
    __builtin_amdgcn_global_load_lds((glb_void*)src, (lds_void*)dst, 16, 0, 0);
}

template <int DT>
struct MM;

template <>
struct MM<1> {  // bf16 operands
    using T = __bf16;
    using Frag = bf16x8;
    static constexpr int kEpc = 8;    // elements per 16-byte chunk
    static constexpr int kSteps = 2;  // fragments' depths per k tile
    // fragment of rows [r0, r0 + 16) and chunks [4 kk, 4 kk + 4) of a KC tile
    static __device__ __forceinline__ Frag read_kc(const char* tile, int r0, int kk, int lane)
    {
        const int row = r0 + (lane & 15);
        const int c = (kk * 4 + (lane >> 4)) ^ (row & 7);
        return *reinterpret_cast<const Frag*>(tile + row * 128 + c * 16);
    }
    static __device__ __forceinline__ int mc_idx(int k) { return ((k >> 3) & 3) * 4 + (k & 3); }
    // the same fragment of an MC tile of COLS columns: lane l of a group of 16 supplies the
    // address of 4 columns of one k and receives the 4 k of one column
    template <int COLS>
    static __device__ __forceinline__ Frag read_mc(const char* tile, int r0, int kk, int lane)
    {
        const int g = lane >> 4, j = lane & 15;
        const int k = kk * 32 + g * 8 + (j >> 2);
        const int gran = (r0 >> 4) ^ (mc_idx(k) & (COLS / 16 - 1));
        const char* p = tile + k * (COLS * 2) + gran * 32 + (j & 3) * 8;
        typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * COLS * 2));
        typedef short s16x8 __attribute__((ext_vector_type(8)));
        const s16x8 v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        return __builtin_bit_cast(Frag, v);
    }
    static __device__ __forceinline__ float widen(T v) { return float(v); }
    static __device__ __forceinline__ T narrow(float v) { return __bf16(v); }
};

// fp32 operands.  An operand is the sum of three bf16 parts, each the rounding of what the ones
// before it leave: all of its 24 bits, down to 2^-134 (bf16's range ends there: operands below 2^-110
// lose their last bits).  A product is formed from the six products of parts that matter, smallest
// first, accumulated in fp32, at a sixth of bf16's rate where the fp32 matrix instruction has a
// sixteenth.  The three left out are together up to 2^-24.0 of the product (the largest found; below
// 2^-23 by their sizes), 2^-27.4 in the mean square of random pairs; fp32 rounds a product by as much.
// An operand that bf16 rounds to infinity (from 3.3962e38 on) has inf - inf among its parts; such
// tiles are formed again by the fp32 instruction (see mm_tile_f32).
template <>
struct MM<0> {
    using T = float;
    static constexpr int kEpc = 4;
    static __device__ __forceinline__ float widen(T v) { return v; }
    static __device__ __forceinline__ T narrow(float v) { return v; }
};
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// 8 neighbouring k of one row: their parts, packed
__device__ __forceinline__ void split8(const float (&v)[8], u32x4 (&part)[3])
{
    typedef __bf16 Pair __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        // two elements at a time: they are rounded, and packed, by one instruction
        float v0 = v[2 * j], v1 = v[2 * j + 1];
#pragma unroll
        for (int q = 0; q < 3; ++q) {
            const uint32_t u = __builtin_bit_cast(uint32_t, Pair{__bf16(v0), __bf16(v1)});
            part[q][j] = u;
            v0 -= __uint_as_float(u << 16);
            v1 -= __uint_as_float(u & 0xffff0000u);
        }
    }
}

__device__ __forceinline__ f32x4 mfma_bf16(bf16x8 b, bf16x8 a, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, a, c, 0, 0, 0);
}

// The order of the tiles.  Workgroups go to the 8 XCDs in turn, each with an L2 of its own:
// run_of gives each XCD one contiguous run of the order, and the order walks columns of kGroupM
// tiles, so that the tiles an XCD works on together share their A and B rows.
constexpr uint32_t kXcds = 8, kGroupM = 8;
__device__ __forceinline__ uint32_t run_of(uint32_t id, uint32_t total)
{
    const uint32_t per = total / kXcds, rem = total % kXcds;
    const uint32_t x = id % kXcds, i = id / kXcds;
    return x * per + (x < rem ? x : rem) + i;
}
__device__ __forceinline__ void tile_at(uint32_t at, uint32_t ntm, uint32_t ntn, uint32_t* tm, uint32_t* tn)
{
    const uint32_t width = kGroupM * ntn;
    const uint32_t g = at / width, in = at % width;
    const uint32_t gm = ntm - g * kGroupM < kGroupM ? ntm - g * kGroupM : kGroupM;
    *tm = g * kGroupM + in % gm;
    *tn = in / gm;
}

// A launch's tiles: `whole` of them as they are, and the `split` last ones of the order as two
// halves of BM / 2 rows each.  With one large tile per CU the last round of a launch leaves CUs
// idle; when at most half of them are left with work, halves of its tiles take half the time.
struct TilePlan {
    uint32_t ntm, ntn, whole, split;
    __host__ __device__ uint32_t blocks() const { return whole + 2 * split; }
};
// Workgroup id's tile, and which half of it (-1: all of it).
__device__ __forceinline__ int tile_of(uint32_t id, const TilePlan& t, uint32_t* tm, uint32_t* tn)
{
    if (id < t.whole) {
        tile_at(run_of(id, t.whole), t.ntm, t.ntn, tm, tn);
        return -1;
    }
    const uint32_t q = run_of(id - t.whole, 2 * t.split);
    tile_at(t.whole + q / 2, t.ntm, t.ntn, tm, tn);
    return int(q & 1);
}

// Geometry of a tile.  DT: 0 fp32, 1 bf16.  BM x BN over WM x WN waves.
// With 2 x 4 waves the A tile lies in LDS as one part per wave row (A_PART rows or columns),
// each loaded by the waves that read it.
template <int DT_, int BM_, int BN_, int WM_, int WN_, bool A_MC_, bool B_MC_>
struct Geo {
    static constexpr int DT = DT_, BM = BM_, BN = BN_, WM = WM_, WN = WN_;
    static constexpr bool A_MC = A_MC_, B_MC = B_MC_;
    static constexpr int BK = 8 * MM<DT>::kEpc;  // 128 bytes of k
    static constexpr int NT = 64 * WM * WN;
    static constexpr int FM = BM / WM / 16, FN = BN / WN / 16;  // fragments per wave
    static constexpr bool GROUPS = WM == 2 && WN == 4;          // the two-group schedule (see mm_loop)
    static constexpr int A_PARTS = GROUPS ? 2 : 1, A_PART = BM / A_PARTS, A_NT = NT / A_PARTS;
    static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;
    static constexpr int B_STAGES = GROUPS ? 3 : 2;
    // bf16: the A buffers, then the B buffers; fp32: one tile of each, in three parts of 64 bytes a row
    static constexpr int LDS = DT == 1 ? 2 * A_BYTES + B_STAGES * B_BYTES : (BM + BN) * 192;
    static constexpr int NA = A_BYTES / 16 / NT, NB = B_BYTES / 16 / NT;  // chunks per thread
    static_assert(A_BYTES % (16 * NT) == 0 && B_BYTES % (16 * NT) == 0, "whole loads per thread");
};

// Chunk i of thread `tid` of THREADS in a tile of ROWS rows (KC) or ROWS columns (MC): which
// row and which 16-byte chunk of k (KC) or which k and chunk of columns (MC) it has to load.
template <int DT, bool MC, int ROWS, int THREADS>
__device__ __forceinline__ void chunk_place(int i, int tid, int* row, int* k)
{
    using M = MM<DT>;
    const int q = i * THREADS + tid;
    if constexpr (!MC) {
        *row = q >> 3;
        *k = ((q & 7) ^ (*row & 7)) * M::kEpc;
    } else {
        constexpr int per = ROWS / M::kEpc;    // chunks per k row
        constexpr int gch = 16 / M::kEpc;      // chunks per 16-element granule
        *k = q / per;
        const int c = q % per;
        const int gran = (c / gch) ^ (M::mc_idx(*k) & (ROWS / 16 - 1));
        *row = (gran * gch + c % gch) * M::kEpc;
    }
}
template <class G>
__device__ __forceinline__ void a_place(int i, int tid, int* row, int* k)
{
    chunk_place<G::DT, G::A_MC, G::A_PART, G::A_NT>(i, tid % G::A_NT, row, k);
    *row += tid / G::A_NT * G::A_PART;
}
template <class G>
__device__ __forceinline__ void b_place(int i, int tid, int* row, int* k)
{
    chunk_place<G::DT, G::B_MC, G::BN, G::NT>(i, tid, row, k);
}
// Byte offset of element (row m, k) of an MC A tile.
template <class G>
__device__ __forceinline__ int a_mc_offset(int m, int k)
{
    using M = MM<G::DT>;
    const int in = m % G::A_PART, gran = (in >> 4) ^ (M::mc_idx(k) & (G::A_PART / 16 - 1));
    return m / G::A_PART * (G::A_PART * 128) + (k * G::A_PART + gran * 16 + (in & 15)) * int(sizeof(typename M::T));
}

// How many of the `total` k lie in k tile t, or a negative number past the last tile.
template <int DT>
__device__ __forceinline__ int k_left(int64_t total, int t)
{
    constexpr int BK = 8 * MM<DT>::kEpc;
    const int64_t left = total - int64_t(t) * BK;
    return left < BK ? int(left) : BK;
}

// The wave's fragments of half `kk` of the k tile in a_tile and b_tile.
template <class G>
__device__ __forceinline__ void mm_read(const char* a_tile, const char* b_tile, int kk, int wm, int wn, int lane,
                                        typename MM<G::DT>::Frag (&a)[G::FM], typename MM<G::DT>::Frag (&b)[G::FN])
{
    using M = MM<G::DT>;
#pragma unroll
    for (int i = 0; i < G::FN; ++i) {
        const int r0 = (wn * G::FN + i) * 16;
        if constexpr (G::B_MC)
            b[i] = M::template read_mc<G::BN>(b_tile, r0, kk, lane);
        else
            b[i] = M::read_kc(b_tile, r0, kk, lane);
    }
    // with one part per wave row, rows count from the part's first
    const char* const part = a_tile + (G::A_PARTS > 1 ? wm * (G::A_PART * 128) : 0);
#pragma unroll
    for (int i = 0; i < G::FM; ++i) {
        const int r0 = ((G::A_PARTS > 1 ? 0 : wm * G::FM) + i) * 16;
        if constexpr (G::A_MC)
            a[i] = M::template read_mc<G::A_PART>(part, r0, kk, lane);
        else
            a[i] = M::read_kc(part, r0, kk, lane);
    }
}

struct NoWork {
    __device__ void operator()(int) const {}
};
// acc += the fragments' product; beside(i) is issued after row i's products.
template <class G, class Beside = NoWork>
__device__ __forceinline__ void mm_mul(const typename MM<G::DT>::Frag (&a)[G::FM],
                                       const typename MM<G::DT>::Frag (&b)[G::FN], f32x4 (&acc)[G::FM][G::FN],
                                       Beside beside = Beside())
{
#pragma unroll
    for (int i = 0; i < G::FM; ++i) {
#pragma unroll
        for (int q = 0; q < G::FN; ++q) {
            const int j = i & 1 ? G::FN - 1 - q : q;  // there and back: every two neighbours share an operand
            acc[i][j] = mfma_bf16(b[j], a[i], acc[i][j]);
        }
        beside(i);
    }
}

// Whether the thread's sums are neither infinite nor NaN: 0 times each is 0.
template <class G>
__device__ __forceinline__ bool all_finite(const f32x4 (&acc)[G::FM][G::FN])
{
    float zero[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < G::FM; ++i)
#pragma unroll
        for (int j = 0; j < G::FN; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) zero[e] = fmaf(acc[i][j][e], 0.0f, zero[e]);
    return zero[0] + zero[1] + zero[2] + zero[3] == 0.0f;
}

// acc += A B^T over the k tile in a_tile and b_tile, for the wave at (wm, wn).
template <class G>
__device__ __forceinline__ void mm_step(const char* a_tile, const char* b_tile, int wm, int wn, int lane, f32x4 (&acc)[G::FM][G::FN])
{
#pragma unroll
    for (int kk = 0; kk < MM<G::DT>::kSteps; ++kk) {
        typename MM<G::DT>::Frag a[G::FM], b[G::FN];
        mm_read<G>(a_tile, b_tile, kk, wm, wn, lane, a, b);
        mm_mul<G>(a, b, acc);
    }
}

// One phase of the two-group schedule ends: nothing moves across, in the compiler or the wave.
__device__ __forceinline__ void phase_end()
{
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ void wait_lds_reads() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
// all but the latest N loads of this wave have arrived
template <int N>
__device__ __forceinline__ void wait_loads()
{
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// The main loop: acc += A B^T over `tiles` k tiles.  a_lane / b_lane: this thread's chunk
// addresses at k = 0; Prob::a_off(t) / b_off(t): bytes to add for k tile t; Prob::valid(t): how
// many k of tile t exist (none past the last tile); the others read zeros on both sides.
template <class G, class Prob>
__device__ __forceinline__ void mm_loop(const Prob& p, const char* const (&a_lane)[G::NA],
                                        const char* const (&b_lane)[G::NB], int tiles, char* lds,
                                        f32x4 (&acc)[G::FM][G::FN])
{
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);  // uniform, and known to be
    const int wm = wave / G::WN, wn = wave % G::WN;

    // this wave's first lane's place: the hardware adds 16 bytes per lane
    char* const a_dst = lds + (G::A_PARTS > 1 ? wm * (G::A_PART * 128) + wn * 1024 : wave * 1024);
    char* const b_dst = lds + 2 * G::A_BYTES + wave * 1024;
    const char* const zero = reinterpret_cast<const char*>(g_zero_chunk);
    // this thread's source addresses of k tile t
    auto a_src = [&](int t, const char* (&src)[G::NA]) {
        const int64_t off = p.a_off(t);
        const int valid = p.valid(t);
#pragma unroll
        for (int i = 0; i < G::NA; ++i) src[i] = a_lane[i] + off;
        if (valid < G::BK) {
            int row, k;
#pragma unroll
            for (int i = 0; i < G::NA; ++i) {
                a_place<G>(i, tid, &row, &k);
                if (k >= valid) src[i] = zero;
            }
        }
    };
    auto b_src = [&](int t, const char* (&src)[G::NB]) {
        const int64_t off = p.b_off(t);
        const int valid = p.valid(t);
#pragma unroll
        for (int i = 0; i < G::NB; ++i) src[i] = b_lane[i] + off;
        if (valid < G::BK) {
            int row, k;
#pragma unroll
            for (int i = 0; i < G::NB; ++i) {
                b_place<G>(i, tid, &row, &k);
                if (k >= valid) src[i] = zero;
            }
        }
    };
    const char* as[G::NA];
    const char* bs[G::NB];
    auto load_a = [&](int buf, int i) { load_to_lds(as[i], a_dst + buf * G::A_BYTES + i * (G::A_NT * 16)); };
    auto load_b = [&](int buf, int i) { load_to_lds(bs[i], b_dst + buf * G::B_BYTES + i * (G::NT * 16)); };
    auto issue_a = [&](int t, int buf) {
        a_src(t, as);
#pragma unroll
        for (int i = 0; i < G::NA; ++i) load_a(buf, i);
    };
    auto issue_b = [&](int t, int buf) {
        b_src(t, bs);
#pragma unroll
        for (int i = 0; i < G::NB; ++i) load_b(buf, i);
    };

    if constexpr (G::GROUPS) {
        static_assert(G::FM == 2 * G::NA && G::NB <= G::FM, "the loads' places among the products");
        // Two groups of four waves (one of each on every SIMD), one phase apart: while one reads
        // its fragments, the other has the matrix cores.  A k tile is four phases of each group:
        // fragments of its first half, products, fragments of its second half, products.  Loads
        // are issued among the products.  In phases of the early group (the late one is a phase
        // behind), tile t is read from phase 4t to 4t + 3, the late group's last, and every read
        // has been waited for when its phase ends.
        //   B has three buffers: tile t + 2's was last read, with tile t - 1, in phase 4t - 1, and
        //   takes its loads in phase 4t + 1 (early) and 4t + 2 (late).
        //   A has two: tile t + 2's was last read, with tile t, by the wave row that loads it, in
        //   phase 4t + 2 (4t + 3), and takes its loads in phase 4t + 3 (4t + 4).
        // Before the end of phase 4t + 3 each wave waits for its own loads of tile t + 1; those
        // issued after them, of B (and A) of tile t + 2, stay under way.  Tile t + 1 is read from
        // phase 4t + 4 on.
        const bool late = wm != 0;
        issue_b(0, 0);
        issue_a(0, 0);
        issue_b(1, 1);
        issue_a(1, 1);
        wait_loads<G::NA + G::NB>();
        phase_end();
        if (late) phase_end();
        typename MM<G::DT>::Frag a[G::FM], b[G::FN];
        int b_buf = 0, b_next = 2;
        for (int t = 0; t < tiles; ++t) {
            const char* const a_tile = lds + (t & 1) * G::A_BYTES;
            const char* const b_tile = lds + 2 * G::A_BYTES + b_buf * G::B_BYTES;
            mm_read<G>(a_tile, b_tile, 0, wm, wn, lane, a, b);
            b_src(t + 2, bs);
            wait_lds_reads();
            phase_end();
            __builtin_amdgcn_s_setprio(1);
            mm_mul<G>(a, b, acc, [&](int i) {
                constexpr int every = G::FM / G::NB;
                if (i % every == every - 1) load_b(b_next, i / every);
            });
            __builtin_amdgcn_s_setprio(0);
            phase_end();
            mm_read<G>(a_tile, b_tile, 1, wm, wn, lane, a, b);
            a_src(t + 2, as);
            wait_lds_reads();
            if (late) wait_loads<G::NB>();
            phase_end();
            __builtin_amdgcn_s_setprio(1);
            mm_mul<G>(a, b, acc, [&](int i) {
                if (i & 1) load_a(t & 1, i >> 1);
            });
            __builtin_amdgcn_s_setprio(0);
            if (!late) wait_loads<G::NA + G::NB>();
            phase_end();
            b_buf = b_buf == 2 ? 0 : b_buf + 1;
            b_next = b_next == 2 ? 0 : b_next + 1;
        }
        wait_loads<0>();  // the loads past the last tile: LDS is free after the loop
        if (!late) phase_end();
        return;
    }
    if (tiles > 0) {
        issue_a(0, 0);
        issue_b(0, 0);
    }
    for (int t = 0; t < tiles; ++t) {
        // tile t has arrived for every wave, and every wave has finished reading tile t-1
        __syncthreads();
        if (t + 1 < tiles) {
            issue_a(t + 1, (t + 1) & 1);
            issue_b(t + 1, (t + 1) & 1);
        }
        mm_step<G>(lds + (t & 1) * G::A_BYTES, lds + 2 * G::A_BYTES + (t & 1) * G::B_BYTES, wm, wn, lane, acc);
    }
}

// ---- fp32 --------------------------------------------------------------------------------------

// A thread's items of one operand's k tile (ROWS rows or columns of it, 32 k), as loaded.
//   KC: an item is 8 k of one row;
//   MC: an item is 8 k of two neighbouring columns.
// Either way the tile lies in LDS with k contiguous, each part a row of 64 bytes whose 16-byte chunk
// c sits at position c ^ (row / 4 % 4).  Elements past the ends of k are zeros, and no element past
// the ends of a row is read, whatever its alignment.
template <bool MC, int ROWS, int NT>
struct Staged {
    static constexpr int ITEMS = MC ? ROWS / 2 * 4 : ROWS * 4, N = (ITEMS + NT - 1) / NT, LEN = MC ? 16 : 8;
    float v[N][LEN];

    static __device__ __forceinline__ bool has(int i, int tid) { return ITEMS % NT == 0 || i * NT + tid < ITEMS; }
    // first row (column) and chunk of k of item i
    static __device__ __forceinline__ void place(int i, int tid, int* row, int* chunk)
    {
        const int q = i * NT + tid;
        if (MC) {
            *row = q % (ROWS / 2) * 2;
            *chunk = q / (ROWS / 2);
        } else {
            *row = q >> 2;
            *chunk = q & 3;
        }
    }
    // p[i]: item i's first element at k tile 0, clamped to a row (column) that exists; two: its second
    // column exists; ld: elements per k (MC); valid: k of this tile that exist
    __device__ __forceinline__ void load(const float* const (&p)[N], const bool (&two)[N], int64_t off, int64_t ld, int valid,
                                         int tid)
    {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            int row, chunk;
            place(i, tid, &row, &chunk);
            const int left = has(i, tid) ? valid - chunk * 8 : 0;
            const float* q = p[i] + off;
            if (!MC) {
                if (left >= 8) {
                    __builtin_memcpy(v[i], q, 32);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[i][e] = e < left ? q[e] : 0.0f;
                }
            } else {
                if (left >= 8 && two[i]) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) __builtin_memcpy(&v[i][2 * e], q + e * ld, 8);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        v[i][2 * e] = e < left ? q[e * ld] : 0.0f;
                        v[i][2 * e + 1] = e < left && two[i] ? q[e * ld + 1] : 0.0f;
                    }
                }
            }
        }
    }
    // tile: three parts of ROWS rows
    __device__ __forceinline__ void store(char* tile, int tid) const
    {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (!has(i, tid)) continue;
            int row, chunk;
            place(i, tid, &row, &chunk);
#pragma unroll
            for (int c = 0; c < (MC ? 2 : 1); ++c) {
                float one[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) one[e] = MC ? v[i][2 * e + c] : v[i][e];
                u32x4 part[3];
                split8(one, part);
                const int r = row + c;
                char* const to = tile + r * 64 + (chunk ^ (r >> 2 & 3)) * 16;
#pragma unroll
                for (int q = 0; q < 3; ++q) *reinterpret_cast<u32x4*>(to + q * (ROWS * 64)) = part[q];
            }
        }
    }
    // tile: ROWS rows of the elements as they are
    __device__ __forceinline__ void store_whole(float* tile, int tid) const
    {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (!has(i, tid)) continue;
            int row, chunk;
            place(i, tid, &row, &chunk);
#pragma unroll
            for (int c = 0; c < (MC ? 2 : 1); ++c)
#pragma unroll
                for (int e = 0; e < 8; ++e) tile[(row + c) * 32 + chunk * 8 + e] = MC ? v[i][2 * e + c] : v[i][e];
        }
    }
};
__device__ __forceinline__ bf16x8 staged_frag(const char* part, int r0, int lane)
{
    const int row = r0 + (lane & 15);
    return *reinterpret_cast<const bf16x8*>(part + row * 64 + ((lane >> 4) ^ (row >> 2 & 3)) * 16);
}

// One workgroup's tile of an fp32 product.  Elements pass through registers, where each is split
// once per workgroup; the next k tile's loads are in flight while this one's products are formed.
// Sums that are not finite are formed again, by the fp32 instruction from the elements
// themselves: an infinity, or a number that bf16 rounds to one, makes all that it takes part in NaN
// above, where infinite or finite results may be due.  The check costs up to 1% of a pass (894 tokens,
// 2560 -> 2 x 1600: 461 -> 462 us; 777, 1001 -> 2 x 2731: 338 -> 341), the rest such tiles alone: the loss
// of 333 tokens of 50257 entries takes 1.34 ms for 0.19 with every second entry at the type's lowest value,
// and 0.19 with them at -1e30.
// Prob: a_at(row, k) / b_at(row, k), the address of an element, rows past the end clamped to the last;
// a_cols() / b_cols(), for MC operands the columns that exist from the tile's first on; a_ld() / b_ld(),
// their elements per k; a_off, b_off (in bytes), valid, tiles, finish as for mm_tile; kSkips, and where
// that is true skips(t, k): rows k of k tile t of B that tiles formed again leave out.
template <class G, class Prob>
__device__ __forceinline__ void mm_tile_f32(const Prob& p, char* lds)
{
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / G::WN, wn = wave % G::WN;
    using SA = Staged<G::A_MC, G::BM, G::NT>;
    using SB = Staged<G::B_MC, G::BN, G::NT>;
    SA sa;
    SB sb;
    const float* pa[SA::N];
    const float* pb[SB::N];
    bool ta[SA::N], tb[SB::N];
    auto set = [&](int thread) {
        int row, chunk;
#pragma unroll
        for (int i = 0; i < SA::N; ++i) {
            SA::place(i, thread, &row, &chunk);
            ta[i] = !G::A_MC || row + 1 < p.a_cols();
            pa[i] = p.a_at(row, SA::has(i, thread) ? chunk * 8 : 0);
        }
#pragma unroll
        for (int i = 0; i < SB::N; ++i) {
            SB::place(i, thread, &row, &chunk);
            tb[i] = !G::B_MC || row + 1 < p.b_cols();
            pb[i] = p.b_at(row, SB::has(i, thread) ? chunk * 8 : 0);
        }
    };
    auto load = [&](int t) {
        sa.load(pa, ta, p.a_off(t) / 4, p.a_ld(), p.valid(t), tid);
        sb.load(pb, tb, p.b_off(t) / 4, p.b_ld(), p.valid(t), tid);
    };
    set(tid);
    f32x4 acc[G::FM][G::FN];
#pragma unroll
    for (int i = 0; i < G::FM; ++i)
#pragma unroll
        for (int j = 0; j < G::FN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    char* const at = lds;
    char* const bt = lds + G::BM * 192;
    __shared__ int odd;  // some sum is not finite
    if (tid == 0) odd = 0;
    if (p.tiles > 0) load(0);
    for (int t = 0; t < p.tiles; ++t) {
        __syncthreads();  // the last tile's readers are done
        sa.store(at, tid);
        sb.store(bt, tid);
        __syncthreads();
        if (t + 1 < p.tiles) load(t + 1);
        bf16x8 b[3][G::FN];
#pragma unroll
        for (int q = 0; q < 3; ++q)
#pragma unroll
            for (int j = 0; j < G::FN; ++j) b[q][j] = staged_frag(bt + q * (G::BN * 64), (wn * G::FN + j) * 16, lane);
        constexpr int kA[6] = {2, 1, 0, 1, 0, 0}, kB[6] = {0, 1, 2, 0, 1, 0};  // smallest first
#pragma unroll
        for (int i = 0; i < G::FM; ++i) {
            bf16x8 a[3];
#pragma unroll
            for (int q = 0; q < 3; ++q) a[q] = staged_frag(at + q * (G::BM * 64), (wm * G::FM + i) * 16, lane);
#pragma unroll
            for (int q = 0; q < 6; ++q)
#pragma unroll
                for (int j = 0; j < G::FN; ++j) acc[i][j] = mfma_bf16(b[kB[q]][j], a[kA[q]], acc[i][j]);
        }
    }
    if (p.tiles > 0) {
        if (!all_finite<G>(acc)) odd = 1;
        __syncthreads();
        if (__builtin_expect(odd, 0)) {
            // formed anew: kept through the loop above, the addresses would cost its registers
            int thread = tid;
            asm volatile("" : "+v"(thread));
            set(thread);
            float* const wa = reinterpret_cast<float*>(lds);
            float* const wb = wa + G::BM * 32;
            // a row of fragments at a time, and finite sums stay as they are: they do not depend on what
            // shares their tile
#pragma unroll
            for (int i = 0; i < G::FM; ++i) {
                f32x4 whole[G::FN];
#pragma unroll
                for (int j = 0; j < G::FN; ++j) whole[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
                for (int t = 0; t < p.tiles; ++t) {
                    load(t);
                    if constexpr (Prob::kSkips) {
                        static_assert(G::B_MC, "k of B are rows that may be left out");
                        const int exist = p.valid(t);
#pragma unroll
                        for (int n = 0; n < SB::N; ++n) {
                            int col, chunk;
                            SB::place(n, tid, &col, &chunk);
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                if (SB::has(n, tid) && chunk * 8 + e < exist && p.skips(t, chunk * 8 + e))
                                    sb.v[n][2 * e] = sb.v[n][2 * e + 1] = 0.0f;
                        }
                    }
                    __syncthreads();
                    sa.store_whole(wa, tid);
                    sb.store_whole(wb, tid);
                    __syncthreads();
#pragma unroll 1
                    for (int e = 0; e < 8; ++e) {
                        // element e of a lane's 8 is the same k on both sides
                        const int from = (lane & 15) * 32 + (lane >> 4) * 8 + e;
                        const float av = wa[(wm * G::FM + i) * 512 + from];
#pragma unroll
                        for (int j = 0; j < G::FN; ++j)
                            whole[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(wb[(wn * G::FN + j) * 512 + from], av, whole[j], 0, 0, 0);
                    }
                }
#pragma unroll
                for (int j = 0; j < G::FN; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (!(fabsf(acc[i][j][e]) < __builtin_inff())) acc[i][j][e] = whole[j][e];
            }
        }
    }
    p.template finish<G>(acc, lds, wm, wn, lane);
}

// One workgroup's tile.  Prob supplies
//   a_chunk(row, k) / b_chunk(row, k): address of the chunk of A (B) whose first element is
//       (tile row `row`, k) at k tile 0, rows past the end clamped to the last;
//   a_off, b_off, valid (see mm_loop), tiles: the number of k tiles;
//   finish<G>(acc, lds, wm, wn, lane): the epilogue.  acc[i][j][e] is C at row
//       (wm FM + i) 16 + lane % 16, column (wn FN + j) 16 + (lane / 16) 4 + e of the tile.
template <class G, class Prob>
__device__ __forceinline__ void mm_tile(const Prob& p, char* lds)
{
    if constexpr (G::DT == 0) {
        mm_tile_f32<G>(p, lds);
        return;
    } else {
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);  // uniform, and known to be
    const char* a_lane[G::NA];
    const char* b_lane[G::NB];
    int row, k;
#pragma unroll
    for (int i = 0; i < G::NA; ++i) {
        a_place<G>(i, tid, &row, &k);
        a_lane[i] = p.a_chunk(row, k);
    }
#pragma unroll
    for (int i = 0; i < G::NB; ++i) {
        b_place<G>(i, tid, &row, &k);
        b_lane[i] = p.b_chunk(row, k);
    }
    f32x4 acc[G::FM][G::FN];
#pragma unroll
    for (int i = 0; i < G::FM; ++i)
#pragma unroll
        for (int j = 0; j < G::FN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    mm_loop<G>(p, a_lane, b_lane, p.tiles, lds, acc);
    p.template finish<G>(acc, lds, wave / G::WN, wave % G::WN, lane);
    }
}

// ---- few rows: the weights stream past them ------------------------------------------------------

// Products of up to kStreamRows rows of x with 2 x 16 rows of weights per workgroup, whose waves
// split k.  A wave reads its part of the 32 rows straight into MFMA operands (lane: row l % 16, 16
// bytes of k per step), the rows of x likewise (every workgroup shares them: they stay in the
// caches), and the waves' sums are joined in LDS.  Bound by reading the weights.
// ALIGNED: every row starts on 16 bytes and k is whole 16-byte chunks; otherwise rows are read as
// they lie, and the last chunk element by element.
constexpr int kStreamWaves = 4;
constexpr int kStreamUnroll = 4;  // steps whose loads are in flight together

template <int DT>
struct Stream;
template <>
struct Stream<1> {
    using Frag = bf16x8;
    static __device__ __forceinline__ f32x4 mul(Frag w, Frag x, f32x4 c) { return mfma_bf16(w, x, c); }
};
template <>
struct Stream<0> {  // the fp32 instruction: its rate does not matter here
    using Frag = f32x4;
    static __device__ __forceinline__ f32x4 mul(Frag w, Frag x, f32x4 c)
    {
        // k is taken in the order (k % 4) * 4 + k / 4 within a step's 16, on both sides alike
#pragma unroll
        for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(w[j], x[j], c, 0, 0, 0);
        return c;
    }
};

template <int DT, bool ALIGNED>
__device__ __forceinline__ typename Stream<DT>::Frag stream_load(const typename MM<DT>::T* p)
{
    typename Stream<DT>::Frag f;
    if constexpr (ALIGNED)
        f = *reinterpret_cast<const typename Stream<DT>::Frag*>(p);
    else
        __builtin_memcpy(&f, p, sizeof(f));
    return f;
}
// the chunk of which `left` elements exist (none: nothing is read)
template <int DT>
__device__ __forceinline__ typename Stream<DT>::Frag stream_tail(const typename MM<DT>::T* p, int64_t left)
{
    typename Stream<DT>::Frag f{};
#pragma unroll
    for (int e = 0; e < MM<DT>::kEpc; ++e)
        if (e < left) f[e] = p[e];
    return f;
}

// c0, c1: this wave's part of the products of w0's and w1's 16 rows (rows of C) with px's MT x 16
// rows.  w0, w1, px: this lane's rows (row l % 16 of each).
template <int DT, int MT, bool ALIGNED>
__device__ __forceinline__ void stream_rows(const typename MM<DT>::T* w0, const typename MM<DT>::T* w1,
                                            const typename MM<DT>::T* const (&px)[MT], int64_t k, f32x4 (&c0)[MT],
                                            f32x4 (&c1)[MT])
{
    using S = Stream<DT>;
    using Frag = typename S::Frag;
    constexpr int KS = 4 * MM<DT>::kEpc;  // k per step
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int kq = int((threadIdx.x & 63) >> 4) * MM<DT>::kEpc;
#pragma unroll
    for (int i = 0; i < MT; ++i) c0[i] = c1[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const int64_t whole = k / KS, steps = (k + KS - 1) / KS;
    int64_t s = wave;
    for (; s + (kStreamUnroll - 1) * kStreamWaves < whole; s += kStreamUnroll * kStreamWaves) {
        Frag a[kStreamUnroll], b[kStreamUnroll], x[kStreamUnroll][MT];
#pragma unroll
        for (int q = 0; q < kStreamUnroll; ++q) {
            const int64_t at = (s + q * kStreamWaves) * KS + kq;
            a[q] = stream_load<DT, ALIGNED>(w0 + at);
            b[q] = stream_load<DT, ALIGNED>(w1 + at);
#pragma unroll
            for (int i = 0; i < MT; ++i) x[q][i] = stream_load<DT, ALIGNED>(px[i] + at);
        }
#pragma unroll
        for (int q = 0; q < kStreamUnroll; ++q)
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                c0[i] = S::mul(a[q], x[q][i], c0[i]);
                c1[i] = S::mul(b[q], x[q][i], c1[i]);
            }
    }
    for (; s < steps; s += kStreamWaves) {
        const int64_t at = s * KS + kq, left = k - at;
        const bool all = left >= MM<DT>::kEpc;
        const Frag a = all ? stream_load<DT, ALIGNED>(w0 + at) : stream_tail<DT>(w0 + at, left);
        const Frag b = all ? stream_load<DT, ALIGNED>(w1 + at) : stream_tail<DT>(w1 + at, left);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const Frag x = all ? stream_load<DT, ALIGNED>(px[i] + at) : stream_tail<DT>(px[i] + at, left);
            c0[i] = S::mul(a, x, c0[i]);
            c1[i] = S::mul(b, x, c1[i]);
        }
    }
}

// The waves' parts joined; finish(i, s0, s1) has, for rows 16 i .. 16 i + 15 of x, the sums whose
// element e is weight row (l / 16) 4 + e, x row 16 i + l % 16.
template <int MT, class Finish>
__device__ __forceinline__ void stream_join(const f32x4 (&c0)[MT], const f32x4 (&c1)[MT], Finish finish)
{
    __shared__ f32x4 part[kStreamWaves][2 * MT][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        part[wave][2 * i][lane] = c0[i];
        part[wave][2 * i + 1][lane] = c1[i];
    }
    __syncthreads();
    for (int i = wave; i < MT; i += kStreamWaves) {
        f32x4 s0 = part[0][2 * i][lane], s1 = part[0][2 * i + 1][lane];
#pragma unroll
        for (int w = 1; w < kStreamWaves; ++w) {
            s0 += part[w][2 * i][lane];
            s1 += part[w][2 * i + 1][lane];
        }
        finish(i, s0, s1);
    }
}

// ---- choosing tiles (host) ---------------------------------------------------------------------

// The tiles: a large one (one workgroup of 8 waves per CU, LDS full) and its half, for bf16 alone;
// a small one and a mini one (4 waves; two and three workgroups per CU), which fill the chip with
// less work and, since fp32 takes six products per pair of fragments, feed it at any size.
template <int DT>
struct Tiles {
    template <bool AM, bool BM_>
    using Small = Geo<DT, 128, 128, 2, 2, AM, BM_>;
    template <bool AM, bool BM_>
    using Mini = Geo<DT, 64, 128, 2, 2, AM, BM_>;
};
template <bool AM, bool BM_>
using LargeTile = Geo<1, 256, 256, 2, 4, AM, BM_>;
template <bool AM, bool BM_>
using HalfTile = Geo<1, 128, 256, 2, 4, AM, BM_>;

// `before`: workgroups of the same launch ahead of these tiles.
inline TilePlan plan_tiles(uint32_t ntm, uint32_t ntn, bool can_split, uint32_t before = 0)
{
    const uint32_t total = ntm * ntn, last = (before + total) % kCUs;
    const uint32_t split = can_split && last <= kCUs / 2 && last < total ? last : 0;
    return {ntm, ntn, total - split, split};
}

}  // namespace
}  // namespace ssk
