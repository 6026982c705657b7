// Matrix-product core of the feed-forward and cross-entropy kernels (gfx950).
//
//   C[m, n] = sum_k A(m, k) B(n, k)
//
// One workgroup of WM x WN waves forms a BM x BN tile of C in its registers, fp32, from
// 16x16 MFMA products; A and B tiles of 8 x 16 bytes per row of k pass through LDS, two
// buffers in turn, loaded from global memory straight to LDS 16 bytes a lane.  Either
// operand is stored with k contiguous (KC: rows of A or B) or with m/n contiguous (MC:
// the transpose), so products with a transposed operand need no transposing pass: the MC
// fragments are read from LDS with the transposing read (bf16) or element by element (fp32).
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
    static constexpr int kEpc = 8;  // elements per 16-byte chunk
    static __device__ __forceinline__ f32x4 mul(Frag b, Frag a, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, a, c, 0, 0, 0);
    }
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

template <>
struct MM<0> {  // fp32 operands
    using T = float;
    using Frag = f32x4;
    static constexpr int kEpc = 4;
    // k is taken in the order (k % 4) * 4 + k / 4 within a fragment's 16, on both sides alike
    static __device__ __forceinline__ f32x4 mul(Frag b, Frag a, f32x4 c)
    {
#pragma unroll
        for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(b[j], a[j], c, 0, 0, 0);
        return c;
    }
    static __device__ __forceinline__ Frag read_kc(const char* tile, int r0, int kk, int lane)
    {
        const int row = r0 + (lane & 15);
        const int c = (kk * 4 + (lane >> 4)) ^ (row & 7);
        return *reinterpret_cast<const Frag*>(tile + row * 128 + c * 16);
    }
    static __device__ __forceinline__ int mc_idx(int k) { return (k >> 2) & 3; }
    template <int COLS>
    static __device__ __forceinline__ Frag read_mc(const char* tile, int r0, int kk, int lane)
    {
        const int k = kk * 16 + (lane >> 4) * 4;
        const int gran = (r0 >> 4) ^ (mc_idx(k) & (COLS / 16 - 1));
        const float* p = reinterpret_cast<const float*>(tile) + k * COLS + gran * 16 + (lane & 15);
        Frag v;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = p[j * COLS];
        return v;
    }
    static __device__ __forceinline__ float widen(T v) { return v; }
    static __device__ __forceinline__ T narrow(float v) { return v; }
};

// Tile of workgroup `id` of ntm x ntn.  Workgroups go to the 8 XCDs in turn, each with an L2
// of its own: each XCD gets one contiguous run of the tile order, and the order walks columns
// of kGroupM tiles, so that the tiles an XCD works on together share their A and B rows.
constexpr int kXcds = 8, kGroupM = 8;
__device__ __forceinline__ void tile_of(uint32_t id, uint32_t ntm, uint32_t ntn, uint32_t* tm, uint32_t* tn)
{
    const uint32_t total = ntm * ntn;
    const uint32_t per = total / kXcds, rem = total % kXcds;
    const uint32_t x = id % kXcds, i = id / kXcds;
    const uint32_t at = x * per + (x < rem ? x : rem) + i;
    const uint32_t width = kGroupM * ntn;
    const uint32_t g = at / width, in = at % width;
    const uint32_t gm = ntm - g * kGroupM < kGroupM ? ntm - g * kGroupM : kGroupM;
    *tm = g * kGroupM + in % gm;
    *tn = in / gm;
}

// Geometry of a tile.  DT: 0 fp32, 1 bf16.  BM x BN over WM x WN waves.
template <int DT_, int BM_, int BN_, int WM_, int WN_, bool A_MC_, bool B_MC_>
struct Geo {
    static constexpr int DT = DT_, BM = BM_, BN = BN_, WM = WM_, WN = WN_;
    static constexpr bool A_MC = A_MC_, B_MC = B_MC_;
    static constexpr int BK = 8 * MM<DT>::kEpc;  // 128 bytes of k
    static constexpr int NT = 64 * WM * WN;
    static constexpr int FM = BM / WM / 16, FN = BN / WN / 16;  // fragments per wave
    static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128, STAGE = A_BYTES + B_BYTES;
    static constexpr int LDS = 2 * STAGE;
    static constexpr int NA = A_BYTES / 16 / NT, NB = B_BYTES / 16 / NT;  // chunks per thread
    static_assert(A_BYTES % (16 * NT) == 0 && B_BYTES % (16 * NT) == 0, "whole loads per thread");
};

// Chunk i of a thread in a tile of ROWS rows (KC) or ROWS columns (MC): which row/column group
// and which 16-byte chunk of k (KC) or which k and chunk of columns (MC) it has to load.
template <class G, bool MC, int ROWS>
__device__ __forceinline__ void chunk_place(int i, int tid, int* row, int* k)
{
    using M = MM<G::DT>;
    const int q = i * G::NT + tid;
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

// acc += A B^T over the k tile in `stage`, for the wave at (wm, wn).
template <class G>
__device__ __forceinline__ void mm_step(const char* stage, int wm, int wn, int lane, f32x4 (&acc)[G::FM][G::FN])
{
    using M = MM<G::DT>;
    const char* const at = stage;
    const char* const bt = at + G::A_BYTES;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
        typename M::Frag a[G::FM], b[G::FN];
#pragma unroll
        for (int i = 0; i < G::FN; ++i) {
            const int r0 = (wn * G::FN + i) * 16;
            if constexpr (G::B_MC)
                b[i] = M::template read_mc<G::BN>(bt, r0, kk, lane);
            else
                b[i] = M::read_kc(bt, r0, kk, lane);
        }
#pragma unroll
        for (int i = 0; i < G::FM; ++i) {
            const int r0 = (wm * G::FM + i) * 16;
            if constexpr (G::A_MC)
                a[i] = M::template read_mc<G::BM>(at, r0, kk, lane);
            else
                a[i] = M::read_kc(at, r0, kk, lane);
        }
#pragma unroll
        for (int i = 0; i < G::FM; ++i)
#pragma unroll
            for (int j = 0; j < G::FN; ++j) acc[i][j] = M::mul(b[j], a[i], acc[i][j]);
    }
}

// The main loop: acc += A B^T over `tiles` k tiles.  a_lane / b_lane: this thread's chunk
// addresses at k = 0; Prob::a_off(t) / b_off(t): bytes to add for k tile t; Prob::valid(t): how
// many k of tile t exist (the others read zeros on both sides).
template <class G, class Prob>
__device__ __forceinline__ void mm_loop(const Prob& p, const char* const (&a_lane)[G::NA],
                                        const char* const (&b_lane)[G::NB], int tiles, char* lds,
                                        f32x4 (&acc)[G::FM][G::FN])
{
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = wave / G::WN, wn = wave % G::WN;

    auto issue = [&](int t, char* stage) {
        const int64_t ao = p.a_off(t), bo = p.b_off(t);
        const int valid = p.valid(t);
        // this wave's first lane's place in the tile: the hardware adds 16 bytes per lane
        char* const dst = stage + wave * 1024;
        if (valid >= G::BK) {
#pragma unroll
            for (int i = 0; i < G::NA; ++i) load_to_lds(a_lane[i] + ao, dst + i * (G::NT * 16));
#pragma unroll
            for (int i = 0; i < G::NB; ++i) load_to_lds(b_lane[i] + bo, dst + G::A_BYTES + i * (G::NT * 16));
        } else {
            int row, k;
#pragma unroll
            for (int i = 0; i < G::NA; ++i) {
                chunk_place<G, G::A_MC, G::BM>(i, tid, &row, &k);
                load_to_lds(k < valid ? a_lane[i] + ao : reinterpret_cast<const char*>(g_zero_chunk),
                            dst + i * (G::NT * 16));
            }
#pragma unroll
            for (int i = 0; i < G::NB; ++i) {
                chunk_place<G, G::B_MC, G::BN>(i, tid, &row, &k);
                load_to_lds(k < valid ? b_lane[i] + bo : reinterpret_cast<const char*>(g_zero_chunk),
                            dst + G::A_BYTES + i * (G::NT * 16));
            }
        }
    };

    issue(0, lds);
    for (int t = 0; t < tiles; ++t) {
        // tile t has arrived for every wave, and every wave has finished reading tile t-1
        __syncthreads();
        if (t + 1 < tiles) issue(t + 1, lds + ((t + 1) & 1) * G::STAGE);
        mm_step<G>(lds + (t & 1) * G::STAGE, wm, wn, lane, acc);
    }
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
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const char* a_lane[G::NA];
    const char* b_lane[G::NB];
    int row, k;
#pragma unroll
    for (int i = 0; i < G::NA; ++i) {
        chunk_place<G, G::A_MC, G::BM>(i, tid, &row, &k);
        a_lane[i] = p.a_chunk(row, k);
    }
#pragma unroll
    for (int i = 0; i < G::NB; ++i) {
        chunk_place<G, G::B_MC, G::BN>(i, tid, &row, &k);
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

}  // namespace
}  // namespace ssk
