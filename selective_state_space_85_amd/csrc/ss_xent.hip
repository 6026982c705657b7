// gfx950 kernels of the softmax cross entropy of a vocabulary projection
//   l = x w^T (n, v),  lse_i = log sum_j exp(l_ij),  loss_i = lse_i - l_i,target
// and its gradients
//   dl_ij = (exp(l_ij - lse_i) - [j = target_i]) dloss_i,  dx = dl w,  dw = dl^T x.
//
// The logits are never stored.  Forward: each 128 columns' tile of logits is reduced, in the
// accumulators that hold it, to a maximum and a sum of exponentials per row; a second kernel
// joins the (maximum, sum) pairs of a row.  Backward: the vocabulary is taken in pieces; a
// piece's logits are formed again and turned into dl in the epilogue (rounded once to the
// operands' type, as the next products' operands must be) in a workspace that the next piece
// reuses, and one launch forms the piece's part of dx (fp32 sums over the pieces, rounded
// after the last) and its rows of dw.  Bound by the matrix cores at training sizes:
// 8192 tokens, 2560 wide, 50257 entries, bf16: forward 1.65 ms (1280 TFLOP/s), backward 5.6 ms
// (1130); 4096, 5120, 131072: 3.9 ms (1420) and 13.8 ms (1200).  What the pieces cost beside the
// products is the sums of dx: 168 MB per piece of 32768 entries in the second.
//
// bf16: a row's target entry of dl, (p - 1) dloss, is far larger than its others, and what
// rounding takes from it would be the largest error of both gradients.  It is kept aside: dx
// gets it times the target's row of w in the epilogue, and a dw tile takes one more k tile
// (per BK tokens whose targets lie in it) of these remainders against those tokens' rows of x.  The
// other entries' rounding does not show beside the outputs' own: 0.00166 of their root mean square
// either way.  Where most targets are the same few entries, their tiles of dw take that many more
// k tiles, unpipelined, and end the launch later; times here are of targets spread evenly.
//
// A row whose target is ignore_index, or lies outside [0, v), has loss 0 and no gradient, whatever
// it holds: its dl is 0, its dx is set to 0 (0 times an infinite weight is NaN), and a dw tile whose
// sums are not all finite is formed again without such rows (0 times a NaN of theirs).
#include "ss_gemm.h"
#include "ss_lm_internal.h"

namespace ssk {
namespace {

__device__ __forceinline__ bool live_target(int64_t t, const XentArgs& a)
{
    return t != a.ignore_index && t >= 0 && t < a.v;
}

// what both products over (x, w) share: rows of x against rows [v0, v0 + cols) of w
template <int DT>
struct XentLogits {
    using T = typename MM<DT>::T;
    const XentArgs& a;
    int64_t m0, n0;  // first row, first column of the vocabulary
    int tiles;

    __device__ const char* a_chunk(int row, int k) const
    {
        int64_t r = m0 + row;
        r = r < a.n ? r : a.n - 1;
        return reinterpret_cast<const char*>(static_cast<const T*>(a.x) + r * a.x_ld + k);
    }
    __device__ const char* b_chunk(int row, int k) const
    {
        int64_t r = n0 + row;
        r = r < a.v ? r : a.v - 1;
        return reinterpret_cast<const char*>(static_cast<const T*>(a.w) + r * a.w_ld + k);
    }
    __device__ int64_t a_off(int t) const { return int64_t(t) * 128; }
    __device__ int64_t b_off(int t) const { return int64_t(t) * 128; }
    __device__ int valid(int t) const { return k_left<DT>(DT == 0 ? a.d : a.d_pad, t); }
    __device__ const float* a_at(int row, int k) const { return reinterpret_cast<const float*>(a_chunk(row, k)); }
    __device__ const float* b_at(int row, int k) const { return reinterpret_cast<const float*>(b_chunk(row, k)); }
    __device__ int64_t a_cols() const { return 0; }
    __device__ int64_t b_cols() const { return 0; }
    __device__ int64_t a_ld() const { return 0; }
    __device__ int64_t b_ld() const { return 0; }
    static constexpr bool kSkips = false;
};

// ---- forward -------------------------------------------------------------------------------

// (m, s) stands for s exp(m): joins another pair.  An all -inf side leaves the other as it is.
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2)
{
    const float top = fmaxf(m, m2);
    // NaN: fmaxf drops it, but its sum is NaN and stays
    const float base = top == -__builtin_inff() ? 0.0f : top;
    s = s * exp2_hw((m - base) * kLog2e) + s2 * exp2_hw((m2 - base) * kLog2e);
    m = top;
}

template <int DT>
struct XentFwdProb : XentLogits<DT> {
    template <class G>
    __device__ void finish(f32x4 (&acc)[G::FM][G::FN], char* lds, int wm, int wn, int lane) const
    {
        const XentArgs& a = this->a;
        // waves of one kXentCols group of columns
        constexpr int kGroup = int(kXentCols) / (G::FN * 16);
        static_assert(kGroup >= 1 && G::BN % kXentCols == 0, "whole groups of columns per tile");
        float* const pm = reinterpret_cast<float*>(lds);           // (WN, BM)
        float* const ps = pm + G::WN * G::BM;
        __syncthreads();  // every wave has read its last operands
#pragma unroll
        for (int i = 0; i < G::FM; ++i) {
            const int r = (wm * G::FM + i) * 16 + (lane & 15);
            const int64_t m = this->m0 + r;
            const int64_t t = m < a.n ? a.target[m] : -1;
            float top = -__builtin_inff();
#pragma unroll
            for (int j = 0; j < G::FN; ++j) {
                const int64_t c = this->n0 + (wn * G::FN + j) * 16 + (lane >> 4) * 4;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (c + e == t && t < a.v) a.target_logit[m] = acc[i][j][e];
                    if (c + e < a.v) top = fmaxf(top, acc[i][j][e]);
                }
            }
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            const float base = top == -__builtin_inff() ? 0.0f : top;
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < G::FN; ++j) {
                const int64_t c = this->n0 + (wn * G::FN + j) * 16 + (lane >> 4) * 4;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (c + e < a.v) sum += exp2_hw((acc[i][j][e] - base) * kLog2e);
            }
            sum += __shfl_xor(sum, 16);
            sum += __shfl_xor(sum, 32);
            if (lane < 16) {
                pm[wn * G::BM + r] = top;
                ps[wn * G::BM + r] = sum;
            }
        }
        __syncthreads();
        for (int q = threadIdx.x; q < G::BM * (G::BN / int(kXentCols)); q += G::NT) {
            const int r = q % G::BM, g = q / G::BM;
            if (this->m0 + r >= a.n || this->n0 + g * kXentCols >= a.v) continue;
            float m = pm[g * kGroup * G::BM + r], s = ps[g * kGroup * G::BM + r];
#pragma unroll
            for (int w = 1; w < kGroup; ++w) join(m, s, pm[(g * kGroup + w) * G::BM + r], ps[(g * kGroup + w) * G::BM + r]);
            const int64_t at = (this->n0 / kXentCols + g) * a.n + this->m0 + r;
            a.part_max[at] = m;
            a.part_sum[at] = s;
        }
    }
};

// H: the geometry of half a tile (G itself where tiles are never halved)
template <class G, class H>
__global__ __launch_bounds__(G::NT) void xent_fwd_kernel(XentArgs a, TilePlan plan)
{
    __shared__ __attribute__((aligned(1024))) char lds[G::LDS];
    uint32_t tm, tn;
    const int half = tile_of(blockIdx.x, plan, &tm, &tn);
    XentFwdProb<G::DT> p{{a, int64_t(tm) * G::BM, int64_t(tn) * G::BN, int((a.d_pad + G::BK - 1) / G::BK)}};
    if (half < 0) {
        mm_tile<G>(p, lds);
        return;
    }
    p.m0 += half * H::BM;
    if (p.m0 < a.n) mm_tile<H>(p, lds);
}

// The pairs of a row, joined: ROWS rows per workgroup, 256 / ROWS threads a row.
template <int ROWS>
__global__ __launch_bounds__(256) void xent_join_kernel(XentArgs a, int64_t groups)
{
    constexpr int LANES = 256 / ROWS;
    __shared__ float sm[LANES][ROWS], ss[LANES][ROWS];
    const int r = threadIdx.x % ROWS, q = threadIdx.x / ROWS;
    const int64_t row = int64_t(blockIdx.x) * ROWS + r;
    float m = -__builtin_inff(), s = 0.0f;
    if (row < a.n) {
#pragma unroll 4
        for (int64_t g = q; g < groups; g += LANES) join(m, s, a.part_max[g * a.n + row], a.part_sum[g * a.n + row]);
    }
    sm[q][r] = m;
    ss[q][r] = s;
    for (int half = LANES / 2; half > 0; half /= 2) {
        __syncthreads();
        if (q < half) {
            join(m, s, sm[q + half][r], ss[q + half][r]);
            sm[q][r] = m;
            ss[q][r] = s;
        }
    }
    if (q != 0 || row >= a.n) return;
    const float lse = m + __builtin_amdgcn_logf(s) * kLn2;
    const int64_t t = a.target[row];
    a.lse[row] = lse;
    a.loss[row] = live_target(t, a) ? lse - a.target_logit[row] : 0.0f;
}

// Few rows: 32 columns of the vocabulary per workgroup.
template <int DT, int MT, bool ALIGNED>
struct XentStream {
    using T = typename MM<DT>::T;
    const XentArgs& a;
    int64_t c0;  // first column
    f32x4 s0[MT], s1[MT];

    __device__ __forceinline__ void run()
    {
        const int lane = threadIdx.x & 63;
        const T* px[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            int64_t m = i * 16 + (lane & 15);
            m = m < a.n ? m : a.n - 1;
            px[i] = static_cast<const T*>(a.x_raw) + m * a.x_raw_ld;
        }
        int64_t r0 = c0 + (lane & 15), r1 = r0 + 16;
        r0 = r0 < a.v ? r0 : a.v - 1;
        r1 = r1 < a.v ? r1 : a.v - 1;
        const T* const w = static_cast<const T*>(a.w_raw);
        stream_rows<DT, MT, ALIGNED>(w + r0 * a.d, w + r1 * a.d, px, a.d, s0, s1);
    }
};

template <int DT, int MT, bool ALIGNED>
__global__ __launch_bounds__(64 * kStreamWaves) void xent_fwd_stream_kernel(XentArgs a)
{
    XentStream<DT, MT, ALIGNED> x{a, int64_t(blockIdx.x) * kXentStreamCols, {}, {}};
    x.run();
    const int lane = threadIdx.x & 63;
    stream_join<MT>(x.s0, x.s1, [&](int i, f32x4 l0, f32x4 l1) {
        const int64_t m = i * 16 + (lane & 15), c = x.c0 + (lane >> 4) * 4;
        const int64_t t = m < a.n ? a.target[m] : -1;
        float top = -__builtin_inff(), sum = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int64_t col = c + (e & 3) + (e & 4) * 4;
            const float v = e < 4 ? l0[e & 3] : l1[e & 3];
            if (col == t && t < a.v) a.target_logit[m] = v;
            if (col < a.v) top = fmaxf(top, v);
        }
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float base = top == -__builtin_inff() ? 0.0f : top;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int64_t col = c + (e & 3) + (e & 4) * 4;
            const float v = e < 4 ? l0[e & 3] : l1[e & 3];
            if (col < a.v) sum += exp2_hw((v - base) * kLog2e);
        }
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        if (lane < 16 && m < a.n) {
            a.part_max[blockIdx.x * a.n + m] = top;
            a.part_sum[blockIdx.x * a.n + m] = sum;
        }
    });
}

// ---- backward ------------------------------------------------------------------------------

// dl of one piece: columns [v0, v0 + cols) of the vocabulary, rows of `pad` elements.
struct Piece {
    int64_t v0, cols, pad;
};

// What of row m's dl is the same for every column.
struct RowOfDl {
    int64_t target;
    bool live;
    float lse, scale;
    __device__ RowOfDl(const XentArgs& a, int64_t m)
        : target(a.target[m]), live(live_target(target, a)), lse(a.lse[m]), scale(a.dloss[m])
    {
    }
};

// Four neighbouring columns c.. of row m from their logits.
template <int DT>
__device__ __forceinline__ void dl_emit(const XentArgs& a, const Piece& p, const RowOfDl& row, int64_t m, int64_t c, f32x4 l)
{
    using T = typename MM<DT>::T;
    if (c - p.v0 >= p.pad) return;
    if (a.few) {  // fp32: nothing is rounded, nothing kept aside
        f32x4 q;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float v = exp2_hw((l[e] - row.lse) * kLog2e) - (c + e == row.target ? 1.0f : 0.0f);
            q[e] = row.live && c + e - p.v0 < p.cols ? v * row.scale : 0.0f;
        }
        *reinterpret_cast<f32x4*>(static_cast<float*>(a.dl) + m * p.pad + (c - p.v0)) = q;
        return;
    }
    typedef T T4 __attribute__((ext_vector_type(4)));
    T4 q;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float v = exp2_hw((l[e] - row.lse) * kLog2e) - (c + e == row.target ? 1.0f : 0.0f);
        // the columns past the piece's end hold zeros: the products read them
        const float full = row.live && c + e - p.v0 < p.cols ? v * row.scale : 0.0f;
        q[e] = MM<DT>::narrow(full);
        if (DT == 1 && row.live && c + e == row.target && c + e - p.v0 < p.cols) a.lo[m] = full - MM<DT>::widen(q[e]);
    }
    *reinterpret_cast<T4*>(static_cast<T*>(a.dl) + m * p.pad + (c - p.v0)) = q;
}

template <int DT>
struct XentDlProb : XentLogits<DT> {
    Piece piece;

    template <class G>
    __device__ void finish(f32x4 (&acc)[G::FM][G::FN], char*, int wm, int wn, int lane) const
    {
        const XentArgs& a = this->a;
#pragma unroll
        for (int i = 0; i < G::FM; ++i) {
            const int64_t m = this->m0 + (wm * G::FM + i) * 16 + (lane & 15);
            if (m >= a.n) continue;
            const RowOfDl row(a, m);
#pragma unroll
            for (int j = 0; j < G::FN; ++j)
                dl_emit<DT>(a, piece, row, m, this->n0 + (wn * G::FN + j) * 16 + (lane >> 4) * 4, acc[i][j]);
        }
    }
};

// Few rows: 32 columns of the piece per workgroup.
template <int DT, int MT, bool ALIGNED>
__global__ __launch_bounds__(64 * kStreamWaves) void xent_dl_stream_kernel(XentArgs a, Piece piece)
{
    XentStream<DT, MT, ALIGNED> x{a, piece.v0 + int64_t(blockIdx.x) * kXentStreamCols, {}, {}};
    x.run();
    const int lane = threadIdx.x & 63;
    stream_join<MT>(x.s0, x.s1, [&](int i, f32x4 l0, f32x4 l1) {
        const int64_t m = i * 16 + (lane & 15), c = x.c0 + (lane >> 4) * 4;
        if (m >= a.n) return;
        const RowOfDl row(a, m);
        dl_emit<DT>(a, piece, row, m, c, l0);
        dl_emit<DT>(a, piece, row, m, c + 16, l1);
    });
}

template <class G, class H>
__global__ __launch_bounds__(G::NT) void xent_dl_kernel(XentArgs a, int64_t v0, int64_t cols, int64_t pad, TilePlan plan)
{
    __shared__ __attribute__((aligned(1024))) char lds[G::LDS];
    uint32_t tm, tn;
    const int half = tile_of(blockIdx.x, plan, &tm, &tn);
    XentDlProb<G::DT> p{
        {a, int64_t(tm) * G::BM, v0 + int64_t(tn) * G::BN, int((a.d_pad + G::BK - 1) / G::BK)}, {v0, cols, pad}};
    if (half < 0) {
        mm_tile<G>(p, lds);
        return;
    }
    p.m0 += half * H::BM;
    if (p.m0 < a.n) mm_tile<H>(p, lds);
}

// The tokens whose targets lie in each group of kXentCols columns, in order.
__global__ __launch_bounds__(256) void xent_list_kernel(XentArgs a)
{
    const int64_t from = int64_t(blockIdx.x) * kXentCols;
    int32_t* const list = a.tokens + int64_t(blockIdx.x) * a.n;
    __shared__ int found[2][4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int count = 0, buf = 0;
    for (int64_t i = 0; i < a.n; i += 256, buf ^= 1) {
        const int64_t tok = i + threadIdx.x;
        const int64_t t = tok < a.n ? a.target[tok] : -1;
        const bool in = t >= from && t < from + kXentCols && live_target(t, a);
        const uint64_t mask = __ballot(in);
        if (lane == 0) found[buf][wave] = __popcll(mask);
        __syncthreads();
        int at = count;
        for (int w = 0; w < 4; ++w) {
            if (w < wave) at += found[buf][w];
            count += found[buf][w];
        }
        if (in) list[at + __popcll(mask & ((uint64_t(1) << lane) - 1))] = int32_t(tok);
    }
    if (threadIdx.x == 0) a.counts[blockIdx.x] = count;
}

// dx += dl w over one piece
template <int DT>
struct XentDxProb {
    using T = typename MM<DT>::T;
    static constexpr int BK = 8 * MM<DT>::kEpc;
    const XentArgs& a;
    int64_t m0, n0, v0, cols, pad;
    int tiles;
    int from;       // this part's first k tile
    float* acc_to;  // this part's sums over the pieces so far; null with one piece and one part
    bool first, last;  // of the pieces; last: and the only part

    __device__ const char* a_chunk(int row, int k) const
    {
        int64_t r = m0 + row;
        r = r < a.n ? r : a.n - 1;
        return reinterpret_cast<const char*>(static_cast<const T*>(a.dl) + r * pad + k);
    }
    __device__ const char* b_chunk(int col, int k) const
    {
        int64_t c = n0 + col;
        c = c < a.d_pad ? c : a.d_pad - MM<DT>::kEpc;
        return reinterpret_cast<const char*>(static_cast<const T*>(a.w) + (v0 + k) * a.w_ld + c);
    }
    __device__ int64_t a_off(int t) const { return int64_t(t + from) * 128; }
    __device__ int64_t b_off(int t) const { return int64_t(t + from) * BK * a.w_ld * int64_t(sizeof(T)); }
    __device__ int valid(int t) const { return k_left<DT>(cols, t + from); }

    __device__ const float* a_at(int row, int k) const { return reinterpret_cast<const float*>(a_chunk(row, k)); }
    __device__ const float* b_at(int col, int k) const
    {
        const int64_t c = n0 + col < a.d ? n0 + col : a.d - 1;
        return static_cast<const float*>(a.w) + (v0 + k) * a.w_ld + c;
    }
    __device__ int64_t a_cols() const { return 0; }
    __device__ int64_t b_cols() const { return a.d - n0; }
    __device__ int64_t a_ld() const { return 0; }
    __device__ int64_t b_ld() const { return a.w_ld; }
    static constexpr bool kSkips = false;

    template <class G>
    __device__ void finish(f32x4 (&acc)[G::FM][G::FN], char*, int wm, int wn, int lane) const
    {
#pragma unroll
        for (int i = 0; i < G::FM; ++i) {
            const int64_t m = m0 + (wm * G::FM + i) * 16 + (lane & 15);
            if (m >= a.n) continue;
            const int64_t t = a.target[m];
            const bool live = live_target(t, a), add = DT == 1 && last && live;
            const float lo = add ? a.lo[m] : 0.0f;
            const T* const wt = static_cast<const T*>(a.w) + (add ? t : 0) * a.w_ld;
#pragma unroll
            for (int j = 0; j < G::FN; ++j) {
                const int64_t c = n0 + (wn * G::FN + j) * 16 + (lane >> 4) * 4;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (c + e >= a.d) continue;
                    float v = acc[i][j][e];
                    if (!first) v += acc_to[m * a.d + c + e];
                    if (add) v = fmaf(lo, MM<DT>::widen(wt[c + e]), v);
                    if (last)
                        static_cast<T*>(a.dx)[m * a.d + c + e] = MM<DT>::narrow(live ? v : 0.0f);
                    else
                        acc_to[m * a.d + c + e] = v;
                }
            }
        }
    }
};

// rows [v0, v0 + cols) of dw = dl^T x
template <int DT>
struct XentDwProb {
    using T = typename MM<DT>::T;
    static constexpr int BK = 8 * MM<DT>::kEpc;
    const XentArgs& a;
    int64_t m0, n0, v0, cols, pad;
    int tiles;
    int first;    // this part's first k tile
    float* part;  // where this part's sums go; null: dw itself
    bool vec;

    __device__ const char* a_chunk(int col, int k) const
    {
        int64_t c = m0 + col;
        c = c < pad ? c : pad - MM<DT>::kEpc;
        return reinterpret_cast<const char*>(static_cast<const T*>(a.dl) + int64_t(k) * pad + c);
    }
    __device__ const char* b_chunk(int col, int k) const
    {
        int64_t c = n0 + col;
        c = c < a.d_pad ? c : a.d_pad - MM<DT>::kEpc;
        return reinterpret_cast<const char*>(static_cast<const T*>(a.x) + int64_t(k) * a.x_ld + c);
    }
    __device__ int64_t a_off(int t) const { return int64_t(t + first) * BK * pad * int64_t(sizeof(T)); }
    __device__ int64_t b_off(int t) const { return int64_t(t + first) * BK * a.x_ld * int64_t(sizeof(T)); }
    __device__ int valid(int t) const { return k_left<DT>(a.n, t + first); }

    __device__ const float* a_at(int col, int k) const
    {
        const int64_t c = m0 + col < pad ? m0 + col : pad - 1;
        return static_cast<const float*>(a.dl) + int64_t(k) * pad + c;
    }
    __device__ const float* b_at(int col, int k) const
    {
        const int64_t c = n0 + col < a.d ? n0 + col : a.d - 1;
        return static_cast<const float*>(a.x) + int64_t(k) * a.x_ld + c;
    }
    __device__ int64_t a_cols() const { return pad - m0; }
    __device__ int64_t b_cols() const { return a.d - n0; }
    __device__ int64_t a_ld() const { return pad; }
    __device__ int64_t b_ld() const { return a.x_ld; }
    // tiles formed again leave out the rows of x without a target
    static constexpr bool kSkips = true;
    __device__ bool skips(int t, int k) const { return !live_target(a.target[int64_t(t + first) * BK + k], a); }

    // bf16: a tile whose sums are not all finite, again
    template <class G>
    __device__ void again(f32x4 (&acc)[G::FM][G::FN], char* lds, int wm, int wn, int lane) const
    {
        const int tid = threadIdx.x;
        int* const odd = reinterpret_cast<int*>(lds);
        __syncthreads();  // every wave has read its last operands
        if (tid == 0) *odd = 0;
        __syncthreads();
        if (!all_finite<G>(acc)) *odd = 1;
        __syncthreads();
        if (!*odd) return;
        char* const a_dst = lds + (G::A_PARTS > 1 ? wm * (G::A_PART * 128) + wn * 1024 : (tid >> 6) * 1024);
        char* const b_dst = lds + 2 * G::A_BYTES + (tid >> 6) * 1024;
        const char* const zero = reinterpret_cast<const char*>(g_zero_chunk);
#pragma unroll
        for (int i = 0; i < G::FM; ++i)
#pragma unroll
            for (int j = 0; j < G::FN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
        for (int t = 0; t < tiles; ++t) {
            const int exist = valid(t);
            __syncthreads();  // the last tile's readers are done
            int col, k;
#pragma unroll
            for (int i = 0; i < G::NA; ++i) {
                a_place<G>(i, tid, &col, &k);
                load_to_lds(k < exist ? a_chunk(col, k) + a_off(t) : zero, a_dst + i * (G::A_NT * 16));
            }
#pragma unroll
            for (int i = 0; i < G::NB; ++i) {
                b_place<G>(i, tid, &col, &k);
                load_to_lds(k < exist && !skips(t, k) ? b_chunk(col, k) + b_off(t) : zero, b_dst + i * (G::NT * 16));
            }
            wait_loads<0>();
            __syncthreads();
            mm_step<G>(lds, lds + 2 * G::A_BYTES, wm, wn, lane, acc);
        }
    }

    // the target entries' remainders
    template <class G>
    __device__ void remainders(f32x4 (&acc)[G::FM][G::FN], char* lds, int wm, int wn, int lane) const
    {
        using M = MM<DT>;
        const int tid = threadIdx.x;
        // the groups of columns that the tile shares with (a mini tile is half of one)
        const int64_t top = m0 + G::BM < cols ? m0 + G::BM : cols;
#pragma unroll 1
        for (int64_t g = (v0 + m0) / kXentCols; g * kXentCols < v0 + top; ++g) {
            const int32_t* const list = a.tokens + g * a.n;
            const int count = a.counts[g];
#pragma unroll 1
            for (int at = 0; at < count; at += BK) {
                __syncthreads();  // the stage's last readers are done
                for (int q = tid; q < G::A_BYTES / 16; q += G::NT)
                    reinterpret_cast<f32x4*>(lds)[q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                int col, k;
#pragma unroll
                for (int i = 0; i < G::NB; ++i) {
                    b_place<G>(i, tid, &col, &k);
                    int64_t c = n0 + col;
                    c = c < a.d_pad ? c : a.d_pad - M::kEpc;
                    const char* src = reinterpret_cast<const char*>(g_zero_chunk);
                    if (at + k < count) src = reinterpret_cast<const char*>(static_cast<const T*>(a.x) + list[at + k] * a.x_ld + c);
                    load_to_lds(src, lds + 2 * G::A_BYTES + (tid >> 6) * 1024 + i * (G::NT * 16));
                }
                __syncthreads();
                if (tid < BK && at + tid < count) {
                    const int tok = list[at + tid];
                    const int m = int(a.target[tok] - v0 - m0);
                    if (m >= 0 && m < G::BM) *reinterpret_cast<T*>(lds + a_mc_offset<G>(m, tid)) = M::narrow(a.lo[tok]);
                }
                __syncthreads();
                mm_step<G>(lds, lds + 2 * G::A_BYTES, wm, wn, lane, acc);
            }
        }
    }

    template <class G>
    __device__ void finish(f32x4 (&acc)[G::FM][G::FN], char* lds, int wm, int wn, int lane) const
    {
        if constexpr (DT == 1) {
            again<G>(acc, lds, wm, wn, lane);
            if (first == 0) remainders<G>(acc, lds, wm, wn, lane);  // by the first part
        }
#pragma unroll
        for (int i = 0; i < G::FM; ++i) {
            const int64_t r = m0 + (wm * G::FM + i) * 16 + (lane & 15);
            if (r >= cols) continue;
            T* const row = static_cast<T*>(a.dw) + (v0 + r) * a.d;
#pragma unroll
            for (int j = 0; j < G::FN; ++j) {
                const int64_t c = n0 + (wn * G::FN + j) * 16 + (lane >> 4) * 4;
                if (part) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (c + e < a.d) part[r * a.d + c + e] = acc[i][j][e];
                } else if (vec && c + 4 <= a.d) {
                    typedef T T4 __attribute__((ext_vector_type(4)));
                    T4 q;
#pragma unroll
                    for (int e = 0; e < 4; ++e) q[e] = MM<DT>::narrow(acc[i][j][e]);
                    *reinterpret_cast<T4*>(row + c) = q;
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (c + e < a.d) row[c + e] = MM<DT>::narrow(acc[i][j][e]);
                }
            }
        }
    }
};

// A part's share of `all` k tiles: the first, and how many (rounding, or a short last piece, may leave
// parts nothing).
__device__ __forceinline__ void share(int64_t all, int64_t parts, uint32_t part, int* first, int* tiles)
{
    const int64_t depth = (all + parts - 1) / parts, from = part * depth, left = all > from ? all - from : 0;
    *first = int(from);
    *tiles = int(left < depth ? left : depth);
}

// Both sets of tiles: dx's, dx_splits times px, and then dw's, dw_splits times pw.  HX, HW: their halves.
template <class GX, class HX, class GW, class HW>
__global__ __launch_bounds__(GX::NT) void xent_grad_kernel(XentArgs a, int64_t v0, int64_t cols, int64_t pad, TilePlan px,
                                                           TilePlan pw, bool first, bool last, bool vec_w)
{
    static_assert(GX::NT == GW::NT && GX::LDS == GW::LDS, "one launch");
    __shared__ __attribute__((aligned(1024))) char lds[GX::LDS];
    uint32_t tm, tn;
    const uint32_t per_x = px.blocks(), n_dx = per_x * uint32_t(a.dx_splits);
    int from, tiles;
    if (blockIdx.x < n_dx) {
        const uint32_t part = blockIdx.x / per_x;
        const int h = tile_of(blockIdx.x % per_x, px, &tm, &tn);
        share((cols + GX::BK - 1) / GX::BK, a.dx_splits, part, &from, &tiles);
        XentDxProb<GX::DT> p{a,    int64_t(tm) * GX::BM, int64_t(tn) * GX::BN, v0, cols, pad, tiles,
                             from, a.dx_acc ? a.dx_acc + int64_t(part) * a.n * a.d : nullptr, first,
                             last && a.dx_splits == 1};
        if (h < 0) {
            mm_tile<GX>(p, lds);
            return;
        }
        p.m0 += h * HX::BM;
        if (p.m0 < a.n) mm_tile<HX>(p, lds);
    } else {
        const uint32_t id = blockIdx.x - n_dx, per_w = pw.blocks(), part = id / per_w;
        const int h = tile_of(id % per_w, pw, &tm, &tn);
        share((a.n + GW::BK - 1) / GW::BK, a.dw_splits, part, &from, &tiles);
        XentDwProb<GW::DT> p{a,    int64_t(tm) * GW::BM, int64_t(tn) * GW::BN, v0, cols, pad, tiles,
                             from, a.dw_part ? a.dw_part + int64_t(part) * cols * a.d : nullptr, vec_w};
        if (h < 0) {
            mm_tile<GW>(p, lds);
            return;
        }
        p.m0 += h * HW::BM;
        if (p.m0 < cols) mm_tile<HW>(p, lds);
    }
}

// A piece's rows of dw from their parts, in order.
template <int DT>
__global__ __launch_bounds__(256) void xent_dw_sum_kernel(XentArgs a, int64_t v0, int64_t cols)
{
    const int64_t n = cols * a.d;
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256) {
        float s = 0.0f;
#pragma unroll 8
        for (int64_t p = 0; p < a.dw_splits; ++p) s += a.dw_part[p * n + i];
        static_cast<typename MM<DT>::T*>(a.dw)[v0 * a.d + i] = MM<DT>::narrow(s);
    }
}

// dx from its parts, in order, and (bf16) its rows' target remainders.
template <int DT>
__global__ __launch_bounds__(256) void xent_dx_sum_kernel(XentArgs a)
{
    using T = typename MM<DT>::T;
    const int64_t n = a.n * a.d;
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256) {
        float s = 0.0f;
#pragma unroll 8
        for (int64_t p = 0; p < a.dx_splits; ++p) s += a.dx_acc[p * n + i];
        const int64_t row = i / a.d, t = a.target[row];
        if (!live_target(t, a))
            s = 0.0f;
        else if (DT == 1)
            s = fmaf(a.lo[row], MM<DT>::widen(static_cast<const T*>(a.w)[t * a.w_ld + i % a.d]), s);
        static_cast<T*>(a.dx)[i] = MM<DT>::narrow(s);
    }
}

// ---- launches --------------------------------------------------------------------------------

template <class G, class H>
hipError_t fwd_tiles(const XentArgs& a, hipStream_t s)
{
    const TilePlan plan = plan_tiles(up(a.n, G::BM), up(a.v, G::BN), H::BM < G::BM);
    xent_fwd_kernel<G, H><<<dim3(plan.blocks()), dim3(G::NT), 0, s>>>(a, plan);
    return hipGetLastError();
}

template <int DT>
hipError_t fwd_tiles_dt(const XentArgs& a, hipStream_t s)
{
    const Tile t = best_tile<DT>(count(a.n, a.v, 256, 256), count(a.n, a.v, 128, 128), count(a.n, a.v, 64, 128));
    if constexpr (DT == 1) {
        if (t == Tile::Large) return fwd_tiles<LargeTile<false, false>, HalfTile<false, false>>(a, s);
    }
    using S = typename Tiles<DT>::template Small<false, false>;
    using M = typename Tiles<DT>::template Mini<false, false>;
    return t == Tile::Mini ? fwd_tiles<M, M>(a, s) : fwd_tiles<S, S>(a, s);
}

template <int DT, int MT>
hipError_t fwd_stream(const XentArgs& a, hipStream_t s)
{
    const dim3 grid(up(a.v, kXentStreamCols)), block(64 * kStreamWaves);
    if (a.aligned)
        xent_fwd_stream_kernel<DT, MT, true><<<grid, block, 0, s>>>(a);
    else
        xent_fwd_stream_kernel<DT, MT, false><<<grid, block, 0, s>>>(a);
    return hipGetLastError();
}

template <int DT>
hipError_t fwd_dt(const XentArgs& a, hipStream_t s)
{
    const hipError_t e = !a.stream   ? fwd_tiles_dt<DT>(a, s)
                         : a.n <= 16 ? fwd_stream<DT, 1>(a, s)
                         : a.n <= 32 ? fwd_stream<DT, 2>(a, s)
                                     : fwd_stream<DT, 4>(a, s);
    if (e != hipSuccess) return e;
    const int64_t groups = up(a.v, a.stream ? kXentStreamCols : kXentCols);
    // few rows: more threads on each
    if (a.n >= 4096)
        xent_join_kernel<16><<<dim3(up(a.n, 16)), dim3(256), 0, s>>>(a, groups);
    else
        xent_join_kernel<2><<<dim3(up(a.n, 2)), dim3(256), 0, s>>>(a, groups);
    return hipGetLastError();
}

template <int DT, int MT>
hipError_t dl_stream(const XentArgs& a, const Piece& p, hipStream_t s)
{
    const dim3 grid(up(p.pad, kXentStreamCols)), block(64 * kStreamWaves);
    if (a.aligned)
        xent_dl_stream_kernel<DT, MT, true><<<grid, block, 0, s>>>(a, p);
    else
        xent_dl_stream_kernel<DT, MT, false><<<grid, block, 0, s>>>(a, p);
    return hipGetLastError();
}

template <class G, class H>
hipError_t dl_tiles(const XentArgs& a, int64_t v0, int64_t cols, int64_t pad, hipStream_t s)
{
    const TilePlan plan = plan_tiles(up(a.n, G::BM), up(pad, G::BN), H::BM < G::BM);
    xent_dl_kernel<G, H><<<dim3(plan.blocks()), dim3(G::NT), 0, s>>>(a, v0, cols, pad, plan);
    return hipGetLastError();
}

template <int DT>
hipError_t dl_tiles_dt(const XentArgs& a, int64_t v0, int64_t cols, int64_t pad, hipStream_t s)
{
    if (a.stream)
        return a.n <= 16   ? dl_stream<DT, 1>(a, {v0, cols, pad}, s)
               : a.n <= 32 ? dl_stream<DT, 2>(a, {v0, cols, pad}, s)
                           : dl_stream<DT, 4>(a, {v0, cols, pad}, s);
    const Tile t = best_tile<DT>(count(a.n, pad, 256, 256), count(a.n, pad, 128, 128), count(a.n, pad, 64, 128));
    if constexpr (DT == 1) {
        if (t == Tile::Large)
            return dl_tiles<LargeTile<false, false>, HalfTile<false, false>>(a, v0, cols, pad, s);
    }
    using S = typename Tiles<DT>::template Small<false, false>;
    using M = typename Tiles<DT>::template Mini<false, false>;
    return t == Tile::Mini ? dl_tiles<M, M>(a, v0, cols, pad, s) : dl_tiles<S, S>(a, v0, cols, pad, s);
}

template <class GX, class HX, class GW, class HW>
hipError_t grad_tiles(const XentArgs& a, int64_t v0, int64_t cols, int64_t pad, hipStream_t s)
{
    const bool can = HX::BM < GX::BM;
    const uint32_t sx = uint32_t(a.dx_splits), sw = uint32_t(a.dw_splits);
    TilePlan px{0, 0, 0, 0}, pw{0, 0, 0, 0};
    // only the last tiles of a launch are halved
    if (a.dx) px = plan_tiles(up(a.n, GX::BM), up(a.d, GX::BN), can && !a.dw && sx == 1);
    if (a.dw) pw = plan_tiles(up(cols, GW::BM), up(a.d, GW::BN), can && sw == 1, px.whole * sx);
    const bool vec = a.d % 4 == 0 && reinterpret_cast<uintptr_t>(a.dw) % (GX::DT == 0 ? 16 : 8) == 0;
    xent_grad_kernel<GX, HX, GW, HW><<<dim3(px.blocks() * sx + pw.blocks() * sw), dim3(GX::NT), 0, s>>>(
        a, v0, cols, pad, px, pw, v0 == 0, v0 + cols == a.v, vec);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.dw || sw == 1) return e;
    const int64_t blocks = (cols * a.d + 255) / 256;
    xent_dw_sum_kernel<GX::DT><<<dim3(unsigned(blocks < 4096 ? blocks : 4096)), dim3(256), 0, s>>>(a, v0, cols);
    return hipGetLastError();
}

template <int DT>
hipError_t grad_tiles_dt(const XentArgs& a, int64_t v0, int64_t cols, int64_t pad, hipStream_t s)
{
    auto tiles = [&](int bm, int bn) {
        return (a.dx ? count(a.n, a.d, bm, bn) * a.dx_splits : 0) + (a.dw ? count(cols, a.d, bm, bn) * a.dw_splits : 0);
    };
    const Tile t = best_tile<DT>(tiles(256, 256), tiles(128, 128), tiles(64, 128));
    if constexpr (DT == 1) {
        if (t == Tile::Large)
            return grad_tiles<LargeTile<false, true>, HalfTile<false, true>, LargeTile<true, true>, HalfTile<true, true>>(
                a, v0, cols, pad, s);
    }
    using T = Tiles<DT>;
    using SX = typename T::template Small<false, true>;
    using SW = typename T::template Small<true, true>;
    using MX = typename T::template Mini<false, true>;
    using MW = typename T::template Mini<true, true>;
    return t == Tile::Mini ? grad_tiles<MX, MX, MW, MW>(a, v0, cols, pad, s)
                           : grad_tiles<SX, SX, SW, SW>(a, v0, cols, pad, s);
}

template <int DT>
hipError_t bwd_dt(const XentArgs& a, hipStream_t s)
{
    if (a.few) {
        const int64_t pad = (a.v + 15) / 16 * 16;
        const hipError_t e = dl_tiles_dt<DT>(a, 0, a.v, pad, s);
        if (e != hipSuccess) return e;
        return launch_few_grad({static_cast<const float*>(a.dl), pad, 0, a.w_raw, nullptr, a.dw, nullptr, a.x_raw,
                                a.x_raw_ld, a.dx ? a.dx_acc : nullptr, a.dx, a.v, a.v, a.n, a.d, a.dx_per, a.dx_splits,
                                a.target, a.ignore_index},
                               DT, s);
    }
    if (DT == 1 && a.dw) {
        xent_list_kernel<<<dim3(up(a.v, kXentCols)), dim3(256), 0, s>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    for (int64_t v0 = 0; v0 < a.v; v0 += a.piece) {
        const int64_t cols = a.v - v0 < a.piece ? a.v - v0 : a.piece;
        const int64_t pad = (cols + 15) / 16 * 16;
        hipError_t e = dl_tiles_dt<DT>(a, v0, cols, pad, s);
        if (e == hipSuccess) e = grad_tiles_dt<DT>(a, v0, cols, pad, s);
        if (e != hipSuccess) return e;
    }
    if (!a.dx || a.dx_splits == 1) return hipSuccess;
    const int64_t blocks = (a.n * a.d + 255) / 256;
    xent_dx_sum_kernel<DT><<<dim3(unsigned(blocks < 4096 ? blocks : 4096)), dim3(256), 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_xent_fwd(const XentArgs& a, int dtype, hipStream_t stream)
{
    (void)hipGetLastError();
    return dtype == 0 ? fwd_dt<0>(a, stream) : fwd_dt<1>(a, stream);
}

hipError_t launch_xent_bwd(const XentArgs& a, int dtype, hipStream_t stream)
{
    (void)hipGetLastError();
    return dtype == 0 ? bwd_dt<0>(a, stream) : bwd_dt<1>(a, stream);
}

}  // namespace ssk
