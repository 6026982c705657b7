// gfx950 kernels of the gated feed-forward projection
//   g = x Wg^T, u = x Wu^T, h = act(g) u          x (m, k), Wg and Wu (f, k), h (m, f)
// and its gradients
//   dg = dh u act'(g), du = dh act(g)
//   dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x.
//
// Forward: one kernel.  A tile's B rows are 32 rows of Wg and the same 32 of Wu in turn for
// each wave column, so that one wave holds g and u of the same elements in its accumulators
// and the product never leaves the registers; g and u are not stored.
// Backward: the same product again with dh in the epilogue gives dg and du (rounded once to
// the operands' type, as the next product's operands must be: of bf16 gradients 0.00235 of their root
// mean square is off for 0.00166 by their own rounding alone, where products of the remainders too
// would double the gradients' time; of a few bf16 tokens what the rounding leaves is kept for the
// weights' gradients, see kGluLoRows), side by side in one (m, 2 f) workspace matrix;
// the second launch holds the tiles of dx (contraction over the 2 f columns of that matrix
// against the rows of Wg, then of Wu) and those of dWg and dWu (its transpose against x)
// together, so that one set's last tiles run beside the other's first.
// All three are bound by the matrix cores at training sizes (k = 2560, f = 6912, bf16, silu):
// forward, 4096 tokens 228 us, 16384 tokens 935 us (1270 and 1240 TFLOP/s); backward, 16384 tokens
// 1090 us for dg and du again and 2.12 ms for the gradients (1060 and 1090 TFLOP/s).  Keeping g and
// u would spare the 1.08 ms and take 4 m f bytes for each layer (453 MB here).
// Few tokens: the weights stream past them (see ss_gemm.h); one token 13.5 us, 5.2 TB/s.
#include "ss_gemm.h"
#include "ss_lm_internal.h"

namespace ssk {
namespace {

// ---- the activation ----------------------------------------------------------------------

constexpr float kGeluA = 0.79788456f;   // sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;

__device__ __forceinline__ float sigmoidf(float v) { return __builtin_amdgcn_rcpf(1.0f + exp2_hw(-v * kLog2e)); }

// gelu's tanh form: 0.5 g (1 + tanh(s)) = g sigmoid(2 s), s = sqrt(2/pi) (g + 0.044715 g^3)
template <int ACT>
__device__ __forceinline__ float act_of(float g)
{
    if constexpr (ACT == kActSilu) return g * sigmoidf(g);
    const float s2 = 2.0f * kGeluA * fmaf(kGeluB * g * g, g, g);
    return g * sigmoidf(s2);
}

// act and its derivative
template <int ACT>
__device__ __forceinline__ void act_grad(float g, float* act, float* slope)
{
    if constexpr (ACT == kActSilu) {
        const float s = sigmoidf(g);
        *act = g * s;
        *slope = fmaf(g * s, 1.0f - s, s);
    } else {
        const float s2 = 2.0f * kGeluA * fmaf(kGeluB * g * g, g, g);
        const float s = sigmoidf(s2);
        *act = g * s;
        *slope = fmaf(g * s * (1.0f - s), 2.0f * kGeluA * fmaf(3.0f * kGeluB * g, g, 1.0f), s);
    }
}

template <int DT>
struct Vec4;
template <>
struct Vec4<0> {
    using V = f32x4;
};
template <>
struct Vec4<1> {
    using V = bf16x4;
};

// 4 neighbouring elements of a row whose first `left` exist; vec: 4-element accesses are aligned
template <int DT>
__device__ __forceinline__ void load4(const typename MM<DT>::T* p, int64_t left, bool vec, float (&v)[4])
{
    if (vec && left >= 4) {
        const auto q = *reinterpret_cast<const typename Vec4<DT>::V*>(p);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = MM<DT>::widen(q[e]);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = e < left ? MM<DT>::widen(p[e]) : 0.0f;
    }
}
template <int DT>
__device__ __forceinline__ void store4(typename MM<DT>::T* p, int64_t left, bool vec, const float (&v)[4])
{
    if (vec && left >= 4) {
        typename Vec4<DT>::V q;
#pragma unroll
        for (int e = 0; e < 4; ++e) q[e] = MM<DT>::narrow(v[e]);
        *reinterpret_cast<typename Vec4<DT>::V*>(p) = q;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < left) p[e] = MM<DT>::narrow(v[e]);
    }
}

// ---- g and u, and what is made of them ----------------------------------------------------

// Four neighbouring features f.. of token m.  BACK: dg and du into the workspace instead of h.
// vec: rows of h (dh) are aligned for 4-element accesses.
template <int DT, int ACT, bool BACK>
__device__ __forceinline__ void glu_emit(const GluArgs& a, int64_t m, int64_t f, f32x4 g, f32x4 u, bool vec)
{
    using T = typename MM<DT>::T;
    if constexpr (!BACK) {
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = act_of<ACT>(g[e]) * u[e];
        if (f < a.f) store4<DT>(static_cast<T*>(a.h) + m * a.f + f, a.f - f, vec, v);
    } else {
        if (f >= a.f_pad) return;
        float d[4] = {0.0f, 0.0f, 0.0f, 0.0f}, dg[4], du[4];
        if (f < a.f) load4<DT>(static_cast<const T*>(a.dh) + m * a.f + f, a.f - f, vec, d);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float act, slope;
            act_grad<ACT>(g[e], &act, &slope);
            // the pad columns f..f_pad hold zeros: later products read them
            const bool in = f + e < a.f;
            dg[e] = in ? d[e] * u[e] * slope : 0.0f;
            du[e] = in ? d[e] * act : 0.0f;
        }
        // f_pad is a multiple of 4: whole groups, aligned
        if (a.few) {
            float* const row = static_cast<float*>(a.dgu) + m * 2 * a.f_pad + f;
            store4<0>(row, 4, true, dg);
            store4<0>(row + a.f_pad, 4, true, du);
            return;
        }
        T* const row = static_cast<T*>(a.dgu) + m * 2 * a.f_pad + f;
        store4<DT>(row, 4, true, dg);
        store4<DT>(row + a.f_pad, 4, true, du);
        if (DT == 1 && a.lo) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                dg[e] -= MM<DT>::widen(MM<DT>::narrow(dg[e]));
                du[e] -= MM<DT>::widen(MM<DT>::narrow(du[e]));
            }
            T* const rest = row + a.m * 2 * a.f_pad;
            store4<DT>(rest, 4, true, dg);
            store4<DT>(rest + a.f_pad, 4, true, du);
        }
    }
}

template <int DT, int ACT, bool BACK>
struct GluProb {
    using T = typename MM<DT>::T;
    const GluArgs& a;
    int64_t m0, f0;  // the tile's first token and first feature
    int tiles;
    bool vec;

    __device__ const char* a_chunk(int row, int k) const
    {
        int64_t r = m0 + row;
        r = r < a.m ? r : a.m - 1;
        return reinterpret_cast<const char*>(static_cast<const T*>(a.x) + r * a.x_ld + k);
    }
    __device__ const char* b_chunk(int row, int k) const
    {
        // 64 tile rows per wave column: 32 of Wg, then the same 32 of Wu
        int64_t r = f0 + (row >> 6) * 32 + (row & 31);
        r = r < a.f ? r : a.f - 1;
        return reinterpret_cast<const char*>(static_cast<const T*>((row & 32) ? a.wu : a.wg) + r * a.w_ld + k);
    }
    __device__ int64_t a_off(int t) const { return int64_t(t) * 128; }
    __device__ int64_t b_off(int t) const { return int64_t(t) * 128; }
    __device__ int valid(int t) const { return k_left<DT>(DT == 0 ? a.k : a.k_pad, t); }
    __device__ const float* a_at(int row, int k) const { return reinterpret_cast<const float*>(a_chunk(row, k)); }
    __device__ const float* b_at(int row, int k) const { return reinterpret_cast<const float*>(b_chunk(row, k)); }
    __device__ int64_t a_cols() const { return 0; }
    __device__ int64_t b_cols() const { return 0; }
    __device__ int64_t a_ld() const { return 0; }
    __device__ int64_t b_ld() const { return 0; }
    static constexpr bool kSkips = false;

    template <class G>
    __device__ void finish(f32x4 (&acc)[G::FM][G::FN], char*, int wm, int wn, int lane) const
    {
        static_assert(G::FN == 4, "a wave column holds 32 + 32 tile rows of B");
#pragma unroll
        for (int i = 0; i < G::FM; ++i) {
            const int64_t m = m0 + (wm * G::FM + i) * 16 + (lane & 15);
            if (m >= a.m) continue;
#pragma unroll
            for (int j = 0; j < 2; ++j)
                glu_emit<DT, ACT, BACK>(a, m, f0 + wn * 32 + j * 16 + (lane >> 4) * 4, acc[i][j], acc[i][j + 2], vec);
        }
    }
};

// H: the geometry of half a tile (G itself where tiles are never halved)
template <class G, class H, int ACT, bool BACK>
__global__ __launch_bounds__(G::NT) void glu_tile_kernel(GluArgs a, TilePlan plan, bool vec)
{
    __shared__ __attribute__((aligned(1024))) char lds[G::LDS];
    uint32_t tm, tf;
    const int half = tile_of(blockIdx.x, plan, &tm, &tf);
    GluProb<G::DT, ACT, BACK> p{a, int64_t(tm) * G::BM, int64_t(tf) * (G::BN / 2),
                                int((a.k_pad + G::BK - 1) / G::BK), vec};
    if (half < 0) {
        mm_tile<G>(p, lds);
        return;
    }
    p.m0 += half * H::BM;
    if (p.m0 < a.m) mm_tile<H>(p, lds);
}

// ---- dx = [dg du] [Wg; Wu] -----------------------------------------------------------------

template <int DT>
struct GluDxProb {
    using T = typename MM<DT>::T;
    static constexpr int BK = 8 * MM<DT>::kEpc;
    const GluArgs& a;
    int64_t m0, n0;
    int half;   // k tiles per half
    int tiles;
    int first;  // this part's first k tile
    float* part;  // where this part's sums go; null: dx itself
    bool vec;

    __device__ const char* a_chunk(int row, int k) const
    {
        int64_t r = m0 + row;
        r = r < a.m ? r : a.m - 1;
        return reinterpret_cast<const char*>(static_cast<const T*>(a.dgu) + r * 2 * a.f_pad + k);
    }
    __device__ const char* b_chunk(int col, int k) const
    {
        int64_t c = n0 + col;
        c = c < a.k_pad ? c : a.k_pad - MM<DT>::kEpc;
        return reinterpret_cast<const char*>(static_cast<const T*>(a.wg) + int64_t(k) * a.w_ld + c);
    }
    __device__ int64_t a_off(int t) const
    {
        t += first;
        return t < half ? int64_t(t) * 128 : int64_t(t - half) * 128 + a.f_pad * int64_t(sizeof(T));
    }
    __device__ int64_t b_off(int t) const
    {
        t += first;
        const int64_t second = reinterpret_cast<intptr_t>(a.wu) - reinterpret_cast<intptr_t>(a.wg);
        const int64_t row = int64_t(BK) * a.w_ld * int64_t(sizeof(T));
        return t < half ? t * row : (t - half) * row + second;
    }
    __device__ int valid(int t) const
    {
        t += first;
        return k_left<DT>(a.f, t < half ? t : t - half);
    }

    __device__ const float* a_at(int row, int k) const { return reinterpret_cast<const float*>(a_chunk(row, k)); }
    __device__ const float* b_at(int col, int k) const
    {
        const int64_t c = n0 + col < a.k ? n0 + col : a.k - 1;
        return static_cast<const float*>(a.wg) + int64_t(k) * a.w_ld + c;
    }
    __device__ int64_t a_cols() const { return 0; }
    __device__ int64_t b_cols() const { return a.k - n0; }
    __device__ int64_t a_ld() const { return 0; }
    __device__ int64_t b_ld() const { return a.w_ld; }
    static constexpr bool kSkips = false;

    template <class G>
    __device__ void finish(f32x4 (&acc)[G::FM][G::FN], char*, int wm, int wn, int lane) const
    {
#pragma unroll
        for (int i = 0; i < G::FM; ++i) {
            const int64_t m = m0 + (wm * G::FM + i) * 16 + (lane & 15);
            if (m >= a.m) continue;
#pragma unroll
            for (int j = 0; j < G::FN; ++j) {
                const int64_t n = n0 + (wn * G::FN + j) * 16 + (lane >> 4) * 4;
                const float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
                if (n >= a.k) continue;
                if (part)
                    store4<0>(part + m * a.k + n, a.k - n, a.k % 4 == 0, v);
                else
                    store4<DT>(static_cast<T*>(a.dx) + m * a.k + n, a.k - n, vec, v);
            }
        }
    }
};

// ---- [dWg; dWu] = [dg du]^T x ----------------------------------------------------------------

template <int DT>
struct GluDwProb {
    using T = typename MM<DT>::T;
    static constexpr int BK = 8 * MM<DT>::kEpc;
    const GluArgs& a;
    int64_t m0, n0;  // m0: first column of dgu (of its 2 f_pad), n0: first column of x
    // rows of dgu: the tokens, and the same again for the remainders (all in one k tile)
    int tiles;
    int first;    // this part's first k tile
    float* part;  // where this part's sums go; null: the gradients themselves
    bool vec;

    __device__ const char* a_chunk(int col, int k) const
    {
        int64_t c = m0 + col;
        c = c < 2 * a.f_pad ? c : 2 * a.f_pad - MM<DT>::kEpc;
        return reinterpret_cast<const char*>(static_cast<const T*>(a.dgu) + int64_t(k) * 2 * a.f_pad + c);
    }
    __device__ const char* b_chunk(int col, int k) const
    {
        int64_t c = n0 + col;
        c = c < a.k_pad ? c : a.k_pad - MM<DT>::kEpc;
        const int64_t token = a.lo && k >= a.m ? k - a.m : k;
        return reinterpret_cast<const char*>(static_cast<const T*>(a.x) + token * a.x_ld + c);
    }
    __device__ int64_t a_off(int t) const { return int64_t(t + first) * BK * 2 * a.f_pad * int64_t(sizeof(T)); }
    __device__ int64_t b_off(int t) const { return int64_t(t + first) * BK * a.x_ld * int64_t(sizeof(T)); }
    __device__ int valid(int t) const { return k_left<DT>(a.lo ? 2 * a.m : a.m, t + first); }

    __device__ const float* a_at(int col, int k) const
    {
        const int64_t c = m0 + col < 2 * a.f_pad ? m0 + col : 2 * a.f_pad - 1;
        return static_cast<const float*>(a.dgu) + int64_t(k) * 2 * a.f_pad + c;
    }
    __device__ const float* b_at(int col, int k) const
    {
        const int64_t c = n0 + col < a.k ? n0 + col : a.k - 1;
        return static_cast<const float*>(a.x) + int64_t(k) * a.x_ld + c;
    }
    __device__ int64_t a_cols() const { return 2 * a.f_pad - m0; }
    __device__ int64_t b_cols() const { return a.k - n0; }
    __device__ int64_t a_ld() const { return 2 * a.f_pad; }
    __device__ int64_t b_ld() const { return a.x_ld; }
    static constexpr bool kSkips = false;

    template <class G>
    __device__ void finish(f32x4 (&acc)[G::FM][G::FN], char*, int wm, int wn, int lane) const
    {
#pragma unroll
        for (int i = 0; i < G::FM; ++i) {
            const int64_t c = m0 + (wm * G::FM + i) * 16 + (lane & 15);
            const bool up = c >= a.f_pad;
            const int64_t f = up ? c - a.f_pad : c;
            if (f >= a.f) continue;
            T* const row = static_cast<T*>(up ? a.dwu : a.dwg) + f * a.k;
#pragma unroll
            for (int j = 0; j < G::FN; ++j) {
                const int64_t n = n0 + (wn * G::FN + j) * 16 + (lane >> 4) * 4;
                const float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
                if (n >= a.k) continue;
                if (part)
                    store4<0>(part + c * a.k + n, a.k - n, a.k % 4 == 0, v);
                else
                    store4<DT>(row + n, a.k - n, vec, v);
            }
        }
    }
};

// A part's share of `all` k tiles: the first, and how many (rounding may leave the last parts nothing).
__device__ __forceinline__ void share(int64_t all, int64_t parts, uint32_t part, int* first, int* tiles)
{
    const int64_t depth = (all + parts - 1) / parts, from = part * depth, left = all > from ? all - from : 0;
    *first = int(from);
    *tiles = int(left < depth ? left : depth);
}

// Both sets of tiles: dx's, dx_splits times px, and then dw's, dw_splits times pw.  HX, HW: their halves.
template <class GX, class HX, class GW, class HW>
__global__ __launch_bounds__(GX::NT) void glu_grad_kernel(GluArgs a, TilePlan px, TilePlan pw, bool vec_x, bool vec_w)
{
    static_assert(GX::NT == GW::NT && GX::LDS == GW::LDS, "one launch");
    __shared__ __attribute__((aligned(1024))) char lds[GX::LDS];
    uint32_t tm, tn;
    const uint32_t per_x = px.blocks(), n_dx = per_x * uint32_t(a.dx_splits);
    int first, tiles;
    if (blockIdx.x < n_dx) {
        const uint32_t part = blockIdx.x / per_x;
        const int h = tile_of(blockIdx.x % per_x, px, &tm, &tn);
        const int half = int((a.f + GX::BK - 1) / GX::BK);
        share(2 * half, a.dx_splits, part, &first, &tiles);
        GluDxProb<GX::DT> p{a,     int64_t(tm) * GX::BM, int64_t(tn) * GX::BN, half, tiles,
                            first, a.dx_part ? a.dx_part + int64_t(part) * a.m * a.k : nullptr, vec_x};
        if (h < 0) {
            mm_tile<GX>(p, lds);
            return;
        }
        p.m0 += h * HX::BM;
        if (p.m0 < a.m) mm_tile<HX>(p, lds);
    } else {
        const uint32_t id = blockIdx.x - n_dx, per_w = pw.blocks(), part = id / per_w;
        const int h = tile_of(id % per_w, pw, &tm, &tn);
        share((a.m + GW::BK - 1) / GW::BK, a.dw_splits, part, &first, &tiles);
        GluDwProb<GW::DT> p{a,     int64_t(tm) * GW::BM, int64_t(tn) * GW::BN, tiles,
                            first, a.dw_part ? a.dw_part + int64_t(part) * 2 * a.f_pad * a.k : nullptr, vec_w};
        if (h < 0) {
            mm_tile<GW>(p, lds);
            return;
        }
        p.m0 += h * HW::BM;
        if (p.m0 < 2 * a.f_pad) mm_tile<HW>(p, lds);
    }
}

// The weights' gradients from their parts, in order.
template <int DT>
__global__ __launch_bounds__(256) void glu_dw_sum_kernel(GluArgs a)
{
    using T = typename MM<DT>::T;
    const int64_t n = a.f * a.k, all = 2 * a.f_pad * a.k;
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < 2 * n; i += int64_t(gridDim.x) * 256) {
        const bool up_half = i >= n;
        const int64_t at = up_half ? i - n + a.f_pad * a.k : i;
        float s = 0.0f;
#pragma unroll 8
        for (int64_t p = 0; p < a.dw_splits; ++p) s += a.dw_part[p * all + at];
        static_cast<T*>(up_half ? a.dwu : a.dwg)[up_half ? i - n : i] = MM<DT>::narrow(s);
    }
}

// dx from its parts, in order.
template <int DT>
__global__ __launch_bounds__(256) void glu_dx_sum_kernel(GluArgs a)
{
    const int64_t n = a.m * a.k;
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256) {
        float s = 0.0f;
#pragma unroll 8
        for (int64_t p = 0; p < a.dx_splits; ++p) s += a.dx_part[p * n + i];
        static_cast<typename MM<DT>::T*>(a.dx)[i] = MM<DT>::narrow(s);
    }
}

// ---- few tokens ---------------------------------------------------------------------------------

// 16 features per workgroup: their rows of Wg and of Wu.
template <int DT, int MT, bool ALIGNED, int ACT, bool BACK>
__global__ __launch_bounds__(64 * kStreamWaves) void glu_stream_kernel(GluArgs a, bool vec)
{
    using T = typename MM<DT>::T;
    const int lane = threadIdx.x & 63;
    const int64_t f0 = int64_t(blockIdx.x) * 16;
    int64_t fr = f0 + (lane & 15);
    fr = fr < a.f ? fr : a.f - 1;
    const T* px[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        int64_t m = i * 16 + (lane & 15);
        m = m < a.m ? m : a.m - 1;
        px[i] = static_cast<const T*>(a.x_raw) + m * a.x_raw_ld;
    }
    f32x4 g[MT], u[MT];
    stream_rows<DT, MT, ALIGNED>(static_cast<const T*>(a.wg_raw) + fr * a.k, static_cast<const T*>(a.wu_raw) + fr * a.k,
                                 px, a.k, g, u);
    stream_join<MT>(g, u, [&](int i, f32x4 gs, f32x4 us) {
        const int64_t m = i * 16 + (lane & 15);
        if (m < a.m) glu_emit<DT, ACT, BACK>(a, m, f0 + (lane >> 4) * 4, gs, us, vec);
    });
}

// ---- padded copy ------------------------------------------------------------------------------

// One 16-byte chunk of a padded row per thread.
template <int DT>
__global__ __launch_bounds__(256) void pad_rows_kernel(const typename MM<DT>::T* src, int64_t ld,
                                                       typename MM<DT>::T* dst, int64_t rows, int64_t cols,
                                                       int64_t chunks)
{
    constexpr int E = MM<DT>::kEpc;
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < rows * chunks; i += int64_t(gridDim.x) * 256) {
        const int64_t r = i / chunks, c = (i - r * chunks) * E;
        const typename MM<DT>::T* p = src + r * ld + c;
        *reinterpret_cast<typename Stream<DT>::Frag*>(dst + i * E) =
            c + E <= cols ? stream_load<DT, false>(p) : stream_tail<DT>(p, cols - c);
    }
}

// ---- launches -----------------------------------------------------------------------------------

template <class G, class H, int ACT, bool BACK>
hipError_t launch_glu_tile(const GluArgs& a, bool vec, hipStream_t s)
{
    const TilePlan plan = plan_tiles(up(a.m, G::BM), up(BACK ? a.f_pad : a.f, G::BN / 2), H::BM < G::BM);
    glu_tile_kernel<G, H, ACT, BACK><<<dim3(plan.blocks()), dim3(G::NT), 0, s>>>(a, plan, vec);
    return hipGetLastError();
}

template <int DT, int ACT, bool BACK>
hipError_t launch_glu_gu(const GluArgs& a, bool vec, hipStream_t s)
{
    const int64_t f = 2 * a.f;  // tile columns: f of Wg and f of Wu
    const Tile t = best_tile<DT>(count(a.m, f, 256, 256), count(a.m, f, 128, 128), count(a.m, f, 64, 128));
    if constexpr (DT == 1) {
        if (t == Tile::Large)
            return launch_glu_tile<LargeTile<false, false>, HalfTile<false, false>, ACT, BACK>(a, vec, s);
    }
    using S = typename Tiles<DT>::template Small<false, false>;
    using M = typename Tiles<DT>::template Mini<false, false>;
    return t == Tile::Mini ? launch_glu_tile<M, M, ACT, BACK>(a, vec, s) : launch_glu_tile<S, S, ACT, BACK>(a, vec, s);
}

template <int DT, int MT, bool BACK>
hipError_t launch_glu_stream_mt(const GluArgs& a, bool vec, hipStream_t s)
{
    const dim3 grid(up(BACK ? a.f_pad : a.f, 16)), block(64 * kStreamWaves);
    if (a.act == kActSilu) {
        if (a.aligned)
            glu_stream_kernel<DT, MT, true, kActSilu, BACK><<<grid, block, 0, s>>>(a, vec);
        else
            glu_stream_kernel<DT, MT, false, kActSilu, BACK><<<grid, block, 0, s>>>(a, vec);
    } else {
        if (a.aligned)
            glu_stream_kernel<DT, MT, true, kActGelu, BACK><<<grid, block, 0, s>>>(a, vec);
        else
            glu_stream_kernel<DT, MT, false, kActGelu, BACK><<<grid, block, 0, s>>>(a, vec);
    }
    return hipGetLastError();
}

template <int DT, bool BACK>
hipError_t launch_glu_stream(const GluArgs& a, bool vec, hipStream_t s)
{
    if (a.m <= 16) return launch_glu_stream_mt<DT, 1, BACK>(a, vec, s);
    if (a.m <= 32) return launch_glu_stream_mt<DT, 2, BACK>(a, vec, s);
    return launch_glu_stream_mt<DT, 4, BACK>(a, vec, s);
}

bool vec_rows(const void* p, int64_t row, int dtype)
{
    return row % 4 == 0 && reinterpret_cast<uintptr_t>(p) % (dtype == 0 ? 16 : 8) == 0;
}

template <int DT>
hipError_t glu_fwd_dt(const GluArgs& a, hipStream_t s)
{
    const bool vec = vec_rows(a.h, a.f, DT);
    if (a.stream) return launch_glu_stream<DT, false>(a, vec, s);
    return a.act == kActSilu ? launch_glu_gu<DT, kActSilu, false>(a, vec, s)
                             : launch_glu_gu<DT, kActGelu, false>(a, vec, s);
}

template <class GX, class HX, class GW, class HW>
hipError_t launch_glu_grad(const GluArgs& a, hipStream_t s)
{
    const bool can = HX::BM < GX::BM;
    const uint32_t sx = uint32_t(a.dx_splits), sw = uint32_t(a.dw_splits);
    TilePlan px{0, 0, 0, 0}, pw{0, 0, 0, 0};
    // only the last tiles of a launch are halved
    if (a.dx) px = plan_tiles(up(a.m, GX::BM), up(a.k, GX::BN), can && !a.dwg && sx == 1);
    if (a.dwg) pw = plan_tiles(up(2 * a.f_pad, GW::BM), up(a.k, GW::BN), can && sw == 1, px.whole * sx);
    const bool vx = vec_rows(a.dx, a.k, GX::DT), vw = vec_rows(a.dwg, a.k, GX::DT) && vec_rows(a.dwu, a.k, GX::DT);
    glu_grad_kernel<GX, HX, GW, HW><<<dim3(px.blocks() * sx + pw.blocks() * sw), dim3(GX::NT), 0, s>>>(a, px, pw, vx, vw);
    hipError_t e = hipGetLastError();
    auto blocks = [](int64_t n) { return dim3(unsigned(n / 256 + 1 < 4096 ? n / 256 + 1 : 4096)); };
    if (e == hipSuccess && a.dx && sx > 1) {
        glu_dx_sum_kernel<GX::DT><<<blocks(a.m * a.k), dim3(256), 0, s>>>(a);
        e = hipGetLastError();
    }
    if (e == hipSuccess && a.dwg && sw > 1) {
        glu_dw_sum_kernel<GX::DT><<<blocks(2 * a.f * a.k), dim3(256), 0, s>>>(a);
        e = hipGetLastError();
    }
    return e;
}

template <int DT>
hipError_t glu_bwd_dt(const GluArgs& a, hipStream_t s)
{
    const bool vec = vec_rows(a.dh, a.f, DT);
    const hipError_t e = a.stream ? launch_glu_stream<DT, true>(a, vec, s)
                         : a.act == kActSilu ? launch_glu_gu<DT, kActSilu, true>(a, vec, s)
                                             : launch_glu_gu<DT, kActGelu, true>(a, vec, s);
    if (e != hipSuccess) return e;
    if (a.few)
        return launch_few_grad({static_cast<const float*>(a.dgu), 2 * a.f_pad, a.f_pad, a.wg_raw, a.wu_raw, a.dwg, a.dwu,
                                a.x_raw, a.x_raw_ld, a.dx_part, a.dx, a.f, 2 * a.f, a.m, a.k, a.dx_per, a.dx_splits, nullptr, 0},
                               DT, s);
    auto tiles = [&](int bm, int bn) {
        return (a.dx ? count(a.m, a.k, bm, bn) * a.dx_splits : 0) + (a.dwg ? count(2 * a.f_pad, a.k, bm, bn) * a.dw_splits : 0);
    };
    const Tile t = best_tile<DT>(tiles(256, 256), tiles(128, 128), tiles(64, 128));
    if constexpr (DT == 1) {
        if (t == Tile::Large)
            return launch_glu_grad<LargeTile<false, true>, HalfTile<false, true>, LargeTile<true, true>,
                                   HalfTile<true, true>>(a, s);
    }
    using T = Tiles<DT>;
    using SX = typename T::template Small<false, true>;
    using SW = typename T::template Small<true, true>;
    using MX = typename T::template Mini<false, true>;
    using MW = typename T::template Mini<true, true>;
    return t == Tile::Mini ? launch_glu_grad<MX, MX, MW, MW>(a, s) : launch_glu_grad<SX, SX, SW, SW>(a, s);
}

}  // namespace

hipError_t launch_pad_rows(const void* src, int64_t ld, void* dst, int64_t rows, int64_t cols, int64_t cols_pad,
                           int dtype, hipStream_t stream)
{
    (void)hipGetLastError();
    const int64_t chunks = cols_pad / (dtype == 0 ? MM<0>::kEpc : MM<1>::kEpc);
    const int64_t blocks = (rows * chunks + 255) / 256;
    const dim3 grid(unsigned(blocks < 16384 ? blocks : 16384));
    if (dtype == 0)
        pad_rows_kernel<0><<<grid, dim3(256), 0, stream>>>(static_cast<const float*>(src), ld, static_cast<float*>(dst),
                                                          rows, cols, chunks);
    else
        pad_rows_kernel<1><<<grid, dim3(256), 0, stream>>>(static_cast<const __bf16*>(src), ld,
                                                          static_cast<__bf16*>(dst), rows, cols, chunks);
    return hipGetLastError();
}

hipError_t launch_glu_fwd(const GluArgs& a, int dtype, hipStream_t stream)
{
    (void)hipGetLastError();
    return dtype == 0 ? glu_fwd_dt<0>(a, stream) : glu_fwd_dt<1>(a, stream);
}

hipError_t launch_glu_bwd(const GluArgs& a, int dtype, hipStream_t stream)
{
    (void)hipGetLastError();
    return dtype == 0 ? glu_bwd_dt<0>(a, stream) : glu_bwd_dt<1>(a, stream);
}

}  // namespace ssk
