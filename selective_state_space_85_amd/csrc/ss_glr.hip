// gfx950 kernels of the gated linear recurrence, per batch row and channel
//   k = c softplus(decay),  a_t = exp(-k sigmoid(r_t))  (0 where reset_t),
//   h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t,  y_t = h_t,
// its backward pass and its single-token form.
//
// The update is an affine map h -> a h + b, and maps compose: (a1, b1) then (a2, b2) is
// (a2 a1, a2 b1 + b2).  A workgroup of 8 waves takes 32 VC channels (VC neighbouring ones per
// lane) and walks its rows in tiles of 16 R: each half wave holds a run of R rows, forms their
// a and b in registers, and its run's composed map; the two halves of a wave are joined by a
// lane exchange, the 8 waves through LDS, and every run then replays its rows from the state
// that enters it.  So the operands are read once and y is written once: the kernel is bound
// by HBM traffic (bf16: 8 bytes per element), with the next tile's loads in flight while a
// tile is worked on.
//
// With few (batch row, channel block) pairs the rows are split in chunks: a first pass forms
// each chunk's composed map, and the second pass starts every chunk from the maps before it.
//
// Backward.  g_t = dL/dh_t = dy_t + a_{t+1} g_{t+1}: the same maps from the end.  Run q_t = a_t g_t
// backward: q -> a (q + dy), so a run's product of a serves both directions.  The states
// h_{t-1} are rebuilt from those kept every 64 rows.
//
// 1 - a^2 = -expm1(-2 k s) is formed without cancellation: as a gate closes a tends to 1 and
// the plain difference would lose every digit.
#include "ss_device.h"
#include "ss_lm_internal.h"

namespace ssk {
namespace {

constexpr int kRunLanes = 32;               // lanes per run: half a wave
constexpr int kGlrWaves = 8;
constexpr int kRuns = 2 * kGlrWaves;        // runs per tile
constexpr int kGlrThreads = 64 * kGlrWaves;
constexpr int kFwdRows = 8, kBwdRows = 4;   // rows per run
static_assert(kRuns * kFwdRows == kGlrChunkUnit && kRuns * kBwdRows == kGlrRows, "tiles and kept states");
static_assert(kGlrRows % kFwdRows == 0, "a kept state falls on a run's start");

// VC neighbouring elements of a row as loaded
template <int DT, int VC>
struct Row;
template <>
struct Row<1, 2> {
    using Raw = uint32_t;
    static __device__ __forceinline__ float get(Raw v, int e)
    {
        return __uint_as_float(e == 0 ? v << 16 : v & 0xffff0000u);
    }
    static __device__ __forceinline__ Raw make(const float (&v)[2])
    {
        return uint32_t(f32_to_bf16_bits(v[0])) | (uint32_t(f32_to_bf16_bits(v[1])) << 16);
    }
};
template <>
struct Row<1, 1> {
    using Raw = uint16_t;
    static __device__ __forceinline__ float get(Raw v, int) { return bf16_bits_to_f32(v); }
    static __device__ __forceinline__ Raw make(const float (&v)[1]) { return f32_to_bf16_bits(v[0]); }
};
template <>
struct Row<0, 2> {
    using Raw = float2;
    static __device__ __forceinline__ float get(Raw v, int e) { return e == 0 ? v.x : v.y; }
    static __device__ __forceinline__ Raw make(const float (&v)[2]) { return make_float2(v[0], v[1]); }
};
template <>
struct Row<0, 1> {
    using Raw = float;
    static __device__ __forceinline__ float get(Raw v, int) { return v; }
    static __device__ __forceinline__ Raw make(const float (&v)[1]) { return v[0]; }
};

template <int DT>
constexpr int64_t elem_bytes = DT == 0 ? 4 : 2;

template <int DT, int VC>
__device__ __forceinline__ typename Row<DT, VC>::Raw load_row(const void* base, int64_t elem)
{
    return *reinterpret_cast<const typename Row<DT, VC>::Raw*>(static_cast<const char*>(base) + elem * elem_bytes<DT>);
}
template <int DT, int VC>
__device__ __forceinline__ void store_row(void* base, int64_t elem, const float (&v)[VC])
{
    *reinterpret_cast<typename Row<DT, VC>::Raw*>(static_cast<char*>(base) + elem * elem_bytes<DT>) =
        Row<DT, VC>::make(v);
}

// sigmoid(v) and 1 - sigmoid(v), both to full relative precision.  The exponent is held below
// 2^126 so that e stays finite and e s tends to 1.
__device__ __forceinline__ float sigmoid2(float v, float* rest)
{
    const float e = exp2_hw(fminf(-v * kLog2e, 126.0f));
    const float s = __builtin_amdgcn_rcpf(1.0f + e);
    *rest = e * s;
    return s;
}

// a = exp(-k s) and m = sqrt(1 - a^2).  Below t = 2 k s = 1/2 the series of 1 - e^-t to t^7
// (truncation t^7/8! < 2e-7 relative), above it 1 - a^2 itself (a^2 < 0.61: no cancellation).
__device__ __forceinline__ void decay_of(float k, float s, float* a, float* m)
{
    const float ks = k * s;
    *a = exp2_hw(-ks * kLog2e);
    const float t = ks + ks;
    float p = fmaf(t, 1.0f / 5040.0f, -1.0f / 720.0f);
    p = fmaf(t, p, 1.0f / 120.0f);
    p = fmaf(t, p, -1.0f / 24.0f);
    p = fmaf(t, p, 1.0f / 6.0f);
    p = fmaf(t, p, -0.5f);
    const float small = fmaf(t * t, p, t);
    *m = __builtin_amdgcn_sqrtf(t < 0.5f ? small : fmaf(-*a, *a, 1.0f));
}

__device__ __forceinline__ float channel_rate(float decay, float c)
{
    return c * (fmaxf(decay, 0.0f) + log1pf(expf(-fabsf(decay))));
}

// a h + b, the update and the composition of maps.  With resets a product of 0 means that
// nothing of h remains, not even a NaN or an infinity (0 times which would be NaN).
template <bool RESET>
__device__ __forceinline__ float carry(float a, float h, float b)
{
    const float v = fmaf(a, h, b);
    return RESET && a == 0.0f ? b : v;
}

// The other half wave's value.
__device__ __forceinline__ float other_half(float v) { return __shfl_xor(v, 32); }

// What a workgroup works on.
template <int VC>
struct Place {
    int64_t b, c, d;   // batch row, chunk, first channel of this lane
    int64_t t0, t1;    // the chunk's rows
    int64_t dc;        // d clamped to a channel that exists: loads stay inside
    bool live;
    __device__ Place(const GlrArgs& a)
    {
        const int64_t cols = (a.dim + kRunLanes * VC - 1) / (kRunLanes * VC);
        const int64_t id = blockIdx.x;
        const int64_t rest = id / cols;
        d = (id % cols) * (kRunLanes * VC) + (threadIdx.x & 31) * VC;
        b = rest % a.batch;
        c = rest / a.batch;
        live = d < a.dim;
        dc = live ? d : 0;
        t0 = c * a.chunk_len;
        t1 = t0 + a.chunk_len < a.seqlen ? t0 + a.chunk_len : a.seqlen;
    }
};

// ---- forward -------------------------------------------------------------------------------

// AGG: only each chunk's composed map (ws_prod, ws_end)
template <int DT, int VC, bool RESET, bool AGG>
__global__ __launch_bounds__(kGlrThreads, 4) void glr_fwd_kernel(GlrArgs a)
{
    constexpr int R = kFwdRows, T = kRuns * R;
    using RW = Row<DT, VC>;
    using Raw = typename RW::Raw;
    const Place<VC> w(a);
    const int wave = threadIdx.x >> 6, half = (threadIdx.x >> 5) & 1, run = wave * 2 + half;
    const int64_t bd = w.b * a.dim + w.dc;

    float k[VC], h[VC], prod[VC];
#pragma unroll
    for (int e = 0; e < VC; ++e) {
        k[e] = channel_rate(a.decay[w.dc + e], a.c);
        h[e] = AGG || !a.h0 ? 0.0f : a.h0[bd + e];
        prod[e] = 1.0f;
    }
    if (!AGG) {
        for (int64_t c = 0; c < w.c; ++c)
#pragma unroll
            for (int e = 0; e < VC; ++e) {
                const int64_t at = c * a.batch * a.dim + bd + e;
                h[e] = carry<RESET>(a.ws_prod[at], h[e], a.ws_end[at]);
            }
    }

    __shared__ float maps[2][kGlrWaves][2 * VC][kRunLanes];
    Raw rx[R], rr[R], ri[R];
    uint8_t rs[R];
    auto load = [&](int64_t tile) {
        const int64_t first = tile + run * R;
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const int64_t t = first + q < a.seqlen ? first + q : a.seqlen - 1;
            const int64_t row = w.b * a.seqlen + t;
            rr[q] = load_row<DT, VC>(a.r, row * a.r_ld + w.dc);
            ri[q] = load_row<DT, VC>(a.i, row * a.i_ld + w.dc);
            rx[q] = load_row<DT, VC>(a.x, row * a.x_ld + w.dc);
            if (RESET) rs[q] = a.reset[row];
        }
    };
    load(w.t0);
    int buf = 0;
    for (int64_t tile = w.t0; tile < w.t1; tile += T, buf ^= 1) {
        const int64_t first = tile + run * R;
        float av[R][VC], bv[R][VC], P[VC], E[VC];
#pragma unroll
        for (int e = 0; e < VC; ++e) {
            P[e] = 1.0f;
            E[e] = 0.0f;
        }
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const bool in = first + q < w.t1;
#pragma unroll
            for (int e = 0; e < VC; ++e) {
                float rest, m;
                const float sr = sigmoid2(RW::get(rr[q], e), &rest);
                const float si = sigmoid2(RW::get(ri[q], e), &rest);
                decay_of(k[e], sr, &av[q][e], &m);
                if (RESET && rs[q]) {
                    av[q][e] = 0.0f;
                    m = 1.0f;
                }
                bv[q][e] = m * si * RW::get(rx[q], e);
                // rows past the end leave the state as it is
                av[q][e] = in ? av[q][e] : 1.0f;
                bv[q][e] = in ? bv[q][e] : 0.0f;
                P[e] *= av[q][e];
                E[e] = carry<RESET>(av[q][e], E[e], bv[q][e]);
            }
        }
        if (tile + T < w.t1) load(tile + T);
        // join the halves of the wave; the earlier half publishes the wave's map
        float P0[VC], E0[VC];
#pragma unroll
        for (int e = 0; e < VC; ++e) {
            P0[e] = other_half(P[e]);
            E0[e] = other_half(E[e]);
            if (half == 0) {
                maps[buf][wave][2 * e][threadIdx.x & 31] = P0[e] * P[e];
                maps[buf][wave][2 * e + 1][threadIdx.x & 31] = carry<RESET>(P0[e], E[e], E0[e]);
            }
        }
        __syncthreads();
        float in[VC];
#pragma unroll
        for (int v = 0; v < kGlrWaves; ++v) {
#pragma unroll
            for (int e = 0; e < VC; ++e) {
                if (v == wave) in[e] = h[e];
                const float p = maps[buf][v][2 * e][threadIdx.x & 31];
                h[e] = carry<RESET>(p, h[e], maps[buf][v][2 * e + 1][threadIdx.x & 31]);
                if (AGG) prod[e] *= p;
            }
        }
        if (!AGG) {
#pragma unroll
            for (int e = 0; e < VC; ++e)
                if (half == 1) in[e] = carry<RESET>(P0[e], in[e], E0[e]);
            if (a.ckpt && w.live && first % kGlrRows == 0 && first < w.t1) {
                const int64_t at = (first / kGlrRows) * a.batch * a.dim + bd;
#pragma unroll
                for (int e = 0; e < VC; ++e) a.ckpt[at + e] = in[e];
            }
            if (a.y && w.live) {
#pragma unroll
                for (int q = 0; q < R; ++q) {
#pragma unroll
                    for (int e = 0; e < VC; ++e) in[e] = carry<RESET>(av[q][e], in[e], bv[q][e]);
                    if (first + q < w.t1) store_row<DT, VC>(a.y, (w.b * a.seqlen + first + q) * a.dim + w.d, in);
                }
            }
        }
    }
    if (run != 0 || !w.live) return;
#pragma unroll
    for (int e = 0; e < VC; ++e) {
        if (AGG) {
            const int64_t at = w.c * a.batch * a.dim + bd + e;
            a.ws_prod[at] = prod[e];
            a.ws_end[at] = h[e];
        } else if (a.h_last && w.c == a.n_chunks - 1) {
            a.h_last[bd + e] = h[e];
        }
    }
}

// ---- backward ------------------------------------------------------------------------------

// AGG: only each chunk's composed map of q, from r and dy (ws_prod, ws_end)
template <int DT, int VC, bool RESET, bool AGG>
__global__ __launch_bounds__(kGlrThreads, 4) void glr_bwd_kernel(GlrArgs a)
{
    constexpr int R = kBwdRows, T = kRuns * R;
    using RW = Row<DT, VC>;
    using Raw = typename RW::Raw;
    const Place<VC> w(a);
    const int wave = threadIdx.x >> 6, half = (threadIdx.x >> 5) & 1, run = wave * 2 + half;
    const int l32 = threadIdx.x & 31;
    const int64_t bd = w.b * a.dim + w.dc;

    float k[VC], q[VC], prod[VC], dk[VC];
#pragma unroll
    for (int e = 0; e < VC; ++e) {
        k[e] = channel_rate(a.decay[w.dc + e], a.c);
        q[e] = AGG || !a.dh_last ? 0.0f : a.dh_last[bd + e];
        prod[e] = 1.0f;
        dk[e] = 0.0f;
    }
    if (!AGG) {
        for (int64_t c = a.n_chunks - 1; c > w.c; --c)
#pragma unroll
            for (int e = 0; e < VC; ++e) {
                const int64_t at = c * a.batch * a.dim + bd + e;
                q[e] = carry<RESET>(a.ws_prod[at], q[e], a.ws_end[at]);
            }
    }

    __shared__ float maps[2][kGlrWaves][3 * VC][kRunLanes];
    Raw rx[R], rr[R], ri[R], rd[R];
    uint8_t rs[R];
    float kept[VC];
    auto load = [&](int64_t tile) {
        const int64_t first = tile + run * R;
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const int64_t t = first + j < a.seqlen ? first + j : a.seqlen - 1;
            const int64_t row = w.b * a.seqlen + t;
            rr[j] = load_row<DT, VC>(a.r, row * a.r_ld + w.dc);
            rd[j] = load_row<DT, VC>(a.dy, row * a.dim + w.dc);
            if (!AGG) {
                ri[j] = load_row<DT, VC>(a.i, row * a.i_ld + w.dc);
                rx[j] = load_row<DT, VC>(a.x, row * a.x_ld + w.dc);
            }
            if (RESET) rs[j] = a.reset[row];
        }
        if (!AGG) {
            const int64_t at = (tile / kGlrRows) * a.batch * a.dim + bd;
#pragma unroll
            for (int e = 0; e < VC; ++e) kept[e] = a.ckpt[at + e];
        }
    };
    const int64_t last = w.t0 + (w.t1 - w.t0 - 1) / T * T;
    load(last);
    int buf = 0;
    for (int64_t tile = last; tile >= w.t0; tile -= T, buf ^= 1) {
        const int64_t first = tile + run * R;
        float av[R][VC], m[R][VC], sr[R][VC], nr[R][VC], si[R][VC], ni[R][VC], x[R][VC], dy[R][VC], h[VC];
        float P[VC], E[VC], Q[VC];
#pragma unroll
        for (int e = 0; e < VC; ++e) {
            P[e] = 1.0f;
            E[e] = Q[e] = 0.0f;
            h[e] = kept[e];
        }
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const bool in = first + j < w.t1;
#pragma unroll
            for (int e = 0; e < VC; ++e) {
                sr[j][e] = sigmoid2(RW::get(rr[j], e), &nr[j][e]);
                decay_of(k[e], sr[j][e], &av[j][e], &m[j][e]);
                if (RESET && rs[j]) {
                    av[j][e] = 0.0f;
                    m[j][e] = 1.0f;
                }
                dy[j][e] = in ? RW::get(rd[j], e) : 0.0f;
                av[j][e] = in ? av[j][e] : 1.0f;
                if (!AGG) {
                    si[j][e] = sigmoid2(RW::get(ri[j], e), &ni[j][e]);
                    x[j][e] = in ? RW::get(rx[j], e) : 0.0f;
                    E[e] = carry<RESET>(av[j][e], E[e], m[j][e] * si[j][e] * x[j][e]);
                }
                P[e] *= av[j][e];
            }
        }
#pragma unroll
        for (int j = R - 1; j >= 0; --j)
#pragma unroll
            for (int e = 0; e < VC; ++e) Q[e] = carry<RESET>(av[j][e], Q[e] + dy[j][e], 0.0f);
        if (tile > w.t0) load(tile - T);

        float Po[VC], Eo[VC], Qo[VC];  // the other half's
#pragma unroll
        for (int e = 0; e < VC; ++e) {
            Po[e] = other_half(P[e]);
            Qo[e] = other_half(Q[e]);
            if (!AGG) Eo[e] = other_half(E[e]);
            if (half == 0) {
                maps[buf][wave][3 * e][l32] = Po[e] * P[e];
                maps[buf][wave][3 * e + 1][l32] = carry<RESET>(P[e], Qo[e], Q[e]);
                if (!AGG) maps[buf][wave][3 * e + 2][l32] = carry<RESET>(Po[e], E[e], Eo[e]);
            }
        }
        __syncthreads();
        float hin[VC], qin[VC];
        if (!AGG) {
#pragma unroll
            for (int v = 0; v < kGlrWaves - 1; ++v)
#pragma unroll
                for (int e = 0; e < VC; ++e)
                    if (v < wave) h[e] = carry<RESET>(maps[buf][v][3 * e][l32], h[e], maps[buf][v][3 * e + 2][l32]);
#pragma unroll
            for (int e = 0; e < VC; ++e) hin[e] = half == 1 ? carry<RESET>(Po[e], h[e], Eo[e]) : h[e];
        }
#pragma unroll
        for (int v = kGlrWaves - 1; v >= 0; --v)
#pragma unroll
            for (int e = 0; e < VC; ++e) {
                if (v == wave) qin[e] = q[e];
                const float p = maps[buf][v][3 * e][l32];
                q[e] = carry<RESET>(p, q[e], maps[buf][v][3 * e + 1][l32]);
                if (AGG) prod[e] *= p;
            }
        if (!AGG) {
            float before[R][VC];  // h_{t-1}
#pragma unroll
            for (int j = 0; j < R; ++j)
#pragma unroll
                for (int e = 0; e < VC; ++e) {
                    before[j][e] = hin[e];
                    hin[e] = carry<RESET>(av[j][e], hin[e], m[j][e] * si[j][e] * x[j][e]);
                }
#pragma unroll
            for (int e = 0; e < VC; ++e)
                if (half == 0) qin[e] = carry<RESET>(Po[e], qin[e], Qo[e]);
#pragma unroll
            for (int j = R - 1; j >= 0; --j) {
                float dx[VC], dr[VC], di[VC];
#pragma unroll
                for (int e = 0; e < VC; ++e) {
                    const float g = qin[e] + dy[j][e];
                    const float gm = g * m[j][e], gms = gm * si[j][e];
                    dx[e] = gms;
                    di[e] = gms * x[j][e] * ni[j][e];
                    // d m / d log a = -a^2 / m; where a rounds to 1 (s so small that m is 0)
                    // its product with ds/dr vanishes
                    const float im = m[j][e] > 0.0f ? __builtin_amdgcn_rcpf(m[j][e]) : 0.0f;
                    const float ga = carry<RESET>(av[j][e], g, 0.0f);
                    const float dm = ga * av[j][e] * im * si[j][e] * x[j][e];
                    const float dla = carry<RESET>(av[j][e], g * before[j][e], 0.0f) - (RESET && av[j][e] == 0.0f ? 0.0f : dm);
                    const float dls = dla * sr[j][e];
                    dr[e] = -k[e] * dls * nr[j][e];
                    if (first + j < w.t1) dk[e] += dls;
                    qin[e] = ga;
                }
                if (w.live && first + j < w.t1) {
                    const int64_t at = (w.b * a.seqlen + first + j) * a.g_ld + w.d;
                    store_row<DT, VC>(a.dx, at, dx);
                    store_row<DT, VC>(a.dr, at, dr);
                    store_row<DT, VC>(a.di, at, di);
                }
            }
        }
    }
    if (AGG) {
        if (run == 0 && w.live)
#pragma unroll
            for (int e = 0; e < VC; ++e) {
                const int64_t at = w.c * a.batch * a.dim + bd + e;
                a.ws_prod[at] = prod[e];
                a.ws_end[at] = q[e];
            }
        return;
    }
    // the runs' sums over their rows, joined in a fixed order
    __syncthreads();
    float* const sums = &maps[0][0][0][0];
    static_assert(kRuns * VC <= 2 * kGlrWaves * 3 * VC, "fits the maps' space");
#pragma unroll
    for (int e = 0; e < VC; ++e) sums[(run * VC + e) * kRunLanes + l32] = dk[e];
    __syncthreads();
    if (run != 0 || !w.live) return;
#pragma unroll
    for (int e = 0; e < VC; ++e) {
        float s = 0.0f;
        for (int v = 0; v < kRuns; ++v) s += sums[(v * VC + e) * kRunLanes + l32];
        a.part_decay[w.c * a.batch * a.dim + bd + e] = s;
        if (a.dh0 && w.c == 0) a.dh0[bd + e] = q[e];
    }
}

// ddecay = -c sigmoid(decay) sum of the parts: one channel per thread, in a fixed order
__global__ __launch_bounds__(64) void glr_decay_kernel(GlrArgs a)
{
    const int64_t d = int64_t(blockIdx.x) * 64 + threadIdx.x;
    if (d >= a.dim) return;
    float s = 0.0f;
    for (int64_t j = 0; j < a.n_chunks * a.batch; ++j) s += a.part_decay[j * a.dim + d];
    float rest;
    a.ddecay[d] = -a.c * sigmoid2(a.decay[d], &rest) * s;
}

// ---- one token ------------------------------------------------------------------------------

template <int DT, int VC>
__global__ __launch_bounds__(256) void glr_step_kernel(GlrStepArgs a)
{
    using RW = Row<DT, VC>;
    const int64_t d = (int64_t(blockIdx.x) * 256 + threadIdx.x) * VC;
    if (d >= a.dim) return;
    float k[VC];
#pragma unroll
    for (int e = 0; e < VC; ++e) k[e] = channel_rate(a.decay[d + e], a.c);
    for (int64_t b = blockIdx.y; b < a.batch; b += gridDim.y) {
        const auto rr = load_row<DT, VC>(a.r, b * a.r_ld + d);
        const auto ri = load_row<DT, VC>(a.i, b * a.i_ld + d);
        const auto rx = load_row<DT, VC>(a.x, b * a.x_ld + d);
        float h[VC];
#pragma unroll
        for (int e = 0; e < VC; ++e) {
            float rest, av, m;
            const float sr = sigmoid2(RW::get(rr, e), &rest);
            const float si = sigmoid2(RW::get(ri, e), &rest);
            decay_of(k[e], sr, &av, &m);
            h[e] = fmaf(av, a.h[b * a.dim + d + e], m * si * RW::get(rx, e));
            a.h[b * a.dim + d + e] = h[e];
        }
        store_row<DT, VC>(a.y, b * a.dim + d, h);
    }
}

// ---- launches ---------------------------------------------------------------------------------

// Two channels per lane need every row of every operand aligned to two elements.
bool even(const void* p, int64_t ld, int dtype)
{
    return p == nullptr || (ld % 2 == 0 && reinterpret_cast<uintptr_t>(p) % (dtype == 0 ? 8 : 4) == 0);
}

template <int DT, int VC, bool RESET>
hipError_t fwd_variant(const GlrArgs& a, hipStream_t s)
{
    const int64_t cols = (a.dim + kRunLanes * VC - 1) / (kRunLanes * VC);
    const int64_t blocks = cols * a.batch * a.n_chunks;
    if (a.n_chunks > 1) {
        // the last chunk's map leads nowhere
        glr_fwd_kernel<DT, VC, RESET, true><<<dim3(unsigned(blocks - cols * a.batch)), dim3(kGlrThreads), 0, s>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    glr_fwd_kernel<DT, VC, RESET, false><<<dim3(unsigned(blocks)), dim3(kGlrThreads), 0, s>>>(a);
    return hipGetLastError();
}

template <int DT, int VC, bool RESET>
hipError_t bwd_variant(const GlrArgs& a, hipStream_t s)
{
    const int64_t cols = (a.dim + kRunLanes * VC - 1) / (kRunLanes * VC);
    const int64_t blocks = cols * a.batch * a.n_chunks;
    if (a.n_chunks > 1) {
        glr_bwd_kernel<DT, VC, RESET, true><<<dim3(unsigned(blocks)), dim3(kGlrThreads), 0, s>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    glr_bwd_kernel<DT, VC, RESET, false><<<dim3(unsigned(blocks)), dim3(kGlrThreads), 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    glr_decay_kernel<<<dim3(unsigned((a.dim + 63) / 64)), dim3(64), 0, s>>>(a);
    return hipGetLastError();
}

template <int DT>
hipError_t fwd_dt(const GlrArgs& a, hipStream_t s)
{
    const bool two = a.dim % 2 == 0 && even(a.x, a.x_ld, DT) && even(a.r, a.r_ld, DT) && even(a.i, a.i_ld, DT) &&
                     even(a.y, a.dim, DT);
    if (a.reset) return two ? fwd_variant<DT, 2, true>(a, s) : fwd_variant<DT, 1, true>(a, s);
    return two ? fwd_variant<DT, 2, false>(a, s) : fwd_variant<DT, 1, false>(a, s);
}

template <int DT>
hipError_t bwd_dt(const GlrArgs& a, hipStream_t s)
{
    const bool two = a.dim % 2 == 0 && even(a.x, a.x_ld, DT) && even(a.r, a.r_ld, DT) && even(a.i, a.i_ld, DT) &&
                     even(a.dy, a.dim, DT) && even(a.dx, a.g_ld, DT) && even(a.dr, a.g_ld, DT) &&
                     even(a.di, a.g_ld, DT);
    if (a.reset) return two ? bwd_variant<DT, 2, true>(a, s) : bwd_variant<DT, 1, true>(a, s);
    return two ? bwd_variant<DT, 2, false>(a, s) : bwd_variant<DT, 1, false>(a, s);
}

template <int DT>
hipError_t step_dt(const GlrStepArgs& a, hipStream_t s)
{
    const bool two = a.dim % 2 == 0 && even(a.x, a.x_ld, DT) && even(a.r, a.r_ld, DT) && even(a.i, a.i_ld, DT) &&
                     even(a.y, a.dim, DT);
    const unsigned rows = unsigned(a.batch < 65535 ? a.batch : 65535);
    if (two)
        glr_step_kernel<DT, 2><<<dim3(unsigned((a.dim + 511) / 512), rows), dim3(256), 0, s>>>(a);
    else
        glr_step_kernel<DT, 1><<<dim3(unsigned((a.dim + 255) / 256), rows), dim3(256), 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_glr_fwd(const GlrArgs& a, int dtype, hipStream_t stream)
{
    (void)hipGetLastError();
    return dtype == 0 ? fwd_dt<0>(a, stream) : fwd_dt<1>(a, stream);
}

hipError_t launch_glr_bwd(const GlrArgs& a, int dtype, hipStream_t stream)
{
    (void)hipGetLastError();
    return dtype == 0 ? bwd_dt<0>(a, stream) : bwd_dt<1>(a, stream);
}

hipError_t launch_glr_step(const GlrStepArgs& a, int dtype, hipStream_t stream)
{
    (void)hipGetLastError();
    return dtype == 0 ? step_dt<0>(a, stream) : step_dt<1>(a, stream);
}

}  // namespace ssk
