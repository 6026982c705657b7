// gfx950 kernels of the gated linear recurrence, per batch row and channel
//   k = c softplus(decay),  a_t = exp(-k sigmoid(r_t))  (0 where reset_t),
//   h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t,  y_t = h_t,
// its backward pass and its single-token form.
//
// The update is an affine map h -> a h + b, and maps compose: (a1, b1) then (a2, b2) is
// (a2 a1, a2 b1 + b2).
//
// Forward: one pass.  A workgroup of 8 waves takes 32 VC channels (VC neighbouring ones per lane)
// of kFwdTile rows: each half wave holds a run of 16 rows, forms their a and b in registers, and
// its run's composed map; halves are joined by a lane exchange, waves through LDS.  The tile's map
// is published, the state entering the tile is found from the tiles before it (see `look_back`), and
// every run replays its rows from the state that enters it.  The operands are read once and y is
// written once: HBM traffic bounds it (bf16: 8 bytes per element, 33 vector instructions).
// (1, 131072, 2048) bf16: 435 us, 4.94 TB/s, as much as a copy of 1 GiB reaches (4.8);
// (8, 2048, 5120) with kept states: 144 us; (3, 1021, 1533) fp32 with resets, one channel per lane: 26 us
// for 16 at a copy's rate, its 576 workgroups on 512 places.  In two passes over r and x (chunks' maps,
// then their states) the first took 840.
//
// Backward.  g_t = dL/dh_t = dy_t + a_{t+1} g_{t+1}: the same maps from the end.  q_t = a_t g_t runs
// backward as q -> a (q + dy), so a run's product of a serves both directions.  A workgroup of 4
// waves walks a chunk of rows in tiles of 32 from its end, the states h_{t-1} rebuilt from those kept
// every 32 rows, the next tile's loads in flight.  (Its values per row are too many for the forward's
// way.)  With few (batch row, channel block) pairs the rows are split in chunks: a first pass over
// r and dy forms each chunk's composed map of q.  (8, 2048, 5120) bf16, 14 bytes per element: 296 us,
// 4.1 TB/s: every tile waits on the one before it, which three workgroups per CU do not hide
// quite.  (3, 1021, 1533) fp32 with resets, cut in 7 chunks of 160 rows: 14 + 38 us.
//
// 1 - a^2 = -expm1(-2 k s) is formed without cancellation: as a gate closes a tends to 1 and
// the plain difference would lose every digit.
#include "ss_device.h"
#include "ss_lm_internal.h"

namespace ssk {
namespace {

constexpr int kRunLanes = 32;  // lanes per run: half a wave
// forward: 8 waves, 16 rows per run
constexpr int kFwdWaves = 8, kFwdThreads = 64 * kFwdWaves, kFwdRows = 16, kFwdTile = 2 * kFwdWaves * kFwdRows;
// backward: 4 waves, 4 rows per run
constexpr int kBwdWaves = 4, kBwdRuns = 2 * kBwdWaves, kBwdThreads = 64 * kBwdWaves, kBwdRows = 4;
static_assert(kFwdThreads == kGlrFwdThreads && kBwdThreads == kGlrBwdThreads && kRunLanes == 32, "launches");
static_assert(kFwdTile == kGlrTile && kBwdRuns * kBwdRows == kGlrRows, "tiles and kept states");
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
        typedef __bf16 Pair __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(Raw, Pair{__bf16(v[0]), __bf16(v[1])});  // one instruction
    }
    static __device__ __forceinline__ Raw load(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff)
    {
        return __builtin_amdgcn_raw_buffer_load_b32(r, voff, soff, 0);
    }
    static __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff, Raw v)
    {
        __builtin_amdgcn_raw_buffer_store_b32(v, r, voff, soff, 0);
    }
};
template <>
struct Row<1, 1> {
    using Raw = uint16_t;
    static __device__ __forceinline__ float get(Raw v, int) { return bf16_bits_to_f32(v); }
    static __device__ __forceinline__ Raw make(const float (&v)[1]) { return f32_to_bf16_bits(v[0]); }
    static __device__ __forceinline__ Raw load(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff)
    {
        return __builtin_amdgcn_raw_buffer_load_b16(r, voff, soff, 0);
    }
    static __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff, Raw v)
    {
        __builtin_amdgcn_raw_buffer_store_b16(v, r, voff, soff, 0);
    }
};
typedef uint32_t Words2 __attribute__((ext_vector_type(2)));
template <>
struct Row<0, 2> {
    using Raw = Words2;
    static __device__ __forceinline__ float get(Raw v, int e) { return __uint_as_float(e == 0 ? v.x : v.y); }
    static __device__ __forceinline__ Raw make(const float (&v)[2])
    {
        return Raw{__float_as_uint(v[0]), __float_as_uint(v[1])};
    }
    static __device__ __forceinline__ Raw load(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff)
    {
        return __builtin_amdgcn_raw_buffer_load_b64(r, voff, soff, 0);
    }
    static __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff, Raw v)
    {
        __builtin_amdgcn_raw_buffer_store_b64(v, r, voff, soff, 0);
    }
};
template <>
struct Row<0, 1> {
    using Raw = uint32_t;
    static __device__ __forceinline__ float get(Raw v, int) { return __uint_as_float(v); }
    static __device__ __forceinline__ Raw make(const float (&v)[1]) { return __float_as_uint(v[0]); }
    static __device__ __forceinline__ Raw load(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff)
    {
        return __builtin_amdgcn_raw_buffer_load_b32(r, voff, soff, 0);
    }
    static __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff, Raw v)
    {
        __builtin_amdgcn_raw_buffer_store_b32(v, r, voff, soff, 0);
    }
};

template <int DT>
constexpr uint32_t elem_bytes = DT == 0 ? 4 : 2;

// The rows of one tile of an operand: row q of this lane's run is a scalar offset away from the
// lane's own.  Rows past the chunk's end and lanes past the last channel fall to the range
// check, which counts the scalar offset with the lane's (a raw buffer's does on gfx9): their loads
// read 0 and their stores are dropped.  The host keeps a tile below 2^31 bytes.
template <int DT, int VC>
struct Rows {
    using RW = Row<DT, VC>;
    uint32_t lane, step;  // this lane's offset in a tile, bytes per row
    __device__ Rows(int64_t ld, int64_t d, bool live, int first)
        : lane(live ? uint32_t(first * ld + d) * elem_bytes<DT> : kIdleOffset), step(uint32_t(ld) * elem_bytes<DT>)
    {
    }
    // base: the operand's first element of the batch row; `rows` from `row` on exist
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t tile(const void* base, int64_t row, int rows) const
    {
        return make_rsrc(static_cast<const char*>(base) + row * int64_t(step), uint32_t(rows) * step);
    }
    __device__ __forceinline__ typename RW::Raw load(__amdgpu_buffer_rsrc_t r, int q) const
    {
        return RW::load(r, lane, uint32_t(q) * step);
    }
    __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t r, int q, const float (&v)[VC]) const
    {
        RW::store(r, lane, uint32_t(q) * step, RW::make(v));
    }
};

template <int DT>
__device__ __forceinline__ const void* offset(const void* p, int64_t elems)
{
    return static_cast<const char*>(p) + elems * elem_bytes<DT>;
}

__device__ __forceinline__ float sigmoid1(float v) { return __builtin_amdgcn_rcpf(1.0f + exp2_hw(-v * kLog2e)); }

// sigmoid(v) and 1 - sigmoid(v), both to full relative precision.  The exponent is held below
// 2^126 so that e stays finite and e s tends to 1.
__device__ __forceinline__ float sigmoid2(float v, float* rest)
{
    const float e = exp2_hw(fminf(-v * kLog2e, 126.0f));
    const float s = __builtin_amdgcn_rcpf(1.0f + e);
    *rest = e * s;
    return s;
}

// a = exp(-k s) and w = 1 - a^2 = 1 - e^-t, t = 2 k s.  Below t = 1/2 a polynomial of
// (1 - e^-t) / t (degree 4, a weighted least-squares fit: 1.04e-7 off at most, 1.6e-7 with every
// step rounded, and w within 2.0e-7), above it 1 - a^2 itself (a^2 < 0.61: no cancellation).
__device__ __forceinline__ void decay_of(float k, float s, float* a, float* w)
{
    *a = exp2_hw((-kLog2e * k) * s);
    const float t = (k + k) * s;
    float p = fmaf(t, 0.00677103829f, -0.0410012789f);
    p = fmaf(t, p, 0.166548148f);
    p = fmaf(t, p, -0.49999249f);
    p = fmaf(t, p, 0.99999994f);
    *w = t < 0.5f ? t * p : fmaf(-*a, *a, 1.0f);
}

__device__ __forceinline__ float channel_rate(float decay, float c)
{
    return c * (fmaxf(decay, 0.0f) + log1pf(expf(-fabsf(decay))));
}

// a h + b, the update and the composition of maps.  With resets a factor of 0 means that
// nothing of h remains, not even a NaN or an infinity (0 times which would be NaN), so a row's a
// and a product of them are 0 at resets alone: elsewhere they are at least the least positive number
// (`factor`, `joined`), which takes nothing from a finite state and leaves the others what they are.
template <bool RESET>
__device__ __forceinline__ float carry(float a, float h, float b)
{
    const float v = fmaf(a, h, b);
    return RESET && a == 0.0f ? b : v;
}
// A factor that is not a reset's; a NaN stays one.
__device__ __forceinline__ float factor(float a) { return __uint_as_float(max(__float_as_uint(a), 1u)); }
// The product of two maps' factors.
template <bool RESET>
__device__ __forceinline__ float joined(float a, float b)
{
    return RESET && (a == 0.0f || b == 0.0f) ? 0.0f : factor(a * b);
}

// The other half wave's value.
__device__ __forceinline__ float other_half(float v) { return __shfl_xor(v, 32); }

// What a workgroup of the backward works on.
template <int VC>
struct Place {
    int64_t b, c, d;   // batch row, chunk, first channel of this lane
    int64_t t0, t1;    // the chunk's rows
    int64_t dc;        // d, or a channel that exists where d does not
    bool live;
    __device__ Place(const GlrArgs& a)
    {
        const uint32_t cols = uint32_t((a.dim + kRunLanes * VC - 1) / (kRunLanes * VC));
        const uint32_t id = blockIdx.x, rest = id / cols;
        d = int64_t(id % cols) * (kRunLanes * VC) + (threadIdx.x & 31) * VC;
        b = rest % uint32_t(a.batch);
        c = rest / uint32_t(a.batch);
        live = d < a.dim;
        dc = live ? d : 0;
        t0 = c * a.chunk_len;
        t1 = t0 + a.chunk_len < a.seqlen ? t0 + a.chunk_len : a.seqlen;
    }
};

// ---- forward -------------------------------------------------------------------------------

// A tile's word for one channel: the state's bits in the low half; above them the product of a
// (0 <= a <= 1: its two top bits are clear) and two flags.  kMap: the halves are the tile's map.
// kState: the low half is the state after the tile.  A word is read and written whole, so nothing
// else has to be ordered with it.  Words start as 0, neither flag set.
constexpr uint32_t kMap = 0x40000000u, kState = 0x80000000u, kMapBits = 0x3fffffffu;
constexpr int kWindow = 16;  // tiles looked back over

__device__ __forceinline__ uint64_t word_of(float a, float h, uint32_t flag)
{
    return (uint64_t((__float_as_uint(a) & kMapBits) | flag) << 32) | __float_as_uint(h);
}
__device__ __forceinline__ void put_word(uint64_t* p, uint64_t v)
{
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t get_word(const uint64_t* p)
{
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The state after tile `tile` - 1 of this lane's channel; `words`: the channel's word of tile 0,
// tiles `step` words apart.  Waits until one of the last kWindow tiles has its state and all
// those after it have their maps, then applies the maps in order: the value is the same whichever
// tile's state was there first, since every tile forms its state by the same chain.
// The wait ends: tiles are handed out in order (a tile's predecessors hold a running workgroup or
// are done), maps are published without waiting for anything, and the earliest unfinished tile
// finds its predecessor's state.
template <bool RESET>
__device__ __forceinline__ float look_back(const uint64_t* words, int64_t step, int64_t tile, bool lane_used)
{
    uint64_t w[kWindow];
    int depth;
    for (;;) {
#pragma unroll
        for (int j = 0; j < kWindow; ++j) w[j] = j < tile && lane_used ? get_word(words + (tile - 1 - j) * step) : 0;
        depth = -1;
        bool open = true;
#pragma unroll
        for (int j = 0; j < kWindow; ++j) {
            const uint32_t top = uint32_t(w[j] >> 32);
            if (open && (top & kState)) depth = j;
            open = open && !(top & kState) && (top & kMap);
        }
        if (__all(depth >= 0 || !lane_used)) break;
        __builtin_amdgcn_s_sleep(1);
    }
    float h = 0.0f;
#pragma unroll
    for (int j = kWindow - 1; j >= 0; --j) {
        const float a = __uint_as_float(uint32_t(w[j] >> 32) & kMapBits), b = __uint_as_float(uint32_t(w[j]));
        if (j < depth) h = carry<RESET>(a, h, b);
        if (j == depth) h = b;
    }
    return h;
}

// The words of a call and its ticket, cleared.
__global__ __launch_bounds__(256) void glr_clear_kernel(uint64_t* words, int64_t count, uint32_t* ticket)
{
    const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (i < count) words[i] = 0;
    if (i == 0) *ticket = 0;
}

template <int DT, int VC, bool RESET>
__global__ __launch_bounds__(kFwdThreads, 4) void glr_fwd_kernel(GlrArgs a)
{
    constexpr int R = kFwdRows, W = kFwdWaves;
    using RW = Row<DT, VC>;
    using Raw = typename RW::Raw;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int half = lane >> 5, run = wave * 2 + half, l32 = lane & 31;

    __shared__ float maps[W][2][kRunLanes * VC];  // (product, end) of each wave's rows
    __shared__ float enter[W][kRunLanes * VC];    // the state entering each wave's rows
    __shared__ uint32_t turn;
    uint32_t id = blockIdx.x;
    if (a.n_tiles > 1) {
        // tiles in the order in which workgroups start: a tile's predecessors have all started
        if (threadIdx.x == 0) turn = atomicAdd(a.ws_ticket, 1u);
        __syncthreads();
        id = __builtin_amdgcn_readfirstlane(turn);
    }
    const uint32_t cols = uint32_t((a.dim + kRunLanes * VC - 1) / (kRunLanes * VC));
    const uint32_t units = cols * uint32_t(a.batch);
    const uint32_t tile = id / units, unit = id % units;
    const int64_t b = unit / cols, d0 = int64_t(unit % cols) * (kRunLanes * VC);
    const int64_t d = d0 + l32 * VC, t0 = int64_t(tile) * kFwdTile;
    const bool live = d < a.dim;
    const int64_t dc = live ? d : 0;
    const int rows = int(a.seqlen - t0 < kFwdTile ? a.seqlen - t0 : kFwdTile);
    const int64_t row0 = b * a.seqlen + t0;

    float k[VC];
#pragma unroll
    for (int e = 0; e < VC; ++e) k[e] = channel_rate(a.decay[dc + e], a.c);
    const Rows<DT, VC> px(a.x_ld, d, live, run * R), pr(a.r_ld, d, live, run * R), pi(a.i_ld, d, live, run * R);
    const auto br = pr.tile(a.r, row0, rows), bi = pi.tile(a.i, row0, rows), bx = px.tile(a.x, row0, rows);

    float av[R][VC], bv[R][VC];
    Raw rx[R], rr[R], ri[R];
    bool rs[R];
#pragma unroll
    for (int q = 0; q < R; ++q) {
        rr[q] = pr.load(br, q);
        ri[q] = pi.load(bi, q);
        rx[q] = px.load(bx, q);
        if (RESET) rs[q] = a.reset[row0 + (run * R + q < rows ? run * R + q : 0)] != 0;
    }
    bool cut = false;  // a reset among the run's rows
#pragma unroll
    for (int q = 0; q < R; ++q)
#pragma unroll
        for (int e = 0; e < VC; ++e) {
            float ww;
            decay_of(k[e], sigmoid1(RW::get(rr[q], e)), &av[q][e], &ww);
            float m = __builtin_amdgcn_sqrtf(ww);
            if (RESET) {
                av[q][e] = rs[q] ? 0.0f : factor(av[q][e]);
                m = rs[q] ? 1.0f : m;
            }
            bv[q][e] = m * sigmoid1(RW::get(ri[q], e)) * RW::get(rx[q], e);
        }
    if (rows < kFwdTile) {
        // rows past the end leave the state as it is
#pragma unroll
        for (int q = 0; q < R; ++q)
#pragma unroll
            for (int e = 0; e < VC; ++e) {
                av[q][e] = run * R + q < rows ? av[q][e] : 1.0f;
                bv[q][e] = run * R + q < rows ? bv[q][e] : 0.0f;
            }
    }
    if (RESET) {
#pragma unroll
        for (int q = 0; q < R; ++q) cut = cut || (rs[q] && run * R + q < rows);
    }
    // the run's map, then the wave's; the earlier half publishes it
    float P[VC], E[VC], P0[VC], E0[VC];
#pragma unroll
    for (int e = 0; e < VC; ++e) {
        P[e] = av[0][e];
        E[e] = bv[0][e];
#pragma unroll
        for (int q = 1; q < R; ++q) {
            P[e] *= av[q][e];
            E[e] = carry<RESET>(av[q][e], E[e], bv[q][e]);
        }
        P[e] = cut ? 0.0f : factor(P[e]);
        P0[e] = other_half(P[e]);
        E0[e] = other_half(E[e]);
        if (half == 0) {
            maps[wave][0][l32 * VC + e] = joined<RESET>(P0[e], P[e]);
            maps[wave][1][l32 * VC + e] = carry<RESET>(P0[e], E[e], E0[e]);
        }
    }
    __syncthreads();
    if (wave == 0) {
        // one channel per lane from here on
        const bool used = lane < kRunLanes * VC;
        const int ch = used ? lane : 0;
        const int64_t at = d0 + ch, state = b * a.dim + at;
        const bool exists = used && at < a.dim;
        float A = 1.0f, S = 0.0f, h;
#pragma unroll
        for (int v = 0; v < W; ++v) {
            const float p = maps[v][0][ch];
            A = joined<RESET>(p, A);
            S = carry<RESET>(p, S, maps[v][1][ch]);
        }
        const int64_t step = int64_t(units) * (kRunLanes * VC);
        uint64_t* const words = a.ws_words + int64_t(unit) * (kRunLanes * VC) + ch;
        if (tile == 0) {
            h = a.h0 && exists ? a.h0[state] : 0.0f;
        } else {
            if (used) put_word(words + tile * step, word_of(A, S, kMap));
            h = look_back<RESET>(words, step, tile, used);
        }
        const float after = carry<RESET>(A, h, S);
        if (tile + 1 < a.n_tiles) {
            if (used) put_word(words + tile * step, word_of(0.0f, after, kState));
        } else if (a.h_last && exists) {
            a.h_last[state] = after;
        }
#pragma unroll
        for (int v = 0; v < W; ++v) {
            if (used) enter[v][ch] = h;
            h = carry<RESET>(maps[v][0][ch], h, maps[v][1][ch]);
        }
    }
    __syncthreads();
    float in[VC];
#pragma unroll
    for (int e = 0; e < VC; ++e) {
        in[e] = enter[wave][l32 * VC + e];
        if (half == 1) in[e] = carry<RESET>(P0[e], in[e], E0[e]);
    }
    if (a.ckpt && (run * R) % kGlrRows == 0 && run * R < rows && live) {
        const int64_t at = ((t0 + run * R) / kGlrRows * a.batch + b) * a.dim + d;
#pragma unroll
        for (int e = 0; e < VC; ++e) a.ckpt[at + e] = in[e];
    }
    if (a.y) {
        const Rows<DT, VC> py(a.dim, d, live, run * R);
        const auto by = py.tile(a.y, row0, rows);
#pragma unroll
        for (int q = 0; q < R; ++q) {
#pragma unroll
            for (int e = 0; e < VC; ++e) in[e] = carry<RESET>(av[q][e], in[e], bv[q][e]);
            py.store(by, q, in);
        }
    }
}

// ---- backward ------------------------------------------------------------------------------

// AGG: only each chunk's composed map of q, from r and dy (ws_prod, ws_end)
template <int DT, int VC, bool RESET, bool AGG>
__global__ __launch_bounds__(kBwdThreads, AGG ? 4 : 3) void glr_bwd_kernel(GlrArgs a)
{
    constexpr int R = kBwdRows, T = kBwdRuns * R;
    using RW = Row<DT, VC>;
    using Raw = typename RW::Raw;
    const Place<VC> w(a);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = (threadIdx.x >> 5) & 1, run = wave * 2 + half, l32 = threadIdx.x & 31;
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

    __shared__ float maps[2][kBwdWaves][3 * VC][kRunLanes];
    const Rows<DT, VC> px(a.x_ld, w.d, w.live, run * R), pr(a.r_ld, w.d, w.live, run * R),
        pi(a.i_ld, w.d, w.live, run * R), pd(a.dim, w.d, w.live, run * R), pg(a.g_ld, w.d, w.live, run * R);
    const int64_t row0 = w.b * a.seqlen;
    Raw rx[R], rr[R], ri[R], rd[R];
    uint8_t rs[R];
    float kept[VC];
    auto load = [&](int64_t tile) {
        const int rows = int(w.t1 - tile < T ? w.t1 - tile : T);
        const auto br = pr.tile(a.r, row0 + tile, rows), bi = pi.tile(a.i, row0 + tile, rows),
                   bx = px.tile(a.x, row0 + tile, rows), bd_ = pd.tile(a.dy, row0 + tile, rows);
#pragma unroll
        for (int j = 0; j < R; ++j) {
            rr[j] = pr.load(br, j);
            rd[j] = pd.load(bd_, j);
            if (!AGG) {
                ri[j] = pi.load(bi, j);
                rx[j] = px.load(bx, j);
            }
            if (RESET) {
                const int64_t t = tile + run * R + j;
                rs[j] = t < a.seqlen ? a.reset[row0 + t] : 0;
            }
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
        const int rows = int(w.t1 - tile < T ? w.t1 - tile : T);
        // c1 = m si: dx = g c1.  bv = c1 x, the update's input.  slope: d log a takes
        // g a (h_{t-1} - (a / w) bv), from dm/dlog a = -a^2 / m and w = m^2.
        float av[R][VC], bv[R][VC], c1[R][VC], slope[R][VC], sr[R][VC], nr[R][VC], ni[R][VC], dy[R][VC], h[VC];
        float P[VC], E[VC], Q[VC];
        bool cut = false;  // a reset among the run's rows
        if (RESET) {
#pragma unroll
            for (int j = 0; j < R; ++j) cut = cut || rs[j];
        }
#pragma unroll
        for (int j = 0; j < R; ++j)
#pragma unroll
            for (int e = 0; e < VC; ++e) {
                float ww;
                sr[j][e] = sigmoid2(RW::get(rr[j], e), &nr[j][e]);
                decay_of(k[e], sr[j][e], &av[j][e], &ww);
                if (RESET) {
                    av[j][e] = rs[j] ? 0.0f : factor(av[j][e]);
                    ww = rs[j] ? 1.0f : ww;
                }
                dy[j][e] = RW::get(rd[j], e);
                if (!AGG) {
                    c1[j][e] = __builtin_amdgcn_sqrtf(ww) * sigmoid2(RW::get(ri[j], e), &ni[j][e]);
                    bv[j][e] = c1[j][e] * RW::get(rx[j], e);
                    // where w underflows (the gate shut), bv is 0 and so is the slope's part: the
                    // least normal number beside w changes nothing else
                    slope[j][e] = av[j][e] * bv[j][e] * __builtin_amdgcn_rcpf(ww + 1.1754944e-38f);
                }
            }
        if (rows < T) {
            // rows past the end pass q on as it is and add nothing to the decay's gradient; their dy,
            // and x, read as 0
#pragma unroll
            for (int j = 0; j < R; ++j)
#pragma unroll
                for (int e = 0; e < VC; ++e) {
                    const bool in = run * R + j < rows;
                    av[j][e] = in ? av[j][e] : 1.0f;
                    sr[j][e] = in ? sr[j][e] : 0.0f;
                }
        }
        if (!AGG) {
#pragma unroll
            for (int e = 0; e < VC; ++e) h[e] = kept[e];
        }
        if (tile > w.t0) load(tile - T);
#pragma unroll
        for (int e = 0; e < VC; ++e) {
            P[e] = av[0][e];
            if (!AGG) E[e] = bv[0][e];
#pragma unroll
            for (int j = 1; j < R; ++j) {
                P[e] *= av[j][e];
                if (!AGG) E[e] = carry<RESET>(av[j][e], E[e], bv[j][e]);
            }
            P[e] = cut ? 0.0f : factor(P[e]);
            Q[e] = carry<RESET>(av[R - 1][e], dy[R - 1][e], 0.0f);
#pragma unroll
            for (int j = R - 2; j >= 0; --j) Q[e] = carry<RESET>(av[j][e], Q[e] + dy[j][e], 0.0f);
        }

        float Po[VC], Eo[VC], Qo[VC];  // the other half's
#pragma unroll
        for (int e = 0; e < VC; ++e) {
            Po[e] = other_half(P[e]);
            Qo[e] = other_half(Q[e]);
            if (!AGG) Eo[e] = other_half(E[e]);
            if (half == 0) {
                maps[buf][wave][3 * e][l32] = joined<RESET>(Po[e], P[e]);
                maps[buf][wave][3 * e + 1][l32] = carry<RESET>(P[e], Qo[e], Q[e]);
                if (!AGG) maps[buf][wave][3 * e + 2][l32] = carry<RESET>(Po[e], E[e], Eo[e]);
            }
        }
        __syncthreads();
        float hin[VC], qin[VC];
        if (!AGG) {
#pragma unroll
            for (int v = 0; v < kBwdWaves - 1; ++v)
                if (v < wave) {
#pragma unroll
                    for (int e = 0; e < VC; ++e)
                        h[e] = carry<RESET>(maps[buf][v][3 * e][l32], h[e], maps[buf][v][3 * e + 2][l32]);
                }
#pragma unroll
            for (int e = 0; e < VC; ++e) hin[e] = half == 1 ? carry<RESET>(Po[e], h[e], Eo[e]) : h[e];
        }
#pragma unroll
        for (int v = kBwdWaves - 1; v >= 0; --v)
#pragma unroll
            for (int e = 0; e < VC; ++e) {
                if (!AGG && v == wave) qin[e] = q[e];
                const float p = maps[buf][v][3 * e][l32];
                q[e] = carry<RESET>(p, q[e], maps[buf][v][3 * e + 1][l32]);
                if (AGG) prod[e] = joined<RESET>(p, prod[e]);
            }
        if (!AGG) {
            float before[R][VC];  // h_{t-1}
#pragma unroll
            for (int j = 0; j < R; ++j)
#pragma unroll
                for (int e = 0; e < VC; ++e) {
                    before[j][e] = hin[e];
                    hin[e] = carry<RESET>(av[j][e], hin[e], bv[j][e]);
                }
#pragma unroll
            for (int e = 0; e < VC; ++e)
                if (half == 0) qin[e] = carry<RESET>(Po[e], qin[e], Qo[e]);
            const auto bx = pg.tile(a.dx, row0 + tile, rows), br = pg.tile(a.dr, row0 + tile, rows),
                       bi = pg.tile(a.di, row0 + tile, rows);
#pragma unroll
            for (int j = R - 1; j >= 0; --j) {
                float dx[VC], dr[VC], di[VC];
#pragma unroll
                for (int e = 0; e < VC; ++e) {
                    const float g = qin[e] + dy[j][e];
                    dx[e] = g * c1[j][e];
                    di[e] = g * bv[j][e] * ni[j][e];
                    qin[e] = carry<RESET>(av[j][e], g, 0.0f);
                    // at a reset nothing of log a's gradient is left, whatever lies before it
                    const float through = before[j][e] - slope[j][e];
                    const float dls = carry<RESET>(av[j][e], g * through, 0.0f) * sr[j][e];
                    dr[e] = -k[e] * dls * nr[j][e];
                    dk[e] += dls;
                }
                pg.store(bx, j, dx);
                pg.store(br, j, dr);
                pg.store(bi, j, di);
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
    static_assert(kBwdRuns * VC <= 2 * kBwdWaves * 3 * VC, "fits the maps' space");
#pragma unroll
    for (int e = 0; e < VC; ++e) sums[(run * VC + e) * kRunLanes + l32] = dk[e];
    __syncthreads();
    if (run != 0 || !w.live) return;
#pragma unroll
    for (int e = 0; e < VC; ++e) {
        float s = 0.0f;
        for (int v = 0; v < kBwdRuns; ++v) s += sums[(v * VC + e) * kRunLanes + l32];
        a.part_decay[w.c * a.batch * a.dim + bd + e] = s;
        if (a.dh0 && w.c == 0) a.dh0[bd + e] = q[e];
    }
}

// ddecay = -c sigmoid(decay) sum of the parts, in a fixed order: 16 channels per workgroup, 16
// threads each, every 16th part per thread.
constexpr int kSumCols = 16, kSumParts = 16;
__global__ __launch_bounds__(kSumCols * kSumParts) void glr_decay_kernel(GlrArgs a)
{
    __shared__ float sums[kSumParts][kSumCols];
    const int c = threadIdx.x % kSumCols, p = threadIdx.x / kSumCols;
    const int64_t d = int64_t(blockIdx.x) * kSumCols + c, parts = a.n_chunks * a.batch;
    float s = 0.0f;
    if (d < a.dim)
        for (int64_t j = p; j < parts; j += kSumParts) s += a.part_decay[j * a.dim + d];
    sums[p][c] = s;
    __syncthreads();
    if (p != 0 || d >= a.dim) return;
    s = 0.0f;
#pragma unroll
    for (int v = 0; v < kSumParts; ++v) s += sums[v][c];
    float rest;
    a.ddecay[d] = -a.c * sigmoid2(a.decay[d], &rest) * s;
}

// ---- one token ------------------------------------------------------------------------------

// VC neighbouring channels per thread, loaded and stored together, and ROWS batch rows whose loads
// are in flight together; the channels' rates are formed once for them.  Bound by HBM traffic
// (bf16: 16 bytes per element), and at few rows by the launch.  256 rows of 5120, bf16: 7.2 us of
// which 4.4 are 21 MB at a copy's rate; one row of 1536: 3.1 us.  With two channels of one row per
// thread the first took 10.1.
template <int DT, int VC>
struct Chunk;  // VC elements
template <>
struct Chunk<0, 4> {
    float4 v;
    __device__ __forceinline__ float get(int e) const { return e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w; }
    static __device__ __forceinline__ Chunk make(const float (&f)[4]) { return {make_float4(f[0], f[1], f[2], f[3])}; }
};
template <>
struct Chunk<1, 4> {
    uint2 v;
    __device__ __forceinline__ float get(int e) const
    {
        const uint32_t u = e < 2 ? v.x : v.y;
        return __uint_as_float(e & 1 ? u & 0xffff0000u : u << 16);
    }
    static __device__ __forceinline__ Chunk make(const float (&f)[4])
    {
        return {make_uint2(Row<1, 2>::make({f[0], f[1]}), Row<1, 2>::make({f[2], f[3]}))};
    }
};
template <int DT>
struct Chunk<DT, 1> {
    typename Row<DT, 1>::Raw v;
    __device__ __forceinline__ float get(int) const { return Row<DT, 1>::get(v, 0); }
    static __device__ __forceinline__ Chunk make(const float (&f)[1]) { return {Row<DT, 1>::make(f)}; }
};

constexpr int kStepThreads = kGlrStepThreads;
template <int DT, int VC, int ROWS>
__global__ __launch_bounds__(kStepThreads) void glr_step_kernel(GlrStepArgs a)
{
    using C = Chunk<DT, VC>;
    using H = Chunk<0, VC>;
    const int64_t d = (int64_t(blockIdx.x) * kStepThreads + threadIdx.x) * VC;
    if (d >= a.dim) return;
    float k[VC];
#pragma unroll
    for (int e = 0; e < VC; ++e) k[e] = channel_rate(a.decay[d + e], a.c);
    for (int64_t b0 = int64_t(blockIdx.y) * ROWS; b0 < a.batch; b0 += int64_t(gridDim.y) * ROWS) {
        C r[ROWS], i[ROWS], x[ROWS];
        H h[ROWS];
#pragma unroll
        for (int q = 0; q < ROWS; ++q) {
            const int64_t b = b0 + q < a.batch ? b0 + q : a.batch - 1;
            r[q] = *static_cast<const C*>(offset<DT>(a.r, b * a.r_ld + d));
            i[q] = *static_cast<const C*>(offset<DT>(a.i, b * a.i_ld + d));
            x[q] = *static_cast<const C*>(offset<DT>(a.x, b * a.x_ld + d));
            h[q] = *reinterpret_cast<const H*>(a.h + b * a.dim + d);
        }
#pragma unroll
        for (int q = 0; q < ROWS; ++q) {
            float v[VC];
#pragma unroll
            for (int e = 0; e < VC; ++e) {
                float av, w;
                decay_of(k[e], sigmoid1(r[q].get(e)), &av, &w);
                const float in = __builtin_amdgcn_sqrtf(w) * sigmoid1(i[q].get(e)) * x[q].get(e);
                v[e] = fmaf(av, h[q].get(e), in);
            }
            if (b0 + q < a.batch) {
                *reinterpret_cast<H*>(a.h + (b0 + q) * a.dim + d) = H::make(v);
                *const_cast<C*>(static_cast<const C*>(offset<DT>(a.y, (b0 + q) * a.dim + d))) = C::make(v);
            }
        }
    }
}

// ---- launches ---------------------------------------------------------------------------------

template <int DT, int VC, bool RESET>
hipError_t fwd_variant(const GlrArgs& a, hipStream_t s)
{
    const int64_t blocks = glr_blocks(a, VC, a.n_tiles);
    if (a.n_tiles > 1) {
        const int64_t words = blocks * (kRunLanes * VC);
        glr_clear_kernel<<<dim3(unsigned((words + 255) / 256)), dim3(256), 0, s>>>(a.ws_words, words, a.ws_ticket);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    glr_fwd_kernel<DT, VC, RESET><<<dim3(unsigned(blocks)), dim3(kFwdThreads), 0, s>>>(a);
    return hipGetLastError();
}

template <int DT, int VC, bool RESET>
hipError_t bwd_variant(const GlrArgs& a, hipStream_t s)
{
    const int64_t blocks = glr_blocks(a, VC, a.n_chunks);
    if (a.n_chunks > 1) {
        glr_bwd_kernel<DT, VC, RESET, true><<<dim3(unsigned(blocks)), dim3(kBwdThreads), 0, s>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    glr_bwd_kernel<DT, VC, RESET, false><<<dim3(unsigned(blocks)), dim3(kBwdThreads), 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    glr_decay_kernel<<<dim3(unsigned((a.dim + kSumCols - 1) / kSumCols)), dim3(kSumCols * kSumParts), 0, s>>>(a);
    return hipGetLastError();
}

template <int DT>
hipError_t fwd_dt(const GlrArgs& a, hipStream_t s)
{
    const bool two = glr_fwd_channels(a, DT) == 2;
    if (a.reset) return two ? fwd_variant<DT, 2, true>(a, s) : fwd_variant<DT, 1, true>(a, s);
    return two ? fwd_variant<DT, 2, false>(a, s) : fwd_variant<DT, 1, false>(a, s);
}

template <int DT>
hipError_t bwd_dt(const GlrArgs& a, hipStream_t s)
{
    const bool two = glr_bwd_channels(a, DT) == 2;
    if (a.reset) return two ? bwd_variant<DT, 2, true>(a, s) : bwd_variant<DT, 1, true>(a, s);
    return two ? bwd_variant<DT, 2, false>(a, s) : bwd_variant<DT, 1, false>(a, s);
}

template <int DT, int VC>
hipError_t step_vec(const GlrStepArgs& a, hipStream_t s)
{
    const int64_t cols = (a.dim + kStepThreads * VC - 1) / (kStepThreads * VC);
    // two rows per thread when that leaves two workgroups per CU
    if (cols * a.batch >= 1024) {
        const int64_t rows = (a.batch + 1) / 2;
        glr_step_kernel<DT, VC, 2><<<dim3(unsigned(cols), unsigned(rows < 65535 ? rows : 65535)), dim3(kStepThreads), 0,
                                     s>>>(a);
    } else {
        glr_step_kernel<DT, VC, 1><<<dim3(unsigned(cols), unsigned(a.batch < 65535 ? a.batch : 65535)),
                                     dim3(kStepThreads), 0, s>>>(a);
    }
    return hipGetLastError();
}

template <int DT>
hipError_t step_dt(const GlrStepArgs& a, hipStream_t s)
{
    return glr_step_channels(a, DT) == 4 ? step_vec<DT, 4>(a, s) : step_vec<DT, 1>(a, s);
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
