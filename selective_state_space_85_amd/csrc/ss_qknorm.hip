// gfx950 kernels of the norms of queries and keys for each head with their position rotation, and
// of its gradients.  For one token and head, with r = 1 / sqrt(mean(x^2) + eps):
//   y = R(pos) (x r w)
// and with g = R(pos)^-1 dy:
//   dw = sum over tokens and heads of g x r,   dx = r (g w - x r mean(g w x r))
// R turns pair i of the first 2 n elements by pos * inv_freq[i].
//
// A head belongs to a group of GL lanes, each with 8 of its elements as 4 pairs; a workgroup takes
// a tile of tokens.  It first forms the tile's cosines and sines, one angle per thread, each once for
// all heads, then its groups of lanes walk the tile's heads in the order in which they lie in memory.
// The angle is a number of turns, reduced in 64 bits before it is rounded: a product of a position
// and a frequency in 32 bits would be off by whole turns far into a long context.
//
// What bounds it: HBM, each input read and each output written once.  bf16: 131072 tokens of 16 + 4 heads of
// 128 forward 256 us, 5.2 TB/s; 16384 tokens of 40 + 40 heads forward 134 us, 5.0 TB/s, backward 217 + 5 us,
// 4.6 TB/s.  One token 4.2 us, the latency of its angles and of one row.  fp32 of an odd pairing, 3063 tokens of
// 12 + 4 heads of 90: 11 us forward, 18 + 4 backward, three rounds of latency for each workgroup.  In the
// backward, loading the next row before the sums of this one: 217 -> 338 us.
#include <hip/hip_runtime.h>

#include "ss_attn_internal.h"
#include "ss_device.h"

namespace ssk {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// four neighbouring elements, in fp32
__device__ __forceinline__ void load4(const float* p, float (&v)[4])
{
    const f32x4 x = *reinterpret_cast<const f32x4*>(p);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = x[e];
}
__device__ __forceinline__ void load4(const uint16_t* p, float (&v)[4])
{
    const u32x2 x = *reinterpret_cast<const u32x2*>(p);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        v[2 * e] = __uint_as_float(x[e] << 16);
        v[2 * e + 1] = __uint_as_float(x[e] & 0xffff0000u);
    }
}
__device__ __forceinline__ void store4(float* p, const float (&v)[4])
{
    *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
}
__device__ __forceinline__ void store4(uint16_t* p, const float (&v)[4])
{
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    *reinterpret_cast<u32x2*>(p) = u32x2{__builtin_bit_cast(uint32_t, bf16x2{__bf16(v[0]), __bf16(v[1])}),
                                         __builtin_bit_cast(uint32_t, bf16x2{__bf16(v[2]), __bf16(v[3])})};
}

// Where a lane's 8 elements lie.  Pair s is (s, s + half), or (2 s, 2 s + 1) if interleaved; past the
// turned pairs the elements go two by two.  VEC: half is a multiple of 4 and the width of 8, so that a lane's
// elements are two runs of four, pairs 4 lane + e; unturned runs need no pairing.  Otherwise they go one by
// one, pairs lane + GL e, so that a group's loads lie side by side (3063 tokens of
// 12 + 4 heads of 90 in fp32: 17.4 -> 11.2 us forward, 24.2 -> 18.2 backward).
template <int DT, bool VEC, bool INTER, int GL>
struct Slots {
    using T = typename Elem<DT>::T;
    int width, half, at;  // at: the lane's first pair
    __device__ __forceinline__ Slots(int w, int h) : width(w), half(h), at(int(threadIdx.x % GL) * (VEC ? 4 : 1)) {}
    __device__ __forceinline__ int pair(int e) const { return at + (VEC ? e : GL * e); }
    __device__ __forceinline__ bool live() const { return VEC ? 2 * at < width : true; }
    __device__ __forceinline__ int run_a() const { return !INTER && at < half ? at : 2 * at; }
    __device__ __forceinline__ int run_b() const { return !INTER && at < half ? at + half : 2 * at + 4; }
    __device__ __forceinline__ int elem_a(int e) const { return !INTER && pair(e) < half ? pair(e) : 2 * pair(e); }
    __device__ __forceinline__ int elem_b(int e) const { return !INTER && pair(e) < half ? pair(e) + half : 2 * pair(e) + 1; }
    template <typename P>
    __device__ __forceinline__ void load(const P* p, float (&a)[4], float (&b)[4]) const
    {
        if constexpr (VEC) {
            // lanes past the width read its first elements and drop them
            float x[4], y[4];
            load4(p + (live() ? run_a() : 0), x);
            load4(p + (live() ? run_b() : 4), y);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float u = INTER ? (e < 2 ? x[2 * e] : y[2 * e - 4]) : x[e];
                const float v = INTER ? (e < 2 ? x[2 * e + 1] : y[2 * e - 3]) : y[e];
                a[e] = live() ? u : 0.0f;
                b[e] = live() ? v : 0.0f;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                a[e] = elem_a(e) < width ? one(p, elem_a(e)) : 0.0f;
                b[e] = elem_b(e) < width ? one(p, elem_b(e)) : 0.0f;
            }
        }
    }
    template <typename P>
    __device__ __forceinline__ void store(P* p, const float (&a)[4], const float (&b)[4]) const
    {
        if constexpr (VEC) {
            if (!live()) return;
            if constexpr (INTER) {
                const float x[4] = {a[0], b[0], a[1], b[1]}, y[4] = {a[2], b[2], a[3], b[3]};
                store4(p + run_a(), x);
                store4(p + run_b(), y);
            } else {
                store4(p + run_a(), a);
                store4(p + run_b(), b);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (elem_a(e) < width) put(p, elem_a(e), a[e]);
                if (elem_b(e) < width) put(p, elem_b(e), b[e]);
            }
        }
    }
    // cosines and sines of the lane's pairs from a token's row of the table
    __device__ __forceinline__ void turns(const float2* row, float (&c)[4], float (&s)[4]) const
    {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool on = pair(e) < half;
            const float2 v = row[on ? pair(e) : 0];
            c[e] = on ? v.x : 1.0f;
            s[e] = on ? v.y : 0.0f;
        }
    }

private:
    static __device__ __forceinline__ float one(const float* p, int i) { return p[i]; }
    static __device__ __forceinline__ float one(const uint16_t* p, int i) { return bf16_bits_to_f32(p[i]); }
    static __device__ __forceinline__ void put(float* p, int i, float v) { p[i] = v; }
    static __device__ __forceinline__ void put(uint16_t* p, int i, float v) { p[i] = f32_to_bf16_bits(v); }
};

// Cosines and sines of the tokens [t0, t0 + n).
__device__ __forceinline__ void fill_table(const QknormArgs& a, float2* table, int64_t t0, int n)
{
    const int half = int(a.half);
    for (int i = threadIdx.x; i < n * half; i += kQknormThreads) {
        const double turns = double(a.pos[t0 + i / half]) * double(a.inv_freq[i % half]) * 0.15915494309189535;
        float s, c;
        sincospif(2.0f * float(turns - rint(turns)), &s, &c);
        table[i] = float2{c, s};
    }
}

template <int GL>
__device__ __forceinline__ float group_sum(float v)
{
#pragma unroll
    for (int m = 1; m < GL; m *= 2) v += __shfl_xor(v, m);
    return v;
}

template <int DT, bool VEC, bool INTER, int GL>
__global__ __launch_bounds__(kQknormThreads) void qknorm_fwd_kernel(QknormArgs a, int tile)
{
    using T = typename Elem<DT>::T;
    __shared__ float2 table[kQknormAngles];
    const int64_t t0 = int64_t(blockIdx.x) * tile;
    const int n = int(a.tokens - t0 < tile ? a.tokens - t0 : tile);
    const int width = int(a.width), half = int(a.half);
    const Slots<DT, VEC, INTER, GL> sl(width, half);
    fill_table(a, table, t0, n);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const QknormSide& s = a.side[i];
        const int heads = int(s.heads);
        float wa[4], wb[4];
        sl.load(s.w, wa, wb);
        // every lane of a group has the same row, and with it the same way through the loop
        for (int row = threadIdx.x / GL; row < n * heads; row += kQknormThreads / GL) {
            const int t = row / heads, h = row % heads;
            float xa[4], xb[4], c[4], sn[4];
            sl.load(static_cast<const T*>(s.x) + (t0 + t) * s.ld + int64_t(h) * width, xa, xb);
            float sum = 0.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) sum = fmaf(xa[e], xa[e], fmaf(xb[e], xb[e], sum));
            const float r = rsqrtf(group_sum<GL>(sum) / float(width) + a.eps);
            sl.turns(table + t * half, c, sn);
            float ya[4], yb[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float p = xa[e] * r * wa[e], q = xb[e] * r * wb[e];
                ya[e] = p * c[e] - q * sn[e];
                yb[e] = q * c[e] + p * sn[e];
            }
            sl.store(static_cast<T*>(s.out) + ((t0 + t) * heads + h) * width, ya, yb);
        }
    }
}

template <int DT, bool VEC, bool INTER, int GL>
__global__ __launch_bounds__(kQknormThreads) void qknorm_bwd_kernel(QknormArgs a, int tile)
{
    using T = typename Elem<DT>::T;
    constexpr int kGroups = kQknormThreads / GL;
    __shared__ float2 table[kQknormAngles];
    __shared__ __align__(16) float sums[kGroups][8 * GL];
    const int width = int(a.width), half = int(a.half);
    const Slots<DT, VEC, INTER, GL> sl(width, half);
    const int group = threadIdx.x / GL;
    float da[2][4] = {}, db[2][4] = {};
    const int64_t tiles = (a.tokens + tile - 1) / tile;
    for (int64_t at = blockIdx.x; at < tiles; at += gridDim.x) {
        const int64_t t0 = at * tile;
        const int n = int(a.tokens - t0 < tile ? a.tokens - t0 : tile);
        __syncthreads();
        fill_table(a, table, t0, n);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const QknormSide& s = a.side[i];
            const int heads = int(s.heads);
            float wa[4], wb[4];
            sl.load(s.w, wa, wb);
            for (int row = group; row < n * heads; row += kGroups) {
                const int t = row / heads, h = row % heads;
                const int64_t flat = ((t0 + t) * heads + h) * width;
                float xa[4], xb[4], ga[4], gb[4], c[4], sn[4];
                sl.load(static_cast<const T*>(s.x) + (t0 + t) * s.ld + int64_t(h) * width, xa, xb);
                sl.load(static_cast<const T*>(s.dy) + flat, ga, gb);
                float sum = 0.0f;
#pragma unroll
                for (int e = 0; e < 4; ++e) sum = fmaf(xa[e], xa[e], fmaf(xb[e], xb[e], sum));
                const float r = rsqrtf(group_sum<GL>(sum) / float(width) + a.eps);
                sl.turns(table + t * half, c, sn);
                float dot = 0.0f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float p = ga[e] * c[e] + gb[e] * sn[e], q = gb[e] * c[e] - ga[e] * sn[e];
                    xa[e] *= r;
                    xb[e] *= r;
                    da[i][e] = fmaf(p, xa[e], da[i][e]);
                    db[i][e] = fmaf(q, xb[e], db[i][e]);
                    ga[e] = p * wa[e];
                    gb[e] = q * wb[e];
                    dot = fmaf(ga[e], xa[e], fmaf(gb[e], xb[e], dot));
                }
                const float m = group_sum<GL>(dot) / float(width);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    ga[e] = r * (ga[e] - xa[e] * m);
                    gb[e] = r * (gb[e] - xb[e] * m);
                }
                sl.store(static_cast<T*>(s.out) + flat, ga, gb);
            }
        }
    }
    // The groups' sums of dw, joined in order.  These joins and the next kernel's are in 64 bits, beside which
    // the rest of either does not notice them: in 32 each addition would round all that is summed so far.
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        __syncthreads();
        sl.store(&sums[group][0], da[i], db[i]);
        __syncthreads();
        for (int c = threadIdx.x; c < width; c += kQknormThreads) {
            double v = 0.0;
            for (int g = 0; g < kGroups; ++g) v += double(sums[g][c]);
            a.part[(i * int64_t(gridDim.x) + blockIdx.x) * width + c] = float(v);
        }
    }
}

// dw[c] = sum of the workgroups' sums: 16 columns x 64 runs of workgroups, the runs joined in order.
constexpr int kSumCols = 16, kSumRuns = 64;
__global__ __launch_bounds__(kSumCols * kSumRuns) void qknorm_sum_kernel(QknormArgs a)
{
    __shared__ double run[kSumRuns][kSumCols];
    const int c = threadIdx.x % kSumCols, g = threadIdx.x / kSumCols;
    const int64_t col = int64_t(blockIdx.x) * kSumCols + c;
    const float* const p = a.part + int64_t(blockIdx.y) * a.blocks * a.width;
    double v = 0.0;
    if (col < a.width)
#pragma unroll 8
        for (int64_t i = g; i < a.blocks; i += kSumRuns) v += double(p[i * a.width + col]);
    run[g][c] = v;
    __syncthreads();
    if (g == 0 && col < a.width) {
        double s = 0.0;
        for (int i = 0; i < kSumRuns; ++i) s += run[i][c];
        a.side[blockIdx.y].dw[col] = float(s);
    }
}

bool runs_of_four(const void* p, int64_t ld, int64_t es)
{
    return reinterpret_cast<uintptr_t>(p) % uintptr_t(4 * es) == 0 && ld % 4 == 0;
}

template <int DT, bool VEC, bool INTER>
hipError_t launch(const QknormArgs& a, bool back, hipStream_t stream)
{
    const int tile = int(qknorm_tile(a.tokens, a.half, back));
    const uint32_t tiles = uint32_t(qknorm_tiles(a.tokens, a.half, false));
    auto go = [&](auto gl) {
        constexpr int GL = decltype(gl)::value;
        if (back) qknorm_bwd_kernel<DT, VEC, INTER, GL><<<uint32_t(a.blocks), kQknormThreads, 0, stream>>>(a, tile);
        else qknorm_fwd_kernel<DT, VEC, INTER, GL><<<tiles, kQknormThreads, 0, stream>>>(a, tile);
        return hipGetLastError();
    };
    using std::integral_constant;
    return a.width <= 64 ? go(integral_constant<int, 8>())
           : a.width <= 128 ? go(integral_constant<int, 16>())
           : a.width <= 256 ? go(integral_constant<int, 32>()) : go(integral_constant<int, 64>());
}

template <int DT>
hipError_t launch(const QknormArgs& a, bool back, hipStream_t stream)
{
    const int64_t es = DT == 0 ? 4 : 2;
    bool vec = a.width % 8 == 0 && a.half % 4 == 0;
    for (const QknormSide& s : a.side)
        vec = vec && runs_of_four(s.x, s.ld, es) && runs_of_four(s.out, s.heads * a.width, es) &&
              runs_of_four(s.w, 4, 4) && (!back || runs_of_four(s.dy, 4, es));
    if (vec) return a.interleaved ? launch<DT, true, true>(a, back, stream) : launch<DT, true, false>(a, back, stream);
    return a.interleaved ? launch<DT, false, true>(a, back, stream) : launch<DT, false, false>(a, back, stream);
}

}  // namespace

hipError_t launch_qknorm_fwd(const QknormArgs& a, int dtype, hipStream_t stream)
{
    return dtype == 0 ? launch<0>(a, false, stream) : launch<1>(a, false, stream);
}

hipError_t launch_qknorm_bwd(const QknormArgs& a, int dtype, hipStream_t stream)
{
    const hipError_t e = dtype == 0 ? launch<0>(a, true, stream) : launch<1>(a, true, stream);
    if (e != hipSuccess) return e;
    qknorm_sum_kernel<<<dim3(uint32_t((a.width + kSumCols - 1) / kSumCols), 2), kSumCols * kSumRuns, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace ssk
