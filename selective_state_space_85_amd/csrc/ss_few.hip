// gfx950 kernels of the gradients of a product x W^T with few rows of x, in one pass over the weights:
//   dx = s W (m, k) and dW = s^T x (rows, k), s (m, rows) the gradient of the product, fp32.
//
// A thread owns 4 neighbouring columns: its x (m x 4 values) and its sums of dx stay in registers
// while it walks a range of W's rows; a row is read once for dx and its dW is written beside it, with
// the row's m factors broadcast from LDS.  2 m multiply-adds per element: at 8 rows still below
// what reading and writing the weights takes (HBM traffic bounds it), with no padding or rounding of
// s on the way.  The ranges' sums of dx are joined by a second kernel, in order.
// One token, 3401 -> 2 x 8588, fp32, forward and backward: 235 us, of which 196 are the weights read
// three times and their gradients written once at a copy's rate; padded copies and tiles took 737.
#include "ss_gemm.h"
#include "ss_lm_internal.h"

namespace ssk {
namespace {

constexpr int kFewThreads = 128, kFewCols = 4, kFewTile = 64;  // rows of s staged together
constexpr int kFewUnroll = 4;                                  // rows of W in flight

template <int DT>
struct Cols;
template <>
struct Cols<0> {
    using V = f32x4;
};
template <>
struct Cols<1> {
    using V = bf16x4;
};

// 4 elements at any alignment, of which `left` exist
template <int DT>
__device__ __forceinline__ void get4(const typename MM<DT>::T* p, int64_t left, float (&v)[4])
{
    if (left >= 4) {
        typename Cols<DT>::V q;
        __builtin_memcpy(&q, p, sizeof(q));
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = MM<DT>::widen(q[e]);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = e < left ? MM<DT>::widen(p[e]) : 0.0f;
    }
}
template <int DT>
__device__ __forceinline__ void put4(typename MM<DT>::T* p, int64_t left, const float (&v)[4])
{
    if (left >= 4) {
        typename Cols<DT>::V q;
#pragma unroll
        for (int e = 0; e < 4; ++e) q[e] = MM<DT>::narrow(v[e]);
        __builtin_memcpy(p, &q, sizeof(q));
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < left) p[e] = MM<DT>::narrow(v[e]);
    }
}

__device__ __forceinline__ bool row_counts(const FewGradArgs& a, int64_t i)
{
    if (!a.target) return true;
    const int64_t t = a.target[i];
    return t != a.ignore_index && t >= 0 && t < a.rows;
}

template <int DT, int MR, bool DX, bool DW>
__global__ __launch_bounds__(kFewThreads) void few_grad_kernel(FewGradArgs a)
{
    using T = typename MM<DT>::T;
    __shared__ float tile[kFewTile][MR];
    const int64_t c = (int64_t(blockIdx.x) * kFewThreads + threadIdx.x) * kFewCols, left = a.k - c;
    const int64_t r0 = int64_t(blockIdx.y) * a.per, r1 = r0 + a.per < a.rows ? r0 + a.per : a.rows;
    float x[MR][4], sum[MR][4];
#pragma unroll
    for (int i = 0; i < MR; ++i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[i][e] = sum[i][e] = 0.0f;
        if (DW && i < a.m && left > 0 && row_counts(a, i)) get4<DT>(static_cast<const T*>(a.x) + i * a.x_ld + c, left, x[i]);
    }
    for (int64_t rb = r0; rb < r1; rb += kFewTile) {
        __syncthreads();
        for (int q = threadIdx.x; q < kFewTile * MR; q += kFewThreads) {
            const int i = q / kFewTile, rr = q % kFewTile;
            const int64_t r = rb + rr;
            const int64_t at = r < a.first ? r : r - a.first + a.s_second;
            tile[rr][i] = r < r1 && i < a.m ? a.s[i * a.s_ld + at] : 0.0f;
        }
        __syncthreads();
        if (left <= 0) continue;
        const int n = int(r1 - rb < kFewTile ? r1 - rb : kFewTile);
        for (int rr = 0; rr < n; rr += kFewUnroll) {
            float w[kFewUnroll][4];
            if (DX) {
#pragma unroll
                for (int u = 0; u < kFewUnroll; ++u) {
                    const int64_t r = rb + (rr + u < n ? rr + u : n - 1);  // past the end: its factors are 0
                    const T* p = r < a.first ? static_cast<const T*>(a.w0) + r * a.k
                                             : static_cast<const T*>(a.w1) + (r - a.first) * a.k;
                    get4<DT>(p + c, left, w[u]);
                }
            }
#pragma unroll
            for (int u = 0; u < kFewUnroll; ++u) {
                float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int i = 0; i < MR; ++i) {
                    const float s = tile[(rr + u) % kFewTile][i];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (DX && rr + u < n) sum[i][e] = fmaf(s, w[u][e], sum[i][e]);
                        if (DW) d[e] = fmaf(s, x[i][e], d[e]);
                    }
                }
                if (DW && rr + u < n) {
                    const int64_t r = rb + rr + u;
                    T* p = r < a.first ? static_cast<T*>(a.dw0) + r * a.k : static_cast<T*>(a.dw1) + (r - a.first) * a.k;
                    put4<DT>(p + c, left, d);
                }
            }
        }
    }
    if (!DX || left <= 0) return;
#pragma unroll
    for (int i = 0; i < MR; ++i)
        if (i < a.m) put4<0>(a.part + (blockIdx.y * a.m + i) * a.k + c, left, sum[i]);
}

// dx from its parts, in order.
template <int DT>
__global__ __launch_bounds__(256) void few_sum_kernel(FewGradArgs a)
{
    const int64_t n = a.m * a.k, i = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (i >= n) return;
    float s = 0.0f;
#pragma unroll 8
    for (int64_t p = 0; p < a.parts; ++p) s += a.part[p * n + i];
    static_cast<typename MM<DT>::T*>(a.dx)[i] = MM<DT>::narrow(row_counts(a, i / a.k) ? s : 0.0f);
}

template <int DT, int MR>
hipError_t few_grad(const FewGradArgs& a, hipStream_t s)
{
    const dim3 grid(up(a.k, kFewThreads * kFewCols), unsigned(a.parts)), block(kFewThreads);
    if (!a.part)
        few_grad_kernel<DT, MR, false, true><<<grid, block, 0, s>>>(a);
    else if (!a.dw0)
        few_grad_kernel<DT, MR, true, false><<<grid, block, 0, s>>>(a);
    else
        few_grad_kernel<DT, MR, true, true><<<grid, block, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.part) return e;
    few_sum_kernel<DT><<<dim3(up(a.m * a.k, 256)), dim3(256), 0, s>>>(a);
    return hipGetLastError();
}

template <int DT>
hipError_t few_dt(const FewGradArgs& a, hipStream_t s)
{
    if (a.m <= 1) return few_grad<DT, 1>(a, s);
    if (a.m <= 4) return few_grad<DT, 4>(a, s);
    return few_grad<DT, int(kFewRows)>(a, s);
}

}  // namespace

hipError_t launch_few_grad(const FewGradArgs& a, int dtype, hipStream_t stream)
{
    (void)hipGetLastError();
    return dtype == 0 ? few_dt<0>(a, stream) : few_dt<1>(a, stream);
}

}  // namespace ssk
