// gfx950 kernels of linear attention beside its walks (ss_lattn.h): the states between segments, the
// sums over heads that share queries and keys, and the single token.
#include <hip/hip_runtime.h>

#include "ss_attn_internal.h"
#include "ss_device.h"

namespace ssk {
namespace {

// ---- states between segments ------------------------------------------------------------
// What segment i leaves, T_i, and the decay over it, f_i, give the state before each:
// S_0 = h0, S_{i+1} = f_i S_i + T_i (T_i alone where the segment has a reset).  One thread per cell of
// the state; S_i takes T_i's place.  16 heads of 128 x 128 in 32 segments: 15 us, 67 MB read and written.
constexpr int kJoinThreads = 256, kAhead = 8;
__global__ __launch_bounds__(kJoinThreads) void join_kernel(LattnArgs a)
{
    const LattnJob& j = a.job[blockIdx.z];
    const int64_t cells = int64_t(j.dk) * j.dv, bh = blockIdx.x, n = a.batch * a.heads;
    for (int64_t c = int64_t(blockIdx.y) * kJoinThreads + threadIdx.x; c < cells; c += int64_t(gridDim.y) * kJoinThreads) {
        const int64_t i = c / j.dv, k = c % j.dv;
        float s = j.h0 ? j.h0[bh * cells + i * j.si + k * j.sj] : 0.0f;
        float* p = j.seg + bh * cells + c;
        const float* f = j.keep + bh;
        // the last segment's T is not there, nor needed; kAhead of the others are read at a time
        const int64_t last = a.segs - 1;
        for (int64_t g = 0; g < last; g += kAhead) {
            float left[kAhead], keep[kAhead];
#pragma unroll
            for (int e = 0; e < kAhead; ++e) {
                left[e] = g + e < last ? p[e * n * cells] : 0.0f;
                keep[e] = g + e < last ? f[e * n] : 0.0f;
            }
#pragma unroll
            for (int e = 0; e < kAhead; ++e) {
                if (g + e >= last) continue;
                p[e * n * cells] = s;
                s = keep[e] < 0.0f ? left[e] : fmaf(keep[e], s, left[e]);
            }
            p += kAhead * n * cells;
            f += kAhead * n;
        }
        j.seg[(last * n + bh) * cells + c] = s;
    }
}

// ---- sums over the heads that share one ---------------------------------------------------
constexpr int kShareThreads = 256;
template <int DT>
__global__ __launch_bounds__(kShareThreads) void share_kernel(const float* part, void* out, int64_t n, int64_t share,
                                                              int64_t width)
{
    using T = typename Elem<DT>::T;
    for (int64_t i = int64_t(blockIdx.x) * kShareThreads + threadIdx.x; i < n; i += int64_t(gridDim.x) * kShareThreads) {
        const float* p = part + i / width * share * width + i % width;
        float s = p[0];
        for (int64_t g = 1; g < share; ++g) s += p[g * width];
        Elem<DT>::store(static_cast<T*>(out), i, s);
    }
}

// ---- one token --------------------------------------------------------------------------
// S <- a S + k v^T, o = scale S^T q: 8 bytes of the state's traffic per cell and nothing to speak of
// beside it.  A workgroup has one (batch row, head) and 128 columns of the state, or fewer where there
// are fewer; 32 threads side by side take 4 columns each, and the 8 groups of them every 8th row, all
// of whose loads are issued before the first is used (ROWS of them at a time).  Their sums of o are
// joined in order.  256 sequences of 40 heads of 128 x 128: 1.34 GB in 275 us, 4.9 TB/s, a large copy's rate
// (490 us with a load and a store in turn); one sequence: 6.5 us, the latency of one round of loads.
constexpr int kStepGroups = kStepThreads / (kStepCols / 4);
template <int DT, bool VEC, int ROWS>
__global__ __launch_bounds__(kStepThreads) void lattn_step_kernel(LattnStepArgs a)
{
    typedef float f32x4 __attribute__((ext_vector_type(4)));
    using T = typename Elem<DT>::T;
    __shared__ __align__(16) float part[kStepGroups][kStepCols + 4];
    __shared__ float sk[kLattnMaxDim], sq[kLattnMaxDim];
    const uint32_t tiles = uint32_t((a.dv + kStepCols - 1) / kStepCols);
    const int dk = int(a.dk), dv = int(a.dv);
    const int c0 = int(blockIdx.x % tiles) * kStepCols;
    const int64_t bh = blockIdx.x / tiles;
    const int64_t b = bh / a.heads, h = bh % a.heads, hk = h / (a.heads / a.qk_heads);
    const int col = c0 + threadIdx.x % (kStepCols / 4) * 4, group = threadIdx.x / (kStepCols / 4);
    const T* const q = static_cast<const T*>(a.q) + b * a.q_ld + hk * dk;
    const T* const k = static_cast<const T*>(a.k) + b * a.k_ld + hk * dk;
    const T* const v = static_cast<const T*>(a.v) + b * a.v_ld + h * dv;
    float* const s = a.h + (bh * dk + group) * dv + col;
    const int64_t step = int64_t(kStepGroups) * dv;
    f32x4 x[ROWS];
    auto load = [&](int i0) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const float* const p = s + (i0 / kStepGroups + i) * step;
            if constexpr (VEC) {
                if (i0 + kStepGroups * i + group < dk && col < dv) x[i] = *reinterpret_cast<const f32x4*>(p);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (i0 + kStepGroups * i + group < dk && col + e < dv) x[i][e] = p[e];
            }
        }
    };
    load(0);
    for (int i = threadIdx.x; i < dk; i += kStepThreads) {
        sk[i] = Elem<DT>::load(k, i);
        sq[i] = Elem<DT>::load(q, i);
    }
    const float decay = float(exp(double(a.log_decay[h])));
    f32x4 vv = {0.0f, 0.0f, 0.0f, 0.0f}, sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (col + e < dv) vv[e] = Elem<DT>::load(v, col + e);
    __syncthreads();
    for (int i0 = 0;;) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const int r = i0 + kStepGroups * i + group;
            if (r >= dk) continue;
            const float kk = sk[r], qq = sq[r];
            float* const p = s + (i0 / kStepGroups + i) * step;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[i][e] = fmaf(decay, x[i][e], kk * vv[e]);
                sum[e] = fmaf(qq, x[i][e], sum[e]);
            }
            if constexpr (VEC) {
                if (col < dv) *reinterpret_cast<f32x4*>(p) = x[i];
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (col + e < dv) p[e] = x[i][e];
            }
        }
        i0 += kStepGroups * ROWS;
        if (i0 >= dk) break;
        load(i0);
    }
    *reinterpret_cast<f32x4*>(&part[group][col - c0]) = sum;
    __syncthreads();
    if (threadIdx.x < kStepCols && c0 + int(threadIdx.x) < dv) {
        float o = 0.0f;
#pragma unroll
        for (int g = 0; g < kStepGroups; ++g) o += part[g][threadIdx.x];
        Elem<DT>::store(static_cast<T*>(a.o), bh * dv + c0 + threadIdx.x, o * a.scale);
    }
}

bool chunks16(const void* p, int64_t ld, int64_t width, int64_t es)
{
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * es % 16 == 0 && width * es % 16 == 0;
}

}  // namespace

hipError_t launch_lattn_join(const LattnArgs& a, hipStream_t stream)
{
    const dim3 grid(static_cast<uint32_t>(a.batch * a.heads),
                    static_cast<uint32_t>((int64_t(a.job[0].dk) * a.job[0].dv + kJoinThreads - 1) / kJoinThreads),
                    static_cast<uint32_t>(a.jobs));
    join_kernel<<<grid, kJoinThreads, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_lattn(const LattnArgs& a, int dtype, hipStream_t stream)
{
    const int64_t es = dtype == 0 ? 4 : 2;
    bool vec = true;
    for (int i = 0; i < a.jobs; ++i) {
        const LattnJob& j = a.job[i];
        vec = vec && chunks16(j.q, j.q_ld, j.dk, es) && chunks16(j.k, j.k_ld, j.dk, es) &&
              chunks16(j.v, j.v_ld, j.dv, es) && reinterpret_cast<uintptr_t>(j.out) % 16 == 0;
    }
    return dtype == 0 ? launch_lattn_f32(a, vec, stream) : launch_lattn_bf16(a, vec, stream);
}

hipError_t launch_lattn_share(const float* part, void* out, int64_t rows, int64_t heads, int64_t share, int64_t width,
                              int dtype, hipStream_t stream)
{
    const int64_t n = rows * (heads / share) * width;
    const int64_t blocks = (n + kShareThreads - 1) / kShareThreads;
    const uint32_t grid = static_cast<uint32_t>(blocks < 8192 ? blocks : 8192);
    if (dtype == 0) share_kernel<0><<<grid, kShareThreads, 0, stream>>>(part, out, n, share, width);
    else share_kernel<1><<<grid, kShareThreads, 0, stream>>>(part, out, n, share, width);
    return hipGetLastError();
}

template <int DT>
static hipError_t step_typed(const LattnStepArgs& a, hipStream_t stream)
{
    const uint32_t grid = static_cast<uint32_t>(lattn_step_groups(a.batch, a.heads, a.dv));
    const bool vec = a.dv % 4 == 0 && reinterpret_cast<uintptr_t>(a.h) % 16 == 0;
    if (vec) lattn_step_kernel<DT, true, 16><<<grid, kStepThreads, 0, stream>>>(a);
    else lattn_step_kernel<DT, false, 8><<<grid, kStepThreads, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_lattn_step(const LattnStepArgs& a, int dtype, hipStream_t stream)
{
    return dtype == 0 ? step_typed<0>(a, stream) : step_typed<1>(a, stream);
}

}  // namespace ssk
