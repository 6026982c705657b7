// gfx950 kernel of sampling from logits.  With the row's tokens in falling order of their logits
// (equal ones by index) and w_j = exp((l_j - l_0) / T), every limit is a prefix of that order, and so
// is what the random number passes over.  So no order is formed: each of top-k, top-p and the random
// number asks for the place in the order at which a running count or sum first reaches a target,
// and that is found by histograms.  Weights are fixed-point numbers of 64 bits: a row's sum fits, sums
// are exact, and neither threads nor atomics change them by their order.
//
// One workgroup has one row.  Bins of equal width in the logit below the largest hold counts and
// weights; their running sums answer which bin a place lies in.  The bin's tokens are copied to LDS
// (or, if they are too many, found in the row again), and histograms over 8 bits at a time of the
// logit's bits, then of the index, lead to the one token.
#include <hip/hip_runtime.h>

#include "ss_attn_internal.h"
#include "ss_device.h"

namespace ssk {
namespace {

constexpr int kThr = 1024;
constexpr int kBins = 2048;   // coarse bins
constexpr int kList = 4096;   // tokens of a bin that fit the LDS
constexpr int kRadix = 256;

// Order-preserving bits of a logit: 0 for the ones that are never taken (NaN, -infinity).
__device__ __forceinline__ uint32_t key_of(float l)
{
    const uint32_t b = __float_as_uint(l + 0.0f);  // -0 and 0 are equal
    const uint32_t k = b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u);
    return l > -INFINITY ? k : 0u;
}
__device__ __forceinline__ float logit_of(uint32_t k)
{
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

struct Shared {
    uint64_t mass[kBins];   // running sums once formed
    uint32_t count[kBins];
    uint32_t key[kList], index[kList];
    uint64_t rmass[kRadix];
    uint32_t rcount[kRadix];
    uint64_t wave_mass[kThr / 64];
    uint32_t wave_count[kThr / 64];
    uint64_t top[kThr / 64];
    uint32_t low[kThr / 64];
    uint32_t found, listed;
};

// The row and what its weights go by.
template <int DT>
struct Row {
    const typename Elem<DT>::T* p;
    int64_t n;
    float top, scale;  // the largest logit; bins per unit of logit
    double rate, unit; // 1 / T; the weight of the largest
    bool infinite;
    __device__ __forceinline__ uint32_t key(int64_t i) const { return key_of(Elem<DT>::load(p, i)); }
    __device__ __forceinline__ int bin(float l) const
    {
        const float f = (top - l) * scale;
        return infinite ? (l < top ? kBins - 1 : 0) : f < float(kBins - 1) ? int(f) : kBins - 1;
    }
    __device__ __forceinline__ uint64_t weight(float l) const
    {
        if (infinite) return l < top ? 0 : uint64_t(unit);
        return uint64_t(rint(exp((double(l) - double(top)) * rate) * unit));
    }
};

// Inclusive running sums over a workgroup's threads.
__device__ __forceinline__ void block_scan(Shared& s, uint64_t& m, uint32_t& c)
{
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint64_t om = __shfl_up(m, d);
        const uint32_t oc = __shfl_up(c, d);
        if (lane >= d) {
            m += om;
            c += oc;
        }
    }
    if (lane == 63) {
        s.wave_mass[w] = m;
        s.wave_count[w] = c;
    }
    __syncthreads();
    for (int i = 0; i < w; ++i) {
        m += s.wave_mass[i];
        c += s.wave_count[i];
    }
    __syncthreads();
}

// Calls f(index, key) for every token of the row that can be taken, this thread's share of them.
template <int DT, typename F>
__device__ __forceinline__ void each(const Row<DT>& r, F f)
{
    for (int64_t i = threadIdx.x; i < r.n; i += kThr) {
        const uint32_t k = r.key(i);
        if (k) f(uint32_t(i), k);
    }
}

// The place in the order at which the count (or the weights) first reaches `target`, 1 <= target <= all:
// its key, the how-manieth of the tokens with that key it is, and the sum of the weights up to it.
struct Place {
    uint32_t key, nth;
    uint64_t mass;
    bool listed;  // whether the list holds its bin
};

template <int DT, bool MASS>
__device__ Place find(Shared& s, const Row<DT>& r, uint64_t target)
{
    // the bin
    __syncthreads();
    for (int b = threadIdx.x; b < kBins; b += kThr) {
        const uint64_t before = b == 0 ? 0 : MASS ? s.mass[b - 1] : s.count[b - 1];
        const uint64_t upto = MASS ? s.mass[b] : s.count[b];
        if (before < target && target <= upto) s.found = uint32_t(b);
    }
    if (threadIdx.x == 0) s.listed = 0;
    __syncthreads();
    const int bin = int(s.found);
    uint64_t mass = bin ? s.mass[bin - 1] : 0;        // of what lies before
    uint64_t count = bin ? s.count[bin - 1] : 0;
    const uint32_t in_bin = s.count[bin] - uint32_t(count);
    Place at;
    at.listed = in_bin <= kList;
    if (at.listed) {
        each(r, [&](uint32_t i, uint32_t k) {
            if (r.bin(logit_of(k)) == bin) {
                const uint32_t slot = atomicAdd(&s.listed, 1u);
                s.key[slot] = k;
                s.index[slot] = i;
            }
        });
        __syncthreads();
    }
    // 8 bits of the key at a time, the largest first
    uint32_t prefix = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
        if (threadIdx.x < kRadix) {
            s.rmass[threadIdx.x] = 0;
            s.rcount[threadIdx.x] = 0;
        }
        __syncthreads();
        auto add = [&](uint32_t, uint32_t k) {
            if (shift < 24 && (k >> (shift + 8)) != prefix) return;
            const int d = 255 - int(k >> shift & 255u);
            atomicAdd(&s.rcount[d], 1u);
            atomicAdd(reinterpret_cast<unsigned long long*>(&s.rmass[d]), r.weight(logit_of(k)));
        };
        if (at.listed) {
            for (uint32_t i = threadIdx.x; i < in_bin; i += kThr) add(0, s.key[i]);
        } else {
            each(r, [&](uint32_t i, uint32_t k) {
                if (r.bin(logit_of(k)) == bin) add(i, k);
            });
        }
        __syncthreads();
        uint64_t m = threadIdx.x < kRadix ? s.rmass[threadIdx.x] : 0;
        uint32_t c = threadIdx.x < kRadix ? s.rcount[threadIdx.x] : 0;
        const uint64_t own_m = m;
        const uint32_t own_c = c;
        block_scan(s, m, c);
        const uint64_t upto = MASS ? mass + m : count + c, before = MASS ? upto - own_m : upto - own_c;
        if (threadIdx.x < kRadix && before < target && target <= upto) {
            s.found = threadIdx.x;
            s.wave_mass[0] = m - own_m;
            s.wave_count[0] = c - own_c;
        }
        __syncthreads();
        prefix = prefix << 8 | (255u - s.found);
        mass += s.wave_mass[0];
        count += s.wave_count[0];
        __syncthreads();
    }
    at.key = prefix;
    const uint64_t w = r.weight(logit_of(prefix));
    at.nth = uint32_t(MASS ? (target - mass + w - 1) / w : target - count);
    at.mass = mass + at.nth * w;
    return at;
}

// The index of the nth token with this key.
template <int DT>
__device__ uint32_t index_of(Shared& s, const Row<DT>& r, const Place& at)
{
    const uint32_t in_list = s.listed;
    uint32_t prefix = 0, before = 0;
    for (int shift = 16; shift >= 0; shift -= 8) {
        if (threadIdx.x < kRadix) s.rcount[threadIdx.x] = 0;
        __syncthreads();
        auto add = [&](uint32_t i, uint32_t k) {
            if (k != at.key || (shift < 16 && (i >> (shift + 8)) != prefix)) return;
            atomicAdd(&s.rcount[i >> shift & 255u], 1u);
        };
        if (at.listed) {
            for (uint32_t i = threadIdx.x; i < in_list; i += kThr) add(s.index[i], s.key[i]);
        } else {
            each(r, add);
        }
        __syncthreads();
        uint64_t m = 0;
        uint32_t c = threadIdx.x < kRadix ? s.rcount[threadIdx.x] : 0;
        const uint32_t own = c;
        block_scan(s, m, c);
        if (threadIdx.x < kRadix && before + c - own < at.nth && at.nth <= before + c) {
            s.found = threadIdx.x;
            s.wave_count[0] = c - own;
        }
        __syncthreads();
        prefix = prefix << 8 | s.found;
        before += s.wave_count[0];
        __syncthreads();
    }
    return prefix;
}

template <int DT>
__global__ __launch_bounds__(kThr) void sample_kernel(SampleArgs a)
{
    __shared__ Shared s;
    const int64_t row = blockIdx.x;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    Row<DT> r;
    r.p = static_cast<const typename Elem<DT>::T*>(a.logits) + row * a.ld;
    r.n = a.vocab;

    // the largest logit with its first place, and the smallest
    uint64_t top = 0;
    uint32_t low = 0xffffffffu;
    each(r, [&](uint32_t i, uint32_t k) {
        const uint64_t v = uint64_t(k) << 32 | (0xffffffffu - i);
        top = v > top ? v : top;
        low = k < low ? k : low;
    });
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint64_t ot = __shfl_xor(top, d);
        const uint32_t ol = __shfl_xor(low, d);
        top = ot > top ? ot : top;
        low = ol < low ? ol : low;
    }
    if (lane == 0) {
        s.top[w] = top;
        s.low[w] = low;
    }
    __syncthreads();
    for (int i = 0; i < kThr / 64; ++i) {
        top = s.top[i] > top ? s.top[i] : top;
        low = s.low[i] < low ? s.low[i] : low;
    }
    const float t = a.temperature ? a.temperature[row] : a.temperature_all;
    if (top == 0 || !(t > 0.0f)) {
        if (threadIdx.x == 0) a.token[row] = top == 0 ? -1 : int64_t(0xffffffffu - uint32_t(top));
        return;
    }

    r.top = logit_of(uint32_t(top >> 32));
    r.infinite = r.top == INFINITY;
    r.rate = 1.0 / double(t);
    // a row's weights sum to less than 2^63, and each fits a double's 52 bits
    const int bits = 64 - __builtin_clzll(uint64_t(r.n));
    const int shift = 62 - bits < 50 ? 62 - bits : 50;
    r.unit = double(uint64_t(1) << shift);
    // bins over what has a weight: exp(-64) of the largest is less than half a unit, whatever the row
    const float depth = fminf(fminf(r.top - logit_of(low), 64.0f * t), 3.0e38f);
    r.scale = depth > 0.0f ? float(kBins - 1) / depth : 0.0f;
    if (!(r.scale < 3.0e38f)) r.scale = 3.0e38f;

    for (int b = threadIdx.x; b < kBins; b += kThr) {
        s.mass[b] = 0;
        s.count[b] = 0;
    }
    __syncthreads();
    const float min_p = a.min_p ? a.min_p[row] : a.min_p_all;
    const double floor_w = min_p > 0.0f ? double(min_p) * r.unit : 0.0;
    uint64_t above = 0;  // the weights that min_p leaves
    each(r, [&](uint32_t, uint32_t k) {
        const float l = logit_of(k);
        const int b = r.bin(l);
        const uint64_t v = r.weight(l);
        atomicAdd(&s.count[b], 1u);
        if (v) atomicAdd(reinterpret_cast<unsigned long long*>(&s.mass[b]), v);
        if (double(v) >= floor_w) above += v;
    });
    __syncthreads();
    // running sums: each thread has neighbouring bins
    {
        constexpr int kPer = kBins / kThr;
        uint64_t m = 0;
        uint32_t c = 0;
        for (int i = 0; i < kPer; ++i) {
            m += s.mass[threadIdx.x * kPer + i];
            c += s.count[threadIdx.x * kPer + i];
        }
        const uint64_t own_m = m;
        const uint32_t own_c = c;
        block_scan(s, m, c);
        m -= own_m;
        c -= own_c;
        for (int i = 0; i < kPer; ++i) {
            m += s.mass[threadIdx.x * kPer + i];
            c += s.count[threadIdx.x * kPer + i];
            s.mass[threadIdx.x * kPer + i] = m;
            s.count[threadIdx.x * kPer + i] = c;
        }
        uint32_t none = 0;
        block_scan(s, above, none);
        if (threadIdx.x == kThr - 1) s.top[0] = above;
        __syncthreads();
        above = s.top[0];
    }
    uint64_t all = s.mass[kBins - 1];
    const int32_t k = a.top_k ? a.top_k[row] : a.top_k_all;
    if (k > 0 && uint32_t(k) < s.count[kBins - 1]) all = find<DT, false>(s, r, uint64_t(k)).mass;
    const float p = a.top_p ? a.top_p[row] : a.top_p_all;
    if (p < 1.0f) {
        const double want = p > 0.0f ? ceil(double(p) * double(all)) : 1.0;
        uint64_t target = want > 1.0 ? uint64_t(want) : 1;
        target = target < all ? target : all;
        all = find<DT, true>(s, r, target).mass;
    }
    if (min_p > 0.0f) {
        const uint64_t first = uint64_t(r.unit);
        const uint64_t kept = above > first ? above : first;
        all = kept < all ? kept : all;
    }
    const float u = a.u[row];
    const double pass = u > 0.0f ? floor(double(u) * double(all)) : 0.0;
    uint64_t target = pass < double(all) ? uint64_t(pass) + 1 : all;
    target = target < all ? target : all;
    const Place at = find<DT, true>(s, r, target);
    const uint32_t token = index_of(s, r, at);
    if (threadIdx.x == 0) a.token[row] = token;
}

}  // namespace

hipError_t launch_sample(const SampleArgs& a, int dtype, hipStream_t stream)
{
    if (dtype == 0) sample_kernel<0><<<uint32_t(a.rows), kThr, 0, stream>>>(a);
    else sample_kernel<1><<<uint32_t(a.rows), kThr, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace ssk
