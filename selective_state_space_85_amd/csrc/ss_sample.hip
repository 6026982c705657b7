// gfx950 kernel of sampling from logits.  With the row's tokens in falling order of their logits
// (equal ones by index) and w_j = exp((l_j - l_0) / T), every limit is a prefix of that order, and so
// is what the random number passes over.  So no order is formed: each of top-k, top-p and the random
// number asks for the place in the order at which a running count or sum first reaches a target.
// Weights are fixed-point numbers of 64 bits: a row's sum fits, sums are exact, and neither threads nor
// atomics change them by their order.
//
// One workgroup has one row and reads it three times (from the caches, but for the first):
//  1. the largest logit and the smallest;
//  2. bins of equal width in the logit, with their weights.  Their running sums tell which bin a place
//     lies in.  With a small top-k no bins of the row are needed: the tokens that are at least the k-th largest
//     of the threads' own maxima hold the first k, fit the LDS, and are binned by count, then by weight;
//  3. the tokens of the bins that the limits leave, to LDS, if they fit there.
// A place is then found among the tokens of its bin: up to 64 of them, by one wave, a token to a lane,
// each counting what comes before it.  More are first cut down by histograms over 8 bits of their logits
// at a time and, where those are equal, of their indices.
//
// What bounds it: one workgroup's passes, scans and barriers, not bytes.  One row of 50257 in bf16, nucleus: 30
// us, of which 3 for the largest logit, 15 for the weights' bins (some 40 instructions and an LDS addition for
// each of 49 tokens a thread), 5-7 for the list, 2-3 for a place.  64 rows of 131072, top-k of 50 and nucleus,
// a row to a CU: 30 us (35 with counts of the whole row, and 23 of them for those).  256 rows of 50257 in fp32
// with settings of their own: 56 us, a workgroup to a CU (85 KB of LDS, 94 registers a thread).
#include <hip/hip_runtime.h>

#include "ss_attn_internal.h"
#include "ss_device.h"

namespace ssk {
namespace {

constexpr int kThr = 1024;
constexpr int kBins = 4096;   // coarse bins
constexpr int kList = 4096;   // tokens that fit the LDS
constexpr int kFew = 64;      // tokens of one wave
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
    uint64_t mass[kBins];   // the bins' weights, running sums once formed
    uint32_t count[kBins];  // the same of their tokens
    uint32_t key[kList], index[kList];
    double root[64];        // 2^(i / 64)
    uint64_t rmass[kRadix];
    uint32_t few_key[kFew], few_index[kFew];
    uint64_t wave_mass[kThr / 64];
    uint32_t wave_count[kThr / 64];
    float top[kThr / 64], low[kThr / 64];
    uint64_t found_mass;
    uint32_t found, found_key, found_index, listed, few;
};

// 8 or 4 elements at any alignment
template <int DT>
struct Piece;
template <>
struct Piece<0> {
    static constexpr int kN = 4;
    typedef float V __attribute__((ext_vector_type(4), aligned(4)));
    V v;
    __device__ __forceinline__ float operator[](int i) const { return v[i]; }
};
template <>
struct Piece<1> {
    static constexpr int kN = 8;
    typedef uint32_t V __attribute__((ext_vector_type(4), aligned(2)));
    V v;
    __device__ __forceinline__ float operator[](int i) const
    {
        return __uint_as_float(i & 1 ? v[i / 2] & 0xffff0000u : v[i / 2] << 16);
    }
};

// The row, and what its weights go by.
template <int DT>
struct Row {
    const typename Elem<DT>::T* p;
    int n;
    float least;  // the smallest logit that can be taken: the lowest number, or infinity if one is there
    // what logits are multiplied with so that differences stay finite: 1, 1 / 4, or 0 for infinities, which
    // are all equal then
    float pre;
    float top, scale;  // the largest logit; bins of counts per unit of logit
    // a logit whose weight is 0 in place of all below it, NaN and -infinity too; plain: it is there and `pre` is 1
    float floor;
    bool plain;
    double rate;       // log2(e) / T; both go by logits times `pre`
    int shift;         // the largest logit's weight is 2^shift
    __device__ __forceinline__ float value(float l) const { return fminf(l, 3.402823466e38f) * pre; }
    // the bin of a count
    __device__ __forceinline__ int count_bin(float l) const { return int(fminf((top - value(l)) * scale, float(kBins - 1))); }
    // The weight 2^shift exp((l - top) / T), rounded, and its bin: 2^t = 2^i root[j] 2^r with t = i + j / 64 + r,
    // |r| <= 1 / 128, 2^r by its series, of which the first term left out is (ln 2 / 128)^6 / 720 = 3.5e-17.
    // Bins are 1 / 64 of a halving wide: the weights of the last one are below 2^-63 of the largest, which is
    // less than half a unit, whatever the row.
    template <bool PLAIN = false>
    __device__ __forceinline__ uint64_t weight(float l, const double* root, int* bin) const
    {
        constexpr double kGrid = 6755399441055744.0 / 64;  // 1.5 * 2^52 / 64: sums are multiples of 1 / 64
        constexpr double kWhole = 4503599627370496.0;      // 2^52: sums are integers
        const double t = PLAIN ? (double(fmaxf(l, floor)) - double(top)) * rate
                               : fmax((double(value(l)) - double(top)) * rate, -1000.0);
        const double g = t + kGrid;
        const int n64 = int(__double_as_longlong(g));  // 64 t, rounded, in the low bits
        const double r = t - (g - kGrid);
        double s = fma(r, 0.0013333558146428441, 0.0096181291076284769);
        s = fma(r, s, 0.055504108664821576);
        s = fma(r, s, 0.24022650695910069);
        s = fma(r, s, 0.69314718055994529) * r;
        const double m = root[n64 & 63];
        const double w = ldexp(fma(m, s, m), (n64 >> 6) + shift);
        *bin = -n64 < kBins - 1 ? -n64 : kBins - 1;
        return uint64_t(__double_as_longlong(w + kWhole)) & 0xfffffffffffffull;
    }
    __device__ __forceinline__ int weight_bin(float l) const
    {
        const double t = fmax((double(value(l)) - double(top)) * rate, -1000.0);
        const int n64 = int(__double_as_longlong(t + 6755399441055744.0 / 64));
        return -n64 < kBins - 1 ? -n64 : kBins - 1;
    }
};

// Some neighbouring pieces of the row, kThr pieces apart, of one thread.
template <int DT, int N>
struct Pieces {
    Piece<DT> v[N];
    int at;
    float least;
    // f(index, logit) for every token
    template <typename F>
    __device__ __forceinline__ void walk(F f)
    {
#pragma unroll
        for (int i = 0; i < N; ++i) {
#pragma unroll
            for (int e = 0; e < Piece<DT>::kN; ++e) f(uint32_t((at + i * kThr) * Piece<DT>::kN + e), v[i][e]);
        }
    }
    // the weights and their bins, 0 for tokens that cannot be taken: four at a time without branches, so that
    // one's table is read while another's series is formed
    template <bool PLAIN, typename F>
    __device__ __forceinline__ void weigh(const Row<DT>& r, const double* root, F f)
    {
#pragma unroll
        for (int i = 0; i < N; ++i) {
#pragma unroll
            for (int q = 0; q < Piece<DT>::kN; q += 4) {
                uint64_t w[4];
                int b[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float l = v[i][q + e];
                    w[e] = r.template weight<PLAIN>(PLAIN || l >= least ? l : 0.0f, root, &b[e]);
                    if (!PLAIN) w[e] = l >= least ? w[e] : 0;
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) f(w[e], b[e]);
            }
        }
    }
};
template <int DT>
struct Single {
    float l;
    int at;
    float least;
    template <typename F>
    __device__ __forceinline__ void walk(F f)
    {
        f(uint32_t(at), l);
    }
    template <bool PLAIN, typename F>
    __device__ __forceinline__ void weigh(const Row<DT>& r, const double* root, F f)
    {
        int b;
        const uint64_t w = r.weight(l >= least ? l : 0.0f, root, &b);
        f(l >= least ? w : 0, b);
    }
};

// Calls f with this thread's share of the row, some tokens at a time.
template <int DT, typename F>
__device__ __forceinline__ void each_few(const Row<DT>& r, F f)
{
    constexpr int kN = Piece<DT>::kN, kAhead = DT == 0 ? 4 : 2;
    const int whole = r.n / kN;
    auto load = [&](int at) { return Piece<DT>{*reinterpret_cast<const typename Piece<DT>::V*>(r.p + int64_t(at) * kN)}; };
    int at = threadIdx.x;
    for (; at + (kAhead - 1) * kThr < whole; at += kAhead * kThr) {
        Pieces<DT, kAhead> v;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) v.v[i] = load(at + i * kThr);
        v.at = at;
        v.least = r.least;
        f(v);
    }
#pragma unroll 1
    for (; at < whole; at += kThr) {
        Pieces<DT, 1> v{{load(at)}, at, r.least};
        f(v);
    }
    const int last = whole * kN + threadIdx.x;
    if (last < r.n) {
        Single<DT> v{Elem<DT>::load(r.p, last), last, r.least};
        f(v);
    }
}

// Calls f(index, logit) for every token of the row, this thread's share of them: for all, and for those
// that can be taken, not NaN and not -infinity.
template <int DT, typename F>
__device__ __forceinline__ void each_any(const Row<DT>& r, F f)
{
    each_few(r, [&](auto& v) { v.walk(f); });
}
template <int DT, typename F>
__device__ __forceinline__ void each(const Row<DT>& r, F f)
{
    each_any(r, [&](uint32_t i, float l) {
        if (l >= r.least) f(i, l);
    });
}

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

// Running sums of the bins' weights or counts, each thread's lying side by side.
template <bool MASS>
__device__ __forceinline__ void scan_bins(Shared& s)
{
    constexpr int kPer = kBins / kThr;
    uint64_t m = 0, mm[kPer] = {};
    uint32_t c = 0, cc[kPer] = {};
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (MASS) m += mm[i] = s.mass[threadIdx.x * kPer + i];
        else c += cc[i] = s.count[threadIdx.x * kPer + i];
    }
    uint64_t before_m = m;
    uint32_t before_c = c;
    block_scan(s, before_m, before_c);
    before_m -= m;
    before_c -= c;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (MASS) s.mass[threadIdx.x * kPer + i] = before_m += mm[i];
        else s.count[threadIdx.x * kPer + i] = before_c += cc[i];
    }
    __syncthreads();
}

// The sum of v over the workgroup.
__device__ __forceinline__ uint64_t block_sum(Shared& s, uint64_t v)
{
    uint32_t none = 0;
    block_scan(s, v, none);
    if (threadIdx.x == kThr - 1) s.found_mass = v;
    __syncthreads();
    return s.found_mass;
}

// The bins' running counts, or weights; returns the sum of the weights that are at least `least`, if that
// is not 0.
template <int DT, bool MASS>
__device__ __forceinline__ uint64_t fill_bins(Shared& s, const Row<DT>& r, uint64_t least)
{
    __syncthreads();
    for (int b = threadIdx.x; b < kBins; b += kThr) {
        if (MASS) s.mass[b] = 0;
        else s.count[b] = 0;
    }
    __syncthreads();
    uint64_t above = 0;
    if (MASS) {
        auto add = [&](uint64_t w, int b) {
            if (w) atomicAdd(reinterpret_cast<unsigned long long*>(&s.mass[b]), w);
            if (least) above += w >= least ? w : 0;
        };
        if (r.plain) each_few(r, [&](auto& v) { v.template weigh<true>(r, s.root, add); });
        else each_few(r, [&](auto& v) { v.template weigh<false>(r, s.root, add); });
    } else {
        each(r, [&](uint32_t, float l) { atomicAdd(&s.count[r.count_bin(l)], 1u); });
    }
    __syncthreads();
    scan_bins<MASS>(s);
    return MASS && least ? block_sum(s, above) : 0;
}

// The bin in whose running sum `target` falls.
template <bool MASS>
__device__ __forceinline__ int bin_of(Shared& s, uint64_t target)
{
    __syncthreads();
    for (int b = threadIdx.x; b < kBins; b += kThr) {
        const uint64_t before = b == 0 ? 0 : MASS ? s.mass[b - 1] : s.count[b - 1];
        const uint64_t upto = MASS ? s.mass[b] : s.count[b];
        if (before < target && target <= upto) s.found = uint32_t(b);
    }
    __syncthreads();
    return int(s.found);
}

// Copies the tokens whose logits lie in [from, to], which holds nothing that cannot be taken, to the list,
// and says whether they fit there.
template <int DT>
__device__ __forceinline__ bool make_list(Shared& s, const Row<DT>& r, float from, float to)
{
    if (threadIdx.x == 0) s.listed = 0;
    __syncthreads();
    // A wave's slots at a time: of at most 16 tokens a thread, the sums over the lanes before it by the bits
    // of their numbers.  One addition for each thread's takes the time of 64.
    each_few(r, [&](auto& v) {
        uint32_t n = 0;
        v.walk([&](uint32_t, float l) { n += l >= from && l <= to; });
        if (__ballot(n != 0) == 0) return;
        uint32_t slot = 0, all = 0;
#pragma unroll
        for (int b = 0; b < 5; ++b) {
            const uint64_t m = __ballot(n >> b & 1);
            slot += __builtin_amdgcn_mbcnt_hi(uint32_t(m >> 32), __builtin_amdgcn_mbcnt_lo(uint32_t(m), 0)) << b;
            all += uint32_t(__builtin_popcountll(m)) << b;
        }
        const uint64_t here = __ballot(true);
        uint32_t base = 0;
        if ((here & ((uint64_t(1) << (threadIdx.x & 63)) - 1)) == 0) base = atomicAdd(&s.listed, all);
        slot += __builtin_amdgcn_readfirstlane(base);
        if (n == 0) return;
        v.walk([&](uint32_t i, float l) {
            if (!(l >= from && l <= to)) return;
            if (slot < kList) {
                s.key[slot] = key_of(l);
                s.index[slot] = i;
            }
            ++slot;
        });
    });
    __syncthreads();
    return s.listed <= kList;
}
// The logit that lies `bins` bins below the largest, or, with up, one that is above it, else below, by what
// rounding may move a bin's border: lists may hold a few tokens more than their bins.
template <int DT, bool MASS>
__device__ __forceinline__ float border(const Row<DT>& r, int bins, bool up)
{
    if (r.pre == 0.0f) return INFINITY;
    // log2(e) / rate is T
    const double width = MASS ? 1.0 / 64 / r.rate : r.scale > 0.0f ? 1.0 / double(r.scale) : 0.0;
    const double l = (double(r.top) - bins * width) / double(r.pre), slack = (fabs(l) + fabs(double(r.top))) * 1e-6;
    if (up) return float(fmin(l + slack, 3.402823466e38));
    return bins >= kBins ? r.least : fmaxf(float(fmax(l - slack, -3.402823466e38)), r.least);
}

// A token, and the weights up to it in the order.
struct Place {
    uint32_t key, index;
    uint64_t mass;
};

// The place at which the count (or the weights) first reaches `target`, 1 <= target <= all, by the bins'
// running counts (or weights).  `listed`: the list holds the tokens that are left (a key of 0 there is one
// that is not); otherwise it is overwritten.  With counts, the weights up to the place are the caller's to find.
template <int DT, bool MASS>
__device__ __forceinline__ Place find(Shared& s, const Row<DT>& r, uint64_t target, bool listed)
{
    const int bin = bin_of<MASS>(s, target);
    // without a list of all that is left, one of the bin
    if (!listed) listed = make_list(s, r, border<DT, MASS>(r, bin + 1, false), border<DT, MASS>(r, bin - 1, true));
    uint64_t before = bin == 0 ? 0 : MASS ? s.mass[bin - 1] : s.count[bin - 1];
    // the tokens among which it lies: those of the bin whose key's bits from key_shift on are key_bits, and
    // the index's from index_shift on
    int key_shift = 32, index_shift = 32;
    uint32_t key_bits = 0, index_bits = 0;
    auto candidates = [&](auto f) {
        auto test = [&](uint32_t i, uint32_t k, float l) {
            if ((MASS ? r.weight_bin(l) : r.count_bin(l)) == bin && (key_shift == 32 || k >> key_shift == key_bits) &&
                (index_shift == 32 || i >> index_shift == index_bits))
                f(i, k, l);
        };
        if (listed) {
            const uint32_t n = s.listed;
            for (uint32_t j = threadIdx.x; j < n; j += kThr)
                if (s.key[j]) test(s.index[j], s.key[j], logit_of(s.key[j]));
        } else {
            each(r, [&](uint32_t i, float l) { test(i, key_of(l), l); });
        }
    };
    for (;;) {
        if (threadIdx.x == 0) s.few = 0;
        __syncthreads();
        candidates([&](uint32_t i, uint32_t k, float) {
            const uint32_t slot = atomicAdd(&s.few, 1u);
            if (slot < kFew) {
                s.few_key[slot] = k;
                s.few_index[slot] = i;
            }
        });
        __syncthreads();
        if (s.few <= kFew) break;
        // the next 8 bits of the key, larger ones first, then of the index, smaller ones first
        const bool by_key = key_shift > 0;
        const int shift = by_key ? key_shift - 8 : index_shift - 8;
        if (threadIdx.x < kRadix) s.rmass[threadIdx.x] = 0;
        __syncthreads();
        candidates([&](uint32_t i, uint32_t k, float l) {
            const uint32_t d = by_key ? 255u - (k >> shift & 255u) : i >> shift & 255u;
            int b;
            atomicAdd(reinterpret_cast<unsigned long long*>(&s.rmass[d]), MASS ? r.weight(l, s.root, &b) : 1ull);
        });
        __syncthreads();
        uint64_t m = threadIdx.x < kRadix ? s.rmass[threadIdx.x] : 0;
        uint32_t none = 0;
        const uint64_t own = m;
        block_scan(s, m, none);
        if (threadIdx.x < kRadix && before + m - own < target && target <= before + m) {
            s.found = threadIdx.x;
            s.found_mass = m - own;
        }
        __syncthreads();
        const uint32_t d = s.found;
        before += s.found_mass;
        if (by_key) {
            key_bits = key_bits << 8 | (255u - d);
            key_shift = shift;
        } else {
            index_bits = index_bits << 8 | d;
            index_shift = shift;
        }
        __syncthreads();
    }
    if (threadIdx.x < 64) {
        const int n = int(s.few), lane = threadIdx.x;
        const uint32_t k = lane < n ? s.few_key[lane] : 0, i = lane < n ? s.few_index[lane] : 0xffffffffu;
        int b;
        const uint64_t w = lane >= n ? 0 : MASS ? r.weight(logit_of(k), s.root, &b) : 1;
        const uint32_t wl = uint32_t(w), wh = uint32_t(w >> 32);
        for (int t = 0; t < n; ++t) {
            const uint32_t ok = __builtin_amdgcn_readlane(k, t), oi = __builtin_amdgcn_readlane(i, t);
            const uint64_t ow = uint64_t(uint32_t(__builtin_amdgcn_readlane(wh, t))) << 32 | uint32_t(__builtin_amdgcn_readlane(wl, t));
            before += ok > k || (ok == k && oi < i) ? ow : 0;
        }
        if (lane < n && before < target && target <= before + w) {
            s.found_key = k;
            s.found_index = i;
            s.found_mass = before + w;
        }
    }
    __syncthreads();
    return {s.found_key, s.found_index, s.found_mass};
}

// The list's running counts in place of the row's.
template <int DT>
__device__ __forceinline__ void count_list(Shared& s, const Row<DT>& r)
{
    __syncthreads();
    for (int b = threadIdx.x; b < kBins; b += kThr) s.count[b] = 0;
    __syncthreads();
    const uint32_t n = s.listed;
    for (uint32_t j = threadIdx.x; j < n; j += kThr)
        if (s.key[j]) atomicAdd(&s.count[r.count_bin(logit_of(s.key[j]))], 1u);
    __syncthreads();
    scan_bins<false>(s);
}

// Lists tokens among which the first `k` are, without counting the row: those that are at least the k-th of
// the threads' largest logits, `own`.  About -kThr ln(1 - k / kThr) of them, if the large ones lie anywhere.
// Says whether there are k threads with one and the tokens fit the list.
template <int DT>
__device__ __forceinline__ bool shortlist(Shared& s, const Row<DT>& r, float own, uint32_t k)
{
    __syncthreads();
    s.key[threadIdx.x] = own >= r.least ? key_of(own) : 0u;
    s.index[threadIdx.x] = threadIdx.x;
    if (threadIdx.x == 0) s.listed = kThr;
    count_list(s, r);
    if (s.count[kBins - 1] < k) return false;
    const Place at = find<DT, false>(s, r, k, true);
    if (!make_list(s, r, logit_of(at.key), INFINITY)) return false;
    count_list(s, r);
    return true;
}

// The sums of the weights, and of those that are at least `least`, up to a place.
template <int DT>
__device__ __forceinline__ void sums_upto(Shared& s, const Row<DT>& r, const Place& at, uint64_t least, uint64_t* all, uint64_t* above)
{
    uint64_t m = 0, a = 0;
    each(r, [&](uint32_t i, float l) {
        const uint32_t k = key_of(l);
        if (k > at.key || (k == at.key && i <= at.index)) {
            int b;
            const uint64_t v = r.weight(l, s.root, &b);
            m += v;
            a += v >= least ? v : 0;
        }
    });
    *all = block_sum(s, m);
    __syncthreads();
    *above = block_sum(s, a);
}

template <int DT>
__global__ __launch_bounds__(kThr) void sample_kernel(SampleArgs a)
{
    __shared__ Shared s;
    const int64_t row = blockIdx.x;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    Row<DT> r;
    r.p = static_cast<const typename Elem<DT>::T*>(a.logits) + row * a.ld;
    r.n = int(a.vocab);
    if (threadIdx.x < 64) s.root[threadIdx.x] = exp2(threadIdx.x / 64.0);

    // the largest logit and the smallest
    r.least = -3.402823466e38f;
    float top = -INFINITY, low = INFINITY;
    each_any(r, [&](uint32_t, float l) {
        top = fmaxf(top, l);  // neither takes NaN
        low = fminf(low, l > -INFINITY ? l : INFINITY);
    });
    const float own = top;  // this thread's largest
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        top = fmaxf(top, __shfl_xor(top, d));
        low = fminf(low, __shfl_xor(low, d));
    }
    if (lane == 0) {
        s.top[w] = top;
        s.low[w] = low;
    }
    __syncthreads();
    for (int i = 0; i < kThr / 64; ++i) {
        top = fmaxf(top, s.top[i]);
        low = fminf(low, s.low[i]);
    }
    const float t = a.temperature ? a.temperature[row] : a.temperature_all;
    if (top == -INFINITY || !(t > 0.0f)) {
        // none, or the first place of the largest
        uint32_t where = 0xffffffffu;
        if (threadIdx.x == 0) s.found = where;
        __syncthreads();
        each(r, [&](uint32_t i, float l) { where = l == top && i < where ? i : where; });
        if (where != 0xffffffffu) atomicMin(&s.found, where);
        __syncthreads();
        if (threadIdx.x == 0) a.token[row] = top == -INFINITY ? -1 : int64_t(s.found);
        return;
    }

    // differences of logits up to 2^126 are finite
    r.pre = fmaxf(fabsf(top), fabsf(low)) < 8.5e37f ? 1.0f : 0.25f;
    if (top == INFINITY) {
        r.least = INFINITY;
        r.pre = 0.0f;
        low = top;
    }
    r.top = r.value(top);
    const double td = r.pre > 0.0f ? double(t) * double(r.pre) : 1.0;
    r.rate = 1.4426950408889634 / td;
    // at 100 T below the largest logit, which rounding moves by less than half of that, or the next number
    // below it: less than 2^-70 of the largest weight
    r.floor = float(double(r.top) - 100.0 * td);
    if (!(r.floor < r.top)) r.floor = logit_of(key_of(r.top) - 1);
    r.plain = r.pre == 1.0f && (double(r.floor) - double(r.top)) * r.rate >= -1000.0;
    // a row's weights sum to less than 2^62, and each fits the 52 bits of a double
    const int bits = 32 - __builtin_clz(uint32_t(r.n));
    r.shift = 62 - bits < 50 ? 62 - bits : 50;
    const uint64_t first = uint64_t(1) << r.shift;
    // bins of counts over the logits that have a weight; the last one has those more than 64 T below the
    // largest, whose weights, below exp(-63), are less than half a unit too
    const float deep = float(fmin(double(r.top) - double(r.value(low)), 64.0 * td));
    r.scale = deep > 0.0f ? fminf(float(kBins - 2) / deep, 3.0e38f) : 0.0f;

    const int32_t k = a.top_k ? a.top_k[row] : a.top_k_all;
    const float min_p = a.min_p ? a.min_p[row] : a.min_p_all;
    const uint64_t least = min_p > 0.0f ? uint64_t(ceil(fmin(double(min_p), 2.0) * double(first))) : 0;
    bool listed = false;
    uint64_t above = 0;  // the weights that min_p leaves
    uint64_t all = 0;    // those that every limit so far leaves
    if (k > 0 && k < r.n) {
        // the bins' counts, and the last of the tokens that top_k leaves
        const bool few = k <= kThr / 8 * 7 && shortlist(s, r, own, uint32_t(k));
        if (!few) fill_bins<DT, false>(s, r, 0);
        const uint32_t can = s.count[kBins - 1];
        const uint32_t keep = uint32_t(k) < can ? uint32_t(k) : can;
        const int bin = bin_of<false>(s, keep);
        if (bin < kBins - 1) {  // otherwise what top_k drops has no weight
            if (few) listed = true;
            else if (s.count[bin] <= kList) listed = make_list(s, r, border<DT, false>(r, bin + 1, false), INFINITY);
            const Place at = find<DT, false>(s, r, keep, listed);
            if (listed) {
                // the bins' weights from the list, without those that top_k drops
                for (int b = threadIdx.x; b < kBins; b += kThr) s.mass[b] = 0;
                __syncthreads();
                for (uint32_t j = threadIdx.x; j < s.listed; j += kThr) {
                    const uint32_t key = s.key[j];
                    if (key < at.key || (key == at.key && s.index[j] > at.index)) {
                        s.key[j] = 0;
                    } else {
                        int b;
                        const uint64_t v = r.weight(logit_of(key), s.root, &b);
                        atomicAdd(reinterpret_cast<unsigned long long*>(&s.mass[b]), v);
                        above += v >= least ? v : 0;
                    }
                }
                __syncthreads();
                scan_bins<true>(s);
                all = s.mass[kBins - 1];
                above = block_sum(s, above);
            } else {
                sums_upto(s, r, at, least, &all, &above);
            }
        }
    }
    if (!listed) {
        const uint64_t sum = fill_bins<DT, true>(s, r, least);
        if (all == 0) {
            all = s.mass[kBins - 1];
            above = sum;
        }
    }
    const float p = a.top_p ? a.top_p[row] : a.top_p_all;
    if (p < 1.0f) {
        const double want = p > 0.0f ? ceil(double(p) * double(all)) : 1.0;
        uint64_t target = want > 1.0 ? uint64_t(want) : 1;
        target = target < all ? target : all;
        // what is left, to the list if it fits: the token is among it
        if (!listed) listed = make_list(s, r, border<DT, true>(r, bin_of<true>(s, target) + 1, false), INFINITY);
        all = find<DT, true>(s, r, target, listed).mass;
    }
    if (min_p > 0.0f) {
        const uint64_t kept = above > first ? above : first;
        all = kept < all ? kept : all;
    }
    const float u = a.u[row];
    const double pass = u > 0.0f ? floor(double(u) * double(all)) : 0.0;
    uint64_t target = pass < double(all) ? uint64_t(pass) + 1 : all;
    target = target < all ? target : all;
    const Place at = find<DT, true>(s, r, target, listed);
    if (threadIdx.x == 0) a.token[row] = at.index;
}

}  // namespace

hipError_t launch_sample(const SampleArgs& a, int dtype, hipStream_t stream)
{
    if (dtype == 0) sample_kernel<0><<<uint32_t(a.rows), kThr, 0, stream>>>(a);
    else sample_kernel<1><<<uint32_t(a.rows), kThr, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace ssk
