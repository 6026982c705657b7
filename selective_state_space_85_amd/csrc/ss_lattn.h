// gfx950 kernel of linear attention with a decay for each head.  With a = exp(log_decay[h]):
//   S_t = a S_{t-1} + k_t v_t^T,   o_t = S_t^T q_t
// taken a chunk of C rows at a time.  With S the state before the chunk, rows t, s of it and
// a^(t - s) for s <= t:
//   o_t = sum_s a^(t - s) (q_t . k_s) v_s + a^(t + 1) S^T q_t
//   S  <- a^C S + sum_s a^(C - 1 - s) k_s v_s^T
// so the work is dense products on the matrix cores; the decays only ever multiply, never divide.
//
// One workgroup walks one (batch row, head, slice of v's columns); each wave owns 32 columns of v
// and holds their part of the state, dk x 32, in fp32 accumulators for the whole walk.  Everything
// is formed transposed, so that accumulators feed the next product without leaving registers:
//   P^T = K Q^T      (s x t; one 32 x 32 block per wave, exchanged through LDS)
//   O^T = S^T Q^T, times a^(t + 1), + V^T P^T     (v columns x t)
//   S   = a^C S + K^T (w V)
// A block of the state in accumulators (rows dk, columns v) is the operand S^T as it stands, up to
// a swap between the halves of a wave (bf16) or as it is (fp32).
//
// Resets cut the sequence: row t sees the rows from the last reset up to t, and the state only if
// none lies in the chunk before or at t.  A chunk's resets are one 64-bit mask.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "ss_attn_internal.h"

namespace ssk {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
// two values rounded to bf16 by one conversion, a in the low half
__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, bf16x2{__bf16(a), __bf16(b)});
}

// What a product of 32 x 32 blocks needs of an element type.  A fragment holds kDepth indices of the
// contraction for 32 rows (or columns) of an operand: lane l has row l % 32 and, of the kDepth
// indices, the kDepth / 2 ones from (l / 32) * kDepth / 2.
template <int DT>
struct Ops;

template <>
struct Ops<1> {  // bf16
    using E = uint16_t;
    using Frag = bf16x8;
    static constexpr int kDepth = 16;
    static constexpr int kEpc = 8;  // elements per 16 bytes
    static __device__ __forceinline__ f32x16 mma(const Frag& a, const Frag& b, const f32x16& c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
    // contraction along a row of LDS: p is this lane's row at its first index
    static __device__ __forceinline__ Frag row(const E* p) { return *reinterpret_cast<const Frag*>(p); }
    // contraction down the columns: rows from `base`, column lane % 32.  Within a group of 16 lanes the
    // transpose read gives lane i, as its element k, element i % 4 of the 4-vector that lane 4 k + i / 4
    // addresses.
    static __device__ __forceinline__ Frag col(const E* base, int pitch, int lane)
    {
        typedef __attribute__((address_space(3))) s16x4* lds_ptr;
        const int j = lane & 15, g = lane >> 4;
        const E* p = base + (8 * (g >> 1) + (j >> 2)) * pitch + 16 * (g & 1) + 4 * (j & 3);
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)p);
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p + 4 * pitch));
        return __builtin_bit_cast(Frag, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
    // rows [kDepth u, kDepth u + kDepth) of an accumulator block as a fragment, each value rounded to
    // bf16.  Registers 8 u .. 8 u + 3 hold rows 0-3 (lower half of the wave) and 4-7 (upper half) of
    // these 16, the next four 8-11 and 12-15: one swap of halves gives the lower half 0-7, the upper 8-15.
    static __device__ __forceinline__ Frag from_acc(const f32x16& c, int u)
    {
        u32x4 r;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t x = pack_bf16(c[8 * u + 2 * i], c[8 * u + 2 * i + 1]);
            const uint32_t y = pack_bf16(c[8 * u + 4 + 2 * i], c[8 * u + 4 + 2 * i + 1]);
            const auto s = __builtin_amdgcn_permlane32_swap(x, y, false, false);
            r[i] = s[0];
            r[2 + i] = s[1];
        }
        return __builtin_bit_cast(Frag, r);
    }
    // acc += a (w . v): the weighted rows in three bf16 parts, each the rounding of what the ones
    // before it leave, so that the state keeps fp32's 24 bits
    static __device__ __forceinline__ void split(const Frag& v, const float (&w)[8], Frag (&part)[3])
    {
        const u32x4 u = __builtin_bit_cast(u32x4, v);
        u32x4 p[3];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float x = bf_lo(u[i]) * w[2 * i], y = bf_hi(u[i]) * w[2 * i + 1];
#pragma unroll
            for (int q = 0; q < 3; ++q) {
                p[q][i] = pack_bf16(x, y);
                x -= bf_lo(p[q][i]);
                y -= bf_hi(p[q][i]);
            }
        }
#pragma unroll
        for (int q = 0; q < 3; ++q) part[q] = __builtin_bit_cast(Frag, p[q]);
    }
    static constexpr int kParts = 3;
    // bits set where one of the fragment's elements is infinite or NaN
    static __device__ __forceinline__ uint32_t not_finite(const Frag& v)
    {
        const u32x4 u = __builtin_bit_cast(u32x4, v);
        uint32_t bad = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) bad |= (u[i] & 0x7f807f80u) + 0x00800080u;
        return bad & 0x80008000u;
    }
    // the fragment with those elements zeroed
    static __device__ __forceinline__ Frag finite_part(const Frag& v)
    {
        u32x4 u = __builtin_bit_cast(u32x4, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t e = u[i] & 0x7f807f80u;
            u[i] &= ((e & 0xffffu) == 0x7f80u ? 0u : 0xffffu) | (e >= 0x7f800000u ? 0u : 0xffff0000u);
        }
        return __builtin_bit_cast(Frag, u);
    }
    // the fragment with the elements of the lane's indices below `from` zeroed
    static __device__ __forceinline__ Frag drop_below(const Frag& v, int index, int from)
    {
        u32x4 u = __builtin_bit_cast(u32x4, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (index + 2 * i < from) u[i] &= 0xffff0000u;
            if (index + 2 * i + 1 < from) u[i] &= 0x0000ffffu;
        }
        return __builtin_bit_cast(Frag, u);
    }
    static __device__ __forceinline__ float widen(E v) { return __uint_as_float(uint32_t(v) << 16); }
    static __device__ __forceinline__ void store4(E* p, const float (&v)[4])
    {
        *reinterpret_cast<u32x2*>(p) = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    }
    static __device__ __forceinline__ void store1(E* p, float v) { *p = __builtin_bit_cast(uint16_t, __bf16(v)); }
};

template <>
struct Ops<0> {  // fp32: the fp32 matrix instruction, four of them to a fragment
    using E = float;
    using Frag = f32x4;
    static constexpr int kDepth = 8;
    static constexpr int kEpc = 4;
    static __device__ __forceinline__ f32x16 mma(const Frag& a, const Frag& b, f32x16 c)
    {
#pragma unroll
        for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[e], b[e], c, 0, 0, 0);
        return c;
    }
    static __device__ __forceinline__ Frag row(const E* p) { return *reinterpret_cast<const Frag*>(p); }
    static __device__ __forceinline__ Frag col(const E* base, int pitch, int lane)
    {
        const E* p = base + 4 * (lane >> 5) * pitch + (lane & 31);
        return Frag{p[0], p[pitch], p[2 * pitch], p[3 * pitch]};
    }
    // accumulator registers 4 u .. 4 u + 3 hold rows 8 u .. 8 u + 3 in the lower half, the next in the upper
    static __device__ __forceinline__ Frag from_acc(const f32x16& c, int u)
    {
        return Frag{c[4 * u], c[4 * u + 1], c[4 * u + 2], c[4 * u + 3]};
    }
    static constexpr int kParts = 1;
    static __device__ __forceinline__ void split(const Frag& v, const float (&w)[4], Frag (&part)[1])
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) part[0][i] = v[i] * w[i];
    }
    static __device__ __forceinline__ uint32_t not_finite(const Frag& v)
    {
        uint32_t bad = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) bad |= (__float_as_uint(v[i]) & 0x7f800000u) + 0x00800000u;
        return bad & 0x80000000u;
    }
    static __device__ __forceinline__ Frag finite_part(Frag v)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if ((__float_as_uint(v[i]) & 0x7f800000u) == 0x7f800000u) v[i] = 0.0f;
        return v;
    }
    static __device__ __forceinline__ Frag drop_below(Frag v, int index, int from)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (index + i < from) v[i] = 0.0f;
        return v;
    }
    static __device__ __forceinline__ float widen(E v) { return v; }
    static __device__ __forceinline__ void store4(E* p, const float (&v)[4])
    {
        *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
    }
    static __device__ __forceinline__ void store1(E* p, float v) { *p = v; }
};

// 16 bytes of a row: elements [c, c + kEpc) of `width`, zero past its end.  VEC: the host has checked
// that rows are whole 16-byte chunks.
template <int DT, bool VEC>
__device__ __forceinline__ u32x4 load_piece(const typename Ops<DT>::E* row, int c, int width, bool live)
{
    constexpr int kEpc = Ops<DT>::kEpc;
    if constexpr (VEC) {
        // no branch: a lane without elements reads the row's first ones and drops them
        const bool in = live && c < width;
        const u32x4 v = *reinterpret_cast<const u32x4*>(row + (in ? c : 0));
        const uint32_t keep = in ? 0xffffffffu : 0u;
        return u32x4{v[0] & keep, v[1] & keep, v[2] & keep, v[3] & keep};
    } else {
        union {
            u32x4 v;
            typename Ops<DT>::E e[kEpc];
        } p;
        p.v = u32x4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < kEpc; ++i)
            if (live && c + i < width) p.e[i] = row[c + i];
        return p.v;
    }
}

// The geometry of one instantiation.  Rows in LDS are padded by 16 bytes.
template <int DT, int DKP, int NW>
struct LattnShape {
    static constexpr int kThreads = 64 * NW;
    // fp32 rows of 256 elements: half a chunk at a time fits the LDS
    static constexpr int kC = DT == 0 && DKP == 256 ? 32 : 64;
    static constexpr int kPad = Ops<DT>::kEpc;
    static constexpr int kKP = DKP + kPad;       // pitch of q and k rows
    static constexpr int kVP = 32 * NW + kPad;   // of v rows
    static constexpr int kPP = kC + kPad;        // of P rows
    static constexpr int kQPieces = kC * DKP / Ops<DT>::kEpc / kThreads;
    static constexpr int kVPieces = kC * 32 * NW / Ops<DT>::kEpc / kThreads;
};

// grid (slices * heads * batch * segments, jobs), slices fastest.
// STATE: forms what each segment leaves in the state, from zero, and nothing else.
template <int DT, int DKP, int NW, bool VEC, bool STATE>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(DT == 0 || DKP == 256 ? 1 : 2))) void lattn_kernel(LattnArgs a)
{
    using O = Ops<DT>;
    using E = typename O::E;
    using Frag = typename O::Frag;
    using G = LattnShape<DT, DKP, NW>;
    constexpr int C = G::kC, kTB = C / 32, kDB = DKP / 32, kDepth = O::kDepth, kHalf = kDepth / 2;
    constexpr int kKS = C / kDepth, kSub = 32 / kDepth;

    __shared__ __align__(16) E sQ[STATE ? 1 : C][G::kKP];
    __shared__ __align__(16) E sK[C][G::kKP];
    __shared__ __align__(16) E sV[C][G::kVP];
    __shared__ __align__(16) E sP[STATE ? 1 : C][G::kPP];
    __shared__ float s_pow[C + 1];      // a^j
    __shared__ float s_leave[2 * C];    // in_scale a^(C - 1 - x), 0 past C

    const LattnJob& j = a.job[blockIdx.y];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, l32 = lane & 31, hl = lane >> 5;
    const int slices = (j.dv + kLattnSlice - 1) / kLattnSlice;
    uint32_t x = blockIdx.x;
    const int v0 = int(x % uint32_t(slices)) * kLattnSlice;
    x /= uint32_t(slices);
    const int64_t H = a.heads, L = a.seqlen;
    const int64_t h = x % uint32_t(H);
    x /= uint32_t(H);
    const int64_t b = x % uint32_t(a.batch), seg = x / uint32_t(a.batch);
    const int64_t row0 = seg * a.seg_len, row1 = row0 + a.seg_len < L ? row0 + a.seg_len : L;
    const int64_t bh = b * H + h, cells = int64_t(j.dk) * j.dv;

    // powers of the decay, in 64 bits: they stand for the whole walk
    const double log_a = double(a.log_decay[h]);
    for (int i = tid; i <= C; i += G::kThreads) s_pow[i] = i == 0 ? 1.0f : float(exp(log_a * i));
    for (int i = tid; i < 2 * C; i += G::kThreads)
        s_leave[i] = i >= C ? 0.0f : i == C - 1 ? j.in_scale : float(exp(log_a * (C - 1 - i)) * double(j.in_scale));

    const E* const pq = static_cast<const E*>(j.q) + b * L * j.q_ld + (h / j.q_share) * j.dk;
    const E* const pk = static_cast<const E*>(j.k) + b * L * j.k_ld + (h / j.k_share) * j.dk;
    const E* const pv = static_cast<const E*>(j.v) + b * L * j.v_ld + (h / j.v_share) * j.dv + v0;
    const int vw = j.dv - v0;  // columns from here on
    const uint8_t* const pr = a.reset ? a.reset + b * L : nullptr;
    const bool rev = j.rev;
    auto token = [&](int64_t r) { return rev ? L - 1 - r : r; };

    // this wave's columns of v, and whether it has any
    const int c0 = 32 * w;
    const bool mine = c0 < vw;

    // ---- the state before the first row ----
    f32x16 st[kDB];
    const bool from_seg = a.segs > 1 && !STATE;
    const float* const h0 = STATE ? nullptr : from_seg ? j.seg + (seg * a.batch * H + bh) * cells : j.h0 ? j.h0 + bh * cells : nullptr;
    const int64_t si = from_seg ? j.dv : j.si, sj = from_seg ? 1 : j.sj;
#pragma unroll
    for (int d = 0; d < kDB; ++d) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int i = 32 * d + 8 * (r >> 2) + 4 * hl + (r & 3);
            st[d][r] = h0 && i < j.dk && c0 + l32 < vw ? h0[i * si + (v0 + c0 + l32) * sj] : 0.0f;
        }
    }

    // ---- a chunk's operands, loaded one chunk ahead ----
    u32x4 fq[STATE ? 1 : G::kQPieces], fk[G::kQPieces], fv[G::kVPieces];
    uint32_t flag = 0;
    auto issue = [&](int64_t t0) {
#pragma unroll
        for (int i = 0; i < G::kQPieces; ++i) {
            const int p = tid + G::kThreads * i, r = p / (DKP / O::kEpc), c = p % (DKP / O::kEpc) * O::kEpc;
            const bool live = t0 + r < row1;
            const int64_t t = live ? token(t0 + r) : 0;
            if constexpr (!STATE) fq[i] = load_piece<DT, VEC>(pq + t * j.q_ld, c, j.dk, live);
            fk[i] = load_piece<DT, VEC>(pk + t * j.k_ld, c, j.dk, live);
        }
#pragma unroll
        for (int i = 0; i < G::kVPieces; ++i) {
            const int p = tid + G::kThreads * i, r = p / (32 * NW / O::kEpc), c = p % (32 * NW / O::kEpc) * O::kEpc;
            const bool live = t0 + r < row1;
            const int64_t t = live ? token(t0 + r) : 0;
            fv[i] = load_piece<DT, VEC>(pv + t * j.v_ld, c, vw, live);
        }
        // whether the state of the row before is dropped on the way to this row: from the end, the
        // reset is the one of the row that was walked before
        flag = 0;
        if (pr) {
            const int64_t r = t0 + lane, t = rev ? L - r : r;
            if (lane < C && r < row1 && t < L) flag = pr[t];
        }
    };

    // decays between this lane's rows of P^T (s) and its column (t): the same in every chunk.  Blocks
    // of P^T: 0 is (s 0-31, t 0-31), 1 is (s 0-31, t 32-63), 2 is (s 32-63, t 32-63).
    constexpr int kBlocks = kTB == 2 ? 3 : 1;
    const bool diag = w != 1 || kTB == 1;
    float pair[16];
    __syncthreads();
    if constexpr (!STATE) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int gap = l32 - (8 * (r >> 2) + 4 * hl + (r & 3)) + (diag ? 0 : 32);
            pair[r] = gap >= 0 ? s_pow[gap] * j.pair_scale : 0.0f;
        }
    }

    issue(row0);
    bool cut = false;  // STATE: whether a reset lies in the segment
    for (int64_t t0 = row0; t0 < row1; t0 += C) {
        const int n = int(row1 - t0 < C ? row1 - t0 : C);  // rows of this chunk
        // ---- the chunk into LDS, the next one's loads on their way ----
#pragma unroll
        for (int i = 0; i < G::kQPieces; ++i) {
            const int p = tid + G::kThreads * i, r = p / (DKP / O::kEpc), c = p % (DKP / O::kEpc) * O::kEpc;
            if constexpr (!STATE) *reinterpret_cast<u32x4*>(&sQ[r][c]) = fq[i];
            *reinterpret_cast<u32x4*>(&sK[r][c]) = fk[i];
        }
#pragma unroll
        for (int i = 0; i < G::kVPieces; ++i) {
            const int p = tid + G::kThreads * i, r = p / (32 * NW / O::kEpc), c = p % (32 * NW / O::kEpc) * O::kEpc;
            *reinterpret_cast<u32x4*>(&sV[r][c]) = fv[i];
        }
        const uint64_t resets = __ballot(flag != 0);
        const int last = resets ? 63 - __builtin_clzll(resets) : 0;  // the last reset's row: what is before leaves nothing
        if (t0 + C < row1) issue(t0 + C);
        __syncthreads();

        // the state of the row before the chunk reaches its first row undecayed if it is the gradient
        // that the last row's state has from outside
        const int e0 = rev && t0 == 0 ? 0 : 1;

        f32x16 o[kTB];
        if constexpr (!STATE) {
            // ---- P^T = K Q^T with its decays, into LDS as P (t, s) ----
#pragma unroll
            for (int blk = 0; blk < kBlocks; ++blk) {
                if (blk % NW != w) continue;
                const int sb = blk == 2 ? 32 : 0, tb = blk == 0 ? 0 : 32;
                f32x16 p;
#pragma unroll
                for (int r = 0; r < 16; ++r) p[r] = 0.0f;
#pragma unroll
                for (int d = 0; d < DKP / kDepth; ++d)
                    p = O::mma(O::row(&sK[sb + l32][d * kDepth + kHalf * hl]), O::row(&sQ[tb + l32][d * kDepth + kHalf * hl]), p);
                const int t = tb + l32;
                // the first row that row t sees
                const uint64_t upto = resets & (~uint64_t(0) >> (63 - t));
                const int from = upto ? 63 - __builtin_clzll(upto) : 0;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int s = sb + 8 * q + 4 * hl;
                    float v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        v[e] = s + e <= t && s + e >= from ? p[4 * q + e] * pair[4 * q + e] : 0.0f;
                    O::store4(&sP[t][s], v);
                }
            }
            // ---- O^T = S^T Q^T ----
            if (mine) {
#pragma unroll
                for (int tb = 0; tb < kTB; ++tb) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) o[tb][r] = 0.0f;
                }
#pragma unroll
                for (int d = 0; d < kDB; ++d) {
#pragma unroll
                    for (int u = 0; u < kSub; ++u) {
                        const Frag s = O::from_acc(st[d], u);
#pragma unroll
                        for (int tb = 0; tb < kTB; ++tb)
                            o[tb] = O::mma(s, O::row(&sQ[32 * tb + l32][32 * d + kDepth * u + kHalf * hl]), o[tb]);
                    }
                }
#pragma unroll
                for (int tb = 0; tb < kTB; ++tb) {
                    const int t = 32 * tb + l32;
                    const bool sees = (resets & (~uint64_t(0) >> (63 - t))) == 0;
                    const float f = s_pow[t + e0] * j.out_scale;
#pragma unroll
                    for (int r = 0; r < 16; ++r) o[tb][r] = sees ? o[tb][r] * f : 0.0f;
                }
            }
            __syncthreads();
        }

        if (mine) {
            Frag vf[kKS];
            uint32_t bad = 0;
#pragma unroll
            for (int ks = 0; ks < kKS; ++ks) {
                vf[ks] = O::col(&sV[ks * kDepth][c0], G::kVP, lane);
                bad |= O::not_finite(vf[ks]);
            }
            if constexpr (!STATE) {
                // ---- O^T += V^T P^T ----
                // a row must not meet an infinity or NaN that it does not see, not even times 0: these are
                // left out of the product and added where they are seen
                const bool odd = __ballot(bad != 0) != 0;
#pragma unroll
                for (int ks = 0; ks < kKS; ++ks) {
                    Frag v = vf[ks];
                    if (odd) v = O::finite_part(v);
#pragma unroll
                    for (int tb = 0; tb < kTB; ++tb)
                        if (ks < (tb + 1) * kSub)
                            o[tb] = O::mma(v, O::row(&sP[32 * tb + l32][ks * kDepth + kHalf * hl]), o[tb]);
                }
                if (odd) {
#pragma unroll
                    for (int tb = 0; tb < kTB; ++tb) {
                        const int t = 32 * tb + l32;
                        const uint64_t upto = resets & (~uint64_t(0) >> (63 - t));
                        const int from = upto ? 63 - __builtin_clzll(upto) : 0;
#pragma unroll 1
                        for (int s = 0; s < 32 * (tb + 1); ++s) {
                            const bool sees = s <= t && s >= from;
                            const float p = O::widen(sP[t][s]);
#pragma unroll
                            for (int r = 0; r < 16; ++r) {
                                const float v = O::widen(sV[s][c0 + 8 * (r >> 2) + 4 * hl + (r & 3)]);
                                o[tb][r] += sees && !(fabsf(v) < INFINITY) ? p * v : 0.0f;
                            }
                        }
                    }
                }
                // ---- store: lane (t, 4 columns at a time) ----
#pragma unroll
                for (int tb = 0; tb < kTB; ++tb) {
                    const int t = 32 * tb + l32;
                    if (t >= n) continue;
                    const int64_t at = ((b * L + token(t0 + t)) * H + h) * j.dv + v0;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int c = c0 + 8 * q + 4 * hl;
                        const float v[4] = {o[tb][4 * q], o[tb][4 * q + 1], o[tb][4 * q + 2], o[tb][4 * q + 3]};
                        if (VEC) {
                            if (c < vw) {
                                if (j.out_f32) Ops<0>::store4(static_cast<float*>(j.out) + at + c, v);
                                else O::store4(static_cast<E*>(j.out) + at + c, v);
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                if (c + e >= vw) continue;
                                if (j.out_f32) static_cast<float*>(j.out)[at + c + e] = v[e];
                                else O::store1(static_cast<E*>(j.out) + at + c + e, v[e]);
                            }
                        }
                    }
                }
            }

            // ---- S = a^n S + K^T (w V) ----
            const float f = resets ? 0.0f : s_pow[n - 1 + e0];
#pragma unroll
            for (int d = 0; d < kDB; ++d) {
#pragma unroll
                for (int r = 0; r < 16; ++r) st[d][r] = resets ? 0.0f : st[d][r] * f;
            }
#pragma unroll
            for (int ks = 0; ks < kKS; ++ks) {
                float wt[kHalf];
#pragma unroll
                for (int i = 0; i < kHalf; ++i) wt[i] = s_leave[ks * kDepth + kHalf * hl + i + C - n];
                Frag v = vf[ks];
                if (resets) v = O::drop_below(v, ks * kDepth + kHalf * hl, last);
                Frag part[O::kParts];
                O::split(v, wt, part);
#pragma unroll
                for (int d = 0; d < kDB; ++d) {
                    Frag k = O::col(&sK[ks * kDepth][32 * d], G::kKP, lane);
                    if (resets) k = O::drop_below(k, ks * kDepth + kHalf * hl, last);
#pragma unroll
                    for (int q = O::kParts - 1; q >= 0; --q) st[d] = O::mma(k, part[q], st[d]);
                }
            }
        }
        cut |= resets != 0;
        __syncthreads();
    }

    if constexpr (STATE) {
        if (v0 == 0 && tid == 0) {
            const int64_t n = row1 - row0 - (rev && row0 == 0 ? 1 : 0);
            j.keep[seg * a.batch * H + bh] = cut ? -1.0f : n == 0 ? 1.0f : float(exp(log_a * double(n)));
        }
    }
    // ---- the state after the last row ----
    float* out = nullptr;
    int64_t oi = j.dv, oj = 1;
    float f = 1.0f;
    if (STATE) {
        out = j.seg + (seg * a.batch * H + bh) * cells;
    } else if (j.h_last && seg == a.segs - 1) {
        out = j.h_last + bh * cells;
        oi = j.si;
        oj = j.sj;
        if (rev) f = pr && pr[0] ? -1.0f : s_pow[1];
    }
    if (out && mine) {
#pragma unroll
        for (int d = 0; d < kDB; ++d) {
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int i = 32 * d + 8 * (r >> 2) + 4 * hl + (r & 3);
                if (i < j.dk && c0 + l32 < vw) out[i * oi + (v0 + c0 + l32) * oj] = f < 0.0f ? 0.0f : st[d][r] * f;
            }
        }
    }
}

template <int DT, int DKP, int NW, bool VEC>
hipError_t launch_shape(const LattnArgs& a, hipStream_t stream)
{
    const int64_t blocks = lattn_slices(a.job[0].dv) * a.heads * a.batch * a.segs;
    const dim3 grid(static_cast<uint32_t>(blocks), static_cast<uint32_t>(a.jobs)), block(64 * NW);
    if (a.segs > 1) {
        lattn_kernel<DT, DKP, NW, VEC, true><<<grid, block, 0, stream>>>(a);
        if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
        if (hipError_t e = launch_lattn_join(a, stream); e != hipSuccess) return e;
    }
    lattn_kernel<DT, DKP, NW, VEC, false><<<grid, block, 0, stream>>>(a);
    return hipGetLastError();
}

// Jobs of one launch have the same widths up to the padding that chooses the instantiation.
template <int DT>
hipError_t launch_typed(const LattnArgs& a, bool vec, hipStream_t stream)
{
    const int dk = a.job[0].dk, dv = a.job[0].dv;
    auto go = [&](auto dkp, auto nw) {
        constexpr int kD = decltype(dkp)::value, kW = decltype(nw)::value;
        return vec ? launch_shape<DT, kD, kW, true>(a, stream) : launch_shape<DT, kD, kW, false>(a, stream);
    };
    using std::integral_constant;
    auto by_dv = [&](auto dkp) {
        return dv <= 64 ? go(dkp, integral_constant<int, 2>()) : go(dkp, integral_constant<int, 4>());
    };
    return dk <= 64 ? by_dv(integral_constant<int, 64>())
                    : dk <= 128 ? by_dv(integral_constant<int, 128>()) : by_dv(integral_constant<int, 256>());
}

}  // namespace
}  // namespace ssk
