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
// a swap between the halves of a wave.  In bf16, S and P are rounded where they become operands: of the
// output that leaves a relative error of 0.0023 with the rounding of the output itself, 0.0017 alone.  As two
// bf16 parts each they leave that alone, in mostly 13-43% more time: 8 x 2048 x 40 heads of 128 forward 237 -> 288 us
// and backward 481 -> 580, 131072 x 16 heads 758 -> 860, 8 x 2048 x 32 heads of 64 forward 95 -> 123 (S alone in
// two parts 259, 530, 811 and 97, P alone 259, 527, 803 and 119).  What is rounded there is gone with its row;
// w V goes in as three bf16 parts, since what is rounded on its way into the state would stay there.
//
// Resets cut the sequence: row t sees the rows from the last reset up to t, and the state only if
// none lies in the chunk before or at t.  A chunk's resets are one 64-bit mask.
//
// What bounds it: with heads of 128 and 64 rows in bf16 a wave has 82 matrix instructions of 32 cycles
// to a chunk, some 560 vector instructions beside them, and some 80 KB of LDS traffic
// to the wave.  Two workgroups on a CU take 7-9 us for a chunk each at the 1.75-2.05 GHz that the card then runs at,
// of which the matrix cores are busy 36-38% and vector instructions are issued in 40%.  bf16, heads of 128:
//   131072 x 16 heads, forward: states between segments 242-333 us (1.07 GB read, 3.2-4.4 TB/s), joined 15,
//     main pass 457-612 (2.15 GB, 3.5-4.7 TB/s)
//   8 x 2048 x 40 heads: forward 206-234 us, 320 walks on 256 CUs (256 of them, of 32 heads: 130-156); gradients,
//     960 walks in one launch, 409-471 us; queries and keys shared by four heads: 726-802, and 2 x 86 for the sums
// fp32, 3 x 1021 x 12 heads of 72 and 91: 16 + 7 + 33 us forward, 29 + 10 + 74 + 10 for the gradients.
// Tried and not kept in bf16: chunks of 32 rows with three workgroups on a CU (28 registers in memory: 8 x
// 2048 x 32 heads 141 -> 285 us) or with two (141 -> 153), rows padded by 32 bytes more in LDS, loads before
// the barrier instead of among the products, P's products among those of S.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>
#include <utility>

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

__device__ __forceinline__ float masked(float v, uint32_t mask) { return __uint_as_float(__float_as_uint(v) & mask); }
// The same by the instruction's name, for values that no matrix instruction wrote: where a half of the
// result is used by itself too, the compiler would convert it a second time.
__device__ __forceinline__ uint32_t pack_named(float a, float b)
{
    uint32_t r;
    asm("v_cvt_pk_bf16_f32 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}

// What a product of 32 x 32 blocks needs of an element type.  A fragment holds 16 indices of the
// contraction for 32 rows (or columns) of an operand: lane l has row l % 32 and, of the 16 indices, the
// 8 from l / 32 * 8.
template <int DT>
struct Ops;

template <>
struct Ops<1> {  // bf16
    using E = uint16_t;
    using Frag = bf16x8;   // an operand of a product
    using VFrag = bf16x8;  // a fragment of v as it is
    static constexpr int kEpc = 8;  // elements per 16 bytes
    static __device__ __forceinline__ f32x16 mma(const Frag& a, const Frag& b, const f32x16& c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
    // blocks of 16 x 16: fragments of 32 indices, lane l has row l % 16 and 8 indices from l / 16 * 8; of the
    // result rows l / 16 * 4 .. + 3 of column l % 16
    static __device__ __forceinline__ f32x4 mma16(const Frag& a, const Frag& b, const f32x4& c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
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
    static __device__ __forceinline__ VFrag vcol(const E* base, int pitch, int lane) { return col(base, pitch, lane); }
    static __device__ __forceinline__ Frag operand(const VFrag& v) { return v; }
    // rows of q, k or P in LDS
    template <int R, int P>
    struct Tile {
        E m[R][P];
        __device__ __forceinline__ void put(int r, int c, const u32x4& v) { *reinterpret_cast<u32x4*>(&m[r][c]) = v; }
        __device__ __forceinline__ Frag row(int r, int c) const { return Ops::row(&m[r][c]); }
        __device__ __forceinline__ Frag col(int r, int c, int lane) const { return Ops::col(&m[r][c], P, lane); }
        __device__ __forceinline__ float value(int r, int c) const { return widen(m[r][c]); }
        // 4 values that no matrix instruction wrote, each under a mask
        __device__ __forceinline__ void store4(int r, int c, const float (&v)[4], const uint32_t (&k)[4])
        {
            *reinterpret_cast<u32x2*>(&m[r][c]) = u32x2{pack_named(masked(v[0], k[0]), masked(v[1], k[1])),
                                                        pack_named(masked(v[2], k[2]), masked(v[3], k[3]))};
        }
    };
    // rows [16 u, 16 u + 16) of an accumulator block as a fragment, each value rounded to
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
    // Rows of v times their weights, in three bf16 parts, each the rounding of what the ones before it
    // leave, so that the state keeps fp32's 24 bits.  In kSteps steps of a few instructions, for the
    // places between products; step i does part i % 3 of elements 2 (i / 3) and 2 (i / 3) + 1.
    static constexpr int kSteps = 12;
    struct Weighing {
        float x, y;
    };
    template <int I>
    static __device__ __forceinline__ void weigh(const Frag& v, const float* w, Frag (&part)[3], Weighing& s)
    {
        constexpr int q = I % 3, i = I / 3;
        const uint32_t u = __builtin_bit_cast(u32x4, v)[i];
        if constexpr (q == 0) {
            s.x = bf_lo(u) * w[2 * i];
            s.y = bf_hi(u) * w[2 * i + 1];
        }
        const uint32_t r = pack_named(s.x, s.y);
        s.x -= bf_lo(r);
        s.y -= bf_hi(r);
        u32x4 p = __builtin_bit_cast(u32x4, part[q]);
        p[i] = r;
        part[q] = __builtin_bit_cast(Frag, p);
    }
    static constexpr int kParts = 3;
    // whether an element of column lane % 32 is infinite or NaN: times a matrix of zeros, they leave NaN
    template <int N>
    static __device__ __forceinline__ bool not_finite(const VFrag (&v)[N])
    {
        const Frag zero = __builtin_bit_cast(Frag, u32x4{0, 0, 0, 0});
        f32x16 c;
#pragma unroll
        for (int r = 0; r < 16; ++r) c[r] = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) c = mma(zero, v[i], c);
        return !(c[0] == 0.0f);
    }
    // the fragment with those elements zeroed
    static __device__ __forceinline__ Frag finite_part(const Frag& v, uint32_t ones)
    {
        u32x4 u = __builtin_bit_cast(u32x4, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t e = u[i] & 0x7f807f80u;
            u[i] &= ((e & 0xffffu) == 0x7f80u ? 0u : ones & 0xffffu) | (e >= 0x7f800000u ? 0u : ones & 0xffff0000u);
        }
        return __builtin_bit_cast(Frag, u);
    }
    // the fragment with the elements of the lane's indices below `from` zeroed
    static __device__ __forceinline__ Frag drop_below(const Frag& v, int index, int from, uint32_t ones)
    {
        u32x4 u = __builtin_bit_cast(u32x4, v);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            u[i] &= (index + 2 * i < from ? 0u : ones & 0xffffu) | (index + 2 * i + 1 < from ? 0u : ones & 0xffff0000u);
        return __builtin_bit_cast(Frag, u);
    }
    static __device__ __forceinline__ float widen(E v) { return __uint_as_float(uint32_t(v) << 16); }
    static __device__ __forceinline__ void store4(E* p, const float (&v)[4])
    {
        *reinterpret_cast<u32x2*>(p) = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    }
};

// fp32 by three bf16 parts of each operand: the leading 8 bits of its 24, of what they leave, and the
// rest, each cut off, not rounded, so that no part overflows and nothing is lost (below 2^-110 the last
// bits are).  Of the nine products of parts the six that matter are formed, smallest first; what is left
// out is below 2^-23 of a product, 2^-25 on average, and fp32 rounds one by up to 2^-24.  That is three
// eighths of the time of the fp32 matrix instruction, which has a sixteenth of bf16's rate.  q, k and P
// lie in LDS as their parts, v as it is.
template <>
struct Ops<0> {
    using E = float;
    struct Frag {
        bf16x8 p[3];
    };
    struct VFrag {
        float v[8];
    };
    static constexpr int kEpc = 4;
    static __device__ __forceinline__ f32x16 mma(const Frag& a, const Frag& b, f32x16 c)
    {
        c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[2], b.p[0], c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[0], b.p[2], c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[1], b.p[1], c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[1], b.p[0], c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[0], b.p[1], c, 0, 0, 0);
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[0], b.p[0], c, 0, 0, 0);
    }
    static __device__ __forceinline__ f32x4 mma16(const Frag& a, const Frag& b, f32x4 c)
    {
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.p[2], b.p[0], c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.p[0], b.p[2], c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.p[1], b.p[1], c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.p[1], b.p[0], c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.p[0], b.p[1], c, 0, 0, 0);
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.p[0], b.p[0], c, 0, 0, 0);
    }
    // the parts of x and y, packed, x in the low halves
    static __device__ __forceinline__ void parts(float x, float y, uint32_t (&p)[3])
    {
#pragma unroll
        for (int q = 0; q < 3; ++q) {
            const uint32_t u = __float_as_uint(x), v = __float_as_uint(y);
            p[q] = __builtin_amdgcn_perm(v, u, 0x07060302u);
            x -= __uint_as_float(u & 0xffff0000u);
            y -= __uint_as_float(v & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ Frag operand(const VFrag& v)
    {
        u32x4 r[3];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t p[3];
            parts(v.v[2 * i], v.v[2 * i + 1], p);
#pragma unroll
            for (int q = 0; q < 3; ++q) r[q][i] = p[q];
        }
        Frag f;
#pragma unroll
        for (int q = 0; q < 3; ++q) f.p[q] = __builtin_bit_cast(bf16x8, r[q]);
        return f;
    }
    template <int R, int P>
    struct Tile {
        uint16_t m[3][R][P];
        __device__ __forceinline__ void put4(int r, int c, float x, float y, float z, float w)
        {
            uint32_t a[3], b[3];
            parts(x, y, a);
            parts(z, w, b);
#pragma unroll
            for (int q = 0; q < 3; ++q) *reinterpret_cast<u32x2*>(&m[q][r][c]) = u32x2{a[q], b[q]};
        }
        __device__ __forceinline__ void put(int r, int c, const u32x4& v)
        {
            put4(r, c, __uint_as_float(v[0]), __uint_as_float(v[1]), __uint_as_float(v[2]), __uint_as_float(v[3]));
        }
        __device__ __forceinline__ void store4(int r, int c, const float (&v)[4], const uint32_t (&k)[4])
        {
            put4(r, c, masked(v[0], k[0]), masked(v[1], k[1]), masked(v[2], k[2]), masked(v[3], k[3]));
        }
        __device__ __forceinline__ Frag row(int r, int c) const
        {
            return Frag{Ops<1>::row(&m[0][r][c]), Ops<1>::row(&m[1][r][c]), Ops<1>::row(&m[2][r][c])};
        }
        __device__ __forceinline__ Frag col(int r, int c, int lane) const
        {
            return Frag{Ops<1>::col(&m[0][r][c], P, lane), Ops<1>::col(&m[1][r][c], P, lane), Ops<1>::col(&m[2][r][c], P, lane)};
        }
        __device__ __forceinline__ float value(int r, int c) const
        {
            return (Ops<1>::widen(m[2][r][c]) + Ops<1>::widen(m[1][r][c])) + Ops<1>::widen(m[0][r][c]);
        }
    };
    static __device__ __forceinline__ VFrag vcol(const E* base, int pitch, int lane)
    {
        const E* p = base + 8 * (lane >> 5) * pitch + (lane & 31);
        VFrag f;
#pragma unroll
        for (int i = 0; i < 8; ++i) f.v[i] = p[i * pitch];
        return f;
    }
    static __device__ __forceinline__ Frag from_acc(const f32x16& c, int u)
    {
        u32x4 r[3];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t x[3], y[3];
            parts(c[8 * u + 2 * i], c[8 * u + 2 * i + 1], x);
            parts(c[8 * u + 4 + 2 * i], c[8 * u + 4 + 2 * i + 1], y);
#pragma unroll
            for (int q = 0; q < 3; ++q) {
                const auto s = __builtin_amdgcn_permlane32_swap(x[q], y[q], false, false);
                r[q][i] = s[0];
                r[q][2 + i] = s[1];
            }
        }
        Frag f;
#pragma unroll
        for (int q = 0; q < 3; ++q) f.p[q] = __builtin_bit_cast(bf16x8, r[q]);
        return f;
    }
    // one operand of three parts, weighed two elements at a step
    static constexpr int kParts = 1;
    static constexpr int kSteps = 4;
    struct Weighing {};
    template <int I>
    static __device__ __forceinline__ void weigh(const VFrag& v, const float* w, Frag (&part)[1], Weighing&)
    {
        uint32_t p[3];
        parts(v.v[2 * I] * w[2 * I], v.v[2 * I + 1] * w[2 * I + 1], p);
#pragma unroll
        for (int q = 0; q < 3; ++q) {
            u32x4 r = __builtin_bit_cast(u32x4, part[0].p[q]);
            r[I] = p[q];
            part[0].p[q] = __builtin_bit_cast(bf16x8, r);
        }
    }
    template <int N>
    static __device__ __forceinline__ bool not_finite(const VFrag (&v)[N])
    {
        float c = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
#pragma unroll
            for (int e = 0; e < 8; ++e) c = fmaf(v[i].v[e], 0.0f, c);
        }
        return !(c == 0.0f);
    }
    static __device__ __forceinline__ VFrag finite_part(VFrag f, uint32_t ones)
    {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t u = __float_as_uint(f.v[i]);
            f.v[i] = __uint_as_float(u & ((u & 0x7f800000u) == 0x7f800000u ? 0u : ones));
        }
        return f;
    }
    static __device__ __forceinline__ VFrag drop_below(VFrag f, int index, int from, uint32_t ones)
    {
#pragma unroll
        for (int i = 0; i < 8; ++i) f.v[i] = masked(f.v[i], index + i < from ? 0u : ones);
        return f;
    }
    static __device__ __forceinline__ float widen(E v) { return v; }
    static __device__ __forceinline__ void store4(E* p, const float (&v)[4])
    {
        *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
    }
};

// An operand's rows of one chunk as a range-checked buffer: loads past its rows give zeros, stores there
// are dropped.  Offsets count bytes from the row that lies lowest in memory; a lane that has nothing to
// load or store adds kNowhere, which no row's offset brings back into a buffer's range (the host keeps
// 64 rows under 2^29 bytes).
constexpr uint32_t kNowhere = 0x80000000u;
typedef __amdgpu_buffer_rsrc_t Rsrc;
__device__ __forceinline__ Rsrc buffer_of(const void* p, uint32_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), short(0), int(bytes), 0x00020000);
}

// How rows are read.  kWhole: the host has checked that they are whole 16-byte chunks at such addresses.
// kAny: at any address, of 16 bytes and more.  kSingle: element by element (8 x 2048 x 32 heads of 125
// in bf16: 707 us, 222 by kAny; of 128 by kWhole 134; 3 x 1021 x 12 heads of 72 and 91 in fp32 with their
// gradients: 186 and 163).
enum Access { kSingle, kWhole, kAny };

// 16 bytes of a row; `at` is kNowhere past the width.  kSingle: the `left` elements there are.  kAny: the
// aligned 16 bytes from the word at which they begin, and the next word where they do not begin with a
// word; a row's last piece ends with the row, so that nothing else of memory is touched.
struct Piece {
    u32x4 v;
    uint32_t x;
};
template <int DT, Access ACC>
__device__ __forceinline__ Piece load_piece(Rsrc r, uint32_t at, int left)
{
    if constexpr (ACC == kWhole) return {__builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0), 0};
    if constexpr (ACC == kAny && DT == 0) return {__builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0), 0};
    if constexpr (ACC == kAny)
        return {__builtin_amdgcn_raw_buffer_load_b128(r, at & ~3u, 0, 0),
                uint32_t(__builtin_amdgcn_raw_buffer_load_b32(r, at & 2u ? (at & ~3u) + 16u : kNowhere, 0, 0))};
    u32x4 v;
    if constexpr (DT == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __builtin_amdgcn_raw_buffer_load_b32(r, i < left ? at + 4 * i : kNowhere, 0, 0);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = uint16_t(__builtin_amdgcn_raw_buffer_load_b16(r, 2 * i < left ? at + 4 * i : kNowhere, 0, 0));
            const uint32_t hi = uint16_t(__builtin_amdgcn_raw_buffer_load_b16(r, 2 * i + 1 < left ? at + 4 * i + 2 : kNowhere, 0, 0));
            v[i] = lo | hi << 16;
        }
    }
    return {v, 0};
}
// The piece's elements.  kAny: without what lies before them, the half of a word and the `over` elements by
// which the piece was moved to end with its row; zeros come in behind.
template <int DT, Access ACC>
__device__ __forceinline__ u32x4 elements(const Piece& p, uint32_t at, int over)
{
    if constexpr (ACC != kAny) return p.v;
    if constexpr (DT == 0) {
        u32x4 w = p.v;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = over & 1 ? (i < 3 ? w[i + 1] : 0u) : w[i];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = over & 2 ? (i < 2 ? w[i + 2] : 0u) : w[i];
        return w;
    }
    // By masks, each move into words of its own: of `over & 2 ? w[i + 1] : w[i]` the compiler makes an index
    // into w, which then lies in memory.
    const uint32_t half = at << 3 & 16u, odd = uint32_t(over) << 4 & 16u;
    const uint32_t two = over & 2 ? 0xffffffffu : 0u, four = over & 4 ? 0xffffffffu : 0u;
    const uint32_t raw[5] = {p.v[0], p.v[1], p.v[2], p.v[3], p.x & 0xffffu};
    uint32_t x[5], y[5], z[6];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __builtin_amdgcn_alignbit(raw[i + 1], raw[i], half);
    x[4] = y[4] = z[4] = z[5] = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = __builtin_amdgcn_alignbit(x[i + 1], x[i], odd);
#pragma unroll
    for (int i = 0; i < 4; ++i) z[i] = (y[i + 1] & two) | (y[i] & ~two);
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = (z[i + 2] & four) | (z[i] & ~four);
    return w;
}

// The same as a store.  kAny: element by element too.
template <int DT, Access ACC>
__device__ __forceinline__ void store_piece(Rsrc r, uint32_t at, int left, const u32x4& v)
{
    if constexpr (ACC == kWhole) {
        __builtin_amdgcn_raw_buffer_store_b128(v, r, at, 0, 0);
    } else if constexpr (DT == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) __builtin_amdgcn_raw_buffer_store_b32(v[i], r, i < left ? at + 4 * i : kNowhere, 0, 0);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            __builtin_amdgcn_raw_buffer_store_b16(uint16_t(v[i]), r, 2 * i < left ? at + 4 * i : kNowhere, 0, 0);
            __builtin_amdgcn_raw_buffer_store_b16(uint16_t(v[i] >> 16), r, 2 * i + 1 < left ? at + 4 * i + 2 : kNowhere, 0, 0);
        }
    }
}

// All bits set.  In a branch that is seldom taken, masks made from it keep the compiler from running
// the branch's arithmetic always and selecting.
__device__ __forceinline__ uint32_t cold()
{
    uint32_t ones = 0xffffffffu;
    asm volatile("" : "+v"(ones));
    return ones;
}

// f(0), f(1), ... f(N - 1), each with its index as a type.
template <int N, typename F, int... I>
__device__ __forceinline__ void unroll_each(F&& f, std::integer_sequence<int, I...>)
{
    (f(std::integral_constant<int, I>()), ...);
}
template <int N, typename F>
__device__ __forceinline__ void unroll(F&& f)
{
    unroll_each<N>(f, std::make_integer_sequence<int, N>());
}

// The geometry of one instantiation.  Rows in LDS are padded by 16 bytes.
template <int DT, int DKP, int NW, Access ACC>
struct LattnShape {
    static constexpr int kThreads = 64 * NW;
    // rows at any address take a register more for each piece on its way
    static constexpr int kC = ACC == kAny ? 32 : lattn_chunk(DT, DKP, 32 * NW);
    static constexpr int kKP = DKP + 8;                       // pitch of q and k rows
    static constexpr int kVP = 32 * NW + Ops<DT>::kEpc;       // of v rows
    static constexpr int kPP = kC + 8;                        // of P rows
    // q and k are loaded as if they had a power of two of columns; the products go by DKP (8 x 512 x 32 heads of
    // 96 in fp32: 84 -> 77 us for 96 beside 128, of 160: 290 -> 232 for 192 beside 256)
    static constexpr int kLoad = DKP <= 64 ? 64 : DKP <= 128 ? 128 : 256;
    static constexpr int kQPieces = kC * kLoad / Ops<DT>::kEpc / kThreads;
    static constexpr int kVPieces = kC * 32 * NW / Ops<DT>::kEpc / kThreads;
    // waves on a SIMD: two, but where their registers do not allow it (8 x 2048 x 32 heads of 201 in bf16: 833 us
    // with two and 28 registers in memory, 667 with one; of 177, which fit two: 587 with one, 405)
    static constexpr int kWaves = (DKP > 128 && (DT == 0 || NW == 2 || (ACC == kAny && DKP == 256))) || (DKP > 64 && DT == 0 && NW == 2) ? 1 : 2;
};

// grid (units rounded up to 8, times jobs); units are slices * heads * batch * segments, slices fastest.
// Workgroups go to the 8 XCDs in turn: the jobs of a unit, which read the same rows in the same order
// (dk and dv), are 8 apart, on one XCD and its L2 (8 x 2048 x 40 heads of 128, gradients: 457 -> 448 us).
// STATE: forms what each segment but the last leaves in the state, from zero, and nothing else.
template <int DT, int DKP, int NW, Access ACC, bool STATE>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(LattnShape<DT, DKP, NW, ACC>::kWaves))) void lattn_kernel(LattnArgs a)
{
    using O = Ops<DT>;
    using E = typename O::E;
    using Frag = typename O::Frag;
    using VFrag = typename O::VFrag;
    using G = LattnShape<DT, DKP, NW, ACC>;
    constexpr int C = G::kC, kTB = C / 32, kDB = DKP / 32, kDepth = 16, kHalf = 8;
    constexpr int kKS = C / kDepth, kSub = 32 / kDepth;

    __shared__ __align__(16) typename O::template Tile<STATE ? 1 : C, G::kKP> sQ;
    __shared__ __align__(16) typename O::template Tile<C, G::kKP> sK;
    __shared__ __align__(16) E sV[C][G::kVP];
    __shared__ __align__(16) typename O::template Tile<STATE ? 1 : C, G::kPP> sP;
    __shared__ float s_enter[C + 1];    // out_scale a^j
    __shared__ float s_pow[C + 1];      // a^j
    __shared__ float s_pair[2 * C];              // pair_scale a^(C - 1 - x), 0 past C
    __shared__ float s_weight[C];                // in_scale a^(C - 1 - s)
    __shared__ __align__(16) float s_leave[C];   // a chunk's weights: the same where it is whole

    uint32_t x = blockIdx.x / (8 * a.jobs) * 8 + blockIdx.x % 8;
    const LattnJob& j = a.job[blockIdx.x / 8 % a.jobs];
    const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    int lane = tid & 63, l32 = lane & 31, hl = lane >> 5;
    // Hides from the compiler that addresses derived from the lane stay the same from chunk to chunk:
    // kept in registers they push others out to memory.
    auto renew = [&] {
        asm volatile("" : "+v"(lane));
        l32 = lane & 31;
        hl = lane >> 5;
    };
    const int slices = (j.dv + kLattnSlice - 1) / kLattnSlice;
    const int v0 = int(x % uint32_t(slices)) * kLattnSlice;
    x /= uint32_t(slices);
    const int64_t H = a.heads, L = a.seqlen;
    const int64_t h = x % uint32_t(H);
    x /= uint32_t(H);
    const int64_t b = x % uint32_t(a.batch), seg = x / uint32_t(a.batch);
    if (seg >= (STATE ? a.segs - 1 : a.segs)) return;  // what the last segment leaves is not needed
    const int64_t row0 = seg * a.seg_len, row1 = row0 + a.seg_len < L ? row0 + a.seg_len : L;
    const int64_t bh = b * H + h, cells = int64_t(j.dk) * j.dv;

    // powers of the decay, in 64 bits: they stand for the whole walk
    const double log_a = double(a.log_decay[h]);
    for (int i = tid; i <= C; i += G::kThreads) {
        const double power = i == 0 ? 1.0 : exp(log_a * i);
        s_pow[i] = float(power);
        s_enter[i] = float(power * double(j.out_scale));
    }
    for (int i = tid; i < 2 * C; i += G::kThreads)
        s_pair[i] = i >= C ? 0.0f : i == C - 1 ? j.pair_scale : float(exp(log_a * (C - 1 - i)) * double(j.pair_scale));
    for (int i = tid; i < C; i += G::kThreads)
        s_weight[i] = s_leave[i] = i == C - 1 ? j.in_scale : float(exp(log_a * (C - 1 - i)) * double(j.in_scale));

    constexpr uint32_t kEs = sizeof(E);
    const char* const pq = static_cast<const char*>(j.q) + (b * L * j.q_ld + (h / j.q_share) * j.dk) * kEs;
    const char* const pk = static_cast<const char*>(j.k) + (b * L * j.k_ld + (h / j.k_share) * j.dk) * kEs;
    const char* const pv = static_cast<const char*>(j.v) + (b * L * j.v_ld + (h / j.v_share) * j.dv) * kEs;
    // the stride of a single row lies between sequences alone, and may be any
    const bool single = L == 1;
    const uint32_t lq = uint32_t(single ? j.dk : j.q_ld) * kEs, lk = uint32_t(single ? j.dk : j.k_ld) * kEs;
    const uint32_t lv = uint32_t(single ? j.dv : j.v_ld) * kEs;
    const uint32_t oes = j.out_f32 ? 4 : kEs, lo = uint32_t(H * j.dv) * oes;
    char* const po = static_cast<char*>(j.out) + (b * L * H * j.dv + h * j.dv + v0) * oes;
    const int vw = j.dv - v0;  // columns from here on
    const int ow = vw < kLattnSlice ? vw : kLattnSlice;  // columns of this workgroup
    const uint8_t* const pr = a.reset ? a.reset + b * L : nullptr;
    const bool rev = j.rev;
    // An operand at the walk's current chunk of C rows: `at` is the row that lies lowest in memory.
    struct Side {
        const char* at;
        uint32_t ld, width;  // bytes
    };
    auto side = [&](const char* p, uint32_t ld, uint32_t width, int t0) {
        return Side{p + (rev ? L - t0 - C : t0) * int64_t(ld), ld, width};
    };
    auto next = [&](Side& s) { s.at += (rev ? -int64_t(C) : int64_t(C)) * int64_t(s.ld); };
    // n of its rows as a buffer, and what to add to the offset of row r in a whole chunk, which is
    // (rev ? C - 1 - r : r) rows: a short chunk lacks its last rows, from the end the lowest in memory.  The
    // buffer begins and ends with a word.
    auto rows = [&](const Side& s, int n) {
        const uint32_t miss = uint32_t(C - n) * s.ld;
        const char* p = s.at + (rev ? miss : 0u);
        uint32_t bytes = n > 0 ? uint32_t(C - 1) * s.ld + s.width - miss : 0;
        if constexpr (ACC == kAny) {
            const uint32_t half = uint32_t(reinterpret_cast<uintptr_t>(p)) & 2u;
            p -= half;
            bytes = n > 0 ? (bytes + half + 3u) & ~3u : 0;
        }
        return buffer_of(p, bytes);
    };
    auto shift = [&](const Side& s, int n) {
        uint32_t by = rev ? 0u - uint32_t(C - n) * s.ld : 0u;
        if constexpr (ACC == kAny) by += uint32_t(reinterpret_cast<uintptr_t>(s.at) + (rev ? uint32_t(C - n) * s.ld : 0u)) & 2u;
        return by;
    };

    const int c0 = 32 * w;  // this wave's columns of v; past the width they are zeros and nothing is stored

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
    constexpr int kQC = G::kLoad / O::kEpc, kVC = 32 * NW / O::kEpc;  // 16-byte pieces of a row
    constexpr int kQR = G::kThreads / kQC, kVR = G::kThreads / kVC;  // rows that the threads load at once
    static_assert(G::kThreads % kQC == 0 && G::kThreads % kVC == 0, "a thread's pieces lie in one column");
    const int qr = tid / kQC, qc = tid % kQC * O::kEpc, vr = tid / kVC, vc = tid % kVC * O::kEpc;
    Piece fq[STATE ? 1 : G::kQPieces], fk[G::kQPieces], fv[G::kVPieces];
    uint32_t flag = 0;
    const Rsrc rr = buffer_of(pr, pr ? uint32_t(L) : 0);
    Side q = side(pq, lq, j.dk * kEs, int(row0)), k = side(pk, lk, j.dk * kEs, int(row0)), v = side(pv, lv, j.dv * kEs, int(row0));
    // results go out a chunk later: the first time nothing does
    Side out = side(po, lo, ow * oes, int(row0) - C);
    u32x4 fo[STATE ? 1 : G::kVPieces];
    int out_rows = 0;
    // a thread's first piece of a whole chunk, and the bytes to the next; by how much a piece is moved to end
    // with its row
    auto first = [&](const Side& s, int r, int c, int width) {
        return (c < width ? uint32_t(c) * kEs : kNowhere) + uint32_t(rev ? C - 1 - r : r) * s.ld;
    };
    auto past = [&](int c, int width) { return ACC == kAny && c < width && c + O::kEpc > width ? c + O::kEpc - width : 0; };
    const int q_past = past(qc, j.dk), v_past = past(v0 + vc, j.dv);
    auto step = [&](const Side& s, int r) { return rev ? 0u - r * s.ld : r * s.ld; };
    const uint32_t oq = first(q, qr, qc, j.dk) - q_past * kEs, ok = first(k, qr, qc, j.dk) - q_past * kEs;
    const uint32_t ov = first(v, vr, v0 + vc, j.dv) - v_past * kEs;
    const uint32_t oo = first(out, vr, vc, ow);
    // The stores and loads of a chunk, one piece at a time, so that they go out between products.  Stores
    // come first: a wait for loads then waits for no store that was issued behind them.
    struct Moves {
        Rsrc out, q, k, v;
        uint32_t ao, aq, ak, av, so, sq, sk, sv;
        int out_rows, rows;
    } mv;
    auto start_store = [&] {
        mv.out = rows(out, out_rows);
        mv.ao = oo + shift(out, out_rows);
        mv.so = step(out, kVR);
        mv.out_rows = out_rows;
        next(out);
    };
    auto start_load = [&](int t0, int n) {
        // whether the state of the row before is dropped on the way to this row: from the end, the
        // reset is the one of the row that was walked before
        const int t = rev ? int(L) - t0 - lane : t0 + lane;
        flag = uint8_t(__builtin_amdgcn_raw_buffer_load_b8(rr, lane < n && t < int(L) ? uint32_t(t) : kNowhere, 0, 0));
        mv.q = rows(q, n);
        mv.k = rows(k, n);
        mv.v = rows(v, n);
        mv.aq = oq + shift(q, n);
        mv.ak = ok + shift(k, n);
        mv.av = ov + shift(v, n);
        mv.sq = step(q, kQR);
        mv.sk = step(k, kQR);
        mv.sv = step(v, kVR);
        mv.rows = n;
        next(q);
        next(k);
        next(v);
    };
    constexpr int kStores = G::kVPieces, kLoads = (STATE ? 1 : 2) * G::kQPieces + G::kVPieces;
    // kAny: the words at a buffer's ends hold elements of rows that are not there
    auto there = [&](uint32_t at, int row, int n) { return DT == 1 && ACC == kAny && row >= n ? kNowhere : at; };
    auto store_one = [&](auto i_v) {
        constexpr int i = decltype(i_v)::value;
        store_piece<DT, ACC>(mv.out, there(mv.ao + i * mv.so, vr + i * kVR, mv.out_rows), ow - vc, fo[i]);
    };
    auto load_one = [&](auto i_v) {
        constexpr int i = decltype(i_v)::value;
        if constexpr (i < G::kVPieces) {
            fv[i] = load_piece<DT, ACC>(mv.v, there(mv.av + i * mv.sv, vr + i * kVR, mv.rows), vw - vc);
        } else if constexpr (i < G::kVPieces + G::kQPieces) {
            constexpr int p = i - G::kVPieces;
            fk[p] = load_piece<DT, ACC>(mv.k, there(mv.ak + p * mv.sk, qr + p * kQR, mv.rows), j.dk - qc);
        } else {
            constexpr int p = i - G::kVPieces - G::kQPieces;
            fq[p] = load_piece<DT, ACC>(mv.q, there(mv.aq + p * mv.sq, qr + p * kQR, mv.rows), j.dk - qc);
        }
    };

    // Blocks of P^T.  Of 64 rows, 32 x 32: (s 0-31, t 0-31), (s 0-31, t 32-63) and (s 32-63, t 32-63); a wave
    // left without one forms the last one too and writes the same numbers, so that every wave runs the same
    // code.  Of 32 rows, 16 x 16, all four.  A lane has column t = tb + lt of its block and, of its rows, four
    // neighbouring ones at a time.
    constexpr bool kWide = kTB == 2;
    constexpr int kBlocks = kWide ? 3 : 4, kRounds = (kBlocks + NW - 1) / NW, kQuads = kWide ? 4 : 1;

    auto block = [&](int i, int& sb, int& tb) {
        if constexpr (kWide) {
            const int blk = w + i * NW < kBlocks ? w + i * NW : kBlocks - 1;
            sb = blk == 2 ? 32 : 0;
            tb = blk == 0 ? 0 : 32;
        } else {
            sb = (w + i * NW) / 2 * 16;
            tb = (w + i * NW) % 2 * 16;
        }
    };
    auto column = [&] { return kWide ? l32 : lane & 15; };
    auto first_row = [&](int quad) { return kWide ? 8 * quad + 4 * hl : 4 * (lane >> 4); };
    // a bit for each register of a block: whether row t comes after row s or is it
    uint32_t causal[kRounds];
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
        int sb, tb;
        block(i, sb, tb);
        causal[i] = 0;
#pragma unroll
        for (int r = 0; r < 4 * kQuads; ++r) causal[i] |= (sb + first_row(r / 4) + r % 4 <= tb + column() ? 1u : 0u) << r;
    }

    const int left0 = int(row1 - row0);
    start_load(int(row0), left0 < C ? left0 : C);
    unroll<kLoads>(load_one);
    bool cut = false;  // STATE: whether a reset lies in the segment
    for (int t0 = int(row0), left = left0; left > 0; t0 += C, left -= C) {
        const int n = left < C ? left : C;  // rows of this chunk
        renew();
        // ---- the chunk into LDS, the next one's loads on their way ----
#pragma unroll
        for (int i = 0; i < G::kQPieces; ++i) {
            if (G::kLoad != DKP && qc >= DKP) break;
            if constexpr (!STATE) sQ.put(qr + i * kQR, qc, elements<DT, ACC>(fq[i], mv.aq + i * mv.sq, q_past));
            sK.put(qr + i * kQR, qc, elements<DT, ACC>(fk[i], mv.ak + i * mv.sk, q_past));
        }
#pragma unroll
        for (int i = 0; i < G::kVPieces; ++i) *reinterpret_cast<u32x4*>(&sV[vr + i * kVR][vc]) = elements<DT, ACC>(fv[i], mv.av + i * mv.sv, v_past);
        const uint64_t resets = __ballot(flag != 0);
        const int last = resets ? 63 - __builtin_clzll(resets) : 0;  // the last reset's row: what is before leaves nothing
        if constexpr (!STATE) {
            start_store();
            unroll<kStores>(store_one);
        }
        start_load(t0 + C, left - C < 0 ? 0 : left - C < C ? left - C : C);
        __syncthreads();
        if constexpr (STATE) unroll<kLoads>(load_one);

        // the state of the row before the chunk reaches its first row undecayed if it is the gradient
        // that the last row's state has from outside
        const int e0 = rev && t0 == 0 ? 0 : 1;

        VFrag vf[kKS];  // this wave's columns of v
        auto columns = [&] {
#pragma unroll
            for (int ks = 0; ks < kKS; ++ks) vf[ks] = O::vcol(&sV[ks * kDepth][c0], G::kVP, lane);
        };
        columns();
        f32x16 o[kTB];
        bool odd = false;  // whether one of them is infinite or NaN
        if constexpr (!STATE) {
            // ---- P^T = K Q^T with its decays, into LDS as P (t, s); O^T = S^T Q^T ----
            typedef std::conditional_t<kWide, f32x16, f32x4> Block;
            Block p[kRounds];
            uint32_t see[kRounds];  // the same for whether row t sees row s
#pragma unroll
            for (int i = 0; i < kRounds; ++i) see[i] = causal[i];
            const int lt = column();
            if (resets) {
                cold();
#pragma unroll
                for (int i = 0; i < kRounds; ++i) {
                    int sb, tb;
                    block(i, sb, tb);
                    // the first row that row t sees
                    const uint64_t upto = resets & (~uint64_t(0) >> (63 - tb - lt));
                    const int from = upto ? 63 - __builtin_clzll(upto) : 0;
#pragma unroll
                    for (int r = 0; r < 4 * kQuads; ++r)
                        if (sb + first_row(r / 4) + r % 4 < from) see[i] &= ~(1u << r);
                }
            }
            // four rows s of a block of P at a time
            auto pairs = [&](auto i_v) {
                constexpr int i = decltype(i_v)::value / kQuads, quad = decltype(i_v)::value % kQuads;
                int sb, tb;
                block(i, sb, tb);
                const int t = tb + lt, s = sb + first_row(quad);
                const float* const f = &s_pair[C - 1 - t + s];
                float x[4];
                uint32_t m[4];
                // every product masked afterwards: a choice would become a branch
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[e] = p[i][4 * quad + e] * f[e];
                    m[e] = uint32_t(__builtin_amdgcn_sbfe(int(see[i]), 4 * quad + e, 1));
                }
                sP.store4(t, s, x, m);
            };
#pragma unroll
            for (int tb = 0; tb < kTB; ++tb) {
#pragma unroll
                for (int r = 0; r < 16; ++r) o[tb][r] = 0.0f;
            }
            // every fragment is read some steps before its product
            constexpr int kSteps = DKP / kDepth, kPieces = kQuads * kRounds;
            unroll<kRounds>([&](auto x_v) {
                constexpr int x = decltype(x_v)::value, kDeep = kWide ? 16 : 32, kTimes = DKP / kDeep, kAhead = kWide ? 3 : 1;
                int sb, tb;
                block(x, sb, tb);
                Frag kq[kAhead + 1][2];
                auto fetch = [&](int i) {
                    const int c = kDeep * i + (kWide ? 8 * hl : 8 * (lane >> 4));
                    kq[i % (kAhead + 1)][0] = sK.row(sb + lt, c);
                    kq[i % (kAhead + 1)][1] = sQ.row(tb + lt, c);
                };
#pragma unroll
                for (int r = 0; r < 4 * kQuads; ++r) p[x][r] = 0.0f;
#pragma unroll
                for (int i = 0; i < kAhead; ++i) fetch(i);
                unroll<kTimes>([&](auto i_v) {
                    constexpr int i = decltype(i_v)::value;
                    if constexpr (i + kAhead < kTimes) fetch(i + kAhead);
                    if constexpr (kWide) p[x] = O::mma(kq[i % (kAhead + 1)][0], kq[i % (kAhead + 1)][1], p[x]);
                    else p[x] = O::mma16(kq[i % (kAhead + 1)][0], kq[i % (kAhead + 1)][1], p[x]);
                    __builtin_amdgcn_sched_barrier(0);
                });
            });
            constexpr int kNext = DT == 1 ? 2 : 1;
            Frag qf[kNext + 1][kTB];
            auto queries = [&](int i) {
#pragma unroll
                for (int tb = 0; tb < kTB; ++tb) qf[i % (kNext + 1)][tb] = sQ.row(32 * tb + l32, kDepth * i + kHalf * hl);
            };
#pragma unroll
            for (int i = 0; i < kNext; ++i) queries(i);
            // the products of S with, between them, the next chunk's loads and the rest of P
            unroll<kSteps>([&](auto i_v) {
                constexpr int i = decltype(i_v)::value;
                if constexpr (i + kNext < kSteps) queries(i + kNext);
                const Frag s = O::from_acc(st[i / kSub], i % kSub);
#pragma unroll
                for (int tb = 0; tb < kTB; ++tb) o[tb] = O::mma(s, qf[i % (kNext + 1)][tb], o[tb]);
                constexpr int m0 = kLoads * i / kSteps, m1 = kLoads * (i + 1) / kSteps;
                unroll<m1 - m0>([&](auto m_v) { load_one(std::integral_constant<int, m0 + decltype(m_v)::value>()); });
                constexpr int p0 = i < 2 ? 0 : kPieces * (i - 2) / (kSteps - 2), p1 = i < 2 ? 0 : kPieces * (i - 1) / (kSteps - 2);
                unroll<p1 - p0>([&](auto m_v) { pairs(std::integral_constant<int, p0 + decltype(m_v)::value>()); });
                __builtin_amdgcn_sched_barrier(0);
            });
            odd = __ballot(O::not_finite(vf)) != 0;
#pragma unroll
            for (int tb = 0; tb < kTB; ++tb) {
                const float f = s_enter[32 * tb + l32 + e0];
#pragma unroll
                for (int r = 0; r < 16; ++r) o[tb][r] *= f;
            }
            if (resets) {
                const uint32_t ones = cold();
#pragma unroll
                for (int tb = 0; tb < kTB; ++tb) {
                    const bool sees = (resets & (~uint64_t(0) >> (63 - 32 * tb - l32))) == 0;
#pragma unroll
                    for (int r = 0; r < 16; ++r) o[tb][r] = masked(o[tb][r], sees ? ones : 0u);
                }
            }
            __syncthreads();
        }
        // what lies before the last reset leaves nothing: P is formed, so those rows of k can go.  The
        // last chunk of a walk may be short: its weights end with its last row.
        if (resets || n < C) {
            const int thread = 64 * w + lane;
            if (resets) {
                for (int p = thread; p < last * (DKP / O::kEpc); p += G::kThreads)
                    sK.put(p / (DKP / O::kEpc), p % (DKP / O::kEpc) * O::kEpc, u32x4{0, 0, 0, 0});
            }
            if (n < C)
                for (int i = thread; i < C; i += G::kThreads) s_leave[i] = i < n ? s_weight[i + C - n] : 0.0f;
            __syncthreads();
        }

        constexpr int kKeys = DT == 0 ? 1 : kDB > 4 ? 2 : kDB;  // fragments of k held for a step, and as many for the next
        Frag part[2][O::kParts], kf[2][kKeys];
        float wt[2][kHalf];
        typename O::Weighing steps;
        auto weights = [&](int ks) {
#pragma unroll
            for (int i = 0; i < kHalf; ++i) wt[ks & 1][i] = s_leave[ks * kDepth + kHalf * hl + i];
        };
        auto keys = [&](int step) {  // kKeys blocks of d of 16 rows
#pragma unroll
            for (int e = 0; e < kKeys; ++e) {
                const int at = step * kKeys + e;
                kf[step & 1][e] = sK.col(at / kDB * kDepth, 32 * (at % kDB), lane);
            }
        };
        auto weigh = [&](auto ks_v, auto lo_v, auto hi_v) {  // steps [lo, hi) of it
            constexpr int ks = decltype(ks_v)::value, lo = decltype(lo_v)::value, hi = decltype(hi_v)::value;
            unroll<hi - lo>([&](auto t) {
                O::template weigh<lo + decltype(t)::value>(vf[ks], wt[ks & 1], part[ks & 1], steps);
            });
        };
        const std::integral_constant<int, 0> zero{};
        const std::integral_constant<int, O::kSteps> all{};
        weights(0);
        const float f = s_pow[n - 1 + e0];  // the decay over the chunk
        if constexpr (!STATE) {
            // ---- O^T += V^T P^T ----
            // a row must not meet an infinity or NaN that it does not see, not even times 0: these are
            // left out of the product and added where they are seen
            if (odd) {
                const uint32_t ones = cold();
#pragma unroll
                for (int ks = 0; ks < kKS; ++ks) vf[ks] = O::finite_part(vf[ks], ones);
            }
            constexpr int kProducts = kTB == 2 ? 3 * kSub : kSub;
            Frag pf[kProducts];
#pragma unroll
            for (int i = 0; i < kProducts; ++i) {
                const int ks = i < 2 * kSub && kTB == 2 ? i / 2 : i - (kTB - 1) * kSub, tb = kTB == 2 && (i >= 2 * kSub || i % 2 == 1);
                pf[i] = sP.row(32 * tb + l32, ks * kDepth + kHalf * hl);
            }
            keys(0);
            weigh(zero, zero, all);  // while P's rows come
            __builtin_amdgcn_sched_barrier(0);
            unroll<kProducts>([&](auto i_v) {
                constexpr int i = decltype(i_v)::value;
                constexpr int ks = i < 2 * kSub && kTB == 2 ? i / 2 : i - (kTB - 1) * kSub, tb = kTB == 2 && (i >= 2 * kSub || i % 2 == 1);
                o[tb] = O::mma(O::operand(vf[ks]), pf[i], o[tb]);
                // the state's own decay beside these
                constexpr int r0 = 16 * kDB * i / kProducts, r1 = 16 * kDB * (i + 1) / kProducts;
                unroll<r1 - r0>([&](auto r_v) {
                    constexpr int r = r0 + decltype(r_v)::value;
                    st[r / 16][r % 16] *= f;
                });
                __builtin_amdgcn_sched_barrier(0);
            });
            if (odd) {
#pragma unroll
                for (int tb = 0; tb < kTB; ++tb) {
                    const int t = 32 * tb + l32;
                    const uint64_t upto = resets & (~uint64_t(0) >> (63 - t));
                    const int from = upto ? 63 - __builtin_clzll(upto) : 0;
#pragma unroll 1
                    for (int s = 0; s < 32 * (tb + 1); ++s) {
                        const bool sees = s <= t && s >= from;
                        const float p = sP.value(t, s);
#pragma unroll
                        for (int r = 0; r < 16; ++r) {
                            const float v = O::widen(sV[s][c0 + 8 * (r >> 2) + 4 * hl + (r & 3)]);
                            o[tb][r] += sees && !(fabsf(v) < INFINITY) ? p * v : 0.0f;
                        }
                    }
                }
                columns();
            }
            if (DT == 1 && j.out_f32) {
                // sums over the heads that share k or q follow: a lane has 4 columns of row t at a time
                const Rsrc b = rows(out, n);
#pragma unroll
                for (int tb = 0; tb < kTB; ++tb) {
                    const int t = 32 * tb + l32;
                    const uint32_t at = uint32_t(rev ? C - 1 - t : t) * lo + shift(out, n) + uint32_t(c0 + 4 * hl) * 4;
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const int c = 8 * (r >> 2) + (r & 3);
                        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(o[tb][r]), b,
                                                              c0 + 4 * hl + c < ow ? at + 4 * c : kNowhere, 0, 0);
                    }
                }
            } else {
                // into the place of this wave's columns of v, which are in its registers: whole rows go
                // out from there
#pragma unroll
                for (int tb = 0; tb < kTB; ++tb) {
#pragma unroll
                    for (int q4 = 0; q4 < 4; ++q4) {
                        const float x[4] = {o[tb][4 * q4], o[tb][4 * q4 + 1], o[tb][4 * q4 + 2], o[tb][4 * q4 + 3]};
                        O::store4(&sV[32 * tb + l32][c0 + 8 * q4 + 4 * hl], x);
                    }
                }
                out_rows = n;
            }
        } else {
            keys(0);
            weigh(zero, zero, all);
#pragma unroll
            for (int d = 0; d < kDB; ++d) {
#pragma unroll
                for (int r = 0; r < 16; ++r) st[d][r] *= f;
            }
        }

        // ---- S = a^n S + K^T (w V) ----
        if (odd || resets) {
            const uint32_t ones = cold();
            if (resets) {
#pragma unroll
                for (int ks = 0; ks < kKS; ++ks) vf[ks] = O::drop_below(vf[ks], ks * kDepth + kHalf * hl, last, ones);
#pragma unroll
                for (int d = 0; d < kDB; ++d) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) st[d][r] = masked(st[d][r], ~ones);
                }
            }
            weigh(zero, zero, all);
        }
        // Each product is followed by a few steps of weighing the next rows: issued in this order, they
        // run beside each other.  The smallest parts come first; neighbouring products are of different
        // blocks of the state and do not wait for one another.
        unroll<kKS>([&](auto ks_v) {
            constexpr int ks = decltype(ks_v)::value, kProducts = O::kParts * kDB;
            if constexpr (ks + 1 < kKS) weights(ks + 1);
            unroll<kProducts>([&](auto i_v) {
                constexpr int i = decltype(i_v)::value, group = i / (O::kParts * kKeys), at = i % (O::kParts * kKeys);
                constexpr int q = O::kParts - 1 - at / kKeys, d = group * kKeys + at % kKeys;
                constexpr int step = (ks * kDB + d) / kKeys;
                if constexpr (at == 0 && step + 1 < kKS * kDB / kKeys) keys(step + 1);
                st[d] = O::mma(kf[step & 1][d % kKeys], part[ks & 1][q], st[d]);
                if constexpr (ks + 1 < kKS)
                    weigh(std::integral_constant<int, ks + 1>(), std::integral_constant<int, O::kSteps * i / kProducts>(),
                          std::integral_constant<int, O::kSteps * (i + 1) / kProducts>());
                __builtin_amdgcn_sched_barrier(0);
            });
        });
        cut |= resets != 0;
        __syncthreads();
        // whole rows of o; the same threads write the next chunk's rows of v there
        if constexpr (!STATE) {
#pragma unroll
            for (int i = 0; i < G::kVPieces; ++i) fo[i] = *reinterpret_cast<const u32x4*>(&sV[vr + i * kVR][vc]);
        }
    }
    if constexpr (!STATE) {
        start_store();
        unroll<kStores>(store_one);
    }

    if constexpr (STATE) {
        if (v0 == 0 && tid == 0) {
            const int64_t n = row1 - row0 - (rev && row0 == 0 ? 1 : 0);
            j.keep[seg * a.batch * H + bh] = cut ? -1.0f : n == 0 ? 1.0f : float(exp(log_a * double(n)));
        }
    }
    renew();
    // ---- the state after the last row ----
    float* to = nullptr;
    int64_t oi = j.dv, oj = 1;
    float f = 1.0f;
    if (STATE) {
        to = j.seg + (seg * a.batch * H + bh) * cells;
    } else if (j.h_last && seg == a.segs - 1) {
        to = j.h_last + bh * cells;
        oi = j.si;
        oj = j.sj;
        if (rev) f = pr && pr[0] ? -1.0f : s_pow[1];
    }
    if (to) {
#pragma unroll
        for (int d = 0; d < kDB; ++d) {
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int i = 32 * d + 8 * (r >> 2) + 4 * hl + (r & 3);
                if (i < j.dk && c0 + l32 < vw) to[i * oi + (v0 + c0 + l32) * oj] = f < 0.0f ? 0.0f : st[d][r] * f;
            }
        }
    }
}

template <int DT, int DKP, int NW, Access ACC>
hipError_t launch_shape(const LattnArgs& a, hipStream_t stream)
{
    auto grid = [&](int64_t segs) { return static_cast<uint32_t>(lattn_groups(a.batch, a.heads, a.job[0].dv, a.jobs, segs)); };
    const dim3 block(64 * NW);
    if (a.segs > 1) {
        lattn_kernel<DT, DKP, NW, ACC, true><<<grid(a.segs - 1), block, 0, stream>>>(a);
        if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
        if (hipError_t e = launch_lattn_join(a, stream); e != hipSuccess) return e;
    }
    lattn_kernel<DT, DKP, NW, ACC, false><<<grid(a.segs), block, 0, stream>>>(a);
    return hipGetLastError();
}

// Jobs of one launch have the same class of widths; the widest chooses the padding of q and k.
template <int DT>
hipError_t launch_typed(const LattnArgs& a, bool vec, hipStream_t stream)
{
    const int dv = a.job[0].dv;
    int dk = 0;
    for (int i = 0; i < a.jobs; ++i) dk = a.job[i].dk > dk ? a.job[i].dk : dk;
    // rows of 16 bytes and more
    bool any = true;
    for (int i = 0; i < a.jobs; ++i) any = any && a.job[i].dk >= Ops<DT>::kEpc && a.job[i].dv >= Ops<DT>::kEpc;
    auto go = [&](auto dkp, auto nw) {
        constexpr int kD = decltype(dkp)::value, kW = decltype(nw)::value;
        if (vec) return launch_shape<DT, kD, kW, kWhole>(a, stream);
        if (any) return launch_shape<DT, kD, kW, kAny>(a, stream);
        // rows of less than 16 bytes: beside v of more than 64 columns only those of q and k, so of up to 64
        if constexpr (kW == 2 || kD == 64) return launch_shape<DT, kD, kW, kSingle>(a, stream);
        return hipErrorInvalidValue;
    };
    using std::integral_constant;
    auto by_dv = [&](auto dkp) {
        return lattn_waves(dv) == 2 ? go(dkp, integral_constant<int, 2>()) : go(dkp, integral_constant<int, 4>());
    };
    return dk <= 64    ? by_dv(integral_constant<int, 64>())
           : dk <= 96  ? by_dv(integral_constant<int, 96>())
           : dk <= 128 ? by_dv(integral_constant<int, 128>())
           : dk <= 192 ? by_dv(integral_constant<int, 192>()) : by_dv(integral_constant<int, 256>());
}

}  // namespace
}  // namespace ssk
