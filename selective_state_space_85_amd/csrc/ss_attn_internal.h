// Internal interface between the C-ABI layer of the linear-attention operators (ss_attn_api.cpp)
// and their gfx950 kernels (ss_lattn.hip, ss_qknorm.hip, ss_sample.hip).  Not installed, not part of
// the ABI.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

namespace ssk {

// ---- linear attention with a decay for each head ---------------------------------------

constexpr int kLattnMaxDim = 256;
// Rows per chunk, the unit that sequences are cut in, for widths dk and dv.  In fp32 the three parts of every
// row fit the LDS for 32, with two workgroups beside each other up to 128 elements.  In bf16 a state above
// 128 x 128 for each four waves, or 64 x 64 for each two, leaves registers for 32 rows with two waves on a
// SIMD (32768 x 8 heads of 256: 459 -> 340 us forward; of 128 and 64: 100 -> 84; of 128, where both fit: 114).
constexpr int lattn_chunk(int dtype, int dk, int dv) { return dtype == 0 || dk > 128 || (dk > 64 && dv <= 64) ? 32 : 64; }

// One walk over the sequence.  Forward, dq, dk and dv are the same operation
//   o_t = sum over s up to t of a^(t - s) (q_t . k_s) v_s  (+ a^(t + 1) h0^T q_t)
// with other operands: (q, k, v); (d_o, v, k); and from the end, (v, d_o, q) and (k, q, d_o).
struct LattnJob {
    const void* q;
    const void* k;
    const void* v;
    int64_t q_ld, k_ld, v_ld;       // elements between two tokens
    int q_share, k_share, v_share;  // heads that share one head of the operand
    int dk, dv;                     // widths of q and k, of v
    void* out;                      // (batch, seqlen, heads, dv) dtype, or fp32 if out_f32
    bool out_f32;
    bool rev;                       // from the last row to the first
    const float* h0;                // (batch, heads, dk x dv) with strides si, sj, or null
    float* h_last;                  // the same strides, or null; rev: times the decay, 0 at a reset of row 0
    int64_t si, sj;
    // of (q_t . k_s), of k_s v_s^T on its way into the state, of what the state gives a row
    float pair_scale, in_scale, out_scale;
    float* seg;   // (segments, batch * heads, dk, dv): what each segment leaves, then the state before it
    float* keep;  // (segments, batch * heads): the decay over each segment, -1 where it has a reset
};

struct LattnArgs {
    LattnJob job[3];
    int jobs;
    const float* log_decay;
    const uint8_t* reset;  // nullable
    int64_t batch, seqlen, heads;
    int64_t seg_len, segs;  // rows of a segment (a multiple of lattn_chunk), segments
};
// Columns of v that one workgroup takes.
constexpr int kLattnSlice = 128;
inline int64_t lattn_slices(int64_t dv) { return (dv + kLattnSlice - 1) / kLattnSlice; }

// Waves of a workgroup, 32 columns of v each.
inline int lattn_waves(int64_t dv) { return dv <= 64 ? 2 : 4; }
// Workgroups of a launch of `jobs` walks over `segs` segments: whole eights of them (lattn_kernel).
inline int64_t lattn_groups(int64_t batch, int64_t heads, int64_t dv, int jobs, int64_t segs)
{
    return (lattn_slices(dv) * heads * batch * segs + 7) / 8 * 8 * jobs;
}

// Jobs of one launch have the same class of widths (lattn_class).
inline int lattn_class(int dk, int dv) { return (dk <= 64 ? 0 : dk <= 128 ? 1 : 2) + 3 * (dv <= 64 ? 0 : int(lattn_slices(dv))); }
// Workgroups of a class that a CU holds beside each other.
inline int64_t lattn_resident(int dtype, int dk, int dv)
{
    return dtype == 0 ? (dk > 128 ? 1 : 2) : dk <= 128 && dv <= 64 ? 4 : 2;
}
hipError_t launch_lattn(const LattnArgs& a, int dtype, hipStream_t stream);
// its parts: the element types' instantiations (vec: every row is whole 16-byte chunks), and the
// states before the segments from what each segment leaves
hipError_t launch_lattn_bf16(const LattnArgs& a, bool vec, hipStream_t stream);
hipError_t launch_lattn_f32(const LattnArgs& a, bool vec, hipStream_t stream);
hipError_t launch_lattn_join(const LattnArgs& a, hipStream_t stream);

// out (rows, heads / share, width) dtype = sums of part (rows, heads, width) over `share` heads
hipError_t launch_lattn_share(const float* part, void* out, int64_t rows, int64_t heads, int64_t share, int64_t width,
                              int dtype, hipStream_t stream);

// One token: workgroups of kStepThreads for each kStepCols columns of a head's state.
constexpr int kStepThreads = 256, kStepCols = 128;
inline int64_t lattn_step_groups(int64_t batch, int64_t heads, int64_t dv)
{
    return batch * heads * ((dv + kStepCols - 1) / kStepCols);
}

struct LattnStepArgs {
    float* h;
    const void* q;
    const void* k;
    const void* v;
    int64_t q_ld, k_ld, v_ld;
    const float* log_decay;
    float scale;
    void* o;
    int64_t batch, qk_heads, heads, dk, dv;
};
hipError_t launch_lattn_step(const LattnStepArgs& a, int dtype, hipStream_t stream);

// ---- norms and rotation of queries and keys --------------------------------------------

constexpr int kQknormMaxDim = 512;
constexpr int64_t kQknormMaxHeads = int64_t(1) << 24;  // the heads of a tile's tokens are counted in 32 bits

constexpr int kQknormThreads = 256;
constexpr int kQknormAngles = 1024;   // of a workgroup's tile of tokens
constexpr int kQknormTile = 16;       // tokens of a tile at most

// Tokens of a tile: as many as its angles allow, fewer where that would leave CUs without work: 2048
// tiles forward (16384 tokens of 40 + 40 heads of 128: 142 us in 1024 tiles, 134 in 2048), 1024 backward
// (221 and 216 there, and 3 us more for the sums of 2048 workgroups).
inline int64_t qknorm_tile(int64_t tokens, int64_t half, bool back)
{
    int64_t n = half ? kQknormAngles / half : kQknormTile;
    n = n < kQknormTile ? n : kQknormTile;
    const int64_t even = back ? tokens / 1024 : tokens / 2048 + (tokens % 2048 != 0);
    n = n < even ? n : even;
    return n > 1 ? n : 1;
}
inline int64_t qknorm_tiles(int64_t tokens, int64_t half, bool back)
{
    const int64_t tile = qknorm_tile(tokens, half, back);
    return tokens / tile + (tokens % tile != 0);
}

struct QknormSide {
    const void* x;   // (tokens, heads, width), rows ld apart
    int64_t ld, heads;
    const float* w;
    void* out;       // forward: the normed and turned x; backward: dx
    const void* dy;  // backward
    float* dw;       // backward
};

struct QknormArgs {
    QknormSide side[2];
    const int64_t* pos;
    const float* inv_freq;
    float eps;
    bool interleaved;
    float* part;  // backward: (2, blocks, width), each workgroup's sums
    int64_t tokens, width, half;
    int64_t blocks;
};
hipError_t launch_qknorm_fwd(const QknormArgs& a, int dtype, hipStream_t stream);
hipError_t launch_qknorm_bwd(const QknormArgs& a, int dtype, hipStream_t stream);

// ---- sampling --------------------------------------------------------------------------

constexpr int64_t kSampleMaxVocab = int64_t(1) << 24;

struct SampleArgs {
    const void* logits;
    int64_t ld;
    const float* u;
    const float* temperature;
    const int32_t* top_k;
    const float* top_p;
    const float* min_p;
    float temperature_all, top_p_all, min_p_all;
    int32_t top_k_all;
    int64_t* token;
    int64_t rows, vocab;
};
hipError_t launch_sample(const SampleArgs& a, int dtype, hipStream_t stream);

}  // namespace ssk
