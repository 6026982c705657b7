// Internal interface between the C-ABI layer of the language-model operators
// (ss_lm_api.cpp) and their gfx950 kernels (ss_glr.hip, ss_glu.hip, ss_xent.hip).
// Not installed, not part of the ABI.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

namespace ssk {

// Rows of x up to which products with weights may stream the weights past them (ss_gemm.h)
// instead of working in tiles.
constexpr int64_t kStreamRows = 64;
// Rows of x up to which the gradients of such products are formed in one pass over the weights
// (ss_few.hip).
constexpr int64_t kFewRows = 8;

// With s (m, rows), x (m, k) and weights W (rows, k): dx = s W in parts, dW = s^T x.  W may lie in
// two matrices, the first `first` rows in w0 and the others in w1.
struct FewGradArgs {
    const float* s;   // rows of s_ld elements; its columns for w1 start at s_second
    int64_t s_ld, s_second;
    const void* w0;
    const void* w1;
    void* dw0;        // null: not wanted
    void* dw1;
    const void* x;
    int64_t x_ld;
    float* part;      // (parts, m, k); null: dx is not wanted
    void* dx;         // (m, k)
    int64_t first, rows, m, k;
    int64_t per, parts;  // rows per part of the sums of dx
    // null, or (m,): rows whose target is ignore_index or outside [0, rows) have s = 0, their dx is
    // 0 and nothing of their x enters dW
    const int64_t* target;
    int64_t ignore_index;
};
hipError_t launch_few_grad(const FewGradArgs& a, int dtype, hipStream_t stream);

// ---- gated feed-forward projection -----------------------------------------------------

constexpr int kActSilu = 0, kActGelu = 1;


// Tokens up to which the weights' gradients in tiles, bf16, use what the rounding of dg and du left
// as well: their sums have few terms to even the roundings out, and a k tile (64 tokens) has
// room for both without another product.
constexpr int64_t kGluLoRows = 32;

struct GluArgs {
    const void* x;   // (m, k), rows x_ld elements apart
    int64_t x_ld;
    const void* wg;  // (f, k), rows w_ld elements apart
    const void* wu;
    int64_t w_ld;
    void* h;         // (m, f); the backward: unused
    const void* dh;  // backward: (m, f)
    void* dgu;       // backward workspace: (m, 2 f_pad), dg in the first half of a row, du in the second
    bool lo;         // and behind them as many rows of what their rounding left (see kGluLoRows)
    void* dx;        // (m, k), nullable
    void* dwg;       // (f, k), nullable (both or neither)
    void* dwu;
    int64_t m, k, f, f_pad;
    int64_t k_pad;   // k rounded up to whole 16-byte chunks; rows of x and w in tiles hold zeros there
    // the operands as the caller gave them: the streaming kernels take any alignment.  Equal to x
    // and the weights unless those are padded copies.
    const void* x_raw;
    int64_t x_raw_ld;
    const void* wg_raw;
    const void* wu_raw;
    bool aligned;    // x_raw and the weights start every row on 16 bytes
    bool stream;     // the products of x and the weights stream the weights
    bool few;        // the backward in one pass over the weights: dgu is fp32
    int act;
    // the backward's sums of dx over 2 f are cut in dx_splits parts when tokens are few
    float* dx_part;  // (dx_splits, m, k) fp32, null with one part in tiles
    int64_t dx_splits;
    int64_t dx_per;  // few: rows of the weights per part
    // and those of the weights' gradients over the tokens when features are few
    float* dw_part;  // (dw_splits, 2 f_pad, k) fp32, null with one part
    int64_t dw_splits;
};

// Copy of `rows` rows of `cols` elements (ld apart) into rows of cols_pad elements, the pad zeroed.
hipError_t launch_pad_rows(const void* src, int64_t ld, void* dst, int64_t rows, int64_t cols, int64_t cols_pad,
                           int dtype, hipStream_t stream);
hipError_t launch_glu_fwd(const GluArgs& a, int dtype, hipStream_t stream);
// The backward's two launches: dgu from x, w, dh; then dx and dw from dgu.
hipError_t launch_glu_bwd(const GluArgs& a, int dtype, hipStream_t stream);

// ---- softmax cross entropy of a vocabulary projection -----------------------------------

// Columns of the vocabulary behind one partial (maximum, sum) pair of a row, in tiles and in the
// streaming kernel.
constexpr int64_t kXentCols = 128, kXentStreamCols = 32;

struct XentArgs {
    const void* x;  // (n, d), rows x_ld elements apart
    int64_t x_ld;
    const void* w;  // (v, d), rows w_ld elements apart
    int64_t w_ld;
    const int64_t* target;  // (n,)
    int64_t ignore_index;
    float* loss;        // forward output (n,)
    float* lse;         // forward output, backward input (n,)
    float* part_max;    // forward workspace: (ceil(v / columns per pair), n)
    float* part_sum;
    float* target_logit;  // forward workspace (n,)
    const float* dloss;   // backward (n,)
    void* dl;             // backward workspace: (n, piece_pad) gradient of one piece's logits
    // bf16 backward workspace: what rounding took from each row's target entry of dl, and per
    // 128 columns of the vocabulary the tokens whose targets lie there, in order, and their number
    float* lo;            // (n,)
    int32_t* tokens;      // (ceil(v / kXentCols), n)
    int32_t* counts;      // (ceil(v / kXentCols),)
    // backward workspace: sums of dx over the pieces, each piece's sum in dx_splits parts, (dx_splits,
    // n, d) fp32; null with one piece and one part
    float* dx_acc;
    int64_t dx_splits;
    int64_t dx_per;  // few: rows of w per part
    // sums of dw over the rows of x in dw_splits parts, (dw_splits, columns of the piece, d) fp32;
    // null with one part
    float* dw_part;
    int64_t dw_splits;
    void* dx;             // (n, d), nullable
    void* dw;             // (v, d), nullable
    int64_t n, d, v;
    int64_t d_pad;        // d rounded up to whole 16-byte chunks
    // as for GluArgs
    const void* x_raw;
    int64_t x_raw_ld;
    const void* w_raw;
    bool aligned, stream, few;
    int64_t piece;        // columns of the vocabulary per piece (the backward)
};

hipError_t launch_xent_fwd(const XentArgs& a, int dtype, hipStream_t stream);
hipError_t launch_xent_bwd(const XentArgs& a, int dtype, hipStream_t stream);

// ---- gated linear recurrence ------------------------------------------------------------

// Rows between two kept states, which is also the backward's tile: it rebuilds a tile's states
// from the one that enters it.  The backward's chunks are whole tiles.
constexpr int64_t kGlrRows = 32;
// Rows of a forward tile.
constexpr int64_t kGlrTile = 256;
// Longest row stride, in elements: a tile stays below 2^31 bytes.
constexpr int64_t kGlrMaxStride = int64_t(1) << 20;

struct GlrArgs {
    const void* x;  // (batch, seqlen, dim), rows *_ld elements apart
    const void* r;
    const void* i;
    int64_t x_ld, r_ld, i_ld;
    const float* decay;    // (dim,)
    float c;
    const float* h0;       // (batch, dim), nullable
    const uint8_t* reset;  // (batch, seqlen), nullable
    void* y;               // (batch, seqlen, dim); null: only the states are wanted
    float* h_last;         // (batch, dim), nullable
    float* ckpt;           // (ceil(seqlen / kGlrRows), batch, dim) states entering every kGlrRows-th row, nullable
    // forward with more than one tile: a word per tile and channel (channels rounded up to
    // whole workgroups), and the next tile to be taken
    uint64_t* ws_words;
    uint32_t* ws_ticket;
    int64_t batch, seqlen, dim;
    int64_t n_tiles;       // ceil(seqlen / kGlrTile)
    // backward; n_chunks > 1: per chunk and channel the affine map of the chunk
    float* ws_prod;        // (n_chunks, batch, dim)
    float* ws_end;         // (n_chunks, batch, dim)
    int64_t chunk_len, n_chunks;  // chunk_len a multiple of kGlrRows
    const void* dy;        // (batch, seqlen, dim)
    const float* dh_last;  // (batch, dim), nullable
    void* dx;              // (batch, seqlen, dim), rows g_ld elements apart
    void* dr;
    void* di;
    int64_t g_ld;
    float* dh0;            // (batch, dim), nullable
    float* part_decay;     // (n_chunks, batch, dim) sums over a chunk's rows
    float* ddecay;         // (dim,)
};

// Rows of `ld` elements from p on start whole groups of n (2 or 4) elements.
inline bool whole_groups(const void* p, int64_t ld, int dtype, int n)
{
    return p == nullptr || (ld % n == 0 && reinterpret_cast<uintptr_t>(p) % uintptr_t((dtype == 0 ? 4 : 2) * n) == 0);
}
// Channels per lane, two where every row of every operand allows it: the forward's, the backward's.
inline int glr_fwd_channels(const GlrArgs& a, int dtype)
{
    return a.dim % 2 == 0 && whole_groups(a.x, a.x_ld, dtype, 2) && whole_groups(a.r, a.r_ld, dtype, 2) &&
                   whole_groups(a.i, a.i_ld, dtype, 2) && whole_groups(a.y, a.dim, dtype, 2)
               ? 2
               : 1;
}
inline int glr_bwd_channels(const GlrArgs& a, int dtype)
{
    return a.dim % 2 == 0 && whole_groups(a.x, a.x_ld, dtype, 2) && whole_groups(a.r, a.r_ld, dtype, 2) &&
                   whole_groups(a.i, a.i_ld, dtype, 2) && whole_groups(a.dy, a.dim, dtype, 2) &&
                   whole_groups(a.dx, a.g_ld, dtype, 2) && whole_groups(a.dr, a.g_ld, dtype, 2) &&
                   whole_groups(a.di, a.g_ld, dtype, 2)
               ? 2
               : 1;
}
// Workgroups of a launch over `spans` tiles or chunks of rows, with that many channels per lane (32 lanes).
inline int64_t glr_blocks(const GlrArgs& a, int channels, int64_t spans)
{
    return (a.dim + 32 * channels - 1) / (32 * channels) * a.batch * spans;
}
// Their threads.
constexpr int kGlrFwdThreads = 512, kGlrBwdThreads = 256;

hipError_t launch_glr_fwd(const GlrArgs& a, int dtype, hipStream_t stream);
hipError_t launch_glr_bwd(const GlrArgs& a, int dtype, hipStream_t stream);

struct GlrStepArgs {
    float* h;  // (batch, dim)
    const void* x;
    const void* r;
    const void* i;  // (batch, dim)
    int64_t x_ld, r_ld, i_ld;
    const float* decay;
    float c;
    void* y;
    int64_t batch, dim;
};
// Channels per thread of the step, and its threads.
inline int glr_step_channels(const GlrStepArgs& a, int dtype)
{
    return whole_groups(a.x, a.x_ld, dtype, 4) && whole_groups(a.r, a.r_ld, dtype, 4) &&
                   whole_groups(a.i, a.i_ld, dtype, 4) && whole_groups(a.y, a.dim, dtype, 4) &&
                   whole_groups(a.h, a.dim, 0, 4)
               ? 4
               : 1;
}
constexpr int kGlrStepThreads = 256;
hipError_t launch_glr_step(const GlrStepArgs& a, int dtype, hipStream_t stream);

}  // namespace ssk
