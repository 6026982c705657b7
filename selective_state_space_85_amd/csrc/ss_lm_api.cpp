// C ABI of the language-model operators (ss_lm.h): argument validation, plans, workspace
// sizing and kernel dispatch.  Validation runs on the host before anything is enqueued.
#include <math.h>
#include <stdint.h>

#include "ss_check.h"
#include "ss_internal.h"
#include "ss_lm.h"
#include "ss_lm_internal.h"
#include "ss_tiles.h"

namespace {

constexpr size_t kBad = static_cast<size_t>(-1);

int64_t elem_size(ss_dtype dtype) { return dtype == SS_F32 ? 4 : 2; }
bool known(ss_dtype dtype) { return dtype == SS_F32 || dtype == SS_BF16; }

ss_status done(hipError_t e)
{
    if (e == hipSuccess) return SS_OK;
    ssk::note_hip_error(e);
    return SS_ERR_HIP;
}

// Regions of a workspace, each from a 256-byte boundary.
struct Regions {
    int64_t at = 0;
    bool ok = true;
    int64_t add(int64_t count, int64_t size)
    {
        int64_t bytes, from;
        if (!ok || !mul(count, size, &bytes) || __builtin_add_overflow(at, int64_t(255), &from)) {
            ok = false;
            return 0;
        }
        if (bytes == 0) return at;  // not there
        from &= ~int64_t(255);
        if (__builtin_add_overflow(from, bytes, &at)) ok = false;
        return from;
    }
};

// Bytes that `rows` rows of `cols` elements, ld elements apart, span.
bool strided_bytes(int64_t rows, int64_t cols, int64_t ld, int64_t es, int64_t* bytes)
{
    int64_t n;
    return mul(rows - 1, ld, &n) && !__builtin_add_overflow(n, cols, &n) && mul(n, es, bytes);
}

// Whether two tensors of the same rows, row length and stride (bytes) share an element.
// Column slices of one tensor interleave without sharing any.
bool strided_overlap(const void* p, const void* q, int64_t bytes, int64_t row, int64_t stride)
{
    if (!overlap(span(p, bytes), span(q, bytes))) return false;
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    const int64_t off = static_cast<int64_t>((a < b ? b - a : a - b) % static_cast<uintptr_t>(stride));
    return off < row || off + row > stride;
}

// Whether a launch fits: HIP takes fewer than 2^32 threads along a grid's axis.
bool launch_fits(int64_t blocks, int64_t threads) { return blocks <= int64_t(UINT32_MAX) / threads; }

ss_status check_workspace(void* workspace, size_t given, int64_t need, const Range* others, size_t count)
{
    if (need == 0) return SS_OK;
    if (!workspace || given < static_cast<size_t>(need)) return SS_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return SS_ERR_INVALID_ARG;
    const Range w = span(workspace, need);
    for (size_t i = 0; i < count; ++i)
        if (overlap(w, others[i])) return SS_ERR_INVALID_ARG;
    return SS_OK;
}

bool any_overlap(const Range* outputs, size_t n_out, const Range* inputs, size_t n_in)
{
    for (size_t i = 0; i < n_out; ++i) {
        for (size_t k = 0; k < n_in; ++k)
            if (overlap(outputs[i], inputs[k])) return true;
        for (size_t k = i + 1; k < n_out; ++k)
            if (overlap(outputs[i], outputs[k])) return true;
    }
    return false;
}

// ---- gated linear recurrence ------------------------------------------------------------

constexpr int64_t kGlrCols = 64;  // channels per workgroup
// The backward with fewer one-chunk workgroups than kGlrWhole leaves CUs idle: the rows are then
// cut until there are kGlrTarget workgroups, in chunks of at least kGlrMinChunk rows (the cut
// costs a pass over r and dy) and at most kGlrMaxChunks of them (a chunk joins the maps of those
// after it itself).  Both passes, whole and cut: (1, 16384, 2048) bf16 900 and 201 us, (4, 2048, 2560)
// 160 and 134, (3, 1021, 1533) fp32 81 and 84; with twice as many chunks 214, 126 and 86.  These have
// 32, 160 and 72 workgroups; between 256 and 768, where whole rows leave some CUs a workgroup short
// of three, nothing was measured.  Kernels of one channel per lane have twice the workgroups counted.
constexpr int64_t kGlrWhole = 256, kGlrTarget = 768, kGlrMinChunk = 128, kGlrMaxChunks = 64;

void glr_plan(int64_t batch, int64_t seqlen, int64_t dim, int64_t* len, int64_t* chunks)
{
    const int64_t unit = ssk::kGlrRows;
    const int64_t blocks = batch * ceil_div(dim, kGlrCols);
    int64_t k = 1;
    if (blocks < kGlrWhole) {
        k = ceil_div(kGlrTarget, blocks);
        const int64_t most = seqlen / kGlrMinChunk;
        k = k < most ? k : most;
        k = k < kGlrMaxChunks ? k : kGlrMaxChunks;
        k = k > 1 ? k : 1;
    }
    *len = ceil_div(ceil_div(seqlen, k), unit) * unit;
    *chunks = ceil_div(seqlen, *len);
}

struct GlrLayout {
    int64_t len, chunks, tiles;
    int64_t ticket, words, prod, end, part, ckpt, total;
};

bool glr_sizes(int64_t batch, int64_t seqlen, int64_t dim)
{
    int64_t n;
    return batch > 0 && seqlen > 0 && dim > 0 && mul(batch, seqlen, &n) && mul(n, dim, &n) && mul(n, 4, &n);
}

// The forward's part is there for the forward, and for a backward without kept states.
bool glr_layout(int64_t batch, int64_t seqlen, int64_t dim, bool back, bool with_ckpt, GlrLayout* w)
{
    if (!glr_sizes(batch, seqlen, dim)) return false;
    glr_plan(batch, seqlen, dim, &w->len, &w->chunks);
    w->tiles = ceil_div(seqlen, ssk::kGlrTile);
    Regions r;
    int64_t words = 0;
    if ((!back || !with_ckpt) && w->tiles > 1 &&
        (!mul(w->tiles * batch, ceil_div(dim, kGlrCols), &words) || !mul(words, kGlrCols, &words)))
        return false;
    w->ticket = r.add(words ? 1 : 0, 4);
    w->words = r.add(words, 8);
    const int64_t maps = back && w->chunks > 1 ? w->chunks * batch * dim : 0;
    w->prod = r.add(maps, 4);
    w->end = r.add(maps, 4);
    w->part = r.add(back ? w->chunks * batch * dim : 0, 4);
    w->ckpt = r.add(back && !with_ckpt ? ceil_div(seqlen, ssk::kGlrRows) * batch * dim : 0, 4);
    w->total = r.at;
    return r.ok;
}

bool glr_grid_ok(int64_t batch, int64_t dim, const GlrLayout& w)
{
    int64_t n, m;
    return mul(batch, ceil_div(dim, kGlrCols / 2), &n) && mul(n, w.chunks, &m) && m <= INT32_MAX && mul(n, w.tiles, &m) &&
           m <= INT32_MAX;
}

bool glr_too_wide(int64_t a, int64_t b, int64_t c, int64_t d)
{
    return a > ssk::kGlrMaxStride || b > ssk::kGlrMaxStride || c > ssk::kGlrMaxStride || d > ssk::kGlrMaxStride;
}

}  // namespace

extern "C" {

size_t ss_glr_ckpt_bytes(int64_t batch, int64_t seqlen, int64_t dim)
{
    int64_t n;
    if (!glr_sizes(batch, seqlen, dim)) return kBad;
    if (!mul(ceil_div(seqlen, ssk::kGlrRows), batch, &n) || !mul(n, dim, &n) || !mul(n, 4, &n)) return kBad;
    return static_cast<size_t>(n);
}

size_t ss_glr_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim)
{
    GlrLayout w;
    return glr_layout(batch, seqlen, dim, false, true, &w) ? static_cast<size_t>(w.total) : kBad;
}

size_t ss_glr_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim, int with_ckpt)
{
    GlrLayout w;
    return glr_layout(batch, seqlen, dim, true, with_ckpt != 0, &w) ? static_cast<size_t>(w.total) : kBad;
}

ss_status ss_glr_fwd(const void* x, int64_t x_row_stride, const void* r, int64_t r_row_stride, const void* i,
                     int64_t i_row_stride, const float* decay, float c, const float* h0, const uint8_t* reset,
                     void* y, float* h_last, float* ckpt, void* workspace, size_t workspace_bytes, int64_t batch,
                     int64_t seqlen, int64_t dim, ss_dtype dtype, hipStream_t stream)
{
    if (!x || !r || !i || !decay || !y) return SS_ERR_INVALID_ARG;
    GlrLayout w;
    if (!glr_layout(batch, seqlen, dim, false, true, &w)) return SS_ERR_INVALID_ARG;
    if (x_row_stride < dim || r_row_stride < dim || i_row_stride < dim) return SS_ERR_INVALID_ARG;
    if (!isfinite(c) || c <= 0.0f) return SS_ERR_INVALID_ARG;
    if (!known(dtype)) return SS_ERR_UNSUPPORTED;
    if (!glr_grid_ok(batch, dim, w) || glr_too_wide(x_row_stride, r_row_stride, i_row_stride, dim))
        return SS_ERR_UNSUPPORTED;
    const int64_t es = elem_size(dtype), rows = batch * seqlen;
    const void* elems[] = {x, r, i, y};
    for (const void* p : elems)
        if (!aligned(p, uintptr_t(es))) return SS_ERR_INVALID_ARG;
    const void* words[] = {decay, h0, h_last, ckpt};
    for (const void* p : words)
        if (!aligned(p, 4)) return SS_ERR_INVALID_ARG;
    int64_t xb, rb, ib;
    if (!strided_bytes(rows, dim, x_row_stride, es, &xb) || !strided_bytes(rows, dim, r_row_stride, es, &rb) ||
        !strided_bytes(rows, dim, i_row_stride, es, &ib))
        return SS_ERR_INVALID_ARG;
    const int64_t state = batch * dim * 4;
    const Range all[] = {span(x, xb), span(r, rb), span(i, ib), span(decay, dim * 4), span(reset, rows),
                         span(h0, state), span(y, rows * dim * es),
                         span(ckpt, static_cast<int64_t>(ss_glr_ckpt_bytes(batch, seqlen, dim))),
                         span(h_last, state)};
    if (any_overlap(all + 6, 3, all, 5)) return SS_ERR_INVALID_ARG;
    for (int k = 6; k < 9; ++k)  // h_last may be h0 itself
        if (overlap(all[k], all[5]) && !(k == 8 && h_last == h0)) return SS_ERR_INVALID_ARG;
    const ss_status st = check_workspace(workspace, workspace_bytes, w.total, all, 9);
    if (st != SS_OK) return st;

    char* const ws = static_cast<char*>(workspace);
    ssk::GlrArgs a{};
    a.x = x;
    a.r = r;
    a.i = i;
    a.x_ld = x_row_stride;
    a.r_ld = r_row_stride;
    a.i_ld = i_row_stride;
    a.decay = decay;
    a.c = c;
    a.h0 = h0;
    a.reset = reset;
    a.y = y;
    a.h_last = h_last;
    a.ckpt = ckpt;
    if (w.tiles > 1) {
        a.ws_words = reinterpret_cast<uint64_t*>(ws + w.words);
        a.ws_ticket = reinterpret_cast<uint32_t*>(ws + w.ticket);
    }
    a.batch = batch;
    a.seqlen = seqlen;
    a.dim = dim;
    a.n_tiles = w.tiles;
    const int dt = dtype == SS_F32 ? 0 : 1;
    if (!launch_fits(ssk::glr_blocks(a, ssk::glr_fwd_channels(a, dt), w.tiles), ssk::kGlrFwdThreads))
        return SS_ERR_UNSUPPORTED;
    return done(ssk::launch_glr_fwd(a, dt, stream));
}

ss_status ss_glr_bwd(const void* x, int64_t x_row_stride, const void* r, int64_t r_row_stride, const void* i,
                     int64_t i_row_stride, const float* decay, float c, const float* h0, const uint8_t* reset,
                     const void* dy, const float* dh_last, const float* ckpt, void* dx, void* dr, void* di,
                     int64_t grad_row_stride, float* ddecay, float* dh0, void* workspace, size_t workspace_bytes,
                     int64_t batch, int64_t seqlen, int64_t dim, ss_dtype dtype, hipStream_t stream)
{
    if (!x || !r || !i || !decay || !dy || !dx || !dr || !di || !ddecay) return SS_ERR_INVALID_ARG;
    GlrLayout w;
    if (!glr_layout(batch, seqlen, dim, true, ckpt != nullptr, &w)) return SS_ERR_INVALID_ARG;
    if (x_row_stride < dim || r_row_stride < dim || i_row_stride < dim || grad_row_stride < dim)
        return SS_ERR_INVALID_ARG;
    if (!isfinite(c) || c <= 0.0f) return SS_ERR_INVALID_ARG;
    if (!known(dtype)) return SS_ERR_UNSUPPORTED;
    if (!glr_grid_ok(batch, dim, w) || glr_too_wide(x_row_stride, r_row_stride, i_row_stride, grad_row_stride))
        return SS_ERR_UNSUPPORTED;
    const int64_t es = elem_size(dtype), rows = batch * seqlen;
    const void* elems[] = {x, r, i, dy, dx, dr, di};
    for (const void* p : elems)
        if (!aligned(p, uintptr_t(es))) return SS_ERR_INVALID_ARG;
    const void* words[] = {decay, h0, dh_last, ckpt, ddecay, dh0};
    for (const void* p : words)
        if (!aligned(p, 4)) return SS_ERR_INVALID_ARG;
    int64_t xb, rb, ib, gb;
    if (!strided_bytes(rows, dim, x_row_stride, es, &xb) || !strided_bytes(rows, dim, r_row_stride, es, &rb) ||
        !strided_bytes(rows, dim, i_row_stride, es, &ib) || !strided_bytes(rows, dim, grad_row_stride, es, &gb))
        return SS_ERR_INVALID_ARG;
    const int64_t state = batch * dim * 4;
    const Range all[] = {span(x, xb), span(r, rb), span(i, ib), span(decay, dim * 4), span(reset, rows),
                         span(h0, state), span(dy, rows * dim * es), span(dh_last, state),
                         span(ckpt, static_cast<int64_t>(ss_glr_ckpt_bytes(batch, seqlen, dim))),
                         span(dx, gb), span(dr, gb), span(di, gb), span(ddecay, dim * 4), span(dh0, state)};
    for (int k = 9; k < 12; ++k) {
        if (any_overlap(all + k, 1, all, 9)) return SS_ERR_INVALID_ARG;
        if (overlap(all[k], all[12]) || overlap(all[k], all[13])) return SS_ERR_INVALID_ARG;
    }
    if (any_overlap(all + 12, 2, all, 9)) return SS_ERR_INVALID_ARG;
    const int64_t row = dim * es, stride = grad_row_stride * es;
    if (strided_overlap(dx, dr, gb, row, stride) || strided_overlap(dx, di, gb, row, stride) ||
        strided_overlap(dr, di, gb, row, stride))
        return SS_ERR_INVALID_ARG;
    const ss_status st = check_workspace(workspace, workspace_bytes, w.total, all, 14);
    if (st != SS_OK) return st;

    char* const ws = static_cast<char*>(workspace);
    ssk::GlrArgs a{};
    a.x = x;
    a.r = r;
    a.i = i;
    a.x_ld = x_row_stride;
    a.r_ld = r_row_stride;
    a.i_ld = i_row_stride;
    a.decay = decay;
    a.c = c;
    a.h0 = h0;
    a.reset = reset;
    if (w.chunks > 1) {
        a.ws_prod = reinterpret_cast<float*>(ws + w.prod);
        a.ws_end = reinterpret_cast<float*>(ws + w.end);
    }
    if (!ckpt && w.tiles > 1) {
        a.ws_words = reinterpret_cast<uint64_t*>(ws + w.words);
        a.ws_ticket = reinterpret_cast<uint32_t*>(ws + w.ticket);
    }
    a.batch = batch;
    a.seqlen = seqlen;
    a.dim = dim;
    a.n_tiles = w.tiles;
    a.chunk_len = w.len;
    a.n_chunks = w.chunks;
    // the kept states: only read from here on when they are the caller's
    a.ckpt = ckpt ? const_cast<float*>(ckpt) : reinterpret_cast<float*>(ws + w.ckpt);
    const int dt = dtype == SS_F32 ? 0 : 1;
    a.dy = dy;
    a.dh_last = dh_last;
    a.dx = dx;
    a.dr = dr;
    a.di = di;
    a.g_ld = grad_row_stride;
    a.dh0 = dh0;
    a.part_decay = reinterpret_cast<float*>(ws + w.part);
    a.ddecay = ddecay;
    if (!launch_fits(ssk::glr_blocks(a, ssk::glr_bwd_channels(a, dt), w.chunks), ssk::kGlrBwdThreads) ||
        (!ckpt && !launch_fits(ssk::glr_blocks(a, ssk::glr_fwd_channels(a, dt), w.tiles), ssk::kGlrFwdThreads)))
        return SS_ERR_UNSUPPORTED;
    if (!ckpt) {
        const hipError_t e = ssk::launch_glr_fwd(a, dt, stream);  // y is null: the states alone
        if (e != hipSuccess) return done(e);
    }
    return done(ssk::launch_glr_bwd(a, dt, stream));
}

ss_status ss_glr_step(float* h, const void* x, int64_t x_row_stride, const void* r, int64_t r_row_stride,
                      const void* i, int64_t i_row_stride, const float* decay, float c, void* y, int64_t batch,
                      int64_t dim, ss_dtype dtype, hipStream_t stream)
{
    if (!h || !x || !r || !i || !decay || !y) return SS_ERR_INVALID_ARG;
    if (!glr_sizes(batch, 1, dim)) return SS_ERR_INVALID_ARG;
    if (x_row_stride < dim || r_row_stride < dim || i_row_stride < dim) return SS_ERR_INVALID_ARG;
    if (!isfinite(c) || c <= 0.0f) return SS_ERR_INVALID_ARG;
    if (!known(dtype)) return SS_ERR_UNSUPPORTED;
    const int64_t es = elem_size(dtype);
    const void* elems[] = {x, r, i, y};
    for (const void* p : elems)
        if (!aligned(p, uintptr_t(es))) return SS_ERR_INVALID_ARG;
    if (!aligned(h, 4) || !aligned(decay, 4)) return SS_ERR_INVALID_ARG;
    int64_t xb, rb, ib;
    if (!strided_bytes(batch, dim, x_row_stride, es, &xb) || !strided_bytes(batch, dim, r_row_stride, es, &rb) ||
        !strided_bytes(batch, dim, i_row_stride, es, &ib))
        return SS_ERR_INVALID_ARG;
    const Range all[] = {span(x, xb), span(r, rb), span(i, ib), span(decay, dim * 4), span(h, batch * dim * 4),
                         span(y, batch * dim * es)};
    if (any_overlap(all + 4, 2, all, 4)) return SS_ERR_INVALID_ARG;
    const ssk::GlrStepArgs a{h, x, r, i, x_row_stride, r_row_stride, i_row_stride, decay, c, y, batch, dim};
    const int dt = dtype == SS_F32 ? 0 : 1;
    if (!launch_fits(ceil_div(dim, ssk::kGlrStepThreads * ssk::glr_step_channels(a, dt)), ssk::kGlrStepThreads))
        return SS_ERR_UNSUPPORTED;
    return done(ssk::launch_glr_step(a, dt, stream));
}

}  // extern "C"

namespace {

// ---- the two matrix operators: x (rows, dim) against weights (cols, dim) ------------------

// Elements per 16 bytes: rows are read in whole 16-byte chunks.
// (fp32 tiles take any alignment.)
int64_t chunk_elems(ss_dtype dtype) { return 16 / elem_size(dtype); }
int64_t padded(int64_t n, ss_dtype dtype) { return ceil_div(n, chunk_elems(dtype)) * chunk_elems(dtype); }

// Every row starts on 16 bytes.
bool whole_rows(const void* p, int64_t ld, ss_dtype dtype) { return aligned(p, 16) && ld % chunk_elems(dtype) == 0; }

// Sizes whose products are formed unchecked below.
bool mat_sizes(int64_t rows, int64_t dim, int64_t cols)
{
    if (rows <= 0 || dim <= 0 || cols <= 0) return false;
    // room for the padding to 16-byte chunks and to tiles
    if (rows > (INT64_MAX >> 16) || dim > (INT64_MAX >> 16) || cols > (INT64_MAX >> 16)) return false;
    const int64_t r = rows + 256, d = dim + 256, c = cols + 256;
    int64_t n;
    return mul(r, d, &n) && mul(n, 16, &n) && mul(c, d, &n) && mul(n, 16, &n) && mul(r, c, &n) && mul(n, 16, &n);
}

// A grid of 128 x 128 tiles (the smaller kind) has to fit one launch.
bool mat_grid_ok(int64_t rows, int64_t cols)
{
    int64_t n;
    return mul(ceil_div(rows, 128), ceil_div(cols, 64), &n) && n <= INT32_MAX / 2;
}

// The threads of a launch of tiles stay below HIP's limit.  Sizes within mat_grid_ok.
template <int DT>
bool tiles_fit(int64_t large, int64_t small, int64_t mini)
{
    return ssk::tile_threads(ssk::best_tile<DT>(large, small, mini), large, small, mini) <= int64_t(UINT32_MAX);
}
// Two outputs of one launch, each in `parts` (0: not wanted).
struct TiledOutput {
    int64_t rows, cols, parts;
};
bool tiles_fit(TiledOutput a, TiledOutput b, ss_dtype dtype)
{
    auto tiles = [&](int bm, int bn) {
        return (a.parts ? ssk::count(a.rows, a.cols, bm, bn) * a.parts : 0) +
               (b.parts ? ssk::count(b.rows, b.cols, bm, bn) * b.parts : 0);
    };
    const int64_t large = tiles(256, 256), small = tiles(128, 128), mini = tiles(64, 128);
    return dtype == SS_F32 ? tiles_fit<0>(large, small, mini) : tiles_fit<1>(large, small, mini);
}
// The one-pass gradients' launches.
bool few_fits(int64_t rows, int64_t dim)
{
    return launch_fits(ceil_div(dim, 512), 128) && launch_fits(ceil_div(rows * dim, 256), 256);
}

// x's checks: its stride and alignment; *pack: it has to be copied to padded rows
ss_status mat_operand(const void* p, int64_t ld, int64_t dim, ss_dtype dtype, bool* pack)
{
    if (ld < dim) return SS_ERR_INVALID_ARG;
    *pack = dtype == SS_BF16 && dim % chunk_elems(dtype) != 0;
    if (*pack || dtype == SS_F32) return aligned(p, uintptr_t(elem_size(dtype))) ? SS_OK : SS_ERR_INVALID_ARG;
    if (!aligned(p, 16) || ld % chunk_elems(dtype) != 0) return SS_ERR_INVALID_ARG;
    return SS_OK;
}

// Parts into which the sums of a rows x dim gradient over `depth` terms are cut.  dx (sums over the
// weights' rows) and the weights' gradients (sums over x's rows) are formed by one launch: where one
// of them has few tiles, each with a far longer sum than the other's, those would end long after
// the rest.  Its sums are cut to the others' length, but not below 16 k tiles, nor into more than fill
// the chip twice over.
int64_t grad_parts(int64_t rows, int64_t dim, int64_t depth, ss_dtype dtype)
{
    const int64_t bk = 8 * chunk_elems(dtype);
    const int64_t own = ceil_div(depth, bk), others = ceil_div(rows, bk);
    const int64_t tiles = ceil_div(rows, 128) * ceil_div(dim, 128);
    int64_t s = own / (others > 16 ? others : 16);
    const int64_t most = 1024 / tiles;
    s = s < most ? s : most;
    return s > 1 ? s : 1;
}

// How the products of `rows` rows of x with `cols` weight rows are formed (both directions), and
// their gradients.
struct RowsPlan {
    bool aligned;  // rows are of whole 16-byte chunks
    bool stream;   // the weights stream past x; else tiles
    bool few;      // the gradients in one pass over the weights
    bool pad;      // padded copies are needed: bf16 tiles read them (in the forward, or the backward)
};
// Streaming reads x again for every 32 weight rows, from the caches, which costs more the more rows
// there are; tiles of 128 weight rows cost the same up to 64 rows, but leave CUs idle while there
// are fewer than 256 of them.  Times in us, streamed and in tiles, k = 2560:
//   bf16,   43 tiles:  1 row 10 19, 64 rows 18 26;   108: 1 row 14 27, 32 rows 21 27, 64 rows 31 27;
//          216 tiles:  8 rows 28 29, 16 rows 32 29;  313: 1 row 33 31;   432: 1 row 53 47, 16 rows 72 48;
//   fp32, 108 tiles: 64 rows 73 103;  216: 32 rows 97 114, 64 rows 162 115;  432: 16 rows 160 170.
// At other k the times' proportions may differ.
// bf16 rows that are not whole 16-byte chunks would need padded copies of the weights for tiles, and
// are always streamed.
// The gradients in one pass save a second reading of the weights (and padded copies), at 2 m
// multiply-adds per element on the vector units.  Times in us of both passes so and in tiles:
//   bf16, 2560 -> 2 x 6912: 1 row 78 88, 4 rows 83 86, 8 rows 98 88;  768 -> 2 x 2048: 1 row 39 33;
//   bf16, 2561 -> 2 x 6913: 1 row 121 188, 8 rows 160 204, 16 rows 237 216;
//   fp32, 2560 -> 2 x 6912: 1 row 119 142, 8 rows 139 149, 16 rows 178 158.
constexpr int64_t kFewAligned = 4, kFewWeights = int64_t(16) << 20;  // bf16: rows, elements of the weights
RowsPlan rows_plan(int64_t rows, int64_t dim, int64_t cols, ss_dtype dtype, bool back)
{
    RowsPlan p;
    p.aligned = dim % chunk_elems(dtype) == 0;
    const int64_t tiles = ceil_div(cols, 128), idle = tiles < 256 ? 256 - tiles : 0;
    if (dtype == SS_F32) {
        p.stream = rows <= 16 || (rows <= ssk::kStreamRows && rows <= idle);
        p.few = rows <= ssk::kFewRows;
    } else if (p.aligned) {
        p.stream = rows <= ssk::kStreamRows && rows * 16 <= idle * 5;
        p.few = rows <= kFewAligned && cols * dim >= kFewWeights;
    } else {
        p.stream = rows <= ssk::kStreamRows;
        p.few = rows <= ssk::kFewRows;
    }
    p.pad = dtype == SS_BF16 && !p.aligned && (back ? !p.few : !p.stream);
    return p;
}

// Parts of dx when few: enough ranges of the weights' rows for eight workgroups (of 512 columns) per
// CU, of at least 8 rows, and few enough that the parts stay a quarter of the weights' size, or small.
// A narrow x has up to 2048 of them, which few_sum_kernel adds by one thread per element: 2 rows, 276
// wide, against 65098 weight rows, loss and gradients, take 147 us for 15 at a copy's rate.
void few_parts(int64_t m, int64_t k, int64_t rows, ss_dtype dtype, int64_t* per, int64_t* parts)
{
    constexpr int64_t kSmall = int64_t(8) << 20;
    int64_t s = 2048 / ceil_div(k, 512);
    const int64_t by_rows = rows / 8;
    int64_t by_size = rows * elem_size(dtype) / (16 * m);
    const int64_t small = kSmall / (4 * m * k);
    by_size = by_size > small ? by_size : small;
    s = s < by_rows ? s : by_rows;
    s = s < by_size ? s : by_size;
    s = s > 1 ? s : 1;
    *per = ceil_div(rows, s);
    *parts = ceil_div(rows, *per);
}

struct GluLayout {
    int64_t k_pad, f_pad, splits, per, dw_splits;
    RowsPlan plan;
    bool pack, lo;
    int64_t x, wg, wu, dgu, part, dw_part, total;
};

bool glu_layout(int64_t m, int64_t k, int64_t f, ss_dtype dtype, bool back, GluLayout* w)
{
    if (!mat_sizes(m, k, f) || !known(dtype)) return false;
    const int64_t es = elem_size(dtype);
    w->k_pad = padded(k, dtype);
    w->f_pad = padded(f, dtype);
    w->plan = rows_plan(m, k, 2 * f, dtype, back);
    w->pack = w->plan.pad;
    Regions r;
    w->x = r.add(w->pack ? m * w->k_pad : 0, es);
    w->wg = r.add(w->pack ? f * w->k_pad : 0, es);
    w->wu = r.add(w->pack ? f * w->k_pad : 0, es);
    w->lo = dtype == SS_BF16 && !w->plan.few && m <= ssk::kGluLoRows;
    w->dgu = r.add(back ? (w->lo ? 2 * m : m) * 2 * w->f_pad : 0, w->plan.few ? 4 : es);
    w->per = 0;
    if (w->plan.few)
        few_parts(m, k, 2 * f, dtype, &w->per, &w->splits);
    else
        w->splits = grad_parts(m, k, 2 * f, dtype);
    int64_t part;
    if (!mul(w->splits, m, &part) || !mul(part, k, &part)) return false;
    w->part = r.add(back && (w->splits > 1 || w->plan.few) ? part : 0, 4);
    w->dw_splits = w->plan.few ? 1 : grad_parts(2 * w->f_pad, k, m, dtype);
    if (!mul(w->dw_splits, 2 * w->f_pad, &part) || !mul(part, k, &part)) return false;
    w->dw_part = r.add(back && w->dw_splits > 1 ? part : 0, 4);
    w->total = r.at;
    return r.ok;
}

struct XentLayout {
    int64_t d_pad, piece, splits, per, dw_splits;
    RowsPlan plan;
    bool pack;
    int64_t x, w, pmax, psum, tl, dl, lo, tokens, counts, acc, dw_part, total;
};

// Columns per piece of the backward: as many as keep the piece's gradient of the logits within
// kXentPieceBytes (it is written once and read twice, so it had better stay in the last-level
// cache), but no fewer than kXentMinPiece (each piece reads and writes the fp32 sums of dx).
// Pieces are evened out, in whole tiles of 256 columns.  Loss and gradients of 8192 tokens, 2560
// wide, 50257 entries with 64 MB, 256 MB and 1 GB: 8.0, 7.5 and 7.5 ms.
constexpr int64_t kXentPieceBytes = int64_t(256) << 20, kXentMinPiece = 4096;

int64_t xent_piece(int64_t n, int64_t v, int64_t es)
{
    int64_t most = kXentPieceBytes / (n * es);
    most = most > kXentMinPiece ? most : kXentMinPiece;
    const int64_t count = ceil_div(v, most);
    const int64_t even = ceil_div(ceil_div(v, count), 256) * 256;
    return even < v ? even : v;
}

bool xent_layout(int64_t n, int64_t d, int64_t v, ss_dtype dtype, bool back, XentLayout* w)
{
    if (!mat_sizes(n, d, v) || !known(dtype)) return false;
    const int64_t es = elem_size(dtype);
    w->d_pad = padded(d, dtype);
    w->plan = rows_plan(n, d, v, dtype, back);
    w->pack = w->plan.pad;
    w->piece = w->plan.few ? v : xent_piece(n, v, es);
    Regions r;
    w->x = r.add(w->pack ? n * w->d_pad : 0, es);
    w->w = r.add(w->pack ? v * w->d_pad : 0, es);
    const int64_t parts = back ? 0 : ceil_div(v, w->plan.stream ? ssk::kXentStreamCols : ssk::kXentCols) * n;
    w->pmax = r.add(parts, 4);
    w->psum = r.add(parts, 4);
    w->tl = r.add(back ? 0 : n, 4);
    w->dl = r.add(back ? n * (ceil_div(w->piece, 16) * 16) : 0, w->plan.few ? 4 : es);
    const bool listed = back && dtype == SS_BF16 && !w->plan.few;
    const int64_t groups = ceil_div(v, ssk::kXentCols);
    w->lo = r.add(listed ? n : 0, 4);
    w->tokens = r.add(listed ? groups * n : 0, 4);
    w->counts = r.add(listed ? groups : 0, 4);
    w->per = 0;
    if (w->plan.few)
        few_parts(n, d, v, dtype, &w->per, &w->splits);
    else
        w->splits = grad_parts(n, d, w->piece, dtype);
    int64_t sums;
    if (!mul(w->splits, n, &sums) || !mul(sums, d, &sums)) return false;
    w->acc = r.add(back && (w->piece < v || w->splits > 1 || w->plan.few) ? sums : 0, 4);
    w->dw_splits = w->plan.few ? 1 : grad_parts(w->piece, d, n, dtype);
    if (!mul(w->dw_splits, w->piece, &sums) || !mul(sums, d, &sums)) return false;
    w->dw_part = r.add(back && w->dw_splits > 1 ? sums : 0, 4);
    w->total = r.at;
    return r.ok;
}

}  // namespace

extern "C" {

size_t ss_glu_workspace_bytes(int64_t tokens, int64_t dim, int64_t features, ss_dtype dtype)
{
    GluLayout w;
    return glu_layout(tokens, dim, features, dtype, false, &w) ? static_cast<size_t>(w.total) : kBad;
}

size_t ss_glu_bwd_workspace_bytes(int64_t tokens, int64_t dim, int64_t features, ss_dtype dtype)
{
    GluLayout w;
    return glu_layout(tokens, dim, features, dtype, true, &w) ? static_cast<size_t>(w.total) : kBad;
}

}  // extern "C"

namespace {

// Both directions: h for the forward; dh, dx, dwg and dwu for the backward.
ss_status glu_impl(const void* x, int64_t x_ld, const void* wg, const void* wu, void* h, const void* dh, void* dx,
                   void* dwg, void* dwu, bool back, ss_activation act, void* workspace, size_t workspace_bytes,
                   int64_t m, int64_t k, int64_t f, ss_dtype dtype, hipStream_t stream)
{
    if (!x || !wg || !wu || (back ? !dh : !h)) return SS_ERR_INVALID_ARG;
    if (back && ((dwg == nullptr) != (dwu == nullptr) || (!dx && !dwg))) return SS_ERR_INVALID_ARG;
    if (!mat_sizes(m, k, f)) return SS_ERR_INVALID_ARG;
    if (!known(dtype) || (act != SS_ACT_SILU && act != SS_ACT_GELU)) return SS_ERR_UNSUPPORTED;
    GluLayout w;
    if (!glu_layout(m, k, f, dtype, back, &w)) return SS_ERR_INVALID_ARG;
    if (!mat_grid_ok(m, f) || !mat_grid_ok(m, k) || !mat_grid_ok(2 * w.f_pad, k)) return SS_ERR_UNSUPPORTED;
    if (w.plan.stream ? !launch_fits(ceil_div(w.f_pad, 16), 256) : !tiles_fit({m, 2 * w.f_pad, 1}, {0, 0, 0}, dtype))
        return SS_ERR_UNSUPPORTED;
    if (back && (w.plan.few ? !few_fits(m, k)
                            : !tiles_fit({m, k, dx ? w.splits : 0}, {2 * w.f_pad, k, dwg ? w.dw_splits : 0}, dtype)))
        return SS_ERR_UNSUPPORTED;
    const int64_t es = elem_size(dtype);
    bool pack;
    ss_status st = mat_operand(x, x_ld, k, dtype, &pack);
    if (st != SS_OK) return st;
    const void* weights[] = {wg, wu};
    for (const void* p : weights) {
        st = mat_operand(p, k, k, dtype, &pack);
        if (st != SS_OK) return st;
    }
    const void* elems[] = {h, dh, dx, dwg, dwu};
    for (const void* p : elems)
        if (!aligned(p, uintptr_t(es))) return SS_ERR_INVALID_ARG;
    int64_t xb;
    if (!strided_bytes(m, k, x_ld, es, &xb)) return SS_ERR_INVALID_ARG;
    const Range all[] = {span(x, xb), span(wg, f * k * es), span(wu, f * k * es), span(dh, m * f * es),
                         span(h, m * f * es), span(dx, m * k * es), span(dwg, f * k * es), span(dwu, f * k * es)};
    if (any_overlap(all + 4, 4, all, 4)) return SS_ERR_INVALID_ARG;
    st = check_workspace(workspace, workspace_bytes, w.total, all, 8);
    if (st != SS_OK) return st;

    char* const ws = static_cast<char*>(workspace);
    const int dt = dtype == SS_F32 ? 0 : 1;
    ssk::GluArgs a{};
    a.x = x;
    a.x_ld = x_ld;
    a.wg = wg;
    a.wu = wu;
    a.w_ld = k;
    a.h = h;
    a.dh = dh;
    a.dgu = ws ? ws + w.dgu : nullptr;
    a.lo = w.lo;
    a.dx = dx;
    a.dwg = dwg;
    a.dwu = dwu;
    a.m = m;
    a.k = k;
    a.f = f;
    a.f_pad = w.f_pad;
    a.k_pad = w.k_pad;
    a.dx_splits = w.splits;
    a.dx_per = w.per;
    a.dx_part = back && dx && (w.splits > 1 || w.plan.few) ? reinterpret_cast<float*>(ws + w.part) : nullptr;
    a.dw_splits = w.dw_splits;
    a.dw_part = back && dwg && w.dw_splits > 1 ? reinterpret_cast<float*>(ws + w.dw_part) : nullptr;
    a.act = act == SS_ACT_SILU ? ssk::kActSilu : ssk::kActGelu;
    a.x_raw = x;
    a.x_raw_ld = x_ld;
    a.wg_raw = wg;
    a.wu_raw = wu;
    a.aligned = w.plan.aligned && whole_rows(x, x_ld, dtype) && whole_rows(wg, k, dtype) && whole_rows(wu, k, dtype);
    a.stream = w.plan.stream;
    a.few = w.plan.few;
    if (w.pack) {
        // after a streamed product, tiles read x for the weights' gradients and the weights for dx
        const bool few = w.plan.stream;
        hipError_t e = hipSuccess;
        if (!few || dwg) e = ssk::launch_pad_rows(x, x_ld, ws + w.x, m, k, w.k_pad, dt, stream);
        if (e == hipSuccess && (!few || dx)) e = ssk::launch_pad_rows(wg, k, ws + w.wg, f, k, w.k_pad, dt, stream);
        if (e == hipSuccess && (!few || dx)) e = ssk::launch_pad_rows(wu, k, ws + w.wu, f, k, w.k_pad, dt, stream);
        if (e != hipSuccess) return done(e);
        a.x = ws + w.x;
        a.wg = ws + w.wg;
        a.wu = ws + w.wu;
        a.x_ld = a.w_ld = w.k_pad;
    }
    return done(back ? ssk::launch_glu_bwd(a, dt, stream) : ssk::launch_glu_fwd(a, dt, stream));
}

ss_status xent_impl(const void* x, int64_t x_ld, const void* weight, const int64_t* target, int64_t ignore_index,
                    float* loss, float* lse_out, const float* lse_in, const float* dloss, void* dx, void* dw,
                    bool back, void* workspace, size_t workspace_bytes, int64_t n, int64_t d, int64_t v,
                    ss_dtype dtype, hipStream_t stream)
{
    if (!x || !weight || !target) return SS_ERR_INVALID_ARG;
    if (back ? (!lse_in || !dloss || (!dx && !dw)) : (!loss || !lse_out)) return SS_ERR_INVALID_ARG;
    if (!mat_sizes(n, d, v)) return SS_ERR_INVALID_ARG;
    if (!known(dtype)) return SS_ERR_UNSUPPORTED;
    XentLayout w;
    if (!xent_layout(n, d, v, dtype, back, &w)) return SS_ERR_INVALID_ARG;
    if (!mat_grid_ok(n, v) || !mat_grid_ok(n, d) || !mat_grid_ok(v, d) || n > INT32_MAX) return SS_ERR_UNSUPPORTED;
    // a piece (the forward's is the whole vocabulary), and the last one
    const int64_t piece = back ? w.piece : v;
    const int64_t pieces[] = {piece, v - (ceil_div(v, piece) - 1) * piece};
    for (const int64_t cols : pieces) {
        const int64_t width = back ? ceil_div(cols, 16) * 16 : cols;
        if (w.plan.stream ? !launch_fits(ceil_div(width, ssk::kXentStreamCols), 256)
                          : !tiles_fit({n, width, 1}, {0, 0, 0}, dtype))
            return SS_ERR_UNSUPPORTED;
        if (back && (w.plan.few ? !few_fits(n, d)
                                : !tiles_fit({n, d, dx ? w.splits : 0}, {cols, d, dw ? w.dw_splits : 0}, dtype)))
            return SS_ERR_UNSUPPORTED;
    }
    // the lists of targets; the forward's join
    if (back ? dw && !launch_fits(ceil_div(v, ssk::kXentCols), 256) : !launch_fits(ceil_div(n, n >= 4096 ? 16 : 2), 256))
        return SS_ERR_UNSUPPORTED;
    const int64_t es = elem_size(dtype);
    bool pack;
    ss_status st = mat_operand(x, x_ld, d, dtype, &pack);
    if (st == SS_OK) st = mat_operand(weight, d, d, dtype, &pack);
    if (st != SS_OK) return st;
    if (!aligned(target, 8) || !aligned(dx, uintptr_t(es)) || !aligned(dw, uintptr_t(es))) return SS_ERR_INVALID_ARG;
    const void* words[] = {loss, lse_out, lse_in, dloss};
    for (const void* p : words)
        if (!aligned(p, 4)) return SS_ERR_INVALID_ARG;
    int64_t xb;
    if (!strided_bytes(n, d, x_ld, es, &xb)) return SS_ERR_INVALID_ARG;
    const Range all[] = {span(x, xb), span(weight, v * d * es), span(target, n * 8), span(lse_in, n * 4),
                         span(dloss, n * 4), span(loss, n * 4), span(lse_out, n * 4), span(dx, n * d * es),
                         span(dw, v * d * es)};
    if (any_overlap(all + 5, 4, all, 5)) return SS_ERR_INVALID_ARG;
    st = check_workspace(workspace, workspace_bytes, w.total, all, 9);
    if (st != SS_OK) return st;

    char* const ws = static_cast<char*>(workspace);
    const int dt = dtype == SS_F32 ? 0 : 1;
    ssk::XentArgs a{};
    a.x = x;
    a.x_ld = x_ld;
    a.w = weight;
    a.w_ld = d;
    a.target = target;
    a.ignore_index = ignore_index;
    a.loss = loss;
    a.lse = back ? const_cast<float*>(lse_in) : lse_out;  // the backward only reads it
    a.dloss = dloss;
    a.dx = dx;
    a.dw = dw;
    a.n = n;
    a.d = d;
    a.v = v;
    a.d_pad = w.d_pad;
    a.piece = w.piece;
    a.part_max = reinterpret_cast<float*>(ws + w.pmax);
    a.part_sum = reinterpret_cast<float*>(ws + w.psum);
    a.target_logit = reinterpret_cast<float*>(ws + w.tl);
    a.dl = ws + w.dl;
    a.lo = reinterpret_cast<float*>(ws + w.lo);
    a.tokens = reinterpret_cast<int32_t*>(ws + w.tokens);
    a.counts = reinterpret_cast<int32_t*>(ws + w.counts);
    a.dx_splits = w.splits;
    a.dw_splits = w.dw_splits;
    a.dw_part = w.dw_splits > 1 ? reinterpret_cast<float*>(ws + w.dw_part) : nullptr;
    a.dx_per = w.per;
    a.dx_acc = w.piece < v || w.splits > 1 || w.plan.few ? reinterpret_cast<float*>(ws + w.acc) : nullptr;
    a.x_raw = x;
    a.x_raw_ld = x_ld;
    a.w_raw = weight;
    a.aligned = w.plan.aligned && whole_rows(x, x_ld, dtype) && whole_rows(weight, d, dtype);
    a.stream = w.plan.stream;
    a.few = w.plan.few;
    if (w.pack) {
        // after a streamed product, tiles read x for dw and w for dx
        const bool few = w.plan.stream;
        hipError_t e = hipSuccess;
        if (!few || dw) e = ssk::launch_pad_rows(x, x_ld, ws + w.x, n, d, w.d_pad, dt, stream);
        if (e == hipSuccess && (!few || dx)) e = ssk::launch_pad_rows(weight, d, ws + w.w, v, d, w.d_pad, dt, stream);
        if (e != hipSuccess) return done(e);
        a.x = ws + w.x;
        a.w = ws + w.w;
        a.x_ld = a.w_ld = w.d_pad;
    }
    return done(back ? ssk::launch_xent_bwd(a, dt, stream) : ssk::launch_xent_fwd(a, dt, stream));
}

}  // namespace

extern "C" {

ss_status ss_glu_fwd(const void* x, int64_t x_row_stride, const void* w_gate, const void* w_up, void* h,
                     ss_activation act, void* workspace, size_t workspace_bytes, int64_t tokens, int64_t dim,
                     int64_t features, ss_dtype dtype, hipStream_t stream)
{
    return glu_impl(x, x_row_stride, w_gate, w_up, h, nullptr, nullptr, nullptr, nullptr, false, act, workspace,
                    workspace_bytes, tokens, dim, features, dtype, stream);
}

ss_status ss_glu_bwd(const void* x, int64_t x_row_stride, const void* w_gate, const void* w_up, const void* dh,
                     void* dx, void* dw_gate, void* dw_up, ss_activation act, void* workspace,
                     size_t workspace_bytes, int64_t tokens, int64_t dim, int64_t features, ss_dtype dtype,
                     hipStream_t stream)
{
    return glu_impl(x, x_row_stride, w_gate, w_up, nullptr, dh, dx, dw_gate, dw_up, true, act, workspace,
                    workspace_bytes, tokens, dim, features, dtype, stream);
}

size_t ss_xent_workspace_bytes(int64_t tokens, int64_t dim, int64_t vocab, ss_dtype dtype)
{
    XentLayout w;
    return xent_layout(tokens, dim, vocab, dtype, false, &w) ? static_cast<size_t>(w.total) : kBad;
}

size_t ss_xent_bwd_workspace_bytes(int64_t tokens, int64_t dim, int64_t vocab, ss_dtype dtype)
{
    XentLayout w;
    return xent_layout(tokens, dim, vocab, dtype, true, &w) ? static_cast<size_t>(w.total) : kBad;
}

ss_status ss_xent_fwd(const void* x, int64_t x_row_stride, const void* w, const int64_t* target,
                      int64_t ignore_index, float* loss, float* lse, void* workspace, size_t workspace_bytes,
                      int64_t tokens, int64_t dim, int64_t vocab, ss_dtype dtype, hipStream_t stream)
{
    return xent_impl(x, x_row_stride, w, target, ignore_index, loss, lse, nullptr, nullptr, nullptr, nullptr, false,
                     workspace, workspace_bytes, tokens, dim, vocab, dtype, stream);
}

ss_status ss_xent_bwd(const void* x, int64_t x_row_stride, const void* w, const int64_t* target,
                      int64_t ignore_index, const float* lse, const float* dloss, void* dx, void* dw,
                      void* workspace, size_t workspace_bytes, int64_t tokens, int64_t dim, int64_t vocab,
                      ss_dtype dtype, hipStream_t stream)
{
    return xent_impl(x, x_row_stride, w, target, ignore_index, nullptr, nullptr, lse, dloss, dx, dw, true, workspace,
                     workspace_bytes, tokens, dim, vocab, dtype, stream);
}

}  // extern "C"
