// C ABI of linear attention, of the norms of its queries and keys, and of sampling (ss_attn.h):
// argument validation, plans, workspace sizing and kernel dispatch.  Validation runs on the host
// before anything is enqueued.
#include <math.h>
#include <stdint.h>

#include <initializer_list>

#include "ss_attn.h"
#include "ss_attn_internal.h"
#include "ss_host.h"

namespace {

// ---- linear attention -------------------------------------------------------------------

struct LattnDims {
    int64_t batch, seqlen, qk_heads, heads, dk, dv;
    int64_t share() const { return heads / qk_heads; }
    int64_t cells() const { return dk * dv; }
    int64_t states() const { return batch * heads * cells(); }
};

// Sizes are positive, heads shared evenly, and every element count of an operand, in bytes, fits 63 bits.
bool lattn_sizes(const LattnDims& d)
{
    int64_t n;
    if (d.batch <= 0 || d.seqlen <= 0 || d.qk_heads <= 0 || d.heads <= 0 || d.dk <= 0 || d.dv <= 0) return false;
    if (d.heads % d.qk_heads != 0) return false;
    return mul(d.batch, d.seqlen, &n) && mul(n, d.heads, &n) && mul(n, d.dk > d.dv ? d.dk : d.dv, &n) && mul(n, 4, &n) &&
           mul(d.batch, d.heads, &n) && mul(n, d.dk, &n) && mul(n, d.dv, &n) && mul(n, 4, &n);
}

bool lattn_widths(const LattnDims& d) { return d.dk <= ssk::kLattnMaxDim && d.dv <= ssk::kLattnMaxDim; }

// How a walk is cut into segments of the sequence: so that a launch has as many workgroups as the CUs hold
// beside each other, in segments of at least two chunks of the kernel's.  The cut costs a pass over k and v that forms the states
// between the segments, two fifths of a walk, and two launches: in bf16 fewer than four segments do not
// pay for it, in fp32 fewer than three.  Whole and cut, us, of 2048 rows in bf16: 16 walks 108 and 34, 64
// walks 109 and 72, 128 walks 116 and 110 (in four), 200 walks 132 and 183 (in two); 16 walks of 256 rows 19
// and 25 (in two), of 512 rows 32 and 27 (in four).  fp32: 64 walks 310 and 127, 128 walks 310 and 237 (in
// four), 192 walks 318 and 354 (in two), 200 walks 311 and 371 (in two).  Segments of one chunk and two, bf16:
// 16 walks of 256 rows 23 and 20 (whole), of 512 rows 25 and 29, of 2048 rows 41 and 35; fp32: 16 walks of
// 128 rows 30 and 25 (whole), of 2048 rows the same.  Of two chunks and four, fp32: 16 walks of 256 rows 31
// and 43 (whole), of 512 rows 33 and 45, of 2048 rows 60 and 56.
constexpr int64_t kLattnMaxSegs = 256;

struct LattnCut {
    int64_t len, segs;  // rows of a segment, segments
};

// For a launch of `jobs` walks with widths dk and dv of each head.
LattnCut lattn_cut(const LattnDims& d, ss_dtype dtype, int jobs, int64_t dk, int64_t dv)
{
    const int dt = dtype == SS_F32 ? 0 : 1;
    const int64_t walks = jobs * d.batch * d.heads * ssk::lattn_slices(dv);
    const int64_t target = 256 * ssk::lattn_resident(dt, int(dk), int(dv)), least = dt == 0 ? 3 : 4, chunk = ssk::lattn_chunk(dt, int(dk), int(dv));
    const int64_t most = d.seqlen / (2 * chunk);
    int64_t k = target / walks;
    k = k < most ? k : most;
    k = k < kLattnMaxSegs ? k : kLattnMaxSegs;
    if (k < least) k = 1;
    const int64_t len = ceil_div(ceil_div(d.seqlen, k), chunk) * chunk;
    return {len, ceil_div(d.seqlen, len)};
}

// Whether the backward's three walks, of widths (dk, dv) and (dv, dk), go in one launch.
bool lattn_together(const LattnDims& d) { return ssk::lattn_class(int(d.dk), int(d.dv)) == ssk::lattn_class(int(d.dv), int(d.dk)); }

struct LattnLayout {
    LattnCut cut[3];  // of each walk: the forward's, or dv's, dk's and dq's
    int64_t seg[3], keep[3], part[2];
    int64_t total;
};

bool lattn_layout(const LattnDims& d, ss_dtype dtype, bool back, LattnLayout* w)
{
    if (!lattn_sizes(d)) return false;
    int64_t walks, n, f;
    if (!mul(d.batch, d.heads, &walks) || !mul(walks, 6, &n)) return false;
    const bool three = back && lattn_together(d);
    w->cut[0] = lattn_cut(d, dtype, three ? 3 : 1, d.dk, d.dv);
    w->cut[1] = w->cut[2] = three ? w->cut[0] : lattn_cut(d, dtype, 2, d.dv, d.dk);
    Regions r;
    for (int i = 0; i < (back ? 3 : 1); ++i) {
        const int64_t segs = w->cut[i].segs;
        if (!mul(segs, d.states(), &n) || !mul(segs, walks, &f)) return false;
        w->seg[i] = r.add(segs > 1 ? n : 0, 4);
        w->keep[i] = r.add(segs > 1 ? f : 0, 4);
    }
    for (int i = 0; i < 2; ++i) w->part[i] = r.add(back && d.share() > 1 ? d.batch * d.seqlen * d.heads * d.dk : 0, 4);
    w->total = r.at;
    return r.ok;
}

// Rows' strides that the kernels' 32-bit offsets over a chunk take, in elements: the inputs', which a
// sequence of one row has none of, and the outputs' (row, 0 where there is no second one).
constexpr int64_t kLattnMaxStride = int64_t(1) << 20;
bool lattn_too_wide(int64_t seqlen, std::initializer_list<int64_t> in, int64_t row, int64_t other)
{
    for (const int64_t ld : in)
        if (seqlen > 1 && ld > kLattnMaxStride) return true;
    return row > kLattnMaxStride || other > kLattnMaxStride;
}

// Whether a launch of `jobs` walks of width dv fits a grid.
bool lattn_fits(const LattnDims& d, int64_t dv, int jobs, int64_t segs)
{
    int64_t n;
    // counted as the kernel's launch does, which then cannot overflow
    return mul(d.batch * d.heads, segs, &n) && n <= UINT32_MAX &&
           launch_fits(ssk::lattn_groups(d.batch, d.heads, dv, jobs, segs), 64 * ssk::lattn_waves(dv));
}

// Whether every launch of a direction fits a grid, and a sequence's rows their counters.
bool lattn_grid_ok(const LattnDims& d, const LattnLayout& w, bool back)
{
    if (d.seqlen >= int64_t(1) << 30) return false;
    if (!back) return lattn_fits(d, d.dv, 1, w.cut[0].segs);
    if (lattn_together(d)) return lattn_fits(d, d.dv, 3, w.cut[0].segs);
    return lattn_fits(d, d.dv, 1, w.cut[0].segs) && lattn_fits(d, d.dk, 2, w.cut[1].segs);
}

size_t lattn_bytes(const LattnDims& d, ss_dtype dtype, bool back)
{
    LattnLayout w;
    if (!known(dtype) || !lattn_sizes(d) || !lattn_widths(d)) return kBad;
    return lattn_layout(d, dtype, back, &w) ? static_cast<size_t>(w.total) : kBad;
}

ssk::LattnArgs lattn_args(const LattnDims& d, const LattnCut& cut, const float* log_decay, const uint8_t* reset)
{
    ssk::LattnArgs a{};
    a.log_decay = log_decay;
    a.reset = reset;
    a.batch = d.batch;
    a.seqlen = d.seqlen;
    a.heads = d.heads;
    a.seg_len = cut.len;
    a.segs = cut.segs;
    return a;
}

}  // namespace

extern "C" {

size_t ss_lattn_workspace_bytes(int64_t batch, int64_t seqlen, int64_t qk_heads, int64_t heads, int64_t k_dim,
                                int64_t v_dim, ss_dtype dtype)
{
    return lattn_bytes({batch, seqlen, qk_heads, heads, k_dim, v_dim}, dtype, false);
}

size_t ss_lattn_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t qk_heads, int64_t heads, int64_t k_dim,
                                    int64_t v_dim, ss_dtype dtype)
{
    return lattn_bytes({batch, seqlen, qk_heads, heads, k_dim, v_dim}, dtype, true);
}

ss_status ss_lattn_fwd(const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride, const void* v,
                       int64_t v_row_stride, const float* log_decay, float scale, const float* h0,
                       const uint8_t* reset, void* o, float* h_last, void* workspace, size_t workspace_bytes,
                       int64_t batch, int64_t seqlen, int64_t qk_heads, int64_t heads, int64_t k_dim, int64_t v_dim,
                       ss_dtype dtype, hipStream_t stream)
{
    if (!q || !k || !v || !log_decay || !o) return SS_ERR_INVALID_ARG;
    const LattnDims d{batch, seqlen, qk_heads, heads, k_dim, v_dim};
    LattnLayout w;
    if (!lattn_sizes(d) || !isfinite(scale)) return SS_ERR_INVALID_ARG;
    if (q_row_stride < qk_heads * k_dim || k_row_stride < qk_heads * k_dim || v_row_stride < heads * v_dim)
        return SS_ERR_INVALID_ARG;
    if (!known(dtype) || !lattn_widths(d)) return SS_ERR_UNSUPPORTED;
    if (!lattn_layout(d, dtype, false, &w)) return SS_ERR_INVALID_ARG;
    if (!lattn_grid_ok(d, w, false) || lattn_too_wide(seqlen, {q_row_stride, k_row_stride, v_row_stride}, heads * v_dim, 0))
        return SS_ERR_UNSUPPORTED;
    const int64_t es = elem_size(dtype), rows = batch * seqlen;
    const void* elems[] = {q, k, v, o};
    for (const void* p : elems)
        if (!aligned(p, uintptr_t(es))) return SS_ERR_INVALID_ARG;
    const void* words[] = {log_decay, h0, h_last};
    for (const void* p : words)
        if (!aligned(p, 4)) return SS_ERR_INVALID_ARG;
    int64_t qb, kb, vb;
    if (!strided_bytes(rows, qk_heads * k_dim, q_row_stride, es, &qb) ||
        !strided_bytes(rows, qk_heads * k_dim, k_row_stride, es, &kb) ||
        !strided_bytes(rows, heads * v_dim, v_row_stride, es, &vb))
        return SS_ERR_INVALID_ARG;
    const int64_t state = d.states() * 4;
    const Range all[] = {span(q, qb), span(k, kb), span(v, vb), span(log_decay, heads * 4), span(reset, rows),
                         span(h0, state), span(o, rows * heads * v_dim * es), span(h_last, state)};
    if (any_overlap(all + 6, 2, all, 5)) return SS_ERR_INVALID_ARG;
    if (overlap(all[6], all[5]) || (overlap(all[7], all[5]) && h_last != h0)) return SS_ERR_INVALID_ARG;
    const ss_status st = check_workspace(workspace, workspace_bytes, w.total, all, 8);
    if (st != SS_OK) return st;

    char* const ws = static_cast<char*>(workspace);
    ssk::LattnArgs a = lattn_args(d, w.cut[0], log_decay, reset);
    ssk::LattnJob& j = a.job[0];
    j = {q, k, v, q_row_stride, k_row_stride, v_row_stride, int(d.share()), int(d.share()), 1, int(k_dim), int(v_dim),
         o, false, false, h0, h_last, v_dim, 1, scale, 1.0f, scale, nullptr, nullptr};
    if (a.segs > 1) {
        j.seg = reinterpret_cast<float*>(ws + w.seg[0]);
        j.keep = reinterpret_cast<float*>(ws + w.keep[0]);
    }
    a.jobs = 1;
    return done(ssk::launch_lattn(a, dtype == SS_F32 ? 0 : 1, stream));
}

ss_status ss_lattn_bwd(const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride, const void* v,
                       int64_t v_row_stride, const float* log_decay, float scale, const float* h0,
                       const uint8_t* reset, const void* d_o, int64_t do_row_stride, const float* dh_last, void* dq,
                       void* dk, void* dv, float* dh0, void* workspace, size_t workspace_bytes, int64_t batch,
                       int64_t seqlen, int64_t qk_heads, int64_t heads, int64_t k_dim, int64_t v_dim, ss_dtype dtype,
                       hipStream_t stream)
{
    if (!q || !k || !v || !log_decay || !d_o || !dq || !dk || !dv) return SS_ERR_INVALID_ARG;
    const LattnDims d{batch, seqlen, qk_heads, heads, k_dim, v_dim};
    LattnLayout w;
    if (!lattn_sizes(d) || !isfinite(scale)) return SS_ERR_INVALID_ARG;
    if (q_row_stride < qk_heads * k_dim || k_row_stride < qk_heads * k_dim || v_row_stride < heads * v_dim ||
        do_row_stride < heads * v_dim)
        return SS_ERR_INVALID_ARG;
    if (!known(dtype) || !lattn_widths(d)) return SS_ERR_UNSUPPORTED;
    if (!lattn_layout(d, dtype, true, &w)) return SS_ERR_INVALID_ARG;
    if (!lattn_grid_ok(d, w, true) ||
        lattn_too_wide(seqlen, {q_row_stride, k_row_stride, v_row_stride, do_row_stride}, heads * k_dim, heads * v_dim))
        return SS_ERR_UNSUPPORTED;
    const int64_t es = elem_size(dtype), rows = batch * seqlen;
    const void* elems[] = {q, k, v, d_o, dq, dk, dv};
    for (const void* p : elems)
        if (!aligned(p, uintptr_t(es))) return SS_ERR_INVALID_ARG;
    const void* words[] = {log_decay, h0, dh_last, dh0};
    for (const void* p : words)
        if (!aligned(p, 4)) return SS_ERR_INVALID_ARG;
    int64_t qb, kb, vb, ob;
    if (!strided_bytes(rows, qk_heads * k_dim, q_row_stride, es, &qb) ||
        !strided_bytes(rows, qk_heads * k_dim, k_row_stride, es, &kb) ||
        !strided_bytes(rows, heads * v_dim, v_row_stride, es, &vb) ||
        !strided_bytes(rows, heads * v_dim, do_row_stride, es, &ob))
        return SS_ERR_INVALID_ARG;
    const int64_t state = d.states() * 4, qk = rows * qk_heads * k_dim * es;
    const Range all[] = {span(q, qb), span(k, kb), span(v, vb), span(d_o, ob), span(log_decay, heads * 4),
                         span(reset, rows), span(h0, state), span(dh_last, state),
                         span(dq, qk), span(dk, qk), span(dv, rows * heads * v_dim * es), span(dh0, state)};
    if (any_overlap(all + 8, 4, all, 8)) return SS_ERR_INVALID_ARG;
    const ss_status st = check_workspace(workspace, workspace_bytes, w.total, all, 12);
    if (st != SS_OK) return st;

    char* const ws = static_cast<char*>(workspace);
    const int share = int(d.share()), ki = int(k_dim), vi = int(v_dim);
    float* const part_q = share > 1 ? reinterpret_cast<float*>(ws + w.part[0]) : nullptr;
    float* const part_k = share > 1 ? reinterpret_cast<float*>(ws + w.part[1]) : nullptr;
    // dq_t = scale sum_s a^(t-s) (d_o_t . v_s) k_s, forwards; its state is S transposed
    const ssk::LattnJob jq = {d_o, v, k, do_row_stride, v_row_stride, k_row_stride, 1, 1, share, vi, ki,
                              part_q ? static_cast<void*>(part_q) : dq, part_q != nullptr, false, h0, nullptr, 1, v_dim,
                              scale, 1.0f, scale, nullptr, nullptr};
    // dk_s = scale sum_t a^(t-s) (v_s . d_o_t) q_t, from the end; its state is G transposed
    const ssk::LattnJob jk = {v, d_o, q, v_row_stride, do_row_stride, q_row_stride, 1, 1, share, vi, ki,
                              part_k ? static_cast<void*>(part_k) : dk, part_k != nullptr, true, dh_last, nullptr, 1,
                              v_dim, scale, scale, 1.0f, nullptr, nullptr};
    // dv_s = scale sum_t a^(t-s) (k_s . q_t) d_o_t, from the end; its state is G
    const ssk::LattnJob jv = {k, q, d_o, k_row_stride, q_row_stride, do_row_stride, share, share, 1, ki, vi, dv, false,
                              true, dh_last, dh0, v_dim, 1, scale, scale, 1.0f, nullptr, nullptr};
    ssk::LattnJob jobs[] = {jv, jk, jq};
    for (int i = 0; i < 3; ++i)
        if (w.cut[i].segs > 1) {
            jobs[i].seg = reinterpret_cast<float*>(ws + w.seg[i]);
            jobs[i].keep = reinterpret_cast<float*>(ws + w.keep[i]);
        }
    const int dt = dtype == SS_F32 ? 0 : 1;
    ssk::LattnArgs a = lattn_args(d, w.cut[0], log_decay, reset);
    a.job[a.jobs++] = jobs[0];
    if (!lattn_together(d)) {
        if (const hipError_t e = ssk::launch_lattn(a, dt, stream); e != hipSuccess) return done(e);
        a = lattn_args(d, w.cut[1], log_decay, reset);
    }
    a.job[a.jobs++] = jobs[1];
    a.job[a.jobs++] = jobs[2];
    if (const hipError_t e = ssk::launch_lattn(a, dt, stream); e != hipSuccess) return done(e);
    if (share > 1) {
        if (const hipError_t e = ssk::launch_lattn_share(part_q, dq, rows, heads, share, k_dim, dt, stream); e != hipSuccess)
            return done(e);
        return done(ssk::launch_lattn_share(part_k, dk, rows, heads, share, k_dim, dt, stream));
    }
    return SS_OK;
}

ss_status ss_lattn_step(float* h, const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride,
                        const void* v, int64_t v_row_stride, const float* log_decay, float scale, void* o,
                        int64_t batch, int64_t qk_heads, int64_t heads, int64_t k_dim, int64_t v_dim, ss_dtype dtype,
                        hipStream_t stream)
{
    if (!h || !q || !k || !v || !log_decay || !o) return SS_ERR_INVALID_ARG;
    const LattnDims d{batch, 1, qk_heads, heads, k_dim, v_dim};
    if (!lattn_sizes(d) || !isfinite(scale)) return SS_ERR_INVALID_ARG;
    if (q_row_stride < qk_heads * k_dim || k_row_stride < qk_heads * k_dim || v_row_stride < heads * v_dim)
        return SS_ERR_INVALID_ARG;
    if (!known(dtype) || !lattn_widths(d)) return SS_ERR_UNSUPPORTED;
    if (batch * heads > UINT32_MAX || !launch_fits(ssk::lattn_step_groups(batch, heads, v_dim), ssk::kStepThreads))
        return SS_ERR_UNSUPPORTED;
    const int64_t es = elem_size(dtype);
    const void* elems[] = {q, k, v, o};
    for (const void* p : elems)
        if (!aligned(p, uintptr_t(es))) return SS_ERR_INVALID_ARG;
    if (!aligned(log_decay, 4) || !aligned(h, 4)) return SS_ERR_INVALID_ARG;
    int64_t qb, kb, vb;
    if (!strided_bytes(batch, qk_heads * k_dim, q_row_stride, es, &qb) ||
        !strided_bytes(batch, qk_heads * k_dim, k_row_stride, es, &kb) ||
        !strided_bytes(batch, heads * v_dim, v_row_stride, es, &vb))
        return SS_ERR_INVALID_ARG;
    const Range all[] = {span(q, qb), span(k, kb), span(v, vb), span(log_decay, heads * 4), span(h, d.states() * 4),
                         span(o, batch * heads * v_dim * es)};
    if (any_overlap(all + 4, 2, all, 4)) return SS_ERR_INVALID_ARG;
    ssk::LattnStepArgs a{h, q, k, v, q_row_stride, k_row_stride, v_row_stride, log_decay, scale, o, batch, qk_heads,
                         heads, k_dim, v_dim};
    return done(ssk::launch_lattn_step(a, dtype == SS_F32 ? 0 : 1, stream));
}

// ---- norms and rotation -----------------------------------------------------------------

}  // extern "C"

namespace {

// Workgroups of the backward, each of which leaves its sums of dw_q and dw_k.
constexpr int64_t kQknormBlocks = 1024;
int64_t qknorm_blocks(int64_t tokens) { return tokens < kQknormBlocks ? tokens : kQknormBlocks; }

bool qknorm_sizes(int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t width)
{
    int64_t n;
    if (tokens <= 0 || q_heads <= 0 || k_heads <= 0 || width <= 0) return false;
    return mul(q_heads > k_heads ? q_heads : k_heads, width, &n) && mul(n, tokens, &n) && mul(n, 4, &n);
}

struct QknormCheck {
    Range all[16];
    int inputs, total;
};

// What the two directions' checks share; `c` then holds the inputs' ranges.
ss_status qknorm_check(const void* q, int64_t q_ld, const void* k, int64_t k_ld, const float* w_q, const float* w_k,
                       const int64_t* pos, const float* inv_freq, float eps, int64_t tokens, int64_t q_heads,
                       int64_t k_heads, int64_t width, int64_t half, ss_dtype dtype, QknormCheck* c)
{
    if (!q || !k || !w_q || !w_k || !pos) return SS_ERR_INVALID_ARG;
    if (!qknorm_sizes(tokens, q_heads, k_heads, width)) return SS_ERR_INVALID_ARG;
    if (half < 0 || half > width / 2 || (half > 0 && !inv_freq)) return SS_ERR_INVALID_ARG;
    if (!isfinite(eps) || eps < 0.0f) return SS_ERR_INVALID_ARG;
    if (q_ld < q_heads * width || k_ld < k_heads * width) return SS_ERR_INVALID_ARG;
    if (!known(dtype) || width > ssk::kQknormMaxDim) return SS_ERR_UNSUPPORTED;
    // the backward, whose launch does not grow with the tokens, takes what the forward does
    if (!launch_fits(ssk::qknorm_tiles(tokens, half, false), ssk::kQknormThreads) || q_heads > ssk::kQknormMaxHeads ||
        k_heads > ssk::kQknormMaxHeads)
        return SS_ERR_UNSUPPORTED;
    const int64_t es = elem_size(dtype);
    if (!aligned(q, uintptr_t(es)) || !aligned(k, uintptr_t(es)) || !aligned(w_q, 4) || !aligned(w_k, 4) ||
        !aligned(pos, 8) || !aligned(inv_freq, 4))
        return SS_ERR_INVALID_ARG;
    int64_t qb, kb;
    if (!strided_bytes(tokens, q_heads * width, q_ld, es, &qb) || !strided_bytes(tokens, k_heads * width, k_ld, es, &kb))
        return SS_ERR_INVALID_ARG;
    c->all[0] = span(q, qb);
    c->all[1] = span(k, kb);
    c->all[2] = span(w_q, width * 4);
    c->all[3] = span(w_k, width * 4);
    c->all[4] = span(pos, tokens * 8);
    c->all[5] = span(half ? inv_freq : nullptr, half * 4);
    c->inputs = c->total = 6;
    return SS_OK;
}

ssk::QknormArgs qknorm_args(const void* q, int64_t q_ld, const void* k, int64_t k_ld, const float* w_q,
                            const float* w_k, const int64_t* pos, const float* inv_freq, float eps, int interleaved,
                            int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t width, int64_t half)
{
    ssk::QknormArgs a{};
    a.side[0].x = q;
    a.side[0].ld = q_ld;
    a.side[0].heads = q_heads;
    a.side[0].w = w_q;
    a.side[1].x = k;
    a.side[1].ld = k_ld;
    a.side[1].heads = k_heads;
    a.side[1].w = w_k;
    a.pos = pos;
    a.inv_freq = inv_freq;
    a.eps = eps;
    a.interleaved = interleaved != 0;
    a.tokens = tokens;
    a.width = width;
    a.half = half;
    return a;
}

}  // namespace

extern "C" {

ss_status ss_qknorm_fwd(const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride, const float* w_q,
                        const float* w_k, const int64_t* pos, const float* inv_freq, float eps, int interleaved,
                        void* qo, void* ko, int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t width,
                        int64_t half_rotary, ss_dtype dtype, hipStream_t stream)
{
    if (!qo || !ko) return SS_ERR_INVALID_ARG;
    QknormCheck c;
    const ss_status st = qknorm_check(q, q_row_stride, k, k_row_stride, w_q, w_k, pos, inv_freq, eps, tokens, q_heads,
                                      k_heads, width, half_rotary, dtype, &c);
    if (st != SS_OK) return st;
    const int64_t es = elem_size(dtype);
    if (!aligned(qo, uintptr_t(es)) || !aligned(ko, uintptr_t(es))) return SS_ERR_INVALID_ARG;
    c.all[c.total++] = span(qo, tokens * q_heads * width * es);
    c.all[c.total++] = span(ko, tokens * k_heads * width * es);
    if (any_overlap(c.all + c.inputs, 2, c.all, c.inputs)) return SS_ERR_INVALID_ARG;
    ssk::QknormArgs a = qknorm_args(q, q_row_stride, k, k_row_stride, w_q, w_k, pos, inv_freq, eps, interleaved, tokens,
                                    q_heads, k_heads, width, half_rotary);
    a.side[0].out = qo;
    a.side[1].out = ko;
    return done(ssk::launch_qknorm_fwd(a, dtype == SS_F32 ? 0 : 1, stream));
}

size_t ss_qknorm_bwd_workspace_bytes(int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t width)
{
    if (!qknorm_sizes(tokens, q_heads, k_heads, width) || width > ssk::kQknormMaxDim) return kBad;
    return static_cast<size_t>(2 * qknorm_blocks(tokens) * width * 4);
}

ss_status ss_qknorm_bwd(const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride, const float* w_q,
                        const float* w_k, const int64_t* pos, const float* inv_freq, float eps, int interleaved,
                        const void* dqo, const void* dko, void* dq, void* dk, float* dw_q, float* dw_k,
                        void* workspace, size_t workspace_bytes, int64_t tokens, int64_t q_heads, int64_t k_heads,
                        int64_t width, int64_t half_rotary, ss_dtype dtype, hipStream_t stream)
{
    if (!dqo || !dko || !dq || !dk || !dw_q || !dw_k) return SS_ERR_INVALID_ARG;
    QknormCheck c;
    ss_status st = qknorm_check(q, q_row_stride, k, k_row_stride, w_q, w_k, pos, inv_freq, eps, tokens, q_heads,
                                k_heads, width, half_rotary, dtype, &c);
    if (st != SS_OK) return st;
    const int64_t es = elem_size(dtype), nq = tokens * q_heads * width * es, nk = tokens * k_heads * width * es;
    const void* elems[] = {dqo, dko, dq, dk};
    for (const void* p : elems)
        if (!aligned(p, uintptr_t(es))) return SS_ERR_INVALID_ARG;
    if (!aligned(dw_q, 4) || !aligned(dw_k, 4)) return SS_ERR_INVALID_ARG;
    c.all[c.total++] = span(dqo, nq);
    c.all[c.total++] = span(dko, nk);
    c.inputs = c.total;
    c.all[c.total++] = span(dq, nq);
    c.all[c.total++] = span(dk, nk);
    c.all[c.total++] = span(dw_q, width * 4);
    c.all[c.total++] = span(dw_k, width * 4);
    if (any_overlap(c.all + c.inputs, size_t(c.total - c.inputs), c.all, size_t(c.inputs))) return SS_ERR_INVALID_ARG;
    ssk::QknormArgs a = qknorm_args(q, q_row_stride, k, k_row_stride, w_q, w_k, pos, inv_freq, eps, interleaved, tokens,
                                    q_heads, k_heads, width, half_rotary);
    a.blocks = qknorm_blocks(tokens);
    st = check_workspace(workspace, workspace_bytes, 2 * a.blocks * width * 4, c.all, size_t(c.total));
    if (st != SS_OK) return st;
    a.side[0].out = dq;
    a.side[0].dy = dqo;
    a.side[0].dw = dw_q;
    a.side[1].out = dk;
    a.side[1].dy = dko;
    a.side[1].dw = dw_k;
    a.part = static_cast<float*>(workspace);
    return done(ssk::launch_qknorm_bwd(a, dtype == SS_F32 ? 0 : 1, stream));
}

// ---- sampling ---------------------------------------------------------------------------

size_t ss_sample_workspace_bytes(int64_t rows, int64_t vocab, ss_dtype dtype)
{
    int64_t n;
    if (rows <= 0 || vocab <= 0 || vocab > ssk::kSampleMaxVocab || !known(dtype) || !mul(rows, vocab, &n) || !mul(n, 4, &n))
        return kBad;
    return 0;
}

ss_status ss_sample(const void* logits, int64_t row_stride, const float* u, const float* temperature,
                    float temperature_all, const int32_t* top_k, int32_t top_k_all, const float* top_p,
                    float top_p_all, const float* min_p, float min_p_all, int64_t* token, void* workspace,
                    size_t workspace_bytes, int64_t rows, int64_t vocab, ss_dtype dtype, hipStream_t stream)
{
    if (!logits || !u || !token || rows <= 0 || vocab <= 0 || row_stride < vocab) return SS_ERR_INVALID_ARG;
    if (!known(dtype) || vocab > ssk::kSampleMaxVocab || rows > INT32_MAX || !launch_fits(rows, 1024))
        return SS_ERR_UNSUPPORTED;
    const int64_t es = elem_size(dtype);
    if (!aligned(logits, uintptr_t(es)) || !aligned(token, 8)) return SS_ERR_INVALID_ARG;
    const void* words[] = {u, temperature, top_k, top_p, min_p};
    for (const void* p : words)
        if (!aligned(p, 4)) return SS_ERR_INVALID_ARG;
    int64_t bytes;
    if (!strided_bytes(rows, vocab, row_stride, es, &bytes)) return SS_ERR_INVALID_ARG;
    const Range all[] = {span(logits, bytes), span(u, rows * 4), span(temperature, rows * 4), span(top_k, rows * 4),
                         span(top_p, rows * 4), span(min_p, rows * 4), span(token, rows * 8)};
    if (any_overlap(all + 6, 1, all, 6)) return SS_ERR_INVALID_ARG;
    const ss_status st = check_workspace(workspace, workspace_bytes, 0, all, 7);
    if (st != SS_OK) return st;
    ssk::SampleArgs a{logits, row_stride, u, temperature, top_k, top_p, min_p, temperature_all, top_p_all, min_p_all,
                      top_k_all, token, rows, vocab};
    return done(ssk::launch_sample(a, dtype == SS_F32 ? 0 : 1, stream));
}

}  // extern "C"
