// host_model.cpp -- argument validation, workspace layout and the choice of
// form of the gated linear recurrence, the norm and the vocabulary loss. Plain
// C++ with no HIP, like host.cpp.
#include <cmath>
#include <cstdint>
#include <string>

#include "vs_host.h"
#include "vs_model.h"

namespace vs {

// ------------------------------------------------- gated linear recurrence
namespace {

const char* gated_problem(int64_t batch, int64_t dim, int64_t L, int& code) {
    if (const char* p = sizes_problem(batch, dim, 1, L, 1, 1, code)) return p;
    code = VS_ERR_UNSUPPORTED;
    if (batch * dim > kMaxGroups) return "2^24 rows (batch x dim) or more are not supported";
    return nullptr;
}

const char* rate_problem(float rate) {
    return std::isfinite(rate) && rate >= 0 ? nullptr : "rate must be finite and >= 0";
}

}  // namespace

// A wave takes 512 tokens at a time, so it wastes on short rows what 16 lanes
// (128 at a time) keep busy: bf16, 64 x 384 rows of 256 14.0 us against 31.7, of 384
// 19.1 against 32.9, of 512 26.5 against 25.4. Rows past 256 tokens need enough
// others beside them, for their chunks follow one another (384 rows of 300: 7.2 us
// against 5.9). Four or eight waves a row where rows alone don't fill the
// machine: 1,536 rows of 16,385 52.8 us with one wave, 44.9 with four, 47.2 with
// eight; 384 of 4,097 11.9, 8.0 and 7.5; 6,144 of 4,097 49.9, 67.3 and 91.9.
GatedForm gated_form(int64_t batch, int64_t dim, int64_t L) {
    const int64_t rows = batch * dim;
    if (L <= 256 || (L <= 384 && rows >= 2048)) return {16, 1};
    if (rows >= 2048 || L <= 1024) return {64, 1};
    if (rows >= 512 || L <= 4096) return {64, 4};
    return {64, 8};
}

size_t gated_ws_bytes(int op, int64_t batch, int64_t dim, int64_t L) {
    int code;
    if (gated_problem(batch, dim, L, code)) return 0;
    const size_t rows = static_cast<size_t>(batch * dim);
    if (op == VS_GATED_SAVED) return rows * static_cast<size_t>(ceil_div(L, gated_form(batch, dim, L).block())) * kF;
    if (op == VS_GATED_GRAD) return rows * kF;           // per row: its part of dlam
    return 0;
}

int prepare_gated(GatedCall& c) {
    clear_error();
    if (c.dtype != VS_F32 && c.dtype != VS_BF16) return fail(VS_ERR_DTYPE, "unknown dtype");
    int code;
    if (const char* p = gated_problem(c.batch, c.dim, c.L, code)) return fail(code, p);
    if (const char* p = rate_problem(c.rate)) return fail(VS_ERR_UNSUPPORTED, p);
    if (!c.x || !c.r || !c.i || !c.lam) return fail(VS_ERR_NULL, "x, r, i and lam must not be NULL");
    if (c.grad) {
        if (!c.dy || !c.dx || !c.dr || !c.di || !c.dlam) return fail(VS_ERR_NULL, "dy, dx, dr, di and dlam must not be NULL");
        if (c.z && !c.dz) return fail(VS_ERR_NULL, "dz must not be NULL when z is given");
        if (!c.z) c.dz = nullptr;
    } else if (!c.y) {
        return fail(VS_ERR_NULL, "y must not be NULL");
    }
    for (int k = 0; k < (c.grad ? 5 : 4); ++k) {
        c.st[k] = c.strides ? Strides{c.strides[2 * k], c.strides[2 * k + 1]} : Strides{c.dim * c.L, c.L};
        if (k == 3 && !c.z) { c.st[k] = Strides{0, 0}; continue; }
        if (int rc = check_strides(c.st[k], c.batch)) return rc;
    }
    c.form = gated_form(c.batch, c.dim, c.L);
    const size_t es = esize(c.dtype), act = static_cast<size_t>(c.batch * c.dim * c.L) * es;
    const size_t states = static_cast<size_t>(c.batch * c.dim) * kF, par = static_cast<size_t>(c.dim) * kF;
    const size_t saved = gated_ws_bytes(VS_GATED_SAVED, c.batch, c.dim, c.L);
    const size_t ws = c.grad ? gated_ws_bytes(VS_GATED_GRAD, c.batch, c.dim, c.L) : 0;
    if ((c.save || c.grad) && (!c.saved || c.saved_bytes < saved))
        return fail(VS_ERR_WORKSPACE, "saved-state buffer missing or smaller than gated_workspace_bytes(VS_GATED_SAVED)");
    if (ws > 0 && (!c.ws || c.ws_bytes < ws)) return fail(VS_ERR_WORKSPACE, "workspace missing or smaller than gated_workspace_bytes()");
    auto span = [&](const void* p, int k) { return Span{p, p ? span_bytes(c.batch, c.dim, c.L, c.st[k], es) : 0}; };
    const Span ins[] = {span(c.x, 0), span(c.r, 1), span(c.i, 2), span(c.z, 3), span(c.grad ? c.dy : nullptr, 4),
                        {c.lam, par}, {c.h0, states}, {c.lengths, static_cast<size_t>(c.batch) * 4},
                        {c.grad ? c.dh_out : nullptr, states}, {c.grad ? c.saved : nullptr, saved}};
    if (int rc = check_aligned(ins, 5, es, "activation pointer misaligned")) return rc;
    if (int rc = check_aligned(ins + 5, 5, 4, "32-bit pointer misaligned")) return rc;
    if (!c.grad) {
        const Span outs[] = {{c.y, act}, {c.h_out, states}, {c.save ? c.saved : nullptr, saved}};
        if (int rc = check_aligned(outs, 1, es, "activation pointer misaligned")) return rc;
        if (int rc = check_aligned(outs + 1, 2, 4, "32-bit pointer misaligned")) return rc;
        return check_overlaps(ins, 10, outs, 3);
    }
    const Span outs[] = {{c.dx, act}, {c.dr, act}, {c.di, act}, {c.dz, act}, {c.dlam, par}, {c.dh0, states}, {c.ws, ws}};
    if (int rc = check_aligned(outs, 4, es, "activation pointer misaligned")) return rc;
    if (int rc = check_aligned(outs + 4, 3, 4, "32-bit pointer misaligned")) return rc;
    return check_overlaps(ins, 10, outs, 7);
}

int prepare_gated_step(GatedStepCall& c) {
    clear_error();
    if (c.dtype != VS_F32 && c.dtype != VS_BF16) return fail(VS_ERR_DTYPE, "unknown dtype");
    int code;
    if (const char* p = sizes_problem(c.batch, c.dim, 1, 1, 1, 1, code)) return fail(code, p);
    if (const char* p = rate_problem(c.rate)) return fail(VS_ERR_UNSUPPORTED, p);
    if (c.slots < 1) return fail(VS_ERR_SHAPE, "the pool must have at least one slot");
    if (c.slots >= (int64_t(1) << 31)) return fail(VS_ERR_UNSUPPORTED, "pools of 2^31 slots or more are not supported");
    if (c.batch * ceil_div(c.dim, 4) > kMaxGroups * 256)
        return fail(VS_ERR_UNSUPPORTED, "a step of 2^34 channels or more is not supported");
    if (!c.x || !c.r || !c.i || !c.lam || !c.h || !c.y) return fail(VS_ERR_NULL, "x, r, i, lam, h and y must not be NULL");
    if ((!c.slot_in || !c.slot_out) && c.slots < c.batch)
        return fail(VS_ERR_SHAPE, "without slot_in or slot_out the pool needs a slot for every row");
    for (int k = 0; k < 4; ++k) {
        c.st[k] = c.strides ? c.strides[k] : c.dim;
        if (c.st[k] < 0) return fail(VS_ERR_SHAPE, "strides must be >= 0");
        if (c.st[k] >= (int64_t(1) << 28)) return fail(VS_ERR_UNSUPPORTED, "row strides of 2^28 elements or more are not supported");
    }
    const size_t es = esize(c.dtype);
    auto span = [&](const void* p, int k) {
        return Span{p, p ? (static_cast<size_t>((c.batch - 1) * c.st[k]) + static_cast<size_t>(c.dim)) * es : 0};
    };
    const size_t idx = static_cast<size_t>(c.batch) * 4;
    const Span ins[] = {span(c.x, 0), span(c.r, 1), span(c.i, 2), span(c.z, 3),
                        {c.lam, static_cast<size_t>(c.dim) * kF}, {c.slot_in, idx}, {c.slot_out, idx}};
    const Span outs[] = {{c.y, static_cast<size_t>(c.batch * c.dim) * es}, {c.h, static_cast<size_t>(c.slots * c.dim) * kF}};
    if (int rc = check_aligned(ins, 4, es, "activation pointer misaligned")) return rc;
    if (int rc = check_aligned(ins + 4, 3, 4, "32-bit pointer misaligned")) return rc;
    if (int rc = check_aligned(outs, 1, es, "activation pointer misaligned")) return rc;
    if (int rc = check_aligned(outs + 1, 1, 4, "state pointer misaligned")) return rc;
    return check_overlaps(ins, 7, outs, 2);
}

// -------------------------------------------------------------------- norm
namespace {

const char* norm_problem(int64_t batch, int64_t dim, int64_t L, int& code) {
    code = VS_ERR_SHAPE;
    if (batch < 1 || dim < 1 || L < 1) return "batch, dim and the sequence length must be >= 1";
    code = VS_ERR_UNSUPPORTED;
    if (dim > kNormMaxDim) return "dim above 8192 is not supported";
    if (L >= kCausalMaxL) return "sequences of 2^27 tokens or more are not supported";
    // launches of fewer than 2^32 threads: up to 1,024 a tile, 64 or more a row
    if (batch >= (int64_t(1) << 26) || (L > 1 && batch * ceil_div(L, 16) >= (int64_t(1) << 22)))
        return "2^26 rows, or 2^22 tiles of 16 tokens, or more are not supported";
    if (!product_below(batch, dim, L, int64_t(1) << 40)) return "outputs of 2^40 elements or more are not supported";
    return nullptr;
}

// a wave a row while it holds the row in 16 bytes a lane, then four, then sixteen
NormForm norm_rows(int64_t dim, int dtype) {
    const int64_t lanes = dtype == VS_BF16 ? 8 : 4;     // entries of 16 bytes
    if (dim <= 64 * lanes) return kNormRow1;
    if (dim <= 256 * lanes) return kNormRow4;
    return kNormRow16;
}

// Tokens of a tile, channel-major. The wider the piece of a row, the fewer lines are
// shared with a neighbouring tile (bf16 8 x 768 x 4,097 with a residual 53.6 us in
// pieces of 64 bytes, 44.3 in pieces of 128; training step of 8 x 384 x 4,097 62.3 and
// 52.2), as long as six sweeps of sixteen waves (the gradient, which holds more:
// eight), eight channels a wave, hold all channels (gradient of 8 x 768 x 4,097:
// 106 us a step; with twelve sweeps 112, sixteen waves 108).
int norm_tile(int64_t dim, bool grad, size_t es) {
    return (dim <= (grad ? 384 : 768) ? kNormWide : kNormNarrow) / static_cast<int>(es);
}

// Batch rows that a channel-major gradient takes in one launch: each tile leaves a
// line of dw's sums, 4 bytes a channel, and rows of one token would leave twice
// what a bf16 activation holds (65,536 x 4,096: 1 GB). One token: as many lines as
// the rows' form has; more: 64 MB of lines, or 4,096. What is past that goes into dw
// launch by launch.
int64_t norm_slab(int64_t batch, int64_t dim, int64_t L, int tile) {
    const int64_t few = dim > 512 ? kNormGroups : 4 * kNormGroups, fit = (int64_t(1) << 24) / dim, tiles = ceil_div(L, tile);
    const int64_t rows = (L == 1 || fit < few ? few : fit) / tiles;
    return rows < 1 ? 1 : rows < batch ? rows : batch;
}

// lines of dw's sums: one for each tile of a launch, or for each wave or workgroup that takes rows
int64_t norm_parts(NormForm f, int64_t batch, int64_t dim, int64_t L, int tile) {
    if (f == kNormColumn) return norm_slab(batch, dim, L, tile) * ceil_div(L, tile);
    const int64_t per = f == kNormRow1 ? 4 : 1, groups = ceil_div(batch, per);
    return (groups < kNormGroups ? groups : kNormGroups) * per;
}

}  // namespace

int prepare_norm(NormCall& c) {
    clear_error();
    if (c.dtype != VS_F32 && c.dtype != VS_BF16) return fail(VS_ERR_DTYPE, "unknown dtype");
    int code;
    if (const char* p = norm_problem(c.batch, c.dim, c.L, code)) return fail(code, p);
    if (!(std::isfinite(c.eps) && c.eps >= 0)) return fail(VS_ERR_UNSUPPORTED, "eps must be finite and >= 0");
    if (!c.x || !c.y) return fail(VS_ERR_NULL, c.grad ? "s and ds must not be NULL" : "x and y must not be NULL");
    if (c.grad && !c.dy) return fail(VS_ERR_NULL, "dy must not be NULL");
    if (!c.grad && !c.residual != !c.sum) return fail(VS_ERR_NULL, "residual and sum must be given together");
    const void* second = c.grad ? c.dy : c.residual;
    const void* ins[] = {c.x, second, c.grad ? c.dsum : nullptr};
    bool rows = c.L == 1;
    for (int k = 0; k < (c.grad ? 3 : 2); ++k) {
        c.st[k] = c.strides ? Strides{c.strides[2 * k], c.strides[2 * k + 1]} : Strides{c.dim * c.L, c.L};
        if (!ins[k]) { c.st[k] = Strides{0, 0}; continue; }
        if (int rc = check_strides(c.st[k], c.batch)) return rc;
        rows = rows && (c.st[k].d == 1 || c.dim == 1);
    }
    c.form = rows ? norm_rows(c.dim, c.dtype) : kNormColumn;
    const int64_t threads = c.form == kNormRow1 ? 64 : c.form == kNormRow4 ? 256 : 1024;
    if (c.batch * ceil_div(c.L, 16) >= (int64_t(1) << 32) / threads)
        return fail(VS_ERR_UNSUPPORTED, "rows of that many channels: launches of 2^32 threads or more are not supported");
    c.tile = norm_tile(c.dim, c.grad, esize(c.dtype));
    c.slab = c.grad && c.dw && c.form == kNormColumn ? norm_slab(c.batch, c.dim, c.L, c.tile) : c.batch;
    c.parts = norm_parts(c.form, c.batch, c.dim, c.L, c.tile);
    const size_t es = esize(c.dtype), act = static_cast<size_t>(c.batch * c.dim * c.L) * es;
    const size_t par = static_cast<size_t>(c.dim) * kF, ws = c.dw ? static_cast<size_t>(c.parts) * par : 0;
    if (ws > 0 && (!c.ws || c.ws_bytes < ws)) return fail(VS_ERR_WORKSPACE, "workspace missing or smaller than norm_workspace_bytes()");
    auto span = [&](int k) { return Span{ins[k], ins[k] ? span_bytes(c.batch, c.dim, c.L, c.st[k], es) : 0}; };
    // the sum may be the residual itself (a stride over one channel, or one row, says nothing)
    const bool inplace = !c.grad && c.sum && c.sum == c.residual && (c.st[1].d == c.L || c.dim == 1) &&
                         (c.st[1].b == c.dim * c.L || c.batch == 1);
    const Span in[] = {span(0), span(1), span(2), {c.w, par}, {c.lengths, static_cast<size_t>(c.batch) * 4}};
    const Span out[] = {{c.y, act}, {c.grad ? nullptr : c.sum, act}, {c.dw, par}, {c.dw ? c.ws : nullptr, ws}};
    if (int rc = check_aligned(in, 3, es, "activation pointer misaligned")) return rc;
    if (int rc = check_aligned(in + 3, 2, 4, "32-bit pointer misaligned")) return rc;
    if (int rc = check_aligned(out, 2, es, "activation pointer misaligned")) return rc;
    if (int rc = check_aligned(out + 2, 2, 4, "32-bit pointer misaligned")) return rc;
    if (!inplace) return check_overlaps(in, 5, out, 4);
    // all but the sum against its residual
    const Span apart[] = {in[0], in[3], in[4]};
    if (int rc = check_overlaps(apart, 3, out, 4)) return rc;
    return check_overlaps(in + 1, 1, out, 1);
}

// --------------------------------------------------------- vocabulary loss
namespace {

const char* vocab_problem(int64_t tokens, int64_t dim, int64_t vocab, int& code) {
    code = VS_ERR_SHAPE;
    if (tokens < 1 || dim < 1 || vocab < 1) return "tokens, dim and vocab must be >= 1";
    code = VS_ERR_UNSUPPORTED;
    if (dim > 65536) return "dim above 65536 is not supported";
    if (tokens >= (int64_t(1) << 24) || vocab >= (int64_t(1) << 24)) return "2^24 tokens or vocabulary entries or more are not supported";
    if (!product_below(tokens, dim, 1, int64_t(1) << 34) || !product_below(vocab, dim, 1, int64_t(1) << 34))
        return "matrices of 2^34 entries or more are not supported";
    if (ceil_div(tokens, 128) * ceil_div(vocab, 128) >= (int64_t(1) << 22)) return "2^36 logits or more are not supported";
    return nullptr;
}

int64_t tiles_of(int64_t m, int64_t n, int64_t tile) { return ceil_div(m, tile) * ceil_div(n, tile); }

// Whether the logits take the larger tile: by rounds of tiles over the chip, one
// larger tile or two smaller ones on a compute unit at a time. A round of smaller
// ones takes 0.65 of a larger one's time in bf16, whose operands are read twice
// as often, and half in fp32, which the matrix cores bound. bf16: 197 x 768 x
// 49,999 scored 26.7 us (smaller tile 30.7), 64 x 1,536 x 32,768 31.4 (larger 44.5),
// the training step of 8,194 x 1,536 x 49,999 4,850 (smaller 5,240); fp32 500 x 768
// x 10,000 scored 98.6 (larger 187).
bool vocab_wide(int64_t m, int64_t n, int dtype) {
    const int64_t wide = ceil_div(tiles_of(m, n, 256), kNumCUs), narrow = ceil_div(tiles_of(m, n, 128), 2 * kNumCUs);
    return 20 * wide <= (dtype == VS_BF16 ? 13 : 10) * narrow;
}

int64_t stages_of(int64_t k, int dtype) { return ceil_div(k * static_cast<int64_t>(esize(dtype)), kVocabStage); }

// both products of a piece run together: no workgroup takes more than its share
// of all stages, or eight, and a product is cut into at most 64
struct Splits { int64_t work; int dx, dw; };
Splits vocab_splits(int64_t dim, int64_t tokens, int64_t n, int64_t tile, int dtype) {
    const int64_t tx = tiles_of(dim, tokens, tile), tw = tiles_of(dim, n, tile), kx = stages_of(n, dtype), kw = stages_of(tokens, dtype);
    const int64_t work = tx * kx + tw * kw, slots = tile == 256 ? kNumCUs : 2 * kNumCUs;
    int64_t share = ceil_div(work, slots);
    share = share < 8 ? 8 : share;
    auto cut = [&](int64_t k) { const int64_t s = ceil_div(k, share); return static_cast<int>(s > 64 ? 64 : s); };
    return {work, cut(kx), cut(kw)};
}

}  // namespace

VocabPlan vocab_plan(bool grad, int64_t tokens, int64_t dim, int64_t vocab, int dtype) {
    VocabPlan p{};
    const size_t es = esize(dtype);
    p.dp = ceil_div(dim, 8) * 8;
    p.pack_w = dim * static_cast<int64_t>(es) % 4 != 0;         // a row starts or ends between words
    size_t off = 0;
    auto take = [&](size_t n) { const size_t at = off; off += al256(n); return at; };
    p.x = take(static_cast<size_t>(tokens * p.dp) * es);
    p.w = take(p.pack_w ? static_cast<size_t>(vocab * p.dp) * es : 0);
    if (!grad) {
        p.wide = vocab_wide(vocab, tokens, dtype);
        p.tiles = static_cast<int>(ceil_div(vocab, p.wide ? 256 : 128));
        p.part = take(static_cast<size_t>(p.tiles) * static_cast<size_t>(tokens) * 2 * kF);
        p.logit = take(static_cast<size_t>(tokens) * kF);
    } else {
        // P of a piece takes up to 512 MB: half of that lets P stay in the memory-side
        // cache, but the products have fewer tiles to share out (bf16 8,194 x 1,536 x
        // 49,999 5,230 us, with 256 MB 5,120; 8,194 x 768 x 32,768 2,045 and 2,211;
        // 4,096 x 768 x 49,152 1,429 and 1,495; fp32 2,049 x 384 x 49,999 2,699 and 2,780)
        int64_t piece = (int64_t(1) << 29) / (tokens * static_cast<int64_t>(es)) / 256 * 256;
        piece = piece < 256 ? 256 : piece;
        // 256 rows of P, also those past the last token, have offsets of 32 bits
        const int64_t most = (int64_t(1) << 24) / static_cast<int64_t>(es);
        piece = piece > most ? most : piece;
        p.pieces = ceil_div(vocab, piece);
        p.piece = ceil_div(ceil_div(vocab, p.pieces), 256) * 256;
        p.pieces = ceil_div(vocab, p.piece);
        const int64_t n = p.piece < vocab ? p.piece : vocab;
        p.prob_wide = vocab_wide(n, tokens, dtype);
        // a quarter of the larger tile's work costs the smaller one 1.3 (fp32: 1.05) quarters
        // (bf16 8,194 x 1,536 x 49,999 4,850 us, with the smaller tile 5,300; 4,097 x 384 x
        // 1,000 59.8, with the larger 72.8; fp32 394 x 384 x 32,768 412 and 545)
        const Splits wide = vocab_splits(dim, tokens, n, 256, dtype), narrow = vocab_splits(dim, tokens, n, 128, dtype);
        p.wide = 80 * wide.work <= (dtype == VS_BF16 ? 26 : 21) * narrow.work;
        p.dx_splits = p.wide ? wide.dx : narrow.dx;
        p.dw_splits = p.wide ? wide.dw : narrow.dw;
        p.P = take(static_cast<size_t>(tokens * (ceil_div(n, 8) * 8)) * es);
        p.part_dx = take(p.dx_splits > 1 ? static_cast<size_t>(p.dx_splits * tokens * dim) * kF : 0);
        p.part_dw = take(p.dw_splits > 1 ? static_cast<size_t>(p.dw_splits * n * dim) * kF : 0);
        p.sum = take(p.pieces > 1 ? static_cast<size_t>(tokens * dim) * kF : 0);
        p.rest = take(dtype == VS_BF16 ? static_cast<size_t>(tokens) * kF : 0);
    }
    p.bytes = off;
    return p;
}

int prepare_vocab(VocabCall& c) {
    clear_error();
    if (c.dtype != VS_F32 && c.dtype != VS_BF16) return fail(VS_ERR_DTYPE, "unknown dtype");
    int code;
    if (const char* p = vocab_problem(c.tokens, c.dim, c.vocab, code)) return fail(code, p);
    if (c.target_bits != 32 && c.target_bits != 64) return fail(VS_ERR_UNSUPPORTED, "targets have 32 or 64 bits");
    c.target64 = c.target_bits == 64;
    if (!c.x || !c.W || !c.target) return fail(VS_ERR_NULL, "x, W and target must not be NULL");
    if (c.grad ? !c.lse_in || !c.dloss || !c.dx || !c.dW : !c.loss || !c.lse)
        return fail(VS_ERR_NULL, c.grad ? "lse, dloss, dx and dW must not be NULL" : "loss and lse must not be NULL");
    if (c.ldx == 0) c.ldx = c.dim;
    if (c.ldx < c.dim) return fail(VS_ERR_SHAPE, "x_stride is smaller than dim");
    if (c.ldx >= (int64_t(1) << 28)) return fail(VS_ERR_UNSUPPORTED, "row strides of 2^28 elements or more are not supported");
    c.plan = vocab_plan(c.grad, c.tokens, c.dim, c.vocab, c.dtype);
    const size_t es = esize(c.dtype);
    if (!c.ws || c.ws_bytes < c.plan.bytes) return fail(VS_ERR_WORKSPACE, "workspace missing or smaller than vocab_workspace_bytes()");
    // reads go by words: x starts, steps and ends on one, or is packed
    c.plan.pack_x = !aligned(c.x, 4) || c.ldx * static_cast<int64_t>(es) % 4 != 0 || c.plan.pack_w || c.ldx > 65536;
    const size_t xs = (static_cast<size_t>((c.tokens - 1) * c.ldx) + static_cast<size_t>(c.dim)) * es, ws = static_cast<size_t>(c.vocab * c.dim) * es;
    const size_t row = static_cast<size_t>(c.tokens) * kF;
    const Span ins[] = {{c.x, xs}, {c.W, ws}, {c.target, static_cast<size_t>(c.tokens) * (c.target64 ? 8 : 4)},
                        {c.grad ? c.lse_in : nullptr, row}, {c.grad ? c.dloss : nullptr, row}};
    if (int rc = check_aligned(ins, 1, es, "x misaligned")) return rc;
    if (int rc = check_aligned(ins + 1, 1, c.plan.pack_w ? es : 4, "W misaligned (4 bytes, 2 where dim is odd)")) return rc;
    if (int rc = check_aligned(ins + 2, 1, c.target64 ? 8 : 4, "target misaligned")) return rc;
    if (int rc = check_aligned(ins + 3, 2, 4, "32-bit pointer misaligned")) return rc;
    if (!aligned(c.ws, 16)) return fail(VS_ERR_ALIGN, "workspace misaligned (16 bytes)");
    if (!c.grad) {
        const Span outs[] = {{c.loss, row}, {c.lse, row}, {c.ws, c.plan.bytes}};
        if (int rc = check_aligned(outs, 2, 4, "32-bit pointer misaligned")) return rc;
        return check_overlaps(ins, 5, outs, 3);
    }
    const Span outs[] = {{c.dx, static_cast<size_t>(c.tokens * c.dim) * es}, {c.dW, ws}, {c.ws, c.plan.bytes}};
    if (int rc = check_aligned(outs, 2, es, "gradient misaligned")) return rc;
    return check_overlaps(ins, 5, outs, 3);
}

}  // namespace vs

// ---------------------------------------------------------------- C ABI
extern "C" {

size_t gated_workspace_bytes(int op, int64_t batch, int64_t dim, int64_t seqlen) {
    return vs::gated_ws_bytes(op, batch, dim, seqlen);
}

size_t norm_workspace_bytes(int64_t batch, int64_t dim, int64_t seqlen) {
    int code;
    if (vs::norm_problem(batch, dim, seqlen, code)) return 0;
    // whichever form the strides and the type lead to
    int64_t parts = 0;
    auto most = [&](vs::NormForm f, int tile) {
        const int64_t n = vs::norm_parts(f, batch, dim, seqlen, tile);
        parts = n > parts ? n : parts;
    };
    for (size_t es : {2, 4}) most(vs::kNormColumn, vs::norm_tile(dim, true, es));
    // past 512 channels a row has four waves or more in either type
    if (seqlen == 1) most(dim > 512 ? vs::kNormRow4 : vs::kNormRow1, 1);
    return static_cast<size_t>(parts * dim) * vs::kF;
}

size_t vocab_workspace_bytes(int op, int64_t tokens, int64_t dim, int64_t vocab, int dtype) {
    int code;
    if ((op != VS_VOCAB_LOSS && op != VS_VOCAB_GRAD) || (dtype != VS_F32 && dtype != VS_BF16) ||
        vs::vocab_problem(tokens, dim, vocab, code))
        return 0;
    return vs::vocab_plan(op == VS_VOCAB_GRAD, tokens, dim, vocab, dtype).bytes;
}

}  // extern "C"
