// host_causal.cpp -- argument validation and workspace layout of the causal
// mixer (convolution, scan, their gradients and single-token forms) and of
// beam search. Plain C++ with no HIP, like host.cpp: everything here is decided
// before a kernel file touches the HIP runtime.
#include <cstdint>
#include <string>

#include "vs_internal.h"

namespace vs {

namespace {

constexpr size_t kF = 4;                 // bytes of an fp32 value

size_t al256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
size_t esize(int dtype) { return dtype == VS_BF16 ? 2 : 4; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// sizes every entry point of the mixer shares; `inner` is dstate or the width
const char* sizes_problem(int64_t batch, int64_t dim, int64_t inner, int64_t L, int64_t inner_low,
                          int64_t inner_high, int& code) {
    code = VS_ERR_SHAPE;
    if (batch < 1 || dim < 1 || L < 1) return "batch, dim and the sequence length must be >= 1";
    if (inner < inner_low) return inner_low == 2 ? "the convolution's width must be >= 2" : "dstate must be >= 1";
    if (batch > 65535) return "batch above 65535 is not supported";
    code = VS_ERR_UNSUPPORTED;
    if (inner > inner_high) return inner_low == 2 ? "a convolution width above 8 is not supported" : "dstate above 16 is not supported";
    if (dim >= kCausalMaxDim) return "dim of 2^20 or more is not supported";
    if (L >= kCausalMaxL) return "sequences of 2^27 tokens or more are not supported";
    // outputs are contiguous: their byte counts stay far below 2^63
    if (!product_below(batch, dim, L, int64_t(1) << 40)) return "outputs of 2^40 elements or more are not supported";
    return nullptr;
}

struct Span { const void* p; size_t n; };

// bytes from the first to past the last element of a [batch][rows][len] tensor
size_t span_bytes(int64_t batch, int64_t rows, int64_t len, const Strides& s, size_t es) {
    return (static_cast<size_t>((batch - 1) * s.b + (rows - 1) * s.d) + static_cast<size_t>(len)) * es;
}

int check_strides(const Strides& s, int64_t batch) {
    if (s.b < 0 || s.d < 0) return fail(VS_ERR_SHAPE, "strides must be >= 0");
    if (s.d >= kCausalMaxL) return fail(VS_ERR_UNSUPPORTED, "channel strides of 2^27 elements or more are not supported");
    if (s.b >= (int64_t(1) << 44) / (batch > 0 ? batch : 1))
        return fail(VS_ERR_UNSUPPORTED, "tensors that span 2^44 elements or more are not supported");
    return VS_OK;
}

int check_aligned(const Span* t, int n, size_t al, const char* what) {
    for (int i = 0; i < n; ++i)
        if (t[i].p && !aligned(t[i].p, al)) return fail(VS_ERR_ALIGN, what);
    return VS_OK;
}

// no output may overlap an input or another output
int check_overlaps(const Span* in, int ni, const Span* out, int no) {
    for (int i = 0; i < no; ++i) {
        for (int j = 0; j < ni; ++j)
            if (overlaps(out[i].p, out[i].n, in[j].p, in[j].n))
                return fail(VS_ERR_ALIAS, "an output or the workspace overlaps an input");
        for (int j = i + 1; j < no; ++j)
            if (overlaps(out[i].p, out[i].n, out[j].p, out[j].n))
                return fail(VS_ERR_ALIAS, "outputs overlap each other or the workspace");
    }
    return VS_OK;
}

}  // namespace

// The forms are chosen by an estimate of their time in shader cycles, from the
// kernels' measured cycles per block of 16 tokens with w workgroups on a
// compute unit (of the 256):
//   narrow scan (16 channels a workgroup)  max(1250, 260 + 750 w)
//   wide scan (64 channels)                max(3300, 2600 w)
//   adjoint (16 channels)                  max(2900, 2100 w)
//   carry launches (64 channels)           max(2450, 1950 w)
// and what the second launch and the folding of p finer pieces add. When they
// were fitted, bf16, both launches together: 8 x 768 x 4,097 tokens narrow 214 us
// uncut, 205 us in 2 pieces of 8; 1 x 768 x 4,097 132 us narrow and uncut; 1 x
// 1,536 x 16,385 570 us narrow, 210 us wide in 21 pieces; 64 x 1,536 x 197 110 us
// narrow, 101 us wide and uncut. Gradient: 8 x 768 x 4,097 553 us uncut, 469 us
// in 2 pieces of 8; 1 x 768 x 4,097 335 us uncut, 87 us in 16 pieces. What is
// chosen now takes, in that order, 190 us, 46 (narrow, 10 pieces of 2), 212, 98;
// gradient 442 and 88 us.
namespace {

int64_t most(int64_t a, int64_t b) { return a > b ? a : b; }

struct Form {
    int64_t channels;
    int64_t least, base, per_wg;        // cycles per block: max(least, base + per_wg w)
    int64_t start, fold;                // a cut adds start (4 + w) and fold (4 + w) for each finer piece
    int64_t max_w;                      // the fullest compute unit that is tried
};
constexpr Form kNarrow{kCausalCh, 1250, 260, 750, 2000, 50, 4}, kWide{kCausalWideCh, 3300, 0, 2600, 3500, 140, 4},
    kAdjoint{kCausalCh, 2900, 0, 2100, 2000, 50, 8};

// the best cut of one form, if it beats `cycles`
void try_form(const Form& f, bool wide, int64_t batch, int64_t dim, int64_t L, ScanCut& best, int64_t& cycles) {
    const int64_t tiles = ceil_div(L, kTileTok), blocks = ceil_div(L, kBlockTok);
    const int64_t wgs = batch * ceil_div(dim, f.channels), carry_wgs = batch * ceil_div(dim, kCausalWideCh);
    auto per_block = [&](int64_t w) { return most(f.least, f.base + f.per_wg * w); };
    const int64_t whole = blocks * per_block(ceil_div(wgs, kNumCUs));
    if (whole < cycles) {
        cycles = whole;
        best = ScanCut{wide, 1, 1, tiles};
    }
    // for each w the most pieces that w workgroups a compute unit hold
    for (int64_t w = 1; w <= f.max_w; ++w) {
        int64_t p = kNumCUs * w / wgs;
        p = p > kCausalMaxPieces ? kCausalMaxPieces : p;
        p = p > tiles ? tiles : p;
        if (p < 2) continue;
        for (int64_t sub = 1; sub <= 8 && p * sub <= tiles && p * sub <= 2 * kCausalMaxPieces; sub *= 2) {
            const int64_t fine = ceil_div(tiles, p * sub);
            const int64_t pieces = ceil_div(tiles, fine * sub);              // no empty pieces
            if (pieces < 2 || batch * pieces * sub > 65535) continue;
            const int64_t wm = ceil_div(wgs * pieces, kNumCUs), wc = ceil_div(carry_wgs * (pieces - 1) * sub, kNumCUs);
            // alone on its compute unit the longest piece counts, else their mean
            const int64_t main = wm == 1 ? 2 * fine * sub : ceil_div(blocks, pieces);
            const int64_t t = main * per_block(wm) + 2 * fine * most(2450, 1950 * wc) +
                              f.start * (4 + w) + f.fold * (4 + w) * pieces * sub;
            if (t < cycles) {
                cycles = t;
                best = ScanCut{wide, static_cast<int>(pieces), static_cast<int>(sub), fine};
            }
        }
    }
}

}  // namespace

ScanCut causal_cut(int64_t batch, int64_t dim, int64_t L) {
    ScanCut best{};
    int64_t cycles = INT64_MAX;
    try_form(kNarrow, false, batch, dim, L, best, cycles);
    try_form(kWide, true, batch, dim, L, best, cycles);
    return best;
}

ScanCut causal_grad_cut(int64_t batch, int64_t dim, int64_t L) {
    ScanCut best{};
    int64_t cycles = INT64_MAX;
    try_form(kAdjoint, false, batch, dim, L, best, cycles);
    return best;
}

// A wave covers kConvGradStep tokens at a time; it takes up to 8 such steps of
// a row where that leaves 16 waves for each of the 1,024 SIMDs (8 x 768 x 4,097
// bf16, 9 steps a row: 3 of them 44 us, 1 58, 8 48).
int64_t conv_grad_segment(int64_t batch, int64_t dim, int64_t L) {
    int64_t steps = batch * dim * ceil_div(L, kConvGradStep) / (16 * 1024);
    steps = steps < 1 ? 1 : (steps > 8 ? 8 : steps);
    return steps * kConvGradStep;
}

size_t causal_saved_layout(int64_t batch, int64_t dim, int64_t dstate, int64_t L, size_t offs[2]) {
    const size_t rows = static_cast<size_t>(batch * dim);
    const size_t nblk = static_cast<size_t>(ceil_div(L, kBlockTok));
    offs[0] = 0;
    offs[1] = al256(rows * nblk * static_cast<size_t>(dstate) * kF);
    return offs[1] + al256(rows * static_cast<size_t>(L) * kF);
}

size_t causal_grad_layout(int64_t batch, int64_t dim, int64_t dstate, int64_t L, size_t offs[4]) {
    const size_t rows = static_cast<size_t>(batch * dim);
    const size_t nblk = static_cast<size_t>(ceil_div(L, kBlockTok));
    const size_t groups = static_cast<size_t>(ceil_div(dim, kCausalCh));
    const ScanCut cut = causal_grad_cut(batch, dim, L);
    const size_t pieces = static_cast<size_t>(cut.pieces), carry = (pieces - 1) * static_cast<size_t>(cut.sub);
    size_t off = 0;
    offs[0] = off; off += al256(static_cast<size_t>(batch) * groups * nblk * 2 * kBlockTok * kRowLanes * kF);
    offs[1] = off; off += al256(rows * pieces * static_cast<size_t>(dstate + 2) * kF);
    offs[2] = off; off += al256(rows * carry * static_cast<size_t>(dstate) * kF);
    offs[3] = off; off += al256(rows * carry * kF);
    return off;
}

size_t causal_ws_bytes(int op, int64_t batch, int64_t dim, int64_t dstate, int64_t L) {
    int code;
    const bool conv = op == VS_S6_CONV_GRAD;
    if (sizes_problem(batch, dim, dstate, L, conv ? 2 : 1, conv ? VS_MAX_CONV_WIDTH : VS_MAX_DSTATE, code)) return 0;
    size_t offs[4];
    const size_t rows = static_cast<size_t>(batch * dim);
    if (op == VS_S6_SCAN) {
        // per finer piece but those of the last: its end state from zero and its sum of delta
        const ScanCut cut = causal_cut(batch, dim, L);
        return rows * static_cast<size_t>((cut.pieces - 1) * cut.sub) * static_cast<size_t>(dstate + 1) * kF;
    }
    if (op == VS_S6_SAVED) return causal_saved_layout(batch, dim, dstate, L, offs);
    if (op == VS_S6_GRAD) return causal_grad_layout(batch, dim, dstate, L, offs);
    if (op == VS_S6_CONV_GRAD)          // per segment of a row: dw and dbias
        return rows * static_cast<size_t>(ceil_div(L, conv_grad_segment(batch, dim, L)) * (dstate + 1)) * kF;
    return 0;
}

int prepare_causal(CausalCall& c) {
    clear_error();
    if (c.dtype != VS_F32 && c.dtype != VS_BF16) return fail(VS_ERR_DTYPE, "unknown dtype");
    if (c.flags & ~VS_FLAG_SOFTPLUS) return fail(VS_ERR_UNSUPPORTED, "the causal scan takes VS_FLAG_SOFTPLUS only");
    int code;
    if (const char* p = sizes_problem(c.batch, c.dim, c.dstate, c.L, 1, VS_MAX_DSTATE, code)) return fail(code, p);
    if (!c.u || !c.delta || !c.B || !c.C || !c.A) return fail(VS_ERR_NULL, "u, delta, B, C and A must not be NULL");
    if (!c.grad && !c.y) return fail(VS_ERR_NULL, "y must not be NULL");
    if (c.grad) {
        if (!c.dy || !c.saved) return fail(VS_ERR_NULL, "dy and saved must not be NULL");
        if (!c.du || !c.ddelta || !c.dB || !c.dC || !c.dA || !c.dD || !c.dbias)
            return fail(VS_ERR_NULL, "every gradient output but dz and dh0 must be given");
        if (c.z && !c.dz) return fail(VS_ERR_NULL, "dz must not be NULL when z is given");
        if (!c.z) c.dz = nullptr;
    }
    const int nst = c.grad ? 6 : 5;
    for (int i = 0; i < nst; ++i) {
        const int64_t rows = i == 3 || i == 4 ? c.dstate : c.dim;
        c.st[i] = c.strides ? Strides{c.strides[2 * i], c.strides[2 * i + 1]} : Strides{rows * c.L, c.L};
        if (i == 2 && !c.z) { c.st[i] = Strides{0, 0}; continue; }
        if (int rc = check_strides(c.st[i], c.batch)) return rc;
    }
    const size_t es = esize(c.dtype);
    const size_t act = static_cast<size_t>(c.batch * c.dim * c.L) * es;
    const size_t bcf = static_cast<size_t>(c.batch * c.dstate * c.L) * kF;
    const size_t par = static_cast<size_t>(c.dim) * kF, pa = par * static_cast<size_t>(c.dstate);
    const size_t states = static_cast<size_t>(c.batch) * pa;
    size_t offs[4];
    const size_t saved = causal_saved_layout(c.batch, c.dim, c.dstate, c.L, offs);
    const size_t ws = c.grad ? causal_grad_layout(c.batch, c.dim, c.dstate, c.L, offs)
                             : causal_ws_bytes(VS_S6_SCAN, c.batch, c.dim, c.dstate, c.L);
    if ((c.save || c.grad) && (!c.saved || c.saved_bytes < saved))
        return fail(VS_ERR_WORKSPACE, "saved-state buffer missing or smaller than s6_workspace_bytes(VS_S6_SAVED)");
    if (ws > 0 && (!c.ws || c.ws_bytes < ws))
        return fail(VS_ERR_WORKSPACE, "workspace missing or smaller than s6_workspace_bytes()");
    const Span acts[] = {{c.u, span_bytes(c.batch, c.dim, c.L, c.st[0], es)},
                         {c.delta, span_bytes(c.batch, c.dim, c.L, c.st[1], es)},
                         {c.z, span_bytes(c.batch, c.dim, c.L, c.st[2], es)},
                         {c.B, span_bytes(c.batch, c.dstate, c.L, c.st[3], es)},
                         {c.C, span_bytes(c.batch, c.dstate, c.L, c.st[4], es)},
                         {c.grad ? c.dy : nullptr, c.grad ? span_bytes(c.batch, c.dim, c.L, c.st[5], es) : 0}};
    const Span params[] = {{c.A, pa}, {c.Dskip, par}, {c.dt_bias, par}, {c.h0, states},
                           {c.lengths, static_cast<size_t>(c.batch) * 4}, {c.grad ? c.dh_out : nullptr, states},
                           {c.grad ? c.saved : nullptr, saved}};
    if (int rc = check_aligned(acts, 6, es, "activation pointer misaligned")) return rc;
    if (int rc = check_aligned(params, 7, 4, "32-bit pointer misaligned")) return rc;
    Span ins[13];
    for (int i = 0; i < 6; ++i) ins[i] = acts[i];
    for (int i = 0; i < 7; ++i) ins[6 + i] = params[i];
    if (!c.grad) {
        const Span outs[] = {{c.y, act}, {c.h_out, states}, {c.save ? c.saved : nullptr, saved}, {c.ws, ws}};
        if (int rc = check_aligned(outs, 1, es, "activation pointer misaligned")) return rc;
        if (int rc = check_aligned(outs + 1, 3, 4, "32-bit pointer misaligned")) return rc;
        return check_overlaps(ins, 13, outs, 4);
    }
    const Span outs[] = {{c.du, act}, {c.ddelta, act}, {c.dz, act}, {c.dB, bcf}, {c.dC, bcf}, {c.dA, pa},
                         {c.dD, par}, {c.dbias, par}, {c.dh0, states}, {c.ws, ws}};
    if (int rc = check_aligned(outs, 3, es, "activation pointer misaligned")) return rc;
    if (int rc = check_aligned(outs + 3, 7, 4, "32-bit pointer misaligned")) return rc;
    return check_overlaps(ins, 13, outs, 10);
}

int prepare_conv(ConvCall& c) {
    clear_error();
    if (c.dtype != VS_F32 && c.dtype != VS_BF16) return fail(VS_ERR_DTYPE, "unknown dtype");
    if (c.flags & ~VS_CONV_SILU) return fail(VS_ERR_UNSUPPORTED, "unknown flag bits");
    int code;
    if (const char* p = sizes_problem(c.batch, c.dim, c.width, c.L, 2, VS_MAX_CONV_WIDTH, code)) return fail(code, p);
    if (!c.x || !c.w) return fail(VS_ERR_NULL, "x and w must not be NULL");
    if (c.grad ? !c.dy || !c.dx || !c.dw || !c.dbias : !c.y)
        return fail(VS_ERR_NULL, c.grad ? "dy, dx, dw and dbias must not be NULL" : "y must not be NULL");
    for (int i = 0; i < (c.grad ? 2 : 1); ++i) {
        c.st[i] = c.strides ? Strides{c.strides[2 * i], c.strides[2 * i + 1]} : Strides{c.dim * c.L, c.L};
        if (int rc = check_strides(c.st[i], c.batch)) return rc;
    }
    const size_t es = esize(c.dtype);
    const size_t act = static_cast<size_t>(c.batch * c.dim * c.L) * es;
    const size_t win = static_cast<size_t>(c.batch * c.dim * (c.width - 1)) * es;
    const size_t par = static_cast<size_t>(c.dim) * kF, pw = par * static_cast<size_t>(c.width);
    const size_t ws = c.grad ? causal_ws_bytes(VS_S6_CONV_GRAD, c.batch, c.dim, c.width, c.L) : 0;
    if (ws > 0 && (!c.ws || c.ws_bytes < ws))
        return fail(VS_ERR_WORKSPACE, "workspace missing or smaller than s6_workspace_bytes()");
    const Span ins[] = {{c.x, span_bytes(c.batch, c.dim, c.L, c.st[0], es)}, {c.window, win},
                        {c.grad ? c.dy : nullptr, c.grad ? span_bytes(c.batch, c.dim, c.L, c.st[1], es) : 0},
                        {c.grad ? c.dwindow_out : nullptr, win},
                        {c.w, pw}, {c.bias, par}, {c.lengths, static_cast<size_t>(c.batch) * 4}};
    if (int rc = check_aligned(ins, 4, es, "activation pointer misaligned")) return rc;
    if (int rc = check_aligned(ins + 4, 3, 4, "32-bit pointer misaligned")) return rc;
    if (!c.grad) {
        const Span outs[] = {{c.y, act}, {c.window_out, win}};
        if (int rc = check_aligned(outs, 2, es, "activation pointer misaligned")) return rc;
        return check_overlaps(ins, 7, outs, 2);
    }
    const Span outs[] = {{c.dx, act}, {c.dwindow, win}, {c.dw, pw}, {c.dbias, par}, {c.ws, ws}};
    if (int rc = check_aligned(outs, 2, es, "activation pointer misaligned")) return rc;
    if (int rc = check_aligned(outs + 2, 3, 4, "32-bit pointer misaligned")) return rc;
    return check_overlaps(ins, 7, outs, 5);
}

namespace {

int check_step(StepCall& c, int nst, int64_t inner_low, int64_t inner_high, size_t pool_el) {
    clear_error();
    if (c.dtype != VS_F32 && c.dtype != VS_BF16) return fail(VS_ERR_DTYPE, "unknown dtype");
    int code;
    if (const char* p = sizes_problem(c.batch, c.dim, c.inner, 1, inner_low, inner_high, code)) return fail(code, p);
    if (c.slots < 1) return fail(VS_ERR_SHAPE, "the pool must have at least one slot");
    if (c.slots >= (int64_t(1) << 31) || !product_below(c.slots, c.dim, c.inner, int64_t(1) << 44))
        return fail(VS_ERR_UNSUPPORTED, "pools of 2^44 elements or 2^31 slots or more are not supported");
    for (int i = 0; i < nst; ++i) {
        const int64_t row = i < 3 ? c.dim : c.inner;
        c.st[i] = c.strides && (nst > 1 || c.strides[i] != 0) ? c.strides[i] : row;
        if (c.st[i] < 0) return fail(VS_ERR_SHAPE, "strides must be >= 0");
        if (c.st[i] >= (int64_t(1) << 28)) return fail(VS_ERR_UNSUPPORTED, "row strides of 2^28 elements or more are not supported");
    }
    const size_t es = esize(c.dtype);
    const size_t par = static_cast<size_t>(c.dim) * kF;
    auto span = [&](const void* p, int i, int64_t len) {
        return Span{p, p ? (static_cast<size_t>((c.batch - 1) * c.st[i]) + static_cast<size_t>(len)) * es : 0};
    };
    Span acts[5] = {span(c.u, 0, c.dim), {}, {}, {}, {}};
    if (nst > 1) {
        acts[1] = span(c.delta, 1, c.dim);
        acts[2] = span(c.z, 2, c.dim);
        acts[3] = span(c.B, 3, c.inner);
        acts[4] = span(c.C, 4, c.inner);
    }
    const size_t idx = static_cast<size_t>(c.batch) * 4;
    const Span params[] = {{c.A, par * static_cast<size_t>(c.inner)}, {c.Dskip, par}, {c.dt_bias, par},
                           {c.slot_in, idx}, {c.slot_out, idx}};
    const Span outs[] = {{c.y, static_cast<size_t>(c.batch * c.dim) * es},
                         {c.pool, static_cast<size_t>(c.slots * c.dim) * pool_el}};
    if (int rc = check_aligned(acts, 5, es, "activation pointer misaligned")) return rc;
    if (int rc = check_aligned(params, 5, 4, "32-bit pointer misaligned")) return rc;
    if (int rc = check_aligned(outs, 1, es, "activation pointer misaligned")) return rc;
    if (int rc = check_aligned(outs + 1, 1, nst > 1 ? 4 : es, "state pointer misaligned")) return rc;
    Span ins[10];
    for (int i = 0; i < 5; ++i) ins[i] = acts[i];
    for (int i = 0; i < 5; ++i) ins[5 + i] = params[i];
    return check_overlaps(ins, 10, outs, 2);
}

// without slot arrays row b uses slot b
int check_slots(const StepCall& c) {
    if ((!c.slot_in || !c.slot_out) && c.slots < c.batch)
        return fail(VS_ERR_SHAPE, "without slot_in or slot_out the pool needs a slot for every row");
    return VS_OK;
}

}  // namespace

int prepare_conv_step(StepCall& c) {
    const size_t es = esize(c.dtype);
    if (int rc = check_step(c, 1, 2, VS_MAX_CONV_WIDTH, static_cast<size_t>(c.inner > 1 ? c.inner - 1 : 1) * es)) return rc;
    if (c.flags & ~VS_CONV_SILU) return fail(VS_ERR_UNSUPPORTED, "unknown flag bits");
    if (!c.u || !c.A || !c.pool || !c.y) return fail(VS_ERR_NULL, "x, w, window and y must not be NULL");
    return check_slots(c);
}

int prepare_scan_step(StepCall& c) {
    if (int rc = check_step(c, 5, 1, VS_MAX_DSTATE, static_cast<size_t>(c.inner > 0 ? c.inner : 1) * kF)) return rc;
    if (c.flags & ~VS_FLAG_SOFTPLUS) return fail(VS_ERR_UNSUPPORTED, "the causal scan takes VS_FLAG_SOFTPLUS only");
    if (!c.u || !c.delta || !c.B || !c.C || !c.A || !c.pool || !c.y)
        return fail(VS_ERR_NULL, "u, delta, B, C, A, h and y must not be NULL");
    return check_slots(c);
}

// ---- beam search
namespace {

bool beam_sizes_ok(int64_t batch, int64_t beams, int64_t vocab) {
    return batch >= 1 && batch <= 65535 && beams >= 1 && beams <= VS_MAX_BEAMS && vocab >= 1 && vocab < (int64_t(1) << 30);
}

}  // namespace

int validate_beam_select(int64_t batch, int64_t beams, int64_t vocab, int dtype, const void* logits,
                         const int64_t* strides, const float* scores, const uint8_t* done, int64_t eos,
                         const float* out_scores, const int32_t* out_parent, const int32_t* out_token,
                         const void* ws, size_t ws_bytes, int64_t st[2]) {
    clear_error();
    if (dtype != VS_F32 && dtype != VS_BF16) return fail(VS_ERR_DTYPE, "unknown dtype");
    if (batch < 1 || beams < 1 || vocab < 1) return fail(VS_ERR_SHAPE, "batch, beams and vocab must be >= 1");
    if (!beam_sizes_ok(batch, beams, vocab))
        return fail(VS_ERR_UNSUPPORTED, "beams above 32, a batch above 65535 or a vocabulary of 2^30 or more is not supported");
    if (!logits || !scores || !out_scores || !out_parent || !out_token)
        return fail(VS_ERR_NULL, "logits, scores and the outputs must not be NULL");
    if (done && (eos < 0 || eos >= vocab)) return fail(VS_ERR_SHAPE, "eos must be in 0..vocab-1");
    st[0] = strides ? strides[0] : beams * vocab;
    st[1] = strides ? strides[1] : vocab;
    if (st[0] < 0 || st[1] < 0) return fail(VS_ERR_SHAPE, "strides must be >= 0");
    if (st[0] >= (int64_t(1) << 40) || st[1] >= (int64_t(1) << 40))
        return fail(VS_ERR_UNSUPPORTED, "strides of 2^40 elements or more are not supported");
    const size_t es = esize(dtype), rows = static_cast<size_t>(batch * beams);
    const size_t need = beam_workspace_bytes(batch, beams, vocab);
    if (!ws || ws_bytes < need) return fail(VS_ERR_WORKSPACE, "workspace missing or smaller than beam_workspace_bytes()");
    const Span ins[] = {{logits, (static_cast<size_t>((batch - 1) * st[0] + (beams - 1) * st[1]) + static_cast<size_t>(vocab)) * es},
                        {scores, rows * 4}, {done, rows}};
    const Span outs[] = {{out_scores, rows * 4}, {out_parent, rows * 4}, {out_token, rows * 4}, {ws, need}};
    if (int rc = check_aligned(ins, 1, es, "logits misaligned")) return rc;
    if (int rc = check_aligned(ins + 1, 1, 4, "32-bit pointer misaligned")) return rc;
    if (int rc = check_aligned(outs, 3, 4, "32-bit pointer misaligned")) return rc;
    if (int rc = check_aligned(outs + 3, 1, 8, "workspace misaligned (8 bytes)")) return rc;
    return check_overlaps(ins, 3, outs, 4);
}

int validate_beam_reorder(int64_t layers, int64_t batch, int64_t beams, int64_t row_bytes,
                          int64_t& layer_bytes, const void* state, const int32_t* parent, const void* out) {
    clear_error();
    if (layers < 1 || batch < 1 || beams < 1 || row_bytes < 1)
        return fail(VS_ERR_SHAPE, "layers, batch, beams and row_bytes must be >= 1");
    if (beams > VS_MAX_BEAMS || batch > 65535 || layers > 65535)
        return fail(VS_ERR_UNSUPPORTED, "beams above 32, or a batch or layers above 65535, are not supported");
    if (row_bytes >= (int64_t(1) << 36)) return fail(VS_ERR_UNSUPPORTED, "rows of 2^36 bytes or more are not supported");
    if (!state || !parent || !out) return fail(VS_ERR_NULL, "state, parent and out must not be NULL");
    const int64_t dense = batch * beams * row_bytes;         // below 2^57
    if (layer_bytes == 0) layer_bytes = dense;
    if (layer_bytes < dense) return fail(VS_ERR_SHAPE, "layer_bytes is smaller than a layer's rows");
    if (layer_bytes >= (int64_t(1) << 58) / layers) return fail(VS_ERR_UNSUPPORTED, "states of 2^58 bytes or more are not supported");
    if (!aligned(parent, 4)) return fail(VS_ERR_ALIGN, "32-bit pointer misaligned");
    const size_t all = static_cast<size_t>(layer_bytes * (layers - 1) + dense);
    if (overlaps(out, all, parent, static_cast<size_t>(batch * beams) * 4)) return fail(VS_ERR_ALIAS, "out overlaps parent");
    if (out != state && overlaps(out, all, state, all)) return fail(VS_ERR_ALIAS, "out partly overlaps state");
    return VS_OK;
}

}  // namespace vs

// ---------------------------------------------------------------- C ABI
extern "C" {

size_t s6_workspace_bytes(int op, int64_t batch, int64_t dim, int64_t dstate, int64_t seqlen) {
    return vs::causal_ws_bytes(op, batch, dim, dstate, seqlen);
}

size_t beam_workspace_bytes(int64_t batch, int64_t beams, int64_t vocab) {
    if (!vs::beam_sizes_ok(batch, beams, vocab)) return 0;
    // per part of a row: `beams` candidates of 8 bytes, then its maximum and its sum
    return static_cast<size_t>(batch * beams * vs::beam_parts(vocab)) * static_cast<size_t>(beams + 1) * 8;
}

}  // extern "C"
