// Drives the host layer of the gated recurrence, the norm and the vocabulary
// loss (csrc/host_model.cpp) with ordinary and extreme arguments under the
// address and undefined-behaviour sanitizers. Addresses are made up: nothing is
// read through them.
#include <cstdint>
#include <cstdio>
#include <cstdlib>

#include "vs_model.h"

namespace {

int failures = 0;
void expect(bool ok, const char* what) {
    if (!ok) {
        std::fprintf(stderr, "FAILED: %s (%s)\n", what, vs::last_error());
        ++failures;
    }
}
void* at(uint64_t i) { return reinterpret_cast<void*>((uint64_t(1) << 44) + (i << 44)); }
float* fp(uint64_t i) { return static_cast<float*>(at(i)); }
const int64_t kBig = INT64_MAX;

vs::GatedCall gated(bool grad) {
    vs::GatedCall c{};
    c.batch = 2; c.dim = 8; c.L = 33; c.dtype = VS_BF16; c.x = at(0); c.r = at(1); c.i = at(2); c.z = at(3); c.lam = fp(4); c.rate = 8.f;
    c.saved = at(5); c.saved_bytes = size_t(1) << 43;
    if (grad) {
        c.grad = true; c.dy = at(6); c.dx = at(7); c.dr = at(8); c.di = at(9); c.dz = at(10); c.dlam = fp(11); c.ws = at(12);
        c.ws_bytes = size_t(1) << 43;
    } else {
        c.save = true; c.y = at(7); c.h_out = fp(8);
    }
    return c;
}
vs::GatedStepCall step() {
    vs::GatedStepCall c{};
    c.batch = 2; c.dim = 8; c.dtype = VS_F32; c.x = at(0); c.r = at(1); c.i = at(2); c.lam = fp(3); c.rate = 1.f; c.h = fp(4); c.slots = 2;
    c.y = at(5);
    return c;
}
vs::NormCall norm(bool grad) {
    vs::NormCall c{};
    c.batch = 2; c.dim = 8; c.L = 33; c.dtype = VS_F32; c.x = at(0); c.w = fp(1); c.eps = 0.f; c.y = at(2);
    if (grad) { c.grad = true; c.dy = at(3); c.dw = fp(4); c.ws = at(5); c.ws_bytes = size_t(1) << 43; }
    else { c.residual = at(3); c.sum = at(3); }
    return c;
}
vs::VocabCall vocab(bool grad) {
    vs::VocabCall c{};
    c.tokens = 5; c.dim = 24; c.vocab = 100; c.dtype = VS_BF16; c.x = at(0); c.W = at(1); c.target = at(2); c.target_bits = 64; c.ws = at(3);
    c.ws_bytes = size_t(1) << 43;
    if (grad) { c.grad = true; c.lse_in = fp(4); c.dloss = fp(5); c.dx = at(6); c.dW = at(7); }
    else { c.loss = fp(4); c.lse = fp(5); }
    return c;
}

template <typename T>
T& made(T c) {
    static T kept;
    return kept = c;
}

}  // namespace

int main() {
    expect(vs::prepare_gated(made(gated(false))) == VS_OK, "an ordinary recurrence");
    expect(vs::prepare_gated(made(gated(true))) == VS_OK, "its gradient");
    expect(vs::prepare_gated_step(made(step())) == VS_OK, "its step");
    expect(vs::prepare_norm(made(norm(false))) == VS_OK, "a norm in place");
    expect(vs::prepare_norm(made(norm(true))) == VS_OK, "its gradient");
    expect(vs::prepare_vocab(made(vocab(false))) == VS_OK, "a loss");
    expect(vs::prepare_vocab(made(vocab(true))) == VS_OK, "its gradient");
    const int64_t extremes[] = {INT64_MIN, -1, 0, 1, 2, 31, 33, 8192, 65535, 65536, int64_t(1) << 20, (int64_t(1) << 24) - 1,
                                (int64_t(1) << 27) - 1, int64_t(1) << 31, int64_t(1) << 44, int64_t(1) << 62, kBig};
    for (int64_t a : extremes)
        for (int64_t b : extremes) {
            int64_t st[10] = {a, b, 264, 33, b, a, 264, 33, a, a};
            vs::GatedCall g = gated(true);
            g.strides = st;
            (void)vs::prepare_gated(g);
            vs::GatedStepCall s = step();
            s.strides = st;
            (void)vs::prepare_gated_step(s);
            for (int k = 0; k < 2; ++k) {
                vs::NormCall n = norm(k);
                n.strides = st;
                (void)vs::prepare_norm(n);
                vs::VocabCall v = vocab(k);
                v.ldx = a;
                v.tokens = b;
                (void)vs::prepare_vocab(v);
            }
            for (int64_t d : extremes) {
                for (int op = -1; op < 3; ++op) {
                    gated_workspace_bytes(op, a, b, d);
                    vocab_workspace_bytes(op, a, b, d, VS_BF16);
                    vocab_workspace_bytes(op, a, b, d, VS_F32);
                }
                norm_workspace_bytes(a, b, d);
                for (int k = 0; k < 2; ++k) {
                    vs::GatedCall c = gated(k);
                    c.batch = a; c.dim = b; c.L = d;
                    (void)vs::prepare_gated(c);
                    vs::NormCall n = norm(k);
                    n.batch = a; n.dim = b; n.L = d;
                    (void)vs::prepare_norm(n);
                    vs::VocabCall v = vocab(k);
                    v.tokens = a; v.dim = b; v.vocab = d;
                    (void)vs::prepare_vocab(v);
                }
                vs::GatedStepCall t = step();
                t.batch = a; t.dim = b; t.slots = d;
                (void)vs::prepare_gated_step(t);
            }
        }
    // forms and plans: every token and entry is covered, launches fit the grid
    const int64_t sizes[] = {1, 2, 31, 32, 33, 100, 127, 128, 129, 255, 257, 500, 1000, 4097, 8194, 49999, 100000, 1000000};
    for (int64_t t : sizes)
        for (int64_t d : sizes)
            for (int64_t v : sizes) {
                if (d > 65536 || t * v >= (int64_t(1) << 36)) continue;
                for (int dtype : {VS_F32, VS_BF16}) {
                    const vs::VocabPlan f = vs::vocab_plan(false, t, d, v, dtype), g = vs::vocab_plan(true, t, d, v, dtype);
                    expect(int64_t(f.tiles) * (f.wide ? 256 : 128) >= v, "tiles cover the vocabulary");
                    expect(g.piece * g.pieces >= v && g.piece * (g.pieces - 1) < v && g.piece % 256 == 0, "pieces cover it, none is empty");
                    expect(f.dp >= d && f.dp % 8 == 0, "packed rows are whole");
                    expect(g.dx_splits >= 1 && g.dw_splits >= 1 && g.dx_splits <= 64 && g.dw_splits <= 64, "splits");
                    expect(f.part + size_t(f.tiles) * size_t(t) * 8 <= f.logit && f.logit + size_t(t) * 4 <= f.bytes, "forward workspace");
                    const size_t n = size_t(g.piece < v ? g.piece : v);
                    expect(g.P + size_t(t) * ((n + 7) / 8 * 8) * (dtype == VS_BF16 ? 2 : 4) <= g.part_dx, "P's place");
                    if (g.dx_splits > 1) expect(g.part_dx + size_t(g.dx_splits) * size_t(t * d) * 4 <= g.part_dw, "dx's parts");
                    if (g.dw_splits > 1) expect(g.part_dw + size_t(g.dw_splits) * n * size_t(d) * 4 <= g.sum, "dW's parts");
                    if (g.pieces > 1) expect(g.sum + size_t(t * d) * 4 <= g.bytes, "the sum of dx");
                }
                const vs::GatedForm form = vs::gated_form(t, d, v);
                expect((form.lanes == 16 && form.waves == 1) || (form.lanes == 64 && (form.waves == 1 || form.waves == 4 || form.waves == 8)),
                       "a form that is built");
            }
    if (failures) return 1;
    std::puts("host model checks ok");
    return 0;
}
