// Drives the host layer of the causal mixer and beam search
// (csrc/host_causal.cpp) with ordinary and extreme arguments under the address
// and undefined-behaviour sanitizers. Addresses are made up: nothing is read
// through them.
#include <cstdint>
#include <cstdio>
#include <cstdlib>

#include "vs_internal.h"

namespace {

int failures = 0;
void expect(bool ok, const char* what) {
    if (!ok) {
        std::fprintf(stderr, "FAILED: %s (%s)\n", what, vs::last_error());
        ++failures;
    }
}
void* at(uint64_t i) { return reinterpret_cast<void*>((uint64_t(1) << 44) + (i << 40)); }
const int64_t kBig = INT64_MAX;

vs::CausalCall scan() {
    vs::CausalCall c{};
    c.batch = 2; c.dim = 8; c.dstate = 16; c.L = 33; c.dtype = VS_BF16; c.flags = VS_FLAG_SOFTPLUS;
    c.u = at(0); c.delta = at(1); c.z = at(2); c.B = at(3); c.C = at(4); c.A = static_cast<float*>(at(5));
    c.y = at(8); c.h_out = static_cast<float*>(at(9)); c.ws = at(10); c.ws_bytes = size_t(1) << 39;
    return c;
}
vs::CausalCall grad() {
    vs::CausalCall c = scan();
    c.y = nullptr; c.h_out = nullptr; c.grad = true; c.dy = at(11); c.saved = at(12); c.saved_bytes = size_t(1) << 39;
    c.du = at(13); c.ddelta = at(14); c.dz = at(15); c.dB = static_cast<float*>(at(16)); c.dC = static_cast<float*>(at(17));
    c.dA = static_cast<float*>(at(18)); c.dD = static_cast<float*>(at(19)); c.dbias = static_cast<float*>(at(20));
    return c;
}
vs::ConvCall conv() {
    vs::ConvCall c{};
    c.batch = 2; c.dim = 8; c.width = 4; c.L = 33; c.dtype = VS_F32; c.x = at(0); c.w = static_cast<float*>(at(1));
    c.y = at(2); c.window_out = at(3);
    return c;
}
vs::StepCall step() {
    vs::StepCall c{};
    c.batch = 2; c.dim = 8; c.inner = 16; c.dtype = VS_F32; c.u = at(0); c.delta = at(1); c.B = at(2); c.C = at(3);
    c.A = static_cast<float*>(at(4)); c.pool = at(5); c.slots = 2; c.y = at(6);
    return c;
}

}  // namespace

int main() {
    const int64_t extremes[] = {INT64_MIN, -1, 0, 1, 2, 15, 16, 17, 65535, 65536, int64_t(1) << 20, int64_t(1) << 27,
                                int64_t(1) << 31, int64_t(1) << 40, int64_t(1) << 62, kBig};
    // every combination of extreme sizes: no overflow, and sizes refused by the calls have no workspace
    for (int64_t a : extremes)
        for (int64_t b : extremes)
            for (int64_t d : extremes) {
                for (int op = -1; op < 5; ++op) s6_workspace_bytes(op, a, b, 16, d);
                s6_workspace_bytes(VS_S6_CONV_GRAD, a, b, d, 100);
                s6_workspace_bytes(VS_S6_GRAD, a, b, d, 100);
                beam_workspace_bytes(a, b, d);
                vs::CausalCall c = scan();
                c.batch = a; c.dim = b; c.L = d;
                c.ws_bytes = 0;
                (void)vs::prepare_causal(c);
                vs::CausalCall g = grad();
                g.batch = a; g.dim = b; g.dstate = d;
                (void)vs::prepare_causal(g);
                vs::ConvCall v = conv();
                v.batch = a; v.dim = b; v.L = d;
                (void)vs::prepare_conv(v);
                vs::StepCall s = step();
                s.batch = a; s.dim = b; s.slots = d;
                (void)vs::prepare_scan_step(s);
                (void)vs::prepare_conv_step(s);
                int64_t st[2], strides[2] = {a, b}, lb = d;
                (void)vs::validate_beam_select(a, b, d, VS_F32, at(0), nullptr, static_cast<float*>(at(1)), nullptr, 0,
                                               static_cast<float*>(at(2)), static_cast<int32_t*>(at(3)), static_cast<int32_t*>(at(4)),
                                               at(5), kBig, st);
                (void)vs::validate_beam_select(3, 4, 100, VS_F32, at(0), strides, static_cast<float*>(at(1)), nullptr, 0,
                                               static_cast<float*>(at(2)), static_cast<int32_t*>(at(3)), static_cast<int32_t*>(at(4)),
                                               at(5), kBig, st);
                (void)vs::validate_beam_reorder(a, b, 4, d, lb, at(0), static_cast<int32_t*>(at(6)), at(1));
                int64_t lb2 = a;
                (void)vs::validate_beam_reorder(b, 2, 4, d, lb2, at(0), static_cast<int32_t*>(at(6)), at(1));
            }
    {
        vs::CausalCall c = scan();
        expect(vs::prepare_causal(c) == VS_OK, "an ordinary scan");
        for (int64_t a : extremes)
            for (int64_t b : extremes) {
                int64_t st[12] = {a, b, 264, 33, a, b, 528, 33, b, a, 264, 33};
                vs::CausalCall s = scan(), g = grad();
                s.strides = g.strides = st;
                (void)vs::prepare_causal(s);
                (void)vs::prepare_causal(g);
            }
        vs::CausalCall g = grad();
        expect(vs::prepare_causal(g) == VS_OK, "an ordinary gradient");
        vs::ConvCall v = conv();
        expect(vs::prepare_conv(v) == VS_OK, "an ordinary convolution");
        vs::StepCall s = step();
        expect(vs::prepare_scan_step(s) == VS_OK, "an ordinary step");
    }
    // a cut leaves no token out, and its launches fit the grid
    const int64_t batches[] = {1, 2, 3, 7, 8, 64, 515, 65535}, dims[] = {1, 24, 100, 384, 768, 1536, 100000},
                  lens[] = {1, 16, 31, 32, 33, 100, 197, 1000, 4097, 16385, 100000, (int64_t(1) << 27) - 1};
    for (int64_t b : batches)
        for (int64_t d : dims)
            for (int64_t l : lens)
                for (int k = 0; k < 2; ++k) {
                    const vs::ScanCut c = k ? vs::causal_grad_cut(b, d, l) : vs::causal_cut(b, d, l);
                    const int64_t piece = c.fine_tiles * c.sub * vs::kTileTok;
                    expect(c.pieces >= 1 && c.sub >= 1 && c.fine_tiles >= 1, "a cut has pieces");
                    expect(piece * c.pieces >= l && piece * (c.pieces - 1) < l, "a cut covers the row, with no empty piece");
                    expect(c.pieces == 1 || b * c.pieces * c.sub <= 65535, "a cut's launches fit the grid");
                    expect(piece < (int64_t(1) << 31), "a piece's length fits an int");
                }
    if (failures) return 1;
    std::puts("host causal checks ok");
    return 0;
}
