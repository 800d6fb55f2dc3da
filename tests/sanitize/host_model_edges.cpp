// Calls at the edge of what the host layer of the gated recurrence, the norm and
// the vocabulary loss accepts (csrc/host_model.cpp), under the address and
// undefined-behaviour sanitizers. Addresses are made up: nothing is read through
// them.
#include <cstdint>
#include <cstdio>

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

vs::NormCall norm(int64_t batch, int64_t dim, int64_t L, const int64_t* strides) {
    vs::NormCall c{};
    c.batch = batch; c.dim = dim; c.L = L; c.dtype = VS_BF16; c.x = at(0); c.w = fp(1); c.eps = 1e-6f; c.y = at(2); c.strides = strides;
    return c;
}

// the sum is the residual itself: whatever stands for the stride of an axis of one
void in_place() {
    const int64_t one_channel[] = {70, 1, 70, 1}, one_row[] = {5, 70, 5, 70}, apart[] = {70, 1, 80, 1};
    vs::NormCall c = norm(4, 1, 70, one_channel);
    c.residual = c.sum = at(3);
    expect(vs::prepare_norm(c) == VS_OK, "in place, one channel");
    c = norm(1, 6, 70, one_row);
    c.residual = c.sum = at(3);
    expect(vs::prepare_norm(c) == VS_OK, "in place, one row");
    c = norm(4, 1, 70, apart);
    c.residual = c.sum = at(3);
    expect(vs::prepare_norm(c) == VS_ERR_ALIAS, "one channel, rows that lie apart");
}

// the workspace of the gradient's sums: what norm_workspace_bytes() says suffices for
// any type and strides, no more lines for one token a row past 4,096 (past 512
// channels 1,024), and 64 MB or that many lines for longer rows
void norm_workspaces() {
    const int64_t batches[] = {1, 2, 3, 700, 1023, 1025, 4097, 8194, 65536, 100000, (int64_t(1) << 22) - 1};
    const int64_t lengths[] = {1, 2, 17, 32, 33, 100, 4097, 21845, 43712, 70000, 100000, (int64_t(1) << 27) - 1};
    for (int64_t batch : batches)
        for (int64_t dim : {1, 24, 384, 385, 512, 513, 768, 769, 1536, 4096, 8192})
            for (int64_t L : lengths) {
                const size_t bytes = norm_workspace_bytes(batch, dim, L);
                if (bytes == 0) continue;                    // sizes that are refused
                const int64_t strides[] = {dim, 1, dim, 1, dim, 1}, apart[] = {2 * dim * L, 2 * L, 2 * dim * L, 2 * L, 2 * dim * L, 2 * L};
                for (int k = 0; k < 6; ++k) {
                    vs::NormCall c = norm(batch, dim, L, k / 2 == 0 ? nullptr : k / 2 == 1 && L == 1 ? strides : apart);
                    c.dtype = k % 2 ? VS_BF16 : VS_F32;
                    c.grad = true; c.dy = at(3); c.dw = fp(4); c.ws = at(5); c.ws_bytes = bytes;
                    expect(vs::prepare_norm(c) == VS_OK || vs::last_error()[0] != 'w', "a workspace of the stated size");
                    if (c.form == vs::kNormColumn) {
                        const int64_t tiles = (L + c.tile - 1) / c.tile;
                        expect(c.slab >= 1 && c.slab <= batch && c.slab * tiles == c.parts, "a slab's tiles");
                    }
                }
                const int64_t few = dim > 512 ? 1024 : 4096, lines = static_cast<int64_t>(bytes) / 4 / dim;
                if (L == 1) expect(lines <= few, "rows of one token: a bounded workspace");
                else expect(lines <= few || lines * dim * 4 <= 64 << 20 || lines <= (L + 15) / 16, "a bounded workspace");
            }
}

// Operands are read by words: rows whose length is no whole number of them are
// packed, also where their stride is one, for the last row may end the caller's memory.
void odd_rows() {
    for (int64_t dim : {1, 24, 25, 26, 63})
        for (int64_t ldx : {dim, dim + 1, dim + 2, int64_t(70000)})
            for (int dtype : {VS_F32, VS_BF16}) {
                vs::VocabCall c{};
                c.tokens = 5; c.dim = dim; c.vocab = 100; c.dtype = dtype; c.x = at(0); c.ldx = ldx; c.W = at(1); c.target = at(2);
                c.target_bits = 64; c.loss = fp(4); c.lse = fp(5); c.ws = at(3); c.ws_bytes = size_t(1) << 43;
                expect(vs::prepare_vocab(c) == VS_OK, "a loss");
                const bool odd = dtype == VS_BF16 && (dim % 2 || ldx % 2);
                expect(c.plan.pack_x == (odd || ldx > 65536) && c.plan.pack_w == (dtype == VS_BF16 && dim % 2), "rows that are packed");
            }
}

// bf16: a gradient's workspace ends with what rounding took off the targets' entries, a token each
void rests() {
    for (int64_t t : {1, 33, 500, 4097, 8194})
        for (int64_t d : {1, 24, 1536})
            for (int64_t v : {1, 257, 49999, 1000000}) {
                const vs::VocabPlan g = vs::vocab_plan(true, t, d, v, VS_BF16);
                expect(g.rest >= g.sum + (g.pieces > 1 ? size_t(t * d) * 4 : 0) && g.rest + size_t(t) * 4 <= g.bytes, "their place");
            }
}

}  // namespace

int main() {
    in_place();
    norm_workspaces();
    odd_rows();
    rests();
    if (failures) return 1;
    std::puts("host model edges ok");
    return 0;
}
