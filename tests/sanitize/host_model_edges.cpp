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

}  // namespace

int main() {
    in_place();
    if (failures) return 1;
    std::puts("host model edges ok");
    return 0;
}
