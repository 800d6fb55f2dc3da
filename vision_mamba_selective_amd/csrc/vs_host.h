// Checks that the host-side files of libvimscan.so share: sizes, strides,
// alignment and overlaps of a call's tensors. Plain C++ with no HIP. Internal.
#pragma once

#include <cstdint>

#include "vs_internal.h"

namespace vs {
namespace {

constexpr size_t kF = 4;                 // bytes of an fp32 value

inline size_t al256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
inline size_t esize(int dtype) { return dtype == VS_BF16 ? 2 : 4; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// sizes every entry point of the mixer shares; `inner` is dstate or the width
inline const char* sizes_problem(int64_t batch, int64_t dim, int64_t inner, int64_t L, int64_t inner_low,
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
inline size_t span_bytes(int64_t batch, int64_t rows, int64_t len, const Strides& s, size_t es) {
    return (static_cast<size_t>((batch - 1) * s.b + (rows - 1) * s.d) + static_cast<size_t>(len)) * es;
}

inline int check_strides(const Strides& s, int64_t batch) {
    if (s.b < 0 || s.d < 0) return fail(VS_ERR_SHAPE, "strides must be >= 0");
    if (s.d >= kCausalMaxL) return fail(VS_ERR_UNSUPPORTED, "channel strides of 2^27 elements or more are not supported");
    if (s.b >= (int64_t(1) << 44) / (batch > 0 ? batch : 1))
        return fail(VS_ERR_UNSUPPORTED, "tensors that span 2^44 elements or more are not supported");
    return VS_OK;
}

inline int check_aligned(const Span* t, int n, size_t al, const char* what) {
    for (int i = 0; i < n; ++i)
        if (t[i].p && !aligned(t[i].p, al)) return fail(VS_ERR_ALIGN, what);
    return VS_OK;
}

// no output may overlap an input or another output
inline int check_overlaps(const Span* in, int ni, const Span* out, int no) {
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
}  // namespace vs
