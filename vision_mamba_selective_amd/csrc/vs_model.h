// Argument records, workspace layouts and choices of form of the gated linear
// recurrence, the norm and the vocabulary loss. Filled and checked by
// host_model.cpp (plain C++, no HIP); read by the kernel files. Internal to
// libvimscan.so.
#pragma once

#include "vs_internal.h"

namespace __attribute__((visibility("hidden"))) vs {

// ---- the gated linear recurrence (gated.hip)
constexpr int kGatedVec = 8;                        // consecutive tokens of one lane
// A row is taken by `lanes` lanes of a wave (16 or 64) or by `waves` whole
// waves (1, 4 or 8), each lane eight tokens at a time; a state is saved for
// every `block` tokens of a row.
struct GatedForm {
    int lanes, waves;
    int block() const { return kGatedVec * lanes; }
};
GatedForm gated_form(int64_t batch, int64_t dim, int64_t L);
size_t gated_ws_bytes(int op, int64_t batch, int64_t dim, int64_t L);

struct GatedCall {
    int64_t batch, dim, L;
    int dtype;
    const void *x, *r, *i, *z, *dy;
    const int64_t* strides;                          // as the caller gave them (may be NULL)
    const float* lam;
    float rate;
    const float* h0;
    const int32_t* lengths;
    void* y;
    float* h_out;
    void* saved;
    size_t saved_bytes;
    void* stream;
    // gradient
    const float* dh_out;
    void *dx, *dr, *di, *dz;
    float *dlam, *dh0;
    void* ws;
    size_t ws_bytes;
    bool save = false, grad = false;
    Strides st[5];                                   // x, r, i, z, dy
    GatedForm form;
};
int prepare_gated(GatedCall& c);

struct GatedStepCall {
    int64_t batch, dim;
    int dtype;
    const void *x, *r, *i, *z;
    const int64_t* strides;
    const float* lam;
    float rate;
    float* h;
    int64_t slots;
    const int32_t *slot_in, *slot_out;
    void* y;
    void* stream;
    int64_t st[4];
};
int prepare_gated_step(GatedStepCall& c);

// ---- the norm (norm.hip)
// Bytes of each channel's row that a workgroup takes, channel-major: the wider
// tile where six sweeps of its waves hold the channels
constexpr int kNormWide = 128, kNormNarrow = 64;
constexpr int64_t kNormMaxDim = 8192;
// workgroups that take the rows of a gradient in turn. The more there are, the more lines
// of dw there are to add up, and the fewer, the fewer loads are in flight; training steps with
// 1,024, 1,536 and 2,048 of them: bf16 8,194 x 1,536 36.4, 37.2 and 40.8 us, fp32 109.9, 113.5
// and 117.3, bf16 with a residual 8,194 x 1,536 51.9, 51.0 and 57.6, x 768 39.0, 35.3 and 41.4, x
// 384 27.6, 31.7 and 37.7: the best count goes with the bytes of a row, by up to 10 %.
constexpr int64_t kNormGroups = 1024;
// channel-major, or rows in 1, 4 or 16 waves: the channels a lane holds bound
// the row's length
enum NormForm { kNormColumn, kNormRow1, kNormRow4, kNormRow16 };
struct NormCall {
    int64_t batch, dim, L;
    int dtype;
    const void *x, *residual;                        // gradient: x is the sum s
    const void *dy, *dsum;
    const int64_t* strides;                          // as the caller gave them (may be NULL)
    const float* w;
    float eps;
    const int32_t* lengths;
    void *y, *sum;                                   // gradient: y is ds
    float* dw;
    void* ws;
    size_t ws_bytes;
    void* stream;
    bool grad = false;
    Strides st[3];                                   // x, residual; gradient: s, dy, dsum
    int tile;                                        // tokens
    NormForm form;
    int64_t parts;                                   // gradient: lines of sums for dw
    int64_t slab;                                    // batch rows of a launch
};
int prepare_norm(NormCall& c);

// ---- the vocabulary loss (vocab.hip)
constexpr int kVocabStage = 128;                     // bytes of k that a product takes at a time
// Tiles are 256 x 256 (wide) or 128 x 128; a product with few of them cuts its k
// into splits.
struct VocabPlan {
    int64_t dp;                                      // row length of packed operands
    bool pack_x, pack_w;
    bool wide;                                       // forward: the logits; gradient: both products
    int tiles;                                       // of the vocabulary, forward
    bool prob_wide;                                  // gradient: the logits
    int dx_splits, dw_splits;
    int64_t piece;                                   // vocabulary entries of a piece of the gradient
    int64_t pieces;
    size_t x, w, part, logit, P, part_dx, part_dw, sum, rest, bytes;    // offsets in the workspace, and its size
};
struct VocabCall {
    int64_t tokens, dim, vocab;
    int dtype;
    const void* x;
    int64_t ldx;
    const void* W;
    const void* target;
    int target_bits;
    float *loss, *lse;
    void* ws;
    size_t ws_bytes;
    void* stream;
    // gradient
    bool grad = false;
    const float *lse_in, *dloss;
    void *dx, *dW;
    int target64;
    VocabPlan plan;
};
VocabPlan vocab_plan(bool grad, int64_t tokens, int64_t dim, int64_t vocab, int dtype);
int prepare_vocab(VocabCall& c);

}  // namespace vs
