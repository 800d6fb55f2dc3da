// Device code shared by the causal scan's forward and gradient kernels: the
// argument records, row lengths, and the staging of B and C in LDS. Internal to
// libvimscan.so.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "vs_device.h"
#include "vs_internal.h"

namespace {

using vs::kRowLanes;
constexpr int kTileTok = vs::kTileTok;      // tokens of B and C staged at a time
// LDS row stride (floats) of a tile: with 36 the 16-byte reads of 16 lanes,
// one row each, fall on distinct banks
constexpr int kTilePad = kTileTok + 4;

struct ScanFwdArgs {
    const void *u, *delta, *z, *B, *C;
    vs::Strides su, sdl, sz, sB, sC;
    const float *A, *Dskip, *dt_bias, *h0;
    const int32_t* lengths;
    void* y;
    float* h_out;
    float *ckpt, *s;        // the saving forward: states at block starts, ungated output
    int64_t dim;
    int L, dstate, nblk;
};

__device__ __forceinline__ int row_length(const int32_t* lengths, int64_t b, int L) {
    if (!lengths) return L;
    const int v = __builtin_amdgcn_readfirstlane(lengths[b]);
    return v < 0 ? 0 : (v > L ? L : v);
}

// a barrier that orders LDS only
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// B and C of one 32-token tile into tile[which][state][token], fp32: 256
// threads, each one token column of four of the 32 rows (B's states, then
// C's). Rows past dstate and tokens past the row's length are zero.
template <typename T>
struct BcStage {
    const T* src[4];
    bool ok[4];
    int col, r0, len;
    uint32_t raw[4];
    bool in;

    template <typename Args>
    __device__ __forceinline__ BcStage(const Args& a, int64_t b, int tid, int len_) {
        col = tid & 31;
        r0 = tid >> 5;
        len = len_;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = (r0 + 8 * i) & 15;
            ok[i] = n < a.dstate;
            const int64_t nc = ok[i] ? n : 0;
            src[i] = i < 2 ? static_cast<const T*>(a.B) + b * a.sB.b + nc * a.sB.d
                           : static_cast<const T*>(a.C) + b * a.sC.b + nc * a.sC.d;
        }
    }
    // only for tiles that hold a token of the row (len >= 1)
    __device__ __forceinline__ void load(int tile) {
        const int t = tile * kTileTok + col;
        in = t < len;
        const int tc = in ? t : len - 1;
#pragma unroll
        for (int i = 0; i < 4; ++i) raw[i] = ld_raw(src[i], tc);
    }
    __device__ __forceinline__ void store(float (&dst)[2][kRowLanes][kTilePad]) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            dst[i >> 1][(r0 + 8 * i) & 15][col] = ok[i] && in ? from_raw<T>(raw[i]) : 0.f;
    }
};

}  // namespace
