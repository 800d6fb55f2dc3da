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
    float *piece_h, *piece_sum;   // the pieces' end states from zero and sums of delta
    int64_t dim;
    int L, dstate, nblk;
    int pieces, piece_len;  // piece_len = sub * fine_len, a multiple of kTileTok
    int sub, fine_len;      // the carry launch cuts every piece into `sub` finer ones
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

// States past dstate have A = B = C = 0 and stay zero, so that they add nothing
// to a sum over the states, as long as all factors are finite: zero times an
// infinity is NaN. So where dstate < 16 a block of tokens whose delta u is not
// finite somewhere in the wave sets those states, and what they give to the
// sums, to zero. A delta that is not finite makes delta u so.
template <typename... F>
__device__ __forceinline__ bool any_non_finite(F... v) {
    return __ballot((... || !(__builtin_fabsf(v) < INFINITY))) != 0;
}

// A few rows of a tensor behind a buffer descriptor: 32-bit byte offsets from
// the first row; reads outside return zero, writes outside are dropped. The
// rows span at most 2^31 bytes (4 rows of at most 2^27 entries).
constexpr uint32_t kDropped = 0xfffffff0u;          // an offset past every descriptor
template <typename T>
using Raw = std::conditional_t<sizeof(T) == 2, uint16_t, uint32_t>;
template <typename T>
struct Rows {
    __amdgpu_buffer_rsrc_t rsrc;
    uint32_t stride;
    __device__ __forceinline__ Rows(const void* p, int64_t first, int64_t rows, int64_t d, int L) {
        const int64_t n = rows > 0 ? (rows - 1) * d + L : 0;
        rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(static_cast<const T*>(p) + (rows > 0 ? first : 0)), 0,
                                                 static_cast<int>(static_cast<uint32_t>(n * static_cast<int64_t>(sizeof(T)))),
                                                 0x00020000);
        stride = static_cast<uint32_t>(d);
    }
    __device__ __forceinline__ uint32_t at(uint32_t row, int t) const {
        return (row * stride + static_cast<uint32_t>(t)) * static_cast<uint32_t>(sizeof(T));
    }
    // `more` bytes further on, the same for the whole wave (a scalar; the range
    // check takes it in)
    __device__ __forceinline__ Raw<T> load(uint32_t off, int more = 0) const {
        if constexpr (sizeof(T) == 2) return __builtin_amdgcn_raw_buffer_load_b16(rsrc, static_cast<int>(off), more, 0);
        else return __builtin_amdgcn_raw_buffer_load_b32(rsrc, static_cast<int>(off), more, 0);
    }
    __device__ __forceinline__ void store(uint32_t off, float v, int more = 0) const {
        if constexpr (sizeof(T) == 2)
            __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, static_cast<__bf16>(v)), rsrc, static_cast<int>(off), more, 0);
        else
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), rsrc, static_cast<int>(off), more, 0);
    }
};

// Four consecutive entries of a row, kept as loaded until they are used.
// Rows start at any element: the accesses are only as aligned as one element.
template <typename T>
struct Four;
template <>
struct Four<float> {
    float v[4];
    __device__ __forceinline__ void load(const float* p) { __builtin_memcpy(v, p, sizeof(v)); }
    // entries first.. of a row of n; zeros past its end
    __device__ __forceinline__ void load_some(const float* p, int first, int n) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = first + i < n ? p[first + i] : 0.f;
    }
    __device__ __forceinline__ float get(int i) const { return v[i]; }
};
template <>
struct Four<uint16_t> {
    uint32_t v[2];
    __device__ __forceinline__ void load(const uint16_t* p) { __builtin_memcpy(v, p, sizeof(v)); }
    __device__ __forceinline__ void load_some(const uint16_t* p, int first, int n) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t lo = first + 2 * i < n ? p[first + 2 * i] : 0u;
            const uint32_t hi = first + 2 * i + 1 < n ? p[first + 2 * i + 1] : 0u;
            v[i] = lo | (hi << 16);
        }
    }
    __device__ __forceinline__ float get(int i) const {
        return __uint_as_float(i & 1 ? v[i / 2] & 0xffff0000u : v[i / 2] << 16);
    }
};
__device__ __forceinline__ void store_four(float* p, const float (&f)[4]) { __builtin_memcpy(p, f, sizeof(f)); }
__device__ __forceinline__ void store_four(uint16_t* p, const float (&f)[4]) {
    typedef __bf16 Vec4 __attribute__((ext_vector_type(4)));
    const Vec4 v = {static_cast<__bf16>(f[0]), static_cast<__bf16>(f[1]), static_cast<__bf16>(f[2]), static_cast<__bf16>(f[3])};
    __builtin_memcpy(p, &v, sizeof(v));
}

// eight of them
template <typename T>
struct Eight {
    Four<T> a, b;
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (sizeof(T) == 2) {
            uint32_t w[4];
            __builtin_memcpy(w, p, sizeof(w));
            a.v[0] = w[0]; a.v[1] = w[1]; b.v[0] = w[2]; b.v[1] = w[3];
        } else {
            a.load(p);
            b.load(p + 4);
        }
    }
    __device__ __forceinline__ void load_some(const T* p, int first, int n) {
        a.load_some(p, first, n);
        b.load_some(p, first + 4, n);
    }
    __device__ __forceinline__ float get(int i) const { return i < 4 ? a.get(i) : b.get(i - 4); }
};
__device__ __forceinline__ void store_eight(float* p, const float (&f)[8]) { __builtin_memcpy(p, f, sizeof(f)); }
__device__ __forceinline__ void store_eight(uint16_t* p, const float (&f)[8]) {
    typedef __bf16 Vec8 __attribute__((ext_vector_type(8)));
    const Vec8 v = {static_cast<__bf16>(f[0]), static_cast<__bf16>(f[1]), static_cast<__bf16>(f[2]), static_cast<__bf16>(f[3]),
                    static_cast<__bf16>(f[4]), static_cast<__bf16>(f[5]), static_cast<__bf16>(f[6]), static_cast<__bf16>(f[7])};
    __builtin_memcpy(p, &v, sizeof(v));
}

// The convolution's view of one lane's eight tokens t0..t0+7: the W - 1 entries
// of the row's line before them and the tokens themselves, zero past the
// row's length. x starts at token 0; win (or NULL) holds the W - 1 entries
// before it.
template <typename T, int W>
__device__ __forceinline__ void conv_line(const T* x, const T* win, int t0, int len, float (&f)[W + 7]) {
    constexpr int P = W - 1;
    if (t0 + 8 <= len) {
        Eight<T> e;
        e.load(x + t0);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[P + i] = e.get(i);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[P + i] = t0 + i < len ? ld(x, t0 + i) : 0.f;
    }
    if (t0 >= 8 && t0 <= len) {
        if constexpr (P <= 4) {
            Four<T> e;
            e.load(x + t0 - 4);
#pragma unroll
            for (int i = 0; i < P; ++i) f[i] = e.get(4 - P + i);
        } else {
            Eight<T> e;
            e.load(x + t0 - 8);
#pragma unroll
            for (int i = 0; i < P; ++i) f[i] = e.get(8 - P + i);
        }
    } else {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int t = t0 - P + i;
            f[i] = t >= 0 ? (t < len ? ld(x, t) : 0.f) : (win ? ld(win, t + P) : 0.f);
        }
    }
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
    template <int ROWS>
    __device__ __forceinline__ void store(float (&dst)[2][ROWS][kTilePad]) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            dst[i >> 1][(r0 + 8 * i) & 15][col] = ok[i] && in ? from_raw<T>(raw[i]) : 0.f;
    }
};

// exp(A sd), the factor of a whole piece's tokens, for a state (or adjoint) h
// that it multiplies. Each token's factor alone leaves a zero and an infinity
// as they are, but all together may underflow to zero or overflow, and zero
// times infinity is NaN: such an h passes through unchanged as long as every
// delta is finite, so that a cut row gives what an uncut one does.
__device__ __forceinline__ float piece_factor(float sd, float A2, float h) {
    constexpr int kZeroOrInf = 0x264, kFinite = 0x1f8;      // classes of v_cmp_class
    const float e = __builtin_amdgcn_exp2f(sd * A2);
    return __builtin_amdgcn_classf(h, kZeroOrInf) && __builtin_amdgcn_classf(sd, kFinite) ? 1.f : e;
}

// The state that the pieces before `piece` leave behind, folded into h: eight
// of the finer pieces' aggregates are in flight at a time; past the last, P = 1
// and h_loc = 0. N states a lane from n0 on, A2 their A log2(e).
template <int N>
__device__ __forceinline__ void fold_pieces(const ScanFwdArgs& a, int64_t b, int64_t d, int piece, int len, int n0,
                                            const float (&A2)[N], float (&h)[N]) {
    constexpr int kFold = 8;
    const int before = min(piece * a.sub, (len + a.fine_len - 1) / a.fine_len);
    const int64_t carry = static_cast<int64_t>(a.pieces - 1) * a.sub;
    for (int p0 = 0; p0 < before; p0 += kFold) {
        float sd[kFold], loc[kFold][N];
#pragma unroll
        for (int k = 0; k < kFold; ++k) {
            const size_t pr = static_cast<size_t>((b * carry + min(p0 + k, before - 1)) * a.dim + d);
            sd[k] = a.piece_sum[pr];
            const float* hp = a.piece_h + pr * a.dstate;
#pragma unroll
            for (int r = 0; r < N; ++r) loc[k][r] = hp[min(n0 + r, a.dstate - 1)];
        }
#pragma unroll
        for (int k = 0; k < kFold; ++k) {
            const bool on = p0 + k < before;
#pragma unroll
            for (int r = 0; r < N; ++r) {
                const float l = on && n0 + r < a.dstate ? loc[k][r] : 0.f;
                h[r] = fmaf(piece_factor(on ? sd[k] : 0.f, A2[r], h[r]), h[r], l);
            }
        }
    }
}

// ---- the wide form: four states a lane, a quad of lanes per channel
constexpr int kWideCh = vs::kCausalWideCh; // channels per workgroup
constexpr int kWidePad = 2 * kRowLanes + 4; // floats per token of the LDS tile

template <int Q>
__device__ __forceinline__ float quad_bcast(float v) { return dpp<Q * 0x55>(v); }

// four values of each lane summed over the quad: lane q returns sum of p_q
__device__ __forceinline__ float quad_transpose_sum(float p0, float p1, float p2, float p3, int lane) {
    const bool odd = (lane & 1) != 0, high = (lane & 2) != 0;
    const float a = p0 + dpp<0xb1>(p0), b = p1 + dpp<0xb1>(p1);      // quad_perm [1,0,3,2]
    const float c = p2 + dpp<0xb1>(p2), d = p3 + dpp<0xb1>(p3);
    const float ab = odd ? b : a, cd = odd ? d : c;
    const float s = ab + dpp<0x4e>(ab), t = cd + dpp<0x4e>(cd);      // quad_perm [2,3,0,1]
    return high ? t : s;
}

}  // namespace
