// Device helpers shared by the kernel translation units: dtype conversion,
// lane moves inside a 16-lane DPP row, the scalar math of the scan and the
// workgroup order over the chip's XCDs. Internal to libvimscan.so.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

namespace {

// The kernels' per-block steps are lambdas over register arrays (token
// sets, tiles' raw words); one left out of line would put those arrays in
// scratch memory.
#define VS_INLINE __attribute__((always_inline))

// ---------------------------------------------------------------- dtype I/O
__device__ __forceinline__ float ld(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float ld(const uint16_t* p, int64_t i) {
    return __uint_as_float(static_cast<uint32_t>(p[i]) << 16);
}
// Raw loads keep the loaded bits untouched so that the conversion (and the
// wait for the load) happens where the value is used, not where it is loaded.
__device__ __forceinline__ uint32_t ld_raw(const float* p, int64_t i) { return __float_as_uint(p[i]); }
__device__ __forceinline__ uint32_t ld_raw(const uint16_t* p, int64_t i) { return p[i]; }
template <typename T>
__device__ __forceinline__ float from_raw(uint32_t r) {
    if constexpr (sizeof(T) == 2) return __uint_as_float(r << 16);
    else return __uint_as_float(r);
}
__device__ __forceinline__ void st(float* p, int64_t i, float v) { p[i] = v; }
// fp32 -> bf16, round to nearest even (v_cvt_pk_bf16_f32 on gfx950).
__device__ __forceinline__ void st(uint16_t* p, int64_t i, float v) {
    p[i] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}

// ------------------------------------------------------------- lane moves
// DPP move whose result feeds a VALU op; the compiler folds it into the
// consumer (v_mul_f32_dpp etc.) when both operands are VGPRs.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xf, 0xf, true));
}
// value of lane I of this 16-lane row, in every lane of the row (row_newbcast)
template <int I>
__device__ __forceinline__ float row_bcast(float v) { return dpp<0x150 + I>(v); }
// acc + row_bcast<I>(v) * w as one v_fmac_f32_dpp. The compiler does not fold
// a DPP move into fmac (whose accumulator is tied to its result), so the
// instruction is written out, and the compiler does not see its DPP read: a
// DPP source needs two wait states after its VALU write. With FIRST the asm
// opens with s_nop 1, for the first of a chain of calls that read one source;
// the later calls of the chain read the same value, written before the
// first. tests/test_dpp_hazards.py checks the rule on every path of the
// built code object.
template <int I, bool FIRST>
__device__ __forceinline__ float row_bcast_fmac(float acc, float v, float w) {
    static_assert(I >= 0 && I < 16, "a lane of the row");
    if constexpr (FIRST)
        asm("s_nop 1\n\tv_fmac_f32_dpp %0, %1, %2 row_newbcast:%3 row_mask:0xf bank_mask:0xf"
            : "+v"(acc) : "v"(v), "v"(w), "i"(I));
    else
        asm("v_fmac_f32_dpp %0, %1, %2 row_newbcast:%3 row_mask:0xf bank_mask:0xf"
            : "+v"(acc) : "v"(v), "v"(w), "i"(I));
    return acc;
}

// Transpose-reduce across the 16 lanes of a row: lane n holds c[i] = its
// state's share of token i's read-out; on return lane j holds the sum over
// the row's lanes of c[j]. Each halving stage pairs lane j with lane j^m. The
// two cross-bank stages (m = 8, 4) write the kept half of each bank (4-lane
// group) with bank-masked DPP adds, 2 per pair, in one asm block: its
// leading s_nop gives the two wait states a DPP read needs after the VALU
// write of its source, and inside the block every DPP source was written at
// least 7 instructions earlier; the trailing s_nop covers the DPP reads that
// follow the block. The in-bank stages (m = 2, 1) add both halves and select.
#define VS_ADD8(T, C, K) \
    "v_add_f32_dpp %[" #T "], %[" #C "], %[" #C "] row_ror:8 row_mask:0xf bank_mask:" K "\n\t"
#define VS_ADD4(V, T, R, K) \
    "v_add_f32_dpp %[" #V "], %[" #T "], %[" #T "] " R " row_mask:0xf bank_mask:" K "\n\t"
__device__ __forceinline__ float row_transpose_sum(const float (&c)[16], int lane) {
    float t0, t1, t2, t3, t4, t5, t6, t7, v0, v1, v2, v3;
    asm("s_nop 1\n\t"
        VS_ADD8(t0, c0, "0x3") VS_ADD8(t0, c8, "0xc")
        VS_ADD8(t1, c1, "0x3") VS_ADD8(t1, c9, "0xc")
        VS_ADD8(t2, c2, "0x3") VS_ADD8(t2, c10, "0xc")
        VS_ADD8(t3, c3, "0x3") VS_ADD8(t3, c11, "0xc")
        VS_ADD8(t4, c4, "0x3") VS_ADD8(t4, c12, "0xc")
        VS_ADD8(t5, c5, "0x3") VS_ADD8(t5, c13, "0xc")
        VS_ADD8(t6, c6, "0x3") VS_ADD8(t6, c14, "0xc")
        VS_ADD8(t7, c7, "0x3") VS_ADD8(t7, c15, "0xc")
        VS_ADD4(v0, t0, "row_ror:12", "0x5") VS_ADD4(v0, t4, "row_ror:4", "0xa")
        VS_ADD4(v1, t1, "row_ror:12", "0x5") VS_ADD4(v1, t5, "row_ror:4", "0xa")
        VS_ADD4(v2, t2, "row_ror:12", "0x5") VS_ADD4(v2, t6, "row_ror:4", "0xa")
        VS_ADD4(v3, t3, "row_ror:12", "0x5") VS_ADD4(v3, t7, "row_ror:4", "0xa")
        "s_nop 1"
        : [t0] "=&v"(t0), [t1] "=&v"(t1), [t2] "=&v"(t2), [t3] "=&v"(t3), [t4] "=&v"(t4),
          [t5] "=&v"(t5), [t6] "=&v"(t6), [t7] "=&v"(t7), [v0] "=&v"(v0), [v1] "=&v"(v1),
          [v2] "=&v"(v2), [v3] "=&v"(v3)
        : [c0] "v"(c[0]), [c1] "v"(c[1]), [c2] "v"(c[2]), [c3] "v"(c[3]), [c4] "v"(c[4]),
          [c5] "v"(c[5]), [c6] "v"(c[6]), [c7] "v"(c[7]), [c8] "v"(c[8]), [c9] "v"(c[9]),
          [c10] "v"(c[10]), [c11] "v"(c[11]), [c12] "v"(c[12]), [c13] "v"(c[13]),
          [c14] "v"(c[14]), [c15] "v"(c[15]));
    const bool b1 = (lane & 2) != 0, b0 = (lane & 1) != 0;
    const float s0 = v0 + dpp<0x4e>(v0), s2 = v2 + dpp<0x4e>(v2);   // quad_perm [2,3,0,1]
    const float s1 = v1 + dpp<0x4e>(v1), s3 = v3 + dpp<0x4e>(v3);
    const float w0 = b1 ? s2 : s0, w1 = b1 ? s3 : s1;
    const float r0 = w0 + dpp<0xb1>(w0), r1 = w1 + dpp<0xb1>(w1);   // quad_perm [1,0,3,2]
    return b0 ? r1 : r0;
}

// ---------------------------------------------------------------- math
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// softplus(x) = max(x, 0) + ln(1 + w), w = e^{-|x|} in (0, 1], with the
// hardware exp2 and log2. Forming v = 1 + w rounds w by r = (v - 1) - w
// (exact in fp32: v - 1 is exact for v in [1, 2], and so is the difference of
// the two nearby values), and ln(v) = ln(1 + w) + r / v. Subtracting r
// leaves an error of |r| w / v <= 2^-24 w, i.e. 2^-24 relative to ln(1 + w).
__device__ __forceinline__ float softplus_f(float x) {
    const float w = __builtin_amdgcn_exp2f(-__builtin_fabsf(x) * kLog2e);
    const float v = 1.f + w;
    const float r = (v - 1.f) - w;
    return fmaf(kLn2, __builtin_amdgcn_logf(v), fmaxf(x, 0.f) - r);
}
// silu(z) = z * sigmoid(z) = z / (1 + e^{-z})
__device__ __forceinline__ float silu_f(float z) {
    return z * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-z * kLog2e));
}

// Workgroups are dispatched to the 8 XCDs (each with its own L2) round-robin
// by linear id. Renumber them so that every XCD receives one contiguous range
// of (batch, channel-group) ids: the workgroups that share a batch's B and C
// then mostly share one L2. A bijection on [0, G): XCD x gets the linear ids
// x, x+8, ..., which map to the range starting at x*(G/8) + min(x, G%8).
constexpr uint32_t kXcds = 8;
__device__ __forceinline__ void xcd_block(uint32_t& cg, uint32_t& bb) {
    const uint32_t G = gridDim.x * gridDim.y;
    const uint32_t lin = blockIdx.x + blockIdx.y * gridDim.x;
    const uint32_t x = lin % kXcds, k = lin / kXcds;
    const uint32_t q = G / kXcds, r = G % kXcds;
    const uint32_t v = x * q + (x < r ? x : r) + k;
    cg = v % gridDim.x;
    bb = v / gridDim.x;
}

template <int I>
struct Unroll {
    template <typename F>
    __device__ __forceinline__ static void run(F&& f) {
        Unroll<I - 1>::run(f);
        f(std::integral_constant<int, I - 1>{});
    }
};
template <>
struct Unroll<0> {
    template <typename F>
    __device__ __forceinline__ static void run(F&&) {}
};

}  // namespace
