// causal_grad.hip -- gfx950 kernels of the causal mixer's gradients: the short
// causal convolution's and the selective scan's (include/vimscan.h has the
// contract).
#include <hip/hip_runtime.h>

#include <cstdint>
#include <string>

#include "vimscan.h"
#include "vs_causal.h"
#include "vs_device.h"
#include "vs_internal.h"

namespace {

using vs::fail;
using vs::Strides;

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

// 1 / (1 + e^{-x}); e^{-x} = inf gives 0
__device__ __forceinline__ float sigmoid_f(float x) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-x * kLog2e));
}

// ------------------------------------------------------------ convolution
struct ConvGradArgs {
    const void *x, *dy, *window, *dwindow_out;
    const float *w, *bias;
    const int32_t* lengths;
    void *dx, *dwindow;
    float* part;            // [batch][segs][dim][W + 1]: dw, dbias of each segment
    Strides sx, sdy;
    int64_t dim;
    int L, segs, seg_len;
    int tw_log2;            // 1 << tw_log2 lanes along a row: 64, or fewer where a whole row fits
};

// A wave takes one segment of one row, 63 x 8 tokens at a time: every lane
// forms dpre of its eight consecutive tokens, and dx[t] = sum_j w[j] dpre[t +
// W-1 - j] takes up to W - 1 later ones from the lane above, so lane 63 only
// supplies its own and lane 0 of the next stride forms them again. Rows of up
// to 248 tokens share a wave (tw lanes each). Each lane sums dw and dbias of
// its tokens; the segment's sums go to its partial row. Bound by memory (x
// and dy read, dx written once) and, nearly as much, by VALU issue: 8 x 768 x
// 4,097 bf16 43 us, 3.7 TB/s, VALU active 86 %.
template <typename T, int W, bool SILU>
__global__ __launch_bounds__(kThreads) void causal_conv_grad_kernel(const ConvGradArgs a) {
    const int tw = 1 << a.tw_log2;
    const int last = tw - 1;                         // the lane that only supplies its dpre
    const int lane = threadIdx.x & last;
    const int64_t b = blockIdx.y;
    int64_t d0 = static_cast<int64_t>(blockIdx.x) * (kThreads >> a.tw_log2) + (threadIdx.x >> a.tw_log2);
    int seg = 0;
    if (a.segs > 1) {                                // uniform; a whole wave to a segment then
        const uint32_t item = blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        d0 = item / static_cast<uint32_t>(a.segs);
        seg = static_cast<int>(item - static_cast<uint32_t>(d0) * static_cast<uint32_t>(a.segs));
    }
    const bool real = d0 < a.dim;                    // lanes past the last row load, and write nothing
    const int64_t d = real ? d0 : a.dim - 1;
    const int len = row_length(a.lengths, b, a.L);
    const T* x = static_cast<const T*>(a.x) + b * a.sx.b + d * a.sx.d;
    const T* dy = static_cast<const T*>(a.dy) + b * a.sdy.b + d * a.sdy.d;
    const size_t wrow = static_cast<size_t>(b * a.dim + d) * (W - 1);
    const T* win = a.window ? static_cast<const T*>(a.window) + wrow : nullptr;
    const T* dwo = a.dwindow_out ? static_cast<const T*>(a.dwindow_out) + wrow : nullptr;
    T* dx = static_cast<T*>(a.dx) + static_cast<size_t>(b * a.dim + d) * a.L;
    float w[W];
#pragma unroll
    for (int j = 0; j < W; ++j) w[j] = a.w[d * W + j];
    const float bias = a.bias ? a.bias[d] : 0.f;
    float dw[W], db = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j] = 0.f;
    const int s0 = seg * a.seg_len, s1 = min(s0 + a.seg_len, a.L);
    for (int base = s0; base < s1; base += vs::kConvGradStep) {     // once where tw < 64
        const int t0 = base + lane * 8;
        float dpre[8 + W - 1];
#pragma unroll
        for (int i = 0; i < 8 + W - 1; ++i) dpre[i] = 0.f;
        if (t0 < len) {
            float f[W + 7];
            conv_line<T, W>(x, win, t0, len, f);
            Eight<T> g;
            if (t0 + 8 <= len) g.load(dy + t0);
            else g.load_some(dy, t0, len);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float pre = bias, v = g.get(i);
#pragma unroll
                for (int j = 0; j < W; ++j) pre = fmaf(w[j], f[i + j], pre);
                if (SILU) {
                    const float sg = sigmoid_f(pre);
                    v *= sg * fmaf(pre, 1.f - sg, 1.f);
                }
                dpre[i] = v;
            }
            if (t0 + 8 > len) {
#pragma unroll
                for (int i = 0; i < 8; ++i) dpre[i] = t0 + i < len ? dpre[i] : 0.f;
            }
            // padding stays out of dw (its dpre is zero, but the entries
            // before it may be infinite)
            auto sums = [&](int n) VS_INLINE {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    db += dpre[i];
#pragma unroll
                    for (int j = 0; j < W; ++j) dw[j] = i < n ? fmaf(dpre[i], f[i + j], dw[j]) : dw[j];
                }
            };
            if (lane < last) {
                if (t0 + 8 <= len) sums(8);
                else sums(len - t0);
            }
        }
#pragma unroll
        for (int k = 0; k < W - 1; ++k) dpre[8 + k] = __shfl_down(dpre[k], 1);
        if (real && lane < last && t0 < s1) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] = 0.f;
#pragma unroll
                for (int k = 0; k < W; ++k) v[i] = fmaf(w[W - 1 - k], dpre[i + k], v[i]);
            }
            if (t0 + 8 + W - 1 > len) {                 // the row's last tokens, and the padding
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int k = t0 + i + W - 1 - len; // the token's place in the outgoing window
                    if (dwo && k >= 0 && t0 + i < len) v[i] += ld(dwo, k);
                    if (t0 + i >= len) v[i] = 0.f;
                }
            }
            if (t0 + 8 <= a.L) {
                store_eight(dx + t0, v);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (t0 + i < a.L) st(dx, t0 + i, v[i]);
            }
        }
        // entry p of the incoming window feeds pre[p - j], j <= p
        if (a.dwindow && base == 0 && lane == 0 && real) {
#pragma unroll
            for (int p = 0; p < W - 1; ++p) {
                float v = 0.f;
#pragma unroll
                for (int j = 0; j <= p; ++j) v = fmaf(w[j], dpre[p - j], v);
                const int k = p - len;                  // short rows hand it on
                if (dwo && k >= 0) v += ld(dwo, k);
                st(static_cast<T*>(a.dwindow) + wrow, p, v);
            }
        }
    }
    float* part = a.part + ((static_cast<size_t>(b) * a.segs + seg) * a.dim + d) * (W + 1);
#pragma unroll
    for (int j = 0; j <= W; ++j) {
        float v = j < W ? dw[j < W ? j : 0] : db;
#pragma unroll
        for (int m = 32; m > 0; m >>= 1)
            if (m < tw) v += __shfl_xor(v, m);
        if (lane == 0 && real) part[j] = v;
    }
}

// dw and dbias: the segments' partial sums added in order, one thread per output
__global__ __launch_bounds__(kThreads) void conv_grad_reduce_kernel(const float* part, float* dw, float* dbias,
                                                                    int64_t n, int64_t parts, int width) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (i >= n) return;
    float s = 0.f;
#pragma unroll 8
    for (int64_t p = 0; p < parts; ++p) s += part[p * n + i];        // eight loads in flight
    const int64_t d = i / (width + 1);
    const int j = static_cast<int>(i % (width + 1));
    if (j < width) dw[d * width + j] = s;
    else dbias[d] = s;
}

// ------------------------------------------------------------------- scan
struct ScanGradArgs {
    const void *u, *delta, *z, *B, *C, *dy;
    Strides su, sdl, sz, sB, sC, sdy;
    const float *A, *Dskip, *dt_bias;
    const int32_t* lengths;
    const float *ckpt, *s, *dh_out;
    void *du, *ddelta, *dz;
    float *dh0;
    float* bc_part;         // [batch][group][nblk][512]: the sums of dB and dC over the group
    float* stat;            // [batch][piece][dim][dstate + 2]: dA, dD, dt_bias of each row
    float *piece_lam, *piece_sum;   // the pieces' adjoints from zero and sums of delta
    int64_t dim;
    int L, dstate, nblk;
    int pieces, piece_len;  // piece_len = sub * fine_len, a multiple of kTileTok
    int sub, fine_len;      // the carry launch cuts every piece into `sub` finer ones
};

// Lanes 0-31 return a[l] + a[l + 32]; lanes 32-63 return b[l - 32] + b[l].
__device__ __forceinline__ float swap32_sum(float a, float b) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// Of the four 16-lane rows, rows 0 and 2 return a's sum over themselves and
// the row above, rows 1 and 3 return b's sum over the row below and themselves.
__device__ __forceinline__ float swap16_sum(float a, float b) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Reverse mode, on the forward kernel's layout (a 16-lane row per channel,
// lane n = state n, 16 channels per workgroup), blocks of 16 tokens taken from
// the row's end. Per block the states are formed again from the one stored at
// its start, keeping h_t and e_t = exp(delta_t A); then the adjoint runs back,
//   lam_t = gy_t C_t + e_{t+1} lam_{t+1},  gy = dy silu(z),
// and with q_t = e_t lam_t h_{t-1}: dA += q delta, dC_t = gy h_t,
// dB_t = lam_t delta u; the sums over states W = sum lam B, V = sum q A are
// transpose reductions inside the row and give du = delta W + gy D and
// dDelta = V + u W. dB and dC are sums over channels: the wave's four rows are
// added by two rounds of lane swaps, the workgroup's waves in LDS, and the
// workgroups' chunks by bc_reduce_kernel, all in a fixed order.
//
// Where the rows are too few to fill the chip the sequence is cut into pieces
// as in the forward pass: the adjoint that leaves a piece at its start is P
// lam + lam_loc, lam the one that enters at its end, so a first launch
// (adjoint_carry_kernel) forms lam_loc and the sum of delta of every piece but
// the first, and each workgroup here folds those of the later pieces. That
// launch has a quarter of this one's workgroups per piece, so it cuts the
// pieces into finer ones.
//
// FULL: 16 states. Otherwise what the lanes past dstate give to W and V is set
// to zero (infinities times their zeros are NaN), in a variant of its own: a
// branch for the blocks that need it takes 139 registers against 127, three
// waves a SIMD instead of four.
//
// Bound by VALU issue: 391 instructions a wave for 16 tokens, 156 of them with
// a DPP operand, VALU active 86 %. 8 x 768 x 4,097 bf16,
// 16 states, in 2 pieces: 348 us here and 52 in the carry launch. The matrix
// cores could add up dB and dC over the channels, but a product with zeros for
// the channels past dim or another block's tokens turns an infinity there into
// NaN, and the lane swaps that it would save are an eighth of the instructions.
template <typename T, bool GATE, bool SOFTPLUS, bool FULL>
__global__ __launch_bounds__(kThreads) void causal_grad_kernel(const ScanGradArgs a) {
    // row kRowLanes stays zero: the B and C of lanes whose channel is past dim
    __shared__ __attribute__((aligned(16))) float tile[2][2][kRowLanes + 1][kTilePad];
    __shared__ float4 red[2][kWaves][2][64];
    const int tid = threadIdx.x;
    if (tid < 4 * kTilePad) tile[tid / (2 * kTilePad)][tid / kTilePad & 1][kRowLanes][tid % kTilePad] = 0.f;
    const int lane = tid & 63;
    const int wave = tid >> 6;
    const int n = lane & 15;
    uint32_t cg, bb;
    xcd_block(cg, bb);
    const int piece = static_cast<int>(bb % static_cast<uint32_t>(a.pieces));     // piece fastest
    const int64_t b = bb / static_cast<uint32_t>(a.pieces);
    const int64_t d0 = static_cast<int64_t>(cg) * vs::kCausalCh + (tid >> 4);
    const bool active = d0 < a.dim;
    const int64_t d = active ? d0 : a.dim - 1;
    const int L = a.L;
    const int len = row_length(a.lengths, b, L);
    const bool n_ok = n < a.dstate;
    const float An = n_ok ? a.A[d * a.dstate + n] : 0.f;
    const float A2 = An * kLog2e;
    const float Dk = a.Dskip ? a.Dskip[d] : 0.f;
    const float bias = a.dt_bias ? a.dt_bias[d] : 0.f;
    const size_t row = static_cast<size_t>(b * a.dim + d);
    // the wave's four rows of each tensor behind a buffer descriptor, as in
    // the forward kernel: no branches around memory in the loop
    const int64_t w0 = static_cast<int64_t>(cg) * vs::kCausalCh + __builtin_amdgcn_readfirstlane(wave) * 4;
    const int64_t wd = w0 < a.dim ? w0 : a.dim - 1;
    const int64_t wrows = w0 < a.dim ? (a.dim - w0 < 4 ? a.dim - w0 : 4) : 1;
    const uint32_t wr = static_cast<uint32_t>(d - wd);
    const Rows<T> u(a.u, b * a.su.b + wd * a.su.d, wrows, a.su.d, L), dl(a.delta, b * a.sdl.b + wd * a.sdl.d, wrows, a.sdl.d, L);
    const Rows<T> z(a.z, GATE ? b * a.sz.b + wd * a.sz.d : 0, GATE ? wrows : 0, a.sz.d, L);
    const Rows<T> dy(a.dy, b * a.sdy.b + wd * a.sdy.d, wrows, a.sdy.d, L);
    const int64_t orow = (b * a.dim + wd) * L;
    const Rows<T> du(a.du, orow, wrows, L, L), dd(a.ddelta, orow, wrows, L, L), dz(a.dz, orow, GATE ? wrows : 0, L, L);
    const Rows<float> s(a.s, orow, GATE ? wrows : 0, L, L);
    const int64_t crow = static_cast<int64_t>(a.nblk) * a.dstate;
    const Rows<float> ck(a.ckpt, (b * a.dim + wd) * crow, wrows, crow, static_cast<int>(crow));
    float* chunk = a.bc_part + (static_cast<size_t>(b) * gridDim.x + cg) * static_cast<size_t>(a.nblk) * 512;
    // this piece's tokens [s0, s1), of which [s0, e) are real
    const int s0 = piece * a.piece_len, s1 = min(s0 + a.piece_len, L), e = min(s1, len);
    const int t_real = active ? len : 0;             // tokens that this lane takes part in

    BcStage<T> stage(a, b, tid, len);
    const int blk0 = s0 / 16;
    const int nblk = e > s0 ? (e + 15) / 16 : blk0;  // blocks [blk0, nblk)
    const int tile0 = s0 / kTileTok;
    const int ntile = e > s0 ? (e + kTileTok - 1) / kTileTok : tile0;
    // Lanes of channels past dim count for nothing in the sums over channels:
    // they hold zeros from here on, B and C among them (their memory is channel
    // dim - 1's, and a zero factor in front of an infinity would be NaN)
    const bool holds = active && n_ok;
    const int bc_row = active ? n : kRowLanes;
    float lamE = a.dh_out && holds ? a.dh_out[row * a.dstate + n] : 0.f;
    // the adjoint that enters at the piece's end: those of the later pieces
    // that hold tokens, the last of them first, eight in flight at a time
    const int later = (piece + 1) * a.sub;           // the first finer piece after this one
    constexpr int kFold = 8;
    for (int p1 = (len + a.fine_len - 1) / a.fine_len - 1; p1 >= later; p1 -= kFold) {
        float sd[kFold], loc[kFold];
#pragma unroll
        for (int k = 0; k < kFold; ++k) {
            const int p = max(p1 - k, later);
            const size_t pr = static_cast<size_t>((b * ((a.pieces - 1) * a.sub) + p - a.sub) * a.dim + d);
            sd[k] = a.piece_sum[pr];
            loc[k] = a.piece_lam[pr * a.dstate + (n_ok ? n : 0)];
        }
#pragma unroll
        for (int k = 0; k < kFold; ++k) {
            const bool on = p1 - k >= later;
            lamE = fmaf(piece_factor(on ? sd[k] : 0.f, A2, lamE), lamE, on && holds ? loc[k] : 0.f);
        }
    }
    lamE = holds ? lamE : 0.f;                       // an infinite sum times A or lamE = 0
    // dA adds up all of a row's tokens in one lane: in fp64, a block's sum at a time
    double dA = 0.;
    float dD = 0.f, db = 0.f;
    struct Tok { Raw<T> u, d, z, g; uint32_t s, h; };
    // each lane's byte offset of token n of block 0 in every tensor; the block
    // comes in as a scalar
    constexpr int kEs = sizeof(T);
    const uint32_t ou = u.at(wr, n), od = dl.at(wr, n), og = dy.at(wr, n), oz = z.at(wr, n), os = s.at(wr, n);
    const uint32_t oh = holds ? ck.at(wr, n) : kDropped, oo = active ? du.at(wr, n) : kDropped;
    auto tok_load = [&](int blk, Tok& k) VS_INLINE {
        const int t0 = blk * 16 * kEs;
        k.u = u.load(ou, t0);
        k.d = dl.load(od, t0);
        k.g = dy.load(og, t0);
        if (GATE) {
            k.z = z.load(oz, t0);
            k.s = s.load(os, blk * 64);
        }
        k.h = ck.load(oh, blk * a.dstate * 4);
    };
    uint64_t again = 0;
    Tok nxt{};
    if (ntile > tile0) {
        stage.load(ntile - 1);
        tok_load(nblk - 1, nxt);
        stage.store(tile[(ntile - 1) & 1]);
    }
    lds_barrier();
    for (int blk = nblk - 1; blk >= blk0; --blk) {
        const int it = blk >> 1, half = blk & 1;
        // the tile below goes to the other buffer while this one is used
        const bool stages = it > tile0 && (half == 1 || blk == nblk - 1);
        if (stages) stage.load(it - 1);
        const Tok cur = nxt;
        tok_load(blk > blk0 ? blk - 1 : blk0, nxt);
        const int t = blk * 16 + n;
        const bool ok = t < t_real;
        const uint32_t out = t < s1 ? oo : kDropped;
        const int out0 = blk * 16 * kEs;
        const float x = from_raw<T>(cur.d) + bias;
        const float dlt = ok ? (SOFTPLUS ? softplus_f(x) : x) : 0.f;
        const float cu = ok ? from_raw<T>(cur.u) : 0.f;
        const float du_ = dlt * cu;
        const float g = from_raw<T>(cur.g);
        float gs = g;
        if (GATE) {
            const float zz = from_raw<T>(cur.z), sg = sigmoid_f(zz);
            gs = g * (zz * sg);
            const float v = g * __uint_as_float(cur.s) * sg * fmaf(zz, 1.f - sg, 1.f);
            dz.store(out, ok ? v : 0.f, out0);
        }
        gs = ok ? gs : 0.f;
        const float4* Bt = reinterpret_cast<const float4*>(&tile[it & 1][0][bc_row][half * 16]);
        const float4* Ct = reinterpret_cast<const float4*>(&tile[it & 1][1][bc_row][half * 16]);
        float Bv[16], Cv[16], hs[16], es[16], wv[16], vv[16], sbc[16];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float4 bq = Bt[q], cq = Ct[q];
            Bv[4 * q] = bq.x; Bv[4 * q + 1] = bq.y; Bv[4 * q + 2] = bq.z; Bv[4 * q + 3] = bq.w;
            Cv[4 * q] = cq.x; Cv[4 * q + 1] = cq.y; Cv[4 * q + 2] = cq.z; Cv[4 * q + 3] = cq.w;
        }
        const float h_in = __uint_as_float(cur.h);
        float h = h_in;
        Unroll<16>::run([&](auto ic) VS_INLINE {
            constexpr int i = decltype(ic)::value;
            es[i] = __builtin_amdgcn_exp2f(row_bcast<i>(dlt) * A2);
            h = fmaf(es[i], h, row_bcast<i>(du_) * Bv[i]);
            hs[i] = h;
        });
        // second copies of the broadcast sources, opaque to the compiler, give
        // every broadcast one use, which folds it into that use as a DPP operand
        float du_m = du_, gs_m = gs;
        asm volatile("" : "+v"(du_m), "+v"(gs_m));
        float dA_blk = 0.f, pb[8], pc[8];
        Unroll<16>::run([&](auto ic) VS_INLINE {
            constexpr int i = 15 - decltype(ic)::value;
            const float lam = row_bcast_fmac<i, i == 15>(lamE, gs, Cv[i]);
            lamE = lam * es[i];
            const float q = lamE * (i > 0 ? hs[i > 0 ? i - 1 : 0] : h_in);
            dA_blk = row_bcast_fmac<i, i == 15>(dA_blk, dlt, q);
            wv[i] = FULL || n_ok ? lam * Bv[i] : 0.f;
            vv[i] = FULL || n_ok ? q * An : 0.f;
            pb[i & 7] = row_bcast<i>(du_m) * lam;
            pc[i & 7] = row_bcast<i>(gs_m) * hs[i];
            // eight steps' products stand before their swaps: a swap that
            // follows its operands' writes at once would wait for them
            if (i % 8 == 0) {
#pragma unroll
                for (int k = 0; k < 8; ++k) sbc[i + k] = swap32_sum(pb[k], pc[k]);
            }
        });
        if (!FULL) lamE = n_ok ? lamE : 0.f;
        const float Rw = row_transpose_sum(wv, lane);
        const float Rv = row_transpose_sum(vv, lane);
        const float ddl = fmaf(cu, Rw, Rv);
        const float dx = ok ? (SOFTPLUS ? ddl * sigmoid_f(x) : ddl) : 0.f;
        du.store(out, ok ? fmaf(dlt, Rw, gs * Dk) : 0.f, out0);
        dd.store(out, dx, out0);
        db += dx;
        dD = fmaf(gs, cu, dD);
        // steps i and i + 8 of the block share a register: row 0 of a wave
        // then holds dB of step i, row 1 dB of i + 8, rows 2 and 3 dC
#pragma unroll
        for (int k = 0; k < 2; ++k)
            red[blk & 1][wave][k][lane] = make_float4(swap16_sum(sbc[4 * k], sbc[4 * k + 8]), swap16_sum(sbc[4 * k + 1], sbc[4 * k + 9]),
                                                      swap16_sum(sbc[4 * k + 2], sbc[4 * k + 10]), swap16_sum(sbc[4 * k + 3], sbc[4 * k + 11]));
        // the padding of a row's last block has delta = 0, but zero times an
        // infinite adjoint or state is NaN: those lanes' sum of that block is
        // formed again after the loop, where registers are free
        if (blk * 16 + 16 > len) {                           // uniform
            again = __ballot(!(__builtin_fabsf(dA_blk) < INFINITY));
            dA_blk = __builtin_fabsf(dA_blk) < INFINITY ? dA_blk : 0.f;
        }
        dA += static_cast<double>(dA_blk);
        if (stages) stage.store(tile[(it - 1) & 1]);
        lds_barrier();
        // a thread adds two of the waves' sums: the chunk is [i / 4][lane][i % 4]
        {
            const int k = wave >> 1, part = wave & 1;
            float2 v = reinterpret_cast<const float2*>(&red[blk & 1][0][k][lane])[part];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) {
                const float2 o = reinterpret_cast<const float2*>(&red[blk & 1][w][k][lane])[part];
                v.x += o.x; v.y += o.y;
            }
            *reinterpret_cast<float2*>(chunk + static_cast<size_t>(blk) * 512 + (k * 64 + lane) * 4 + part * 2) = v;
        }
    }
    if (again != 0) {                                // uniform
        const int t0 = (nblk - 1) * 16;
        const float x = from_raw<T>(dl.load(od, t0 * kEs)) + bias, zz = GATE ? from_raw<T>(z.load(oz, t0 * kEs)) : 0.f;
        const bool ok = t0 + n < t_real;
        const float dlt = ok ? (SOFTPLUS ? softplus_f(x) : x) : 0.f;
        const float du_ = ok ? dlt * from_raw<T>(u.load(ou, t0 * kEs)) : 0.f;
        float gs = from_raw<T>(dy.load(og, t0 * kEs));
        if (GATE) gs *= zz * sigmoid_f(zz);
        const int64_t nc = n_ok ? n : 0;
        const T* Bn = static_cast<const T*>(a.B) + b * a.sB.b + nc * a.sB.d + t0;
        const T* Cn = static_cast<const T*>(a.C) + b * a.sC.b + nc * a.sC.d + t0;
        float lam = a.dh_out && holds ? a.dh_out[row * a.dstate + n] : 0.f, sum = 0.f;
        for (int i = len - 1 - t0; i >= 0; --i) {
            // the state before token i, from the block's first one
            float h = __uint_as_float(ck.load(oh, (nblk - 1) * a.dstate * 4));
            for (int j = 0; j < i; ++j)
                h = fmaf(__builtin_amdgcn_exp2f(__shfl(dlt, j, 16) * A2), h, __shfl(du_, j, 16) * ld(Bn, j));
            const float dt = __shfl(dlt, i, 16);
            lam = fmaf(__shfl(gs, i, 16), ld(Cn, i), lam) * __builtin_amdgcn_exp2f(dt * A2);
            sum = fmaf(dt, lam * h, sum);
        }
        dA += (again >> lane) & 1 ? static_cast<double>(sum) : 0.;
    }
    float* stat = a.stat + (static_cast<size_t>(b * a.pieces + piece) * a.dim + d) * (a.dstate + 2);
    if (active && n_ok) {
        stat[n] = static_cast<float>(dA);
        if (a.dh0 && piece == 0) a.dh0[row * a.dstate + n] = lamE;
    }
    // dD and dt_bias: the row's lanes hold its tokens' shares
#pragma unroll
    for (int m = 8; m > 0; m >>= 1) {
        dD += __shfl_xor(dD, m);
        db += __shfl_xor(db, m);
    }
    if (active && n == 0) {
        stat[a.dstate] = dD;
        stat[a.dstate + 1] = db;
    }
    // the gradients of the padding
    for (int t = nblk * 16 + n; active && t < s1; t += 16) {
        du.store(du.at(wr, t), 0.f);
        dd.store(dd.at(wr, t), 0.f);
        if (GATE) dz.store(dz.at(wr, t), 0.f);
    }
}

// The adjoint that a piece's tokens leave at its start from zero at its end,
// and their sum of delta: lamE <- exp(delta_t A) (lamE + gy_t C_t) from the
// piece's last token to its first. The wide form of the forward scan (four
// states a lane, 64 channels a workgroup), without a read-out. Bound by VALU
// issue: half of 8 x 768 x 4,097 bf16 52 us.
template <typename T, bool GATE, bool SOFTPLUS>
__global__ __launch_bounds__(kThreads) void adjoint_carry_kernel(const ScanGradArgs a) {
    constexpr int kPad = kRowLanes + 4;
    __shared__ __attribute__((aligned(16))) float tile[2][kTileTok][kPad];
    const int tid = threadIdx.x;
    const int q = tid & 3;
    uint32_t cg, bb;
    xcd_block(cg, bb);
    const uint32_t np = static_cast<uint32_t>((a.pieces - 1) * a.sub);
    const int slot = static_cast<int>(bb % np);          // finer piece slot + sub
    const int64_t b = bb / np;
    const int64_t d0 = static_cast<int64_t>(cg) * kWideCh + (tid >> 2);
    const bool active = d0 < a.dim;
    const int64_t d = active ? d0 : a.dim - 1;
    const int len = row_length(a.lengths, b, a.L);
    const int s0 = (slot + a.sub) * a.fine_len, e = min(min(s0 + a.fine_len, a.L), len);
    if (e <= s0) return;                                 // no later piece is folded either
    float A2[4], lam[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int n = 4 * q + r;
        A2[r] = n < a.dstate ? a.A[d * a.dstate + n] * kLog2e : 0.f;
        lam[r] = 0.f;
    }
    const float bias = a.dt_bias ? a.dt_bias[d] : 0.f;
    const T* dl = static_cast<const T*>(a.delta) + b * a.sdl.b + d * a.sdl.d;
    const T* z = static_cast<const T*>(a.z) + b * a.sz.b + d * a.sz.d;
    const T* dy = static_cast<const T*>(a.dy) + b * a.sdy.b + d * a.sdy.d;
    // C: thread (state tid / 8, tokens 4k..4k+3) of the first 128
    const int sr = (tid >> 3) & 15, sk = (tid & 7) * 4;
    const bool s_ok = sr < a.dstate, stager = tid < 128;
    const T* ssrc = static_cast<const T*>(a.C) + b * a.sC.b + (s_ok ? sr : 0) * a.sC.d;
    Four<T> sraw, rd, rz, rg;
    auto stage_load = [&](int t0) VS_INLINE {
        const int t = t0 + sk;
        if (t + 4 <= len) sraw.load(ssrc + t);
        else sraw.load_some(ssrc, t, len);
    };
    auto stage_store = [&](float (&dst)[kTileTok][kPad]) VS_INLINE {
        if (stager)
#pragma unroll
            for (int i = 0; i < 4; ++i) dst[sk + i][sr] = s_ok ? sraw.get(i) : 0.f;
    };
    auto tok_load = [&](int t0) VS_INLINE {
        const int t = t0 + 4 * q;
        if (t0 + 16 <= len) {                            // uniform
            rd.load(dl + t);
            rg.load(dy + t);
            if (GATE) rz.load(z + t);
        } else {
            rd.load_some(dl, t, len);
            rg.load_some(dy, t, len);
            if (GATE) rz.load_some(z, t, len);
        }
    };
    const int ntile = (e - s0 + kTileTok - 1) / kTileTok;
    stage_load(s0 + (ntile - 1) * kTileTok);
    tok_load(s0 + (e - s0 - 1) / 16 * 16);
    stage_store(tile[(ntile - 1) & 1]);
    float sdl = 0.f;
    for (int it = ntile - 1; it >= 0; --it) {
        const int t_tile = s0 + it * kTileTok;
        lds_barrier();
        if (it > 0) stage_load(t_tile - kTileTok);
#pragma unroll
        for (int half = 1; half >= 0; --half) {
            const int t0 = t_tile + half * 16;
            if (t0 >= e) continue;                       // uniform
            float dlt[4], gs[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool ok = t0 + 4 * q + i < e;
                const float x = rd.get(i) + bias;
                dlt[i] = ok ? (SOFTPLUS ? softplus_f(x) : x) : 0.f;
                gs[i] = rg.get(i);
                if (GATE) {
                    const float zz = rz.get(i);
                    gs[i] *= zz * sigmoid_f(zz);
                }
                gs[i] = ok ? gs[i] : 0.f;
                sdl += dlt[i];
            }
            if (t0 > s0) tok_load(t0 - 16);
            Unroll<16>::run([&](auto ic) VS_INLINE {
                constexpr int i = 15 - decltype(ic)::value;
                // as in the forward form: keep the exponentials of later tokens from moving up
                if (i % 4 == 3) asm volatile("" : "+v"(dlt[0]), "+v"(dlt[1]), "+v"(dlt[2]), "+v"(dlt[3]), "+v"(lam[0]));
                const float4 Cv = *reinterpret_cast<const float4*>(&tile[it & 1][half * 16 + i][4 * q]);
                const float dt = quad_bcast<i / 4>(dlt[i % 4]), g = quad_bcast<i / 4>(gs[i % 4]);
                lam[0] = __builtin_amdgcn_exp2f(dt * A2[0]) * fmaf(g, Cv.x, lam[0]);
                lam[1] = __builtin_amdgcn_exp2f(dt * A2[1]) * fmaf(g, Cv.y, lam[1]);
                lam[2] = __builtin_amdgcn_exp2f(dt * A2[2]) * fmaf(g, Cv.z, lam[2]);
                lam[3] = __builtin_amdgcn_exp2f(dt * A2[3]) * fmaf(g, Cv.w, lam[3]);
            });
        }
        if (it > 0) stage_store(tile[(it - 1) & 1]);
    }
    sdl += dpp<0xb1>(sdl);
    sdl += dpp<0x4e>(sdl);
    if (active) {
        const size_t pr = static_cast<size_t>((b * static_cast<int64_t>(np) + slot) * a.dim + d);
        if (q == 0) a.piece_sum[pr] = sdl;
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (4 * q + r < a.dstate) a.piece_lam[pr * a.dstate + 4 * q + r] = lam[r];
    }
}

struct BcReduceArgs {
    const float *part, *stat;
    const int32_t* lengths;
    float *dB, *dC, *dA, *dD, *dbias;
    int64_t stat_rows, dim;  // stat_rows: batch rows times pieces
    int L, dstate, nblk, groups;
    int tok_wgs;            // workgroups over the tokens of a batch row
};

// dB and dC: the workgroups' chunks added in order; a thread takes four
// tokens of one state. The workgroups past tok_wgs of batch row 0 add dA, dD
// and dt_bias over the batch rows and their pieces, one thread per output.
// Bound by memory: 8 x 768 x 4,097, 203 MB of chunks in 46 us, 4.5 TB/s.
__global__ __launch_bounds__(kThreads) void bc_reduce_kernel(const BcReduceArgs a) {
    const int tid = threadIdx.x;
    const int64_t b = blockIdx.y;
    if (static_cast<int>(blockIdx.x) >= a.tok_wgs) {
        const int per = a.dstate + 2;
        const int64_t n = a.dim * per;
        const int64_t i = static_cast<int64_t>(blockIdx.x - a.tok_wgs) * kThreads + tid;
        if (b != 0 || i >= n) return;
        float s = 0.f;
#pragma unroll 8
        for (int64_t r = 0; r < a.stat_rows; ++r) s += a.stat[r * n + i];
        const int64_t d = i / per;
        const int k = static_cast<int>(i % per);
        if (k < a.dstate) a.dA[d * a.dstate + k] = s;
        else if (k == a.dstate) a.dD[d] = s;
        else a.dbias[d] = s;
        return;
    }
    // a block of 16 tokens takes 128 threads, thread (k, l) the four tokens
    // 4 k + 8 ((l / 16) % 2).. of dB (l < 32) or dC, state l % 16
    const int lane = tid & 63, n = lane & 15;
    const int blk = static_cast<int>(blockIdx.x) * 2 + (tid >> 7);
    const int t = blk * 16 + ((lane >> 4) & 1) * 8 + ((tid >> 6) & 1) * 4;
    if (t >= a.L || n >= a.dstate) return;
    const int len = row_length(a.lengths, b, a.L);
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (t < len) {
        const float* p = a.part + (static_cast<size_t>(b) * a.groups * a.nblk + blk) * 512 + (tid & 127) * 4;
#pragma unroll 4
        for (int g = 0; g < a.groups; ++g) {
            const float4 o = *reinterpret_cast<const float4*>(p + static_cast<size_t>(g) * a.nblk * 512);
            v[0] += o.x; v[1] += o.y; v[2] += o.z; v[3] += o.w;
        }
    }
    float* out = (lane >> 5 ? a.dC : a.dB) + (b * a.dstate + n) * static_cast<int64_t>(a.L) + t;
    // tokens of the block past the length: zero times an adjoint or a state
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = t + k < len ? v[k] : 0.f;
    if (t + 4 <= a.L) {
        store_four(out, v);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (t + k < a.L) out[k] = v[k];
    }
}

// -------------------------------------------------------------- launching
int launched() {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(VS_ERR_HIP, std::string("kernel launch: ") + hipGetErrorString(e));
    return VS_OK;
}

template <typename T>
int launch_conv_grad(const vs::ConvCall& c) {
    ConvGradArgs a{};
    a.x = c.x; a.dy = c.dy; a.window = c.window; a.dwindow_out = c.dwindow_out; a.w = c.w; a.bias = c.bias;
    a.lengths = c.lengths; a.dx = c.dx; a.dwindow = c.dwindow; a.part = static_cast<float*>(c.ws);
    a.sx = c.st[0]; a.sdy = c.st[1]; a.dim = c.dim; a.L = static_cast<int>(c.L);
    a.seg_len = static_cast<int>(vs::conv_grad_segment(c.batch, c.dim, c.L));
    a.segs = static_cast<int>((c.L + a.seg_len - 1) / a.seg_len);
    a.tw_log2 = 1;
    while (a.tw_log2 < 6 && ((1 << a.tw_log2) - 1) * vs::kConvVec < c.L) ++a.tw_log2;
    const int64_t per = kThreads >> a.tw_log2;
    const int64_t wgs = (c.dim * a.segs + per - 1) / per;
    if (wgs > vs::kMaxGroups) return fail(VS_ERR_UNSUPPORTED, "too many tokens and channels for one launch");
    const dim3 grid(static_cast<unsigned>(wgs), static_cast<unsigned>(c.batch));
    const hipStream_t st = static_cast<hipStream_t>(c.stream);
    switch (c.width) {
#define VS_CASE(w)                                                                                                       \
    case w:                                                                                                              \
        if (c.flags & VS_CONV_SILU)                                                                                      \
            hipLaunchKernelGGL((causal_conv_grad_kernel<T, w, true>), grid, dim3(kThreads), 0, st, a);                   \
        else                                                                                                             \
            hipLaunchKernelGGL((causal_conv_grad_kernel<T, w, false>), grid, dim3(kThreads), 0, st, a);                  \
        break;
    VS_CASE(2) VS_CASE(3) VS_CASE(4) VS_CASE(5) VS_CASE(6) VS_CASE(7) VS_CASE(8)
#undef VS_CASE
    }
    if (int rc = launched()) return rc;
    const int64_t n = c.dim * (c.width + 1);
    hipLaunchKernelGGL(conv_grad_reduce_kernel, dim3(static_cast<unsigned>((n + kThreads - 1) / kThreads)), dim3(kThreads), 0, st,
                       static_cast<const float*>(c.ws), c.dw, c.dbias, n, c.batch * a.segs, static_cast<int>(c.width));
    return launched();
}

template <typename T, bool FULL>
void launch_grad(const ScanGradArgs& a, dim3 grid, const vs::CausalCall& c) {
    const dim3 blk(kThreads);
    const hipStream_t st = static_cast<hipStream_t>(c.stream);
    const bool sp = c.flags & VS_FLAG_SOFTPLUS;
    if (c.z && sp) hipLaunchKernelGGL((causal_grad_kernel<T, true, true, FULL>), grid, blk, 0, st, a);
    else if (c.z) hipLaunchKernelGGL((causal_grad_kernel<T, true, false, FULL>), grid, blk, 0, st, a);
    else if (sp) hipLaunchKernelGGL((causal_grad_kernel<T, false, true, FULL>), grid, blk, 0, st, a);
    else hipLaunchKernelGGL((causal_grad_kernel<T, false, false, FULL>), grid, blk, 0, st, a);
}

template <typename T>
int launch_scan_grad(const vs::CausalCall& c) {
    size_t so[2], wo[4];
    vs::causal_saved_layout(c.batch, c.dim, c.dstate, c.L, so);
    vs::causal_grad_layout(c.batch, c.dim, c.dstate, c.L, wo);
    ScanGradArgs a{};
    a.u = c.u; a.delta = c.delta; a.z = c.z; a.B = c.B; a.C = c.C; a.dy = c.dy;
    a.su = c.st[0]; a.sdl = c.st[1]; a.sz = c.st[2]; a.sB = c.st[3]; a.sC = c.st[4]; a.sdy = c.st[5];
    a.A = c.A; a.Dskip = c.Dskip; a.dt_bias = c.dt_bias; a.lengths = c.lengths;
    a.ckpt = reinterpret_cast<const float*>(static_cast<const char*>(c.saved) + so[0]);
    a.s = reinterpret_cast<const float*>(static_cast<const char*>(c.saved) + so[1]);
    a.dh_out = c.dh_out; a.du = c.du; a.ddelta = c.ddelta; a.dz = c.dz; a.dh0 = c.dh0;
    a.bc_part = reinterpret_cast<float*>(static_cast<char*>(c.ws) + wo[0]);
    a.stat = reinterpret_cast<float*>(static_cast<char*>(c.ws) + wo[1]);
    a.dim = c.dim; a.L = static_cast<int>(c.L); a.dstate = static_cast<int>(c.dstate);
    a.nblk = static_cast<int>((c.L + vs::kBlockTok - 1) / vs::kBlockTok);
    const unsigned groups = static_cast<unsigned>((c.dim + vs::kCausalCh - 1) / vs::kCausalCh);
    const vs::ScanCut cut = vs::causal_grad_cut(c.batch, c.dim, c.L);
    a.pieces = cut.pieces;
    a.sub = cut.sub;
    a.fine_len = static_cast<int>(cut.fine_tiles * kTileTok);
    a.piece_len = a.fine_len * a.sub;
    const dim3 grid(groups, static_cast<unsigned>(c.batch * a.pieces)), blk(kThreads);
    const hipStream_t st = static_cast<hipStream_t>(c.stream);
    const bool sp = c.flags & VS_FLAG_SOFTPLUS;
    if (a.pieces > 1) {
        a.piece_lam = reinterpret_cast<float*>(static_cast<char*>(c.ws) + wo[2]);
        a.piece_sum = reinterpret_cast<float*>(static_cast<char*>(c.ws) + wo[3]);
        const dim3 cgrid(static_cast<unsigned>((c.dim + kWideCh - 1) / kWideCh), static_cast<unsigned>(c.batch * (a.pieces - 1) * a.sub));
        if (c.z && sp) hipLaunchKernelGGL((adjoint_carry_kernel<T, true, true>), cgrid, blk, 0, st, a);
        else if (c.z) hipLaunchKernelGGL((adjoint_carry_kernel<T, true, false>), cgrid, blk, 0, st, a);
        else if (sp) hipLaunchKernelGGL((adjoint_carry_kernel<T, false, true>), cgrid, blk, 0, st, a);
        else hipLaunchKernelGGL((adjoint_carry_kernel<T, false, false>), cgrid, blk, 0, st, a);
        if (int rc = launched()) return rc;
    }
    if (c.dstate == kRowLanes) launch_grad<T, true>(a, grid, c);
    else launch_grad<T, false>(a, grid, c);
    if (int rc = launched()) return rc;
    BcReduceArgs r{};
    r.part = a.bc_part; r.stat = a.stat; r.lengths = c.lengths; r.dB = c.dB; r.dC = c.dC; r.dA = c.dA; r.dD = c.dD;
    r.dbias = c.dbias; r.stat_rows = c.batch * a.pieces; r.dim = c.dim; r.L = a.L; r.dstate = a.dstate; r.nblk = a.nblk;
    r.groups = static_cast<int>(groups);
    r.tok_wgs = (a.L + 31) / 32;
    const int64_t stat_wgs = (c.dim * (c.dstate + 2) + kThreads - 1) / kThreads;
    hipLaunchKernelGGL(bc_reduce_kernel, dim3(static_cast<unsigned>(r.tok_wgs + stat_wgs), static_cast<unsigned>(c.batch)),
                       blk, 0, st, r);
    return launched();
}

}  // namespace

// ---------------------------------------------------------------- C ABI
extern "C" {

int s6_causal_conv_grad(int64_t batch, int64_t dim, int64_t width, int64_t seqlen, int dtype,
                        int flags, const void* x, const void* dy, const int64_t* strides,
                        const float* w, const float* bias, const void* window,
                        const int32_t* lengths, const void* dwindow_out, void* dx, float* dw,
                        float* dbias, void* dwindow, void* workspace, size_t workspace_bytes,
                        void* stream) {
    vs::ConvCall c{};
    c.batch = batch; c.dim = dim; c.width = width; c.L = seqlen; c.dtype = dtype; c.flags = flags;
    c.x = x; c.dy = dy; c.strides = strides; c.w = w; c.bias = bias; c.window = window; c.lengths = lengths;
    c.grad = true; c.dwindow_out = dwindow_out; c.dx = dx; c.dw = dw; c.dbias = dbias; c.dwindow = dwindow;
    c.ws = workspace; c.ws_bytes = workspace_bytes; c.stream = stream;
    if (int rc = vs::prepare_conv(c)) return rc;
    return dtype == VS_BF16 ? launch_conv_grad<uint16_t>(c) : launch_conv_grad<float>(c);
}

int s6_causal_scan_grad(int64_t batch, int64_t dim, int64_t dstate, int64_t seqlen, int dtype,
                        int flags, const void* u, const void* delta, const void* z, const void* B,
                        const void* C, const void* dy, const int64_t* strides, const float* A,
                        const float* Dskip, const float* dt_bias, const int32_t* lengths,
                        const void* saved, size_t saved_bytes, const float* dh_out, void* du,
                        void* ddelta, void* dz, float* dB, float* dC, float* dA, float* dD,
                        float* ddt_bias, float* dh0, void* workspace, size_t workspace_bytes,
                        void* stream) {
    vs::CausalCall c{};
    c.batch = batch; c.dim = dim; c.dstate = dstate; c.L = seqlen; c.dtype = dtype; c.flags = flags;
    c.u = u; c.delta = delta; c.z = z; c.B = B; c.C = C; c.dy = dy; c.strides = strides; c.A = A;
    c.Dskip = Dskip; c.dt_bias = dt_bias; c.lengths = lengths; c.saved = const_cast<void*>(saved);
    c.saved_bytes = saved_bytes; c.dh_out = dh_out; c.du = du; c.ddelta = ddelta; c.dz = dz; c.dB = dB;
    c.dC = dC; c.dA = dA; c.dD = dD; c.dbias = ddt_bias; c.dh0 = dh0; c.ws = workspace;
    c.ws_bytes = workspace_bytes; c.stream = stream; c.grad = true;
    if (int rc = vs::prepare_causal(c)) return rc;
    return dtype == VS_BF16 ? launch_scan_grad<uint16_t>(c) : launch_scan_grad<float>(c);
}

}  // extern "C"
