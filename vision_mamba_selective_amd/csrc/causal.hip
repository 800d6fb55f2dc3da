// causal.hip -- gfx950 kernels of the causal mixer's forward pass: the short
// causal convolution and the selective scan of prompts, and their single-token
// forms on pools of states (include/vimscan.h has the contract).
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

// ------------------------------------------------------------ convolution
struct ConvArgs {
    const void *x, *window;
    const float *w, *bias;
    const int32_t* lengths;
    void *y, *window_out;
    Strides sx;
    int64_t dim;
    int L;
    int tw_log2;            // 1 << tw_log2 threads along the tokens of a row, at most kThreads
    int segs;               // workgroups along a row
};

// y = silu(bias + sum_j w[j] line[t + j]): a lane takes eight consecutive
// tokens of a row (one or two 16-byte loads, and a second load of the W - 1
// entries before them, which the caches hold); short rows share a workgroup.
// Each entry of x comes from HBM once. 8 x 768 x 4,097 bf16 28 us, 3.7 TB/s read
// and written (a plain copy reaches 5.1), VALU active 61 %. Padding goes
// through the straddling lane's entry-by-entry path: rows of 2,049 to 4,097
// tokens take 32 us for 92 MB.
template <typename T, int W, bool SILU>
__global__ __launch_bounds__(kThreads) void causal_conv_kernel(const ConvArgs a) {
    const int tid = threadIdx.x;
    const int tw = 1 << a.tw_log2, rows = kThreads >> a.tw_log2;
    const int64_t b = blockIdx.y;
    const unsigned group = blockIdx.x / static_cast<unsigned>(a.segs);
    const int seg = static_cast<int>(blockIdx.x - group * static_cast<unsigned>(a.segs));
    const int j = tid & (tw - 1);
    const int64_t d = static_cast<int64_t>(group) * rows + (tid >> a.tw_log2);
    if (d >= a.dim) return;
    const int len = row_length(a.lengths, b, a.L);
    const T* x = static_cast<const T*>(a.x) + b * a.sx.b + d * a.sx.d;
    const T* win = a.window ? static_cast<const T*>(a.window) + (b * a.dim + d) * (W - 1) : nullptr;
    float w[W];
#pragma unroll
    for (int j = 0; j < W; ++j) w[j] = a.w[d * W + j];
    const float bias = a.bias ? a.bias[d] : 0.f;
    T* y = static_cast<T*>(a.y) + (b * a.dim + d) * a.L;
    const int t0 = (seg * tw + j) * vs::kConvVec;
    if (t0 < a.L) {
        float f[W + 7], v[8];
        conv_line<T, W>(x, win, t0, len, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] = bias;
#pragma unroll
            for (int j = 0; j < W; ++j) v[i] = fmaf(w[j], f[i + j], v[i]);
            if (SILU) v[i] = silu_f(v[i]);
        }
        if (t0 + 8 <= len) {
            store_eight(y + t0, v);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (t0 + i < a.L) st(y, t0 + i, t0 + i < len ? v[i] : 0.f);
        }
    }
    // the row's last W - 1 line entries, unchanged in their type
    if (a.window_out && seg == 0) {
        T* wo = static_cast<T*>(a.window_out) + (b * a.dim + d) * (W - 1);
        for (int k = j; k < W - 1; k += tw) {
            const int p = len + k;
            wo[k] = p >= W - 1 ? x[p - (W - 1)] : (win ? win[p] : static_cast<T>(0));
        }
    }
}

struct ConvStepArgs {
    const void* x;
    const float *w, *bias;
    void* window;
    const int32_t *slot_in, *slot_out;
    void* y;
    int64_t sx, slots, dim;
    int silu;
};

// One token of each row, a thread per channel. Bound by the launch at small
// sizes (64 x 1,536 bf16 3 us), then by memory: 515 x 1,536 6 us, 13 MB.
template <typename T, int W>
__global__ __launch_bounds__(kThreads) void conv_step_kernel(const ConvStepArgs a) {
    const int64_t d = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    const int64_t b = blockIdx.y;
    if (d >= a.dim) return;
    T* y = static_cast<T*>(a.y) + b * a.dim + d;
    const int64_t si = a.slot_in ? a.slot_in[b] : b, so = a.slot_out ? a.slot_out[b] : b;
    if (si < 0 || so < 0 || si >= a.slots || so >= a.slots) {
        st(y, 0, 0.f);
        return;
    }
    const T* in = static_cast<const T*>(a.window) + (si * a.dim + d) * (W - 1);
    T line[W];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) line[j] = in[j];
    line[W - 1] = static_cast<const T*>(a.x)[b * a.sx + d];
    float v = a.bias ? a.bias[d] : 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) v = fmaf(a.w[d * W + j], ld(line, j), v);
    T* out = static_cast<T*>(a.window) + (so * a.dim + d) * (W - 1);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) out[j] = line[j + 1];
    st(y, 0, a.silu ? silu_f(v) : v);
}

// ------------------------------------------------------------------- scan
// One recurrence per 16-lane DPP row, lane n = state n; a workgroup holds 16
// channels of one batch row. Tokens go in blocks of 16: lane j of a row loads
// token j, forms its delta and delta u once, and the row broadcasts them; the
// read-out C . h of the 16 tokens is a transpose reduction inside the row.
// B and C of 32 tokens (a tile) are staged in LDS for the workgroup's
// channels, double-buffered, one barrier per tile. Padding (t >= length)
// enters as delta = 0 and zero u, B: it leaves the state as it is whatever
// the padded memory holds. Where that evens out the load of the compute units
// the sequence is cut into a few pieces, as described for the wide form below.
// VALU issue takes most of the time: 165 instructions a wave for 16 tokens, 62
// of them with a DPP operand and 20 transcendental, which cost two to four
// times a plain one's slot: 626 cycles, 100 us of the 169 that the saving form
// takes for 8 x 768 x 4,097 bf16, 16 states, in 2 pieces (carry launch 49), VALU
// active 76 %; without saving both together 190. With rows of 2,049 to 4,097
// tokens, a quarter less work, the launch takes 147 us: an XCD holds one batch
// row there, and the longest row's is the last to end.
template <typename T, bool GATE, bool SOFTPLUS, bool SAVE>
__global__ __launch_bounds__(kThreads) void causal_scan_kernel(const ScanFwdArgs a) {
    __shared__ __attribute__((aligned(16))) float tile[2][2][kRowLanes][kTilePad];
    const int tid = threadIdx.x;
    const int lane = tid & 63;
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
    const float A2 = n_ok ? a.A[d * a.dstate + n] * kLog2e : 0.f;
    const float Dk = a.Dskip ? a.Dskip[d] : 0.f;
    const float bias = a.dt_bias ? a.dt_bias[d] : 0.f;
    const size_t row = static_cast<size_t>(b * a.dim + d);
    float* ck = SAVE ? a.ckpt + row * static_cast<size_t>(a.nblk) * a.dstate : nullptr;

    // The wave's four rows of a tensor are read and written through a buffer
    // descriptor: a lane holds one running byte offset per tensor, reads past
    // the rows return zero and writes there are dropped, so nothing in the
    // loop branches around memory.
    const int64_t w0 = static_cast<int64_t>(cg) * vs::kCausalCh + __builtin_amdgcn_readfirstlane(tid >> 6) * 4;
    const int64_t wd = w0 < a.dim ? w0 : a.dim - 1;
    const int64_t wrows = w0 < a.dim ? (a.dim - w0 < 4 ? a.dim - w0 : 4) : 1;
    const uint32_t wr = static_cast<uint32_t>(d - wd);
    const Rows<T> u(a.u, b * a.su.b + wd * a.su.d, wrows, a.su.d, L), dl(a.delta, b * a.sdl.b + wd * a.sdl.d, wrows, a.sdl.d, L);
    const Rows<T> z(a.z, GATE ? b * a.sz.b + wd * a.sz.d : 0, GATE ? wrows : 0, a.sz.d, L);
    const int64_t orow = (b * a.dim + wd) * L;
    const Rows<T> y(a.y, orow, wrows, L, L);
    const Rows<float> s(a.s, SAVE ? orow : 0, SAVE && GATE ? wrows : 0, L, L);
    // this piece's tokens [s0, s1), of which [s0, e) are real
    const int s0 = piece * a.piece_len, s1 = min(s0 + a.piece_len, L), e = min(s1, len);
    uint32_t ou = u.at(wr, s0 + n), od = dl.at(wr, s0 + n), oz = z.at(wr, s0 + n);
    uint32_t oy = y.at(wr, s0 + n), os = s.at(wr, s0 + n);
    const int t_lim = active ? s1 : 0;          // tokens whose outputs this lane may write

    BcStage<T> stage(a, b, tid, len);
    float h = a.h0 && n_ok ? a.h0[row * a.dstate + n] : 0.f;
    const int tile0 = s0 / kTileTok;
    const int ntile = e > s0 ? (e + kTileTok - 1) / kTileTok : tile0;      // tiles [tile0, ntile)
    Raw<T> ru[2], rd[2], rz[2];
    auto tok_load = [&]() VS_INLINE {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            ru[k] = u.load(ou + k * 16 * sizeof(T));
            rd[k] = dl.load(od + k * 16 * sizeof(T));
            if (GATE) rz[k] = z.load(oz + k * 16 * sizeof(T));
        }
        ou += kTileTok * sizeof(T);
        od += kTileTok * sizeof(T);
        oz += kTileTok * sizeof(T);
    };
    if (ntile > tile0) {
        stage.load(tile0);
        tok_load();
        stage.store(tile[tile0 & 1]);
    }
    if (piece > 0) {
        const float A1[1] = {A2};
        float h1[1] = {h};
        fold_pieces<1>(a, b, d, piece, len, n, A1, h1);
        h = n_ok ? h1[0] : 0.f;
    }
    for (int it = tile0; it < ntile; ++it) {
        lds_barrier();
        if (it + 1 < ntile) stage.load(it + 1);
        Raw<T> cu_[2], cd_[2], cz_[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) { cu_[k] = ru[k]; cd_[k] = rd[k]; cz_[k] = rz[k]; }
        tok_load();                             // past the row: zero, or another row's, unused
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int t = it * kTileTok + half * 16 + n;
            if (half == 1 && it * kTileTok + 16 >= len) {          // uniform: nothing but padding
                y.store(t < t_lim ? oy + 16 * static_cast<uint32_t>(sizeof(T)) : kDropped, 0.f);
                break;
            }
            const bool ok = t < len;
            const float x = from_raw<T>(cd_[half]) + bias;
            const float dlt = ok ? (SOFTPLUS ? softplus_f(x) : x) : 0.f;
            const float cu = ok ? from_raw<T>(cu_[half]) : 0.f;
            const float du = dlt * cu;
            if (SAVE && active && n_ok && it * 2 + half < a.nblk)
                ck[static_cast<size_t>(it * 2 + half) * a.dstate + n] = h;
            const float4* Bt = reinterpret_cast<const float4*>(&tile[it & 1][0][n][half * 16]);
            const float4* Ct = reinterpret_cast<const float4*>(&tile[it & 1][1][n][half * 16]);
            float Bv[16], Cv[16], c[16];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float4 bq = Bt[q], cq = Ct[q];
                Bv[4 * q] = bq.x; Bv[4 * q + 1] = bq.y; Bv[4 * q + 2] = bq.z; Bv[4 * q + 3] = bq.w;
                Cv[4 * q] = cq.x; Cv[4 * q + 1] = cq.y; Cv[4 * q + 2] = cq.z; Cv[4 * q + 3] = cq.w;
            }
            Unroll<16>::run([&](auto ic) VS_INLINE {
                constexpr int i = decltype(ic)::value;
                const float e = __builtin_amdgcn_exp2f(row_bcast<i>(dlt) * A2);
                h = fmaf(e, h, row_bcast<i>(du) * Bv[i]);
                c[i] = h * Cv[i];
            });
            if (a.dstate < kRowLanes && any_non_finite(du)) {      // uniform
#pragma unroll
                for (int i = 0; i < 16; ++i) c[i] = n_ok ? c[i] : 0.f;
                h = n_ok ? h : 0.f;
            }
            const float sum = fmaf(Dk, cu, row_transpose_sum(c, lane));
            float v = sum;
            if (GATE) v *= silu_f(from_raw<T>(cz_[half]));
            const bool wr_ok = t < t_lim;
            if (SAVE && GATE) s.store(wr_ok ? os + half * 16 * 4 : kDropped, sum);
            y.store(wr_ok ? oy + half * 16 * static_cast<uint32_t>(sizeof(T)) : kDropped, ok ? v : 0.f);
        }
        oy += kTileTok * sizeof(T);
        if (SAVE) os += kTileTok * 4;
        if (it + 1 < ntile) stage.store(tile[(it + 1) & 1]);
    }
    // the piece with the row's last token (the first one for an empty row) has its final state
    if (a.h_out && active && n_ok && (len > 0 ? s0 < len && len <= s1 : piece == 0)) a.h_out[row * a.dstate + n] = h;
    // the outputs of the padding past the last tile
    for (int t = ntile * kTileTok + n; t < t_lim; t += 16) {
        y.store(oy, 0.f);
        oy += 16 * sizeof(T);
    }
}

// The same scan with four states in a lane: a wave holds 16 channels, lane q
// of a channel's quad states 4q..4q+3, a workgroup 64 channels of one piece
// of one batch row's tokens. Lane q loads the block's tokens 4q..4q+3 (one
// wide load per tensor), forms their delta and delta u, and the quad
// broadcasts them into the multiplications as DPP operands; the read-out sums
// four states in the lane and finishes in the quad (9 instructions for four
// tokens). B and C of 32 tokens stand in LDS as [token][B | C].
//
// Against one state per lane this takes about a fifth fewer instruction slots
// per state update, but a quarter of the waves: it is the form for sequences
// cut into pieces. A piece's effect on the state is h -> P h + h_loc with P =
// exp(A sum of delta), so a first launch (CARRY) scans every piece but the
// last from zero, with no read-out, and stores h_loc and the sum of delta;
// the second folds those of the earlier pieces into its own starting state
// and scans its tokens in full. Bound by VALU issue like the narrow form: 1 x
// 1,536 x 16,385 bf16 in 21 pieces 140 us and 97 us for the carry, VALU active
// 76 and 72 %, 212 us together where they follow at once (uncut, the narrow
// form takes 570). Two other layouts were slower there: one channel a lane with
// 16 states in registers (375 us: two waves a SIMD), and the broadcasts as moves
// in front of plain multiplications (6 % more than as DPP operands).
template <typename T, bool GATE, bool SOFTPLUS, bool SAVE, bool CARRY>
__global__ __launch_bounds__(kThreads) void causal_scan4_kernel(const ScanFwdArgs a) {
    __shared__ __attribute__((aligned(16))) float tile[2][kTileTok][kWidePad];
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int q = lane & 3;
    uint32_t cg, bb;
    xcd_block(cg, bb);
    // grid.y enumerates (batch, piece), piece fastest; the carry launch leaves the last piece out
    const uint32_t np = static_cast<uint32_t>(CARRY ? (a.pieces - 1) * a.sub : a.pieces);
    const int piece = static_cast<int>(bb % np);
    const int64_t b = bb / np;
    const int64_t d0 = static_cast<int64_t>(cg) * kWideCh + (tid >> 2);
    const bool active = d0 < a.dim;
    const int64_t d = active ? d0 : a.dim - 1;
    const int L = a.L;
    const int len = row_length(a.lengths, b, L);
    // this piece's tokens [s0, s1) and, of those, the real ones [s0, e)
    const int plen = CARRY ? a.fine_len : a.piece_len;
    const int s0 = min(piece * plen, L), s1 = min(s0 + plen, L), e = min(s1, len);
    const size_t row = static_cast<size_t>(b * a.dim + d);
    float A2[4], h[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int n = 4 * q + r;
        A2[r] = n < a.dstate ? a.A[d * a.dstate + n] * kLog2e : 0.f;
        h[r] = 0.f;
    }
    const float Dk = !CARRY && a.Dskip ? a.Dskip[d] : 0.f;
    const float bias = a.dt_bias ? a.dt_bias[d] : 0.f;
    const T* u = static_cast<const T*>(a.u) + b * a.su.b + d * a.su.d;
    const T* dl = static_cast<const T*>(a.delta) + b * a.sdl.b + d * a.sdl.d;
    const T* z = static_cast<const T*>(a.z) + b * a.sz.b + d * a.sz.d;
    T* y = static_cast<T*>(a.y) + row * static_cast<size_t>(L);
    float* s = SAVE ? a.s + row * static_cast<size_t>(L) : nullptr;
    float* ck = SAVE ? a.ckpt + row * static_cast<size_t>(a.nblk) * a.dstate : nullptr;

    // ---- staging: thread (row r of B | C, tokens 4k..4k+3)
    const int sr = tid >> 3, sk = (tid & 7) * 4;
    const bool s_ok = (sr & 15) < a.dstate;
    const int64_t sn = s_ok ? sr & 15 : 0;
    const T* ssrc = sr < 16 ? static_cast<const T*>(a.B) + b * a.sB.b + sn * a.sB.d
                            : static_cast<const T*>(a.C) + b * a.sC.b + sn * a.sC.d;
    Four<T> sraw;
    auto stage_load = [&](int t0) VS_INLINE {
        const int t = t0 + sk;
        if (t + 4 <= len) sraw.load(ssrc + t);
        else sraw.load_some(ssrc, t, len);
    };
    auto stage_store = [&](float (&dst)[kTileTok][kWidePad]) VS_INLINE {
#pragma unroll
        for (int i = 0; i < 4; ++i) dst[sk + i][sr] = s_ok ? sraw.get(i) : 0.f;
    };
    Four<T> ru, rd, rz;
    auto tok_load = [&](int t0) VS_INLINE {
        const int t = t0 + 4 * q;
        if (t0 + 16 <= len) {                                  // uniform
            ru.load(u + t);
            rd.load(dl + t);
            if (GATE && !CARRY) rz.load(z + t);
        } else {
            ru.load_some(u, t, len);
            rd.load_some(dl, t, len);
            if (GATE && !CARRY) rz.load_some(z, t, len);
        }
    };
    const int ntile = e > s0 ? (e - s0 + kTileTok - 1) / kTileTok : 0;
    if (ntile > 0) {
        stage_load(s0);
        tok_load(s0);
        stage_store(tile[0]);
    }
    // ---- the state that the earlier pieces leave
    if (!CARRY) {
        if (a.h0) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (4 * q + r < a.dstate) h[r] = a.h0[row * a.dstate + 4 * q + r];
        }
        fold_pieces<4>(a, b, d, piece, len, 4 * q, A2, h);
#pragma unroll
        for (int r = 0; r < 4; ++r) h[r] = 4 * q + r < a.dstate ? h[r] : 0.f;      // an infinite sum times A = 0
    }
    float sdl = 0.f;
    for (int it = 0; it < ntile; ++it) {
        const int t_tile = s0 + it * kTileTok;
        lds_barrier();
        const bool more = it + 1 < ntile;
        if (more) stage_load(t_tile + kTileTok);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int t0 = t_tile + half * 16;
            if (t0 >= e) break;                                // uniform
            float dlt[4], du[4], uu[4], zz[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = rd.get(i) + bias;
                dlt[i] = SOFTPLUS ? softplus_f(x) : x;
                uu[i] = ru.get(i);
                zz[i] = GATE && !CARRY ? rz.get(i) : 0.f;
            }
            if (t0 + 16 > e) {                                 // uniform: the row's last block
#pragma unroll
                for (int i = 0; i < 4; ++i) dlt[i] = t0 + 4 * q + i < e ? dlt[i] : 0.f;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                du[i] = dlt[i] * uu[i];
                if (CARRY) sdl += dlt[i];
            }
            if (t0 + 16 < e) tok_load(t0 + 16);
            if (SAVE && active) {
                float* c = ck + static_cast<size_t>(t0 >> 4) * a.dstate + 4 * q;
                if ((a.dstate & 3) == 0) {                     // uniform; rows of 16-byte multiples
                    if (4 * q < a.dstate) __builtin_memcpy(c, h, sizeof(h));
                } else {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (4 * q + r < a.dstate) c[r] = h[r];
                }
            }
            float p[16];
            // clean: states past dstate are set back to zero at every token
            auto tokens = [&](auto clean) VS_INLINE { Unroll<16>::run([&](auto ic) VS_INLINE {
                constexpr int i = decltype(ic)::value;
                // the exponentials do not wait for the states: left free, all
                // 64 of a block are formed at its start and held in
                // registers, so each four tokens' steps are tied to the state
                // that the tokens before them left
                if (i % 4 == 0) asm volatile("" : "+v"(dlt[0]), "+v"(dlt[1]), "+v"(dlt[2]), "+v"(dlt[3]), "+v"(h[0]));
                const float* row_bc = tile[it & 1][half * 16 + i];
                const float4 Bv = *reinterpret_cast<const float4*>(row_bc + 4 * q);
                const float dt = quad_bcast<i / 4>(dlt[i % 4]), dx = quad_bcast<i / 4>(du[i % 4]);
                h[0] = fmaf(__builtin_amdgcn_exp2f(dt * A2[0]), h[0], dx * Bv.x);
                h[1] = fmaf(__builtin_amdgcn_exp2f(dt * A2[1]), h[1], dx * Bv.y);
                h[2] = fmaf(__builtin_amdgcn_exp2f(dt * A2[2]), h[2], dx * Bv.z);
                h[3] = fmaf(__builtin_amdgcn_exp2f(dt * A2[3]), h[3], dx * Bv.w);
                if (decltype(clean)::value) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) h[r] = 4 * q + r < a.dstate ? h[r] : 0.f;
                }
                if (!CARRY) {
                    const float4 Cv = *reinterpret_cast<const float4*>(row_bc + kRowLanes + 4 * q);
                    p[i] = fmaf(h[3], Cv.w, fmaf(h[2], Cv.z, fmaf(h[1], Cv.y, h[0] * Cv.x)));
                }
            }); };
            // the carry launch has no read-out: what its unused states hold goes nowhere
            if (!CARRY && a.dstate < kRowLanes && any_non_finite(du[0], du[1], du[2], du[3])) tokens(std::true_type{});
            else tokens(std::false_type{});
            if (!CARRY) {
                float v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[i] = fmaf(Dk, uu[i], quad_transpose_sum(p[i], p[4 + i], p[8 + i], p[12 + i], lane));
                const int t = t0 + 4 * q;
                if (active) {
                    if (SAVE && GATE) {
                        if (t0 + 16 <= e) store_four(s + t, v);
                        else
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (t + i < e) s[t + i] = v[i];
                    }
                    if (GATE) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) v[i] *= silu_f(zz[i]);
                    }
                    if (t0 + 16 <= e) store_four(y + t, v);
                    else
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (t + i < s1) st(y, t + i, t + i < e ? v[i] : 0.f);
                }
            }
        }
        if (more) stage_store(tile[(it + 1) & 1]);
    }
    if (CARRY) {
        sdl += dpp<0xb1>(sdl);
        sdl += dpp<0x4e>(sdl);
        if (active) {
            // [batch][finer piece][dim]: sums of delta, and end states [...][dstate]
            const size_t pr = static_cast<size_t>((b * static_cast<int64_t>(np) + piece) * a.dim + d);
            if (q == 0) a.piece_sum[pr] = sdl;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (4 * q + r < a.dstate) a.piece_h[pr * a.dstate + 4 * q + r] = h[r];
        }
        return;
    }
    // the piece with the row's last token (the first one for an empty row) has its final state
    if (a.h_out && active && (len > 0 ? s0 < len && len <= s1 : piece == 0)) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (4 * q + r < a.dstate) a.h_out[row * a.dstate + 4 * q + r] = h[r];
    }
    // outputs of the padding past the last block: lanes along the tokens of
    // the wave's 16 channels
    const int zf = e > s0 ? s0 + (e - s0 + 15) / 16 * 16 : s0;
    if (zf < s1) {
        const int64_t w0 = static_cast<int64_t>(cg) * kWideCh + (tid >> 6) * 16;
        for (int c = 0; c < 16 && w0 + c < a.dim; ++c) {
            T* yr = static_cast<T*>(a.y) + static_cast<size_t>(b * a.dim + w0 + c) * L;
            for (int t = zf + lane; t < s1; t += 64) st(yr, t, 0.f);
        }
    }
}

// one token of each row on the pool: four lanes per channel, lane q of a quad
// holds states 4q..4q+3
struct ScanStepArgs {
    const void *u, *delta, *z, *B, *C;
    const float *A, *Dskip, *dt_bias;
    float* h;
    const int32_t *slot_in, *slot_out;
    void* y;
    int64_t st[5], slots, dim, batch;
    int dstate;
};

// ROWS batch rows per thread keep several rows' states in flight and read A
// once for them; it is 4 where that still leaves every compute unit 4
// workgroups (515 x 1,536 bf16 26 us with 4, 35 with 1; 64 x 1,536 6.9 with 4,
// 6.1 with 1). VEC: dstate a multiple of 4 (16-byte accesses of the states).
// Bound by memory: each state is read and written once, 4.1 TB/s at 515 x 1,536.
template <typename T, bool GATE, bool SOFTPLUS, bool VEC, int ROWS>
__global__ __launch_bounds__(kThreads) void scan_step_kernel(const ScanStepArgs a) {
    const int64_t d = static_cast<int64_t>(blockIdx.x) * (kThreads / 4) + (threadIdx.x >> 2);
    const int q = threadIdx.x & 3;
    if (d >= a.dim) return;                          // whole quads
    float A2[4];
    const float* A = a.A + d * a.dstate + 4 * q;
#pragma unroll
    for (int r = 0; r < 4; ++r) A2[r] = 4 * q + r < a.dstate ? A[r] * kLog2e : 0.f;
    const float bias = a.dt_bias ? a.dt_bias[d] : 0.f;
    const float Dk = a.Dskip ? a.Dskip[d] : 0.f;
    // states past dstate: read as zero, never written
    const bool lane_ok = 4 * q < a.dstate;
    int64_t so[ROWS];
    bool live[ROWS];
    float h[ROWS][4], Bv[ROWS][4], Cv[ROWS][4], u[ROWS], x[ROWS], z[ROWS];
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
        const int64_t b0 = static_cast<int64_t>(blockIdx.y) * ROWS + k;
        const bool row = b0 < a.batch;
        const int64_t b = row ? b0 : a.batch - 1;
        const int64_t si = a.slot_in ? a.slot_in[b] : b;
        so[k] = a.slot_out ? a.slot_out[b] : b;
        live[k] = row && si >= 0 && si < a.slots && so[k] >= 0 && so[k] < a.slots;
        const float* hi = a.h + ((live[k] ? si : 0) * a.dim + d) * a.dstate + 4 * q;
        const T* B = static_cast<const T*>(a.B) + b * a.st[3] + 4 * q;
        const T* C = static_cast<const T*>(a.C) + b * a.st[4] + 4 * q;
        if (VEC) {
            Four<T> fb, fc;
#pragma unroll
            for (int r = 0; r < 4; ++r) h[k][r] = Bv[k][r] = Cv[k][r] = 0.f;
            if (lane_ok) {
                __builtin_memcpy(h[k], hi, sizeof(h[k]));
                fb.load(B);
                fc.load(C);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    Bv[k][r] = fb.get(r);
                    Cv[k][r] = fc.get(r);
                }
            }
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const bool ok = 4 * q + r < a.dstate;
                h[k][r] = ok ? hi[r] : 0.f;
                Bv[k][r] = ok ? ld(B, r) : 0.f;
                Cv[k][r] = ok ? ld(C, r) : 0.f;
            }
        }
        u[k] = ld(static_cast<const T*>(a.u), b * a.st[0] + d);
        x[k] = ld(static_cast<const T*>(a.delta), b * a.st[1] + d) + bias;
        z[k] = GATE ? ld(static_cast<const T*>(a.z), b * a.st[2] + d) : 0.f;
    }
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
        const int64_t b = static_cast<int64_t>(blockIdx.y) * ROWS + k;
        const float dlt = SOFTPLUS ? softplus_f(x[k]) : x[k];
        const float du = dlt * u[k];
        float sum = 0.f;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float v = fmaf(__builtin_amdgcn_exp2f(dlt * A2[r]), h[k][r], du * Bv[k][r]);
            h[k][r] = (VEC ? lane_ok : 4 * q + r < a.dstate) ? v : 0.f;     // an infinite du is NaN times zero
            sum = fmaf(h[k][r], Cv[k][r], sum);
        }
        sum += dpp<0xb1>(sum);                       // quad_perm [1,0,3,2]
        sum += dpp<0x4e>(sum);                       // quad_perm [2,3,0,1]
        if (live[k]) {
            float* ho = a.h + (so[k] * a.dim + d) * a.dstate + 4 * q;
            if (VEC) {
                if (lane_ok) __builtin_memcpy(ho, h[k], sizeof(h[k]));
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (4 * q + r < a.dstate) ho[r] = h[k][r];
            }
        }
        float v = fmaf(Dk, u[k], sum);
        if (GATE) v *= silu_f(z[k]);
        if (q == 0 && b < a.batch) st(static_cast<T*>(a.y) + b * a.dim + d, 0, live[k] ? v : 0.f);
    }
}

// -------------------------------------------------------------- launching
int launched() {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(VS_ERR_HIP, std::string("kernel launch: ") + hipGetErrorString(e));
    return VS_OK;
}

template <typename F>
int with_width(int64_t width, F&& f) {
    switch (width) {
    case 2: f(std::integral_constant<int, 2>{}); break;
    case 3: f(std::integral_constant<int, 3>{}); break;
    case 4: f(std::integral_constant<int, 4>{}); break;
    case 5: f(std::integral_constant<int, 5>{}); break;
    case 6: f(std::integral_constant<int, 6>{}); break;
    case 7: f(std::integral_constant<int, 7>{}); break;
    default: f(std::integral_constant<int, 8>{}); break;
    }
    return launched();
}

template <typename T>
int launch_conv(const vs::ConvCall& c) {
    ConvArgs a{};
    a.x = c.x; a.window = c.window; a.w = c.w; a.bias = c.bias; a.lengths = c.lengths;
    a.y = c.y; a.window_out = c.window_out; a.sx = c.st[0]; a.dim = c.dim;
    a.L = static_cast<int>(c.L);
    while ((1 << a.tw_log2) < kThreads && (vs::kConvVec << a.tw_log2) < c.L) ++a.tw_log2;
    const int64_t per = vs::kConvVec << a.tw_log2;
    a.segs = static_cast<int>((c.L + per - 1) / per);
    const int64_t rows = kThreads >> a.tw_log2, groups = (c.dim + rows - 1) / rows * a.segs;
    if (groups > vs::kMaxGroups) return fail(VS_ERR_UNSUPPORTED, "too many tokens and channels for one launch");
    const dim3 grid(static_cast<unsigned>(groups), static_cast<unsigned>(c.batch));
    return with_width(c.width, [&](auto w) {
        constexpr int W = decltype(w)::value;
        const hipStream_t st = static_cast<hipStream_t>(c.stream);
        if (c.flags & VS_CONV_SILU) hipLaunchKernelGGL((causal_conv_kernel<T, W, true>), grid, dim3(kThreads), 0, st, a);
        else hipLaunchKernelGGL((causal_conv_kernel<T, W, false>), grid, dim3(kThreads), 0, st, a);
    });
}

template <typename T>
int launch_conv_step(const vs::StepCall& c) {
    ConvStepArgs a{};
    a.x = c.u; a.w = c.A; a.bias = c.dt_bias; a.window = c.pool; a.slot_in = c.slot_in; a.slot_out = c.slot_out;
    a.y = c.y; a.sx = c.st[0]; a.slots = c.slots; a.dim = c.dim; a.silu = c.flags & VS_CONV_SILU;
    const dim3 grid(static_cast<unsigned>((c.dim + kThreads - 1) / kThreads), static_cast<unsigned>(c.batch));
    return with_width(c.inner, [&](auto w) {
        hipLaunchKernelGGL((conv_step_kernel<T, decltype(w)::value>), grid, dim3(kThreads), 0,
                           static_cast<hipStream_t>(c.stream), a);
    });
}

template <typename T, bool VEC, int ROWS>
void launch_step(const ScanStepArgs& a, dim3 grid, const vs::StepCall& c) {
    const dim3 blk(kThreads);
    const hipStream_t st = static_cast<hipStream_t>(c.stream);
    const bool sp = c.flags & VS_FLAG_SOFTPLUS;
    if (c.z && sp) hipLaunchKernelGGL((scan_step_kernel<T, true, true, VEC, ROWS>), grid, blk, 0, st, a);
    else if (c.z) hipLaunchKernelGGL((scan_step_kernel<T, true, false, VEC, ROWS>), grid, blk, 0, st, a);
    else if (sp) hipLaunchKernelGGL((scan_step_kernel<T, false, true, VEC, ROWS>), grid, blk, 0, st, a);
    else hipLaunchKernelGGL((scan_step_kernel<T, false, false, VEC, ROWS>), grid, blk, 0, st, a);
}

template <typename T>
int launch_scan_step(const vs::StepCall& c) {
    ScanStepArgs a{};
    a.u = c.u; a.delta = c.delta; a.z = c.z; a.B = c.B; a.C = c.C; a.A = c.A; a.Dskip = c.Dskip; a.dt_bias = c.dt_bias;
    a.h = static_cast<float*>(c.pool); a.slot_in = c.slot_in; a.slot_out = c.slot_out; a.y = c.y;
    for (int i = 0; i < 5; ++i) a.st[i] = c.st[i];
    a.slots = c.slots; a.dim = c.dim; a.dstate = static_cast<int>(c.inner);
    a.batch = c.batch;
    const int64_t groups = (c.dim + kThreads / 4 - 1) / (kThreads / 4);
    const bool vec = c.inner % 4 == 0 && vs::aligned(c.pool, 16);
    if (groups * ((c.batch + 3) / 4) >= 4 * vs::kNumCUs) {
        const dim3 grid(static_cast<unsigned>(groups), static_cast<unsigned>((c.batch + 3) / 4));
        if (vec) launch_step<T, true, 4>(a, grid, c);
        else launch_step<T, false, 4>(a, grid, c);
    } else {
        const dim3 grid(static_cast<unsigned>(groups), static_cast<unsigned>(c.batch));
        if (vec) launch_step<T, true, 1>(a, grid, c);
        else launch_step<T, false, 1>(a, grid, c);
    }
    return launched();
}

template <typename T, bool SAVE>
int launch_scan(const vs::CausalCall& c) {
    ScanFwdArgs a{};
    a.u = c.u; a.delta = c.delta; a.z = c.z; a.B = c.B; a.C = c.C;
    a.su = c.st[0]; a.sdl = c.st[1]; a.sz = c.st[2]; a.sB = c.st[3]; a.sC = c.st[4];
    a.A = c.A; a.Dskip = c.Dskip; a.dt_bias = c.dt_bias; a.h0 = c.h0; a.lengths = c.lengths;
    a.y = c.y; a.h_out = c.h_out; a.dim = c.dim; a.L = static_cast<int>(c.L);
    a.dstate = static_cast<int>(c.dstate);
    a.nblk = static_cast<int>((c.L + vs::kBlockTok - 1) / vs::kBlockTok);
    if (SAVE) {
        size_t offs[2];
        vs::causal_saved_layout(c.batch, c.dim, c.dstate, c.L, offs);
        a.ckpt = reinterpret_cast<float*>(static_cast<char*>(c.saved) + offs[0]);
        a.s = reinterpret_cast<float*>(static_cast<char*>(c.saved) + offs[1]);
    }
    const dim3 blk(kThreads);
    const hipStream_t st = static_cast<hipStream_t>(c.stream);
    const bool sp = c.flags & VS_FLAG_SOFTPLUS;
    const vs::ScanCut cut = vs::causal_cut(c.batch, c.dim, c.L);
    a.pieces = cut.pieces;
    a.sub = cut.sub;
    a.fine_len = static_cast<int>(cut.fine_tiles * kTileTok);
    a.piece_len = a.fine_len * a.sub;
    const unsigned wide = static_cast<unsigned>((c.dim + kWideCh - 1) / kWideCh);
    if (a.pieces > 1) {
        const int64_t carry = static_cast<int64_t>(a.pieces - 1) * a.sub;
        a.piece_h = static_cast<float*>(c.ws);
        a.piece_sum = a.piece_h + c.batch * carry * c.dim * c.dstate;
        const dim3 cgrid(wide, static_cast<unsigned>(c.batch * carry));
        if (sp) hipLaunchKernelGGL((causal_scan4_kernel<T, false, true, false, true>), cgrid, blk, 0, st, a);
        else hipLaunchKernelGGL((causal_scan4_kernel<T, false, false, false, true>), cgrid, blk, 0, st, a);
        if (int rc = launched()) return rc;
    }
    const unsigned rows = static_cast<unsigned>(c.batch * a.pieces);
    if (cut.wide) {
        const dim3 grid(wide, rows);
        if (c.z && sp) hipLaunchKernelGGL((causal_scan4_kernel<T, true, true, SAVE, false>), grid, blk, 0, st, a);
        else if (c.z) hipLaunchKernelGGL((causal_scan4_kernel<T, true, false, SAVE, false>), grid, blk, 0, st, a);
        else if (sp) hipLaunchKernelGGL((causal_scan4_kernel<T, false, true, SAVE, false>), grid, blk, 0, st, a);
        else hipLaunchKernelGGL((causal_scan4_kernel<T, false, false, SAVE, false>), grid, blk, 0, st, a);
    } else {
        const dim3 grid(static_cast<unsigned>((c.dim + vs::kCausalCh - 1) / vs::kCausalCh), rows);
        if (c.z && sp) hipLaunchKernelGGL((causal_scan_kernel<T, true, true, SAVE>), grid, blk, 0, st, a);
        else if (c.z) hipLaunchKernelGGL((causal_scan_kernel<T, true, false, SAVE>), grid, blk, 0, st, a);
        else if (sp) hipLaunchKernelGGL((causal_scan_kernel<T, false, true, SAVE>), grid, blk, 0, st, a);
        else hipLaunchKernelGGL((causal_scan_kernel<T, false, false, SAVE>), grid, blk, 0, st, a);
    }
    return launched();
}

}  // namespace

// ---------------------------------------------------------------- C ABI
extern "C" {

int s6_causal_conv(int64_t batch, int64_t dim, int64_t width, int64_t seqlen, int dtype, int flags,
                   const void* x, const int64_t* strides, const float* w, const float* bias,
                   const void* window, const int32_t* lengths, void* y, void* window_out,
                   void* stream) {
    vs::ConvCall c{};
    c.batch = batch; c.dim = dim; c.width = width; c.L = seqlen; c.dtype = dtype; c.flags = flags;
    c.x = x; c.strides = strides; c.w = w; c.bias = bias; c.window = window; c.lengths = lengths;
    c.y = y; c.window_out = window_out; c.stream = stream;
    if (int rc = vs::prepare_conv(c)) return rc;
    return dtype == VS_BF16 ? launch_conv<uint16_t>(c) : launch_conv<float>(c);
}

int s6_conv_step(int64_t batch, int64_t dim, int64_t width, int dtype, int flags, const void* x,
                 int64_t x_stride, const float* w, const float* bias, void* window, int64_t slots,
                 const int32_t* slot_in, const int32_t* slot_out, void* y, void* stream) {
    vs::StepCall c{};
    c.batch = batch; c.dim = dim; c.inner = width; c.dtype = dtype; c.flags = flags; c.u = x;
    c.strides = &x_stride; c.A = w; c.dt_bias = bias; c.pool = window; c.slots = slots;
    c.slot_in = slot_in; c.slot_out = slot_out; c.y = y; c.stream = stream;
    if (int rc = vs::prepare_conv_step(c)) return rc;
    return dtype == VS_BF16 ? launch_conv_step<uint16_t>(c) : launch_conv_step<float>(c);
}

int s6_causal_scan_saved(int64_t batch, int64_t dim, int64_t dstate, int64_t seqlen, int dtype,
                         int flags, const void* u, const void* delta, const void* z, const void* B,
                         const void* C, const int64_t* strides, const float* A, const float* Dskip,
                         const float* dt_bias, const float* h0, const int32_t* lengths, void* y,
                         float* h_out, void* saved, size_t saved_bytes, void* workspace,
                         size_t workspace_bytes, void* stream) {
    vs::CausalCall c{};
    c.batch = batch; c.dim = dim; c.dstate = dstate; c.L = seqlen; c.dtype = dtype; c.flags = flags;
    c.u = u; c.delta = delta; c.z = z; c.B = B; c.C = C; c.strides = strides; c.A = A; c.Dskip = Dskip;
    c.dt_bias = dt_bias; c.h0 = h0; c.lengths = lengths; c.y = y; c.h_out = h_out; c.saved = saved;
    c.saved_bytes = saved_bytes; c.ws = workspace; c.ws_bytes = workspace_bytes; c.stream = stream;
    c.save = true;
    if (int rc = vs::prepare_causal(c)) return rc;
    return dtype == VS_BF16 ? launch_scan<uint16_t, true>(c) : launch_scan<float, true>(c);
}

int s6_causal_scan(int64_t batch, int64_t dim, int64_t dstate, int64_t seqlen, int dtype, int flags,
                   const void* u, const void* delta, const void* z, const void* B, const void* C,
                   const int64_t* strides, const float* A, const float* Dskip, const float* dt_bias,
                   const float* h0, const int32_t* lengths, void* y, float* h_out, void* workspace,
                   size_t workspace_bytes, void* stream) {
    vs::CausalCall c{};
    c.batch = batch; c.dim = dim; c.dstate = dstate; c.L = seqlen; c.dtype = dtype; c.flags = flags;
    c.u = u; c.delta = delta; c.z = z; c.B = B; c.C = C; c.strides = strides; c.A = A; c.Dskip = Dskip;
    c.dt_bias = dt_bias; c.h0 = h0; c.lengths = lengths; c.y = y; c.h_out = h_out;
    c.ws = workspace; c.ws_bytes = workspace_bytes; c.stream = stream;
    if (int rc = vs::prepare_causal(c)) return rc;
    return dtype == VS_BF16 ? launch_scan<uint16_t, false>(c) : launch_scan<float, false>(c);
}

int s6_scan_step(int64_t batch, int64_t dim, int64_t dstate, int dtype, int flags, const void* u,
                 const void* delta, const void* z, const void* B, const void* C,
                 const int64_t* strides, const float* A, const float* Dskip, const float* dt_bias,
                 float* h, int64_t slots, const int32_t* slot_in, const int32_t* slot_out, void* y,
                 void* stream) {
    vs::StepCall c{};
    c.batch = batch; c.dim = dim; c.inner = dstate; c.dtype = dtype; c.flags = flags; c.u = u; c.delta = delta;
    c.z = z; c.B = B; c.C = C; c.strides = strides; c.A = A; c.Dskip = Dskip; c.dt_bias = dt_bias; c.pool = h;
    c.slots = slots; c.slot_in = slot_in; c.slot_out = slot_out; c.y = y; c.stream = stream;
    if (int rc = vs::prepare_scan_step(c)) return rc;
    return dtype == VS_BF16 ? launch_scan_step<uint16_t>(c) : launch_scan_step<float>(c);
}

}  // extern "C"
