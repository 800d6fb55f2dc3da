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
    int L, silu;
    int tw;                 // threads along the tokens of a row: a power of two, at most kThreads
    int segs;               // workgroups along a row
};

constexpr int kConvTok = 4;     // tokens of one thread, tw apart

// y = silu(bias + sum_j w[j] line[t + j]): a thread takes kConvTok tokens of
// one row, tw apart, so that loads and stores of a wave are contiguous; short
// rows share a workgroup. Bound by memory: each entry of x comes from HBM
// once, the taps' repeats from the caches.
template <typename T, int W>
__global__ __launch_bounds__(kThreads) void causal_conv_kernel(const ConvArgs a) {
    const int tid = threadIdx.x;
    const int rows = kThreads / a.tw;
    const int64_t b = blockIdx.y;
    const int seg = static_cast<int>(blockIdx.x % static_cast<unsigned>(a.segs));
    const int64_t d = static_cast<int64_t>(blockIdx.x / static_cast<unsigned>(a.segs)) * rows + tid / a.tw;
    if (d >= a.dim) return;
    const int len = row_length(a.lengths, b, a.L);
    const T* x = static_cast<const T*>(a.x) + b * a.sx.b + d * a.sx.d;
    const T* win = a.window ? static_cast<const T*>(a.window) + (b * a.dim + d) * (W - 1) : nullptr;
    // entry p of the row's line [window | x]
    auto line = [&](int p) {
        if (p >= W - 1) return ld(x, p - (W - 1));
        return win ? ld(win, p) : 0.f;
    };
    float w[W];
#pragma unroll
    for (int j = 0; j < W; ++j) w[j] = a.w[d * W + j];
    const float bias = a.bias ? a.bias[d] : 0.f;
    T* y = static_cast<T*>(a.y) + (b * a.dim + d) * a.L;
    const int t0 = seg * a.tw * kConvTok + tid % a.tw;
#pragma unroll
    for (int i = 0; i < kConvTok; ++i) {
        const int t = t0 + i * a.tw;
        if (t >= a.L) break;
        float v = 0.f;
        if (t < len) {
            v = bias;
#pragma unroll
            for (int j = 0; j < W; ++j) v = fmaf(w[j], line(t + j), v);
            if (a.silu) v = silu_f(v);
        }
        st(y, t, v);
    }
    // the row's last W - 1 line entries, unchanged in their type
    const int j = tid % a.tw;
    if (a.window_out && seg == 0) {
        T* wo = static_cast<T*>(a.window_out) + (b * a.dim + d) * (W - 1);
        for (int k = j; k < W - 1; k += a.tw) {
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

// one token of each row, a thread per channel
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
// the padded memory holds.
template <typename T, bool GATE, bool SOFTPLUS, bool SAVE>
__global__ __launch_bounds__(kThreads) void causal_scan_kernel(const ScanFwdArgs a) {
    __shared__ __attribute__((aligned(16))) float tile[2][2][kRowLanes][kTilePad];
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int n = lane & 15;
    uint32_t cg, bb;
    xcd_block(cg, bb);
    const int64_t b = bb;
    const int64_t d0 = static_cast<int64_t>(cg) * vs::kCausalCh + (tid >> 4);
    const bool active = d0 < a.dim;
    const int64_t d = active ? d0 : a.dim - 1;
    const int L = a.L;
    const int len = row_length(a.lengths, b, L);
    const bool n_ok = n < a.dstate;
    const float A2 = n_ok ? a.A[d * a.dstate + n] * kLog2e : 0.f;
    const float Dk = a.Dskip ? a.Dskip[d] : 0.f;
    const float bias = a.dt_bias ? a.dt_bias[d] : 0.f;
    const T* u = static_cast<const T*>(a.u) + b * a.su.b + d * a.su.d;
    const T* dl = static_cast<const T*>(a.delta) + b * a.sdl.b + d * a.sdl.d;
    const T* z = static_cast<const T*>(a.z) + b * a.sz.b + d * a.sz.d;
    const size_t row = static_cast<size_t>(b * a.dim + d);
    T* y = static_cast<T*>(a.y) + row * static_cast<size_t>(L);
    float* s = SAVE ? a.s + row * static_cast<size_t>(L) : nullptr;
    float* ck = SAVE ? a.ckpt + row * static_cast<size_t>(a.nblk) * a.dstate : nullptr;

    BcStage<T> stage(a, b, tid, len);
    float h = a.h0 && n_ok ? a.h0[row * a.dstate + n] : 0.f;
    const int ntile = (len + kTileTok - 1) / kTileTok;
    if (ntile > 0) {
        stage.load(0);
        stage.store(tile[0]);
    }
    for (int it = 0; it < ntile; ++it) {
        lds_barrier();
        if (it + 1 < ntile) stage.load(it + 1);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int blk = it * 2 + half;
            const int t = blk * 16 + n;
            const bool ok = t < len;
            const int tc = ok ? t : len - 1;
            const float x = ld(dl, tc) + bias;
            const float dlt = ok ? (SOFTPLUS ? softplus_f(x) : x) : 0.f;
            const float cu = ok ? ld(u, tc) : 0.f;
            const float du = dlt * cu;
            if (SAVE && active && n_ok && blk < a.nblk) ck[static_cast<size_t>(blk) * a.dstate + n] = h;
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
            const float sum = fmaf(Dk, cu, row_transpose_sum(c, lane));
            if (active && t < L) {
                if (SAVE && GATE) s[t] = sum;
                float v = sum;
                if (GATE) v *= silu_f(ld(z, tc));
                st(y, t, ok ? v : 0.f);
            }
        }
        if (it + 1 < ntile) stage.store(tile[(it + 1) & 1]);
    }
    if (a.h_out && active && n_ok) a.h_out[row * a.dstate + n] = h;
    // the outputs of the padding past the last tile
    if (active)
        for (int t = ntile * kTileTok + n; t < L; t += 16) st(y, t, 0.f);
}

// one token of each row on the pool: four lanes per channel, lane q of a quad
// holds states q, q + 4, ... (vector loads where dstate is 16)
struct ScanStepArgs {
    const void *u, *delta, *z, *B, *C;
    const float *A, *Dskip, *dt_bias;
    float* h;
    const int32_t *slot_in, *slot_out;
    void* y;
    int64_t st[5], slots, dim;
    int dstate;
};

template <typename T, bool GATE, bool SOFTPLUS>
__global__ __launch_bounds__(kThreads) void scan_step_kernel(const ScanStepArgs a) {
    const int64_t d = static_cast<int64_t>(blockIdx.x) * (kThreads / 4) + (threadIdx.x >> 2);
    const int q = threadIdx.x & 3;
    const int64_t b = blockIdx.y;
    if (d >= a.dim) return;                          // whole quads
    T* y = static_cast<T*>(a.y) + b * a.dim + d;
    const int64_t si = a.slot_in ? a.slot_in[b] : b, so = a.slot_out ? a.slot_out[b] : b;
    if (si < 0 || so < 0 || si >= a.slots || so >= a.slots) {
        if (q == 0) st(y, 0, 0.f);
        return;
    }
    const float cu = ld(static_cast<const T*>(a.u), b * a.st[0] + d);
    const float x = ld(static_cast<const T*>(a.delta), b * a.st[1] + d) + (a.dt_bias ? a.dt_bias[d] : 0.f);
    const float dlt = SOFTPLUS ? softplus_f(x) : x;
    const float du = dlt * cu;
    const T* B = static_cast<const T*>(a.B) + b * a.st[3];
    const T* C = static_cast<const T*>(a.C) + b * a.st[4];
    const float* hi = a.h + (si * a.dim + d) * a.dstate;
    float* ho = a.h + (so * a.dim + d) * a.dstate;
    const float* A = a.A + d * a.dstate;
    float sum = 0.f;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int n = 4 * q + r;
        if (n < a.dstate) {
            const float v = fmaf(__builtin_amdgcn_exp2f(dlt * (A[n] * kLog2e)), hi[n], du * ld(B, n));
            ho[n] = v;
            sum = fmaf(v, ld(C, n), sum);
        }
    }
    sum += dpp<0xb1>(sum);                           // quad_perm [1,0,3,2]
    sum += dpp<0x4e>(sum);                           // quad_perm [2,3,0,1]
    if (q == 0) {
        float v = fmaf(a.Dskip ? a.Dskip[d] : 0.f, cu, sum);
        if (GATE) v *= silu_f(ld(static_cast<const T*>(a.z), b * a.st[2] + d));
        st(y, 0, v);
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
    a.L = static_cast<int>(c.L); a.silu = c.flags & VS_CONV_SILU;
    a.tw = 4;
    while (a.tw < kThreads && a.tw < c.L) a.tw *= 2;
    const int64_t per = static_cast<int64_t>(a.tw) * kConvTok;
    a.segs = static_cast<int>((c.L + per - 1) / per);
    const int64_t rows = kThreads / a.tw, groups = (c.dim + rows - 1) / rows * a.segs;
    if (groups >= (int64_t(1) << 31)) return fail(VS_ERR_UNSUPPORTED, "too many tokens and channels for one launch");
    const dim3 grid(static_cast<unsigned>(groups), static_cast<unsigned>(c.batch));
    return with_width(c.width, [&](auto w) {
        hipLaunchKernelGGL((causal_conv_kernel<T, decltype(w)::value>), grid, dim3(kThreads), 0,
                           static_cast<hipStream_t>(c.stream), a);
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

template <typename T>
int launch_scan_step(const vs::StepCall& c) {
    ScanStepArgs a{};
    a.u = c.u; a.delta = c.delta; a.z = c.z; a.B = c.B; a.C = c.C; a.A = c.A; a.Dskip = c.Dskip; a.dt_bias = c.dt_bias;
    a.h = static_cast<float*>(c.pool); a.slot_in = c.slot_in; a.slot_out = c.slot_out; a.y = c.y;
    for (int i = 0; i < 5; ++i) a.st[i] = c.st[i];
    a.slots = c.slots; a.dim = c.dim; a.dstate = static_cast<int>(c.inner);
    const dim3 grid(static_cast<unsigned>((c.dim + kThreads / 4 - 1) / (kThreads / 4)), static_cast<unsigned>(c.batch));
    const dim3 blk(kThreads);
    const hipStream_t st = static_cast<hipStream_t>(c.stream);
    const bool sp = c.flags & VS_FLAG_SOFTPLUS;
    if (c.z && sp) hipLaunchKernelGGL((scan_step_kernel<T, true, true>), grid, blk, 0, st, a);
    else if (c.z) hipLaunchKernelGGL((scan_step_kernel<T, true, false>), grid, blk, 0, st, a);
    else if (sp) hipLaunchKernelGGL((scan_step_kernel<T, false, true>), grid, blk, 0, st, a);
    else hipLaunchKernelGGL((scan_step_kernel<T, false, false>), grid, blk, 0, st, a);
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
    const dim3 grid(static_cast<unsigned>((c.dim + vs::kCausalCh - 1) / vs::kCausalCh), static_cast<unsigned>(c.batch));
    const dim3 blk(kThreads);
    const hipStream_t st = static_cast<hipStream_t>(c.stream);
    const bool sp = c.flags & VS_FLAG_SOFTPLUS;
    if (c.z && sp) hipLaunchKernelGGL((causal_scan_kernel<T, true, true, SAVE>), grid, blk, 0, st, a);
    else if (c.z) hipLaunchKernelGGL((causal_scan_kernel<T, true, false, SAVE>), grid, blk, 0, st, a);
    else if (sp) hipLaunchKernelGGL((causal_scan_kernel<T, false, true, SAVE>), grid, blk, 0, st, a);
    else hipLaunchKernelGGL((causal_scan_kernel<T, false, false, SAVE>), grid, blk, 0, st, a);
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
