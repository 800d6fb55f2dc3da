// gated.hip -- the gated linear recurrence: with k = rate softplus(lam),
//     s_t = k sigmoid(r_t), a_t = exp(-s_t), v_t = sqrt(1 - a_t^2) sigmoid(i_t) x_t
//     h_t = a_t h_{t-1} + v_t,  y_t = h_t silu(z_t)
// its gradient, and its form for single tokens on a pool of states.
//
// A lane takes eight consecutive tokens. Their composition is one affine map
// h -> P h + H, and maps compose associatively, (P2, H2) o (P1, H1) =
// (P1 P2, P2 H1 + H2): a DPP scan over the lanes of a row gives every lane the
// state before its tokens, from which it walks them once more. One step of 64
// lanes covers 512 tokens, so that the state passes between steps with two
// multiply-adds, and each input is read once.
//
// The gradient walks the steps backwards. Its adjoint mu_t = a_t lambda_t,
// lambda_t = dL/dh_t = gy_t + mu_{t+1}, is the same kind of recurrence with the
// same a, so each step composes mu -> P mu + M from the later lanes to the
// earlier ones. The states inside a step are made again from the one that the
// forward pass saved at its start (4 bytes for 512 tokens).
#include <hip/hip_runtime.h>

#include <cstdint>

#include "vimscan.h"
#include "vs_causal.h"
#include "vs_model.h"

namespace {

constexpr int kVec = vs::kGatedVec;

struct GatedArgs {
    const void *x, *r, *i, *z, *dy;
    vs::Strides sx, sr, si, sz, sdy;
    const float *lam, *h0, *dh_out;
    float rate;
    const int32_t* lengths;
    void* y;
    float* h_out;
    float* saved;           // [rows][nblk]: the state before each block of tokens
    void *dx, *dr, *di, *dz;
    float *dlam, *dh0, *part;
    uint32_t rows, dim;
    int L, nblk;
};

// NaN stays NaN (fmaxf would drop it)
__device__ __forceinline__ float at_least(float v, float low) { return __builtin_elementwise_maximum(v, low); }
__device__ __forceinline__ float sigmoid_f(float v) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-v * kLog2e));
}
constexpr float kTiny = 0x1p-126f;

// s, a = exp(-s) and q = 1 - a^2 from u = 1 - a, q = u (2 - u). Below s = 1/4
// u = s p(s), with p the interpolation of (1 - exp(-s)) / s at Chebyshev points
// of [0, 1/4] (degree 4, off by 5e-9): 1 - exp(-s) would cancel, and a = 1 - u is
// rounded to nearest, where the hardware's exp2 leans to one side: over the
// thousands of tokens that such decays remember that adds up (off by 1e-5 of
// the state at decays of 0.999). a is held at 2^-126 or more: a zero would turn
// an infinite state into NaN.
struct Decay {
    float s, a, q;
    __device__ __forceinline__ void set(float k, float sr) {
        s = k * sr;
        const float e = __builtin_amdgcn_exp2f(at_least(-s * kLog2e, -126.f));
        float p = fmaf(s, 0.007514301f, -0.041491f);
        p = fmaf(s, p, 0.16665113f);
        p = fmaf(s, p, -0.49999952f);
        p = fmaf(s, p, 1.f);
        const bool slow = s < 0.25f;
        const float u = slow ? s * p : 1.f - e;
        a = slow ? 1.f - u : e;
        q = u * (2.f - u);
    }
    __device__ __forceinline__ void none() { s = 0.f; a = 1.f; q = 0.f; }
};

// ------------------------------------------------------------- lane scans
// lanes that CTRL gives no source, or that ROWS leaves out, see `none`
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ float dpp_or(float none, float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(none), __float_as_int(v), CTRL, ROWS, 0xf, false));
}
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ void compose(float& P, float& H) {
    const float p = dpp_or<CTRL, ROWS>(1.f, P), h = dpp_or<CTRL, ROWS>(0.f, H);
    H = fmaf(P, h, H);
    P = at_least(P * p, kTiny);
}
// inclusive composition over the lanes before, G lanes a row
template <int G>
__device__ __forceinline__ void scan_up(float& P, float& H) {
    compose<0x111>(P, H);                                // row_shr 1, 2, 4, 8
    compose<0x112>(P, H);
    compose<0x114>(P, H);
    compose<0x118>(P, H);
    if constexpr (G == 64) {
        compose<0x142, 0xa>(P, H);                       // row_bcast 15 into rows 1 and 3
        compose<0x143, 0xc>(P, H);                       // row_bcast 31 into rows 2 and 3
    }
}
__device__ __forceinline__ float lane_value(float v, int lane) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}
// of an inclusive scan over the lanes before: the composition of the lanes
// before this one, and that of all
template <int G>
__device__ __forceinline__ void before_and_all(float P, float H, float& Pb, float& Hb, float& Pa, float& Ha) {
    if constexpr (G == 64) {
        Pb = dpp_or<0x138>(1.f, P);                      // wave_shr 1
        Hb = dpp_or<0x138>(0.f, H);
        Pa = lane_value(P, 63);
        Ha = lane_value(H, 63);
    } else {
        Pb = dpp_or<0x111>(1.f, P);
        Hb = dpp_or<0x111>(0.f, H);
        Pa = row_bcast<15>(P);
        Ha = row_bcast<15>(H);
    }
}
// the same towards the earlier lanes: the composition of the later lanes, and that of all
template <int G>
__device__ __forceinline__ void later_and_all(float P, float M, int lane, float& Pl, float& Ml, float& Pa, float& Ma) {
    compose<0x101>(P, M);                                // row_shl 1, 2, 4, 8
    compose<0x102>(P, M);
    compose<0x104>(P, M);
    compose<0x108>(P, M);
    Pl = dpp_or<0x101>(1.f, P);
    Ml = dpp_or<0x101>(0.f, M);
    if constexpr (G == 16) {
        Pa = row_bcast<0>(P);
        Ma = row_bcast<0>(M);
    } else {
        // rows of 16 lanes, from the last to the first
        const float P3 = lane_value(P, 48), M3 = lane_value(M, 48);
        const float P2 = lane_value(P, 32), M2 = fmaf(P2, M3, lane_value(M, 32)), P32 = at_least(P2 * P3, kTiny);
        const float P1 = lane_value(P, 16), M1 = fmaf(P1, M2, lane_value(M, 16)), P321 = at_least(P1 * P32, kTiny);
        const float P0 = lane_value(P, 0);
        Ma = fmaf(P0, M1, lane_value(M, 0));
        Pa = at_least(P0 * P321, kTiny);
        const float pr = lane < 16 ? P321 : lane < 32 ? P32 : lane < 48 ? P3 : 1.f;
        const float mr = lane < 16 ? M1 : lane < 32 ? M2 : lane < 48 ? M3 : 0.f;
        Ml = fmaf(Pl, mr, Ml);
        Pl = at_least(Pl * pr, kTiny);
    }
}

// ------------------------------------------------------------------ tokens
// eight tokens from t on of a row with len real ones, zeros past them
template <typename T>
__device__ __forceinline__ void load_tokens(Eight<T>& e, const T* p, int t, int len) {
    if (t + kVec <= len) e.load(p + t);
    else e.load_some(p, t, len);
}
template <typename T>
__device__ __forceinline__ void store_tokens(T* p, int t, int L, const float (&f)[kVec]) {
    if (t + kVec <= L) {
        store_eight(p + t, f);
    } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j)
            if (t + j < L) st(p, t + j, f[j]);
    }
}

// What a lane knows of its row. Rows past the last are walked with no tokens
// and nothing stored.
template <typename T, int G, int NW>
struct RowLane {
    uint32_t row, b, d;
    int lane, wave, len, L;
    __device__ __forceinline__ explicit RowLane(const GatedArgs& a) {
        const uint32_t tid = threadIdx.x;
        const uint32_t id = NW > 1 ? blockIdx.x : (blockIdx.x * blockDim.x + tid) / G;
        const bool real = id < a.rows;
        row = real ? id : a.rows - 1;
        b = row / a.dim;
        d = row - b * a.dim;
        lane = tid & (G - 1);
        wave = NW > 1 ? tid >> 6 : 0;
        L = real ? a.L : 0;
        len = L;
        if (a.lengths) len = min(max(a.lengths[b], 0), L);
    }
    __device__ __forceinline__ const T* in(const void* p, const vs::Strides& s) const {
        return static_cast<const T*>(p) + static_cast<int64_t>(b) * s.b + static_cast<int64_t>(d) * s.d;
    }
    __device__ __forceinline__ T* out(void* p, int L_) const { return static_cast<T*>(p) + static_cast<int64_t>(row) * L_; }
};

template <int NW>
struct Exchange {
    float P[2][NW], H[2][NW];
};

// ----------------------------------------------------------------- forward
template <typename T, int G, int NW, bool GATED>
__global__ __launch_bounds__(NW > 4 ? 64 * NW : 256) void gated_scan_kernel(const GatedArgs a) {
    constexpr int kBlock = kVec * G, kChunk = kBlock * NW;
    __shared__ Exchange<NW> ex;
    const RowLane<T, G, NW> w(a);
    const T *x = w.in(a.x, a.sx), *r = w.in(a.r, a.sr), *ig = w.in(a.i, a.si), *z = GATED ? w.in(a.z, a.sz) : nullptr;
    T* y = w.out(a.y, a.L);
    const float k = a.rate * softplus_f(a.lam[w.d]);
    float h = a.h0 ? a.h0[w.row] : 0.f;

    Eight<T> ex_, er, ei, ez;
    int t = w.wave * kBlock + w.lane * kVec;
    auto load = [&](int at) VS_INLINE {
        load_tokens(ex_, x, at, w.len);
        load_tokens(er, r, at, w.len);
        load_tokens(ei, ig, at, w.len);
        if constexpr (GATED) load_tokens(ez, z, at, w.len);
    };
    load(t);
    const int chunks = (a.L + kChunk - 1) / kChunk;
    for (int c = 0; c < chunks; ++c, t += kChunk) {
        float al[kVec], v[kVec], g[kVec];
        float P = 1.f, H = 0.f;
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            Decay e;
            e.set(k, sigmoid_f(er.get(j)));
            float in = __builtin_amdgcn_sqrtf(e.q) * sigmoid_f(ei.get(j)) * ex_.get(j);
            if (t + j >= w.len) { e.a = 1.f; in = 0.f; }
            al[j] = e.a;
            v[j] = in;
            if constexpr (GATED) g[j] = silu_f(ez.get(j));
            H = fmaf(e.a, H, in);
            P *= e.a;
        }
        P = at_least(P, kTiny);
        load(t + kChunk);
        scan_up<G>(P, H);
        float Pb, Hb, Pa, Ha;
        before_and_all<G>(P, H, Pb, Hb, Pa, Ha);
        float start = h;                                  // the state before this wave's block
        if constexpr (NW > 1) {
            const int buf = c & 1;
            if (w.lane == 0) { ex.P[buf][w.wave] = Pa; ex.H[buf][w.wave] = Ha; }
            __syncthreads();
#pragma unroll
            for (int o = 0; o < NW; ++o) {
                if (o == w.wave) start = h;
                h = fmaf(ex.P[buf][o], h, ex.H[buf][o]);
            }
        } else {
            h = fmaf(Pa, h, Ha);
        }
        if (a.saved && w.lane == 0 && t < w.L) a.saved[static_cast<size_t>(w.row) * a.nblk + t / kBlock] = start;
        float s = fmaf(Pb, start, Hb);
        float f[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            s = fmaf(al[j], s, v[j]);
            f[j] = s;
            if constexpr (GATED) f[j] *= g[j];
            if (t + j >= w.len) f[j] = 0.f;
        }
        store_tokens(y, t, w.L, f);
    }
    if (a.h_out && w.lane == 0 && w.wave == 0 && w.L > 0) a.h_out[w.row] = h;
}

// ---------------------------------------------------------------- gradient
// The states' scale in dlam: G = dL/ds s, so dL/dlam = sum G (dk/dlam) / k =
// sum G sigmoid(lam) / softplus(lam), which tends to sum G for small lam.
__device__ __forceinline__ float lam_slope(float lam) { return lam < -20.f ? 1.f : sigmoid_f(lam) / softplus_f(lam); }

template <typename T, int G, int NW, bool GATED>
__global__ __launch_bounds__(NW > 4 ? 64 * NW : 256) void gated_grad_kernel(const GatedArgs a) {
    constexpr int kBlock = kVec * G, kChunk = kBlock * NW;
    __shared__ Exchange<NW> ex;
    const RowLane<T, G, NW> w(a);
    const T *x = w.in(a.x, a.sx), *r = w.in(a.r, a.sr), *ig = w.in(a.i, a.si), *z = GATED ? w.in(a.z, a.sz) : nullptr;
    const T* dy = w.in(a.dy, a.sdy);
    T *dx = w.out(a.dx, a.L), *dr = w.out(a.dr, a.L), *di = w.out(a.di, a.L), *dz = GATED ? w.out(a.dz, a.L) : nullptr;
    const float* saved = a.saved + static_cast<size_t>(w.row) * a.nblk;
    const float lam = a.lam[w.d], k = a.rate * softplus_f(lam);
    float mu = a.dh_out ? a.dh_out[w.row] : 0.f;
    float sum = 0.f;

    const int chunks = (a.L + kChunk - 1) / kChunk;
    for (int c = chunks - 1; c >= 0; --c) {
        const int t = c * kChunk + w.wave * kBlock + w.lane * kVec;
        Eight<T> ex_, er, ei, ez, ey;
        load_tokens(ex_, x, t, w.len);
        load_tokens(er, r, t, w.len);
        load_tokens(ei, ig, t, w.len);
        load_tokens(ey, dy, t, w.len);
        if constexpr (GATED) load_tokens(ez, z, t, w.len);
        const float start = t < w.len ? saved[t / kBlock] : 0.f;
        Decay e[kVec];
        float sr[kVec], si[kVec], rq[kVec], v[kVec];
        float P = 1.f, H = 0.f;
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            sr[j] = sigmoid_f(er.get(j));
            si[j] = sigmoid_f(ei.get(j));
            e[j].set(k, sr[j]);
            if (t + j >= w.len) e[j].none();
            rq[j] = e[j].q < 1e-36f ? 0.f : __builtin_amdgcn_rsqf(e[j].q);
            v[j] = t + j < w.len ? e[j].q * rq[j] * si[j] * ex_.get(j) : 0.f;
            H = fmaf(e[j].a, H, v[j]);
            P *= e[j].a;
        }
        P = at_least(P, kTiny);
        float Pi = P, Pb, Hb, Pa, Ha;
        scan_up<G>(Pi, H);
        before_and_all<G>(Pi, H, Pb, Hb, Pa, Ha);
        float hb[kVec], gy[kVec], M = 0.f;
        float h = fmaf(Pb, start, Hb), fz[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            hb[j] = h;
            h = fmaf(e[j].a, h, v[j]);
            gy[j] = ey.get(j);
            if constexpr (GATED) {
                const float zv = ez.get(j), sz = sigmoid_f(zv);
                fz[j] = t + j < w.len ? gy[j] * h * sz * fmaf(zv, 1.f - sz, 1.f) : 0.f;
                gy[j] *= zv * sz;
            }
        }
        if constexpr (GATED) store_tokens(dz, t, w.L, fz);
#pragma unroll
        for (int j = kVec - 1; j >= 0; --j) M = e[j].a * (gy[j] + M);
        float Pl, Ml;
        later_and_all<G>(P, M, w.lane, Pl, Ml, Pa, Ha);
        float from = mu;                                  // mu after this wave's block
        if constexpr (NW > 1) {
            const int buf = c & 1;
            if (w.lane == 0) { ex.P[buf][w.wave] = Pa; ex.H[buf][w.wave] = Ha; }
            __syncthreads();
#pragma unroll
            for (int o = NW - 1; o >= 0; --o) {
                if (o == w.wave) from = mu;
                mu = fmaf(ex.P[buf][o], mu, ex.H[buf][o]);
            }
        } else {
            mu = fmaf(Pa, mu, Ha);
        }
        float m = fmaf(Pl, from, Ml), fx[kVec], fr[kVec], fi[kVec];
#pragma unroll
        for (int j = kVec - 1; j >= 0; --j) {
            const float lt = gy[j] + m;
            const bool on = t + j < w.len;
            fx[j] = on ? lt * e[j].q * rq[j] * si[j] : 0.f;
            fi[j] = on ? lt * v[j] * (1.f - si[j]) : 0.f;
            // s dL/ds: through m, a^2 s / m sigmoid(i) x, and through a, -s a h_before
            const float through = e[j].a * e[j].a * (e[j].s * rq[j]) * si[j] * ex_.get(j);
            const float gs = on && !(e[j].s < 1e-36f) ? lt * (through - e[j].s * e[j].a * hb[j]) : 0.f;
            fr[j] = gs * (1.f - sr[j]);
            sum += gs;
            m = e[j].a * lt;
        }
        store_tokens(dx, t, w.L, fx);
        store_tokens(dr, t, w.L, fr);
        store_tokens(di, t, w.L, fi);
    }
    if (a.dh0 && w.lane == 0 && w.wave == 0 && w.L > 0) a.dh0[w.row] = mu;
    // the row's part of dlam: lanes, then waves, in a fixed order
#pragma unroll
    for (int o = 1; o < G; o *= 2) sum += __shfl_xor(sum, o, 64);
    if constexpr (NW > 1) {
        __syncthreads();
        if (w.lane == 0) ex.P[0][w.wave] = sum;
        __syncthreads();
        sum = 0.f;
#pragma unroll
        for (int o = 0; o < NW; ++o) sum += ex.P[0][o];
    }
    if (w.lane == 0 && w.wave == 0 && w.L > 0) a.part[w.row] = sum;
}

// dlam: the rows of each channel, in 64 bits (their terms have either sign)
__global__ __launch_bounds__(256) void gated_lam_kernel(const GatedArgs a) {
    const uint32_t d = blockIdx.x * 256 + threadIdx.x;
    if (d >= a.dim) return;
    double s = 0;
    for (uint32_t row = d; row < a.rows; row += a.dim) s += a.part[row];
    a.dlam[d] = static_cast<float>(s * lam_slope(a.lam[d]));
}

// ------------------------------------------------------------ single tokens
struct GatedStepArgs {
    const void *x, *r, *i, *z;
    int64_t sx, sr, si, sz;
    const float* lam;
    float rate;
    float* h;
    const int32_t *slot_in, *slot_out;
    void* y;
    uint32_t dim, groups;            // groups of four channels a row
    uint64_t total;
    int64_t slots;
};

// Four channels a thread. A row whose slot is outside the pool gives zeros and
// touches no state.
template <typename T, bool GATED>
__global__ __launch_bounds__(256) void gated_step_kernel(const GatedStepArgs a) {
    const uint64_t id = static_cast<uint64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (id >= a.total) return;
    const uint32_t b = static_cast<uint32_t>(id / a.groups), d0 = (static_cast<uint32_t>(id) - b * a.groups) * 4;
    const int64_t in = a.slot_in ? a.slot_in[b] : b, to = a.slot_out ? a.slot_out[b] : b;
    T* y = static_cast<T*>(a.y) + static_cast<int64_t>(b) * a.dim;
    const bool on = in >= 0 && in < a.slots && to >= 0 && to < a.slots;
    const int n = static_cast<int>(a.dim);
    Four<T> x, r, ig, z;
    Four<float> lam, h;
    float f[4], s[4];
    auto load = [&](auto& e, const auto* p) VS_INLINE {
        if (static_cast<int>(d0) + 4 <= n) e.load(p + d0);
        else e.load_some(p, static_cast<int>(d0), n);
    };
    auto put = [&](auto* p, const float (&v)[4]) VS_INLINE {
        if (static_cast<int>(d0) + 4 <= n) {
            store_four(p + d0, v);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (static_cast<int>(d0) + j < n) st(p, d0 + j, v[j]);
        }
    };
    if (!on) {
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = 0.f;
        put(y, f);
        return;
    }
    load(x, static_cast<const T*>(a.x) + static_cast<int64_t>(b) * a.sx);
    load(r, static_cast<const T*>(a.r) + static_cast<int64_t>(b) * a.sr);
    load(ig, static_cast<const T*>(a.i) + static_cast<int64_t>(b) * a.si);
    if constexpr (GATED) load(z, static_cast<const T*>(a.z) + static_cast<int64_t>(b) * a.sz);
    load(lam, a.lam);
    load(h, a.h + in * a.dim);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        Decay e;
        e.set(a.rate * softplus_f(lam.get(j)), sigmoid_f(r.get(j)));
        s[j] = fmaf(e.a, h.get(j), __builtin_amdgcn_sqrtf(e.q) * sigmoid_f(ig.get(j)) * x.get(j));
        f[j] = s[j];
        if constexpr (GATED) f[j] *= silu_f(z.get(j));
    }
    put(a.h + to * a.dim, s);
    put(y, f);
}

// ------------------------------------------------------------------ launch
int launched() {
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? VS_OK : vs::fail(VS_ERR_HIP, std::string("kernel launch: ") + hipGetErrorString(e));
}

GatedArgs arguments(const vs::GatedCall& c) {
    GatedArgs a{};
    a.x = c.x; a.r = c.r; a.i = c.i; a.z = c.z; a.dy = c.dy;
    a.sx = c.st[0]; a.sr = c.st[1]; a.si = c.st[2]; a.sz = c.st[3]; a.sdy = c.st[4];
    a.lam = c.lam; a.h0 = c.h0; a.dh_out = c.dh_out; a.rate = c.rate; a.lengths = c.lengths;
    a.y = c.y; a.h_out = c.h_out; a.saved = c.save || c.grad ? static_cast<float*>(c.saved) : nullptr;
    a.dx = c.dx; a.dr = c.dr; a.di = c.di; a.dz = c.dz; a.dlam = c.dlam; a.dh0 = c.dh0; a.part = static_cast<float*>(c.ws);
    a.rows = static_cast<uint32_t>(c.batch * c.dim); a.dim = static_cast<uint32_t>(c.dim);
    a.L = static_cast<int>(c.L); a.nblk = static_cast<int>((c.L + c.form.block() - 1) / c.form.block());
    return a;
}

template <typename T, int G, int NW, bool GATED>
void launch_form(const vs::GatedCall& c, const GatedArgs& a) {
    constexpr uint32_t threads = NW > 1 ? 64 * NW : 256, rows = NW > 1 ? 1 : threads / G;
    const dim3 grid((a.rows + rows - 1) / rows);
    const auto s = static_cast<hipStream_t>(c.stream);
    if (c.grad) gated_grad_kernel<T, G, NW, GATED><<<grid, threads, 0, s>>>(a);
    else gated_scan_kernel<T, G, NW, GATED><<<grid, threads, 0, s>>>(a);
}

template <typename T, bool GATED>
int launch_gated(const vs::GatedCall& c) {
    const GatedArgs a = arguments(c);
    if (c.form.lanes == 16) launch_form<T, 16, 1, GATED>(c, a);
    else if (c.form.waves == 1) launch_form<T, 64, 1, GATED>(c, a);
    else if (c.form.waves == 4) launch_form<T, 64, 4, GATED>(c, a);
    else launch_form<T, 64, 8, GATED>(c, a);
    if (c.grad) gated_lam_kernel<<<(a.dim + 255) / 256, 256, 0, static_cast<hipStream_t>(c.stream)>>>(a);
    return launched();
}

int run(vs::GatedCall& c) {
    if (int rc = vs::prepare_gated(c)) return rc;
    if (c.dtype == VS_BF16) return c.z ? launch_gated<uint16_t, true>(c) : launch_gated<uint16_t, false>(c);
    return c.z ? launch_gated<float, true>(c) : launch_gated<float, false>(c);
}

vs::GatedCall call(int64_t batch, int64_t dim, int64_t L, int dtype, const void* x, const void* r, const void* i, const void* z,
                   const int64_t* strides, const float* lam, float rate, const int32_t* lengths, void* stream) {
    vs::GatedCall c{};
    c.batch = batch; c.dim = dim; c.L = L; c.dtype = dtype; c.x = x; c.r = r; c.i = i; c.z = z; c.strides = strides;
    c.lam = lam; c.rate = rate; c.lengths = lengths; c.stream = stream;
    return c;
}

}  // namespace

extern "C" {

int gated_scan(int64_t batch, int64_t dim, int64_t seqlen, int dtype, const void* x, const void* r,
               const void* i, const void* z, const int64_t* strides, const float* lam, float rate,
               const float* h0, const int32_t* lengths, void* y, float* h_out, void* stream) {
    vs::GatedCall c = call(batch, dim, seqlen, dtype, x, r, i, z, strides, lam, rate, lengths, stream);
    c.h0 = h0; c.y = y; c.h_out = h_out;
    return run(c);
}

int gated_scan_saved(int64_t batch, int64_t dim, int64_t seqlen, int dtype, const void* x,
                     const void* r, const void* i, const void* z, const int64_t* strides,
                     const float* lam, float rate, const float* h0, const int32_t* lengths, void* y,
                     float* h_out, void* saved, size_t saved_bytes, void* stream) {
    vs::GatedCall c = call(batch, dim, seqlen, dtype, x, r, i, z, strides, lam, rate, lengths, stream);
    c.h0 = h0; c.y = y; c.h_out = h_out; c.saved = saved; c.saved_bytes = saved_bytes; c.save = true;
    return run(c);
}

int gated_scan_grad(int64_t batch, int64_t dim, int64_t seqlen, int dtype, const void* x,
                    const void* r, const void* i, const void* z, const void* dy,
                    const int64_t* strides, const float* lam, float rate, const int32_t* lengths,
                    const void* saved, size_t saved_bytes, const float* dh_out, void* dx, void* dr,
                    void* di, void* dz, float* dlam, float* dh0, void* workspace,
                    size_t workspace_bytes, void* stream) {
    vs::GatedCall c = call(batch, dim, seqlen, dtype, x, r, i, z, strides, lam, rate, lengths, stream);
    c.dy = dy; c.saved = const_cast<void*>(saved); c.saved_bytes = saved_bytes; c.dh_out = dh_out;
    c.dx = dx; c.dr = dr; c.di = di; c.dz = dz; c.dlam = dlam; c.dh0 = dh0; c.ws = workspace;
    c.ws_bytes = workspace_bytes; c.grad = true;
    return run(c);
}

int gated_scan_step(int64_t batch, int64_t dim, int dtype, const void* x, const void* r,
                    const void* i, const void* z, const int64_t* strides, const float* lam,
                    float rate, float* h, int64_t slots, const int32_t* slot_in,
                    const int32_t* slot_out, void* y, void* stream) {
    vs::GatedStepCall c{};
    c.batch = batch; c.dim = dim; c.dtype = dtype; c.x = x; c.r = r; c.i = i; c.z = z; c.strides = strides;
    c.lam = lam; c.rate = rate; c.h = h; c.slots = slots; c.slot_in = slot_in; c.slot_out = slot_out; c.y = y;
    c.stream = stream;
    if (int rc = vs::prepare_gated_step(c)) return rc;
    GatedStepArgs a{};
    a.x = x; a.r = r; a.i = i; a.z = z; a.sx = c.st[0]; a.sr = c.st[1]; a.si = c.st[2]; a.sz = c.st[3];
    a.lam = lam; a.rate = rate; a.h = h; a.slot_in = slot_in; a.slot_out = slot_out; a.y = y; a.slots = slots;
    a.dim = static_cast<uint32_t>(dim); a.groups = (a.dim + 3) / 4; a.total = static_cast<uint64_t>(batch) * a.groups;
    const dim3 grid(static_cast<uint32_t>((a.total + 255) / 256));
    const auto s = static_cast<hipStream_t>(stream);
    if (dtype == VS_BF16) {
        if (z) gated_step_kernel<uint16_t, true><<<grid, 256, 0, s>>>(a);
        else gated_step_kernel<uint16_t, false><<<grid, 256, 0, s>>>(a);
    } else {
        if (z) gated_step_kernel<float, true><<<grid, 256, 0, s>>>(a);
        else gated_step_kernel<float, false><<<grid, 256, 0, s>>>(a);
    }
    return launched();
}

}  // extern "C"
