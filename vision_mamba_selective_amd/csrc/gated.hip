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
constexpr float kSlow = 0.25f * kLog2e;

// With w = s log2(e): a = 2^-w, u = 1 - a and q = 1 - a^2 = u (2 - u). Below
// s = 1/4 u = w p(w), with p the interpolation of (1 - 2^-w) / w at Chebyshev
// points (degree 4, off by 1.2e-8): 1 - 2^-w would cancel, and a = 1 - u is rounded
// to nearest, where the hardware's exp2 leans to one side: over the thousands of
// tokens that such decays remember that adds up (off by 1e-5 of the state at
// decays of 0.999). a is held at 2^-126 or more: a zero would turn an infinite
// state into NaN. A row whose gate can't reach 1/4 (SLOW) needs no other case: a
// sixth of a token's instructions (bf16, 4 x 768 x 2,048: 13.1 us with it, 13.9
// without; 8 x 768 x 4,097, which waits for memory, 50.0 and 50.5).
struct Decay {
    float w, a, q;
    template <bool SLOW>
    __device__ __forceinline__ void set(float k2, float sr) {
        w = k2 * sr;
        float p = fmaf(w, 0.0012023085f, -0.00957758f);
        p = fmaf(w, p, 0.055498935f);
        p = fmaf(w, p, -0.24022627f);
        p = fmaf(w, p, 0.6931472f);
        float u = w * p;
        a = 1.f - u;
        if constexpr (!SLOW) {
            const float e = __builtin_amdgcn_exp2f(at_least(-w, -126.f));
            const bool slow = w < kSlow;
            u = slow ? u : 1.f - e;
            a = slow ? a : e;
        }
        q = u * (2.f - u);
    }
    __device__ __forceinline__ void none() { w = 0.f; a = 1.f; q = 0.f; }
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
// token t of a row: a scalar base and 32 bits of offset (t is below 2^28)
template <typename P>
__device__ __forceinline__ P* at_token(P* row, int t) {
    typedef std::conditional_t<std::is_const_v<P>, const char, char> Byte;
    return reinterpret_cast<P*>(reinterpret_cast<Byte*>(row) + static_cast<uint32_t>(t) * static_cast<uint32_t>(sizeof(P)));
}
// V tokens of a lane from t on (eight, or one in a row's short last block);
// PART: of a row with len real ones, zeros past them
template <typename T, int V>
struct Tokens {
    Eight<T> e;
    template <bool PART>
    __device__ __forceinline__ void load(const T* p, int t, int len) {
        if (!PART || t + V <= len) e.load(at_token(p, t));
        else e.load_some(p, t, len);
    }
    __device__ __forceinline__ float get(int j) const { return e.get(j); }
};
template <typename T>
struct Tokens<T, 1> {
    uint32_t raw;
    template <bool PART>
    __device__ __forceinline__ void load(const T* p, int t, int len) { raw = t < len ? ld_raw(p, t) : 0u; }
    __device__ __forceinline__ float get(int) const { return from_raw<T>(raw); }
};
template <bool PART, typename T, int V>
__device__ __forceinline__ void store_tokens(T* p, int t, int L, const float (&f)[V]) {
    if constexpr (V == 8) {
        if (!PART || t + V <= L) return store_eight(at_token(p, t), f);
    }
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (t + j < L) st(p, t + j, f[j]);
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
        if constexpr (G == 64) row = __builtin_amdgcn_readfirstlane(row);   // its pointers are scalars
        b = row / a.dim;
        d = row - b * a.dim;
        lane = tid & (G - 1);
        wave = NW > 1 ? __builtin_amdgcn_readfirstlane(tid >> 6) : 0;
        L = real ? a.L : 0;
        len = L;
        if (a.lengths) len = min(max(a.lengths[b], 0), L);
        if constexpr (G == 64) len = __builtin_amdgcn_readfirstlane(len);
    }
    // the wave's first token of chunk c, and this lane's
    __device__ __forceinline__ int block_start(int c) const { return (c * NW + wave) * kVec * G; }
    __device__ __forceinline__ int start(int c) const { return block_start(c) + lane * kVec; }
    // whether any token of the wave's block is real, and whether all are (the
    // same for the wave, which may be the only one of its row to go that way)
    __device__ __forceinline__ bool live(int c) const {
        if constexpr (G == 64) return block_start(c) < len;
        else return __ballot(start(c) < len) != 0;
    }
    __device__ __forceinline__ bool full(int c) const {
        if constexpr (G == 64) return block_start(c) + kVec * G <= len;
        else return __ballot(start(c) + kVec > len) == 0;
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

// What the waves of a row hand each other: the composition of each one's block.
// A wave is at most one barrier ahead, so two buffers do.
template <int NW, bool LATER>
__device__ __forceinline__ float pass_on(Exchange<NW>& ex, int buf, int wave, int lane, float P, float H, float& carry) {
    float mine = carry;
    if constexpr (NW > 1) {
        if (lane == 0) { ex.P[buf][wave] = P; ex.H[buf][wave] = H; }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < NW; ++k) {
            const int o = LATER ? NW - 1 - k : k;
            if (o == wave) mine = carry;
            carry = fmaf(ex.P[buf][o], carry, ex.H[buf][o]);
        }
    } else {
        carry = fmaf(P, carry, H);
    }
    return mine;
}

typedef std::integral_constant<int, kVec> Wide;
typedef std::integral_constant<int, 1> Narrow;
// A row's last chunk of at most 64 tokens is taken one token a lane, by the first
// wave: with eight a row of 4,097 would spend a ninth of its time on one token.
template <int G, int NW>
__device__ __forceinline__ bool narrow_end(int L) {
    return G == 64 && L > kVec * G * NW && (L - 1) % (kVec * G * NW) < 64;
}

// ----------------------------------------------------------------- forward
// Bound by memory where there are rows enough (8 x 768 x 4,097 bf16 of ragged
// lengths 50 us, 4.0 TB/s, VALU issue 56 %; 1 x 1,536 x 16,385 without a gate 45 us,
// 4.5 TB/s); else by the chain of its steps (1 x 384 x 197 fp32 6 us, most of it the
// launch). The next block is read while one is worked on.
template <typename T, int G, int NW, bool GATED>
__global__ __launch_bounds__(NW > 4 ? 64 * NW : 256) void gated_scan_kernel(const GatedArgs a) {
    constexpr int kChunk = kVec * G * NW;
    __shared__ Exchange<NW> ex;
    const RowLane<T, G, NW> w(a);
    const T *x = w.in(a.x, a.sx), *r = w.in(a.r, a.sr), *ig = w.in(a.i, a.si), *z = GATED ? w.in(a.z, a.sz) : nullptr;
    T* y = w.out(a.y, a.L);
    const float k2 = a.rate * softplus_f(a.lam[w.d]) * kLog2e;
    const bool slow = __ballot(!(k2 < kSlow)) == 0;
    float h = a.h0 ? a.h0[w.row] : 0.f;

    // one block: composition of its tokens, of the lanes, of the waves, then the tokens again
    auto block = [&](auto vec, auto is_slow, auto is_part, auto& tx, auto& tr, auto& ti, auto& tz, int t, int c, auto&& next) VS_INLINE {
        constexpr int V = decltype(vec)::value;
        constexpr bool SLOW = decltype(is_slow)::value, PART = decltype(is_part)::value;
        float al[V], v[V], g[V];
        float P = 1.f, H = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            Decay e;
            e.template set<SLOW>(k2, sigmoid_f(tr.get(j)));
            float in = __builtin_amdgcn_sqrtf(e.q) * (sigmoid_f(ti.get(j)) * tx.get(j));
            if (PART && t + j >= w.len) { e.a = 1.f; in = 0.f; }
            al[j] = e.a;
            v[j] = in;
            if constexpr (GATED) g[j] = silu_f(tz.get(j));
            H = fmaf(e.a, H, in);
            P *= e.a;
        }
        P = at_least(P, kTiny);
        next();
        scan_up<G>(P, H);
        float Pb, Hb, Pa, Ha;
        before_and_all<G>(P, H, Pb, Hb, Pa, Ha);
        const float start = pass_on<NW, false>(ex, c & 1, w.wave, w.lane, Pa, Ha, h);
        if (a.saved && w.lane == 0 && w.L > 0) a.saved[static_cast<size_t>(w.row) * a.nblk + c * NW + w.wave] = start;
        float s = fmaf(Pb, start, Hb);
        float f[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            s = fmaf(al[j], s, v[j]);
            f[j] = s;
            if constexpr (GATED) f[j] *= g[j];
            if (PART && t + j >= w.len) f[j] = 0.f;
        }
        store_tokens<PART>(y, t, w.L, f);
    };

    Tokens<T, kVec> tx, tr, ti, tz;
    auto load = [&](int c) VS_INLINE {
        if (!w.live(c)) return;
        const int t = w.start(c);
        if (w.full(c)) {
            tx.template load<false>(x, t, w.len);
            tr.template load<false>(r, t, w.len);
            ti.template load<false>(ig, t, w.len);
            if constexpr (GATED) tz.template load<false>(z, t, w.len);
        } else {
            tx.template load<true>(x, t, w.len);
            tr.template load<true>(r, t, w.len);
            ti.template load<true>(ig, t, w.len);
            if constexpr (GATED) tz.template load<true>(z, t, w.len);
        }
    };
    const int chunks = (a.L + kChunk - 1) / kChunk, wide = chunks - (narrow_end<G, NW>(a.L) ? 1 : 0);
    load(0);
    for (int c = 0; c < wide; ++c) {
        const int t = w.start(c);
        auto next = [&]() VS_INLINE {
            if (c + 1 < wide) load(c + 1);
        };
        if (!w.live(c)) {                                  // padding
            pass_on<NW, false>(ex, c & 1, w.wave, w.lane, 1.f, 0.f, h);
            const float f[kVec] = {};
            store_tokens<true>(y, t, w.L, f);
        } else if (!w.full(c)) {
            block(Wide{}, std::false_type{}, std::true_type{}, tx, tr, ti, tz, t, c, next);
        } else if (slow) {
            block(Wide{}, std::true_type{}, std::false_type{}, tx, tr, ti, tz, t, c, next);
        } else {
            block(Wide{}, std::false_type{}, std::false_type{}, tx, tr, ti, tz, t, c, next);
        }
    }
    if constexpr (G == 64) {
        if (wide < chunks && w.wave > 0) {
            pass_on<NW, false>(ex, wide & 1, w.wave, w.lane, 1.f, 0.f, h);
        } else if (wide < chunks) {
            const int t = wide * kChunk + w.lane;
            Tokens<T, 1> nx, nr, ni, nz;
            nx.template load<true>(x, t, w.len);
            nr.template load<true>(r, t, w.len);
            ni.template load<true>(ig, t, w.len);
            if constexpr (GATED) nz.template load<true>(z, t, w.len);
            block(Narrow{}, std::false_type{}, std::true_type{}, nx, nr, ni, nz, t, wide, [] {});
        }
    }
    if (a.h_out && w.lane == 0 && w.wave == 0 && w.L > 0) a.h_out[w.row] = h;
}

// ---------------------------------------------------------------- gradient
// The states' scale in dlam: G = dL/ds s, so dL/dlam = sum G (dk/dlam) / k =
// sum G sigmoid(lam) / softplus(lam), which tends to sum G for small lam.
__device__ __forceinline__ float lam_slope(float lam) { return lam < -20.f ? 1.f : sigmoid_f(lam) / softplus_f(lam); }

// Nine streams (five read, four written), so memory again: 8 x 768 x 4,097 bf16 93 us,
// 472 MB at 5.1 TB/s, VALU issue 67 %. The states are made again from the saved
// ones: keeping them all would be a tenth stream in fp32. A block's inputs are read
// in two parts, as the registers of the former's become free.
template <typename T, int G, int NW, bool GATED>
__global__ __launch_bounds__(NW > 4 ? 64 * NW : 256) void gated_grad_kernel(const GatedArgs a) {
    constexpr int kChunk = kVec * G * NW;
    __shared__ Exchange<NW> ex;
    const RowLane<T, G, NW> w(a);
    const T *x = w.in(a.x, a.sx), *r = w.in(a.r, a.sr), *ig = w.in(a.i, a.si), *z = GATED ? w.in(a.z, a.sz) : nullptr;
    const T* dy = w.in(a.dy, a.sdy);
    T *dx = w.out(a.dx, a.L), *dr = w.out(a.dr, a.L), *di = w.out(a.di, a.L), *dz = GATED ? w.out(a.dz, a.L) : nullptr;
    const float* saved = a.saved + static_cast<size_t>(w.row) * a.nblk;
    const float k2 = a.rate * softplus_f(a.lam[w.d]) * kLog2e;
    const bool slow = __ballot(!(k2 < kSlow)) == 0;
    float mu = a.dh_out ? a.dh_out[w.row] : 0.f;
    // dlam's sum, a block's tokens in 32 bits and the blocks in 64: a row of 2^24
    // tokens has 32,768 for each lane, which in 32 bits were off by 3e-4 of their sum.
    // Rows of 16 lanes have at most three blocks.
    std::conditional_t<G == 16, float, double> total = 0;

    auto block = [&](auto vec, auto is_slow, auto is_part, auto& tx, auto& tr, auto& ti, auto& tz, auto& ty, float& first, int t, int c,
                     auto&& next) VS_INLINE {
        constexpr int V = decltype(vec)::value;
        constexpr bool SLOW = decltype(is_slow)::value, PART = decltype(is_part)::value;
        const float start = first;
        float al[V], sr[V], si[V], rq[V], m[V], in[V];     // m = sqrt(q), rq = 1 / m, in = sigmoid(i) x (0 at padding)
        float P = 1.f, H = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            sr[j] = sigmoid_f(tr.get(j));
            si[j] = sigmoid_f(ti.get(j));
            Decay e;
            e.template set<SLOW>(k2, sr[j]);
            in[j] = si[j] * tx.get(j);
            if (PART && t + j >= w.len) {
                e.none();
                in[j] = 0.f;
            }
            al[j] = e.a;
            rq[j] = e.q < 1e-36f ? 0.f : __builtin_amdgcn_rsqf(e.q);
            m[j] = e.q * rq[j];
            H = fmaf(al[j], H, m[j] * in[j]);
            P *= al[j];
        }
        P = at_least(P, kTiny);
        next(std::false_type{});
        float Pi = P, Pb, Hb, Pa, Ha;
        scan_up<G>(Pi, H);
        before_and_all<G>(Pi, H, Pb, Hb, Pa, Ha);
        float hb[V], gy[V], M = 0.f;
        float h = fmaf(Pb, start, Hb), fz[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            hb[j] = h;
            h = fmaf(al[j], h, m[j] * in[j]);
            gy[j] = ty.get(j);
            if constexpr (GATED) {
                const float zv = tz.get(j), sz = sigmoid_f(zv), dsz = gy[j] * sz;
                fz[j] = dsz * h * fmaf(zv, 1.f - sz, 1.f);
                if (PART && t + j >= w.len) fz[j] = 0.f;
                gy[j] = dsz * zv;
            }
        }
        next(std::true_type{});
        if constexpr (GATED) store_tokens<PART>(dz, t, w.L, fz);
#pragma unroll
        for (int j = V - 1; j >= 0; --j) M = al[j] * (gy[j] + M);
        float Pl, Ml;
        later_and_all<G>(P, M, w.lane, Pl, Ml, Pa, Ha);
        const float from = pass_on<NW, true>(ex, c & 1, w.wave, w.lane, Pa, Ha, mu);
        float back = fmaf(Pl, from, Ml), sum = 0.f, fx[V], fr[V], fi[V];
#pragma unroll
        for (int j = V - 1; j >= 0; --j) {
            const bool on = !PART || t + j < w.len;
            const float lt = gy[j] + back, lm = lt * m[j];
            back = al[j] * lt;
            fx[j] = on ? lm * si[j] : 0.f;
            fi[j] = on ? lm * in[j] * (1.f - si[j]) : 0.f;
            // s dL/ds (over ln 2): through m, a^2 s / m in, and through a, -s a h_before
            const float gs = on && rq[j] != 0.f ? k2 * sr[j] * back * fmaf(al[j] * rq[j], in[j], -hb[j]) : 0.f;
            fr[j] = gs * fmaf(-sr[j], kLn2, kLn2);
            sum += gs;
        }
        total += sum;
        store_tokens<PART>(dx, t, w.L, fx);
        store_tokens<PART>(dr, t, w.L, fr);
        store_tokens<PART>(di, t, w.L, fi);
    };

    const int chunks = (a.L + kChunk - 1) / kChunk, wide = chunks - (narrow_end<G, NW>(a.L) ? 1 : 0);
    if constexpr (G == 64) {
        if (wide < chunks && w.wave > 0) {
            pass_on<NW, true>(ex, wide & 1, w.wave, w.lane, 1.f, 0.f, mu);
        } else if (wide < chunks) {
            const int t = wide * kChunk + w.lane;
            Tokens<T, 1> nx, nr, ni, nz, ny;
            nx.template load<true>(x, t, w.len);
            nr.template load<true>(r, t, w.len);
            ni.template load<true>(ig, t, w.len);
            ny.template load<true>(dy, t, w.len);
            if constexpr (GATED) nz.template load<true>(z, t, w.len);
            float first = w.L > 0 ? saved[wide * NW] : 0.f;
            block(Narrow{}, std::false_type{}, std::true_type{}, nx, nr, ni, nz, ny, first, t, wide, [](auto) {});
        }
    }
    Tokens<T, kVec> tx, tr, ti, tz, ty;
    float first = 0.f;
    // a block's inputs in two parts: those that the recurrence reads, and those that the gate does
    auto load_part = [&](int c, auto part, auto gate) VS_INLINE {
        constexpr bool PART = decltype(part)::value;
        const int t = w.start(c);
        if constexpr (!decltype(gate)::value) {
            tx.template load<PART>(x, t, w.len);
            tr.template load<PART>(r, t, w.len);
            ti.template load<PART>(ig, t, w.len);
            first = w.L > 0 ? saved[c * NW + w.wave] : 0.f;
        } else {
            ty.template load<PART>(dy, t, w.len);
            if constexpr (GATED) tz.template load<PART>(z, t, w.len);
        }
    };
    auto load = [&](int c, auto gate) VS_INLINE {
        if (c < 0 || !w.live(c)) return;
        if (w.full(c)) load_part(c, std::false_type{}, gate);
        else load_part(c, std::true_type{}, gate);
    };
    load(wide - 1, std::false_type{});
    load(wide - 1, std::true_type{});
    for (int c = wide - 1; c >= 0; --c) {
        const int t = w.start(c);
        auto next = [&](auto gate) VS_INLINE { load(c - 1, gate); };
        if (!w.live(c)) {                                  // padding
            pass_on<NW, true>(ex, c & 1, w.wave, w.lane, 1.f, 0.f, mu);
            const float f[kVec] = {};
            store_tokens<true>(dx, t, w.L, f);
            store_tokens<true>(dr, t, w.L, f);
            store_tokens<true>(di, t, w.L, f);
            if constexpr (GATED) store_tokens<true>(dz, t, w.L, f);
            next(std::false_type{});
            next(std::true_type{});
        } else if (!w.full(c)) {
            block(Wide{}, std::false_type{}, std::true_type{}, tx, tr, ti, tz, ty, first, t, c, next);
        } else if (slow) {
            block(Wide{}, std::true_type{}, std::false_type{}, tx, tr, ti, tz, ty, first, t, c, next);
        } else {
            block(Wide{}, std::false_type{}, std::false_type{}, tx, tr, ti, tz, ty, first, t, c, next);
        }
    }
    if (a.dh0 && w.lane == 0 && w.wave == 0 && w.L > 0) a.dh0[w.row] = mu;
    // the row's part of dlam: lanes, then waves, in a fixed order
#pragma unroll
    for (int o = 1; o < G; o *= 2) total += __shfl_xor(total, o, 64);
    float sum = static_cast<float>(total);
    if constexpr (NW > 1) {
        __syncthreads();
        if (w.lane == 0) ex.P[0][w.wave] = sum;
        __syncthreads();
        sum = 0.f;
#pragma unroll
        for (int o = 0; o < NW; ++o) sum += ex.P[0][o];
    }
    if (w.lane == 0 && w.wave == 0 && w.L > 0) a.part[w.row] = sum * kLn2;
}

// dlam: the rows of each channel, in 64 bits (their terms have either sign). One
// chain of reads for each channel, eight rows at a time: 4 us for a batch of 8, 16 of
// 64, 122 of 512 (384 channels). A launch of its own because it needs every row.
__global__ __launch_bounds__(256) void gated_lam_kernel(const GatedArgs a) {
    const uint32_t d = blockIdx.x * 256 + threadIdx.x;
    if (d >= a.dim) return;
    double s = 0;
    // eight rows in flight
    for (uint32_t row = d; row < a.rows; row += 8 * a.dim) {
        float v[8];
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j) v[j] = row + j * a.dim < a.rows ? a.part[row + j * a.dim] : 0.f;
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j) s += v[j];
    }
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
// touches no state. 515 x 1,536 bf16: 5 us for 14 MB, most of it the launch.
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
        e.set<false>(a.rate * softplus_f(lam.get(j)) * kLog2e, sigmoid_f(r.get(j)));
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
