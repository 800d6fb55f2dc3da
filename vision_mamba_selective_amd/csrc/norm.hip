// norm.hip -- the root-mean-square norm with the residual's addition,
//     s = x + residual (rounded to the activations' type), q = 1 / sqrt(mean_d s^2 + eps),
//     y = s q w
// and its gradient
//     ds = dsum + q (w dy) - s q^3 mean_d(w dy s),  dw = sum over tokens of dy s q
// for channel-major prompts [batch][dim][L] and for rows [tokens][dim].
//
// Channel-major: a workgroup takes a tile, 128 (64) bytes of tokens of all channels.
// A lane holds 16 bytes of tokens of one channel, a wave 8 (16) channels; the
// sweeps' s stay in registers between the sum of squares and the scaling, so that
// every input is read once. Rows: a wave or a workgroup takes a row, in the same
// way.
//
// dw is summed in a fixed order: per tile of tokens (or per workgroup, which
// takes every n-th row) into the workspace, then over those in 64 bits.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "vimscan.h"
#include "vs_device.h"
#include "vs_model.h"

namespace {

// 16 bytes of consecutive entries, kept as loaded; rows start at any element
template <typename T>
struct Pack {
    static constexpr int N = 16 / static_cast<int>(sizeof(T));
    uint32_t v[4];
    __device__ __forceinline__ void load(const T* p) { __builtin_memcpy(v, p, 16); }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = 0;
    }
    // entries first .. first + N - 1 of a row of n, zeros past it
    __device__ __forceinline__ void load(const T* p, int first, int n) {
        if (first + N <= n) return load(p + first);
        zero();
#pragma unroll 1
        for (int i = n - 1; i >= first; --i) up(ld_raw(p, i));
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(T) == 2) return __uint_as_float(i & 1 ? v[i / 2] & 0xffff0000u : v[i / 2] << 16);
        else return __uint_as_float(v[i]);
    }
    // rounds to nearest even
    __device__ __forceinline__ void set(const float (&f)[N]) {
        if constexpr (sizeof(T) == 2) {
            typedef __bf16 Vec8 __attribute__((ext_vector_type(8)));
            const Vec8 b = {static_cast<__bf16>(f[0]), static_cast<__bf16>(f[1]), static_cast<__bf16>(f[2]), static_cast<__bf16>(f[3]),
                            static_cast<__bf16>(f[4]), static_cast<__bf16>(f[5]), static_cast<__bf16>(f[6]), static_cast<__bf16>(f[7])};
            __builtin_memcpy(v, &b, 16);
        } else {
            __builtin_memcpy(v, f, 16);
        }
    }
    template <bool FULL = false>
    __device__ __forceinline__ void store(T* p, int first, int n) const {
        if (FULL || first + N <= n) {
            __builtin_memcpy(p + first, v, 16);
        } else {
            Pack<T> o;
#pragma unroll
            for (int i = 0; i < 4; ++i) o.v[i] = v[i];
#pragma unroll 1
            for (int i = first; i < n; ++i) {
                if constexpr (sizeof(T) == 2) p[i] = static_cast<uint16_t>(o.v[0]);
                else p[i] = __uint_as_float(o.v[0]);
                o.down();
            }
        }
    }
    // all entries one place down, or up with one put in (as v_alignbyte: a shift
    // of 128 bits would go through scratch memory)
    __device__ __forceinline__ void down() {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t above = i < 3 ? v[i + 1] : 0u;
            v[i] = sizeof(T) == 2 ? __builtin_amdgcn_alignbyte(above, v[i], 2) : above;
        }
    }
    __device__ __forceinline__ void up(uint32_t in) {
#pragma unroll
        for (int i = 3; i >= 0; --i) {
            const uint32_t below = i > 0 ? v[i - 1] : sizeof(T) == 2 ? in << 16 : in;
            v[i] = sizeof(T) == 2 ? __builtin_amdgcn_alignbyte(v[i], below, 2) : below;
        }
    }
    // `places` down and zeros for all but the first `keep` entries
    __device__ __forceinline__ void cut(int places, int keep) {
#pragma unroll 1
        for (int i = 0; i < places && i < N; ++i) down();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 2) v[i] = keep >= 2 * i + 2 ? v[i] : keep == 2 * i + 1 ? v[i] & 0xffffu : 0u;
            else v[i] = keep > i ? v[i] : 0u;
        }
    }
    // opaque to the compiler from here on: it would keep the widened values, twice the registers
    __device__ __forceinline__ void settle() {
#pragma unroll
        for (int i = 0; i < 4; ++i) asm("" : "+v"(v[i]));
    }
};

// 1 / sqrt(v) by the hardware's approximation, off by one unit in the last place (an exact
// root and division would leave results off by 5.0e-8 instead of 6.0e-8 of their size).
// It takes subnormal numbers for zeros: they are scaled up first.
__device__ __forceinline__ float inverse_root(float v) {
    const bool low = v < 0x1p-100f;
    const float r = __builtin_amdgcn_rsqf(low ? v * 0x1p64f : v);
    return low ? r * 0x1p32f : r;
}

// weights first .. first + N - 1, ones without weights and past the last
template <int N>
__device__ __forceinline__ void weights(const float* w, int first, int n, float (&f)[N]) {
    if (w && first + N <= n) {
        __builtin_memcpy(f, w + first, sizeof(f));
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = w && first + i < n ? w[first + i] : 1.f;
    }
}

struct NormArgs {
    const void *x, *res, *dy, *dsum;        // gradient: x is s
    vs::Strides sx, sres, sdy, sdsum;
    const float* w;
    float eps, inv_dim;
    const int32_t* lengths;
    void *y, *sum;                          // gradient: y is ds
    float *part, *dw;
    int64_t rows;                           // the batch
    int dim, L, tiles;                      // tiles of a batch row
    int parts;
    int add;                                // dw already holds the sums of other rows
};

template <typename T>
__device__ __forceinline__ const T* at(const void* p, int64_t off) { return static_cast<const T*>(p) + off; }

// ------------------------------------------------------------ channel-major

// A lane's place in its workgroup's tile: N tokens from t on of one channel of
// each sweep of W waves. It loads 16 bytes from `from` on, which is t except where
// these would pass the row's end: there the entries are moved down afterwards,
// and entries at and past the row's length become zeros. None of that is asked
// for in a full tile, whose code is its own.
// TL lanes stand side by side along the tokens: a tile is TL times 16 bytes of each row.
template <typename T, int W, int TL>
struct Column {
    static constexpr int N = Pack<T>::N, kTl = TL, kCh = 64 / kTl, kTile = kTl * N;
    static constexpr int kSweep = kCh * W;              // channels of a sweep
    int lane, wave, t, from, ch, len, L;
    bool full, empty, few;   // the whole tile holds tokens, or none of it, or the row has at most N there (the same for the workgroup)
    int64_t b;
    uint32_t tile;
    // `tokens` of a tile, where that isn't this form's
    __device__ __forceinline__ explicit Column(const NormArgs& a, int tokens = kTile) {
        // neighbouring tiles share the lines at their border: contiguous ranges of tiles to each XCD
        uint32_t zero;
        xcd_block(tile, zero);
        b = tile / a.tiles;
        lane = threadIdx.x & 63;
        wave = threadIdx.x >> 6;
        const int t0 = static_cast<int>(tile - b * a.tiles) * tokens;
        L = a.L;
        t = t0 + lane % kTl * N;
        from = min(t, L - N);
        ch = wave * kCh + lane / kTl;
        len = a.lengths ? __builtin_amdgcn_readfirstlane(min(max(a.lengths[b], 0), L)) : L;
        full = t0 + tokens <= len;
        empty = t0 >= len;
        few = L - t0 <= N;
    }
    template <bool FULL>
    __device__ __forceinline__ void load(Pack<T>& p, const T* row) const {
        if (FULL) {
            p.load(row + t);
        } else if (TL > 1 || L >= N) {
            p.load(row + from);
        } else {             // rows shorter than a load have one tile, of few tokens
            p.zero();
#pragma unroll 1
            for (int i = len - 1; i >= t; --i) p.up(ld_raw(row, i));
        }
    }
    // what load() gave, made zero past the row's length
    template <bool FULL>
    __device__ __forceinline__ void trim(Pack<T>& p) const {
        if (!FULL) p.cut(TL > 1 || L >= N ? t - from : 0, len - t);
    }
    // a tile without tokens
    __device__ __forceinline__ void clear(T* out, int dim) const {
        Pack<T> none;
        none.zero();
        for (int c = ch; c < dim; c += kSweep) none.store(out + static_cast<int64_t>(c) * L, t, L);
    }
};

// A row's last tile of few tokens (one of 1,025 or 4,097) takes a channel a lane, in
// fewer sweeps: as wide as the others it is the last to end, for its sweeps wait
// for one another (bf16 training step of 8 x 768 x 4,097 126 -> 114 us). A lane's load
// holds 8 of them (fp32: 4), so more keep the wide form (forward pass of 8 x 768 with a residual,
// inputs in the last-level cache: 4,096 tokens 34.8 us, 4,097 38.9, 4,104 38.2, 4,105
// 49.8, 4,128 46.0).
template <int HOLD, int TL>
constexpr int kFew = (HOLD + TL - 1) / TL;

// sums over the workgroup's channels of each lane's tokens
template <typename T, int W, int TL>
__device__ __forceinline__ void column_sum(const Column<T, W, TL>& c, float (&v)[Pack<T>::N], float* red) {
    constexpr int N = Pack<T>::N, kTl = TL;
#pragma unroll
    for (int o = kTl; o < 64; o *= 2)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor(v[i], o, 64);
    if (c.lane < kTl) {
#pragma unroll
        for (int i = 0; i < N; ++i) red[(c.wave * kTl + c.lane) * N + i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.f;
#pragma unroll 4                        // of all waves' lines at once, the reads would take 128 registers
    for (int o = 0; o < W; ++o)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += red[(o * kTl + c.lane % kTl) * N + i];
}

template <typename T, int W, int HOLD, bool ADD, bool FULL, bool REST, int TL>
__device__ __forceinline__ void norm_column(const NormArgs& a, const Column<T, W, TL>& c, float* red) {
    constexpr int N = Pack<T>::N;
    const T* x = at<T>(a.x, c.b * a.sx.b);
    const T* res = ADD ? at<T>(a.res, c.b * a.sres.b) : nullptr;
    const int64_t base = c.b * a.dim * static_cast<int64_t>(a.L);
    T *y = static_cast<T*>(a.y) + base, *sum = ADD ? static_cast<T*>(a.sum) + base : nullptr;
    Pack<T> held[HOLD], r[HOLD];
    float ss[N], hw[HOLD];
#pragma unroll
    for (int i = 0; i < N; ++i) ss[i] = 0.f;
    // the loads of all sweeps are in flight before the first is waited for
    auto read = [&](int ch, Pack<T>& s, Pack<T>& r) VS_INLINE {
        c.template load<FULL>(s, x + ch * a.sx.d);
        if constexpr (ADD) c.template load<FULL>(r, res + ch * a.sres.d);
    };
    auto take = [&](int ch, Pack<T>& s, Pack<T>& r) VS_INLINE {
        c.template trim<FULL>(s);
        if constexpr (ADD) {
            c.template trim<FULL>(r);
            float f[N];
#pragma unroll
            for (int i = 0; i < N; ++i) f[i] = s.get(i) + r.get(i);
            s.set(f);
            s.template store<FULL>(sum + static_cast<int64_t>(ch) * a.L, c.t, a.L);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) ss[i] = fmaf(s.get(i), s.get(i), ss[i]);
        s.settle();
    };
#pragma unroll
    for (int k = 0; k < HOLD; ++k) {
        const int ch = c.ch + k * (Column<T, W, TL>::kSweep);
        hw[k] = a.w && ch < a.dim ? a.w[ch] : 1.f;
        if (ch < a.dim) read(ch, held[k], r[k]);
    }
#pragma unroll
    for (int k = 0; k < HOLD; ++k) {
        const int ch = c.ch + k * (Column<T, W, TL>::kSweep);
        if (ch < a.dim) take(ch, held[k], r[k]);
    }
    for (int ch = c.ch + HOLD * (Column<T, W, TL>::kSweep); REST && ch < a.dim; ch += (Column<T, W, TL>::kSweep)) {
        Pack<T> s, q;
        read(ch, s, q);
        take(ch, s, q);
    }
    column_sum(c, ss, red);
    float q[N];
#pragma unroll
    for (int i = 0; i < N; ++i) q[i] = inverse_root(fmaf(ss[i], a.inv_dim, a.eps));
    auto put = [&](int ch, float w, const Pack<T>& s) VS_INLINE {
        float f[N];
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = FULL || c.t + i < c.len ? s.get(i) * q[i] * w : 0.f;
        Pack<T> o;
        o.set(f);
        o.template store<FULL>(y + static_cast<int64_t>(ch) * a.L, c.t, a.L);
    };
#pragma unroll
    for (int k = 0; k < HOLD; ++k) {
        const int ch = c.ch + k * (Column<T, W, TL>::kSweep);
        if (ch < a.dim) put(ch, hw[k], held[k]);
    }
    // channels past what is held: read again (the lane's own entries of the sum, or x)
    for (int ch = c.ch + HOLD * (Column<T, W, TL>::kSweep); REST && ch < a.dim; ch += (Column<T, W, TL>::kSweep)) {
        Pack<T> s;
        if constexpr (ADD) {
            s.load(sum + static_cast<int64_t>(ch) * a.L, c.t, a.L);
        } else {
            c.template load<FULL>(s, x + ch * a.sx.d);
            c.template trim<FULL>(s);
        }
        put(ch, a.w ? a.w[ch] : 1.f, s);
    }
}

// Bound by memory: 8 x 768 x 4,097 bf16 with a residual, four streams of 50 MB, 44.3
// us, 4.5 TB/s
template <typename T, int W, int HOLD, bool ADD, int TL>
__global__ __launch_bounds__(64 * W) void norm_column_kernel(const NormArgs a) {
    typedef Column<T, W, TL> Col;
    constexpr bool kRest = TL == 4;                  // else all channels are held
    __shared__ float red[W * Col::kTile];
    const Col c(a);
    if (c.full) {
        norm_column<T, W, HOLD, ADD, true, kRest>(a, c, red);
    } else if (c.empty) {
        const int64_t base = c.b * a.dim * static_cast<int64_t>(a.L);
        c.clear(static_cast<T*>(a.y) + base, a.dim);
        if constexpr (ADD) c.clear(static_cast<T*>(a.sum) + base, a.dim);
    } else if (c.few) {
        norm_column<T, W, kFew<HOLD, TL>, ADD, false, kRest>(a, Column<T, W, 1>(a, Col::kTile), red);
    } else {
        norm_column<T, W, HOLD, ADD, false, kRest>(a, c, red);
    }
}

template <typename T, int W, int HOLD, bool FULL, bool REST, int TL>
__device__ __forceinline__ void norm_column_grad(const NormArgs& a, const Column<T, W, TL>& c, float* red, uint4 (*held)[64 * W]) {
    constexpr int N = Pack<T>::N, kTl = TL;
    const T *s = at<T>(a.x, c.b * a.sx.b), *dy = at<T>(a.dy, c.b * a.sdy.b);
    const T* dsum = a.dsum ? at<T>(a.dsum, c.b * a.sdsum.b) : nullptr;
    T* ds = static_cast<T*>(a.y) + c.b * a.dim * static_cast<int64_t>(a.L);
    float* part = a.part ? a.part + static_cast<size_t>(c.tile) * a.dim : nullptr;
    Pack<T> hs[HOLD];
    float ss[N], sd[N];
#pragma unroll
    for (int i = 0; i < N; ++i) ss[i] = sd[i] = 0.f;
    auto read = [&](int ch, Pack<T>& ps, Pack<T>& py) VS_INLINE {
        c.template load<FULL>(ps, s + ch * a.sx.d);
        c.template load<FULL>(py, dy + ch * a.sdy.d);
    };
    auto take = [&](int ch, Pack<T>& ps, Pack<T>& py) VS_INLINE {
        c.template trim<FULL>(ps);
        c.template trim<FULL>(py);
        const float w = a.w ? a.w[ch] : 1.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            ss[i] = fmaf(ps.get(i), ps.get(i), ss[i]);
            sd[i] = fmaf(w * py.get(i), ps.get(i), sd[i]);
        }
    };
    {
        // two sweeps ahead: asked for all at once, the loads of a unit's two
        // workgroups come in one burst (bf16 8 x 768 x 4,097 training step, before
        // the last tile's own form: 131 us, three ahead 126.5, two 126.1)
        Pack<T> hy[2];
#pragma unroll
        for (int k = 0; k < 2 && k < HOLD; ++k) {
            const int ch = c.ch + k * (Column<T, W, TL>::kSweep);
            if (ch < a.dim) read(ch, hs[k], hy[k]);
        }
#pragma unroll
        for (int k = 0; k < HOLD; ++k) {
            const int ch = c.ch + k * (Column<T, W, TL>::kSweep), next = ch + 2 * (Column<T, W, TL>::kSweep);
            Pack<T>& py = hy[k % 2];
            if (ch < a.dim) take(ch, hs[k], py);
            hs[k].settle();
            held[k][threadIdx.x] = uint4{py.v[0], py.v[1], py.v[2], py.v[3]};
            if (k + 2 < HOLD && next < a.dim) read(next, hs[k + 2], py);
        }
    }
    for (int ch = c.ch + HOLD * (Column<T, W, TL>::kSweep); REST && ch < a.dim; ch += (Column<T, W, TL>::kSweep)) {
        Pack<T> ps, py;
        read(ch, ps, py);
        take(ch, ps, py);
    }
    auto more = [&](int ch, Pack<T>& g) VS_INLINE {
        if (dsum) c.template load<FULL>(g, dsum + ch * a.sdsum.d);
    };
    // dsum two sweeps ahead: its first loads are on their way while the waves meet,
    // and none stands behind a sweep's stores (8 x 768 x 4,097: 108 -> 106 us a step)
    Pack<T> hg[2];
#pragma unroll
    for (int k = 0; k < 2 && k < HOLD; ++k) {
        const int ch = c.ch + k * (Column<T, W, TL>::kSweep);
        if (ch < a.dim) more(ch, hg[k]);
    }
    column_sum(c, ss, red);
    column_sum(c, sd, red + W * Column<T, W, TL>::kTile);
    float q[N], m[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        q[i] = inverse_root(fmaf(ss[i], a.inv_dim, a.eps));
        m[i] = q[i] * (sd[i] * a.inv_dim);
    }
    auto put = [&](int ch, const Pack<T>& ps, const Pack<T>& py, Pack<T>& g) VS_INLINE {
        const float w = a.w ? a.w[ch] : 1.f;
        if (dsum) c.template trim<FULL>(g);
        float f[N], dw = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            // by the normed value u: the square of q alone may be infinite
            const float u = ps.get(i) * q[i], yv = py.get(i);
            const float d = q[i] * (w * yv - u * m[i]);
            const bool on = FULL || c.t + i < c.len;
            f[i] = on ? (dsum ? g.get(i) + d : d) : 0.f;
            dw = on ? fmaf(yv, u, dw) : dw;
        }
        Pack<T> o;
        o.set(f);
        o.template store<FULL>(ds + static_cast<int64_t>(ch) * a.L, c.t, a.L);
        if (part) {
#pragma unroll
            for (int o2 = 1; o2 < kTl; o2 *= 2) dw += __shfl_xor(dw, o2, 64);
            if (c.lane % kTl == 0) part[ch] = dw;
        }
    };
#pragma unroll
    for (int k = 0; k < HOLD; ++k) {
        const int ch = c.ch + k * (Column<T, W, TL>::kSweep);
        const uint4 y = held[k][threadIdx.x];
        Pack<T> py;
        py.v[0] = y.x; py.v[1] = y.y; py.v[2] = y.z; py.v[3] = y.w;
        const int next = ch + 2 * (Column<T, W, TL>::kSweep);
        if (ch < a.dim) put(ch, hs[k], py, hg[k % 2]);
        if (k + 2 < HOLD && next < a.dim) more(next, hg[k % 2]);
    }
    for (int ch = c.ch + HOLD * (Column<T, W, TL>::kSweep); REST && ch < a.dim; ch += (Column<T, W, TL>::kSweep)) {
        Pack<T> ps, py, g;
        read(ch, ps, py);
        more(ch, g);
        c.template trim<FULL>(ps);
        c.template trim<FULL>(py);
        put(ch, ps, py, g);
    }
}

// Three streams read and one written, at 768 channels in pieces of 64 bytes: 57 us,
// 3.5 TB/s
template <typename T, int W, int HOLD, int TL>
__global__ __launch_bounds__(64 * W, HOLD > 6 ? 2 : 4) void norm_column_grad_kernel(const NormArgs a) {
    typedef Column<T, W, TL> Col;
    constexpr bool kRest = TL == 4 && HOLD > 6;      // else all channels are held
    __shared__ float red[2 * W * Col::kTile];
    // dy is held in LDS: in registers, s and dy together leave a compute unit one
    // workgroup, whose loads and stores then take turns
    __shared__ uint4 held[HOLD][64 * W];
    const Col c(a);
    if (c.full) {
        norm_column_grad<T, W, HOLD, true, kRest>(a, c, red, held);
    } else if (c.empty) {
        c.clear(static_cast<T*>(a.y) + c.b * a.dim * static_cast<int64_t>(a.L), a.dim);
        if (a.part)
            for (int ch = threadIdx.x; ch < a.dim; ch += 64 * W) a.part[static_cast<size_t>(c.tile) * a.dim + ch] = 0.f;
    } else if (c.few) {
        norm_column_grad<T, W, kFew<HOLD, TL>, false, kRest>(a, Column<T, W, 1>(a, Col::kTile), red, held);
    } else {
        norm_column_grad<T, W, HOLD, false, kRest>(a, c, red, held);
    }
}

// -------------------------------------------------------------------- rows
// W waves a row; one-wave rows stand four to a workgroup
template <int W>
struct RowOf {
    int lane, wave, tid;
    __device__ __forceinline__ RowOf() {
        lane = threadIdx.x & 63;
        wave = threadIdx.x >> 6;
        tid = W == 1 ? lane : static_cast<int>(threadIdx.x);
    }
    __device__ __forceinline__ float sum(float v, float* red) const {
#pragma unroll
        for (int o = 1; o < 64; o *= 2) v += __shfl_xor(v, o, 64);
        if constexpr (W > 1) {
            if (lane == 0) red[wave] = v;
            __syncthreads();
            v = 0.f;
#pragma unroll
            for (int o = 0; o < W; ++o) v += red[o];
        }
        return v;
    }
    // two at once, with one barrier (gradient of fp32 rows, 8,194 x 1,536: 118 -> 110 us a step)
    __device__ __forceinline__ void sums(float& v, float& u, float (*red)[2]) const {
#pragma unroll
        for (int o = 1; o < 64; o *= 2) {
            v += __shfl_xor(v, o, 64);
            u += __shfl_xor(u, o, 64);
        }
        if constexpr (W > 1) {
            if (lane == 0) { red[wave][0] = v; red[wave][1] = u; }
            __syncthreads();
            v = u = 0.f;
#pragma unroll
            for (int o = 0; o < W; ++o) { v += red[o][0]; u += red[o][1]; }
        }
    }
};

// Bound by memory (8,194 x 1,536 bf16: 50 MB in 10.3 us), 64 rows by the launch (3 us)
template <typename T, int W, int HOLD, bool ADD>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W) void norm_row_kernel(const NormArgs a) {
    constexpr int N = Pack<T>::N, kStep = 64 * W * N;
    __shared__ float red[W];
    const RowOf<W> r;
    const int64_t b = W == 1 ? static_cast<int64_t>(blockIdx.x) * 4 + r.wave : blockIdx.x;
    if (W == 1 && b >= a.rows) return;
    const int n = a.lengths && a.lengths[b] < 1 ? 0 : a.dim;          // an empty row reads nothing
    const T* x = at<T>(a.x, b * a.sx.b);
    const T* res = ADD ? at<T>(a.res, b * a.sres.b) : nullptr;
    T *y = static_cast<T*>(a.y) + b * a.dim, *sum = ADD ? static_cast<T*>(a.sum) + b * a.dim : nullptr;
    Pack<T> s[HOLD];
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < HOLD; ++k) {
        const int i0 = k * kStep + r.tid * N;
        if (i0 >= a.dim) continue;
        s[k].load(x, i0, n);
        if constexpr (ADD) {
            Pack<T> o;
            o.load(res, i0, n);
            float f[N];
#pragma unroll
            for (int i = 0; i < N; ++i) f[i] = s[k].get(i) + o.get(i);
            s[k].set(f);
            s[k].store(sum, i0, a.dim);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) ss = fmaf(s[k].get(i), s[k].get(i), ss);
    }
    const float q = inverse_root(fmaf(r.sum(ss, red), a.inv_dim, a.eps));
#pragma unroll
    for (int k = 0; k < HOLD; ++k) {
        const int i0 = k * kStep + r.tid * N;
        if (i0 >= a.dim) continue;
        float f[N], w[N];
        weights(a.w, i0, a.dim, w);
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = n ? s[k].get(i) * q * w[i] : 0.f;
        s[k].set(f);
        s[k].store(y, i0, a.dim);
    }
}

// Every gridDim.x-th row (or four of them), the sums of dw in registers: 8,194 x
// 1,536 bf16 22.7 us, 75 MB (14.7 us of them) and the workgroups' lines of dw, 6 MB. A
// row that leaves lanes of its waves empty waits for its loads and barriers instead:
// fp32 8,194 x 1,536, where 384 of 1,024 lanes hold anything, 72 us for 151 MB.
template <typename T, int W, int HOLD>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W) void norm_row_grad_kernel(const NormArgs a) {
    constexpr int N = Pack<T>::N, kStep = 64 * W * N;
    __shared__ float red[2][W][2];
    const RowOf<W> r;
    float dw[HOLD][N], before[HOLD][N];
#pragma unroll
    for (int k = 0; k < HOLD; ++k)
#pragma unroll
        for (int i = 0; i < N; ++i) dw[k][i] = before[k][i] = 0.f;
    const int64_t first = W == 1 ? static_cast<int64_t>(blockIdx.x) * 4 + r.wave : blockIdx.x;
    const int64_t step = static_cast<int64_t>(gridDim.x) * (W == 1 ? 4 : 1);
    // the next row is read while this one is worked on
    Pack<T> ps[HOLD], py[HOLD], pg[HOLD];
    int n = 0;
    auto read = [&](int64_t b) VS_INLINE {
        n = a.lengths && a.lengths[b] < 1 ? 0 : a.dim;                // an empty row reads nothing
        const T *s = at<T>(a.x, b * a.sx.b), *dy = at<T>(a.dy, b * a.sdy.b);
        const T* dsum = a.dsum ? at<T>(a.dsum, b * a.sdsum.b) : nullptr;
#pragma unroll
        for (int k = 0; k < HOLD; ++k) {
            const int i0 = k * kStep + r.tid * N;
            ps[k].load(s, i0, n);
            py[k].load(dy, i0, n);
            if (dsum) pg[k].load(dsum, i0, n);
        }
    };
    if (first < a.rows) read(first);
    int odd = 0, left = 64;
    for (int64_t b = first; b < a.rows; b += step, odd ^= 1) {
        T* ds = static_cast<T*>(a.y) + b * a.dim;
        const bool real = n != 0;
        Pack<T> hs[HOLD], hy[HOLD], hg[HOLD];
        float ss = 0.f, sd = 0.f;
#pragma unroll
        for (int k = 0; k < HOLD; ++k) {
            hs[k] = ps[k];
            hy[k] = py[k];
            hg[k] = pg[k];
            hs[k].settle();
            hy[k].settle();
        }
        if (b + step < a.rows) read(b + step);
#pragma unroll
        for (int k = 0; k < HOLD; ++k) {
            float w[N];
            weights(a.w, k * kStep + r.tid * N, a.dim, w);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                ss = fmaf(hs[k].get(i), hs[k].get(i), ss);
                sd = fmaf(w[i] * hy[k].get(i), hs[k].get(i), sd);
            }
        }
        r.sums(ss, sd, red[odd]);
        const float q = inverse_root(fmaf(ss, a.inv_dim, a.eps)), m = q * (sd * a.inv_dim);
#pragma unroll
        for (int k = 0; k < HOLD; ++k) {
            const int i0 = k * kStep + r.tid * N;
            if (i0 >= a.dim) continue;
            float f[N], w[N];
            weights(a.w, i0, a.dim, w);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float u = hs[k].get(i) * q, yv = hy[k].get(i);
                const float d = q * (w[i] * yv - u * m);
                f[i] = real ? (a.dsum ? hg[k].get(i) + d : d) : 0.f;
                if (real) dw[k][i] = fmaf(yv, u, dw[k][i]);
            }
            Pack<T> o;
            o.set(f);
            o.store(ds, i0, a.dim);
        }
        // 64 rows at a time: a lane may take 16,384, whose terms one after another
        // would be off by 1.7e-4 of their sum
        if (--left == 0) {
            left = 64;
#pragma unroll
            for (int k = 0; k < HOLD; ++k)
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    before[k][i] += dw[k][i];
                    dw[k][i] = 0.f;
                }
        }
    }
    if (!a.part) return;
    float* part = a.part + static_cast<size_t>(W == 1 ? blockIdx.x * 4 + r.wave : blockIdx.x) * a.dim;
#pragma unroll
    for (int k = 0; k < HOLD; ++k)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int at_ = k * kStep + r.tid * N + i;
            if (at_ < a.dim) part[at_] = before[k][i] + dw[k][i];
        }
}

// dw from the parts: 16 channels a workgroup, 64 lines of parts side by side. In 64
// bits: a call may have 4 million parts, 65,536 for each thread, whose sum in 32 would
// be off by 7e-4 where they agree in sign. 5 us for 1,032 parts of 768 channels, a
// chain of reads; few channels with many parts leave most compute units idle.
constexpr int kDwCh = 16, kDwLines = 64;
__global__ __launch_bounds__(kDwCh* kDwLines) void norm_dw_kernel(const NormArgs a) {
    __shared__ double red[kDwLines][kDwCh + 1];
    const int ch = blockIdx.x * kDwCh + threadIdx.x % kDwCh, line = threadIdx.x / kDwCh;
    double s = 0;
    if (ch < a.dim)
#pragma unroll 8
        for (int p = line; p < a.parts; p += kDwLines) s += a.part[static_cast<size_t>(p) * a.dim + ch];
    red[line][threadIdx.x % kDwCh] = s;
    __syncthreads();
    if (threadIdx.x < kDwCh && ch < a.dim) {
        s = a.add ? a.dw[ch] : 0.f;
        for (int o = 0; o < kDwLines; ++o) s += red[o][threadIdx.x];
        a.dw[ch] = static_cast<float>(s);
    }
}

// ------------------------------------------------------------------ launch
template <typename T>
constexpr int kRowHold = static_cast<int>(vs::kNormMaxDim) / (1024 * Pack<T>::N);   // the longest rows, in 16 waves

template <typename T, bool ADD>
void launch_rows(const NormArgs& a, const vs::NormCall& c, hipStream_t s) {
    const dim3 four(static_cast<uint32_t>((c.batch + 3) / 4)), one(static_cast<uint32_t>(c.batch));
    switch (c.form) {
        case vs::kNormRow1: norm_row_kernel<T, 1, 1, ADD><<<four, 256, 0, s>>>(a); break;
        case vs::kNormRow4: norm_row_kernel<T, 4, 1, ADD><<<one, 256, 0, s>>>(a); break;
        default: norm_row_kernel<T, 16, kRowHold<T>, ADD><<<one, 1024, 0, s>>>(a); break;
    }
}
// the sweeps that are held: as few as the channels need
template <typename T, bool ADD, int TL, int W, int HOLD, int... MORE>
void launch_column(const NormArgs& a, uint32_t tiles, hipStream_t s) {
    if constexpr (sizeof...(MORE) > 0)
        if (a.dim > HOLD * Column<T, W, TL>::kSweep) return launch_column<T, ADD, TL, W, MORE...>(a, tiles, s);
    norm_column_kernel<T, W, HOLD, ADD, TL><<<tiles, 64 * W, 0, s>>>(a);
}
template <typename T, bool ADD>
void launch_columns(const NormArgs& a, const vs::NormCall& c, hipStream_t s) {
    const uint32_t tiles = static_cast<uint32_t>(c.batch * a.tiles);
    // Sixteen waves, each with half the sweeps: with at most two workgroups for a
    // compute unit they halve what each wave waits for (fp32 8 x 384 x 1,025:
    // 12.6 -> 10.9 us), and past six sweeps of eight waves these would leave a unit
    // one workgroup (fp32 8 x 768 x 4,097 44.8 -> 39.7 us, bf16 4 x 1,536 x 4,097
    // with a residual 60.6 -> 58.7).
    if (c.tile != vs::kNormWide / static_cast<int>(sizeof(T))) launch_column<T, ADD, 4, 16, 6>(a, tiles, s);
    else if (tiles <= 512 || a.dim > 6 * Column<T, 8, 8>::kSweep) launch_column<T, ADD, 8, 16, 1, 3, 6>(a, tiles, s);
    else launch_column<T, ADD, 8, 8, 2, 6>(a, tiles, s);
}
template <typename T, int TL, int W, int HOLD, int... MORE>
void launch_column_grad(const NormArgs& a, uint32_t tiles, hipStream_t s) {
    if constexpr (sizeof...(MORE) > 0)
        if (a.dim > HOLD * Column<T, W, TL>::kSweep) return launch_column_grad<T, TL, W, MORE...>(a, tiles, s);
    norm_column_grad_kernel<T, W, HOLD, TL><<<tiles, 64 * W, 0, s>>>(a);
}
void launch_dw(const NormArgs& a, hipStream_t s) {
    if (a.dw) norm_dw_kernel<<<dim3((a.dim + kDwCh - 1) / kDwCh), kDwCh * kDwLines, 0, s>>>(a);
}
template <typename T>
void launch_grad(const NormArgs& a, const vs::NormCall& c, hipStream_t s) {
    if (c.form == vs::kNormColumn) {
        // the batch rows whose lines of dw the workspace holds, one such slab after another
        for (int64_t b = 0; b < c.batch; b += c.slab) {
            const int64_t rows = c.batch - b < c.slab ? c.batch - b : c.slab;
            NormArgs p = a;
            p.x = static_cast<const T*>(a.x) + b * a.sx.b;
            p.dy = static_cast<const T*>(a.dy) + b * a.sdy.b;
            if (a.dsum) p.dsum = static_cast<const T*>(a.dsum) + b * a.sdsum.b;
            if (a.lengths) p.lengths = a.lengths + b;
            p.y = static_cast<T*>(a.y) + b * a.dim * a.L;
            p.rows = rows;
            p.add = b > 0;
            const uint32_t tiles = static_cast<uint32_t>(rows * a.tiles);
            p.parts = static_cast<int>(tiles);
            if (c.tile == vs::kNormWide / static_cast<int>(sizeof(T))) launch_column_grad<T, 8, 8, 2, 6>(p, tiles, s);
            else launch_column_grad<T, 4, 8, 6, 12>(p, tiles, s);
            launch_dw(p, s);
        }
    } else {
        const dim3 grid(static_cast<uint32_t>(c.form == vs::kNormRow1 ? a.parts / 4 : a.parts));
        switch (c.form) {
            case vs::kNormRow1: norm_row_grad_kernel<T, 1, 1><<<grid, 256, 0, s>>>(a); break;
            case vs::kNormRow4: norm_row_grad_kernel<T, 4, 1><<<grid, 256, 0, s>>>(a); break;
            default: norm_row_grad_kernel<T, 16, kRowHold<T>><<<grid, 1024, 0, s>>>(a); break;
        }
        launch_dw(a, s);
    }
}

int run(vs::NormCall& c) {
    if (int rc = vs::prepare_norm(c)) return rc;
    NormArgs a{};
    a.x = c.x; a.res = c.residual; a.dy = c.dy; a.dsum = c.dsum;
    a.sx = c.st[0]; a.sres = c.st[1]; a.sdy = c.st[1]; a.sdsum = c.st[2];
    a.w = c.w; a.eps = c.eps; a.inv_dim = 1.f / static_cast<float>(c.dim); a.lengths = c.lengths;
    a.y = c.y; a.sum = c.sum; a.part = c.dw ? static_cast<float*>(c.ws) : nullptr; a.dw = c.dw;
    a.rows = c.batch; a.dim = static_cast<int>(c.dim); a.L = static_cast<int>(c.L);
    a.tiles = static_cast<int>((c.L + c.tile - 1) / c.tile);
    a.parts = static_cast<int>(c.parts);
    const auto s = static_cast<hipStream_t>(c.stream);
    const bool bf16 = c.dtype == VS_BF16;
    if (c.grad) {
        if (bf16) launch_grad<uint16_t>(a, c, s);
        else launch_grad<float>(a, c, s);
    } else if (c.form == vs::kNormColumn) {
        if (bf16) c.residual ? launch_columns<uint16_t, true>(a, c, s) : launch_columns<uint16_t, false>(a, c, s);
        else c.residual ? launch_columns<float, true>(a, c, s) : launch_columns<float, false>(a, c, s);
    } else {
        if (bf16) c.residual ? launch_rows<uint16_t, true>(a, c, s) : launch_rows<uint16_t, false>(a, c, s);
        else c.residual ? launch_rows<float, true>(a, c, s) : launch_rows<float, false>(a, c, s);
    }
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? VS_OK : vs::fail(VS_ERR_HIP, std::string("kernel launch: ") + hipGetErrorString(e));
}

}  // namespace

extern "C" {

int rms_norm(int64_t batch, int64_t dim, int64_t seqlen, int dtype, const void* x, const void* residual,
             const int64_t* strides, const float* w, float eps, const int32_t* lengths, void* y, void* sum,
             void* stream) {
    vs::NormCall c{};
    c.batch = batch; c.dim = dim; c.L = seqlen; c.dtype = dtype; c.x = x; c.residual = residual; c.strides = strides;
    c.w = w; c.eps = eps; c.lengths = lengths; c.y = y; c.sum = sum; c.stream = stream;
    return run(c);
}

int rms_norm_grad(int64_t batch, int64_t dim, int64_t seqlen, int dtype, const void* s, const void* dy,
                  const void* dsum, const int64_t* strides, const float* w, float eps, const int32_t* lengths,
                  void* ds, float* dw, void* workspace, size_t workspace_bytes, void* stream) {
    vs::NormCall c{};
    c.batch = batch; c.dim = dim; c.L = seqlen; c.dtype = dtype; c.x = s; c.dy = dy; c.dsum = dsum; c.strides = strides;
    c.w = w; c.eps = eps; c.lengths = lengths; c.y = ds; c.dw = dw; c.ws = workspace; c.ws_bytes = workspace_bytes;
    c.stream = stream; c.grad = true;
    return run(c);
}

}  // extern "C"
