// vocab.hip -- softmax cross entropy of a linear head over a large vocabulary,
// without keeping the logits, and its gradient: with l = x W^T,
//     lse_t = log sum_v exp(l_tv),  loss_t = lse_t - l_t,target(t)
//     P_tv = (exp(l_tv - lse_t) - [v = target(t)]) dloss_t
//     dx = P W,  dW = P^T x.
//
// Three matrix products share one kernel body (matrix cores, 32 x 32 tiles,
// fp32 accumulation). It computes out[n][m] = sum_k A(m, k) B(n, k), so that a
// lane's accumulators are 16 rows m of one column n:
//   logits  m a vocabulary entry, n a token: a token's maximum and its sum of
//           exponentials are taken inside the lane, and its row of P is
//           written in runs of four entries
//   dx      m a channel, n a token, k the vocabulary
//   dW      m a channel, n a vocabulary entry, k the tokens
// An operand lies in memory with its k side by side (x and W for the logits, P
// for dx) or with its rows side by side (W for dx, x and P for dW). Both are
// copied to LDS as they lie, 128 bytes of k a stage, straight from the buffer
// without a register; the second kind is turned on the way from LDS to the
// registers (ds_read_b64_tr_b16, or single words in fp32), so nothing is
// transposed in memory.
//
// The forward pass leaves a maximum and a sum for each token and tile of the
// vocabulary, 8 bytes for 256 logits. The gradient takes the vocabulary in
// pieces: logits again, P of the piece into the workspace, then both products
// that read it. P is held in the operands' type, as the matrix cores take it. In bf16
// its entries are off by half a step, at random, which a sum of many averages out; but
// a token's largest is its target's, -dloss less a little, so what rounding took
// off that one is kept in fp32 and added to both products.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "vimscan.h"
#include "vs_device.h"
#include "vs_model.h"

namespace {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(16))) float f32x16;
typedef __attribute__((ext_vector_type(4))) short v4s;
typedef __attribute__((ext_vector_type(8))) short v8s;
typedef __attribute__((address_space(3))) void lds_void;

constexpr int kStage = vs::kVocabStage;          // bytes of k a stage

enum Epilogue { kLse, kProb, kSum };

struct GemmArgs {
    const void *A, *B;
    int64_t lda, ldb;               // elements
    int M, N, K;
    int tiles_m, tiles_n;
    int k_split;                    // k of one split (a multiple of a stage's)
    // logits, dx
    const void* target;
    int target64;
    int v0, vocab;                  // the vocabulary entry of m = 0; entries in all
    float *part_max, *part_sum, *target_logit;      // kLse: [tiles_m][N], [N]
    const float *lse, *dloss;       // kProb
    void* P;                        // [N][ldp]
    int ldp;
    float* rest;                    // bf16: what rounding took off the targets' entries of P, [tokens]; a product that has it adds it
    const void* rows;               // dx: W from entry 0
    // kSum: sum[n][m] = (add ? sum : 0) + product, or out in the operands' type
    void* out;
    int64_t ldo;
    float* sum;                     // [N][M], or one for each split
    int add;
};

template <typename T>
struct Types;
template <>
struct Types<uint16_t> {
    typedef bf16x8 Frag;
    static __device__ __forceinline__ void mma(const Frag& a, const Frag& b, f32x16& c) {
        c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
};
template <>
struct Types<float> {
    typedef f32x4 Frag;
    // lane half h holds k = 4 h .. 4 h + 3 of the step's eight: each instruction takes one of both halves
    static __device__ __forceinline__ void mma(const Frag& a, const Frag& b, f32x16& c) {
#pragma unroll
        for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[j], b[j], c, 0, 0, 0);
    }
};

// One operand's tile: R rows of a stage. The 16-byte chunks of a line of LDS
// are permuted so that the fragment reads fall on distinct banks; a chunk's
// place is chosen by the address that its lane reads from.
template <typename T, bool OUTER, int R, int WAVES>
struct Operand {
    static constexpr int kEs = sizeof(T), kBk = kStage / kEs, kBytes = R * kStage;
    static constexpr int kLine = OUTER ? R * kEs : kStage;          // bytes of a line of LDS
    static constexpr int kLanes = kLine / 16;                       // lanes to a line
    static constexpr int kLines = 64 / kLanes;                      // lines of one instruction
    static constexpr int kIters = kBytes / 1024 / WAVES;
    static_assert(kLanes <= 64 && kIters >= 1 && kBytes % (1024 * WAVES) == 0, "whole instructions");
    static_assert(WAVES % 4 == 0, "a lane's chunk is the same in every instruction");

    const char* base;
    int64_t ld;              // bytes
    int64_t bytes;           // from base to the operand's end
    uint32_t off;            // this lane's first chunk
    int wave;
    // fragment reads
    uint32_t at[4];

    static __device__ __forceinline__ int turn(int line) {
        if constexpr (!OUTER) return (line >> 1) & 7;
        else if constexpr (kEs == 2) return 4 * (line & 3);
        else return 8 * ((line >> 2) & 1);
    }
    // The range check goes by words: one that an odd row's end shares with what
    // follows counts as part of the operand (only packed rows and P's are odd:
    // they are padded).
    static __device__ __forceinline__ int64_t whole(int64_t bytes) { return (bytes + 3) & ~int64_t(3); }
    // rows from `first` on of an operand with `rows` of them and K in all
    __device__ __forceinline__ void open(const void* p, int64_t ld_, int first, int rows, int K, int lane, int wave_) {
        ld = ld_ * kEs;
        wave = wave_;
        const int line = wave * kLines + lane / kLanes, chunk = lane % kLanes ^ turn(line);
        if constexpr (OUTER) {
            base = static_cast<const char*>(p) + static_cast<int64_t>(first) * kEs;
            bytes = (K - 1) * ld + whole(static_cast<int64_t>(rows - first) * kEs);
        } else {
            base = static_cast<const char*>(p) + first * ld;
            bytes = (rows - first - 1) * ld + whole(static_cast<int64_t>(K) * kEs);
        }
        off = static_cast<uint32_t>(line * ld) + chunk * 16;
    }
    // the stage from k on; reads past the operand's end return zeros
    __device__ __forceinline__ void load(char* lds, int k) const {
        const int64_t skip = OUTER ? k * ld : static_cast<int64_t>(k) * kEs;
        const int64_t left = bytes - skip;
        const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base + skip), 0,
                                                            static_cast<int>(left < 0x7fffffff ? (left > 0 ? left : 0) : 0x7fffffff), 0x00020000);
#pragma unroll
        for (int i = 0; i < kIters; ++i)
            // all of the offset in the lane's part, which the range check goes by
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void*)(lds + (i * WAVES + wave) * 1024), 16,
                                                     static_cast<int>(off + static_cast<uint32_t>(i * WAVES * kLines * ld)), 0, 0, 0);
    }
    // where entry `at` of a line of LDS stands
    static __device__ __forceinline__ int place(int line, int at) { return line * kLine + ((at * kEs / 16) ^ turn(line)) * 16 + at * kEs % 16; }
    // a stage of rows from k on, those of list[0..n-1] (its low 16 bits, from k); zeros behind them
    __device__ __forceinline__ void pick(char* lds, int k, const int* list, int n, int lane) const {
        static_assert(OUTER, "a row of the operand is a line");
        const int64_t left = bytes - k * ld;
        const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base + k * ld), 0,
                                                            static_cast<int>(left < 0x7fffffff ? left : 0x7fffffff), 0x00020000);
#pragma unroll
        for (int i = 0; i < kIters; ++i) {
            const int line = (i * WAVES + wave) * kLines + lane / kLanes;
            const uint32_t at_ = line < n ? static_cast<uint32_t>((list[line] & 0xffff) * ld) + (lane % kLanes ^ turn(line)) * 16 : 0x80000000u;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void*)(lds + (i * WAVES + wave) * 1024), 16, static_cast<int>(at_), 0, 0, 0);
        }
    }
    static __device__ __forceinline__ void clear(char* lds, int tid) {
        for (int i = tid * 16; i < kBytes; i += WAVES * 64 * 16) *reinterpret_cast<f32x4*>(lds + i) = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    // zeros for k >= n of a stage in LDS
    __device__ __forceinline__ void cut(char* lds, int n, int tid) const {
        if constexpr (OUTER) {
            for (int i = n * kLine + tid * 16; i < kBytes; i += WAVES * 64 * 16) *reinterpret_cast<f32x4*>(lds + i) = f32x4{0.f, 0.f, 0.f, 0.f};
        } else {
            for (int i = tid; i < R * kBk; i += WAVES * 64) {
                const int row = i / kBk, k = i % kBk;
                if (k >= n) *reinterpret_cast<T*>(lds + place(row, k)) = 0;
            }
        }
    }
    // prepares the fragments of 32 rows each from row w0 of the tile on
    __device__ __forceinline__ void aim(int w0, int lane) {
        const int r = lane & 31, h = lane >> 5, i = lane & 15;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            if constexpr (!OUTER) at[s] = (w0 + r) * kStage + ((2 * s + h) ^ turn(r)) * 16;      // of step s
            else if constexpr (kEs == 2)                                                        // of fragment s
                at[s] = (8 * h + i / 4) * kLine + (((w0 / 8 + s * 4) ^ turn(i / 4)) + (r / 16) * 2 + (i % 4) / 2) * 16 + (i & 1) * 8;
            else at[s] = 4 * h * kLine + (((w0 + s * 32 + r) / 4) ^ (8 * h)) * 16 + (r & 3) * 4;
        }
    }
    __device__ __forceinline__ typename Types<T>::Frag read(const char* lds, int f, int s) const {
        typename Types<T>::Frag v;
        if constexpr (!OUTER) {
            v = *reinterpret_cast<const typename Types<T>::Frag*>(lds + at[s] + f * 32 * kStage);
        } else if constexpr (kEs == 2) {
            typedef __attribute__((address_space(3))) v4s* Ptr;
            const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Ptr)(lds + at[f] + 16 * s * kLine));
            const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Ptr)(lds + at[f] + (16 * s + 4) * kLine));
            v = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const float*>(lds + at[f] + (8 * s + j) * kLine);
        }
        return v;
    }
};

__device__ __forceinline__ int64_t target_of(const GemmArgs& a, int t) {
    return a.target64 ? static_cast<const int64_t*>(a.target)[t] : static_cast<const int32_t*>(a.target)[t];
}
// whether a token's target is an entry of the vocabulary
__device__ __forceinline__ bool kept(const GemmArgs& a, int64_t target) { return target >= 0 && target < a.vocab; }

// four consecutive entries of a row of n
__device__ __forceinline__ void put_four(float* p, int at, int n, const float (&f)[4]) {
    if (at + 4 <= n) __builtin_memcpy(p + at, f, 16);
    else
        for (int i = 0; i < 4; ++i)
            if (at + i < n) p[at + i] = f[i];
}

// Of a run of tokens those whose targets are entries of a tile of dW, in order: token
// (16 bits) and entry, and the rest of its entry of P
constexpr int kHits = 2048;
struct Hits {
    int list[kHits];
    uint16_t rest[kHits];
    int count[8];
};
// A workgroup's LDS: two stages of both operands, in arrays of their own, so
// that a stage's reads do not wait for the next one's loads.
struct Lds {
    char *a0, *a1, *b0, *b1;
    Hits* hits;
};

// what a wave has written to its part of LDS is there for its other lanes
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// Rows of out (n, 32 of them) by columns (m, MW of them) of one wave, from the
// accumulators' order to whole rows: through the wave's own part of LDS, 16 bytes
// of a row a lane. Chunks are permuted by the row, so that neither side meets on
// a bank. f(i, r) is the value of accumulator r of fragment i.
template <typename T, int BM, int WM, typename F>
__device__ __forceinline__ void write_rows(const Lds& s, int wave, int lane, T* out, int64_t ld, int rows, int cols, F&& f) {
    constexpr int kEs = sizeof(T), MW = BM / WM, kRow = MW * kEs, kRegion = 32 * kRow, kPer = BM * kStage / kRegion;
    constexpr int kChunks = kRow / 16, kN = 16 / kEs;
    const int k = wave / kPer;
    char* lds = (k == 0 ? s.a0 : k == 1 ? s.a1 : k == 2 ? s.b0 : s.b1) + wave % kPer * kRegion;
    const int n = lane & 31, h = lane >> 5;
#pragma unroll
    for (int i = 0; i < MW / 32; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int m = (32 * i + 8 * q + 4 * h) * kEs;
            T v[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) st(v, r, f(i, 4 * q + r));
            __builtin_memcpy(lds + n * kRow + ((m / 16) ^ (n & (kChunks - 1) & 15)) * 16 + m % 16, v, sizeof(v));
        }
    wave_sync();
#pragma unroll
    for (int k2 = 0; k2 < 32 * kChunks / 64; ++k2) {
        const int row = (k2 * 64 + lane) / kChunks, c = lane % kChunks;
        T v[kN];
        __builtin_memcpy(v, lds + row * kRow + (c ^ (row & (kChunks - 1) & 15)) * 16, 16);
        if (row >= rows) continue;
        T* to = out + row * ld + c * kN;
        if (c * kN + kN <= cols) __builtin_memcpy(to, v, 16);
        else
#pragma unroll
            for (int j = 0; j < kN; ++j)
                if (c * kN + j < cols) to[j] = v[j];
    }
    wave_sync();
}

// a barrier that the copies to LDS this wave has asked for are behind
__device__ __forceinline__ void landed() {
    __builtin_amdgcn_s_waitcnt(0x0f70);              // vmcnt(0)
    __syncthreads();
}

// One tile of a product, of the split `z` of its k.
template <typename T, int BM, int BN, int WM, int WN, bool AO, bool BO, Epilogue EPI>
__device__ __forceinline__ void gemm_tile(const GemmArgs& a, int tile, int z, const Lds& lds) {
    constexpr int kWaves = WM * WN, MF = BM / WM / 32, NF = BN / WN / 32;
    static_assert(MF <= 4 && NF <= 4, "fragments of a wave");
    typedef Operand<T, AO, BM, kWaves> OpA;
    typedef Operand<T, BO, BN, kWaves> OpB;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    // eight columns of tiles at a time, so that the tiles that run together share rows of both operands in an L2
    int tm, tn;
    {
        const int band = tile / (8 * a.tiles_m), width = min(8, a.tiles_n - band * 8), in = tile - band * 8 * a.tiles_m;
        tm = in / width;
        tn = band * 8 + in % width;
    }
    const int m0 = tm * BM, n0 = tn * BN;
    const int k_lo = z * a.k_split, k_hi = min(a.K, k_lo + a.k_split);

    OpA A;
    OpB B;
    A.open(a.A, a.lda, m0, a.M, a.K, lane, wave);
    B.open(a.B, a.ldb, n0, a.N, a.K, lane, wave);
    A.aim(wm * (BM / WM), lane);
    B.aim(wn * (BN / WN), lane);
    f32x16 acc[MF][NF];
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
        for (int j = 0; j < NF; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

    auto multiply = [&](char* pa, char* pb) VS_INLINE {
        // a step's fragments are read while the matrix cores work on the last one's
        typename Types<T>::Frag fa[2][MF], fb[2][NF];
        auto read = [&](int s) VS_INLINE {
#pragma unroll
            for (int j = 0; j < NF; ++j) fb[s & 1][j] = B.read(pb, j, s);
#pragma unroll
            for (int i = 0; i < MF; ++i) fa[s & 1][i] = A.read(pa, i, s);
        };
        read(0);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            if (s < 3) read(s + 1);
#pragma unroll
            for (int i = 0; i < MF; ++i)
#pragma unroll
                for (int j = 0; j < NF; ++j) Types<T>::mma(fa[s & 1][i], fb[s & 1][j], acc[i][j]);
        }
        landed();
    };
    auto stage = [&](char* pa, char* pb, int k) VS_INLINE {
        if (k + OpA::kBk > k_hi) {
            A.cut(pa, k_hi - k, tid);
            B.cut(pb, k_hi - k, tid);
            __syncthreads();
        }
        multiply(pa, pb);
    };
    A.load(lds.a0, k_lo);
    B.load(lds.b0, k_lo);
    landed();
    int k = k_lo;
    for (; k + OpA::kBk < k_hi; k += 2 * OpA::kBk) {
        A.load(lds.a1, k + OpA::kBk);
        B.load(lds.b1, k + OpA::kBk);
        stage(lds.a0, lds.b0, k);
        if (k + 2 * OpA::kBk < k_hi) {
            A.load(lds.a0, k + 2 * OpA::kBk);
            B.load(lds.b0, k + 2 * OpA::kBk);
        }
        stage(lds.a1, lds.b1, k + OpA::kBk);
    }
    if (k < k_hi) stage(lds.a0, lds.b0, k);

    // The targets' entries of P, near -dloss, outweigh the others, so that what their
    // rounding took off would add to a result's own in full (bf16 8,194 x 1,536 x 49,999: off
    // by 0.0023 of dx and dW where 0.0017 is the last rounding). dW: in stages of their
    // own, those of the split's tokens whose targets are entries of the tile (one or two
    // behind 128; as many again where the vocabulary is one tile).
    if constexpr (EPI == kSum && BO && sizeof(T) == 2) {
        if (a.rest) {
            constexpr int kThreads = 64 * kWaves;
            Hits& hits = *lds.hits;
            auto entry = [&](int t) VS_INLINE {
                const int64_t v = t < k_hi ? target_of(a, t) : -1, in = v - a.v0 - n0;
                return kept(a, v) && in >= 0 && in < BN && n0 + in < a.N ? static_cast<int>(in) : -1;
            };
            int set0 = -1, set1 = -1;                                // what a lane has set in its line of b0 and b1
            bool clear = false;
            for (int t0 = k_lo; t0 < k_hi; t0 += kHits) {
                const int per = (min(kHits, k_hi - t0) + kThreads - 1) / kThreads, mine = t0 + tid * per;
                uint32_t found = 0;
#pragma unroll 4
                for (int j = 0; j < per; ++j) found |= (entry(mine + j) >= 0 ? 1u : 0u) << j;
                // this thread's place in the list: tokens stay in order
                int before = __builtin_popcount(found), all = 0;
                const int own = before;
#pragma unroll
                for (int o = 1; o < 64; o *= 2) {
                    const int up = __shfl_up(before, o, 64);
                    before += lane >= o ? up : 0;
                }
                if (lane == 63) hits.count[wave] = before;
                __syncthreads();
                before -= own;
                for (int w = 0; w < kWaves; ++w) {
                    const int n = hits.count[w];
                    before += w < wave ? n : 0;
                    all += n;
                }
                for (; found; found &= found - 1, ++before) {
                    const int t = mine + __builtin_ctz(found);
                    hits.list[before] = (t - t0) | entry(t) << 16;
                    st(hits.rest, before, a.rest[t]);
                }
                if (all > 0 && !clear) {
                    OpB::clear(lds.b0, tid);
                    OpB::clear(lds.b1, tid);
                    clear = true;
                }
                __syncthreads();
                auto fill = [&](char* pa, char* pb, int s, int& set) VS_INLINE {
                    A.pick(pa, t0, hits.list + s, all - s, lane);
                    if (tid < OpA::kBk) {
                        T* line = reinterpret_cast<T*>(pb);
                        if (set >= 0) line[set] = 0;
                        set = s + tid < all ? OpB::place(tid, hits.list[s + tid] >> 16) / OpB::kEs : -1;
                        if (set >= 0) line[set] = hits.rest[s + tid];
                    }
                };
                if (all > 0) {
                    fill(lds.a0, lds.b0, 0, set0);
                    landed();
                }
                for (int s = 0; s < all; s += 2 * OpA::kBk) {
                    if (s + OpA::kBk < all) fill(lds.a1, lds.b1, s + OpA::kBk, set1);
                    multiply(lds.a0, lds.b0);
                    if (s + 2 * OpA::kBk < all) fill(lds.a0, lds.b0, s + 2 * OpA::kBk, set0);
                    if (s + OpA::kBk < all) multiply(lds.a1, lds.b1);
                }
            }
        }
    }

    // acc[i][j][r] of a lane: row m0 + wm BM / WM + 32 i + 8 (r / 4) + 4 (lane / 32) + r % 4, column n0 + wn BN / WN + 32 j + lane % 32
    const int mw = m0 + wm * (BM / WM) + 4 * (lane >> 5), nw = n0 + wn * (BN / WN) + (lane & 31);
    if constexpr (EPI == kLse) {
        float* red = reinterpret_cast<float*>(lds.a0);               // [2][WM][BN]
        if (m0 + BM > a.M) {
#pragma unroll
            for (int i = 0; i < MF; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const bool out = mw + 32 * i + 8 * (r / 4) + r % 4 >= a.M;
#pragma unroll
                    for (int j = 0; j < NF; ++j) acc[i][j][r] = out ? -INFINITY : acc[i][j][r];
                }
        }
#pragma unroll
        for (int j = 0; j < NF; ++j) {
            const int n = nw + 32 * j;
            float mx = -INFINITY;
#pragma unroll
            for (int i = 0; i < MF; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) mx = fmaxf(mx, acc[i][j][r]);
            mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
            const float top = mx == -INFINITY ? 0.f : mx, from = top * kLog2e;
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < MF; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) sum += __builtin_amdgcn_exp2f(fmaf(acc[i][j][r], kLog2e, -from));
            sum += __shfl_xor(sum, 32, 64);
            // what rounding `from` took off each exponent: 2.4e-4 where logits are near 4,096
            sum *= __builtin_amdgcn_exp2f(fmaf(-top, kLog2e, from));
            if (lane < 32) {
                red[wm * BN + n - n0] = mx;
                red[(WM + wm) * BN + n - n0] = sum;
            }
            // the target's logit, where this wave holds it
            const int64_t t = n < a.N ? target_of(a, n) - a.v0 - mw : -1;
            const bool here = t >= 0 && t < BM / WM && (t & 4) == 0 && t + mw < a.M;
            if (__ballot(here)) {
#pragma unroll
                for (int i = 0; i < MF; ++i)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        if (here && t == 32 * i + 8 * (r / 4) + r % 4) a.target_logit[n] = acc[i][j][r];
            }
        }
        __syncthreads();
        for (int c = tid; c < BN; c += 64 * kWaves) {
            if (n0 + c >= a.N) break;
            float mx = red[c], sum = 0.f;
#pragma unroll
            for (int o = 1; o < WM; ++o) mx = fmaxf(mx, red[o * BN + c]);
            const float safe = mx == -INFINITY ? 0.f : mx;
#pragma unroll
            for (int o = 0; o < WM; ++o) sum += red[(WM + o) * BN + c] * __builtin_amdgcn_exp2f((red[o * BN + c] - safe) * kLog2e);
            a.part_max[static_cast<int64_t>(tm) * a.N + n0 + c] = mx;
            a.part_sum[static_cast<int64_t>(tm) * a.N + n0 + c] = sum;
        }
    } else if constexpr (EPI == kProb) {
#pragma unroll
        for (int j = 0; j < NF; ++j) {
            const int n = nw + 32 * j, nc = min(n, a.N - 1);
            const int64_t t = target_of(a, nc);
            const bool on = kept(a, t);
            const float lse = a.lse[nc], shift = lse * kLog2e, g = on ? a.dloss[nc] : 0.f;
            // with what rounding `shift` took off each exponent
            const float gp = g * __builtin_amdgcn_exp2f(fmaf(-lse, kLog2e, shift));
            // the target's place among this lane's rows, and its entry
            const int64_t hot = t - a.v0 - mw;
            float top = 0.f;
            const int first = n0 + wn * (BN / WN) + 32 * j, mf = m0 + wm * (BM / WM);
            write_rows<T, BM, WM>(lds, wave, lane, static_cast<T*>(a.P) + static_cast<int64_t>(first) * a.ldp + mf, a.ldp, a.N - first, a.ldp - mf,
                                  [&](int i, int r) VS_INLINE {
                                      const int m = 32 * i + 8 * (r / 4) + r % 4;
                                      const float p = __builtin_amdgcn_exp2f(fmaf(acc[i][j][r], kLog2e, -shift));
                                      const float e = on && mw + m < a.M ? fmaf(p, gp, hot == m ? -g : 0.f) : 0.f;
                                      if constexpr (sizeof(T) == 2) top = hot == m ? e : top;
                                      return e;
                                  });
            if constexpr (sizeof(T) == 2) {
                // this lane's rows are 4 of every 8, from its mw on
                if (hot >= 0 && hot < BM / WM && (hot & 4) == 0 && mw + hot < a.M && n < a.N && on) {
                    const float kept_part = static_cast<float>(static_cast<__bf16>(top));
                    a.rest[n] = __builtin_isfinite(kept_part) ? top - kept_part : 0.f;
                }
            }
        }
    } else {
        const bool split = a.k_split < a.K;
        // dx: the rest of the target's entry times its row of W
        if constexpr (!BO && sizeof(T) == 2) {
            if (a.rest && z == 0) {
#pragma unroll
                for (int j = 0; j < NF; ++j) {
                    const int n = nw + 32 * j;
                    const int64_t v = target_of(a, min(n, a.N - 1));
                    if (n >= a.N || !kept(a, v)) continue;
                    const float rest = a.rest[n];
                    const T* row = static_cast<const T*>(a.rows) + v * a.lda;
#pragma unroll
                    for (int i = 0; i < MF; ++i)
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const int m = mw + 32 * i + 8 * q;
                            T w[4] = {};
                            if (m + 4 <= a.M) __builtin_memcpy(w, row + m, sizeof(w));
                            else
#pragma unroll
                                for (int r = 0; r < 4; ++r)
                                    if (m + r < a.M) w[r] = row[m + r];
#pragma unroll
                            for (int r = 0; r < 4; ++r) acc[i][j][4 * q + r] = fmaf(rest, ld(w, r), acc[i][j][4 * q + r]);
                        }
                }
            }
        }
#pragma unroll
        for (int j = 0; j < NF; ++j) {
            const int n = nw + 32 * j, first = n0 + wn * (BN / WN) + 32 * j, mf = m0 + wm * (BM / WM);
            float* sum = a.sum ? a.sum + (static_cast<int64_t>(split ? z : 0) * a.N + min(n, a.N - 1)) * a.M : nullptr;
            // a token that is left out: its row of P is zeros, but an infinity in W would make NaN of them
            const bool on = BO || kept(a, target_of(a, min(n, a.N - 1)));
            if (a.out && !split) {
                write_rows<T, BM, WM>(lds, wave, lane, static_cast<T*>(a.out) + static_cast<int64_t>(first) * a.ldo + mf, a.ldo, a.N - first,
                                      a.M - mf, [&](int i, int r) VS_INLINE {
                                          const int m = mw + 32 * i + 8 * (r / 4) + r % 4;
                                          return on ? acc[i][j][r] + (a.add && m < a.M ? sum[m] : 0.f) : 0.f;
                                      });
                continue;
            }
            if (n >= a.N) continue;
#pragma unroll
            for (int i = 0; i < MF; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int m = mw + 32 * i + 8 * q;
                    if (m >= a.M) continue;
                    float f[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) f[r] = on ? acc[i][j][4 * q + r] + (a.add && !split && m + r < a.M ? sum[m + r] : 0.f) : 0.f;
                    put_four(sum, m, a.M, f);
                }
        }
    }
}

// Workgroups are dealt to the XCDs in turn: each gets one contiguous range of the
// tiles 0..n-1 (of those of `more` behind them).
struct Range { int first, count; };
__device__ __forceinline__ Range xcd_range(int n, int x) {
    const int q = n / static_cast<int>(kXcds), r = n % static_cast<int>(kXcds);
    return {x * q + min(x, r), q + (x < r ? 1 : 0)};
}

#define VS_GEMM_LDS(T, AO, BO)                                                                          \
    __shared__ __attribute__((aligned(1024))) char sA0[Operand<T, AO, BM, WM * WN>::kBytes];            \
    __shared__ __attribute__((aligned(1024))) char sA1[Operand<T, AO, BM, WM * WN>::kBytes];            \
    __shared__ __attribute__((aligned(1024))) char sB0[Operand<T, BO, BN, WM * WN>::kBytes];            \
    __shared__ __attribute__((aligned(1024))) char sB1[Operand<T, BO, BN, WM * WN>::kBytes];            \
    Lds lds{sA0, sA1, sB0, sB1, nullptr};

// Bound by the matrix cores and by what they wait for: 8,194 x 1,536 x 49,999 bf16 scored
// in 1,080 us (up to 1,160 on other cards), 1.17 PFLOP/s (59 % of their cycles; the
// library's product of these sizes alone, which writes its logits, 1,083 us). With P
// half of the vocabulary takes 680 us for 540 of product: a tile's 131 KB are written
// with no other tile on the compute unit to work meanwhile. 197 x 768 x 49,999: 25 us
// for 77 MB of W, 196 of 256 units busy. fp32 394 x 384 x 32,768: 100 us, matrix cores
// 80 %, and 394 tokens fill 77 % of two tiles.
template <typename T, int BM, int BN, int WM, int WN, Epilogue EPI>
__global__ __launch_bounds__(64 * WM * WN) void vocab_logits_kernel(const GemmArgs a) {
    VS_GEMM_LDS(T, false, false)
    const int x = blockIdx.x % kXcds, k = blockIdx.x / kXcds;
    gemm_tile<T, BM, BN, WM, WN, false, false, EPI>(a, xcd_range(gridDim.x, x).first + k, 0, lds);
}

// dx and dW of a piece in one launch: the tiles of dx, whose k is the longer one
// with large pieces, first, and those of dW in the room that they leave. Bound by
// the matrix cores: half of 8,194 x 1,536 x 49,999 bf16 1,280 us, 0.98 PFLOP/s (47 % of
// their cycles); fp32 394 x 384 x 32,768 202 us, 98 TFLOP/s of the useful products (73 %).
template <typename T, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void vocab_grads_kernel(const GemmArgs dx, const GemmArgs dw, int n_dx) {
    VS_GEMM_LDS(T, true, true)
    if constexpr (sizeof(T) == 2) {
        __shared__ Hits hits;
        lds.hits = &hits;
    }
    const int x = blockIdx.x % kXcds, k = blockIdx.x / kXcds;
    const Range all = xcd_range(gridDim.x, x), one = xcd_range(n_dx, x);
    if (k < one.count) {
        const int v = one.first + k, tiles = dx.tiles_m * dx.tiles_n;
        gemm_tile<T, BM, BN, WM, WN, true, false, kSum>(dx, v % tiles, v / tiles, lds);
    } else {
        const int v = all.first - one.first + k - one.count, tiles = dw.tiles_m * dw.tiles_n;
        gemm_tile<T, BM, BN, WM, WN, true, true, kSum>(dw, v % tiles, v / tiles, lds);
    }
}

// ------------------------------------------------------------- around them
// rows of `dim` entries into rows of `dp`, zeros behind them; with targets, rows
// that they leave out become zeros
struct PackArgs {
    const void* in;
    int64_t ld;
    void* out;
    int64_t rows;
    int dim, dp;
    const void* target;
    int target64, vocab;
};
template <typename T>
__global__ __launch_bounds__(256) void vocab_pack_kernel(const PackArgs a) {
    const int per = a.dp / 8;                       // runs of eight
    const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (id >= a.rows * per) return;
    const int64_t row = id / per;
    const int c = static_cast<int>(id - row * per) * 8;
    bool on = true;
    if (a.target) {
        const int64_t t = a.target64 ? static_cast<const int64_t*>(a.target)[row] : static_cast<const int32_t*>(a.target)[row];
        on = t >= 0 && t < a.vocab;
    }
    const T* in = static_cast<const T*>(a.in) + row * a.ld;
    T v[8];
    if (on && c + 8 <= a.dim) {
        __builtin_memcpy(v, in + c, sizeof(v));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = on && c + i < a.dim ? in[c + i] : T(0);
    }
    __builtin_memcpy(static_cast<T*>(a.out) + row * a.dp + c, v, sizeof(v));
}

// A token's tiles into its lse and loss: 16 tokens a workgroup, 16 lines of tiles;
// one dependent chain, 4 to 8 us
struct LseArgs {
    const float *part_max, *part_sum, *target_logit;
    const void* target;
    int target64, vocab, tiles;
    int tokens;
    float *loss, *lse;
};
__global__ __launch_bounds__(256) void vocab_lse_kernel(const LseArgs a) {
    __shared__ float red[2][16][17];
    const int c = threadIdx.x & 15, line = threadIdx.x >> 4, t = blockIdx.x * 16 + c;
    float mx = -INFINITY, sum = 0.f;
    if (t < a.tokens)
        for (int v = line; v < a.tiles; v += 16 * 8) {         // eight tiles in flight
            float m[8], s[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int64_t at = static_cast<int64_t>(min(v + 16 * j, a.tiles - 1)) * a.tokens + t;
                m[j] = v + 16 * j < a.tiles ? a.part_max[at] : -INFINITY;
                s[j] = v + 16 * j < a.tiles ? a.part_sum[at] : 0.f;
            }
            float top = mx;
#pragma unroll
            for (int j = 0; j < 8; ++j) top = fmaxf(top, m[j]);
            const float safe = top == -INFINITY ? 0.f : top;
            sum *= __builtin_amdgcn_exp2f((mx - safe) * kLog2e);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum += s[j] * __builtin_amdgcn_exp2f((m[j] - safe) * kLog2e);
            mx = top;
        }
    red[0][line][c] = mx;
    red[1][line][c] = sum;
    __syncthreads();
    if (line || t >= a.tokens) return;
#pragma unroll
    for (int o = 1; o < 16; ++o) mx = fmaxf(mx, red[0][o][c]);
    const float safe = mx == -INFINITY ? 0.f : mx;
    sum = 0.f;
#pragma unroll
    for (int o = 0; o < 16; ++o) sum += red[1][o][c] * __builtin_amdgcn_exp2f((red[0][o][c] - safe) * kLog2e);
    // the loss from differences: of lse, rounded at the logits' size, it would lose what they are away from zero
    const float rest = logf(sum);
    a.lse[t] = safe + rest;
    const int64_t g = a.target64 ? static_cast<const int64_t*>(a.target)[t] : static_cast<const int32_t*>(a.target)[t];
    a.loss[t] = g >= 0 && g < a.vocab ? (safe - a.target_logit[t]) + rest : 0.f;
}

// the splits of a product, in order
struct JoinArgs {
    const float* part;
    int splits;
    int64_t count;                  // entries of one split
    int M;
    float* sum;                     // added to and written where there is no out
    int add;
    void* out;
    int64_t ldo;
};
template <typename T>
__global__ __launch_bounds__(256) void vocab_join_kernel(const JoinArgs a) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= a.count) return;
    float s = a.add ? a.sum[i] : 0.f;
    for (int z = 0; z < a.splits; ++z) s += a.part[z * a.count + i];
    if (a.out) st(static_cast<T*>(a.out) + i / a.M * a.ldo, i % a.M, s);
    else a.sum[i] = s;
}

// ------------------------------------------------------------------ launch
int ceil_div(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }

template <typename T>
void cut(GemmArgs& a, bool wide, int splits) {
    const int tile = wide ? 256 : 128;
    a.tiles_m = ceil_div(a.M, tile);
    a.tiles_n = ceil_div(a.N, tile);
    constexpr int kBk = kStage / static_cast<int>(sizeof(T));
    a.k_split = ceil_div(ceil_div(a.K, kBk), splits) * kBk;      // no split is empty
}

template <typename T, Epilogue EPI>
void logits(GemmArgs a, bool wide, hipStream_t s) {
    cut<T>(a, wide, 1);
    const uint32_t grid = static_cast<uint32_t>(a.tiles_m) * static_cast<uint32_t>(a.tiles_n);
    if (wide) vocab_logits_kernel<T, 256, 256, 2, 4, EPI><<<grid, 512, 0, s>>>(a);
    else vocab_logits_kernel<T, 128, 128, 2, 2, EPI><<<grid, 256, 0, s>>>(a);
}

// a product's splits into its `out`, or its `sum`
template <typename T>
void join(const GemmArgs& a, const float* part, int splits, hipStream_t s) {
    JoinArgs j{};
    j.part = part; j.splits = splits; j.count = static_cast<int64_t>(a.N) * a.M; j.M = a.M; j.sum = a.sum; j.add = a.add;
    j.out = a.out; j.ldo = a.ldo;
    vocab_join_kernel<T><<<ceil_div(j.count, 256), 256, 0, s>>>(j);
}

// both products of a piece; those that cut their k leave their parts in part_dx and part_dw
template <typename T>
void products(GemmArgs dx, GemmArgs dw, const vs::VocabPlan& p, float* part_dx, float* part_dw, hipStream_t s) {
    cut<T>(dx, p.wide, p.dx_splits);
    cut<T>(dw, p.wide, p.dw_splits);
    const int nx = ceil_div(dx.K, dx.k_split), nw = ceil_div(dw.K, dw.k_split);
    GemmArgs gx = dx, gw = dw;
    if (nx > 1) gx.sum = part_dx;
    if (nw > 1) gw.sum = part_dw;
    const int n_dx = dx.tiles_m * dx.tiles_n * nx, n_dw = dw.tiles_m * dw.tiles_n * nw;
    const uint32_t grid = static_cast<uint32_t>(n_dx + n_dw);
    if (p.wide) vocab_grads_kernel<T, 256, 256, 2, 4><<<grid, 512, 0, s>>>(gx, gw, n_dx);
    else vocab_grads_kernel<T, 128, 128, 2, 2><<<grid, 256, 0, s>>>(gx, gw, n_dx);
    if (nx > 1) join<T>(dx, part_dx, nx, s);
    if (nw > 1) join<T>(dw, part_dw, nw, s);
}

template <typename T>
void pack(const void* in, int64_t ld, void* out, int64_t rows, const vs::VocabCall& c, const void* target, hipStream_t s) {
    PackArgs a{};
    a.in = in; a.ld = ld; a.out = out; a.rows = rows; a.dim = static_cast<int>(c.dim); a.dp = static_cast<int>(c.plan.dp);
    a.target = target; a.target64 = c.target64; a.vocab = static_cast<int>(c.vocab);
    vocab_pack_kernel<T><<<ceil_div(rows * (a.dp / 8), 256), 256, 0, s>>>(a);
}

template <typename T>
int launch(const vs::VocabCall& c) {
    const auto s = static_cast<hipStream_t>(c.stream);
    const vs::VocabPlan& p = c.plan;
    char* ws = static_cast<char*>(c.ws);
    const T *x = static_cast<const T*>(c.x), *W = static_cast<const T*>(c.W);
    int64_t ldx = c.ldx, ldw = c.dim;
    if (c.grad || p.pack_x) {
        pack<T>(x, ldx, ws + p.x, c.tokens, c, c.grad ? c.target : nullptr, s);
        x = reinterpret_cast<const T*>(ws + p.x);
        ldx = p.dp;
    }
    if (p.pack_w) {
        pack<T>(W, ldw, ws + p.w, c.vocab, c, nullptr, s);
        W = reinterpret_cast<const T*>(ws + p.w);
        ldw = p.dp;
    }
    GemmArgs l{};
    l.A = W; l.lda = ldw; l.B = x; l.ldb = ldx; l.N = static_cast<int>(c.tokens); l.K = static_cast<int>(c.dim);
    l.target = c.target; l.target64 = c.target64; l.vocab = static_cast<int>(c.vocab);
    if (!c.grad) {
        l.M = static_cast<int>(c.vocab);
        l.part_max = reinterpret_cast<float*>(ws + p.part);
        l.part_sum = l.part_max + static_cast<int64_t>(p.tiles) * c.tokens;
        l.target_logit = reinterpret_cast<float*>(ws + p.logit);
        logits<T, kLse>(l, p.wide, s);
        LseArgs e{};
        e.part_max = l.part_max; e.part_sum = l.part_sum; e.target_logit = l.target_logit; e.target = c.target; e.target64 = c.target64;
        e.vocab = l.vocab; e.tiles = p.tiles; e.tokens = l.N; e.loss = c.loss; e.lse = c.lse;
        vocab_lse_kernel<<<ceil_div(c.tokens, 16), 256, 0, s>>>(e);
    } else {
        float* sum = reinterpret_cast<float*>(ws + p.sum);
        for (int64_t v0 = 0; v0 < c.vocab; v0 += p.piece) {
            const int n = static_cast<int>(c.vocab - v0 < p.piece ? c.vocab - v0 : p.piece);
            const bool last = v0 + n == c.vocab;
            l.A = W + v0 * ldw; l.M = n; l.v0 = static_cast<int>(v0);
            l.lse = c.lse_in; l.dloss = c.dloss; l.P = ws + p.P;
            if (sizeof(T) == 2) l.rest = reinterpret_cast<float*>(ws + p.rest);
            l.ldp = ceil_div(n, 8) * 8;                 // rows of whole 16 bytes
            logits<T, kProb>(l, p.prob_wide, s);
            GemmArgs dx{}, dw{};
            dx.A = W + v0 * ldw; dx.lda = ldw; dx.B = l.P; dx.ldb = l.ldp;
            dx.M = static_cast<int>(c.dim); dx.N = static_cast<int>(c.tokens); dx.K = n;
            dx.target = dw.target = c.target; dx.target64 = dw.target64 = c.target64; dx.vocab = dw.vocab = l.vocab; dw.v0 = l.v0;
            dx.rest = last ? l.rest : nullptr; dx.rows = W; dw.rest = l.rest;    // dx: every piece's, once all are there
            dx.add = v0 > 0; dx.sum = p.pieces > 1 ? sum : nullptr;
            dx.out = last ? c.dx : nullptr; dx.ldo = c.dim;
            dw.A = x; dw.lda = ldx; dw.B = l.P; dw.ldb = l.ldp;
            dw.M = static_cast<int>(c.dim); dw.N = n; dw.K = static_cast<int>(c.tokens);
            dw.out = static_cast<T*>(c.dW) + v0 * c.dim; dw.ldo = c.dim;
            products<T>(dx, dw, p, reinterpret_cast<float*>(ws + p.part_dx), reinterpret_cast<float*>(ws + p.part_dw), s);
        }
    }
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? VS_OK : vs::fail(VS_ERR_HIP, std::string("kernel launch: ") + hipGetErrorString(e));
}

int run(vs::VocabCall& c) {
    if (int rc = vs::prepare_vocab(c)) return rc;
    return c.dtype == VS_BF16 ? launch<uint16_t>(c) : launch<float>(c);
}

}  // namespace

extern "C" {

int vocab_loss(int64_t tokens, int64_t dim, int64_t vocab, int dtype, const void* x, int64_t x_stride,
               const void* W, const void* target, int target_bits, float* loss, float* lse,
               void* workspace, size_t workspace_bytes, void* stream) {
    vs::VocabCall c{};
    c.tokens = tokens; c.dim = dim; c.vocab = vocab; c.dtype = dtype; c.x = x; c.ldx = x_stride; c.W = W; c.target = target;
    c.target_bits = target_bits; c.loss = loss; c.lse = lse; c.ws = workspace; c.ws_bytes = workspace_bytes; c.stream = stream;
    return run(c);
}

int vocab_loss_grad(int64_t tokens, int64_t dim, int64_t vocab, int dtype, const void* x, int64_t x_stride,
                    const void* W, const void* target, int target_bits, const float* lse, const float* dloss,
                    void* dx, void* dW, void* workspace, size_t workspace_bytes, void* stream) {
    vs::VocabCall c{};
    c.tokens = tokens; c.dim = dim; c.vocab = vocab; c.dtype = dtype; c.x = x; c.ldx = x_stride; c.W = W; c.target = target;
    c.target_bits = target_bits; c.lse_in = lse; c.dloss = dloss; c.dx = dx; c.dW = dW; c.ws = workspace;
    c.ws_bytes = workspace_bytes; c.stream = stream; c.grad = true;
    return run(c);
}

}  // extern "C"
