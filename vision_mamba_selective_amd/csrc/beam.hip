// beam.hip -- gfx950 kernels of beam search: the choice among beams x
// vocabulary, and moving the states of the chosen beams (include/vimscan.h has
// the contract).
#include <hip/hip_runtime.h>

#include <cstdint>
#include <string>

#include "vimscan.h"
#include "vs_device.h"
#include "vs_internal.h"

namespace {

using vs::fail;

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kPart = static_cast<int>(vs::kBeamPart);   // entries of one workgroup's part of a row
constexpr int kPer = kPart / kThreads;      // and of one thread: chunks of 8 consecutive ones
constexpr int kChunks = kPer / 8;

struct SelectArgs {
    const void* logits;
    const float* scores;
    const uint8_t* done;
    float* out_scores;
    int32_t *out_parent, *out_token;
    uint64_t* keys;         // [row][part][beams]: the part's best, best first
    float2* sums;           // [row][part]: maximum and sum of exp(x - maximum)
    int64_t sb, sk;
    int64_t batch, vocab, eos;
    int beams, parts;
};

// Order-preserving: larger floats get larger integers; -inf is 0x007fffff.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x);
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t o) {
    return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu));
}
// Candidates are compared as 64-bit integers: the value, then the lower index
// first. Every candidate has a key of its own, and 0 is below all of them.
__device__ __forceinline__ uint64_t make_key(float x, uint32_t index) {
    return (static_cast<uint64_t>(ordered(x)) << 32) | static_cast<uint32_t>(~index);
}
__device__ __forceinline__ float key_value(uint64_t k) { return from_ordered(static_cast<uint32_t>(k >> 32)); }
__device__ __forceinline__ uint32_t key_index(uint64_t k) { return ~static_cast<uint32_t>(k); }

// ---- reductions over a wave, every lane gets the result: quads and rows by
// DPP (after the first two steps a quad is uniform, so mirroring eight lanes
// pairs the quads), the four rows by lane swaps
template <typename F>
__device__ __forceinline__ float wave_reduce(float v, F&& f) {
    v = f(v, dpp<0xb1>(v));                                      // quad_perm [1,0,3,2]
    v = f(v, dpp<0x4e>(v));                                      // quad_perm [2,3,0,1]
    v = f(v, dpp<0x141>(v));                                     // row_half_mirror
    v = f(v, dpp<0x140>(v));                                     // row_mirror
    auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = f(__uint_as_float(r[0]), __uint_as_float(r[1]));
    r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return f(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float wave_max(float v) {
    return wave_reduce(v, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ float wave_sum(float v) {
    return wave_reduce(v, [](float a, float b) { return a + b; });
}
// the sum over this lane and those below it
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_add(int v) {
    return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, false);
}
__device__ __forceinline__ int wave_prefix(int v) {
    v = dpp_add<0x111, 0xf>(v);                                  // row_shr 1, 2, 4, 8
    v = dpp_add<0x112, 0xf>(v);
    v = dpp_add<0x114, 0xf>(v);
    v = dpp_add<0x118, 0xf>(v);
    v = dpp_add<0x142, 0xa>(v);                                  // row_bcast 15: rows 1 and 3
    return dpp_add<0x143, 0xc>(v);                               // row_bcast 31: rows 2 and 3
}
__device__ __forceinline__ uint64_t lane_key(uint64_t k, int lane) {
    const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(k), lane);
    const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(k >> 32), lane);
    return (static_cast<uint64_t>(hi) << 32) | lo;
}
// how many of the first n lanes' keys are above this lane's
__device__ __forceinline__ int wave_rank(uint64_t key, int n) {
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += lane_key(key, j) > key ? 1 : 0;
    return rank;
}
__device__ __forceinline__ uint64_t wave_max64(uint64_t v) {
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) {
        const uint32_t lo = __shfl_xor(static_cast<int>(v), m), hi = __shfl_xor(static_cast<int>(v >> 32), m);
        const uint64_t o = (static_cast<uint64_t>(hi) << 32) | lo;
        v = o > v ? o : v;
    }
    return v;
}

// eight consecutive entries of a row that starts at any element
__device__ __forceinline__ void load_eight(const float* p, float (&f)[8]) { __builtin_memcpy(f, p, sizeof(f)); }
__device__ __forceinline__ void load_eight(const uint16_t* p, float (&f)[8]) {
    uint32_t w[4];
    __builtin_memcpy(w, p, sizeof(w));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
// One part of one row: its `beams` best entries, its maximum and its sum of
// exponentials. A thread holds 32 entries in registers, a wave 2,048. Of a
// wave only the entries above a threshold that at least `beams` of its lanes
// reach are candidates, with the first entries equal to it: they go to a
// list in LDS (some twenty of 2,048 for 8 beams), are ranked by counting, and
// the four waves' best ranked again. GROUPS = 8, 16 or 32 >= beams: the
// threshold is the smallest of that many lane groups' maxima (each group has
// an entry at or above it). Where the list cannot hold what that leaves, the
// threshold becomes the beams-th largest maximum of a lane: fewer than `beams`
// lanes of 32 entries are above that.
// 64 x 8 beams x 49,999 bf16 24 us. The logits' 47 MB would take 9 us, the 663
// VALU instructions a wave about 10 at their issue costs (the counter, in steps
// of four cycles, has the VALU active 81 %). The rest has not been taken apart:
// its steps follow one another (the prefix sum, the second read of the
// candidates, their ranking, and the last one by one wave). The smallest GROUPS is taken: for
// those 8 beams 31 us with 16 and 63 with 32, whose longer lists leave fewer
// workgroups a compute unit; as many logits take, with the merge, 55 us at 32 x
// 16 beams and 168 at 16 x 32. With 64 entries a thread 29 us.
template <typename T, int GROUPS>
__global__ __launch_bounds__(kThreads) void beam_part_kernel(const SelectArgs a) {
    constexpr int kMost = kPer * (GROUPS - 1);
    __shared__ uint64_t list[kWaves][kMost + GROUPS];
    __shared__ uint64_t best[kWaves][GROUPS];
    __shared__ float2 wsum[kWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const uint32_t row32 = blockIdx.x / static_cast<uint32_t>(a.parts);
    const int part = static_cast<int>(blockIdx.x - row32 * static_cast<uint32_t>(a.parts));
    const int64_t row = row32;
    if (a.done && a.done[row]) return;
    const int K = a.beams;
    const uint32_t seq = row32 / static_cast<uint32_t>(K);
    const T* x = static_cast<const T*>(a.logits) + seq * a.sb + (row32 - seq * static_cast<uint32_t>(K)) * a.sk;
    const int64_t first = static_cast<int64_t>(part) * kPart;
    const int n = static_cast<int>(a.vocab - first < kPart ? a.vocab - first : kPart);
    x += first;
    // entry j of chunk c: index c * 2048 + tid * 8 + j. NaN and what lies past
    // the row count as -inf
    float v[kPer];
    if (n == kPart) {                                     // uniform
        float f[kChunks][8];
#pragma unroll
        for (int c = 0; c < kChunks; ++c) load_eight(x + c * kThreads * 8 + tid * 8, f[c]);
#pragma unroll
        for (int i = 0; i < kPer; ++i) v[i] = fmaxf(f[i / 8][i % 8], -INFINITY);
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int j = (i / 8) * kThreads * 8 + tid * 8 + i % 8;
            const float f = ld(x, j < n ? j : n - 1);
            v[i] = j < n ? fmaxf(f, -INFINITY) : -INFINITY;
        }
    }
    float mine = v[0];
#pragma unroll
    for (int i = 1; i < kPer; ++i) mine = fmaxf(mine, v[i]);
    // lane groups of 64 / GROUPS: their maxima, then the smallest of those
    auto hi = [](float p, float q) { return fmaxf(p, q); };
    float group = mine;
    if (GROUPS <= 32) group = hi(group, dpp<0xb1>(group));
    if (GROUPS <= 16) group = hi(group, dpp<0x4e>(group));
    if (GROUPS <= 8) group = hi(group, dpp<0x141>(group));
    float low = wave_reduce(group, [](float p, float q) { return fminf(p, q); });
    const float top = wave_max(group);
    // ---- the wave's candidates: the entries at or above the threshold, whose
    // indices go to the list as they come ...
    uint64_t* mylist = list[wave];
    uint32_t at_least = 0;                                // bit 31 - i: entry i
#pragma unroll
    for (int i = 0; i < kPer; ++i) at_least = at_least + at_least + (v[i] >= low ? 1u : 0u);
    int held = __popc(at_least);
    int place = wave_prefix(held);
    int total = __builtin_amdgcn_readlane(place, 63);
    place -= held;
    if (total <= kMost + GROUPS) {
        while (at_least != 0) {
            const int i = __clz(static_cast<int>(at_least));
            at_least &= ~(0x80000000u >> i);
            mylist[place++] = static_cast<uint32_t>((i >> 3) * kThreads * 8 + tid * 8 + (i & 7));
        }
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
        // ... and become keys with a second read of the entries
        for (int i = lane; i < total; i += 64) {
            const int j = static_cast<int>(mylist[i]);
            const float e = fmaxf(ld(x, j < n ? j : n - 1), -INFINITY);
            mylist[i] = j < n ? make_key(e + 0.f, static_cast<uint32_t>(first + j)) : 0;
        }
    } else {
        // too many equal ones, or too many above a low threshold: raise it,
        // take those above it and the first K equal to it
        bool off = false;                                 // this lane's maximum was taken
        for (int r = 0; r < K; ++r) {
            low = wave_max(off ? -INFINITY : mine);
            const uint64_t at = __ballot(!off && mine == low);
            if (lane == __ffsll(static_cast<unsigned long long>(at)) - 1) off = true;
        }
        held = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) held += v[i] > low ? 1 : 0;
        place = wave_prefix(held);
        total = __builtin_amdgcn_readlane(place, 63);
        place -= held;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (v[i] > low)
                mylist[place++] = make_key(v[i] + 0.f, static_cast<uint32_t>(first + (i / 8) * kThreads * 8 + tid * 8 + i % 8));
        }
        int ties = 0;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const int i0 = c * kThreads * 8 + tid * 8;
            uint32_t eq = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) eq |= (v[8 * c + j] == low && i0 + j < n ? 1u : 0u) << j;
            if (ties < K && __ballot(eq != 0) != 0) {
                const int mineq = __popc(eq), upto = wave_prefix(mineq);
                int r = ties + upto - mineq;
                while (eq != 0 && r < K) {
                    const int j = __ffs(static_cast<int>(eq)) - 1;
                    eq &= eq - 1;
                    mylist[total + r++] = make_key(low + 0.f, static_cast<uint32_t>(first + i0 + j));
                }
                ties = min(ties + __builtin_amdgcn_readlane(upto, 63), K);
            }
        }
        total += ties;
    }
    // ---- the wave's best K, by counting the larger ones
    if (lane < GROUPS) best[wave][lane] = 0;
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    if (total <= 64) {
        const uint64_t k = lane < total ? mylist[lane] : 0;
        const int rank = wave_rank(k, total);
        if (k != 0 && rank < K) best[wave][rank] = k;
    } else {
        for (int i = lane; i < total; i += 64) {
            const uint64_t k = mylist[i];
            int rank = 0;
            for (int j = 0; j < total; ++j) rank += mylist[j] > k ? 1 : 0;
            if (rank < K) best[wave][rank] = k;
        }
    }
    // ---- the sum of exponentials; a maximum of +inf: the number of its entries
    float s = 0.f;
    if (top == INFINITY) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) s += v[i] == INFINITY ? 1.f : 0.f;
    } else if (top != -INFINITY) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) s += __builtin_amdgcn_exp2f((v[i] - top) * kLog2e);
    }
    s = wave_sum(s);
    if (lane == 0) wsum[wave] = make_float2(top, s);
    __syncthreads();
    // ---- the workgroup's: four sorted lists, and four sums
    uint64_t* out = a.keys + (row * a.parts + part) * K;
    if (kWaves * GROUPS <= 64) {
        if (wave == 0) {
            const uint64_t k = lane < kWaves * GROUPS ? best[lane / GROUPS][lane % GROUPS] : 0;
            const int rank = wave_rank(k, kWaves * GROUPS);
            if (k != 0 && rank < K) out[rank] = k;
        }
    } else if (tid < kWaves * GROUPS) {
        const uint64_t k = best[tid / GROUPS][tid % GROUPS];
        int rank = 0;
        for (int w = 0; w < kWaves; ++w)
            for (int j = 0; j < K; ++j) rank += best[w][j] > k ? 1 : 0;
        if (k != 0 && rank < K) out[rank] = k;
    }
    if (tid == 0) {
        float m = fmaxf(fmaxf(wsum[0].x, wsum[1].x), fmaxf(wsum[2].x, wsum[3].x)), sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
            if (wsum[w].x == m) sum += wsum[w].y;
            else if (wsum[w].x != -INFINITY && m != INFINITY) sum += wsum[w].y * __builtin_amdgcn_exp2f((wsum[w].x - m) * kLog2e);
        a.sums[row * a.parts + part] = make_float2(m, sum);
    }
    // a part of fewer than K entries leaves the rest of its places empty
    if (n < K && tid >= n && tid < K) out[tid] = 0;
}

constexpr int kMergeThreads = 512;
constexpr int kMergeWaves = kMergeThreads / 64;
constexpr int kMergeRegs = 4;               // keys of one lane that stay in registers

// One sequence: each wave joins the parts of its beams (the softmax's maximum
// and sum, the beam's best candidates and their scores), then all candidates
// are ranked by counting. Bound by latency: 64 sequences of 8 beams 6 us.
__global__ __launch_bounds__(kMergeThreads) void beam_merge_kernel(const SelectArgs a) {
    __shared__ uint64_t cand[VS_MAX_BEAMS * VS_MAX_BEAMS];     // by score, then beam and rank
    __shared__ uint32_t token[VS_MAX_BEAMS * VS_MAX_BEAMS];
    __shared__ uint64_t picks[kMergeWaves][VS_MAX_BEAMS];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t b = blockIdx.x;
    const int K = a.beams;
    for (int k = wave; k < K; k += kMergeWaves) {
        const int64_t row = b * K + k;
        const float score = a.scores[row];
        if (a.done && a.done[row]) {
            if (lane < K) {
                const int64_t t = lane == 0 ? a.eos : (lane - 1 < a.eos ? lane - 1 : lane);
                float v = lane == 0 ? score : -INFINITY;
                v = v != v ? -INFINITY : v + 0.f;
                cand[k * K + lane] = t < a.vocab ? make_key(v, static_cast<uint32_t>(k * K + lane)) : 0;
                token[k * K + lane] = static_cast<uint32_t>(t);
            }
            continue;
        }
        const uint64_t* keys = a.keys + row * a.parts * K;
        const int64_t n = static_cast<int64_t>(a.parts) * K;
        uint64_t mine[kMergeRegs];
#pragma unroll
        for (int i = 0; i < kMergeRegs; ++i) mine[i] = lane + 64 * i < n ? keys[lane + 64 * i] : 0;
        float top = -INFINITY, sum = 0.f;
        for (int64_t p = lane; p < a.parts; p += 64) {
            const float2 e = a.sums[row * a.parts + p];
            if (e.x > top) {
                sum = top == -INFINITY || e.x == INFINITY ? e.y : fmaf(sum, __builtin_amdgcn_exp2f((top - e.x) * kLog2e), e.y);
                top = e.x;
            } else if (e.x == top) {
                sum += e.y;
            } else if (e.x != -INFINITY && top != INFINITY) {
                sum = fmaf(e.y, __builtin_amdgcn_exp2f((e.x - top) * kLog2e), sum);
            }
        }
        const float all = wave_max(top);
        if (top != all) sum = top == -INFINITY || all == INFINITY ? 0.f : sum * __builtin_amdgcn_exp2f((top - all) * kLog2e);
        top = all;
        sum = wave_sum(sum);
        // lane r: the beam's candidate r
        uint64_t pick = 0;
        if (n <= 64) {
            const int rank = wave_rank(mine[0], static_cast<int>(n));
            if (mine[0] != 0 && rank < K) picks[wave][rank] = mine[0];
            __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
            const int64_t found = a.vocab < K ? a.vocab : K;
            if (lane < found) pick = picks[wave][lane];
            __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
        } else {
            uint64_t last = ~uint64_t(0);
            for (int r = 0; r < K; ++r) {
                uint64_t best = 0;
#pragma unroll
                for (int i = 0; i < kMergeRegs; ++i)
                    if (mine[i] < last && mine[i] > best) best = mine[i];
                for (int64_t i = lane + 64 * kMergeRegs; i < n; i += 64) {
                    const uint64_t e = keys[i];
                    if (e < last && e > best) best = e;
                }
                best = wave_max64(best);
                last = best;
                if (lane == r) pick = best;
            }
        }
        if (lane < K) {
            const float x = key_value(pick);
            // (x - top) - log(sum): top + log(sum) would round away what log(sum)
            // holds where the logits are far from zero
            const float below = x == top ? 0.f : x - top;  // -inf, too, where only top is +inf
            float v = x == -INFINITY ? -INFINITY : below - logf(sum);
            v = score + v + 0.f;
            if (v != v) v = -INFINITY;
            cand[k * K + lane] = pick ? make_key(v, static_cast<uint32_t>(k * K + lane)) : 0;
            token[k * K + lane] = key_index(pick);
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < K * K; i += kMergeThreads) {
        const uint64_t key = cand[i];
        int rank = 0;
        for (int j = 0; j < K * K; ++j) rank += cand[j] > key ? 1 : 0;
        if (key != 0 && rank < K) {
            a.out_scores[b * K + rank] = key_value(key);
            a.out_parent[b * K + rank] = static_cast<int32_t>(b * K + i / K);
            a.out_token[b * K + rank] = static_cast<int32_t>(token[i]);
        }
    }
}

// --------------------------------------------------------------- reordering
using Vec16 = uint32_t __attribute__((ext_vector_type(4)));

struct ReorderArgs {
    const char* state;
    const int32_t* parent;
    char* out;
    int64_t row_bytes, layer_bytes, cols;
    int beams;
};

// A thread takes one column of a sequence's rows: it loads every row that some
// beam needs from another, then stores them, so the rows may be moved in
// place. Rows that keep their place are left alone there. Bound by memory: 24
// layers of 16 x 8 rows of 48 KB 27 us, 5.7 TB/s read and written.
template <typename V, int K>
__global__ __launch_bounds__(kThreads) void beam_reorder_kernel(const ReorderArgs a) {
    // the first column of the workgroup and its sequence are scalars, so that
    // every row's address is one, and a thread adds only its own offset
    const int64_t col0 = static_cast<int64_t>(blockIdx.x) * kThreads;
    if (col0 + static_cast<int64_t>(threadIdx.x) >= a.cols) return;
    const int64_t base = static_cast<int64_t>(blockIdx.z) * a.layer_bytes +
                         static_cast<int64_t>(blockIdx.y) * a.beams * a.row_bytes + col0 * static_cast<int64_t>(sizeof(V));
    const uint32_t off = threadIdx.x * static_cast<uint32_t>(sizeof(V));
    const int32_t* parent = a.parent + static_cast<int64_t>(blockIdx.y) * a.beams;
    const int32_t first = static_cast<int32_t>(blockIdx.y) * a.beams;
    const bool in_place = a.state == a.out;
    int from[K];
#pragma unroll
    for (int i = 0; i < K; ++i) {
        const int p = __builtin_amdgcn_readfirstlane(parent[i < a.beams ? i : 0]) - first;
        from[i] = i < a.beams && p >= 0 && p < a.beams ? p : i;
    }
    // the loads stand in a straight line: a beam that needs none repeats another's
    int some = -1;
#pragma unroll
    for (int i = K - 1; i >= 0; --i)
        if (i < a.beams && (from[i] != i || !in_place)) some = from[i];
    if (some < 0) return;
    V v[K];
#pragma unroll
    for (int i = 0; i < K; ++i) {
        const int f = i < a.beams && (from[i] != i || !in_place) ? from[i] : some;
        v[i] = *reinterpret_cast<const V*>(a.state + (base + f * a.row_bytes) + off);
    }
#pragma unroll
    for (int i = 0; i < K; ++i)
        if (i < a.beams && (from[i] != i || !in_place))
            *reinterpret_cast<V*>(a.out + (base + i * a.row_bytes) + off) = v[i];
}

int launched() {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(VS_ERR_HIP, std::string("kernel launch: ") + hipGetErrorString(e));
    return VS_OK;
}

template <typename T>
void launch_parts(const SelectArgs& a, dim3 grid, hipStream_t st) {
    if (a.beams <= 8) hipLaunchKernelGGL((beam_part_kernel<T, 8>), grid, dim3(kThreads), 0, st, a);
    else if (a.beams <= 16) hipLaunchKernelGGL((beam_part_kernel<T, 16>), grid, dim3(kThreads), 0, st, a);
    else hipLaunchKernelGGL((beam_part_kernel<T, 32>), grid, dim3(kThreads), 0, st, a);
}

template <typename V>
int launch_reorder(ReorderArgs a, int64_t layers, int64_t batch, hipStream_t st) {
    a.cols = a.row_bytes / static_cast<int64_t>(sizeof(V));
    const int64_t wgs = (a.cols + kThreads - 1) / kThreads;
    if (wgs > vs::kMaxGroups) return fail(VS_ERR_UNSUPPORTED, "rows too long for one launch");
    const dim3 grid(static_cast<unsigned>(wgs), static_cast<unsigned>(batch), static_cast<unsigned>(layers));
    if (a.beams <= 4) hipLaunchKernelGGL((beam_reorder_kernel<V, 4>), grid, dim3(kThreads), 0, st, a);
    else if (a.beams <= 8) hipLaunchKernelGGL((beam_reorder_kernel<V, 8>), grid, dim3(kThreads), 0, st, a);
    else if (a.beams <= 16) hipLaunchKernelGGL((beam_reorder_kernel<V, 16>), grid, dim3(kThreads), 0, st, a);
    else hipLaunchKernelGGL((beam_reorder_kernel<V, 32>), grid, dim3(kThreads), 0, st, a);
    return launched();
}

}  // namespace

// ---------------------------------------------------------------- C ABI
extern "C" {

int beam_select(int64_t batch, int64_t beams, int64_t vocab, int dtype, const void* logits,
                const int64_t* strides, const float* scores, const uint8_t* done, int64_t eos,
                float* out_scores, int32_t* out_parent, int32_t* out_token, void* workspace,
                size_t workspace_bytes, void* stream) {
    int64_t st[2];
    if (int rc = vs::validate_beam_select(batch, beams, vocab, dtype, logits, strides, scores, done, eos, out_scores,
                                          out_parent, out_token, workspace, workspace_bytes, st))
        return rc;
    SelectArgs a{};
    a.logits = logits; a.scores = scores; a.done = done; a.out_scores = out_scores; a.out_parent = out_parent;
    a.out_token = out_token; a.sb = st[0]; a.sk = st[1]; a.batch = batch; a.vocab = vocab; a.eos = eos;
    a.beams = static_cast<int>(beams);
    a.parts = static_cast<int>(vs::beam_parts(vocab));
    const int64_t wgs = batch * beams * a.parts;
    if (wgs > vs::kMaxGroups) return fail(VS_ERR_UNSUPPORTED, "batch * beams * vocab too large for one launch");
    a.keys = static_cast<uint64_t*>(workspace);
    a.sums = reinterpret_cast<float2*>(a.keys + wgs * beams);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const dim3 grid(static_cast<unsigned>(wgs));
    if (dtype == VS_BF16) launch_parts<uint16_t>(a, grid, s);
    else launch_parts<float>(a, grid, s);
    if (int rc = launched()) return rc;
    hipLaunchKernelGGL(beam_merge_kernel, dim3(static_cast<unsigned>(batch)), dim3(kMergeThreads), 0, s, a);
    return launched();
}

int beam_reorder(int64_t layers, int64_t batch, int64_t beams, int64_t row_bytes,
                 int64_t layer_bytes, const void* state, const int32_t* parent, void* out,
                 void* stream) {
    if (int rc = vs::validate_beam_reorder(layers, batch, beams, row_bytes, layer_bytes, state, parent, out)) return rc;
    ReorderArgs a{};
    a.state = static_cast<const char*>(state); a.parent = parent; a.out = static_cast<char*>(out);
    a.row_bytes = row_bytes; a.layer_bytes = layer_bytes; a.beams = static_cast<int>(beams);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    // the widest access that every row's address and length allow
    auto fits = [&](int64_t n) {
        return row_bytes % n == 0 && layer_bytes % n == 0 && vs::aligned(state, static_cast<size_t>(n)) &&
               vs::aligned(out, static_cast<size_t>(n));
    };
    if (fits(16)) return launch_reorder<Vec16>(a, layers, batch, st);
    if (fits(4)) return launch_reorder<uint32_t>(a, layers, batch, st);
    if (fits(2)) return launch_reorder<uint16_t>(a, layers, batch, st);
    return launch_reorder<uint8_t>(a, layers, batch, st);
}

}  // extern "C"
