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
constexpr int kPart = 8192;                 // entries of one workgroup's part of a row
constexpr int kPer = kPart / kThreads;      // and of one thread

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

__device__ __forceinline__ uint64_t shfl_xor64(uint64_t v, int m) {
    const uint32_t lo = __shfl_xor(static_cast<int>(v), m), hi = __shfl_xor(static_cast<int>(v >> 32), m);
    return (static_cast<uint64_t>(hi) << 32) | lo;
}
__device__ __forceinline__ uint64_t wave_max64(uint64_t v) {
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) {
        const uint64_t o = shfl_xor64(v, m);
        v = o > v ? o : v;
    }
    return v;
}

// One part of one row: its `beams` best entries, its maximum and its sum of
// exponentials. A thread holds its entries in registers; the best are taken
// one at a time, each the largest key below the last.
template <typename T>
__global__ __launch_bounds__(kThreads) void beam_part_kernel(const SelectArgs a) {
    __shared__ uint64_t wbest[2][kWaves];
    __shared__ float wsum[kWaves];
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x / static_cast<unsigned>(a.parts);
    const int part = static_cast<int>(blockIdx.x % static_cast<unsigned>(a.parts));
    if (a.done && a.done[row]) return;
    const T* x = static_cast<const T*>(a.logits) + (row / a.beams) * a.sb + (row % a.beams) * a.sk;
    const int64_t first = static_cast<int64_t>(part) * kPart;
    const int count = static_cast<int>(a.vocab - first < kPart ? a.vocab - first : kPart);
    float v[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int j = i * kThreads + tid;
        float e = -INFINITY;
        if (j < count) e = ld(x, first + j) + 0.f;            // -0 counts as 0
        v[i] = e != e ? -INFINITY : e;
    }
    uint64_t last = ~uint64_t(0);
    float top = 0.f;
    for (int r = 0; r < a.beams; ++r) {
        uint64_t best = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int j = i * kThreads + tid;
            const uint64_t k = make_key(v[i], static_cast<uint32_t>(first + j));
            if (j < count && k < last && k > best) best = k;
        }
        best = wave_max64(best);
        if ((tid & 63) == 0) wbest[r & 1][tid >> 6] = best;
        __syncthreads();
        best = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) best = wbest[r & 1][w] > best ? wbest[r & 1][w] : best;
        if (r == 0) top = key_value(best);
        last = best;
        if (tid == 0) a.keys[(row * a.parts + part) * a.beams + r] = best;
    }
    // a maximum of +inf: the sum counts its entries
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const float e = top == INFINITY ? (v[i] == INFINITY ? 1.f : 0.f)
                                        : (v[i] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((v[i] - top) * kLog2e));
        s += e;
    }
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) s += __shfl_xor(s, m);
    if ((tid & 63) == 0) wsum[tid >> 6] = s;
    __syncthreads();
    if (tid == 0) a.sums[row * a.parts + part] = make_float2(top, wsum[0] + wsum[1] + wsum[2] + wsum[3]);
}

// One sequence: each wave joins the parts of its beams (the softmax's maximum
// and sum, the beam's best candidates and their scores), then the first wave
// takes the best of all.
__global__ __launch_bounds__(kThreads) void beam_merge_kernel(const SelectArgs a) {
    __shared__ uint64_t cand[VS_MAX_BEAMS * VS_MAX_BEAMS];     // by score, then beam and rank
    __shared__ uint32_t token[VS_MAX_BEAMS * VS_MAX_BEAMS];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t b = blockIdx.x;
    const int K = a.beams;
    for (int k = wave; k < K; k += kWaves) {
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
        float top = -INFINITY, sum = 0.f;
        for (int64_t p = lane; p < a.parts; p += 64) top = fmaxf(top, a.sums[row * a.parts + p].x);
#pragma unroll
        for (int m = 32; m > 0; m >>= 1) top = fmaxf(top, __shfl_xor(top, m));
        for (int64_t p = lane; p < a.parts; p += 64) {
            const float2 e = a.sums[row * a.parts + p];
            if (top == INFINITY) sum += e.x == INFINITY ? e.y : 0.f;
            else if (e.x != -INFINITY) sum += e.y * __builtin_amdgcn_exp2f((e.x - top) * kLog2e);
        }
#pragma unroll
        for (int m = 32; m > 0; m >>= 1) sum += __shfl_xor(sum, m);
        const float lse = top == INFINITY ? 0.f : top + logf(sum);
        const uint64_t* keys = a.keys + row * a.parts * K;
        const int64_t n = static_cast<int64_t>(a.parts) * K;
        uint64_t last = ~uint64_t(0);
        for (int r = 0; r < K; ++r) {
            uint64_t best = 0;
            for (int64_t i = lane; i < n; i += 64) {
                const uint64_t e = keys[i];
                if (e < last && e > best) best = e;
            }
            best = wave_max64(best);
            last = best;
            if (lane == 0) {
                const float x = key_value(best);
                float v = x == -INFINITY ? -INFINITY : (top == INFINITY ? (x == INFINITY ? -logf(sum) : -INFINITY) : x - lse);
                v = score + v + 0.f;
                if (v != v) v = -INFINITY;
                cand[k * K + r] = best ? make_key(v, static_cast<uint32_t>(k * K + r)) : 0;
                token[k * K + r] = key_index(best);
            }
        }
    }
    __syncthreads();
    if (wave != 0) return;
    uint64_t last = ~uint64_t(0);
    for (int r = 0; r < K; ++r) {
        uint64_t best = 0;
        for (int i = lane; i < K * K; i += 64) {
            const uint64_t e = cand[i];
            if (e < last && e > best) best = e;
        }
        best = wave_max64(best);
        last = best;
        if (lane == 0) {
            const uint32_t i = key_index(best);
            a.out_scores[b * K + r] = key_value(best);
            a.out_parent[b * K + r] = static_cast<int32_t>(b * K + i / K);
            a.out_token[b * K + r] = static_cast<int32_t>(token[i]);
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
// place. Rows that keep their place are left alone there.
template <typename V, int K>
__global__ __launch_bounds__(kThreads) void beam_reorder_kernel(const ReorderArgs a) {
    const int64_t col = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (col >= a.cols) return;
    const int64_t base = static_cast<int64_t>(blockIdx.z) * a.layer_bytes +
                         static_cast<int64_t>(blockIdx.y) * a.beams * a.row_bytes + col * static_cast<int64_t>(sizeof(V));
    const int32_t* parent = a.parent + static_cast<int64_t>(blockIdx.y) * a.beams;
    const int32_t first = static_cast<int32_t>(blockIdx.y) * a.beams;
    const bool in_place = a.state == a.out;
    V v[K];
    int from[K];
#pragma unroll
    for (int i = 0; i < K; ++i) {
        from[i] = i;
        if (i < a.beams) {
            const int p = __builtin_amdgcn_readfirstlane(parent[i]) - first;
            from[i] = p >= 0 && p < a.beams ? p : i;
            if (from[i] != i || !in_place)
                v[i] = *reinterpret_cast<const V*>(a.state + base + from[i] * a.row_bytes);
        }
    }
#pragma unroll
    for (int i = 0; i < K; ++i)
        if (i < a.beams && (from[i] != i || !in_place))
            *reinterpret_cast<V*>(a.out + base + i * a.row_bytes) = v[i];
}

int launched() {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(VS_ERR_HIP, std::string("kernel launch: ") + hipGetErrorString(e));
    return VS_OK;
}

template <typename V>
int launch_reorder(ReorderArgs a, int64_t layers, int64_t batch, hipStream_t st) {
    a.cols = a.row_bytes / static_cast<int64_t>(sizeof(V));
    const int64_t wgs = (a.cols + kThreads - 1) / kThreads;
    if (wgs >= (int64_t(1) << 31)) return fail(VS_ERR_UNSUPPORTED, "rows too long for one launch");
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
    a.parts = static_cast<int>((vocab + kPart - 1) / kPart);
    const int64_t wgs = batch * beams * a.parts;
    if (wgs >= (int64_t(1) << 31)) return fail(VS_ERR_UNSUPPORTED, "batch * beams * vocab too large for one launch");
    a.keys = static_cast<uint64_t*>(workspace);
    a.sums = reinterpret_cast<float2*>(a.keys + wgs * beams);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const dim3 grid(static_cast<unsigned>(wgs));
    if (dtype == VS_BF16) hipLaunchKernelGGL((beam_part_kernel<uint16_t>), grid, dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL((beam_part_kernel<float>), grid, dim3(kThreads), 0, s, a);
    if (int rc = launched()) return rc;
    hipLaunchKernelGGL(beam_merge_kernel, dim3(static_cast<unsigned>(batch)), dim3(kThreads), 0, s, a);
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
