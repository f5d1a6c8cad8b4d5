// The processing of logits in front of a selection on gfx950: penalties for the
// tokens of a history, biases, a mask of allowed tokens. With n the number of
// times token t stands in the row's history, m of them past its prompt:
//   n > 0:        x = x > 0 ? x / repetition : x * repetition
//   m > 0:        x = x - (frequency m + presence)
//   a bias for t: x = x + bias (of several the last)
//   t forbidden:  x = -inf
// in fp32, rounded once to the logits' type.
//
// One workgroup per chunk of a row. It counts the history's tokens of its chunk
// in LDS, one word per logit (integer atomics: the order does not matter), and
// walks its logits once, 16 bytes per lane. A vector whose tokens are all
// forbidden is written without being read; in place, a vector that nothing
// changes is neither read nor written.
#include "logits_launch.h"

namespace kda {
namespace {

constexpr float NEG_INF = -__builtin_inff();
// A logit's word: tokens past the prompt, whether the prompt has it, whether it has a bias.
constexpr uint32_t PAST = 0x3fffffffu, BIASED = 1u << 30, PROMPT = 1u << 31;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

template <int DT>
struct Elem;
template <>
struct Elem<KDA_FP32> {
    typedef float T;
    static __device__ __forceinline__ float up(float x) { return x; }
    static __device__ __forceinline__ float down(float x) { return x; }
};
template <>
struct Elem<KDA_BF16> {
    typedef __bf16 T;
    static __device__ __forceinline__ float up(__bf16 x) { return (float)x; }
    static __device__ __forceinline__ __bf16 down(float x) { return (__bf16)x; }
};
template <>
struct Elem<KDA_FP16> {
    typedef _Float16 T;
    static __device__ __forceinline__ float up(_Float16 x) { return (float)x; }
    static __device__ __forceinline__ _Float16 down(float x) { return (_Float16)x; }
};

// What a row's logits go through (uniform).
struct Row {
    float repetition, frequency, presence;
    bool repeat, count;
    const float* bias;
    uint32_t mask_none;  // all ones where there is no mask
};

__device__ __forceinline__ float process(float x, uint32_t word, const int32_t* slot, const Row& r) {
    if (word) {
        const uint32_t m = word & PAST;
        if (r.repeat && (word & ~BIASED)) x = x > 0.f ? x / r.repetition : x * r.repetition;
        if (r.count && m) x -= r.frequency * (float)m + r.presence;
        if (word & BIASED) x += r.bias[*slot - 1];
    }
    return x;
}

template <int DT, bool LISTS>
__global__ __launch_bounds__(kLogitsThreads) void process_logits(LogitsArgs a) {
    typedef Elem<DT> E;
    typedef typename E::T T;
    constexpr int VEC = 16 / (int)sizeof(T);  // logits of a vector
    extern __shared__ __align__(16) uint32_t lds[];
    uint32_t* const word = lds;                    // [chunk]
    int32_t* const slot = (int32_t*)lds + a.chunk;  // [chunk] where there are biases: 1 + the entry
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x / a.splits;
    const int v0 = (int)(blockIdx.x % a.splits) * a.chunk;
    const int n = a.x.vocab - v0 < a.chunk ? a.x.vocab - v0 : a.chunk;
    const T* const in = (const T*)a.x.logits + row * a.x.row_stride + v0;
    T* const out = (T*)a.x.out + row * a.x.out_stride + v0;
    const bool in_place = a.x.out == a.x.logits;
    const uint32_t* const allowed = a.x.allowed ? a.x.allowed + row * a.x.allowed_stride + (v0 >> 5) : nullptr;

    Row r = {};
    if constexpr (LISTS) {
        for (int i = tid * 4; i < n; i += kLogitsThreads * 4) {  // the chunk is a multiple of 4
            *(u32x4*)(word + i) = u32x4{0, 0, 0, 0};
            if (a.x.n_bias) *(u32x4*)(slot + i) = u32x4{0, 0, 0, 0};
        }
        __syncthreads();
        if (a.x.tokens) {
            int len = a.x.max_tokens, prompt = 0;
            if (a.x.lengths) {
                len = a.x.lengths[row];
                len = len < 0 ? 0 : len < a.x.max_tokens ? len : a.x.max_tokens;
            }
            if (a.x.prompt_lengths) prompt = a.x.prompt_lengths[row];
            r.repeat = a.x.repetition != nullptr;
            r.count = a.x.frequency || a.x.presence;
            if (r.repeat) r.repetition = a.x.repetition[row];
            if (a.x.frequency) r.frequency = a.x.frequency[row];
            if (a.x.presence) r.presence = a.x.presence[row];
            const int32_t* const tokens = a.x.tokens + row * a.x.token_stride;
            // without a repetition penalty the prompt does not count
            for (int i = (r.repeat || prompt < 0 ? 0 : prompt) + tid; i < len; i += kLogitsThreads) {
                const uint32_t t = (uint32_t)(tokens[i] - v0);
                if (t < (uint32_t)n) {
                    if (i < prompt) atomicOr(word + t, PROMPT);
                    else atomicAdd(word + t, 1u);
                }
            }
        }
        if (a.x.n_bias) {
            r.bias = a.x.bias + row * a.x.bias_stride;
            const int32_t* const tokens = a.x.bias_tokens + row * a.x.bias_stride;
            for (int i = tid; i < a.x.n_bias; i += kLogitsThreads) {
                const uint32_t t = (uint32_t)(tokens[i] - v0);
                if (t < (uint32_t)n) {
                    atomicOr(word + t, BIASED);
                    atomicMax(slot + t, i + 1);
                }
            }
        }
        __syncthreads();
    }

    for (int i = tid * VEC; i + VEC <= n; i += kLogitsThreads * VEC) {
        constexpr uint32_t ALL = (1u << VEC) - 1;
        const uint32_t bits = allowed ? allowed[i >> 5] >> (i & 31) & ALL : ALL;
        uint32_t w[VEC] = {};
        uint32_t any = 0;
        if constexpr (LISTS) {
#pragma unroll
            for (int j = 0; j < VEC; j += 4) {
                const u32x4 x = *(const u32x4*)(word + i + j);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    w[j + e] = x[e];
                    any |= x[e];
                }
            }
        }
        if (in_place && !any && bits == ALL) continue;
        T x[VEC];
        if (bits == 0) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) x[e] = E::down(NEG_INF);
        } else {
            __builtin_memcpy(x, __builtin_assume_aligned(in + i, sizeof(T)), 16);
            if (any)
#pragma unroll
                for (int e = 0; e < VEC; ++e) x[e] = E::down(process(E::up(x[e]), w[e], slot + i + e, r));
            if (bits != ALL)
#pragma unroll
                for (int e = 0; e < VEC; ++e) x[e] = bits >> e & 1 ? x[e] : E::down(NEG_INF);
        }
        __builtin_memcpy(__builtin_assume_aligned(out + i, sizeof(T)), x, 16);
    }
    // the logits behind the row's last whole vector
    const int i = n / VEC * VEC + tid;
    if (i < n) {
        const bool ok = !allowed || allowed[i >> 5] >> (i & 31) & 1;
        float x = NEG_INF;
        if (ok) {
            x = E::up(in[i]);
            if constexpr (LISTS) x = process(x, word[i], slot + i, r);
        }
        out[i] = E::down(x);
    }
}

template <int DT>
void launch(const LogitsArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)((int64_t)a.x.rows * a.splits)), block(kLogitsThreads);
    const size_t lds = (size_t)a.chunk * 4 * (a.x.n_bias ? 2 : 1);
    if (a.x.tokens || a.x.n_bias) hipLaunchKernelGGL((process_logits<DT, true>), grid, block, lds, s, a);
    else hipLaunchKernelGGL((process_logits<DT, false>), grid, block, 0, s, a);
}

}  // namespace

hipError_t launch_logits(const LogitsArgs& a, hipStream_t s) {
    if (a.x.dtype == KDA_FP32) launch<KDA_FP32>(a, s);
    else if (a.x.dtype == KDA_BF16) launch<KDA_BF16>(a, s);
    else launch<KDA_FP16>(a, s);
    return hipGetLastError();
}

}  // namespace kda
