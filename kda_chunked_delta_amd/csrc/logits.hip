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
// in LDS, one word per logit, and lists those that it meets (integer atomics:
// neither the counts nor the results depend on their order). All logits are then
// copied under the mask, 16 bytes per lane, and the few listed ones and those
// with a bias taken one by one: a division for every logit of every wavefront
// that holds a listed one took 15 us more for 256 rows of 131072. What
// is all forbidden is written without being read; in place, nothing is copied.
#include "logits_launch.h"

namespace kda {
namespace {

constexpr float NEG_INF = -__builtin_inff();
// The words of a chunk: how often a token stands past the prompt, whether it has
// a bias, and whether the prompt has it, in 16 bits where the history is shorter
// than 2^14 tokens (half the LDS, twice the logits per scan of the history), else
// in 32.
template <bool HALF>
struct Words {
    static constexpr int BITS = HALF ? 16 : 32;
    static constexpr uint32_t PROMPT = 1u << (BITS - 1), BIASED = 1u << (BITS - 2), PAST = BIASED - 1;
    uint32_t* base;
    __device__ __forceinline__ uint32_t get(uint32_t t) const { return HALF ? ((const uint16_t*)base)[t] : base[t]; }
    __device__ __forceinline__ void set(uint32_t t, uint32_t x) const {
        if constexpr (HALF) ((uint16_t*)base)[t] = (uint16_t)x;
        else base[t] = x;
    }
    // These give the word before. (A count stays below 2^14: no carry into the other half.)
    __device__ __forceinline__ uint32_t add(uint32_t t) const {
        if constexpr (HALF) return atomicAdd(base + (t >> 1), 1u << (16 * (t & 1))) >> (16 * (t & 1)) & 0xffffu;
        else return atomicAdd(base + t, 1u);
    }
    __device__ __forceinline__ uint32_t mark(uint32_t t) const {
        if constexpr (HALF) return atomicOr(base + (t >> 1), PROMPT << (16 * (t & 1))) >> (16 * (t & 1)) & 0xffffu;
        else return atomicOr(base + t, PROMPT);
    }
    __device__ __forceinline__ void raise(uint32_t t, uint32_t x) const {  // to x at least
        if constexpr (HALF) {
            uint32_t* const p = base + (t >> 1);
            const int at = 16 * (t & 1);
            uint32_t seen = *(volatile uint32_t*)p;
            while ((seen >> at & 0xffffu) < x) {
                const uint32_t old = atomicCAS(p, seen, (seen & ~(0xffffu << at)) | x << at);
                if (old == seen) break;
                seen = old;
            }
        } else {
            atomicMax(base + t, x);
        }
    }
};
constexpr int BATCH = 4;  // loads of 16 bytes in flight together

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
};

template <bool HALF>
__device__ __forceinline__ float penalise(float x, uint32_t word, const Row& r) {
    typedef Words<HALF> W;
    const uint32_t m = word & W::PAST;
    if (r.repeat && (word & ~W::BIASED)) x = x > 0.f ? x / r.repetition : x * r.repetition;
    if (r.count && m) x -= r.frequency * (float)m + r.presence;
    return x;
}

// LISTS: 0 without a history and biases, 1 with words of 16 bits, 2 of 32.
template <int DT, int LISTS, int THREADS>
__global__ __launch_bounds__(THREADS) void process_logits(LogitsArgs a) {
    typedef Elem<DT> E;
    typedef typename E::T T;
    constexpr int VEC = 16 / (int)sizeof(T);  // logits of a vector
    typedef Words<LISTS == 1> W;
    extern __shared__ __align__(16) uint32_t lds[];
    const W words{lds};  // [chunk]
    uint16_t* const list = (uint16_t*)lds + a.chunk * (W::BITS / 16);  // [the lesser of chunk and max_tokens]
    __shared__ uint32_t n_list;
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x / a.splits;
    const int v0 = (int)(blockIdx.x % a.splits) * a.chunk;
    const int n = a.x.vocab - v0 < a.chunk ? a.x.vocab - v0 : a.chunk;
    const T* const in = (const T*)a.x.logits + row * a.x.row_stride + v0;
    T* const out = (T*)a.x.out + row * a.x.out_stride + v0;
    const bool in_place = a.x.out == a.x.logits;
    const uint32_t* const allowed = a.x.allowed ? a.x.allowed + row * a.x.allowed_stride + (v0 >> 5) : nullptr;

    constexpr uint32_t ALL = (1u << VEC) - 1;
    constexpr int STEP = THREADS * VEC;  // logits from one of a lane's vectors to its next
    // The lane's vectors i0, i0 + STEP, ..: their bits of the mask, and the logits of those that need them.
    uint32_t bits[BATCH];
    u32x4 x[BATCH];
    auto fetch = [&](int i0) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            const int i = i0 + j * STEP;
            bits[j] = ALL;
            if (allowed && i + VEC <= n) bits[j] = allowed[i >> 5] >> (i & 31) & ALL;
        }
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            const int i = i0 + j * STEP;
            if (i + VEC <= n && bits[j] && !(in_place && bits[j] == ALL))
                __builtin_memcpy(&x[j], __builtin_assume_aligned(in + i, sizeof(T)), 16);
        }
    };
    const bool copies = !in_place || allowed;
    if (copies) fetch(tid * VEC);  // on their way while the words are made

    Row r = {};
    const int32_t* const tokens = LISTS > 0 && a.x.tokens ? a.x.tokens + row * a.x.token_stride : nullptr;
    const int32_t* const bias_tokens = LISTS > 0 && a.x.n_bias ? a.x.bias_tokens + row * a.x.bias_stride : nullptr;
    uint64_t last = 0;  // of the lane's entries with a bias, those that count: the last ones of their tokens
    if constexpr (LISTS > 0) {
        const int quads = tokens ? a.x.max_tokens / 4 : 0;
        int32_t tok[BATCH][4];
        auto fetch_tokens = [&](int q0) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < BATCH; ++j)
                if (q0 + j * THREADS < quads)
                    __builtin_memcpy(tok[j], __builtin_assume_aligned(tokens + 4 * (q0 + j * THREADS), 4), 16);
        };
        fetch_tokens(tid);
        int len = 0, prompt = 0;
        if (tokens) {
            len = a.x.max_tokens;
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
        }
        for (int i = tid * 16; i < n * (W::BITS / 8); i += THREADS * 16)
            *(u32x4*)((uint8_t*)lds + i) = u32x4{0, 0, 0, 0};
        if (tid == 0) n_list = 0;
        __syncthreads();
        if (bias_tokens) {
            auto each_bias = [&](auto f) __attribute__((always_inline)) {
                for (int i = tid, k = 0; i < a.x.n_bias; i += THREADS, ++k) {
                    const uint32_t t = (uint32_t)bias_tokens[i] - (uint32_t)v0;
                    if (t < (uint32_t)n) f(t, i, k);
                }
            };
            each_bias([&](uint32_t t, int i, int) { words.raise(t, (uint32_t)i + 1); });
            __syncthreads();
            each_bias([&](uint32_t t, int i, int k) {  // the others see the last one's number, or its mark
                if (words.get(t) != (uint32_t)i + 1) return;
                last |= (uint64_t)1 << k;
                words.set(t, W::BIASED);
            });
            __syncthreads();
        }
        if (tokens) {
            // without a repetition penalty the prompt does not count
            const int first = r.repeat ? 0 : prompt;
            auto count = [&](int32_t token, int i) __attribute__((always_inline)) {
                const uint32_t t = (uint32_t)token - (uint32_t)v0;
                if (t < (uint32_t)n && i >= first && i < len)
                    if ((i < prompt ? words.mark(t) : words.add(t)) == 0)
                        list[atomicAdd(&n_list, 1u)] = (uint16_t)t;
            };
            constexpr int MANY = THREADS * BATCH;  // quads of a batch
            int q = 0;
            if (first >= 4 * MANY) q = first / (4 * MANY) * MANY;  // batches before that are left out
            for (; 4 * q < len; q += MANY) {
                if (q > 0) fetch_tokens(q + tid);
#pragma unroll
                for (int j = 0; j < BATCH; ++j) {
                    const int at = q + tid + j * THREADS;
                    if (at < quads)
#pragma unroll
                        for (int e = 0; e < 4; ++e) count(tok[j][e], 4 * at + e);
                }
            }
            if (4 * quads + tid < len) count(tokens[4 * quads + tid], 4 * quads + tid);
        }
    }

    if (copies) {
        for (int i0 = tid * VEC; i0 + VEC <= n; i0 += STEP * BATCH) {
            if (i0 >= STEP) fetch(i0);
#pragma unroll
            for (int j = 0; j < BATCH; ++j) {
                const int i = i0 + j * STEP;
                if (i + VEC > n || (in_place && bits[j] == ALL)) continue;
                T y[VEC];
                __builtin_memcpy(y, &x[j], 16);
                if (bits[j] != ALL)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) y[e] = bits[j] >> e & 1 ? y[e] : E::down(NEG_INF);
                __builtin_memcpy(__builtin_assume_aligned(out + i, sizeof(T)), y, 16);
            }
        }
        // the logits behind the row's last whole vector
        const int i = n / VEC * VEC + tid;
        if (i < n) out[i] = !allowed || allowed[i >> 5] >> (i & 31) & 1 ? in[i] : E::down(NEG_INF);
    }
    if constexpr (LISTS > 0) {
        // in place, a logit is still what it was, or -inf behind the mask
        auto ok = [&](uint32_t t) { return !allowed || allowed[t >> 5] >> (t & 31) & 1; };
        __syncthreads();
        for (uint32_t p = tid; p < n_list; p += THREADS) {
            const uint32_t t = list[p];
            if (ok(t)) out[t] = E::down(penalise<LISTS == 1>(E::up(in[t]), words.get(t), r));
        }
        const float* const bias = a.x.bias + row * a.x.bias_stride;
        for (int i = tid, k = 0; last >> k; i += THREADS, ++k)
            if (last >> k & 1) {
                const uint32_t t = (uint32_t)bias_tokens[i] - (uint32_t)v0;
                if (ok(t)) out[t] = E::down(penalise<LISTS == 1>(E::up(in[t]), words.get(t), r) + bias[i]);
            }
    }
}

template <int DT>
void launch(const LogitsArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)((int64_t)a.x.rows * a.splits)), block(a.threads);
    if (a.lists == 1) hipLaunchKernelGGL((process_logits<DT, 1, kLogitsListThreads>), grid, block, a.lds, s, a);
    else if (a.lists == 2) hipLaunchKernelGGL((process_logits<DT, 2, kLogitsListThreads>), grid, block, a.lds, s, a);
    else hipLaunchKernelGGL((process_logits<DT, 0, kLogitsThreads>), grid, block, 0, s, a);
}

}  // namespace

hipError_t launch_logits(const LogitsArgs& a, hipStream_t s) {
    if (a.x.dtype == KDA_FP32) launch<KDA_FP32>(a, s);
    else if (a.x.dtype == KDA_BF16) launch<KDA_BF16>(a, s);
    else launch<KDA_FP16>(a, s);
    return hipGetLastError();
}

}  // namespace kda
