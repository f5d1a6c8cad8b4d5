// Beam search's selection on gfx950. For beam w of a batch entry with logits
// x_w and running score s_w, candidate (w, t) has the value
//   s_w + x_wt - logsumexp(x_w);
// a finished beam has one candidate, its end token, at its own score. The n
// best candidates are kept, in the order of value, then of w * vocab + t.
//
// The logits are read once. beam_rows gives each chunk of a row to one
// workgroup, which keeps it in registers: the chunk's maximum, its sum of
// exp(x - maximum), and its n first (logit, token) keys, which are also its
// first by value. beam_pick joins the chunks: the log-sum-exp of each row and
// every value in fp64 (candidates of two beams can lie closer than fp32
// resolves), then n times the best head of the sorted lists.
#include "kda.h"
#include "state_pool_launch.h"

namespace kda {
namespace {

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LOG2E_LO = (float)(1.4426950408889634 - (double)LOG2E);
constexpr float LN2 = 0.6931471805599453f;
constexpr float NEG_INF = -__builtin_huge_valf();

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// fp32 order as unsigned order; -0 counts as 0, NaN as -inf.
__device__ __forceinline__ uint32_t sortable(float x) {
    const uint32_t u = __float_as_uint(x);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unsortable(uint32_t k) {
    return __uint_as_float(k ^ (k >> 31 ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ float clean(float x) { return x != x ? NEG_INF : x + 0.0f; }

// A key orders by logit, then by lower token; 0 is no candidate.
__device__ __forceinline__ uint64_t key_of(uint32_t s, uint32_t token) { return (uint64_t)s << 32 | ~token; }

template <int DT>
struct Elem;
template <>
struct Elem<KDA_FP32> {
    static constexpr int SIZE = 4;
    static __device__ __forceinline__ float get(const u32x4& v, int j) { return __uint_as_float(v[j]); }
    static __device__ __forceinline__ float at(const void* p, int64_t i) { return ((const float*)p)[i]; }
};
template <>
struct Elem<KDA_BF16> {
    static constexpr int SIZE = 2;
    static __device__ __forceinline__ float get(const u32x4& v, int j) {
        return __uint_as_float(j & 1 ? v[j >> 1] & 0xffff0000u : v[j >> 1] << 16);
    }
    static __device__ __forceinline__ float at(const void* p, int64_t i) {
        return __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16);
    }
};
template <>
struct Elem<KDA_FP16> {
    static constexpr int SIZE = 2;
    static __device__ __forceinline__ float half(uint32_t u) {
        return (float)__builtin_bit_cast(_Float16, (uint16_t)u);
    }
    static __device__ __forceinline__ float get(const u32x4& v, int j) {
        return half(j & 1 ? v[j >> 1] >> 16 : v[j >> 1] & 0xffffu);
    }
    static __device__ __forceinline__ float at(const void* p, int64_t i) { return half(((const uint16_t*)p)[i]); }
};

template <class T>
__device__ __forceinline__ T wave_max(T x) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const T y = __shfl_xor(x, d, 64);
        x = y > x ? y : x;
    }
    return x;
}

// 16 bytes from an address aligned to an element only.
template <int DT>
__device__ __forceinline__ u32x4 load16(const uint8_t* p) {
    u32x4 v;
    __builtin_memcpy(&v, __builtin_assume_aligned(p, Elem<DT>::SIZE), 16);
    return v;
}

// VECS 16-byte vectors per thread. A chunk's elements and the order of its sums
// depend on the row's length alone, not on its address: equal rows get equal
// sums, and their candidates tie. exp(x - m) is exp2 of (x - m) log2(e) with
// the product's rounding put back in, added in pairs and then in fp64, which
// leaves exp2's own last bit (2^-23) and one rounding (2^-24) at most.
template <int DT, int VECS>
__global__ __launch_bounds__(256) void beam_rows(BeamArgs a) {
    constexpr int PER = 16 / Elem<DT>::SIZE, N = VECS * PER;
    __shared__ uint64_t s_key[256];
    __shared__ uint64_t s_cand[kBeamPickMax * N];
    __shared__ float s_max[4];
    __shared__ double s_sum[4];
    __shared__ uint64_t s_edge;
    __shared__ int s_count;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int split = blockIdx.x % a.splits;
    const int64_t row = blockIdx.x / a.splits;
    if (a.finished && a.finished[row]) return;
    const uint8_t* base = (const uint8_t*)a.logits + row * a.row_stride * Elem<DT>::SIZE;
    const int first = split * a.chunk;
    float x[N];
    uint32_t best_s = 0, best_t = 0;
    float m = NEG_INF;
    if (tid == 0) s_count = 0;
    bool any = false;
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
        const int t0 = first + (i * 256 + tid) * PER;
        u32x4 v = {0, 0, 0, 0};
        const bool whole = t0 + PER <= a.vocab;
        if (whole) v = load16<DT>(base + (int64_t)t0 * Elem<DT>::SIZE);
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int t = t0 + j;
            float y = NEG_INF;
            if (whole) y = clean(Elem<DT>::get(v, j));
            else if (t < a.vocab) y = clean(Elem<DT>::at(base, t));
            x[i * PER + j] = y;
            m = y > m ? y : m;
            const uint32_t s = sortable(y);
            if (t < a.vocab && (!any || s > best_s)) {
                best_s = s;
                best_t = (uint32_t)t;
                any = true;
            }
        }
    }
    const uint64_t mine = any ? key_of(best_s, best_t) : 0;
    m = wave_max(m);
    if (lane == 0) s_max[wave] = m;
    s_key[tid] = mine;
    __syncthreads();
    m = fmaxf(fmaxf(s_max[0], s_max[1]), fmaxf(s_max[2], s_max[3]));
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < VECS; ++i)
#pragma unroll
        for (int j = 0; j < PER; j += 2) {
            float e[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const float y = x[i * PER + j + u], d = y - m;
                const float hi = d * LOG2E;
                const float lo = __builtin_fmaf(d, LOG2E, -hi) + d * LOG2E_LO;
                const float p = __builtin_amdgcn_exp2f(hi);
                // exp2 of a large negative number is 0, and y - m is 0 - 0 or
                // inf - inf where both are the maximum: that counts as 1
                e[u] = y == m ? 1.f : p > 0.f ? __builtin_fmaf(p, lo * LN2, p) : 0.f;
                if (first + (i * 256 + tid) * PER + j + u >= a.vocab) e[u] = 0.f;
            }
            sum += (double)(e[0] + e[1]);
        }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d, 64);
    if (lane == 0) s_sum[wave] = sum;
    // the n-th of the threads' first keys: the chunk's n first keys are at or
    // above it, and only n threads have keys there
    int rank = 0;
    for (int i = 0; i < 256; ++i) rank += s_key[i] > mine || (s_key[i] == mine && i < tid);
    if (rank == a.n - 1) s_edge = mine;
    __syncthreads();
    const uint64_t edge = s_edge;
    if (mine >= edge && mine != 0)
#pragma unroll
        for (int i = 0; i < VECS; ++i)
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                const int t = first + (i * 256 + tid) * PER + j;
                const uint64_t k = key_of(sortable(x[i * PER + j]), (uint32_t)t);
                if (t < a.vocab && k >= edge) s_cand[atomicAdd(&s_count, 1)] = k;
            }
    __syncthreads();
    const int count = s_count;
    uint64_t* out = a.keys + (row * a.splits + split) * a.n;
    for (int i = tid; i < count; i += 256) {
        const uint64_t k = s_cand[i];
        int r = 0;
        for (int j = 0; j < count; ++j) r += s_cand[j] > k;
        if (r < a.n) out[r] = k;
    }
    for (int i = count + tid; i < a.n; i += 256) out[i] = 0;
    if (tid == 0) {
        a.maxima[row * a.splits + split] = m;
        a.sums[row * a.splits + split] = s_sum[0] + s_sum[1] + s_sum[2] + s_sum[3];
    }
}

// A candidate of the selection: higher value first, then the lower beam, then
// the larger key (the candidates of one beam go by logit, which resolves more
// than the value does).
struct Cand {
    double v;
    uint32_t beam;  // NO_BEAM: none
    uint64_t key;
};
constexpr uint32_t NO_BEAM = 0xffffffffu;
__device__ __forceinline__ bool before(const Cand& x, const Cand& y) {
    return x.v > y.v || (x.v == y.v && (x.beam < y.beam || (x.beam == y.beam && x.key > y.key)));
}

// What a row adds to its logits.
constexpr int ROW_PLAIN = 0, ROW_EMPTY = 1, ROW_FINISHED = 2;

// Keys of a batch entry that are staged in LDS (48 KiB); larger entries are
// read from memory.
constexpr int PICK_LDS_KEYS = 6144;

// One wavefront per batch entry. A row is `splits` sorted lists, or one list
// made up on the spot: a finished beam's end token and then -inf, or -inf
// throughout (no logit or score above -inf). Each lane keeps the best head of
// its lists; a round takes the best of the lanes, and its owner moves on.
template <bool STAGED>
__global__ __launch_bounds__(64) void beam_pick(BeamArgs a) {
    __shared__ double s_log[kBeamMax];
    __shared__ float s_top[kBeamMax], s_score[kBeamMax];
    __shared__ int s_kind[kBeamMax];
    __shared__ uint64_t s_keys[STAGED ? PICK_LDS_KEYS : 1];
    extern __shared__ uint16_t s_pos[];  // [beams * splits] entries taken of each list
    const int lane = threadIdx.x;
    const int64_t row0 = (int64_t)blockIdx.x * a.beams;
    const int lists = a.beams * a.splits;
    const uint64_t* keys = a.keys + row0 * a.splits * a.n;
    if constexpr (STAGED)
        for (int i = lane; i < lists * a.n; i += 64) s_keys[i] = keys[i];
    // maximum and sum of the rows: `span` lanes (a power of two) per row
    const int span = a.beams > 32 ? 1 : a.beams > 16 ? 2 : a.beams > 8 ? 4 : a.beams > 4 ? 8 : 16;
    {
        const int w = lane / span, sub = lane % span;
        const bool row = w < a.beams && !(a.finished && a.finished[row0 + w]);
        const float* mx = a.maxima + (row0 + w) * a.splits;
        const double* sm = a.sums + (row0 + w) * a.splits;
        float top = NEG_INF;
        if (row)
            for (int i = sub; i < a.splits; i += span) top = mx[i] > top ? mx[i] : top;
        for (int d = 1; d < span; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
        double sum = 0;
        if (row)
            for (int i = sub; i < a.splits; i += span)
                sum += mx[i] == top ? sm[i] : sm[i] * exp((double)mx[i] - (double)top);
        for (int d = 1; d < span; d <<= 1) sum += __shfl_xor(sum, d, 64);
        if (w < a.beams && sub == 0) {
            const float sc = clean(a.scores[row0 + w]);
            s_kind[w] = !row ? ROW_FINISHED : top == NEG_INF || sc == NEG_INF ? ROW_EMPTY : ROW_PLAIN;
            s_top[w] = top;
            s_score[w] = sc;
            s_log[w] = log(sum);
        }
    }
    for (int l = lane; l < lists; l += 64) s_pos[l] = 0;
    __syncthreads();
    const double none = -__builtin_huge_val();
    auto head = [&](int l) {
        const int w = l / a.splits, pos = s_pos[l];
        Cand c{none, NO_BEAM, 0};
        const int kind = s_kind[w];
        if (kind == ROW_PLAIN) {
            const uint64_t k = pos < a.n ? (STAGED ? s_keys[l * a.n + pos] : keys[(int64_t)l * a.n + pos]) : 0;
            if (k) {
                const float x = unsortable((uint32_t)(k >> 32)), top = s_top[w];
                c.beam = w;
                c.key = k;
                if (x > NEG_INF) c.v = (x == top ? 0.0 : (double)x - (double)top) - s_log[w] + (double)s_score[w];
                if (c.v != c.v) c.v = none;  // no probability, at a score of +inf
            }
        } else if (l % a.splits == 0) {
            const float sc = s_score[w];
            // a finished beam's end token leads, unless it is itself at -inf: then its place is that of its index
            const bool lead = kind == ROW_FINISHED && sc > NEG_INF;
            const int t = !lead ? pos : pos == 0 ? a.eos : pos - 1 < a.eos ? pos - 1 : pos;
            if (t < a.vocab) {
                c.beam = w;
                c.key = key_of(sortable(lead && pos == 0 ? 0.f : NEG_INF), (uint32_t)t);
                if (lead && pos == 0) c.v = sc;
            }
        }
        return c;
    };
    Cand best;
    int from;
    auto rescan = [&] {
        best = Cand{none, NO_BEAM, 0};
        from = 0;
        for (int l = lane; l < lists; l += 64) {
            const Cand c = head(l);
            if (before(c, best)) {
                best = c;
                from = l;
            }
        }
    };
    rescan();
    for (int i = 0; i < a.n; ++i) {
        double top = best.v;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) top = fmax(top, __shfl_xor(top, d, 64));
        uint64_t at = __ballot(best.v == top && best.beam != NO_BEAM);
        if (at & (at - 1)) {  // equal values: compare the rest
            Cand w = best.v == top ? best : Cand{none, NO_BEAM, 0};
            uint32_t beam = w.beam;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const uint32_t o = __shfl_xor(beam, d, 64);
                beam = o < beam ? o : beam;
            }
            uint64_t key = w.beam == beam ? w.key : 0;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const uint64_t o = __shfl_xor((unsigned long long)key, d, 64);
                key = o > key ? o : key;
            }
            at = __ballot(best.v == top && best.beam == beam && best.key == key);
        }
        if (at >> lane & 1) {
            const int64_t o = (int64_t)blockIdx.x * a.n + i;
            const int32_t token = (int32_t)~(uint32_t)best.key;
            a.out_scores[o] = (float)best.v;
            a.out_parents[o] = (int32_t)best.beam;
            a.out_tokens[o] = token;
            if (a.out_finished) a.out_finished[o] = token == a.eos || s_kind[best.beam] == ROW_FINISHED;
            s_pos[from] += 1;
            rescan();
        }
    }
}

template <int DT>
hipError_t rows(const BeamArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)((int64_t)a.batch * a.beams * a.splits)), block(256);
    constexpr int PER = 16 / Elem<DT>::SIZE;
    const int vecs = a.chunk / (256 * PER);
    if (vecs * PER == 32) hipLaunchKernelGGL((beam_rows<DT, 32 / PER>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((beam_rows<DT, 8 / PER>), grid, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_beam_rows(const BeamArgs& a, int dtype, hipStream_t s) {
    if (dtype == KDA_FP32) return rows<KDA_FP32>(a, s);
    if (dtype == KDA_BF16) return rows<KDA_BF16>(a, s);
    return rows<KDA_FP16>(a, s);
}

hipError_t launch_beam_pick(const BeamArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)a.batch), block(64);
    const int64_t lists = (int64_t)a.beams * a.splits;
    if (lists * a.n <= PICK_LDS_KEYS) hipLaunchKernelGGL(beam_pick<true>, grid, block, (size_t)lists * 2, s, a);
    else hipLaunchKernelGGL(beam_pick<false>, grid, block, (size_t)lists * 2, s, a);
    return hipGetLastError();
}

}  // namespace kda
