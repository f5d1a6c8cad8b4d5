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
// resolves), then the n best entries of the sorted lists.
#include "kda.h"
#include "state_pool_launch.h"

namespace kda {
namespace {

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LOG2E_LO = (float)(1.4426950408889634 - (double)LOG2E);
constexpr double LN2 = 0.6931471805599453;
// Up to this maximum a chunk's exponentials are taken as they are: e^48 and its
// sums are far inside fp32, and what flushes to zero (logits below -87) is below
// e^-39 of the maximum's term. Beyond it, with |x - m| < 32, x and m are both
// multiples of 2^-19 (|x| > 16, |m| > 32), and so is their difference, which
// 24 bits hold; terms further off are below e^-32 of the maximum's.
constexpr float REF_MAX = 48.f;
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

__device__ __forceinline__ void set16(u32x4& v, int j, uint32_t x) {
    v[j >> 1] = j & 1 ? (v[j >> 1] & 0xffffu) | x << 16 : x;
}

template <int DT>
struct Elem;
template <>
struct Elem<KDA_FP32> {
    static constexpr int SIZE = 4;
    static constexpr uint32_t NONE = 0xff800000u;  // -inf
    static __device__ __forceinline__ float get(const u32x4& v, int j) { return __uint_as_float(v[j]); }
    static __device__ __forceinline__ void set(u32x4& v, int j, uint32_t x) { v[j] = x; }
    static __device__ __forceinline__ uint32_t raw(const void* p, int64_t i) { return ((const uint32_t*)p)[i]; }
};
template <>
struct Elem<KDA_BF16> {
    static constexpr int SIZE = 2;
    static __device__ __forceinline__ float get(const u32x4& v, int j) {
        return __uint_as_float(j & 1 ? v[j >> 1] & 0xffff0000u : v[j >> 1] << 16);
    }
    static constexpr uint32_t NONE = 0xff80u;
    static __device__ __forceinline__ void set(u32x4& v, int j, uint32_t x) { set16(v, j, x); }
    static __device__ __forceinline__ uint32_t raw(const void* p, int64_t i) { return ((const uint16_t*)p)[i]; }
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
    static constexpr uint32_t NONE = 0xfc00u;
    static __device__ __forceinline__ void set(u32x4& v, int j, uint32_t x) { set16(v, j, x); }
    static __device__ __forceinline__ uint32_t raw(const void* p, int64_t i) { return ((const uint16_t*)p)[i]; }
};

__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) x = fmaxf(x, __shfl_xor(x, d, 64));
    return x;
}

// 16 bytes from an address aligned to an element only.
template <int DT>
__device__ __forceinline__ u32x4 load16(const uint8_t* p) {
    u32x4 v;
    __builtin_memcpy(&v, __builtin_assume_aligned(p, Elem<DT>::SIZE), 16);
    return v;
}

// The n-th largest key of a wavefront's 64 (n <= 64; keys differ, or are 0):
// the value bit by bit from ballots, then the token among the lanes that hold
// that value.
__device__ __forceinline__ uint64_t nth_key(uint32_t value, uint32_t token, int n) {
    uint32_t v = 0;
#pragma unroll
    for (int b = 31; b >= 0; --b) {
        const uint32_t c = v | 1u << b;
        v = __popcll(__ballot(value >= c)) >= n ? c : v;
    }
    if (v == 0) return 0;
    uint64_t tied = __ballot(value == v);
    int left = n - __popcll(__ballot(value > v));  // how many of the tied ones count
    uint32_t t = 0;
    while (left-- > 0) {
        uint32_t low = tied >> (threadIdx.x & 63) & 1 ? token : 0xffffffffu;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const uint32_t o = __shfl_xor(low, d, 64);
            low = o < low ? o : low;
        }
        t = low;
        tied &= ~__ballot(token == low && (tied >> (threadIdx.x & 63) & 1));
    }
    return key_of(v, t);
}

// One workgroup of 256 threads per chunk of a row, N elements per thread in
// VECS 16-byte vectors.
//
// Sums. A chunk's elements and the order of its sums depend on the row's
// length alone, not on its address: equal rows get equal sums, and their
// candidates tie. Terms are exp(x - r) with r = 0 where the maximum m allows it,
// so that no bit of x is lost (x - m in fp32 is off by 2^-21 from |x - m| = 8 on,
// the same way for equal logits), and r = m beyond REF_MAX, where x - m is exact
// as long as the term counts. exp(d) is exp2 of d log2(e); that product's rounding
// is put back in by a sum of its own, sum(exp2 * rounding). The exponentials are
// added in pairs and then in fp64, which leaves exp2's own last bit (2^-23) and
// one rounding (2^-24) at most.
//
// Keys. The 256 threads form 64 groups of 4 (one lane of each wavefront). The
// n-th largest of the groups' first keys is a lower edge of the chunk's n first
// keys, and only n groups have keys at or above it: those (at most 4 n N, in
// practice little more than n) are ranked by counting.
//
// Measured on 32 x 8 rows of 131072 bf16 logits, n = 16 (67 MB): 28 us, 2.4 TB/s,
// half of it the stream and half vector instructions: the exponentials, the
// first keys (a compare and two selects per logit) and the edge (71 us with the
// edge from ranks over all 256 threads' first keys). Every load of a thread is
// in flight at once.
template <int DT, int VECS>
__global__ __launch_bounds__(kBeamThreads) void beam_rows(BeamArgs a) {
    constexpr int PER = 16 / Elem<DT>::SIZE, N = VECS * PER;
    extern __shared__ uint64_t s_cand[];  // [4 n N]
    __shared__ uint32_t s_value[4][64], s_token[4][64];
    __shared__ float s_max[4];
    __shared__ double s_sum[4], s_scale;
    __shared__ uint64_t s_edge;
    __shared__ int s_count;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int split = blockIdx.x % a.splits;
    const int64_t row = blockIdx.x / a.splits;
    if (a.finished && a.finished[row]) return;
    const uint8_t* base = (const uint8_t*)a.logits + row * a.row_stride * Elem<DT>::SIZE;
    const int first = split * a.chunk + tid * PER;  // vector i starts at first + 256 PER i
    u32x4 x[VECS];
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
        const int t0 = first + i * 256 * PER;
        if (t0 + PER <= a.vocab) {
            x[i] = load16<DT>(base + (int64_t)t0 * Elem<DT>::SIZE);
        } else {
#pragma unroll
            for (int j = 0; j < PER; ++j)
                Elem<DT>::set(x[i], j, t0 + j < a.vocab ? Elem<DT>::raw(base, t0 + j) : Elem<DT>::NONE);
        }
    }
    if (tid == 0) s_count = 0;
    // the thread's first key: NaN never compares greater; all -inf leaves the first token
    float best = NEG_INF;
    int at = 0;
#pragma unroll
    for (int i = 0; i < VECS; ++i)
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const float y = Elem<DT>::get(x[i], j);
            if (y > best) {
                best = y;
                at = i * 256 * PER + j;
            }
        }
    const bool any = first < a.vocab;
    s_value[wave][lane] = any ? sortable(best + 0.0f) : 0u;
    s_token[wave][lane] = (uint32_t)(first + at);
    const float wm = wave_max(best);
    if (lane == 0) s_max[wave] = wm;
    __syncthreads();
    if (wave == 0) {
        uint32_t v = s_value[0][lane], t = s_token[0][lane];
#pragma unroll
        for (int w = 1; w < 4; ++w) {
            const uint32_t ov = s_value[w][lane], ot = s_token[w][lane];
            if (ov > v || (ov == v && ot < t)) {
                v = ov;
                t = ot;
            }
        }
        const uint64_t edge = nth_key(v, t, a.n);
        if (lane == 0) s_edge = edge;
    }
    const float m = fmaxf(fmaxf(s_max[0], s_max[1]), fmaxf(s_max[2], s_max[3]));
    const float ref = __builtin_fabsf(m) <= REF_MAX ? 0.f : m;
    if (wave == 1) {  // the sum is handed on relative to the maximum; the first wavefront forms the edge meanwhile
        const double f = ref == m ? 1.0 : exp(-(double)m);
        if (lane == 0) s_scale = f;
    }
    double sum = 0.0;
    if (__builtin_isinf(m)) {  // no logit above -inf: all count as 1; or some at +inf, which share the row
#pragma unroll
        for (int i = 0; i < VECS; ++i)
#pragma unroll
            for (int j = 0; j < PER; ++j)
                if (first + i * 256 * PER + j < a.vocab && Elem<DT>::get(x[i], j) == m) sum += 1.0;
    } else {
        float rest = 0.f;  // sum of exp2(hi) * lo
#pragma unroll
        for (int i = 0; i < VECS; ++i)
#pragma unroll
            for (int j = 0; j < PER; j += 2) {
                float e[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    // -inf and NaN become -200, whose exponential is 0
                    const float d = fmaxf(Elem<DT>::get(x[i], j + u) - ref, -200.f);
                    const float hi = d * LOG2E;
                    const float lo = __builtin_fmaf(d, LOG2E_LO, __builtin_fmaf(d, LOG2E, -hi));
                    e[u] = __builtin_amdgcn_exp2f(hi);
                    rest = __builtin_fmaf(e[u], lo, rest);
                }
                sum += (double)(e[0] + e[1]);
            }
        sum += (double)rest * LN2;
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d, 64);
    if (lane == 0) s_sum[wave] = sum;
    __syncthreads();
    const uint64_t edge = s_edge;
    const float edge_value = edge ? unsortable((uint32_t)(edge >> 32)) : NEG_INF;
    if (any && best >= edge_value)
#pragma unroll
        for (int i = 0; i < VECS; ++i)
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                const float y = clean(Elem<DT>::get(x[i], j));
                const int t = first + i * 256 * PER + j;
                if (y >= edge_value && t < a.vocab) {
                    const uint64_t k = key_of(sortable(y), (uint32_t)t);
                    if (k >= edge) s_cand[atomicAdd(&s_count, 1)] = k;
                }
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
        a.sums[row * a.splits + split] = (s_sum[0] + s_sum[1] + s_sum[2] + s_sum[3]) * s_scale;
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

// Keys of a batch entry that are staged in LDS, and lists that a lane then keeps
// the heads of in registers; larger entries are read from memory.
constexpr int PICK_LDS_KEYS = 5632, PICK_LANE_LISTS = 4;
constexpr int PICK_RANKED = 512;  // candidates that are ranked by counting

// Unsigned order of a candidate's value; 0 is no candidate.
__device__ __forceinline__ uint64_t order_of(const Cand& c) {
    const uint64_t bits = __builtin_bit_cast(uint64_t, c.v);
    return c.beam == NO_BEAM ? 0 : bits ^ (bits >> 63 ? ~0ull : 1ull << 63);
}

// The larger of two unsigned numbers over the wavefront, by DPP.
__device__ __forceinline__ uint32_t wave_umax(uint32_t x) {
#define KDA_UMAX(CTRL)                                                                               \
    {                                                                                                \
        const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xF, 0xF, false); \
        x = o > x ? o : x;                                                                           \
    }
    KDA_UMAX(0x111) KDA_UMAX(0x112) KDA_UMAX(0x114) KDA_UMAX(0x118) KDA_UMAX(0x142) KDA_UMAX(0x143)
#undef KDA_UMAX
    return (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
}

// One workgroup per batch entry. A row is `splits` sorted lists, or one list
// made up on the spot: a finished beam's end token and then -inf, or -inf
// throughout (no logit or score above -inf). All wavefronts stage the keys. The
// n-th best of 256 entries, the first of every list (by the upper bits of the
// value), is a lower edge of the n best; the candidates at or above it, little
// more than n, are ranked by counting. Where more than PICK_RANKED tie, and
// where the keys do not fit LDS, the first wavefront takes n rounds: each lane
// keeps the heads of its lists, the best of them goes out and its owner moves
// on. Bound by latency: 32 entries of 8 beams and 128 lists with n = 16 take
// 11 us, of which 3 are the launch (23 with the rounds on lists in memory); 32
// lists with n = 16 as many (16 by rounds).
template <bool STAGED>
__global__ __launch_bounds__(kBeamThreads) void beam_pick(BeamArgs a) {
    __shared__ double s_log[kBeamMax];
    __shared__ float s_top[kBeamMax], s_score[kBeamMax];
    __shared__ int s_kind[kBeamMax];
    __shared__ uint64_t s_keys[STAGED ? PICK_LDS_KEYS : 1];
    __shared__ uint64_t s_order[STAGED ? PICK_RANKED : 1], s_key[STAGED ? PICK_RANKED : 1];
    __shared__ uint32_t s_beam[STAGED ? PICK_RANKED : 1], s_first[STAGED ? 64 * PICK_LANE_LISTS : 1], s_edge;
    __shared__ int s_count;
    extern __shared__ uint16_t s_pos[];  // [beams * splits] entries taken of each list
    const int tid = threadIdx.x, lane = tid & 63;
    const int64_t row0 = (int64_t)blockIdx.x * a.beams;
    const int lists = a.beams * a.splits;
    const uint64_t* keys = a.keys + row0 * a.splits * a.n;
    if constexpr (STAGED) {
        const int total = lists * a.n;
        for (int base = tid; base < total; base += 8 * 256) {  // eight loads in flight
            uint64_t k[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) k[j] = keys[base + 256 * j < total ? base + 256 * j : base];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (base + 256 * j < total) s_keys[base + 256 * j] = k[j];
        }
    }
    // maximum and sum of the rows: 16 lanes per row
    for (int w0 = 0; w0 < a.beams; w0 += 16) {
        const int w = w0 + (tid >> 4), sub = tid & 15;
        const bool row = w < a.beams && !(a.finished && a.finished[row0 + w]);
        const float* mx = a.maxima + (row0 + w) * a.splits;
        const double* sm = a.sums + (row0 + w) * a.splits;
        const float m0 = row && sub < a.splits ? mx[sub] : NEG_INF;
        const double s0 = row && sub < a.splits ? sm[sub] : 0;
        float top = m0;
        if (row)
            for (int i = sub + 16; i < a.splits; i += 16) top = mx[i] > top ? mx[i] : top;
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
        auto part = [&](float m, double s) { return m == top ? s : s * exp((double)m - (double)top); };
        double sum = part(m0, s0);
        if (row)
            for (int i = sub + 16; i < a.splits; i += 16) sum += part(mx[i], sm[i]);
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) sum += __shfl_xor(sum, d, 64);
        if (w < a.beams && sub == 0) {
            const float sc = clean(a.scores[row0 + w]);
            s_kind[w] = !row ? ROW_FINISHED : top == NEG_INF || sc == NEG_INF ? ROW_EMPTY : ROW_PLAIN;
            s_top[w] = top;
            s_score[w] = sc;
            s_log[w] = log(sum);
        }
    }
    if constexpr (!STAGED)
        for (int l = tid; l < lists; l += 256) s_pos[l] = 0;
    if (tid == 0) s_count = 0;
    __syncthreads();
    const double none = -__builtin_huge_val();
    // entry `pos` of list l, which belongs to beam w: its key (0: none) and value
    auto entry = [&](int l, int w, int pos, bool first_list) __attribute__((always_inline)) {
        Cand c{none, NO_BEAM, 0};
        const int kind = s_kind[w];
        const float sc = s_score[w];
        if (kind == ROW_PLAIN) {
            c.key = pos < a.n ? (STAGED ? s_keys[l * a.n + pos] : keys[(int64_t)l * a.n + pos]) : 0;
            const float x = unsortable((uint32_t)(c.key >> 32)), top = s_top[w];
            if (c.key && x > NEG_INF) {
                const double v = (x == top ? 0.0 : (double)x - (double)top) - s_log[w] + (double)sc;
                c.v = v == v ? v + 0.0 : none;  // NaN: no probability, at a score of +inf
            }
        } else if (first_list) {
            // a finished beam's end token leads, unless it is itself at -inf: then its place is that of its index
            const bool lead = kind == ROW_FINISHED && sc > NEG_INF;
            const int t = !lead ? pos : pos == 0 ? a.eos : pos - 1 < a.eos ? pos - 1 : pos;
            if (t < a.vocab) c.key = key_of(sortable(lead && pos == 0 ? 0.f : NEG_INF), (uint32_t)t);
            if (lead && pos == 0) c.v = (double)sc + 0.0;
        }
        if (c.key) c.beam = (uint32_t)w;
        return c;
    };
    auto emit = [&](int i, double v, uint32_t beam, uint64_t key) __attribute__((always_inline)) {
        const int64_t o = (int64_t)blockIdx.x * a.n + i;
        const int32_t token = (int32_t)~(uint32_t)key;
        a.out_scores[o] = (float)v;
        a.out_parents[o] = (int32_t)beam;
        a.out_tokens[o] = token;
        if (a.out_finished) a.out_finished[o] = token == a.eos || s_kind[beam] == ROW_FINISHED;
    };
    Cand best;
    int from;
    // the lane's lists lane + 64q
    Cand head[PICK_LANE_LISTS];
    int pos[PICK_LANE_LISTS], beam[PICK_LANE_LISTS];
    auto choose = [&]() __attribute__((always_inline)) {
        best = Cand{none, NO_BEAM, 0};
        from = 0;
        if constexpr (STAGED) {
#pragma unroll
            for (int q = 0; q < PICK_LANE_LISTS; ++q)
                if (before(head[q], best)) {
                    best = head[q];
                    from = q;
                }
        } else {
            for (int l = lane; l < lists; l += 64) {
                const Cand c = entry(l, l / a.splits, s_pos[l], l % a.splits == 0);
                if (before(c, best)) {
                    best = c;
                    from = l;
                }
            }
        }
    };
    if constexpr (STAGED) {
        // the threads share the lists evenly, each every `step`-th entry of one
        const int shift = lists > 1 ? 32 - __builtin_clz(lists - 1) : 0, step = 256 >> shift;
        const int l = tid >> (8 - shift), w = l / a.splits;
        int i = tid & (step - 1);
        Cand c{none, NO_BEAM, 0};
        if (l < lists && i < a.n) c = entry(l, w, i, l == w * a.splits);
        uint64_t order = order_of(c);
        s_first[tid] = (uint32_t)(order >> 32);
        __syncthreads();
        if (tid < 64) {
            uint32_t x[4], v = 0;
#pragma unroll
            for (int q = 0; q < 4; ++q) x[q] = s_first[lane + 64 * q];
#pragma unroll
            for (int b = 31; b >= 12; --b) {  // 8 bits of a double's mantissa are enough
                const uint32_t e = v | 1u << b;
                int count = 0;
#pragma unroll
                for (int q = 0; q < 4; ++q) count += __popcll(__ballot(x[q] >= e));
                v = count >= a.n ? e : v;
            }
            if (tid == 0) s_edge = v;
        }
        __syncthreads();
        const uint32_t edge = s_edge;
        while (order != 0 && (uint32_t)(order >> 32) >= edge) {
            const int at = atomicAdd(&s_count, 1);
            if (at < PICK_RANKED) {
                s_order[at] = order;
                s_beam[at] = c.beam;
                s_key[at] = c.key;
            }
            if ((i += step) >= a.n) break;
            c = entry(l, w, i, l == w * a.splits);
            order = order_of(c);
        }
        __syncthreads();
        const int count = s_count;
        if (count <= PICK_RANKED) {
            for (int i = tid; i < count; i += 256) {
                const uint64_t order = s_order[i], key = s_key[i];
                const uint32_t beam = s_beam[i];
                int rank = 0;
                for (int j = 0; j < count; ++j) {
                    const uint64_t o = s_order[j];
                    rank += o > order || (o == order && (s_beam[j] < beam || (s_beam[j] == beam && s_key[j] > key)));
                }
                const uint64_t bits = order >> 63 ? order ^ 1ull << 63 : ~order;
                if (rank < a.n) emit(rank, __builtin_bit_cast(double, bits), beam, key);
            }
            return;
        }
    }
    if (tid >= 64) return;
    if constexpr (STAGED) {
#pragma unroll
        for (int q = 0; q < PICK_LANE_LISTS; ++q) {
            const int l = lane + 64 * q;
            pos[q] = 0;
            beam[q] = l < lists ? l / a.splits : 0;
            head[q] = l < lists ? entry(l, beam[q], 0, l == beam[q] * a.splits) : Cand{none, NO_BEAM, 0};
        }
    }
    choose();
    for (int i = 0; i < a.n; ++i) {
        const uint64_t order = order_of(best);
        const uint32_t hi = wave_umax((uint32_t)(order >> 32));
        uint64_t at = __ballot((uint32_t)(order >> 32) == hi);
        if (at & (at - 1)) {  // the rest of the value, then beam and key
            const uint32_t lo = wave_umax(at >> lane & 1 ? (uint32_t)order : 0u);
            at = __ballot((at >> lane & 1) && (uint32_t)order == lo);
            const uint32_t beam = ~wave_umax(at >> lane & 1 ? ~best.beam : 0u);
            at = __ballot((at >> lane & 1) && best.beam == beam);
            const uint32_t k1 = wave_umax(at >> lane & 1 ? (uint32_t)(best.key >> 32) : 0u);
            at = __ballot((at >> lane & 1) && (uint32_t)(best.key >> 32) == k1);
            const uint32_t k0 = wave_umax(at >> lane & 1 ? (uint32_t)best.key : 0u);
            at = __ballot((at >> lane & 1) && (uint32_t)best.key == k0);
        }
        if (at >> lane & 1 && best.beam != NO_BEAM) {
            emit(i, best.v, best.beam, best.key);
            if constexpr (STAGED) {
#pragma unroll
                for (int q = 0; q < PICK_LANE_LISTS; ++q)
                    if (q == from) {
                        const int l = lane + 64 * q;
                        head[q] = entry(l, beam[q], ++pos[q], l == beam[q] * a.splits);
                    }
            } else {
                s_pos[from] += 1;
            }
            choose();
        }
    }
}

template <int DT>
hipError_t rows(const BeamArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)((int64_t)a.batch * a.beams * a.splits)), block(kBeamThreads);
    constexpr int PER = 16 / Elem<DT>::SIZE;
    const int vecs = a.chunk / (256 * PER);
    const size_t lds = (size_t)4 * a.n * vecs * PER * sizeof(uint64_t);
    if (vecs * PER == 32) hipLaunchKernelGGL((beam_rows<DT, 32 / PER>), grid, block, lds, s, a);
    else hipLaunchKernelGGL((beam_rows<DT, 8 / PER>), grid, block, lds, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_beam_rows(const BeamArgs& a, int dtype, hipStream_t s) {
    if (dtype == KDA_FP32) return rows<KDA_FP32>(a, s);
    if (dtype == KDA_BF16) return rows<KDA_BF16>(a, s);
    return rows<KDA_FP16>(a, s);
}

hipError_t launch_beam_pick(const BeamArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)a.batch), block(kBeamThreads);
    const int64_t lists = (int64_t)a.beams * a.splits;
    if (lists * a.n <= PICK_LDS_KEYS && lists <= 64 * PICK_LANE_LISTS)
        hipLaunchKernelGGL(beam_pick<true>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(beam_pick<false>, grid, block, (size_t)lists * 2, s, a);
    return hipGetLastError();
}

}  // namespace kda
