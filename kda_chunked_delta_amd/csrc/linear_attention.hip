// Linear attention with one decay per head on gfx950 (CDNA4): chunked prefill
// and recurrent decode over a 128 x 128 fp32 state per head:
//   S_t = exp(g_t) S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t
// with a log-decay g per token and head, or one per head for all tokens.
//
// Chunked form. For a chunk of rows r = 0 .. 31 with start state S and G_r the
// running sum of g inside the chunk:
//   A = lower((q_r . k_i) exp(G_r - G_i))
//   O = scale (diag(exp(G)) Q S + A V)
//   S <- exp(G_31) S + K^T diag(exp(G_31 - G)) V
// The decay is one number per row: it scales rows of results, and V on its way
// into the state, never q and k, which go to the matrix instructions as they
// are in memory. What is computed in fp32 and then multiplied is rounded so:
//   - diag(exp(G_31 - G)) V becomes the sum of three bf16 numbers, all 24 bits of
//     its mantissa, since the state keeps its sum: one bf16 would leave up to 2^-8 of
//     each token in an fp32 state, two 2^-17 (2e-6 of its norm). The third part costs
//     7 to 8% (16 prompts of 2048 tokens and 64 heads 424 and 461 us);
//   - A becomes a pair hi + lo (2^-17): a rounding of one of its few large values
//     would reach a whole row of an output, and not average out (2 to 3%);
//   - the copy of S that Q S multiplies becomes one bf16 (2^-8 at most of each
//     value). It is read and not kept: its rounding reaches one output, as a sum over
//     128 channels that is rounded to bf16 itself, 1.7e-3 of its norm, and adds up to
//     2.3e-3 with that. A pair would leave the 1.7e-3, for 16 more products a chunk:
//     1.29 against 1.12 us with 8 workgroups, 522 against 453 us for the 16 prompts,
//     195 against 169 for eight packed ones. (The gated delta rule reads its state into
//     what it writes next, and takes the pair.)
// All sums are fp32, the running sum of g is fp64 (differences of it are taken).
// A decay near 1 is applied as its difference to 1, so that its error does not add up
// over the chunks that a state remembers. What is left of an fp32 state's error is the
// rounding of its sums, some seven a chunk without a preferred sign: 6e-8 of its norm
// after 32 tokens, 3e-7 after 1024, 9e-7 after 8192, 2.6e-6 after 65536, with slow
// decays, and a third of that in the segments of a plan. (A decay that is a few steps
// of the state's last bit a chunk is rounded to whole ones: 3.7e-6 after 65536 tokens
// of -1e-8.)
#include "chunk_tiles.hpp"
#include "linear_attention_launch.h"

#include <mutex>

namespace kda {
namespace {

static_assert(kLaChunk == TILE_ROWS);

// Per-row values of a chunk, fp32 [4][32]: the running log2-decay as hi + lo,
// exp(G) and exp(G_31 - G). Then the chunk's decay exp(G_31) as the state takes it: {1, d}
// where it is 1 + d in [1/2, 2], the state becoming S + d S, else {p, 0}, p S.
constexpr int LS_H = 0, LS_L = 32, LS_GAM = 64, LS_LAST = 96, LS_STEP = 128, LS_FLOATS = 132;

constexpr double LN2 = 0.6931471805599453;
// e^y - 1 for |y| <= ln 2, its series up to y^10 / 10! (1e-8 of the value is left out).
__device__ __forceinline__ float expm1_small(float y) {
    constexpr float c[9] = {1.f / 3628800, 1.f / 362880, 1.f / 40320, 1.f / 5040, 1.f / 720,
                            1.f / 120,     1.f / 24,     1.f / 6,     1.f / 2};
    float q = c[0];
#pragma unroll
    for (int i = 1; i < 9; ++i) q = __builtin_fmaf(q, y, c[i]);
    return __builtin_fmaf(y * y, q, y);
}

// One fp32 number for a decay near 1 is off by up to 2^-25, and with a fixed
// log-decay by the same in every chunk that the state remembers: 2048 chunks of
// -1e-6, -1e-5 and -3e-5 a token left the state 1e-5, 9e-6 and 2e-5 off. d is off by
// 2^-23 of what the chunk forgets instead, whatever the number of chunks.
//
// One wavefront: x = the log-decay of row lane & 31, after the log2-decay of the
// tokens behind the chunk, which the last values get in addition. Returns the
// chunk's log2-decay. {p, d} go with outputs alone.
template <bool OUT>
__device__ __forceinline__ double row_scan(float x, double after, int lane, float* gs) {
    const int r = lane & 31;
    x *= LOG2E;
    double G = x < LOG2_FLOOR ? LOG2_FLOOR : x;
#pragma unroll
    for (int d = 1; d < TILE_ROWS; d <<= 1) {
        const double y = __shfl_up(G, d, 32);
        if (r >= d) G += y;
    }
    const double all = __shfl(G, 31, 32);
    const float hi = (float)G;
    if (lane < TILE_ROWS) {
        gs[LS_H + r] = hi;
        gs[LS_L + r] = (float)(G - (double)hi);
        gs[LS_GAM + r] = exp2_hw(hi);
        gs[LS_LAST + r] = exp2_hw((float)(all - G + after));
    }
    if (OUT && lane == 31) {
        const bool near = all >= -1.0 && all <= 1.0;
        gs[LS_STEP] = near ? 1.f : exp2_hw(hi);
        gs[LS_STEP + 1] = near ? expm1_small((float)(all * LN2)) : 0.f;
    }
    return all;
}

// Rows lane & 31 of a tile, the granule of step s of channel tile t: 4t + 2s + h.
__device__ __forceinline__ u32x4 row32(const uint8_t* tile, int at_row, int t, int s) {
    return *(const u32x4*)(tile + (at_row ^ ((4 * t + 2 * s) << 4)));
}

// A of a chunk as the operand of A V, hi and lo: [2][step s 2][lane 64][8 bf16], lane
// l holding token l & 31 and the keys 16s + 8 (j >> 2) + 4 (l >> 5) + (j & 3).
// One wavefront forms the 16 x 16 tile of tokens 16 rt .. and keys 16 ct .. :
// lane (gg, m) has token 16 rt + m and keys 16 ct + 4 gg + b, half a lane's
// entry. Tile (0, 1) is zero; it is cleared once and never written.
constexpr int A_LO = 2048, A_BYTES = 4096;
__device__ __forceinline__ uint8_t* a_tile(uint8_t* rec, int rt, int ct, int lane) {
    const int gg = lane >> 4, m = lane & 15;
    return rec + ct * 1024 + (32 * (gg & 1) + 16 * rt + m) * 16 + 8 * (gg >> 1);
}
__device__ __forceinline__ u32x4 row16(const uint8_t* tile, int row0, int p, int lane) {
    return *(const u32x4*)(tile + tile_off(row0 + (lane & 15), 4 * p + (lane >> 4)));
}
template <int RT, int CT>
__device__ __forceinline__ void form_a(const uint8_t* Q, const uint8_t* K, const float* gs, float scale, uint8_t* rec,
                                       int lane) {
    const int gg = lane >> 4, m = lane & 15;
    f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int p = 0; p < 4; ++p) x = mfma_k32(row16(K, 16 * CT, p, lane), row16(Q, 16 * RT, p, lane), x);
    const f32x4 hv = *(const f32x4*)(gs + LS_H + 16 * CT + 4 * gg), lv = *(const f32x4*)(gs + LS_L + 16 * CT + 4 * gg);
    const float hm = gs[LS_H + 16 * RT + m], lm = gs[LS_L + 16 * RT + m];
#pragma unroll
    for (int b = 0; b < 4; ++b)
        x[b] = CT < RT || 4 * gg + b <= m ? scale * x[b] * pair_decay(hm, lm, hv[b], lv[b]) : 0.f;
    const HiLo y = split4(x);
    *(u32x2*)a_tile(rec, RT, CT, lane) = y.h;
    *(u32x2*)(a_tile(rec, RT, CT, lane) + A_LO) = y.l;
}

// A wait for the wavefront's LDS traffic that the compiler counts: it then knows
// that loads issued before have come, and does not wait for later ones instead.
__device__ __forceinline__ void counted_wait() {
    sched_fence();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
    asm volatile("" ::: "memory");
    sched_fence();
}

// Sixteen weighted values of a lane as three bf16 operands a + b + c that make
// them up (8 bits of mantissa each).
struct Split3 {
    u32x4 a[2], b[2], c[2];
};
// Their formation in parts, to go beside other products. Values 2n and 2n + 1 of
// the lane's 16, first weighted (x), then what is left of them.
template <int N>
__device__ __forceinline__ void weigh(f32x16& x, const u32x4 (&v)[2], const f32x4 (&w)[4], u32x4 (&to)[2]) {
    const uint32_t p = v[N >> 2][N & 3];
    x[2 * N] = w[N >> 1][2 * (N & 1)] * bf16_lo(p);
    x[2 * N + 1] = w[N >> 1][2 * (N & 1) + 1] * bf16_hi(p);
    to[N >> 2][N & 3] = pack_bf16(x[2 * N], x[2 * N + 1]);
}

// f(0), f(1), .. f(N - 1) with the number as a constant.
template <int N, class F>
__device__ __forceinline__ void unrolled(F f) {
    if constexpr (N > 0) {
        unrolled<N - 1>(f);
        f(std::integral_constant<int, N - 1>{});
    }
}

// Prefill: one workgroup per (unit, head), in a software pipeline with one
// barrier per chunk. In interval i
//   wavefronts 4 .. 7 advance the state over chunk i (32 value columns each)
//     and form its output;
//   wavefronts 0 .. 3 issue the direct-to-LDS loads of q, k and v of chunk
//     i + AHEAD (8 rows each), which stay in flight for AHEAD - 2 intervals;
//     0, 1 and 2 form a tile of A of chunk i + 1 each, 3 the row values of chunk
//     i + 2, and loads the log-decays of chunk i + AHEAD + 1.
// The output leaves through LDS: the state wavefronts put theirs of chunk i into
// a tile, and wavefronts 0 .. 3 store whole rows of it in interval i + 1.
// Without OUT (a segment's end state from zero) the chunks are taken from the
// last to the first, V weighted by the decay up to the segment's end: the state
// is never scaled, and the workgroup stops where that decay is zero in fp32
// (below 2^-160), after a few chunks of a head that forgets fast. Not where a
// log-decay before is above zero, which could bring earlier tokens back, or NaN.
// Ring slots: the tiles AHEAD + 1 chunks, A and the output 2, the row values 3.
//
// Bound by memory where every compute unit is at work: 4.6 to 4.75 TB/s of q, k, v
// and o, where a copy of 1 GiB reaches 5.15 (1.73 us a chunk for 256 workgroups; 16
// prompts of 2048 tokens and 64 heads 453 to 465 us; at this load the clock falls, so
// that products count too). With fewer workgroups by the chain of chunks, 1.10 us each
// (1.12 with decays near 1) with 8 to 32 of them, 1.15 with 128. The chain's 2700
// cycles are 40 products of 32 cycles (8 of S Q, 24 of K^T V, 4 of A V, 4 of V's rests)
// and some 250 vector instructions of 4 on each state wavefront, which its SIMD issues
// one after the other, and those of the operand wavefront beside it.
// Steps that were measured, us a chunk with 8 workgroups: LDS loads next to their
// use 1.24; loads, products and vector instructions issued in turn and a phase
// ahead, A by three wavefronts instead of one 1.17; the state's wavefronts first on
// their SIMD 1.06; decays near 1 as a difference 1.12. Outputs as rows through LDS
// instead of 32 bytes per token and wavefront: 457 to 430 us for the 16 prompts. Not
// better: 8 state wavefronts of 16 columns on 16x16x32 products (1.20 a chunk; every
// operand is read twice as often), 3 to 8 chunks of loads ahead, heads in the order of
// the XCDs.
constexpr int AHEAD = 4;
constexpr int N_TILE = AHEAD + 1, N_A = 2, N_O = 2, N_GS = 3, N_G = AHEAD + 2;
constexpr int LEAD = AHEAD + 1;  // intervals before chunk 0
template <bool OUT>
struct Lds {
    alignas(16) uint8_t k[N_TILE][TILE_BYTES];
    alignas(16) uint8_t v[N_TILE][TILE_BYTES];
    alignas(16) uint8_t q[OUT ? N_TILE : 1][OUT ? TILE_BYTES : 16];
    alignas(16) uint8_t a[OUT ? N_A : 1][OUT ? A_BYTES : 16];
    alignas(16) uint8_t o[OUT ? N_O : 1][OUT ? TILE_BYTES : 16];
    alignas(16) float gs[N_GS][LS_FLOATS];
    alignas(16) float g[N_G][64];  // the loads write 64 lanes; rows past the chunk hold zeros
    int stop;                      // without OUT: the step from which on no token counts
};

// What a workgroup works on (uniform).
struct Work {
    const uint8_t *q, *k, *v;  // the unit's first rows of its head
    const float* g;
    uint8_t* out;                // as v
    uint32_t st_qk, st_v, st_g;  // bytes from row to row
    int n_tok, n_chunks;
    float scale;
    float* decay;  // without OUT: gets the log2-decay over the unit's tokens
};

// One wavefront: whether a log-decay of the unit's first n > 0 tokens is not at most 0.
__device__ __forceinline__ bool grows(const Work& w, int n, int lane) {
    constexpr int AT_ONCE = 8;  // loads in flight together
    if (w.st_g == 0) n = 1;
    bool found = false;
    for (int t0 = 0; t0 < n; t0 += 64 * AT_ONCE) {
        float x[AT_ONCE];
#pragma unroll
        for (int j = 0; j < AT_ONCE; ++j) {
            const int t = t0 + 64 * j + lane;
            x[j] = *(const float*)((const uint8_t*)w.g + (size_t)(t < n ? t : n - 1) * w.st_g);
        }
#pragma unroll
        for (int j = 0; j < AT_ONCE; ++j) found |= !(x[j] <= 0.f);
    }
    return __builtin_amdgcn_ballot_w64(found) != 0;
}

template <int ROLE, bool OUT, bool NT>
__device__ __forceinline__ void produce(const Work& w, Lds<OUT>& lds, int lane) {
    Ring<N_TILE> tile;
    Ring<N_A> ra;
    Ring<N_GS> gs;
    Ring<N_G> rg;
    // the chunk of step c
    auto place = [&](int c) { return OUT ? c : w.n_chunks - 1 - c; };
    auto load = [&](const uint8_t* base, uint32_t stride, int at, int rows, uint8_t* to)
                    __attribute__((always_inline)) {
        const auto rsrc = chunk_rsrc(base + (size_t)(at < 0 ? 0 : at) * TILE_ROWS * stride, (uint32_t)rows * stride);
        load_rows<NT>(rsrc, stride, 2 * ROLE, lane, to);
        load_rows<NT>(rsrc, stride, 2 * ROLE + 1, lane, to);
    };
    // rows 8 ROLE .. of the output of chunk c (none before the first), 2 stores
    auto store = [&](int c) __attribute__((always_inline)) {
        const auto rsrc = chunk_rsrc(w.out + (size_t)(c < 0 ? 0 : c) * TILE_ROWS * w.st_v,
                                     (uint32_t)rows_of_chunk(w.n_tok, c) * w.st_v);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int row = 8 * ROLE + 4 * j + (lane >> 4);
            const u32x4 x = *(const u32x4*)(lds.o[c & 1] + tile_off(row, lane & 15));
            __builtin_amdgcn_raw_buffer_store_b128(x, rsrc, (int)(row * w.st_v + (lane & 15) * 16), 0,
                                                   NT ? 2 : 0);
        }
    };
    double after = 0.0;    // ROLE 3 without OUT: the log2-decay of the chunks scanned
    bool to_start = false;  // and whether those before have to be scanned whatever it is
    int end = w.n_chunks;
    if constexpr (ROLE == 3 && !OUT) lds.stop = end;
    // ring position j is step i + j
    for (int i = -LEAD; i < end; ++i) {
        const int c = i + AHEAD, at = place(c), rows = rows_of_chunk(w.n_tok, at);
        load(w.k, w.st_qk, at, rows, lds.k[tile.at[AHEAD]]);
        load(w.v, w.st_v, at, rows, lds.v[tile.at[AHEAD]]);
        if constexpr (OUT) load(w.q, w.st_qk, at, rows, lds.q[tile.at[AHEAD]]);
        if constexpr (OUT) store(i - 1);
        if constexpr (ROLE == 3) {  // a fixed decay has st_g = 0
            const int at_g = place(c + 1), left = rows_of_chunk(w.n_tok, at_g);
            const uint32_t range = __builtin_amdgcn_readfirstlane(left ? (uint32_t)(left - 1) * w.st_g + 4 : 0u);
            const auto rsrc =
                chunk_rsrc((const uint8_t*)w.g + (size_t)(at_g < 0 ? 0 : at_g) * TILE_ROWS * w.st_g, range);
            const uint32_t off = lane < left ? (uint32_t)lane * w.st_g : 0x7ffffffcu;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rsrc, (__attribute__((address_space(3))) void*)lds.g[rg.at[AHEAD + 1]], 4, (int)off, 0, 0, 0);
            if (i + 2 >= 0 && i + 2 < end) {
                const bool gone = !OUT && __builtin_amdgcn_ballot_w64(after <= LOG2_FLOOR) != 0 && !to_start;
                if (__builtin_expect(gone, 0)) to_start = grows(w, (place(i + 2) + 1) * TILE_ROWS, lane);
                if (gone && !to_start) {
                    end = i + 2;
                    lds.stop = end;
                } else {
                    const double all = row_scan<OUT>(lds.g[rg.at[2]][lane & 31], after, lane, lds.gs[gs.at[2]]);
                    if constexpr (!OUT) after += all;
                }
            }
        }
        if constexpr (ROLE < 3 && OUT)  // tiles (0, 0), (1, 0) and (1, 1)
            if (i + 1 >= 0 && i + 1 < w.n_chunks)
                form_a<(ROLE > 0), (ROLE > 1)>(lds.q[tile.at[1]], lds.k[tile.at[1]], lds.gs[gs.at[1]], w.scale,
                                               lds.a[ra.at[1]], lane);
        // what the last AHEAD - 2 intervals issued may be on its way; the loads before have landed
        constexpr int ISSUED = (OUT ? 8 : 4) + (ROLE == 3 ? 1 : 0);
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(ISSUED * (AHEAD - 2)) : "memory");
        lds_barrier();
        if constexpr (ROLE != 3 && !OUT) end = __builtin_amdgcn_readfirstlane(lds.stop);
        tile.next();
        ra.next();
        gs.next();
        rg.next();
    }
    if constexpr (OUT) {
        if (w.n_chunks > 0) store(w.n_chunks - 1);
    } else if constexpr (ROLE == 3) {
        if (lane == 0) *w.decay = (float)after;
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load into LDS outlives the workgroup
}

template <bool OUT, bool NT>
__global__ __launch_bounds__(kLaThreads) void la_prefill(LaArgs a) {
    extern __shared__ __align__(16) uint8_t lds_raw[];
    Lds<OUT>& lds = *(Lds<OUT>*)lds_raw;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int hd = blockIdx.x % a.H;
    const LaUnit un = a.units[blockIdx.x / a.H];
    // the unit's tokens, clamped into the sequence and the inputs
    int64_t beg = a.cu[un.seq], end = a.cu[un.seq + 1];
    end = end > a.Tt ? a.Tt : end;
    beg = (beg < 0 ? 0 : beg) + un.tok0;
    end = end < beg + un.n_tok ? end : beg + un.n_tok;
    const int n_tok = __builtin_amdgcn_readfirstlane(end > beg ? (int)(end - beg) : 0);
    const int n_chunks = (int)(((int64_t)n_tok + TILE_ROWS - 1) / TILE_ROWS);
    const uint32_t st_v = (uint32_t)a.H * (D * 2);

    if (wave < 4) {
        Work w;
        const int64_t row = beg * a.H + hd, row_qk = (beg * a.Hk + hd / a.group) * (D * 2);
        w.q = (const uint8_t*)a.q + row_qk;
        w.k = (const uint8_t*)a.k + row_qk;
        w.v = (const uint8_t*)a.v + row * (D * 2);
        w.g = a.g + (a.g_fixed ? hd : row);
        w.out = (uint8_t*)a.out + row * (D * 2);
        w.st_qk = (uint32_t)a.Hk * (D * 2);
        w.st_v = st_v;
        w.st_g = a.g_fixed ? 0u : (uint32_t)a.H * 4;
        w.n_tok = n_tok;
        w.n_chunks = n_chunks;
        w.scale = a.scale;
        w.decay = OUT ? nullptr : a.decays + (int64_t)un.out * a.H + hd;
        if (wave == 0) produce<0, OUT, NT>(w, lds, lane);
        else if (wave == 1) produce<1, OUT, NT>(w, lds, lane);
        else if (wave == 2) produce<2, OUT, NT>(w, lds, lane);
        else produce<3, OUT, NT>(w, lds, lane);
        return;
    }

    // wavefronts 4 .. 7: the state, 32 value columns each. Each shares its SIMD
    // with an operand wavefront, whose work is to fall beside the products.
    __builtin_amdgcn_s_setprio(2);
    const int col0 = 32 * (wave & 3);
    const int h = lane >> 5, odd = (lane >> 4) & 1, r = (lane >> 2) & 3, c = lane & 3;
    f32x16 S[4];
    // the element of the 128 x 128 state that element 4a + b of tile t is on this lane
    const int at0 = 8 * h * D + col0 + value_col(lane & 31);
    auto each = [&](auto f) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                S[t][i] = f(at0 + (32 * t + 16 * (i >> 3) + (i & 7)) * D, S[t][i]);
    };
    const int64_t own = ((int64_t)un.seq * a.H + hd) * (D * D);
    if (un.in >= 0) {
        const float* p = a.slots + ((int64_t)un.in * a.H + hd) * (D * D);
        each([&](int at, float) { return p[at]; });
    } else if (un.in == LA_INITIAL && a.s0) {
        if (a.state_bf16) {
            const uint16_t* p = (const uint16_t*)a.s0 + own;
            each([&](int at, float) { return __uint_as_float((uint32_t)p[at] << 16); });
        } else {
            const float* p = (const float*)a.s0 + own;
            each([&](int at, float) { return p[at]; });
        }
    } else {
        each([&](int, float) { return 0.f; });
    }
    if constexpr (OUT)
        if (wave < 4 + N_A)
            for (int part = 0; part < A_BYTES; part += A_LO)
                *(u32x2*)(a_tile(lds.a[wave - 4], 0, 1, lane) + part) = u32x2{0, 0};
    for (int i = -LEAD; i < 0; ++i) lds_barrier();
    Ring<N_TILE> tile;
    Ring<N_A> ra;
    Ring<N_GS> gs;
#pragma unroll
    for (int i = 0; i < LEAD; ++i) {
        tile.next();
        ra.next();
        gs.next();
    }
    const int at_row = opaque(tile_off(lane & 31, h));
    // K^T: lane row l & 31 of tile t is channel 32t + 16 odd + 8 (i >> 2 & 1) + 4 (i >> 3) + (i & 3), i = l & 15
    const int at_col0 = opaque(tile_off(4 * h + r, 2 * odd + (c & 1)) + 8 * (c >> 1));
    const int at_col1 = opaque(tile_off(8 + 4 * h + r, 2 * odd + (c & 1)) + 8 * (c >> 1));
    const int at_o = opaque(tile_off(lane & 31, (col0 >> 3) + 2 * h));
    const int at_v0 = opaque(tile_off(4 * h + r, (col0 >> 3) + 2 * (c & 1) + odd) + 8 * (c >> 1));
    const int at_v1 = opaque(tile_off(8 + 4 * h + r, (col0 >> 3) + 2 * (c & 1) + odd) + 8 * (c >> 1));
    auto columns = [&](const uint8_t* tile, int at0, int at1) __attribute__((always_inline)) {
        const u32x2 x = lds_load_tr16(tile + at0), y = lds_load_tr16(tile + at1);
        return u32x4{x.x, x.y, y.x, y.y};
    };
    // While one chunk is worked on, Q, V and the first half of K^T of the next are read (they have landed an interval
    // before) and its V is weighted: LDS and VALU work beside the products. V: rows 16s + 8 (j >> 2) + 4h + (j & 3) of
    // the lane's column value_col(l & 31).
    u32x4 qf[4][2], kt[4][2], vw[2];
    f32x4 last[4];
    Split3 w;
    auto fetch_v = [&](int slot, const float* row) __attribute__((always_inline)) {
#pragma unroll
        for (int s = 0; s < 2; ++s) vw[s] = columns(lds.v[slot] + 4096 * s, at_v0, at_v1);
#pragma unroll
        for (int a = 0; a < 4; ++a) last[a] = *(const f32x4*)(row + LS_LAST + 8 * a + 4 * h);
    };
    u32x2 step = {0, 0};
    float gam_row = 0.f;
    int n_steps = n_chunks;
    auto fetch_gam = [&](const float* row) __attribute__((always_inline)) {
        if constexpr (OUT) {
            step = *(const u32x2*)(row + LS_STEP);
            gam_row = a.scale * row[LS_GAM + (lane & 31)];
        } else {
            n_steps = lds.stop;
        }
    };
    auto fetch_q = [&](int slot, int t, int s) __attribute__((always_inline)) {
        if constexpr (OUT) qf[t][s] = row32(lds.q[slot], at_row, t, s);
    };
    auto fetch_k = [&](int slot, int t, int s) __attribute__((always_inline)) {
        kt[t][s] = columns(lds.k[slot] + 4096 * s, at_col0 ^ (4 * t << 4), at_col1 ^ (4 * t << 4));
    };
    fetch_gam(lds.gs[gs.at[0]]);
    fetch_v(tile.at[0], lds.gs[gs.at[0]]);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        fetch_q(tile.at[0], t, 0);
        fetch_q(tile.at[0], t, 1);
        fetch_k(tile.at[0], t, 0);
    }
    const MinusOne neg = minus_one(lane);
    {
        f32x16 x;
        unrolled<8>([&](auto n) __attribute__((always_inline)) { weigh<n()>(x, vw, last, w.a); });
        x = rest_of(x, w.a, neg);
        pack_rows(x, w.b);
        x = rest_of(x, w.b, neg);
        pack_rows(x, w.c);
    }
    counted_wait();
    for (int i = 0; i < (OUT ? n_chunks : __builtin_amdgcn_readfirstlane(n_steps)); ++i) {
        const uint32_t p = __builtin_amdgcn_readfirstlane(step.x), d = __builtin_amdgcn_readfirstlane(step.y);
        const float gm = gam_row;
        const u32x4 v0 = vw[0], v1 = vw[1];
        u32x4 ah[2], al[2], sb[2];
        f32x16 o = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if constexpr (OUT) pack_rows(S[0], sb);
        sched_fence();
        // o = S Q. A product of the matrix unit takes 32 cycles and leaves room for some five vector
        // instructions, so they are issued in turn, with the LDS loads of what comes next.
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            u32x4 after[2];
            if constexpr (OUT) {
                o = mfma_32(sb[0], qf[t][0], o);
                sched_fence();
                if (t < 3) pack_rows(S[t + 1], after);
            }
            if (t == 0) fetch_v(tile.at[1], lds.gs[gs.at[1]]);
            if (t == 1 || t == 2) {
                fetch_k(tile.at[0], 2 * t - 2, 1);
                fetch_k(tile.at[0], 2 * t - 1, 1);
            }
            if constexpr (OUT) {
                sched_fence();
                o = mfma_32(sb[1], qf[t][1], o);
                sched_fence();
                sb[0] = after[0];
                sb[1] = after[1];
            }
            sched_fence();
        }
        // S decays. (One of the two at most. Branches round each tile, or one with two sides, cost registers for copies
        // of S, and a chunk 15 to 30%; S + d S beside the products above and p S in a branch 2% where d counts and 12%
        // where p does, against 5 and 4 for this.)
        if (OUT && p != 0x3f800000) {
#pragma unroll
            for (int t = 0; t < 4; ++t) S[t] = __uint_as_float(p) * S[t];
        }
        if (OUT && d != 0) {
#pragma unroll
            for (int t = 0; t < 4; ++t) S[t] = __builtin_elementwise_fma(f32x16(__uint_as_float(d)), S[t], S[t]);
        }
        sched_fence();
        // S += K^T (weighted V), beside the weighting for the next chunk
        Split3 next;
        f32x16 x;
        unrolled<24>([&](auto m) __attribute__((always_inline)) {
            constexpr int n = m(), s = n / 12, k = n / 4 % 3, t = n % 4;
            S[t] = mfma_32(kt[t][s], k == 0 ? w.c[s] : k == 1 ? w.b[s] : w.a[s], S[t]);
            if constexpr (n < 8) weigh<n>(x, vw, last, next.a);
            if constexpr (n < 8) fetch_q(tile.at[1], n / 2, n % 2);
            if constexpr (n >= 12 && n % 2 == 0 && n < 20) fetch_k(tile.at[1], n / 2 - 6, 0);
            if constexpr (n == 8) x = rest_of(x, next.a, neg);
            if constexpr (n == 13) fetch_gam(lds.gs[gs.at[1]]);
            if constexpr (n == 14) pack_rows(x, next.b);
            if constexpr (n == 15) x = rest_of(x, next.b, neg);
            if constexpr (n == 21) pack_rows(x, next.c);
            sched_fence();
            if constexpr (OUT) {
                if constexpr (n == 8 || n == 9) {
                    constexpr int at = (n - 8) * 1024;
                    ah[n - 8] = *(const u32x4*)(lds.a[ra.at[0]] + at + lane * 16);
                    al[n - 8] = *(const u32x4*)(lds.a[ra.at[0]] + A_LO + at + lane * 16);
                }
                if constexpr (n > 8 && n <= 12) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[4 * (n - 9) + e] *= gm;
                }
                if constexpr (n == 12 || n == 13) o = mfma_32(n == 12 ? v0 : v1, al[n == 13], o);
                if constexpr (n == 14 || n == 15) o = mfma_32(n == 14 ? v0 : v1, ah[n == 15], o);
                if constexpr (n == 19 || n == 20) {  // token l & 31, element 4a + b being value column 16h + 4a + b
                    constexpr int j = n - 19;
                    const u32x2 p = pack4(quarter(o, 2 * j)), q = pack4(quarter(o, 2 * j + 1));
                    *(u32x4*)(lds.o[i & 1] + (at_o ^ (j << 4))) = u32x4{p.x, p.y, q.x, q.y};
                }
                sched_fence();
            }
        });
        w = next;
        counted_wait();
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        sched_fence();
        tile.next();
        ra.next();
        gs.next();
    }
    if (un.out >= 0) {
        float* p = a.slots + ((int64_t)un.out * a.H + hd) * (D * D);
        each([&](int at, float s) { return p[at] = s; });
    } else if (un.out == LA_FINAL && a.sT) {
        if (a.state_bf16) {
            uint16_t* p = (uint16_t*)a.sT + own;
            each([&](int at, float s) {
                p[at] = (uint16_t)pack_bf16(s, 0.f);
                return s;
            });
        } else {
            float* p = (float*)a.sT + own;
            each([&](int at, float s) { return p[at] = s; });
        }
    }
}

// The states between segments: slot 0 gets the initial state, and slot s + 1,
// which holds the end state of segment s from zero, is added the decayed slot s. The
// decays come as logarithms, and one near 1 is applied as in a chunk: its error does not
// add up over the segments (2048 of one chunk, -4e-8 a token: 4e-5 of the state before).
// The others are applied as two roots, for what a state that has grown keeps of them below
// 2^-126.
// One thread per four elements of a state; the loads of DEEP segments are in flight
// while the DEEP before are added: 64 segments of 4 heads (16 MiB) take 10 us.
constexpr int DEEP = 8;
static_assert(kLaMergeTiles * kLaMergeThreads * 4 == D * D);
__global__ __launch_bounds__(kLaMergeThreads) void la_merge(LaMergeArgs a) {
    const int tile = blockIdx.x % kLaMergeTiles, ih = blockIdx.x / kLaMergeTiles, hd = ih % a.H;
    const LaMerge it = a.items[ih / a.H];
    const int at = (tile * kLaMergeThreads + threadIdx.x) * 4;
    const int64_t own = ((int64_t)it.seq * a.H + hd) * (D * D) + at;
    float* const first = a.slots + ((int64_t)it.slot0 * a.H + hd) * (D * D) + at;
    const int64_t step = (int64_t)a.H * (D * D);
    const int lane = threadIdx.x & 63;
    // A segment of 64 per lane: its log2-decay (behind the end, the last one's again).
    auto load_x = [&](int s) { return a.decays[(int64_t)(it.slot0 + (s < it.n ? s : it.n - 1)) * a.H + hd]; };
    // The states of DEEP segments from s0 on, likewise.
    auto load = [&](int s0, f32x4 (&b)[DEEP]) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < DEEP; ++j) b[j] = *(const f32x4*)(first + (s0 + j < it.n ? s0 + j : it.n - 1) * step);
    };
    float x = load_x(1 + lane);
    f32x4 b[DEEP];
    load(1, b);
    f32x4 c = {0.f, 0.f, 0.f, 0.f};
    if (a.s0 && a.state_bf16) {
        const u32x2 y = *(const u32x2*)((const uint16_t*)a.s0 + own);
        c = f32x4{bf16_lo(y.x), bf16_hi(y.x), bf16_lo(y.y), bf16_hi(y.y)};
    } else if (a.s0) {
        c = *(const f32x4*)((const float*)a.s0 + own);
    }
    *(f32x4*)first = c;
    float lane_d = 0.f, lane_p = 0.f;
    uint64_t nears = 0;
    auto add = [&](int s0, bool all) __attribute__((always_inline)) {
        const int from = (s0 - 1) & 63;
        if (from == 0) {  // d of each lane's segment, and what c is multiplied with before
            if (s0 > 1) x = load_x(s0 + lane);
            const bool near = x >= -1.f && x <= 1.f;
            const float half = exp2_hw(0.5f * x);
            lane_d = near ? expm1_small(x * (float)LN2) : half;
            lane_p = near ? 1.f : half;
            nears = __builtin_amdgcn_ballot_w64(near);
        }
#pragma unroll
        for (int j = 0; j < DEEP; ++j) {
            const float d = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(lane_d), from + j));
            const float p = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(lane_p), from + j));
            const bool near = nears >> (from + j) & 1;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float y = __builtin_fmaf(d, p * c[e], b[j][e]);
                c[e] = near ? c[e] + y : y;
            }
            if (all || s0 + j < it.n) *(f32x4*)(first + (s0 + j) * step) = c;
        }
    };
    int s0 = 1;
    for (; s0 + DEEP < it.n; s0 += DEEP) {
        f32x4 next[DEEP];
        load(s0 + DEEP, next);
        sched_fence();
        add(s0, true);
#pragma unroll
        for (int j = 0; j < DEEP; ++j) b[j] = next[j];
    }
    add(s0, false);
}

// Decode. With S the state before a token and gam = exp(g), for value column j:
//   o_j = scale (gam sum_r q_r S_rj + (q . k) v_j),   S'_rj = gam S_rj + k_r v_j
// with a gam in [1/2, 2] as 1 + d, S + (d S + k v) (256 sequences 192 us, 190 with the product).
// One wavefront per (sequence, head, 32-column tile) keeps its part of the
// state in registers over all T tokens: lane (rs, cg) = (lane >> 3, lane & 7)
// owns rows 16rs .. + 15 of columns 4cg .. + 3, so a load instruction covers
// eight whole 128-byte lines, the sums need three lane exchanges and the
// kernel needs neither LDS nor a barrier. Bound by HBM: 256 sequences of 32 heads
// take 190 to 193 us (5.6 TB/s); one sequence takes 4, the latency of the launch and of
// one load after another.
//
// States beyond 128 MiB, half the last-level cache, are read and written with
// the nontemporal hint, as the gated delta rule's decode does, which moves the
// same bytes and measured both sides.
static_assert(kLaDecodeThreads == 64 * 4);  // a wavefront per 32-column tile

template <bool NT>
__global__ __launch_bounds__(kLaDecodeThreads) void la_decode(LaDecodeArgs a) {
    const int lane = threadIdx.x & 63, tile = threadIdx.x >> 6;
    const int64_t nh = blockIdx.x;
    const int64_t n = nh / a.H;
    const int hd = (int)(nh % a.H), hq = hd / a.group;
    const int rs = lane >> 3, col = 32 * tile + 4 * (lane & 7);
    const int64_t slot = a.slots ? (int64_t)a.slots[n] : n;
    if (slot < 0 || slot >= a.n_slots) {
        for (int t = rs; t < a.T; t += 8) *(uint2*)(a.out + ((n * a.T + t) * a.H + hd) * D + col) = uint2{0u, 0u};
        return;
    }
    f32x4* st = (f32x4*)(a.state + (slot * a.H + hd) * (D * D) + (16 * rs) * D + col);
    f32x4 s[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        if constexpr (NT) s[i] = __builtin_nontemporal_load(st + i * (D / 4));
        else s[i] = st[i * (D / 4)];
    }
    struct Token {
        u32x4 k[2], q[2];
        u32x2 v;
        float g;
    };
    auto load = [&](int t) __attribute__((always_inline)) {
        const int64_t row = (n * a.T + t) * a.H + hd, rq = (n * a.T + t) * a.Hk + hq;
        const u32x4* kp = (const u32x4*)(a.k + rq * D + 16 * rs);
        const u32x4* qp = (const u32x4*)(a.q + rq * D + 16 * rs);
        return Token{{kp[0], kp[1]}, {qp[0], qp[1]}, *(const u32x2*)(a.v + row * D + col),
                     a.g[a.g_fixed ? hd : row]};
    };
    Token next = load(0);  // each a token ahead
    for (int t = 0; t < a.T; ++t) {
        const int64_t row = (n * a.T + t) * a.H + hd;
        const Token now = next;
        if (t + 1 < a.T) next = load(t + 1);
        const u32x4 (&k2)[2] = now.k, (&q2)[2] = now.q;
        const u32x2 vb = now.v;
        // the decay as one + d: as in the prefill, the error of one near 1 does not add up, here over the tokens of a
        // generation (4096 of -1e-6 left a state 3.4e-5 off, now 2.7e-6)
        const bool near = __builtin_fabsf(now.g) <= (float)LN2;
        const float d = near ? expm1_small(now.g) : exp2_hw(now.g * LOG2E), one = near ? 1.f : 0.f, gam = one + d;
        float k[16], q[16], qk = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            k[2 * i] = bf16_lo(k2[i >> 2][i & 3]);
            k[2 * i + 1] = bf16_hi(k2[i >> 2][i & 3]);
            q[2 * i] = bf16_lo(q2[i >> 2][i & 3]);
            q[2 * i + 1] = bf16_hi(q2[i >> 2][i & 3]);
        }
        const f32x4 v = {bf16_lo(vb.x), bf16_hi(vb.x), bf16_lo(vb.y), bf16_hi(vb.y)};
        f32x4 sb = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            qk = __builtin_fmaf(q[i], k[i], qk);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                sb[j] = __builtin_fmaf(q[i], s[i][j], sb[j]);
                s[i][j] = __builtin_fmaf(one, s[i][j], __builtin_fmaf(d, s[i][j], k[i] * v[j]));
            }
        }
#pragma unroll
        for (int d = 8; d < 64; d <<= 1) {
            qk += __shfl_xor(qk, d, 64);
#pragma unroll
            for (int j = 0; j < 4; ++j) sb[j] += __shfl_xor(sb[j], d, 64);
        }
        f32x4 o;
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = a.scale * __builtin_fmaf(gam, sb[j], qk * v[j]);
        if (rs == 0) *(u32x2*)(a.out + row * D + col) = pack4(o);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        if constexpr (NT) __builtin_nontemporal_store(s[i], st + i * (D / 4));
        else st[i * (D / 4)] = s[i];
    }
}

template <bool OUT, bool NT>
hipError_t run_la_prefill(const LaArgs& a, hipStream_t s) {
    // more LDS than the default limit, allowed once per device and process
    static std::mutex mu;
    static uint64_t done[4] = {0, 0, 0, 0};
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    {
        std::lock_guard<std::mutex> lk(mu);
        if (dev >= 256 || !(done[dev >> 6] >> (dev & 63) & 1)) {
            e = hipFuncSetAttribute((const void*)la_prefill<OUT, NT>, hipFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)sizeof(Lds<OUT>));
            if (e != hipSuccess) return e;
            if (dev < 256) done[dev >> 6] |= 1ull << (dev & 63);
        }
    }
    hipLaunchKernelGGL((la_prefill<OUT, NT>), dim3((unsigned)(a.n_units * a.H)), dim3(kLaThreads), sizeof(Lds<OUT>), s,
                       a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_la_prefill(const LaArgs& a, bool with_out, hipStream_t s) {
    if (a.n_units == 0) return hipSuccess;
    // What the last-level cache (256 MiB) cannot hold is streamed with the
    // nontemporal hint: 472 us without and 461 with it for 16 prompts of 2048 tokens and
    // 64 heads (2 GiB), 191 and 187 for 65536 tokens of 8 heads. Not in the segments' pass,
    // which leaves k and v to the second one (178 us, and 190 with the hint there, when measured).
    const bool nt = (size_t)a.Tt * (a.H + a.Hk) * (4 * D) > ((size_t)256 << 20);
    if (!with_out) return run_la_prefill<false, false>(a, s);
    return nt ? run_la_prefill<true, true>(a, s) : run_la_prefill<true, false>(a, s);
}

hipError_t launch_la_merge(const LaMergeArgs& a, hipStream_t s) {
    hipLaunchKernelGGL(la_merge, dim3((unsigned)(a.n_items * a.H * kLaMergeTiles)), dim3(kLaMergeThreads), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_la_decode(const LaDecodeArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)(a.n_seqs * a.H)), block(kLaDecodeThreads);
    const bool nt = (size_t)a.n_seqs * a.H * (D * D * 4) > ((size_t)128 << 20);
    if (nt) hipLaunchKernelGGL(la_decode<true>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(la_decode<false>, grid, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace kda
