// The gated delta rule on gfx950 (CDNA4): chunked prefill and recurrent decode
// over a 128 x 128 fp32 state per head, with one log-decay per token and head:
//   S_t = (I - beta_t k_t k_t^T) exp(g_t) S_{t-1} + beta_t k_t v_t^T,   o_t = scale S_t^T q_t
//
// Chunked form. For a chunk of rows r = 0 .. 31 with start state S, G_r the
// running sum of g inside the chunk and gam_r = exp(G_r):
//   L  = strict-lower(beta_r (k_r . k_i) exp(G_r - G_i)),   T' = (I + L)^-1 diag(beta)
//   A  = lower((q_r . k_i) exp(G_r - G_i))
//   U  = T' (V - diag(gam) K S)
//   O  = scale (diag(gam) Q S + A U)
//   S <- gam_31 S + K^T diag(exp(G_31 - G)) U
// The decay is one number per row, so it scales rows of results and never the
// operands q, k and v: those go to the matrix instructions as they are in
// memory. What is computed (S, V - K S, T', A, U) is split into a pair of bf16
// numbers hi + lo, which carries 16 bits of mantissa; products of two such
// pairs leave out lo * lo (2^-18 of the product). All sums are fp32, the
// running sum of g is fp64 (differences of it are taken), so states keep about
// 2^-18 per step against the 2^-9 of single bf16 operands. Zeros of L, T' and A
// multiply whatever is there: a value that is not finite reaches all rows of its
// chunk.
#include "gated_delta_launch.h"
#include "kda_device.hpp"

#include <mutex>

namespace kda {
namespace {

constexpr int GC = kGdChunk;
constexpr int TILE_BYTES = GC * D * 2;  // one chunk of q, k or v of one head (8 KiB)

// LDS tiles hold token rows of 256 bytes; the 16-byte granules of row r are
// permuted by XOR with gd_swz(r). Row fragments (16 rows, one granule) and the
// transposing loads (4 rows of each 16-lane group, 4 granules) then both touch
// 16 distinct granule positions.
__device__ __forceinline__ int gd_swz(int row) { return ((row & 3) << 2) | ((row >> 2) & 3); }
__device__ __forceinline__ int tile_off(int row, int gi) { return row * 256 + ((gi ^ gd_swz(row)) << 4); }

// Rows 4i .. 4i + 3 of a tile by one direct-to-LDS load. Rows past the
// descriptor's range become zeros.
__device__ __forceinline__ void load_rows(__amdgpu_buffer_rsrc_t rsrc, uint32_t stride, int i, int lane,
                                          uint8_t* tile) {
    const int row = 4 * i + (lane >> 4);
    const uint32_t off = (uint32_t)row * stride + (((lane & 15) ^ gd_swz(row)) << 4);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (__attribute__((address_space(3))) void*)(tile + 1024 * i), 16,
                                             (int)off, 0, 0, 0);
}

// Per-row values of a chunk, fp32 [5][32]: the running log2-decay as hi + lo,
// gam, exp(G_31 - G) and beta.
constexpr int GS_H = 0, GS_L = 32, GS_GAM = 64, GS_LAST = 96, GS_BETA = 128, GS_FLOATS = 160;
// Below this log2-decay a token's decay is zero in fp32 and stands for any
// smaller one (-inf included), which keeps the running sum finite.
constexpr float GD_LOG2_FLOOR = -160.0f;

// One wavefront: x = the log-decay and b = beta of row lane & 31.
__device__ __forceinline__ void row_scan(float x, float b, int lane, float* gs) {
    const int r = lane & 31;
    x *= LOG2E;
    double G = x < GD_LOG2_FLOOR ? GD_LOG2_FLOOR : x;
#pragma unroll
    for (int d = 1; d < GC; d <<= 1) {
        const double y = __shfl_up(G, d, 32);
        if (r >= d) G += y;
    }
    const double all = __shfl(G, 31, 32);
    const float hi = (float)G;
    if (lane < GC) {
        gs[GS_H + r] = hi;
        gs[GS_L + r] = (float)(G - (double)hi);
        gs[GS_GAM + r] = exp2_hw(hi);
        gs[GS_LAST + r] = exp2_hw((float)(all - G));
        gs[GS_BETA + r] = b;
    }
}

__device__ __forceinline__ u32x4 row_frag(const uint8_t* tile, int row0, int p, int lane) {
    return *(const u32x4*)(tile + tile_off(row0 + (lane & 15), 4 * p + (lane >> 4)));
}

// 16 x 16 Gram over 128 channels: lane (gg, m) gets a_{ra + 4gg + v} . b_{rb + m}.
__device__ __forceinline__ f32x4 gram(const uint8_t* a, int ra, const uint8_t* b, int rb, int lane) {
    f32x4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int p = 0; p < 4; ++p) c = mfma_k32(row_frag(a, ra, p, lane), row_frag(b, rb, p, lane), c);
    return c;
}

struct HiLo {
    u32x2 h, l;
};
__device__ __forceinline__ HiLo split4(const f32x4& x) {
    HiLo r;
    r.h = pack4(x);
    r.l = pack4(x[0] - bf16_lo(r.h.x), x[1] - bf16_hi(r.h.x), x[2] - bf16_lo(r.h.y), x[3] - bf16_hi(r.h.y));
    return r;
}

// T' and A of a chunk as operands of 32x32x16 products: [step s 2][hi, lo]
// [lane 64][8 bf16], lane l holding row l & 31 and columns 16s + 8 (j >> 2) +
// 4 (l >> 5) + (j & 3). The wavefront that forms 16 x 16 tile (rt, ct) holds
// row 16rt + m, columns 16ct + 4gg + v on lane (gg, m): half a lane's entry.
// Tile (0, 1) is zero; it is cleared once and never written.
constexpr int REC4 = 4096;
__device__ __forceinline__ void put_tile(uint8_t* rec, int rt, int ct, int lane, const f32x4& x) {
    const int gg = lane >> 4, m = lane & 15;
    uint8_t* at = rec + ct * 2048 + (32 * (gg & 1) + 16 * rt + m) * 16 + 8 * (gg >> 1);
    const HiLo s = split4(x);
    *(u32x2*)at = s.h;
    *(u32x2*)(at + 1024) = s.l;
}

__device__ __forceinline__ float pair_decay(float hr, float lr, float hi, float li) {
    return exp2_hw((hr - hi) + (lr - li));
}

// Scratch of the inverse: 16 x 16 fp32 matrices with a row stride of 20 floats.
constexpr int LSTR = 20;
constexpr int LMAT = 16 * LSTR;

// Diagonal tile td of T' on one wavefront. (I + L)^-1 is found by columns:
// lane (gg, m) holds u[s] = T[m][4gg + s], and step K subtracts L[m][K] T[K][c]
// from the rows below (a DPP broadcast of lane K inside a multiply-add, 15
// dependent steps of 4). The unscaled tile stays behind for the off-diagonal
// one, T00 as rows of LSTR floats in lt, T11 by lane in t11.
template <int TD>
__device__ __forceinline__ void diag_tile(const uint8_t* K, const float* gs, float* lt, float* inv, uint8_t* rec_t,
                                          int lane) {
    const int gg = lane >> 4, m = lane & 15, r0 = 16 * TD;
    const f32x4 a = gram(K, r0, K, r0, lane);  // k_m . k_{4gg + v}
    const f32x4 hv = *(const f32x4*)(gs + GS_H + r0 + 4 * gg), lv = *(const f32x4*)(gs + GS_L + r0 + 4 * gg);
    const f32x4 bv = *(const f32x4*)(gs + GS_BETA + r0 + 4 * gg);
    const float hm = gs[GS_H + r0 + m], lm = gs[GS_L + r0 + m], bm = gs[GS_BETA + r0 + m];
    f32x4 row;  // -L[m][4gg + v]
#pragma unroll
    for (int v = 0; v < 4; ++v) row[v] = 4 * gg + v < m ? -bm * a[v] * pair_decay(hm, lm, hv[v], lv[v]) : 0.f;
    *(f32x4*)(lt + m * LSTR + 4 * gg) = row;
    float l[16];  // -L[m][K]
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const f32x4 x = *(const f32x4*)(lt + m * LSTR + 4 * q);
#pragma unroll
        for (int v = 0; v < 4; ++v) l[4 * q + v] = x[v];
    }
    f32x4 u;
#pragma unroll
    for (int s = 0; s < 4; ++s) u[s] = (4 * gg + s == m) ? 1.f : 0.f;
    // A DPP read needs two wait states after the write of its source: three
    // other instructions stand between them in the block, a nop before it.
#define GD_STEP(K, L)                                                      \
    "v_fmac_f32_dpp %0, %0, " L " row_newbcast:" K " row_mask:0xf bank_mask:0xf\n\t" \
    "v_fmac_f32_dpp %1, %1, " L " row_newbcast:" K " row_mask:0xf bank_mask:0xf\n\t" \
    "v_fmac_f32_dpp %2, %2, " L " row_newbcast:" K " row_mask:0xf bank_mask:0xf\n\t" \
    "v_fmac_f32_dpp %3, %3, " L " row_newbcast:" K " row_mask:0xf bank_mask:0xf\n\t"
    float u0 = u[0], u1 = u[1], u2 = u[2], u3 = u[3];
    asm("s_nop 1\n\t"
        GD_STEP("0", "%4")
        GD_STEP("1", "%5")
        GD_STEP("2", "%6")
        GD_STEP("3", "%7")
        GD_STEP("4", "%8")
        GD_STEP("5", "%9")
        GD_STEP("6", "%10")
        GD_STEP("7", "%11")
        GD_STEP("8", "%12")
        GD_STEP("9", "%13")
        GD_STEP("10", "%14")
        GD_STEP("11", "%15")
        GD_STEP("12", "%16")
        GD_STEP("13", "%17")
        GD_STEP("14", "%18")
        "s_nop 1"
        : "+v"(u0), "+v"(u1), "+v"(u2), "+v"(u3)
        : "v"(l[0]), "v"(l[1]), "v"(l[2]), "v"(l[3]), "v"(l[4]), "v"(l[5]), "v"(l[6]), "v"(l[7]), "v"(l[8]), "v"(l[9]),
          "v"(l[10]), "v"(l[11]), "v"(l[12]), "v"(l[13]), "v"(l[14]));
#undef GD_STEP
    u = f32x4{u0, u1, u2, u3};
    if constexpr (TD == 0) *(f32x4*)(inv + m * LSTR + 4 * gg) = u;
    else *(f32x4*)(inv + lane * 4) = u;
    put_tile(rec_t, TD, TD, lane, u * bv);
}

// L10 as lane (gg, m) -> L10[4gg + v][m].
__device__ __forceinline__ f32x4 lower_tile(const uint8_t* K, const float* gs, int lane) {
    const int gg = lane >> 4, m = lane & 15;
    const f32x4 a = gram(K, 16, K, 0, lane);
    const f32x4 hv = *(const f32x4*)(gs + GS_H + 16 + 4 * gg), lv = *(const f32x4*)(gs + GS_L + 16 + 4 * gg);
    const f32x4 bv = *(const f32x4*)(gs + GS_BETA + 16 + 4 * gg);
    const float hm = gs[GS_H + m], lm = gs[GS_L + m];
    f32x4 r;
#pragma unroll
    for (int v = 0; v < 4; ++v) r[v] = bv[v] * a[v] * pair_decay(hv[v], lv[v], hm, lm);
    return r;
}

// T10 = -T11 L10 T00, as its transpose -T00^T (L10^T T11^T) on fp32 matrix
// instructions: every operand is then in the layout it was formed in (step s
// takes k = 4gg + s from each lane), and the result is lane (gg, m) ->
// T10[m][4gg + v], the record's layout.
__device__ __forceinline__ void off_diagonal(const f32x4& l10, const float* t00, const float* t11, const float* gs,
                                             uint8_t* rec_t, int lane) {
    const int gg = lane >> 4, m = lane & 15;
    const f32x4 b = *(const f32x4*)(t11 + lane * 4);
    f32x4 a, y = {0.f, 0.f, 0.f, 0.f}, z = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < 4; ++s) a[s] = t00[(4 * gg + s) * LSTR + m];
#pragma unroll
    for (int s = 0; s < 4; ++s) y = mfma_f32_k4(l10[s], b[s], y);
#pragma unroll
    for (int s = 0; s < 4; ++s) z = mfma_f32_k4(a[s], y[s], z);
    const f32x4 bv = *(const f32x4*)(gs + GS_BETA + 4 * gg);
    put_tile(rec_t, 1, 0, lane, -z * bv);
}

// A (masked, decayed q-k products, times the output's scale) to its record.
__device__ __forceinline__ void qk_tiles(const uint8_t* Q, const uint8_t* K, const float* gs, float scale,
                                         uint8_t* rec_a, int lane) {
    const int gg = lane >> 4, m = lane & 15;
#pragma unroll
    for (int rt = 0; rt < 2; ++rt)
#pragma unroll
        for (int ct = 0; ct <= rt; ++ct) {
            const f32x4 a = gram(K, 16 * ct, Q, 16 * rt, lane);  // k_{4gg + v} . q_m
            const f32x4 hv = *(const f32x4*)(gs + GS_H + 16 * ct + 4 * gg);
            const f32x4 lv = *(const f32x4*)(gs + GS_L + 16 * ct + 4 * gg);
            const float hm = gs[GS_H + 16 * rt + m], lm = gs[GS_L + 16 * rt + m];
            f32x4 r;
#pragma unroll
            for (int v = 0; v < 4; ++v)
                r[v] = (ct < rt || 4 * gg + v <= m) ? scale * a[v] * pair_decay(hm, lm, hv[v], lv[v]) : 0.f;
            put_tile(rec_a, rt, ct, lane, r);
        }
}

// 32 x 32 products. A and B operands: lane l holds row (column) l & 31 and 8
// of the 16 summed indices, those of its half h = l >> 5. Result: lane l holds
// column l & 31 and rows 8a + 4h + b in element 4a + b.
typedef float f32x16 __attribute__((ext_vector_type(16)));
__device__ __forceinline__ f32x16 mfma_32(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}
__device__ __forceinline__ f32x4 quarter(const f32x16& x, int a) {
    return f32x4{x[4 * a], x[4 * a + 1], x[4 * a + 2], x[4 * a + 3]};
}
// Elements 8s .. 8s + 7 of a result as the operand of step s of a product that
// sums over its rows: the lane's 8 indices are rows 16s + 8 (j >> 2) + 4h + (j & 3).
struct Operand {
    u32x4 h[2], l[2];
};
__device__ __forceinline__ void pack_rows(const f32x16& x, u32x4 (&y)[2]) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const u32x2 a = pack4(quarter(x, 2 * s)), b = pack4(quarter(x, 2 * s + 1));
        y[s] = u32x4{a.x, a.y, b.x, b.y};
    }
}
// The rest x - hi of a tile is formed by the matrix unit, as x + (-1) hi with
// the operand of -1 in minus_one[s]. It is exact, and two matrix instructions
// stand in for 32 vector ones, which bound the chain otherwise.
struct MinusOne {
    u32x4 s[2];
};
__device__ __forceinline__ MinusOne minus_one(int lane) {
    const int row = lane & 31, h = lane >> 5;
    MinusOne m;
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const int r = row - (16 * s + 8 * (w >> 1) + 4 * h + 2 * (w & 1));  // 0: the low half, 1: the high
            m.s[s][w] = r == 0 ? 0x0000bf80u : r == 1 ? 0xbf800000u : 0u;
        }
    return m;
}
__device__ __forceinline__ f32x16 rest_of(const f32x16& x, const u32x4 (&hi)[2], const MinusOne& m) {
    return mfma_32(m.s[1], hi[1], mfma_32(m.s[0], hi[0], x));
}

// The state of one wavefront: 32 value columns in four tiles of 32 channels.
// Row 8a + 4h + b of tile t is channel 32t + 16 (a >> 1) + 8h + 4 (a & 1) + b,
// so that step s of tile t takes 8 consecutive channels 32t + 16s + 8h ..
// from each lane of the other operand. Column n of the tiles is value column
// value_col(n), so that a lane's 16 rows of a transposed result are 16
// consecutive value columns.
__device__ __forceinline__ int value_col(int n) { return 16 * ((n >> 2) & 1) + 4 * (n >> 3) + (n & 3); }

// A lane's place in an LDS tile, from which the places of the other steps
// follow by an exclusive or. (Kept from the optimiser, which would hold every
// place in a register of its own.)
__device__ __forceinline__ int opaque(int x) {
    asm("" : "+v"(x));
    return x;
}

// Nothing is scheduled across sched_fence.
__device__ __forceinline__ void sched_fence() { __builtin_amdgcn_sched_barrier(0); }
// Fixes the place of what forms or uses x among the other pins.
template <class T>
__device__ __forceinline__ void pin(T& x) { asm volatile("" : "+v"(x)); }
// What is left of a chunk's output when its state is done: o (scaled by gam)
// and the operands of A U.
struct Rest {
    f32x16 o;
    Operand u, a;
};

// o += A U: token l & 31, element 4a + b being value column 16h + 4a + b.
__device__ __forceinline__ void finish_output(Rest& x) {
#pragma unroll
    for (int s = 0; s < 2; ++s) x.o = mfma_32(x.u.l[s], x.a.h[s], x.o);
#pragma unroll
    for (int s = 0; s < 2; ++s) x.o = mfma_32(x.u.h[s], x.a.l[s], x.o);
#pragma unroll
    for (int s = 0; s < 2; ++s) x.o = mfma_32(x.u.h[s], x.a.h[s], x.o);
}

__device__ __forceinline__ Operand load_record(const uint8_t* rec, int lane) {
    Operand r;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        r.h[s] = *(const u32x4*)(rec + s * 2048 + lane * 16);
        r.l[s] = *(const u32x4*)(rec + s * 2048 + 1024 + lane * 16);
    }
    return r;
}

// Advances the state over one chunk and, with OUT, finishes and stores the
// output of the one before it. The matrix unit is to be busy throughout (76
// instructions of 32 cycles with OUT): the last chunk's A U and K S go beside
// the split and the scaling of S, Q S beside R = V - diag(gam) K S and beside
// W, K^T W beside the split of U. LDS operands are read a phase ahead.
template <bool OUT, class Store>
__device__ __forceinline__ void chunk_step(const uint8_t* Q, const uint8_t* K, const uint8_t* V, const uint8_t* rec_t,
                                           const uint8_t* rec_a, const float* gs, float scale, int col0, int lane,
                                           const MinusOne& neg, f32x16 (&S)[4], Rest& rest, Store store) {
    const int h = lane >> 5, odd = (lane >> 4) & 1, r = (lane >> 2) & 3, c = lane & 3;
    const f32x16 zero = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    // rows l & 31, the granule of step s of tile t: 4t + 2s + h
    const int at_row = opaque(tile_off(lane & 31, h));
    auto row32 = [&](const uint8_t* tile, int t, int s) __attribute__((always_inline)) {
        return *(const u32x4*)(tile + (at_row ^ ((4 * t + 2 * s) << 4)));
    };
    u32x4 kf[4][2];
    const float gc = gs[GS_GAM + 31];
#pragma unroll
    for (int t = 0; t < (OUT ? 4 : 1); ++t)  // without OUT, a tile ahead: 168 registers are there
#pragma unroll
        for (int s = 0; s < 2; ++s) kf[t][s] = row32(K, t, s);
    if constexpr (OUT) finish_output(rest);
    sched_fence();
    // K S
    Operand sb[4];
    f32x16 P = zero, below;
    u32x4 qf[4][2];
    f32x4 gam[4];
    u32x2 vw[4];
    auto low = [&](int t, const f32x16& x) __attribute__((always_inline)) {  // lo of S's tile t, then its scaling
        pack_rows(x, sb[t].l);
#pragma unroll
        for (int s = 0; s < 2; ++s) P = mfma_32(kf[t][s], sb[t].l[s], P);
        S[t] = gc * S[t];
    };
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        pack_rows(S[t], sb[t].h);
        const f32x16 x = rest_of(S[t], sb[t].h, neg);
#pragma unroll
        for (int s = 0; s < 2; ++s) P = mfma_32(kf[t][s], sb[t].h[s], P);
        if constexpr (OUT) {
            if (t == 1) store(rest.o);
            if (t > 0) low(t - 1, below);  // a tile behind, so that the matrix unit does not wait
            below = x;
        } else {  // the other wavefront of the SIMD fills the wait
            if (t < 3) {
#pragma unroll
                for (int s = 0; s < 2; ++s) kf[t + 1][s] = row32(K, t + 1, s);
            }
            low(t, x);
        }
        if (t == 3) {
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                gam[a] = *(const f32x4*)(gs + GS_GAM + 8 * a + 4 * h);
                // rows 8a + 4h + r, the lane's column value_col(l & 31)
                vw[a] = lds_load_tr16(V + tile_off(8 * a + 4 * h + r, (col0 >> 3) + 2 * (c & 1) + odd) + 8 * (c >> 1));
            }
        }
        sched_fence();
    }
    if constexpr (OUT) {
#pragma unroll
        for (int s = 0; s < 4; ++s) qf[s >> 1][s & 1] = row32(Q, s >> 1, s & 1);
        low(3, below);
        sched_fence();
    }
    // R = V - diag(gam) K S
    f32x16 o = zero;
    int done = 0;
    auto qs = [&](int n) __attribute__((always_inline)) {  // the next n of Q S
        if constexpr (OUT) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < n) {
                    const int q = done + k, t = q >> 2, s = q & 1;
                    pin(qf[t][s]);
                    o = mfma_32(q & 2 ? sb[t].l[s] : sb[t].h[s], qf[t][s], o);
                }
            done += n;
        }
        sched_fence();
    };
    f32x16 R;
    Operand T;
    qs(2);
#pragma unroll
    for (int a = 0; a < 4; ++a) {
        f32x4 x = {__builtin_fmaf(-gam[a][0], P[4 * a], bf16_lo(vw[a].x)),
                   __builtin_fmaf(-gam[a][1], P[4 * a + 1], bf16_hi(vw[a].x)),
                   __builtin_fmaf(-gam[a][2], P[4 * a + 2], bf16_lo(vw[a].y)),
                   __builtin_fmaf(-gam[a][3], P[4 * a + 3], bf16_hi(vw[a].y))};
        pin(x);
#pragma unroll
        for (int b = 0; b < 4; ++b) R[4 * a + b] = x[b];
        if (a == 1) T = load_record(rec_t, lane);
        qs(1);
    }
    Operand rb;
    pack_rows(R, rb.h);
    const f32x16 R_below = rest_of(R, rb.h, neg);
    if constexpr (OUT) {
#pragma unroll
        for (int s = 4; s < 8; ++s) qf[s >> 1][s & 1] = row32(Q, s >> 1, s & 1);
    }
    sched_fence();
    qs(2);
    // U = T' R
    f32x16 U = zero;
#pragma unroll
    for (int s = 0; s < 2; ++s) U = mfma_32(T.l[s], rb.h[s], U);
#pragma unroll
    for (int s = 0; s < 2; ++s) U = mfma_32(T.h[s], rb.h[s], U);
    pack_rows(R_below, rb.l);
    f32x4 last[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) last[a] = *(const f32x4*)(gs + GS_LAST + 8 * a + 4 * h);
    float gm = 0.f;
    if constexpr (OUT) gm = scale * gs[GS_GAM + (lane & 31)];
#pragma unroll
    for (int s = 0; s < 2; ++s) U = mfma_32(T.h[s], rb.l[s], U);
    sched_fence();
    // K^T: lane row l & 31 of tile t is channel 32t + 16 odd + 8 (i >> 2 & 1) + 4 (i >> 3) + (i & 3), i = l & 15
    const int at_col0 = opaque(tile_off(4 * h + r, 2 * odd + (c & 1)) + 8 * (c >> 1));
    const int at_col1 = opaque(tile_off(8 + 4 * h + r, 2 * odd + (c & 1)) + 8 * (c >> 1));
    u32x4 kt[4][2];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const u32x2 k0 = lds_load_tr16(K + (at_col0 ^ (4 * t << 4)) + 4096 * s);
            const u32x2 k1 = lds_load_tr16(K + (at_col1 ^ (4 * t << 4)) + 4096 * s);
            kt[t][s] = u32x4{k0.x, k0.y, k1.x, k1.y};
        }
    sched_fence();
    qs(3);
    // W = diag(exp(G_31 - G)) U
    f32x16 W;
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) W[4 * a + b] = last[a][b] * U[4 * a + b];
    Operand wb;
    pack_rows(W, wb.h);
    const f32x16 W_below = rest_of(W, wb.h, neg);
    if constexpr (OUT) rest.a = load_record(rec_a, lane);
    sched_fence();
    qs(5);
    pack_rows(W_below, wb.l);
    sched_fence();
    // S += K^T W beside the split of U
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int t = 0; t < 4; ++t) S[t] = mfma_32(kt[t][s], wb.h[s], S[t]);
    if constexpr (OUT) {
        pack_rows(U, rest.u.h);
        rest.o = gm * o;
        const f32x16 U_below = rest_of(U, rest.u.h, neg);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int t = 0; t < 4; ++t) S[t] = mfma_32(kt[t][s], wb.l[s], S[t]);
        pack_rows(U_below, rest.u.l);
    } else {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int t = 0; t < 4; ++t) S[t] = mfma_32(kt[t][s], wb.l[s], S[t]);
    }
    sched_fence();
}

// Prefill: one workgroup per (unit, head), in a software pipeline with one
// barrier per chunk. In interval i
//   wavefronts 4 .. 7 advance the state over chunk i (32 columns each); without
//     OUT, wavefronts 8 .. 11 do the same for the transfer M of the unit's
//     tokens, the end state from the identity with V = 0, on the same operands;
//   wavefronts 0 .. 3 form the operands of later chunks: 0, 1 and 2 the tiles
//     of (I + L)^-1 of chunk i + 2 and 3 its A, wavefront 2 also T10 of chunk
//     i + 1 (from the tiles published by the last barrier), 2 or (without OUT)
//     3 the row values of chunk i + 3, and all four issue the loads of q, k (chunk i + 4) and v
//     (chunk i + 2), which must have landed by the end of interval i + 1.
// Bound by the chain of chunks: 1.7 us each with few units (2.25 without OUT),
// 2.2 (2.9) when every compute unit is at work and the clock falls from 2.4 to
// 2.0 GHz. The matrix units are then busy for 45% of the cycles, vector
// instructions issue for a third; products and splits of one chunk wait for
// each other. Measured: 65536 tokens of 8 heads, 190 us without OUT (230 with a
// workgroup each for B and M) and 157 with; eight prompts of 512 to 4096 tokens
// and 32 heads, 240 us (first kernel, on 16x16x32 products and without the
// pipeline: 544).
// Ring slots: q and k 5 chunks, v and the operands 3, the row values 4.
constexpr int N_QK = 5, N_V = 3, N_REC = 3, N_GS = 4;
constexpr int DEPTH = 4;  // intervals from a chunk's first load to its use
template <bool OUT>
struct Lds {
    alignas(16) uint8_t k[N_QK][TILE_BYTES];
    alignas(16) uint8_t q[OUT ? N_QK : 1][TILE_BYTES];  // without OUT: zeros, the V of a transfer
    alignas(16) uint8_t v[N_V][TILE_BYTES];
    alignas(16) uint8_t t[N_REC][REC4];
    alignas(16) uint8_t a[OUT ? N_REC : 1][REC4];
    alignas(16) float gs[N_GS][GS_FLOATS];
    alignas(16) float lt[2 * LMAT];
    alignas(16) float t00[2][LMAT], t11[2][256];
};

// Ring positions of chunks i .. i + N - 1 (uniform).
template <int N>
struct Ring {
    int at[N];
    __device__ __forceinline__ Ring() {
#pragma unroll
        for (int j = 0; j < N; ++j) at[j] = j;
    }
    __device__ __forceinline__ void next() {
        const int first = at[0];
#pragma unroll
        for (int j = 0; j + 1 < N; ++j) at[j] = at[j + 1];
        at[N - 1] = first;
    }
};

// Valid rows of chunk c of a unit of n tokens (0 outside it).
__device__ __forceinline__ int rows_of_chunk(int n, int c) {
    const int left = n - c * GC;
    return __builtin_amdgcn_readfirstlane(c < 0 || left <= 0 ? 0 : left < GC ? left : GC);
}

// What a workgroup works on (uniform).
struct GdWork {
    const uint8_t *q, *k, *v;  // the unit's first rows of its head
    const float* g;            // beta at the same index
    const void* beta;
    uint32_t st_qk, st_v;      // bytes from row to row
    int H, n_tok, n_chunks;
    float scale;
    bool beta_bf16;
};

// The loop of operand wavefront ROLE (a loop per role: values that one role
// carries from interval to interval would make the others wait for its loads).
template <int ROLE, bool OUT>
__device__ __forceinline__ void produce(const GdWork& w, Lds<OUT>& lds, int lane) {
    Ring<N_QK> qk;
    Ring<N_V> rv;
    Ring<N_REC> rec;
    Ring<N_GS> gs;
    // a chunk's rows by the four wavefronts, 8 each
    auto load = [&](const uint8_t* base, uint32_t stride, int c, int rows, uint8_t* tile)
                    __attribute__((always_inline)) {
        const auto rsrc = chunk_rsrc(base + (size_t)(c < 0 ? 0 : c) * GC * stride, (uint32_t)rows * stride);
        load_rows(rsrc, stride, 2 * ROLE, lane, tile);
        load_rows(rsrc, stride, 2 * ROLE + 1, lane, tile);
    };
    constexpr int SCAN = OUT ? 2 : 3;  // who forms the row values: the A of OUT takes wavefront 3 longer
    float x = 0.f;  // SCAN: log-decay of row lane & 31, and its beta's bits
    uint32_t b = 0;
    f32x4 l10 = {0.f, 0.f, 0.f, 0.f};
    // ring position j is chunk i + j
    for (int i = -DEPTH; i < w.n_chunks; ++i) {
        const int par = i & 1, rows = rows_of_chunk(w.n_tok, i + 4);
        load(w.v, w.st_v, i + 2, rows_of_chunk(w.n_tok, i + 2), lds.v[rv.at[2]]);
        load(w.k, w.st_qk, i + 4, rows, lds.k[qk.at[4]]);
        if constexpr (OUT) load(w.q, w.st_qk, i + 4, rows, lds.q[qk.at[4]]);
        const bool inside = i + 2 >= 0 && i + 2 < w.n_chunks;
        const float* g = lds.gs[gs.at[2]];
        const uint8_t* K = lds.k[qk.at[2]];
        if constexpr (ROLE == 0) {
            if (inside) diag_tile<0>(K, g, lds.lt, lds.t00[par], lds.t[rec.at[2]], lane);
        } else if constexpr (ROLE == 1) {
            if (inside) diag_tile<1>(K, g, lds.lt + LMAT, lds.t11[par], lds.t[rec.at[2]], lane);
        } else if constexpr (ROLE == 3 && OUT) {
            if (inside) qk_tiles(lds.q[qk.at[2]], K, g, w.scale, lds.a[rec.at[2]], lane);
        } else if constexpr (ROLE == 2) {
            if (i + 1 >= 0 && i + 1 < w.n_chunks)
                off_diagonal(l10, lds.t00[par ^ 1], lds.t11[par ^ 1], lds.gs[gs.at[1]], lds.t[rec.at[1]], lane);
            if (inside) l10 = lower_tile(K, g, lane);
        }
        if constexpr (ROLE == SCAN) {
            row_scan(x, w.beta_bf16 ? __uint_as_float(b << 16) : __uint_as_float(b), lane, lds.gs[gs.at[3]]);
            const uint32_t at = (uint32_t)(lane & 31) * (uint32_t)w.H, n = rows ? (uint32_t)(rows - 1) * w.H + 1 : 0u;
            const size_t c = (size_t)(i + 4) * GC * w.H;
            x = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(chunk_rsrc(w.g + c, n * 4),
                                                                               (int)(at * 4), 0, 0));
            if (w.beta_bf16)
                b = __builtin_amdgcn_raw_buffer_load_b16(chunk_rsrc((const uint16_t*)w.beta + c, n * 2), (int)(at * 2),
                                                         0, 0);
            else
                b = __builtin_amdgcn_raw_buffer_load_b32(chunk_rsrc((const float*)w.beta + c, n * 4), (int)(at * 4), 0,
                                                         0);
        }
        // the loads of the last interval have landed: at most this one's (q, k, v; g and beta) are still on their way
        constexpr int ISSUED = (OUT ? 6 : 4) + (ROLE == SCAN ? 2 : 0);
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(ISSUED) : "memory");
        lds_barrier();
        qk.next();
        rv.next();
        rec.next();
        gs.next();
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load into LDS outlives the workgroup
}

template <bool OUT>
constexpr int kThreads = OUT ? kGdThreads : kGdSegmentThreads;
static_assert(kThreads<true> == 64 * (4 + 4) && kThreads<false> == 64 * (4 + 8));

template <bool OUT>
__global__ __launch_bounds__(kThreads<OUT>) void gd_prefill(GdArgs a) {
    extern __shared__ __align__(16) uint8_t lds_raw[];
    Lds<OUT>& lds = *(Lds<OUT>*)lds_raw;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int h = blockIdx.x % a.H;
    const GdUnit un = a.units[blockIdx.x / a.H];
    // the unit's tokens, clamped into the sequence and the inputs
    int64_t beg = a.cu[un.seq], end = a.cu[un.seq + 1];
    end = end > a.Tt ? a.Tt : end;
    beg = (beg < 0 ? 0 : beg) + un.tok0;
    end = end < beg + un.n_tok ? end : beg + un.n_tok;
    const int n_tok = __builtin_amdgcn_readfirstlane(end > beg ? (int)(end - beg) : 0);
    const int n_chunks = (n_tok + GC - 1) / GC;
    const uint32_t st_v = (uint32_t)a.H * (D * 2);

    if (wave < 4) {
        GdWork w;
        const int64_t row = beg * a.H + h, row_qk = (beg * a.Hk + h / a.group) * (D * 2);
        w.q = (const uint8_t*)a.q + row_qk;
        w.k = (const uint8_t*)a.k + row_qk;
        w.v = (const uint8_t*)a.v + row * (D * 2);
        w.g = a.g + row;
        w.beta = a.beta_bf16 ? (const void*)((const uint16_t*)a.beta + row) : (const void*)((const float*)a.beta + row);
        w.st_qk = (uint32_t)a.Hk * (D * 2);
        w.st_v = st_v;
        w.H = a.H;
        w.n_tok = n_tok;
        w.n_chunks = n_chunks;
        w.scale = a.scale;
        w.beta_bf16 = a.beta_bf16;
        if (wave == 0) produce<0, OUT>(w, lds, lane);
        else if (wave == 1) produce<1, OUT>(w, lds, lane);
        else if (wave == 2) produce<2, OUT>(w, lds, lane);
        else produce<3, OUT>(w, lds, lane);
        return;
    }

    // wavefronts 4 .. 7: the state, 32 value columns each. Each shares its SIMD
    // with one operand wavefront and goes first (measured: 247 us without, 232
    // with, on eight prompts of 512 to 4096 tokens and 32 heads). Without OUT,
    // wavefronts 8 .. 11 advance the transfer of the same tokens.
    __builtin_amdgcn_s_setprio(2);
    const int col0 = 32 * (wave & 3);
    const bool transfer = !OUT && wave >= 8;
    const int in = transfer ? GD_IDENTITY : un.in, out = transfer ? un.out_m : un.out;
    if (transfer && out < 0) {
        for (int i = -DEPTH; i < n_chunks; ++i) lds_barrier();
        return;
    }
    if (transfer)
        for (int i = (wave & 3) * 64 + lane; i < TILE_BYTES / 16; i += 256)
            *(u32x4*)(lds.q[0] + 16 * i) = u32x4{0, 0, 0, 0};
    // tile (0, 1) of every operand record
    for (int i = (wave & 3) * 64 + lane; !transfer && i < N_REC * 2 * 64; i += 256) {
        const int slot = i >> 7, at = 2048 + (i >> 6 & 1) * 1024 + (32 * (i >> 4 & 1) + (i & 15)) * 16;
        if (!(i >> 5 & 1)) {
            *(u32x4*)(lds.t[slot] + at) = u32x4{0, 0, 0, 0};
            if constexpr (OUT) *(u32x4*)(lds.a[slot] + at) = u32x4{0, 0, 0, 0};
        }
    }
    f32x16 S[4];
    // the element of the 128 x 128 state that element 4a + b of tile t is on this lane
    const int at0 = 8 * (lane >> 5) * D + col0 + value_col(lane & 31);
    auto each = [&](auto f) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                S[t][i] = f(at0 + (32 * t + 16 * (i >> 3) + (i & 7)) * D, S[t][i]);
    };
    const int64_t own = ((int64_t)un.seq * a.H + h) * (D * D);
    if (in >= 0) {
        const float* p = a.carries + ((int64_t)in * a.H + h) * (D * D);
        each([&](int at, float) { return p[at]; });
    } else if (in == GD_INITIAL && a.s0) {
        if (a.state_bf16) {
            const uint16_t* p = (const uint16_t*)a.s0 + own;
            each([&](int at, float) { return __uint_as_float((uint32_t)p[at] << 16); });
        } else {
            const float* p = (const float*)a.s0 + own;
            each([&](int at, float) { return p[at]; });
        }
    } else {
        const float one = in == GD_IDENTITY ? 1.f : 0.f;
        each([&](int at, float) { return at % (D + 1) == 0 ? one : 0.f; });
    }
    for (int i = -DEPTH; i < 0; ++i) lds_barrier();
    uint8_t* ob = (uint8_t*)a.out + (beg * a.H + h) * (D * 2);
    Ring<N_QK> qk;
    Ring<N_V> rv;
    Ring<N_REC> rec;
    Ring<N_GS> gs;
    for (int i = 0; i < DEPTH; ++i) {
        qk.next();
        rv.next();
        rec.next();
        gs.next();
    }
    const MinusOne neg = minus_one(lane);
    Rest rest = {};
    // the output rows of chunk i (none before the first)
    auto store = [&](int i, const f32x16& o) __attribute__((always_inline)) {
        const uint32_t bytes = (uint32_t)rows_of_chunk(n_tok, i) * st_v;
        const auto rsrc = chunk_rsrc(ob + (size_t)(i < 0 ? 0 : i) * GC * st_v, bytes);
        const int at = (int)((lane & 31) * st_v) + (col0 + 16 * (lane >> 5)) * 2;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const u32x2 x = pack4(quarter(o, 2 * j)), y = pack4(quarter(o, 2 * j + 1));
            __builtin_amdgcn_raw_buffer_store_b128(u32x4{x.x, x.y, y.x, y.y}, rsrc, at + 16 * j, 0, 0);
        }
    };
    for (int i = 0; i < n_chunks; ++i) {
        chunk_step<OUT>(lds.q[OUT ? qk.at[0] : 0], lds.k[qk.at[0]],
                        transfer ? lds.q[0] : lds.v[rv.at[0]], lds.t[rec.at[0]],
                        lds.a[OUT ? rec.at[0] : 0], lds.gs[gs.at[0]], a.scale, col0, lane, neg, S, rest,
                        [&](const f32x16& o) __attribute__((always_inline)) { store(i - 1, o); });
        lds_barrier();
        qk.next();
        rv.next();
        rec.next();
        gs.next();
    }
    if constexpr (OUT) {
        finish_output(rest);
        store(n_chunks - 1, rest.o);
    }
    if (transfer) {  // hi and lo in gd_merge's order: [channel / 16][column / 32][hi, lo][lane][8]
        uint16_t* p = (uint16_t*)(a.sums + ((int64_t)out * a.H + h) * (D * D));
        each([&](int at, float s) {
            const int ch = at / D, col = at % D;
            const int to = 16 * (col >> 3 & 3) + (ch & 15);
            uint16_t* dst = p + (ch >> 4) * 4096 + (col >> 5) * 1024 + to * 8 + (col & 7);
            const uint32_t hi = pack_bf16(s, 0.f);
            dst[0] = (uint16_t)hi;
            dst[512] = (uint16_t)pack_bf16(s - bf16_lo(hi), 0.f);
            return s;
        });
    } else if (out >= 0) {
        float* p = a.sums + ((int64_t)out * a.H + h) * (D * D);
        each([&](int at, float s) { return p[at] = s; });
    } else if (out == GD_FINAL && a.sT) {
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

// carry_0 = the initial state, carry_1 = the end state of segment 0, then
// carry_{s+1} = M_s carry_s + B_s. One workgroup of 8 wavefronts per (item,
// head, 16-column tile); wavefront w forms channels 16w .. 16w + 15. M comes as
// hi + lo pairs in the order of the operands; each wavefront splits its part of
// the carry and passes it on through LDS, double-buffered, once per segment.
// The steps are serial, so M and B are loaded two steps ahead. Bound by what
// one compute unit loads, 72 KiB a step: 30 steps take 32 us, and took 56 with
// M as rows, whose 64-byte pieces a load instruction fetches at half the rate
// (splitting M here or three steps ahead made no difference to either).
constexpr int CSTR = D + 8;  // bf16 per column of the carry in LDS
constexpr int AHEAD = 2;
__global__ __launch_bounds__(kGdMergeThreads) void gd_merge(GdMergeArgs a) {
    __shared__ __align__(16) uint16_t carry[2][2][16 * CSTR];  // [step parity][hi, lo]
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, gg = lane >> 4, m = lane & 15;
    // the column tiles of a head are n_items * H apart: with a multiple of 8
    // heads they share an XCD, whose L2 then reads M once
    const int heads = a.n_items * a.H;
    const int ct = blockIdx.x / heads, ih = blockIdx.x % heads, h = ih % a.H;
    const GdMerge it = a.items[ih / a.H];
    const int col = 16 * ct + m, ch = 16 * wave + 4 * gg;
    auto at = [&](int slot) { return ((int64_t)slot * a.H + h) * (D * D) + ch * D + col; };
    struct Step {
        u32x4 h[4], l[4];
        f32x4 b;
    };
    auto load = [&](Step& x, int s) __attribute__((always_inline)) {  // segment s, or the last transfer there is
        s = s < it.n - 2 ? s : it.n - 2;
        const uint8_t* M = (const uint8_t*)(a.sums + ((int64_t)(it.sum0 + 2 * s) * a.H + h) * (D * D)) + wave * 8192 +
                           lane * 16;
        const float* B = a.sums + at(it.sum0 + 2 * s - 1);
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            x.h[p] = *(const u32x4*)(M + 2048 * p);
            x.l[p] = *(const u32x4*)(M + 2048 * p + 1024);
        }
#pragma unroll
        for (int v = 0; v < 4; ++v) x.b[v] = B[v * D];
    };
    Step x[AHEAD];
    if (it.n > 2) {
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) load(x[j], 1 + j);
    }
    auto put = [&](int s, const f32x4& c) __attribute__((always_inline)) {
        float* dst = a.carries + at(it.carry0 + s);
#pragma unroll
        for (int v = 0; v < 4; ++v) dst[v * D] = c[v];
    };
    f32x4 c, c0 = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int v = 0; v < 4; ++v) c[v] = a.sums[at(it.sum0) + v * D];
    if (a.s0 && a.state_bf16) {
#pragma unroll
        for (int v = 0; v < 4; ++v)
            c0[v] = __uint_as_float((uint32_t)((const uint16_t*)a.s0)[at(it.seq) + v * D] << 16);
    } else if (a.s0) {
#pragma unroll
        for (int v = 0; v < 4; ++v) c0[v] = ((const float*)a.s0)[at(it.seq) + v * D];
    }
    put(0, c0);
    put(1, c);
    auto step = [&](Step& x, int s) __attribute__((always_inline)) {
        uint16_t(*buf)[16 * CSTR] = carry[s & 1];
        const HiLo own = split4(c);
        *(u32x2*)(buf[0] + m * CSTR + ch) = own.h;
        *(u32x2*)(buf[1] + m * CSTR + ch) = own.l;
        lds_barrier();
        c = x.b;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const u32x4 bh = *(const u32x4*)(buf[0] + m * CSTR + 32 * p + 8 * gg);
            const u32x4 bl = *(const u32x4*)(buf[1] + m * CSTR + 32 * p + 8 * gg);
            c = mfma_k32(x.l[p], bh, c);
            c = mfma_k32(x.h[p], bl, c);
            c = mfma_k32(x.h[p], bh, c);
        }
        load(x, s + AHEAD);
        put(s + 1, c);
    };
    int s = 1;
    for (; s + AHEAD < it.n; s += AHEAD)
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) step(x[j], s + j);
#pragma unroll
    for (int j = 0; j + 1 < AHEAD; ++j)
        if (s + j + 1 < it.n) step(x[j], s + j);
}

// Decode. With S the state before a token and gam = exp(g), for value column j:
//   a_j = gam sum_r k_r S_rj,  b_j = gam sum_r q_r S_rj,  e_j = v_j - a_j
//   S'_rj = gam S_rj + (beta k_r) e_j,   o_j = scale (b_j + beta (q . k) e_j)
// One wavefront per (sequence, head, 32-column tile) keeps its part of the
// state in registers over all T tokens: lane (rs, cg) = (lane >> 3, lane & 7)
// owns rows 16rs .. + 15 of columns 4cg .. + 3, so a load instruction covers
// eight whole 128-byte lines, the sums need three lane exchanges and the
// kernel needs neither LDS nor a barrier. Bound by HBM: 128 KiB of state
// traffic per (sequence, head) against 1 KiB per token; 256 sequences of 32
// heads take 193 us (5.6 TB/s). One sequence takes 7 us, which is the latency
// of the launch and of one load after another.
//
// States beyond 128 MiB, half the last-level cache, are read and written with
// the nontemporal hint. Where the states are not in that cache (several layers
// take turns) it is faster at every size: 51 us against 56 for 64 sequences of
// 32 heads (128 MiB), 62 against 70 for 80. Where a call finds the states of
// the one before, it costs: 49 against 43, 60 against 53, and 196 against 217
// from 352 MiB on.
static_assert(kGdDecodeThreads == 64 * 4);  // a wavefront per 32-column tile

template <bool NT>
__global__ __launch_bounds__(kGdDecodeThreads) void gd_decode(GdDecodeArgs a) {
    const int lane = threadIdx.x & 63, tile = threadIdx.x >> 6;
    const int64_t nh = blockIdx.x;
    const int64_t n = nh / a.H;
    const int h = (int)(nh % a.H), hq = h / a.group;
    const int rs = lane >> 3, col = 32 * tile + 4 * (lane & 7);
    const int64_t slot = a.slots ? (int64_t)a.slots[n] : n;
    if (slot < 0 || slot >= a.n_slots) {
        for (int t = rs; t < a.T; t += 8) *(uint2*)(a.out + ((n * a.T + t) * a.H + h) * D + col) = uint2{0u, 0u};
        return;
    }
    f32x4* st = (f32x4*)(a.state + (slot * a.H + h) * (D * D) + (16 * rs) * D + col);
    f32x4 s[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        if constexpr (NT) s[i] = __builtin_nontemporal_load(st + i * (D / 4));
        else s[i] = st[i * (D / 4)];
    }
    for (int t = 0; t < a.T; ++t) {
        const int64_t row = (n * a.T + t) * a.H + h, rq = (n * a.T + t) * a.Hk + hq;
        const u32x4* kp = (const u32x4*)(a.k + rq * D + 16 * rs);
        const u32x4* qp = (const u32x4*)(a.q + rq * D + 16 * rs);
        const u32x4 k2[2] = {kp[0], kp[1]}, q2[2] = {qp[0], qp[1]};
        const u32x2 vb = *(const u32x2*)(a.v + row * D + col);
        const float beta = a.beta[row], gam = exp2_hw(a.g[row] * LOG2E);
        float k[16], q[16], qk = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            k[2 * i] = bf16_lo(k2[i >> 2][i & 3]);
            k[2 * i + 1] = bf16_hi(k2[i >> 2][i & 3]);
            q[2 * i] = bf16_lo(q2[i >> 2][i & 3]);
            q[2 * i + 1] = bf16_hi(q2[i >> 2][i & 3]);
        }
        f32x4 sa = {0.f, 0.f, 0.f, 0.f}, sb = sa;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            qk = __builtin_fmaf(q[i], k[i], qk);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                sa[j] = __builtin_fmaf(k[i], s[i][j], sa[j]);
                sb[j] = __builtin_fmaf(q[i], s[i][j], sb[j]);
            }
        }
#pragma unroll
        for (int d = 8; d < 64; d <<= 1) {
            qk += __shfl_xor(qk, d, 64);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                sa[j] += __shfl_xor(sa[j], d, 64);
                sb[j] += __shfl_xor(sb[j], d, 64);
            }
        }
        const f32x4 v = {bf16_lo(vb.x), bf16_hi(vb.x), bf16_lo(vb.y), bf16_hi(vb.y)};
        f32x4 e, o;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            e[j] = __builtin_fmaf(-gam, sa[j], v[j]);
            o[j] = a.scale * __builtin_fmaf(beta * qk, e[j], gam * sb[j]);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][j] = __builtin_fmaf(gam, s[i][j], (beta * k[i]) * e[j]);
        if (rs == 0) *(u32x2*)(a.out + row * D + col) = pack4(o);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        if constexpr (NT) __builtin_nontemporal_store(s[i], st + i * (D / 4));
        else st[i * (D / 4)] = s[i];
    }
}

}  // namespace

template <bool OUT>
hipError_t run_gd_prefill(const GdArgs& a, hipStream_t s) {
    // more LDS than the default limit, allowed once per device and process
    static std::mutex mu;
    static uint64_t done[4] = {0, 0, 0, 0};
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    {
        std::lock_guard<std::mutex> lk(mu);
        if (dev >= 256 || !(done[dev >> 6] >> (dev & 63) & 1)) {
            e = hipFuncSetAttribute((const void*)gd_prefill<OUT>, hipFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)sizeof(Lds<OUT>));
            if (e != hipSuccess) return e;
            if (dev < 256) done[dev >> 6] |= 1ull << (dev & 63);
        }
    }
    const dim3 grid((unsigned)(a.n_units * a.H)), block(kThreads<OUT>);
    hipLaunchKernelGGL((gd_prefill<OUT>), grid, block, sizeof(Lds<OUT>), s, a);
    return hipGetLastError();
}

hipError_t launch_gd_prefill(const GdArgs& a, bool with_out, hipStream_t s) {
    if (a.n_units == 0) return hipSuccess;
    return with_out ? run_gd_prefill<true>(a, s) : run_gd_prefill<false>(a, s);
}

hipError_t launch_gd_merge(const GdMergeArgs& a, hipStream_t s) {
    hipLaunchKernelGGL(gd_merge, dim3((unsigned)(a.n_items * a.H * kGdMergeTiles)), dim3(kGdMergeThreads),
                       0, s, a);
    return hipGetLastError();
}

hipError_t launch_gd_decode(const GdDecodeArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)(a.n_seqs * a.H)), block(kGdDecodeThreads);
    const bool nt = (size_t)a.n_seqs * a.H * (D * D * 4) > ((size_t)128 << 20);
    if (nt) hipLaunchKernelGGL(gd_decode<true>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(gd_decode<false>, grid, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace kda
