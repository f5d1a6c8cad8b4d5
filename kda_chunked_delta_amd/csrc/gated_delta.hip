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
// 2^-18 per step against the 2^-9 of single bf16 operands.
#include "gated_delta_launch.h"
#include "kda_device.hpp"

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
__device__ __forceinline__ void load_rows(__amdgpu_buffer_rsrc_t rsrc, uint32_t stride, int i, int lane, uint8_t* tile) {
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

// T' and A of a chunk as operands of 16x16x32 products: [row tile 2][hi, lo]
// [lane 64][8 bf16], lane (gg, m) holding row m of the row tile and columns
// 4gg + j (j < 4) and 16 + 4gg + j - 4 (j >= 4).
constexpr int REC4 = 4096;
__device__ __forceinline__ void put_half(uint8_t* rec, int rt, int half, int lane, const f32x4& x) {
    const HiLo s = split4(x);
    *(u32x2*)(rec + ((rt * 2 + 0) * 64 + lane) * 16 + 8 * half) = s.h;
    *(u32x2*)(rec + ((rt * 2 + 1) * 64 + lane) * 16 + 8 * half) = s.l;
}

__device__ __forceinline__ float pair_decay(float hr, float lr, float hi, float li) {
    return exp2_hw((hr - hi) + (lr - li));
}

// Scratch of the inverse, fp32: two 16 x 16 matrices per diagonal tile with a
// row stride of 20 floats, T00 as lane (gg, m) -> T00[4gg + s][m], T11 as
// lane (gg, m) -> T11[m][4gg + s].
constexpr int LSTR = 20;
constexpr int LMAT = 16 * LSTR;

// (I + L)^-1 of a diagonal 16 x 16 tile on one wavefront, both as t[s] =
// T[4gg + s][m] (by rows) and u[s] = T[m][4gg + s] (by columns): 15 dependent
// steps of a DPP broadcast and a multiply-subtract each.
template <bool ROWS>
__device__ __forceinline__ void invert_tile(const float* lt, int lane, f32x4& t, f32x4& u) {
    const int gg = lane >> 4, m = lane & 15;
    float lr[16], lc[16];  // L[m][K], L[K][m]
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const f32x4 a = *(const f32x4*)(lt + m * LSTR + 4 * q);
#pragma unroll
        for (int v = 0; v < 4; ++v) lr[4 * q + v] = a[v];
        if constexpr (ROWS) {
            const f32x4 b = *(const f32x4*)(lt + LMAT + m * LSTR + 4 * q);
#pragma unroll
            for (int v = 0; v < 4; ++v) lc[4 * q + v] = b[v];
        }
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) t[s] = u[s] = (4 * gg + s == m) ? 1.f : 0.f;
    auto step = [&](auto kc) __attribute__((always_inline)) {
        constexpr int K = decltype(kc)::value;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            u[s] -= lr[K] * row_newbcast<K>(u[s]);
            if constexpr (ROWS) t[s] -= lc[15 - K] * row_newbcast<15 - K>(t[s]);
        }
    };
    step(std::integral_constant<int, 0>{});  step(std::integral_constant<int, 1>{});
    step(std::integral_constant<int, 2>{});  step(std::integral_constant<int, 3>{});
    step(std::integral_constant<int, 4>{});  step(std::integral_constant<int, 5>{});
    step(std::integral_constant<int, 6>{});  step(std::integral_constant<int, 7>{});
    step(std::integral_constant<int, 8>{});  step(std::integral_constant<int, 9>{});
    step(std::integral_constant<int, 10>{}); step(std::integral_constant<int, 11>{});
    step(std::integral_constant<int, 12>{}); step(std::integral_constant<int, 13>{});
    step(std::integral_constant<int, 14>{});
}

// Diagonal tile td of T': its rows go to the record, the unscaled inverse to
// the scratch of the off-diagonal tile (T00 by rows, T11 by columns).
template <int TD>
__device__ __forceinline__ void diag_tile(const uint8_t* K, const float* gs, float* lt, float* inv, uint8_t* rec_t,
                                          int lane) {
    const int gg = lane >> 4, m = lane & 15, r0 = 16 * TD;
    const f32x4 a = gram(K, r0, K, r0, lane);  // k_{4gg + v} . k_m
    const f32x4 hv = *(const f32x4*)(gs + GS_H + r0 + 4 * gg), lv = *(const f32x4*)(gs + GS_L + r0 + 4 * gg);
    const f32x4 bv = *(const f32x4*)(gs + GS_BETA + r0 + 4 * gg);
    const float hm = gs[GS_H + r0 + m], lm = gs[GS_L + r0 + m], bm = gs[GS_BETA + r0 + m];
    f32x4 row, col;  // L[m][4gg + v], L[4gg + v][m]
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        row[v] = 4 * gg + v < m ? bm * a[v] * pair_decay(hm, lm, hv[v], lv[v]) : 0.f;
        col[v] = m < 4 * gg + v ? bv[v] * a[v] * pair_decay(hv[v], lv[v], hm, lm) : 0.f;
    }
    *(f32x4*)(lt + m * LSTR + 4 * gg) = row;
    if constexpr (TD == 0) *(f32x4*)(lt + LMAT + m * LSTR + 4 * gg) = col;
    f32x4 t, u;
    invert_tile<TD == 0>(lt, lane, t, u);
    *(f32x4*)(inv + lane * 4) = TD == 0 ? t : u;
    put_half(rec_t, TD, TD, lane, u * bv);
    if constexpr (TD == 0) put_half(rec_t, 0, 1, lane, f32x4{0.f, 0.f, 0.f, 0.f});
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
    const f32x4 a = *(const f32x4*)(t00 + lane * 4), b = *(const f32x4*)(t11 + lane * 4);
    f32x4 y = {0.f, 0.f, 0.f, 0.f}, z = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < 4; ++s) y = mfma_f32_k4(l10[s], b[s], y);
#pragma unroll
    for (int s = 0; s < 4; ++s) z = mfma_f32_k4(a[s], y[s], z);
    const f32x4 bv = *(const f32x4*)(gs + GS_BETA + 4 * (lane >> 4));
    put_half(rec_t, 1, 0, lane, -z * bv);
}

// A (masked, decayed q-k products) to its record.
__device__ __forceinline__ void qk_tiles(const uint8_t* Q, const uint8_t* K, const float* gs, uint8_t* rec_a, int lane) {
    const int gg = lane >> 4, m = lane & 15;
#pragma unroll
    for (int rt = 0; rt < 2; ++rt)
#pragma unroll
        for (int ct = 0; ct < 2; ++ct) {
            f32x4 r = {0.f, 0.f, 0.f, 0.f};
            if (ct <= rt) {
                const f32x4 a = gram(K, 16 * ct, Q, 16 * rt, lane);  // k_{4gg + v} . q_m
                const f32x4 hv = *(const f32x4*)(gs + GS_H + 16 * ct + 4 * gg);
                const f32x4 lv = *(const f32x4*)(gs + GS_L + 16 * ct + 4 * gg);
                const float hm = gs[GS_H + 16 * rt + m], lm = gs[GS_L + 16 * rt + m];
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    r[v] = (ct < rt || 4 * gg + v <= m) ? a[v] * pair_decay(hm, lm, hv[v], lv[v]) : 0.f;
            }
            put_half(rec_a, rt, ct, lane, r);
        }
}

// The state of one wavefront: NT tiles of 16 value columns. S[2p + e][n] holds,
// on lane (gg, m), channels 32p + 8gg + 4e + v of column 16n + m: two tiles
// together are one 16x16x32 operand with 8 consecutive channels per lane.
template <int NT>
struct State {
    f32x4 s[8][NT];
};

// Advances the state over one chunk; with OUT, o[rt][n] gets the unscaled
// output of token 16rt + m, columns 16n + 4gg + v.
template <int NT, bool OUT>
__device__ __forceinline__ void chunk_step(const uint8_t* Q, const uint8_t* K, const uint8_t* V, const uint8_t* rec_t,
                                           const uint8_t* rec_a, const float* gs, int col0, int lane, State<NT>& st,
                                           f32x4 (&o)[2][NT]) {
    const int gg = lane >> 4, m = lane & 15, tr = (lane >> 2) & 3, tc = lane & 3;
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    f32x4 P[2][NT];
#pragma unroll
    for (int rt = 0; rt < 2; ++rt)
#pragma unroll
        for (int n = 0; n < NT; ++n) P[rt][n] = o[rt][n] = zero;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        u32x4 sh[NT], sl[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const HiLo a = split4(st.s[2 * p][n]), b = split4(st.s[2 * p + 1][n]);
            sh[n] = u32x4{a.h.x, a.h.y, b.h.x, b.h.y};
            sl[n] = u32x4{a.l.x, a.l.y, b.l.x, b.l.y};
        }
#pragma unroll
        for (int rt = 0; rt < 2; ++rt) {
            const u32x4 kf = row_frag(K, 16 * rt, p, lane);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                P[rt][n] = mfma_k32(kf, sh[n], P[rt][n]);
                P[rt][n] = mfma_k32(kf, sl[n], P[rt][n]);
            }
            if constexpr (OUT) {
                const u32x4 qf = row_frag(Q, 16 * rt, p, lane);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    o[rt][n] = mfma_k32(sh[n], qf, o[rt][n]);
                    o[rt][n] = mfma_k32(sl[n], qf, o[rt][n]);
                }
            }
        }
    }
    // R = V - diag(gam) P, then U = T' R
    u32x4 rh[NT], rl[NT], uh[NT], ul[NT], wh[NT], wl[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        HiLo r[2];
#pragma unroll
        for (int rt = 0; rt < 2; ++rt) {
            const f32x4 gam = *(const f32x4*)(gs + GS_GAM + 16 * rt + 4 * gg);
            const u32x2 vw = lds_load_tr16(V + tile_off(16 * rt + 4 * gg + tr, (col0 >> 3) + 2 * n + (tc >> 1)) +
                                           8 * (tc & 1));
            r[rt] = split4(f32x4{bf16_lo(vw.x) - gam[0] * P[rt][n][0], bf16_hi(vw.x) - gam[1] * P[rt][n][1],
                                 bf16_lo(vw.y) - gam[2] * P[rt][n][2], bf16_hi(vw.y) - gam[3] * P[rt][n][3]});
        }
        rh[n] = u32x4{r[0].h.x, r[0].h.y, r[1].h.x, r[1].h.y};
        rl[n] = u32x4{r[0].l.x, r[0].l.y, r[1].l.x, r[1].l.y};
    }
    f32x4 U[2][NT];
#pragma unroll
    for (int rt = 0; rt < 2; ++rt) {
        const u32x4 th = *(const u32x4*)(rec_t + ((rt * 2 + 0) * 64 + lane) * 16);
        const u32x4 tl = *(const u32x4*)(rec_t + ((rt * 2 + 1) * 64 + lane) * 16);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            f32x4 u = mfma_k32(tl, rh[n], zero);
            u = mfma_k32(th, rl[n], u);
            U[rt][n] = mfma_k32(th, rh[n], u);
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        HiLo w[2], u[2];
#pragma unroll
        for (int rt = 0; rt < 2; ++rt) {
            const f32x4 last = *(const f32x4*)(gs + GS_LAST + 16 * rt + 4 * gg);
            w[rt] = split4(last * U[rt][n]);
            if constexpr (OUT) u[rt] = split4(U[rt][n]);
        }
        wh[n] = u32x4{w[0].h.x, w[0].h.y, w[1].h.x, w[1].h.y};
        wl[n] = u32x4{w[0].l.x, w[0].l.y, w[1].l.x, w[1].l.y};
        if constexpr (OUT) {
            uh[n] = u32x4{u[0].h.x, u[0].h.y, u[1].h.x, u[1].h.y};
            ul[n] = u32x4{u[0].l.x, u[0].l.y, u[1].l.x, u[1].l.y};
        }
    }
    // S = gam_31 S + K^T W
    const float gc = gs[GS_GAM + 31];
#pragma unroll
    for (int t = 0; t < 8; ++t) {
        const int gi = 4 * (t >> 1) + tc, e = 8 * (t & 1);
        const u32x2 k0 = lds_load_tr16(K + tile_off(4 * gg + tr, gi) + e);
        const u32x2 k1 = lds_load_tr16(K + tile_off(16 + 4 * gg + tr, gi) + e);
        const u32x4 kt = {k0.x, k0.y, k1.x, k1.y};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            f32x4 s = gc * st.s[t][n];
            s = mfma_k32(kt, wl[n], s);
            st.s[t][n] = mfma_k32(kt, wh[n], s);
        }
    }
    if constexpr (OUT) {
#pragma unroll
        for (int rt = 0; rt < 2; ++rt) {
            const float gam = gs[GS_GAM + 16 * rt + m];
            const u32x4 ah = *(const u32x4*)(rec_a + ((rt * 2 + 0) * 64 + lane) * 16);
            const u32x4 al = *(const u32x4*)(rec_a + ((rt * 2 + 1) * 64 + lane) * 16);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                f32x4 x = gam * o[rt][n];
                x = mfma_k32(ul[n], ah, x);
                x = mfma_k32(uh[n], al, x);
                o[rt][n] = mfma_k32(uh[n], ah, x);
            }
        }
    }
}

__device__ __forceinline__ float load_state(const void* p, int64_t i, bool bf16) {
    return bf16 ? __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16) : ((const float*)p)[i];
}

// The channel of row v of tile t on lane group gg.
__device__ __forceinline__ int state_channel(int t, int gg, int v) { return 32 * (t >> 1) + 8 * gg + 4 * (t & 1) + v; }

template <int NT, bool OUT>
__global__ __launch_bounds__(512) void gd_prefill(GdArgs a) {
    constexpr int COLS = 64 * NT, NCT = D / COLS;
    __shared__ __align__(16) uint8_t sQ[TILE_BYTES], sK[TILE_BYTES], sV[TILE_BYTES], sT_[REC4], sA[REC4];
    __shared__ __align__(16) float gs[GS_FLOATS], lt[3 * LMAT], t00[256], t11[256];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int gg = lane >> 4, m = lane & 15;
    const int ct = blockIdx.x % NCT, uh = blockIdx.x / NCT;
    const int h = uh % a.H;
    const GdUnit un = a.units[uh / a.H];
    // the unit's tokens, clamped into the sequence and the inputs
    int64_t beg = a.cu[un.seq], end = a.cu[un.seq + 1];
    end = end > a.Tt ? a.Tt : end;
    beg = (beg < 0 ? 0 : beg) + un.tok0;
    end = end < beg + un.n_tok ? end : beg + un.n_tok;
    const int n_tok = __builtin_amdgcn_readfirstlane(end > beg ? (int)(end - beg) : 0);
    const int n_chunks = (n_tok + GC - 1) / GC;
    const uint32_t st_qk = (uint32_t)a.Hk * (D * 2), st_v = (uint32_t)a.H * (D * 2);
    const uint8_t* qb = (const uint8_t*)a.q + (beg * a.Hk + h / a.group) * (D * 2);
    const uint8_t* kb = (const uint8_t*)a.k + (beg * a.Hk + h / a.group) * (D * 2);
    const uint8_t* vb = (const uint8_t*)a.v + (beg * a.H + h) * (D * 2);
    uint8_t* ob = (uint8_t*)a.out + (beg * a.H + h) * (D * 2);

    const bool chain = wave >= 4;  // wavefronts 4 .. 7 hold the state
    const int col0 = ct * COLS + (wave - 4) * (16 * NT);
    State<NT> st;
    if (chain) {
        const void* src = un.in >= 0 ? (const void*)(a.carries + ((int64_t)un.in * a.H + h) * (D * D))
                                     : (const void*)a.s0;
        const bool b16 = un.in < 0 && a.state_bf16;
        const int64_t base = un.in >= 0 ? 0 : ((int64_t)un.seq * a.H + h) * (D * D);
        const bool load = un.in >= 0 || (un.in == GD_INITIAL && a.s0);
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const int ch = state_channel(t, gg, v), col = col0 + 16 * n + m;
                    st.s[t][n][v] = load ? load_state(src, base + ch * D + col, b16)
                                         : (un.in == GD_IDENTITY && ch == col ? 1.f : 0.f);
                }
    }
    for (int ci = 0; ci < n_chunks; ++ci) {
        const int left = n_tok - ci * GC, nrows = left < GC ? left : GC;
        __syncthreads();  // the tiles of the last chunk are free
        {
            const size_t cq = (size_t)ci * GC * st_qk, cv = (size_t)ci * GC * st_v;
            load_rows(chunk_rsrc(kb + cq, (uint32_t)nrows * st_qk), st_qk, wave, lane, sK);
            load_rows(chunk_rsrc(vb + cv, un.with_v ? (uint32_t)nrows * st_v : 0u), st_v, wave, lane, sV);
            if constexpr (OUT) load_rows(chunk_rsrc(qb + cq, (uint32_t)nrows * st_qk), st_qk, wave, lane, sQ);
        }
        if (wave == 0) {
            const int r = lane & 31;
            float x = 0.f, b = 0.f;
            if (r < nrows) {
                const int64_t i = (beg + ci * GC + r) * a.H + h;
                x = a.g[i];
                b = a.beta_bf16 ? __uint_as_float((uint32_t)((const uint16_t*)a.beta)[i] << 16)
                                : ((const float*)a.beta)[i];
            }
            row_scan(x, b, lane, gs);
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        f32x4 l10 = {0.f, 0.f, 0.f, 0.f};
        if (wave == 0) diag_tile<0>(sK, gs, lt, t00, sT_, lane);
        else if (wave == 1) diag_tile<1>(sK, gs, lt + 2 * LMAT, t11, sT_, lane);
        else if (wave == 2) l10 = lower_tile(sK, gs, lane);
        else if (OUT && wave == 3) qk_tiles(sQ, sK, gs, sA, lane);
        __syncthreads();
        if (wave == 2) off_diagonal(l10, t00, t11, gs, sT_, lane);
        __syncthreads();
        if (chain) {
            f32x4 o[2][NT];
            chunk_step<NT, OUT>(sQ, sK, sV, sT_, sA, gs, col0, lane, st, o);
            if constexpr (OUT) {
                const auto rsrc = chunk_rsrc(ob + (size_t)ci * GC * st_v, (uint32_t)nrows * st_v);
#pragma unroll
                for (int rt = 0; rt < 2; ++rt)
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const f32x4 x = a.scale * o[rt][n];
                        __builtin_amdgcn_raw_buffer_store_b64(pack4(x), rsrc,
                                                              (int)((16 * rt + m) * st_v + (col0 + 16 * n + 4 * gg) * 2),
                                                              0, 0);
                    }
            }
        }
    }
    if (chain && (un.out >= 0 || (un.out == GD_FINAL && a.sT))) {
        const bool b16 = un.out < 0 && a.state_bf16;
        const int64_t base = ((int64_t)(un.out >= 0 ? un.out : un.seq) * a.H + h) * (D * D);
        float* f = un.out >= 0 ? a.sums : (float*)a.sT;
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const int64_t i = base + state_channel(t, gg, v) * D + col0 + 16 * n + m;
                    if (b16) ((uint16_t*)a.sT)[i] = (uint16_t)pack_bf16(st.s[t][n][v], 0.f);
                    else f[i] = st.s[t][n][v];
                }
    }
}

// carry_0 = the initial state, carry_1 = the end state of segment 0, then
// carry_{s+1} = M_s carry_s + B_s. One workgroup of 8 wavefronts per (item,
// head, 16-column tile); wavefront w forms channels 16w .. 16w + 15, with M and
// the carry as hi + lo pairs. The carry goes from wavefront to wavefront
// through LDS, once per segment.
constexpr int CSTR = D + 4;  // floats per column of the carry in LDS
__global__ __launch_bounds__(512) void gd_merge(GdMergeArgs a) {
    __shared__ __align__(16) float carry[16 * CSTR];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, gg = lane >> 4, m = lane & 15;
    const int ct = blockIdx.x % 8, ih = blockIdx.x / 8, h = ih % a.H;
    const GdMerge it = a.items[ih / a.H];
    const int col = 16 * ct + m, ch = 16 * wave + 4 * gg;
    auto at = [&](int slot) { return ((int64_t)slot * a.H + h) * (D * D) + ch * D + col; };
    f32x4 c;
    if (it.n < 2) return;
    for (int s = 0; s < 2; ++s) {
        float* dst = a.carries + at(it.carry0 + s);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            c[v] = s ? a.sums[at(it.sum0) + v * D] : a.s0 ? load_state(a.s0, at(it.seq) + v * D, a.state_bf16) : 0.f;
            dst[v * D] = c[v];
        }
    }
    for (int s = 1; s + 1 < it.n; ++s) {
        *(f32x4*)(carry + m * CSTR + ch) = c;
        const int64_t bm = at(it.sum0 + 2 * s - 1);
        const float* M = a.sums + ((int64_t)(it.sum0 + 2 * s) * a.H + h) * (D * D) + (16 * wave + m) * D + 8 * gg;
#pragma unroll
        for (int v = 0; v < 4; ++v) c[v] = a.sums[bm + v * D];
        __syncthreads();
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const HiLo a0 = split4(*(const f32x4*)(M + 32 * p)), a1 = split4(*(const f32x4*)(M + 32 * p + 4));
            const float* cc = carry + m * CSTR + 32 * p + 8 * gg;
            const HiLo b0 = split4(*(const f32x4*)cc), b1 = split4(*(const f32x4*)(cc + 4));
            const u32x4 ah = {a0.h.x, a0.h.y, a1.h.x, a1.h.y}, al = {a0.l.x, a0.l.y, a1.l.x, a1.l.y};
            const u32x4 bh = {b0.h.x, b0.h.y, b1.h.x, b1.h.y}, bl = {b0.l.x, b0.l.y, b1.l.x, b1.l.y};
            c = mfma_k32(al, bh, c);
            c = mfma_k32(ah, bl, c);
            c = mfma_k32(ah, bh, c);
        }
        __syncthreads();
        float* dst = a.carries + at(it.carry0 + s + 1);
#pragma unroll
        for (int v = 0; v < 4; ++v) dst[v * D] = c[v];
    }
}

// Decode. With S the state before a token and gam = exp(g), for value column j:
//   a_j = gam sum_r k_r S_rj,  b_j = gam sum_r q_r S_rj,  e_j = v_j - a_j
//   S'_rj = gam S_rj + (beta k_r) e_j,   o_j = scale (b_j + beta (q . k) e_j)
// One wavefront per (sequence, head, 32-column tile) keeps its part of the
// state in registers over all T tokens: lane (rs, cg) = (lane >> 3, lane & 7)
// owns rows 16rs .. + 15 of columns 4cg .. + 3, so a load instruction covers
// eight whole 128-byte lines, the sums need three lane exchanges and the
// kernel needs neither LDS nor a barrier. Bound by HBM: 128 KiB of state
// traffic per (sequence, head) against 1 KiB per token.
constexpr int DEC_W = 4;  // wavefronts (32-column tiles) per workgroup

template <bool NT>
__global__ __launch_bounds__(64 * DEC_W) void gd_decode(GdDecodeArgs a) {
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

hipError_t launch_gd_prefill(const GdArgs& a, bool with_out, hipStream_t s) {
    if (a.n_units == 0) return hipSuccess;
    const dim3 grid((unsigned)(a.n_units * a.H)), block(512);
    if (with_out) hipLaunchKernelGGL((gd_prefill<2, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((gd_prefill<2, false>), grid, block, 0, s, a);
    return hipGetLastError();
}

hipError_t launch_gd_merge(const GdMergeArgs& a, hipStream_t s) {
    hipLaunchKernelGGL(gd_merge, dim3((unsigned)(a.n_items * a.H * 8)), dim3(512), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_gd_decode(const GdDecodeArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)(a.n_seqs * a.H)), block(64 * DEC_W);
    const bool nt = (size_t)a.n_seqs * a.H * (D * D * 4) > ((size_t)128 << 20);
    if (nt) hipLaunchKernelGGL(gd_decode<true>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(gd_decode<false>, grid, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace kda
