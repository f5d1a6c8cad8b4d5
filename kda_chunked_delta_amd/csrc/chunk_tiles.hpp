// Device building blocks of the chunked kernels with one decay per token and
// head (gated_delta.hip, linear_attention.hip): chunks of 32 token rows in LDS,
// and 32 x 32 matrix products on a 128 x 128 state held in registers.
#pragma once
#include "kda_device.hpp"

namespace kda {

constexpr int TILE_ROWS = 32;                  // tokens per chunk
constexpr int TILE_BYTES = TILE_ROWS * D * 2;  // one chunk of q, k or v of one head (8 KiB)

// LDS tiles hold token rows of 256 bytes; the 16-byte granules of row r are
// permuted by XOR with tile_swz(r). Row fragments (16 rows, one granule) and the
// transposing loads (4 rows of each 16-lane group, 4 granules) then both touch
// 16 distinct granule positions.
__device__ __forceinline__ int tile_swz(int row) { return ((row & 3) << 2) | ((row >> 2) & 3); }
__device__ __forceinline__ int tile_off(int row, int gi) { return row * 256 + ((gi ^ tile_swz(row)) << 4); }

// Rows 4i .. 4i + 3 of a tile by one direct-to-LDS load. Rows past the
// descriptor's range become zeros. NT: with the nontemporal hint.
template <bool NT = false>
__device__ __forceinline__ void load_rows(__amdgpu_buffer_rsrc_t rsrc, uint32_t stride, int i, int lane,
                                          uint8_t* tile) {
    const int row = 4 * i + (lane >> 4);
    const uint32_t off = (uint32_t)row * stride + (((lane & 15) ^ tile_swz(row)) << 4);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (__attribute__((address_space(3))) void*)(tile + 1024 * i), 16,
                                             (int)off, 0, 0, NT ? 2 : 0);
}

// Below this log2-decay a token's decay is zero in fp32 and stands for any
// smaller one (-inf included), which keeps the running sum finite.
constexpr float LOG2_FLOOR = -160.0f;
// e^(G_r - G_i) from two running sums of log2-decays in hi + lo form.
__device__ __forceinline__ float pair_decay(float hr, float lr, float hi, float li) {
    return exp2_hw((hr - hi) + (lr - li));
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
    const int left = n - c * TILE_ROWS;
    return __builtin_amdgcn_readfirstlane(c < 0 || left <= 0 ? 0 : left < TILE_ROWS ? left : TILE_ROWS);
}

}  // namespace kda
