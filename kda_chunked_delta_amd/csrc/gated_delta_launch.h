// Internal interface between the host code and the kernels of the gated delta
// rule (gated_delta.hip). Not part of the public C ABI.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

constexpr int kGdChunk = 32;  // tokens per chunk of the gated delta prefill

// Threads of a workgroup: the prefill's (one per unit and head) with output and
// for a segment's end state and transfer, the merge's (kGdMergeTiles per
// sequence and head) and the decode's (one per sequence and head).
constexpr int kGdThreads = 512, kGdSegmentThreads = 768, kGdMergeThreads = 512, kGdDecodeThreads = 256;
constexpr int kGdMergeTiles = 8;

// A run of tokens of one sequence, advanced by one workgroup per head. `in` and
// `out` name the state it starts from and where its end state goes.
struct GdUnit {
    int32_t seq;
    int32_t tok0;   // first token within the sequence
    int32_t n_tok;  // tokens to run (may be 0)
    int32_t in;     // GD_ZERO, GD_INITIAL, GD_IDENTITY, or a carry slot (>= 0)
    int32_t out;    // GD_NONE, GD_FINAL, or a summary slot (>= 0)
    int32_t out_m;  // where the transfer of the tokens goes: GD_NONE or a summary slot
};
enum : int32_t { GD_ZERO = -1, GD_INITIAL = -2, GD_IDENTITY = -3 };
enum : int32_t { GD_NONE = -1, GD_FINAL = -2 };

// The segments 0 .. n - 1 of one sequence. Carry slot carry0 + s holds the
// state before segment s; summary slot sum0 the end state of segment 0, slots
// sum0 + 2 s - 1 and sum0 + 2 s the end state B_s from zero and the transfer
// M_s of segment s = 1 .. n - 2 (M as pairs of bf16 in the merge's own order).
struct GdMerge {
    int32_t seq;
    int32_t n;
    int32_t carry0;
    int32_t sum0;
};

struct GdArgs {
    const uint16_t* q;   // [Tt][Hk][128] bf16
    const uint16_t* k;
    const uint16_t* v;   // [Tt][H][128] bf16
    const float* g;      // [Tt][H] log-decay
    const void* beta;    // [Tt][H] fp32, or bf16 when beta_bf16
    const int32_t* cu;   // device cu_seqlens
    int64_t Tt;
    int32_t H, Hk, group;
    const GdUnit* units;
    int32_t n_units;
    const void* s0;      // may be null: zero initial states
    void* sT;            // may be null
    const float* carries;  // [slots][H][128][128]
    float* sums;           // [slots][H][128][128]
    uint16_t* out;
    float scale;
    int32_t beta_bf16, state_bf16;
};

struct GdMergeArgs {
    const GdMerge* items;
    int32_t n_items;
    int32_t H;
    const void* s0;
    int32_t state_bf16;
    const float* sums;
    float* carries;
};

struct GdDecodeArgs {
    const uint16_t* q;     // [n_seqs][T][Hk][128] bf16
    const uint16_t* k;
    const uint16_t* v;     // [n_seqs][T][H][128] bf16
    const float* g;        // [n_seqs][T][H]
    const float* beta;     // [n_seqs][T][H]
    float* state;          // [n_slots][H][128][128], read and written
    uint16_t* out;
    int32_t n_seqs, T, H, Hk, group;
    float scale;
    const int32_t* slots;  // null: sequence n uses state[n]
    int32_t n_slots;
};

hipError_t launch_gd_prefill(const GdArgs& a, bool with_out, hipStream_t s);
hipError_t launch_gd_merge(const GdMergeArgs& a, hipStream_t s);
hipError_t launch_gd_decode(const GdDecodeArgs& a, hipStream_t s);

}  // namespace kda
