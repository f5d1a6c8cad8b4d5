// Internal interface between the host code and the kernels of linear attention
// (linear_attention.hip). Not part of the public C ABI.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

constexpr int kLaChunk = 32;  // tokens per chunk of the prefill

// Threads of a workgroup: the prefill's (one per unit and head), the merge's
// (kLaMergeTiles per sequence and head) and the decode's (one per sequence and head).
constexpr int kLaThreads = 512, kLaMergeThreads = 256, kLaDecodeThreads = 256;
constexpr int kLaMergeTiles = 16;

// A run of tokens of one sequence, advanced by one workgroup per head. `in` and
// `out` name the state it starts from and where its end state goes.
struct LaUnit {
    int32_t seq;
    int32_t tok0;   // first token within the sequence
    int32_t n_tok;  // tokens to run (may be 0)
    int32_t in;     // LA_ZERO, LA_INITIAL, or a slot (>= 0)
    int32_t out;    // LA_NONE, LA_FINAL, or a slot (>= 0)
};
enum : int32_t { LA_ZERO = -1, LA_INITIAL = -2 };
enum : int32_t { LA_NONE = -1, LA_FINAL = -2 };

// The segments 0 .. n - 1 of one sequence. Slot slot0 + s is to hold the state
// before segment s; before the merge, slot slot0 + s + 1 holds the end state of
// segment s from zero and that slot's decay the sum of g over segment s, times log2(e).
struct LaMerge {
    int32_t seq;
    int32_t n;
    int32_t slot0;
};

struct LaArgs {
    const uint16_t* q;   // [Tt][Hk][128] bf16
    const uint16_t* k;
    const uint16_t* v;   // [Tt][H][128] bf16
    const float* g;      // log-decay [Tt][H], or [H] when g_fixed
    const int32_t* cu;   // device cu_seqlens
    int64_t Tt;
    int32_t H, Hk, group;
    const LaUnit* units;
    int32_t n_units;
    const void* s0;      // may be null: zero initial states
    void* sT;            // may be null
    float* slots;        // [n_slots][H][128][128]
    float* decays;       // [n_slots][H], logarithms to base 2
    uint16_t* out;
    float scale;
    int32_t g_fixed, state_bf16;
};

struct LaMergeArgs {
    const LaMerge* items;
    int32_t n_items;
    int32_t H;
    const void* s0;
    int32_t state_bf16;
    float* slots;
    const float* decays;
};

struct LaDecodeArgs {
    const uint16_t* q;     // [n_seqs][T][Hk][128] bf16
    const uint16_t* k;
    const uint16_t* v;     // [n_seqs][T][H][128] bf16
    const float* g;        // [n_seqs][T][H], or [H] when g_fixed
    float* state;          // [n_slots][H][128][128], read and written
    uint16_t* out;
    int32_t n_seqs, T, H, Hk, group;
    float scale;
    const int32_t* slots;  // null: sequence n uses state[n]
    int32_t n_slots;
    int32_t g_fixed;
};

hipError_t launch_la_prefill(const LaArgs& a, bool with_out, hipStream_t s);
hipError_t launch_la_merge(const LaMergeArgs& a, hipStream_t s);
hipError_t launch_la_decode(const LaDecodeArgs& a, hipStream_t s);

}  // namespace kda
