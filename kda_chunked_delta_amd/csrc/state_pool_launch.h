// Internal interface between the host code (state_pool.cpp) and the kernels
// of the state pool's pages (state_pool.hip) and of beam search's selection
// (beam_select.hip). Not part of the public C ABI.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

struct PoolView {
    uint8_t* base;
    int64_t layer_stride;  // bytes from a page of one layer to the same page of the next
    int64_t page_bytes;    // a multiple of 16
    int32_t n_layers, n_pages;
};

constexpr int kPoolCopyMax = 1024;   // pairs of one pool copy
constexpr int kPoolForkMax = 8192;   // requests of one fork
constexpr int kMoveThreads = 256;    // threads of a workgroup that moves part of a page
constexpr int kMovePart = kMoveThreads * 64;  // bytes of that part
constexpr int kBeamThreads = 256;    // threads of a workgroup of the selection
constexpr int kBeamMax = 64;         // beams of one batch entry
constexpr int kBeamPickMax = 64;     // candidates selected per batch entry

// Page src[i] (page i when src is null) to page dst[i], i < n; pairs with an
// index outside the pool or src == dst are skipped, no destination may be a
// source.
hipError_t launch_pool_move(const PoolView& p, const int32_t* src, const int32_t* dst, int32_t n, hipStream_t s);
hipError_t launch_pool_copy(const PoolView& p, const int32_t* src, const int32_t* dst, int32_t n, hipStream_t s);
hipError_t launch_pool_fork_plan(uint8_t* used, int32_t n_pages, const int32_t* src, int32_t* dst, int32_t n,
                                 hipStream_t s);
hipError_t launch_pool_free(uint8_t* used, int32_t n_pages, const int32_t* pages, int32_t n, hipStream_t s);
hipError_t launch_pool_compact_plan(uint8_t* used, int32_t n_pages, int32_t* table, int32_t n_table, int32_t* newpos,
                                    int32_t* n_live, hipStream_t s);
hipError_t launch_beam_reorder(const PoolView& p, const int32_t* slots, const int32_t* parents, int32_t* new_slots,
                               int32_t batch, int32_t beams, hipStream_t s);

struct BeamArgs {
    const void* logits;
    int64_t row_stride;  // elements
    const float* scores;
    const uint8_t* finished;  // may be null
    int32_t eos;              // < 0: none
    int32_t batch, beams, vocab, n;
    int32_t splits, chunk;    // chunks of a row, elements of a chunk
    uint64_t* keys;           // [batch * beams][splits][n]
    double* sums;             // [batch * beams][splits]
    float* maxima;            // [batch * beams][splits]
    float* out_scores;
    int32_t* out_parents;
    int32_t* out_tokens;
    uint8_t* out_finished;    // null without eos
};

// dtype: a kda_dtype value
hipError_t launch_beam_rows(const BeamArgs& a, int dtype, hipStream_t s);
hipError_t launch_beam_pick(const BeamArgs& a, hipStream_t s);

}  // namespace kda
