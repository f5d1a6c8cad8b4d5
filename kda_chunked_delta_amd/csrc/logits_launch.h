// Internal interface between the host code and the kernel of the processing of
// logits (logits.hip). Not part of the public C ABI.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "kda.h"

namespace kda {

// Threads of a workgroup, without and with a history or biases.
constexpr int kLogitsThreads = 256, kLogitsListThreads = 512;
constexpr int kLogitsBiasMax = 8192;   // of a row: fewer than 2^14, and than 64 per thread
constexpr int kLogitsShort = 1 << 14;  // histories below this are counted in 16 bits

struct LogitsArgs {
    kda_logits x;    // as the caller gave them, checked
    int32_t chunk;   // logits of a row per workgroup, a multiple of 32
    int32_t splits;  // chunks per row
    int32_t lists;   // 0: no history and biases, 1: words of 16 bits, 2: of 32
    int32_t threads;
    int32_t lds;     // bytes
};

// What a workgroup takes of a row: 8192 logits, or 2048 where that leaves the 256
// compute units with fewer than two workgroups each. With lists, which every
// workgroup of a row goes through, 16384 or 4096. 8192 in place of 16384 with
// words of 32 bits (64 KiB of LDS otherwise), and for a history of more than 4096
// tokens, whose list takes the LDS of a third workgroup per compute unit (41 KiB each
// with 4096 tokens, 49 with 8192, of 160): 256 rows of 131072 took 37 us with histories of
// 4096 tokens, 39 with 8192 logits; with histories of 8192 tokens (fp32) 92, and 82.
constexpr int32_t kLogitsSmallest = 2048;
inline void split_logits(LogitsArgs* a) {
    kda_logits& x = a->x;
    // a history that no penalty asks for is not looked at, and takes no room
    if (!x.tokens || !(x.repetition || x.frequency || x.presence)) x.max_tokens = 0;
    if (x.max_tokens == 0) x.tokens = nullptr;
    a->lists = !x.tokens && !x.n_bias ? 0 : x.max_tokens < kLogitsShort ? 1 : 2;
    a->threads = a->lists ? kLogitsListThreads : kLogitsThreads;
    const int32_t large = a->lists == 1 && x.max_tokens <= 4096 ? 16384 : 8192;
    const int32_t small = a->lists ? 2 * kLogitsSmallest : kLogitsSmallest;
    a->chunk = (int64_t)x.rows * ((x.vocab - 1) / large + 1) >= 512 ? large : small;
    a->splits = (x.vocab - 1) / a->chunk + 1;
    const int32_t listed = std::min(a->chunk, x.max_tokens);
    a->lds = a->chunk * (a->lists == 1 ? 2 : 4) + (listed * 2 + 15) / 16 * 16;
}

hipError_t launch_logits(const LogitsArgs& a, hipStream_t s);

}  // namespace kda
