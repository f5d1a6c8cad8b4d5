// Internal interface between the host code and the kernel of the processing of
// logits (logits.hip). Not part of the public C ABI.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

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

hipError_t launch_logits(const LogitsArgs& a, hipStream_t s);

}  // namespace kda
