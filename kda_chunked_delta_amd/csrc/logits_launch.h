// Internal interface between the host code and the kernel of the processing of
// logits (logits.hip). Not part of the public C ABI.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kda.h"

namespace kda {

constexpr int kLogitsThreads = 256;

struct LogitsArgs {
    kda_logits x;    // as the caller gave them, checked
    int32_t chunk;   // logits of a row per workgroup
    int32_t splits;  // chunks per row
};

hipError_t launch_logits(const LogitsArgs& a, hipStream_t s);

}  // namespace kda
