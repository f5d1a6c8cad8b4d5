// Internals shared by the host sources: error reporting, the plan, the
// context with its per-stream workspace arenas, and timed launches. Not part
// of the public C ABI.
#pragma once
#include <hip/hip_runtime.h>

#include <mutex>
#include <unordered_map>
#include <vector>

#include "gated_delta_launch.h"
#include "kda.h"
#include "kda_launch.h"
#include "linear_attention_launch.h"

namespace kda {

// Records the calling thread's error message and returns st.
kda_status fail(kda_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
kda_status hip_fail(hipError_t e, const char* what);
// Whether [a, a + na) and [b, b + nb) share a byte (NULL or empty: never).
bool overlap(const void* a, size_t na, const void* b, size_t nb);
inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
// Whether a grid of this many workgroups can be launched: HIP takes fewer than 2^32 threads.
inline bool launchable(int64_t workgroups, int threads) { return workgroups <= (int64_t)UINT32_MAX / threads; }

// Makes a device current for a scope.
struct DeviceScope {
    int prev = -1, cur = -1;
    hipError_t enter(int device) {
        hipError_t e = hipGetDevice(&prev);
        if (e != hipSuccess) return e;
        cur = device;
        return prev == device ? hipSuccess : hipSetDevice(device);
    }
    ~DeviceScope() { if (cur >= 0 && prev >= 0 && prev != cur) (void)hipSetDevice(prev); }
};

}  // namespace kda

// ---------------------------------------------------------------------------
// plan
// ---------------------------------------------------------------------------
struct kda_plan {
    kda_plan_info info{};
    std::vector<int32_t> cu;            // host copy of cu_seqlens
    std::vector<kda::ChunkDesc> chunks;     // K1 items (global chunk order)
    std::vector<kda::UnitDesc> units;        // K2 units, launch order
    std::vector<kda::MergeDesc> merges;      // CP merge items
    std::vector<kda::UnitDesc> fixups;       // warm-start segments, as rerun from their carry
    std::vector<kda::UnitDesc> cp_units;     // warm-start CP: the segmented fallback's K2 units
    std::vector<kda::UnitDesc> alt_units;    // split plans: the batch unsplit (the exact path)
    std::vector<kda::UnitDesc> k1_units;     // segmented pipeline: K1 with the B summaries, one per K2 unit
    std::vector<kda::MergeSeg> merge_segs;   // segmented pipeline: one merge workgroup row per segment
    // Gated delta rule plans (kda_plan_gated_delta) have these tables instead;
    // their units above are for inspection only. off_b holds the summaries.
    bool gated = false;
    std::vector<kda::GdUnit> gd_units;  // main launch
    std::vector<kda::GdUnit> gd_pre;    // segments' end states and transfers
    std::vector<kda::GdMerge> gd_merges;
    // Linear attention plans (kda_plan_linear_attention) have these. off_carry
    // holds the slots' states, off_b their decays.
    bool linear = false;
    std::vector<kda::LaUnit> la_units;  // main launch
    std::vector<kda::LaUnit> la_pre;    // segments' end states
    std::vector<kda::LaMerge> la_merges;
    // workspace layout (byte offsets into the arena)
    size_t off_rec = 0, off_b = 0, off_m = 0, off_mlive = 0, off_carry = 0;
    size_t off_spec_states = 0, off_spec_flags = 0, off_gate = 0;
    // device copy of the tables
    int device = -1;
    void* dev_tables = nullptr;
    size_t dev_off_chunks = 0, dev_off_units = 0, dev_off_merges = 0, dev_off_fixups = 0;
    size_t dev_off_cp_units = 0, dev_off_alt_units = 0, dev_off_k1_units = 0, dev_off_merge_segs = 0;
    // Speculation feedback, outside graph capture: a speculative call (the
    // first, then every 64th) copies its outcome (split plans: the speculation
    // flags; warm-start CP: the gate) into pinned host memory and records an
    // event; a later call
    // that finds the copy complete and a failure in it turns speculation off
    // for this plan, which then runs its exact path (unsplit serial, or the
    // segmented pipeline ungated). Results are the same bits either way.
    mutable std::mutex spec_mu;
    mutable int32_t* spec_host = nullptr;
    mutable size_t spec_words = 0;
    mutable hipEvent_t spec_event = nullptr;
    mutable bool spec_pending = false;
    mutable bool spec_off = false;
    mutable uint64_t spec_calls = 0;  // the outcome is copied on the first call and every 64th
};

// ---------------------------------------------------------------------------
// context and arena
// ---------------------------------------------------------------------------
struct Arena {
    void* ptr = nullptr;
    size_t bytes = 0;
    // A call captured into a graph bakes this address into the graph, which
    // may be replayed at any time after: such memory is never freed before
    // kda_destroy (growing or evicting the arena retires it instead).
    bool captured = false;
};

struct TimedLaunch {
    const char* name;
    hipEvent_t beg, end;
};

struct kda_ctx {
    int device = 0;
    int n_cus = 0;
    hipDeviceProp_t prop{};
    std::mutex mu;
    std::unordered_map<hipStream_t, Arena> arenas;
    std::vector<void*> retired;  // arena memory that served a graph capture, freed in kda_destroy
    void* scratch = nullptr;     // this device's copy of the static scratch (kda_prefill_noalloc)
    bool poison = false;
    bool timing = false;
    std::vector<TimedLaunch> events;  // pool, reused across calls
    int n_timed = 0;
};

static const size_t kMaxArenas = 16;
static const int kMaxTimedLaunches = 4096;

// Run `launch` on `stream`; while the context's timing is on, bracket it with
// a pair of HIP events from the context's pool (ctx->mu held by the caller).
template <class F>
static hipError_t timed_launch(kda_ctx* ctx, hipStream_t stream, const char* name, F&& launch) {
    if (!ctx->timing) return launch();
    if (ctx->n_timed >= kMaxTimedLaunches) return launch();  // log full: run untimed
    if ((int)ctx->events.size() <= ctx->n_timed) {
        TimedLaunch t{name, nullptr, nullptr};
        hipError_t ee = hipEventCreate(&t.beg);
        if (ee == hipSuccess) ee = hipEventCreate(&t.end);
        if (ee != hipSuccess) return ee;
        ctx->events.push_back(t);
    }
    TimedLaunch& t = ctx->events[ctx->n_timed++];
    t.name = name;
    hipError_t ee = hipEventRecord(t.beg, stream);
    if (ee == hipSuccess) ee = launch();
    if (ee == hipSuccess) ee = hipEventRecord(t.end, stream);
    return ee;
}
