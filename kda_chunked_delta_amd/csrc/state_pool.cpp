// Host side of the state pool's pages and of beam search's selection: argument
// checks and dispatch behind the C ABI of include/kda.h.
#include <climits>

#include "kda_internal.h"
#include "state_pool_launch.h"

using namespace kda;

namespace {

struct Buffer {
    const void* p;
    size_t n;
    const char* name;
};

kda_status check_pool(const char* who, const kda_pool* p) {
    if (!p) return fail(KDA_ERR_INVALID, "%s: pool is NULL", who);
    if (p->n_layers < 1 || p->n_pages < 0)
        return fail(KDA_ERR_INVALID, "%s: the pool needs n_layers >= 1 and n_pages >= 0 (got %d, %d)", who,
                    p->n_layers, p->n_pages);
    if (p->page_bytes < 16 || p->page_bytes % 16 || p->page_bytes > ((int64_t)1 << 40))
        return fail(KDA_ERR_INVALID, "%s: page_bytes must be a multiple of 16, up to 2^40 (got %lld)", who,
                    (long long)p->page_bytes);
    if (p->n_layers > 1 && (p->layer_stride % 16 || p->layer_stride / p->page_bytes < p->n_pages))
        return fail(KDA_ERR_INVALID, "%s: layer_stride must be a multiple of 16 and hold n_pages pages (got %lld)",
                    who, (long long)p->layer_stride);
    if (p->n_pages > 0 && !p->base) return fail(KDA_ERR_INVALID, "%s: the pool's base is NULL", who);
    if ((uintptr_t)p->base % 16) return fail(KDA_ERR_INVALID, "%s: the pool's base is not 16-byte aligned", who);
    return KDA_OK;
}

size_t pool_extent(const kda_pool* p) {
    return (size_t)(p->n_layers - 1) * (size_t)p->layer_stride + (size_t)p->n_pages * (size_t)p->page_bytes;
}

PoolView view(const kda_pool* p) {
    return PoolView{(uint8_t*)p->base, p->n_layers > 1 ? p->layer_stride : 0, p->page_bytes, p->n_layers, p->n_pages};
}

// Needed, aligned to `align`, and apart from the pool (when given) and from each other.
kda_status check_buffers(const char* who, const kda_pool* pool, const Buffer* b, int n, size_t align) {
    for (int i = 0; i < n; ++i) {
        if (b[i].n == 0) continue;
        if (!b[i].p) return fail(KDA_ERR_INVALID, "%s: %s is NULL", who, b[i].name);
        if ((uintptr_t)b[i].p % align)
            return fail(KDA_ERR_INVALID, "%s: %s is not %zu-byte aligned", who, b[i].name, align);
        if (pool && overlap(pool->base, pool_extent(pool), b[i].p, b[i].n))
            return fail(KDA_ERR_ALIAS, "%s: the pool overlaps %s", who, b[i].name);
    }
    return KDA_OK;
}

// Runs `launch` with ctx's device current.
template <class F>
kda_status on_device(kda_ctx* ctx, hipStream_t stream, const char* who, F&& body) {
    std::lock_guard<std::mutex> lk(ctx->mu);
    DeviceScope scope;
    hipError_t e = scope.enter(ctx->device);
    if (e != hipSuccess) return hip_fail(e, who);
    e = body();
    return e == hipSuccess ? KDA_OK : hip_fail(e, who);
}

// Chunks of a row: 8192 elements per workgroup, or 2048 where that leaves the
// chip with fewer than two workgroups per compute unit, or where the room for
// a chunk's candidates (4 n per element and thread) would pass 32 KiB. Measured,
// both kernels, 8192 and 2048: 4 rows of 32000, 20 and 16 us; 128 rows, 18 and
// 18; 256 rows of 131072, 39 and 108. The rule looks at beam_rows alone: 8 to 24
// rows of 131072 get 64 chunks each, which beam_pick cannot stage (39 to 67 us).
void beam_split(int64_t rows, int64_t vocab, int32_t n, int32_t* chunk, int32_t* splits) {
    *chunk = n <= 32 && rows * ((vocab + 8191) / 8192) >= 512 ? 8192 : 2048;
    *splits = (int32_t)((vocab + *chunk - 1) / *chunk);
}

}  // namespace

extern "C" {

kda_status kda_pool_copy_validate(const kda_pool* pool, const int32_t* src, const int32_t* dst, int32_t n) {
    const char* const who = "kda_pool_copy";
    kda_status st = check_pool(who, pool);
    if (st != KDA_OK) return st;
    if (n < 0 || n > kPoolCopyMax)
        return fail(KDA_ERR_INVALID, "%s: n must be in [0, %d] (got %d)", who, kPoolCopyMax, n);
    if ((pool->page_bytes / 128 + 1) * pool->n_layers > INT32_MAX)
        return fail(KDA_ERR_INVALID, "%s: page_bytes * n_layers too large", who);
    const Buffer b[] = {{src, (size_t)n * 4, "src"}, {dst, (size_t)n * 4, "dst"}};
    return check_buffers(who, pool, b, 2, 4);
}

kda_status kda_pool_copy(kda_ctx* ctx, const kda_pool* pool, const int32_t* src, const int32_t* dst, int32_t n,
                         hipStream_t stream) {
    if (!ctx) return fail(KDA_ERR_INVALID, "kda_pool_copy: ctx is NULL");
    const kda_status st = kda_pool_copy_validate(pool, src, dst, n);
    if (st != KDA_OK || n == 0 || pool->n_pages == 0) return st;
    return on_device(ctx, stream, "kda_pool_copy", [&] {
        return timed_launch(ctx, stream, "pool_copy", [&] { return launch_pool_copy(view(pool), src, dst, n, stream); });
    });
}

kda_status kda_pool_fork_validate(const kda_pool* pool, const uint8_t* used, const int32_t* src, const int32_t* dst,
                                  int32_t n) {
    const char* const who = "kda_pool_fork";
    kda_status st = check_pool(who, pool);
    if (st != KDA_OK) return st;
    if (n < 0 || n > kPoolForkMax)
        return fail(KDA_ERR_INVALID, "%s: n must be in [0, %d] (got %d)", who, kPoolForkMax, n);
    const Buffer b[] = {{src, (size_t)n * 4, "src"}, {dst, (size_t)n * 4, "dst"}};
    const Buffer u[] = {{used, (size_t)pool->n_pages, "used"}};
    if ((st = check_buffers(who, pool, b, 2, 4)) != KDA_OK || (st = check_buffers(who, pool, u, 1, 1)) != KDA_OK)
        return st;
    if (overlap(dst, b[1].n, src, b[0].n) || overlap(dst, b[1].n, used, u[0].n) || overlap(src, b[0].n, used, u[0].n))
        return fail(KDA_ERR_ALIAS, "%s: used, src and dst overlap", who);
    return KDA_OK;
}

kda_status kda_pool_fork(kda_ctx* ctx, const kda_pool* pool, uint8_t* used, const int32_t* src, int32_t* dst,
                         int32_t n, hipStream_t stream) {
    if (!ctx) return fail(KDA_ERR_INVALID, "kda_pool_fork: ctx is NULL");
    const kda_status st = kda_pool_fork_validate(pool, used, src, dst, n);
    if (st != KDA_OK || n == 0) return st;
    return on_device(ctx, stream, "kda_pool_fork", [&] {
        hipError_t e = timed_launch(ctx, stream, "pool_fork_plan", [&] {
            return launch_pool_fork_plan(used, pool->n_pages, src, dst, n, stream);
        });
        if (e != hipSuccess) return e;
        return timed_launch(ctx, stream, "pool_move", [&] { return launch_pool_move(view(pool), src, dst, n, stream); });
    });
}

kda_status kda_pool_free_validate(int32_t n_pages, const uint8_t* used, const int32_t* pages, int32_t n) {
    const char* const who = "kda_pool_free";
    if (n_pages < 0 || n < 0)
        return fail(KDA_ERR_INVALID, "%s: n_pages and n must be >= 0 (got %d, %d)", who, n_pages, n);
    const Buffer b[] = {{pages, (size_t)n * 4, "pages"}}, u[] = {{used, (size_t)n_pages, "used"}};
    kda_status st = check_buffers(who, nullptr, b, 1, 4);
    if (st != KDA_OK || (st = check_buffers(who, nullptr, u, 1, 1)) != KDA_OK) return st;
    if (overlap(used, (size_t)n_pages, pages, (size_t)n * 4)) return fail(KDA_ERR_ALIAS, "%s: used overlaps pages", who);
    return KDA_OK;
}

kda_status kda_pool_free(kda_ctx* ctx, int32_t n_pages, uint8_t* used, const int32_t* pages, int32_t n,
                         hipStream_t stream) {
    if (!ctx) return fail(KDA_ERR_INVALID, "kda_pool_free: ctx is NULL");
    const kda_status st = kda_pool_free_validate(n_pages, used, pages, n);
    if (st != KDA_OK || n == 0) return st;
    return on_device(ctx, stream, "kda_pool_free", [&] {
        return timed_launch(ctx, stream, "pool_free", [&] { return launch_pool_free(used, n_pages, pages, n, stream); });
    });
}

kda_status kda_pool_compact_validate(const kda_pool* pool, const uint8_t* used, const int32_t* table, int32_t n_table,
                                     const int32_t* new_pages, const int32_t* n_live) {
    const char* const who = "kda_pool_compact";
    kda_status st = check_pool(who, pool);
    if (st != KDA_OK) return st;
    if (n_table < 0) return fail(KDA_ERR_INVALID, "%s: n_table must be >= 0 (got %d)", who, n_table);
    const Buffer b[] = {{table, (size_t)n_table * 4, "table"}, {new_pages, (size_t)pool->n_pages * 4, "new_pages"},
                        {n_live, 4, "n_live"}, {used, (size_t)pool->n_pages, "used"}};
    if ((st = check_buffers(who, pool, b, 3, 4)) != KDA_OK || (st = check_buffers(who, pool, b + 3, 1, 1)) != KDA_OK)
        return st;
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < i; ++j)
            if (overlap(b[i].p, b[i].n, b[j].p, b[j].n))
                return fail(KDA_ERR_ALIAS, "%s: %s overlaps %s", who, b[i].name, b[j].name);
    return KDA_OK;
}

kda_status kda_pool_compact(kda_ctx* ctx, const kda_pool* pool, uint8_t* used, int32_t* table, int32_t n_table,
                            int32_t* new_pages, int32_t* n_live, hipStream_t stream) {
    if (!ctx) return fail(KDA_ERR_INVALID, "kda_pool_compact: ctx is NULL");
    const kda_status st = kda_pool_compact_validate(pool, used, table, n_table, new_pages, n_live);
    if (st != KDA_OK) return st;
    return on_device(ctx, stream, "kda_pool_compact", [&] {
        hipError_t e = timed_launch(ctx, stream, "pool_compact_plan", [&] {
            return launch_pool_compact_plan(used, pool->n_pages, table, n_table, new_pages, n_live, stream);
        });
        if (e != hipSuccess) return e;
        return timed_launch(ctx, stream, "pool_move", [&] {
            return launch_pool_move(view(pool), nullptr, new_pages, pool->n_pages, stream);
        });
    });
}

kda_status kda_beam_reorder_validate(const kda_pool* pool, const int32_t* slots, const int32_t* parents,
                                     const int32_t* new_slots, int32_t batch, int32_t beams) {
    const char* const who = "kda_beam_reorder";
    kda_status st = check_pool(who, pool);
    if (st != KDA_OK) return st;
    if (batch < 0 || beams < 1 || beams > kBeamMax)
        return fail(KDA_ERR_INVALID, "%s: batch must be >= 0 and beams in [1, %d] (got %d, %d)", who, kBeamMax, batch,
                    beams);
    const int64_t items = (int64_t)batch * beams;
    const int64_t parts = (pool->page_bytes + kMovePart - 1) / kMovePart;  // up to 2^26
    if (items > INT32_MAX || !launchable(items * parts, kMoveThreads))
        return fail(KDA_ERR_INVALID, "%s: batch * beams * page_bytes too large", who);
    const size_t n = (size_t)items * 4;
    const Buffer b[] = {{slots, n, "slots"}, {parents, n, "parents"}, {new_slots, n, "new_slots"}};
    if ((st = check_buffers(who, pool, b, 3, 4)) != KDA_OK) return st;
    if (overlap(new_slots, n, slots, n) || overlap(new_slots, n, parents, n))
        return fail(KDA_ERR_ALIAS, "%s: new_slots overlaps slots or parents", who);
    return KDA_OK;
}

kda_status kda_beam_reorder(kda_ctx* ctx, const kda_pool* pool, const int32_t* slots, const int32_t* parents,
                            int32_t* new_slots, int32_t batch, int32_t beams, hipStream_t stream) {
    if (!ctx) return fail(KDA_ERR_INVALID, "kda_beam_reorder: ctx is NULL");
    const kda_status st = kda_beam_reorder_validate(pool, slots, parents, new_slots, batch, beams);
    if (st != KDA_OK || batch == 0) return st;
    return on_device(ctx, stream, "kda_beam_reorder", [&] {
        return timed_launch(ctx, stream, "beam_reorder", [&] {
            return launch_beam_reorder(view(pool), slots, parents, new_slots, batch, beams, stream);
        });
    });
}

size_t kda_beam_select_workspace_bytes(int32_t batch, int32_t beams, int32_t vocab, int32_t n) {
    if (batch < 1 || beams < 1 || vocab < 1 || n < 1) return 0;
    int32_t chunk, splits;
    beam_split((int64_t)batch * beams, vocab, n, &chunk, &splits);
    return (size_t)batch * beams * splits * ((size_t)n * 8 + 8 + 4);
}

kda_status kda_beam_select_validate(int32_t batch, int32_t beams, int32_t vocab, int32_t n, const void* logits,
                                    kda_dtype dtype, int64_t row_stride, const float* scores, const uint8_t* finished,
                                    int32_t eos, const float* out_scores, const int32_t* out_parents,
                                    const int32_t* out_tokens, const uint8_t* out_finished, const void* workspace,
                                    size_t workspace_bytes) {
    const char* const who = "kda_beam_select";
    if (batch < 0 || beams < 1 || beams > kBeamMax || vocab < 1)
        return fail(KDA_ERR_INVALID, "%s: batch must be >= 0, beams in [1, %d] and vocab >= 1 (got %d, %d, %d)", who,
                    kBeamMax, batch, beams, vocab);
    if (n < 1 || n > kBeamPickMax || (int64_t)beams * vocab < n)
        return fail(KDA_ERR_INVALID, "%s: n must be in [1, %d] and at most beams * vocab (got %d)", who, kBeamPickMax,
                    n);
    if (dtype != KDA_FP32 && dtype != KDA_BF16 && dtype != KDA_FP16)
        return fail(KDA_ERR_INVALID, "%s: unknown dtype %d", who, (int)dtype);
    if ((int64_t)beams * vocab > INT32_MAX)
        return fail(KDA_ERR_INVALID, "%s: beams * vocab too large (%lld)", who, (long long)beams * vocab);
    if (row_stride < vocab)
        return fail(KDA_ERR_INVALID, "%s: row_stride must be at least vocab (got %lld)", who, (long long)row_stride);
    if (finished && (eos < 0 || eos >= vocab))
        return fail(KDA_ERR_INVALID, "%s: finished beams need eos in [0, vocab) (got %d)", who, eos);
    if (eos >= vocab) return fail(KDA_ERR_INVALID, "%s: eos must be below vocab (got %d)", who, eos);
    if ((eos >= 0) != (out_finished != nullptr) && batch > 0)
        return fail(KDA_ERR_INVALID, "%s: out_finished goes with eos >= 0", who);
    if (batch == 0) return KDA_OK;
    const int64_t rows = (int64_t)batch * beams;
    int32_t chunk, splits;
    beam_split(rows, vocab, n, &chunk, &splits);
    if (!launchable(rows * splits, kBeamThreads) || (int64_t)beams * splits > 24 * 1024)
        return fail(KDA_ERR_INVALID, "%s: batch * beams * vocab too large", who);
    const size_t size = dtype == KDA_FP32 ? 4 : 2, R = (size_t)rows, K = (size_t)batch * n;
    const Buffer b[] = {{out_scores, K * 4, "out_scores"}, {out_parents, K * 4, "out_parents"},
                        {out_tokens, K * 4, "out_tokens"}, {scores, R * 4, "scores"}};
    const Buffer c[] = {{out_finished, out_finished ? K : 0, "out_finished"}, {finished, finished ? R : 0, "finished"}};
    const Buffer l[] = {{logits, ((R - 1) * (size_t)row_stride + vocab) * size, "logits"}};
    const size_t need = kda_beam_select_workspace_bytes(batch, beams, vocab, n);
    const Buffer ws[] = {{workspace, need, "workspace"}};
    kda_status st;
    if ((st = check_buffers(who, nullptr, b, 4, 4)) != KDA_OK || (st = check_buffers(who, nullptr, c, 2, 1)) != KDA_OK ||
        (st = check_buffers(who, nullptr, l, 1, size)) != KDA_OK || (st = check_buffers(who, nullptr, ws, 1, 16)) != KDA_OK)
        return st;
    if (workspace_bytes < need)
        return fail(KDA_ERR_INVALID, "%s: needs a workspace of %zu bytes (got %zu)", who, need, workspace_bytes);
    const Buffer outs[] = {b[0], b[1], b[2], c[0], ws[0]}, ins[] = {b[3], c[1], l[0]};
    for (int i = 0; i < 5; ++i) {
        for (const Buffer& x : ins)
            if (overlap(outs[i].p, outs[i].n, x.p, x.n))
                return fail(KDA_ERR_ALIAS, "%s: %s overlaps %s", who, outs[i].name, x.name);
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n))
                return fail(KDA_ERR_ALIAS, "%s: %s overlaps %s", who, outs[i].name, outs[j].name);
    }
    return KDA_OK;
}

kda_status kda_beam_select(kda_ctx* ctx, int32_t batch, int32_t beams, int32_t vocab, int32_t n, const void* logits,
                           kda_dtype dtype, int64_t row_stride, const float* scores, const uint8_t* finished,
                           int32_t eos, float* out_scores, int32_t* out_parents, int32_t* out_tokens,
                           uint8_t* out_finished, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    if (!ctx) return fail(KDA_ERR_INVALID, "kda_beam_select: ctx is NULL");
    const kda_status st = kda_beam_select_validate(batch, beams, vocab, n, logits, dtype, row_stride, scores, finished,
                                                   eos, out_scores, out_parents, out_tokens, out_finished, workspace,
                                                   workspace_bytes);
    if (st != KDA_OK || batch == 0) return st;
    BeamArgs a{logits, row_stride, scores, finished, eos, batch, beams, vocab, n};
    beam_split((int64_t)batch * beams, vocab, n, &a.chunk, &a.splits);
    const size_t lists = (size_t)batch * beams * a.splits;
    a.keys = (uint64_t*)workspace;
    a.sums = (double*)(a.keys + lists * n);
    a.maxima = (float*)(a.sums + lists);
    a.out_scores = out_scores;
    a.out_parents = out_parents;
    a.out_tokens = out_tokens;
    a.out_finished = out_finished;
    return on_device(ctx, stream, "kda_beam_select", [&] {
        hipError_t e = timed_launch(ctx, stream, "beam_rows", [&] { return launch_beam_rows(a, dtype, stream); });
        if (e != hipSuccess) return e;
        return timed_launch(ctx, stream, "beam_pick", [&] { return launch_beam_pick(a, stream); });
    });
}

}  // extern "C"
