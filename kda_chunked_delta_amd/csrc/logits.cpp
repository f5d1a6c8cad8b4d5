// Host side of the processing of logits: argument checks and dispatch of
// logits.hip behind the C ABI of include/kda.h.
#include "kda_internal.h"
#include "logits_launch.h"

using namespace kda;

namespace {

struct Buffer {
    const void* p;
    size_t n;
    size_t align;
    const char* name;
};

// Bytes from the first row's start to the last row's end.
size_t extent(int64_t rows, int64_t stride, int64_t n, size_t size) {
    return rows > 0 && n > 0 ? (size_t)((rows - 1) * stride + n) * size : 0;
}

}  // namespace

extern "C" {

kda_status kda_logits_process_validate(const kda_logits* x) {
    const char* const who = "kda_logits_process";
    if (!x) return fail(KDA_ERR_INVALID, "%s: the arguments are NULL", who);
    if (x->rows < 0 || x->vocab < 1)
        return fail(KDA_ERR_INVALID, "%s: rows must be >= 0 and vocab >= 1 (got %d, %d)", who, x->rows, x->vocab);
    if (x->dtype != KDA_FP32 && x->dtype != KDA_BF16 && x->dtype != KDA_FP16)
        return fail(KDA_ERR_INVALID, "%s: unknown dtype %d", who, (int)x->dtype);
    if (x->max_tokens < 0 || x->max_tokens >= 1 << 30)
        return fail(KDA_ERR_INVALID, "%s: max_tokens must be in [0, 2^30) (got %d)", who, x->max_tokens);
    if (x->n_bias < 0 || x->n_bias > kLogitsBiasMax)
        return fail(KDA_ERR_INVALID, "%s: n_bias must be in [0, %d] (got %d)", who, kLogitsBiasMax, x->n_bias);
    if (x->row_stride < x->vocab || x->out_stride < x->vocab)
        return fail(KDA_ERR_INVALID, "%s: row_stride and out_stride must be at least vocab (got %lld, %lld)", who,
                    (long long)x->row_stride, (long long)x->out_stride);
    const int64_t words = ((int64_t)x->vocab + 31) / 32;
    const struct { int64_t stride, n; const void* p; const char* name; } strides[] = {
        {x->token_stride, x->max_tokens, x->tokens, "token_stride"},
        {x->bias_stride, x->n_bias, x->n_bias ? x->bias : nullptr, "bias_stride"},
        {x->allowed_stride, words, x->allowed, "allowed_stride"}};
    for (const auto& s : strides)
        if (s.p && s.stride != 0 && s.stride < s.n)
            return fail(KDA_ERR_INVALID, "%s: %s must be 0 or at least a row's %lld entries (got %lld)", who, s.name,
                        (long long)s.n, (long long)s.stride);
    const int64_t most = (int64_t)1 << 40;
    if (x->row_stride > most || x->out_stride > most || x->token_stride > most || x->bias_stride > most ||
        x->allowed_stride > most)
        return fail(KDA_ERR_INVALID, "%s: strides must be at most 2^40", who);
    if (!x->tokens && x->max_tokens > 0) return fail(KDA_ERR_INVALID, "%s: tokens is NULL", who);
    const int64_t splits = ((int64_t)x->vocab + 2 * kLogitsSmallest - 1) / (2 * kLogitsSmallest);
    if (!launchable(x->rows * splits, kLogitsListThreads))
        return fail(KDA_ERR_INVALID, "%s: rows * vocab too large", who);
    if (x->rows == 0) return KDA_OK;
    // from the first row's start to the last one's end, 2^60 entries keep the bytes in 64 bits
    for (const int64_t stride : {x->row_stride, x->out_stride, x->tokens ? x->token_stride : 0,
                                 x->n_bias ? x->bias_stride : 0, x->allowed ? x->allowed_stride : 0})
        if ((x->rows - 1) * (stride >> 20) >= (int64_t)1 << 40)
            return fail(KDA_ERR_INVALID, "%s: rows * stride must be below 2^60 (got %d, %lld)", who, x->rows,
                        (long long)stride);
    const size_t size = x->dtype == KDA_FP32 ? 4 : 2, R = (size_t)x->rows;
    if (!x->logits || !x->out) return fail(KDA_ERR_INVALID, "%s: %s is NULL", who, x->logits ? "out" : "logits");
    if (x->n_bias && (!x->bias || !x->bias_tokens))
        return fail(KDA_ERR_INVALID, "%s: %s is NULL", who, x->bias ? "bias_tokens" : "bias");
    const Buffer out = {x->out, extent(x->rows, x->out_stride, x->vocab, size), size, "out"};
    const Buffer in = {x->logits, extent(x->rows, x->row_stride, x->vocab, size), size, "logits"};
    const Buffer ins[] = {
        in, {x->tokens, extent(x->rows, x->token_stride, x->max_tokens, 4), 4, "tokens"},
        {x->lengths, R * 4, 4, "lengths"}, {x->prompt_lengths, R * 4, 4, "prompt_lengths"},
        {x->repetition, R * 4, 4, "repetition"}, {x->frequency, R * 4, 4, "frequency"},
        {x->presence, R * 4, 4, "presence"},
        {x->n_bias ? x->bias_tokens : nullptr, extent(x->rows, x->bias_stride, x->n_bias, 4), 4, "bias_tokens"},
        {x->n_bias ? x->bias : nullptr, extent(x->rows, x->bias_stride, x->n_bias, 4), 4, "bias"},
        {x->allowed, extent(x->rows, x->allowed_stride, words, 4), 4, "allowed"}};
    if ((uintptr_t)out.p % size) return fail(KDA_ERR_INVALID, "%s: out is not %zu-byte aligned", who, size);
    for (const Buffer& b : ins) {
        if (b.p && (uintptr_t)b.p % b.align)
            return fail(KDA_ERR_INVALID, "%s: %s is not %zu-byte aligned", who, b.name, b.align);
        if (&b == ins && x->logits == x->out) {
            if (x->row_stride != x->out_stride && x->rows > 1)
                return fail(KDA_ERR_ALIAS, "%s: in place, out_stride has to be row_stride", who);
            continue;
        }
        if (overlap(out.p, out.n, b.p, b.n)) return fail(KDA_ERR_ALIAS, "%s: out overlaps %s", who, b.name);
    }
    return KDA_OK;
}

kda_status kda_logits_process(kda_ctx* ctx, const kda_logits* x, hipStream_t stream) {
    if (!ctx) return fail(KDA_ERR_INVALID, "kda_logits_process: ctx is NULL");
    const kda_status st = kda_logits_process_validate(x);
    if (st != KDA_OK || x->rows == 0) return st;
    LogitsArgs a{};
    a.x = *x;
    split_logits(&a);
    if (a.x.logits == a.x.out && !a.x.tokens && !a.x.n_bias && !a.x.allowed) return KDA_OK;  // nothing changes
    std::lock_guard<std::mutex> lk(ctx->mu);
    DeviceScope scope;
    hipError_t e = scope.enter(ctx->device);
    if (e != hipSuccess) return hip_fail(e, "kda_logits_process: selecting the device");
    e = timed_launch(ctx, stream, "logits_process", [&] { return launch_logits(a, stream); });
    return e == hipSuccess ? KDA_OK : hip_fail(e, "logits_process launch");
}

}  // extern "C"
