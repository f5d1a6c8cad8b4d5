// Host side of linear attention: plans, argument checks and dispatch of
// linear_attention.hip behind the C ABI of include/kda.h.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>
#include <memory>
#include <new>

#include "kda_internal.h"

using namespace kda;

namespace {

constexpr int32_t kMaxHeads = 1 << 17;  // 32 token rows of one tensor stay below 2^31 bytes

// Cost model of a plan, microseconds on MI355X, fitted to launches of 8 to 1024
// units: what a chunk of a unit takes at least, with output and without, and at
// what rate the whole chip (256 compute units) moves the bytes of a chunk (32 KiB
// with output, 16 without); a launch beside its chunks; a segment's step of the merge.
constexpr double kFullUs = 1.13, kPreUs = 0.82, kBytesPerUs = 5.0e6, kLaunchUs = 6.0, kMergeUs = 0.1;

// A launch of units, H heads each: bound by the chain of the longest one, by
// the workgroups that share a compute unit, or by memory.
double launch_us(int64_t units, int64_t chunks, int longest, int H, int n_cus, double per_chunk, double bytes) {
    if (units == 0) return 0;
    const double n = (double)units * H, total = (double)chunks * H;
    const double chain = n <= n_cus ? longest : std::max((double)longest, total / n_cus + 0.9 * longest);
    return kLaunchUs + std::max(chain * per_chunk, total * bytes / kBytesPerUs);
}

int segments_of(int chunks, int seg) { return seg > 0 && chunks > seg ? (chunks + seg - 1) / seg : 1; }

double plan_us(const std::vector<int>& nch, int H, int n_cus, int seg) {
    int64_t units = 0, chunks = 0, pre_units = 0, pre_chunks = 0;
    int longest = 0, pre_longest = 0, most = 1;
    for (int c : nch) {
        const int n = segments_of(c, seg), len = (c + n - 1) / n;
        most = std::max(most, n);
        units += n;
        chunks += c;
        longest = std::max(longest, len);
        if (n > 1) {
            pre_units += n - 1;
            pre_chunks += (int64_t)c * (n - 1) / n;
            pre_longest = std::max(pre_longest, len);
        }
    }
    double us = launch_us(units, chunks, longest, H, n_cus, kFullUs, 32768);
    if (most > 1)
        us += launch_us(pre_units, pre_chunks, pre_longest, H, n_cus, kPreUs, 16384) + kLaunchUs + most * kMergeUs;
    return us;
}

kda_status build(int32_t n_cus, const int32_t* cu, int32_t n_seqs, int32_t H, int32_t dk, int32_t dv,
                 kda_cp_mode mode, int32_t seg_chunks, kda_plan** out) {
    const char* const who = "kda_plan_linear_attention";
    if (!out) return fail(KDA_ERR_INVALID, "%s: out is NULL", who);
    *out = nullptr;
    if (dk != 128 || dv != 128)
        return fail(KDA_ERR_UNSUPPORTED, "%s: dk = dv = 128 required (got dk=%d dv=%d)", who, dk, dv);
    if (H < 1 || H > kMaxHeads) return fail(KDA_ERR_INVALID, "%s: H must be in [1, %d] (got %d)", who, kMaxHeads, H);
    if (n_seqs < 1) return fail(KDA_ERR_INVALID, "%s: n_seqs must be >= 1 (got %d)", who, n_seqs);
    if (!cu) return fail(KDA_ERR_INVALID, "%s: cu_seqlens_host is NULL", who);
    if (n_cus < 1) return fail(KDA_ERR_INVALID, "%s: n_cus must be >= 1 (got %d)", who, n_cus);
    if (mode != KDA_CP_OFF && mode != KDA_CP_ON && mode != KDA_CP_AUTO)
        return fail(KDA_ERR_INVALID, "%s: unknown cp mode %d", who, (int)mode);
    if (seg_chunks < 0) return fail(KDA_ERR_INVALID, "%s: seg_chunks must be >= 0 (got %d)", who, seg_chunks);
    if (cu[0] != 0) return fail(KDA_ERR_INVALID, "%s: cu_seqlens[0] must be 0 (got %d)", who, cu[0]);
    for (int i = 0; i < n_seqs; ++i)
        if (cu[i + 1] < cu[i])
            return fail(KDA_ERR_INVALID, "%s: cu_seqlens decreases at index %d (%d -> %d)", who, i, cu[i], cu[i + 1]);

    std::vector<int> nch(n_seqs);
    int64_t total = 0;
    int longest = 0;
    for (int i = 0; i < n_seqs; ++i) {
        nch[i] = (int)(((int64_t)cu[i + 1] - cu[i] + kLaChunk - 1) / kLaChunk);
        total += nch[i];
        longest = std::max(longest, nch[i]);
    }
    // segment length: given, or the cheapest that cuts the longest sequence into
    // 2, 3, .. 64, 66, .. parts of at least four chunks
    const double t_serial = plan_us(nch, H, n_cus, 0);
    double t_cp = -1;
    int seg = 0;
    if (mode != KDA_CP_OFF) {
        if (seg_chunks > 0) {
            seg = seg_chunks;
            t_cp = plan_us(nch, H, n_cus, seg);
        } else {
            for (int n = 2; n <= longest / 4; n += std::max(1, n / 32)) {
                const int c = (longest + n - 1) / n;
                const double t = plan_us(nch, H, n_cus, c);
                if (t_cp < 0 || t < t_cp) {
                    t_cp = t;
                    seg = c;
                }
            }
            if (mode == KDA_CP_AUTO && 0.95 * t_serial <= t_cp) seg = 0;
        }
    }
    auto p = std::make_unique<kda_plan>();
    p->linear = true;
    p->cu.assign(cu, cu + n_seqs + 1);
    int n_slots = 0, n_cp = 0;
    for (int i = 0; i < n_seqs; ++i) {
        const int n = segments_of(nch[i], seg);
        const int64_t L = (int64_t)cu[i + 1] - cu[i];
        if (n > 1) {
            p->la_merges.push_back(LaMerge{i, n, n_slots});
            ++n_cp;
        }
        for (int s = 0; s < n; ++s) {
            const int c0 = (int)((int64_t)nch[i] * s / n), c1 = (int)((int64_t)nch[i] * (s + 1) / n);
            const int64_t t0 = (int64_t)c0 * kLaChunk, t1 = std::min((int64_t)c1 * kLaChunk, L);
            p->la_units.push_back(LaUnit{i, (int32_t)t0, (int32_t)(t1 - t0), n > 1 ? n_slots + s : LA_INITIAL,
                                         s + 1 == n ? LA_FINAL : LA_NONE});
            if (s + 1 < n)
                p->la_pre.push_back(LaUnit{i, (int32_t)t0, (int32_t)(t1 - t0), LA_ZERO, n_slots + s + 1});
            UnitDesc u{};
            u.seq = i;
            u.chunk0 = c0;
            u.n_chunks = c1 - c0;
            u.segment = s;
            u.n_segments = n;
            p->units.push_back(u);
        }
        if (n > 1) n_slots += n;
    }
    // longest first, so that the last workgroups to start are short
    auto longer = [](const LaUnit& a, const LaUnit& b) { return a.n_tok > b.n_tok; };
    std::stable_sort(p->la_units.begin(), p->la_units.end(), longer);
    std::stable_sort(p->la_pre.begin(), p->la_pre.end(), longer);
    std::stable_sort(p->units.begin(), p->units.end(),
                     [](const UnitDesc& a, const UnitDesc& b) { return a.n_chunks > b.n_chunks; });
    if (!launchable((int64_t)p->la_units.size() * H, kLaThreads) ||
        !launchable((int64_t)p->la_merges.size() * H * kLaMergeTiles, kLaMergeThreads))
        return fail(KDA_ERR_INVALID, "%s: too many work units (%zu units, %d heads)", who, p->la_units.size(), H);
    p->off_carry = 0;
    p->off_b = (size_t)n_slots * H * kStateBytes;  // the slots' decays
    kda_plan_info& in = p->info;
    in.n_seqs = n_seqs;
    in.H = H;
    in.dk = dk;
    in.dv = dv;
    in.total_tokens = cu[n_seqs];
    in.total_chunks = (int32_t)total;
    in.uses_cp = n_cp > 0;
    in.n_units = (int32_t)p->la_units.size();
    in.n_cp_seqs = n_cp;
    in.n_prescan = (int32_t)p->la_pre.size();
    in.n_carry_slots = n_slots;
    in.max_unit_chunks = p->units[0].n_chunks;
    in.n_cus = n_cus;
    in.workspace_bytes = align_up(p->off_b + (size_t)n_slots * H * 4, 16);
    in.est_serial_us = t_serial;
    in.est_cp_us = t_cp;
    in.est_split_us = in.est_warm_cp_us = -1.0;
    *out = p.release();
    return KDA_OK;
}

kda_status upload(kda_plan* p, int device) {
    const size_t n_units = p->la_units.size() * sizeof(LaUnit), n_pre = p->la_pre.size() * sizeof(LaUnit);
    const size_t n_merge = p->la_merges.size() * sizeof(LaMerge);
    p->dev_off_units = 0;
    p->dev_off_k1_units = align_up(n_units, 256);
    p->dev_off_merges = align_up(p->dev_off_k1_units + n_pre, 256);
    std::vector<uint8_t> host(p->dev_off_merges + n_merge, 0);
    memcpy(&host[0], p->la_units.data(), n_units);
    if (n_pre) memcpy(&host[p->dev_off_k1_units], p->la_pre.data(), n_pre);
    if (n_merge) memcpy(&host[p->dev_off_merges], p->la_merges.data(), n_merge);
    DeviceScope scope;
    hipError_t e = scope.enter(device);
    if (e != hipSuccess) return hip_fail(e, "kda_plan_linear_attention: selecting the device");
    void* d = nullptr;
    e = hipMalloc(&d, host.size());
    if (e == hipSuccess) e = hipMemcpy(d, host.data(), host.size(), hipMemcpyHostToDevice);
    if (e != hipSuccess) {
        if (d) (void)hipFree(d);
        return hip_fail(e, "kda_plan_linear_attention: uploading plan tables");
    }
    p->dev_tables = d;
    p->device = device;
    return KDA_OK;
}

struct Buffer {
    const void* p;
    size_t n;
    const char* name;
};

}  // namespace

extern "C" {

kda_status kda_plan_linear_attention_host(int32_t n_cus, const int32_t* cu_seqlens_host, int32_t n_seqs, int32_t H,
                                          int32_t dk, int32_t dv, kda_cp_mode mode, int32_t seg_chunks,
                                          kda_plan** out) {
    try {
        return build(n_cus, cu_seqlens_host, n_seqs, H, dk, dv, mode, seg_chunks, out);
    } catch (const std::bad_alloc&) {
        return fail(KDA_ERR_INVALID, "kda_plan_linear_attention: out of host memory");
    }
}

kda_status kda_plan_linear_attention(kda_ctx* ctx, const int32_t* cu_seqlens_host, int32_t n_seqs, int32_t H,
                                     int32_t dk, int32_t dv, kda_cp_mode mode, int32_t seg_chunks, kda_plan** out) {
    if (!ctx) return fail(KDA_ERR_INVALID, "kda_plan_linear_attention: ctx is NULL");
    try {
        kda_status st = build(ctx->n_cus, cu_seqlens_host, n_seqs, H, dk, dv, mode, seg_chunks, out);
        if (st != KDA_OK) return st;
        std::unique_ptr<kda_plan> p(*out);
        *out = nullptr;
        st = upload(p.get(), ctx->device);
        if (st == KDA_OK) *out = p.release();
        return st;
    } catch (const std::bad_alloc&) {
        return fail(KDA_ERR_INVALID, "kda_plan_linear_attention: out of host memory");
    }
}

kda_status kda_linear_attention_prefill_validate(const kda_plan* p, const kda_linear_opts* opts, const void* q,
                                                 const void* k, const void* v, const float* g, const int32_t* cu_dev,
                                                 float scale, const void* s0, const void* sT, const void* out,
                                                 const void* workspace, size_t workspace_bytes) {
    const char* const who = "kda_linear_attention_prefill";
    if (!p) return fail(KDA_ERR_INVALID, "%s: plan is NULL", who);
    if (!p->linear) return fail(KDA_ERR_INVALID, "%s: the plan is not one of kda_plan_linear_attention", who);
    const kda_plan_info& in = p->info;
    if (opts && opts->qk_heads < 0)
        return fail(KDA_ERR_INVALID, "%s: qk_heads must be >= 0 (got %d)", who, opts->qk_heads);
    const int32_t qk_heads = opts && opts->qk_heads > 0 ? opts->qk_heads : in.H;
    const bool state16 = opts && opts->state_bf16, fixed = opts && opts->g_fixed;
    if (in.H % qk_heads != 0)
        return fail(KDA_ERR_INVALID, "%s: the plan's %d value heads are not a multiple of %d q/k heads", who, in.H,
                    qk_heads);
    if (!std::isfinite(scale)) return fail(KDA_ERR_INVALID, "%s: scale is not finite", who);
    if (!cu_dev) return fail(KDA_ERR_INVALID, "%s: cu_seqlens is NULL", who);
    if ((uintptr_t)cu_dev % 4) return fail(KDA_ERR_INVALID, "%s: cu_seqlens is not 4-byte aligned", who);
    const size_t Tt = (size_t)in.total_tokens, H = (size_t)in.H, N = (size_t)in.n_seqs;
    const size_t n_qk = Tt * (size_t)qk_heads * 256, n_act = Tt * H * 256;
    const size_t n_state = N * H * 128 * 128 * (state16 ? 2 : 4);
    const Buffer ins[] = {{q, n_qk, "q"}, {k, n_qk, "k"}, {v, n_act, "v"}, {g, (fixed ? H : Tt * H) * 4, "g"},
                          {cu_dev, (N + 1) * 4, "cu_seqlens"}, {s0, n_state, "initial_state"}};
    const Buffer outs[] = {{out, n_act, "out"}, {sT, n_state, "final_state"},
                           {workspace, in.workspace_bytes, "workspace"}};
    if (Tt > 0) {
        const size_t align[] = {16, 16, 16, 4};
        for (int i = 0; i < 4; ++i) {
            if (!ins[i].p) return fail(KDA_ERR_INVALID, "%s: %s is NULL", who, ins[i].name);
            if ((uintptr_t)ins[i].p % align[i])
                return fail(KDA_ERR_INVALID, "%s: %s is not %zu-byte aligned", who, ins[i].name, align[i]);
        }
        if (!out) return fail(KDA_ERR_INVALID, "%s: out is NULL", who);
        if ((uintptr_t)out % 16) return fail(KDA_ERR_INVALID, "%s: out is not 16-byte aligned", who);
    }
    if ((uintptr_t)s0 % 16) return fail(KDA_ERR_INVALID, "%s: initial_state is not 16-byte aligned", who);
    if ((uintptr_t)sT % 16) return fail(KDA_ERR_INVALID, "%s: final_state is not 16-byte aligned", who);
    if (in.workspace_bytes > 0) {
        if (!workspace || workspace_bytes < in.workspace_bytes)
            return fail(KDA_ERR_INVALID, "%s: the plan needs a workspace of %zu bytes (got %zu)", who,
                        in.workspace_bytes, workspace ? workspace_bytes : (size_t)0);
        if ((uintptr_t)workspace % 16) return fail(KDA_ERR_INVALID, "%s: workspace is not 16-byte aligned", who);
    }
    for (const Buffer& o : outs)
        for (const Buffer& i : ins) {
            if (o.p == sT && i.p == s0 && s0 == sT) continue;  // updated in place
            if (overlap(o.p, o.n, i.p, i.n)) return fail(KDA_ERR_ALIAS, "%s: %s overlaps %s", who, o.name, i.name);
        }
    for (int i = 0; i < 3; ++i)
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n))
                return fail(KDA_ERR_ALIAS, "%s: %s overlaps %s", who, outs[i].name, outs[j].name);
    return KDA_OK;
}

kda_status kda_linear_attention_prefill(kda_ctx* ctx, const kda_plan* p, const kda_linear_opts* opts, const void* q,
                                        const void* k, const void* v, const float* g, const int32_t* cu_dev,
                                        float scale, const void* s0, void* sT, void* out, void* workspace,
                                        size_t workspace_bytes, hipStream_t stream) {
    if (!ctx) return fail(KDA_ERR_INVALID, "kda_linear_attention_prefill: ctx is NULL");
    kda_status st = kda_linear_attention_prefill_validate(p, opts, q, k, v, g, cu_dev, scale, s0, sT, out, workspace,
                                                          workspace_bytes);
    if (st != KDA_OK) return st;
    if (!p->dev_tables)
        return fail(KDA_ERR_INVALID, "kda_linear_attention_prefill: plan has no device tables (host-only plan?)");
    if (p->device != ctx->device)
        return fail(KDA_ERR_INVALID, "kda_linear_attention_prefill: plan is for device %d, context for device %d",
                    p->device, ctx->device);
    std::lock_guard<std::mutex> lk(ctx->mu);
    DeviceScope scope;
    hipError_t e = scope.enter(ctx->device);
    if (e != hipSuccess) return hip_fail(e, "kda_linear_attention_prefill: selecting the device");
    const uint8_t* tabs = (const uint8_t*)p->dev_tables;
    LaArgs a{};
    a.q = (const uint16_t*)q;
    a.k = (const uint16_t*)k;
    a.v = (const uint16_t*)v;
    a.g = g;
    a.cu = cu_dev;
    a.Tt = p->info.total_tokens;
    a.H = p->info.H;
    a.Hk = opts && opts->qk_heads > 0 ? opts->qk_heads : a.H;
    a.group = a.H / a.Hk;
    a.s0 = s0;
    a.sT = sT;
    a.slots = (float*)((uint8_t*)workspace + p->off_carry);
    a.decays = (float*)((uint8_t*)workspace + p->off_b);
    a.out = (uint16_t*)out;
    a.scale = scale;
    a.g_fixed = opts && opts->g_fixed;
    a.state_bf16 = opts && opts->state_bf16;
    if (!p->la_merges.empty()) {
        LaArgs b = a;
        b.units = (const LaUnit*)(tabs + p->dev_off_k1_units);
        b.n_units = (int32_t)p->la_pre.size();
        e = timed_launch(ctx, stream, "linear_attention_segments", [&] { return launch_la_prefill(b, false, stream); });
        if (e != hipSuccess) return hip_fail(e, "linear attention segment launch");
        const LaMergeArgs m{(const LaMerge*)(tabs + p->dev_off_merges), (int32_t)p->la_merges.size(), a.H, s0,
                            a.state_bf16, a.slots, a.decays};
        e = timed_launch(ctx, stream, "linear_attention_merge", [&] { return launch_la_merge(m, stream); });
        if (e != hipSuccess) return hip_fail(e, "linear attention merge launch");
    }
    a.units = (const LaUnit*)(tabs + p->dev_off_units);
    a.n_units = (int32_t)p->la_units.size();
    e = timed_launch(ctx, stream, "linear_attention", [&] { return launch_la_prefill(a, true, stream); });
    if (e != hipSuccess) return hip_fail(e, "linear attention launch");
    return KDA_OK;
}

kda_status kda_linear_attention_decode_validate(int32_t n_seqs, int32_t n_tokens, int32_t H, int32_t qk_heads,
                                                int32_t dk, int32_t dv, const void* q, const void* k, const void* v,
                                                const float* g, int32_t g_fixed, float scale, const float* state,
                                                int32_t n_slots, const int32_t* slots, const void* out) {
    const char* const who = "kda_linear_attention_decode";
    if (dk != 128 || dv != 128)
        return fail(KDA_ERR_UNSUPPORTED, "%s: dk = dv = 128 required (got dk=%d dv=%d)", who, dk, dv);
    if (n_seqs < 0 || n_tokens < 0 || H < 1)
        return fail(KDA_ERR_INVALID, "%s: n_seqs and n_tokens must be >= 0 and H >= 1 (got %d, %d, %d)", who, n_seqs,
                    n_tokens, H);
    if (qk_heads < 1 || H % qk_heads != 0)
        return fail(KDA_ERR_INVALID, "%s: %d value heads are not a multiple of %d q/k heads", who, H, qk_heads);
    if (n_slots < 0) return fail(KDA_ERR_INVALID, "%s: n_slots must be >= 0 (got %d)", who, n_slots);
    if (!slots && n_slots != n_seqs)
        return fail(KDA_ERR_INVALID, "%s: without a slot table the state holds n_seqs = %d states, not %d", who,
                    n_seqs, n_slots);
    if (!launchable((int64_t)n_seqs * H, kLaDecodeThreads))
        return fail(KDA_ERR_INVALID, "%s: n_seqs * H too large (%lld)", who, (long long)n_seqs * H);
    if (!std::isfinite(scale)) return fail(KDA_ERR_INVALID, "%s: scale is not finite", who);
    if (n_seqs == 0 || n_tokens == 0) return KDA_OK;
    const size_t rows = (size_t)n_seqs * n_tokens, n_act = rows * H * 256, n_qk = rows * qk_heads * 256;
    const Buffer ins[] = {{q, n_qk, "q"}, {k, n_qk, "k"}, {v, n_act, "v"},
                          {g, (g_fixed ? (size_t)H : rows * H) * 4, "g"}, {slots, (size_t)n_seqs * 4, "slots"}};
    for (int i = 0; i < 4; ++i) {
        const int align = i < 3 ? 16 : 4;
        if (!ins[i].p) return fail(KDA_ERR_INVALID, "%s: %s is NULL", who, ins[i].name);
        if ((uintptr_t)ins[i].p % align)
            return fail(KDA_ERR_INVALID, "%s: %s is not %d-byte aligned", who, ins[i].name, align);
    }
    if (!out) return fail(KDA_ERR_INVALID, "%s: out is NULL", who);
    if ((uintptr_t)out % 16) return fail(KDA_ERR_INVALID, "%s: out is not 16-byte aligned", who);
    if (n_slots > 0 && !state) return fail(KDA_ERR_INVALID, "%s: state is NULL", who);
    if ((uintptr_t)state % 16) return fail(KDA_ERR_INVALID, "%s: state is not 16-byte aligned", who);
    if ((uintptr_t)slots % 4) return fail(KDA_ERR_INVALID, "%s: slots is not 4-byte aligned", who);
    const size_t n_state = (size_t)n_slots * H * kStateBytes;
    for (const Buffer& b : ins) {
        if (overlap(out, n_act, b.p, b.n)) return fail(KDA_ERR_ALIAS, "%s: out overlaps %s", who, b.name);
        if (overlap(state, n_state, b.p, b.n)) return fail(KDA_ERR_ALIAS, "%s: state overlaps %s", who, b.name);
    }
    if (overlap(out, n_act, state, n_state)) return fail(KDA_ERR_ALIAS, "%s: out overlaps state", who);
    return KDA_OK;
}

kda_status kda_linear_attention_decode(kda_ctx* ctx, int32_t n_seqs, int32_t n_tokens, int32_t H, int32_t qk_heads,
                                       int32_t dk, int32_t dv, const void* q, const void* k, const void* v,
                                       const float* g, int32_t g_fixed, float scale, float* state, int32_t n_slots,
                                       const int32_t* slots, void* out, hipStream_t stream) {
    if (!ctx) return fail(KDA_ERR_INVALID, "kda_linear_attention_decode: ctx is NULL");
    const kda_status st = kda_linear_attention_decode_validate(n_seqs, n_tokens, H, qk_heads, dk, dv, q, k, v, g,
                                                               g_fixed, scale, state, n_slots, slots, out);
    if (st != KDA_OK || n_seqs == 0 || n_tokens == 0) return st;
    std::lock_guard<std::mutex> lk(ctx->mu);
    DeviceScope scope;
    hipError_t e = scope.enter(ctx->device);
    if (e != hipSuccess) return hip_fail(e, "kda_linear_attention_decode: selecting the device");
    const LaDecodeArgs a{(const uint16_t*)q, (const uint16_t*)k, (const uint16_t*)v, g, state, (uint16_t*)out,
                         n_seqs, n_tokens, H, qk_heads, H / qk_heads, scale, slots, n_slots, g_fixed};
    e = timed_launch(ctx, stream, "linear_attention_decode", [&] { return launch_la_decode(a, stream); });
    if (e != hipSuccess) return hip_fail(e, "linear attention decode launch");
    return KDA_OK;
}

}  // extern "C"
