// Host side of the gated delta rule: plans, argument checks and dispatch of
// gated_delta.hip behind the C ABI of include/kda.h.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>
#include <functional>
#include <memory>
#include <new>
#include <queue>

#include "gated_delta_launch.h"
#include "kda_internal.h"

using namespace kda;

namespace {

constexpr int32_t kMaxHeads = 1 << 17;  // 32 token rows of one tensor stay below 2^31 bytes

// Cost model of a plan, microseconds on MI355X, fitted to launches of 8 to 2048
// units of 8 to 2048 chunks: a chunk of a unit with output, one of a segment's
// end state and transfer, what a launch of either takes beside its chunks, a
// merge step and the rest of a merge. Chunks take kBusy more while every compute
// unit is at work: matrix instructions at that rate lower the clock.
constexpr double kFullUs = 1.7, kPreUs = 2.25, kBusy = 0.28, kUnitUs = 7.0, kMergeUs = 1.0, kMergeLaunchUs = 5.0;

// A launch of units of these chunk counts (longest first), H heads each: one
// workgroup per compute unit, the next one to whichever is free first.
double launch_us(std::vector<int> chunks, int H, int n_cus, double per_chunk) {
    if (chunks.empty()) return 0;
    std::sort(chunks.begin(), chunks.end(), std::greater<int>());
    const int64_t n = (int64_t)chunks.size() * H;
    double total = 0;
    for (int c : chunks) total += (double)c * H;
    if (n > 16384) return kUnitUs + per_chunk * (1 + kBusy) * (total / n_cus + chunks[0]);
    std::priority_queue<double, std::vector<double>, std::greater<double>> busy;
    double end = 0;
    for (int c : chunks)
        for (int h = 0; h < H; ++h) {
            double t = 0;
            if ((int)busy.size() == n_cus) {
                t = busy.top();
                busy.pop();
            }
            t += kUnitUs + per_chunk * c;
            busy.push(t);
            end = std::max(end, t);
        }
    return end * (1 + kBusy * per_chunk * total / (end * n_cus));
}

int segments_of(int chunks, int seg) { return seg > 0 && chunks > seg ? (chunks + seg - 1) / seg : 1; }

double plan_us(const std::vector<int>& nch, int H, int n_cus, int seg) {
    std::vector<int> main, pre;
    int most = 1, items = 0;
    for (int c : nch) {
        const int n = segments_of(c, seg);
        most = std::max(most, n);
        items += n > 1;
        for (int s = 0; s < n; ++s) {
            const int len = (int)((int64_t)c * (s + 1) / n - (int64_t)c * s / n);
            main.push_back(len);
            if (s + 1 < n) pre.push_back(len);
        }
    }
    double us = launch_us(main, H, n_cus, kFullUs);
    if (most > 1) {
        const double rounds = std::max(1.0, 8.0 * items * H / n_cus);  // 8 workgroups per item and head
        us += launch_us(pre, H, n_cus, kPreUs) + (most - 2) * rounds * kMergeUs + kMergeLaunchUs;
    }
    return us;
}

kda_status build(int32_t n_cus, const int32_t* cu, int32_t n_seqs, int32_t H, int32_t dk, int32_t dv,
                 kda_cp_mode mode, int32_t seg_chunks, kda_plan** out) {
    if (!out) return fail(KDA_ERR_INVALID, "kda_plan_gated_delta: out is NULL");
    *out = nullptr;
    if (dk != 128 || dv != 128)
        return fail(KDA_ERR_UNSUPPORTED, "kda_plan_gated_delta: dk = dv = 128 required (got dk=%d dv=%d)", dk, dv);
    if (H < 1 || H > kMaxHeads)
        return fail(KDA_ERR_INVALID, "kda_plan_gated_delta: H must be in [1, %d] (got %d)", kMaxHeads, H);
    if (n_seqs < 1) return fail(KDA_ERR_INVALID, "kda_plan_gated_delta: n_seqs must be >= 1 (got %d)", n_seqs);
    if (!cu) return fail(KDA_ERR_INVALID, "kda_plan_gated_delta: cu_seqlens_host is NULL");
    if (n_cus < 1) return fail(KDA_ERR_INVALID, "kda_plan_gated_delta: n_cus must be >= 1 (got %d)", n_cus);
    if (mode != KDA_CP_OFF && mode != KDA_CP_ON && mode != KDA_CP_AUTO)
        return fail(KDA_ERR_INVALID, "kda_plan_gated_delta: unknown cp mode %d", (int)mode);
    if (seg_chunks < 0)
        return fail(KDA_ERR_INVALID, "kda_plan_gated_delta: seg_chunks must be >= 0 (got %d)", seg_chunks);
    if (cu[0] != 0) return fail(KDA_ERR_INVALID, "kda_plan_gated_delta: cu_seqlens[0] must be 0 (got %d)", cu[0]);
    for (int i = 0; i < n_seqs; ++i)
        if (cu[i + 1] < cu[i])
            return fail(KDA_ERR_INVALID, "kda_plan_gated_delta: cu_seqlens decreases at index %d (%d -> %d)", i, cu[i],
                        cu[i + 1]);

    std::vector<int> nch(n_seqs);
    int64_t total = 0;
    int longest = 0;
    for (int i = 0; i < n_seqs; ++i) {
        nch[i] = (int)(((int64_t)cu[i + 1] - cu[i] + kGdChunk - 1) / kGdChunk);
        total += nch[i];
        longest = std::max(longest, nch[i]);
    }
    // segment length: given, or the cheapest of a geometric range
    const double t_serial = plan_us(nch, H, n_cus, 0);
    double t_cp = -1;
    int seg = 0;
    if (mode != KDA_CP_OFF) {
        if (seg_chunks > 0) {
            seg = seg_chunks;
            t_cp = plan_us(nch, H, n_cus, seg);
        } else {
            for (int c = 4; c < longest; c += std::max(1, c / 4)) {
                const double t = plan_us(nch, H, n_cus, c);
                if (t_cp < 0 || t < t_cp) {
                    t_cp = t;
                    seg = c;
                }
            }
            // segments do more work for a shorter chain: cut only for what the model is sure of
            if (mode == KDA_CP_AUTO && 0.93 * t_serial <= t_cp) seg = 0;
        }
    }
    auto p = std::make_unique<kda_plan>();
    p->gated = true;
    p->cu.assign(cu, cu + n_seqs + 1);
    int n_carry = 0, n_sum = 0, n_cp = 0;
    for (int i = 0; i < n_seqs; ++i) {
        const int n = segments_of(nch[i], seg), L = cu[i + 1] - cu[i];
        if (n > 1) {
            p->gd_merges.push_back(GdMerge{i, n, n_carry, n_sum});
            ++n_cp;
        }
        for (int s = 0; s < n; ++s) {
            const int c0 = (int)((int64_t)nch[i] * s / n), c1 = (int)((int64_t)nch[i] * (s + 1) / n);
            const int t0 = c0 * kGdChunk, nt = (int)(std::min((int64_t)c1 * kGdChunk, (int64_t)L) - t0);
            p->gd_units.push_back(GdUnit{i, t0, nt, n > 1 ? n_carry + s : GD_INITIAL, s + 1 == n ? GD_FINAL : GD_NONE,
                                         GD_NONE});
            if (s + 1 < n) {
                if (s == 0) p->gd_pre.push_back(GdUnit{i, t0, nt, GD_INITIAL, n_sum, GD_NONE});
                else p->gd_pre.push_back(GdUnit{i, t0, nt, GD_ZERO, n_sum + 2 * s - 1, n_sum + 2 * s});
            }
            UnitDesc u{};
            u.seq = i;
            u.chunk0 = c0;
            u.n_chunks = c1 - c0;
            u.segment = s;
            u.n_segments = n;
            p->units.push_back(u);
        }
        if (n > 1) {
            n_carry += n;
            n_sum += 2 * n - 3;
        }
    }
    // longest first, so that the last workgroups to start are short
    auto longer = [](const GdUnit& a, const GdUnit& b) { return a.n_tok > b.n_tok; };
    std::stable_sort(p->gd_units.begin(), p->gd_units.end(), longer);
    std::stable_sort(p->gd_pre.begin(), p->gd_pre.end(), longer);
    std::stable_sort(p->units.begin(), p->units.end(),
                     [](const UnitDesc& a, const UnitDesc& b) { return a.n_chunks > b.n_chunks; });
    if (!launchable((int64_t)p->gd_units.size() * H, kGdThreads) ||
        !launchable((int64_t)p->gd_pre.size() * H, kGdSegmentThreads) ||
        !launchable((int64_t)p->gd_merges.size() * H * kGdMergeTiles, kGdMergeThreads)) {
        return fail(KDA_ERR_INVALID, "kda_plan_gated_delta: too many work units (%zu units, %d heads)",
                    p->gd_units.size(), H);
    }
    p->off_b = 0;
    p->off_carry = (size_t)n_sum * H * kStateBytes;
    kda_plan_info& in = p->info;
    in.n_seqs = n_seqs;
    in.H = H;
    in.dk = dk;
    in.dv = dv;
    in.total_tokens = cu[n_seqs];
    in.total_chunks = (int32_t)total;
    in.uses_cp = n_cp > 0;
    in.n_units = (int32_t)p->gd_units.size();
    in.n_cp_seqs = n_cp;
    in.n_prescan = n_sum;
    in.n_carry_slots = n_carry;
    in.max_unit_chunks = p->units[0].n_chunks;
    in.n_cus = n_cus;
    in.workspace_bytes = p->off_carry + (size_t)n_carry * H * kStateBytes;
    in.est_serial_us = t_serial;
    in.est_cp_us = t_cp;
    in.est_split_us = in.est_warm_cp_us = -1.0;
    *out = p.release();
    return KDA_OK;
}

kda_status upload(kda_plan* p, int device) {
    const size_t n_units = p->gd_units.size() * sizeof(GdUnit), n_pre = p->gd_pre.size() * sizeof(GdUnit);
    const size_t n_merge = p->gd_merges.size() * sizeof(GdMerge);
    p->dev_off_units = 0;
    p->dev_off_k1_units = align_up(n_units, 256);
    p->dev_off_merges = align_up(p->dev_off_k1_units + n_pre, 256);
    std::vector<uint8_t> host(p->dev_off_merges + n_merge, 0);
    memcpy(&host[0], p->gd_units.data(), n_units);
    if (n_pre) memcpy(&host[p->dev_off_k1_units], p->gd_pre.data(), n_pre);
    if (n_merge) memcpy(&host[p->dev_off_merges], p->gd_merges.data(), n_merge);
    DeviceScope scope;
    hipError_t e = scope.enter(device);
    if (e != hipSuccess) return hip_fail(e, "kda_plan_gated_delta: selecting the device");
    void* d = nullptr;
    e = hipMalloc(&d, host.size());
    if (e == hipSuccess) e = hipMemcpy(d, host.data(), host.size(), hipMemcpyHostToDevice);
    if (e != hipSuccess) {
        if (d) (void)hipFree(d);
        return hip_fail(e, "kda_plan_gated_delta: uploading plan tables");
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

kda_status kda_plan_gated_delta_host(int32_t n_cus, const int32_t* cu_seqlens_host, int32_t n_seqs, int32_t H,
                                     int32_t dk, int32_t dv, kda_cp_mode mode, int32_t seg_chunks, kda_plan** out) {
    try {
        return build(n_cus, cu_seqlens_host, n_seqs, H, dk, dv, mode, seg_chunks, out);
    } catch (const std::bad_alloc&) {
        return fail(KDA_ERR_INVALID, "kda_plan_gated_delta: out of host memory");
    }
}

kda_status kda_plan_gated_delta(kda_ctx* ctx, const int32_t* cu_seqlens_host, int32_t n_seqs, int32_t H, int32_t dk,
                                int32_t dv, kda_cp_mode mode, int32_t seg_chunks, kda_plan** out) {
    if (!ctx) return fail(KDA_ERR_INVALID, "kda_plan_gated_delta: ctx is NULL");
    try {
        kda_status st = build(ctx->n_cus, cu_seqlens_host, n_seqs, H, dk, dv, mode, seg_chunks, out);
        if (st != KDA_OK) return st;
        std::unique_ptr<kda_plan> p(*out);
        *out = nullptr;
        st = upload(p.get(), ctx->device);
        if (st == KDA_OK) *out = p.release();
        return st;
    } catch (const std::bad_alloc&) {
        return fail(KDA_ERR_INVALID, "kda_plan_gated_delta: out of host memory");
    }
}

kda_status kda_gated_delta_prefill_validate(const kda_plan* p, const kda_prefill_opts* opts, const void* q,
                                            const void* k, const void* v, const float* g, const void* beta,
                                            const int32_t* cu_dev, float scale, const void* s0, const void* sT,
                                            const void* out, const void* workspace, size_t workspace_bytes) {
    const char* const who = "kda_gated_delta_prefill";
    if (!p) return fail(KDA_ERR_INVALID, "%s: plan is NULL", who);
    if (!p->gated) return fail(KDA_ERR_INVALID, "%s: the plan is a KDA plan (use kda_plan_gated_delta)", who);
    const kda_plan_info& in = p->info;
    if (opts && opts->qk_heads < 0)
        return fail(KDA_ERR_INVALID, "%s: qk_heads must be >= 0 (got %d)", who, opts->qk_heads);
    const int32_t qk_heads = opts && opts->qk_heads > 0 ? opts->qk_heads : in.H;
    const bool beta16 = opts && opts->beta_bf16, state16 = opts && opts->state_bf16;
    if (in.H % qk_heads != 0)
        return fail(KDA_ERR_INVALID, "%s: the plan's %d value heads are not a multiple of %d q/k heads", who, in.H,
                    qk_heads);
    if (!std::isfinite(scale)) return fail(KDA_ERR_INVALID, "%s: scale is not finite", who);
    if (!cu_dev) return fail(KDA_ERR_INVALID, "%s: cu_seqlens is NULL", who);
    if ((uintptr_t)cu_dev % 4) return fail(KDA_ERR_INVALID, "%s: cu_seqlens is not 4-byte aligned", who);
    const size_t Tt = (size_t)in.total_tokens, H = (size_t)in.H, N = (size_t)in.n_seqs;
    const size_t n_qk = Tt * (size_t)qk_heads * 256, n_act = Tt * H * 256;
    const size_t n_state = N * H * 128 * 128 * (state16 ? 2 : 4);
    const Buffer ins[] = {{q, n_qk, "q"}, {k, n_qk, "k"}, {v, n_act, "v"}, {g, Tt * H * 4, "g"},
                          {beta, Tt * H * (beta16 ? 2 : 4), "beta"}, {cu_dev, (N + 1) * 4, "cu_seqlens"},
                          {s0, n_state, "initial_state"}};
    const Buffer outs[] = {{out, n_act, "out"}, {sT, n_state, "final_state"}, {workspace, in.workspace_bytes, "workspace"}};
    if (Tt > 0) {
        const size_t align[] = {16, 16, 16, 4, (size_t)(beta16 ? 2 : 4)};
        for (int i = 0; i < 5; ++i) {
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

kda_status kda_gated_delta_prefill(kda_ctx* ctx, const kda_plan* p, const kda_prefill_opts* opts, const void* q,
                                   const void* k, const void* v, const float* g, const void* beta,
                                   const int32_t* cu_dev, float scale, const void* s0, void* sT, void* out,
                                   void* workspace, size_t workspace_bytes, hipStream_t stream) {
    if (!ctx) return fail(KDA_ERR_INVALID, "kda_gated_delta_prefill: ctx is NULL");
    kda_status st = kda_gated_delta_prefill_validate(p, opts, q, k, v, g, beta, cu_dev, scale, s0, sT, out, workspace,
                                                     workspace_bytes);
    if (st != KDA_OK) return st;
    if (!p->dev_tables)
        return fail(KDA_ERR_INVALID, "kda_gated_delta_prefill: plan has no device tables (host-only plan?)");
    if (p->device != ctx->device)
        return fail(KDA_ERR_INVALID, "kda_gated_delta_prefill: plan is for device %d, context for device %d",
                    p->device, ctx->device);
    std::lock_guard<std::mutex> lk(ctx->mu);
    DeviceScope scope;
    hipError_t e = scope.enter(ctx->device);
    if (e != hipSuccess) return hip_fail(e, "kda_gated_delta_prefill: selecting the device");
    const uint8_t* tabs = (const uint8_t*)p->dev_tables;
    GdArgs a{};
    a.q = (const uint16_t*)q;
    a.k = (const uint16_t*)k;
    a.v = (const uint16_t*)v;
    a.g = g;
    a.beta = beta;
    a.cu = cu_dev;
    a.Tt = p->info.total_tokens;
    a.H = p->info.H;
    a.Hk = opts && opts->qk_heads > 0 ? opts->qk_heads : a.H;
    a.group = a.H / a.Hk;
    a.s0 = s0;
    a.sT = sT;
    a.sums = (float*)((uint8_t*)workspace + p->off_b);
    float* carries = (float*)((uint8_t*)workspace + p->off_carry);
    a.carries = carries;
    a.out = (uint16_t*)out;
    a.scale = scale;
    a.beta_bf16 = opts && opts->beta_bf16;
    a.state_bf16 = opts && opts->state_bf16;
    if (!p->gd_merges.empty()) {
        GdArgs b = a;
        b.units = (const GdUnit*)(tabs + p->dev_off_k1_units);
        b.n_units = (int32_t)p->gd_pre.size();
        e = timed_launch(ctx, stream, "gated_delta_segments", [&] { return launch_gd_prefill(b, false, stream); });
        if (e != hipSuccess) return hip_fail(e, "gated delta segment launch");
        const GdMergeArgs m{(const GdMerge*)(tabs + p->dev_off_merges), (int32_t)p->gd_merges.size(), a.H, s0,
                            a.state_bf16, a.sums, carries};
        e = timed_launch(ctx, stream, "gated_delta_merge", [&] { return launch_gd_merge(m, stream); });
        if (e != hipSuccess) return hip_fail(e, "gated delta merge launch");
    }
    a.units = (const GdUnit*)(tabs + p->dev_off_units);
    a.n_units = (int32_t)p->gd_units.size();
    e = timed_launch(ctx, stream, "gated_delta", [&] { return launch_gd_prefill(a, true, stream); });
    if (e != hipSuccess) return hip_fail(e, "gated delta launch");
    return KDA_OK;
}

kda_status kda_gated_delta_decode_validate(int32_t n_seqs, int32_t n_tokens, int32_t H, int32_t qk_heads, int32_t dk,
                                           int32_t dv, const void* q, const void* k, const void* v, const float* g,
                                           const float* beta, float scale, const float* state, int32_t n_slots,
                                           const int32_t* slots, const void* out) {
    const char* const who = "kda_gated_delta_decode";
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
    if (!launchable((int64_t)n_seqs * H, kGdDecodeThreads))
        return fail(KDA_ERR_INVALID, "%s: n_seqs * H too large (%lld)", who, (long long)n_seqs * H);
    if (!std::isfinite(scale)) return fail(KDA_ERR_INVALID, "%s: scale is not finite", who);
    if (n_seqs == 0 || n_tokens == 0) return KDA_OK;
    const size_t rows = (size_t)n_seqs * n_tokens, n_act = rows * H * 256, n_qk = rows * qk_heads * 256;
    const Buffer ins[] = {{q, n_qk, "q"}, {k, n_qk, "k"}, {v, n_act, "v"}, {g, rows * H * 4, "g"},
                          {beta, rows * H * 4, "beta"}, {slots, (size_t)n_seqs * 4, "slots"}};
    for (int i = 0; i < 5; ++i) {
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

kda_status kda_gated_delta_decode(kda_ctx* ctx, int32_t n_seqs, int32_t n_tokens, int32_t H, int32_t qk_heads,
                                  int32_t dk, int32_t dv, const void* q, const void* k, const void* v, const float* g,
                                  const float* beta, float scale, float* state, int32_t n_slots, const int32_t* slots,
                                  void* out, hipStream_t stream) {
    if (!ctx) return fail(KDA_ERR_INVALID, "kda_gated_delta_decode: ctx is NULL");
    const kda_status st = kda_gated_delta_decode_validate(n_seqs, n_tokens, H, qk_heads, dk, dv, q, k, v, g, beta,
                                                          scale, state, n_slots, slots, out);
    if (st != KDA_OK || n_seqs == 0 || n_tokens == 0) return st;
    std::lock_guard<std::mutex> lk(ctx->mu);
    DeviceScope scope;
    hipError_t e = scope.enter(ctx->device);
    if (e != hipSuccess) return hip_fail(e, "kda_gated_delta_decode: selecting the device");
    const GdDecodeArgs a{(const uint16_t*)q, (const uint16_t*)k, (const uint16_t*)v, g, beta, state, (uint16_t*)out,
                         n_seqs, n_tokens, H, qk_heads, H / qk_heads, scale, slots, n_slots};
    e = timed_launch(ctx, stream, "gated_delta_decode", [&] { return launch_gd_decode(a, stream); });
    if (e != hipSuccess) return hip_fail(e, "gated delta decode launch");
    return KDA_OK;
}

}  // extern "C"
