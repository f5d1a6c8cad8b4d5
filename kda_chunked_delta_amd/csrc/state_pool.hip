// Pages of a state pool on gfx950: copying, forking, freeing and compacting
// pages, and the reordering of a beam batch's states. A page is one slot of a
// pool (H states of 64 KiB; with several layers, one page per layer), so all
// of it is bound by HBM: two bytes moved per byte of a copied page.
#include "state_pool_launch.h"

namespace kda {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// A workgroup copies kMovePart bytes at a time: 4 vectors per thread in flight.
constexpr int MOVE_VEC = kMovePart / (kMoveThreads * 16);

// Part `part` of one page to another, by kMoveThreads threads. Read and written with the
// nontemporal hint: 64 forks of 2 MiB pages (256 MiB moved) take 43 us, 6.2 TB/s,
// where a plain copy of 1 GiB runs at 5.2.
__device__ __forceinline__ void move_part(const PoolView& p, int layer, int src, int dst, int part) {
    const uint8_t* s = p.base + layer * p.layer_stride + src * p.page_bytes;
    uint8_t* d = p.base + layer * p.layer_stride + dst * p.page_bytes;
    const int64_t at = (int64_t)part * kMovePart + threadIdx.x * 16;
    u32x4 x[MOVE_VEC];
#pragma unroll
    for (int i = 0; i < MOVE_VEC; ++i)
        if (at + i * 4096 < p.page_bytes) x[i] = __builtin_nontemporal_load((const u32x4*)(s + at + i * 4096));
#pragma unroll
    for (int i = 0; i < MOVE_VEC; ++i)
        if (at + i * 4096 < p.page_bytes) __builtin_nontemporal_store(x[i], (u32x4*)(d + at + i * 4096));
}

__device__ __forceinline__ bool in_pool(const PoolView& p, int page) { return page >= 0 && page < p.n_pages; }

__global__ __launch_bounds__(kMoveThreads) void pool_move(PoolView p, const int32_t* src, const int32_t* dst, int32_t n,
                                                 int32_t parts) {
    const int64_t per = (int64_t)parts * p.n_layers, total = per * n;
    for (int64_t f = blockIdx.x; f < total; f += gridDim.x) {
        const int i = (int)(f / per), rest = (int)(f % per);
        const int a = src ? src[i] : i, b = dst[i];
        if (a == b || !in_pool(p, a) || !in_pool(p, b)) continue;
        move_part(p, rest / parts, a, b, rest % parts);
    }
}

// Copies as if every source were read before any destination is written: each
// workgroup holds its part (2^log_vecs vectors) of every source page in
// registers, J vectors per thread, before it writes. Of several pairs with one
// destination the last wins. Vectors that nothing is copied from are read from
// the pool's first bytes, so that the loads need no branches (with them the
// compiler spilled the vectors: 40 us for two pages of 2 MiB instead of 8).
// Rotations of 2 MiB pages: 16 in 11.5 us, 64 in 37, and 256, in parts of 512
// bytes, in 269 (4.0 TB/s).
template <int J>
__global__ __launch_bounds__(1024) void pool_copy(PoolView p, const int32_t* src, const int32_t* dst, int32_t n,
                                                  int32_t first_part, int32_t parts, int32_t log_vecs) {
    __shared__ int32_t to[kPoolCopyMax], from[kPoolCopyMax];
    const int tid = threadIdx.x;
    int d = -1;
    if (tid < n) {
        const int a = src[tid], b = dst[tid];
        if (in_pool(p, a) && in_pool(p, b)) d = b;
        from[tid] = a;
        to[tid] = d;
    }
    __syncthreads();
    if (d >= 0)
        for (int j = tid + 1; j < n; ++j)
            if (to[j] == d) d = -2;
    __syncthreads();
    if (tid < n) to[tid] = d;
    __syncthreads();
    const int at_part = first_part + blockIdx.x, layer = at_part / parts, part = at_part % parts;
    uint8_t* base = p.base + layer * p.layer_stride;
    // vector f of the workgroup: pair f >> log_vecs, a row of consecutive vectors of its page
    const int64_t first = (int64_t)part << log_vecs;
    u32x4 x[J];
    uint8_t* w[J];  // where it goes
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int f = tid + j * 1024, i = f >> log_vecs;
        const int64_t at = (first + (f & ((1 << log_vecs) - 1))) * 16;
        const int t = i < n ? to[i] : -1;
        const bool ok = t >= 0 && at < p.page_bytes;
        x[j] = *(const u32x4*)(ok ? base + from[i] * p.page_bytes + at : p.base);
        w[j] = ok ? base + t * p.page_bytes + at : nullptr;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < J; ++j)
        if (w[j]) *(u32x4*)w[j] = x[j];
}

// Exclusive prefix sum of x over 1024 threads; `all` gets the total. s_sum:
// 17 ints of LDS, free again after the call.
__device__ __forceinline__ int block_scan(int x, int* s_sum, int& all) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int y = x;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int z = __shfl_up(y, d, 64);
        if (lane >= d) y += z;
    }
    if (lane == 63) s_sum[wave] = y;
    __syncthreads();
    if (threadIdx.x == 0) {
        int t = 0;
        for (int w = 0; w < 16; ++w) {
            const int c = s_sum[w];
            s_sum[w] = t;
            t += c;
        }
        s_sum[16] = t;
    }
    __syncthreads();
    all = s_sum[16];
    const int r = s_sum[wave] + y - x;
    __syncthreads();
    return r;
}

// Request i gets the free page of its rank among the requests with a used
// source, in page order. One workgroup.
__global__ __launch_bounds__(1024) void pool_fork_plan(uint8_t* used, int32_t n_pages, const int32_t* src,
                                                       int32_t* dst, int32_t n) {
    __shared__ int32_t s_sum[17], s_free[kPoolForkMax];
    const int tid = threadIdx.x;
    int want = 0;
    int rank[kPoolForkMax / 1024];
#pragma unroll
    for (int j = 0; j < kPoolForkMax / 1024; ++j) {
        rank[j] = -1;
        if (j * 1024 < n) {
            const int i = j * 1024 + tid, a = i < n ? src[i] : -1;
            const bool ok = a >= 0 && a < n_pages && used[a];
            int all;
            const int r = block_scan(ok, s_sum, all);
            if (ok) rank[j] = want + r;
            want += all;
        }
    }
    int found = 0;
    for (int p0 = 0; p0 < n_pages && found < want; p0 += 1024) {
        const int pg = p0 + tid;
        const bool fr = pg < n_pages && !used[pg];
        int all;
        const int r = found + block_scan(fr, s_sum, all);
        if (fr && r < want) s_free[r] = pg;
        found += all;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPoolForkMax / 1024; ++j) {
        const int i = j * 1024 + tid;
        if (i < n) {
            const int d = rank[j] >= 0 && rank[j] < found ? s_free[rank[j]] : -1;
            dst[i] = d;
            if (d >= 0) used[d] = 1;
        }
    }
}

__global__ __launch_bounds__(256) void pool_free(uint8_t* used, int32_t n_pages, const int32_t* pages, int32_t n) {
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    const int pg = pages[i];
    if (pg >= 0 && pg < n_pages) used[pg] = 0;
}

// newpos[p] = the place of used page p among the first `live` pages: itself if
// it lies there, else the hole of its rank; -1 for a free page. One workgroup.
// The list of holes is kept in newpos behind the first `live` entries; the
// final entries replace it from the last page down, because page p's rank
// among the pages to move is at most p - live.
__global__ __launch_bounds__(1024) void pool_compact_plan(uint8_t* used, int32_t n_pages, int32_t* table,
                                                          int32_t n_table, int32_t* newpos, int32_t* n_live) {
    __shared__ int32_t s_sum[17];
    const int tid = threadIdx.x;
    int live = 0;
    for (int p0 = 0; p0 < n_pages; p0 += 1024) {
        int all;
        block_scan(p0 + tid < n_pages && used[p0 + tid], s_sum, all);
        live += all;
    }
    int holes = 0;
    for (int p0 = 0; p0 < live; p0 += 1024) {
        const int pg = p0 + tid;
        const bool hole = pg < live && !used[pg];
        int all;
        const int r = holes + block_scan(hole, s_sum, all);
        if (hole) newpos[live + r] = pg;
        if (pg < live) newpos[pg] = hole ? -1 : pg;
        holes += all;
    }
    __syncthreads();
    int behind = holes;  // pages to move at or after the current tile's end
    for (int p0 = (n_pages - 1) / 1024 * 1024; p0 + 1024 > live && p0 >= 0; p0 -= 1024) {
        const int pg = p0 + tid;
        const bool mv = pg < n_pages && pg >= live && used[pg];
        int all;
        const int r = block_scan(mv, s_sum, all);
        behind -= all;
        const int to = mv ? newpos[live + behind + r] : -1;
        __syncthreads();
        if (pg < n_pages && pg >= live) newpos[pg] = to;
    }
    __syncthreads();
    for (int pg = tid; pg < n_pages; pg += 1024) used[pg] = pg < live;
    for (int i = tid; i < n_table; i += 1024) {
        const int t = table[i];
        table[i] = t >= 0 && t < n_pages ? newpos[t] : -1;
    }
    if (tid == 0) *n_live = live;
}

// Reordering of a beam batch. The first beam that continues parent q keeps q's
// page; every other beam takes, in beam order, a page of the parents that no
// beam continues (beams without a valid parent last, and uncopied). Sources
// (pages of parents that go on) and destinations (pages of parents that do
// not) are disjoint. One workgroup per part of one beam's page; each works the
// plan of its batch entry out for itself, one beam per lane, which costs less
// than a launch of its own. 16 entries of 4 beams and 32 heads: 25 us, 5.2 TB/s.
__global__ __launch_bounds__(kMoveThreads) void beam_reorder(PoolView p, const int32_t* slots, const int32_t* parents,
                                                    int32_t* new_slots, int32_t beams, int32_t parts) {
    __shared__ int32_t s_target;
    const int item = blockIdx.x / parts, part = blockIdx.x % parts;
    const int w = item % beams;
    const int64_t row = (int64_t)(item / beams) * beams;
    if (threadIdx.x < 64) {
        const int l = threadIdx.x;
        int q = l < beams ? parents[row + l] : -1;
        if (q >= beams) q = -1;
        bool first = q >= 0, gone = l < beams;
        for (int i = 0; i < beams; ++i) {
            const int qi = __shfl(q, i, 64);
            if (qi == q && i < l) first = false;
            if (qi == l) gone = false;
        }
        const uint64_t extra = __ballot(q >= 0 && !first), none = __ballot(l < beams && q < 0);
        uint64_t free = __ballot(gone);
        const uint64_t below = (1ull << w) - 1;
        int target = __shfl(q, w, 64);
        const bool is_extra = extra >> w & 1, is_none = none >> w & 1;
        if (is_extra || is_none) {
            int r = is_extra ? __popcll(extra & below) : __popcll(extra) + __popcll(none & below);
            for (; r > 0; --r) free &= free - 1;
            target = __ffsll((unsigned long long)free) - 1;
        }
        if (l == 0) s_target = target;
    }
    __syncthreads();
    const int to = slots[row + s_target], q = parents[row + w];
    if (part == 0 && threadIdx.x == 0) new_slots[row + w] = to;
    if (q < 0 || q >= beams) return;
    const int from = slots[row + q];
    if (from == to || !in_pool(p, from) || !in_pool(p, to)) return;
    for (int layer = 0; layer < p.n_layers; ++layer) move_part(p, layer, from, to, part);
}

int parts_of(const PoolView& p) { return (int)((p.page_bytes + kMovePart - 1) / kMovePart); }

}  // namespace

hipError_t launch_pool_move(const PoolView& p, const int32_t* src, const int32_t* dst, int32_t n, hipStream_t s) {
    const int parts = parts_of(p);
    const int64_t total = (int64_t)parts * p.n_layers * n;
    if (total == 0 || p.n_pages == 0) return hipSuccess;
    hipLaunchKernelGGL(pool_move, dim3((unsigned)(total < 4096 ? total : 4096)), dim3(kMoveThreads), 0, s, p, src, dst, n,
                       parts);
    return hipGetLastError();
}

hipError_t launch_pool_copy(const PoolView& p, const int32_t* src, const int32_t* dst, int32_t n, hipStream_t s) {
    // vectors of a part: 64 KiB down to 128 bytes, n parts within 8 vectors of
    // 1024 threads, and a page in parts for every compute unit if it has them
    int log_vecs = 12;
    while (log_vecs > 3 && ((int64_t)n << log_vecs > 8 * 1024 ||
                            ((p.page_bytes / 16 * p.n_layers) >> log_vecs) < 512))
        --log_vecs;
    const int64_t parts = ((p.page_bytes / 16 - 1) >> log_vecs) + 1;
    const int64_t vectors = (int64_t)n << log_vecs, total = parts * p.n_layers;
    const auto kernel = vectors <= 1024 ? pool_copy<1> : vectors <= 4096 ? pool_copy<4> : pool_copy<8>;
    // parts are apart from each other; a launch takes fewer than 2^32 threads (512 MiB in parts of 128 bytes)
    constexpr int64_t MOST = UINT32_MAX / 1024;
    for (int64_t first = 0; first < total; first += MOST) {
        const dim3 grid((unsigned)(total - first < MOST ? total - first : MOST));
        hipLaunchKernelGGL(kernel, grid, dim3(1024), 0, s, p, src, dst, n, (int)first, (int)parts, log_vecs);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch_pool_fork_plan(uint8_t* used, int32_t n_pages, const int32_t* src, int32_t* dst, int32_t n,
                                 hipStream_t s) {
    hipLaunchKernelGGL(pool_fork_plan, dim3(1), dim3(1024), 0, s, used, n_pages, src, dst, n);
    return hipGetLastError();
}

hipError_t launch_pool_free(uint8_t* used, int32_t n_pages, const int32_t* pages, int32_t n, hipStream_t s) {
    hipLaunchKernelGGL(pool_free, dim3((unsigned)(((int64_t)n + 255) / 256)), dim3(256), 0, s, used, n_pages, pages,
                       n);
    return hipGetLastError();
}

hipError_t launch_pool_compact_plan(uint8_t* used, int32_t n_pages, int32_t* table, int32_t n_table, int32_t* newpos,
                                    int32_t* n_live, hipStream_t s) {
    hipLaunchKernelGGL(pool_compact_plan, dim3(1), dim3(1024), 0, s, used, n_pages, table, n_table, newpos, n_live);
    return hipGetLastError();
}

hipError_t launch_beam_reorder(const PoolView& p, const int32_t* slots, const int32_t* parents, int32_t* new_slots,
                               int32_t batch, int32_t beams, hipStream_t s) {
    const int parts = parts_of(p);
    hipLaunchKernelGGL(beam_reorder, dim3((unsigned)((int64_t)batch * beams * parts)), dim3(kMoveThreads), 0, s, p,
                       slots, parents, new_slots, beams, parts);
    return hipGetLastError();
}

}  // namespace kda
