// pages.cu -- the page table of a paged cache: taking and freeing pages,
// forking sequences, moving the pages in use together.  Everything stays on the
// device, so the calls can be captured and no length is read by the host.
//
// A table [B, M] holds the pages of each sequence (-1: none), refs [n_pages]
// how many table entries name a page; a page is free when its count is 0.
// Pages are always taken in ascending order, for the table entries that need
// one in (row, slot) order, so the result does not depend on the schedule: the
// only atomics are integer adds and minima whose order does not matter.
//
// Each call is one kernel on one cluster of 8 CTAs (256 warps): the phases are
// separated by cluster barriers instead of launches, and eight SMs read the
// table and the counts.  The work is a few bytes per entry; what bounds it is
// the latency of a phase (a barrier and a dependent load), so the phases are few.
// Ranks come from one pass of ballots: every warp owns a contiguous range of
// pages (or entries), publishes its count, and after the barrier all 256 counts
// are scanned by each CTA for itself.
#include <climits>

#include "device.cuh"
#include "internal.h"

namespace gqa {

constexpr int kPgCtas = 8;                   // one portable cluster
constexpr int kPgThreads = 1024;
constexpr int kPgWarps = kPgCtas * kPgThreads / 32;

__device__ __forceinline__ void cluster_barrier() {
    // release / acquire at cluster scope, after a device-wide fence for the
    // global writes of the phase
    __threadfence();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The contiguous range of [0, n) that warp gw owns, in multiples of 32.
struct PgRange {
    long long begin, end;
    __device__ PgRange(long long n, int gw) {
        const long long seg = (n + 32ll * kPgWarps - 1) / (32ll * kPgWarps) * 32;
        begin = min(n, seg * gw);
        end = min(n, begin + seg);
    }
};

// Exclusive prefix sums of 256 counts published in global memory; total in out[256].
__device__ __forceinline__ void pg_scan(const int *counts, int (&out)[kPgWarps + 1], int (&tmp)[8]) {
    const int t = threadIdx.x, lane = t & 31, w = t >> 5;
    int v = 0, x = 0;
    if (t < kPgWarps) {
        v = x = __ldcg(counts + t);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += y;
        }
        if (lane == 31) tmp[w] = x;
    }
    __syncthreads();
    if (t < kPgWarps) {
        for (int i = 0; i < w; ++i) x += tmp[i];
        out[t] = x - v;
        if (t == kPgWarps - 1) out[kPgWarps] = x;
    }
    __syncthreads();
}

struct PgParams {
    int32_t *table, *refs, *seqlens;
    const int32_t *lengths, *parents;
    int32_t *moves;
    int B, M, n_pages, page, cap;
    int *status;
    // workspace
    int *count_a, *count_b;                  // one per warp
    int *list_a, *list_b, *list_c;           // n_pages each
    int *rows;                               // 4 B
    int *entries;                            // B M
};

__device__ __forceinline__ int ld(const int *p) { return __ldcg(p); }

// Entry as a page, -1 for none; an entry beyond the pool counts as none.
__device__ __forceinline__ int valid_page(int e, int n_pages, int *status) {
    if (e >= n_pages) {
        record_status(status, GQA_ERR_INVALID_ARG);
        return -1;
    }
    return e < 0 ? -1 : e;
}

// Free pages of this warp's range, counted.
__device__ __forceinline__ int count_free(const PgParams &p, int gw, int lane) {
    const PgRange r(p.n_pages, gw);
    int n = 0;
    for (long long i = r.begin; i < r.end; i += 32) {
        const bool free = i + lane < r.end && ld(p.refs + i + lane) <= 0;
        n += __popc(__ballot_sync(0xffffffffu, free));
    }
    return n;
}

// The first `want` free pages of the pool, in order, into list_a, each with one reference.
__device__ __forceinline__ void take_free(const PgParams &p, int gw, int lane, int rank, int want) {
    const PgRange r(p.n_pages, gw);
    for (long long i = r.begin; i < r.end && rank < want; i += 32) {
        const bool free = i + lane < r.end && ld(p.refs + i + lane) <= 0;
        const uint32_t m = __ballot_sync(0xffffffffu, free);
        const int k = rank + __popc(m & ((1u << lane) - 1));
        if (free && k < want) {
            p.list_a[k] = static_cast<int>(i + lane);
            p.refs[i + lane] = 1;
        }
        rank += __popc(m);
    }
}

// Pages for the rows' lengths: entries at and past ceil(length / page) are
// released, missing ones below it get the lowest free pages.
__global__ void __cluster_dims__(kPgCtas, 1, 1) __launch_bounds__(kPgThreads, 1)
pages_resize_kernel(const PgParams p) {
    __shared__ int need[kPgWarps + 1], avail[kPgWarps + 1], tmp[8];
    const int lane = threadIdx.x & 31, gw = (blockIdx.x * kPgThreads + threadIdx.x) >> 5;
    const long long n = static_cast<long long>(p.B) * p.M;
    const PgRange r(n, gw);
    auto keep = [&](int b) {                  // slots that row b shall hold
        const int L = p.lengths[b];
        const long long k = L <= 0 ? 0 : (static_cast<long long>(L) + p.page - 1) / p.page;
        if (L < 0 || k > p.M) record_status(p.status, GQA_ERR_INVALID_ARG);
        return static_cast<int>(min(k, static_cast<long long>(p.M)));
    };
    int count = 0;
    for (long long i = r.begin; i < r.end; i += 32) {
        const long long at = i + lane;
        bool want = false;
        if (at < r.end) {
            const int b = static_cast<int>(at / p.M), s = static_cast<int>(at % p.M);
            const int raw = p.table[at], e = valid_page(raw, p.n_pages, p.status);
            if (s < keep(b)) {
                want = e < 0;
            } else {
                if (e >= 0 && atomicSub(p.refs + e, 1) <= 0)
                    record_status(p.status, GQA_ERR_INVALID_ARG);
                if (raw != -1) p.table[at] = -1;
            }
        }
        count += __popc(__ballot_sync(0xffffffffu, want));
    }
    if (lane == 0) p.count_a[gw] = count;
    cluster_barrier();
    const int free = count_free(p, gw, lane);
    if (lane == 0) p.count_b[gw] = free;
    cluster_barrier();
    pg_scan(p.count_a, need, tmp);
    pg_scan(p.count_b, avail, tmp);
    if (need[kPgWarps] == 0) return;          // the same for every CTA
    take_free(p, gw, lane, avail[gw], need[kPgWarps]);
    cluster_barrier();
    if (need[kPgWarps] > avail[kPgWarps] && gw == 0 && lane == 0)
        record_status(p.status, GQA_ERR_PAGES);
    int rank = need[gw];
    for (long long i = r.begin; i < r.end; i += 32) {
        const long long at = i + lane;
        bool want = false;
        if (at < r.end) {
            const int e = p.table[at];        // this warp's own range
            want = static_cast<int>(at % p.M) < keep(static_cast<int>(at / p.M)) &&
                   (e < 0 || e >= p.n_pages);
        }
        const uint32_t m = __ballot_sync(0xffffffffu, want);
        const int k = rank + __popc(m & ((1u << lane) - 1));
        if (want) p.table[at] = k < avail[kPgWarps] ? ld(p.list_a + k) : -1;
        rank += __popc(m);
    }
}

// New row b = old row parents[b].  rows: [heir | length | source page or -1 | rank].
__global__ void __cluster_dims__(kPgCtas, 1, 1) __launch_bounds__(kPgThreads, 1)
pages_fork_kernel(const PgParams p) {
    __shared__ int need[kPgWarps + 1], avail[kPgWarps + 1], tmp[8];
    const int lane = threadIdx.x & 31, gw = (blockIdx.x * kPgThreads + threadIdx.x) >> 5;
    const int gt = blockIdx.x * kPgThreads + threadIdx.x;
    int *heir = p.rows, *length = heir + p.B, *source = length + p.B, *rank_of = source + p.B;
    auto parent = [&](int b) {
        const int x = p.parents[b];
        return x >= 0 && x < p.B ? x : -1;
    };
    for (int b = gt; b < p.B; b += kPgCtas * kPgThreads) {
        heir[b] = INT_MAX;
        if (p.parents[b] >= p.B) record_status(p.status, GQA_ERR_INVALID_ARG);
    }
    cluster_barrier();
    // the parent's own row goes on in its last page, else its first child does
    for (int b = gt; b < p.B; b += kPgCtas * kPgThreads) {
        const int x = parent(b);
        if (x >= 0) atomicMin(heir + x, x == b ? -1 : b);
    }
    cluster_barrier();
    // new lengths, and which rows need a page for a copy of the last one
    const PgRange rb(p.B, gw);
    int count = 0;
    for (long long i = rb.begin; i < rb.end; i += 32) {
        bool want = false;
        if (i + lane < rb.end) {
            const int b = static_cast<int>(i + lane), x = parent(b);
            int L = x >= 0 ? p.seqlens[x] : 0, src = -1;
            if (L < 0 || L > p.M * p.page) {
                record_status(p.status, GQA_ERR_INVALID_ARG);
                L = L < 0 ? 0 : p.M * p.page;
            }
            if (x >= 0 && x != b && ld(heir + x) != b && L % p.page > 0) {
                src = valid_page(p.table[static_cast<size_t>(x) * p.M + L / p.page], p.n_pages, p.status);
                if (src < 0) record_status(p.status, GQA_ERR_INVALID_ARG);
                want = src >= 0;
            }
            length[b] = L;
            source[b] = src;
        }
        count += __popc(__ballot_sync(0xffffffffu, want));
    }
    if (lane == 0) p.count_a[gw] = count;
    // new rows, and the references that changed rows drop and gain
    const long long n = static_cast<long long>(p.B) * p.M;
    for (long long at = gt; at < n; at += kPgCtas * kPgThreads) {
        const int b = static_cast<int>(at / p.M), s = static_cast<int>(at % p.M), x = parent(b);
        const int old = p.table[at];
        int now = old;
        if (x != b) {
            now = -1;
            if (x >= 0) {
                const int L = max(0, p.seqlens[x]);
                if (s < L / p.page || ld(heir + x) == b) now = p.table[static_cast<size_t>(x) * p.M + s];
            }
            now = valid_page(now, p.n_pages, p.status);
            const int gone = valid_page(old, p.n_pages, p.status);
            if (gone != now) {
                if (gone >= 0) atomicSub(p.refs + gone, 1);
                if (now >= 0) atomicAdd(p.refs + now, 1);
            }
        }
        p.entries[at] = now;
    }
    cluster_barrier();
    const int free = count_free(p, gw, lane);
    if (lane == 0) p.count_b[gw] = free;
    cluster_barrier();
    pg_scan(p.count_a, need, tmp);
    pg_scan(p.count_b, avail, tmp);
    const int want = need[kPgWarps], have = min(want, avail[kPgWarps]);
    take_free(p, gw, lane, avail[gw], want);
    int rank = need[gw];
    for (long long i = rb.begin; i < rb.end; i += 32) {
        const bool w = i + lane < rb.end && source[i + lane] >= 0;      // this warp's own rows
        const uint32_t m = __ballot_sync(0xffffffffu, w);
        if (i + lane < rb.end) rank_of[i + lane] = w ? rank + __popc(m & ((1u << lane) - 1)) : -1;
        rank += __popc(m);
    }
    cluster_barrier();
    if (gt == 0) {
        p.moves[0] = have;
        p.moves[1] = p.moves[2] = 0;
        if (want > have) record_status(p.status, GQA_ERR_PAGES);
    }
    for (long long at = gt; at < n; at += kPgCtas * kPgThreads) {
        const int b = static_cast<int>(at / p.M), s = static_cast<int>(at % p.M);
        const int k = ld(rank_of + b), L = ld(length + b);
        int e = p.entries[at];                // written by this thread
        if (k >= 0 && s == L / p.page) e = k < have ? ld(p.list_a + k) : -1;
        p.table[at] = e;
    }
    for (int b = gt; b < p.B; b += kPgCtas * kPgThreads) {
        const int k = ld(rank_of + b), L = ld(length + b);
        p.seqlens[b] = L;
        if (k >= 0 && k < have) {
            p.moves[3 * (1 + k)] = ld(source + b);
            p.moves[3 * (1 + k) + 1] = ld(p.list_a + k);
            p.moves[3 * (1 + k) + 2] = L % p.page;
        }
    }
}

// Used pages at and past their number move, in order, to the free pages below it.
__global__ void __cluster_dims__(kPgCtas, 1, 1) __launch_bounds__(kPgThreads, 1)
pages_compact_kernel(const PgParams p) {
    __shared__ int used[kPgWarps + 1], tmp[8], s_below;
    const int lane = threadIdx.x & 31, gw = (blockIdx.x * kPgThreads + threadIdx.x) >> 5;
    const int gt = blockIdx.x * kPgThreads + threadIdx.x;
    const PgRange r(p.n_pages, gw);
    const int mine = static_cast<int>(r.end - r.begin) - count_free(p, gw, lane);
    if (lane == 0) p.count_a[gw] = mine;
    cluster_barrier();
    pg_scan(p.count_a, used, tmp);
    const int n_used = used[kPgWarps];
    // used pages below n_used: whole ranges, and the part of the one that n_used cuts
    if (threadIdx.x < 32) {
        const long long seg = (p.n_pages + 32ll * kPgWarps - 1) / (32ll * kPgWarps) * 32;
        const int cut = static_cast<int>(min(static_cast<long long>(kPgWarps), n_used / seg));
        int below = used[cut];                // cut = 256: all of them
        for (long long i = seg * cut; i < n_used; i += 32) {
            const bool u = i + lane < n_used && ld(p.refs + i + lane) > 0;
            below += __popc(__ballot_sync(0xffffffffu, u));
        }
        if (lane == 0) s_below = below;
    }
    __syncthreads();
    const int below = s_below, n_moves = n_used - below;
    // list_a: free pages below n_used; list_b: used pages past it; list_c: the
    // move of each page past it, -1 for none
    int rank = used[gw];
    for (long long i = r.begin; i < r.end; i += 32) {
        const bool in = i + lane < r.end;
        const int id = static_cast<int>(i + lane);
        const bool u = in && ld(p.refs + id) > 0;
        const uint32_t m = __ballot_sync(0xffffffffu, u);
        const int k = rank + __popc(m & ((1u << lane) - 1));     // used pages before id
        if (in) {
            if (id < n_used) {
                if (!u) p.list_a[id - k] = id;
            } else {
                if (u) p.list_b[k - below] = id;
                p.list_c[id] = u ? k - below : -1;
            }
        }
        rank += __popc(m);
    }
    cluster_barrier();
    if (gt == 0) {
        p.moves[0] = n_moves;
        p.moves[1] = p.moves[2] = 0;
    }
    for (int k = gt; k < n_moves; k += kPgCtas * kPgThreads) {
        const int from = ld(p.list_b + k), to = ld(p.list_a + k);
        p.refs[to] = ld(p.refs + from);
        p.refs[from] = 0;
        p.moves[3 * (1 + k)] = from;
        p.moves[3 * (1 + k) + 1] = to;
        p.moves[3 * (1 + k) + 2] = p.page;
    }
    const long long n = static_cast<long long>(p.B) * p.M;
    for (long long at = gt; at < n; at += kPgCtas * kPgThreads) {
        const int e = valid_page(p.table[at], p.n_pages, p.status);
        if (e < n_used) continue;
        const int k = ld(p.list_c + e);
        if (k >= 0) p.table[at] = ld(p.list_a + k);
        else record_status(p.status, GQA_ERR_INVALID_ARG);       // an entry without a reference
    }
}

static size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Workspace: counts of 2 x 256 warps | 4 ints per row | 3 lists of pages | a copy of the table.
struct PgWorkspace {
    size_t off_rows, off_lists, list, off_entries, bytes;
    PgWorkspace(int B, int M, int n_pages) {
        off_rows = 2 * kPgWarps * sizeof(int);
        off_lists = off_rows + align256(4 * static_cast<size_t>(B) * sizeof(int));
        list = align256(static_cast<size_t>(n_pages) * sizeof(int));
        off_entries = off_lists + 3 * list;
        bytes = off_entries + align256(static_cast<size_t>(B) * M * sizeof(int));
    }
};

// Checks shared by the three calls; fills p's table part and the workspace.
static int pages_setup(PgParams &p, int32_t *table, int32_t *refs, int B, int M, int n_pages, int page,
                       void *workspace, size_t workspace_bytes) {
    if (B < 0 || M < 1)
        return set_error(GQA_ERR_INVALID_ARG, "B=%d must be >= 0 and M=%d page slots >= 1", B, M);
    if (n_pages < 1) return set_error(GQA_ERR_INVALID_ARG, "n_pages=%d must be >= 1", n_pages);
    if (page < 1) return set_error(GQA_ERR_INVALID_ARG, "page=%d must be >= 1", page);
    if (static_cast<long long>(M) * page > 0x7fffffffLL || static_cast<long long>(B) * M > 0x7fffffffLL)
        return set_error(GQA_ERR_UNSUPPORTED, "M=%d x page=%d rows or B=%d x M entries exceed an int", M,
                         page, B);
    if (B > 0)
        if (int rc = check_ptr(table, 4, "table")) return rc;
    if (int rc = check_ptr(refs, 4, "refs")) return rc;
    const PgWorkspace ws(B, M, n_pages);
    if (int rc = check_workspace(workspace, workspace_bytes, ws.bytes)) return rc;
    uint8_t *base = static_cast<uint8_t *>(workspace);
    p.table = table;
    p.refs = refs;
    p.B = B;
    p.M = M;
    p.n_pages = n_pages;
    p.page = page;
    p.count_a = reinterpret_cast<int *>(base);
    p.count_b = p.count_a + kPgWarps;
    p.rows = reinterpret_cast<int *>(base + ws.off_rows);
    p.list_a = reinterpret_cast<int *>(base + ws.off_lists);
    p.list_b = reinterpret_cast<int *>(base + ws.off_lists + ws.list);
    p.list_c = reinterpret_cast<int *>(base + ws.off_lists + 2 * ws.list);
    p.entries = reinterpret_cast<int *>(base + ws.off_entries);
    return GQA_OK;
}

static int pages_launch(void (*kern)(PgParams), PgParams &p, gqa_stream_t stream, const char *what) {
    if (int rc = require_sm100()) return rc;
    p.status = device_status_ptr();
    if (!p.status) return GQA_ERR_CUDA;
    kern<<<kPgCtas, kPgThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
    return check_cuda(cudaGetLastError(), what);
}

}  // namespace gqa

using namespace gqa;

extern "C" size_t gqa_pages_workspace_size(int B, int M, int n_pages) {
    if (B < 0 || M < 1 || n_pages < 1) return 0;
    return PgWorkspace(B, M, n_pages).bytes;
}

extern "C" int gqa_pages_resize(int32_t *table, int32_t *refs, const int32_t *lengths, int B, int M,
                                int n_pages, int page, void *workspace, size_t workspace_bytes,
                                gqa_stream_t stream) {
    clear_error();
    PgParams p{};
    if (int rc = pages_setup(p, table, refs, B, M, n_pages, page, workspace, workspace_bytes)) return rc;
    if (B == 0) return GQA_OK;
    if (int rc = check_ptr(lengths, 4, "lengths")) return rc;
    p.lengths = lengths;
    return pages_launch(pages_resize_kernel, p, stream, "pages_resize_kernel launch");
}

extern "C" int gqa_pages_fork(int32_t *table, int32_t *refs, int32_t *seqlens, const int32_t *parents,
                              int32_t *moves, int B, int M, int n_pages, int page, void *workspace,
                              size_t workspace_bytes, gqa_stream_t stream) {
    clear_error();
    PgParams p{};
    if (int rc = pages_setup(p, table, refs, B, M, n_pages, page, workspace, workspace_bytes)) return rc;
    if (int rc = check_ptr(moves, 4, "moves")) return rc;
    if (B > 0) {
        if (int rc = check_ptr(seqlens, 4, "seqlens")) return rc;
        if (int rc = check_ptr(parents, 4, "parents")) return rc;
    }
    p.seqlens = seqlens;
    p.parents = parents;
    p.moves = moves;
    return pages_launch(pages_fork_kernel, p, stream, "pages_fork_kernel launch");
}

extern "C" int gqa_pages_compact(int32_t *table, int32_t *refs, int32_t *moves, int B, int M,
                                 int n_pages, int page, void *workspace, size_t workspace_bytes,
                                 gqa_stream_t stream) {
    clear_error();
    PgParams p{};
    if (int rc = pages_setup(p, table, refs, B, M, n_pages, page, workspace, workspace_bytes)) return rc;
    if (int rc = check_ptr(moves, 4, "moves")) return rc;
    p.moves = moves;
    return pages_launch(pages_compact_kernel, p, stream, "pages_compact_kernel launch");
}
