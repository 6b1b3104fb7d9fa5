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
// Rows, table and pages are spread over the warps from three different starts, so that
// for small sizes each warp has one of them and their loads run side by side.
// Ranks come from ballots: every warp owns a contiguous range of pages, and one of
// the table, publishes its counts, and after the barrier all 256 counts are scanned
// by each CTA for itself.  The entry that needs the k-th page is listed under k, so
// that the warp that finds the k-th free page can hand it out without a further
// phase: two barriers a call.  Forking 256 rows of 128 slots took 16.0 us with five
// barriers, 11.0 us with two and 8.6 us with the loads side by side, 4 rows 10.9, 9.4
// and 6.2 us; freeing and taking the 4600 pages of 96 rows 15.1, 12.6 and 10.4 us.
#include <climits>

#include "cache8.cuh"

namespace gqa {

constexpr int kPgCtas = 8;                   // one portable cluster
constexpr int kPgThreads = 1024;
constexpr int kPgWarps = kPgCtas * kPgThreads / 32;

// Everything the cluster's threads wrote before is visible to its threads after
// (release and acquire at cluster scope, global memory included).
__device__ __forceinline__ void cluster_barrier() {
    __syncwarp();                             // the aligned form wants whole warps
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The contiguous range of [0, n) that warp gw owns, in multiples of `unit`.
struct PgRange {
    int begin, end;
    __device__ PgRange(int n, int unit, int gw) {
        const long long seg = (static_cast<long long>(n) + unit * kPgWarps - 1) / (unit * kPgWarps) * unit;
        begin = static_cast<int>(min(static_cast<long long>(n), seg * gw));
        end = static_cast<int>(min(static_cast<long long>(n), begin + seg));
    }
};

// Exclusive prefix sums of the 256 counts that the warps published, total in out[256];
// mine: count number threadIdx.x, loaded by the caller as early as it can.
__device__ __forceinline__ int published(const int *counts) {
    return threadIdx.x < kPgWarps ? __ldcg(counts + threadIdx.x) : 0;
}
__device__ __forceinline__ void pg_scan(int mine, int (&out)[kPgWarps + 1], int (&tmp)[8]) {
    const int t = threadIdx.x, lane = t & 31, w = t >> 5;
    int x = mine;
    if (t < kPgWarps) {
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += y;
        }
        if (lane == 31) tmp[w] = x;
    }
    __syncthreads();
    if (t < kPgWarps) {
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (i < w) x += tmp[i];
        out[t] = x - mine;
        if (t == kPgWarps - 1) out[kPgWarps] = x;
    }
    __syncthreads();
}

// Number of this warp among the cluster's, from the k-th of three starts.
__device__ __forceinline__ int pg_warp(int k) {
    const int w = static_cast<int>(threadIdx.x >> 5) * kPgCtas + blockIdx.x;
    return (w + k * (kPgWarps / 3)) % kPgWarps;
}

constexpr int kPgMaxForkRows = 49152;        // 192 KB of shared memory
constexpr int kPgSlots = 256;                // slots of a piece of a table row, 8 per lane

struct PgParams {
    int32_t *table, *refs, *seqlens;
    const int32_t *lengths, *parents;
    int32_t *moves;
    int B, M, n_pages, page;
    int row_pieces;                          // ceil(M / kPgSlots)
    int *status;
    // workspace
    int *count_a, *count_b;                  // one per warp
    int *list_a, *list_b, *list_c;           // lists of pages (n_pages) or table entries (B M)
    int *rows;                               // 8 B
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

// Free pages of a warp's range: counted, then handed out.
struct FreePages {
    PgRange r;
    int warp, count = 0;
    uint32_t first = 0;                       // the first 32 pages' free ones

    __device__ FreePages(const PgParams &p) : r(p.n_pages, 32, pg_warp(2)), warp(pg_warp(2)) {
        const int lane = threadIdx.x & 31;
        for (int i = r.begin; i < r.end; i += 32) {
            const uint32_t m = __ballot_sync(0xffffffffu, i + lane < r.end && ld(p.refs + i + lane) <= 0);
            if (i == r.begin) first = m;
            count += __popc(m);
        }
    }
    // hand(k, page) for the pool's k-th free page, k < want; rank: of this range's first
    template <class F>
    __device__ void hand_out(const PgParams &p, int rank, int want, F hand) const {
        const int lane = threadIdx.x & 31;
        for (int i = r.begin; i < r.end && rank < want; i += 32) {
            const uint32_t m = i == r.begin ? first
                                            : __ballot_sync(0xffffffffu, i + lane < r.end &&
                                                                             ld(p.refs + i + lane) <= 0);
            const int k = rank + __popc(m & ((1u << lane) - 1));
            if ((m >> lane & 1) && k < want) {
                p.refs[i + lane] = 1;
                hand(k, i + lane);
            }
            rank += __popc(m);
        }
    }
};

// Pages for the rows' lengths: entries at and past ceil(length / page) are
// released, missing ones below it get the lowest free pages.  list_a: the entry
// that needs the k-th page.
__global__ void __cluster_dims__(kPgCtas, 1, 1) __launch_bounds__(kPgThreads, 1)
pages_resize_kernel(const PgParams p) {
    dependents_may_launch();
    wait_for_stream();
    __shared__ int need[kPgWarps + 1], avail[kPgWarps + 1], tmp[8];
    const int lane = threadIdx.x & 31, gw = pg_warp(0);
    const PgRange r(p.B * p.row_pieces, 1, gw);
    constexpr int kPer = kPgSlots / 32;
    auto keep = [&](int b) {                  // slots that row b shall hold
        const int L = p.lengths[b];
        const int k = L <= 0 ? 0 : (L - 1) / p.page + 1;
        if (lane == 0 && (L < 0 || k > p.M)) record_status(p.status, GQA_ERR_INVALID_ARG);
        return min(k, p.M);
    };
    // piece i of the table: its row, first slot and entries (-1 past the row's end)
    int e[kPer];
    auto load = [&](int i, int &b, int &s0) {
        b = i / p.row_pieces;
        s0 = (i - b * p.row_pieces) * kPgSlots + lane;
        const int32_t *row = p.table + static_cast<size_t>(b) * p.M;
#pragma unroll
        for (int x = 0; x < kPer; ++x) e[x] = s0 + 32 * x < p.M ? row[s0 + 32 * x] : -1;
    };
    int count = 0;
    for (int i = r.begin; i < r.end; ++i) {
        int b, s0;
        load(i, b, s0);
        const int k = keep(b);
        int32_t *row = p.table + static_cast<size_t>(b) * p.M;
#pragma unroll
        for (int x = 0; x < kPer; ++x) {
            const int s = s0 + 32 * x, v = valid_page(e[x], p.n_pages, p.status);
            if (s >= k && v >= 0 && atomicSub(p.refs + v, 1) <= 0)
                record_status(p.status, GQA_ERR_INVALID_ARG);
            if (e[x] != -1 && (s >= k || v < 0)) row[s] = -1;
            count += __popc(__ballot_sync(0xffffffffu, s < k && v < 0));
        }
    }
    if (lane == 0) p.count_a[gw] = count;
    cluster_barrier();
    const int needed = published(p.count_a);
    const FreePages pages(p);
    if (lane == 0) p.count_b[pages.warp] = pages.count;
    pg_scan(needed, need, tmp);
    const int want = need[kPgWarps];
    if (want == 0) return;                    // the same for every CTA
    if (count > 0) {
        int rank = need[gw];
        for (int i = r.begin; i < r.end; ++i) {
            int b, s0;
            load(i, b, s0);                   // this warp's own range
            const int k = keep(b);
#pragma unroll
            for (int x = 0; x < kPer; ++x) {
                const int s = s0 + 32 * x;
                const bool w = s < k && e[x] < 0;
                const uint32_t m = __ballot_sync(0xffffffffu, w);
                if (w) p.list_a[rank + __popc(m & ((1u << lane) - 1))] = b * p.M + s;
                rank += __popc(m);
            }
        }
    }
    cluster_barrier();
    pg_scan(published(p.count_b), avail, tmp);
    if (want > avail[kPgWarps] && gw == 0 && lane == 0) record_status(p.status, GQA_ERR_PAGES);
    pages.hand_out(p, avail[pages.warp], want, [&](int k, int page) { p.table[ld(p.list_a + k)] = page; });
}

// New row b = old row parents[b].  needs: {row, its source page, its length, -} of the
// row that needs the k-th page; shared memory: per parent, the row that goes on in its
// last page.
__global__ void __cluster_dims__(kPgCtas, 1, 1) __launch_bounds__(kPgThreads, 1)
pages_fork_kernel(const PgParams p) {
    dependents_may_launch();
    wait_for_stream();
    extern __shared__ int heir[];
    __shared__ int need[kPgWarps + 1], avail[kPgWarps + 1], tmp[8];
    const int lane = threadIdx.x & 31;
    auto parent = [&](int b) {
        const int x = p.parents[b];
        return x >= 0 && x < p.B ? x : -1;
    };
    // the parent's own row goes on in its last page, else its first child does
    for (int b = threadIdx.x; b < p.B; b += kPgThreads) heir[b] = INT_MAX;
    __syncthreads();
    for (int b = threadIdx.x; b < p.B; b += kPgThreads) {
        const int x = parent(b);
        if (x >= 0) atomicMin(heir + x, x == b ? -1 : b);
        if (p.parents[b] >= p.B) record_status(p.status, GQA_ERR_INVALID_ARG);
    }
    __syncthreads();
    auto full_slots = [&](int b, int x) {     // slots that row b takes over from row x
        return x < 0 ? 0 : (heir[x] == b ? p.M : max(0, p.seqlens[x]) / p.page);
    };
    // new lengths, and which rows need a page for a copy of the last one
    const int row_warp = pg_warp(1);
    const PgRange rb(p.B, 1, row_warp);
    int count = 0, src = -1, L = 0;           // of this lane's last row
    for (int i = rb.begin; i < rb.end; i += 32) {
        src = -1;
        if (i + lane < rb.end) {
            const int b = i + lane, x = parent(b);
            L = x >= 0 ? p.seqlens[x] : 0;
            if (L < 0 || L > p.M * p.page) {
                record_status(p.status, GQA_ERR_INVALID_ARG);
                L = L < 0 ? 0 : p.M * p.page;
            }
            if (x >= 0 && x != b && heir[x] != b && L % p.page > 0) {
                src = valid_page(p.table[static_cast<size_t>(x) * p.M + L / p.page], p.n_pages, p.status);
                if (src < 0) record_status(p.status, GQA_ERR_INVALID_ARG);
            }
            p.rows[b] = L;
            p.rows[p.B + b] = src;
        }
        count += __popc(__ballot_sync(0xffffffffu, src >= 0));
    }
    if (lane == 0) p.count_a[row_warp] = count;
    // new rows, and the references that changed rows drop and gain
    const PgRange r(p.B * p.row_pieces, 1, pg_warp(0));
    constexpr int kPer = kPgSlots / 32;
    int now[kPer] = {};                       // of the last piece
    for (int i = r.begin; i < r.end; ++i) {
        const int b = i / p.row_pieces, s0 = (i - b * p.row_pieces) * kPgSlots + lane, x = parent(b);
        if (x == b) continue;
        const size_t to = static_cast<size_t>(b) * p.M, from = static_cast<size_t>(max(x, 0)) * p.M;
        const int full = full_slots(b, x);
        int old[kPer];
#pragma unroll
        for (int y = 0; y < kPer; ++y) {
            const int s = s0 + 32 * y;
            old[y] = s < p.M ? p.table[to + s] : -1;
            now[y] = s < p.M && s < full ? p.table[from + s] : -1;
        }
#pragma unroll
        for (int y = 0; y < kPer; ++y) {
            const int s = s0 + 32 * y, off = valid_page(old[y], p.n_pages, p.status);
            now[y] = valid_page(now[y], p.n_pages, p.status);
            if (now[y] != off) {
                if (off >= 0) atomicSub(p.refs + off, 1);
                if (now[y] >= 0) atomicAdd(p.refs + now[y], 1);
            }
            if (s < p.M && i + 1 < r.end) p.entries[to + s] = now[y];
        }
    }
    cluster_barrier();
    const int needed = published(p.count_a);
    const FreePages pages(p);
    if (lane == 0) p.count_b[pages.warp] = pages.count;
    pg_scan(needed, need, tmp);
    const int want = need[kPgWarps];
    int4 *needs = reinterpret_cast<int4 *>(p.rows + 4 * static_cast<size_t>(p.B));
    if (count > 0) {
        int rank = need[row_warp];
        for (int i = rb.begin; i < rb.end; i += 32) {
            const int b = i + lane;
            if (rb.end - rb.begin > 32) {     // this warp's own rows
                src = b < rb.end ? p.rows[p.B + b] : -1;
                L = b < rb.end ? p.rows[b] : 0;
            }
            const uint32_t m = __ballot_sync(0xffffffffu, src >= 0);
            if (src >= 0) needs[rank + __popc(m & ((1u << lane) - 1))] = make_int4(b, src, L, 0);
            rank += __popc(m);
        }
    }
    // rows without a page of their own to come: the table (every old row has been read)
    for (int i = r.begin; i < r.end; ++i) {
        const int b = i / p.row_pieces, s0 = (i - b * p.row_pieces) * kPgSlots + lane, x = parent(b);
        if (x == b) continue;
#pragma unroll
        for (int y = 0; y < kPer; ++y) {
            const int s = s0 + 32 * y;
            if (s < p.M)
                p.table[static_cast<size_t>(b) * p.M + s] =
                    i + 1 < r.end ? p.entries[static_cast<size_t>(b) * p.M + s] : now[y];
        }
    }
    cluster_barrier();
    pg_scan(published(p.count_b), avail, tmp);
    const int have = min(want, avail[kPgWarps]);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        p.moves[0] = have;
        p.moves[1] = p.moves[2] = 0;
        if (want > have) record_status(p.status, GQA_ERR_PAGES);
    }
    pages.hand_out(p, avail[pages.warp], want, [&](int k, int page) {
        const int4 n = __ldcg(needs + k);
        p.table[static_cast<size_t>(n.x) * p.M + n.z / p.page] = page;
        p.moves[3 * (1 + k)] = n.y;
        p.moves[3 * (1 + k) + 1] = page;
        p.moves[3 * (1 + k) + 2] = n.z % p.page;
    });
    for (int i = rb.begin + lane; i < rb.end; i += 32)
        p.seqlens[i] = rb.end - rb.begin > 32 ? p.rows[i] : L;
}

// Used pages at and past their number move, in order, to the free pages below it.
__global__ void __cluster_dims__(kPgCtas, 1, 1) __launch_bounds__(kPgThreads, 1)
pages_compact_kernel(const PgParams p) {
    dependents_may_launch();
    wait_for_stream();
    __shared__ int used[kPgWarps + 1], tmp[8], s_below;
    const int lane = threadIdx.x & 31;
    const int gt = threadIdx.x * kPgCtas + blockIdx.x;
    const FreePages pages(p);
    const PgRange r = pages.r;
    if (lane == 0) p.count_a[pages.warp] = r.end - r.begin - pages.count;
    cluster_barrier();
    pg_scan(published(p.count_a), used, tmp);
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
    int rank = used[pages.warp];
    for (int i = r.begin; i < r.end; i += 32) {
        const int id = i + lane;
        const bool in = id < r.end;
        const bool u = in && (i == r.begin ? !(pages.first >> lane & 1) : ld(p.refs + id) > 0);
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
    const PgRange rt(p.B * p.row_pieces, 1, pg_warp(0));
    for (int i = rt.begin; i < rt.end; ++i) {
        const int b = i / p.row_pieces, s0 = (i - b * p.row_pieces) * kPgSlots + lane;
        int32_t *row = p.table + static_cast<size_t>(b) * p.M;
        int e[kPgSlots / 32];
#pragma unroll
        for (int x = 0; x < kPgSlots / 32; ++x) e[x] = s0 + 32 * x < p.M ? row[s0 + 32 * x] : -1;
#pragma unroll
        for (int x = 0; x < kPgSlots / 32; ++x) {
            if (valid_page(e[x], p.n_pages, p.status) < n_used) continue;
            const int k = ld(p.list_c + e[x]);
            if (k >= 0) row[s0 + 32 * x] = ld(p.list_a + k);
            else record_status(p.status, GQA_ERR_INVALID_ARG);   // an entry without a reference
        }
    }
}

static size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Workspace: counts of 2 x 256 warps | 8 ints per row | as many ints as the table has
// entries (entries, or the list of those that need a page) | 3 lists of pages.
struct PgWorkspace {
    size_t off_rows, off_entries, off_lists, list, bytes;
    PgWorkspace(int B, int M, int n_pages) {
        off_rows = 2 * kPgWarps * sizeof(int);
        off_entries = off_rows + align256(8 * static_cast<size_t>(B) * sizeof(int));
        off_lists = off_entries + align256(static_cast<size_t>(B) * M * sizeof(int));
        list = align256(static_cast<size_t>(n_pages) * sizeof(int));
        bytes = off_lists + 3 * list;
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
    p.row_pieces = (M + kPgSlots - 1) / kPgSlots;
    p.list_a = reinterpret_cast<int *>(base + ws.off_lists);
    p.list_b = reinterpret_cast<int *>(base + ws.off_lists + ws.list);
    p.list_c = reinterpret_cast<int *>(base + ws.off_lists + 2 * ws.list);
    p.entries = reinterpret_cast<int *>(base + ws.off_entries);
    return GQA_OK;
}

static int pages_launch(void (*kern)(PgParams), PgParams &p, size_t smem, gqa_stream_t stream,
                        const char *what) {
    if (int rc = require_sm100()) return rc;
    p.status = device_status_ptr();
    if (!p.status) return GQA_ERR_CUDA;
    return launch_dependent(kern, kPgCtas, kPgThreads, smem, reinterpret_cast<cudaStream_t>(stream), what, p);
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
    p.list_a = p.entries;                    // one place per table entry
    return pages_launch(pages_resize_kernel, p, 0, stream, "pages_resize_kernel launch");
}

extern "C" int gqa_pages_fork(int32_t *table, int32_t *refs, int32_t *seqlens, const int32_t *parents,
                              int32_t *moves, int B, int M, int n_pages, int page, void *workspace,
                              size_t workspace_bytes, gqa_stream_t stream) {
    clear_error();
    PgParams p{};
    if (int rc = pages_setup(p, table, refs, B, M, n_pages, page, workspace, workspace_bytes)) return rc;
    if (B > kPgMaxForkRows)
        return set_error(GQA_ERR_UNSUPPORTED, "pages_fork: B=%d rows exceed %d", B, kPgMaxForkRows);
    if (int rc = check_ptr(moves, 4, "moves")) return rc;
    if (B > 0) {
        if (int rc = check_ptr(seqlens, 4, "seqlens")) return rc;
        if (int rc = check_ptr(parents, 4, "parents")) return rc;
    }
    p.seqlens = seqlens;
    p.parents = parents;
    p.moves = moves;
    const size_t smem = static_cast<size_t>(B) * sizeof(int);
    static CtxSlot setup;
    if (int rc = require_sm100()) return rc;
    if (int rc = once_per_context(setup, [&](int) {
            return check_cuda(cudaFuncSetAttribute(pages_fork_kernel,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   kPgMaxForkRows * sizeof(int)),
                              "cudaFuncSetAttribute(pages_fork)");
        }))
        return rc;
    return pages_launch(pages_fork_kernel, p, smem, stream, "pages_fork_kernel launch");
}

extern "C" int gqa_pages_compact(int32_t *table, int32_t *refs, int32_t *moves, int B, int M,
                                 int n_pages, int page, void *workspace, size_t workspace_bytes,
                                 gqa_stream_t stream) {
    clear_error();
    PgParams p{};
    if (int rc = pages_setup(p, table, refs, B, M, n_pages, page, workspace, workspace_bytes)) return rc;
    if (int rc = check_ptr(moves, 4, "moves")) return rc;
    p.moves = moves;
    return pages_launch(pages_compact_kernel, p, 0, stream, "pages_compact_kernel launch");
}
