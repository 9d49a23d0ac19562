// kvp.cu -- bookkeeping of the paged KV cache on the device: reserving, forking and
// freeing, compacting (include/kvcache.h).  All results are whole numbers and do
// not depend on the order in which threads run: counts are integer atomics, free
// pages go out lowest id first.
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/kvcache.h"
#include "attn_internal.h"
#include "ptx.cuh"

namespace tme {

int device_setup_public(unsigned int** status);   // abi.cu

namespace {

// The planning kernels run as one CTA: they are chains of a few scans, bound by latency
// (reserve: 3.9 us at 512 pages, 40 us at 65537 pages; times in this file are in a graph).
constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
// The planning's steps depend on one another through the pages' counts, the list of
// free ids and a few numbers per sequence, and each step costs a round trip of the
// memory those are in: they live in shared memory up to this many bytes (2 ints a
// page, 5 a sequence, reassign's rows beside them when they fit, too), in the
// workspace past it.  A fork of 64 sequences over 2049 pages, its copies included:
// 11.7 us against 14.5; of 96 over 19201 pages: 18.9 against 31.8.
constexpr size_t kSharedBytes = 200 * 1024;
// Table entries that compact's planning CTA renumbers itself; more take a second
// kernel (2304 entries 7.2 us against 8.3, 16K 19.1 against 19.5, 64K 91.7 against
// 89.1).
constexpr int64_t kRemapEntries = 16 * 1024;

struct PageParams {
    int* table;
    int* lens;
    int* refs;
    const int* arg;        // n_new or parents
    int* src;              // pairs to copy
    int* dst;
    int* info;
    int* granted;          // reserve: info[0] again, or null
    unsigned int* status;
    int* scratch;          // workspace: scratch_ints() (when not in shared memory)
    int* ids;              // workspace: new id of each page (compact's second kernel)
    int* table2;           // workspace [n_seqs][max_pages]
    const int* table_in;   // compact
    const int* refs_in;
    int n_seqs, max_pages, n_pages, page, window, sinks;
};

size_t scratch_ints(int n_seqs, int n_pages) {
    return 2 * static_cast<size_t>(n_pages) + 5 * static_cast<size_t>(n_seqs);
}

// The planning's working arrays.
template <bool SHARED>
struct Scratch {
    int* count;    // [n_pages] holders of each page after the call
    int* ids;      // [n_pages] free ids, lowest first; compact: new ids
    int* len;      // [n_seqs]
    int* arg;      // [n_seqs] tokens to add, or parent
    int* keeper;   // [n_seqs]
    int* base;     // [n_seqs]
    int* tail;     // [n_seqs]
    __device__ __forceinline__ explicit Scratch(const PageParams& p) {
        extern __shared__ int s_scratch[];
        count = SHARED ? s_scratch : p.scratch;
        ids = count + p.n_pages;
        len = ids + p.n_pages;
        arg = len + p.n_seqs;
        keeper = arg + p.n_seqs;
        base = keeper + p.n_seqs;
        tail = base + p.n_seqs;
    }
    // What atomics of this CTA change is read past the first-level cache.
    __device__ __forceinline__ static int get(const int* p) { return SHARED ? *p : __ldcg(p); }
};

// Exclusive prefix sum of one value per thread over the CTA, and the total.
__device__ __forceinline__ int block_scan(int x, int* total) {
    __shared__ int s[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += y;
    }
    __syncthreads();   // the previous call's readers are done with s
    if (lane == 31) s[warp] = inc;
    __syncthreads();
    const int w = s[lane];
    int winc = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, winc, d);
        if (lane >= d) winc += y;
    }
    *total = __shfl_sync(0xffffffffu, winc, 31);
    return __shfl_sync(0xffffffffu, winc - w, warp) + inc - x;
}

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

__device__ __forceinline__ bool in_pool(const PageParams& p, int id) {
    return id >= 0 && id < p.n_pages;
}

// Calls f(i, refs[i]) for every page, 8 loads of a thread in flight.
template <typename F>
__device__ __forceinline__ void for_pages(const PageParams& p, const int* refs, F&& f) {
    for (int i0 = 0; i0 < p.n_pages; i0 += 8 * kThreads) {
        int r[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int i = i0 + k * kThreads + static_cast<int>(threadIdx.x);
            r[k] = i < p.n_pages ? __ldcg(refs + i) : 0;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int i = i0 + k * kThreads + static_cast<int>(threadIdx.x);
            if (i < p.n_pages) f(i, r[k]);
        }
    }
}

// Loads the counts; returns how many pages are free (after a barrier).
template <bool SHARED>
__device__ int load_counts(const PageParams& p, const Scratch<SHARED>& m, const int* refs) {
    int free = 0;
    for_pages(p, refs, [&](int i, int r) {
        m.count[i] = r;
        free += r == 0;
    });
    int total;
    block_scan(free, &total);
    return total;
}

// Writes the counts back.
template <bool SHARED>
__device__ void store_counts(const PageParams& p, const Scratch<SHARED>& m) {
    if constexpr (SHARED) {
        for (int i = threadIdx.x; i < p.n_pages; i += kThreads) p.refs[i] = m.count[i];
    } else {
        for_pages(p, m.count, [&](int i, int r) { p.refs[i] = r; });
    }
}

// Lists the lowest `want` free ids in order; returns how many there are in all.  16
// pages a thread and step (4 in shared memory, whose pools are smaller).
template <bool SHARED>
__device__ int list_free(const PageParams& p, const Scratch<SHARED>& m, int want) {
    constexpr int K = SHARED ? 4 : 16;
    int n = 0;
    for (int i0 = 0; i0 < p.n_pages; i0 += K * kThreads) {
        const int i = i0 + K * static_cast<int>(threadIdx.x);
        int r[K], mine = 0;
#pragma unroll
        for (int k = 0; k < K; ++k) r[k] = i + k < p.n_pages ? m.get(m.count + i + k) : 1;
#pragma unroll
        for (int k = 0; k < K; ++k) mine += r[k] == 0;
        int total;
        int at = n + block_scan(mine, &total);
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (r[k] == 0) {
                if (at < want) m.ids[at] = i + k;
                ++at;
            }
        n += total;
    }
    __syncthreads();
    return n;
}

template <bool SHARED>
__global__ void __launch_bounds__(kThreads) kvp_reserve_kernel(const PageParams p) {
    const Scratch<SHARED> m(p);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    __shared__ int s_bad;
    if (tid == 0) s_bad = 0;
    for (int c = tid; c < p.n_seqs; c += kThreads) {
        m.len[c] = p.lens[c];
        m.arg[c] = p.arg[c];
    }
    const int before = load_counts(p, m, p.refs);
    // pages each sequence needs
    const int64_t cap = static_cast<int64_t>(p.max_pages) * p.page;
    int need = 0;
    for (int c0 = 0; c0 < p.n_seqs; c0 += kThreads) {
        const int c = c0 + tid;
        int want = 0;
        if (c < p.n_seqs) {
            const int len = m.len[c];
            int n = m.arg[c];
            if (n < 0 || len < 0) {
                atomicOr(p.status, kStatusPage);
                n = 0;
            }
            if (n > 0 && static_cast<int64_t>(len) + n > cap) {
                s_bad = 1;
                n = 0;
            }
            m.arg[c] = n;
            want = n > 0 ? ceil_div(len + n, p.page) - ceil_div(len, p.page) : 0;
        }
        int total;
        const int at = block_scan(want, &total);
        if (c < p.n_seqs) m.base[c] = need + at;
        need += total;
    }
    __syncthreads();
    // pages that windows leave behind: columns [j0, j1), which no later query sees
    const int j0 = ceil_div(p.sinks, p.page);
    auto past = [&](int c) {
        if (p.window <= 0 || m.arg[c] <= 0) return 0;
        const int first = m.len[c] - p.window + 1;   // first position a new query sees
        return min(first > 0 ? first / p.page : 0, p.max_pages);
    };
    // Calls f(column, page) for those still held, from the newest down to the first
    // 32 columns that an earlier call has dealt with.
    auto leave = [&](int c, auto&& f) {
        const int* row = p.table + static_cast<int64_t>(c) * p.max_pages;
        for (int j1 = past(c); j1 > j0; j1 -= 32) {
            const int j = j1 - 32 + lane;
            const int id = j >= j0 ? row[j] : -1;
            if (in_pool(p, id)) f(j, id);
            if (__any_sync(0xffffffffu, !in_pool(p, id))) break;
        }
    };
    if (p.window > 0) {
        for (int c = warp; c < p.n_seqs; c += kWarps)
            leave(c, [&](int, int id) { atomicSub(m.count + id, 1); });
        __syncthreads();
    }
    const int free = list_free(p, m, need);
    const bool done = s_bad == 0 && need <= free;
    if (tid == 0) {
        p.info[0] = done;
        if (p.granted) *p.granted = done;
        p.info[1] = done ? need : 0;
        p.info[2] = done ? free - before : 0;
        p.info[3] = done ? free - need : before;
        if (!done) atomicOr(p.status, kStatusPool);
    }
    if (!done) return;
    for (int c = warp; c < p.n_seqs; c += kWarps) {
        int* row = p.table + static_cast<int64_t>(c) * p.max_pages;
        leave(c, [&](int j, int) { row[j] = -1; });
        const int len = m.len[c], n = m.arg[c];
        if (n > 0) {
            const int first = ceil_div(len, p.page), want = ceil_div(len + n, p.page) - first;
            for (int k = lane; k < want; k += 32) {
                const int id = m.ids[m.base[c] + k];
                row[first + k] = id;
                atomicExch(m.count + id, 1);
            }
            if (lane == 0) p.lens[c] = len + n;
        }
    }
    __syncthreads();
    store_counts(p, m);
}

template <bool SHARED>
__global__ void __launch_bounds__(kThreads) kvp_reassign_kernel(const PageParams p, bool rows_shared) {
    asm volatile("griddepcontrol.launch_dependents;");   // the copies may set up meanwhile
    const Scratch<SHARED> m(p);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int* table2 = SHARED && rows_shared ? m.tail + p.n_seqs : p.table2;
    const int cap = p.max_pages * p.page;
    for (int c = tid; c < p.n_seqs; c += kThreads) {
        int q = p.arg[c];
        if (q < -1 || q >= p.n_seqs) {   // a bad parent keeps the sequence
            atomicOr(p.status, kStatusPage);
            q = c;
        }
        m.arg[c] = q;
        m.len[c] = min(max(p.lens[c], 0), cap);
        m.keeper[c] = 0x7fffffff;
    }
    const int before = load_counts(p, m, p.refs);
    for (int c = tid; c < p.n_seqs; c += kThreads) {
        const int q = m.arg[c];
        if (q >= 0) atomicMin(m.keeper + q, q == c ? -1 : c);
    }
    __syncthreads();
    // Children that do not keep their parent's partly filled last page copy it.
    int n_copy = 0;
    for (int c0 = 0; c0 < p.n_seqs; c0 += kThreads) {
        const int c = c0 + tid;
        int tail = -1;
        if (c < p.n_seqs) {
            const int q = m.arg[c];
            if (q >= 0 && q != c && m.len[q] % p.page != 0 && m.get(m.keeper + q) != c) {
                const int j = m.len[q] / p.page;
                if (in_pool(p, p.table[static_cast<int64_t>(q) * p.max_pages + j])) tail = j;
            }
            m.tail[c] = tail;
        }
        int total;
        const int at = block_scan(tail >= 0 ? 1 : 0, &total);
        if (c < p.n_seqs) m.base[c] = n_copy + at;
        n_copy += total;
    }
    __syncthreads();
    // New rows of the changed sequences aside, and the counts they leave.
    auto columns = [&](int c, int* had, int* has) {
        const int q = m.arg[c];
        *had = ceil_div(m.len[c], p.page);
        *has = q >= 0 ? ceil_div(m.len[q], p.page) : 0;
        return max(*had, *has);
    };
    for (int c = warp; c < p.n_seqs; c += kWarps) {
        const int q = m.arg[c];
        if (q == c) continue;
        int had, has;
        const int cols = columns(c, &had, &has);
        const int tail = m.tail[c];
        const int64_t row = static_cast<int64_t>(c) * p.max_pages;
        const int64_t from = static_cast<int64_t>(q) * p.max_pages;
        for (int j = lane; j < cols; j += 32) {
            const int old = j < had ? p.table[row + j] : -1;
            const int id = j < has ? p.table[from + j] : -1;
            if (in_pool(p, old)) atomicSub(m.count + old, 1);
            if (in_pool(p, id) && j != tail) atomicAdd(m.count + id, 1);
            table2[row + j] = id;
        }
    }
    __syncthreads();
    const int free = list_free(p, m, n_copy);
    const bool done = n_copy <= free;
    if (tid == 0) {
        p.info[0] = done;
        p.info[1] = done ? n_copy : 0;
        p.info[2] = done ? free - before : 0;
        p.info[3] = done ? free - n_copy : before;
        if (!done) atomicOr(p.status, kStatusPool);
    }
    if (!done) return;
    for (int c = warp; c < p.n_seqs; c += kWarps) {
        const int q = m.arg[c];
        if (q == c) continue;
        int had, has;
        const int cols = columns(c, &had, &has);
        const int tail = m.tail[c], at = m.base[c];
        const int64_t row = static_cast<int64_t>(c) * p.max_pages;
        for (int j = lane; j < cols; j += 32) {
            int id = table2[row + j];   // this lane wrote it
            if (j == tail) {
                p.src[at] = id;
                id = m.ids[at];
                p.dst[at] = id;
                atomicExch(m.count + id, 1);
            }
            p.table[row + j] = id;
        }
        if (lane == 0) p.lens[c] = q >= 0 ? m.len[q] : 0;
    }
    __syncthreads();
    store_counts(p, m);
}

// New ids of the held pages (ids: -1 not held, the page itself, or the free id it
// moves to), refs_out, the moves and, for a small table, table_out.
template <bool SHARED>
__global__ void __launch_bounds__(kThreads) kvp_compact_kernel(const PageParams p, int64_t entries) {
    asm volatile("griddepcontrol.launch_dependents;");   // what follows may set up meanwhile
    const Scratch<SHARED> m(p);
    const int tid = threadIdx.x;
    int held = 0;
    for_pages(p, p.refs_in, [&](int i, int r) {
        m.count[i] = r;
        held += r > 0;
    });
    int total;
    block_scan(held, &total);
    held = total;
    // holes below `held` and pages past it, each in order; both counts of a step
    // travel in one scan (at most 4 * 1024 each, 16 bits)
    int holes = 0, movers = 0;
    for (int i0 = 0; i0 < p.n_pages; i0 += 4 * kThreads) {
        const int i = i0 + 4 * tid;
        int kind[4], mine = 0;   // 0, 1 a hole, 1 << 16 a mover
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const bool in = i + k < p.n_pages;
            const int r = in ? m.count[i + k] : 0;
            kind[k] = !in ? 0 : i + k < held ? (r > 0 ? 0 : 1) : (r > 0 ? 1 << 16 : 0);
            mine += kind[k];
        }
        int both;
        const int at = block_scan(mine, &both);
        int h = holes + (at & 0xffff), v = movers + (at >> 16);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (kind[k] == 1) p.dst[h++] = i + k;
            if (kind[k] > 1) p.src[v++] = i + k;
        }
        holes += both & 0xffff;
        movers += both >> 16;
    }
    __syncthreads();
    for (int i = tid; i < p.n_pages; i += kThreads) {
        const int r = m.count[i];
        m.ids[i] = r > 0 ? i : -1;
        p.refs[i] = i < held && r > 0 ? r : 0;
    }
    __syncthreads();
    for (int k = tid; k < movers; k += kThreads) {   // as many holes as movers
        const int from = p.src[k], to = p.dst[k];
        m.ids[from] = to;
        p.refs[to] = m.count[from];
    }
    if (tid == 0) {
        p.info[0] = 1;
        p.info[1] = movers;
        p.info[2] = held;
        p.info[3] = p.n_pages - held;
    }
    __syncthreads();
    if (entries <= kRemapEntries) {
        for (int i = tid; i < static_cast<int>(entries); i += kThreads) {
            const int id = p.table_in[i];
            p.table[i] = in_pool(p, id) ? m.ids[id] : id;
        }
    } else {
        for (int i = tid; i < p.n_pages; i += kThreads) p.ids[i] = m.ids[i];
    }
}

__global__ void __launch_bounds__(256) kvp_remap_kernel(const PageParams p, int64_t n) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= n) return;
    const int id = p.table_in[i];
    p.table[i] = in_pool(p, id) ? p.ids[id] : id;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
size_t pad256(size_t b) { return (b + 255) & ~size_t(255); }

int check_pages(int n_seqs, int max_pages, int n_pages) {
    if (n_seqs <= 0 || max_pages <= 0 || n_pages <= 0) return ATTN_ERR_INVALID;
    if (static_cast<int64_t>(n_seqs) * max_pages > (1ll << 30) || n_pages > (1 << 30))
        return ATTN_ERR_UNSUPPORTED;
    return ATTN_OK;
}

// Lays the workspace out; ws may be null (the size alone).
size_t lay_out(PageParams* p, void* ws, int n_seqs, int max_pages, int n_pages) {
    char* at = static_cast<char*>(ws);
    size_t off = 0;
    auto take = [&](int** ptr, size_t n) {
        *ptr = ws ? reinterpret_cast<int*>(at + off) : nullptr;
        off += pad256(n * sizeof(int));
    };
    take(&p->scratch, scratch_ints(n_seqs, n_pages));
    take(&p->ids, n_pages);
    take(&p->table2, static_cast<size_t>(n_seqs) * max_pages);
    return off;
}

// Launches a planning kernel: `shared` when its working arrays fit shared memory.
template <typename... Args>
cudaError_t launch_plan(SmemLimit& limit, void (*shared)(Args...), void (*global)(Args...),
                        const PageParams& p, size_t more, cudaStream_t stream, Args... args) {
    const size_t bytes = scratch_ints(p.n_seqs, p.n_pages) * sizeof(int) + more;
    if (bytes > kSharedBytes) return launch_kernel(global, dim3(1), dim3(kThreads), 0, stream, args...);
    const cudaError_t e = limit.raise(shared, static_cast<int>(kSharedBytes));
    if (e != cudaSuccess) return e;
    return launch_kernel(shared, dim3(1), dim3(kThreads), bytes, stream, args...);
}

int prepare(PageParams* p, void* ws, size_t bytes, int n_seqs, int max_pages, int n_pages) {
    const int rc = check_pages(n_seqs, max_pages, n_pages);
    if (rc != ATTN_OK) return rc;
    if (!ws) return ATTN_ERR_INVALID;
    if (!aligned16(ws)) return ATTN_ERR_ALIGN;
    if (bytes < lay_out(p, ws, n_seqs, max_pages, n_pages)) return ATTN_ERR_WORKSPACE;
    p->n_seqs = n_seqs;
    p->max_pages = max_pages;
    p->n_pages = n_pages;
    return device_setup_public(&p->status);
}

bool page_ok(int page) { return page == 16 || page == 32 || page == 64 || page == 128; }

}  // namespace
}  // namespace tme

using namespace tme;

extern "C" size_t kvp_workspace_size(int n_seqs, int max_pages, int n_pages) {
    if (check_pages(n_seqs, max_pages, n_pages) != ATTN_OK) return 0;
    PageParams p{};
    return lay_out(&p, nullptr, n_seqs, max_pages, n_pages);
}

extern "C" int kvp_reserve(int* table, int* lens, int* refs, const int* n_new, int n_seqs,
                           int max_pages, int n_pages, int page, int window, int sinks, int* info,
                           void* workspace, size_t workspace_bytes, void* stream) {
    return kvp_reserve_step(table, lens, refs, n_new, n_seqs, max_pages, n_pages, page, window, sinks,
                            info, nullptr, workspace, workspace_bytes, stream);
}

extern "C" int kvp_reserve_step(int* table, int* lens, int* refs, const int* n_new, int n_seqs,
                                int max_pages, int n_pages, int page, int window, int sinks,
                                int* info, int* granted, void* workspace, size_t workspace_bytes,
                                void* stream) {
    if (!table || !lens || !refs || !n_new || !info) return ATTN_ERR_INVALID;
    if (window < 0 || sinks < 0) return ATTN_ERR_INVALID;
    if (!page_ok(page)) return page <= 0 ? ATTN_ERR_INVALID : ATTN_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(max_pages) * page > (1ll << 30)) return ATTN_ERR_UNSUPPORTED;
    const void* ptrs[] = {table, lens, refs, n_new, info, granted};
    for (const void* ptr : ptrs)
        if (!aligned4(ptr)) return ATTN_ERR_ALIGN;
    PageParams p{};
    const int rc = prepare(&p, workspace, workspace_bytes, n_seqs, max_pages, n_pages);
    if (rc != ATTN_OK) return rc;
    p.table = table;
    p.lens = lens;
    p.refs = refs;
    p.arg = n_new;
    p.info = info;
    p.granted = granted;
    p.page = page;
    // no position is past 2^30: larger ones mean all of them
    p.window = window > (1 << 30) ? 1 << 30 : window;
    p.sinks = sinks > (1 << 30) ? 1 << 30 : sinks;
    static SmemLimit limit;
    return launch_plan(limit, kvp_reserve_kernel<true>, kvp_reserve_kernel<false>, p, 0,
                       static_cast<cudaStream_t>(stream), p) == cudaSuccess
               ? ATTN_OK
               : ATTN_ERR_CUDA;
}

extern "C" int kvp_reassign(int* table, int* lens, int* refs, const int* parents, int n_seqs,
                            int max_pages, int n_pages, int page, int* copy_src, int* copy_dst,
                            int* info, void* workspace, size_t workspace_bytes, void* stream) {
    if (!table || !lens || !refs || !parents || !copy_src || !copy_dst || !info)
        return ATTN_ERR_INVALID;
    if (!page_ok(page)) return page <= 0 ? ATTN_ERR_INVALID : ATTN_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(max_pages) * page > (1ll << 30)) return ATTN_ERR_UNSUPPORTED;
    const void* ptrs[] = {table, lens, refs, parents, copy_src, copy_dst, info};
    for (const void* ptr : ptrs)
        if (!aligned4(ptr)) return ATTN_ERR_ALIGN;
    PageParams p{};
    const int rc = prepare(&p, workspace, workspace_bytes, n_seqs, max_pages, n_pages);
    if (rc != ATTN_OK) return rc;
    p.table = table;
    p.lens = lens;
    p.refs = refs;
    p.arg = parents;
    p.src = copy_src;
    p.dst = copy_dst;
    p.info = info;
    p.page = page;
    const size_t rows = static_cast<size_t>(n_seqs) * max_pages * sizeof(int);
    const bool rows_shared = scratch_ints(n_seqs, n_pages) * sizeof(int) + rows <= kSharedBytes;
    static SmemLimit limit;
    return launch_plan(limit, kvp_reassign_kernel<true>, kvp_reassign_kernel<false>, p,
                       rows_shared ? rows : 0, static_cast<cudaStream_t>(stream), p, rows_shared) == cudaSuccess
               ? ATTN_OK
               : ATTN_ERR_CUDA;
}

extern "C" int kvp_compact(const int* table, const int* refs, int* table_out, int* refs_out,
                           int n_seqs, int max_pages, int n_pages, int* move_src, int* move_dst,
                           int* info, void* workspace, size_t workspace_bytes, void* stream) {
    if (!table || !refs || !table_out || !refs_out || !move_src || !move_dst || !info)
        return ATTN_ERR_INVALID;
    const void* ptrs[] = {table, refs, table_out, refs_out, move_src, move_dst, info};
    for (const void* ptr : ptrs)
        if (!aligned4(ptr)) return ATTN_ERR_ALIGN;
    PageParams p{};
    const int rc = prepare(&p, workspace, workspace_bytes, n_seqs, max_pages, n_pages);
    if (rc != ATTN_OK) return rc;
    p.table_in = table;
    p.refs_in = refs;
    p.table = table_out;
    p.refs = refs_out;
    p.src = move_src;
    p.dst = move_dst;
    p.info = info;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int64_t n = static_cast<int64_t>(n_seqs) * max_pages;
    static SmemLimit limit;
    cudaError_t e = launch_plan(limit, kvp_compact_kernel<true>, kvp_compact_kernel<false>, p, 0, st, p, n);
    if (e == cudaSuccess && n > kRemapEntries)
        e = launch_dependent(kvp_remap_kernel, (n + 255) / 256, 256, 0, st, p, n);
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}
