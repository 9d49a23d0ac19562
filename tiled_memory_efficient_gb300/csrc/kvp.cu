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

constexpr int kThreads = 1024;   // the planning kernels run as one CTA

struct PageParams {
    int* table;
    int* lens;
    int* refs;
    const int* arg;        // n_new or parents
    int* src;              // pairs to copy
    int* dst;
    int* info;
    unsigned int* status;
    int* refs2;            // workspace: refs after the call [n_pages]
    int* ids;              // workspace: free ids, lowest first [n_pages]; compact: new id of a page
    int* keeper;           // workspace [n_seqs]
    int* base;             // workspace [n_seqs]
    int* tail;             // workspace [n_seqs]
    int* new_len;          // workspace [n_seqs]
    int* table2;           // workspace [n_seqs][max_pages]
    const int* table_in;   // compact
    const int* refs_in;
    int n_seqs, max_pages, n_pages, page, window, sinks;
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

__device__ __forceinline__ int block_sum(int x) {
    int total;
    block_scan(x, &total);
    return total;
}

// Counters that atomics of this CTA change are read past the first-level cache.
__device__ __forceinline__ int counter(const int* p) { return __ldcg(p); }

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Lists the free ids (refs2 = 0) in order; returns how many there are.
__device__ int list_free(const PageParams& p) {
    int count = 0;
    for (int i0 = 0; i0 < p.n_pages; i0 += kThreads) {
        const int i = i0 + static_cast<int>(threadIdx.x);
        const bool free = i < p.n_pages && counter(p.refs2 + i) == 0;
        int total;
        const int at = block_scan(free ? 1 : 0, &total);
        if (free) p.ids[count + at] = i;
        count += total;
    }
    __syncthreads();
    return count;
}

__device__ __forceinline__ bool in_pool(const PageParams& p, int id) {
    return id >= 0 && id < p.n_pages;
}

__global__ void __launch_bounds__(kThreads) kvp_reserve_kernel(const PageParams p) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    __shared__ int s_bad;
    if (tid == 0) s_bad = 0;
    for (int i = tid; i < p.n_pages; i += kThreads) p.refs2[i] = p.refs[i];
    __syncthreads();
    // pages each sequence needs; those its window leaves behind are released
    const int64_t cap = static_cast<int64_t>(p.max_pages) * p.page;
    int need = 0;
    for (int c0 = 0; c0 < p.n_seqs; c0 += kThreads) {
        const int c = c0 + tid;
        int want = 0;
        if (c < p.n_seqs) {
            const int len = p.lens[c];
            int n = p.arg[c];
            if (n < 0 || len < 0) {
                atomicOr(p.status, kStatusPage);
                n = 0;
            }
            if (n > 0 && static_cast<int64_t>(len) + n > cap) {
                s_bad = 1;
                n = 0;
            }
            want = n > 0 ? ceil_div(len + n, p.page) - ceil_div(len, p.page) : 0;
        }
        int total;
        const int at = block_scan(want, &total);
        if (c < p.n_seqs) p.base[c] = need + at;
        need += total;
    }
    auto evicted = [&](int c, int* j0, int* j1) {   // columns [j0, j1) no later query sees
        const int len = p.lens[c];
        *j0 = *j1 = 0;
        if (p.window <= 0 || p.arg[c] <= 0 || len < 0) return;
        *j0 = ceil_div(p.sinks, p.page);
        const int past = len - p.window + 1;   // first position a new query sees
        *j1 = min(past > 0 ? past / p.page : 0, p.max_pages);
    };
    for (int c = warp; c < p.n_seqs; c += kThreads / 32) {
        int j0, j1;
        evicted(c, &j0, &j1);
        for (int j = j0 + lane; j < j1; j += 32) {
            const int id = p.table[static_cast<int64_t>(c) * p.max_pages + j];
            if (in_pool(p, id)) atomicSub(p.refs2 + id, 1);
        }
    }
    __syncthreads();
    int before = 0;
    for (int i = tid; i < p.n_pages; i += kThreads) before += p.refs[i] == 0;
    before = block_sum(before);
    const int free = list_free(p);
    const bool done = s_bad == 0 && need <= free;
    if (tid == 0) {
        p.info[0] = done;
        p.info[1] = done ? need : 0;
        p.info[2] = done ? free - before : 0;
        p.info[3] = done ? free - need : before;
        if (!done) atomicOr(p.status, kStatusPool);
    }
    if (!done) return;
    for (int c = warp; c < p.n_seqs; c += kThreads / 32) {
        int j0, j1;
        evicted(c, &j0, &j1);
        int* row = p.table + static_cast<int64_t>(c) * p.max_pages;
        for (int j = j0 + lane; j < j1; j += 32) row[j] = -1;
        const int len = p.lens[c], n = p.arg[c];
        if (n > 0 && len >= 0) {
            const int first = ceil_div(len, p.page), want = ceil_div(len + n, p.page) - first;
            for (int k = lane; k < want; k += 32) {
                const int id = p.ids[p.base[c] + k];
                row[first + k] = id;
                atomicExch(p.refs2 + id, 1);
            }
            __syncwarp();
            if (lane == 0) p.lens[c] = len + n;
        }
    }
    __syncthreads();
    for (int i = tid; i < p.n_pages; i += kThreads) p.refs[i] = counter(p.refs2 + i);
}

__global__ void __launch_bounds__(kThreads) kvp_reassign_kernel(const PageParams p) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i < p.n_pages; i += kThreads) p.refs2[i] = p.refs[i];
    for (int c = tid; c < p.n_seqs; c += kThreads) p.keeper[c] = 0x7fffffff;
    __syncthreads();
    auto parent = [&](int c) {   // a bad one keeps the sequence
        const int q = p.arg[c];
        return q < -1 || q >= p.n_seqs ? c : q;
    };
    auto length = [&](int c) { return c < 0 ? 0 : min(max(p.lens[c], 0), p.max_pages * p.page); };
    for (int c = tid; c < p.n_seqs; c += kThreads) {
        const int q = parent(c);
        if (q != p.arg[c]) atomicOr(p.status, kStatusPage);
        if (q >= 0) atomicMin(p.keeper + q, q == c ? -1 : c);
    }
    __syncthreads();
    // Children that do not keep their parent's partly filled last page copy it.
    int n_copy = 0;
    for (int c0 = 0; c0 < p.n_seqs; c0 += kThreads) {
        const int c = c0 + tid;
        int tail = -1;
        if (c < p.n_seqs) {
            const int q = parent(c), len = length(q);
            if (q >= 0 && q != c && len % p.page != 0 && counter(p.keeper + q) != c &&
                in_pool(p, p.table[static_cast<int64_t>(q) * p.max_pages + len / p.page]))
                tail = len / p.page;
            p.tail[c] = tail;
            p.new_len[c] = q == c ? p.lens[c] : len;
        }
        int total;
        const int at = block_scan(tail >= 0 ? 1 : 0, &total);
        if (c < p.n_seqs) p.base[c] = n_copy + at;
        n_copy += total;
    }
    __syncthreads();
    // New rows of the changed sequences aside, and the counts they leave.
    auto columns = [&](int c, int q) {
        return max(ceil_div(length(c), p.page), ceil_div(length(q), p.page));
    };
    for (int c = warp; c < p.n_seqs; c += kThreads / 32) {
        const int q = parent(c);
        if (q == c) continue;
        const int64_t row = static_cast<int64_t>(c) * p.max_pages;
        const int had = ceil_div(length(c), p.page), has = ceil_div(length(q), p.page);
        const int tail = p.tail[c];
        for (int j = lane; j < columns(c, q); j += 32) {
            if (j < had && in_pool(p, p.table[row + j])) atomicSub(p.refs2 + p.table[row + j], 1);
            int id = -1;
            if (j < has) {
                id = p.table[static_cast<int64_t>(q) * p.max_pages + j];
                if (in_pool(p, id) && j != tail) atomicAdd(p.refs2 + id, 1);
            }
            p.table2[row + j] = id;
        }
    }
    __syncthreads();
    int before = 0;
    for (int i = tid; i < p.n_pages; i += kThreads) before += p.refs[i] == 0;
    before = block_sum(before);
    const int free = list_free(p);
    const bool done = n_copy <= free;
    if (tid == 0) {
        p.info[0] = done;
        p.info[1] = done ? n_copy : 0;
        p.info[2] = done ? free - before : 0;
        p.info[3] = done ? free - n_copy : before;
        if (!done) atomicOr(p.status, kStatusPool);
    }
    if (!done) return;
    for (int c = warp; c < p.n_seqs; c += kThreads / 32) {
        const int q = parent(c);
        if (q == c) continue;
        const int64_t row = static_cast<int64_t>(c) * p.max_pages;
        const int tail = p.tail[c], at = p.base[c];
        const int cols = max(ceil_div(length(c), p.page), ceil_div(p.new_len[c], p.page));
        for (int j = lane; j < cols; j += 32) {
            int id = p.table2[row + j];
            if (j == tail) {
                p.src[at] = id;
                id = p.ids[at];
                p.dst[at] = id;
                atomicExch(p.refs2 + id, 1);
            }
            p.table[row + j] = id;
        }
    }
    __syncthreads();
    for (int c = tid; c < p.n_seqs; c += kThreads) p.lens[c] = p.new_len[c];
    for (int i = tid; i < p.n_pages; i += kThreads) p.refs[i] = counter(p.refs2 + i);
}

// New ids of the held pages: ids[i] = -1 (not held), i, or the free id it moves
// to; refs_out and the moves.
__global__ void __launch_bounds__(kThreads) kvp_compact_kernel(const PageParams p) {
    const int tid = threadIdx.x;
    int held = 0;
    for (int i = tid; i < p.n_pages; i += kThreads) held += p.refs_in[i] > 0;
    held = block_sum(held);
    int holes = 0, movers = 0;
    for (int i0 = 0; i0 < p.n_pages; i0 += kThreads) {
        const int i = i0 + tid;
        const int r = i < p.n_pages ? p.refs_in[i] : 0;
        const bool hole = i < held && r <= 0, mover = i >= held && i < p.n_pages && r > 0;
        int n_hole, n_mover;
        const int a = block_scan(hole ? 1 : 0, &n_hole), b = block_scan(mover ? 1 : 0, &n_mover);
        if (hole) p.dst[holes + a] = i;
        if (mover) {
            p.src[movers + b] = i;
            p.refs2[movers + b] = r;   // refs_out may be refs
        }
        if (i < p.n_pages) p.ids[i] = r > 0 ? i : -1;
        holes += n_hole;
        movers += n_mover;
    }
    __syncthreads();
    for (int i = tid; i < p.n_pages; i += kThreads) {
        const int r = p.refs_in[i];
        p.refs[i] = i < held && r > 0 ? r : 0;
    }
    __syncthreads();
    for (int k = tid; k < movers; k += kThreads) {   // as many holes as movers
        p.ids[p.src[k]] = p.dst[k];
        p.refs[p.dst[k]] = p.refs2[k];
    }
    if (tid == 0) {
        p.info[0] = 1;
        p.info[1] = movers;
        p.info[2] = held;
        p.info[3] = p.n_pages - held;
    }
}

__global__ void __launch_bounds__(256) kvp_remap_kernel(const PageParams p, int64_t n) {
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
    take(&p->refs2, n_pages);
    take(&p->ids, n_pages);
    take(&p->keeper, n_seqs);
    take(&p->base, n_seqs);
    take(&p->tail, n_seqs);
    take(&p->new_len, n_seqs);
    take(&p->table2, static_cast<size_t>(n_seqs) * max_pages);
    return off;
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
    if (!table || !lens || !refs || !n_new || !info) return ATTN_ERR_INVALID;
    if (window < 0 || sinks < 0) return ATTN_ERR_INVALID;
    if (!page_ok(page)) return page <= 0 ? ATTN_ERR_INVALID : ATTN_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(max_pages) * page > (1ll << 30)) return ATTN_ERR_UNSUPPORTED;
    const void* ptrs[] = {table, lens, refs, n_new, info};
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
    p.page = page;
    // no position is past 2^30: larger ones mean all of them
    p.window = window > (1 << 30) ? 1 << 30 : window;
    p.sinks = sinks > (1 << 30) ? 1 << 30 : sinks;
    return launch_kernel(kvp_reserve_kernel, dim3(1), dim3(kThreads), 0,
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
    return launch_kernel(kvp_reassign_kernel, dim3(1), dim3(kThreads), 0,
                         static_cast<cudaStream_t>(stream), p) == cudaSuccess
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
    cudaError_t e = launch_kernel(kvp_compact_kernel, dim3(1), dim3(kThreads), 0, st, p);
    const int64_t n = static_cast<int64_t>(n_seqs) * max_pages;
    if (e == cudaSuccess)
        e = launch_kernel(kvp_remap_kernel, dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), 0,
                          st, p, n);
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}
