// kv8.cu -- the paged 8-bit KV cache: appending, attention, page copies.
//
// Cache layout and semantics: include/kvcache.h.  A decode step over a cache reads
// 2 D bytes per cached token and KV head and does 4 G D operations on them, so
// it is bound by memory: the kernels here are built to keep every SM's share of
// the reads in flight and to spend few instructions per byte.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "../../include/kvcache.h"
#include "attn_internal.h"
#include "kv8_attn.cuh"

namespace tme {
namespace {

// ------------------------------------------------------------------ append

struct AppendParams {
    const uint16_t* src[2];   // k, v
    uint8_t* pages[2];
    float* scales[2];
    const int* table;
    const int* lens;
    const int* n_new;
    const int* granted;
    unsigned int* status;
    int64_t sb, sh, st;
    int B, Hkv, T, n_pages, max_pages, n_slots;
};

constexpr int kAppendThreads = 128;

// Largest finite magnitude of n packed pairs, as fp32 bits.  Magnitudes order like
// their bits, so the pairs' maximum is taken on the 16-bit fields; only where it
// is an infinity or NaN are those left out one by one.
template <bool BF16, int N>
__device__ __forceinline__ uint32_t amax_bits(const uint4 (&w)[N]) {
    constexpr uint32_t kInf = BF16 ? 0x7f80u : 0x7c00u;
    uint32_t u = 0u;
#pragma unroll
    for (int i = 0; i < N; ++i)
        u = __vmaxu2(u, __vmaxu2(__vmaxu2(w[i].x & 0x7fff7fffu, w[i].y & 0x7fff7fffu),
                                 __vmaxu2(w[i].z & 0x7fff7fffu, w[i].w & 0x7fff7fffu)));
    uint32_t top = max(u & 0xffffu, u >> 16);
    if (top >= kInf) {
        top = 0u;
#pragma unroll 1
        for (int i = 0; i < 4 * N; ++i) {
            uint32_t x = 0u;   // (a register array takes no run-time index)
#pragma unroll
            for (int k = 0; k < N; ++k) {
                if (i == 4 * k) x = w[k].x;
                if (i == 4 * k + 1) x = w[k].y;
                if (i == 4 * k + 2) x = w[k].z;
                if (i == 4 * k + 3) x = w[k].w;
            }
            const uint32_t lo = x & 0x7fffu, hi = (x >> 16) & 0x7fffu;
            top = max(top, max(lo < kInf ? lo : 0u, hi < kInf ? hi : 0u));
        }
    }
    return __float_as_uint(unpack16<BF16>(top).x);
}

// One CTA per (sequence, page it may touch, KV head, keys or values): the page's
// new tokens are read once into registers (NV 16-byte vectors a thread, PAGE * D
// = 1024 NV), their largest magnitude gives the scale, then they are rounded
// and written; earlier tokens of the page are read only when the scale grew.
// A single token a sequence is bound by a launch (3.7 us in a graph), a prompt by the CTAs'
// turns: 2 x 8190 tokens, 8 KV heads, D = 128 read 67 MB and write 34 in 16.4 us cold, of
// which 31 are still in the second-level cache at the end; DRAM is 54% busy and the issue
// slots 57%.  3.4 waves of CTAs load, meet a barrier and store, with nothing between a
// CTA's stores and the next one's loads.  64 registers a thread leave 8 CTAs of 16 KB (64-token
// pages, D = 128) in flight on an SM, and the tokens are asked for before the page's id.
template <int D, int PAGE, bool BF16>
__global__ void __launch_bounds__(kAppendThreads, PAGE * D > 8192 ? 5 : 8)
    kv8_append_kernel(const AppendParams p) {
    constexpr int NV = PAGE * D / 8 / kAppendThreads;
    static_assert(NV >= 1, "a thread holds at least one vector");
    constexpr int VPT = D / 8;                        // vectors per token
    constexpr int STEP = kAppendThreads / VPT;        // tokens between a thread's vectors
    asm volatile("griddepcontrol.launch_dependents;");   // the attention may set up meanwhile
    int id = static_cast<int>(blockIdx.x);
    const int which = id & 1;
    id >>= 1;
    const int h = id % p.Hkv;
    id /= p.Hkv;
    const int slot = id % p.n_slots;
    const int b = id / p.n_slots;
    const int len = p.lens[b];
    const int n = p.n_new ? p.n_new[b] : p.T;
    const int granted = p.granted ? *p.granted : 1;   // 0: lens does not hold the tokens
    if (n == 0 || granted == 0) return;
    if (n < 0 || n > p.T || n > len || (len - 1) / PAGE >= p.max_pages) {
        if (threadIdx.x == 0) atomicOr(p.status, kStatusPage);
        return;
    }
    const int start = len - n;
    const int pj = start / PAGE + slot;
    const int t0 = pj * PAGE;
    if (t0 >= len) return;
    const int pid = p.table[static_cast<int64_t>(b) * p.max_pages + pj];
    const int pos0 = t0 + static_cast<int>(threadIdx.x) / VPT;   // position of the first vector
    const uint16_t* src = p.src[which] + b * p.sb + h * p.sh + (pos0 - start) * p.st +
                          threadIdx.x % VPT * 8;
    uint4 w[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int pos = pos0 + i * STEP;
        w[i] = make_uint4(0u, 0u, 0u, 0u);
        if (pos >= start && pos < len) w[i] = __ldcs(reinterpret_cast<const uint4*>(src + i * (STEP * p.st)));
    }
    if (pid < 0 || pid >= p.n_pages) {
        if (threadIdx.x == 0) atomicOr(p.status, kStatusPage);
        return;
    }
    uint8_t* dst = p.pages[which] + (static_cast<int64_t>(pid) * p.Hkv + h) * (PAGE * D) + threadIdx.x * 8;
    float* scale = p.scales[which] + static_cast<int64_t>(pid) * p.Hkv + h;
    const float s_old = t0 < start ? *scale : 0.0f;
    uint32_t u = __reduce_max_sync(0xffffffffu, amax_bits<BF16>(w));
    __shared__ uint32_t s_max[kAppendThreads / 32];
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = u;
    __syncthreads();   // also: every thread has read the old scale
#pragma unroll
    for (int i = 0; i < kAppendThreads / 32; ++i) u = max(u, s_max[i]);
    int e = amax_exp(__uint_as_float(u));
    const int e_old = t0 < start ? scale_exp(s_old) : e;
    e = max(e, e_old);
    if (threadIdx.x == 0) *scale = exp2i(e);
    const float inv = exp2i(-e);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int pos = pos0 + i * STEP;
        if (pos >= start && pos < len) {
            const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
            uint32_t r[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = unpack16<BF16>(x[j]);
                r[j] = f32_to_e4m3x2(f.x * inv, f.y * inv);
            }
            *reinterpret_cast<uint2*>(dst + i * (kAppendThreads * 8)) =
                make_uint2(r[0] | (r[1] << 16), r[2] | (r[3] << 16));
        }
    }
    if (e != e_old) raise_tokens<kAppendThreads * 8, STEP>(dst, pos0, min(start, t0 + PAGE), e_old, e);
}

template <int D, int PAGE>
cudaError_t launch_append(bool bf16, const AppendParams& p, cudaStream_t stream) {
    const int64_t ctas = static_cast<int64_t>(p.B) * p.n_slots * p.Hkv * 2;
    const dim3 grid(static_cast<unsigned>(ctas)), block(kAppendThreads);
    return bf16 ? launch_kernel(kv8_append_kernel<D, PAGE, true>, grid, block, 0, stream, p)
                : launch_kernel(kv8_append_kernel<D, PAGE, false>, grid, block, 0, stream, p);
}

// ------------------------------------------------------------------ attention
//
// The kernel is in kv8_attn.cuh.

// Combines the partial results of the units that lie in several CTAs: a warp per
// row, kMergeRows rows of one (sequence, unit) per CTA.  Lanes hold the CTAs' LSEs,
// 32 at a time, so the loads of the partial outputs depend on nothing but each
// other's sum.  Empty sequences get out = 0 and lse = -inf here.
constexpr int kMergeRows = 4;

template <int D, bool BF16, int NR>
__global__ void __launch_bounds__(kMergeRows * 32) kv8_merge_kernel(const AttnParams p) {
    constexpr int V = D / 32, kThreads = kMergeRows * 32;
    const int U = p.Hkv * p.n_rb;
    const int chunks = (min(8 * NR, p.rows) + kMergeRows - 1) / kMergeRows;   // of a row block
    const int unit = static_cast<int>(blockIdx.x / chunks);
    const int b = unit / U, u = unit % U;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.launch_dependents;");   // the next kernel may set up
    // Launched as a programmatic dependent of the attention kernel, which lets this
    // one start after its own wait: the lengths are complete here, the partial
    // results after the wait below.
    // tiles of all sequences, and of those before b: each warp for itself, or
    // (many sequences) the CTA together
    const bool alone = p.B <= 128, granted = step_granted(p);
    int all = 0, before = 0;
    for (int i = alone ? lane : threadIdx.x; i < p.B; i += alone ? 32 : kThreads) {
        const int len = p.lens[i], n = seq_of(p, len, queries_of(p, granted, i, len)).n;
        all += n;
        if (i < b) before += n;
    }
    all = __reduce_add_sync(0xffffffffu, all);
    before = __reduce_add_sync(0xffffffffu, before);
    if (!alone) {
        __shared__ int s_sum[2][kMergeRows];
        if (lane == 0) {
            s_sum[0][warp] = all;
            s_sum[1][warp] = before;
        }
        __syncthreads();
        all = before = 0;
#pragma unroll
        for (int i = 0; i < kMergeRows; ++i) {
            all += s_sum[0][i];
            before += s_sum[1][i];
        }
    }
    const int row0 = u % p.n_rb * (8 * NR);
    const int r = static_cast<int>(blockIdx.x % chunks) * kMergeRows + warp;   // within the block
    const int len = p.lens[b], n = seq_of(p, len, queries_of(p, granted, b, len)).n;
    const Shares sh(all * U, p.ctas);
    const int first = before * U + u * n;
    int c0 = 0, c1 = -1;   // the CTAs that hold part of the unit
    if (n > 0) {
        c0 = sh.owner(first);
        c1 = sh.owner(first + n - 1);
    }
    const int second = n > 0 && first > sh.begin(c0) ? 1 : 0;   // slot of c0's part
    asm volatile("griddepcontrol.wait;" ::: "memory");   // in every thread: this grid ends after that one
    if (r >= min(8 * NR, p.rows - row0) || c0 == c1) return;   // c0 == c1: written by that CTA
    auto part_row = [&](int cta) {
        return static_cast<int64_t>(2 * cta + (cta == c0 ? second : 0)) * (8 * NR) + r;
    };
    float M = -INFINITY, sum = 0.0f, acc[V] = {};
    for (int base = c0; base <= c1; base += 32) {
        const int cnt = min(32, c1 + 1 - base);
        const float L = lane < cnt ? p.part_lse[part_row(base + lane)] : -INFINITY;
        float M1 = fmaxf(M, L);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) M1 = fmaxf(M1, __shfl_xor_sync(0xffffffffu, M1, d));
        const float al = M == -INFINITY ? 0.0f : ex2_ftz(M - M1);
        const float w = L == -INFINITY ? 0.0f : ex2_ftz(L - M1);
        M = M1;
        sum *= al;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] *= al;
#pragma unroll 8
        for (int k = 0; k < cnt; ++k) {
            const float wk = __shfl_sync(0xffffffffu, w, k);
            const float* src = p.part_o + part_row(base + k) * D + lane * V;
            float x[V];
            if constexpr (V == 4) {
                const float4 y = *reinterpret_cast<const float4*>(src);
                x[0] = y.x, x[1] = y.y, x[2] = y.z, x[3] = y.w;
            } else {
                const float2 y = *reinterpret_cast<const float2*>(src);
                x[0] = y.x, x[1] = y.y;
            }
            sum += wk;
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = fmaf(wk, x[i], acc[i]);
        }
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    const int64_t row = (static_cast<int64_t>(b) * p.Hkv + u / p.n_rb) * p.rows + row0 + r;
    uint16_t* out = static_cast<uint16_t*>(p.out) + row * D + lane * V;
#pragma unroll
    for (int i = 0; i < V; i += 2)
        *reinterpret_cast<uint32_t*>(out + i) = pack2<BF16>(acc[i] * inv, acc[i + 1] * inv);
    if (lane == 0)
        p.lse[row] = sum == 0.0f ? -INFINITY : (M + lg2_approx(sum)) * 0.6931471805599453f;
}

template <int D, bool BF16, int NR>
cudaError_t launch_merge(const AttnParams& p, cudaStream_t stream) {
    const int rows = 8 * NR < p.rows ? 8 * NR : p.rows;
    const int64_t ctas = static_cast<int64_t>(p.B) * p.Hkv * p.n_rb *
                         ((rows + kMergeRows - 1) / kMergeRows);
    return launch_dependent(kv8_merge_kernel<D, BF16, NR>, ctas, kMergeRows * 32, 0, stream, p);
}

// ------------------------------------------------------------------ page copies

struct CopyParams {
    uint8_t* pages[2];
    float* scales[2];
    const int* src;
    const int* dst;
    const int* count;
    unsigned int* status;
    int max_count, n_layers, n_pages, Hkv;
    int vecs;   // 16-byte vectors of a page (all heads)
};

// CTAs take (pair, layer, keys or values) items in turn, as many as the device
// holds: the count of pairs is only known there.  4 vectors in flight a thread.
// Bound by memory: a compaction's 59 MB are read and written in 19.6 us cold, 6.0 TB/s (40
// of the written MB are still in the second-level cache then); its plan takes 7.5 us before.
constexpr int kCopyThreads = 256, kCopyCtasPerSm = 8;
__global__ void __launch_bounds__(kCopyThreads) kv8_copy_kernel(const CopyParams p) {
    // Launched as a programmatic dependent of the kernel that lists the pairs.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t items = 2 * static_cast<int64_t>(min(*p.count, p.max_count)) * p.n_layers;
    for (int64_t id = blockIdx.x; id < items; id += gridDim.x) {
        const int which = static_cast<int>(id & 1);
        const int layer = static_cast<int>((id >> 1) % p.n_layers);
        const int i = static_cast<int>((id >> 1) / p.n_layers);
        const int a = p.src[i], b = p.dst[i];
        if (a < 0 || a >= p.n_pages || b < 0 || b >= p.n_pages) {
            if (threadIdx.x == 0) atomicOr(p.status, kStatusPage);
            continue;
        }
        const int64_t base = static_cast<int64_t>(layer) * p.n_pages;
        const uint4* from = reinterpret_cast<const uint4*>(p.pages[which]) + (base + a) * p.vecs;
        uint4* to = reinterpret_cast<uint4*>(p.pages[which]) + (base + b) * p.vecs;
        for (int x = threadIdx.x; x < p.vecs; x += 4 * kCopyThreads) {
            uint4 w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (x + kCopyThreads * k < p.vecs) w[k] = from[x + kCopyThreads * k];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (x + kCopyThreads * k < p.vecs) to[x + kCopyThreads * k] = w[k];
        }
        for (int x = threadIdx.x; x < p.Hkv; x += kCopyThreads)
            p.scales[which][(base + b) * p.Hkv + x] = p.scales[which][(base + a) * p.Hkv + x];
    }
}

// ------------------------------------------------------------------ host

}  // namespace
}  // namespace tme

using namespace tme;

extern "C" int kv8_append(const void* k, const void* v, void* k_pages, void* v_pages,
                          float* k_scale, float* v_scale, const int* table, const int* lens,
                          const int* n_new, int B, int Hkv, int T, int D, int page, int n_pages,
                          int max_pages, long long stride_b, long long stride_h,
                          long long stride_t, int dtype, void* stream) {
    return kv8_append_step(k, v, k_pages, v_pages, k_scale, v_scale, table, lens, n_new, nullptr, B,
                           Hkv, T, D, page, n_pages, max_pages, stride_b, stride_h, stride_t, dtype,
                           stream);
}

extern "C" int kv8_append_step(const void* k, const void* v, void* k_pages, void* v_pages,
                               float* k_scale, float* v_scale, const int* table, const int* lens,
                               const int* n_new, const int* granted, int B, int Hkv, int T, int D,
                               int page, int n_pages, int max_pages, long long stride_b,
                               long long stride_h, long long stride_t, int dtype, void* stream) {
    if (!k || !v || !k_pages || !v_pages || !k_scale || !v_scale || !table || !lens)
        return ATTN_ERR_INVALID;
    int rc = check_cache(B, Hkv, D, page, n_pages, max_pages);
    if (rc != ATTN_OK) return rc;
    if (T <= 0 || (dtype != ATTN_F16 && dtype != ATTN_BF16)) return ATTN_ERR_INVALID;
    if (stride_b < 0 || stride_h < 0 || stride_t < 0) return ATTN_ERR_INVALID;
    const void* ptrs[] = {k, v, k_pages, v_pages};
    const void* words[] = {k_scale, v_scale, table, lens, n_new, granted};
    if (!aligned(ptrs, 16) || !aligned(words, 4)) return ATTN_ERR_ALIGN;
    if (stride_b % 8 || stride_h % 8 || stride_t % 8) return ATTN_ERR_ALIGN;
    const int64_t slots = (static_cast<int64_t>(T) + page - 2) / page + 1;
    if (slots * B * Hkv * 2 > 0x7fffffffll) return ATTN_ERR_UNSUPPORTED;
    AppendParams p{};
    rc = device_setup_public(&p.status);
    if (rc != ATTN_OK) return rc;
    p.src[0] = static_cast<const uint16_t*>(k);
    p.src[1] = static_cast<const uint16_t*>(v);
    p.pages[0] = static_cast<uint8_t*>(k_pages);
    p.pages[1] = static_cast<uint8_t*>(v_pages);
    p.scales[0] = k_scale;
    p.scales[1] = v_scale;
    p.table = table;
    p.lens = lens;
    p.n_new = n_new;
    p.granted = granted;
    p.sb = stride_b;
    p.sh = stride_h;
    p.st = stride_t;
    p.B = B;
    p.Hkv = Hkv;
    p.T = T;
    p.n_pages = n_pages;
    p.max_pages = max_pages;
    p.n_slots = static_cast<int>(slots);
    const bool bf16 = dtype == ATTN_BF16;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaErrorInvalidValue;
#define TME_APPEND(d, pg) \
    if (D == d && page == pg) e = launch_append<d, pg>(bf16, p, st);
    TME_APPEND(64, 16)
    TME_APPEND(64, 32)
    TME_APPEND(64, 64)
    TME_APPEND(64, 128)
    TME_APPEND(128, 16)
    TME_APPEND(128, 32)
    TME_APPEND(128, 64)
    TME_APPEND(128, 128)
#undef TME_APPEND
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

namespace tme {
namespace {
int check_kv8_attn(int B, int Hq, int Hkv, int Nq, int D) {
    if (B <= 0 || Hq <= 0 || Hkv <= 0 || Nq <= 0 || D <= 0 || Hq % Hkv != 0) return ATTN_ERR_INVALID;
    if (D != 64 && D != 128) return ATTN_ERR_UNSUPPORTED;
    if (B > kMaxBatch) return ATTN_ERR_UNSUPPORTED;
    const int64_t rows = static_cast<int64_t>(Hq / Hkv) * Nq;
    const int64_t units = static_cast<int64_t>(B) * Hkv * ((rows + 31) / 32);
    if (rows > (1 << 30) || units > (1 << 27)) return ATTN_ERR_UNSUPPORTED;
    return ATTN_OK;
}
}  // namespace

int attn_params(AttnParams* out_p, const void* q, const void* k_pages, const void* v_pages,
                const float* k_scale, const float* v_scale, const int* table, const int* lens,
                const int* n_new, const int* granted, void* out, float* lse, void* workspace,
                size_t workspace_bytes, size_t needed, int B, int Hq, int Hkv, int Nq, int D, int page,
                int n_pages, int max_pages, float scale, int window, int sinks, int dtype) {
    if (!q || !k_pages || !v_pages || !k_scale || !v_scale || !table || !lens || !out || !lse ||
        !workspace)
        return ATTN_ERR_INVALID;
    int rc = check_kv8_attn(B, Hq, Hkv, Nq, D);
    if (rc != ATTN_OK) return rc;
    rc = check_cache(B, Hkv, D, page, n_pages, max_pages);
    if (rc != ATTN_OK) return rc;
    if (dtype != ATTN_F16 && dtype != ATTN_BF16) return ATTN_ERR_INVALID;
    if (!(scale > 0.0f) || !std::isfinite(scale)) return ATTN_ERR_INVALID;
    if (window < 0 || sinks < 0) return ATTN_ERR_INVALID;
    const void* ptrs[] = {q, k_pages, v_pages, out, lse, workspace};
    const void* words[] = {k_scale, v_scale, table, lens, n_new, granted};
    if (!aligned(ptrs, 16) || !aligned(words, 4)) return ATTN_ERR_ALIGN;
    if (workspace_bytes < needed) return ATTN_ERR_WORKSPACE;
    // the kernels count tiles of all sequences' table capacity in 32 bits
    if (static_cast<int64_t>(B) * Hkv * ((static_cast<int64_t>(Hq / Hkv) * Nq + 31) / 32) *
            ((static_cast<int64_t>(max_pages) * page + 31) / 32) > 0x7fffffffll)
        return ATTN_ERR_UNSUPPORTED;
    AttnParams p{};
    rc = device_setup_public(&p.status);
    if (rc != ATTN_OK) return rc;
    const int sms = device_sms();
    if (sms <= 0) return ATTN_ERR_CUDA;
    const int64_t rows = static_cast<int64_t>(Hq / Hkv) * Nq;
    const int nr = row_tiles(rows);
    p.q = q;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.table = table;
    p.lens = lens;
    p.n_new = n_new;
    p.granted = granted;
    p.out = out;
    p.lse = lse;
    p.ctas = sms;
    const size_t n_part = 2 * static_cast<size_t>(sms) * 8 * nr;
    p.part_o = static_cast<float*>(workspace);
    p.part_lse = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                          pad256(n_part * D * sizeof(float)));
    p.B = B;
    p.Hkv = Hkv;
    p.rows = static_cast<int>(rows);
    p.n_rb = static_cast<int>((rows + 8 * nr - 1) / (8 * nr));
    p.Nq = Nq;
    p.page_shift = page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7;
    p.tile_shift = D == 64 && nr < 4 ? 6 : 5;
    p.n_pages = n_pages;
    p.max_pages = max_pages;
    // no position is past max_pages * page <= 2^30: larger ones mean all
    const int most = max_pages * page;
    p.window = window > most ? most : window;
    p.sinks = sinks > most ? most : sinks;
    p.scale_log2 = scale * 1.4426950408889634f;
    *out_p = p;
    return ATTN_OK;
}

// The attention and the merge behind it.
int attn_launch(const AttnParams& p, const void* k_pages, const void* v_pages, int D, int page, bool bf16,
                cudaStream_t st) {
    cudaError_t e = launch_attention<false>(p, k_pages, v_pages, D, page, bf16, st);
    if (e != cudaSuccess) return ATTN_ERR_CUDA;
    const int nr = row_tiles(p.rows);
    e = cudaErrorInvalidValue;
#define TME_MERGE(d, b, n) \
    if (D == d && bf16 == b && nr == n) e = launch_merge<d, b, n>(p, st);
    TME_MERGE(64, false, 1)
    TME_MERGE(64, false, 2)
    TME_MERGE(64, false, 4)
    TME_MERGE(64, true, 1)
    TME_MERGE(64, true, 2)
    TME_MERGE(64, true, 4)
    TME_MERGE(128, false, 1)
    TME_MERGE(128, false, 2)
    TME_MERGE(128, false, 4)
    TME_MERGE(128, true, 1)
    TME_MERGE(128, true, 2)
    TME_MERGE(128, true, 4)
#undef TME_MERGE
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}
}  // namespace tme

extern "C" size_t kv8_attn_workspace_size(int B, int Hq, int Hkv, int Nq, int D) {
    if (check_kv8_attn(B, Hq, Hkv, Nq, D) != ATTN_OK) return 0;
    const int sms = device_sms();
    return part_bytes(static_cast<int64_t>(Hq / Hkv) * Nq, D, sms > 0 ? sms : 1);
}

extern "C" int kv8_attn(const void* q, const void* k_pages, const void* v_pages,
                        const float* k_scale, const float* v_scale, const int* table,
                        const int* lens, void* out, float* lse, void* workspace,
                        size_t workspace_bytes, int B, int Hq, int Hkv, int Nq, int D, int page,
                        int n_pages, int max_pages, float scale, int window, int sinks, int dtype,
                        void* stream) {
    return kv8_attn_step(q, k_pages, v_pages, k_scale, v_scale, table, lens, nullptr, nullptr, out, lse,
                         workspace, workspace_bytes, B, Hq, Hkv, Nq, D, page, n_pages, max_pages,
                         scale, window, sinks, dtype, stream);
}

extern "C" int kv8_attn_step(const void* q, const void* k_pages, const void* v_pages,
                             const float* k_scale, const float* v_scale, const int* table,
                             const int* lens, const int* n_new, const int* granted, void* out,
                             float* lse, void* workspace, size_t workspace_bytes, int B, int Hq,
                             int Hkv, int Nq, int D, int page, int n_pages, int max_pages,
                             float scale, int window, int sinks, int dtype, void* stream) {
    AttnParams p;
    int rc = attn_params(&p, q, k_pages, v_pages, k_scale, v_scale, table, lens, n_new, granted, out, lse,
                         workspace, workspace_bytes, kv8_attn_workspace_size(B, Hq, Hkv, Nq, D), B, Hq, Hkv,
                         Nq, D, page, n_pages, max_pages, scale, window, sinks, dtype);
    if (rc != ATTN_OK) return rc;
    return attn_launch(p, k_pages, v_pages, D, page, dtype == ATTN_BF16, static_cast<cudaStream_t>(stream));
}

extern "C" int kv8_copy_pages(void* k_pages, void* v_pages, float* k_scale, float* v_scale,
                              const int* src, const int* dst, const int* count, int max_count,
                              int n_layers, int Hkv, int page, int D, int n_pages, void* stream) {
    if (!k_pages || !v_pages || !k_scale || !v_scale || !src || !dst || !count)
        return ATTN_ERR_INVALID;
    int rc = check_cache(1, Hkv, D, page, n_pages, 1);
    if (rc != ATTN_OK) return rc;
    if (max_count < 0 || n_layers <= 0) return ATTN_ERR_INVALID;
    const void* ptrs[] = {k_pages, v_pages};
    const void* words[] = {k_scale, v_scale, src, dst, count};
    if (!aligned(ptrs, 16) || !aligned(words, 4)) return ATTN_ERR_ALIGN;
    if (max_count == 0) return ATTN_OK;
    if (static_cast<int64_t>(max_count) * n_layers * 2 > 0x7fffffffll ||
        static_cast<int64_t>(Hkv) * page * D / 16 > (1 << 30))
        return ATTN_ERR_UNSUPPORTED;
    CopyParams p{};
    rc = device_setup_public(&p.status);
    if (rc != ATTN_OK) return rc;
    p.pages[0] = static_cast<uint8_t*>(k_pages);
    p.pages[1] = static_cast<uint8_t*>(v_pages);
    p.scales[0] = k_scale;
    p.scales[1] = v_scale;
    p.src = src;
    p.dst = dst;
    p.count = count;
    p.max_count = max_count;
    p.n_layers = n_layers;
    p.n_pages = n_pages;
    p.Hkv = Hkv;
    p.vecs = Hkv * page * D / 16;
    const int sms = device_sms();
    const int64_t items = static_cast<int64_t>(max_count) * n_layers * 2;
    const int64_t most = static_cast<int64_t>(sms > 0 ? sms : 1) * kCopyCtasPerSm;
    return launch_dependent(kv8_copy_kernel, items < most ? items : most, kCopyThreads, 0,
                            static_cast<cudaStream_t>(stream), p) == cudaSuccess
               ? ATTN_OK
               : ATTN_ERR_CUDA;
}
