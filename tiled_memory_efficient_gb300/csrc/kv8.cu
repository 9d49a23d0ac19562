// kv8.cu -- the paged 8-bit KV cache: appending, attention, page copies.
//
// Cache layout and semantics: include/kvcache.h.  A decode step over a cache reads
// 2 D bytes per cached token and KV head and does 4 G D operations on them, so
// it is bound by memory: the kernels here are built to keep every SM's share of
// the reads in flight and to spend few instructions per byte.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/kvcache.h"
#include "attn_internal.h"
#include "ptx.cuh"

namespace tme {

// abi.cu
int device_setup_public(unsigned int** status);
int make_byte_map_public(CUtensorMap* map, const void* base, int D, int rows, int64_t groups,
                         int box_rows);

namespace {

// ------------------------------------------------------------------ e4m3

constexpr int kMinExp = -126;   // of a page's scale 2^e (448 * 2^120 is past bf16's range)
constexpr int kMaxExp = 120;

// Two e4m3 values (16 bits) as two fp16 values: exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
        : "=r"(r)
        : "r"(w));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x2_hi_to_f16x2(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}"
        : "=r"(r)
        : "r"(w));
    return r;
}
__device__ __forceinline__ float2 f16x2_to_f32(uint32_t w) {
    float a, b;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\t"
        "cvt.f32.f16 %1, hi;\n\t}"
        : "=f"(a), "=f"(b)
        : "r"(w));
    return make_float2(a, b);
}
// Two fp32 values rounded to e4m3 (nearest even, clamped to +-448; first in the low byte).
__device__ __forceinline__ uint32_t f32_to_e4m3x2(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}
__device__ __forceinline__ float exp2i(int e) {   // 2^e, -126 <= e <= 127
    return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}
// Exponent of a stored scale (a power of two; anything else is brought into range).
__device__ __forceinline__ int scale_exp(float s) {
    const int e = static_cast<int>((__float_as_uint(s) >> 23) & 0xffu) - 127;
    return min(max(e, kMinExp), kMaxExp);
}
// Smallest e with amax <= 448 * 2^e = 1.75 * 2^(e + 8), clamped.
__device__ __forceinline__ int amax_exp(float amax) {
    const uint32_t u = __float_as_uint(amax);
    int e = static_cast<int>(u >> 23) - 127 - 8;
    if ((u & 0x7fffffu) > 0x600000u) ++e;
    return min(max(e, kMinExp), kMaxExp);
}

template <bool BF16>
__device__ __forceinline__ float2 unpack16(uint32_t w) {
    if constexpr (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    else return f16x2_to_f32(w);
}

// ------------------------------------------------------------------ append

struct AppendParams {
    const uint16_t* src[2];   // k, v
    uint8_t* pages[2];
    float* scales[2];
    const int* table;
    const int* lens;
    const int* n_new;
    unsigned int* status;
    int64_t sb, sh, st;
    int B, Hkv, T, n_pages, max_pages, n_slots;
};

constexpr int kAppendThreads = 128;

// One CTA per (sequence, page it may touch, KV head, keys or values): the page's
// new tokens are read once into registers (NV 16-byte vectors a thread, PAGE * D
// = 1024 NV), their largest magnitude gives the scale, then they are rounded
// and written; earlier tokens of the page are read only when the scale grew.
template <int D, int PAGE, bool BF16>
__global__ void __launch_bounds__(kAppendThreads) kv8_append_kernel(const AppendParams p) {
    constexpr int NV = PAGE * D / 8 / kAppendThreads;
    static_assert(NV >= 1, "a thread holds at least one vector");
    constexpr int VPT = D / 8;   // vectors per token
    int64_t id = blockIdx.x;
    const int which = static_cast<int>(id & 1);
    id >>= 1;
    const int h = static_cast<int>(id % p.Hkv);
    id /= p.Hkv;
    const int slot = static_cast<int>(id % p.n_slots);
    const int b = static_cast<int>(id / p.n_slots);
    const int len = p.lens[b];
    const int n = p.n_new ? p.n_new[b] : p.T;
    if (n == 0) return;
    if (n < 0 || n > p.T || n > len || (len - 1) / PAGE >= p.max_pages) {
        if (threadIdx.x == 0) atomicOr(p.status, kStatusPage);
        return;
    }
    const int start = len - n;
    const int pj = start / PAGE + slot;
    const int t0 = pj * PAGE;
    if (t0 >= len) return;
    const int pid = p.table[static_cast<int64_t>(b) * p.max_pages + pj];
    if (pid < 0 || pid >= p.n_pages) {
        if (threadIdx.x == 0) atomicOr(p.status, kStatusPage);
        return;
    }
    const uint16_t* src = p.src[which] + b * p.sb + h * p.sh;
    uint8_t* dst = p.pages[which] + (static_cast<int64_t>(pid) * p.Hkv + h) * (PAGE * D);
    float* scale = p.scales[which] + static_cast<int64_t>(pid) * p.Hkv + h;
    const float s_old = t0 < start ? *scale : 0.0f;

    uint4 w[NV];
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = threadIdx.x + i * kAppendThreads;
        const int pos = t0 + c / VPT;
        w[i] = make_uint4(0u, 0u, 0u, 0u);
        if (pos >= start && pos < len)
            w[i] = *reinterpret_cast<const uint4*>(src + (pos - start) * p.st + c % VPT * 8);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = unpack16<BF16>(x[j]);
            const float a = fabsf(f.x), c = fabsf(f.y);
            amax = fmaxf(amax, a <= 3.4028235e38f ? a : 0.0f);   // finite ones only
            amax = fmaxf(amax, c <= 3.4028235e38f ? c : 0.0f);
        }
    }
    // magnitudes order like their bits
    uint32_t u = __reduce_max_sync(0xffffffffu, __float_as_uint(amax));
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
    const float redo = e_old - e < -100 ? 0.0f : exp2i(e_old - e);   // 448 * 2^-100 rounds to 0
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = threadIdx.x + i * kAppendThreads;
        const int pos = t0 + c / VPT;
        uint2* at = reinterpret_cast<uint2*>(dst + c * 8);
        if (pos >= start && pos < len) {
            const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
            uint32_t r[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = unpack16<BF16>(x[j]);
                r[j] = f32_to_e4m3x2(f.x * inv, f.y * inv);
            }
            *at = make_uint2(r[0] | (r[1] << 16), r[2] | (r[3] << 16));
        } else if (pos < start && e != e_old) {
            const uint2 o = *at;
            const uint32_t x[2] = {o.x, o.y};
            uint32_t r[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t y = x[j >> 1];
                const float2 f = f16x2_to_f32((j & 1) ? e4m3x2_hi_to_f16x2(y) : e4m3x2_to_f16x2(y));
                r[j] = f32_to_e4m3x2(f.x * redo, f.y * redo);
            }
            *at = make_uint2(r[0] | (r[1] << 16), r[2] | (r[3] << 16));
        }
    }
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
// Work is counted in tiles of 32 tokens: sequence b has n_b visible ones (its sink
// tiles and then its window's, or all) for each of its U = Hkv * row blocks
// units.  The CTAs of one wave cut the concatenation of all (sequence, unit)
// lists into equal shares, so the balance does not depend on the lengths; a unit
// that lies in one CTA is written out directly, the others leave fp32 partial
// results that kv8_merge_kernel combines.
//
// Inside a CTA every warp works on its own: tiles w, w + 8, ... of the share,
// through a ring of kStages (K, V) slots that it alone fills (TMA, an mbarrier
// each) and empties, so warps meet only where a unit ends.  Lane s owns slot s:
// it follows the slot's tiles through the table and issues their copies.
//
// Products run on mma.sync m16n8k16 with the tokens (scores) or the head
// dimensions (output) as its 16 rows and up to 8 query rows as its columns:
// S^T = K Q^T, O^T += V^T P^T.  The tensor core is not what bounds this kernel (a
// tile of 32 tokens is 8 KB at D = 128, about 180 cycles of one SM's share of the
// memory, and 32 small products), and registers hold P between the two products.
// K and V become fp16 exactly (e4m3x2 -> f16x2); the dimensions of a K row and
// the tokens of a V column may meet the product in any order that its other
// operand shares, which is how 16-byte shared loads feed both (kTok below).

constexpr int kWarps = 8;
constexpr int kAttnThreads = kWarps * 32;
constexpr int kTile = 32;         // tokens per tile
constexpr int kMaxBatch = 2048;   // sequences per call (their tile counts live in shared memory)
constexpr int kMinShare = kWarps; // tiles per CTA, at least (one per warp)

struct AttnParams {
    const void* q;
    const float* k_scale;
    const float* v_scale;
    const int* table;
    const int* lens;
    void* out;
    float* lse;
    float* part_o;     // [2 * ctas][rows of a block][D]
    float* part_lse;   // [2 * ctas][rows of a block], log2 domain
    unsigned int* status;
    int B, Hkv, rows, n_rb;   // rows = G * Nq of a KV head, row blocks
    int Nq, page, n_pages, max_pages;
    int window, sinks, ctas;
    float scale_log2;
};

// The visible tiles of a sequence.
struct Seq {
    int len, first;        // positions held; position of the first query (may be < 0)
    int lo;                // first position inside a window of some query
    int n_sink, skip, n;   // tiles [0, n_sink) and [n_sink + skip, ...), n in all
};
__device__ __forceinline__ Seq seq_of(const AttnParams& p, int len) {
    Seq s;
    s.len = min(max(len, 0), p.max_pages * p.page);
    s.first = s.len - p.Nq;
    s.lo = p.window > 0 ? max(s.first - p.window + 1, 0) : 0;
    const int lo_tile = s.lo / kTile;
    s.n_sink = min((p.sinks + kTile - 1) / kTile, lo_tile);
    s.skip = lo_tile - s.n_sink;
    s.n = (s.len + kTile - 1) / kTile - s.skip;
    return s;
}
__device__ __forceinline__ int seq_token(const Seq& s, int v) {   // first token of tile v of the list
    return (v < s.n_sink ? v : v + s.skip) * kTile;
}

// Shares: CTA c takes [c T / n, (c + 1) T / n) of the T tiles, n CTAs.
__device__ __forceinline__ int shares(int64_t T, int ctas) {
    const int64_t n = (T + kMinShare - 1) / kMinShare;
    return static_cast<int>(n < ctas ? n : ctas);
}

// Token that row m of a 16-token product tile stands for (both halves of 8
// alike).  The 16-byte shared loads of K (lanes g = m, chunk t) and of V (lanes
// t = m / 2, chunk g) then meet every bank once in each group of 8 lanes (16 for
// 8-byte loads), given the swizzle TMA wrote.
template <int D>
__device__ __forceinline__ int tok8(int m) {
    return D == 128 ? (m & 1 ? (m & 6) ^ 5 : m & 6)          // 0 5 2 7 4 1 6 3
                    : (0x65742130 >> (4 * ((m & 7)))) & 7;   // 0 3 1 2 4 7 5 6
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 r;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "r"(a)
                 : "memory");
    return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 r;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a) : "memory");
    return r;
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

template <int D>
struct AttnCfg {
    static constexpr int kStages = D == 128 ? 3 : 6;
    static constexpr int kHalf = kTile * D;         // bytes of K (or V) of a tile
    static constexpr int kSlot = 2 * kHalf;
    static constexpr int kRing = kWarps * kStages * kSlot;          // 192 KB
    static constexpr int kMergeOff = kRing;                         // 8 warps x 8 rows x 64 fp32
    static constexpr int kLseOff = kMergeOff + kWarps * 8 * 64 * 4;
    static constexpr int kBarOff = kLseOff + kWarps * 8 * 4;
    static constexpr int kMiscOff = kBarOff + kWarps * kStages * 8;
    static constexpr int kPreOff = kMiscOff + 64;                   // B + 1 ints
    static int smem_bytes(int B) { return kPreOff + (B + 1) * 4 + 1024; }
};

template <int D, bool BF16, int NR>
__global__ void __launch_bounds__(kAttnThreads, 1)
    kv8_attn_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                    const AttnParams p) {
    using C = AttnCfg<D>;
    constexpr int ST = C::kStages;
    constexpr int KC = D / 64;         // 16-byte chunks of a K row per lane
    constexpr int MT = D / 16;         // 16-dimension tiles of O^T
    constexpr int VB = D / 8;          // bytes of a V row per lane (16 or 8)
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    float* s_merge = reinterpret_cast<float*>(smem + C::kMergeOff);   // [warp][8 rows][64]
    float* s_lse = reinterpret_cast<float*>(smem + C::kLseOff);       // [warp][8 rows]
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMiscOff);
    int* s_warp = reinterpret_cast<int*>(smem + C::kMiscOff + 16);    // [8]
    int* s_pre = reinterpret_cast<int*>(smem + C::kPreOff);           // [B + 1]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kWarps * ST; ++i) mbar_init(&bars[i], 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    // exclusive prefix sums of the sequences' tile counts
    int carry = 0;
    for (int b0 = 0; b0 < p.B; b0 += kAttnThreads) {
        const int b = b0 + static_cast<int>(threadIdx.x);
        int len = 0;
        if (b < p.B) {
            len = p.lens[b];
            if (blockIdx.x == 0 && (len < 0 || len > p.max_pages * p.page))
                atomicOr(p.status, kStatusPage);
        }
        const int n = b < p.B ? seq_of(p, len).n : 0;
        int x = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += y;
        }
        if (lane == 31) s_warp[warp] = x;
        __syncthreads();
        int before = carry, all = carry;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            if (i < warp) before += s_warp[i];
            all += s_warp[i];
        }
        if (b < p.B) s_pre[b] = before + x - n;
        carry = all;
        __syncthreads();
    }
    if (threadIdx.x == 0) s_pre[p.B] = carry;
    __syncthreads();
    const int U = p.Hkv * p.n_rb;
    const int64_t T = static_cast<int64_t>(carry) * U;
    const int n_cta = shares(T, p.ctas);
    const int c = static_cast<int>(blockIdx.x);
    if (c >= n_cta) return;   // nothing in flight, no barrier left
    const int64_t g0 = c * T / n_cta, g1 = (c + 1) * T / n_cta;

    // (sequence, unit, tile) of a position in the concatenated lists; b moves forward only
    auto locate = [&](int64_t x, int& b, int& u, int& v) {
        while (x >= static_cast<int64_t>(s_pre[b + 1]) * U) ++b;
        const int n = s_pre[b + 1] - s_pre[b];
        const int64_t r = x - static_cast<int64_t>(s_pre[b]) * U;
        u = static_cast<int>(r / n);
        v = static_cast<int>(r - static_cast<int64_t>(u) * n);
    };

    // ---- this lane's slot (lanes 0 .. ST - 1)
    uint8_t* ring = smem + warp * (ST * C::kSlot);
    uint64_t* full = bars + warp * ST;
    const int box = min(p.page, kTile);    // tokens per TMA box
    const int boxes = kTile / box;         // 1, or 2 of 16 tokens
    int64_t next = g0 + warp + kWarps * lane;   // next tile of this lane's slot
    int nb = 0;                                 // its sequence
    // scales of the tile in the slot: pages of its two 16-token halves
    float ks0 = 0.0f, ks1 = 0.0f, vs0 = 0.0f, vs1 = 0.0f;
    int bad = 0;                                // bit i: half i has no readable page
    int issued = 0;
    auto issue = [&]() {
        if (next >= g1) return;
        int u, v;
        locate(next, nb, u, v);
        next += kWarps * ST;
        const Seq s = seq_of(p, p.lens[nb]);
        const int tok = seq_token(s, v);
        const int h = u / p.n_rb;
        uint8_t* dst = ring + lane * C::kSlot;
        mbar_arrive_expect_tx(&full[lane], C::kSlot);
        bad = 0;
        ++issued;
        for (int i = 0; i < boxes; ++i) {
            const int x = tok + i * box;
            // a box no query sees need not have a page
            const bool seen = x < s.len && (x + box > s.lo || x < p.sinks);
            int pid = -1;
            if (seen) pid = p.table[static_cast<int64_t>(nb) * p.max_pages + x / p.page];
            const bool ok = pid >= 0 && pid < p.n_pages;
            if (seen && !ok) atomicOr(p.status, kStatusPage);
            if (!ok) bad |= boxes == 1 ? 3 : 1 << i;
            // past the pool the copy fills zeros
            const int z = ok ? pid * p.Hkv + h : p.n_pages * p.Hkv;
            tma_load_3d(&tmK, &full[lane], dst + i * 16 * D, 0, x % p.page, z);
            tma_load_3d(&tmV, &full[lane], dst + C::kHalf + i * 16 * D, 0, x % p.page, z);
            const float a = ok ? p.k_scale[z] : 1.0f, e = ok ? p.v_scale[z] : 1.0f;
            if (i == 0) {
                ks0 = a;
                vs0 = e;
            }
            if (i == 1 || boxes == 1) {
                ks1 = a;
                vs1 = e;
            }
        }
    };
    if (lane < ST) issue();

    // ---- fragment addresses (the same in every tile)
    uint32_t k_at[2][KC], v_at[2];   // K: token rows g / g + 8, chunks t (+ 4); V: rows 2t, 2t + 1
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = tok8<D>(g) + 8 * i;
#pragma unroll
        for (int cc = 0; cc < KC; ++cc) {
            const int ch = t + 4 * cc;
            k_at[i][cc] = r * D + 16 * (D == 128 ? ch ^ (r & 7) : ch ^ ((r >> 1) & 3));
        }
        const int rv = tok8<D>(2 * t + i);
        v_at[i] = D == 128 ? rv * D + 16 * (g ^ (rv & 7))
                           : rv * D + 16 * ((g >> 1) ^ ((rv >> 1) & 3)) + 8 * (g & 1);
    }
    const int tok_a = tok8<D>(g);          // tokens of this lane's score rows: tok_a, tok_a + 8
    const int tok_v0 = tok8<D>(2 * t), tok_v1 = tok8<D>(2 * t + 1);

    // ---- the share, unit by unit
    int64_t mine = g0 + warp;   // this warp's next tile
    int it = 0;                 // tiles this warp has done
    int b = 0, u, v;
    locate(g0, b, u, v);
    int64_t unit0 = g0 - v;     // the unit's first tile in the concatenated lists
    while (unit0 < g1) {
        while (s_pre[b + 1] == s_pre[b]) ++b;   // empty sequences
        const Seq s = seq_of(p, p.lens[b]);
        const int h = u / p.n_rb, rb = u % p.n_rb;
        const int64_t unit1 = unit0 + s.n;
        const int64_t end = unit1 < g1 ? unit1 : g1;
        const int row0 = rb * (8 * NR);
        const int64_t head_row = (static_cast<int64_t>(b) * p.Hkv + h) * p.rows;   // of q, out, lse

        // Q as fp16 B fragments: lane (g, t) holds dimensions 16 (t + 4 cc) .. + 15 of row g.
        // bf16 rows are scaled by a power of two first (their largest magnitude
        // to [2^14, 2^15)), which the scores take back: fp16 then holds every
        // value down to 2^-28 of the row's largest exactly.
        uint32_t qf[NR][KC][8];
        float f_row[NR][2];   // softmax scale of this lane's score columns 2t, 2t + 1
#pragma unroll
        for (int nt = 0; nt < NR; ++nt) {
            const int r = row0 + nt * 8 + g;
            uint32_t w[KC][8];
#pragma unroll
            for (int cc = 0; cc < KC; ++cc) {
                const uint4* src = reinterpret_cast<const uint4*>(
                    static_cast<const uint16_t*>(p.q) + (head_row + r) * D + 16 * (t + 4 * cc));
                const uint4 z = make_uint4(0u, 0u, 0u, 0u);
                const uint4 lo = r < p.rows ? src[0] : z, hi = r < p.rows ? src[1] : z;
                w[cc][0] = lo.x, w[cc][1] = lo.y, w[cc][2] = lo.z, w[cc][3] = lo.w;
                w[cc][4] = hi.x, w[cc][5] = hi.y, w[cc][6] = hi.z, w[cc][7] = hi.w;
            }
            int shift = 0;   // the row is scaled by 2^shift
            if constexpr (BF16) {
                uint32_t ex = 0u;   // largest finite bf16 exponent field
#pragma unroll
                for (int cc = 0; cc < KC; ++cc)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t a = (w[cc][i] >> 7) & 0xffu, e = (w[cc][i] >> 23) & 0xffu;
                        ex = max(ex, max(a < 255u ? a : 0u, e < 255u ? e : 0u));
                    }
                ex = max(ex, __shfl_xor_sync(0xffffffffu, ex, 1));
                ex = max(ex, __shfl_xor_sync(0xffffffffu, ex, 2));
                shift = ex == 0u ? 0 : min(14 + 127 - static_cast<int>(ex), 126);
                const float up = exp2i(shift);
#pragma unroll
                for (int cc = 0; cc < KC; ++cc)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 x = unpack16<true>(w[cc][i]);
                        w[cc][i] = pack2<false>(x.x * up, x.y * up);
                    }
            }
#pragma unroll
            for (int cc = 0; cc < KC; ++cc)
#pragma unroll
                for (int i = 0; i < 8; ++i) qf[nt][cc][i] = w[cc][i];
            // lane 8t (row 2t) and lane 8t + 4 (row 2t + 1) know this lane's columns' shifts
            f_row[nt][0] = p.scale_log2 * exp2i(-__shfl_sync(0xffffffffu, shift, 8 * t));
            f_row[nt][1] = p.scale_log2 * exp2i(-__shfl_sync(0xffffffffu, shift, 8 * t + 4));
        }

        // running state of this lane's columns (rows 2t, 2t + 1 of each 8): m the
        // largest score, l the sum of 2^(score - m) over this lane's tokens, R
        // the largest score + log2(value scale), O^T scaled by 2^-R
        float m[NR][2], l[NR][2], R[NR][2], o[NR][MT][4];
#pragma unroll
        for (int nt = 0; nt < NR; ++nt) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m[nt][e] = -INFINITY;
                R[nt][e] = -INFINITY;
                l[nt][e] = 0.0f;
            }
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.0f;
        }

        for (; mine < end; mine += kWarps, ++it) {
            const int slot = it % ST;
            const int tok = seq_token(s, static_cast<int>(mine - unit0));
            // scales of the two 16-token halves, from the slot's lane
            const float fk[2] = {__shfl_sync(0xffffffffu, ks0, slot), __shfl_sync(0xffffffffu, ks1, slot)};
            const float lv[2] = {
                static_cast<float>(scale_exp(__shfl_sync(0xffffffffu, vs0, slot))),
                static_cast<float>(scale_exp(__shfl_sync(0xffffffffu, vs1, slot)))};
            const int bad_t = __shfl_sync(0xffffffffu, bad, slot);
            warp_wait(&full[slot], (it / ST) & 1, abort_flag, p.status);
            const uint32_t sk = smem_u32(ring + slot * C::kSlot), sv = sk + C::kHalf;

            // S^T: 2 halves of 16 tokens
            float sc[2][NR][4];
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
                for (int nt = 0; nt < NR; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[hf][nt][e] = 0.0f;
#pragma unroll
                for (int cc = 0; cc < KC; ++cc) {
                    const uint4 r0 = lds128(sk + hf * 16 * D + k_at[0][cc]);
                    const uint4 r1 = lds128(sk + hf * 16 * D + k_at[1][cc]);
                    const uint32_t x0[4] = {r0.x, r0.y, r0.z, r0.w}, x1[4] = {r1.x, r1.y, r1.z, r1.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t a0 = e4m3x2_to_f16x2(x0[i]), a2 = e4m3x2_hi_to_f16x2(x0[i]);
                        const uint32_t a1 = e4m3x2_to_f16x2(x1[i]), a3 = e4m3x2_hi_to_f16x2(x1[i]);
#pragma unroll
                        for (int nt = 0; nt < NR; ++nt)
                            mma16816(sc[hf][nt], a0, a1, a2, a3, qf[nt][cc][2 * i], qf[nt][cc][2 * i + 1]);
                    }
                }
            }
            // scores in log2 units; edge tiles hide what a row does not see
            const bool edge = bad_t != 0 || tok + kTile - 1 > s.first ||
                              (p.window > 0 && tok <= s.len - 1 - p.window && tok + kTile > p.sinks);
#pragma unroll
            for (int nt = 0; nt < NR; ++nt)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const float f0 = f_row[nt][0] * fk[hf], f1 = f_row[nt][1] * fk[hf];
                    sc[hf][nt][0] *= f0;
                    sc[hf][nt][1] *= f1;
                    sc[hf][nt][2] *= f0;
                    sc[hf][nt][3] *= f1;
                }
            if (edge) {
#pragma unroll
                for (int nt = 0; nt < NR; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int pos = s.first + (row0 + nt * 8 + 2 * t + (e & 1)) % p.Nq;
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            const int key = tok + hf * 16 + tok_a + 8 * (e >> 1);
                            const bool see = !((bad_t >> hf) & 1) && key <= pos &&
                                             (p.window <= 0 || key > pos - p.window || key < p.sinks);
                            if (!see) sc[hf][nt][e] = -INFINITY;
                        }
                    }
            }
            // running maxima: rescale only when one of them moves
            bool grow = false;
            float mx[NR][2], ax[NR][2];
#pragma unroll
            for (int nt = 0; nt < NR; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float h0 = fmaxf(sc[0][nt][e], sc[0][nt][e + 2]);
                    const float h1 = fmaxf(sc[1][nt][e], sc[1][nt][e + 2]);
                    mx[nt][e] = fmaxf(h0, h1);
                    ax[nt][e] = fmaxf(h0 + lv[0], h1 + lv[1]);
                    grow = grow || mx[nt][e] > m[nt][e] || ax[nt][e] > R[nt][e];
                }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int nt = 0; nt < NR; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float a = mx[nt][e], x = ax[nt][e];
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) {
                            a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, d));
                            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
                        }
                        const float m1 = fmaxf(m[nt][e], a), R1 = fmaxf(R[nt][e], x);
                        if (m1 > m[nt][e]) l[nt][e] *= ex2_ftz(m[nt][e] - m1);   // from -inf: 0 * 0
                        if (R1 > R[nt][e]) {
                            const float al = ex2_ftz(R[nt][e] - R1);
#pragma unroll
                            for (int i = 0; i < MT; ++i) {
                                o[nt][i][e] *= al;
                                o[nt][i][e + 2] *= al;
                            }
                        }
                        m[nt][e] = m1;
                        R[nt][e] = R1;
                    }
            }
            // p = 2^(s - m) into l; P^T = 2^(s + log2 vs - R), fp16 (at most 1: rounded by
            // 2^-11 of itself, and 2^-25 of the largest at the far end)
            uint32_t pf[2][NR][2];
#pragma unroll
            for (int nt = 0; nt < NR; ++nt) {
                float nm[2], nR[2][2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    nm[e] = m[nt][e] == -INFINITY ? 0.0f : m[nt][e];
                    const float r = R[nt][e] == -INFINITY ? 0.0f : R[nt][e];
                    nR[0][e] = lv[0] - r;
                    nR[1][e] = lv[1] - r;
                }
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    float w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        l[nt][e & 1] += ex2_ftz(sc[hf][nt][e] - nm[e & 1]);
                        w[e] = ex2_ftz(sc[hf][nt][e] + nR[hf][e & 1]);
                    }
                    pf[hf][nt][0] = movmatrix_trans(pack2<false>(w[0], w[1]));
                    pf[hf][nt][1] = movmatrix_trans(pack2<false>(w[2], w[3]));
                }
            }
            // O^T += V^T P^T
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                uint32_t r[4][VB / 4];   // tokens 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t a = sv + hf * 16 * D + (i >> 1) * 8 * D + v_at[i & 1];
                    if constexpr (VB == 16) {
                        const uint4 x = lds128(a);
                        r[i][0] = x.x, r[i][1] = x.y, r[i][2] = x.z, r[i][3] = x.w;
                    } else {
                        const uint2 x = lds64(a);
                        r[i][0] = x.x, r[i][1] = x.y;
                    }
                }
                if (edge) {
                    // rows no query sees may hold anything, NaN too: zero them
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int key = tok + hf * 16 + (i >> 1) * 8 + ((i & 1) ? tok_v1 : tok_v0);
                        if (((bad_t >> hf) & 1) || key >= s.len || (key < s.lo && key >= p.sinks)) {
#pragma unroll
                            for (int j = 0; j < VB / 4; ++j) r[i][j] = 0u;
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < VB / 4; ++j) {
                    // pairs of tokens for each of the word's 4 dimensions
                    const uint32_t a01 = __byte_perm(r[0][j], r[1][j], 0x5140);
                    const uint32_t a23 = __byte_perm(r[0][j], r[1][j], 0x7362);
                    const uint32_t b01 = __byte_perm(r[2][j], r[3][j], 0x5140);
                    const uint32_t b23 = __byte_perm(r[2][j], r[3][j], 0x7362);
                    const uint32_t a0 = e4m3x2_to_f16x2(a01), a1 = e4m3x2_hi_to_f16x2(a01);
                    const uint32_t a2 = e4m3x2_to_f16x2(b01), a3 = e4m3x2_hi_to_f16x2(b01);
                    const uint32_t c0 = e4m3x2_to_f16x2(a23), c1 = e4m3x2_hi_to_f16x2(a23);
                    const uint32_t c2 = e4m3x2_to_f16x2(b23), c3 = e4m3x2_hi_to_f16x2(b23);
#pragma unroll
                    for (int nt = 0; nt < NR; ++nt) {
                        mma16816(o[nt][2 * j], a0, a1, a2, a3, pf[hf][nt][0], pf[hf][nt][1]);
                        mma16816(o[nt][2 * j + 1], c0, c1, c2, c3, pf[hf][nt][0], pf[hf][nt][1]);
                    }
                }
            }
            __syncwarp();   // every lane has read the slot
            if (lane == slot) issue();
        }

        // ---- the unit ends here for this CTA: combine the 8 warps
        const bool whole = unit0 >= g0 && unit1 <= g1;
        const int part = 2 * c + (unit0 <= g0 ? 0 : 1);
#pragma unroll 1
        for (int nt = 0; nt < NR; ++nt) {
            if (row0 + nt * 8 >= p.rows) break;
            float inv[2], lse2[2];
            // (nt is a run-time index here: pick the registers)
            float mm[2], ll[2], RR[2], oo[MT][4];
#pragma unroll
            for (int k = 0; k < NR; ++k)
                if (k == nt) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        mm[e] = m[k][e];
                        ll[e] = l[k][e];
                        RR[e] = R[k][e];
                    }
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) oo[i][e] = o[k][i][e];
                }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = ll[e];
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
                lse2[e] = x == 0.0f ? -INFINITY : mm[e] + lg2_approx(x);   // a NaN stays one
                inv[e] = x == 0.0f ? 0.0f : ex2_ftz(RR[e] - mm[e]) / x;
            }
            if (g == 0) {
                s_lse[warp * 8 + 2 * t] = lse2[0];
                s_lse[warp * 8 + 2 * t + 1] = lse2[1];
            }
#pragma unroll 1
            for (int half = 0; half < D / 64; ++half) {
                // dimensions VB g + 8 half .. + 7 of rows 2t, 2t + 1 (64 columns in all)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float x[4];
#pragma unroll
                    for (int k = 0; k < D / 64; ++k)
                        if (k == half) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) x[e] = oo[4 * k + i][e] * inv[e & 1];
                        }
                    float* at = s_merge + (warp * 8 + 2 * t) * 64 + 8 * g + 2 * i;
                    *reinterpret_cast<float2*>(at) = make_float2(x[0], x[2]);
                    *reinterpret_cast<float2*>(at + 64) = make_float2(x[1], x[3]);
                }
                __syncthreads();
                // 256 threads: row threadIdx / 32, two columns each
                const int r = warp, row = row0 + nt * 8 + r;
                float M = -INFINITY;
#pragma unroll
                for (int k = 0; k < kWarps; ++k) M = fmaxf(M, s_lse[k * 8 + r]);
                float sum = 0.0f, ox = 0.0f, oy = 0.0f;
#pragma unroll
                for (int k = 0; k < kWarps; ++k) {
                    const float L = s_lse[k * 8 + r];
                    const float wk = L == -INFINITY ? 0.0f : ex2_ftz(L - M);
                    const float2 x = *reinterpret_cast<const float2*>(s_merge + (k * 8 + r) * 64 + 2 * lane);
                    sum += wk;
                    ox = fmaf(wk, x.x, ox);
                    oy = fmaf(wk, x.y, oy);
                }
                const float n = sum == 0.0f ? 0.0f : 1.0f / sum;
                // column 2 lane of this half: dimension VB (lane / 4) + 8 half + 2 (lane % 4)
                const int dim = VB * g + 8 * half + 2 * t;
                const float L = sum == 0.0f ? -INFINITY : M + lg2_approx(sum);
                if (row < p.rows) {
                    if (whole) {
                        *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) +
                                                     (head_row + row) * D + dim) =
                            pack2<BF16>(ox * n, oy * n);
                        if (half == 0 && lane == 0) p.lse[head_row + row] = L * 0.6931471805599453f;
                    } else {
                        const int64_t pr = static_cast<int64_t>(part) * (8 * NR) + nt * 8 + r;
                        *reinterpret_cast<float2*>(p.part_o + pr * D + dim) = make_float2(ox * n, oy * n);
                        if (half == 0 && lane == 0) p.part_lse[pr] = L;
                    }
                }
                __syncthreads();
            }
        }
        unit0 = unit1;
        if (++u == U) {
            u = 0;
            ++b;
        }
    }
    // After a wait that gave up, copies may still be on their way into this
    // CTA's shared memory: wait for the last one of each slot (bounded).
    if (*abort_flag && lane < ST && issued > 0)
        mbar_wait_bounded(&full[lane], (issued - 1) & 1, p.status);
}

// Combines the partial results of the units that lie in several CTAs, one CTA per
// (sequence, unit); empty sequences get out = 0 and lse = -inf here.
template <int D, bool BF16, int NR>
__global__ void __launch_bounds__(256) kv8_merge_kernel(const AttnParams p) {
    const int U = p.Hkv * p.n_rb;
    const int b = static_cast<int>(blockIdx.x / U), u = static_cast<int>(blockIdx.x % U);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // tiles of all sequences, and of those before b
    int all = 0, before = 0;
    for (int i = threadIdx.x; i < p.B; i += 256) {
        const int n = seq_of(p, p.lens[i]).n;
        all += n;
        if (i < b) before += n;
    }
    all = __reduce_add_sync(0xffffffffu, all);
    before = __reduce_add_sync(0xffffffffu, before);
    __shared__ int s_sum[2][8];
    if (lane == 0) {
        s_sum[0][warp] = all;
        s_sum[1][warp] = before;
    }
    __syncthreads();
    all = before = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        all += s_sum[0][i];
        before += s_sum[1][i];
    }
    const Seq s = seq_of(p, p.lens[b]);
    const int64_t T = static_cast<int64_t>(all) * U;
    const int n_cta = shares(T, p.ctas);
    const int64_t first = static_cast<int64_t>(before) * U + static_cast<int64_t>(u) * s.n;
    const int h = u / p.n_rb, row0 = u % p.n_rb * (8 * NR);
    const int64_t head_row = (static_cast<int64_t>(b) * p.Hkv + h) * p.rows;
    const int rows = min(8 * NR, p.rows - row0);
    // Launched as a programmatic dependent of the attention kernel: what follows
    // reads its partial results.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int c0 = 0, c1 = -1;   // the CTAs that hold part of it
    if (s.n > 0) {
        c0 = static_cast<int>(((first + 1) * n_cta - 1) / T);
        c1 = static_cast<int>(((first + s.n) * n_cta - 1) / T);
        if (c0 == c1) return;   // written by that CTA
    }
    constexpr int V = D / 32;
    for (int r = warp; r < rows; r += 8) {
        float M = -INFINITY, sum = 0.0f, acc[V] = {};
        for (int cta = c0; cta <= c1; ++cta) {
            const int slot = 2 * cta + (cta == c0 && first > c0 * T / n_cta ? 1 : 0);
            const int64_t pr = static_cast<int64_t>(slot) * (8 * NR) + r;
            const float L = p.part_lse[pr];
            float x[V];
#pragma unroll
            for (int i = 0; i < V; ++i) x[i] = p.part_o[pr * D + lane * V + i];
            if (L == -INFINITY) continue;
            const float M1 = fmaxf(M, L), al = ex2_ftz(M - M1), w = ex2_ftz(L - M1);
            sum = sum * al + w;
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = acc[i] * al + w * x[i];
            M = M1;
        }
        const float n = sum == 0.0f ? 0.0f : 1.0f / sum;
        uint16_t* out = static_cast<uint16_t*>(p.out) + (head_row + row0 + r) * D + lane * V;
#pragma unroll
        for (int i = 0; i < V; i += 2)
            *reinterpret_cast<uint32_t*>(out + i) = pack2<BF16>(acc[i] * n, acc[i + 1] * n);
        if (lane == 0)
            p.lse[head_row + row0 + r] =
                sum == 0.0f ? -INFINITY : (M + lg2_approx(sum)) * 0.6931471805599453f;
    }
}

template <int D, bool BF16, int NR>
cudaError_t launch_attn(const CUtensorMap& tmK, const CUtensorMap& tmV, const AttnParams& p,
                        cudaStream_t stream) {
    auto kern = kv8_attn_kernel<D, BF16, NR>;
    const int smem = AttnCfg<D>::smem_bytes(p.B);
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    e = launch_kernel(kern, dim3(static_cast<unsigned>(p.ctas)), dim3(kAttnThreads), smem, stream,
                      tmK, tmV, p);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(p.B) * p.Hkv * p.n_rb);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv8_merge_kernel<D, BF16, NR>, p);
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

// One CTA per (pair, layer, keys or values), 4 vectors in flight a thread.
__global__ void __launch_bounds__(256) kv8_copy_kernel(const CopyParams p) {
    const int64_t id = blockIdx.x;
    const int which = static_cast<int>(id & 1);
    const int layer = static_cast<int>((id >> 1) % p.n_layers);
    const int i = static_cast<int>((id >> 1) / p.n_layers);
    if (i >= min(*p.count, p.max_count)) return;
    const int a = p.src[i], b = p.dst[i];
    if (a < 0 || a >= p.n_pages || b < 0 || b >= p.n_pages) {
        if (threadIdx.x == 0) atomicOr(p.status, kStatusPage);
        return;
    }
    const int64_t base = static_cast<int64_t>(layer) * p.n_pages;
    const uint4* from = reinterpret_cast<const uint4*>(p.pages[which]) + (base + a) * p.vecs;
    uint4* to = reinterpret_cast<uint4*>(p.pages[which]) + (base + b) * p.vecs;
    for (int x = threadIdx.x; x < p.vecs; x += 1024) {
        uint4 w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (x + 256 * k < p.vecs) w[k] = from[x + 256 * k];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (x + 256 * k < p.vecs) to[x + 256 * k] = w[k];
    }
    for (int x = threadIdx.x; x < p.Hkv; x += 256)
        p.scales[which][(base + b) * p.Hkv + x] = p.scales[which][(base + a) * p.Hkv + x];
}

// ------------------------------------------------------------------ host

template <int N>
bool aligned(const void* const (&ptrs)[N], uintptr_t bytes) {
    for (const void* p : ptrs)
        if (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) return false;
    return true;
}

bool page_ok(int page) { return page == 16 || page == 32 || page == 64 || page == 128; }

// Sizes of a cache that every call shares.
int check_cache(int B, int Hkv, int D, int page, int n_pages, int max_pages) {
    if (B <= 0 || Hkv <= 0 || D <= 0 || page <= 0 || n_pages <= 0 || max_pages <= 0)
        return ATTN_ERR_INVALID;
    if (D != 64 && D != 128) return ATTN_ERR_UNSUPPORTED;
    if (!page_ok(page)) return ATTN_ERR_UNSUPPORTED;
    // positions, and (page, head) coordinates of a copy, are 32-bit signed
    if (static_cast<int64_t>(max_pages) * page > (1ll << 30)) return ATTN_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(n_pages) * Hkv > (1ll << 30)) return ATTN_ERR_UNSUPPORTED;
    return ATTN_OK;
}

int device_sms() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0) {
        cudaGetLastError();
        return 0;
    }
    return sms;
}

size_t pad256(size_t b) { return (b + 255) & ~size_t(255); }

// 8-row tiles of a row block: 1, 2 or 4.
int row_tiles(int64_t rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : 4; }

size_t part_bytes(int64_t rows, int D, int ctas) {
    const size_t n = 2 * static_cast<size_t>(ctas) * 8 * row_tiles(rows);
    return pad256(n * D * sizeof(float)) + pad256(n * sizeof(float));
}

// The [n_pages * Hkv][page][D] bytes of a pool, boxes of min(page, 32) tokens.
int make_page_map(CUtensorMap* map, const void* base, int D, int page, int64_t pages) {
    return make_byte_map_public(map, base, D, page, pages, page < kTile ? page : kTile);
}

}  // namespace
}  // namespace tme

using namespace tme;

extern "C" int kv8_append(const void* k, const void* v, void* k_pages, void* v_pages,
                          float* k_scale, float* v_scale, const int* table, const int* lens,
                          const int* n_new, int B, int Hkv, int T, int D, int page, int n_pages,
                          int max_pages, long long stride_b, long long stride_h,
                          long long stride_t, int dtype, void* stream) {
    if (!k || !v || !k_pages || !v_pages || !k_scale || !v_scale || !table || !lens)
        return ATTN_ERR_INVALID;
    int rc = check_cache(B, Hkv, D, page, n_pages, max_pages);
    if (rc != ATTN_OK) return rc;
    if (T <= 0 || (dtype != ATTN_F16 && dtype != ATTN_BF16)) return ATTN_ERR_INVALID;
    if (stride_b < 0 || stride_h < 0 || stride_t < 0) return ATTN_ERR_INVALID;
    const void* ptrs[] = {k, v, k_pages, v_pages};
    const void* words[] = {k_scale, v_scale, table, lens, n_new};
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
    if (rows > (1 << 30) || units > (1 << 30)) return ATTN_ERR_UNSUPPORTED;
    return ATTN_OK;
}
}  // namespace
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
    const void* words[] = {k_scale, v_scale, table, lens};
    if (!aligned(ptrs, 16) || !aligned(words, 4)) return ATTN_ERR_ALIGN;
    if (workspace_bytes < kv8_attn_workspace_size(B, Hq, Hkv, Nq, D)) return ATTN_ERR_WORKSPACE;
    AttnParams p{};
    rc = device_setup_public(&p.status);
    if (rc != ATTN_OK) return rc;
    const int sms = device_sms();
    if (sms <= 0) return ATTN_ERR_CUDA;
    CUtensorMap tmK, tmV;
    const int64_t pages = static_cast<int64_t>(n_pages) * Hkv;
    if (make_page_map(&tmK, k_pages, D, page, pages) != ATTN_OK ||
        make_page_map(&tmV, v_pages, D, page, pages) != ATTN_OK)
        return ATTN_ERR_CUDA;
    const int64_t rows = static_cast<int64_t>(Hq / Hkv) * Nq;
    const int nr = row_tiles(rows);
    p.q = q;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.table = table;
    p.lens = lens;
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
    p.page = page;
    p.n_pages = n_pages;
    p.max_pages = max_pages;
    // no position is past max_pages * page <= 2^30: larger ones mean all
    const int most = max_pages * page;
    p.window = window > most ? most : window;
    p.sinks = sinks > most ? most : sinks;
    p.scale_log2 = scale * 1.4426950408889634f;
    const bool bf16 = dtype == ATTN_BF16;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaErrorInvalidValue;
#define TME_ATTN(d, b, n) \
    if (D == d && bf16 == b && nr == n) e = launch_attn<d, b, n>(tmK, tmV, p, st);
    TME_ATTN(64, false, 1)
    TME_ATTN(64, false, 2)
    TME_ATTN(64, false, 4)
    TME_ATTN(64, true, 1)
    TME_ATTN(64, true, 2)
    TME_ATTN(64, true, 4)
    TME_ATTN(128, false, 1)
    TME_ATTN(128, false, 2)
    TME_ATTN(128, false, 4)
    TME_ATTN(128, true, 1)
    TME_ATTN(128, true, 2)
    TME_ATTN(128, true, 4)
#undef TME_ATTN
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
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
    const unsigned ctas = static_cast<unsigned>(max_count) * n_layers * 2;
    return launch_kernel(kv8_copy_kernel, dim3(ctas), dim3(256), 0, static_cast<cudaStream_t>(stream),
                         p) == cudaSuccess
               ? ATTN_OK
               : ATTN_ERR_CUDA;
}
