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
    if (e != e_old) {   // the earlier tokens, to the larger scale
        const float redo = e_old - e < -100 ? 0.0f : exp2i(e_old - e);   // 448 * 2^-100 rounds to 0
#pragma unroll 1
        for (int pos = pos0; pos < start && pos < t0 + PAGE; pos += STEP) {
            uint2* at = reinterpret_cast<uint2*>(dst + (pos - pos0) / STEP * (kAppendThreads * 8));
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
// Work is counted in tiles of 32 or 64 tokens: sequence b has n_b visible ones (its sink
// tiles and then its window's, or all) for each of its U = Hkv * row blocks
// units.  The CTAs of one wave cut the concatenation of all (sequence, unit)
// lists into equal shares, so the balance does not depend on the lengths; a unit
// that lies in one CTA is written out directly, the others leave fp32 partial
// results that kv8_merge_kernel combines.
//
// Inside a CTA every warp works on its own: tiles w, w + W, ... of the share (W warps),
// through a ring of kStages (K, V) slots that it alone fills (TMA, an mbarrier
// each) and empties, so warps meet only where a unit ends.  Lane s owns slot s:
// it follows the slot's tiles through the table, a tile ahead of the copies it
// issues, so that no copy waits for its page id.
//
// Products run on mma.sync m16n8k16 with the tokens (scores) or the head
// dimensions (output) as its 16 rows and up to 8 query rows as its columns:
// S^T = K Q^T, O^T += V^T P^T.  The tensor core is not what bounds this kernel (a
// tile of 32 tokens is 8 KB at D = 128, about 350 cycles of one SM's share of the
// memory, and 32 small products), and registers hold P between the two products.
// With 32 query rows Q comes from shared memory instead of registers, which the
// accumulators fill.
// K and V become fp16 exactly (e4m3x2 -> f16x2); the dimensions of a K row and
// the tokens of a V column may meet the product in any order that its other
// operand shares, which is how 16-byte shared loads feed both (tok8 below).
//
// Bound by memory where caches are long: 32 sequences of 200 to 32768 tokens, 8 KV
// heads, D = 128 stream 962 MB in 154 us, 6.2 TB/s, 92% of a plain copy's rate; 8 of 64K
// tokens, 2 KV heads, D = 64, 134 MB in 31 us with the merge, calls in a graph.  Short ones by
// latency: 8 of 256 tokens take 4.9 us in a graph, launch, the chain of lengths, page ids and
// tiles, and merge.  With 32 query rows the same chain is three times as long (4 drafts of 7
// heads, 516 visible tokens: 17 us): a unit's end brings 8 warps' 32 rows together through
// shared memory, twice where a share of 4 tiles crosses into the next head, and all of that
// code runs once, so that warps stand 3.6 of 14 cycles per instruction waiting for
// instructions, 3.1 at barriers and 3.0 for shared memory.

// Warps per CTA: 12 of them with 2 slots each instead of 3 took 5.4 us against 4.8 (8
// sequences of 256 tokens, D = 64) and 51.4 against 50.4 (64K tokens, D = 128).
constexpr int kWarps = 8;
constexpr int kAttnThreads = kWarps * 32;
// Tiles per CTA, at least: 12 of them put 8 sequences of 256 tokens on 6 CTAs, several
// units each, 13.4 us against 5.4.
constexpr int kMinShare = 4;
constexpr int kMaxBatch = 1024;   // sequences per call (their tile counts live in shared memory)

struct AttnParams {
    const void* q;
    const float* k_scale;
    const float* v_scale;
    const int* table;
    const int* lens;
    const int* n_new;     // queries of a sequence that stand at a position (null: all Nq)
    const int* granted;   // 0: none does (null: 1)
    void* out;
    float* lse;
    float* part_o;     // [2 * ctas][rows of a block][D]
    float* part_lse;   // [2 * ctas][rows of a block], log2 domain
    unsigned int* status;
    int B, Hkv, rows, n_rb;   // rows = G * Nq of a KV head, row blocks
    int Nq, page_shift, n_pages, max_pages;
    int window, sinks, ctas, tile_shift;
    float scale_log2;
};

// The visible tiles of a sequence.
struct Seq {
    int len, nq, first;    // positions held; queries; position of the first one (may be < 0)
    int lo;                // first position inside a window of some query
    int n_sink, skip, n;   // tiles [0, n_sink) and [n_sink + skip, ...), n in all
};
__device__ __forceinline__ Seq seq_of(const AttnParams& p, int len, int nq) {
    Seq s;
    const int up = (1 << p.tile_shift) - 1;
    s.len = min(max(len, 0), p.max_pages << p.page_shift);
    s.nq = nq;
    s.first = s.len - nq;
    s.lo = p.window > 0 ? max(s.first - p.window + 1, 0) : 0;
    const int lo_tile = s.lo >> p.tile_shift;
    s.n_sink = min((p.sinks + up) >> p.tile_shift, lo_tile);
    s.skip = lo_tile - s.n_sink;
    s.n = nq > 0 ? ((s.len + up) >> p.tile_shift) - s.skip : 0;
    return s;
}
__device__ __forceinline__ bool step_granted(const AttnParams& p) { return !p.granted || *p.granted != 0; }
// Queries of sequence b of that length; -1: a count that does not fit.
__device__ __forceinline__ int queries_of(const AttnParams& p, bool granted, int b, int len) {
    if (!granted) return 0;
    if (!p.n_new) return p.Nq;
    const int n = p.n_new[b];
    return n < 0 || n > p.Nq || n > min(len, p.max_pages << p.page_shift) ? -1 : n;
}
__device__ __forceinline__ int seq_tile(const Seq& s, int v) {   // tile v of the list
    return v < s.n_sink ? v : v + s.skip;
}

// Shares: the T tiles are cut into n runs of q or q + 1 tiles (the first rem of them).
// T < 2^31 (checked on the host).
struct Shares {
    int n, q, rem;
    __device__ __forceinline__ Shares(int T, const AttnParams& p) {
        n = min((T + kMinShare - 1) / kMinShare, p.ctas);
        q = n > 0 ? static_cast<int>(static_cast<unsigned>(T) / static_cast<unsigned>(n)) : 0;
        rem = T - q * n;
    }
    __device__ __forceinline__ int begin(int c) const { return c * q + min(c, rem); }
    __device__ __forceinline__ int owner(int x) const {   // CTA that holds tile x
        const int big = rem * (q + 1);
        return x < big ? x / (q + 1) : rem + (x - big) / q;
    }
};

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
                 : "r"(a));
    return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 r;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a));
    return r;
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// 4-byte asynchronous copy global -> shared, and an arrival on a barrier once this
// thread's copies so far have landed (the barrier counts it).
__device__ __forceinline__ void cp_async4(void* dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)),
                 "l"(reinterpret_cast<uint64_t>(src))
                 : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// What a slot's lane leaves beside its tile: the scales and page ids of its 16-token
// quarters' boxes (up to 4), and which boxes hold nothing readable.
struct SlotInfo {
    float ks[4], vs[4];
    int pid[4];   // of the lane's next tile
    int bad;      // bit i: box i
    int pad[3];
};

// Tokens of a tile: 8 KB of keys and values (a warp's share of the loop's fixed work
// is then the same for both head dimensions), 4 KB where 32 rows' scores leave no
// registers for more.
template <int D, int NR>
constexpr int tile_tokens() { return D == 64 && NR < 4 ? 64 : 32; }

template <int D, int NR>
struct AttnCfg {
    static constexpr int kTile = tile_tokens<D, NR>();
    // 192 KB of slots; 128 KB with more rows, whose combination takes more room
    static constexpr int kStages = (NR == 1 ? 192 : 128) * 1024 / kWarps / (2 * D * kTile);
    static constexpr int kHalf = kTile * D;         // bytes of K (or V) of a tile
    static constexpr bool kQSmem = NR == 4;
    static constexpr int kSlot = 2 * kHalf;
    static constexpr int kRing = kWarps * kStages * kSlot;          // 192 KB
    static constexpr int kMergeOff = kRing;                         // [warp][8 NR rows][64] fp32
    static constexpr int kLseOff = kMergeOff + kWarps * NR * 8 * 64 * 4;
    static constexpr int kInfoOff = kLseOff + kWarps * NR * 8 * 4;  // a slot each
    static constexpr int kQOff = kInfoOff + kWarps * kStages * static_cast<int>(sizeof(SlotInfo));
    static constexpr int kBarOff = kQOff + (kQSmem ? NR * 8 * D * 2 + NR * 8 * 4 : 0);
    static constexpr int kMiscOff = kBarOff + kWarps * kStages * 8;
    static constexpr int kPreOff = kMiscOff + 8 * kWarps;                   // B + 1 ints, then 2 B
    static constexpr int smem_bytes(int B) { return kPreOff + (3 * B + 1) * 4; }
    static_assert(smem_bytes(kMaxBatch) <= 227 * 1024, "shared memory of a CTA");
};

// ONE: a tile lies in one page (page >= the tile's tokens); else it takes 2 or 4 boxes.
template <int D, bool BF16, int NR, bool ONE>
__global__ void __launch_bounds__(kAttnThreads, 1)
    kv8_attn_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                    const AttnParams p) {
    using C = AttnCfg<D, NR>;
    constexpr int ST = C::kStages, kTile = C::kTile;
    constexpr int NQ = kTile / 16;     // 16-token quarters of a tile (2 or 4)
    constexpr int KC = D / 64;         // 16-byte chunks of a K row per lane
    constexpr int MT = D / 16;         // 16-dimension tiles of O^T
    constexpr int VB = D / 8;          // bytes of a V row per lane (16 or 8)
    extern __shared__ __align__(1024) uint8_t smem[];
    float* s_merge = reinterpret_cast<float*>(smem + C::kMergeOff);   // [warp][8 NR rows][64]
    float* s_lse = reinterpret_cast<float*>(smem + C::kLseOff);       // [warp][8 NR rows]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOff) + warp * ST;   // this warp's slots
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMiscOff) + warp;
    int* s_warp = reinterpret_cast<int*>(smem + C::kMiscOff + 4 * kWarps);   // [kWarps]
    int* s_pre = reinterpret_cast<int*>(smem + C::kPreOff);           // [B + 1] tiles before
    int* s_len = s_pre + p.B + 1;                                     // [B]
    int* s_nq = s_len + p.B;                                          // [B] queries

    if (lane == 0) {
        // a slot's phase: its copies' bytes, and its lane's small copies
        for (int i = 0; i < ST; ++i) mbar_init(&full[i], 2);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    // Launched as a programmatic dependent of the kernel before it (an append, as
    // a rule), whose writes it reads from here on; the merge may set up already.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    // exclusive prefix sums of the sequences' tile counts
    const bool granted = step_granted(p);
    int carry = 0;
    for (int b0 = 0; b0 < p.B; b0 += kAttnThreads) {
        const int b = b0 + static_cast<int>(threadIdx.x);
        int len = 0, nq = 0;
        if (b < p.B) {
            len = p.lens[b];
            nq = queries_of(p, granted, b, len);
            if (blockIdx.x == 0 && (len < 0 || len > p.max_pages << p.page_shift || nq < 0))
                atomicOr(p.status, kStatusPage);
        }
        const int n = b < p.B ? seq_of(p, len, nq).n : 0;
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
        if (b < p.B) {
            s_pre[b] = before + x - n;
            s_len[b] = len;
            s_nq[b] = nq;
        }
        carry = all;
        if (b0 + kAttnThreads < p.B) __syncthreads();   // s_warp is written again
    }
    if (threadIdx.x == 0) s_pre[p.B] = carry;
    __syncthreads();
    const int U = p.Hkv * p.n_rb;
    const Shares sh(carry * U, p);
    const int c = static_cast<int>(blockIdx.x);
    if (c >= sh.n) return;   // nothing in flight, no barrier left
    const int g0 = sh.begin(c), g1 = sh.begin(c + 1);

    // KV head of a unit (unit = head * n_rb + row block; one block, as a rule)
    auto head_of = [&](int u_) { return p.n_rb == 1 ? u_ : u_ / p.n_rb; };

    // ---- the first unit, and Q of a unit as B fragments: lane (g, t) holds
    // dimensions 16 (t + 4 cc) .. + 15 of row g of each 8.  The raw rows are asked
    // for ahead of their unit; make_q makes them fp16.  bf16 rows are scaled by a
    // power of two first (their largest magnitude to [2^14, 2^15)), which the
    // scores take back: fp16 then holds every value down to 2^-28 of the row's
    // largest exactly.  They stay in registers, or (kQSmem) warp w prepares the 8
    // rows w and leaves them in shared memory as [row tile][word pair][lane], and
    // the factors behind them.
    int b = 0;   // the last sequence that starts at or before g0: not an empty one
    for (int hi = p.B - 1; b < hi;) {
        const int mid = (b + hi + 1) >> 1;
        if (s_pre[mid] * U <= g0) b = mid;
        else hi = mid - 1;
    }
    const int n_first = s_pre[b + 1] - s_pre[b];
    int u = static_cast<int>(static_cast<unsigned>(g0 - s_pre[b] * U) / static_cast<unsigned>(n_first));
    const int v_first = g0 - s_pre[b] * U - u * n_first;
    int unit0 = g0 - v_first;   // the unit's first tile in the concatenated lists
    constexpr int QN = C::kQSmem ? 1 : NR;
    uint32_t qf[QN][KC][8];
    float f_row[NR][2];   // softmax scale of this lane's score columns 2t, 2t + 1
    uint32_t* s_q = reinterpret_cast<uint32_t*>(smem + C::kQOff);
    float* s_f = reinterpret_cast<float*>(smem + C::kQOff + NR * 8 * D * 2);
    auto load_q = [&](int b_, int u_) {
        const int h_ = head_of(u_);
        const int64_t head = (static_cast<int64_t>(b_) * p.Hkv + h_) * p.rows;
#pragma unroll
        for (int nt = 0; nt < QN; ++nt) {
            if (C::kQSmem && warp >= NR) continue;
            const int r = (u_ - h_ * p.n_rb) * (8 * NR) + (C::kQSmem ? warp : nt) * 8 + g;
#pragma unroll
            for (int cc = 0; cc < KC; ++cc) {
                const uint4* src = reinterpret_cast<const uint4*>(
                    static_cast<const uint16_t*>(p.q) + (head + r) * D + 16 * (t + 4 * cc));
                const uint4 z = make_uint4(0u, 0u, 0u, 0u);
                const uint4 lo = r < p.rows ? src[0] : z, hi = r < p.rows ? src[1] : z;
                uint32_t* w = qf[nt][cc];
                w[0] = lo.x, w[1] = lo.y, w[2] = lo.z, w[3] = lo.w;
                w[4] = hi.x, w[5] = hi.y, w[6] = hi.z, w[7] = hi.w;
            }
        }
    };
    auto make_q = [&]() {
#pragma unroll
        for (int nt = 0; nt < QN; ++nt) {
            if (C::kQSmem && warp >= NR) continue;
            int shift = 0;   // the row is scaled by 2^shift
            if constexpr (BF16) {
                uint32_t ex = 0u;   // largest finite bf16 exponent field
#pragma unroll
                for (int cc = 0; cc < KC; ++cc)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t x = qf[nt][cc][i];
                        const uint32_t a = (x >> 7) & 0xffu, e = (x >> 23) & 0xffu;
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
                        const float2 x = unpack16<true>(qf[nt][cc][i]);
                        qf[nt][cc][i] = pack2<false>(x.x * up, x.y * up);
                    }
            }
            if constexpr (C::kQSmem) {
#pragma unroll
                for (int cc = 0; cc < KC; ++cc)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        *reinterpret_cast<uint2*>(s_q + ((warp * KC + cc) * 4 + i) * 64 + 2 * lane) =
                            make_uint2(qf[0][cc][2 * i], qf[0][cc][2 * i + 1]);
                if (t == 0) s_f[warp * 8 + g] = p.scale_log2 * exp2i(-shift);
            } else {
                // lane 8t (row 2t) and lane 8t + 4 (row 2t + 1) know this lane's columns' shifts
                f_row[nt][0] = p.scale_log2 * exp2i(-__shfl_sync(0xffffffffu, shift, 8 * t));
                f_row[nt][1] = p.scale_log2 * exp2i(-__shfl_sync(0xffffffffu, shift, 8 * t + 4));
            }
        }
        if constexpr (C::kQSmem) {
            __syncthreads();   // (barriers of the previous unit's end came after its last read)
#pragma unroll
            for (int nt = 0; nt < NR; ++nt) {
                f_row[nt][0] = s_f[nt * 8 + 2 * t];
                f_row[nt][1] = s_f[nt * 8 + 2 * t + 1];
            }
        }
    };
    load_q(b, u);

    // ---- this lane's slot (lanes 0 .. ST - 1).  Page ids and scales travel by
    // asynchronous copies into the slot's SlotInfo: a load into a register would
    // hold up every lane that reads its own copy of that register.
    uint8_t* ring = smem + warp * (ST * C::kSlot);
    SlotInfo* infos = reinterpret_cast<SlotInfo*>(smem + C::kInfoOff) + warp * ST;
    const int box_shift = ONE ? p.tile_shift : p.page_shift;   // tokens per TMA box
    const int boxes = ONE ? 1 : kTile >> box_shift;
    // quarters that a box covers: quarter hf lies in box hf >> q_shift
    const int q_shift = box_shift - 4;
    int left = 0;                               // tiles of this lane not issued yet
    int nb = 0, nu = 0, nv = 0, nh = 0, nn = 0; // the next one: sequence, unit, list index; KV head; list length
    int n_sink = 0, n_skip = 0, n_len = 0, n_lo = 0;   // of its sequence (Seq)
    const int* nrow = nullptr;                  // and its table row
    int ntok = 0, nseen = 0;                    // its first token; boxes some query sees
    int issued = 0;
    auto enter = [&]() {   // a new sequence
        const Seq x = seq_of(p, s_len[nb], s_nq[nb]);
        nn = x.n;
        n_sink = x.n_sink;
        n_skip = x.skip;
        n_len = x.len;
        n_lo = x.lo;
        nrow = p.table + static_cast<int64_t>(nb) * p.max_pages;
    };
    // Asks for the page ids of the next tile; a box no query sees need not have a page.
    auto fetch = [&]() {
        if (left == 0) return;
        if (nv >= nn) {
            do {
                nv -= nn;
                if (++nu == U) {
                    nu = 0;
                    do ++nb;
                    while (s_pre[nb + 1] == s_pre[nb]);
                    enter();
                }
            } while (nv >= nn);
            nh = head_of(nu);
        }
        ntok = (nv < n_sink ? nv : nv + n_skip) << p.tile_shift;
        if constexpr (ONE) {
            cp_async4(&infos[lane].pid[0], nrow + (ntok >> p.page_shift));
        } else {
            nseen = 0;
            for (int i = 0; i < boxes; ++i) {
                const int x = ntok + (i << box_shift);
                if (x < n_len && (x + (1 << box_shift) > n_lo || x < p.sinks)) {
                    nseen |= 1 << i;
                    cp_async4(&infos[lane].pid[i], nrow + (x >> p.page_shift));
                }
            }
        }
        cp_async_commit();
    };
    const int n_heads = p.n_pages * p.Hkv;   // past the pool copies fill zeros
    const uint32_t dst0 = smem_u32(ring + lane * C::kSlot);
    auto issue = [&]() {
        if (left == 0) return;
        --left;
        SlotInfo* in = infos + lane;
        cp_async_wait_all();   // the ids, asked for a whole turn of the ring ago
        const volatile int* pids = in->pid;
        int bad = 0;
        if constexpr (ONE) {
            const int pid = pids[0];
            if (pid < 0 || pid >= p.n_pages) {
                bad = 1;
                in->ks[0] = in->vs[0] = 1.0f;
                atomicOr(p.status, kStatusPage);
            }
            in->bad = bad;
            mbar_arrive_expect_tx(&full[lane], C::kSlot);   // releases the stores above, too
            const int y = ntok & ((1 << p.page_shift) - 1);
            const int z = bad ? n_heads : pid * p.Hkv + nh;
            tma_load_3d_at(&tmK, &full[lane], dst0, 0, y, z);
            tma_load_3d_at(&tmV, &full[lane], dst0 + C::kHalf, 0, y, z);
            if (!bad) {
                cp_async4(&in->ks[0], p.k_scale + z);
                cp_async4(&in->vs[0], p.v_scale + z);
            }
        } else {
            for (int i = 0; i < boxes; ++i) {
                const int pid = (nseen >> i) & 1 ? pids[i] : -1;
                if (pid < 0 || pid >= p.n_pages) {
                    bad |= 1 << i;
                    in->ks[i] = in->vs[i] = 1.0f;
                    if ((nseen >> i) & 1) atomicOr(p.status, kStatusPage);
                }
            }
            in->bad = bad;
            mbar_arrive_expect_tx(&full[lane], C::kSlot);
            for (int i = 0; i < boxes; ++i) {
                const bool ok = !((bad >> i) & 1);
                const int z = ok ? pids[i] * p.Hkv + nh : n_heads;
                const uint32_t at = dst0 + (i << box_shift) * D;   // a box is a page: row 0
                tma_load_3d_at(&tmK, &full[lane], at, 0, 0, z);
                tma_load_3d_at(&tmV, &full[lane], at + C::kHalf, 0, 0, z);
                if (ok) {
                    cp_async4(&in->ks[i], p.k_scale + z);
                    cp_async4(&in->vs[i], p.v_scale + z);
                }
            }
        }
        cp_async_arrive(&full[lane]);
        ++issued;
        nv += kWarps * ST;
        fetch();
    };
    if (lane < ST) {
        const int first = g0 + warp + kWarps * lane;
        if (first < g1) {
            left = (g1 - first + kWarps * ST - 1) / (kWarps * ST);
            nb = b;
            nu = u;
            nv = v_first + first - g0;   // fetch carries it into later units
            nh = head_of(nu);
            enter();
        }
        fetch();
        issue();
    }

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
    int mine = g0 + warp;       // this warp's next tile
    int slot = 0;               // of that tile
    uint32_t phase = 0;         // and its turn of the ring
    while (unit0 < g1) {
        const Seq s = seq_of(p, s_len[b], s_nq[b]);
        const int h = head_of(u), row0 = (u - h * p.n_rb) * (8 * NR);
        const int unit1 = unit0 + s.n, end = min(unit1, g1);
        const int64_t head_row = (static_cast<int64_t>(b) * p.Hkv + h) * p.rows;   // of q, out, lse
        make_q();

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

        for (; mine < end; mine += kWarps) {
            const int tok = seq_tile(s, mine - unit0) * kTile;
            warp_wait(&full[slot], phase, abort_flag, p.status);
            const uint32_t sk = smem_u32(ring + slot * C::kSlot), sv = sk + C::kHalf;
            const volatile SlotInfo* in = infos + slot;
            const int bad = in->bad;
            float fk[NQ], lv[NQ];   // of each quarter: key scale, log2 of the value scale
            if constexpr (ONE) {
                const float a = in->ks[0], e = static_cast<float>(scale_exp(in->vs[0]));
#pragma unroll
                for (int hf = 0; hf < NQ; ++hf) {
                    fk[hf] = a;
                    lv[hf] = e;
                }
            } else {
#pragma unroll
                for (int hf = 0; hf < NQ; ++hf) {
                    fk[hf] = in->ks[hf >> q_shift];
                    lv[hf] = static_cast<float>(scale_exp(in->vs[hf >> q_shift]));
                }
            }
            // bit hf: the quarter has no readable page
            auto bad_quarter = [&](int hf) { return ONE ? bad != 0 : ((bad >> (hf >> q_shift)) & 1) != 0; };

            // S^T of the tile's quarters
            float sc[NQ][NR][4];
#pragma unroll
            for (int hf = 0; hf < NQ; ++hf)
#pragma unroll
                for (int nt = 0; nt < NR; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[hf][nt][e] = 0.0f;
#pragma unroll
            for (int cc = 0; cc < KC; ++cc) {
                uint4 x[NQ][2];
#pragma unroll
                for (int hf = 0; hf < NQ; ++hf) {
                    x[hf][0] = lds128(sk + hf * 16 * D + k_at[0][cc]);
                    x[hf][1] = lds128(sk + hf * 16 * D + k_at[1][cc]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint2 qv[NR];
#pragma unroll
                    for (int nt = 0; nt < NR; ++nt) {
                        if constexpr (C::kQSmem)
                            qv[nt] = lds64(smem_u32(s_q + ((nt * KC + cc) * 4 + i) * 64 + 2 * lane));
                        else
                            qv[nt] = make_uint2(qf[nt][cc][2 * i], qf[nt][cc][2 * i + 1]);
                    }
#pragma unroll
                    for (int hf = 0; hf < NQ; ++hf) {
                        const uint32_t x0 = i == 0   ? x[hf][0].x
                                            : i == 1 ? x[hf][0].y
                                            : i == 2 ? x[hf][0].z
                                                     : x[hf][0].w;
                        const uint32_t x1 = i == 0   ? x[hf][1].x
                                            : i == 1 ? x[hf][1].y
                                            : i == 2 ? x[hf][1].z
                                                     : x[hf][1].w;
                        const uint32_t a0 = e4m3x2_to_f16x2(x0), a2 = e4m3x2_hi_to_f16x2(x0);
                        const uint32_t a1 = e4m3x2_to_f16x2(x1), a3 = e4m3x2_hi_to_f16x2(x1);
#pragma unroll
                        for (int nt = 0; nt < NR; ++nt)
                            mma16816(sc[hf][nt], a0, a1, a2, a3, qv[nt].x, qv[nt].y);
                    }
                }
            }
            // scores in log2 units; edge tiles hide what a row does not see
            const bool edge = bad != 0 || tok + kTile - 1 > s.first || s.nq < p.Nq ||
                              (p.window > 0 && tok <= s.len - 1 - p.window && tok + kTile > p.sinks);
#pragma unroll
            for (int nt = 0; nt < NR; ++nt)
#pragma unroll
                for (int hf = 0; hf < NQ; ++hf) {
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
                        const int i = (row0 + nt * 8 + 2 * t + (e & 1)) % p.Nq;
                        const int pos = i < s.nq ? s.first + i : -1;
#pragma unroll
                        for (int hf = 0; hf < NQ; ++hf) {
                            const int key = tok + hf * 16 + tok_a + 8 * (e >> 1);
                            const bool see = !bad_quarter(hf) && key <= pos &&
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
                    float a = -INFINITY, x = -INFINITY;
#pragma unroll
                    for (int hf = 0; hf < NQ; ++hf) {
                        const float y = fmaxf(sc[hf][nt][e], sc[hf][nt][e + 2]);
                        a = fmaxf(a, y);
                        x = fmaxf(x, y + lv[hf]);
                    }
                    mx[nt][e] = a;
                    ax[nt][e] = x;
                    grow = grow || a > m[nt][e] || x > R[nt][e];
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
            uint32_t pf[NQ][NR][2];
#pragma unroll
            for (int nt = 0; nt < NR; ++nt) {
                float nm[2], nr[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    nm[e] = m[nt][e] == -INFINITY ? 0.0f : m[nt][e];
                    nr[e] = R[nt][e] == -INFINITY ? 0.0f : R[nt][e];
                }
#pragma unroll
                for (int hf = 0; hf < NQ; ++hf) {
                    float w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        l[nt][e & 1] += ex2_ftz(sc[hf][nt][e] - nm[e & 1]);
                        w[e] = ex2_ftz(sc[hf][nt][e] + (lv[hf] - nr[e & 1]));
                    }
                    pf[hf][nt][0] = movmatrix_trans(pack2<false>(w[0], w[1]));
                    pf[hf][nt][1] = movmatrix_trans(pack2<false>(w[2], w[3]));
                }
            }
            // O^T += V^T P^T
#pragma unroll
            for (int hf = 0; hf < NQ; ++hf) {
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
                        if (bad_quarter(hf) || key >= s.len || (key < s.lo && key >= p.sinks)) {
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
            if (++slot == ST) {
                slot = 0;
                phase ^= 1u;
            }
        }

        // ---- the unit ends here for this CTA: combine the warps.  The next unit's Q
        // is asked for first.
        const bool whole = unit0 >= g0 && unit1 <= g1;
        const int part = 2 * c + (unit0 <= g0 ? 0 : 1);
        unit0 = unit1;
        if (++u == U) {
            u = 0;
            do ++b;
            while (unit0 < g1 && s_pre[b + 1] == s_pre[b]);   // empty sequences
        }
        if (unit0 < g1) load_q(b, u);
        // Every warp's LSE of each row to shared memory; then lane i weighs row i of
        // the unit (mod 8 NR), and this lane's columns take their rows' factors.
        float up[NR][2];   // brings O^T to real units, then to the warp's share of the row
#pragma unroll
        for (int nt = 0; nt < NR; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = l[nt][e];
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
                if (g == 0)
                    s_lse[(warp * NR + nt) * 8 + 2 * t + e] =
                        x == 0.0f ? -INFINITY : m[nt][e] + lg2_approx(x);   // a NaN stays one
                up[nt][e] = x == 0.0f ? 0.0f : ex2_ftz(R[nt][e] - m[nt][e]) / x;
            }
        __syncthreads();
        float sum = 0.0f;   // of row lane % (8 NR): 0 when it sees nothing
        {
            const int i = lane % (8 * NR);
            float a[kWarps], M = -INFINITY;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                a[k] = s_lse[k * (8 * NR) + i];
                M = fmaxf(M, a[k]);
            }
#pragma unroll
            for (int k = 0; k < kWarps; ++k) sum += a[k] == -INFINITY ? 0.0f : ex2_ftz(a[k] - M);
            const float own = s_lse[warp * (8 * NR) + i];
            const float share = sum == 0.0f || own == -INFINITY ? 0.0f : ex2_ftz(own - M) / sum;
#pragma unroll
            for (int nt = 0; nt < NR; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    up[nt][e] *= __shfl_sync(0xffffffffu, share, nt * 8 + 2 * t + e);
            if (warp == 0 && lane < 8 * NR && row0 + i < p.rows) {
                const float L = sum == 0.0f ? -INFINITY : M + lg2_approx(sum);
                if (whole) p.lse[head_row + row0 + i] = L * 0.6931471805599453f;
                else p.part_lse[static_cast<int64_t>(part) * (8 * NR) + i] = L;
            }
        }
        // the warps' shares of O, 64 dimensions at a time: per lane the next 8 of its
        // dimensions of rows 2t, 2t + 1 of each 8
#pragma unroll
        for (int half = 0; half < D / 64; ++half) {
            if (half > 0) __syncthreads();   // the previous step's sums are made
#pragma unroll
            for (int nt = 0; nt < NR; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float(&x)[4] = o[nt][4 * half + i];
                    float* at = s_merge + ((warp * NR + nt) * 8 + 2 * t) * 64 + 8 * g + 2 * i;
                    *reinterpret_cast<float2*>(at) = make_float2(x[0] * up[nt][0], x[2] * up[nt][0]);
                    *reinterpret_cast<float2*>(at + 64) = make_float2(x[1] * up[nt][1], x[3] * up[nt][1]);
                }
            __syncthreads();
            // a row per warp and turn, two columns a lane: dimension VB g + 8 half + 2t
            for (int r = warp; r < min(8 * NR, p.rows - row0); r += kWarps) {
                float ox = 0.0f, oy = 0.0f;
#pragma unroll
                for (int k = 0; k < kWarps; ++k) {
                    const float2 x =
                        *reinterpret_cast<const float2*>(s_merge + (k * NR * 8 + r) * 64 + 2 * lane);
                    ox += x.x;
                    oy += x.y;
                }
                // a row that sees nothing is 0 beside a NaN that others see, too
                if (__shfl_sync(0xffffffffu, sum, r) == 0.0f) ox = oy = 0.0f;
                const int dim = VB * g + 8 * half + 2 * t;
                if (whole)
                    *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) +
                                                 (head_row + row0 + r) * D + dim) = pack2<BF16>(ox, oy);
                else
                    *reinterpret_cast<float2*>(
                        p.part_o + (static_cast<int64_t>(part) * (8 * NR) + r) * D + dim) =
                        make_float2(ox, oy);
            }
        }
    }
    // After a wait that gave up, copies may still be on their way into this
    // CTA's shared memory: wait for the last one of each slot (bounded).
    if (*abort_flag && lane < ST && issued > 0)
        mbar_wait_bounded(&full[lane], (issued - 1) & 1, p.status);
}

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
    const Shares sh(all * U, p);
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

template <int D, bool BF16, int NR, bool ONE>
cudaError_t launch_attn(const CUtensorMap& tmK, const CUtensorMap& tmV, AttnParams p,
                        cudaStream_t stream) {
    auto kern = kv8_attn_kernel<D, BF16, NR, ONE>;
    p.tile_shift = AttnCfg<D, NR>::kTile == 64 ? 6 : 5;
    const int smem = AttnCfg<D, NR>::smem_bytes(p.B);
    static SmemLimit limit;
    cudaError_t e = limit.raise(kern, AttnCfg<D, NR>::smem_bytes(kMaxBatch));
    if (e != cudaSuccess) return e;
    e = launch_dependent(kern, p.ctas, kAttnThreads, smem, stream, tmK, tmV, p);
    if (e != cudaSuccess) return e;
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

// SM count of the current device (0 without one), asked for once per device.
int device_sms() {
    static std::atomic<int> known[64];
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    if (dev < 64 && (sms = known[dev].load(std::memory_order_relaxed)) > 0) return sms;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0) {
        cudaGetLastError();
        return 0;
    }
    if (dev < 64) known[dev].store(sms, std::memory_order_relaxed);
    return sms;
}

size_t pad256(size_t b) { return (b + 255) & ~size_t(255); }

// 8-row tiles of a row block: 1, 2 or 4.
int row_tiles(int64_t rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : 4; }

size_t part_bytes(int64_t rows, int D, int ctas) {
    const size_t n = 2 * static_cast<size_t>(ctas) * 8 * row_tiles(rows);
    return pad256(n * D * sizeof(float)) + pad256(n * sizeof(float));
}

// The [n_pages * Hkv][page][D] bytes of a pool, boxes of at most a tile's tokens.
int make_page_map(CUtensorMap* map, const void* base, int D, int page, int64_t pages, int nr) {
    const int tile = D == 64 && nr < 4 ? tile_tokens<64, 1>() : tile_tokens<128, 1>();
    return make_byte_map_public(map, base, D, page, pages, page < tile ? page : tile);
}

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
    if (workspace_bytes < kv8_attn_workspace_size(B, Hq, Hkv, Nq, D)) return ATTN_ERR_WORKSPACE;
    // the kernels count tiles of all sequences' table capacity in 32 bits
    if (static_cast<int64_t>(B) * Hkv * ((static_cast<int64_t>(Hq / Hkv) * Nq + 31) / 32) *
            ((static_cast<int64_t>(max_pages) * page + 31) / 32) > 0x7fffffffll)
        return ATTN_ERR_UNSUPPORTED;
    AttnParams p{};
    rc = device_setup_public(&p.status);
    if (rc != ATTN_OK) return rc;
    const int sms = device_sms();
    if (sms <= 0) return ATTN_ERR_CUDA;
    CUtensorMap tmK, tmV;
    const int64_t pages = static_cast<int64_t>(n_pages) * Hkv;
    const int64_t rows = static_cast<int64_t>(Hq / Hkv) * Nq;
    const int nr = row_tiles(rows);
    if (make_page_map(&tmK, k_pages, D, page, pages, nr) != ATTN_OK ||
        make_page_map(&tmV, v_pages, D, page, pages, nr) != ATTN_OK)
        return ATTN_ERR_CUDA;
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
    if (D == d && bf16 == b && nr == n)                                              \
        e = page >= tile_tokens<d, n>() ? launch_attn<d, b, n, true>(tmK, tmV, p, st) \
                                        : launch_attn<d, b, n, false>(tmK, tmV, p, st);
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
    const int sms = device_sms();
    const int64_t items = static_cast<int64_t>(max_count) * n_layers * 2;
    const int64_t most = static_cast<int64_t>(sms > 0 ? sms : 1) * kCopyCtasPerSm;
    return launch_dependent(kv8_copy_kernel, items < most ? items : most, kCopyThreads, 0,
                            static_cast<cudaStream_t>(stream), p) == cudaSuccess
               ? ATTN_OK
               : ATTN_ERR_CUDA;
}
