// kv8.cuh -- what the translation units of the paged 8-bit cache share: e4m3 and the
// pages' power-of-two scales on the device, the checks of a call on the host.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "../../include/kvcache.h"
#include "ptx.cuh"

namespace tme {

// abi.cu
int device_setup_public(unsigned int** status);

struct AttnParams;

// kv8.cu: checks a cache attention's arguments (the workspace for `needed` bytes) and fills its
// parameters.
int attn_params(AttnParams* p, const void* q, const void* k_pages, const void* v_pages,
                const float* k_scale, const float* v_scale, const int* table, const int* lens,
                const int* n_new, const int* granted, void* out, float* lse, void* workspace,
                size_t workspace_bytes, size_t needed, int B, int Hq, int Hkv, int Nq, int D, int page,
                int n_pages, int max_pages, float scale, int window, int sinks, int dtype);
// kv8_shared_attn.cu: the attention behind a shared prefix, without the merge.
int attn_launch_shared(const AttnParams& p, const void* k_pages, const void* v_pages, int D, int page, bool bf16,
                       cudaStream_t stream);

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

// A thread's tokens of a page before `end`, STEP apart from pos on (their bytes BYTES apart from `at`), to
// the larger scale 2^e.
template <int BYTES, int STEP>
__device__ __forceinline__ void raise_tokens(uint8_t* at, int pos, int end, int e_old, int e) {
    const float redo = e_old - e < -100 ? 0.0f : exp2i(e_old - e);   // 448 * 2^-100 rounds to 0
#pragma unroll 1
    for (; pos < end; pos += STEP, at += BYTES) {
        const uint2 o = *reinterpret_cast<const uint2*>(at);
        const uint32_t x[2] = {o.x, o.y};
        uint32_t r[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t y = x[j >> 1];
            const float2 f = f16x2_to_f32((j & 1) ? e4m3x2_hi_to_f16x2(y) : e4m3x2_to_f16x2(y));
            r[j] = f32_to_e4m3x2(f.x * redo, f.y * redo);
        }
        *reinterpret_cast<uint2*>(at) = make_uint2(r[0] | (r[1] << 16), r[2] | (r[3] << 16));
    }
}

// ------------------------------------------------------------------ attention

// Tiles per CTA, at least: 12 of them put 8 sequences of 256 tokens on 6 CTAs, several
// units each, 13.4 us against 5.4.
constexpr int kMinShare = 4;
constexpr int kMaxBatch = 1024;   // sequences per call (their tile counts live in shared memory)

}  // namespace

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
    // attention over a shared prefix (null: none): the plan, and the rows of sequences that
    // share, over the positions after their prefix
    const int* plan;
    int least_runs;    // runs that a plan's groups have to save in all,
    int least_members; // and sequences that each of them has to have, where the plan leaves the choice
    float* own_o;      // [B, Hq, Nq][D]
    float* own_lse;    // [B, Hq, Nq], log2 domain
    unsigned int* status;
    int B, Hkv, rows, n_rb;   // rows = G * Nq of a KV head, row blocks
    int Nq, page_shift, n_pages, max_pages;
    int window, sinks, ctas, tile_shift;
    float scale_log2;
};

namespace {

// The visible tiles of a sequence.
struct Seq {
    int len, nq, first;    // positions held; queries; position of the first one (may be < 0)
    int lo;                // first position inside a window of some query, or past the shared prefix
    int n_sink, skip, n;   // tiles [0, n_sink) and [n_sink + skip, ...), n in all
};
__device__ __forceinline__ Seq seq_of(const AttnParams& p, int len, int nq, int start = 0) {
    Seq s;
    const int up = (1 << p.tile_shift) - 1;
    s.len = min(max(len, 0), p.max_pages << p.page_shift);
    s.nq = nq;
    s.first = s.len - nq;
    s.lo = p.window > 0 ? max(s.first - p.window + 1, 0) : start;
    const int lo_tile = s.lo >> p.tile_shift;
    s.n_sink = min((p.sinks + up) >> p.tile_shift, lo_tile);
    s.skip = lo_tile - s.n_sink;
    s.n = nq > 0 ? max(((s.len + up) >> p.tile_shift) - s.skip, 0) : 0;
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
    __device__ __forceinline__ Shares(int T, int ctas, int least = kMinShare) {
        n = min((T + least - 1) / least, ctas);
        q = n > 0 ? static_cast<int>(static_cast<unsigned>(T) / static_cast<unsigned>(n)) : 0;
        rem = T - q * n;
    }
    __device__ __forceinline__ int begin(int c) const { return c * q + min(c, rem); }
    __device__ __forceinline__ int owner(int x) const {   // CTA that holds tile x
        const int big = rem * (q + 1);
        return x < big ? x / (q + 1) : rem + (x - big) / q;
    }
};

// Behind a shared prefix each warp of the attention has a share (up to 16 query rows; with
// more the CTA has), of this many tiles at least.
// Its units (a sequence's tiles of one KV head) begin with kOwnSteps steps beside their tiles: the queries
// and the rows of the unit before take about as long, and a short sequence brings a run of such units
// (128 sequences with 1 to 1000 positions of their own, 8 KV heads of 128: the whole call 87 us, 94.7
// with equal tiles; 1 step 89.6, 2 to 4 alike).  With more than 16 rows a CTA's eight warps end a unit
// together, which takes as long as some 32 tiles: 64 sequences of 20 to 1000 positions behind 8192, five queries, 32:8
// heads of 128, the whole call 125 us, 225 with equal tiles; with 200 positions each beside 32 sequences of 16384
// that share nothing 369 and 1341 (kv8_attn 563), 14:2 of 64 142 and 456 (203); 16 steps 495 and 170, 64 394 and 152.
constexpr int kAttnWarps = 8, kWarpMinShare = 2, kOwnSteps = 3, kOwnStepsCta = 32;
inline __host__ __device__ int own_steps(int rows) { return rows <= 16 ? kOwnSteps : kOwnStepsCta; }
inline __host__ __device__ int own_workers(int ctas, int rows) { return rows <= 16 ? ctas * kAttnWarps : ctas; }
__device__ __forceinline__ Shares own_shares(const AttnParams& p, int T) {
    return Shares(T, own_workers(p.ctas, p.rows), p.rows <= 16 ? kWarpMinShare : kMinShare);
}

// What kvp_find_shared leaves: a header (magic, groups, n_seqs, runs that all of them save or kPlanAlways), then
// arrays of n_seqs words.  Group g are the sequences members[first[g] .. + count[g]), in ascending order; the first
// `blocks[g]` runs of kShareBlock positions of all of them lie in the pages of the first one's table row.
constexpr int kShareBlock = 128;
constexpr int kPlanMagic = 0x5a4e0002;
constexpr int kPlanAlways = 0x7fffffff;   // a plan that is followed whatever it saves
struct Plan {
    const int* w;
    int n, least;   // sequences; members of a group that is followed
    __device__ __forceinline__ Plan(const int* words, int n_seqs, int least_members)
        : w(words), n(n_seqs), least(words[3] == kPlanAlways ? 0 : least_members) {}
    // Whether it is a plan for as many sequences at all, and whether it is worth while.
    __device__ __forceinline__ bool ok() const { return w[0] == kPlanMagic && w[2] == n; }
    __device__ __forceinline__ bool ok(int least_runs) const { return ok() && w[3] >= least_runs; }
    __device__ __forceinline__ int groups() const { return min(max(w[1], 0), n); }
    __device__ __forceinline__ int at(int array, int i) const { return w[4 + array * n + i]; }
    __device__ __forceinline__ int first(int g) const { return min(max(at(0, g), 0), n); }
    __device__ __forceinline__ int count(int g) const { return min(max(at(1, g), 0), n - first(g)); }
    // (masks, no branches: a load behind one would wait for what decides it)
    __device__ __forceinline__ int blocks(int g) const { return max(at(2, g), 0) & -static_cast<int>(at(1, g) >= least); }
    __device__ __forceinline__ int member(int i) const { return min(max(at(3, i), 0), n - 1); }
    __device__ __forceinline__ int group(int b) const { return min(at(4, b), n - 1); }   // -1: none
    __device__ __forceinline__ int rank(int b) const { return at(5, b); }
    // positions that sequence b shares (a multiple of kShareBlock), with how many others and itself
    __device__ __forceinline__ int start(int b) const {
        return max(at(6, b), 0) & ~(kShareBlock - 1) & -static_cast<int>(at(7, b) >= least);
    }
};
constexpr int kPlanArrays = 8, kPlanScratch = 3;

// ------------------------------------------------------------------ host

template <int N>
bool aligned(const void* const (&ptrs)[N], uintptr_t bytes) {
    for (const void* p : ptrs)
        if (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) return false;
    return true;
}

inline bool page_ok(int page) { return page == 16 || page == 32 || page == 64 || page == 128; }

// Sizes of a cache that every call shares.
inline int check_cache(int B, int Hkv, int D, int page, int n_pages, int max_pages) {
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
inline int device_sms() {
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

inline size_t pad256(size_t b) { return (b + 255) & ~size_t(255); }

// 8-row tiles of a row block: 1, 2 or 4.
inline int row_tiles(int64_t rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : 4; }

inline size_t part_bytes(int64_t rows, int D, int ctas) {
    const size_t n = 2 * static_cast<size_t>(ctas) * 8 * row_tiles(rows);
    return pad256(n * D * sizeof(float)) + pad256(n * sizeof(float));
}

}  // namespace
}  // namespace tme
