// kv8_attn.cuh -- the attention kernel of the paged 8-bit cache, for the plain call (kv8.cu) and
// for what sequences see behind a shared prefix (kv8_shared_attn.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn_internal.h"
#include "kv8.cuh"
#include "ptx.cuh"

namespace tme {

// abi.cu
int make_byte_map_public(CUtensorMap* map, const void* base, int D, int rows, int64_t groups,
                         int box_rows);

namespace {

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
constexpr int kWarps = kAttnWarps;
constexpr int kAttnThreads = kWarps * 32;
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
    static constexpr int kPreOff = kMiscOff + 8 * kWarps;                   // B + 1 ints, then 2 B or (SHARED) 3 B
    static constexpr int smem_bytes(int B, bool shared) { return kPreOff + ((shared ? 4 : 3) * B + 1) * 4; }
    static_assert(smem_bytes(kMaxBatch, true) <= 227 * 1024, "shared memory of a CTA");
};

// ONE: a tile lies in one page (page >= the tile's tokens); else it takes 2 or 4 boxes.
// SHARED: behind a shared prefix's attention (kv8_shared.cu): a sequence's tiles start after its prefix,
// and its rows go to own_o and own_lse in fp32, for the merge with the prefix's.  What is left behind
// a prefix is short, a few tiles a unit, and the end of a unit that 8 warps share costs more than its
// tiles: up to 16 query rows each warp therefore takes a share of its own, whose units it
// ends by itself (128 sequences of 1 to 1000 positions, 8 KV heads, D = 128: 77 us so, 36 alone).
template <int D, bool BF16, int NR, bool ONE, bool SHARED>
__global__ void __launch_bounds__(kAttnThreads, 1)
    kv8_attn_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                    const AttnParams p) {
    using C = AttnCfg<D, NR>;
    constexpr bool ALONE = SHARED && NR < 4;   // every warp has a share of its own (below)
    constexpr int ST = C::kStages, kTile = C::kTile;
    constexpr int STEP = ALONE ? 1 : kWarps;   // tiles from one of a warp's to its next
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
    int* s_held = reinterpret_cast<int*>(smem + C::kLseOff);          // SHARED (before s_lse is used): [kWarps]
    int* s_pre = reinterpret_cast<int*>(smem + C::kPreOff);           // [B + 1] tiles before
    int* s_len = s_pre + p.B + 1;                                     // [B]
    int* s_nq = s_len + p.B;                                          // [B] queries
    int* s_start = s_nq + p.B;                                        // SHARED: [B] positions of the prefix
    auto start_of = [&](int b_) { return SHARED ? s_start[b_] : 0; };
    // SHARED (up to 2^20 queries, 1024 sequences): beside them how many sequences before hold tiles
    constexpr int kNqBits = 21;
    static_assert(kMaxBatch <= 1 << (31 - kNqBits), "a word holds both");
    auto queries = [&](int b_) { return SHARED ? (s_nq[b_] & ((1 << kNqBits) - 1)) - 1 : s_nq[b_]; };

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
    // SHARED: that kernel is the shared prefix's, of which nothing is read here: it let
    // this one start after its own wait, so what was before it is complete, and is waited
    // for at the end, so that the merge finds both.
    if constexpr (!SHARED) asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    // exclusive prefix sums of the sequences' tile counts
    const bool granted = step_granted(p);
    int carry = 0, held = 0;   // tiles, SHARED: sequences with any
    for (int b0 = 0; b0 < p.B; b0 += kAttnThreads) {
        const int b = b0 + static_cast<int>(threadIdx.x);
        int len = 0, nq = 0, start = 0;
        if (b < p.B) {
            len = p.lens[b];
            nq = queries_of(p, granted, b, len);
            if constexpr (SHARED) {
                const Plan plan(p.plan, p.B, p.least_members);
                start = plan.start(b);   // (asked for beside the header)
                if (!plan.ok(p.least_runs)) start = 0;
            }
            if (blockIdx.x == 0 && (len < 0 || len > p.max_pages << p.page_shift || nq < 0))
                atomicOr(p.status, kStatusPage);
        }
        const int n = b < p.B ? seq_of(p, len, nq, start).n : 0;
        int x = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += y;
        }
        if (lane == 31) s_warp[warp] = x;
        int z = 0;   // SHARED: sequences before in the turn that hold tiles
        if constexpr (SHARED) {
            const unsigned any = __ballot_sync(0xffffffffu, n > 0);
            z = __popc(any & ((1u << lane) - 1u));
            if (lane == 0) s_held[warp] = __popc(any);
        }
        __syncthreads();
        int before = carry, all = carry;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            if (i < warp) before += s_warp[i];
            all += s_warp[i];
        }
        if constexpr (SHARED) {
            z += held;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) {
                if (i < warp) z += s_held[i];
                held += s_held[i];
            }
        }
        if (b < p.B) {
            s_pre[b] = before + x - n;
            s_len[b] = len;
            s_nq[b] = SHARED ? (nq + 1) | (z << kNqBits) : nq;
            if constexpr (SHARED) s_start[b] = start;
        }
        carry = all;
        if (b0 + kAttnThreads < p.B) __syncthreads();   // s_warp is written again
    }
    if (threadIdx.x == 0) s_pre[p.B] = carry;
    __syncthreads();
    const int U = p.Hkv * p.n_rb;
    constexpr int K = ALONE ? kOwnSteps : kOwnStepsCta;   // SHARED: a unit's steps beside its tiles
    const Shares sh = SHARED ? own_shares(p, (carry + K * held) * U) : Shares(carry * U, p.ctas);
    // (consecutive shares of warps on different SMs)
    const int c = static_cast<int>(blockIdx.x) + (ALONE ? warp * p.ctas : 0);
    // SHARED: the tile that step x of the concatenated units leads to; its sequence, KV head and place in its
    // list.  Two probes a lane (at most 1024 sequences).
    auto tile_at = [&](int x, int* b_, int* u_, int* v_) {
        auto steps = [&](int i) { return (s_pre[i] + K * (s_nq[i] >> kNqBits)) * U; };
        const int gap = (p.B + 31) >> 5, i = lane * gap;
        const int base = (__popc(__ballot_sync(0xffffffffu, i < p.B && steps(min(i, p.B - 1)) <= x)) - 1) * gap;
        const int k = base + lane;
        *b_ = base - 1 +
              __popc(__ballot_sync(0xffffffffu, lane < gap && k < p.B && steps(min(k, p.B - 1)) <= x));
        const int n = s_pre[*b_ + 1] - s_pre[*b_], off = x - steps(*b_);
        *u_ = static_cast<int>(static_cast<unsigned>(off) / static_cast<unsigned>(n + K));
        *v_ = max(off - *u_ * (n + K) - K, 0);
        return s_pre[*b_] * U + *u_ * n + *v_;
    };
    int g0 = 0, g1 = 0, b = 0, u = 0, v_first = 0;
    if (c < sh.n) {
        g0 = sh.begin(c), g1 = sh.begin(c + 1);
        if constexpr (SHARED) {
            int b1, u1, v1;
            g1 = c + 1 < sh.n ? tile_at(g1, &b1, &u1, &v1) : carry * U;
            g0 = tile_at(g0, &b, &u, &v_first);
        }
    }
    if (g0 >= g1) {   // nothing in flight, no barrier left
        if constexpr (SHARED) asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }

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
    if constexpr (!SHARED) {
        // the last sequence that starts at or before g0: not an empty one
        for (int hi = p.B - 1; b < hi;) {
            const int mid = (b + hi + 1) >> 1;
            if (s_pre[mid] * U <= g0) b = mid;
            else hi = mid - 1;
        }
        const int n_first = s_pre[b + 1] - s_pre[b];
        u = static_cast<int>(static_cast<unsigned>(g0 - s_pre[b] * U) / static_cast<unsigned>(n_first));
        v_first = g0 - s_pre[b] * U - u * n_first;
    }
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
        const Seq x = seq_of(p, s_len[nb], queries(nb), start_of(nb));
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
        nv += STEP * ST;
        fetch();
    };
    if (lane < ST) {
        const int first = g0 + (ALONE ? 0 : warp) + STEP * lane;
        if (first < g1) {
            left = (g1 - first + STEP * ST - 1) / (STEP * ST);
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
    int mine = g0 + (ALONE ? 0 : warp);   // this warp's next tile
    int slot = 0;               // of that tile
    uint32_t phase = 0;         // and its turn of the ring
    while (unit0 < g1) {
        const Seq s = seq_of(p, s_len[b], queries(b), start_of(b));
        const bool joins = start_of(b) > 0;   // the rows join a shared prefix's
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

        for (; mine < end; mine += STEP) {
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
        if constexpr (ALONE) {
            // this warp alone: lane (g, t) holds dimensions VB g .. + VB - 1 of rows 2t, 2t + 1 of each 8
#pragma unroll
            for (int nt = 0; nt < NR; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = l[nt][e];
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
                    const int i = nt * 8 + 2 * t + e;
                    if (row0 + i >= p.rows) continue;
                    const bool empty = x == 0.0f;   // sees nothing: 0, beside a NaN that others see, too
                    const float L = empty ? -INFINITY : m[nt][e] + lg2_approx(x);   // a NaN stays one
                    const float f = empty ? 0.0f : ex2_ftz(R[nt][e] - m[nt][e]) / x;
                    const int64_t row = head_row + row0 + i, at = static_cast<int64_t>(part) * (8 * NR) + i;
                    if (g == 0) {
                        if (!whole) p.part_lse[at] = L;
                        else if (joins) p.own_lse[row] = L;
                        else p.lse[row] = L * 0.6931471805599453f;
                    }
                    float y[VB];
#pragma unroll
                    for (int k = 0; k < VB / 2; ++k) {
                        y[2 * k] = empty ? 0.0f : o[nt][k][e] * f;
                        y[2 * k + 1] = empty ? 0.0f : o[nt][k][e + 2] * f;
                    }
                    if (whole && !joins) {
                        uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + row * D + VB * g);
#pragma unroll
                        for (int k = 0; k < VB / 8; ++k)
                            dst[k] = make_uint4(pack2<BF16>(y[8 * k], y[8 * k + 1]), pack2<BF16>(y[8 * k + 2], y[8 * k + 3]),
                                                pack2<BF16>(y[8 * k + 4], y[8 * k + 5]),
                                                pack2<BF16>(y[8 * k + 6], y[8 * k + 7]));
                    } else {
                        float4* dst = reinterpret_cast<float4*>((whole ? p.own_o + row * D : p.part_o + at * D) + VB * g);
#pragma unroll
                        for (int k = 0; k < VB / 4; ++k)
                            dst[k] = make_float4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
                    }
                }
        } else {
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
                if (SHARED && whole && joins) p.own_lse[head_row + row0 + i] = L;
                else if (whole) p.lse[head_row + row0 + i] = L * 0.6931471805599453f;
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
                if (SHARED && whole && joins)
                    *reinterpret_cast<float2*>(p.own_o + (head_row + row0 + r) * D + dim) = make_float2(ox, oy);
                else if (whole)
                    *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) +
                                                 (head_row + row0 + r) * D + dim) = pack2<BF16>(ox, oy);
                else
                    *reinterpret_cast<float2*>(
                        p.part_o + (static_cast<int64_t>(part) * (8 * NR) + r) * D + dim) =
                        make_float2(ox, oy);
            }
        }
        }
    }
    // After a wait that gave up, copies may still be on their way into this
    // CTA's shared memory: wait for the last one of each slot (bounded).
    if (*abort_flag && lane < ST && issued > 0)
        mbar_wait_bounded(&full[lane], (issued - 1) & 1, p.status);
    if constexpr (SHARED) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ------------------------------------------------------------------ host

// The [n_pages * Hkv][page][D] bytes of a pool, boxes of at most a tile's tokens.
int make_page_map(CUtensorMap* map, const void* base, int D, int page, int64_t pages, int nr) {
    const int tile = D == 64 && nr < 4 ? tile_tokens<64, 1>() : tile_tokens<128, 1>();
    return make_byte_map_public(map, base, D, page, pages, page < tile ? page : tile);
}

template <int D, bool BF16, int NR, bool ONE, bool SHARED>
cudaError_t launch_attn(const CUtensorMap& tmK, const CUtensorMap& tmV, const AttnParams& p,
                        cudaStream_t stream) {
    auto kern = kv8_attn_kernel<D, BF16, NR, ONE, SHARED>;
    static SmemLimit limit;
    const cudaError_t e = limit.raise(kern, AttnCfg<D, NR>::smem_bytes(kMaxBatch, SHARED));
    if (e != cudaSuccess) return e;
    return launch_dependent(kern, p.ctas, kAttnThreads, AttnCfg<D, NR>::smem_bytes(p.B, SHARED), stream, tmK, tmV, p);
}

// The attention alone; its merge is the caller's.
template <bool SHARED>
cudaError_t launch_attention(const AttnParams& p, const void* k_pages, const void* v_pages, int D, int page,
                             bool bf16, cudaStream_t st) {
    CUtensorMap tmK, tmV;
    const int64_t pages = static_cast<int64_t>(p.n_pages) * p.Hkv;
    const int nr = row_tiles(p.rows);
    if (make_page_map(&tmK, k_pages, D, page, pages, nr) != ATTN_OK ||
        make_page_map(&tmV, v_pages, D, page, pages, nr) != ATTN_OK)
        return cudaErrorInvalidValue;
    cudaError_t e = cudaErrorInvalidValue;
#define TME_ATTN(d, b, n) \
    if (D == d && bf16 == b && nr == n) {                                                          \
        static_assert(tile_tokens<d, n>() == (d == 64 && n < 4 ? 64 : 32), "p.tile_shift");         \
        e = page >= tile_tokens<d, n>() ? launch_attn<d, b, n, true, SHARED>(tmK, tmV, p, st)       \
                                        : launch_attn<d, b, n, false, SHARED>(tmK, tmV, p, st);     \
    }
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
    return e;
}

}  // namespace
}  // namespace tme
