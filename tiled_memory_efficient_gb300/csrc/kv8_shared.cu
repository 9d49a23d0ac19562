// kv8_shared.cu -- attention over the paged 8-bit cache for sequences that share a
// prefix (include/kvcache.h): which sequences those are, the prefix's attention for
// all of them at once, and the merge with what each sees of its own.
//
// softmax(q K^T) V over positions [0, len) is the sum over [0, s) and [s, len), each
// with its own maximum and sum, weighted by exp(LSE - LSE of both).  The part [s, len) is
// kv8_attn's; over [0, s) the rows of a group's sequences (G Nq each of a KV head) stand together as
// one matrix, so its keys and values are read once for all of them and the two products
// become matrix products with 128 rows or more: work for tcgen05, bound by it and by the
// exponentials where the single sequence's attention is bound by memory.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/kvcache.h"
#include "attn_internal.h"
#include "kv8.cuh"
#include "ptx.cuh"

namespace tme {
namespace {

// ------------------------------------------------------------------ the prefix's attention

constexpr int kPreRows = 128;       // rows of a Q tile, keys of a K/V tile
constexpr int kPreMinShare = 2;     // tiles per CTA, at least
constexpr float kPreThreshold = 8.0f;   // powers of two a score may outgrow the reference by

struct PreParams {
    AttnParams a;
    const uint8_t* k_pages;
    const uint8_t* v_pages;
    float* row_o;      // [B, Hq, Nq][D]: units that lie in one CTA
    float* row_lse;    // [B, Hq, Nq], log2 domain
    float* part_o;     // [2 * ctas][rows of a block][D]: the others
    float* part_lse;
};

// What the producer leaves beside a raw tile: keys are kf times their fp16 values, the accumulator's
// values 2^ev; bad: pages (bits) that hold nothing readable; scaled: whether some page's keys (1) or
// values (2) are moved by a power of two on their way to fp16, and by which (two fp16 each).
struct TileInfo {
    float kf;
    int ev, bad, scaled;
    uint32_t factor[2][8];
};
constexpr int kInfos = 8;   // of them: the softmax may be four tiles behind the producer

// QT: Q tiles of a CTA (128 rows each).
template <int D, int QT>
struct PreCfg {
    static constexpr int kTile16 = kPreRows * D * 2;    // 128 x D, fp16
    static constexpr int kRaw = kPreRows * D;           // 128 x D, e4m3
    // K and V take turns; shared memory is full at D = 128 with two Q tiles
    static constexpr int kRawSlots = D == 64 ? 8 : QT == 1 ? 4 : 2;
    static constexpr int kKOff = QT * kTile16;
    static constexpr int kVOff = kKOff + 2 * kTile16;
    static constexpr int kRawOff = kVOff + 2 * kTile16;
    static constexpr int kInfoOff = kRawOff + kRawSlots * kRaw;
    static constexpr int kBarOff = kInfoOff + kInfos * static_cast<int>(sizeof(TileInfo));
    static constexpr int kBars = 2 * kRawSlots + 8 + kInfos + 2 + 2 + QT * 2 + 1;
    static constexpr int kMiscOff = kBarOff + kBars * 8;
    static constexpr int kSmem = kMiscOff + 16 + 1024;
    static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
    static constexpr int kSoftmaxWarps = 4 * QT, kConvWarp = kSoftmaxWarps, kMmaWarp = kConvWarp + 4,
                         kProducerWarp = kMmaWarp + 1, kThreads = (kProducerWarp + 1) * 32;
    static constexpr int kRowBlock = QT * kPreRows;
};

// Tiles, units and rows of a group.  The shares are cut from its units' steps: to begin a unit (its queries
// on their way, the rows of the one before written) takes about as long as kUnitSteps tiles, so that a CTA
// which ends one unit and begins another has as many tiles less: four groups of 12 sequences with three
// queries under 5008 positions (4 KV heads, D = 128) 36.5 us instead of 39.9 with equal tiles, 64 samples
// under 32K positions (2 KV heads, D = 64) 32.9 instead of 33.8; 2 to 6 steps measure alike.
constexpr int kUnitSteps = 3;
struct Group {
    int blocks, n_rb, units, rows;
    __device__ __forceinline__ int unit_steps() const { return blocks > 0 ? blocks + kUnitSteps : 0; }
    __device__ __forceinline__ int steps() const { return units * unit_steps(); }
    // tiles before step s of the group
    __device__ __forceinline__ int tiles_before(int s) const {
        const int u = s / unit_steps();
        return u * blocks + max(s - u * unit_steps() - kUnitSteps, 0);
    }
};
__device__ __forceinline__ Group group_of(const AttnParams& p, const Plan& plan, int g, int row_block) {
    Group x;
    x.blocks = min(plan.blocks(g), (p.max_pages << p.page_shift) / kShareBlock);
    x.rows = plan.count(g) * p.rows;   // at most 2^30 (checked on the host)
    x.n_rb = (x.rows + row_block - 1) / row_block;
    x.units = p.Hkv * x.n_rb;
    return x;
}
// Steps of all groups, and (`before`) of those before one; each warp for itself.  `mine`: group `lane`, asked for
// with the header.
__device__ __forceinline__ int all_steps(const AttnParams& p, const Plan& plan, int groups, int row_block,
                                         const Group& mine, int before = 0, int* lead = nullptr) {
    const int lane = threadIdx.x & 31;
    int all = 0, first = 0;
    for (int g = lane; g < groups; g += 32) {
        const int n = (g == lane ? mine : group_of(p, plan, g, row_block)).steps();
        all += n;
        if (g < before) first += n;
    }
    if (lead) *lead = __reduce_add_sync(0xffffffffu, first);
    return __reduce_add_sync(0xffffffffu, all);
}

// A CTA's share of the tiles, part by part (a part: consecutive tiles of one unit).  Every role
// walks it for itself.
struct Walk {
    Group x;
    int g, u, v;      // group, unit within it, first tile of the part within the unit
    int left;         // tiles of the share from the part on
    __device__ __forceinline__ int tiles() const { return min(x.blocks - v, left); }
    __device__ __forceinline__ void next(const AttnParams& p, const Plan& plan, int groups, int row_block) {
        left -= tiles();
        v = 0;
        if (left > 0 && ++u == x.units) {
            u = 0;
            do ++g, x = group_of(p, plan, g, row_block);
            while (x.steps() == 0 && g + 1 < groups);
            if (x.steps() == 0) left = 0;   // (a plan that changed meanwhile: no endless walk)
        }
    }
    __device__ __forceinline__ int head() const { return u / x.n_rb; }
    __device__ __forceinline__ int row0(int row_block) const { return (u - head() * x.n_rb) * row_block; }
};
// The share of a CTA that starts at step g0 and ends at g1 (g0 < g1): its first tile, and how many.
__device__ __forceinline__ Walk walk_from(const AttnParams& p, const Plan& plan, int groups, int row_block,
                                          const Group& mine, int g0, int g1) {
    const int lane = threadIdx.x & 31;
    Walk w{};
    int carry = 0, tiles = 0;
    bool found = false;
    for (int base = 0; base < groups; base += 32) {
        const int g = base + lane;
        Group x{};
        if (g < groups) x = base == 0 ? mine : group_of(p, plan, g, row_block);
        const int n = x.steps();
        int sum = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, sum, d);
            if (lane >= d) sum += y;
        }
        const int begin = carry + sum - n;   // of the lane's group
        const int lo = max(g0, begin), hi = min(g1, carry + sum);
        if (lo < hi) tiles += x.tiles_before(hi - begin) - x.tiles_before(lo - begin);
        const unsigned past = __ballot_sync(0xffffffffu, carry + sum > g0);
        if (past && !found) {
            const int at = __ffs(past) - 1;
            const int off = g0 - __shfl_sync(0xffffffffu, begin, at);
            w.g = base + at;
            w.x.blocks = __shfl_sync(0xffffffffu, x.blocks, at);
            w.x.n_rb = __shfl_sync(0xffffffffu, x.n_rb, at);
            w.x.units = __shfl_sync(0xffffffffu, x.units, at);
            w.x.rows = __shfl_sync(0xffffffffu, x.rows, at);
            w.u = off / w.x.unit_steps();
            w.v = max(off - w.u * w.x.unit_steps() - kUnitSteps, 0);
            found = true;
        }
        carry += __shfl_sync(0xffffffffu, sum, 31);
        if (carry >= g1) break;
    }
    w.left = __reduce_add_sync(0xffffffffu, tiles);
    return w;
}

// 16 e4m3 values as fp16, times 2^d (d <= 0, as two fp16 in `factor`; 1: not multiplied).
__device__ __forceinline__ void convert16(const uint4& x, uint32_t factor, bool scaled, uint4* lo, uint4* hi) {
    const uint32_t in[4] = {x.x, x.y, x.z, x.w};
    uint32_t r[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r[2 * i] = e4m3x2_to_f16x2(in[i]);
        r[2 * i + 1] = e4m3x2_hi_to_f16x2(in[i]);
    }
    if (scaled) {
#pragma unroll
        for (int i = 0; i < 8; ++i) asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(r[i]) : "r"(factor));
    }
    *lo = make_uint4(r[0], r[1], r[2], r[3]);
    *hi = make_uint4(r[4], r[5], r[6], r[7]);
}
// 2^d as two fp16 values; 0 below the smallest one (the values it would scale are under 2^-33
// of the largest that the tile can hold).
__device__ __forceinline__ uint32_t pow2_f16x2(int d) {
    const uint32_t h = d >= -14 ? static_cast<uint32_t>(d + 15) << 10 : d >= -24 ? 1u << (d + 24) : 0u;
    return h | (h << 16);
}

// (no "memory": what reads it is behind a fence, and other loads may pass)
__device__ __forceinline__ void sts128(uint32_t a, const uint4& x) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w));
}
__device__ __forceinline__ uint4 lds128v(uint32_t a) {
    uint4 r;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
    return r;
}

// One CTA per SM, each an equal share of all groups' (KV head, row block, tile of 128 keys): the
// roles are those of the dense forward, but the keys and values arrive as e4m3 pages in a
// ring of raw tiles (one bulk copy a page) and four warps rewrite them as fp16 operands (exact; a page
// whose scale is below the tile's largest is moved by that power of two, exact down to 2^-15 of
// it), swizzled as TMA would have written them.  The value scale that the accumulator stands at
// only grows within a unit, by whole tiles, and joins the softmax's rescale.  A part of a unit ends in fp32
// rows with their LSE, for kv8_shared_merge_kernel.
//   warps 0 .. 4 QT - 1   softmax, a thread per row: one pass over S in TMEM, P over S as fp16
//   then 4 warps          converters
//   then 1 warp           tcgen05.mma issue: QT = 2 PV_0, S_0', PV_1, S_1', so that one tile's softmax
//                         runs beside the other's products; QT = 1 two S buffers, S' before PV
//   then 1 warp           producer: page ids, scales, bulk copies
// Bound by a tile's chain, scores, softmax, product, of which two are in flight: at D = 128 3750 cycles a step of
// 128 keys and 256 rows, where the products take 2048 (D = 64: 3300 and 1024), and by both ends of a part: 6 to 9
// us until the first scores, 3 to 4 for its rows.  128 sequences, 32:8 heads, D = 128 under 16K positions 42 us behind
// the call before (46 by itself, the tensor pipe 30% and issue slots 42% busy); 64 samples, 14:2 heads, D = 64 under
// 32K 20 us (24, 15% and 35%).  Two Q
// tiles a CTA (QT) take those 51.5 us instead of 62.5 with one, and 25 instead of 29, in an earlier state of both.
template <int D, bool BF16, int QT>
__global__ void __launch_bounds__(PreCfg<D, QT>::kThreads, 1)
    kv8_prefix_kernel(const __grid_constant__ PreParams p) {
    using C = PreCfg<D, QT>;
    constexpr int RS = C::kRawSlots, NI = RS / 2, RB = C::kRowBlock;
    static_assert(kInfos >= NI + 3, "a tile's info outlives its softmax");
    constexpr int kOCol = 256;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    TileInfo* infos = reinterpret_cast<TileInfo*>(smem + C::kInfoOff);          // [kInfos]
    uint64_t* raw_full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);       // [RS]
    uint64_t* raw_empty = raw_full + RS;     // [RS]
    uint64_t* k_full = raw_empty + RS;       // [2] the fp16 tile is written
    uint64_t* k_empty = k_full + 2;          // [2]
    uint64_t* v_full = k_empty + 2;          // [2]
    uint64_t* v_empty = v_full + 2;          // [2]
    uint64_t* info_full = v_empty + 2;       // [kInfos]
    uint64_t* s_full = info_full + kInfos;        // [2] QT = 2: of tile t; QT = 1: of S buffer x & 1
    uint64_t* pv_done = s_full + 2;          // [2] PV of tile t done
    uint64_t* p_full = pv_done + 2;          // [QT]
    uint64_t* q_full = p_full + QT;          // [QT]
    uint64_t* mma_done = q_full + QT;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kMiscOff);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const AttnParams& a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // As the attention behind it: reads from here on what earlier kernels wrote; that one may
    // set up and start (it reads nothing of this one's).
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const Plan plan(a.plan, a.B, a.least_members);
    const Group mine = group_of(a, plan, min(lane, a.B - 1), RB);   // (asked for beside the header)
    const bool granted = step_granted(a);
    if (!plan.ok()) {   // the sequences are then each for itself
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.status, kStatusPage);
        return;
    }
    const int groups = granted && plan.ok(a.least_runs) ? plan.groups() : 0;
    const int T = all_steps(a, plan, groups, RB, mine);
    const Shares sh(T, a.ctas, kPreMinShare);
    const int cta = static_cast<int>(blockIdx.x);
    if (cta >= sh.n) return;   // nothing to wait for
    Walk w = walk_from(a, plan, groups, RB, mine, sh.begin(cta), sh.begin(cta + 1));
    const int total = w.left;
    if (total <= 0) return;    // (the steps before a unit's first tile)
    auto next = [&](Walk& x) { x.next(a, plan, groups, RB); };
    auto active = [&](const Walk& x, int t) { return x.row0(RB) + t * kPreRows < x.x.rows; };

    if (threadIdx.x == C::kConvWarp * 32) {
        for (int i = 0; i < RS; ++i) {
            mbar_init(&raw_full[i], 1);
            mbar_init(&raw_empty[i], 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&k_full[i], 4);
            mbar_init(&k_empty[i], 1);
            mbar_init(&v_full[i], 4);
            mbar_init(&v_empty[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&pv_done[i], 1);
        }
        for (int i = 0; i < kInfos; ++i) mbar_init(&info_full[i], 1);
        for (int t = 0; t < QT; ++t) {
            mbar_init(&p_full[t], kPreRows);
            mbar_init(&q_full[t], kPreRows);
        }
        mbar_init(mma_done, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == C::kMmaWarp) tmem_alloc(tmem_slot, 512);
    // Each role looks up what it can before the barriers and TMEM are there, and comes here once.
    uint32_t tmem = 0;
    auto ready = [&]() {
        tc_fence_before();
        asm volatile("bar.sync 0;" ::: "memory");
        tc_fence_after();
        tmem = *tmem_slot;
    };

    // Every wait is bounded: one that gives up sets the abort flag, at which all others return
    // at once, so each role's loops run to their end (or leave) without blocking.
    if (warp < C::kSoftmaxWarps) {
        // ------------------------------------------------------------ softmax
        ready();
        const int t = warp >> 2, quad = warp & 3;
        const int rl = quad * 32 + lane;
        const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
        const uint32_t tO = tmem + lane_base + kOCol + t * D;
        const uint32_t sQ = smem_u32(smem + t * C::kTile16);
        // this thread's row of the part: whether it exists, its position (-1: sees nothing), its
        // place among all rows, its scores' factor
        bool exists = false;
        int pos = -1;
        int row_id = 0;
        float f_row = 0.0f;
        // Q of a part's tile t: each thread its own row, bf16 brought into fp16's range by a power of
        // two first (as in kv8_attn).  S of the part before has been computed.
        auto load_q = [&](const Walk& x) {
            const int r = x.row0(RB) + t * kPreRows + rl;
            exists = r < x.x.rows;
            pos = -1;
            const uint4* src = nullptr;
            if (exists) {
                const int m = r / a.rows, rr = r - m * a.rows;
                const int b = plan.member(plan.first(x.g) + m);
                const int len = a.lens[b], nq = queries_of(a, granted, b, len);
                const int i = rr % a.Nq;
                if (i < nq) pos = min(max(len, 0), a.max_pages << a.page_shift) - nq + i;
                row_id = (b * a.Hkv + x.head()) * a.rows + rr;
                src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + static_cast<int64_t>(row_id) * D);
            }
            uint4 q[D / 8];   // the whole row at once: one trip to memory
#pragma unroll
            for (int k = 0; k < D / 8; ++k) q[k] = exists ? src[k] : make_uint4(0u, 0u, 0u, 0u);
            int shift = 0;
            if constexpr (BF16) {
                uint32_t ex = 0u;   // largest finite exponent field
#pragma unroll
                for (int k = 0; k < D / 8; ++k) {
                    const uint32_t y[4] = {q[k].x, q[k].y, q[k].z, q[k].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t lo = (y[e] >> 7) & 0xffu, hi = (y[e] >> 23) & 0xffu;
                        ex = max(ex, max(lo < 255u ? lo : 0u, hi < 255u ? hi : 0u));
                    }
                }
                shift = ex == 0u ? 0 : min(14 + 127 - static_cast<int>(ex), 126);
            }
            const float up = exp2i(shift);
            f_row = a.scale_log2 * exp2i(-shift);
#pragma unroll
            for (int k = 0; k < D / 8; ++k) {
                if constexpr (BF16) {
                    uint32_t y[4] = {q[k].x, q[k].y, q[k].z, q[k].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 v = unpack16<true>(y[e]);
                        y[e] = pack2<false>(v.x * up, v.y * up);
                    }
                    q[k] = make_uint4(y[0], y[1], y[2], y[3]);
                }
                sts128(sQ + (k >> 3) * (kPreRows * 128) + rl * 128 + (((k & 7) ^ (rl & 7)) << 4), q[k]);
            }
            fence_proxy_async_smem();
            mbar_arrive(&q_full[t]);
        };
        int x = 0;          // tile of the share
        uint32_t ns = 0;    // tiles of this Q tile so far
        bool ok = true;
        // the part whose rows are still to be written (its Q tile's next rows are loaded first)
        bool pending = false, mine = false, live = false, whole = false;
        int my_row = 0, part = 0, ev = 0;
        float m = -INFINITY, l = 0.0f;
#pragma unroll 1
        for (;;) {
            const bool more = w.left > 0, act = more && active(w, t);
            if (act) load_q(w);
            if (pending) {
                ok = warp_wait(&pv_done[t], (ns - 1) & 1u, abort_flag, a.status);
                if (!ok) break;
                tc_fence_after();
                const bool empty = !live || l == 0.0f;   // (a NaN is not)
                const float inv = empty ? 0.0f : 1.0f / l, scale = exp2i(ev);
                const int at = whole ? my_row : part * RB + t * kPreRows + rl;
                float* dst = (whole ? p.row_o : p.part_o) + static_cast<int64_t>(at) * D;
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    tmem_ld32(tO + c * 32, o);
                    tmem_wait_ld();
                    reg_fence(o);
                    if (mine) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t y[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                y[k] = empty ? 0u : __float_as_uint(__uint_as_float(o[8 * i + k]) * inv * scale);
                            st_global_v8(dst + c * 32 + 8 * i, y);
                        }
                    }
                }
                if (mine) (whole ? p.row_lse : p.part_lse)[at] = empty ? -INFINITY : m + lg2_approx(l);
                tc_fence_before();
                pending = false;
            }
            if (!more) break;
            const int n = w.tiles();
            if (!act) {
                x += n;
                next(w);
                continue;
            }
            mine = exists;
            my_row = row_id;
            const int my_pos = pos;
            const float my_f = f_row;
            live = __any_sync(0xffffffffu, my_pos >= 0);
            const int min_pos = __reduce_min_sync(0xffffffffu, mine ? my_pos : 0x7fffffff);
            m = -INFINITY, l = 0.0f;
            ev = 0;
#pragma unroll 1
            for (int j = 0; j < n && ok; ++j, ++x, ++ns) {
                const uint32_t buf = QT == 1 ? (ns & 1u) : static_cast<uint32_t>(t);
                const uint32_t tS = tmem + lane_base + buf * 128;
                ok = warp_wait(&info_full[x % kInfos], (x / kInfos) & 1, abort_flag, a.status);
                ok = ok && warp_wait(&s_full[buf], QT == 1 ? (ns >> 1) & 1u : ns & 1u, abort_flag, a.status);
                if (!ok) break;
                tc_fence_after();
                const volatile TileInfo* in = infos + x % kInfos;
                // (not 0, where both factors are tiny: what is hidden below is -inf times it; the scores,
                // at most 2^32, are nothing beside 1 there)
                const float f = fmaxf(my_f * in->kf, 0x1p-126f);
                const int ev_now = in->ev, bad = in->bad;
                // QT = 1: S of this tile went out ahead of the last PV.  A warp that arrived for this tile
                // while another has yet to for the last one would complete that phase in its place; and O is
                // not to be touched before that PV is done.
                auto last_pv = [&]() {
                    if (QT == 1 && j > 0) ok = warp_wait(&pv_done[t], (ns - 1) & 1u, abort_flag, a.status);
                    return ok;
                };
                if (!live) {   // a warp with no row that sees anything keeps the counts
                    if (!last_pv()) break;
                    mbar_arrive(&p_full[t]);
                    continue;
                }
                const int key0 = (w.v + j) * kPreRows;
                if (bad != 0 || key0 + kPreRows - 1 > min_pos) {
                    // what the rows do not see, in place in TMEM, 32 keys at a time (tiles that hold the
                    // queries' own positions, and bad pages, are rare: not in the other tiles' code)
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        uint32_t s[32];
                        tmem_ld32(tS + c * 32, s);
                        tmem_wait_ld();
                        reg_fence(s);
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const int k = c * 32 + i;
                            if (key0 + k > my_pos || ((bad >> (k >> a.page_shift)) & 1)) s[i] = __float_as_uint(-INFINITY);
                        }
                        tmem_st32(tS + c * 32, s);
                    }
                    tmem_wait_st();
                }
                // One pass over S, 32 keys at a time, in a loop: the four roles run different code on each SM
                // sub-partition, and what is unrolled waits for its instructions.  The reference m moves,
                // by whole powers of two, where a score outgrows it by more than 2^kPreThreshold:
                // the terms of the keys before are then moved by as much, exactly.
                float al = 1.0f;   // what the sum, and O, are moved by
                uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    uint32_t now[32], pk[16];
                    tmem_ld32(tS + c * 32, now);
                    tmem_wait_ld();
                    reg_fence(now);
                    float y0 = __uint_as_float(now[0]), y1 = __uint_as_float(now[1]);
                    float y2 = __uint_as_float(now[2]), y3 = __uint_as_float(now[3]);
#pragma unroll
                    for (int i = 4; i < 28; i += 8) {
                        y0 = fmax3(y0, __uint_as_float(now[i]), __uint_as_float(now[i + 1]));
                        y1 = fmax3(y1, __uint_as_float(now[i + 2]), __uint_as_float(now[i + 3]));
                        y2 = fmax3(y2, __uint_as_float(now[i + 4]), __uint_as_float(now[i + 5]));
                        y3 = fmax3(y3, __uint_as_float(now[i + 6]), __uint_as_float(now[i + 7]));
                    }
                    y0 = fmax3(y0, __uint_as_float(now[28]), __uint_as_float(now[29]));
                    y1 = fmax3(y1, __uint_as_float(now[30]), __uint_as_float(now[31]));
                    const float m_new = ceilf(fmaxf(m, fmaxf(fmaxf(y0, y1), fmaxf(y2, y3)) * f));
                    const bool need = m_new > m + kPreThreshold;
                    if (__any_sync(0xffffffffu, need)) {
                        // (from -inf: every term so far is 0)
                        const int d = need ? static_cast<int>(fmaxf(m - m_new, -1000.0f)) : 0;
                        const float by = need ? ex2_ftz(m - m_new) : 1.0f;
                        al *= by;
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[i] = fmul2(acc[i], f2(by, by));
                        m = need ? m_new : m;
                        const uint32_t by16 = pow2_f16x2(d);
                        tmem_wait_st();
                        for (int e = 0; e < c; ++e) {
                            tmem_ld16(tS + e * 16, pk);
                            tmem_wait_ld();
                            reg_fence(pk);
#pragma unroll
                            for (int i = 0; i < 16; ++i) asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(pk[i]) : "r"(by16));
                            tmem_st16(tS + e * 16, pk);
                        }
                    }
                    const float m_sub = m == -INFINITY ? 0.0f : m;
                    const uint64_t f2s = f2(f, f), nm2 = f2(-m_sub, -m_sub);
#pragma unroll
                    for (int i = 0; i < 32; i += 2)
                        pk[i >> 1] = softmax_pair<false>(now[i], now[i + 1], f2s, nm2, acc[(i >> 1) & 3]);
                    // (columns 16 c .. + 15: of scores that are read)
                    tmem_st16(tS + c * 16, pk);
                }
                const uint64_t a2 = fadd2(fadd2(acc[0], acc[1]), fadd2(acc[2], acc[3]));
                l = l * al + (f2lo(a2) + f2hi(a2));
                const int up = j > 0 ? ev_now - ev : 0;   // the value scale grew by 2^up
                ev = ev_now;
                if (!last_pv()) break;
                if (j > 0 && __any_sync(0xffffffffu, al != 1.0f || up > 0)) {
                    tc_fence_after();
                    const float o_al = al * exp2i(-min(up, 126));
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32];
                        tmem_ld32(tO + c * 32, o);
                        tmem_wait_ld();
                        reg_fence(o);
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * o_al);
                        tmem_st32(tO + c * 32, o);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&p_full[t]);
            }
            if (!ok) break;
            // where this part's rows go
            whole = w.v == 0 && n == w.x.blocks;
            part = 2 * cta + (w.left == total ? 0 : 1);
            pending = true;
            next(w);
        }
    } else if (warp < C::kMmaWarp) {
        // ------------------------------------------------------------ converters
        ready();
        const int ct = threadIdx.x - C::kConvWarp * 32;
        constexpr int KB = D / 64;                // column blocks of an fp16 tile
        // 8 lanes hold chunks 0 .. 3 of a column block in two neighbouring rows (D = 128: of block a in the even
        // row and of the other one in the odd row, a in turn), so that both their loads and their stores,
        // units 2 j and 2 j + 1 of the row's swizzled 128 bytes, meet every bank once.
        const int cj = ct & 3, cs = (ct >> 2) & 1, cr = 2 * (ct >> 3) + cs;   // row modulo 32
        const uint32_t lo_at = cr * 128 + (((2 * cj) ^ (cr & 7)) << 4);
        const uint32_t hi_at = cr * 128 + (((2 * cj + 1) ^ (cr & 7)) << 4);
        bool ok = true;
        for (int x = 0; x < total && ok; ++x) {
            const TileInfo* in = infos + x % kInfos;
#pragma unroll 1
            for (int which = 0; which < 2; ++which) {
                const int slot = (2 * x) % RS + which;
                ok = warp_wait(&raw_full[slot], static_cast<uint32_t>(x / NI) & 1u, abort_flag, a.status);
                uint64_t* empty = which == 0 ? &k_empty[x & 1] : &v_empty[x & 1];
                if (ok && x >= 2) ok = warp_wait(empty, ((x - 2) >> 1) & 1, abort_flag, a.status);
                if (!ok) break;
                const uint32_t src = smem_u32(smem + C::kRawOff + slot * C::kRaw) + cr * D + cj * 16;
                const uint32_t dst = smem_u32(smem + (which == 0 ? C::kKOff : C::kVOff) + (x & 1) * C::kTile16);
                const int bad = in->bad;
                const bool scaled = (in->scaled >> which) & 1;
                // 32 rows a turn, asked for a turn ahead
                uint4 raw[KB], ahead[KB];
#pragma unroll
                for (int e = 0; e < KB; ++e) raw[e] = lds128v(src + (KB == 1 ? 0 : cs ^ e) * 64);
#pragma unroll 1
                for (int i = 0; i < kPreRows; i += 32) {
                    if (i + 32 < kPreRows) {
#pragma unroll
                        for (int e = 0; e < KB; ++e)
                            ahead[e] = lds128v(src + (i + 32) * D + (KB == 1 ? 0 : cs ^ e) * 64);
                    }
                    const int pg = (i + cr) >> a.page_shift;
                    uint32_t factor = 0u;
                    if (scaled) factor = in->factor[which][pg];
                    const bool drop = (bad >> pg) & 1;
#pragma unroll
                    for (int e = 0; e < KB; ++e) {
                        uint4 lo, hi;
                        convert16(raw[e], factor, scaled, &lo, &hi);
                        if (drop) lo = hi = make_uint4(0u, 0u, 0u, 0u);
                        const uint32_t to = dst + (KB == 1 ? 0 : cs ^ e) * (kPreRows * 128) + i * 128;
                        sts128(to + lo_at, lo);
                        sts128(to + hi_at, hi);
                        raw[e] = ahead[e];
                    }
                }
                // the tensor core reads these bytes after the arrival below
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&raw_empty[slot]);
                    mbar_arrive(which == 0 ? &k_full[x & 1] : &v_full[x & 1]);
                }
            }
        }
    } else if (warp == C::kMmaWarp) {
        // ------------------------------------------------------------ MMA issue
        ready();
        constexpr uint32_t idesc_s = idesc_f16(kPreRows, kPreRows, false, false);
        constexpr uint32_t idesc_o = idesc_f16(kPreRows, D, false, true);
        constexpr uint64_t kTileStep = C::kTile16 >> 4, kBlk = (kPreRows * 128) >> 4;
        const uint64_t dq0 = smem_desc_sw128(smem_u32(smem), 16, 1024);
        const uint64_t dk0 = smem_desc_sw128(smem_u32(smem + C::kKOff), 16, 1024);
        const uint64_t dv0 = smem_desc_sw128(smem_u32(smem + C::kVOff), kPreRows * 128, 1024);
        uint32_t ns[2] = {0u, 0u}, np[2] = {0u, 0u}, nq[2] = {0u, 0u};
        auto issue_s = [&](int t, int x, bool last) {
            const int st = x & 1;
            warp_wait(&k_full[st], (x >> 1) & 1, abort_flag, a.status);
            tc_fence_after();
            const uint32_t buf = QT == 1 ? (ns[t] & 1u) : static_cast<uint32_t>(t);
#pragma unroll
            for (int kb = 0; kb < D / 64; ++kb)
                mma_ss_k64(tmem + buf * 128, dq0 + t * kTileStep + kb * kBlk, dk0 + st * kTileStep + kb * kBlk,
                           idesc_s, kb > 0 ? 1u : 0u);
            mma_commit_elect(&s_full[buf]);
            if (last) mma_commit_elect(&k_empty[st]);
            ++ns[t];
        };
        auto issue_pv = [&](int t, int x, bool first, bool last) {
            const int st = x & 1;
            warp_wait(&v_full[st], (x >> 1) & 1, abort_flag, a.status);
            warp_wait(&p_full[t], np[t] & 1u, abort_flag, a.status);
            tc_fence_after();
            const uint32_t buf = QT == 1 ? (np[t] & 1u) : static_cast<uint32_t>(t);
            mma_ts_k128(tmem + kOCol + t * D, tmem + buf * 128, dv0 + st * kTileStep, idesc_o, first ? 0u : 1u);
            mma_commit_elect(&pv_done[t]);
            if (last) mma_commit_elect(&v_empty[st]);
            ++np[t];
        };
        int x = 0;
        while (w.left > 0 && __all_sync(0xffffffffu, *abort_flag == 0)) {
            const int n = w.tiles();
            const bool two = QT == 2 && active(w, 1);   // (tile 0 always has rows)
            warp_wait(&q_full[0], nq[0]++ & 1u, abort_flag, a.status);
            issue_s(0, x, !two);
            if (two) {
                warp_wait(&q_full[QT - 1], nq[1]++ & 1u, abort_flag, a.status);
                issue_s(QT - 1, x, true);
            }
            for (int j = 0; j < n; ++j) {
                if (QT == 1) {
                    if (j + 1 < n) issue_s(0, x + j + 1, true);
                    issue_pv(0, x + j, j == 0, true);
                } else {
                    issue_pv(0, x + j, j == 0, !two);
                    if (j + 1 < n) issue_s(0, x + j + 1, !two);
                    if (two) {
                        issue_pv(QT - 1, x + j, j == 0, true);
                        if (j + 1 < n) issue_s(QT - 1, x + j + 1, true);
                    }
                }
            }
            x += n;
            next(w);
        }
        mma_commit_elect(mma_done);
        mbar_wait_bounded(mma_done, 0, a.status);
    } else if (warp == C::kProducerWarp) {
        // ------------------------------------------------------------ producer
        const int ppt = 1 << (7 - a.page_shift), page_bytes = D << a.page_shift;
        // a lane per page of the tile: its id two tiles ahead, its scales one
        Walk ahead = w;
        int vv = 0;   // tile of `ahead`'s part
        // the table row of the group's first sequence (looked up when the group changes: two loads that wait for
        // each other)
        auto row_of_group = [&]() { return a.table + static_cast<int64_t>(plan.member(plan.first(ahead.g))) * a.max_pages; };
        const int* row = row_of_group();
        struct Page {
            int pid, h;
            bool fresh;   // the first tile of a part
            float ks, vs;
        };
        int head = ahead.head();
        auto fetch = [&]() {
            Page r{-1, 0, vv == 0, 1.0f, 1.0f};
            if (ahead.left <= 0) return r;
            if (lane < ppt) r.pid = row[(ahead.v + vv) * ppt + lane];
            r.h = head;
            if (++vv == ahead.tiles()) {
                vv = 0;
                const int g = ahead.g;
                next(ahead);
                if (ahead.left > 0) {
                    head = ahead.head();
                    if (ahead.g != g) row = row_of_group();
                }
            }
            return r;
        };
        auto scales = [&](Page& r) {
            if (r.pid >= 0 && r.pid < a.n_pages) {
                const int64_t at = static_cast<int64_t>(r.pid) * a.Hkv + r.h;
                r.ks = a.k_scale[at];
                r.vs = a.v_scale[at];
            }
        };
        Page now = fetch(), soon = fetch();
        scales(now);
        ready();
        int issued = 0;   // raw tiles, K and V in turn
        int ev = -1000;   // value scale of the accumulator: none yet
        for (int x = 0; x < total; ++x) {
            const Page later = fetch();
            scales(soon);
            const bool good = lane < ppt && now.pid >= 0 && now.pid < a.n_pages;
            const unsigned all_good = __ballot_sync(0xffffffffu, good);
            const unsigned bad = ((1u << ppt) - 1u) & ~all_good;
            const uint32_t bytes = static_cast<uint32_t>(__popc(all_good)) * page_bytes;
            const int64_t at = (static_cast<int64_t>(now.pid) * a.Hkv + now.h) * page_bytes;
            bool ok = true;
#pragma unroll 1
            for (int which = 0; which < 2; ++which) {
                const int slot = (2 * x) % RS + which;
                if (x >= NI)
                    ok = warp_wait(&raw_empty[slot], static_cast<uint32_t>(x / NI - 1) & 1u, abort_flag, a.status);
                if (!ok) break;
                if (which == 0) {
                    // the keys' largest scale; the values', of the unit's part so far
                    const int ke = good ? scale_exp(now.ks) : -1000, ve = good ? scale_exp(now.vs) : -1000;
                    int top = __reduce_max_sync(0xffffffffu, ke);
                    if (now.fresh) ev = -1000;
                    ev = max(ev, __reduce_max_sync(0xffffffffu, ve));
                    const int ev_now = ev == -1000 ? 0 : ev;
                    if (top == -1000) top = 0;
                    TileInfo* in = infos + x % kInfos;
                    if (lane < ppt) {
                        in->factor[0][lane] = good ? pow2_f16x2(ke - top) : 0u;
                        in->factor[1][lane] = good ? pow2_f16x2(ve - ev_now) : 0u;
                    }
                    const int scaled = (__any_sync(0xffffffffu, good && ke != top) ? 1 : 0) |
                                       (__any_sync(0xffffffffu, good && ve != ev_now) ? 2 : 0);
                    if (lane == 0) {
                        in->kf = exp2i(top);
                        in->ev = ev_now;
                        in->bad = static_cast<int>(bad);
                        in->scaled = scaled;
                        if (bad) atomicOr(a.status, kStatusPage);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&info_full[x % kInfos]);
                }
                if (lane == 0) mbar_arrive_expect_tx(&raw_full[slot], bytes);   // releases the stores above, too
                __syncwarp();
                if (good)
                    bulk_load(smem + C::kRawOff + slot * C::kRaw + lane * page_bytes,
                              (which == 0 ? p.k_pages : p.v_pages) + at, page_bytes, &raw_full[slot]);
                ++issued;
            }
            if (!ok) break;
            now = soon;
            soon = later;
        }
        // No copy may still be on its way into shared memory that the CTA gives up.
        __syncwarp();
        if (lane == 0)
            for (int y = max(issued - RS, 0); y < issued; ++y)
                mbar_wait_bounded(&raw_full[y % RS], static_cast<uint32_t>(y / RS) & 1u, a.status);
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == C::kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------ merge

// A warp per row, or (WPR) a CTA's four: the row's results over the prefix and over its own positions, each
// whole or in the parts that several CTAs left.  Rows of sequences that share nothing and lie in
// one CTA are written already.  It finds its parts beside the kernels before it; behind them a row is two trips to
// memory: 4 to 6 us for 896 rows of some 40 parts, 13 for 4096 rows of 10 (25 MB), whose last CTAs find room late.
constexpr int kMergeWarps = 4;
constexpr int kMergeRowsAlone = 8;   // rows per SM up to which a CTA takes one

template <int D, bool BF16, int WPR>
__global__ void __launch_bounds__(kMergeWarps * 32)
    kv8_shared_merge_kernel(const __grid_constant__ PreParams p, int row_block, int row8) {
    const AttnParams& a = p.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    asm volatile("griddepcontrol.launch_dependents;");   // the next kernel may set up
    const int64_t row = WPR == 1 ? static_cast<int64_t>(blockIdx.x) * kMergeWarps + warp : blockIdx.x;
    const bool real = row < static_cast<int64_t>(a.B) * a.Hkv * a.rows;
    const int u = real ? static_cast<int>(row / a.rows) : 0;   // (sequence, KV head)
    const int b = u / a.Hkv, h = u - b * a.Hkv, rr = static_cast<int>(row - static_cast<int64_t>(u) * a.rows);
    const Plan plan(a.plan, a.B, a.least_members);
    const Group mine = group_of(a, plan, min(lane, a.B - 1), row_block);
    const bool granted = step_granted(a), planned = plan.ok(a.least_runs);
    // own positions: the tiles of all sequences, and of those before b
    int all = 0, before = 0, n = 0;   // (of units: their first steps, too)
    const int K = own_steps(a.rows);
    for (int i = lane; i < a.B; i += 32) {
        const int len = a.lens[i];
        const int k = seq_of(a, len, queries_of(a, granted, i, len), planned ? plan.start(i) : 0).n;
        const int steps = k > 0 ? k + K : 0;
        all += steps;
        if (i < b) before += steps;
        if (i == b) n = k;
    }
    all = __reduce_add_sync(0xffffffffu, all);
    before = __reduce_add_sync(0xffffffffu, before);
    n = __reduce_add_sync(0xffffffffu, n);
    const int U = a.Hkv * a.n_rb;
    int c0 = 0, c1 = -1, second = 0, r_own = 0;
    if (n > 0) {
        const Shares sh = own_shares(a, all * U);
        const int first = before * U + (h * a.n_rb + rr / row8) * (n + K);
        c0 = sh.owner(first + K);
        c1 = sh.owner(first + K + n - 1);
        second = first > sh.begin(c0) ? 1 : 0;
        r_own = rr % row8;
    }
    // the prefix
    const int groups = planned && granted ? plan.groups() : 0;
    const int g = real && groups > 0 ? plan.group(b) : -1;
    int d0 = 0, d1 = -1, second_pre = 0, r_pre = 0;
    int lead = 0;
    const int T = all_steps(a, plan, groups, row_block, mine, g, &lead);
    if (g >= 0 && g < groups) {
        const Group x = group_of(a, plan, g, row_block);
        const int64_t r = static_cast<int64_t>(plan.rank(b)) * a.rows + rr;
        if (x.blocks > 0 && r >= 0 && r < x.rows) {
            const Shares sh(T, a.ctas, kPreMinShare);
            const int first = lead + (h * x.n_rb + static_cast<int>(r / row_block)) * x.unit_steps();
            d0 = sh.owner(first + kUnitSteps);
            d1 = sh.owner(first + kUnitSteps + x.blocks - 1);
            second_pre = first > sh.begin(d0) ? 1 : 0;
            r_pre = static_cast<int>(r % row_block);
        }
    }
    const bool shares = planned && plan.start(b) > 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");   // in every thread: this grid ends after those
    if (!real || (!shares && n > 0 && c0 == c1)) return;
    // Two runs of results, over its own positions and over the prefix: each `n` rows of a buffer, `step`
    // apart, the first one `add` further on.  Eight of a run are in flight at once, and the code is kept
    // small: it runs once, and a warp waits longer for instructions than for their data.
    const bool own_whole = c0 == c1 && shares, pre_whole = d0 == d1;
    constexpr int LPR = D / 4, PER = 32 / LPR;   // lanes of a row, four dimensions each; results side by side
    const int sub = lane / LPR, col = lane % LPR * 4;
    float M = -INFINITY, sum = 0.0f, acc[4] = {};
#pragma unroll 1
    for (int run = 0; run < 2; ++run) {
        const bool own = run == 0, whole = own ? own_whole : pre_whole;
        const int n_run = own ? c1 - c0 + 1 : d1 - d0 + 1, step = 2 * (own ? row8 : row_block);
        const int add = whole ? 0 : own ? second * row8 : second_pre * row_block;
        const int64_t at = whole ? row : static_cast<int64_t>(own ? c0 : d0) * step + (own ? r_own : r_pre);
        const float* l = (own ? (whole ? a.own_lse : a.part_lse) : (whole ? p.row_lse : p.part_lse)) + at;
        const float* o = (own ? (whole ? a.own_o : a.part_o) : (whole ? p.row_o : p.part_o)) + at * D + col;
#pragma unroll 1
        for (int k = sub + (WPR > 1 ? warp * 8 * PER : 0); k < n_run; k += WPR * 8 * PER) {
            float L[8], top = M;
            float4 y[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int i = k + u * PER, off = i * step + (i == 0 ? add : 0);
                L[u] = -INFINITY;
                y[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (i < n_run) {
                    L[u] = l[off];
                    y[u] = *reinterpret_cast<const float4*>(o + static_cast<int64_t>(off) * D);
                }
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) top = fmaxf(top, L[u]);
            const float al = M == -INFINITY ? 0.0f : ex2_ftz(M - top);
            M = top;
            sum *= al;
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] *= al;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const float w = L[u] == -INFINITY ? 0.0f : ex2_ftz(L[u] - M);
                sum += w;
                acc[0] = fmaf(w, y[u].x, acc[0]);
                acc[1] = fmaf(w, y[u].y, acc[1]);
                acc[2] = fmaf(w, y[u].z, acc[2]);
                acc[3] = fmaf(w, y[u].w, acc[3]);
            }
        }
    }
    if constexpr (PER == 2) {   // the two halves' sums
        const float other = __shfl_xor_sync(0xffffffffu, M, 16), top = fmaxf(M, other);
        const float al = M == -INFINITY ? 0.0f : ex2_ftz(M - top);
        M = top;
        sum *= al;
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            acc[i] *= al;
            acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], 16);
        }
    }
    if constexpr (WPR > 1) {   // the warps' sums
        __shared__ float s_m[WPR], s_sum[WPR];
        __shared__ __align__(16) float s_acc[WPR][D];
        if (lane == 0) s_m[warp] = M, s_sum[warp] = sum;
        if (sub == 0) *reinterpret_cast<float4*>(&s_acc[warp][col]) = make_float4(acc[0], acc[1], acc[2], acc[3]);
        __syncthreads();
        if (warp != 0) return;
        for (int w = 1; w < WPR; ++w) M = fmaxf(M, s_m[w]);
        sum = acc[0] = acc[1] = acc[2] = acc[3] = 0.0f;
        for (int w = 0; w < WPR; ++w) {
            const float al = s_m[w] == -INFINITY ? 0.0f : ex2_ftz(s_m[w] - M);
            const float4 y = *reinterpret_cast<const float4*>(&s_acc[w][col]);
            sum = fmaf(s_sum[w], al, sum);
            acc[0] = fmaf(y.x, al, acc[0]);
            acc[1] = fmaf(y.y, al, acc[1]);
            acc[2] = fmaf(y.z, al, acc[2]);
            acc[3] = fmaf(y.w, al, acc[3]);
        }
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    if (sub == 0)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row * D + col) =
            sum == 0.0f ? make_uint2(0u, 0u)
                        : make_uint2(pack2<BF16>(acc[0] * inv, acc[1] * inv), pack2<BF16>(acc[2] * inv, acc[3] * inv));
    if (lane == 0) a.lse[row] = sum == 0.0f ? -INFINITY : (M + lg2_approx(sum)) * 0.6931471805599453f;
}

// ------------------------------------------------------------------ the plan

struct FindParams {
    const int* table;
    const int* lens;
    int* plan;
    int B, max_pages, page_shift, min_saved;
};
constexpr int kFindThreads = 128;

// Columns of a run of kShareBlock positions.
__device__ __forceinline__ int block_cols(const FindParams& p) { return kShareBlock >> p.page_shift; }
// Runs that a sequence's length and table hold in full.
__device__ __forceinline__ int full_blocks(const FindParams& p, int len) {
    return min(max(len, 0), p.max_pages << p.page_shift) / kShareBlock;
}

// How far sequence b should share, a CTA each: of the depths at which its last page is also the one of
// r - 1 others', that which leaves it the least to read, depth (r - 1) / r saved.  (Pages
// of a sequence that several hold are those of its whole beginning; the next kernel looks.)
__global__ void __launch_bounds__(kFindThreads) kvp_depth_kernel(const FindParams p) {
    asm volatile("griddepcontrol.launch_dependents;");
    __shared__ float s_gain[kFindThreads / 32];
    __shared__ int s_at[kFindThreads / 32];
    __shared__ int s_full[kMaxBatch];
    const int b = static_cast<int>(blockIdx.x), cols = block_cols(p);
    for (int k = threadIdx.x; k < p.B; k += kFindThreads) s_full[k] = full_blocks(p, p.lens[k]);
    __syncthreads();
    const int n = s_full[b];
    const int64_t stride = p.max_pages;
    float gain = 0.0f;
    int at = -1;
    for (int base = 0; base < n; base += kFindThreads) {
        const int i = base + static_cast<int>(threadIdx.x);
        int r = 0;
        if (i < n) {
            const int c = (i + 1) * cols - 1, pid = p.table[b * stride + c];
            const int* other = p.table + c;
#pragma unroll 1
            for (int k0 = 0; k0 < p.B; k0 += 16) {   // sixteen in flight
                int x[16];
#pragma unroll
                for (int u = 0; u < 16; ++u) x[u] = k0 + u < p.B ? other[(k0 + u) * stride] : -1;
#pragma unroll
                for (int u = 0; u < 16; ++u) r += k0 + u < p.B && x[u] == pid && s_full[min(k0 + u, kMaxBatch - 1)] > i;
            }
            if (pid < 0) r = 0;
        }
        const float x = r > 1 ? static_cast<float>(i + 1) * static_cast<float>(r - 1) / static_cast<float>(r) : 0.0f;
        if (x > gain) gain = x, at = i;
        if (!__syncthreads_or(r > 1)) break;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const float x = __shfl_xor_sync(0xffffffffu, gain, d);
        const int y = __shfl_xor_sync(0xffffffffu, at, d);
        if (x > gain || (x == gain && y > at)) gain = x, at = y;
    }
    if ((threadIdx.x & 31) == 0) s_gain[threadIdx.x >> 5] = gain, s_at[threadIdx.x >> 5] = at;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int k = 1; k < kFindThreads / 32; ++k)
            if (s_gain[k] > gain || (s_gain[k] == gain && s_at[k] > at)) gain = s_gain[k], at = s_at[k];
        int* scratch = p.plan + 4 + kPlanArrays * p.B;
        scratch[b] = at + 1;                                                          // depth, 0: none
        scratch[p.B + b] = at >= 0 ? p.table[b * stride + (at + 1) * cols - 1] : -1;   // its last page
    }
}

// Whose group: the first sequence of the same depth and last page, if all pages before are
// its, too (-1: none).
__global__ void __launch_bounds__(kFindThreads) kvp_leader_kernel(const FindParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    __shared__ int s_first;
    const int b = static_cast<int>(blockIdx.x);
    int* scratch = p.plan + 4 + kPlanArrays * p.B;
    const int depth = scratch[b], key = scratch[p.B + b];
    if (threadIdx.x == 0) s_first = b;
    __syncthreads();
    if (depth > 0)
        for (int k = threadIdx.x; k < b; k += kFindThreads)
            if (scratch[k] == depth && scratch[p.B + k] == key) atomicMin(&s_first, k);
    __syncthreads();
    const int first = s_first, cols = depth * block_cols(p);
    const int64_t stride = p.max_pages;
    int same = depth > 0;
    if (first != b)
        for (int c = threadIdx.x; c < cols; c += kFindThreads)
            if (p.table[b * stride + c] != p.table[first * stride + c]) same = 0;
    same = __syncthreads_and(same);
    if (threadIdx.x == 0) scratch[2 * p.B + b] = same ? first : -1;
}

// The plan, one CTA: groups of two or more that save enough, in the order of their first sequences.
constexpr int kPlanThreads = 1024;
// Of a plan that leaves the choice to the attention: what a group saves, in positions.  (It is made before the heads are
// known, and takes out what does not matter: beside 64 sequences under 8192 positions, 16 groups of 8 under 512, 1024 and
// 2048 more left for themselves and read once, us: 14:2 heads of 64 29.4 and 29.0, 31.0 and 29.7, 34.9 and 31.7;
// 32:8 of 128 65 and 63, 79 and 69, 110 and 83.  Of 4 under 1024, 2048 and 4096: 29.4 and 28.8, 31.4 and 30.1,
// 35.3 and 36.7; 61 and 59, 76 and 73, 112 and 99.)
constexpr int kGroupMinSaved = 8192;
__global__ void __launch_bounds__(kPlanThreads) kvp_plan_kernel(const FindParams p) {
    __shared__ int s_leader[kMaxBatch], s_count[kMaxBatch], s_group[kMaxBatch], s_off[kMaxBatch];
    __shared__ int s_warp[2][32];
    __shared__ unsigned long long s_saved;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int b = static_cast<int>(threadIdx.x), lane = b & 31, warp = b >> 5;
    const int* scratch = p.plan + 4 + kPlanArrays * p.B;
    const int depth = b < p.B ? scratch[b] : 0, leader = b < p.B ? scratch[2 * p.B + b] : -1;
    s_leader[b] = leader;
    s_count[b] = 0;
    if (b == 0) s_saved = 0;
    __syncthreads();
    if (leader >= 0) atomicAdd(&s_count[leader], 1);
    __syncthreads();
    // leaders of groups that stay
    const int64_t saved = static_cast<int64_t>(s_count[b] - 1) * depth * kShareBlock;
    const bool stays = leader == b && s_count[b] > 1 && saved >= (p.min_saved < 0 ? kGroupMinSaved : p.min_saved);
    if (stays) atomicAdd(&s_saved, static_cast<unsigned long long>(saved / kShareBlock));   // (integers: any order)
    int g = stays ? 1 : 0, off = stays ? s_count[b] : 0;   // prefix sums over the sequences
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, g, d), y = __shfl_up_sync(0xffffffffu, off, d);
        if (lane >= d) g += x, off += y;
    }
    if (lane == 31) s_warp[0][warp] = g, s_warp[1][warp] = off;
    __syncthreads();
    int groups = 0, members = 0;
    for (int i = 0; i < kPlanThreads / 32; ++i) {
        if (i < warp) g += s_warp[0][i], off += s_warp[1][i];
        groups += s_warp[0][i];
        members += s_warp[1][i];
    }
    s_group[b] = stays ? g - 1 : -1;
    s_off[b] = stays ? off - s_count[b] : 0;
    __syncthreads();
    auto put = [&](int array, int i, int x) { p.plan[4 + array * p.B + i] = x; };
    if (stays) {
        put(0, g - 1, off - s_count[b]);
        put(1, g - 1, s_count[b]);
        put(2, g - 1, depth);
    }
    if (b >= groups && b < p.B) {   // entries of no group
        put(0, b, 0);
        put(1, b, 0);
        put(2, b, 0);
    }
    if (b >= members && b < p.B) put(3, b, 0);
    if (b < p.B) {
        const int mine = leader >= 0 ? s_group[leader] : -1;
        int rank = 0;
        if (mine >= 0) {
            for (int k = 0; k < b; ++k) rank += s_leader[k] == leader;
            put(3, s_off[leader] + rank, b);
        }
        put(4, b, mine);
        put(5, b, rank);
        put(6, b, mine >= 0 ? depth * kShareBlock : 0);
        put(7, b, mine >= 0 ? s_count[leader] : 0);
    }
    if (b == 0) {
        p.plan[1] = groups;
        p.plan[2] = p.B;
        p.plan[3] = p.min_saved < 0 ? static_cast<int>(min(s_saved, 0x7ffffffeull)) : kPlanAlways;
        p.plan[0] = kPlanMagic;
    }
}

// ------------------------------------------------------------------ host

// Keys and values that a plan's groups save by reading prefixes once, from which on it is followed where it leaves
// that to the attention.  Every sequence for itself against the prefixes once, us: 128 sequences of 512
// shared positions, 8 KV heads of 128 (133 MB) 34 and 38, of 1024 (266 MB) 48 and 39; 32 sequences of 2048
// (130 MB) 26 and 25; 128 sequences of 2048, 2 KV heads of 64 (67 MB) 21 and 23, of 4096 (133 MB) 29 and 24.
// (With many rows less is worth while: 16 sequences with 64 queries behind 4096 positions, 32:8 heads of 128, 126 MB, 413
// and 186, behind 256, 8 MB, 122 and 131; there a plan made with a number of positions asks for it.)
constexpr int64_t kWorthBytes = 128ll << 20;
// And the sequences that a group has to have there.  A run of 128 positions of a KV head takes an SM about 1.9 us
// here, for two rows as for 256, and each sequence for itself 0.3 to 0.4 us (D = 64, up to 16 rows, in part from L2) or
// 0.6 to 0.8 (D = 128).  Groups under 16384 positions, for themselves and read once, us: 14:2 heads of 64, 12 of 4 35 and
// 49, 8 of 6 35 and 39, 6 of 8 35 and 35, two queries 9 of 5 43 and 45, 8 of 6 45 and 43; 32:8 of 128, 24 of 2 254 and
// 323, 16 of 3 250 and 225, four queries 256 and 334, 256 and 235.  With more rows each sequence for itself takes
// longer: five queries, 48 of 2 283 and 170, 790 and 683 (three, 14:2 heads of 64, 149 and 157): any group is followed.
int least_members(int D, int64_t rows) { return rows > 16 ? 2 : D == 128 ? 3 : rows > 8 ? 6 : 8; }

// Rows of a CTA of the prefix kernel: one Q tile where all the batch's rows of a KV head fit it.
int prefix_tiles(int B, int64_t rows) { return B * rows <= kPreRows ? 1 : 2; }

struct SharedSizes {
    size_t own_part, own_o, own_lse, row_o, row_lse, part_o, part_lse;
    size_t total() const { return own_part + own_o + own_lse + row_o + row_lse + part_o + part_lse; }
};
SharedSizes shared_sizes(int B, int Hq, int Hkv, int Nq, int D, int sms) {
    const int64_t rows = static_cast<int64_t>(Hq / Hkv) * Nq;
    const size_t all = static_cast<size_t>(B) * Hq * Nq;
    const size_t parts = 2 * static_cast<size_t>(sms) * prefix_tiles(B, rows) * kPreRows;
    return {part_bytes(rows, D, own_workers(sms, static_cast<int>(rows))),
            pad256(all * D * sizeof(float)),   pad256(all * sizeof(float)),
            pad256(all * D * sizeof(float)),   pad256(all * sizeof(float)),
            pad256(parts * D * sizeof(float)), pad256(parts * sizeof(float))};
}

template <int D, bool BF16, int QT>
cudaError_t launch_prefix(const PreParams& p, cudaStream_t stream) {
    auto kern = kv8_prefix_kernel<D, BF16, QT>;
    static SmemLimit limit;
    const cudaError_t e = limit.raise(kern, PreCfg<D, QT>::kSmem);
    if (e != cudaSuccess) return e;
    return launch_dependent(kern, p.a.ctas, PreCfg<D, QT>::kThreads, PreCfg<D, QT>::kSmem, stream, p);
}

template <int D, bool BF16>
cudaError_t launch_shared_merge(const PreParams& p, int row_block, int row8, cudaStream_t stream) {
    const int64_t rows = static_cast<int64_t>(p.a.B) * p.a.Hkv * p.a.rows;
    // Few rows have many parts, which four warps take together: 896 rows (64 samples under 32K positions) 36.3 us
    // the whole call and 33.7, two sequences of 64K for themselves 39 and 22; 2304 rows with a warp each 40,
    // with four 47 (few parts, and four times the CTAs).
    if (rows <= static_cast<int64_t>(kMergeRowsAlone) * p.a.ctas)
        return launch_dependent(kv8_shared_merge_kernel<D, BF16, kMergeWarps>, static_cast<unsigned>(rows),
                                kMergeWarps * 32, 0, stream, p, row_block, row8);
    return launch_dependent(kv8_shared_merge_kernel<D, BF16, 1>,
                            static_cast<unsigned>((rows + kMergeWarps - 1) / kMergeWarps), kMergeWarps * 32, 0,
                            stream, p, row_block, row8);
}

}  // namespace
}  // namespace tme

using namespace tme;

extern "C" size_t kvp_plan_words(int n_seqs) {
    if (n_seqs <= 0 || n_seqs > kMaxBatch) return 0;
    return 4 + static_cast<size_t>(kPlanArrays + kPlanScratch) * n_seqs;
}

extern "C" int kvp_find_shared(const int* table, const int* lens, int n_seqs, int max_pages, int page,
                               int min_saved, int* plan, void* stream) {
    if (!table || !lens || !plan || n_seqs <= 0 || max_pages <= 0 || page <= 0 || min_saved < -1)
        return ATTN_ERR_INVALID;
    if (n_seqs > kMaxBatch) return ATTN_ERR_UNSUPPORTED;
    int rc = check_cache(n_seqs, 1, 64, page, 1, max_pages);
    if (rc != ATTN_OK) return rc;
    const void* words[] = {table, lens, plan};
    if (!aligned(words, 4)) return ATTN_ERR_ALIGN;
    unsigned int* status;
    if ((rc = device_setup_public(&status)) != ATTN_OK) return rc;
    const int shift = page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7;
    const FindParams p{table, lens, plan, n_seqs, max_pages, shift, min_saved};
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = launch_kernel(kvp_depth_kernel, dim3(n_seqs), dim3(kFindThreads), 0, st, p);
    if (e == cudaSuccess) e = launch_dependent(kvp_leader_kernel, n_seqs, kFindThreads, 0, st, p);
    if (e == cudaSuccess) e = launch_dependent(kvp_plan_kernel, 1, kPlanThreads, 0, st, p);
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

extern "C" size_t kv8_attn_shared_workspace_size(int B, int Hq, int Hkv, int Nq, int D) {
    if (kv8_attn_workspace_size(B, Hq, Hkv, Nq, D) == 0) return 0;
    const int sms = device_sms();
    return shared_sizes(B, Hq, Hkv, Nq, D, sms > 0 ? sms : 1).total();
}

extern "C" int kv8_attn_shared(const void* q, const void* k_pages, const void* v_pages,
                               const float* k_scale, const float* v_scale, const int* table,
                               const int* lens, const int* n_new, const int* granted, const int* plan,
                               void* out, float* lse, void* workspace, size_t workspace_bytes, int B,
                               int Hq, int Hkv, int Nq, int D, int page, int n_pages, int max_pages,
                               float scale, int dtype, void* stream) {
    if (!plan) return ATTN_ERR_INVALID;
    if (reinterpret_cast<uintptr_t>(plan) & 3) return ATTN_ERR_ALIGN;
    PreParams p{};
    int rc = attn_params(&p.a, q, k_pages, v_pages, k_scale, v_scale, table, lens, n_new, granted, out, lse,
                         workspace, workspace_bytes, kv8_attn_shared_workspace_size(B, Hq, Hkv, Nq, D), B,
                         Hq, Hkv, Nq, D, page, n_pages, max_pages, scale, 0, 0, dtype);
    if (rc != ATTN_OK) return rc;
    const int64_t rows = static_cast<int64_t>(Hq / Hkv) * Nq;
    const int qt = prefix_tiles(B, rows), row_block = qt * kPreRows;
    // steps of all groups, and rows, are counted in 32 bits; B / 2 groups at most
    const int64_t blocks = (static_cast<int64_t>(B) * rows + row_block - 1) / row_block + B / 2;
    if (static_cast<int64_t>(B) * Hkv * ((rows + 31) / 32) *
            ((static_cast<int64_t>(max_pages) * page + 31) / 32 + own_steps(p.a.rows)) > 0x7fffffffll)
        return ATTN_ERR_UNSUPPORTED;
    const int64_t unit = static_cast<int64_t>(max_pages) * page / kShareBlock + kUnitSteps + 1;
    if (rows > 1 << 20 || static_cast<int64_t>(B) * Hq * Nq > 0x7fffffffll || blocks * Hkv * unit > 0x7fffffffll ||
        (static_cast<int64_t>(B) * Hkv * rows + kMergeWarps - 1) / kMergeWarps > 0x7fffffffll)
        return ATTN_ERR_UNSUPPORTED;
    const SharedSizes z = shared_sizes(B, Hq, Hkv, Nq, D, p.a.ctas);
    char* at = static_cast<char*>(workspace) + z.own_part;
    // (as many parts as there are shares)
    p.a.part_lse = reinterpret_cast<float*>(at - pad256(2 * static_cast<size_t>(own_workers(p.a.ctas, p.a.rows)) * 8 *
                                                        row_tiles(rows) * sizeof(float)));
    auto take = [&](size_t bytes) {
        float* r = reinterpret_cast<float*>(at);
        at += bytes;
        return r;
    };
    p.a.plan = plan;
    const int64_t run_bytes = 2ll * Hkv * D * kShareBlock, least = (kWorthBytes + run_bytes - 1) / run_bytes;
    p.a.least_runs = static_cast<int>(least);
    p.a.least_members = least_members(D, rows);
    p.a.own_o = take(z.own_o);
    p.a.own_lse = take(z.own_lse);
    p.row_o = take(z.row_o);
    p.row_lse = take(z.row_lse);
    p.part_o = take(z.part_o);
    p.part_lse = take(z.part_lse);
    p.k_pages = static_cast<const uint8_t*>(k_pages);
    p.v_pages = static_cast<const uint8_t*>(v_pages);
    const bool bf16 = dtype == ATTN_BF16;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaErrorInvalidValue;
#define TME_PREFIX(d, b, n) \
    if (D == d && bf16 == b && qt == n) e = launch_prefix<d, b, n>(p, st);
    TME_PREFIX(64, false, 1)
    TME_PREFIX(64, false, 2)
    TME_PREFIX(64, true, 1)
    TME_PREFIX(64, true, 2)
    TME_PREFIX(128, false, 1)
    TME_PREFIX(128, false, 2)
    TME_PREFIX(128, true, 1)
    TME_PREFIX(128, true, 2)
#undef TME_PREFIX
    if (e != cudaSuccess) return ATTN_ERR_CUDA;
    rc = attn_launch_shared(p.a, k_pages, v_pages, D, page, bf16, st);
    if (rc != ATTN_OK) return rc;
    const int row8 = 8 * row_tiles(rows);
    e = D == 64 ? (bf16 ? launch_shared_merge<64, true>(p, row_block, row8, st)
                        : launch_shared_merge<64, false>(p, row_block, row8, st))
                : (bf16 ? launch_shared_merge<128, true>(p, row_block, row8, st)
                        : launch_shared_merge<128, false>(p, row_block, row8, st));
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}
