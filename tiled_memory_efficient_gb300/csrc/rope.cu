// rope.cu -- rotary positions: queries and keys (include/rope.h), and the append to
// the paged 8-bit cache that turns its keys on the way.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "../../include/rope.h"
#include "attn_internal.h"
#include "kv8.cuh"
#include "rope.cuh"

namespace tme {
namespace {

// ------------------------------------------------------------------ queries and keys

// New tokens of sequence b of that length (T at most, the table holds `most` positions): -1 for a
// count that does not fit, 0 without room.
__device__ __forceinline__ int tokens_of(const int* granted, const int* n_new, int b, int T, int len, int most) {
    if (granted && *granted == 0) return 0;
    const int n = n_new ? n_new[b] : T;
    if (n == 0) return 0;
    return n < 0 || n > T || n > len || len > most ? -1 : n;
}

struct RopeParams {
    RopeView f;
    const uint16_t* x[2];   // q, k
    uint16_t* y[2];
    int64_t xs[2][3], ys[2][3];   // batch, head, row strides
    const int* pos;
    int64_t pos_b, pos_n;
    int start, B, N, Hq, heads;
    // positions of a cache's newest tokens instead (lens null: none)
    const int* lens;
    const int* n_new;
    const int* granted;
    int most;                     // positions that the table holds
    int tok_shift;                // tokens of a CTA
    int per_thread;               // heads a thread takes, kRopeBatch at most
};

// CTAs of two warps, each for itself at its barrier: rows of 2 x 8192 tokens with 32 heads of 128 take
// 43 us a pass with 64 threads, 44 with 128 and 47 with 256.
constexpr int kRopeThreads = 64;

// Bound by memory: every value is read and written once.  A CTA takes a few tokens and a range of heads;
// a thread 16 dimensions (an item) of one token and up to four of the heads, all of which it asks for
// before the CTA makes its sines, each once.  (Each thread making the sines of its own item for all
// heads that it takes: 16384 tokens of 16 heads of 64 in 15.5 us against 13.2, 64 tokens of 40 heads
// of 128 in 3.6 against 2.6.)  2 x 8192 tokens, 32 heads of 128: 268 MB in 43 us, 6.2 TB/s.
template <int D, bool BF16, int MODE>
__global__ void __launch_bounds__(kRopeThreads, 8) rope_kernel(const __grid_constant__ RopeParams p) {
    constexpr int items = D / 16, kItemShift = D == 128 ? 3 : 2;
    __shared__ __align__(16) float s_cos[kRopeThreads * 8], s_sin[kRopeThreads * 8];   // [token][place of pair]
    // What was before is complete from here on; what is behind may set up.  (Behind an append's prompts, which
    // did the same before they let this one start: they are waited for at the end.)
    if (!p.lens) asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int item = static_cast<int>(threadIdx.x) & (items - 1);
    const int tl = (static_cast<int>(threadIdx.x) >> kItemShift) & ((1 << p.tok_shift) - 1);
    const int hg = static_cast<int>(threadIdx.x) >> (kItemShift + p.tok_shift);   // the thread's first head
    const int step = kRopeThreads >> (kItemShift + p.tok_shift);
    const int tok = (static_cast<int>(blockIdx.x) << p.tok_shift) + tl;
    const bool inside = tok < p.B * p.N;
    const int b = inside ? tok / p.N : 0, n = inside ? tok - b * p.N : 0;
    const int first = static_cast<int>(blockIdx.y) * p.per_thread * step;
    RopeRows t;
    t.x0 = p.x[0] + b * p.xs[0][0] + n * p.xs[0][2];
    t.x1 = p.x[1] + b * p.xs[1][0] + n * p.xs[1][2];
    t.y0 = p.y[0] + b * p.ys[0][0] + n * p.ys[0][2];
    t.y1 = p.y[1] + b * p.ys[1][0] + n * p.ys[1][2];
    t.xh0 = p.xs[0][1], t.xh1 = p.xs[1][1], t.yh0 = p.ys[0][1], t.yh1 = p.ys[1][1];
    t.first = p.Hq;
    int pos;
    bool live = true;
    if (p.lens) {
        const int len = p.lens[b], fresh = tokens_of(p.granted, p.n_new, b, p.N, len, p.most);
        live = n < fresh;
        pos = len - fresh + n;
    } else {
        pos = p.pos ? p.pos[b * p.pos_b + n * p.pos_n] : p.start + n;
    }
    // Pairs in eights, an item's, whose first fours come before all second fours: a token's items
    // read whole lines.
    auto place = [&](int pair) { return tl * (D / 2) + ((pair >> 2) & 1) * (D / 4) + (pair >> 3) * 4 + (pair & 3); };
    auto sines = [&](float (&c)[8], float (&s)[8]) {
        for (int pair = hg * items + item; 2 * pair < p.f.rot; pair += step * items) {
            const float2 cs = rope_cs(p.f.turns, pair, pos, p.f.amp);
            s_cos[place(pair)] = cs.x;
            s_sin[place(pair)] = cs.y * p.f.sign;
        }
        __syncthreads();
        if constexpr (MODE == kRopeScalar) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {   // (places past the last pair: read, not used)
                const int at = place(item_pair<MODE>(item, items, j));
                c[j] = s_cos[at];
                s[j] = s_sin[at];
            }
        } else {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const float4 cc = *reinterpret_cast<const float4*>(s_cos + place(8 * item + 4 * g));
                const float4 ss = *reinterpret_cast<const float4*>(s_sin + place(8 * item + 4 * g));
                c[4 * g] = cc.x, c[4 * g + 1] = cc.y, c[4 * g + 2] = cc.z, c[4 * g + 3] = cc.w;
                s[4 * g] = ss.x, s[4 * g + 1] = ss.y, s[4 * g + 2] = ss.z, s[4 * g + 3] = ss.w;
            }
        }
    };
    const int end = inside ? min(first + p.per_thread * step, p.heads) : 0;
    rope_item<BF16, MODE>(p.f, t, item, items, first + hg, step, end, live, sines);
    if (p.lens) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Tokens and heads of a CTA: heads a thread as many as leave every SM two CTAs; tokens so that the heads
// fill the CTAs and the sines are few (a sine costs about as much as two thirds of an item).
struct RopeSplit {
    int tok_shift, per_thread;
    int64_t x, y;
};
RopeSplit split_rope(int64_t tokens, int heads, int D, int rot) {
    const int item_shift = D == 128 ? 3 : 2;
    RopeSplit best{};
    for (int k = kRopeBatch; k >= 1; k >>= 1) {
        double least = 0.0;
        for (int ts = 0; kRopeThreads >> (item_shift + ts); ++ts) {
            const int per = (kRopeThreads >> (item_shift + ts)) * k;   // heads of a CTA
            const int64_t x = (tokens + (int64_t(1) << ts) - 1) >> ts, y = (heads + per - 1) / per;
            const int sines = ((rot / 2 << ts) + kRopeThreads - 1) / kRopeThreads;   // a thread
            const double cost = static_cast<double>(x) * static_cast<double>(y) * (3 * k + 2 * sines);
            if (least > 0.0 && cost >= least) continue;
            least = cost;
            best = {ts, k, x, y};
        }
        if (best.x * best.y >= 2 * device_sms()) break;
    }
    return best;
}

template <int D, bool BF16>
cudaError_t launch_rope(RopeParams p, cudaStream_t stream) {
    const RopeSplit s = split_rope(static_cast<int64_t>(p.B) * p.N, p.heads, D, p.f.rot);
    p.tok_shift = s.tok_shift;
    p.per_thread = s.per_thread;
    const dim3 grid(static_cast<unsigned>(s.x), static_cast<unsigned>(s.y)), block(kRopeThreads);
    void (*kern)(RopeParams) = p.f.mode == kRopeHalf    ? rope_kernel<D, BF16, kRopeHalf>
                               : p.f.mode == kRopeInter ? rope_kernel<D, BF16, kRopeInter>
                                                        : rope_kernel<D, BF16, kRopeScalar>;
    return launch_dependent(kern, grid, block, 0, stream, p);
}
cudaError_t launch_rope(const RopeParams& p, int D, bool bf16, cudaStream_t stream) {
    if (D == 128) return bf16 ? launch_rope<128, true>(p, stream) : launch_rope<128, false>(p, stream);
    return bf16 ? launch_rope<64, true>(p, stream) : launch_rope<64, false>(p, stream);
}

// Heads a thread of a step's queries takes of `heads`, given the threads that one head needs: as many as
// leave the device its threads, at least two.
int heads_per_thread(int64_t threads, int heads) {
    const int64_t want = static_cast<int64_t>(device_sms() > 0 ? device_sms() : 1) * 1024;
    int64_t parts = (want + threads - 1) / threads;
    const int most = (heads + 1) / 2;
    if (parts > most) parts = most;
    return static_cast<int>((heads + parts - 1) / parts);
}

int check_rope(int D, int rot, int interleaved, float amplitude, const unsigned long long* turns) {
    if (!turns) return ATTN_ERR_INVALID;
    if (rot < 2 || rot > D || rot % 2) return ATTN_ERR_INVALID;
    if (interleaved != 0 && interleaved != 1) return ATTN_ERR_INVALID;
    if (!(amplitude > 0.0f) || !std::isfinite(amplitude)) return ATTN_ERR_INVALID;
    if (reinterpret_cast<uintptr_t>(turns) & 7) return ATTN_ERR_ALIGN;
    return ATTN_OK;
}

// The strides of a tensor: none negative, all multiples of 16 bytes.
int check_strides(const long long* s) {
    for (int i = 0; i < 3; ++i)
        if (s[i] < 0) return ATTN_ERR_INVALID;
    for (int i = 0; i < 3; ++i)
        if (s[i] % 8) return ATTN_ERR_ALIGN;
    return ATTN_OK;
}
bool same_strides(const long long* a, const long long* b) {
    return a[0] == b[0] && a[1] == b[1] && a[2] == b[2];
}

// ------------------------------------------------------------------ append

struct AppendRopeParams {
    RopeView f;
    const uint16_t* src[2];   // k, v
    uint8_t* pages[2];
    float* scales[2];
    const uint16_t* q;
    uint16_t* q_out;
    const int* table;
    const int* lens;
    const int* n_new;
    const int* granted;
    unsigned int* status;
    int64_t sb, sh, st, qb, qh, qt, ob, oh, ot;
    int B, Hq, Hkv, T, n_pages, max_pages, n_slots, page_shift;
    int heads;        // of a page that a CTA takes in turn (prompts)
    int page_ctas;    // CTAs of pages; the others turn queries (steps)
    int q_threads;    // threads that one head's queries need
    int q_chunk;      // heads a thread of those takes
};

// The tokens that slot `slot` of sequence b's new ones has on its page.
struct PageTokens {
    int n, start, t0, lo, hi, pid;   // new tokens; position of the first; of the page's first; new ones on it
    int64_t head;                    // (page, head) of head 0
    __device__ __forceinline__ bool find(const AppendRopeParams& p, int b, int slot, bool report) {
        const int len = p.lens[b];
        n = tokens_of(p.granted, p.n_new, b, p.T, len, p.max_pages << p.page_shift);
        if (n <= 0) {
            if (n < 0 && report) atomicOr(p.status, kStatusPage);
            return false;
        }
        start = len - n;
        const int col = (start >> p.page_shift) + slot;
        t0 = col << p.page_shift;
        if (t0 >= len) return false;
        lo = max(start, t0);
        hi = min(len, t0 + (1 << p.page_shift));
        pid = p.table[static_cast<int64_t>(b) * p.max_pages + col];
        if (pid < 0 || pid >= p.n_pages) {
            if (report) atomicOr(p.status, kStatusPage);
            return false;
        }
        head = static_cast<int64_t>(pid) * p.Hkv;
        return true;
    }
};

// The other half of each of a vector's pairs: dimensions d0 .. d0 + 7 of the row at `row` hold x (words w), and
// neighbouring lanes the row's other vectors (every lane of the warp takes part).
template <bool BF16>
__device__ __forceinline__ void other_halves(const RopeView& f, const uint4& w, const float (&x)[8], int d0,
                                             const uint16_t* row, bool fresh, float (&o)[8]) {
    const int half = f.rot >> 1;
    if (f.mode == kRopeHalf) {
        const int away = d0 < f.rot ? (d0 < half ? half / 8 : -(half / 8)) : 0;
        const uint32_t y[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 e = rope_unpack<BF16>(__shfl_sync(0xffffffffu, y[j], (threadIdx.x + away) & 31));
            o[2 * j] = e.x;
            o[2 * j + 1] = e.y;
        }
    } else if (f.mode == kRopeInter) {
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = x[j ^ 1];
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int d = d0 + j;
            o[j] = fresh && d < f.rot ? rope_load<BF16>(row + (d < half ? d + half : d - half)) : 0.0f;
        }
    }
}
// Pair of dimension d, and whether it is the pair's first half.
__device__ __forceinline__ int pair_of(const RopeView& f, int d) {
    return f.mode == kRopeInter ? d >> 1 : d < f.rot >> 1 ? d : d - (f.rot >> 1);
}
__device__ __forceinline__ bool first_of(const RopeView& f, int d) {
    return f.mode == kRopeInter ? !(d & 1) : d < f.rot >> 1;
}
__device__ __forceinline__ float finite_max(float top, const float (&y)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float a = fabsf(y[j]);
        top = fmaxf(top, a < INFINITY ? a : 0.0f);   // false for a NaN, too
    }
    return top;
}
template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& w, float (&y)[8]) {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 e = rope_unpack<BF16>(x[j]);
        y[2 * j] = e.x;
        y[2 * j + 1] = e.y;
    }
}
__device__ __forceinline__ uint2 quantise8(const float (&y)[8], float inv) {
    uint32_t r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j] = f32_to_e4m3x2(y[2 * j] * inv, y[2 * j + 1] * inv);
    return make_uint2(r[0] | (r[1] << 16), r[2] | (r[3] << 16));
}

// Prompts: one CTA per (sequence, page it may touch, keys or values), `heads` KV heads in turn.  A thread
// holds two rows' items (rope_item's, the two halves of each pair in one thread); the next two heads' are
// on their way to shared memory meanwhile.  The page's sines are made once for all of the CTA's heads:
// each pair's for its position at every fourth token, the three beside it by one turn of that by the angle of
// one or two tokens.  They are then off by 2^-21.8 at most (2^-24.3 rms, over 2^24 random frequencies and
// positions), where every one made for its position is by 2^-23.0 (2^-24.9), at 24.4 us instead of what follows.  2 x
// 8190 tokens, 8 KV heads, D = 128, 67 MB read and 34 written: 21.8 us (one head ahead in registers takes 1.6
// longer, four ahead 2.8; in 64 registers a thread 1.1), bound by each head's chain of turn, maximum, barrier,
// scale and store in three CTAs an SM; the plain append, without sines, takes 14.8.  Pairs that no vector holds
// whole (kRopeScalar) are read and written by the element: 48.2 with 40 of the dimensions turning.
template <int D>
constexpr int prompt_threads(int page) { return page * (D / 32); }
// CTAs of an SM up to which a page's heads are cut (the sines are made once a CTA): 8 take 21.6 us there.
constexpr int kPromptCtas = 4;
constexpr int kPromptThreads = 512;   // at most: pages of 128 tokens, D = 128
constexpr int kPromptAhead = 2;       // heads on their way, a power of two

// 16 bytes global -> shared, asynchronously; 0 instead if not `real`.
__device__ __forceinline__ void copy16(void* dst, const void* src, bool real) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(real ? 16 : 0)
                 : "memory");
}

// Largest finite magnitude of a thread's values: an infinity sends it to the slow look.
__device__ __forceinline__ float item_max(const float (&y)[2][16]) {
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) top = fmaxf(top, fabsf(y[i][j]));   // (a NaN is passed over)
    if (top < INFINITY) return top;
    top = 0.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) top = fmaxf(top, fabsf(y[i][j]) < INFINITY ? fabsf(y[i][j]) : 0.0f);
    return top;
}

template <int D, bool BF16, int MODE>
__global__ void __maxnreg__(80) kv8_append_rope_kernel(const __grid_constant__ AppendRopeParams p) {
    constexpr int items = D / 16;
    extern __shared__ __align__(16) float s_cos[];   // [token][pitch] of the page, then the sines
    __shared__ uint32_t s_max[2][kPromptThreads / 32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");   // what is behind may set up meanwhile
    int id = static_cast<int>(blockIdx.x);
    const int which = id & 1;
    id >>= 1;
    const int parts = (p.Hkv + p.heads - 1) / p.heads, part = id % parts;
    id /= parts;
    const int b = id / p.n_slots;
    PageTokens t;
    if (!t.find(p, b, id - b * p.n_slots, threadIdx.x == 0)) return;
    const int h0 = part * p.heads, h1 = min(h0 + p.heads, p.Hkv);
    const int page = 1 << p.page_shift, step = page >> 1;   // the thread's rows: tok and tok + step
    const int tok = static_cast<int>(threadIdx.x) / items, item = static_cast<int>(threadIdx.x) % items;
    const int half = p.f.rot >> 1;
    const bool keys = which == 0;
    // whether the item turns, and its two vectors (MODE 2: of the values)
    const bool turns = keys && (MODE == kRopeScalar ? item < half : 8 * item < half);
    const bool whole = MODE != kRopeHalf || 8 * item < half;
    const int d0 = MODE != kRopeHalf ? 16 * item : whole ? 8 * item : p.f.rot + 16 * (item - (p.f.rot >> 4));
    const int d1 = MODE != kRopeHalf || !whole ? d0 + 8 : d0 + half;
    auto pair_of = [&](int j) { return MODE == kRopeScalar ? item + j * items : 8 * item + j; };
    // MODE 2, keys: a pair's dimensions (two that stay past the turned ones)
    auto first = [&](int j) { const int i = pair_of(j); return i < half ? i : 2 * i; };
    auto second = [&](int j) { const int i = pair_of(j); return i < half ? i + half : 2 * i + 1; };
    const uint16_t* src = p.src[which] + b * p.sb + (t.t0 + tok - t.start) * p.st;
    bool fresh[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) fresh[i] = t.t0 + tok + i * step >= t.lo && t.t0 + tok + i * step < t.hi;
    // A thread's vectors of a head travel into shared memory that it alone reads (0 where a token is not new);
    // MODE 2's keys are read element by element where they are used.
    const bool copies = MODE != kRopeScalar || !keys;
    const int pitch = (half + 7) & ~7;
    float* s_sin = s_cos + (pitch << p.page_shift);
    uint4* s_raw = reinterpret_cast<uint4*>(s_sin + (pitch << p.page_shift)) + threadIdx.x;
    auto ask = [&](int h) {
        if (copies && h < h1) {
            uint4* to = s_raw + (h & (kPromptAhead - 1)) * 4 * blockDim.x;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint16_t* row = fresh[i] ? src + h * p.sh + i * step * p.st : p.src[which];
                copy16(to + (2 * i) * blockDim.x, row + (fresh[i] ? d0 : 0), fresh[i]);
                copy16(to + (2 * i + 1) * blockDim.x, row + (fresh[i] ? d1 : 0), fresh[i]);
            }
        }
        cp_async_commit();
    };
    for (int i = 0; i < kPromptAhead; ++i) ask(h0 + i);
    // Pairs of a token's row of sines: in eights (an item's), whose first fours come before all second
    // fours, so that a token's items read whole lines; past the last pair a turn by nothing.
    auto place = [&](int pair) { return ((pair >> 2) & 1) * (pitch >> 1) + (pair >> 3) * 4 + (pair & 3); };
    if (keys) {
        // a thread one pair (there are as many threads, at least) at every so many fours of tokens
        const int shift = pitch > 32 ? 6 : pitch > 16 ? 5 : pitch > 8 ? 4 : 3;
        const int pair = static_cast<int>(threadIdx.x) & ((1 << shift) - 1);
        if (pair < pitch) {
            const unsigned long long turn = pair < half ? __ldg(p.f.turns + pair) : 0ull;
            const float amp = pair < half ? p.f.amp : 1.0f;
            const float2 one = rope_cs(turn, 1.0f), two = rope_cs(2 * turn, 1.0f);
            for (int x = 4 * (static_cast<int>(threadIdx.x) >> shift); x < page; x += 4 * (static_cast<int>(blockDim.x) >> shift)) {
                const float2 m = rope_cs(rope_phase(turn, t.t0 + x + 2), amp);
                float *c = s_cos + x * pitch + place(pair), *s = s_sin + x * pitch + place(pair);
                c[0] = m.x * two.x + m.y * two.y, s[0] = m.y * two.x - m.x * two.y;
                c[pitch] = m.x * one.x + m.y * one.y, s[pitch] = m.y * one.x - m.x * one.y;
                c[2 * pitch] = m.x, s[2 * pitch] = m.y;
                c[3 * pitch] = m.x * one.x - m.y * one.y, s[3 * pitch] = m.y * one.x + m.x * one.y;
            }
        }
        __syncthreads();
    }
#pragma unroll 1
    for (int h = h0; h < h1; ++h) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kPromptAhead - 1) : "memory");   // this head's are there
        float y[2][16];   // the items' first vectors, then their second ones
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t w[8];
            if (copies) {
                const uint4* from = s_raw + ((h & (kPromptAhead - 1)) * 4 + 2 * i) * blockDim.x;
                const uint4 lo = from[0], hi = from[blockDim.x];
                w[0] = lo.x, w[1] = lo.y, w[2] = lo.z, w[3] = lo.w;
                w[4] = hi.x, w[5] = hi.y, w[6] = hi.z, w[7] = hi.w;
            } else {
                const uint16_t* row = src + h * p.sh + i * step * p.st;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    w[j] = fresh[i] ? row[first(2 * j)] | static_cast<uint32_t>(row[first(2 * j + 1)]) << 16 : 0u;
                    w[4 + j] = fresh[i] ? row[second(2 * j)] | static_cast<uint32_t>(row[second(2 * j + 1)]) << 16 : 0u;
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 e = rope_unpack<BF16>(w[j]);
                y[i][2 * j] = e.x;
                y[i][2 * j + 1] = e.y;
            }
        }
        ask(h + kPromptAhead);
        if (turns) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int row = (tok + i * step) * pitch;
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    float c[4], s[4];
                    if constexpr (MODE == kRopeScalar) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int at = row + place(min(pair_of(4 * g + j), half - 1));
                            c[j] = s_cos[at];
                            s[j] = s_sin[at];
                        }
                    } else {
                        const float4 cc = *reinterpret_cast<const float4*>(s_cos + row + g * (pitch >> 1) + 4 * item);
                        const float4 ss = *reinterpret_cast<const float4*>(s_sin + row + g * (pitch >> 1) + 4 * item);
                        c[0] = cc.x, c[1] = cc.y, c[2] = cc.z, c[3] = cc.w;
                        s[0] = ss.x, s[1] = ss.y, s[2] = ss.z, s[3] = ss.w;
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float& a = MODE == kRopeInter ? y[i][8 * g + 2 * j] : y[i][4 * g + j];
                        float& e = MODE == kRopeInter ? y[i][8 * g + 2 * j + 1] : y[i][8 + 4 * g + j];
                        if (MODE != kRopeHalf && pair_of(4 * g + j) >= half) continue;   // (0 * inf is none)
                        const float x = a;
                        a = x * c[j] - e * s[j];
                        e = e * c[j] + x * s[j];
                    }
                }
            }
        }
        uint8_t* dst = p.pages[which] + (((t.head + h) << p.page_shift) + tok) * D;
        float* scale = p.scales[which] + t.head + h;
        const float s_old = t.t0 < t.start ? *scale : 0.0f;
        // largest finite magnitude: positive floats order like their bits
        uint32_t u = __reduce_max_sync(0xffffffffu, __float_as_uint(item_max(y)));
        if ((threadIdx.x & 31) == 0) s_max[h & 1][threadIdx.x >> 5] = u;
        __syncthreads();   // also: every thread has read the old scale
        for (int i = 0; i < static_cast<int>(blockDim.x) / 32; ++i) u = max(u, s_max[h & 1][i]);
        int e = amax_exp(__uint_as_float(u));
        const int e_old = t.t0 < t.start ? scale_exp(s_old) : e;
        e = max(e, e_old);
        if (threadIdx.x == 0) *scale = exp2i(e);
        const float inv = exp2i(-e);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (!fresh[i]) continue;
            uint32_t r[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) r[j] = f32_to_e4m3x2(y[i][2 * j] * inv, y[i][2 * j + 1] * inv);
            uint8_t* row = dst + i * step * D;
            if (MODE == kRopeScalar && keys) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    row[first(j)] = static_cast<uint8_t>(r[j >> 1] >> (8 * (j & 1)));
                    row[second(j)] = static_cast<uint8_t>(r[4 + (j >> 1)] >> (8 * (j & 1)));
                }
            } else {
                *reinterpret_cast<uint2*>(row + d0) = make_uint2(r[0] | (r[1] << 16), r[2] | (r[3] << 16));
                *reinterpret_cast<uint2*>(row + d1) = make_uint2(r[4] | (r[5] << 16), r[6] | (r[7] << 16));
            }
        }
        if (e != e_old)   // (each vector of an old token is one thread's, whoever's its new values are)
            for (int i = 0; i < 2; ++i) {
                const int pos = t.t0 + tok + i * step;
                raise_tokens<0, 1>(dst + i * step * D + 16 * item, pos, min(t.lo, pos + 1), e_old, e);
                raise_tokens<0, 1>(dst + i * step * D + 16 * item + 8, pos, min(t.lo, pos + 1), e_old, e);
            }
    }
}

// Steps of a few tokens: one warp per (sequence, page, KV head, keys or values), whose new tokens it
// holds whole; the CTAs behind those turn the queries.  A step is bound by its launch and two trips to memory:
// 64 single tokens, 32 query and 8 KV heads, D = 128 in 3.7 us (a CTA per page and head, as prompts had
// them, 9.9).
constexpr int kStepThreads = 128;
template <int D>
constexpr int step_tokens() { return 4 * (32 / (D / 8)); }   // tokens a warp holds: four turns of it

template <int D, bool BF16>
__global__ void __launch_bounds__(kStepThreads) kv8_step_rope_kernel(const __grid_constant__ AppendRopeParams p) {
    constexpr int VPT = D / 8, TPI = 32 / VPT, items = D / 16;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");   // the attention may set up meanwhile
    if (static_cast<int>(blockIdx.x) >= p.page_ctas) {
        // queries
        const int64_t id = static_cast<int64_t>(blockIdx.x - p.page_ctas) * kStepThreads + threadIdx.x;
        const int part = static_cast<int>(id / p.q_threads);
        if (part * p.q_chunk >= p.Hq) return;
        const int item = static_cast<int>(id) & (items - 1);   // (q_threads is a multiple of items)
        const int tok = static_cast<int>(id - static_cast<int64_t>(part) * p.q_threads) / items;
        const int h0 = part * p.q_chunk, h1 = min(h0 + p.q_chunk, p.Hq);
        const int b = tok / p.T, t = tok - b * p.T;
        const int len = p.lens[b];
        const int n = tokens_of(p.granted, p.n_new, b, p.T, len, p.max_pages << p.page_shift);
        RopeRows r;
        r.x0 = r.x1 = p.q + b * p.qb + t * p.qt;
        r.y0 = r.y1 = p.q_out + b * p.ob + t * p.ot;
        r.xh0 = r.xh1 = p.qh;
        r.yh0 = r.yh1 = p.oh;
        r.first = p.Hq;
        const bool live = t < n;
        const int pos = len - n + t;
        auto turn = [&](auto mode) {
            constexpr int MODE = decltype(mode)::value;
            rope_item<BF16, MODE>(p.f, r, item, items, h0, 1, h1, live, [&](float (&c)[8], float (&s)[8]) {
                if (live) item_sines<MODE>(p.f, item, items, pos, c, s);
            });
        };
        if (p.f.mode == kRopeHalf) turn(std::integral_constant<int, kRopeHalf>());
        else if (p.f.mode == kRopeInter) turn(std::integral_constant<int, kRopeInter>());
        else turn(std::integral_constant<int, kRopeScalar>());
        return;
    }
    int id = static_cast<int>(blockIdx.x) * (kStepThreads / 32) + static_cast<int>(threadIdx.x >> 5);
    const int which = id & 1;
    id >>= 1;
    const int h = id % p.Hkv;
    id /= p.Hkv;
    const int b = id / p.n_slots, lane = threadIdx.x & 31;
    PageTokens t;
    if (b >= p.B || !t.find(p, b, id - b * p.n_slots, lane == 0)) return;
    const int tok = lane / VPT, d0 = lane % VPT * 8;
    const uint16_t* src = p.src[which] + b * p.sb + h * p.sh;
    uint8_t* page = p.pages[which] + ((t.head + h) << p.page_shift) * D + d0;
    float* scale = p.scales[which] + t.head + h;
    const float s_old = t.t0 < t.start ? *scale : 0.0f;
    uint4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int pos = t.lo + i * TPI + tok;
        w[i] = make_uint4(0u, 0u, 0u, 0u);
        if (pos < t.hi) w[i] = *reinterpret_cast<const uint4*>(src + (pos - t.start) * p.st + d0);
    }
    float y[4][8], top = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        unpack8<BF16>(w[i], y[i]);
        const int pos = t.lo + i * TPI + tok;
        if (which == 0 && t.lo + i * TPI < t.hi) {   // (the same in all lanes)
            float o[8];
            other_halves<BF16>(p.f, w[i], y[i], d0, src + (pos - t.start) * p.st, pos < t.hi, o);
            if (d0 < p.f.rot && pos < t.hi) {
                float2 cs = make_float2(1.0f, 0.0f);
                float r[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if ((p.f.mode != kRopeInter || !(j & 1)) && d0 + j < p.f.rot)
                        cs = rope_cs(p.f.turns, pair_of(p.f, d0 + j), pos, p.f.amp);
                    r[j] = fmaf(first_of(p.f, d0 + j) ? -o[j] : o[j], cs.y, y[i][j] * cs.x);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (d0 + j < p.f.rot) y[i][j] = r[j];
            }
        }
        top = finite_max(top, y[i]);
    }
    int e = amax_exp(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top))));
    const int e_old = t.t0 < t.start ? scale_exp(s_old) : e;
    e = max(e, e_old);
    __syncwarp();   // every lane has read the old scale
    if (lane == 0) *scale = exp2i(e);
    const float inv = exp2i(-e);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int pos = t.lo + i * TPI + tok;
        if (pos < t.hi) *reinterpret_cast<uint2*>(page + (pos - t.t0) * D) = quantise8(y[i], inv);
    }
    if (e != e_old) raise_tokens<TPI * D, TPI>(page + tok * D, t.t0 + tok, t.lo, e_old, e);
}

template <int D, bool BF16>
cudaError_t launch_step(AppendRopeParams p, cudaStream_t stream) {
    constexpr int kWarps = kStepThreads / 32;
    int64_t ctas = (static_cast<int64_t>(p.B) * p.n_slots * p.Hkv * 2 + kWarps - 1) / kWarps;
    p.page_ctas = static_cast<int>(ctas);
    if (p.q) {
        p.q_threads = p.B * p.T * (D / 16);
        p.q_chunk = heads_per_thread(p.q_threads, p.Hq);
        const int64_t parts = (p.Hq + p.q_chunk - 1) / p.q_chunk;
        ctas += (parts * p.q_threads + kStepThreads - 1) / kStepThreads;
    }
    return launch_dependent(kv8_step_rope_kernel<D, BF16>, dim3(static_cast<unsigned>(ctas)), dim3(kStepThreads), 0,
                            stream, p);
}

template <int D, bool BF16, int MODE>
cudaError_t launch_prompt(AppendRopeParams p, cudaStream_t stream) {
    auto kern = kv8_append_rope_kernel<D, BF16, MODE>;
    static SmemLimit limit;
    // a page's cosines and sines, and the heads ahead: at most
    constexpr int kMost = 128 * D * static_cast<int>(sizeof(float)) + kPromptAhead * 64 * prompt_threads<D>(128);
    const cudaError_t e = limit.raise(kern, kMost);
    if (e != cudaSuccess) return e;
    // heads in turn as long as every SM still has some CTAs
    const int64_t pages = static_cast<int64_t>(p.B) * p.n_slots * 2;
    int64_t most = (static_cast<int64_t>(device_sms()) * kPromptCtas + pages - 1) / pages;   // CTAs of a page
    if (most < 1) most = 1;
    p.heads = most >= p.Hkv ? 1 : static_cast<int>((p.Hkv + most - 1) / most);
    const int64_t ctas = pages * ((p.Hkv + p.heads - 1) / p.heads);
    const int pitch = (p.f.rot / 2 + 7) & ~7;
    const int threads = prompt_threads<D>(1 << p.page_shift);
    const size_t smem = ((sizeof(float) * 2 * pitch) << p.page_shift) + kPromptAhead * 64 * threads;
    return launch_dependent(kern, dim3(static_cast<unsigned>(ctas)), dim3(threads), static_cast<int>(smem), stream, p);
}
template <int D, bool BF16>
cudaError_t launch_prompt(const AppendRopeParams& p, cudaStream_t stream) {
    switch (p.f.mode) {
        case kRopeHalf: return launch_prompt<D, BF16, kRopeHalf>(p, stream);
        case kRopeInter: return launch_prompt<D, BF16, kRopeInter>(p, stream);
        default: return launch_prompt<D, BF16, kRopeScalar>(p, stream);
    }
}

}  // namespace
}  // namespace tme

using namespace tme;

extern "C" int rope_apply(const void* q, const void* k, void* q_out, void* k_out,
                          const unsigned long long* turns, const int* positions, int start, int B,
                          int Hq, int Hk, int N, int D, int rot, int interleaved, float amplitude,
                          int transposed, const long long* strides, int dtype, void* stream) {
    if (!q || !q_out || !strides || (k == nullptr) != (k_out == nullptr) || (k == nullptr) != (Hk == 0))
        return ATTN_ERR_INVALID;
    if (B <= 0 || Hq <= 0 || Hk < 0 || N <= 0 || D <= 0) return ATTN_ERR_INVALID;
    if (D != 64 && D != 128) return ATTN_ERR_UNSUPPORTED;
    if ((dtype != ATTN_F16 && dtype != ATTN_BF16) || (transposed != 0 && transposed != 1))
        return ATTN_ERR_INVALID;
    int rc = check_rope(D, rot, interleaved, amplitude, turns);
    if (rc != ATTN_OK) return rc;
    const long long *sq = strides, *sk = strides + 3, *oq = strides + 6, *ok = strides + 9;
    for (const long long* s : {sq, sk, oq, ok}) {
        if (!k && (s == sk || s == ok)) continue;
        if ((rc = check_strides(s)) != ATTN_OK) return rc;
    }
    if ((q == q_out && !same_strides(sq, oq)) || (k && k == k_out && !same_strides(sk, ok)))
        return ATTN_ERR_INVALID;
    const void* ptrs[] = {q, k, q_out, k_out};
    const void* words[] = {positions};
    if (!aligned(ptrs, 16) || !aligned(words, 4)) return ATTN_ERR_ALIGN;
    if (!positions && static_cast<int64_t>(start) + N > 0x7fffffffll) return ATTN_ERR_UNSUPPORTED;
    // a thread's number (16 dimensions of a token) is 32-bit, and so are its grid's rows
    if (static_cast<int64_t>(B) * N > 1 << 27 || static_cast<int64_t>(Hq) + Hk > 65535) return ATTN_ERR_UNSUPPORTED;
    unsigned int* status;
    if ((rc = device_setup_public(&status)) != ATTN_OK) return rc;
    RopeParams p{};
    p.f = {turns, rot, rope_mode(rot, interleaved), amplitude, transposed ? -1.0f : 1.0f};
    const void* in[2] = {q, k ? k : q};
    void* out[2] = {q_out, k ? k_out : q_out};
    for (int w = 0; w < 2; ++w) {
        p.x[w] = static_cast<const uint16_t*>(in[w]);
        p.y[w] = static_cast<uint16_t*>(out[w]);
        for (int i = 0; i < 3; ++i) {
            p.xs[w][i] = (w == 1 && k ? sk : sq)[i];
            p.ys[w][i] = (w == 1 && k ? ok : oq)[i];
        }
    }
    p.pos = positions;
    p.pos_b = positions ? strides[12] : 0;
    p.pos_n = positions ? strides[13] : 0;
    p.start = start;
    p.B = B;
    p.N = N;
    p.Hq = Hq;
    p.heads = Hq + Hk;
    const cudaError_t e = launch_rope(p, D, dtype == ATTN_BF16, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

extern "C" int kv8_append_rope(const void* k, const void* v, void* k_pages, void* v_pages,
                               float* k_scale, float* v_scale, const int* table, const int* lens,
                               const int* n_new, const int* granted, const void* q, void* q_out,
                               const unsigned long long* turns, int rot, int interleaved,
                               float amplitude, int B, int Hq, int Hkv, int T, int D, int page,
                               int n_pages, int max_pages, const long long* strides, int dtype,
                               void* stream) {
    if (!k || !v || !k_pages || !v_pages || !k_scale || !v_scale || !table || !lens || !strides ||
        (q == nullptr) != (q_out == nullptr))
        return ATTN_ERR_INVALID;
    int rc = check_cache(B, Hkv, D, page, n_pages, max_pages);
    if (rc != ATTN_OK) return rc;
    if (T <= 0 || (q && Hq <= 0) || (dtype != ATTN_F16 && dtype != ATTN_BF16)) return ATTN_ERR_INVALID;
    if ((rc = check_rope(D, rot, interleaved, amplitude, turns)) != ATTN_OK) return rc;
    for (int i = 0; i < (q ? 3 : 1); ++i)
        if ((rc = check_strides(strides + 3 * i)) != ATTN_OK) return rc;
    if (q && q == q_out && !same_strides(strides + 3, strides + 6)) return ATTN_ERR_INVALID;
    const void* ptrs[] = {k, v, k_pages, v_pages, q, q_out};
    const void* words[] = {k_scale, v_scale, table, lens, n_new, granted};
    if (!aligned(ptrs, 16) || !aligned(words, 4)) return ATTN_ERR_ALIGN;
    // positions past the last one that a sequence's pages could take are 32-bit, too
    if (static_cast<int64_t>(T) + static_cast<int64_t>(max_pages) * page + 2 * page > 0x7fffffffll)
        return ATTN_ERR_UNSUPPORTED;
    const int64_t slots = (static_cast<int64_t>(T) + page - 2) / page + 1;
    if (slots * B * Hkv * 2 > 0x7fffffffll) return ATTN_ERR_UNSUPPORTED;
    // the queries' CTAs come on top, fewer than one per 16 of their rows
    if (q && (static_cast<int64_t>(B) * T > 1 << 27 || Hq > 65535 ||
              slots * B * Hkv * 2 + static_cast<int64_t>(B) * T * Hq / 16 + 1 > 0x7fffffffll))
        return ATTN_ERR_UNSUPPORTED;
    AppendRopeParams p{};
    if ((rc = device_setup_public(&p.status)) != ATTN_OK) return rc;
    p.f = {turns, rot, rope_mode(rot, interleaved), amplitude, 1.0f};
    p.src[0] = static_cast<const uint16_t*>(k);
    p.src[1] = static_cast<const uint16_t*>(v);
    p.pages[0] = static_cast<uint8_t*>(k_pages);
    p.pages[1] = static_cast<uint8_t*>(v_pages);
    p.scales[0] = k_scale;
    p.scales[1] = v_scale;
    p.q = static_cast<const uint16_t*>(q);
    p.q_out = static_cast<uint16_t*>(q_out);
    p.table = table;
    p.lens = lens;
    p.n_new = n_new;
    p.granted = granted;
    p.sb = strides[0], p.sh = strides[1], p.st = strides[2];
    if (q) {
        p.qb = strides[3], p.qh = strides[4], p.qt = strides[5];
        p.ob = strides[6], p.oh = strides[7], p.ot = strides[8];
    }
    p.B = B;
    p.Hq = q ? Hq : 0;
    p.Hkv = Hkv;
    p.T = T;
    p.n_pages = n_pages;
    p.max_pages = max_pages;
    p.n_slots = static_cast<int>(slots);
    p.page_shift = page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7;
    const bool bf16 = dtype == ATTN_BF16;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaErrorInvalidValue;
    if (T <= (D == 64 ? step_tokens<64>() : step_tokens<128>())) {
        e = D == 64 ? (bf16 ? launch_step<64, true>(p, st) : launch_step<64, false>(p, st))
                    : (bf16 ? launch_step<128, true>(p, st) : launch_step<128, false>(p, st));
        return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
    }
    e = D == 64 ? (bf16 ? launch_prompt<64, true>(p, st) : launch_prompt<64, false>(p, st))
                : (bf16 ? launch_prompt<128, true>(p, st) : launch_prompt<128, false>(p, st));
    if (e == cudaSuccess && q) {   // a kernel of their own, that starts in the pages' tail
        RopeParams r{};
        r.f = p.f;
        for (int w = 0; w < 2; ++w) {
            r.x[w] = p.q;
            r.y[w] = p.q_out;
            r.xs[w][0] = p.qb, r.xs[w][1] = p.qh, r.xs[w][2] = p.qt;
            r.ys[w][0] = p.ob, r.ys[w][1] = p.oh, r.ys[w][2] = p.ot;
        }
        r.lens = lens;
        r.n_new = n_new;
        r.granted = granted;
        r.most = max_pages << p.page_shift;
        r.B = B;
        r.N = T;
        r.Hq = r.heads = Hq;
        e = launch_rope(r, D, bf16, st);
    }
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}
