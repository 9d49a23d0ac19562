// rope.cu -- rotary positions: queries and keys (include/rope.h), and the append to
// the paged 8-bit cache that turns its keys on the way.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/rope.h"
#include "attn_internal.h"
#include "kv8.cuh"
#include "rope.cuh"

namespace tme {
namespace {

// ------------------------------------------------------------------ queries and keys

struct RopeParams {
    RopeView f;
    const uint16_t* x[2];   // q, k
    uint16_t* y[2];
    int64_t xs[2][3], ys[2][3];   // batch, head, row strides
    const int* pos;
    int64_t pos_b, pos_n;
    int start, B, N, Hq, heads;
    int item_shift, chunk;        // 16-dimension items of a row; heads a thread takes
    int total;                    // threads of a block row that have work
};

constexpr int kRopeThreads = 256;

// A thread takes 16 dimensions of one token and `chunk` heads, so that one set of
// sines serves them all; neighbouring threads take neighbouring items of a token.
template <bool BF16, int MODE>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
    const int id = static_cast<int>(blockIdx.x) * kRopeThreads + static_cast<int>(threadIdx.x);
    if (id >= p.total) return;
    const int items = 1 << p.item_shift, item = id & (items - 1), tok = id >> p.item_shift;
    const int b = tok / p.N, n = tok - b * p.N;
    const int h0 = static_cast<int>(blockIdx.y) * p.chunk;
    RopeRows t;
    t.x0 = p.x[0] + b * p.xs[0][0] + n * p.xs[0][2];
    t.x1 = p.x[1] + b * p.xs[1][0] + n * p.xs[1][2];
    t.y0 = p.y[0] + b * p.ys[0][0] + n * p.ys[0][2];
    t.y1 = p.y[1] + b * p.ys[1][0] + n * p.ys[1][2];
    t.xh0 = p.xs[0][1], t.xh1 = p.xs[1][1], t.yh0 = p.ys[0][1], t.yh1 = p.ys[1][1];
    t.first = p.Hq;
    const int pos = p.pos ? p.pos[b * p.pos_b + n * p.pos_n] : p.start + n;
    rope_item<BF16, MODE>(p.f, t, item, items, pos, h0, min(h0 + p.chunk, p.heads), true);
}

template <bool BF16>
cudaError_t launch_rope(const RopeParams& p, cudaStream_t stream) {
    const dim3 grid((p.total + kRopeThreads - 1) / kRopeThreads, (p.heads + p.chunk - 1) / p.chunk);
    const dim3 block(kRopeThreads);
    switch (p.f.mode) {
        case kRopeHalf: return launch_kernel(rope_kernel<BF16, kRopeHalf>, grid, block, 0, stream, p);
        case kRopeInter: return launch_kernel(rope_kernel<BF16, kRopeInter>, grid, block, 0, stream, p);
        default: return launch_kernel(rope_kernel<BF16, kRopeScalar>, grid, block, 0, stream, p);
    }
}

// Heads a thread takes of `heads`, given the threads that one head needs: as many as leave
// the device its threads, at least two.
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
    int B, Hq, Hkv, T, n_pages, max_pages, n_slots;
    int page_ctas;    // CTAs of pages; the others turn queries
    int q_threads;    // threads that one head's queries need
    int q_chunk;      // heads a thread of those takes
};

// New tokens of sequence b (-1: a count that does not fit; 0 without room).
template <int PAGE>
__device__ __forceinline__ int tokens_of(const AppendRopeParams& p, int b, int len) {
    if (p.granted && *p.granted == 0) return 0;
    const int n = p.n_new ? p.n_new[b] : p.T;
    if (n == 0) return 0;
    return n < 0 || n > p.T || n > len || (len - 1) / PAGE >= p.max_pages ? -1 : n;
}

template <int D, int PAGE>
struct AppendRopeCfg {
    static constexpr int kThreads = PAGE * D / 8 < 256 ? PAGE * D / 8 : 256;
    static constexpr int NV = PAGE * D / 8 / kThreads;   // 16-byte vectors a thread holds
    static constexpr int VPT = D / 8;                    // vectors per token
    static constexpr int STEP = kThreads / VPT;          // tokens between a thread's vectors
};

// One CTA per (sequence, page it may touch, KV head, keys or values) as in the plain
// append: the page's new tokens in registers (fp32, since turned keys are rounded
// once), their largest magnitude gives the scale, then the e4m3 bytes.  A thread's vectors are
// STEP tokens apart: it makes the sines of its first one and of STEP positions, and turns from
// one to the next by these (4 multiply-adds a pair; at most 7 steps, each off by 2^-23).  A pair's other
// half comes from another lane of the token.
template <int D, int PAGE, bool BF16>
__global__ void __launch_bounds__(AppendRopeCfg<D, PAGE>::kThreads)
    kv8_append_rope_kernel(const __grid_constant__ AppendRopeParams p) {
    using C = AppendRopeCfg<D, PAGE>;
    constexpr int NV = C::NV, VPT = C::VPT, STEP = C::STEP;
    asm volatile("griddepcontrol.launch_dependents;");   // the attention may set up meanwhile
    if (static_cast<int>(blockIdx.x) >= p.page_ctas) {
        // queries
        constexpr int items = D / 16;
        const int64_t id = static_cast<int64_t>(blockIdx.x - p.page_ctas) * C::kThreads + threadIdx.x;
        const int part = static_cast<int>(id / p.q_threads);
        if (part * p.q_chunk >= p.Hq) return;
        const int item = static_cast<int>(id) & (items - 1);   // (q_threads is a multiple of items)
        const int tok = static_cast<int>(id - static_cast<int64_t>(part) * p.q_threads) / items;
        const int h0 = part * p.q_chunk, h1 = min(h0 + p.q_chunk, p.Hq);
        const int b = tok / p.T, t = tok - b * p.T;
        const int len = p.lens[b], n = tokens_of<PAGE>(p, b, len);
        RopeRows r;
        r.x0 = r.x1 = p.q + b * p.qb + t * p.qt;
        r.y0 = r.y1 = p.q_out + b * p.ob + t * p.ot;
        r.xh0 = r.xh1 = p.qh;
        r.yh0 = r.yh1 = p.oh;
        r.first = p.Hq;
        const bool live = t < n;
        if (p.f.mode == kRopeHalf) rope_item<BF16, kRopeHalf>(p.f, r, item, items, len - n + t, h0, h1, live);
        else if (p.f.mode == kRopeInter) rope_item<BF16, kRopeInter>(p.f, r, item, items, len - n + t, h0, h1, live);
        else rope_item<BF16, kRopeScalar>(p.f, r, item, items, len - n + t, h0, h1, live);
        return;
    }
    int id = static_cast<int>(blockIdx.x);
    const int which = id & 1;
    id >>= 1;
    const int h = id % p.Hkv;
    id /= p.Hkv;
    const int slot = id % p.n_slots;
    const int b = id / p.n_slots;
    const int len = p.lens[b];
    const int n = tokens_of<PAGE>(p, b, len);
    if (n == 0) return;
    if (n < 0) {
        if (threadIdx.x == 0) atomicOr(p.status, kStatusPage);
        return;
    }
    const int start = len - n;
    const int pj = start / PAGE + slot;
    const int t0 = pj * PAGE;
    if (t0 >= len) return;
    const int pid = p.table[static_cast<int64_t>(b) * p.max_pages + pj];
    const int pos0 = t0 + static_cast<int>(threadIdx.x) / VPT;   // position of the first vector
    const int d0 = static_cast<int>(threadIdx.x) % VPT * 8;
    const uint16_t* row = p.src[which] + b * p.sb + h * p.sh;
    uint4 w[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int pos = pos0 + i * STEP;
        w[i] = make_uint4(0u, 0u, 0u, 0u);
        if (pos >= start && pos < len)
            w[i] = __ldcs(reinterpret_cast<const uint4*>(row + (pos - start) * p.st + d0));
    }
    if (pid < 0 || pid >= p.n_pages) {
        if (threadIdx.x == 0) atomicOr(p.status, kStatusPage);
        return;
    }
    float y[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 e = rope_unpack<BF16>(x[j]);
            y[i][2 * j] = e.x;
            y[i][2 * j + 1] = e.y;
        }
    }
    if (which == 0) {
        const int half = p.f.rot >> 1, mode = p.f.mode;
        // this vector's dimensions: which turn (bits), their pairs' cosines and the
        // sines that the other half of the pair takes, now and over STEP positions
        const int turn = d0 >= p.f.rot ? 0 : (p.f.rot - d0 >= 8 ? 0xff : (1 << (p.f.rot - d0)) - 1);
        float c[8], s[8], cd[8], sd[8];
        const int first = start > pos0 ? (start - pos0 + STEP - 1) / STEP : 0;   // first new vector
        const int pos1 = pos0 + first * STEP, end = min(len, t0 + PAGE);
        if (turn != 0 && pos1 < end) {
            const bool more = pos1 + STEP < end;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int d = d0 + j;
                if (mode == kRopeInter && (j & 1)) {   // the same pair's other half
                    c[j] = c[j - 1], s[j] = -s[j - 1];
                    cd[j] = cd[j - 1], sd[j] = -sd[j - 1];
                    continue;
                }
                c[j] = cd[j] = 1.0f;
                s[j] = sd[j] = 0.0f;
                if (d >= p.f.rot) continue;
                const bool low = mode == kRopeInter || d < half;
                const int i = mode == kRopeInter ? d >> 1 : low ? d : d - half;
                const float2 cs = rope_cs(p.f.turns, i, pos1, p.f.amp);
                c[j] = cs.x, s[j] = low ? -cs.y : cs.y;
                if (more) {
                    const float2 dd = rope_cs(p.f.turns, i, STEP, 1.0f);
                    cd[j] = dd.x, sd[j] = low ? -dd.y : dd.y;
                }
            }
        }
        const int away = mode == kRopeHalf && d0 < p.f.rot ? (d0 < half ? half / 8 : -(half / 8)) : 0;
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int pos = pos0 + i * STEP;
            const bool fresh = pos >= start && pos < len;
            float o[8];   // the pairs' other halves
            if (mode == kRopeHalf) {   // (every lane takes part)
                const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 e = rope_unpack<BF16>(__shfl_sync(0xffffffffu, x[j], lane + away));
                    o[2 * j] = e.x;
                    o[2 * j + 1] = e.y;
                }
            } else if (mode == kRopeInter) {
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = y[i][j ^ 1];
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int d = d0 + j;
                    o[j] = fresh && d < p.f.rot
                               ? rope_load<BF16>(row + (pos - start) * p.st + (d < half ? d + half : d - half))
                               : 0.0f;
                }
            }
            if (!fresh || turn == 0) continue;
            float r[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) r[j] = fmaf(o[j], s[j], y[i][j] * c[j]);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if ((turn >> j) & 1) y[i][j] = r[j];
            if (i + 1 < NV) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float cn = fmaf(-s[j], sd[j], c[j] * cd[j]);
                    s[j] = fmaf(s[j], cd[j], c[j] * sd[j]);
                    c[j] = cn;
                }
            }
        }
    }
    uint8_t* dst = p.pages[which] + (static_cast<int64_t>(pid) * p.Hkv + h) * (PAGE * D) + threadIdx.x * 8;
    float* scale = p.scales[which] + static_cast<int64_t>(pid) * p.Hkv + h;
    const float s_old = t0 < start ? *scale : 0.0f;
    // largest finite magnitude: positive floats order like their bits
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float a = fabsf(y[i][j]);
            top = fmaxf(top, a < INFINITY ? a : 0.0f);   // false for a NaN, too
        }
    uint32_t u = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
    __shared__ uint32_t s_max[C::kThreads / 32];
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = u;
    __syncthreads();   // also: every thread has read the old scale
#pragma unroll
    for (int i = 0; i < C::kThreads / 32; ++i) u = max(u, s_max[i]);
    int e = amax_exp(__uint_as_float(u));
    const int e_old = t0 < start ? scale_exp(s_old) : e;
    e = max(e, e_old);
    if (threadIdx.x == 0) *scale = exp2i(e);
    const float inv = exp2i(-e);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int pos = pos0 + i * STEP;
        if (pos >= start && pos < len) {
            uint32_t r[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) r[j] = f32_to_e4m3x2(y[i][2 * j] * inv, y[i][2 * j + 1] * inv);
            *reinterpret_cast<uint2*>(dst + i * (C::kThreads * 8)) =
                make_uint2(r[0] | (r[1] << 16), r[2] | (r[3] << 16));
        }
    }
    if (e != e_old) raise_tokens<C::kThreads * 8, STEP>(dst, pos0, min(start, t0 + PAGE), e_old, e);
}

template <int D, int PAGE>
cudaError_t launch_append_rope(bool bf16, AppendRopeParams p, cudaStream_t stream) {
    using C = AppendRopeCfg<D, PAGE>;
    int64_t ctas = static_cast<int64_t>(p.B) * p.n_slots * p.Hkv * 2;
    p.page_ctas = static_cast<int>(ctas);
    if (p.q) {
        p.q_threads = p.B * p.T * (D / 16);
        p.q_chunk = heads_per_thread(p.q_threads, p.Hq);
        const int64_t parts = (p.Hq + p.q_chunk - 1) / p.q_chunk;
        ctas += (parts * p.q_threads + C::kThreads - 1) / C::kThreads;
    }
    if (ctas > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    const dim3 grid(static_cast<unsigned>(ctas)), block(C::kThreads);
    return bf16 ? launch_kernel(kv8_append_rope_kernel<D, PAGE, true>, grid, block, 0, stream, p)
                : launch_kernel(kv8_append_rope_kernel<D, PAGE, false>, grid, block, 0, stream, p);
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
    p.item_shift = D == 128 ? 3 : 2;
    p.total = (B * N) << p.item_shift;
    p.chunk = heads_per_thread(p.total, p.heads);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == ATTN_BF16 ? launch_rope<true>(p, st) : launch_rope<false>(p, st);
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
    const bool bf16 = dtype == ATTN_BF16;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaErrorInvalidValue;
#define TME_APPEND(d, pg) \
    if (D == d && page == pg) e = launch_append_rope<d, pg>(bf16, p, st);
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
