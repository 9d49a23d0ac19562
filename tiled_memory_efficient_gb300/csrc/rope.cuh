// rope.cuh -- rotary positions on the device, shared by rope.cu's kernels.
//
// Pair i of a row at position p turns by p * f_i radians.  The frequencies come as
// fractions of a turn in 64-bit fixed point, turns[i] = f_i / (2 pi) * 2^64 mod 2^64:
// p * turns[i] mod 2^64 is then the angle in turns, exact in integers however far the
// position (in fp32 an angle of 10^5 radians is off by 0.004).  Its upper 32 bits, as a
// signed fraction of half a turn, go through sincospif, whose argument needs no further
// reduction: cosine and sine are right to about 2^-23.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace tme {
namespace {

// How a head's row is paired, and how the kernels reach a pair's two halves.
constexpr int kRopeHalf = 0;     // (d, d + rot / 2), rot a multiple of 16: whole 16-byte vectors
constexpr int kRopeInter = 1;    // (2 i, 2 i + 1)
constexpr int kRopeScalar = 2;   // (d, d + rot / 2), any even rot: element by element

inline int rope_mode(int rot, int interleaved) {
    return interleaved ? kRopeInter : rot % 16 == 0 ? kRopeHalf : kRopeScalar;
}

// What every rotation needs.
struct RopeView {
    const unsigned long long* turns;   // [rot / 2]
    int rot, mode;
    float amp;    // of cosine and sine
    float sign;   // -1: the transposed rotation
};

// (cosine, sine) * scale of an angle, a 64-bit fraction of a turn.
__device__ __forceinline__ float2 rope_cs(unsigned long long phase, float amp) {
    const int top = static_cast<int>(static_cast<uint32_t>((phase + 0x80000000ull) >> 32));
    float s, c;
    sincospif(static_cast<float>(top) * 0x1p-31f, &s, &c);
    return make_float2(c * amp, s * amp);
}
// The angle of frequency `turn` at position pos, and what pair i turns by there.
__device__ __forceinline__ unsigned long long rope_phase(unsigned long long turn, int pos) {
    return static_cast<unsigned long long>(static_cast<long long>(pos)) * turn;
}
__device__ __forceinline__ float2 rope_cs(const unsigned long long* turns, int i, int pos, float amp) {
    return rope_cs(rope_phase(__ldg(turns + i), pos), amp);
}

template <bool BF16>
__device__ __forceinline__ float2 rope_unpack(uint32_t w) {
    if constexpr (BF16) {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    } else {
        float a, b;
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\t"
            "cvt.f32.f16 %1, hi;\n\t}"
            : "=f"(a), "=f"(b)
            : "r"(w));
        return make_float2(a, b);
    }
}
template <bool BF16>
__device__ __forceinline__ float rope_load(const uint16_t* x) {
    return rope_unpack<BF16>(static_cast<uint32_t>(*x)).x;
}
template <bool BF16>
__device__ __forceinline__ uint16_t rope_round(float x) {
    return static_cast<uint16_t>(pack2<BF16>(x, 0.0f));
}

// The rows of one token: heads [0, first) of one tensor, the others of a second one.
struct RopeRows {
    const uint16_t *x0, *x1;   // the token's row of head 0
    uint16_t *y0, *y1;
    int64_t xh0, xh1, yh0, yh1;   // elements between heads
    int first;
    __device__ __forceinline__ const uint16_t* in(int h) const {
        return h < first ? x0 + h * xh0 : x1 + (h - first) * xh1;
    }
    __device__ __forceinline__ uint16_t* out(int h) const {
        return h < first ? y0 + h * yh0 : y1 + (h - first) * yh1;
    }
};

constexpr int kRopeBatch = 4;   // heads in flight a thread

// Pair p of 8 of item `item`: MODE 0 and 1 hold neighbours, MODE 2 every items-th.
template <int MODE>
__device__ __forceinline__ int item_pair(int item, int items, int p) {
    return MODE == kRopeScalar ? item + p * items : 8 * item + p;
}

// The sines of an item's 8 pairs, made where they are used.
template <int MODE>
__device__ __forceinline__ void item_sines(const RopeView& f, int item, int items, int pos, float (&c)[8], float (&s)[8]) {
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        c[p] = 1.0f, s[p] = 0.0f;
        const int pair = item_pair<MODE>(item, items, p);
        if (2 * pair < f.rot) {
            const float2 cs = rope_cs(f.turns, pair, pos, f.amp);
            c[p] = cs.x, s[p] = cs.y * f.sign;
        }
    }
}

// 16 of the D dimensions of one token's heads h0, h0 + step, ... below h1, with the sines that
// sines(c, s) gives, called once by every thread while the first heads are on their way.  `live`
// false: they become zeros.  What a rotation in place leaves alone is not touched.
template <bool BF16, int MODE, typename Sines>
__device__ __forceinline__ void rope_item(const RopeView& f, const RopeRows& t, int item, int items, int h0,
                                          int step, int h1, bool live, Sines sines) {
    const int half = f.rot >> 1;
    float c[8], s[8];
    if constexpr (MODE == kRopeScalar) {
        sines(c, s);
        for (int h = h0; h < h1; h += step) {
            const uint16_t* x = t.in(h);
            uint16_t* y = t.out(h);
            float a[8], b[8];
#pragma unroll
            for (int p = 0; p < 8; ++p) {   // (pairs past the rotated ones: two dimensions that stay)
                const int i = item_pair<MODE>(item, items, p), d0 = i < half ? i : 2 * i, d1 = i < half ? i + half : 2 * i + 1;
                a[p] = live ? rope_load<BF16>(x + d0) : 0.0f;
                b[p] = live ? rope_load<BF16>(x + d1) : 0.0f;
            }
#pragma unroll
            for (int p = 0; p < 8; ++p) {
                const int i = item_pair<MODE>(item, items, p), d0 = i < half ? i : 2 * i, d1 = i < half ? i + half : 2 * i + 1;
                const bool turn = live && i < half;
                if (!turn && live && x == y) continue;
                y[d0] = rope_round<BF16>(turn ? a[p] * c[p] - b[p] * s[p] : a[p]);
                y[d1] = rope_round<BF16>(turn ? b[p] * c[p] + a[p] * s[p] : b[p]);
            }
        }
    } else {
        // the item's two vectors, and whether they turn as halves of pairs
        const bool turns = MODE == kRopeInter ? 16 * item < f.rot : 8 * item < half;
        const int d0 = MODE == kRopeInter ? 16 * item : turns ? 8 * item : f.rot + 16 * (item - (f.rot >> 4));
        const int d1 = MODE == kRopeInter ? d0 + 8 : turns ? d0 + half : d0 + 8;
        uint4 va[kRopeBatch], vb[kRopeBatch];
        auto load = [&](int h) {
#pragma unroll
            for (int u = 0; u < kRopeBatch; ++u) {
                va[u] = vb[u] = make_uint4(0u, 0u, 0u, 0u);
                if (h + u * step < h1 && live) {
                    const uint16_t* x = t.in(h + u * step);
                    va[u] = *reinterpret_cast<const uint4*>(x + d0);
                    vb[u] = *reinterpret_cast<const uint4*>(x + d1);
                }
            }
        };
        load(h0);
        sines(c, s);
        for (int h = h0; h < h1; h += kRopeBatch * step) {
            if (h != h0) load(h);
#pragma unroll
            for (int u = 0; u < kRopeBatch; ++u) {
                if (h + u * step >= h1) continue;
                uint16_t* y = t.out(h + u * step);
                uint32_t a[4] = {va[u].x, va[u].y, va[u].z, va[u].w};
                uint32_t b[4] = {vb[u].x, vb[u].y, vb[u].z, vb[u].w};
                if (live && turns) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 e = rope_unpack<BF16>(a[j]), o = rope_unpack<BF16>(b[j]);
                        if constexpr (MODE == kRopeHalf) {
                            a[j] = pack2<BF16>(e.x * c[2 * j] - o.x * s[2 * j], e.y * c[2 * j + 1] - o.y * s[2 * j + 1]);
                            b[j] = pack2<BF16>(o.x * c[2 * j] + e.x * s[2 * j], o.y * c[2 * j + 1] + e.y * s[2 * j + 1]);
                        } else {   // word j is pair j of the item, word j of the second vector pair 4 + j
                            if (8 * item + j < half) a[j] = pack2<BF16>(e.x * c[j] - e.y * s[j], e.y * c[j] + e.x * s[j]);
                            if (8 * item + 4 + j < half)
                                b[j] = pack2<BF16>(o.x * c[4 + j] - o.y * s[4 + j], o.y * c[4 + j] + o.x * s[4 + j]);
                        }
                    }
                } else if (live && y == t.in(h + u * step)) {
                    continue;   // in place, and nothing turns
                }
                *reinterpret_cast<uint4*>(y + d0) = make_uint4(a[0], a[1], a[2], a[3]);
                *reinterpret_cast<uint4*>(y + d1) = make_uint4(b[0], b[1], b[2], b[3]);
            }
        }
    }
}

}  // namespace
}  // namespace tme
