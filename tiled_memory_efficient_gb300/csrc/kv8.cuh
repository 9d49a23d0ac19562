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

}  // namespace
}  // namespace tme
