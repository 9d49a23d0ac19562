// window.cuh -- the visible set of sliding-window attention with sinks, shared by
// the forward and backward kernels.
//
// The query at key position p sees the keys j <= p with j > p - window or j <
// sinks.  A Q tile whose first row stands at position min_pos meets its sink
// tiles [0, n_sink) and then one run of 128-key tiles that starts `skip` tiles
// later; entry v of that list is key tile v (v < n_sink) or v + skip.  The tiles
// between them are never loaded, so a tile of R rows costs at most (window + R)
// / 128 + 2 key tiles and its sink tiles whatever the sequence length.
#pragma once

#include <cstdint>

namespace tme {

struct KeyList {
    int n_sink = 0, skip = 0;
    __device__ __forceinline__ int tile(int v) const { return v < n_sink ? v : v + skip; }
};

__device__ __forceinline__ KeyList key_list(int64_t min_pos, int window, int sinks) {
    KeyList kl;
    const int64_t lo = min_pos - window + 1;   // first key inside a window
    const int lo_tile = lo > 0 ? static_cast<int>(static_cast<uint64_t>(lo) >> 7) : 0;
    kl.n_sink = min((sinks + 127) / 128, lo_tile);
    kl.skip = lo_tile - kl.n_sink;
    return kl;
}

// Do queries at positions [min_pos, max_pos] need a per-key mask on keys [key0,
// last]?  Not when the first of them sees up to `last` and the last of them
// sees key0 through its window (or all those keys are sinks).
__device__ __forceinline__ bool window_edge(int key0, int last, int min_pos, int max_pos,
                                            int window, int sinks) {
    return last > min_pos || (key0 <= max_pos - window && last >= sinks);
}

// Bits [0, n) of 32.
__device__ __forceinline__ uint32_t bits_below(int n) {
    return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
}

}  // namespace tme
