// The part of a context that a decode's query sees through a window and the
// first tokens.
#pragma once

#include <stdint.h>

namespace pkv {

// The blocks of a context that hold a position its last token sees.
struct Visible {
    int ctx, w0;            // clamped context; the window's first position
    int sink_blocks, skip;  // entry v of the list is logical block v, or v + skip from sink_blocks on
    int count;
    bool bad;
    // p: max_blocks, window, sinks
    template <typename P>
    __device__ __forceinline__ Visible(const P &p, int context) {
        bad = context < 0 || context > p.max_blocks * 16;
        ctx = min(max(context, 0), p.max_blocks * 16);
        const int nblk = (ctx + 15) >> 4;
        w0 = max(ctx - p.window, 0);
        sink_blocks = min((p.sinks + 15) >> 4, nblk);
        skip = max((w0 >> 4) - sink_blocks, 0);
        count = nblk - skip;
    }
    __device__ __forceinline__ int logical(int v) const { return v < sink_blocks ? v : v + skip; }
    // the visible positions of logical block j, one bit each (never none):
    // before ctx, and in the window or among the first tokens
    __device__ __forceinline__ uint32_t bits(int j, int sinks) const {
        const int t0 = j * 16;
        const int lim = min(ctx - t0, 16), first = min(max(w0 - t0, 0), 16), sk = min(max(sinks - t0, 0), 16);
        return ((1u << lim) - 1u) & ((0xffffu << first) | ((1u << sk) - 1u)) & 0xffffu;
    }
};

}  // namespace pkv
