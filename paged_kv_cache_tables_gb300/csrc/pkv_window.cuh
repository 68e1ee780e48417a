// What a window and the first tokens let a decode's query see of its context, and
// a prefill unit's rows of theirs; stores of a unit's rows.
#pragma once

#include <stdint.h>

#include "pkv_device.cuh"

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

// One unit of work, as the scheduler publishes it (tiles == 0: no more).
// Positions count along the list of pages.
struct WpUnit {
    int tiles;        // key tiles walked
    int h, row0;      // KV head; first row of q / out
    int tokens;       // rows of the unit (tile A first)
    int first;        // position of the first row
    int ctx;          // end of the context
    int wpos;         // first position of the first row's window
    int pad;
};

// Rows [a0, a1) and [b0, b1) of the key tile at key0 that no row of the unit
// sees, in pages that are read: past the context, and between the first tokens
// and the window.
struct WpHidden {
    int a0, a1, b0, b1;
    __device__ __forceinline__ WpHidden(const WpUnit &u, int key0, int sinks, int keys)
        : a0(max(u.ctx - key0, 0)), a1(min(keys, ((u.ctx + 15) & ~15) - key0)), b0(max(sinks - key0, 0)),
          b1(min(u.wpos - key0, keys)) {}
    __device__ __forceinline__ bool any() const { return a0 < a1 || b0 < b1; }
    __device__ __forceinline__ bool has(int r) const { return (r >= a0 && r < a1) || (r >= b0 && r < b1); }
};

// 128 bytes of a warp's rows from shared memory to the output, asynchronously.
__device__ __forceinline__ void store_rows(const CUtensorMap *map, const void *src, int column, int head, int token) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(column), "r"(head), "r"(token), "r"(smem_addr(src))
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// Until what this thread's stores read may be overwritten.
__device__ __forceinline__ void stores_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

// Until this thread's stores are complete.
__device__ __forceinline__ void stores_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

}  // namespace pkv
