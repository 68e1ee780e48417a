// The step's metadata on the GPU: block tables grown from a device free list,
// slot map, positions, cumulative and context lengths from the sequences'
// lengths (pkv_step_tables), and blocks returned to the list
// (pkv_release_blocks).
//
// Mathematics.  Sequence s holds len_s tokens in ceil(len_s / 16) blocks and
// gets new_s more, so it takes need_s = ceil((len_s + new_s) / 16) -
// ceil(len_s / 16) blocks.  With the exclusive prefix sums cu (of new) and bx
// (of need), block k of the step is the k-th id from the end of the free list
// and belongs to the last s with bx_s <= k; token t of the step belongs to the
// last s with cu_s <= t and sits at position len_s + t - cu_s.
//
// What bounds it: of few sequences latency, the launch, the reads of the lengths,
// the scan and the reads of ids being a chain of round trips, 2.9 us for 256
// sequences.  The step of 4,020 sequences and 127,780 rows writes 1.6 MB, 0.24 us
// at the measured copy rate, and takes 8.2 us: the launch of 16 CTAs 1.0, the scan
// of all lengths, repeated in each of them, 3.5, two rounds of bisection, ids and
// stores 3.7.
// So everything is one launch without a workspace: a small step is one CTA;
// a larger one is one cluster of CTAs, each of which scans all lengths itself
// (at most 16,384 of them, out of L2) and fills its share of the outputs, its
// token's sequence found by bisection of the scans in shared memory.  The
// cluster's barrier between the reads and the writes is what lets the outputs
// replace the inputs in place.
#include <cuda_runtime.h>

#include "pkv.h"
#include "pkv_cluster.cuh"
#include "pkv_device.cuh"
#include "pkv_host.h"

namespace pkv {

constexpr int kTabThreads = 1024;
constexpr int kTabBatch = 4;     // sequences whose lengths a thread has under way
constexpr int kTabCluster = 16;   // more than the portable 8: opted into at the first launch

struct TablesParams {
    const int32_t *seq_lens, *new_lens;
    int32_t *block_tables;
    const int32_t *free_list;
    const int32_t *free_count;
    int32_t *free_count_out;
    int32_t *context_lens, *cu_seqlens;
    int64_t *slot_mapping;
    int32_t *token_pos;
    int *dev_status;
    int S, max_blocks, free_capacity, num_blocks, max_tokens;
    bool vec;   // slot_mapping and token_pos are 16-byte aligned
};

struct Pair64 {
    int64_t a, b;
};

// A pair of sums that stay at 2^32 - 1 once they get there (adding so is
// associative): more than any count that is allowed.
struct PairSat {
    uint32_t a, b;
};

__device__ __forceinline__ uint32_t add_sat(uint32_t x, uint32_t y) { return x + y < x ? 0xffffffffu : x + y; }

// Inclusive scan over the CTA.
__device__ __forceinline__ PairSat cta_scan(PairSat v, PairSat *sh, PairSat *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    auto scan = [&](PairSat x) {
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t a = __shfl_up_sync(0xffffffffu, x.a, off), b = __shfl_up_sync(0xffffffffu, x.b, off);
            if (lane >= off) x = {add_sat(x.a, a), add_sat(x.b, b)};
        }
        return x;
    };
    v = scan(v);
    if (lane == 31) sh[warp] = v;
    __syncthreads();
    if (warp == 0) sh[lane] = scan(lane < warps ? sh[lane] : PairSat{0, 0});
    __syncthreads();
    if (warp > 0) v = {add_sat(v.a, sh[warp - 1].a), add_sat(v.b, sh[warp - 1].b)};
    *total = sh[31];
    return v;
}

// The last index s in [0, n) with prefix[s] <= x (prefix non-decreasing,
// prefix[0] = 0 <= x): with x below the total, the one entry that holds x.
__device__ __forceinline__ int last_at_most(const int *prefix, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (prefix[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// Blocks that n tokens behind l take.
__device__ __forceinline__ uint32_t blocks_needed(uint32_t l, uint32_t n) { return ((l + n + 15) >> 4) - ((l + 15) >> 4); }

__global__ void __launch_bounds__(kTabThreads, 1) step_tables_kernel(const TablesParams p) {
    extern __shared__ int tab_smem[];
    __shared__ PairSat sh_scan[32];
    __shared__ int sh_bad;
    const int S = p.S;
    int *cu = tab_smem;          // [S + 1] tokens before each sequence
    int *bx = cu + S + 1;        // [S + 1] blocks taken before each sequence
    int *len = bx + S + 1;       // [S]
    const int tid = threadIdx.x, nt = blockDim.x;
    const int rank = (int)cluster_ctarank(), ranks = (int)cluster_nctarank();
    // no early signal to the next kernel: the decode entry points read
    // context_lens, written here, before their own wait
    pdl_wait_primary();
    if (tid == 0) sh_bad = 0;
    __syncthreads();

    // ---- lengths, checked; a thread takes `per` neighbouring sequences ----
    const int per = (S + nt - 1) / nt;
    const int s_lo = min(S, tid * per), s_hi = min(S, s_lo + per);
    const int64_t limit = (int64_t)p.max_blocks * 16;
    const int count = p.free_count[0];
    int bad = 0;
    PairSat sum{0, 0};
    for (int s0 = s_lo; s0 < s_hi; s0 += kTabBatch) {
        int ls[kTabBatch], ns[kTabBatch];   // on their way together
#pragma unroll
        for (int i = 0; i < kTabBatch; ++i) {
            ls[i] = s0 + i < s_hi ? p.seq_lens[s0 + i] : 0;
            ns[i] = s0 + i < s_hi ? p.new_lens[s0 + i] : 0;
        }
#pragma unroll
        for (int i = 0; i < kTabBatch; ++i) {
            if (s0 + i >= s_hi) break;
            const int l = ls[i], n = ns[i];
            len[s0 + i] = l;
            cu[s0 + i] = n;
            if (l < 0 || (int64_t)l + max(n, 0) > limit) {
                bad |= PKV_DEV_BAD_CONTEXT;
            } else if (n < 0 || n > p.max_tokens) {
                bad |= PKV_DEV_BAD_CHUNK;
            } else {
                sum.a = add_sat(sum.a, n);
                sum.b += blocks_needed(l, n);   // (a table has at most 2^26 entries)
            }
        }
    }
    PairSat total;
    const PairSat incl = cta_scan(sum, sh_scan, &total);
    if (total.a > (uint32_t)p.max_tokens) bad |= PKV_DEV_BAD_CHUNK;
    if (count < 0 || count > p.free_capacity || total.b > (uint32_t)count) bad |= PKV_DEV_FREE_LIST;
    if (bad) atomicOr(&sh_bad, bad);
    {
        // (of use only where all lengths and sums are good)
        uint32_t a = incl.a - sum.a, b = incl.b - sum.b;
        for (int s = s_lo; s < s_hi; ++s) {
            const int l = len[s], n = cu[s];
            cu[s] = (int)a;
            bx[s] = (int)b;
            a += n;
            b += blocks_needed(l, n);
        }
    }
    if (tid == 0) {
        cu[S] = (int)total.a;
        bx[S] = (int)total.b;
    }
    // every CTA has read the lengths and the count before any of them writes
    // (the outputs may be the same arrays); also this CTA's barrier for the
    // scans and the verdict
    __syncthreads();
    if (ranks > 1) cluster_sync();
    const bool fail = sh_bad != 0;
    if (fail && rank == 0 && tid == 0) set_status(p.dev_status, sh_bad);

    // ---- per-sequence outputs ----
    // warps in turn over the CTAs, so that few rows are spread over all of them
    // (4,000 rows: 6.9 us; CTA after CTA 9.3 us)
    const int gt = ((tid >> 5) * ranks + rank) * 32 + (tid & 31), gn = ranks * nt;
    for (int s = gt; s <= S; s += gn) {
        p.cu_seqlens[s] = fail ? 0 : cu[s];
        if (s < S) p.context_lens[s] = fail ? len[s] : len[s] + (cu[s + 1] - cu[s]);
    }
    if (gt == 0) p.free_count_out[0] = fail ? count : count - bx[S];

    // ---- the blocks taken (a thread's first id is on its way while the tokens
    // are laid out) ----
    const int taken = fail ? 0 : bx[S], tokens = fail ? 0 : cu[S];
    const int32_t *top = p.free_list + count - 1;   // the k-th block taken is top[-k]
    const int32_t first_id = gt < taken ? top[-gt] : 0;
    int status = 0;

    // ---- slots and positions: a row's block is the sequence's open block (in
    // its table) or one of those taken now ----
    auto entry = [&](int s, int t, int32_t &pos) {   // of row t of sequence s
        pos = len[s] + (t - cu[s]);
        const int j = pos >> 4, old = (len[s] + 15) >> 4;
        return j < old ? p.block_tables + (int64_t)s * p.max_blocks + j : top - (bx[s] + j - old);
    };
    auto slot_of = [&](int32_t id, int32_t pos) {
        if (id >= 0 && id < p.num_blocks) return (int64_t)id * 16 + (pos & 15);
        status |= PKV_DEV_BAD_BLOCK_ID;
        return (int64_t)-1;
    };
    if (p.max_tokens <= gn) {
        // a row a thread: no walk from one row to the next (256 rows: 2.9 us instead
        // of 3.4 in fours)
        if (gt < p.max_tokens) {
            int64_t slot = -1;
            int32_t pos = 0;
            if (gt < tokens) {
                const int32_t id = *entry(last_at_most(cu, S, gt), gt, pos);
                slot = slot_of(id, pos);
            }
            p.slot_mapping[gt] = slot;
            p.token_pos[gt] = pos;
        }
    } else {
        // four rows a thread
        for (int64_t t0 = (int64_t)gt * 4; t0 < p.max_tokens; t0 += (int64_t)gn * 4) {
            int64_t slot[4];
            int32_t pos[4], id[4];
            int s = t0 < tokens ? last_at_most(cu, S, (int)t0) : 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                id[e] = -1;
                pos[e] = 0;
                if (t0 + e < tokens) {
                    const int t = (int)t0 + e;
                    while (cu[s + 1] <= t) ++s;   // skips sequences without new tokens
                    id[e] = *entry(s, t, pos[e]);
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) slot[e] = t0 + e < tokens ? slot_of(id[e], pos[e]) : -1;
            if (p.vec && t0 + 4 <= p.max_tokens) {
                reinterpret_cast<longlong2 *>(p.slot_mapping + t0)[0] = make_longlong2(slot[0], slot[1]);
                reinterpret_cast<longlong2 *>(p.slot_mapping + t0)[1] = make_longlong2(slot[2], slot[3]);
                *reinterpret_cast<int4 *>(p.token_pos + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (t0 + e < p.max_tokens) {
                        p.slot_mapping[t0 + e] = slot[e];
                        p.token_pos[t0 + e] = pos[e];
                    }
            }
        }
    }
    for (int k = gt; k < taken; k += gn) {
        const int s = last_at_most(bx, S, k);
        const int32_t id = k == gt ? first_id : top[-k];
        if (id < 0 || id >= p.num_blocks) status |= PKV_DEV_BAD_BLOCK_ID;
        p.block_tables[(int64_t)s * p.max_blocks + ((len[s] + 15) >> 4) + (k - bx[s])] = id;
    }
    if (status) set_status(p.dev_status, status);
}

// ---------------------------------------------------------------- release

struct ReleaseParams {
    int32_t *block_tables;
    const int32_t *seq_lens, *finished;
    int32_t *free_list;
    int32_t *free_count;
    int32_t *counts;     // workspace: [S] blocks each row gives back, then the list's count before the call
    int *dev_status;
    int S, max_blocks, free_capacity, num_blocks, window, sinks;
    bool vec;            // the table's rows are 16-byte aligned
};

// Table entries [lo, hi) of sequence s that the call gives back.
__device__ __forceinline__ void release_range(const ReleaseParams &p, int s, int &lo, int &hi, int &status) {
    int64_t l = __ldcg(p.seq_lens + s);
    const bool finished = p.finished != nullptr && __ldcg(p.finished + s) != 0;
    if (l < 0 || l > (int64_t)p.max_blocks * 16) {
        status |= PKV_DEV_BAD_CONTEXT;
        l = l < 0 ? 0 : (int64_t)p.max_blocks * 16;
    }
    const int nb = (int)((l + 15) >> 4);
    lo = hi = 0;
    if (finished) {
        hi = nb;
    } else if (p.window > 0) {
        // the next token sits at position l and sees positions from
        // l - window + 1 on: a block before that whole is out of the window
        const int64_t first = l - p.window + 1;
        lo = (int)(((int64_t)p.sinks + 15) >> 4);
        hi = first > 0 ? min(nb, (int)(first >> 4)) : 0;
        if (hi < lo) hi = lo;
    }
}

// A warp a row, 128 neighbouring entries a load; the blocks go on the list in the
// order of the rows and of the blocks within a row.  A running row is walked from
// its first tokens' blocks on in every call, through the entries given back before.
// Two forms.  Up to
// kRelSmallRows rows are one launch: a cluster of CTAs counts its rows' blocks,
// exchanges the CTAs' totals through distributed shared memory and moves the
// blocks.  More rows are two launches over the whole GPU: one counts into the
// workspace, the other sums the counts of the rows before its own (each CTA reads
// them all, out of L2) and moves.  4,000 rows of up to 2,048 blocks take 11.9 us
// so, and took 49 us in one cluster of 16 CTAs of 1,024 threads.  Up to 256 rows,
// in one launch and in two: 256 rows of up to 512 blocks 5.2 and 4.7 us, 64 of them
// 3.7 and 3.6, 256 of up to 2,048 8.2 and 8.6, 64 of them 6.8 and 7.5; and 2.2 us of
// host time a call instead of 4.1 (a launch, and the workspace).  Loads under way in a warp: few rows want the chain
// of a long row short, many rows want registers for more warps (256 rows of up to
// 2,048 blocks: 10.1 us with four and 11.5 with two, 4,000 of up to 333 13.4 and
// 12.3, a copy of the table and the list included).
constexpr int kRelThreads = 256;
constexpr int kRelSmallLoads = 4, kRelLoads = 2;
constexpr int kRelSmallWarps = 16;
constexpr int kRelSmallRows = kTabCluster * kRelSmallWarps;

// visit(j, ids): of the entries [lo, hi) of row s, those at j .. j + 3, of this
// lane and load, that are given back (others -1); a load of the warp is 128 neighbouring entries, and the
// loads come in order
template <int LOADS, typename F>
__device__ __forceinline__ void walk_row(const ReleaseParams &p, int s, int lo, int hi, int lane, int &status, F visit) {
    const int32_t *row = p.block_tables + (int64_t)s * p.max_blocks;
    for (int j0 = lo & ~3; j0 < hi; j0 += 128 * LOADS) {
        int4 id[LOADS];
#pragma unroll
        for (int u = 0; u < LOADS; ++u) {
            const int j = j0 + 128 * u + 4 * lane;
            id[u] = make_int4(-1, -1, -1, -1);
            if (p.vec) {
                if (j < hi) id[u] = *reinterpret_cast<const int4 *>(row + j);
            } else {
                if (j < hi) id[u].x = row[j];
                if (j + 1 < hi) id[u].y = row[j + 1];
                if (j + 2 < hi) id[u].z = row[j + 2];
                if (j + 3 < hi) id[u].w = row[j + 3];
            }
        }
#pragma unroll
        for (int u = 0; u < LOADS; ++u) {
            const int j = j0 + 128 * u + 4 * lane;
            int32_t e[4] = {id[u].x, id[u].y, id[u].z, id[u].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (j + i < lo || j + i >= hi) e[i] = -1;
                if (e[i] >= p.num_blocks) {
                    status |= PKV_DEV_BAD_BLOCK_ID;
                    e[i] = -1;
                }
            }
            visit(j, e);
        }
    }
}

// Blocks of row s given back (all lanes get the count).
template <int LOADS>
__device__ __forceinline__ int count_row(const ReleaseParams &p, int s, int &lo, int &hi, int lane) {
    int status = 0, n = 0;
    release_range(p, s, lo, hi, status);
    walk_row<LOADS>(p, s, lo, hi, lane, status, [&](int, const int32_t(&e)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) n += e[i] >= 0;
    });
    if (status) set_status(p.dev_status, status);
    return __reduce_add_sync(0xffffffffu, n);
}

// Moves row s's blocks to free_list[at..].
template <int LOADS>
__device__ __forceinline__ void move_row(const ReleaseParams &p, int s, int lo, int hi, int lane, int64_t at) {
    int ignored = 0;
    int32_t *row = p.block_tables + (int64_t)s * p.max_blocks;
    const unsigned before = (1u << lane) - 1u;
    walk_row<LOADS>(p, s, lo, hi, lane, ignored, [&](int j, const int32_t(&e)[4]) {
        int mine = 0, all = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const unsigned m = __ballot_sync(0xffffffffu, e[i] >= 0);
            mine += __popc(m & before);
            all += __popc(m);
        }
        int32_t *to = p.free_list + at + mine;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (e[i] >= 0) {
                *to++ = e[i];
                row[j + i] = -1;
            }
        at += all;
    });
}

__global__ void __launch_bounds__(kRelSmallWarps * 32) release_small_kernel(const ReleaseParams p) {
    __shared__ int sh_count[kRelSmallWarps];
    __shared__ int sh_total;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = (int)cluster_ctarank(), ranks = (int)cluster_nctarank();
    const int s = rank * kRelSmallWarps + warp;
    pdl_wait_primary();
    pdl_launch_dependents();
    const int count = p.free_count[0];
    int lo = 0, hi = 0;
    const int n = s < p.S ? count_row<kRelSmallLoads>(p, s, lo, hi, lane) : 0;
    if (lane == 0) sh_count[warp] = n;
    __syncthreads();
    int64_t at = 0, all = 0;
    int mine = 0;
#pragma unroll
    for (int w = 0; w < kRelSmallWarps; ++w) {
        if (w < warp) at += sh_count[w];
        mine += sh_count[w];   // (a table has fewer than 2^31 entries)
    }
    if (threadIdx.x == 0) sh_total = mine;
    cluster_sync();
    for (int r = 0; r < ranks; ++r) {
        const int t = ld_cluster_s32(cluster_addr(&sh_total, (uint32_t)r));
        if (r < rank) at += t;
        all += t;
    }
    // every CTA has read the totals and the count: they may change now, and a
    // CTA may leave
    cluster_sync();
    if (count < 0 || count > p.free_capacity || count + all > p.free_capacity) {
        if (rank == 0 && threadIdx.x == 0) set_status(p.dev_status, PKV_DEV_FREE_LIST);
        return;
    }
    if (rank == 0 && threadIdx.x == 0) p.free_count[0] = count + (int)all;
    if (n > 0) move_row<kRelSmallLoads>(p, s, lo, hi, lane, count + at);
}

__global__ void __launch_bounds__(kRelThreads) release_count_kernel(const ReleaseParams p) {
    const int lane = threadIdx.x & 31, s = blockIdx.x * (kRelThreads / 32) + (threadIdx.x >> 5);
    pdl_wait_primary();
    pdl_launch_dependents();
    if (blockIdx.x == 0 && threadIdx.x == 0) p.counts[p.S] = p.free_count[0];
    if (s >= p.S) return;
    int lo, hi;
    const int n = count_row<kRelLoads>(p, s, lo, hi, lane);
    if (lane == 0) p.counts[s] = n;
}

__global__ void __launch_bounds__(kRelThreads) release_move_kernel(const ReleaseParams p) {
    __shared__ Pair64 sh_sum[kRelThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int first = blockIdx.x * (kRelThreads / 32), s = first + warp;
    // the lengths do not come from the launch before, which waited for the one they
    // come from before it let this one start; they are read past the L1 cache
    int lo = 0, hi = 0, reported = 0;
    if (s < p.S) release_range(p, s, lo, hi, reported);
    pdl_wait_primary();
    pdl_launch_dependents();
    // blocks given back by the rows before this CTA's, and by all
    Pair64 sum{0, 0};
    constexpr int kBatch = 16;   // loads under way
    for (int i0 = tid; i0 < p.S; i0 += kBatch * kRelThreads) {
        int n[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int i = i0 + u * kRelThreads;
            n[u] = i < p.S ? p.counts[i] : 0;
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            sum.b += n[u];
            if (i0 + u * kRelThreads < first) sum.a += n[u];
        }
    }
    // and by this CTA's rows, one in each of its first lanes
    const int near = lane < kRelThreads / 32 && first + lane < p.S ? p.counts[first + lane] : 0;
    const int count = p.counts[p.S];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        sum.a += __shfl_xor_sync(0xffffffffu, sum.a, o);
        sum.b += __shfl_xor_sync(0xffffffffu, sum.b, o);
    }
    if (lane == 0) sh_sum[warp] = sum;
    __syncthreads();
    int64_t at = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kRelThreads / 32; ++w) {
        at += sh_sum[w].a;
        all += sh_sum[w].b;
    }
    if (count < 0 || count > p.free_capacity || count + all > p.free_capacity) {
        if (blockIdx.x == 0 && tid == 0) set_status(p.dev_status, PKV_DEV_FREE_LIST);
        return;
    }
    if (blockIdx.x == 0 && tid == 0) p.free_count[0] = count + (int)all;
    if (__shfl_sync(0xffffffffu, near, warp) == 0) return;
    at += __reduce_add_sync(0xffffffffu, lane < warp ? near : 0);
    move_row<kRelLoads>(p, s, lo, hi, lane, count + at);
}

}  // namespace pkv

extern "C" int pkv_step_tables(const int32_t *seq_lens, const int32_t *new_lens, int num_seqs, int32_t *block_tables,
                               int max_blocks_per_seq, const int32_t *free_list, int free_capacity,
                               const int32_t *free_count, int32_t *free_count_out, int num_blocks, int block_size,
                               int32_t *context_lens, int32_t *cu_seqlens, int64_t *slot_mapping, int32_t *token_pos,
                               int max_tokens, int *dev_status, void *stream) {
    pkv::NvtxRange nvtx_range("pkv_step_tables");
    using namespace pkv;
    if (num_seqs < 0 || max_blocks_per_seq <= 0 || free_capacity < 0 || num_blocks <= 0 || max_tokens < 0)
        return PKV_ERR_INVALID_ARG;
    if (block_size != 16 || num_seqs > PKV_TABLES_MAX_SEQS || max_blocks_per_seq > (1 << 26)) return PKV_ERR_UNSUPPORTED;
    if (!free_count || !free_count_out || !cu_seqlens) return PKV_ERR_INVALID_ARG;
    if (num_seqs > 0 && (!seq_lens || !new_lens || !block_tables || !context_lens)) return PKV_ERR_INVALID_ARG;
    if (max_tokens > 0 && (!slot_mapping || !token_pos)) return PKV_ERR_INVALID_ARG;
    if (free_capacity > 0 && !free_list) return PKV_ERR_INVALID_ARG;
    if (!aligned(seq_lens, 4) || !aligned(new_lens, 4) || !aligned(block_tables, 4) || !aligned(free_list, 4) ||
        !aligned(free_count, 4) || !aligned(free_count_out, 4) || !aligned(context_lens, 4) ||
        !aligned(cu_seqlens, 4) || !aligned(slot_mapping, 8) || !aligned(token_pos, 4))
        return PKV_ERR_INVALID_ARG;
    int sms = 0;
    int rc = current_sm_count(&sms);
    if (rc != PKV_OK) return rc;
    static unsigned long long attr_set = 0;
    constexpr int kMaxSmem = (3 * PKV_TABLES_MAX_SEQS + 2) * 4;
    if (!done_on_device(&attr_set)) {
        cudaError_t e = cudaFuncSetAttribute(step_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(step_tables_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return cuda_fail(e);
        mark_done_on_device(&attr_set);
    }
    TablesParams prm;
    prm.seq_lens = seq_lens;
    prm.new_lens = new_lens;
    prm.block_tables = block_tables;
    prm.free_list = free_list;
    prm.free_count = free_count;
    prm.free_count_out = free_count_out;
    prm.context_lens = context_lens;
    prm.cu_seqlens = cu_seqlens;
    prm.slot_mapping = slot_mapping;
    prm.token_pos = token_pos;
    prm.dev_status = dev_status;
    prm.S = num_seqs;
    prm.max_blocks = max_blocks_per_seq;
    prm.free_capacity = free_capacity;
    prm.num_blocks = num_blocks;
    prm.max_tokens = max_tokens;
    prm.vec = aligned(slot_mapping, 16) && aligned(token_pos, 16);
    // One CTA while it has a thread for each row, else a cluster; its scan of few
    // sequences is quicker with fewer warps (1,400 sequences: 4.1 us in CTAs of 512
    // threads, 4.5 in 1,024; 2,000 and 20 x 512 rows: 5.2 and 4.8; 16 sequences and
    // 900 rows: 3.0 us in one CTA, 2.7 in 16).
    const bool small = num_seqs <= 256 && max_tokens <= 256;
    const int threads = small ? 256 : num_seqs <= 1536 ? 512 : kTabThreads;
    cudaError_t e = launch_cluster(step_tables_kernel, small ? 1 : kTabCluster, small ? 1 : kTabCluster, threads,
                                   (size_t)(3 * num_seqs + 2) * 4, static_cast<cudaStream_t>(stream), prm);
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? PKV_OK : cuda_fail(e);
}

extern "C" size_t pkv_release_workspace_size(int num_seqs) {
    return num_seqs <= pkv::kRelSmallRows ? 0 : ((size_t)num_seqs + 1) * sizeof(int32_t);
}

extern "C" int pkv_release_blocks(int32_t *block_tables, int max_blocks_per_seq, const int32_t *seq_lens,
                                  const int32_t *finished, int num_seqs, int window, int num_sinks, int32_t *free_list,
                                  int free_capacity, int32_t *free_count, int num_blocks, int block_size,
                                  void *workspace, size_t workspace_bytes, int *dev_status, void *stream) {
    pkv::NvtxRange nvtx_range("pkv_release_blocks");
    using namespace pkv;
    if (num_seqs < 0 || max_blocks_per_seq <= 0 || free_capacity < 0 || num_blocks <= 0 || window < 0 || num_sinks < 0)
        return PKV_ERR_INVALID_ARG;
    if (block_size != 16 || num_seqs > PKV_TABLES_MAX_SEQS || max_blocks_per_seq > (1 << 26)) return PKV_ERR_UNSUPPORTED;
    if ((int64_t)num_seqs * max_blocks_per_seq >= (int64_t)1 << 31) return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PKV_OK;
    if (!block_tables || !seq_lens || !free_list || !free_count) return PKV_ERR_INVALID_ARG;
    if (!aligned(block_tables, 4) || !aligned(seq_lens, 4) || !aligned(finished, 4) || !aligned(free_list, 4) ||
        !aligned(free_count, 4))
        return PKV_ERR_INVALID_ARG;
    const bool small = num_seqs <= kRelSmallRows;
    if (!small && (!workspace || !aligned(workspace, 4) || workspace_bytes < pkv_release_workspace_size(num_seqs)))
        return PKV_ERR_WORKSPACE;
    ReleaseParams prm;
    prm.block_tables = block_tables;
    prm.seq_lens = seq_lens;
    prm.finished = finished;
    prm.free_list = free_list;
    prm.free_count = free_count;
    prm.counts = static_cast<int32_t *>(workspace);
    prm.dev_status = dev_status;
    prm.S = num_seqs;
    prm.max_blocks = max_blocks_per_seq;
    prm.free_capacity = free_capacity;
    prm.num_blocks = num_blocks;
    prm.window = window;
    prm.sinks = num_sinks;
    prm.vec = aligned(block_tables, 16) && max_blocks_per_seq % 4 == 0;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (small) {
        static unsigned long long attr_set = 0;
        if (!done_on_device(&attr_set)) {
            e = cudaFuncSetAttribute(release_small_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e != cudaSuccess) return cuda_fail(e);
            mark_done_on_device(&attr_set);
        }
        int ranks = 1;
        while (ranks * kRelSmallWarps < num_seqs) ranks *= 2;
        e = launch_cluster(release_small_kernel, ranks, ranks, kRelSmallWarps * 32, 0, st, prm);
    } else {
        const int grid = (num_seqs + kRelThreads / 32 - 1) / (kRelThreads / 32);
        e = launch_pdl(release_count_kernel, dim3(grid), dim3(kRelThreads), 0, st, prm);
        if (e == cudaSuccess) e = launch_pdl(release_move_kernel, dim3(grid), dim3(kRelThreads), 0, st, prm);
    }
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? PKV_OK : cuda_fail(e);
}
