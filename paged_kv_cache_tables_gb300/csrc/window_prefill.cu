// Prefill attention over a sliding window and the first tokens of a paged
// context, on the 5th-generation tensor cores (pkv_paged_window_prefill_attention).
//
// Mathematics.  Row i of chunk c sits at position p = ctx_c - q_len_c + i and
// sees position t iff t <= p and (t > p - window or t < sinks).  Over key tiles
// of 128 positions, with the running maximum m and sum l of the softmax in fp32:
//     P = 2^(scale2 S - m),  l = l a + sum P,  O = O a + P V,  a = 2^(m_old - m),
// where m only moves when a row's maximum grows by more than 2^8 (P and O stay
// far inside fp32's range, and O is rarely touched).
//
// What is walked.  A unit of work is 2 x 128 MMA rows (two adjacent tiles A and B
// of 128 / G tokens x the G query heads that share a KV head; or tile A alone,
// where that fills the GPU better), against the
// pages that one of its rows sees: those of the first tokens, then those from
// its first row's window on, as one list of pages (page v of the list is logical
// page v, or v + skip past the first tokens' pages) cut into key tiles of 8.
// Positions past the first tokens' pages are kept less 16 skip throughout, so
// that they count along the list.  Other pages are not read: their table
// entries may be anything.
//
// Warps (persistent; 12 of them):
//   0      TMA and scheduler: takes the CTA's units one after another (its own,
//          then those of CTAs that have not been launched yet, which it cancels:
//          clusterlaunchcontrol), publishes each unit's numbers in a ring of
//          two, loads Q and the K / V tiles, 8 pages of 16 each, a page one box
//   1, 2   issue the MMAs of query tile A, B: S = Q K^T (both operands in shared
//          memory), O += P V (P in tensor memory over S), in two parts of the
//          keys, the first while the softmax still works on the second
//   3      clears V rows that no row of the unit sees, in pages read for their
//          neighbours (they may hold anything, and 0 x NaN must not reach O)
//   4-11   softmax: a warpgroup a query tile, a row per thread
// While one tile's softmax runs, the tensor cores work on the other's products:
// the two issuers take turns, P V of a key tile and S of the next one turn.  Left
// to themselves the tiles fall into step, both softmaxes at once and then both
// products (with P rounded once, 3,500 to 3,750 cycles a key tile for the two, in
// turns 2,650 to 2,900).
// Loads, products and softmax run across the units: while a unit's outputs are
// stored, the next one's Q, K and V arrive.
//
// P goes to the tensor cores as a 16-bit value and its 16-bit rounding residual, two
// products with V: about 16 significant bits, as in the other attention kernels.  P
// rounded once would err by half a step of each weight (2^-8 sum p|v| for bf16), as
// much as the output's own rounding: against 64 bits 0.0023 relative instead of
// 0.0017, and past 2e-3 where a row sees few keys.  What it would save: 445 us
// instead of 641 below, 60 instead of 80.
// Three chunks of 3,500 to 4,100 rows x 32 heads, window 4,096, head_dim 128: 641
// us, 740 GFLOP of the rows' own products at 1,155 TFLOP/s (61 % of the measured
// cuBLAS burst), 1,110 with the residual's at 1,732 (91 %); 32-bit output 695 to 716.
// 8 chunks of 512, window 1,024: 80 us (92).  What bounds it: the tensor cores' turns,
// the masks of a unit's first and last key tiles, and at a unit's end its outputs and
// the wait for the next Q.
// Measured with P rounded once (445 us), and left: the next unit worked out while the last
// tile runs (head_dim 64: 368 -> 395 us, 3 x 4000: 445 -> 442) and its Q loaded to
// a third slot (3 x 4000: 457 -> 464, 8 x 2,048: 178 -> 193, before outputs were
// staged), units halved for the last round of CTAs (453 -> 487 us).
// Before the tiles took turns (then 509 to 515 us): 64-key tiles with two score
// buffers each (S then runs ahead, but an N = 64 product costs as much as N = 128,
// since reading Q out of shared memory bounds both: 633 us); two warpgroups a tile
// (677 us); a polynomial for every eighth exp2 (550 us); four parts of P instead of
// two (616 us); P by the maximum so far, the tile's own taken beside it (565 us).
#include <cuda_runtime.h>

#include <cmath>
#include <cstdio>
#include <type_traits>

#include "pkv.h"
#include "pkv_cluster.cuh"
#include "pkv_device.cuh"
#include "pkv_host.h"
#include "pkv_tc.cuh"

namespace pkv {

constexpr int kWpThreads = 384;
// registers per thread: the launch gives every thread kWpLaunchRegs; the first
// warpgroup drops to kWpLowRegs and the two softmax warpgroups rise to
// kWpHighRegs, which must not exceed what the drop frees
constexpr int kWpLaunchRegs = 168;
constexpr int kWpLowRegs = 88;
constexpr int kWpHighRegs = 208;
static_assert(128 * kWpLowRegs + 256 * kWpHighRegs <= kWpThreads * kWpLaunchRegs, "register split");
constexpr int kWpRows = 128;    // MMA rows = (token, head) pairs per query tile
constexpr int kWpKeys = 128;    // keys per K/V tile
constexpr int kWpPages = kWpKeys / 16;
constexpr int kWpStages = 2;
constexpr uint64_t kWpWaitNs = 2000000000ull;
// tensor memory: S / P of query tile t at column 256 t, O at 256 t + 128
constexpr uint32_t kWpTmemCols = 512;

struct WindowPrefillParams {
    void *out;
    const int32_t *cu_seqlens;
    const int32_t *block_tables;
    const int32_t *context_lens;
    int *dev_status;
    int max_blocks, num_blocks, Hq, Hkv, G;
    int rtok, units_per_seq;
    int window, sinks, total_q, max_q_len;
    float scale_log2;
    bool boxes;   // a warp's 32 rows are whole tokens: tout has a box for them
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

struct WpBars {
    uint64_t unit_full[2], unit_empty[2], cancel;
    uint64_t q_full, q_empty;
    uint64_t k_full[kWpStages], v_full[kWpStages], k_empty[kWpStages], v_empty[kWpStages];
    uint64_t v_clean[kWpStages];
    uint64_t s_full[2], p_full[2][2], o_done[2];   // per query tile (and part of its keys)
    uint64_t turn[2];                              // a query tile's turn at the tensor cores
};

// A K or V tile is its pages one after another; a page holds, for each group of
// 8 rows, the 64-column halves of those rows, each an 8 x 128-byte swizzle atom.
template <int D>
struct WpShape {
    static constexpr int HALVES = D / 64;
    static constexpr int Q_HALF = kWpRows * 128;            // 128 rows x 64 columns
    static constexpr int Q_BYTES = HALVES * Q_HALF;
    static constexpr int GROUP = HALVES * 1024;             // 8 rows
    static constexpr int PAGE = 2 * GROUP;
    static constexpr int TILE = kWpPages * PAGE;
    static constexpr int STAGE_BYTES = 2 * TILE;            // K then V
    // 32-key groups of P after which the first part of P V may start.  Three
    // chunks of 3,500-4,100 rows, window 4,096, after one, two and three groups:
    // 538, 536 and 547 us with head_dim 64; 632, 641 and 644 with 128.
    static constexpr int FIRST_PART = 2;
    static constexpr int OFF_Q = 0;                         // tile A, then tile B
    static constexpr int OFF_KV = 2 * Q_BYTES;
    static constexpr int OFF_OUT = OFF_KV + kWpStages * STAGE_BYTES;   // outputs on their way out: 128 bytes of 32 rows a warp
    static constexpr int OFF_UNIT = OFF_OUT + 8 * 4096;
    static constexpr int OFF_CANCEL = OFF_UNIT + 2 * (int)sizeof(WpUnit);
    static constexpr int OFF_BAR = OFF_CANCEL + 16;
    static constexpr int SMEM_BYTES = 1024 + OFF_BAR + (int)sizeof(WpBars) + 16;
};
static_assert(WpShape<128>::SMEM_BYTES <= 227 * 1024, "shared memory");

// One page of a cache (see encode_page_map) into shared memory.
__device__ __forceinline__ void load_page(void *dst, const CUtensorMap *map, int group, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %2, %2, %3}], [%4];" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(group), "r"(smem_addr(bar))
        : "memory");
}

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

// WIDE: a 32-bit output.  TILES: query tiles of a unit, 2, or 1 (A alone)
template <typename T, int D, bool WIDE, int TILES>
__global__ void __launch_bounds__(kWpThreads, 1)
    window_prefill_kernel(const WindowPrefillParams p, const __grid_constant__ CUtensorMap tk,
                          const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap tq,
                          const __grid_constant__ CUtensorMap tout) {
    using Sh = WpShape<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    WpBars *bars = reinterpret_cast<WpBars *>(sm + Sh::OFF_BAR);
    WpUnit *units = reinterpret_cast<WpUnit *>(sm + Sh::OFF_UNIT);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 1);
    volatile int *gave_up = reinterpret_cast<volatile int *>(tmem_slot + 1);   // a wait of this CTA ran out

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars->unit_full[i], 1);
            mbar_init(&bars->unit_empty[i], TILES == 2 ? 11 : 6);   // warps 1 to 11, or those of tile A and the cleaner
            mbar_init(&bars->s_full[i], 1);
            mbar_init(&bars->p_full[i][0], 4);
            mbar_init(&bars->p_full[i][1], 4);
            mbar_init(&bars->o_done[i], 1);
            mbar_init(&bars->turn[i], 1);
        }
        mbar_init(&bars->cancel, 1);
        mbar_init(&bars->q_full, 1);
        mbar_init(&bars->q_empty, TILES);   // each query tile's products
        for (int s = 0; s < kWpStages; ++s) {
            mbar_init(&bars->k_full[s], 1);
            mbar_init(&bars->v_full[s], 1);
            mbar_init(&bars->k_empty[s], TILES);
            mbar_init(&bars->v_empty[s], TILES + 1);   // and the cleaner, which must not fall a phase behind
            mbar_init(&bars->v_clean[s], 1);
        }
        *gave_up = 0;
        fence_mbar_init();
        prefetch_tensormap(&tq);
        prefetch_tensormap(&tk);
        prefetch_tensormap(&tv);
    }
    if (warp == 1) {
        tc::tmem_alloc(tmem_slot, kWpTmemCols);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const uint32_t sbase = smem_addr(sm);
    // inputs may come from the previous kernel on the stream (the append)
    pdl_wait_primary();
    pdl_launch_dependents();

    // A wait that gives up after kWpWaitNs, or once another one of the CTA has.
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (mbar_try_wait(bar, parity & 1u)) return true;
        const uint64_t t0 = global_timer_ns();
        while (!mbar_try_wait(bar, parity & 1u)) {
            if (*gave_up) return false;
            if (global_timer_ns() - t0 > kWpWaitNs) {
                *gave_up = 1;
                set_status(p.dev_status, PKV_DEV_WAIT_TIMEOUT);
                return false;
            }
        }
        return true;
    };
    auto wait_all = [&](uint64_t *bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)); };

    if (warp < 4) {
        tc::setmaxnreg_dec<kWpLowRegs>();
        if (warp == 0) {
            // ---------------- scheduler and TMA producer ----------------
            int place = blockIdx.x;
            int n = 0;              // units published
            uint32_t g = 0;         // key tiles loaded
            uint32_t asked = 0;     // places asked for
            bool ok = true;
            bool asking = false;
            auto ask = [&]() {
                if (!asking && lane == 0) {
                    mbar_arrive_expect_tx(&bars->cancel, 16);
                    cancel_next_cta(sm + Sh::OFF_CANCEL, &bars->cancel);
                }
                asked += !asking;
                asking = true;
            };
            while (ok) {
                // place -> unit; chunk by chunk, the last pair of tiles first, the KV heads side by side
                const int h = place % p.Hkv;
                const int rest = place / p.Hkv;
                const int unit = p.units_per_seq - 1 - rest % p.units_per_seq;
                const int c = rest / p.units_per_seq;
                const int q0 = __ldg(p.cu_seqlens + c);
                const int q_len = __ldg(p.cu_seqlens + c + 1) - q0;
                const int ctx = __ldg(p.context_lens + c);
                const int i0 = unit * TILES * p.rtok;
                int bad = 0;
                // (rows past max_q_len have no unit)
                if (q_len < 0 || q_len > ctx || q_len > p.max_q_len || q0 < 0 || q_len > p.total_q - q0)
                    bad = PKV_DEV_BAD_CHUNK;
                else if (ctx > p.max_blocks * 16)
                    bad = PKV_DEV_BAD_CONTEXT;
                if (bad && unit == 0 && lane == 0) set_status(p.dev_status, bad);
                if (!bad && i0 < q_len) {
                    WpUnit u = {};
                    u.h = h;
                    u.row0 = q0 + i0;
                    u.tokens = min(TILES * p.rtok, q_len - i0);
                    u.first = ctx - q_len + i0;
                    u.wpos = max(u.first - p.window + 1, 0);
                    const int sink_pages = min((p.sinks + 15) / 16, (ctx + 15) / 16);
                    const int skip = max(u.wpos / 16 - sink_pages, 0);
                    u.first -= 16 * skip;
                    u.wpos -= 16 * skip;
                    u.ctx = ctx - 16 * skip;
                    u.tiles = (u.first + u.tokens - 1) / kWpKeys + 1;
                    if (n >= 2) ok = wait_all(&bars->unit_empty[n & 1], (uint32_t)(n / 2 - 1));
                    if (!ok) break;
                    if (lane == 0) {
                        units[n & 1] = u;
                        tc::mbar_arrive_cta(&bars->unit_full[n & 1]);
                    }
                    const int32_t *row = p.block_tables + (int64_t)c * p.max_blocks;
                    const int pages = (u.ctx + 15) / 16;
                    // lane i < 8 reads the block id of page i of the tile, one tile ahead
                    auto wanted = [&](int j) { return lane < kWpPages && j * kWpPages + lane < pages; };
                    auto fetch = [&](int j) {
                        const int v = j * kWpPages + lane;
                        return wanted(j) ? __ldg(row + (v < sink_pages ? v : v + skip)) : 0;
                    };
                    int blk_next = fetch(0);
                    for (int j = 0; ok && j < u.tiles; ++j, ++g) {
                        // the next place is asked for near the unit's end: a
                        // CTA that takes one sooner holds it back from others
                        // (8 x 512 rows: 73.9 us when asked for at its start)
                        if (j + 2 >= u.tiles) ask();
                        const int blk = blk_next;
                        if (j + 1 < u.tiles) blk_next = fetch(j + 1);
                        int y = p.num_blocks * p.Hkv * 2;      // 8-row group past the pool: zero fill
                        if (wanted(j)) {
                            if (blk >= 0 && blk < p.num_blocks)
                                y = (blk * p.Hkv + h) * 2;
                            else
                                set_status(p.dev_status, PKV_DEV_BAD_BLOCK_ID);
                        }
                        int ys[kWpPages];
#pragma unroll
                        for (int pg = 0; pg < kWpPages; ++pg) ys[pg] = __shfl_sync(0xffffffffu, y, pg);
                        const int st = (int)(g % kWpStages);
                        uint8_t *kd = sm + Sh::OFF_KV + st * Sh::STAGE_BYTES, *vd = kd + Sh::TILE;
                        if (lane == 0) {
                            // a K slot is free once both S products of its last tile are done
                            if (g >= kWpStages) ok = wait(&bars->k_empty[st], g / kWpStages - 1);
                            if (ok) {
                                mbar_arrive_expect_tx(&bars->k_full[st], Sh::TILE);
#pragma unroll
                                for (int pg = 0; pg < kWpPages; ++pg)
                                    load_page(kd + pg * Sh::PAGE, &tk, ys[pg], &bars->k_full[st]);
                            }
                            if (ok && j == 0) {
                                // Q is free once the unit before has no S product left
                                if (n > 0) ok = wait(&bars->q_empty, (uint32_t)(n - 1));
                                if (ok) {
                                    mbar_arrive_expect_tx(&bars->q_full, (uint32_t)(TILES * Sh::HALVES * p.G * p.rtok * 128));
#pragma unroll
                                    for (int t = 0; t < TILES; ++t)
#pragma unroll
                                        for (int hf = 0; hf < Sh::HALVES; ++hf)
                                            tc::tma_load_3d(sm + Sh::OFF_Q + t * Sh::Q_BYTES + hf * Sh::Q_HALF, &tq, hf * 64,
                                                            h * p.G, u.row0 + t * p.rtok, &bars->q_full);
                                }
                            }
                            // a V slot is free once both P V products of its last tile (and its cleaning) are done
                            if (ok && g >= kWpStages) ok = wait(&bars->v_empty[st], g / kWpStages - 1);
                            if (ok) {
                                mbar_arrive_expect_tx(&bars->v_full[st], Sh::TILE);
#pragma unroll
                                for (int pg = 0; pg < kWpPages; ++pg)
                                    load_page(vd + pg * Sh::PAGE, &tv, ys[pg], &bars->v_full[st]);
                            }
                        }
                        ok = __shfl_sync(0xffffffffu, ok, 0);
                    }
                    ++n;
                }
                if (!ok) break;
                ask();
                ok = wait_all(&bars->cancel, asked - 1);
                if (!ok) break;
                asking = false;
                place = cancelled_cta(sm + Sh::OFF_CANCEL);
                fence_proxy_async_smem();   // the answer is read before the next one is written
                __syncwarp();
                if (place < 0) break;
            }
            // no more units (after a wait that ran out the others leave by themselves)
            if (ok && n >= 2) ok = wait_all(&bars->unit_empty[n & 1], (uint32_t)(n / 2 - 1));
            if (ok && lane == 0) {
                units[n & 1].tiles = 0;
                tc::mbar_arrive_cta(&bars->unit_full[n & 1]);
            }
            if (!ok && lane == 0) {
                // what is under way must land before the CTA leaves
                if (asking) mbar_wait(&bars->cancel, (asked - 1) & 1u, kWpWaitNs / 8);
                for (int st = 0; st < kWpStages; ++st) {
                    if (g > (uint32_t)st) {
                        const uint32_t last = (g - 1 - st) / kWpStages;
                        mbar_wait(&bars->k_full[st], last & 1u, kWpWaitNs / 8);
                        mbar_wait(&bars->v_full[st], last & 1u, kWpWaitNs / 8);
                    }
                }
                if (n > 0) mbar_wait(&bars->q_full, (uint32_t)(n - 1) & 1u, kWpWaitNs / 8);
            }
        } else if (warp < 3) {
            // ---------------- MMA issuer of query tile t ----------------
            // The whole warp walks the schedule, so the waits and the
            // descriptor arithmetic are warp-uniform; one elected lane issues
            // each MMA and commit.
            const int t = warp - 1;
            const bool leader = tc::elect_one();
            constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
            constexpr uint32_t idesc_s = tc::idesc_f16(kBf16, false, false, kWpRows, kWpKeys);
            constexpr uint32_t idesc_o = tc::idesc_f16(kBf16, false, true, kWpRows, D);
            const uint32_t d_s = tmem + t * 256, d_o = d_s + 128;
            const uint64_t q_desc = tc::smem_desc_sw128(sbase + Sh::OFF_Q + t * Sh::Q_BYTES, 16, 1024);
            const uint64_t k_desc = tc::smem_desc_sw128(sbase + Sh::OFF_KV, 16, Sh::GROUP);
            const uint64_t v_desc = tc::smem_desc_sw128(sbase + Sh::OFF_KV + Sh::TILE, 1024, Sh::GROUP);
            uint32_t g = 0;     // key tiles done
            // The two tiles take turns: P V of a key tile and S of the next are
            // one turn, so that a tile's softmax runs beside the other's turn.
            auto pass_turn = [&]() {
                if (TILES == 2 && lane == 0) tc::mbar_arrive_cta(&bars->turn[1 - t]);
            };
            auto issue_s = [&](uint32_t k, bool last, bool pass) {   // S = Q K^T of key tile k, the unit's last?
                if (!wait_all(&bars->k_full[k % kWpStages], k / kWpStages)) return false;
                tc::fence_after_sync();
                const uint64_t kb = k_desc + (uint64_t)(((k % kWpStages) * Sh::STAGE_BYTES) >> 4);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t qo = ((kk >> 2) * Sh::Q_HALF + (kk & 3) * 32) >> 4;
                    const uint32_t ko = ((kk >> 2) * 1024 + (kk & 3) * 32) >> 4;
                    if (pass && kk == D / 16 - 2) pass_turn();   // on its way while the rest is issued
                    if (leader) tc::mma_f16_ss(d_s, q_desc + qo, kb + ko, idesc_s, kk > 0);
                }
                if (leader) {
                    tc::mma_commit(&bars->s_full[t]);
                    tc::mma_commit(&bars->k_empty[k % kWpStages]);
                    if (last) tc::mma_commit(&bars->q_empty);
                }
                return true;
            };
            for (int n = 0; t < TILES; ++n) {
                bool ok = wait_all(&bars->unit_full[n & 1], (uint32_t)(n / 2));
                if (!ok) break;
                const WpUnit u = units[n & 1];
                const int tiles = u.tiles;
                __syncwarp();
                if (lane == 0) tc::mbar_arrive_cta(&bars->unit_empty[n & 1]);
                if (tiles == 0) break;
                // (S may be written: the product that read P over it was issued before)
                ok = wait_all(&bars->q_full, (uint32_t)n) && issue_s(g, tiles == 1, false);
                for (int j = 0; ok && j < tiles; ++j, ++g) {
                    const uint64_t vb = v_desc + (uint64_t)(((g % kWpStages) * Sh::STAGE_BYTES) >> 4);
                    const bool dirty = WpHidden(u, j * kWpKeys, p.sinks, kWpKeys).any();
                    ok = wait_all(dirty ? &bars->v_clean[g % kWpStages] : &bars->v_full[g % kWpStages], g / kWpStages);
                    if (TILES == 2 && (t == 1 || g > 0)) ok = ok && wait_all(&bars->turn[t], t == 1 ? g : g - 1);
#pragma unroll
                    for (int part = 0; part < 2; ++part) {
                        // P of a unit's first tile is there only after the unit before's O was read
                        ok = ok && wait_all(&bars->p_full[t][part], g);
                        if (!ok) break;
                        tc::fence_after_sync();
#pragma unroll
                        for (int kk = part ? 2 * Sh::FIRST_PART : 0; kk < (part ? kWpPages : 2 * Sh::FIRST_PART); ++kk) {
                            // O (+)= P V, a page at a time
                            const uint32_t ph = d_s + 32 * (kk >> 1) + 8 * (kk & 1);
                            const uint64_t vp = vb + (uint32_t)(kk * Sh::PAGE >> 4);
                            if (leader) {
                                tc::mma_f16_ts(d_o, ph, vp, idesc_o, j > 0 || kk > 0);
                                tc::mma_f16_ts(d_o, ph + 16, vp, idesc_o, true);   // the weights' rounding residual
                            }
                        }
                    }
                    if (!ok) break;
                    if (leader) {
                        tc::mma_commit(&bars->v_empty[g % kWpStages]);
                        if (j + 1 == tiles) tc::mma_commit(&bars->o_done[t]);
                    }
                    if (j + 1 < tiles)
                        ok = issue_s(g + 1, j + 2 == tiles, true);
                    else
                        pass_turn();
                }
                if (!ok) break;
            }
        }
        else {
            // ---------------- cleaner of V ----------------
            uint32_t g = 0;
            bool ok = true;
            for (int n = 0; ok; ++n) {
                ok = wait_all(&bars->unit_full[n & 1], (uint32_t)(n / 2));
                if (!ok) break;
                const WpUnit u = units[n & 1];
                __syncwarp();
                if (lane == 0) tc::mbar_arrive_cta(&bars->unit_empty[n & 1]);
                if (u.tiles == 0) break;
                for (int j = 0; ok && j < u.tiles; ++j, ++g) {
                    const int st = (int)(g % kWpStages);
                    ok = wait_all(&bars->v_full[st], g / kWpStages);
                    const WpHidden hid(u, j * kWpKeys, p.sinks, kWpKeys);
                    if (hid.any()) {
                        // four rows at a time, eight lanes a 128-byte row half
                        uint8_t *v = sm + Sh::OFF_KV + st * Sh::STAGE_BYTES + Sh::TILE + (lane & 7) * 16;
                        for (int r = lane >> 3; r < kWpKeys; r += 4)
                            if (hid.has(r))
#pragma unroll
                                for (int hf = 0; hf < Sh::HALVES; ++hf)
                                    *reinterpret_cast<uint4 *>(v + (r >> 3) * Sh::GROUP + hf * 1024 + (r & 7) * 128) =
                                        make_uint4(0u, 0u, 0u, 0u);
                        fence_proxy_async_smem();
                    }
                    __syncwarp();
                    if (lane == 0) {
                        tc::mbar_arrive_cta(&bars->v_clean[st]);
                        tc::mbar_arrive_cta(&bars->v_empty[st]);
                    }
                }
            }
        }
    } else {
        tc::setmaxnreg_inc<kWpHighRegs>();
        // ---------------- softmax: tile t, one row per thread ----------------
        const int t = (warp - 4) >> 2;
        const int lane_base = 32 * (warp & 3);          // tensor-memory lanes this warp may touch
        const int r = lane_base + lane;                 // row within the tile
        const uint32_t scol = tmem + ((uint32_t)lane_base << 16) + t * 256;   // the scores, then P
        const uint32_t ocol = scol + 128;
        const uint64_t scale2 = f2_pack(p.scale_log2, p.scale_log2);
        uint32_t g = 0;                                 // key tiles taken
        bool ok = t < TILES;
        for (int n = 0; ok; ++n) {
            ok = wait_all(&bars->unit_full[n & 1], (uint32_t)(n / 2));
            if (!ok) break;
            const WpUnit u = units[n & 1];
            __syncwarp();
            if (lane == 0) tc::mbar_arrive_cta(&bars->unit_empty[n & 1]);
            if (u.tiles == 0) break;
            const int tok = t * p.rtok + r / p.G, head = r % p.G;
            const bool valid = r < p.G * p.rtok && tok < u.tokens;
            const int pos = u.first + (valid ? tok : u.tokens - 1);   // padding rows see the last row's keys
            float m_used = -INFINITY, l = 0.f;
            for (int j = 0; j < u.tiles; ++j, ++g) {
                ok = wait_all(&bars->s_full[t], g);
                if (!ok) break;
                tc::fence_after_sync();
                const int key0 = j * kWpKeys;
                float v[kWpKeys];
#pragma unroll
                for (int cc = 0; cc < kWpKeys; cc += 32) tc::tmem_ld32(scol + cc, *reinterpret_cast<float(*)[32]>(v + cc));
                tc::tmem_wait_ld();
                // hidden: past the row's position; below its window and behind the first tokens
                const int lim = pos - key0, low = lim - p.window + 1, sk = p.sinks - key0;
                if (__any_sync(0xffffffffu, lim < kWpKeys - 1 || (low > 0 && sk < kWpKeys))) {
                    auto below = [](int n) { return n >= 32 ? 0xffffffffu : (n <= 0 ? 0u : (1u << n) - 1u); };
#pragma unroll
                    for (int cc = 0; cc < kWpKeys; cc += 32) {
                        const uint32_t see = below(lim + 1 - cc) & (~below(low - cc) | below(sk - cc));
                        if (__any_sync(0xffffffffu, see != 0xffffffffu)) {
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!(see & (1u << e))) v[cc + e] = -INFINITY;
                        }
                    }
                }
                float mx4[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
                for (int pr = 0; pr < (kWpKeys - 4) / 2; ++pr)
                    mx4[pr & 3] = fmax3(mx4[pr & 3], v[4 + 2 * pr], v[5 + 2 * pr]);
                // scale_log2 > 0, so the scaled maximum is the maximum scaled
                const float mx = fmax3(fmaxf(mx4[0], mx4[1]), mx4[2], mx4[3]) * p.scale_log2;
                const bool first = m_used == -INFINITY;
                const float m_new = fmaxf(m_used, mx);
                const bool rescale = !first && m_new > m_used + 8.f;
                const float alpha = rescale ? exp2_approx(m_used - m_new) : 1.f;
                if (first || rescale) m_used = m_new;
                // O was last written by the P V product before, which the tensor
                // core finished before this tile's S (issued after it) completed
                if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll 1
                    for (int cc = 0; cc < D; cc += 32) {
                        float o[32];
                        tc::tmem_ld32(ocol + cc, o);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] *= alpha;
                        tc::tmem_st32(ocol + cc, o);
                    }
                }
                // P = 2^(x - m_used) over the same columns, 32 keys at a time: 16
                // columns of rounded pairs, then 16 of residual pairs.
                // A row that has seen no key yet has nothing to subtract.
                const float sub = m_used == -INFINITY ? 0.f : m_used;
                const uint64_t negm2 = f2_pack(-sub, -sub);
                uint64_t sum2[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
                for (int cc = 0; cc < kWpKeys / 32; ++cc) {
                    uint32_t hi[16], lo[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float a, b;
                        f2_unpack(f2_fma(f2_pack(v[32 * cc + 2 * e], v[32 * cc + 2 * e + 1]), scale2, negm2), a, b);
                        a = exp2_approx(a);
                        b = exp2_approx(b);
                        const uint64_t ab = f2_pack(a, b);
                        sum2[e & 1] = f2_add(sum2[e & 1], ab);
                        pack2_split2<T>(ab, a, b, hi[e], lo[e]);
                    }
                    tc::tmem_st16(scol + cc * 32, hi);
                    tc::tmem_st16(scol + cc * 32 + 16, lo);
                    if (cc == Sh::FIRST_PART - 1 || cc == 3) {   // a part of P is ready
                        tc::tmem_wait_st();
                        tc::fence_before_sync();
                        __syncwarp();
                        if (lane == 0) tc::mbar_arrive_cta(&bars->p_full[t][cc == 3]);
                    }
                }
                float s0, s1, s2, s3;
                f2_unpack(sum2[0], s0, s1);
                f2_unpack(sum2[1], s2, s3);
                l = l * alpha + ((s0 + s1) + (s2 + s3));
            }
            ok = ok && wait_all(&bars->o_done[t], (uint32_t)n);
            if (!ok) break;
            tc::fence_after_sync();
            const float inv = 1.f / l;
            // 128 bytes of each row at a time: a thread has a row of O, but stores
            // want a row's bytes side by side, so they change hands in shared memory
            // (16-byte chunks, swizzled as TMA swizzles).  Straight from the rows, 32
            // lines an instruction, 8 x 2,048 rows take 178 us instead of 169.  Where
            // the warp's 32 rows are whole tokens TMA stores them, beside the next
            // 128 bytes or the next unit: 162 us instead of 165 (8 x 1,000-1,500 rows
            // of 8 heads, window 128: 21.9 and 22.8; 3 x 4000: 445 and 440; all with
            // P rounded once).
            constexpr int kCols = WIDE ? 32 : 64;      // a 32-bit output or a 16-bit one
            constexpr int kSize = WIDE ? 4 : 2;
            const int64_t at = valid ? ((int64_t)(u.row0 + tok) * p.Hq + (int64_t)u.h * p.G + head) * D * kSize : -1;
            uint8_t *stage = sm + Sh::OFF_OUT + (warp - 4) * 4096;
            const bool box = !WIDE && p.boxes && __all_sync(0xffffffffu, valid);
#pragma unroll 1
            for (int cc = 0; cc < D; cc += kCols) {
                float v[kCols];
#pragma unroll
                for (int e = 0; e < kCols; e += 32) tc::tmem_ld32(ocol + cc + e, *reinterpret_cast<float(*)[32]>(v + e));
                tc::tmem_wait_ld();
                if (lane == 0) stores_read();
                __syncwarp();
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    uint4 w;
                    if constexpr (WIDE)
                        w = make_uint4(__float_as_uint(v[4 * e] * inv), __float_as_uint(v[4 * e + 1] * inv),
                                       __float_as_uint(v[4 * e + 2] * inv), __float_as_uint(v[4 * e + 3] * inv));
                    else
                        w = make_uint4(pack2<T>(v[8 * e] * inv, v[8 * e + 1] * inv),
                                       pack2<T>(v[8 * e + 2] * inv, v[8 * e + 3] * inv),
                                       pack2<T>(v[8 * e + 4] * inv, v[8 * e + 5] * inv),
                                       pack2<T>(v[8 * e + 6] * inv, v[8 * e + 7] * inv));
                    *reinterpret_cast<uint4 *>(stage + lane * 128 + ((e ^ (lane & 7)) << 4)) = w;
                }
                if (box) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) store_rows(&tout, stage, cc, u.h * p.G, u.row0 + tok);
                    continue;
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int row = 4 * i + (lane >> 3);
                    const uint4 w = *reinterpret_cast<const uint4 *>(stage + row * 128 + (((lane ^ row) & 7) << 4));
                    const int64_t to = __shfl_sync(0xffffffffu, at, row);
                    if (to >= 0) *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(p.out) + to + cc * kSize + (lane & 7) * 16) = w;
                }
                __syncwarp();
            }
            // O has been read: ordered before this unit's successor's P, whose
            // arrival lets the tensor core write O again
            tc::fence_before_sync();
        }
        if (lane == 0) stores_done();
    }

    tc::fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, kWpTmemCols);
    }
}

// A cache as (64 columns, 8 rows, column halves, groups of 8 rows): a box of two
// groups is one (block, KV head) page in the order of WpShape, in one load.
// Groups past the pool read 0.
static int encode_page_map(CUtensorMap *map, const void *base, int num_blocks, int num_kv_heads, int head_dim) {
    const uint64_t row = (uint64_t)head_dim * 2;
    const uint64_t dims[4] = {64, 8, (uint64_t)head_dim / 64, (uint64_t)num_blocks * num_kv_heads * 2};
    const uint64_t strides[3] = {row, 128, 8 * row};
    const uint32_t box[4] = {64, 8, (uint32_t)head_dim / 64, 2};
    return encode_tiled_map(map, base, 4, dims, strides, box);
}

template <typename T, int D, bool WIDE, int TILES>
static int launch_window_prefill(const WindowPrefillParams &prm, const CUtensorMap &tk, const CUtensorMap &tv,
                                 const CUtensorMap &tq, const CUtensorMap &tout, int grid, cudaStream_t stream) {
    using Sh = WpShape<D>;
    // the register split inside the kernel waits for registers that only exist
    // if the compiled count is the one it was sized for: check it (once; the
    // answer does not change) and refuse to launch otherwise
    static int regs_ok = 0;   // 0 unknown, 1 as sized, -1 not
    if (regs_ok == 0) {
        cudaFuncAttributes fa;
        cudaError_t e = cudaFuncGetAttributes(&fa, window_prefill_kernel<T, D, WIDE, TILES>);
        if (e != cudaSuccess) return cuda_fail(e);
        regs_ok = fa.numRegs == kWpLaunchRegs ? 1 : -1;
        if (regs_ok < 0) {
            char msg[128];
            std::snprintf(msg, sizeof msg, "window prefill kernel compiled to %d registers per thread, its split needs %d",
                          fa.numRegs, kWpLaunchRegs);
            set_error_message(msg);
        }
    }
    if (regs_ok < 0) return PKV_ERR_UNSUPPORTED;
    static unsigned long long attr_set = 0;   // per instantiation and device
    if (!done_on_device(&attr_set)) {
        cudaError_t e = cudaFuncSetAttribute(window_prefill_kernel<T, D, WIDE, TILES>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::SMEM_BYTES);
        if (e != cudaSuccess) return cuda_fail(e);
        mark_done_on_device(&attr_set);
    }
    cudaError_t e = launch_pdl(window_prefill_kernel<T, D, WIDE, TILES>, dim3(grid), dim3(kWpThreads), Sh::SMEM_BYTES, stream,
                               prm, tk, tv, tq, tout);
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? PKV_OK : cuda_fail(e);
}

}  // namespace pkv

extern "C" int pkv_paged_window_prefill_attention(void *out, const void *q, const int32_t *cu_seqlens, int num_seqs,
                                                  int max_q_len, int total_q, const void *k_cache, const void *v_cache,
                                                  const int32_t *block_tables, int max_blocks_per_seq,
                                                  const int32_t *context_lens, int num_blocks, int num_q_heads,
                                                  int num_kv_heads, int head_dim, int block_size, int window,
                                                  int num_sinks, float scale, int dtype, int out_dtype, int *dev_status,
                                                  void *stream) {
    pkv::NvtxRange nvtx_range("pkv_paged_window_prefill_attention");
    using namespace pkv;
    if (num_seqs < 0 || max_q_len < 0 || total_q < 0 || num_blocks <= 0 || num_kv_heads <= 0 || num_q_heads <= 0 ||
        max_blocks_per_seq <= 0 || window <= 0 || num_sinks < 0)
        return PKV_ERR_INVALID_ARG;
    if (num_q_heads % num_kv_heads != 0) return PKV_ERR_INVALID_ARG;
    const int G = num_q_heads / num_kv_heads;
    if (G > 16 || block_size != 16 || (head_dim != 64 && head_dim != 128)) return PKV_ERR_UNSUPPORTED;
    if (dtype != PKV_DTYPE_F16 && dtype != PKV_DTYPE_BF16) return PKV_ERR_UNSUPPORTED;
    if (out_dtype != dtype && out_dtype != PKV_DTYPE_F32) return PKV_ERR_UNSUPPORTED;
    if (!(std::isfinite(scale) && scale > 0.f)) return PKV_ERR_INVALID_ARG;
    if ((int64_t)num_blocks * num_kv_heads * block_size >= (int64_t)1 << 31) return PKV_ERR_UNSUPPORTED;
    if (max_blocks_per_seq > (1 << 26)) return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0 || max_q_len == 0 || total_q == 0) return PKV_OK;
    if (!out || !q || !cu_seqlens || !k_cache || !v_cache || !block_tables || !context_lens) return PKV_ERR_INVALID_ARG;
    // the query tile is fetched by TMA and output rows are stored as 16-byte vectors
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !aligned(cu_seqlens, 4) || !aligned(block_tables, 4) || !aligned(context_lens, 4))
        return PKV_ERR_INVALID_ARG;
    int sms = 0;
    int rc = current_sm_count(&sms);
    if (rc != PKV_OK) return rc;
    const int rtok = kWpRows / G;
    // query tiles of a unit: two, which share every K and V tile; or one, when
    // all units then run at once and a step of 128 keys has one tile's products
    // (two / one, us, window 1,024: 512 rows behind up to 4,096 26.2 / 23.6, behind
    // 4,096 24.1 / 23.4; 2 x 256 rows 24.2 / 22.2; 16 rows 23.9 / 22.9; three chunks of
    // 3,500-4,100 rows, which fill the GPU either way, with P rounded once: 449 / 776).
    // A 32-bit output always takes two.
    auto units_of = [&](int tiles) { return ((int64_t)max_q_len + tiles * rtok - 1) / (tiles * rtok); };
    const bool one = out_dtype != PKV_DTYPE_F32 && num_seqs * units_of(1) * num_kv_heads <= sms;
    const int qtiles = one ? 1 : 2;
    const int64_t grid = (int64_t)num_seqs * units_of(qtiles) * num_kv_heads;
    if (grid >= (int64_t)1 << 31) return PKV_ERR_UNSUPPORTED;
    const int units = (int)units_of(qtiles);
    CUtensorMap tk, tv, tq;
    rc = encode_page_map(&tk, k_cache, num_blocks, num_kv_heads, head_dim);
    if (rc != PKV_OK) return rc;
    rc = encode_page_map(&tv, v_cache, num_blocks, num_kv_heads, head_dim);
    if (rc != PKV_OK) return rc;
    // q as [total_q][Hq][head_dim]: a box of 64 columns x G heads x rtok tokens; rows past total_q read 0
    const uint64_t dims[3] = {(uint64_t)head_dim, (uint64_t)num_q_heads, (uint64_t)total_q};
    const uint64_t strides[2] = {(uint64_t)head_dim * 2, (uint64_t)num_q_heads * head_dim * 2};
    const uint32_t box[3] = {64, (uint32_t)G, (uint32_t)rtok};
    rc = encode_tiled_map(&tq, q, 3, dims, strides, box);
    if (rc != PKV_OK) return rc;
    WindowPrefillParams prm;
    prm.boxes = out_dtype == dtype && 32 % G == 0;
    CUtensorMap tout = tq;
    if (prm.boxes) {
        const uint32_t rows[3] = {64, (uint32_t)G, 32u / (uint32_t)G};
        rc = encode_tiled_map(&tout, out, 3, dims, strides, rows);
        if (rc != PKV_OK) return rc;
    }
    prm.out = out;
    prm.cu_seqlens = cu_seqlens;
    prm.block_tables = block_tables;
    prm.context_lens = context_lens;
    prm.dev_status = dev_status;
    prm.max_blocks = max_blocks_per_seq;
    prm.num_blocks = num_blocks;
    prm.Hq = num_q_heads;
    prm.Hkv = num_kv_heads;
    prm.G = G;
    prm.rtok = rtok;
    prm.units_per_seq = units;

    const int64_t capacity = (int64_t)max_blocks_per_seq * 16;
    prm.window = window < capacity ? window : (int)capacity;   // no context is longer
    prm.sinks = num_sinks < capacity ? num_sinks : (int)capacity;
    prm.total_q = total_q;
    prm.max_q_len = max_q_len;
    prm.scale_log2 = scale * 1.4426950408889634f;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    auto launch = [&](auto type, auto wide, auto tiles) {
        using T = decltype(type);
        constexpr bool W = decltype(wide)::value;
        constexpr int N = decltype(tiles)::value;
        return head_dim == 128 ? launch_window_prefill<T, 128, W, N>(prm, tk, tv, tq, tout, (int)grid, st)
                               : launch_window_prefill<T, 64, W, N>(prm, tk, tv, tq, tout, (int)grid, st);
    };
    using Yes = std::true_type;
    using No = std::false_type;
    std::integral_constant<int, 1> tile;
    std::integral_constant<int, 2> tiles;
    const bool bf16 = dtype == PKV_DTYPE_BF16;
    if (out_dtype == PKV_DTYPE_F32)
        return bf16 ? launch(__nv_bfloat16(), Yes(), tiles) : launch(__half(), Yes(), tiles);
    if (one) return bf16 ? launch(__nv_bfloat16(), No(), tile) : launch(__half(), No(), tile);
    return bf16 ? launch(__nv_bfloat16(), No(), tiles) : launch(__half(), No(), tiles);
}
