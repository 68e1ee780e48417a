// Prefill attention over the cache held in 8 bits, on the 5th-generation tensor
// cores (pkv_paged_prefill_attention_e4m3).
//
// Mathematics.  As window_prefill.cu, with K_t = k_t a_j and V_t = v_t b_j, k and v
// the e4m3 codes and a, b the scales of t's page j.  Over key tiles of 128
// positions:
//     y_t = scale2 f a_j (q' . k_t) + log2 b_j,   P_t = 2^(y_t - m + 7),
//     l = l c + sum P_t / b_j,   O = O c + P v,   c = 2^(m_old - m),   out = O / l,
// m a maximum of y so far, moved on when a page's P sum to more than 2^15: P stays
// below that, and the largest at least 2^7, whatever the scales are.
//
// Both products run on the codes without their scales:
//   S = q' k^T   in 8 bits (kind::f8f6f4, twice the rate of 16): K goes from the
//                cache to the tensor cores as it is.  A query row is f times the
//                sum of terms, each the rounding of what the ones before leave, f
//                the power of two with its largest element in (224, 448]: one of
//                e4m3's four bits, then of e5m2's three, whose range goes down to
//                2^-16 where e4m3's ends at 2^-9.  Two terms hold bf16's 8 bits, three
//                fp16's 11, of elements down to 2^-13.8 of the row's largest;
//                smaller ones are off by at most 2^-21.8 of it, or 2^-24.8 in fp16 (with
//                e4m3 terms alone: down to 2^-9.8 and 2^-6.8, off by 2^-17.8).  As
//                many steps as in 16 bits, or one and a half times for fp16.
//   O += P v     in fp16: v is converted on the way (exact), P is value and residual,
//                two products, for any output.  (With P rounded once, 2^-11 of a
//                weight, 3 x 4,000 rows of bf16 would take 538 us instead of 724, and
//                outputs would be the 32-bit ones rounded no longer.)
// (P in e4m3 terms would take four: as many steps, and a conversion of every weight
// four times instead of V's once a tile.)
//
// What is walked and the unit of work: as in window_prefill.cu.  Warps (persistent;
// 12 of them):
//   0      TMA and scheduler: takes units, publishes them, loads K and V tiles of
//          codes, 8 pages of 16, a page one box, and the pages' scales (a, log2 b)
//   1      one thread issues the MMAs of both query tiles, turn by turn
//   2, 3   V's codes to fp16, in the layout of an MN-major operand; rows that no row
//          of the unit sees become zero (they may hold NaN codes)
//   4-11   softmax: a warpgroup a query tile, a row per thread; its rows' terms are
//          made by head_dim / 8 lanes each, the next unit's while the last P V of this
//          one runs
// Units go out longest first, found by bisection over up to 32 chunks a lane each
// (us, and chunk by chunk: 8 x 512 behind 0 to 4,096 tokens 140 and 154, 5 x 2,000 of
// head_dim 64 97 and 107; 3 x 4,000 behind a window, whose units are alike, 694 and
// 681).  Where one query tile a unit leaves SMs without one, the unit's keys go to
// the CTAs of a cluster, and the parts are joined through its shared memory (us, and in
// one CTA a unit: 16 rows behind 4,080 17.9 and 62; 50 behind 20,000 94 and 284).
//
// What bounds it: a key tile for two query tiles of head_dim 128 is 2,048 cycles of
// products and half as many again for the residual's, and a chain, S, softmax, P V,
// of which two run at a time; the tensor pipe is active for 70 to 77 % of the time.
// us in bf16, fp16 and bf16 with 32-bit outputs, and over a 16-bit cache in bf16: 8 chunks
// of 512 rows behind 0 to 4,096 tokens 141, 157, 154 and 147, where products of 16
// bits without a residual would take 74; 3 x 4,000 rows, window 4,096, 690, 742, 714
// and 673 for 392; 5 prompts of 2,000, head_dim 64, 94, 97, 98 and 94 for 25, bound by
// the softmax and the issue of products that are half as long.  (Means over three
// sets of contexts; the products' time is of the same ones.)
// Measured and left (3 x 4,000 unless stated): a fourth warpgroup for V and the scales,
// an issuer each for the query tiles; two threads a row, both warpgroups on one
// query tile; a suspended wait; P V from a third of P: none faster.  P in columns of
// its own (head_dim 64), S ahead of the softmax: the query tiles fall into step, 15 %
// slower.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <type_traits>

#include "pkv.h"
#include "pkv_cluster.cuh"
#include "pkv_device.cuh"
#include "pkv_host.h"
#include "pkv_quant.cuh"
#include "pkv_tc.cuh"
#include "pkv_window.cuh"

namespace pkv {

constexpr int kQpThreads = 384;
// registers per thread: the launch gives every thread kQpLaunchRegs; the first
// warpgroup drops and the two softmax warpgroups rise, by no more in all
constexpr int kQpLaunchRegs = 168;
constexpr int kQpLowRegs = 88;
constexpr int kQpHighRegs = 208;
static_assert(128 * (kQpLowRegs + 2 * kQpHighRegs) <= kQpThreads * kQpLaunchRegs, "register split");
constexpr int kQpRows = 128;    // MMA rows = (token, head) pairs per query tile
constexpr int kQpKeys = 128;    // keys per K/V tile
constexpr int kQpPages = kQpKeys / 16;
constexpr int kQpScaleStages = 3;
constexpr uint64_t kQpWaitNs = 2000000000ull;
// tensor memory: S / P of query tile t at column 256 t, O at 256 t + 128
constexpr uint32_t kQpTmemCols = 512;

struct QuantPrefillParams {
    void *out;
    const void *q;
    const float *scales;
    const int32_t *cu_seqlens;
    const int32_t *block_tables;
    const int32_t *context_lens;
    int *dev_status;
    int max_blocks, num_blocks, Hq, Hkv, G;
    int rtok, num_seqs, units_per_seq;
    int window, sinks, total_q, max_q_len;
    float scale_log2;
    bool sorted;  // units by length, longest first
    bool boxes;   // a warp's 32 rows are whole tokens: tout has a box for them
};

struct QpUnit : WpUnit {
    int tile0;                     // the CTA's first key tile of them (u.tiles: its own)
    int chunk, sink_pages, skip;   // page v of the list is logical page v, or v + skip from sink_pages on
};

struct QpBars {
    uint64_t unit_full[2], unit_empty[2], cancel;
    uint64_t q_full[2];                                    // per query tile
    uint64_t k_full[2], k_empty[2];
    uint64_t codes_full[2], codes_empty[2];                // V's codes
    uint64_t v_full[2], v_empty[2];                        // V in fp16
    uint64_t scales_full[kQpScaleStages], scales_empty[kQpScaleStages];
    uint64_t s_full[2], p_full[2][2], half_done[2], o_done[2];   // per query tile (and half of its keys)
};

template <typename T, int D>
struct QpShape {
    static constexpr int TERMS = std::is_same<T, __half>::value ? 3 : 2;
    static constexpr int Q_TERM = kQpRows * D;             // a query tile's codes of one term
    static constexpr int Q_BYTES = TERMS * Q_TERM;
    static constexpr int CODE_PAGE = 16 * D;
    static constexpr int CODE_TILE = kQpPages * CODE_PAGE;
    // V in fp16: a page after another; a page holds, for each group of 8 rows, the
    // 64-column halves of those rows, each an 8 x 128-byte swizzle atom
    static constexpr int HALVES = D / 64;
    static constexpr int GROUP = HALVES * 1024;            // 8 rows
    static constexpr int PAGE = 2 * GROUP;
    static constexpr int TILE = kQpPages * PAGE;
    static constexpr int OFF_Q = 0;                        // tile A, then tile B
    static constexpr int OFF_K = 2 * Q_BYTES;
    static constexpr int OFF_CODES = OFF_K + 2 * CODE_TILE;
    static constexpr int OFF_V = OFF_CODES + 2 * CODE_TILE;
    static constexpr int OFF_OUT = OFF_V + 2 * TILE;       // outputs on their way out: 128 bytes of 32 rows a warp
    // where there is no room for them, the warp's rows of the query's first term
    // take them, and the next unit's terms are made behind them
    static constexpr bool OWN_OUT = !(TERMS == 3 && D == 128);
    static constexpr int OFF_SCALES = OFF_OUT + (OWN_OUT ? 8 * 4096 : 0);
    static constexpr int OFF_CANCEL = OFF_SCALES + kQpScaleStages * kQpPages * 8;
    static constexpr int OFF_UNIT = OFF_CANCEL + 16;
    static constexpr int OFF_BAR = (OFF_UNIT + 2 * (int)sizeof(QpUnit) + 7) & ~7;
    static constexpr int SMEM_BYTES = 1024 + OFF_BAR + (int)sizeof(QpBars) + 16;
};
static_assert(QpShape<__nv_bfloat16, 128>::SMEM_BYTES <= 227 * 1024 && QpShape<__half, 128>::SMEM_BYTES <= 227 * 1024,
              "shared memory");

// One page of codes (see encode_code_page_map) into shared memory.
__device__ __forceinline__ void load_code_page(void *dst, const CUtensorMap *map, int row, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(smem_addr(bar))
        : "memory");
}

// Byte offset of 16-byte piece c of row r in a tile of codes (K-major operand;
// 128-byte rows under 128-byte swizzle, 64-byte rows under 64-byte swizzle).
template <int D>
__device__ __forceinline__ uint32_t code_piece(int r, int c) {
    return D == 128 ? (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)) : (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

// WIDE: a 32-bit output.  TILES: query tiles of a unit, 2, or 1 (A alone; the CTAs
// of a cluster share its keys)
template <typename T, int D, bool WIDE, int TILES>
__global__ void __launch_bounds__(kQpThreads, 1)
    quant_prefill_kernel(const QuantPrefillParams p, const __grid_constant__ CUtensorMap tk,
                         const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap tout) {
    using Sh = QpShape<T, D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    QpBars *bars = reinterpret_cast<QpBars *>(sm + Sh::OFF_BAR);
    QpUnit *units = reinterpret_cast<QpUnit *>(sm + Sh::OFF_UNIT);
    float2 *page_scales = reinterpret_cast<float2 *>(sm + Sh::OFF_SCALES);   // [stage][page] a, log2 b
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 1);
    // What the CTAs of a cluster that share a unit tell one another: a row's m and l,
    // where the query was; its O, by weight, where V was.
    float2 *stats = reinterpret_cast<float2 *>(sm + Sh::OFF_Q);
    const int rank = TILES == 1 ? (int)cluster_ctarank() : 0, ranks = TILES == 1 ? (int)cluster_nctarank() : 1;
    volatile int *gave_up = reinterpret_cast<volatile int *>(tmem_slot + 1);   // a wait of this CTA ran out

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars->unit_full[i], 1);
            mbar_init(&bars->unit_empty[i], 4 * TILES + 3);   // softmax of each tile, issuer, converters
            mbar_init(&bars->q_full[i], 4);
            mbar_init(&bars->k_full[i], 1);
            mbar_init(&bars->k_empty[i], 1);
            mbar_init(&bars->codes_full[i], 1);
            mbar_init(&bars->codes_empty[i], 2);
            mbar_init(&bars->v_full[i], 2);
            mbar_init(&bars->v_empty[i], 1);
            mbar_init(&bars->s_full[i], 1);
            mbar_init(&bars->p_full[i][0], 4);
            mbar_init(&bars->p_full[i][1], 4);
            mbar_init(&bars->half_done[i], 1);
            mbar_init(&bars->o_done[i], 1);
        }
        for (int i = 0; i < kQpScaleStages; ++i) {
            mbar_init(&bars->scales_full[i], 1);
            mbar_init(&bars->scales_empty[i], 4 * TILES);
        }
        mbar_init(&bars->cancel, 1);
        *gave_up = 0;
        units[0].tokens = 0;
        fence_mbar_init();
        prefetch_tensormap(&tk);
        prefetch_tensormap(&tv);
    }
    if (warp == 1) {
        tc::tmem_alloc(tmem_slot, kQpTmemCols);
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

    // A wait that gives up after kQpWaitNs, or once another one of the CTA has.
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (mbar_try_wait(bar, parity & 1u)) return true;
        const uint64_t t0 = global_timer_ns();
        while (!mbar_try_wait(bar, parity & 1u)) {
            if (*gave_up) return false;
            if (global_timer_ns() - t0 > kQpWaitNs) {
                *gave_up = 1;
                set_status(p.dev_status, PKV_DEV_WAIT_TIMEOUT);
                return false;
            }
        }
        return true;
    };
    auto wait_all = [&](uint64_t *bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)); };
    // the n-th unit, once it is published; whether there is one
    auto take_unit = [&](int n, QpUnit &u) {
        const bool ok = wait_all(&bars->unit_full[n & 1], (uint32_t)(n / 2));
        if (!ok) return false;
        u = units[n & 1];
        __syncwarp();
        if (lane == 0) tc::mbar_arrive_cta(&bars->unit_empty[n & 1]);
        return u.tiles > 0;
    };
    auto tile0 = [](const QpUnit &u) { return TILES == 1 ? u.tile0 : 0; };
    // the block id of page v of a unit's list; -1: none is wanted there
    auto page_id = [&](const QpUnit &u, int v) {
        if (16 * v >= u.ctx) return -1;
        return __ldg(p.block_tables + (int64_t)u.chunk * p.max_blocks + (v < u.sink_pages ? v : v + u.skip));
    };

    if (warp < 4) {
        tc::setmaxnreg_dec<kQpLowRegs>();
        if (warp == 0) {
            // ---------------- scheduler and TMA producer ----------------
            int place = blockIdx.x / ranks;
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
            const int R = TILES * p.rtok;   // tokens of a unit
            // a chunk's rows, tokens (none of one that is refused) and context; why it is refused
            auto chunk_of = [&](int c, int &q0, int &q_len, int &ctx) {
                q0 = __ldg(p.cu_seqlens + c);
                q_len = __ldg(p.cu_seqlens + c + 1) - q0;
                ctx = __ldg(p.context_lens + c);
                int bad = 0;
                // (rows past max_q_len have no unit)
                if (q_len < 0 || q_len > ctx || q_len > p.max_q_len || q0 < 0 || q_len > p.total_q - q0)
                    bad = PKV_DEV_BAD_CHUNK;
                else if (ctx > p.max_blocks * 16)
                    bad = PKV_DEV_BAD_CONTEXT;
                if (bad) q_len = 0;
                return bad;
            };
            // Units in order of their contexts, longest first, where a lane can hold a chunk
            // each: a unit's level is the number of units' lengths before it in its context,
            // so a chunk has one unit in each of `count` levels from `level` on.
            const bool sorted = TILES == 2 && p.sorted;
            int my_q0 = 0, my_q_len = 0, my_ctx = 0, level = 0, count = 0;
            if (sorted && lane < p.num_seqs) {
                const int bad = chunk_of(lane, my_q0, my_q_len, my_ctx);
                if (bad && blockIdx.x == 0) set_status(p.dev_status, bad);
                level = (my_ctx - my_q_len) / R;
                count = (my_q_len + R - 1) / R;
            }
            __syncwarp();
            while (ok) {
                // place -> unit; the KV heads side by side
                const int h = place % p.Hkv;
                const int rest = place / p.Hkv;
                int c, unit, q0, q_len, ctx;
                if (sorted) {
                    // the lowest level that at most `rest` units are above, and of its units the
                    // one that is left
                    auto above = [&](int x) { return (int)__reduce_add_sync(0xffffffffu, min(max(level + count - x, 0), count)); };
                    int lo = 0, hi = (int)__reduce_max_sync(0xffffffffu, level + count);
                    while (lo < hi) {
                        const int mid = (lo + hi) >> 1;
                        if (above(mid + 1) <= rest)
                            hi = mid;
                        else
                            lo = mid + 1;
                    }
                    const bool has = lane < p.num_seqs && lo >= level && lo < level + count;
                    const uint32_t with = __ballot_sync(0xffffffffu, has);
                    const int nth = rest - above(lo + 1);
                    const uint32_t hit = __ballot_sync(0xffffffffu, has && __popc(with & ((1u << lane) - 1u)) == nth);
                    c = hit ? __ffs(hit) - 1 : 0;
                    unit = lo - __shfl_sync(0xffffffffu, level, c);
                    q0 = __shfl_sync(0xffffffffu, my_q0, c);
                    q_len = __shfl_sync(0xffffffffu, my_q_len, c);
                    ctx = __shfl_sync(0xffffffffu, my_ctx, c);
                    if (!hit) unit = q_len = 0;   // a place behind the last unit
                } else {
                    // chunk by chunk, the last unit first
                    unit = p.units_per_seq - 1 - rest % p.units_per_seq;
                    c = rest / p.units_per_seq;
                    const int bad = chunk_of(c, q0, q_len, ctx);
                    if (bad && unit == 0 && lane == 0) set_status(p.dev_status, bad);
                }
                const int i0 = unit * R;
                if (i0 < q_len) {
                    QpUnit u = {};
                    u.h = h;
                    u.chunk = c;
                    u.row0 = q0 + i0;
                    u.tokens = min(R, q_len - i0);
                    u.first = ctx - q_len + i0;
                    u.wpos = max(u.first - p.window + 1, 0);
                    u.sink_pages = min((p.sinks + 15) / 16, (ctx + 15) / 16);
                    u.skip = max(u.wpos / 16 - u.sink_pages, 0);
                    u.first -= 16 * u.skip;
                    u.wpos -= 16 * u.skip;
                    u.ctx = ctx - 16 * u.skip;
                    u.tiles = (u.first + u.tokens - 1) / kQpKeys + 1;
                    if constexpr (TILES == 1) {   // the CTA's part of the key tiles: none, where there are few
                        const int all = u.tiles;
                        u.tile0 = all * rank / ranks;   // (fewer than 2^27 tiles)
                        u.tiles = all * (rank + 1) / ranks - u.tile0;
                        if (u.tiles == 0) {
                            if (lane == 0) units[0] = u;
                            break;
                        }
                    }
                    if (n >= 2) ok = wait_all(&bars->unit_empty[n & 1], (uint32_t)(n / 2 - 1));
                    if (!ok) break;
                    if (lane == 0) {
                        units[n & 1] = u;
                        tc::mbar_arrive_cta(&bars->unit_full[n & 1]);
                    }
                    // its query rows on their way to L2: they are read when the unit before is
                    // done (us with and without, 16-bit outputs: 3 x 4,000 rows 694 and 712, in
                    // fp16 742 and 770; 8 x 512 140 and 148, 157 and 162; 32-bit outputs alike.
                    // Heads of 64, whose rows are half as long, bf16 and fp16: 3 x 4,000 613 and
                    // 600, 641 and 623; 8 x 512 128 and 126, 134 and 130; 5 x 2,000 98 and 97, 103
                    // and 100)
                    if constexpr (D == 128) {
                        const int lines = p.G * (D / 64);   // of 128 bytes, of a token
                        const uint8_t *rows = static_cast<const uint8_t *>(p.q) + ((int64_t)u.row0 * p.Hq + (int64_t)h * p.G) * (D * 2);
                        for (int i = lane; i < u.tokens * lines; i += 32) {
                            const int tk = i / lines;
                            asm volatile("prefetch.global.L2 [%0];" ::"l"(rows + (int64_t)tk * p.Hq * (D * 2) + (i - tk * lines) * 128));
                        }
                    }
                    // lane i < 8 reads the block id of page i of the tile, one tile ahead
                    int blk_next = lane < kQpPages ? page_id(u, tile0(u) * kQpPages + lane) : -1;
                    for (int j = 0; ok && j < u.tiles; ++j, ++g) {
                        // the next place is asked for near the unit's end (see window_prefill.cu)
                        if (TILES == 2 && j + 2 >= u.tiles) ask();
                        const int blk = blk_next;
                        const int v = (tile0(u) + j) * kQpPages + lane;
                        if (j + 1 < u.tiles) blk_next = lane < kQpPages ? page_id(u, v + kQpPages) : -1;
                        int y = p.num_blocks * p.Hkv * 16;     // row past the pool: zero fill
                        if (lane < kQpPages && 16 * v < u.ctx) {
                            if (blk >= 0 && blk < p.num_blocks)
                                y = (blk * p.Hkv + h) * 16;
                            else
                                set_status(p.dev_status, PKV_DEV_BAD_BLOCK_ID);
                        }
                        // its scales: on their way while the slots are waited for
                        float2 sc = make_float2(1.f, 1.f);
                        if (lane < kQpPages && 16 * v < u.ctx && blk >= 0 && blk < p.num_blocks)
                            sc = __ldg(reinterpret_cast<const float2 *>(p.scales) + (int64_t)blk * p.Hkv + h);
                        const int st = (int)(g & 1);
                        uint8_t *kd = sm + Sh::OFF_K + st * Sh::CODE_TILE, *vd = sm + Sh::OFF_CODES + st * Sh::CODE_TILE;
                        // a K slot is free once both S products of its last tile are done
                        if (g >= 2) ok = wait_all(&bars->k_empty[st], g / 2 - 1);
                        if (ok) {
                            if (lane == 0) mbar_arrive_expect_tx(&bars->k_full[st], Sh::CODE_TILE);
                            __syncwarp();
                            if (lane < kQpPages) load_code_page(kd + lane * Sh::CODE_PAGE, &tk, y, &bars->k_full[st]);
                        }
                        // a slot of V's codes once they have been converted
                        if (ok && g >= 2) ok = wait_all(&bars->codes_empty[st], g / 2 - 1);
                        if (ok) {
                            if (lane == 0) mbar_arrive_expect_tx(&bars->codes_full[st], Sh::CODE_TILE);
                            __syncwarp();
                            if (lane < kQpPages) load_code_page(vd + lane * Sh::CODE_PAGE, &tv, y, &bars->codes_full[st]);
                        }
                        const int sst = (int)(g % kQpScaleStages);
                        if (ok && g >= kQpScaleStages) ok = wait_all(&bars->scales_empty[sst], g / kQpScaleStages - 1);
                        if (ok) {
                            if (lane < kQpPages) page_scales[sst * kQpPages + lane] = make_float2(sc.x, log2_approx(sc.y));
                            __syncwarp();
                            if (lane == 0) tc::mbar_arrive_cta(&bars->scales_full[sst]);
                        }
                    }
                    ++n;
                }
                if (TILES == 1 || !ok) break;   // (one query tile: every unit has its CTAs)
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
                if (asking) mbar_wait(&bars->cancel, (asked - 1) & 1u, kQpWaitNs / 8);
                for (int st = 0; st < 2; ++st) {
                    if (g > (uint32_t)st) {
                        const uint32_t last = (g - 1 - st) / 2;
                        mbar_wait(&bars->k_full[st], last & 1u, kQpWaitNs / 8);
                        mbar_wait(&bars->codes_full[st], last & 1u, kQpWaitNs / 8);
                    }
                }
            }
        } else if (warp == 1) {
            // ---------------- MMA issuer ----------------
            // One thread: it waits alone (a wait of the whole warp costs a vote and two
            // meetings, there are six a key tile, and with them this loop, not the
            // products, was what products of head_dim 64 waited for: 91 us for 81, 5
            // prompts of 2,000).  The query tiles take turns: P V of a key tile and S of
            // the next are one turn, so that a tile's softmax runs beside the other's turn.
            if (tc::elect_one()) {
                // (the query's first term is e4m3, the others e5m2; K e4m3)
                constexpr uint32_t idesc_s = tc::idesc_f8(false, false, kQpRows, kQpKeys);
                constexpr uint32_t idesc_s5 = tc::idesc_f8(true, false, kQpRows, kQpKeys);
                constexpr uint32_t idesc_o = tc::idesc_f16(false, false, true, kQpRows, D);
                auto code_desc = [&](uint32_t at) { return D == 128 ? tc::smem_desc_sw128(at, 16, 1024) : tc::smem_desc_sw64(at, 16, 512); };
                // descriptors: the upper half, and the lower one of each operand's first byte
                const uint32_t code_high = (uint32_t)(code_desc(0) >> 32);
                const uint32_t q_low = (uint32_t)code_desc(sbase + Sh::OFF_Q), k_low = (uint32_t)code_desc(sbase + Sh::OFF_K);
                const uint64_t v_desc = tc::smem_desc_sw128(sbase + Sh::OFF_V, 1024, Sh::GROUP);
                const uint32_t v_high = (uint32_t)(v_desc >> 32), v_low = (uint32_t)v_desc;
                uint32_t g = 0;     // key tiles done
                auto issue_s = [&](int t, uint32_t k) {   // S = Q K^T of query tile t and key tile k
                    if (t == 0 && !wait(&bars->k_full[k & 1], k / 2)) return false;
                    tc::fence_after_sync();
                    const uint32_t qb = q_low + ((t * Sh::Q_BYTES) >> 4), kb = k_low + (((k & 1) * Sh::CODE_TILE) >> 4);
                    constexpr int STEPS = D / 32;
#pragma unroll
                    for (int i = 0; i < Sh::TERMS * STEPS; ++i) {
                        const uint32_t qo = ((i / STEPS) * Sh::Q_TERM + (i % STEPS) * 32) >> 4, ko = ((i % STEPS) * 32) >> 4;
                        tc::mma_f8_ss(tmem + t * 256, qb + qo, kb + ko, code_high, i < STEPS ? idesc_s : idesc_s5, i > 0);
                    }
                    tc::mma_commit(&bars->s_full[t]);
                    if (t == TILES - 1) tc::mma_commit(&bars->k_empty[k & 1]);
                    return true;
                };
                for (int n = 0;; ++n) {
                    if (!wait(&bars->unit_full[n & 1], (uint32_t)(n / 2))) break;
                    const int tiles = units[n & 1].tiles;
                    tc::mbar_arrive_cta(&bars->unit_empty[n & 1]);
                    if (tiles == 0) break;
                    bool ok = true;
                    // (S may be written: the product that read P over it was issued before)
#pragma unroll
                    for (int t = 0; t < TILES; ++t) ok = ok && wait(&bars->q_full[t], (uint32_t)n) && issue_s(t, g);
                    for (int j = 0; ok && j < tiles; ++j, ++g) {
                        const uint32_t vb = v_low + (((g & 1) * Sh::TILE) >> 4);
                        ok = wait(&bars->v_full[g & 1], g / 2);
#pragma unroll
                        for (int t = 0; t < TILES; ++t) {
                            const uint32_t d_s = tmem + t * 256, d_o = d_s + 128;
#pragma unroll
                            for (int part = 0; part < 2; ++part) {
                                // P of a unit's first tile is there only after the unit before's O was read
                                ok = ok && wait(&bars->p_full[t][part], g);
                                if (!ok) break;
                                tc::fence_after_sync();
#pragma unroll
                                for (int kk = part * kQpPages / 2; kk < (part + 1) * kQpPages / 2; ++kk) {
                                    // O (+)= P V, a page at a time
                                    const uint32_t ph = d_s + 32 * (kk >> 1) + 8 * (kk & 1);
                                    const uint32_t vp = vb + (uint32_t)(kk * Sh::PAGE >> 4);
                                    tc::mma_f16_ts(d_o, ph, vp, v_high, idesc_o, j > 0 || kk > 0);
                                    tc::mma_f16_ts(d_o, ph + 16, vp, v_high, idesc_o, true);   // the weights' rounding residual
                                }
                                if (part == 0) tc::mma_commit(&bars->half_done[t]);
                            }
                            if (!ok) break;
                            if (t == TILES - 1) tc::mma_commit(&bars->v_empty[g & 1]);
                            if (j + 1 == tiles) tc::mma_commit(&bars->o_done[t]);
                            else ok = issue_s(t, g + 1);
                        }
                    }
                    if (!ok) break;
                }
            }
            __syncwarp();
        } else {
            // ---------------- V's codes to fp16 ----------------
            // A warp takes 64 rows, 8 rows x 4 pieces of 16 codes at a time, each lane a
            // piece; the rows of lanes k and k + 4 differ in their lowest and third bit,
            // so that neither the loads nor the stores meet a bank twice.
            const int piece = lane & 3, k = lane >> 2;
            const int row = (k >> 1) ^ ((k & 1) * 5);
            uint32_t g = 0;
            bool ok = true;
            QpUnit u;
            for (int n = 0; ok && take_unit(n, u); ++n) {
                for (int j = 0; ok && j < u.tiles; ++j, ++g) {
                    const int st = (int)(g & 1);
                    ok = wait_all(&bars->codes_full[st], g / 2);
                    if (g >= 2) ok = ok && wait_all(&bars->v_empty[st], g / 2 - 1);
                    if (!ok) break;
                    const uint32_t from = sbase + Sh::OFF_CODES + st * Sh::CODE_TILE;
                    const uint32_t to = sbase + Sh::OFF_V + st * Sh::TILE;
                    const WpHidden hid(u, (tile0(u) + j) * kQpKeys, p.sinks, kQpKeys);
                    const bool any = hid.any();
                    // two groups of 8 rows at a time, the next ones' codes on their way
                    uint4 codes[2][2][Sh::HALVES];
                    auto load = [&](int i) {
#pragma unroll
                        for (int e = 0; e < 2; ++e)
#pragma unroll
                            for (int hf = 0; hf < Sh::HALVES; ++hf)
                                codes[i & 1][e][hf] = lds128(from + code_piece<D>((warp - 2) * 64 + (2 * i + e) * 8 + row, 4 * hf + piece));
                    };
                    load(0);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (i < 3) load(i + 1);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int r0 = (warp - 2) * 64 + (2 * i + e) * 8;
                            const bool gone = any && hid.has(r0 + row);
#pragma unroll
                            for (int hf = 0; hf < Sh::HALVES; ++hf) {
                                uint4 c = codes[i & 1][e][hf];
                                if (any && gone) c = make_uint4(0u, 0u, 0u, 0u);
                                uint4 lo, hi;
                                e4m3x4_to_f16x4(c.x, lo.x, lo.y);
                                e4m3x4_to_f16x4(c.y, lo.z, lo.w);
                                e4m3x4_to_f16x4(c.z, hi.x, hi.y);
                                e4m3x4_to_f16x4(c.w, hi.z, hi.w);
                                const uint32_t at = to + (r0 >> 3) * Sh::GROUP + hf * 1024 + row * 128;
                                st_shared_v4(at + (((2 * piece) ^ row) << 4), lo);
                                st_shared_v4(at + (((2 * piece + 1) ^ row) << 4), hi);
                            }
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tc::mbar_arrive_cta(&bars->v_full[st]);
                        tc::mbar_arrive_cta(&bars->codes_empty[st]);
                    }
                }
            }
        }
    } else {
        tc::setmaxnreg_inc<kQpHighRegs>();
        // ---------------- softmax: tile t, one row per thread ----------------
        const int t = (warp - 4) >> 2;
        const int lane_base = 32 * (warp & 3);          // tensor-memory lanes this warp may touch
        const int r = lane_base + lane;                 // row within the tile
        const uint32_t scol = tmem + ((uint32_t)lane_base << 16) + t * 256;   // the scores, then P
        const uint32_t ocol = scol + 128;
        const int tok = t * p.rtok + r / p.G, head = r % p.G;
        // This warp's rows of the query as terms; what this thread's row has its scores
        // multiplied by.  LANES lanes take a row, eight elements each.
        auto split_query = [&](const QpUnit &u) {
            constexpr int LANES = D / 8, ROWS = 32 / LANES;    // rows at a time
            constexpr int N = 32 / ROWS;
            const int sub = lane / LANES, piece = lane % LANES;
            const uint32_t to = sbase + Sh::OFF_Q + t * Sh::Q_BYTES;
            const uint4 *from = reinterpret_cast<const uint4 *>(static_cast<const T *>(p.q) +
                                                                ((int64_t)u.row0 * p.Hq + (int64_t)u.h * p.G) * D) + piece;
            const int mine_at = r < p.G * p.rtok && tok < u.tokens ? (tok * p.Hq + head) * LANES : -1;
            uint4 x[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int at = __shfl_sync(0xffffffffu, mine_at, i * ROWS + sub);
                x[i] = make_uint4(0u, 0u, 0u, 0u);
                if (at >= 0) x[i] = __ldg(from + at);
            }
            float scale = 0.f;
            // (a loop, and the rows moved up in it: unrolled, this code, which runs once a
            // unit, takes longer to come from memory than to run: 8 x 512 rows a fifth
            // longer.  Four rows at a time or two: 140 us and 147, 3 x 4,000 694 and 706, with
            // 32-bit outputs 153 and 148, 715 and 701; others within 1 %)
            constexpr int PER = 4;
#pragma unroll 1
            for (int i0 = 0; i0 < N; i0 += PER) {
#pragma unroll
                for (int i2 = 0; i2 < PER; ++i2) {
                    const int i = i0 + i2;
                    const uint32_t w[4] = {x[i2].x, x[i2].y, x[i2].z, x[i2].w};
                    const uint32_t top2 = __vmaxu2(__vmaxu2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu),
                                                   __vmaxu2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
                    uint32_t top = max(top2 & 0xffffu, top2 >> 16);
#pragma unroll
                    for (int m = 1; m < LANES; m *= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, m));
                    const bool finite = top < (std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u);
                    const float s = block_scale(finite ? pair_to_f32<T>(top).x : 0.f, -126);
                    const float inv = __uint_as_float((254u << 23) - __float_as_uint(s));   // (s is a power of two)
                    // (a query that is not finite has no finite output)
                    const float mine = __shfl_sync(0xffffffffu, finite ? s : __uint_as_float(0x7fffffffu), (lane % ROWS) * LANES);
                    if (lane / ROWS == i) scale = mine;
                    float v[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 f = pair_to_f32<T>(w[e]);
                        v[2 * e] = f.x * inv;
                        v[2 * e + 1] = f.y * inv;
                    }
                    const int rr = lane_base + i * ROWS + sub;
                    const uint32_t at = to + code_piece<D>(rr, piece >> 1) + (piece & 1) * 8;
#pragma unroll
                    for (int term = 0; term < Sh::TERMS; ++term) {
                        uint32_t c[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            uint32_t lo, hi;
                            if (term == 0) {
                                c[e] = to_e4m3x4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
                                e4m3x4_to_f16x4(c[e], lo, hi);
                            } else {
                                c[e] = to_e5m2x4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
                                e5m2x4_to_f16x4(c[e], lo, hi);
                            }
                            const float2 fl = f16x2_to_f32(lo), fh = f16x2_to_f32(hi);
                            v[4 * e] -= fl.x;
                            v[4 * e + 1] -= fl.y;
                            v[4 * e + 2] -= fh.x;
                            v[4 * e + 3] -= fh.y;
                        }
                        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at + term * Sh::Q_TERM), "r"(c[0]), "r"(c[1]) : "memory");
                    }
                }
#pragma unroll
                for (int k = PER; k < N; ++k) x[k - PER] = x[k];
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive_cta(&bars->q_full[t]);
            return scale * p.scale_log2;
        };
        uint32_t g = 0;                                 // key tiles taken
        QpUnit u;
        bool ok = t < TILES && take_unit(0, u);
        if (TILES == 1 && t == 0 && !ok) stats[r] = make_float2(-INFINITY, 0.f);   // no key of this CTA's
        float rowscale = 0.f;
        if (ok) rowscale = split_query(u);
        for (int n = 0; ok; ++n) {
            const bool valid = r < p.G * p.rtok && tok < u.tokens;
            const int pos = u.first + (valid ? tok : u.tokens - 1);   // padding rows see the last row's keys
            float m_used = -INFINITY, l = 0.f;
            for (int j = 0; j < u.tiles; ++j, ++g) {
                const int st = (int)(g % kQpScaleStages);
                ok = wait_all(&bars->scales_full[st], g / kQpScaleStages) && wait_all(&bars->s_full[t], g);
                if (!ok) break;
                tc::fence_after_sync();
                // Half of the keys at a time, and no look for the largest y first: the code,
                // unrolled for 128 keys, does not stay in the instruction cache (a tenth
                // slower).
#pragma unroll 1
                for (int part = 0; part < 2; ++part) {
                    constexpr int kHalf = kQpKeys / 2;
                    float v[kHalf];
                    tc::tmem_ld32(scol + part * kHalf, *reinterpret_cast<float(*)[32]>(v));
                    tc::tmem_ld32(scol + part * kHalf + 32, *reinterpret_cast<float(*)[32]>(v + 32));
                    // y = v f + lb with f, lb of the key's page.  f is kept from falling to 0
                    // (rows or keys of zeros have tiny scales), where a hidden v, -infinity,
                    // would make NaN of it; |v| is below 2^25, so y moves by less than 2^-101.
                    float f[kHalf / 16], lb[kHalf / 16];
#pragma unroll
                    for (int pg = 0; pg < kHalf / 16; ++pg) {
                        const float2 sc = page_scales[(st * 2 + part) * (kHalf / 16) + pg];
                        f[pg] = fmax_nan(sc.x * rowscale, 0x1p-126f);
                        lb[pg] = sc.y;
                    }
                    tc::tmem_wait_ld();
                    // hidden: past the row's position; below its window and behind the first tokens
                    const int key0 = (tile0(u) + j) * kQpKeys + part * kHalf;
                    const int lim = pos - key0, low = lim - p.window + 1, sk = p.sinks - key0;
                    if (__any_sync(0xffffffffu, lim < kHalf - 1 || (low > 0 && sk < kHalf))) {
                        auto below = [](int n) { return n >= 32 ? 0xffffffffu : (n <= 0 ? 0u : (1u << n) - 1u); };
#pragma unroll
                        for (int cc = 0; cc < kHalf; cc += 32) {
                            const uint32_t see = below(lim + 1 - cc) & (~below(low - cc) | below(sk - cc));
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!(see & (1u << e))) v[cc + e] = -INFINITY;
                        }
                    }
                    // A row that has no maximum yet takes this half's (O has not been
                    // written for it, or only with weights of 0).  Others go on with the
                    // one they have, and look whether it still serves by the sums of P: a
                    // page's sum of at most 2^15 has no weight above.
                    bool raise = m_used == -INFINITY;
                    float sum = 0.f;
#pragma unroll 1
                    for (int go = 0; go < 2; ++go) {   // (raised to the largest y there is, it serves)
                        if (__any_sync(0xffffffffu, raise)) {
                            // m_used becomes the largest y so far; O and l follow.  O was last
                            // written by the P V product of the tile before, which the tensor
                            // core finished before this tile's S (issued after it) completed,
                            // or by the first half's
                            if (part == 1) ok = wait_all(&bars->half_done[t], g);
                            if (!ok) break;
                            tc::fence_after_sync();
                            float mx = m_used;
#pragma unroll
                            for (int pg = 0; pg < kHalf / 16; ++pg) {
                                float a = fmaxf(v[16 * pg], v[16 * pg + 1]), b = fmaxf(v[16 * pg + 2], v[16 * pg + 3]);
#pragma unroll
                                for (int e = 4; e < 16; e += 4) {
                                    a = fmax3(a, v[16 * pg + e], v[16 * pg + e + 1]);
                                    b = fmax3(b, v[16 * pg + e + 2], v[16 * pg + e + 3]);
                                }
                                mx = fmaxf(mx, fmaf(fmaxf(a, b), f[pg], lb[pg]));   // (f > 0)
                            }
                            const float alpha = raise && m_used > -INFINITY ? exp2_approx(m_used - mx) : 1.f;
                            if (raise) m_used = mx;
                            l *= alpha;
                            if (__any_sync(0xffffffffu, alpha != 1.f)) {
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
                        }
                        // P = 2^(y - m_used + 7) over the same columns, a page at a time: 8
                        // columns of rounded pairs (and 16 further 8 of residual pairs).
                        // (A row that has seen no key yet has nothing to subtract.)
                        const float off = (m_used == -INFINITY ? 0.f : m_used) - 7.f;
                        float top = 0.f;
                        sum = 0.f;
#pragma unroll
                        for (int pg = 0; pg < kHalf / 16; ++pg) {
                            const float c = lb[pg] - off;
                            const uint64_t f2 = f2_pack(f[pg], f[pg]), c2 = f2_pack(c, c);
                            uint64_t sum2 = f2_pack(0.f, 0.f);
                            uint32_t hi[8], lo[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                float a, b;
                                f2_unpack(f2_fma(f2_pack(v[16 * pg + 2 * e], v[16 * pg + 2 * e + 1]), f2, c2), a, b);
                                a = exp2_approx(a);
                                b = exp2_approx(b);
                                const uint64_t ab = f2_pack(a, b);
                                sum2 = f2_add(sum2, ab);
                                pack2_split2<__half>(ab, a, b, hi[e], lo[e]);
                            }
                            float s0, s1;
                            f2_unpack(sum2, s0, s1);
                            s0 += s1;
                            top = fmaxf(top, s0);
                            sum = fmaf(s0, exp2_approx(-lb[pg]), sum);
                            const uint32_t to = scol + part * kHalf + 32 * (pg >> 1) + 8 * (pg & 1);
                            tc::tmem_st8(to, hi);
                            tc::tmem_st8(to + 16, lo);
                        }
                        raise = top > 32768.f;
                        if (!__any_sync(0xffffffffu, raise)) break;
                        tc::tmem_wait_st();   // (stores to the same columns need not keep their order)
                    }
                    if (!ok) break;
                    l += sum;
                    tc::tmem_wait_st();   // a part of P is ready
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive_cta(&bars->p_full[t][part]);
                }
                if (!ok) break;
                if (lane == 0) tc::mbar_arrive_cta(&bars->scales_empty[st]);
            }
            if (!ok) break;
            // the next unit's query: this one's S products are done
            QpUnit u_next;
            bool more = false;
            float rowscale_next = 0.f;
            if constexpr (Sh::OWN_OUT) {
                more = take_unit(n + 1, u_next);
                if (more) rowscale_next = split_query(u_next);
            }
            ok = wait_all(&bars->o_done[t], (uint32_t)n);
            if (!ok) break;
            tc::fence_after_sync();
            if (TILES == 1 && ranks > 1) {
                stats[r] = make_float2(m_used, l);
                break;
            }
            const float inv = 1.f / l;
            // 128 bytes of each row at a time, through shared memory (see window_prefill.cu)
            constexpr int kCols = WIDE ? 32 : 64;      // a 32-bit output or a 16-bit one
            constexpr int kSize = WIDE ? 4 : 2;
            const int64_t at = valid ? ((int64_t)(u.row0 + tok) * p.Hq + (int64_t)u.h * p.G + head) * D * kSize : -1;
            uint8_t *stage = Sh::OWN_OUT ? sm + Sh::OFF_OUT + (warp - 4) * 4096
                                         : sm + Sh::OFF_Q + t * Sh::Q_BYTES + (warp & 3) * 4096;
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
            if constexpr (!Sh::OWN_OUT) {
                more = take_unit(n + 1, u_next);
                if (lane == 0) stores_read();
                __syncwarp();
                if (more) rowscale_next = split_query(u_next);
            }
            if (!more) break;
            u = u_next;
            rowscale = rowscale_next;
        }
        if (lane == 0) stores_done();
        if constexpr (TILES == 1) {
            if (ranks > 1) {
                // ---- the parts of a unit: each CTA brings its O to the row's largest m and
                // total l, and sums a slice of the rows over the CTAs, in their order ----
                __syncwarp();
                cluster_sync();
                const int tokens = units[0].tokens, row0 = units[0].row0, h = units[0].h;
                float *part = reinterpret_cast<float *>(sm + Sh::OFF_V);
                if (t == 0 && units[0].tiles > 0) {
                    float m = -INFINITY, total = 0.f;
                    for (int c = 0; c < ranks; ++c) m = fmaxf(m, ld_cluster_f32x2(cluster_addr(stats + r, c)).x);
                    for (int c = 0; c < ranks; ++c) {
                        const float2 s = ld_cluster_f32x2(cluster_addr(stats + r, c));
                        total = fmaf(s.y, exp2_approx(s.x - m), total);
                    }
                    // (a query that is not finite has no m, and NaN for its weight)
                    const float w = exp2_approx(stats[r].x - m) / total;
#pragma unroll 1
                    for (int cc = 0; cc < D; cc += 32) {
                        float o[32];
                        tc::tmem_ld32(ocol + cc, o);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            *reinterpret_cast<float4 *>(part + r * D + (((cc / 4 + e) ^ (r & 7)) << 2)) =
                                make_float4(o[4 * e] * w, o[4 * e + 1] * w, o[4 * e + 2] * w, o[4 * e + 3] * w);
                    }
                }
                __syncwarp();
                cluster_sync();
                constexpr int LANES = D / 4, ROWS = 32 / LANES;   // lanes a row, rows a warp at a time
                const int end = kQpRows * (rank + 1) / ranks;
#pragma unroll 1
                for (int row = kQpRows * rank / ranks + (warp - 4) * ROWS + lane / LANES; row < end; row += 8 * ROWS) {
                    const int tk = row / p.G, col = (lane % LANES) * 4;
                    if (row >= p.G * p.rtok || tk >= tokens) continue;
                    float m = -INFINITY;
                    for (int c = 0; c < ranks; ++c) m = fmaxf(m, ld_cluster_f32x2(cluster_addr(stats + row, c)).x);
                    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int c = 0; c < ranks; ++c) {
                        // (where a CTA saw no key of the row's, nothing may be there)
                        if (ld_cluster_f32x2(cluster_addr(stats + row, c)).x == -INFINITY && m > -INFINITY) continue;
                        const float4 x = ld_cluster_f32x4(cluster_addr(part + row * D + (((col >> 2) ^ (row & 7)) << 2), c));
                        sum.x += x.x;
                        sum.y += x.y;
                        sum.z += x.z;
                        sum.w += x.w;
                    }
                    const int64_t at = ((int64_t)(row0 + tk) * p.Hq + (int64_t)h * p.G + row % p.G) * D + col;
                    if constexpr (WIDE)
                        *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at) = sum;
                    else
                        *reinterpret_cast<uint2 *>(static_cast<T *>(p.out) + at) = make_uint2(pack2<T>(sum.x, sum.y), pack2<T>(sum.z, sum.w));
                }
            }
        }
    }
    if constexpr (TILES == 1) {
        // (and a CTA's shared memory outlives its readers)
        __syncwarp();
        if (ranks > 1) {
            if (warp < 4) {
                cluster_sync();
                cluster_sync();
            }
            cluster_sync();
        }
    }

    tc::fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, kQpTmemCols);
    }
}

// A cache of codes as rows of head_dim bytes, a (block, KV head) page of 16 a box.
// Rows past the pool read 0.
static int encode_code_page_map(CUtensorMap *map, const void *base, int num_blocks, int num_kv_heads, int head_dim) {
    const uint64_t dims[2] = {(uint64_t)head_dim / 2, (uint64_t)num_blocks * num_kv_heads * 16};   // in 16-bit elements
    const uint64_t strides[1] = {(uint64_t)head_dim};
    const uint32_t box[2] = {(uint32_t)head_dim / 2, 16};
    return encode_tiled_map(map, base, 2, dims, strides, box, head_dim);
}

template <typename T, int D, bool WIDE, int TILES>
static int launch_quant_prefill(const QuantPrefillParams &prm, const CUtensorMap &tk, const CUtensorMap &tv,
                                const CUtensorMap &tout, int grid, int ranks, cudaStream_t stream) {
    using Sh = QpShape<T, D>;
    const auto kernel = quant_prefill_kernel<T, D, WIDE, TILES>;
    // the register split inside the kernel waits for registers that only exist
    // if the compiled count is the one it was sized for: check it (once; the
    // answer does not change) and refuse to launch otherwise
    static int regs_ok = 0;   // 0 unknown, 1 as sized, -1 not
    if (regs_ok == 0) {
        cudaFuncAttributes fa;
        cudaError_t e = cudaFuncGetAttributes(&fa, kernel);
        if (e != cudaSuccess) return cuda_fail(e);
        regs_ok = fa.numRegs == kQpLaunchRegs ? 1 : -1;
        if (regs_ok < 0) {
            char msg[128];
            std::snprintf(msg, sizeof msg, "8-bit prefill kernel compiled to %d registers per thread, its split needs %d",
                          fa.numRegs, kQpLaunchRegs);
            set_error_message(msg);
        }
    }
    if (regs_ok < 0) return PKV_ERR_UNSUPPORTED;
    static unsigned long long attr_set = 0;   // per instantiation and device
    if (!done_on_device(&attr_set)) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::SMEM_BYTES);
        if (e != cudaSuccess) return cuda_fail(e);
        mark_done_on_device(&attr_set);
    }
    cudaError_t e;
    if constexpr (TILES == 1)
        e = launch_cluster(kernel, grid * ranks, ranks, kQpThreads, Sh::SMEM_BYTES, stream, prm, tk, tv, tout);
    else
        e = launch_pdl(kernel, dim3(grid), dim3(kQpThreads), Sh::SMEM_BYTES, stream, prm, tk, tv, tout);
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? PKV_OK : cuda_fail(e);
}

}  // namespace pkv

extern "C" int pkv_paged_prefill_attention_e4m3(void *out, const void *q, const int32_t *cu_seqlens, int num_seqs, int max_q_len,
                                                int total_q, const void *k_cache, const void *v_cache, const float *kv_scales,
                                                const int32_t *block_tables, int max_blocks_per_seq,
                                                const int32_t *context_lens, int num_blocks, int num_q_heads, int num_kv_heads,
                                                int head_dim, int block_size, int window, int num_sinks, float scale, int dtype,
                                                int out_dtype, int *dev_status, void *stream) {
    pkv::NvtxRange nvtx_range("pkv_paged_prefill_attention_e4m3");
    using namespace pkv;
    if (max_q_len < 0 || total_q < 0) return PKV_ERR_INVALID_ARG;
    int rc = quant_attention_refusal(num_seqs, num_blocks, num_q_heads, num_kv_heads, head_dim, block_size, max_blocks_per_seq,
                                     window, num_sinks, scale, dtype, out_dtype);
    if (rc != PKV_OK) return rc;
    if (num_seqs == 0 || max_q_len == 0 || total_q == 0) return PKV_OK;
    if (!out || !q || !cu_seqlens || !k_cache || !v_cache || !kv_scales || !block_tables || !context_lens)
        return PKV_ERR_INVALID_ARG;
    // query rows are read and output rows stored as 16-byte vectors
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(kv_scales, 8) ||
        !aligned(cu_seqlens, 4) || !aligned(block_tables, 4) || !aligned(context_lens, 4))
        return PKV_ERR_INVALID_ARG;
    int sms = 0;
    rc = current_sm_count(&sms);
    if (rc != PKV_OK) return rc;
    const int G = num_q_heads / num_kv_heads;
    const int rtok = kQpRows / G;
    // query tiles of a unit: two, which share every K and V tile; or one, when
    // all units then run at once and a step of 128 keys has one tile's products
    const int most_q = std::min(max_q_len, total_q);   // rows that a chunk can have
    auto units_of = [&](int tiles) { return ((int64_t)most_q + tiles * rtok - 1) / (tiles * rtok); };
    const bool one = num_seqs * units_of(1) * num_kv_heads <= sms;
    const int qtiles = one ? 1 : 2;
    int64_t grid = (int64_t)num_seqs * units_of(qtiles) * num_kv_heads;
    if (grid >= (int64_t)1 << 31) return PKV_ERR_UNSUPPORTED;
    // where most SMs would have none, a unit's keys go to the CTAs of a cluster,
    // two key tiles each or more if contexts fill their tables
    const int64_t capacity = (int64_t)max_blocks_per_seq * 16;
    const int64_t keys = window < capacity && num_sinks < capacity - window ? (int64_t)window + num_sinks + max_q_len : capacity;
    int ranks = 1;
    while (one && ranks < 8 && grid * ranks * 2 <= sms && ranks * 2 * 2 * kQpKeys <= keys) ranks *= 2;
    CUtensorMap tk, tv;
    rc = encode_code_page_map(&tk, k_cache, num_blocks, num_kv_heads, head_dim);
    if (rc != PKV_OK) return rc;
    rc = encode_code_page_map(&tv, v_cache, num_blocks, num_kv_heads, head_dim);
    if (rc != PKV_OK) return rc;
    QuantPrefillParams prm;
    prm.boxes = out_dtype == dtype && 32 % G == 0;
    CUtensorMap tout = tk;
    if (prm.boxes) {
        const uint64_t dims[3] = {(uint64_t)head_dim, (uint64_t)num_q_heads, (uint64_t)total_q};
        const uint64_t strides[2] = {(uint64_t)head_dim * 2, (uint64_t)num_q_heads * head_dim * 2};
        const uint32_t rows[3] = {64, (uint32_t)G, 32u / (uint32_t)G};
        rc = encode_tiled_map(&tout, out, 3, dims, strides, rows);
        if (rc != PKV_OK) return rc;
    }
    prm.out = out;
    prm.q = q;
    prm.scales = kv_scales;
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
    prm.num_seqs = num_seqs;
    prm.units_per_seq = (int)units_of(qtiles);
    prm.sorted = num_seqs <= 32 && grid > sms;
    // sorted units leave no place empty between them: as many places as total_q rows
    // in num_seqs chunks can make units
    if (prm.sorted) grid = std::min(grid, ((int64_t)total_q / (qtiles * rtok) + num_seqs) * num_kv_heads);
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
        return head_dim == 128 ? launch_quant_prefill<T, 128, W, N>(prm, tk, tv, tout, (int)grid, ranks, st)
                               : launch_quant_prefill<T, 64, W, N>(prm, tk, tv, tout, (int)grid, ranks, st);
    };
    auto typed = [&](auto type) {
        std::integral_constant<int, 1> tile;
        std::integral_constant<int, 2> tiles;
        if (out_dtype == PKV_DTYPE_F32) return one ? launch(type, std::true_type(), tile) : launch(type, std::true_type(), tiles);
        return one ? launch(type, std::false_type(), tile) : launch(type, std::false_type(), tiles);
    };
    return dtype == PKV_DTYPE_BF16 ? typed(__nv_bfloat16()) : typed(__half());
}
