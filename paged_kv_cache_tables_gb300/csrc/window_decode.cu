// Decode attention over a sliding window and the first tokens of a paged
// context (pkv_paged_window_decode_attention).
//
// Mathematics.  The query of sequence s sits at position p = ctx_s - 1 and
// sees position t iff t <= p and (t > p - window or t < sinks):
//     out = sum_t softmax_t(scale * q . K_t) V_t  over those t,
// taken a few blocks at a time with the running maximum m and sum l of the
// softmax in fp32: their scores x give m' = max(m, x), weights 2^(x - m'), and
// l and the accumulator are scaled by 2^(m - m') (m is left alone until it
// grows by more than 2^8).  Parts of a range combine the same
// way: with M = max m_i, out = sum acc_i 2^(m_i - M) / sum l_i 2^(m_i - M).
//
// What is read.  Only blocks that hold a visible position: the blocks of the
// first tokens, then those from the window's first block on.  They form one
// list of `visible` blocks, in which entry v stands for logical block v, or
// v + skip past the first tokens' blocks.  Table entries between may be
// anything (blocks released to the pool).
//
// One cluster of CTAs takes a (sequence, KV head) range, each CTA an equal
// run of its visible blocks, the warps of a CTA every fourth one.  A warp runs
// its own ring of shared-memory slots: lane 0 issues the TMA loads of a
// block's K and V tiles (128-byte swizzle), the warp pulls both into MMA
// fragments, hands the slot back and computes S = Q K^T and O^T += V^T P^T
// with the query heads of the group as one (padded) row tile.  The warps'
// parts meet in shared memory, the CTAs' parts through distributed shared
// memory, so there is no workspace, no second launch, and the order of every
// sum is fixed by the call's sizes (which choose the split) and the lengths.
//
// What bounds it: HBM.  256 sequences x 8 KV heads, window 1,024 (597 MB of
// visible K and V): 90.6 us, 97 % of the measured copy rate; 16 x 8, window
// 8,000: 78.7 us, 98 %; 7 x 8 of it 37.4 us, 91 % (5 CTAs a range fill 280 of
// 304 places).  Small calls are a chain of latencies (launch, length, table
// entry, tile, products, cluster): 3 to 5 us.  Measured and left: persistent
// CTAs of 8 warps that stream from range to range, ranges taken by cluster
// launch control: 122 us for the 256 sequences, since what a CTA holds ahead it
// holds back from idle SMs at the end, and what it does not hold ahead it waits
// for.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "pkv.h"
#include "pkv_cluster.cuh"
#include "pkv_device.cuh"
#include "pkv_host.h"
#include "pkv_window.cuh"

namespace pkv {

constexpr int kWinWarps = 4;
constexpr int kWinMaxCluster = 16;
constexpr uint64_t kWinWaitNs = 2000000000ull;   // a tile that has not landed in 2 s never will

struct WindowDecodeParams {
    void *out;
    const void *q;
    const int32_t *block_tables;
    const int32_t *context_lens;
    int *dev_status;
    int max_blocks, num_blocks, Hq, Hkv, G;
    int window, sinks;
    float scale_log2;   // scale * log2(e): scores in base-2 units
    int out_dtype;
};

// Two forms.  FEW, for ranges that all fit on the GPU at once (split over
// clusters): long rings, two blocks a step, since a warp's time for a block is
// a chain of latencies that two share.  MANY, for more ranges: three CTAs an SM
// with shorter rings and one block a step, so that CTAs that start and end
// hide behind one that streams.  us, FEW / MANY: 256 sequences x 8 heads of up
// to 65 blocks 94.0 / 91.4, of up to 9 blocks 39.7 / 33.1; 200 x 2 of up to 20
// 14.8 / 11.8; one wave: 7 x 8 of 505 blocks 37.8 / 42.6, 32 x 8 of 33 14.4 / 15.3.
// Groups above 8 heads are built as FEW alone: 256 sequences x 2 heads of 65 blocks
// 39.5 us (visible bytes 22.6), 1,024 113 (90.2), 1,024 of 9 blocks 62 (20.4).
template <int D, bool MANY>
struct WindowShape {
    static constexpr int HALVES = D / 64;               // 64-element (128-byte) column halves
    static constexpr int HALF_BYTES = 64 * 16 * 2;
    static constexpr int TILE_BYTES = HALVES * HALF_BYTES;
    static constexpr int STAGE_BYTES = 2 * TILE_BYTES;  // K then V
    static constexpr int STAGES = D == 128 ? (MANY ? 2 : 3) : 4;
    static constexpr int STEP = MANY ? 1 : 2;           // blocks a warp takes at a time
    static constexpr int PER_SM = D == 128 && !MANY ? 2 : 3;
    static constexpr int RING_BYTES = kWinWarps * STAGES * STAGE_BYTES;
    // behind the ring: barriers, then (m, l) of each warp and of the CTA
    static constexpr int OFF_ML = RING_BYTES + kWinWarps * STAGES * 8;
    static constexpr int SMEM_BYTES = 1024 + OFF_ML + (kWinWarps + 1) * 32 * 4;
};

// Issues the TMA loads of block `blk`'s K and V tiles of KV head h into a ring
// slot (one lane).
template <int D, bool MANY>
__device__ __forceinline__ void issue_block(const WindowDecodeParams &p, const CUtensorMap *tk, const CUtensorMap *tv,
                                            uint8_t *slot, uint64_t *bar, int blk, int h, uint64_t policy) {
    using Sh = WindowShape<D, MANY>;
    const bool bad_blk = blk < 0 || blk >= p.num_blocks;
    if (bad_blk) set_status(p.dev_status, PKV_DEV_BAD_BLOCK_ID);
    // past the end for a bad block id: the load fills zeros
    const int y = bad_blk ? p.num_blocks * p.Hkv * 16 : (blk * p.Hkv + h) * 16;
    mbar_arrive_expect_tx(bar, Sh::STAGE_BYTES);
#pragma unroll
    for (int hf = 0; hf < Sh::HALVES; ++hf) {
        tma_load_2d(slot + hf * Sh::HALF_BYTES, tk, hf * 64, y, bar, policy);
        tma_load_2d(slot + Sh::TILE_BYTES + hf * Sh::HALF_BYTES, tv, hf * 64, y, bar, policy);
    }
}

// A warp's part of a range: query fragments (rows = heads of the group, padded
// to 16), accumulator, running maximum and sum.
template <typename T, int D, int NT, bool MANY>
struct WarpPart {
    using Sh = WindowShape<D, MANY>;
    static constexpr int STEP = Sh::STEP;
    uint32_t qa[D / 16][4];
    float acc[D / 16][NT][4];
    float m_run[NT], l_run[NT];

    // q: G rows of D elements
    __device__ __forceinline__ void start(const uint32_t *q, int G, int lane) {
        const int g = lane >> 2, t4 = lane & 3;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const int c0 = (kk * 16 + 2 * t4) >> 1;
            qa[kk][0] = g < G ? q[g * (D / 2) + c0] : 0u;
            qa[kk][2] = g < G ? q[g * (D / 2) + c0 + 4] : 0u;
            if constexpr (NT == 1) {   // group of at most 8 heads: rows 8..15 are padding
                qa[kk][1] = 0u;
                qa[kk][3] = 0u;
            } else {
                qa[kk][1] = g + 8 < G ? q[(g + 8) * (D / 2) + c0] : 0u;
                qa[kk][3] = g + 8 < G ? q[(g + 8) * (D / 2) + c0 + 4] : 0u;
            }
        }
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
            for (int pn = 0; pn < NT; ++pn)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[mt][pn][e] = 0.f;
#pragma unroll
        for (int pn = 0; pn < NT; ++pn) {
            m_run[pn] = -INFINITY;
            l_run[pn] = 0.f;
        }
    }

    // STEP blocks of 16 tokens in ring slots at `slot`, bit t of `bits` set
    // where token t of them is seen (some token of the first block is).
    // `release` runs once the slots have been read.
    template <typename F>
    __device__ __forceinline__ void attend(const uint32_t (&slot)[STEP], uint32_t bits, float scale_log2, int lane,
                                           F release) {
        const int t4 = lane & 3, mi = lane >> 3;
        const int row = ((mi >> 1) << 3) + (lane & 7);   // token row this lane addresses
        const int sw = row & 7;                           // 128-byte swizzle phase of that row
        auto at = [&](int kk) {
            const int chunk = ((kk & 3) << 1) + (mi & 1);
            return (uint32_t)((kk >> 2) * Sh::HALF_BYTES + row * 128 + ((chunk ^ sw) << 4));
        };
        // S = Q K^T, two chains per 8-token tile
        float s0[2 * STEP][4], s1[2 * STEP][4];
#pragma unroll
        for (int nt = 0; nt < 2 * STEP; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s0[nt][e] = s1[nt][e] = 0.f;
#pragma unroll
        for (int b = 0; b < STEP; ++b) {
            uint32_t kf[D / 16][4];
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) ldsm_x4(slot[b] + at(kk), kf[kk][0], kf[kk][1], kf[kk][2], kf[kk][3]);
#pragma unroll
            for (int kk = 0; kk < D / 16; kk += 2) {
                mma_16816<T>(s0[2 * b], qa[kk], kf[kk][0], kf[kk][1]);
                mma_16816<T>(s0[2 * b + 1], qa[kk], kf[kk][2], kf[kk][3]);
                mma_16816<T>(s1[2 * b], qa[kk + 1], kf[kk + 1][0], kf[kk + 1][1]);
                mma_16816<T>(s1[2 * b + 1], qa[kk + 1], kf[kk + 1][2], kf[kk + 1][3]);
            }
        }
        uint32_t vf[STEP][D / 16][4];
#pragma unroll
        for (int b = 0; b < STEP; ++b)
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
                ldsm_x4_t(slot[b] + Sh::TILE_BYTES + at(kk), vf[b][kk][0], vf[b][kk][1], vf[b][kk][2], vf[b][kk][3]);
        release();

        float pr[2 * STEP][2 * NT];
        float alpha[NT];
        bool moved = false;
#pragma unroll
        for (int pn = 0; pn < NT; ++pn) {
            float x[2 * STEP][2];
            float mx = -INFINITY;
#pragma unroll
            for (int nt = 0; nt < 2 * STEP; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float v = (s0[nt][pn * 2 + e] + s1[nt][pn * 2 + e]) * scale_log2;
                    x[nt][e] = (bits >> (nt * 8 + 2 * t4 + e)) & 1u ? v : -INFINITY;
                    mx = fmaxf(mx, x[nt][e]);
                }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            // the maximum is only moved when it grows by more than 2^8
            const bool move = m_run[pn] == -INFINITY || mx > m_run[pn] + 8.f;
            const float m_new = move ? fmaxf(m_run[pn], mx) : m_run[pn];
            // no finite score so far (keys of infinities): nothing to subtract
            const float sub = m_new == -INFINITY ? 0.f : m_new;
            alpha[pn] = move ? exp2_approx(m_run[pn] - sub) : 1.f;
            moved |= move;
            m_run[pn] = m_new;
            float rs = 0.f;
#pragma unroll
            for (int nt = 0; nt < 2 * STEP; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    pr[nt][pn * 2 + e] = exp2_approx(x[nt][e] - sub);
                    rs += pr[nt][pn * 2 + e];
                }
            l_run[pn] = l_run[pn] * alpha[pn] + rs;
        }
        // hidden positions may hold anything (even NaN): clear their V values
        // in the fragments, so that 0 x garbage cannot reach the accumulator.
        // Registers 0/1 hold tokens 2 t4 (low half) and 2 t4 + 1, 2/3 the same
        // tokens + 8.
        if (bits != (uint32_t)((1ull << (16 * STEP)) - 1u)) {
#pragma unroll
            for (int b = 0; b < STEP; ++b) {
                const uint32_t w = bits >> (16 * b + 2 * t4);
                const uint32_t m01 = (w & 1u ? 0x0000ffffu : 0u) | (w & 2u ? 0xffff0000u : 0u);
                const uint32_t m23 = (w & 0x100u ? 0x0000ffffu : 0u) | (w & 0x200u ? 0xffff0000u : 0u);
#pragma unroll
                for (int mt = 0; mt < D / 16; ++mt) {
                    vf[b][mt][0] &= m01;
                    vf[b][mt][1] &= m01;
                    vf[b][mt][2] &= m23;
                    vf[b][mt][3] &= m23;
                }
            }
        }
        if (__any_sync(0xffffffffu, moved))
#pragma unroll
            for (int pn = 0; pn < NT; ++pn) {
                const float a_lo = __shfl_sync(0xffffffffu, alpha[pn], 8 * t4);
                const float a_hi = __shfl_sync(0xffffffffu, alpha[pn], 8 * t4 + 4);
#pragma unroll
                for (int mt = 0; mt < D / 16; ++mt) {
                    acc[mt][pn][0] *= a_lo;
                    acc[mt][pn][1] *= a_hi;
                    acc[mt][pn][2] *= a_lo;
                    acc[mt][pn][3] *= a_hi;
                }
            }
        // O^T += V^T P^T, P as a rounded 16-bit value and its rounding
        // residual: the weights keep about 16 significant bits
#pragma unroll
        for (int b = 0; b < STEP; ++b) {
            uint32_t pb0[NT][2], pb1[NT][2];
#pragma unroll
            for (int pn = 0; pn < NT; ++pn) {
                pack2_split<T>(pr[2 * b][pn * 2], pr[2 * b][pn * 2 + 1], pb0[pn][0], pb0[pn][1]);
                pack2_split<T>(pr[2 * b + 1][pn * 2], pr[2 * b + 1][pn * 2 + 1], pb1[pn][0], pb1[pn][1]);
            }
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
                    for (int pn = 0; pn < NT; ++pn) mma_16816<T>(acc[mt][pn], vf[b][mt], pb0[pn][r], pb1[pn][r]);
        }
    }

    // The rows' sums over their lanes; lane t4 == 0 of row g then holds row
    // 8 pn + g's in l_run[pn].
    __device__ __forceinline__ void finish() {
#pragma unroll
        for (int pn = 0; pn < NT; ++pn) {
            l_run[pn] += __shfl_xor_sync(0xffffffffu, l_run[pn], 1);
            l_run[pn] += __shfl_xor_sync(0xffffffffu, l_run[pn], 2);
        }
    }

    // (m, l) of the heads at ml[head], ml[16 + head]; accumulators at part[head * D + d].
    __device__ __forceinline__ void store(float *ml, float *part, int G, int lane) const {
        const int g = lane >> 2, t4 = lane & 3;
#pragma unroll
        for (int pn = 0; pn < NT; ++pn) {
            if (t4 == 0) {
                ml[pn * 8 + g] = m_run[pn];
                ml[16 + pn * 8 + g] = l_run[pn];
            }
            const int ha = pn * 8 + 2 * t4, hb = ha + 1;
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt) {
                const int d0 = mt * 16 + g;
                if (ha < G) {
                    part[ha * D + d0] = acc[mt][pn][0];
                    part[ha * D + d0 + 8] = acc[mt][pn][2];
                }
                if (hb < G) {
                    part[hb * D + d0] = acc[mt][pn][1];
                    part[hb * D + d0 + 8] = acc[mt][pn][3];
                }
            }
        }
    }
};

template <typename T, int D, int NT, bool MANY>
__global__ void __launch_bounds__(kWinWarps * 32, NT == 1 ? WindowShape<D, MANY>::PER_SM : 2)
    window_decode_kernel(const WindowDecodeParams p, const __grid_constant__ CUtensorMap tk,
                         const __grid_constant__ CUtensorMap tv) {
    using Sh = WindowShape<D, MANY>;
    constexpr int STAGES = Sh::STAGES, STEP = Sh::STEP;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Sh::RING_BYTES);
    float *ml = reinterpret_cast<float *>(smem + Sh::OFF_ML);   // [warp][m 16, l 16], then the CTA's
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = (int)cluster_ctarank(), ranks = (int)cluster_nctarank();
    const int range = blockIdx.x / ranks;
    const int G = p.G, s = range / p.Hkv, h = range - s * p.Hkv;

    uint8_t *wring = smem + warp * STAGES * Sh::STAGE_BYTES;
    uint64_t *wbar = bars + warp * STAGES;
    if (lane == 0) {
        for (int st = 0; st < STAGES; ++st) mbar_init(&wbar[st], 1);
        fence_mbar_init();
        if (warp == 0) {
            prefetch_tensormap(&tk);
            prefetch_tensormap(&tv);
        }
    }
    __syncwarp();
    pdl_wait_primary();
    pdl_launch_dependents();

    // ---- the range's visible blocks, and this warp's share ----
    const Visible vis(p, __ldg(p.context_lens + s));
    if (vis.bad && tid == 0 && rank == 0 && h == 0) set_status(p.dev_status, PKV_DEV_BAD_CONTEXT);
    const int v_lo = (int)((int64_t)vis.count * rank / ranks), v_hi = (int)((int64_t)vis.count * (rank + 1) / ranks);
    const int n = max(0, (v_hi - v_lo - warp + kWinWarps - 1) / kWinWarps);
    auto logical = [&](int i) { return vis.logical(v_lo + warp + kWinWarps * i); };
    const int32_t *row = p.block_tables + (int64_t)s * p.max_blocks;
    int ids = lane < n ? __ldg(row + logical(lane)) : 0;     // lane i: the id of this warp's block 32 k + i
    const uint64_t policy = l2_policy_evict_first();
    auto issue = [&](int i) {
        const int blk = __shfl_sync(0xffffffffu, ids, i & 31);
        if (lane == 0)
            issue_block<D, MANY>(p, &tk, &tv, wring + (i % STAGES) * Sh::STAGE_BYTES, &wbar[i % STAGES], blk, h, policy);
    };
    int issued = 0;
    for (; issued < min(n, STAGES); ++issued) issue(issued);

    WarpPart<T, D, NT, MANY> part_w;
    part_w.start(reinterpret_cast<const uint32_t *>(static_cast<const T *>(p.q) + ((int64_t)s * p.Hq + (int64_t)h * G) * D),
                 G, lane);
    const uint32_t ring_addr = smem_addr(wring);

    bool timed_out = false;
    int i = 0;   // blocks taken
    while (i < n) {
        // an odd block out is taken with itself, the second time all hidden
        const int k = min(STEP, n - i);
        uint32_t slot[STEP], bits = 0;
        bool ok = true;
#pragma unroll
        for (int b = 0; b < STEP; ++b) {
            const int x = i + min(b, k - 1);
            ok = ok && mbar_wait(&wbar[x % STAGES], (uint32_t)(x / STAGES) & 1u, kWinWaitNs);
            slot[b] = ring_addr + (x % STAGES) * Sh::STAGE_BYTES;
            if (b < k) bits |= vis.bits(logical(x), p.sinks) << (16 * b);
        }
        if (!__all_sync(0xffffffffu, ok)) {
            timed_out = true;
            break;
        }
        i += k;
        part_w.attend(slot, bits, p.scale_log2, lane, [&] {
            fence_proxy_async_smem();
            __syncwarp();
            for (int u = 0; u < k && issued < n; ++u, ++issued) {
                if ((issued & 31) == 0) ids = issued + lane < n ? __ldg(row + logical(issued + lane)) : 0;
                issue(issued);
            }
        });
    }
    if (timed_out) {
        if (lane == 0) set_status(p.dev_status, PKV_DEV_WAIT_TIMEOUT);
        // what is still in flight must land before the ring is used again
        for (int k = i; k < issued; ++k) mbar_wait(&wbar[k % STAGES], (uint32_t)(k / STAGES) & 1u, kWinWaitNs / 8);
    }

    // ---- the warps' parts: (m, l) per head, accumulators [warp][head][d] over the ring ----
    __syncthreads();   // every warp is done with its slots
    float *part = reinterpret_cast<float *>(smem);
    const int GD = G * D;
    part_w.finish();
    part_w.store(ml + warp * 32, part + warp * GD, G, lane);
    __syncthreads();
    float *comb = part + kWinWarps * GD;   // the CTA's accumulators, unnormalised
    float *cml = ml + kWinWarps * 32;
    const int64_t ob = ((int64_t)s * p.Hq + (int64_t)h * G) * D;
    for (int e = tid; e < GD; e += kWinWarps * 32) {
        const int hh = e / D;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWinWarps; ++w) M = fmaxf(M, ml[w * 32 + hh]);
        const float sub = M == -INFINITY ? 0.f : M;
        float o = 0.f, L = 0.f;
#pragma unroll
        for (int w = 0; w < kWinWarps; ++w) {
            const float f = exp2_approx(ml[w * 32 + hh] - sub);
            o += f * part[w * GD + e];
            L += f * ml[w * 32 + 16 + hh];
        }
        if (ranks == 1) {
            store_out<T>(p.out, p.out_dtype, ob + e, vis.count > 0 ? o / L : 0.f);
        } else {
            comb[e] = o;
            if (e % D == 0) {
                cml[hh] = M;
                cml[16 + hh] = L;
            }
        }
    }
    if (ranks == 1) return;

    // ---- the CTAs' parts: each CTA of the cluster joins a slice of the outputs ----
    cluster_sync();
    const int slice = (GD + ranks - 1) / ranks;
    const int e_hi = min(GD, (rank + 1) * slice);
    for (int e = rank * slice + tid; e < e_hi; e += kWinWarps * 32) {
        const int hh = e / D;
        float M = -INFINITY, o = 0.f, L = 0.f;
        // four CTAs' values on their way at a time, joined in the order of the ranks
        for (int r0 = 0; r0 < ranks; r0 += 4) {
            float m[4], l[4], x[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const uint32_t r = (uint32_t)min(r0 + u, ranks - 1);
                m[u] = ld_cluster_f32(cluster_addr(cml + hh, r));
                l[u] = ld_cluster_f32(cluster_addr(cml + 16 + hh, r));
                x[u] = ld_cluster_f32(cluster_addr(comb + e, r));
                if (r0 + u >= ranks) m[u] = -INFINITY;
            }
            const float Mn = fmaxf(fmaxf(fmaxf(M, m[0]), fmaxf(m[1], m[2])), m[3]);
            const float sub = Mn == -INFINITY ? 0.f : Mn;
            const float f0 = exp2_approx(M - sub);
            o *= f0;
            L *= f0;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float f = exp2_approx(m[u] - sub);
                o += f * x[u];
                L += f * l[u];
            }
            M = Mn;
        }
        store_out<T>(p.out, p.out_dtype, ob + e, vis.count > 0 ? o / L : 0.f);
    }
    cluster_sync();   // a CTA's shared memory outlives its readers
}

template <typename T, int D, int NT, bool MANY>
static int launch_window_decode(const WindowDecodeParams &prm, const CUtensorMap &tk, const CUtensorMap &tv, int grid,
                                int ranks, cudaStream_t stream) {
    constexpr int kSmem = WindowShape<D, MANY>::SMEM_BYTES;
    static unsigned long long attr_set = 0;   // per instantiation and device
    if (!done_on_device(&attr_set)) {
        cudaError_t e = cudaFuncSetAttribute(window_decode_kernel<T, D, NT, MANY>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(window_decode_kernel<T, D, NT, MANY>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return cuda_fail(e);
        mark_done_on_device(&attr_set);
    }
    cudaError_t e = launch_cluster(window_decode_kernel<T, D, NT, MANY>, grid, ranks, kWinWarps * 32, kSmem, stream, prm, tk,
                                   tv);
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? PKV_OK : cuda_fail(e);
}

// The form and the CTAs per range, from the number of ranges, the blocks that
// one can have, and whether MANY is built for the group size.
template <typename T, int D>
static int window_decode(const WindowDecodeParams &prm, const CUtensorMap &tk, const CUtensorMap &tv, int64_t ranges,
                         int64_t blocks, int sms, cudaStream_t stream) {
    constexpr int kFew = WindowShape<D, false>::PER_SM, kMany = WindowShape<D, true>::PER_SM;
    // CTAs per range: as many as all fit on the GPU at once, each with at least
    // two blocks a warp.  A second wave of clusters costs more than it evens
    // out: 16 sequences x 8 heads x 65 blocks take 14.9 us in 256 CTAs and 19.1
    // us in 512; 4 x 8 x 257 14.2 us in 256 and 24.3 us in 512.
    int ranks = (int)std::min<int64_t>({kWinMaxCluster, 2 * sms / ranges, blocks / (2 * kWinWarps)});
    if (ranks > 8 && ranks < kWinMaxCluster) ranks = 8;
    // a call of few CTAs is bound by a warp's chain of latencies: one block a
    // warp, up to a CTA per SM (8 ranges of 17 blocks: 5.6 -> 4.2 us)
    ranks = std::max(ranks, (int)std::min<int64_t>({8, sms / ranges, blocks / kWinWarps}));
    if (ranks < 1) ranks = 1;
    const int grid = (int)(ranges * ranks);
    if (prm.G > 8) return launch_window_decode<T, D, 2, false>(prm, tk, tv, grid, ranks, stream);
    // ranges of equal length pay for the last wave: its CTAs at half or a third
    // of an SM's rate each (64 x 8 ranges of 65 blocks: 45.2 us in 1.7 waves of
    // two, 50.8 us in 1.1 waves of three).  Of many waves, or of short ranges,
    // MANY is the better one all the same.
    auto waves = [&](int per_sm) { return (ranges + per_sm * sms - 1) / (per_sm * sms) * per_sm; };
    if (ranges > 2 * sms && (ranges >= 6 * sms || blocks <= 32 || waves(kMany) <= waves(kFew)))
        return launch_window_decode<T, D, 1, true>(prm, tk, tv, grid, ranks, stream);
    return launch_window_decode<T, D, 1, false>(prm, tk, tv, grid, ranks, stream);
}

}  // namespace pkv

extern "C" int pkv_paged_window_decode_attention(void *out, const void *q, const void *k_cache, const void *v_cache,
                                                 const int32_t *block_tables, int max_blocks_per_seq,
                                                 const int32_t *context_lens, int num_seqs, int num_blocks,
                                                 int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                                 int window, int num_sinks, float scale, int dtype, int out_dtype,
                                                 int *dev_status, void *stream) {
    pkv::NvtxRange nvtx_range("pkv_paged_window_decode_attention");
    using namespace pkv;
    if (num_seqs < 0 || num_blocks <= 0 || num_kv_heads <= 0 || num_q_heads <= 0 || max_blocks_per_seq <= 0 ||
        window <= 0 || num_sinks < 0)
        return PKV_ERR_INVALID_ARG;
    if (num_q_heads % num_kv_heads != 0) return PKV_ERR_INVALID_ARG;
    const int G = num_q_heads / num_kv_heads;
    if (G > 16 || block_size != 16 || (head_dim != 64 && head_dim != 128)) return PKV_ERR_UNSUPPORTED;
    if (dtype != PKV_DTYPE_F16 && dtype != PKV_DTYPE_BF16) return PKV_ERR_UNSUPPORTED;
    if (out_dtype != dtype && out_dtype != PKV_DTYPE_F32) return PKV_ERR_UNSUPPORTED;
    if (!(std::isfinite(scale) && scale > 0.f)) return PKV_ERR_INVALID_ARG;
    if ((int64_t)num_blocks * num_kv_heads * block_size >= (int64_t)1 << 31) return PKV_ERR_UNSUPPORTED;
    if ((int64_t)num_seqs * max_blocks_per_seq >= (int64_t)1 << 31 || max_blocks_per_seq > (1 << 26))
        return PKV_ERR_UNSUPPORTED;
    if ((int64_t)num_seqs * num_kv_heads * kWinMaxCluster >= (int64_t)1 << 31) return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PKV_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens) return PKV_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !aligned(block_tables, 4) || !aligned(context_lens, 4))
        return PKV_ERR_INVALID_ARG;
    int sms = 0;
    int rc = current_sm_count(&sms);
    if (rc != PKV_OK) return rc;
    CUtensorMap tk, tv;
    rc = encode_cache_map(&tk, k_cache, num_blocks, num_kv_heads, block_size, head_dim);
    if (rc != PKV_OK) return rc;
    rc = encode_cache_map(&tv, v_cache, num_blocks, num_kv_heads, block_size, head_dim);
    if (rc != PKV_OK) return rc;
    WindowDecodeParams prm;
    prm.out = out;
    prm.q = q;
    prm.block_tables = block_tables;
    prm.context_lens = context_lens;
    prm.dev_status = dev_status;
    prm.max_blocks = max_blocks_per_seq;
    prm.num_blocks = num_blocks;
    prm.Hq = num_q_heads;
    prm.Hkv = num_kv_heads;
    prm.G = G;
    const int64_t capacity = (int64_t)max_blocks_per_seq * 16;
    prm.window = window < capacity ? window : (int)capacity;   // no context is longer
    prm.sinks = num_sinks < capacity ? num_sinks : (int)capacity;
    prm.scale_log2 = scale * 1.4426950408889634f;
    prm.out_dtype = out_dtype;
    const int64_t most = ((int64_t)prm.sinks + 15) / 16 + ((int64_t)window + 14) / 16 + 1;
    const int64_t blocks = std::min<int64_t>(most, max_blocks_per_seq);
    const int64_t ranges = (int64_t)num_seqs * num_kv_heads;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dtype == PKV_DTYPE_BF16)
        return head_dim == 128 ? window_decode<__nv_bfloat16, 128>(prm, tk, tv, ranges, blocks, sms, st)
                               : window_decode<__nv_bfloat16, 64>(prm, tk, tv, ranges, blocks, sms, st);
    return head_dim == 128 ? window_decode<__half, 128>(prm, tk, tv, ranges, blocks, sms, st)
                           : window_decode<__half, 64>(prm, tk, tv, ranges, blocks, sms, st);
}
