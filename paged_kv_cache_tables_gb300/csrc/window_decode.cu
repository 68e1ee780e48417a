// Decode attention over a sliding window and the first tokens of a paged
// context (pkv_paged_window_decode_attention).
//
// Mathematics.  The query of sequence s sits at position p = ctx_s - 1 and
// sees position t iff t <= p and (t > p - window or t < sinks):
//     out = sum_t softmax_t(scale * q . K_t) V_t  over those t,
// taken block by block with the running maximum m and sum l of the softmax in
// fp32: a block's scores x give m' = max(m, x), weights 2^(x - m'), and l and
// the accumulator are scaled by 2^(m - m').  Parts of a range combine the same
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
// sum is fixed by the lengths alone.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "pkv.h"
#include "pkv_cluster.cuh"
#include "pkv_device.cuh"
#include "pkv_host.h"

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

template <int D>
struct WindowShape {
    static constexpr int HALVES = D / 64;               // 64-element (128-byte) column halves
    static constexpr int HALF_BYTES = 64 * 16 * 2;
    static constexpr int TILE_BYTES = HALVES * HALF_BYTES;
    static constexpr int STAGE_BYTES = 2 * TILE_BYTES;  // K then V
    static constexpr int STAGES = D == 128 ? 3 : 6;
    static constexpr int RING_BYTES = kWinWarps * STAGES * STAGE_BYTES;
    // behind the ring: barriers, then (m, l) of each warp and of the CTA
    static constexpr int OFF_ML = RING_BYTES + kWinWarps * STAGES * 8;
    static constexpr int SMEM_BYTES = 1024 + OFF_ML + (kWinWarps + 1) * 32 * 4;
};

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kWinWarps * 32, 2)
    window_decode_kernel(const WindowDecodeParams p, const __grid_constant__ CUtensorMap tk,
                         const __grid_constant__ CUtensorMap tv) {
    using Sh = WindowShape<D>;
    constexpr int STAGES = Sh::STAGES;
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
    int ctx = __ldg(p.context_lens + s);
    if (ctx < 0 || ctx > p.max_blocks * 16) {
        if (tid == 0 && rank == 0 && h == 0) set_status(p.dev_status, PKV_DEV_BAD_CONTEXT);
        ctx = ctx < 0 ? 0 : p.max_blocks * 16;
    }
    const int nblk = (ctx + 15) >> 4;
    const int w0 = max(ctx - p.window, 0);                   // the window's first position
    const int sink_blocks = min((p.sinks + 15) >> 4, nblk);
    const int skip = max((w0 >> 4) - sink_blocks, 0);
    const int visible = nblk - skip;
    const int v_lo = (int)((int64_t)visible * rank / ranks), v_hi = (int)((int64_t)visible * (rank + 1) / ranks);
    const int n = max(0, (v_hi - v_lo - warp + kWinWarps - 1) / kWinWarps);
    auto logical = [&](int i) {
        const int v = v_lo + warp + kWinWarps * i;
        return v < sink_blocks ? v : v + skip;
    };
    const int32_t *row = p.block_tables + (int64_t)s * p.max_blocks;
    int ids = lane < n ? __ldg(row + logical(lane)) : 0;     // lane i: the id of this warp's block 32 k + i
    const uint64_t policy = l2_policy_evict_first();
    auto issue = [&](int i) {
        const int blk = __shfl_sync(0xffffffffu, ids, i & 31);
        if (lane == 0) {
            const bool bad_blk = blk < 0 || blk >= p.num_blocks;
            if (bad_blk) set_status(p.dev_status, PKV_DEV_BAD_BLOCK_ID);
            // past the end for a bad block id: the load fills zeros
            const int y = bad_blk ? p.num_blocks * p.Hkv * 16 : (blk * p.Hkv + h) * 16;
            uint64_t *bar = &wbar[i % STAGES];
            mbar_arrive_expect_tx(bar, Sh::STAGE_BYTES);
            uint8_t *kdst = wring + (i % STAGES) * Sh::STAGE_BYTES;
#pragma unroll
            for (int hf = 0; hf < Sh::HALVES; ++hf) {
                tma_load_2d(kdst + hf * Sh::HALF_BYTES, &tk, hf * 64, y, bar, policy);
                tma_load_2d(kdst + Sh::TILE_BYTES + hf * Sh::HALF_BYTES, &tv, hf * 64, y, bar, policy);
            }
        }
    };
    int issued = 0;
    for (; issued < min(n, STAGES); ++issued) issue(issued);

    // ---- query fragments: rows = heads of the group, padded to 16 ----
    const int g = lane >> 2, t4 = lane & 3;
    uint32_t qa[D / 16][4];
    {
        const uint32_t *qbase =
            reinterpret_cast<const uint32_t *>(static_cast<const T *>(p.q) + ((int64_t)s * p.Hq + (int64_t)h * G) * D);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const int c0 = (kk * 16 + 2 * t4) >> 1;
            qa[kk][0] = g < G ? __ldg(qbase + g * (D / 2) + c0) : 0u;
            qa[kk][2] = g < G ? __ldg(qbase + g * (D / 2) + c0 + 4) : 0u;
            if constexpr (NT == 1) {   // group of at most 8 heads: rows 8..15 are padding
                qa[kk][1] = 0u;
                qa[kk][3] = 0u;
            } else {
                qa[kk][1] = g + 8 < G ? __ldg(qbase + (g + 8) * (D / 2) + c0) : 0u;
                qa[kk][3] = g + 8 < G ? __ldg(qbase + (g + 8) * (D / 2) + c0 + 4) : 0u;
            }
        }
    }
    float acc[D / 16][NT][4];
    float m_run[NT], l_run[NT];
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
    const int mi = lane >> 3;
    const int ld_row = ((mi >> 1) << 3) + (lane & 7);   // token row this lane addresses
    const int ld_sw = ld_row & 7;                        // 128-byte swizzle phase of that row
    const uint32_t ring_addr = smem_addr(wring);

    bool timed_out = false;
    int i = 0;
    for (; i < n; ++i) {
        if (!__all_sync(0xffffffffu, mbar_wait(&wbar[i % STAGES], (uint32_t)(i / STAGES) & 1u, kWinWaitNs))) {
            timed_out = true;
            break;
        }
        const uint32_t kbase = ring_addr + (i % STAGES) * Sh::STAGE_BYTES;
        const uint32_t vbase = kbase + Sh::TILE_BYTES;
        // the block's fragments into registers, then its slot back to the TMA engine
        uint32_t kf[D / 16][4], vf[D / 16][4];
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const int chunk = ((kk & 3) << 1) + (mi & 1);
            const uint32_t off = (kk >> 2) * Sh::HALF_BYTES + ld_row * 128 + ((chunk ^ ld_sw) << 4);
            ldsm_x4(kbase + off, kf[kk][0], kf[kk][1], kf[kk][2], kf[kk][3]);
            ldsm_x4_t(vbase + off, vf[kk][0], vf[kk][1], vf[kk][2], vf[kk][3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (issued < n) {
            if ((issued & 31) == 0) ids = issued + lane < n ? __ldg(row + logical(issued + lane)) : 0;
            issue(issued);
            ++issued;
        }

        // S = Q K^T over the block's 16 tokens, two chains per 8-token tile
        float sacc[2][4], sacc2[2][4];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) sacc[nt][e] = sacc2[nt][e] = 0.f;
#pragma unroll
        for (int kk = 0; kk < D / 16; kk += 2) {
            mma_16816<T>(sacc[0], qa[kk], kf[kk][0], kf[kk][1]);
            mma_16816<T>(sacc[1], qa[kk], kf[kk][2], kf[kk][3]);
            mma_16816<T>(sacc2[0], qa[kk + 1], kf[kk + 1][0], kf[kk + 1][1]);
            mma_16816<T>(sacc2[1], qa[kk + 1], kf[kk + 1][2], kf[kk + 1][3]);
        }

        // the block's visible tokens, one bit each (never none): before ctx,
        // and in the window or among the first tokens
        const int t0 = logical(i) * 16;
        const int lim = min(ctx - t0, 16), first = min(max(w0 - t0, 0), 16), sk = min(max(p.sinks - t0, 0), 16);
        const uint32_t bits = ((1u << lim) - 1u) & ((0xffffu << first) | ((1u << sk) - 1u)) & 0xffffu;
        float pr[2][4];
        float alpha[NT];
#pragma unroll
        for (int pn = 0; pn < NT; ++pn) {
            float x[2][2];
            float mx = -INFINITY;
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int tok = nt * 8 + 2 * t4 + e;
                    const float v = (sacc[nt][pn * 2 + e] + sacc2[nt][pn * 2 + e]) * p.scale_log2;
                    x[nt][e] = (bits >> tok) & 1u ? v : -INFINITY;
                    mx = fmaxf(mx, x[nt][e]);
                }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const float m_new = fmaxf(m_run[pn], mx);
            // no finite score so far (keys of infinities): nothing to subtract
            const float sub = m_new == -INFINITY ? 0.f : m_new;
            alpha[pn] = exp2_approx(m_run[pn] - sub);
            m_run[pn] = m_new;
            float rs = 0.f;
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
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
        if (bits != 0xffffu) {
            const uint32_t b = bits >> (2 * t4);
            const uint32_t m01 = (b & 1u ? 0x0000ffffu : 0u) | (b & 2u ? 0xffff0000u : 0u);
            const uint32_t m23 = (b & 0x100u ? 0x0000ffffu : 0u) | (b & 0x200u ? 0xffff0000u : 0u);
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt) {
                vf[mt][0] &= m01;
                vf[mt][1] &= m01;
                vf[mt][2] &= m23;
                vf[mt][3] &= m23;
            }
        }
        // rescale the accumulator (only when a row's maximum moved), O^T += V^T P^T
        bool moved = false;
#pragma unroll
        for (int pn = 0; pn < NT; ++pn) moved |= alpha[pn] != 1.f;
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
        // P as a rounded 16-bit value and its rounding residual: the weights
        // keep about 16 significant bits
        uint32_t pb0[NT][2], pb1[NT][2];
#pragma unroll
        for (int pn = 0; pn < NT; ++pn) {
            pack2_split<T>(pr[0][pn * 2], pr[0][pn * 2 + 1], pb0[pn][0], pb0[pn][1]);
            pack2_split<T>(pr[1][pn * 2], pr[1][pn * 2 + 1], pb1[pn][0], pb1[pn][1]);
        }
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt) {
#pragma unroll
            for (int pn = 0; pn < NT; ++pn) {
                mma_16816<T>(acc[mt][pn], vf[mt], pb0[pn][0], pb1[pn][0]);
                mma_16816<T>(acc[mt][pn], vf[mt], pb0[pn][1], pb1[pn][1]);
            }
        }
    }
    if (timed_out) {
        if (lane == 0) set_status(p.dev_status, PKV_DEV_WAIT_TIMEOUT);
        // what is still in flight must land before the ring is used again
        for (int k = i + 1; k < issued; ++k) mbar_wait(&wbar[k % STAGES], (uint32_t)(k / STAGES) & 1u, kWinWaitNs / 8);
    }

    // ---- the warps' parts: (m, l) per head, accumulators [warp][head][d] over the ring ----
    __syncthreads();   // every warp is done with its slots
    float *part = reinterpret_cast<float *>(smem);
    const int GD = G * D;
#pragma unroll
    for (int pn = 0; pn < NT; ++pn) {
        float l = l_run[pn];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if (t4 == 0) {
            ml[warp * 32 + pn * 8 + g] = m_run[pn];
            ml[warp * 32 + 16 + pn * 8 + g] = l;
        }
        const int ha = pn * 8 + 2 * t4, hb = ha + 1;
        float *wp = part + warp * GD;
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt) {
            const int d0 = mt * 16 + g;
            if (ha < G) {
                wp[ha * D + d0] = acc[mt][pn][0];
                wp[ha * D + d0 + 8] = acc[mt][pn][2];
            }
            if (hb < G) {
                wp[hb * D + d0] = acc[mt][pn][1];
                wp[hb * D + d0 + 8] = acc[mt][pn][3];
            }
        }
    }
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
            store_out<T>(p.out, p.out_dtype, ob + e, visible > 0 ? o / L : 0.f);
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
        store_out<T>(p.out, p.out_dtype, ob + e, visible > 0 ? o / L : 0.f);
    }
    cluster_sync();   // a CTA's shared memory outlives its readers
}

template <typename T, int D, int NT>
static int launch_window_decode(const WindowDecodeParams &prm, const CUtensorMap &tk, const CUtensorMap &tv, int grid,
                                int ranks, cudaStream_t stream) {
    static unsigned long long attr_set = 0;   // per instantiation and device
    if (!done_on_device(&attr_set)) {
        cudaError_t e = cudaFuncSetAttribute(window_decode_kernel<T, D, NT>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, WindowShape<D>::SMEM_BYTES);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(window_decode_kernel<T, D, NT>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return cuda_fail(e);
        mark_done_on_device(&attr_set);
    }
    cudaError_t e = launch_cluster(window_decode_kernel<T, D, NT>, grid, ranks, kWinWarps * 32,
                                   WindowShape<D>::SMEM_BYTES, stream, prm, tk, tv);
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? PKV_OK : cuda_fail(e);
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
    if (!aligned(q, 4) || !aligned(out, 4) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
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
    // CTAs per range: as many as all fit on the GPU at once (two per SM), each
    // with at least two blocks a warp.  A second wave of clusters costs more
    // than it evens out: 16 sequences x 8 heads x 65 blocks take 14.9 us in 256
    // CTAs and 19.1 us in 512; 4 x 8 x 257 14.2 us in 256 and 24.3 us in 512.
    const int64_t ranges = (int64_t)num_seqs * num_kv_heads;
    const int64_t most = ((int64_t)prm.sinks + 15) / 16 + ((int64_t)window + 14) / 16 + 1;
    const int64_t blocks = most < max_blocks_per_seq ? most : max_blocks_per_seq;
    int ranks = (int)std::min<int64_t>({kWinMaxCluster, 2 * sms / ranges, blocks / (2 * kWinWarps)});
    if (ranks > 8 && ranks < kWinMaxCluster) ranks = 8;
    if (ranks < 1) ranks = 1;
    const int grid = (int)(ranges * ranks);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool wide = G > 8;
    if (dtype == PKV_DTYPE_BF16) {
        if (head_dim == 128)
            return wide ? launch_window_decode<__nv_bfloat16, 128, 2>(prm, tk, tv, grid, ranks, st)
                        : launch_window_decode<__nv_bfloat16, 128, 1>(prm, tk, tv, grid, ranks, st);
        return wide ? launch_window_decode<__nv_bfloat16, 64, 2>(prm, tk, tv, grid, ranks, st)
                    : launch_window_decode<__nv_bfloat16, 64, 1>(prm, tk, tv, grid, ranks, st);
    }
    if (head_dim == 128)
        return wide ? launch_window_decode<__half, 128, 2>(prm, tk, tv, grid, ranks, st)
                    : launch_window_decode<__half, 128, 1>(prm, tk, tv, grid, ranks, st);
    return wide ? launch_window_decode<__half, 64, 2>(prm, tk, tv, grid, ranks, st)
                : launch_window_decode<__half, 64, 1>(prm, tk, tv, grid, ranks, st);
}
