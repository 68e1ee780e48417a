// Decode attention over the cache held in 8 bits
// (pkv_paged_decode_attention_e4m3).
//
// Mathematics.  As window_decode.cu, with K_t = k_t a_j and V_t = v_t b_j, k and
// v the e4m3 codes and a, b the scales of t's block j.  The codes become fp16
// exactly; a multiplies the scores, and b is taken into the softmax: with
//     y_t = scale2 a_j (q . k_t) + log2 b_j,   P_t = 2^(y_t - m + 7),  m >= y_t - 8,
// m the running maximum of y, O = sum P_t v_t and l = sum P_t / b_j give out = O / l.
// So P is below 2^15 and about 2^7 for the weight that counts most, whatever the
// scales are, and meets v as an fp16 value: rounded once (11 bits) for a bf16
// output, whose own rounding is 8 times coarser, else with its rounding
// residual.  A bf16 query is brought to fp16 by a power of two per head that puts
// its largest element into [1, 2): elements below 2^-14 of that lose bits, 2^-25
// of the largest at most.
//
// Layout.  A 16-byte piece of a row goes to one lane, so that a fragment's
// dimensions (for S) and output rows (for O^T) are not in their order in memory
// but in an order that suits these loads:
//   S^T = K Q^T     lane (g, t4) takes 16 dimensions 16 (t4 + 4 j) .. of tokens
//                   rho(g) and rho(g) + 8
//   O^T += V^T P^T  lane (g, t4) takes head_dim / 8 dimensions from g on, of tokens
//                   rho(2 t4), rho(2 t4 + 1), and 8 further; bytes of two tokens
//                   are put side by side before they are converted
// rho permutes the tokens of a group of 8 so that neither load meets a bank
// twice under TMA's 128-byte swizzle (a shared-memory row of 128 bytes is one
// token's codes, or with head_dim 64 two tokens').  With tokens as the rows of
// both products neither pays for absent heads beyond 8, a lane's scores and its
// accumulator columns belong to the same two heads, and P^T is P of S^T
// transposed, 8 x 8 at a time (movmatrix).
#include <cuda_runtime.h>

#include <algorithm>

#include "pkv.h"
#include "pkv_cluster.cuh"
#include "pkv_device.cuh"
#include "pkv_host.h"
#include "pkv_quant.cuh"
#include "pkv_window.cuh"

namespace pkv {

constexpr int kQdWarps = 4;
constexpr int kQdMaxCluster = 16;
constexpr uint64_t kQdWaitNs = 2000000000ull;   // a tile that has not landed in 2 s never will

struct QuantDecodeParams {
    void *out;
    const void *q;
    const float *scales;
    const int32_t *block_tables;
    const int32_t *context_lens;
    int *dev_status;
    int max_blocks, num_blocks, Hq, Hkv, G;
    int window, sinks;
    float scale_log2;   // scale * log2(e): scores in base-2 units
    int out_dtype;
};

// Two forms, as in window_decode.cu: FEW for ranges that all fit on the GPU at
// once, MANY for more.
template <int D, bool MANY>
struct QuantShape {
    static constexpr int TILE_BYTES = 16 * D;
    static constexpr int BLOCK_BYTES = 2 * TILE_BYTES;  // K then V
    static constexpr int STEP = 2;                      // blocks a warp takes at a time: a slot of its ring
    static constexpr int SLOT_BYTES = STEP * BLOCK_BYTES;
    static constexpr int SLOTS = D == 128 ? (MANY ? 2 : 3) : 4;
    static constexpr int PER_SM = D == 128 && !MANY ? 2 : 3;
    static constexpr int RING_BYTES = kQdWarps * SLOTS * SLOT_BYTES;
    // behind the ring: barriers, then (m, l) of each warp and of the CTA
    static constexpr int OFF_ML = RING_BYTES + kQdWarps * SLOTS * 8;
    static constexpr int SMEM_BYTES = 1024 + OFF_ML + (kQdWarps + 1) * 32 * 4;
    static_assert((kQdWarps + 1) * 16 * D * 4 <= RING_BYTES, "the parts take the ring's place");
};

// The token of a group of 8 that stands at place n of a fragment.
template <int D>
__device__ __forceinline__ int token_at(int n) {
    if constexpr (D == 128) return n ^ ((n & 1) << 2);
    const int i = n >> 1, x = (i & 1) | ((i & 2) << 1);
    return n & 1 ? x ^ 3 : x;
}

// Byte offset of 16-byte piece c of token t's codes in a tile.
template <int D>
__device__ __forceinline__ uint32_t piece_at(int t, int c) {
    if constexpr (D == 128) return (uint32_t)(t * 128 + ((c ^ (t & 7)) << 4));
    const int r = t >> 1;
    return (uint32_t)(r * 128 + ((((t & 1) * 4 + c) ^ (r & 7)) << 4));
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}

__device__ __forceinline__ uint2 lds64(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}

// Four 16-bit elements as two fp16 pairs times f.
template <typename T>
__device__ __forceinline__ void query4(uint2 x, float f, uint32_t &a, uint32_t &b) {
    if constexpr (std::is_same<T, __half>::value) {
        a = x.x;
        b = x.y;
    } else {
        a = pack2<__half>(__uint_as_float(x.x << 16) * f, __uint_as_float(x.x & 0xffff0000u) * f);
        b = pack2<__half>(__uint_as_float(x.y << 16) * f, __uint_as_float(x.y & 0xffff0000u) * f);
    }
}

// The transpose of an 8 x 8 matrix of 16-bit elements, a pair a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// A warp's part of a range.  The heads of the group are columns, 8 to a tile
// (NT tiles): lane (g, t4) has those at 2 t4 and 2 t4 + 1 of each.
template <typename T, int D, int NT, bool MANY, bool RES>
struct QuantPart {
    using Sh = QuantShape<D, MANY>;
    static constexpr int STEP = Sh::STEP;
    static constexpr int KT = D / 16;        // steps of 16 dimensions, and of 16 output rows
    static constexpr int NW = D / 32;        // 4-byte words of a token's codes that a lane takes of V
    uint32_t qb[KT][NT][2];
    float acc[KT][NT][4];                    // [output rows][tile][row g heads 2, row g + 8 heads 2]
    float m_run[NT][2], off[NT][2];          // running maximum; what P subtracts
    float l_run[NT][2];
    float qscale[NT][2];                     // a head's score scale, its query's power of two taken back

    // q: G rows of D elements
    __device__ __forceinline__ void start(const T *q, int G, float scale_log2, int lane) {
        const int g = lane >> 2, t4 = lane & 3;
#pragma unroll
        for (int pn = 0; pn < NT; ++pn) {
            const int row = pn * 8 + g;
            uint2 x[KT];
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < D / 64; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint2 *at = reinterpret_cast<const uint2 *>(q + row * D + 16 * (t4 + 4 * j) + 4 * i);
                    x[4 * j + i] = row < G ? *at : make_uint2(0u, 0u);
                    const uint2 w = x[4 * j + i];
                    top = max(max(top, max(w.x & 0x7fffu, (w.x >> 16) & 0x7fffu)), max(w.y & 0x7fffu, (w.y >> 16) & 0x7fffu));
                }
            float f = 1.f, back = 1.f;
            if constexpr (!std::is_same<T, __half>::value) {
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int e = min(max((int)(top >> 7), 1), 253);          // exponent field of the largest
                f = __uint_as_float((uint32_t)(254 - e) << 23);
                back = __uint_as_float((uint32_t)e << 23);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) qscale[pn][e] = __shfl_sync(0xffffffffu, back, 4 * (2 * t4 + e)) * scale_log2;
#pragma unroll
            for (int kk = 0; kk < KT; ++kk) query4<T>(x[kk], f, qb[kk][pn][0], qb[kk][pn][1]);
#pragma unroll
            for (int mt = 0; mt < KT; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[mt][pn][e] = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m_run[pn][e] = -INFINITY;
                off[pn][e] = -7.f;
                l_run[pn][e] = 0.f;
            }
        }
    }

    // STEP blocks of 16 tokens in the ring slot at `slot`, of scales ks, vs; bit t
    // of `bits` set where token t of them is seen (all of them: `all`).
    // `release` runs once the slot has been read.
    template <typename F>
    __device__ __forceinline__ void attend(uint32_t slot, const float (&ks)[STEP], const float (&vs)[STEP], uint32_t bits,
                                           bool all, int lane, F release) {
        const int g = lane >> 2, t4 = lane & 3;
        // S^T = K Q^T, two chains a block
        float s[STEP][2][NT][4];
#pragma unroll
        for (int b = 0; b < STEP; ++b)
#pragma unroll
            for (int pn = 0; pn < NT; ++pn)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[b][0][pn][e] = s[b][1][pn][e] = 0.f;
        const int tok_k = token_at<D>(g);
#pragma unroll
        for (int b = 0; b < STEP; ++b)
#pragma unroll
            for (int j = 0; j < D / 64; ++j) {
                const uint4 k0 = lds128(slot + b * Sh::BLOCK_BYTES + piece_at<D>(tok_k, t4 + 4 * j));
                const uint4 k1 = lds128(slot + b * Sh::BLOCK_BYTES + piece_at<D>(tok_k + 8, t4 + 4 * j));
                const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t a[4];
                    e4m3x4_to_f16x4(w0[i], a[0], a[2]);
                    e4m3x4_to_f16x4(w1[i], a[1], a[3]);
#pragma unroll
                    for (int pn = 0; pn < NT; ++pn)
                        mma_16816<__half>(s[b][i & 1][pn], a, qb[4 * j + i][pn][0], qb[4 * j + i][pn][1]);
                }
            }
        // [block][token rho(2 t4), rho(2 t4 + 1), and those + 8][words]
        uint32_t vw[STEP][4][NW];
#pragma unroll
        for (int b = 0; b < STEP; ++b)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int tok = token_at<D>(2 * t4 + (u & 1)) + 8 * (u >> 1);
                const uint32_t tile = slot + b * Sh::BLOCK_BYTES + Sh::TILE_BYTES;
                if constexpr (D == 128) {
                    const uint4 v = lds128(tile + piece_at<D>(tok, g));
                    vw[b][u][0] = v.x, vw[b][u][1] = v.y, vw[b][u][2] = v.z, vw[b][u][3] = v.w;
                } else {
                    const uint2 v = lds64(tile + piece_at<D>(tok, g >> 1) + (g & 1) * 8);
                    vw[b][u][0] = v.x, vw[b][u][1] = v.y;
                }
            }
        release();

        // y in place of the scores: [block][tile][token rho(g) heads 2, token rho(g) + 8 heads 2]
        float y[STEP][NT][4], rv[STEP];
        bool past = false;
#pragma unroll
        for (int b = 0; b < STEP; ++b) {
            const float lv = __log2f(vs[b]);
            rv[b] = exp2_approx(-lv);
#pragma unroll
            for (int pn = 0; pn < NT; ++pn)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    y[b][pn][e] = fmaf(s[b][0][pn][e] + s[b][1][pn][e], qscale[pn][e & 1] * ks[b], lv);
                    if (!all && !((bits >> (16 * b + tok_k + 8 * (e >> 1))) & 1u)) y[b][pn][e] = -INFINITY;
                    past |= y[b][pn][e] > m_run[pn][e & 1] + 8.f;
                }
        }
        // the maximum is only moved when it grows by more than 2^8
        if (__any_sync(0xffffffffu, past)) {
#pragma unroll
            for (int pn = 0; pn < NT; ++pn)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mx = fmaxf(y[0][pn][e], y[0][pn][e + 2]);
#pragma unroll
                    for (int b = 1; b < STEP; ++b) mx = fmaxf(mx, fmaxf(y[b][pn][e], y[b][pn][e + 2]));
#pragma unroll
                    for (int d = 4; d < 32; d *= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                    if (mx > m_run[pn][e] + 8.f) {
                        const float alpha = exp2_approx(m_run[pn][e] - mx);
                        m_run[pn][e] = mx;
                        off[pn][e] = mx - 7.f;
                        l_run[pn][e] *= alpha;
#pragma unroll
                        for (int mt = 0; mt < KT; ++mt) {
                            acc[mt][pn][e] *= alpha;
                            acc[mt][pn][e + 2] *= alpha;
                        }
                    }
                }
        }
        // hidden positions may hold anything (even NaN codes): zero, so that 0 x
        // garbage cannot reach the accumulator
        if (!all) {
#pragma unroll
            for (int b = 0; b < STEP; ++b)
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int tok = token_at<D>(2 * t4 + (u & 1)) + 8 * (u >> 1);
                    const uint32_t keep = (bits >> (16 * b + tok)) & 1u ? 0xffffffffu : 0u;
#pragma unroll
                    for (int i = 0; i < NW; ++i) vw[b][u][i] &= keep;
                }
        }
#pragma unroll
        for (int b = 0; b < STEP; ++b) {
            // P^T fragments: tokens 0..7 and 8..15 of the block; value, residual
            uint32_t pb[NT][2][2];
#pragma unroll
            for (int pn = 0; pn < NT; ++pn) {
                float w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = exp2_approx(y[b][pn][e] - off[pn][e & 1]);
                l_run[pn][0] = fmaf(w[0] + w[2], rv[b], l_run[pn][0]);
                l_run[pn][1] = fmaf(w[1] + w[3], rv[b], l_run[pn][1]);
                if constexpr (RES) {
                    pack2_split<__half>(w[0], w[1], pb[pn][0][0], pb[pn][0][1]);
                    pack2_split<__half>(w[2], w[3], pb[pn][1][0], pb[pn][1][1]);
                } else {
                    pb[pn][0][0] = pack2<__half>(w[0], w[1]);
                    pb[pn][1][0] = pack2<__half>(w[2], w[3]);
                }
#pragma unroll
                for (int r = 0; r < (RES ? 2 : 1); ++r) {
                    pb[pn][0][r] = transpose8(pb[pn][0][r]);
                    pb[pn][1][r] = transpose8(pb[pn][1][r]);
                }
            }
#pragma unroll
            for (int i = 0; i < NW; ++i)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    // dimensions 4 i + 2 half, + 1 of the lane's: two tokens' bytes side by side
                    const uint32_t sel = half ? 0x7362u : 0x5140u;
                    uint32_t a[4];
                    e4m3x4_to_f16x4(__byte_perm(vw[b][0][i], vw[b][1][i], sel), a[0], a[1]);
                    e4m3x4_to_f16x4(__byte_perm(vw[b][2][i], vw[b][3][i], sel), a[2], a[3]);
#pragma unroll
                    for (int r = 0; r < (RES ? 2 : 1); ++r)
#pragma unroll
                        for (int pn = 0; pn < NT; ++pn)
                            mma_16816<__half>(acc[2 * i + half][pn], a, pb[pn][0][r], pb[pn][1][r]);
                }
        }
    }

    // (m, l) of the heads at ml[head], ml[16 + head]; accumulators at part[head * D + d].
    __device__ __forceinline__ void store(float *ml, float *part, int G, int lane) {
        const int g = lane >> 2, t4 = lane & 3;
#pragma unroll
        for (int pn = 0; pn < NT; ++pn)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int head = pn * 8 + 2 * t4 + e;
                float l = l_run[pn][e];
#pragma unroll
                for (int d = 4; d < 32; d *= 2) l += __shfl_xor_sync(0xffffffffu, l, d);
                if (g == 0) {
                    ml[head] = m_run[pn][e];
                    ml[16 + head] = l;
                }
                if (head < G)
#pragma unroll
                    for (int mt = 0; mt < KT; ++mt)
                        *reinterpret_cast<float2 *>(part + head * D + g * (D / 8) + 2 * mt) =
                            make_float2(acc[mt][pn][e], acc[mt][pn][e + 2]);
            }
    }
};

template <typename T, int D, int NT, bool MANY, bool RES>
__global__ void __launch_bounds__(kQdWarps * 32, NT == 1 ? QuantShape<D, MANY>::PER_SM : 2)
    quant_decode_kernel(const QuantDecodeParams p, const __grid_constant__ CUtensorMap tk,
                        const __grid_constant__ CUtensorMap tv) {
    using Sh = QuantShape<D, MANY>;
    constexpr int SLOTS = Sh::SLOTS, STEP = Sh::STEP;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Sh::RING_BYTES);
    float *ml = reinterpret_cast<float *>(smem + Sh::OFF_ML);   // [warp][m 16, l 16], then the CTA's
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = (int)cluster_ctarank(), ranks = (int)cluster_nctarank();
    const int range = blockIdx.x / ranks;
    const int G = p.G, s = range / p.Hkv, h = range - s * p.Hkv;

    uint8_t *wring = smem + warp * SLOTS * Sh::SLOT_BYTES;
    uint64_t *wbar = bars + warp * SLOTS;
    if (lane == 0) {
        for (int st = 0; st < SLOTS; ++st) mbar_init(&wbar[st], 1);
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
    const int n = max(0, (v_hi - v_lo - warp + kQdWarps - 1) / kQdWarps);
    auto logical = [&](int i) { return vis.logical(v_lo + warp + kQdWarps * i); };
    const int32_t *row = p.block_tables + (int64_t)s * p.max_blocks;
    const uint64_t policy = l2_policy_evict_first();
    // lane i: the id and the scales of this warp's block 32 k + i, and the scales of 32 (k - 1) + i
    int id = 0;
    float2 sc = make_float2(1.f, 1.f), sc_before = sc;
    auto fetch = [&](int k) {
        sc_before = sc;
        id = 32 * k + lane < n ? __ldg(row + logical(32 * k + lane)) : 0;
        const bool ok = 32 * k + lane < n && id >= 0 && id < p.num_blocks;
        sc = ok ? __ldg(reinterpret_cast<const float2 *>(p.scales) + (int64_t)id * p.Hkv + h) : make_float2(1.f, 1.f);
    };
    const int steps = (n + STEP - 1) / STEP;
    auto issue = [&](int i) {   // step i's blocks into slot i % SLOTS
        const int k = min(STEP, n - STEP * i);
        int blk[STEP];
#pragma unroll
        for (int b = 0; b < STEP; ++b) blk[b] = __shfl_sync(0xffffffffu, id, (STEP * i + b) & 31);
        if (lane == 0) {
            uint8_t *slot = wring + (i % SLOTS) * Sh::SLOT_BYTES;
            uint64_t *bar = &wbar[i % SLOTS];
            mbar_arrive_expect_tx(bar, k * Sh::BLOCK_BYTES);
#pragma unroll
            for (int b = 0; b < STEP; ++b) {
                if (b >= k) break;
                const bool bad = blk[b] < 0 || blk[b] >= p.num_blocks;
                if (bad) set_status(p.dev_status, PKV_DEV_BAD_BLOCK_ID);
                // past the end for a bad block id: the load fills zeros
                constexpr int kRows = D / 8;   // 128-byte rows of a tile
                const int y = bad ? p.num_blocks * p.Hkv * kRows : (blk[b] * p.Hkv + h) * kRows;
                tma_load_2d(slot + b * Sh::BLOCK_BYTES, &tk, 0, y, bar, policy);
                tma_load_2d(slot + b * Sh::BLOCK_BYTES + Sh::TILE_BYTES, &tv, 0, y, bar, policy);
            }
        }
    };
    fetch(0);
    int issued = 0;   // steps
    for (; issued < min(steps, SLOTS); ++issued) issue(issued);

    QuantPart<T, D, NT, MANY, RES> part_w;
    part_w.start(static_cast<const T *>(p.q) + ((int64_t)s * p.Hq + (int64_t)h * G) * D, G, p.scale_log2, lane);
    const uint32_t ring_addr = smem_addr(wring);
    // entries [full_lo, full_hi) of the list are blocks that are seen whole
    const int full_lo = ((vis.w0 + 15) >> 4) - vis.skip, full_hi = (vis.ctx >> 4) - vis.skip;

    int i = 0;   // steps taken
    for (; i < steps; ++i) {
        const bool ok = mbar_wait(&wbar[i % SLOTS], (uint32_t)(i / SLOTS) & 1u, kQdWaitNs);
        if (!__all_sync(0xffffffffu, ok)) break;
        const int v0 = v_lo + warp + kQdWarps * STEP * i;
        const bool all = v0 >= full_lo && v0 + kQdWarps * (STEP - 1) < min(full_hi, v_hi);
        uint32_t bits = (uint32_t)((1ull << (16 * STEP)) - 1u);
        if (!all) {
            bits = 0;
#pragma unroll
            for (int b = 0; b < STEP; ++b)
                if (STEP * i + b < n) bits |= vis.bits(logical(STEP * i + b), p.sinks) << (16 * b);
        }
        // (the 32 blocks of the last step issued, or those before)
        const bool now = STEP * i / 32 == STEP * (issued - 1) / 32;
        float ks[STEP], vs[STEP];
#pragma unroll
        for (int b = 0; b < STEP; ++b) {
            ks[b] = __shfl_sync(0xffffffffu, now ? sc.x : sc_before.x, (STEP * i + b) & 31);
            vs[b] = __shfl_sync(0xffffffffu, now ? sc.y : sc_before.y, (STEP * i + b) & 31);
        }
        part_w.attend(ring_addr + (i % SLOTS) * Sh::SLOT_BYTES, ks, vs, bits, all, lane, [&] {
            fence_proxy_async_smem();
            __syncwarp();
            if (issued < steps) {
                if ((STEP * issued & 31) == 0) fetch(STEP * issued / 32);
                issue(issued++);
            }
        });
    }
    if (i < steps) {
        if (lane == 0) set_status(p.dev_status, PKV_DEV_WAIT_TIMEOUT);
        // what is still in flight must land before the ring is used again
        for (int k = i; k < issued; ++k) mbar_wait(&wbar[k % SLOTS], (uint32_t)(k / SLOTS) & 1u, kQdWaitNs / 8);
    }

    // ---- the warps' parts: (m, l) per head, accumulators [warp][head][d] over the ring ----
    __syncthreads();   // every warp is done with its slots
    float *part = reinterpret_cast<float *>(smem);
    const int GD = G * D;
    part_w.store(ml + warp * 32, part + warp * GD, G, lane);
    __syncthreads();
    float *comb = part + kQdWarps * GD;   // the CTA's accumulators, unnormalised
    float *cml = ml + kQdWarps * 32;
    const int64_t ob = ((int64_t)s * p.Hq + (int64_t)h * G) * D;
    for (int e = tid; e < GD; e += kQdWarps * 32) {
        const int hh = e / D;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kQdWarps; ++w) M = fmaxf(M, ml[w * 32 + hh]);
        const float sub = M == -INFINITY ? 0.f : M;
        float o = 0.f, L = 0.f;
#pragma unroll
        for (int w = 0; w < kQdWarps; ++w) {
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
    for (int e = rank * slice + tid; e < e_hi; e += kQdWarps * 32) {
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

template <typename T, int D, int NT, bool MANY, bool RES>
static int launch_quant_decode(const QuantDecodeParams &prm, const CUtensorMap &tk, const CUtensorMap &tv, int grid, int ranks,
                               cudaStream_t stream) {
    constexpr int kSmem = QuantShape<D, MANY>::SMEM_BYTES;
    static unsigned long long attr_set = 0;   // per instantiation and device
    if (!done_on_device(&attr_set)) {
        cudaError_t e = cudaFuncSetAttribute(quant_decode_kernel<T, D, NT, MANY, RES>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(quant_decode_kernel<T, D, NT, MANY, RES>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return cuda_fail(e);
        mark_done_on_device(&attr_set);
    }
    cudaError_t e = launch_cluster(quant_decode_kernel<T, D, NT, MANY, RES>, grid, ranks, kQdWarps * 32, kSmem, stream, prm, tk, tv);
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? PKV_OK : cuda_fail(e);
}

// The form and the CTAs per range, from the number of ranges, the blocks that
// one can have, and whether MANY is built for the group size.
template <typename T, int D, bool RES>
static int quant_decode(const QuantDecodeParams &prm, const CUtensorMap &tk, const CUtensorMap &tv, int64_t ranges,
                        int64_t blocks, int sms, cudaStream_t stream) {
    constexpr int kFew = QuantShape<D, false>::PER_SM, kMany = QuantShape<D, true>::PER_SM;
    // CTAs per range: as many as all fit on the GPU at once, each with at least two blocks a warp
    int ranks = (int)std::min<int64_t>({kQdMaxCluster, 2 * sms / ranges, blocks / (2 * kQdWarps)});
    if (ranks > 8 && ranks < kQdMaxCluster) ranks = 8;
    // a call of few CTAs is bound by a warp's chain of latencies: one block a warp, up to a CTA per SM
    ranks = std::max(ranks, (int)std::min<int64_t>({8, sms / ranges, blocks / kQdWarps}));
    if (ranks < 1) ranks = 1;
    const int grid = (int)(ranges * ranks);
    if (prm.G > 8) return launch_quant_decode<T, D, 2, false, RES>(prm, tk, tv, grid, ranks, stream);
    auto waves = [&](int per_sm) { return (ranges + per_sm * sms - 1) / (per_sm * sms) * per_sm; };
    if (ranges > 2 * sms && (ranges >= 6 * sms || blocks <= 32 || waves(kMany) <= waves(kFew)))
        return launch_quant_decode<T, D, 1, true, RES>(prm, tk, tv, grid, ranks, stream);
    return launch_quant_decode<T, D, 1, false, RES>(prm, tk, tv, grid, ranks, stream);
}

// A cache of codes as rows of 128 bytes (a token's, or with head_dim 64 two tokens'); a box is a tile.  Rows past the
// pool read 0.
static int encode_code_map(CUtensorMap *map, const void *base, int num_blocks, int num_kv_heads, int head_dim) {
    const uint64_t dims[2] = {64, (uint64_t)num_blocks * num_kv_heads * head_dim / 8};   // in 16-bit elements
    const uint64_t strides[1] = {128};
    const uint32_t box[2] = {64, (uint32_t)head_dim / 8};
    return encode_tiled_map(map, base, 2, dims, strides, box);
}

}  // namespace pkv

extern "C" int pkv_paged_decode_attention_e4m3(void *out, const void *q, const void *k_cache, const void *v_cache,
                                               const float *kv_scales, const int32_t *block_tables, int max_blocks_per_seq,
                                               const int32_t *context_lens, int num_seqs, int num_blocks, int num_q_heads,
                                               int num_kv_heads, int head_dim, int block_size, int window, int num_sinks,
                                               float scale, int dtype, int out_dtype, int *dev_status, void *stream) {
    pkv::NvtxRange nvtx_range("pkv_paged_decode_attention_e4m3");
    using namespace pkv;
    int rc = quant_attention_refusal(num_seqs, num_blocks, num_q_heads, num_kv_heads, head_dim, block_size, max_blocks_per_seq,
                                     window, num_sinks, scale, dtype, out_dtype);
    if (rc != PKV_OK) return rc;
    if ((int64_t)num_seqs * num_kv_heads * kQdMaxCluster >= (int64_t)1 << 31) return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PKV_OK;
    if (!out || !q || !k_cache || !v_cache || !kv_scales || !block_tables || !context_lens) return PKV_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(kv_scales, 8) ||
        !aligned(block_tables, 4) || !aligned(context_lens, 4))
        return PKV_ERR_INVALID_ARG;
    int sms = 0;
    rc = current_sm_count(&sms);
    if (rc != PKV_OK) return rc;
    CUtensorMap tk, tv;
    rc = encode_code_map(&tk, k_cache, num_blocks, num_kv_heads, head_dim);
    if (rc != PKV_OK) return rc;
    rc = encode_code_map(&tv, v_cache, num_blocks, num_kv_heads, head_dim);
    if (rc != PKV_OK) return rc;
    QuantDecodeParams prm;
    prm.out = out;
    prm.q = q;
    prm.scales = kv_scales;
    prm.block_tables = block_tables;
    prm.context_lens = context_lens;
    prm.dev_status = dev_status;
    prm.max_blocks = max_blocks_per_seq;
    prm.num_blocks = num_blocks;
    prm.Hq = num_q_heads;
    prm.Hkv = num_kv_heads;
    prm.G = num_q_heads / num_kv_heads;
    const int64_t capacity = (int64_t)max_blocks_per_seq * 16;
    prm.window = window < capacity ? window : (int)capacity;   // no context is longer
    prm.sinks = num_sinks < capacity ? num_sinks : (int)capacity;
    prm.scale_log2 = scale * 1.4426950408889634f;
    prm.out_dtype = out_dtype;
    const int64_t most = ((int64_t)prm.sinks + 15) / 16 + ((int64_t)window + 14) / 16 + 1;
    const int64_t blocks = std::min<int64_t>(most, max_blocks_per_seq);
    const int64_t ranges = (int64_t)num_seqs * num_kv_heads;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    auto run = [&](auto type, auto residual) {
        using T = decltype(type);
        constexpr bool RES = decltype(residual)::value;
        return head_dim == 128 ? quant_decode<T, 128, RES>(prm, tk, tv, ranges, blocks, sms, st)
                               : quant_decode<T, 64, RES>(prm, tk, tv, ranges, blocks, sms, st);
    };
    if (dtype == PKV_DTYPE_F16) return run(__half(), std::true_type());
    return out_dtype == PKV_DTYPE_F32 ? run(__nv_bfloat16(), std::true_type()) : run(__nv_bfloat16(), std::false_type());
}
