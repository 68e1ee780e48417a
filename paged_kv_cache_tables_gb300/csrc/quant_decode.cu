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
//   S = Q K^T       lane (g, t4) takes 16 dimensions 16 (t4 + 4 j) .. of token rho(g)
//   O^T += V^T P^T  lane (g, t4) takes head_dim / 8 dimensions from g on, of tokens
//                   rho(2 t4), rho(2 t4 + 1), and 8 further; bytes of two tokens
//                   are put side by side before they are converted
// rho permutes the tokens of a group of 8 so that neither load meets a bank
// twice under TMA's 128-byte swizzle (a shared-memory row of 128 bytes is one
// token's codes, or with head_dim 64 two tokens').
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
    static constexpr int STAGE_BYTES = 2 * TILE_BYTES;  // K then V
    static constexpr int STAGES = D == 128 ? (MANY ? 4 : 6) : 8;
    static constexpr int STEP = 2;                      // blocks a warp takes at a time
    static constexpr int PER_SM = D == 128 && !MANY ? 2 : 3;
    static constexpr int RING_BYTES = kQdWarps * STAGES * STAGE_BYTES;
    // behind the ring: barriers, then (m, l) of each warp and of the CTA
    static constexpr int OFF_ML = RING_BYTES + kQdWarps * STAGES * 8;
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

// A warp's part of a range: query fragments (rows = heads of the group, padded
// to 16), accumulator, running maximum and sum.
template <typename T, int D, int NT, bool MANY, bool RES>
struct QuantPart {
    using Sh = QuantShape<D, MANY>;
    static constexpr int STEP = Sh::STEP;
    static constexpr int KT = D / 16;        // steps of 16 dimensions, and of 16 output rows
    static constexpr int NW = D / 32;        // 4-byte words of a token's codes that a lane takes of V
    uint32_t qa[KT][4];
    float acc[KT][NT][4];
    float m_run[NT], l_run[NT];
    float qscale[NT];                        // a head's score scale, its query's power of two taken back

    // q: G rows of D elements
    __device__ __forceinline__ void start(const T *q, int G, float scale_log2, int lane) {
        const int g = lane >> 2, t4 = lane & 3;
#pragma unroll
        for (int kk = 0; kk < KT; ++kk) qa[kk][1] = qa[kk][3] = 0u;   // rows 8..15, for groups of at most 8
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
            qscale[pn] = back * scale_log2;
#pragma unroll
            for (int kk = 0; kk < KT; ++kk) query4<T>(x[kk], f, qa[kk][pn], qa[kk][pn + 2]);
        }
#pragma unroll
        for (int mt = 0; mt < KT; ++mt)
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

    // STEP blocks of 16 tokens in ring slots at `slot`, of scales ks, vs; bit t of
    // `bits` set where token t of them is seen (some token of the first block
    // is).  `release` runs once the slots have been read.
    template <typename F>
    __device__ __forceinline__ void attend(const uint32_t (&slot)[STEP], const float (&ks)[STEP], const float (&vs)[STEP],
                                           uint32_t bits, int lane, F release) {
        const int g = lane >> 2, t4 = lane & 3;
        float s[2 * STEP][4];
#pragma unroll
        for (int nt = 0; nt < 2 * STEP; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
#pragma unroll
        for (int b = 0; b < STEP; ++b)
#pragma unroll
            for (int j = 0; j < D / 64; ++j) {
                const int tok = token_at<D>(g);
                const uint4 k0 = lds128(slot[b] + piece_at<D>(tok, t4 + 4 * j));
                const uint4 k1 = lds128(slot[b] + piece_at<D>(tok + 8, t4 + 4 * j));
                const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t x, y;
                    e4m3x4_to_f16x4(w0[i], x, y);
                    mma_16816<__half>(s[2 * b], qa[4 * j + i], x, y);
                    e4m3x4_to_f16x4(w1[i], x, y);
                    mma_16816<__half>(s[2 * b + 1], qa[4 * j + i], x, y);
                }
            }
        // [block][token rho(2 t4), rho(2 t4 + 1), and those + 8][words]
        uint32_t vw[STEP][4][NW];
#pragma unroll
        for (int b = 0; b < STEP; ++b)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int tok = token_at<D>(2 * t4 + (u & 1)) + 8 * (u >> 1);
                if constexpr (D == 128) {
                    const uint4 v = lds128(slot[b] + Sh::TILE_BYTES + piece_at<D>(tok, g));
                    vw[b][u][0] = v.x, vw[b][u][1] = v.y, vw[b][u][2] = v.z, vw[b][u][3] = v.w;
                } else {
                    const uint2 v = lds64(slot[b] + Sh::TILE_BYTES + piece_at<D>(tok, g >> 1) + (g & 1) * 8);
                    vw[b][u][0] = v.x, vw[b][u][1] = v.y;
                }
            }
        release();

        float lv[STEP], rv[STEP];
#pragma unroll
        for (int b = 0; b < STEP; ++b) {
            lv[b] = __log2f(vs[b]);
            rv[b] = exp2_approx(-lv[b]);
        }
        const bool all = bits == (uint32_t)((1ull << (16 * STEP)) - 1u);
        float pr[2 * STEP][2 * NT];
        float alpha[NT];
        bool moved = false;
#pragma unroll
        for (int pn = 0; pn < NT; ++pn) {
            float x[2 * STEP][2];
            float mx = -INFINITY;
#pragma unroll
            for (int nt = 0; nt < 2 * STEP; ++nt) {
                const float f = qscale[pn] * ks[nt >> 1];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    x[nt][e] = fmaf(s[nt][pn * 2 + e], f, lv[nt >> 1]);
                    if (!all && !((bits >> (nt * 8 + token_at<D>(2 * t4 + e))) & 1u)) x[nt][e] = -INFINITY;
                    mx = fmaxf(mx, x[nt][e]);
                }
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
            l_run[pn] *= alpha[pn];
#pragma unroll
            for (int b = 0; b < STEP; ++b) {
                float rs = 0.f;
#pragma unroll
                for (int nt = 2 * b; nt < 2 * b + 2; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        pr[nt][pn * 2 + e] = exp2_approx(x[nt][e] - (sub - 7.f));
                        rs += pr[nt][pn * 2 + e];
                    }
                l_run[pn] = fmaf(rs, rv[b], l_run[pn]);
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
        if (__any_sync(0xffffffffu, moved))
#pragma unroll
            for (int pn = 0; pn < NT; ++pn) {
                const float a_lo = __shfl_sync(0xffffffffu, alpha[pn], 8 * t4);
                const float a_hi = __shfl_sync(0xffffffffu, alpha[pn], 8 * t4 + 4);
#pragma unroll
                for (int mt = 0; mt < KT; ++mt) {
                    acc[mt][pn][0] *= a_lo;
                    acc[mt][pn][1] *= a_hi;
                    acc[mt][pn][2] *= a_lo;
                    acc[mt][pn][3] *= a_hi;
                }
            }
#pragma unroll
        for (int b = 0; b < STEP; ++b) {
            uint32_t pb0[NT][2], pb1[NT][2];
#pragma unroll
            for (int pn = 0; pn < NT; ++pn) {
                if constexpr (RES) {
                    pack2_split<__half>(pr[2 * b][pn * 2], pr[2 * b][pn * 2 + 1], pb0[pn][0], pb0[pn][1]);
                    pack2_split<__half>(pr[2 * b + 1][pn * 2], pr[2 * b + 1][pn * 2 + 1], pb1[pn][0], pb1[pn][1]);
                } else {
                    pb0[pn][0] = pack2<__half>(pr[2 * b][pn * 2], pr[2 * b][pn * 2 + 1]);
                    pb1[pn][0] = pack2<__half>(pr[2 * b + 1][pn * 2], pr[2 * b + 1][pn * 2 + 1]);
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
                        for (int pn = 0; pn < NT; ++pn) mma_16816<__half>(acc[2 * i + half][pn], a, pb0[pn][r], pb1[pn][r]);
                }
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
            for (int mt = 0; mt < KT; ++mt) {
                const int d0 = g * (D / 8) + 2 * mt;
                if (ha < G) *reinterpret_cast<float2 *>(part + ha * D + d0) = make_float2(acc[mt][pn][0], acc[mt][pn][2]);
                if (hb < G) *reinterpret_cast<float2 *>(part + hb * D + d0) = make_float2(acc[mt][pn][1], acc[mt][pn][3]);
            }
        }
    }
};

template <typename T, int D, int NT, bool MANY, bool RES>
__global__ void __launch_bounds__(kQdWarps * 32, NT == 1 ? QuantShape<D, MANY>::PER_SM : 2)
    quant_decode_kernel(const QuantDecodeParams p, const __grid_constant__ CUtensorMap tk,
                        const __grid_constant__ CUtensorMap tv) {
    using Sh = QuantShape<D, MANY>;
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
    auto issue = [&](int i) {
        const int blk = __shfl_sync(0xffffffffu, id, i & 31);
        if (lane == 0) {
            const bool bad = blk < 0 || blk >= p.num_blocks;
            if (bad) set_status(p.dev_status, PKV_DEV_BAD_BLOCK_ID);
            // past the end for a bad block id: the load fills zeros
            constexpr int kRows = D / 8;   // 128-byte rows of a tile
            const int y = bad ? p.num_blocks * p.Hkv * kRows : (blk * p.Hkv + h) * kRows;
            uint8_t *slot = wring + (i % STAGES) * Sh::STAGE_BYTES;
            uint64_t *bar = &wbar[i % STAGES];
            mbar_arrive_expect_tx(bar, Sh::STAGE_BYTES);
            tma_load_2d(slot, &tk, 0, y, bar, policy);
            tma_load_2d(slot + Sh::TILE_BYTES, &tv, 0, y, bar, policy);
        }
    };
    fetch(0);
    int issued = 0;
    for (; issued < min(n, STAGES); ++issued) issue(issued);

    QuantPart<T, D, NT, MANY, RES> part_w;
    part_w.start(static_cast<const T *>(p.q) + ((int64_t)s * p.Hq + (int64_t)h * G) * D, G, p.scale_log2, lane);
    const uint32_t ring_addr = smem_addr(wring);

    bool timed_out = false;
    int i = 0;   // blocks taken
    while (i < n) {
        // an odd block out is taken with itself, the second time all hidden
        const int k = min(STEP, n - i);
        uint32_t slot[STEP], bits = 0;
        float ks[STEP], vs[STEP];
        bool ok = true;
#pragma unroll
        for (int b = 0; b < STEP; ++b) {
            const int x = i + min(b, k - 1);
            ok = ok && mbar_wait(&wbar[x % STAGES], (uint32_t)(x / STAGES) & 1u, kQdWaitNs);
            slot[b] = ring_addr + (x % STAGES) * Sh::STAGE_BYTES;
            if (b < k) bits |= vis.bits(logical(x), p.sinks) << (16 * b);
            // (the 32 blocks of the last one issued, or those before)
            const bool now = x / 32 == (issued - 1) / 32;
            ks[b] = __shfl_sync(0xffffffffu, now ? sc.x : sc_before.x, x & 31);
            vs[b] = __shfl_sync(0xffffffffu, now ? sc.y : sc_before.y, x & 31);
        }
        if (!__all_sync(0xffffffffu, ok)) {
            timed_out = true;
            break;
        }
        i += k;
        part_w.attend(slot, ks, vs, bits, lane, [&] {
            fence_proxy_async_smem();
            __syncwarp();
            for (int u = 0; u < k && issued < n; ++u, ++issued) {
                if ((issued & 31) == 0) fetch(issued / 32);
                issue(issued);
            }
        });
    }
    if (timed_out) {
        if (lane == 0) set_status(p.dev_status, PKV_DEV_WAIT_TIMEOUT);
        // what is still in flight must land before the ring is used again
        for (int k = i; k < issued; ++k) mbar_wait(&wbar[k % STAGES], (uint32_t)(k / STAGES) & 1u, kQdWaitNs / 8);
    }

    // ---- the warps' parts: (m, l) per head, accumulators [warp][head][d] over the ring ----
    __syncthreads();   // every warp is done with its slots
    float *part = reinterpret_cast<float *>(smem);
    const int GD = G * D;
    part_w.finish();
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
