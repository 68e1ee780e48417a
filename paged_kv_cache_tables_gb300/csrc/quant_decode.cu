// Decode attention over the cache held in 8 bits
// (pkv_paged_decode_attention_e4m3).
//
// Mathematics.  As window_decode.cu, with K_t = k_t a_j and V_t = v_t b_j, k and
// v the e4m3 codes and a, b the scales of t's block j.  a multiplies the scores,
// and b is taken into the softmax: with
//     y_t = scale2 a_j (q . k_t) + log2 b_j,   P_t = 2^(y_t - m + 7),  m >= y_t - 8,
// m the running maximum of y, O = sum P_t v_t and l = sum P_t / b_j give out = O / l.
// So P is below 2^15 and about 2^7 for the weight that counts most, whatever the
// scales are, and goes to the tensor cores as fp16 value and fp16 rounding
// residual, against codes converted to fp16 (exact).
//
// The codes of K are multiplied as they are: a query is split into e4m3 terms,
//     q = f (t_0 + t_1 / 16 [+ t_2 / 256]),
// f a power of two per head that puts its largest element into [128, 256).  Each
// term takes four bits, so two hold a bf16 element exactly, down to 2^-13 of the
// head's largest, and three an fp16 one, down to 2^-14; smaller ones are off by at
// most 2^-21 of it, or 2^-25.
//
// Layout.  Tokens are the rows of S^T = K Q^T, head_dim those of O^T = V^T P^T.
// Four heads are the eight columns of a tile: of S^T a head's two terms, of P^T
// its value and its residual, so that one product takes both, and a lane's
// scores, weights and accumulators belong to one head.  P^T is P transposed, 8 x 8
// at a time (movmatrix).  A 16-byte piece of a row goes to one lane, so that the
// dimensions of a fragment are not in their order in memory but in one that suits
// these loads:
//   S^T   lane (g, t4) takes 16 dimensions 16 (t4 + 4 j) .. of tokens rho(g), rho(g) + 8
//   O^T   lane (g, t4) takes head_dim / 8 dimensions from g on, of tokens
//         rho(2 t4), rho(2 t4 + 1), and 8 further; bytes of two tokens are put
//         side by side before they are converted
// rho permutes the tokens of a group of 8 so that neither load meets a bank
// twice, the pieces of a 128-byte row (one token's codes, or with head_dim 64 two
// tokens') being swizzled by the row.
//
// A cluster of CTAs takes a (sequence, KV head) range, as in window_decode.cu; each
// warp runs a ring of its own, filled by 16-byte asynchronous copies.
//
// What bounds it: HBM.  256 sequences x 8 KV heads of 1,400 tokens (740 MB of codes
// and scales): 112.5 us, 97 % of the measured copy rate (a 16-bit cache, twice the
// bytes, 205); fp16 queries, whose third term is a product more, 120.  7 x 8 of
// 60,000 to 131,072: 208 us, 97 % of the floor of the lengths that were timed.  256 of
// 32 to 8,192 tokens: 118 us, 95 % (fp16 123): what is left there is the order (below)
// and the last ranges.  With a window of 1,024 and 64 first tokens 57, 84 %: a range
// is at most 69 blocks and starts with its length, table and scales; 64 x 8 behind a
// window of 4,096 89, 90 %.  Groups of 8 heads: 78 us for 372 MB (70 %), bound by the
// products and the softmax, 350 instructions a block and warp instead of 200; of 16
// 67 for 188 MB (42 %), two ranges that load and convert the same blocks.
// Measured and left: codes of K converted to fp16 and tokens as columns, 390
// instructions a block, 119 us; with tokens as rows, 290, 113 us; TMA instead of
// the copies, whose issue costs a lane 48 cycles and some 20 instructions a tile, 7
// x 131,072: 228 us, small calls up to 6 % more; heads as rows, with P^T in place
// without a transpose, 320 instructions, 117 us.
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

struct QuantDecodeParams {
    void *out;
    const void *q, *k_cache, *v_cache;
    const float *scales;
    const int32_t *block_tables;
    const int32_t *context_lens;
    int *dev_status;
    int num_seqs, max_blocks, num_blocks, Hq, Hkv, G;
    int parts;          // of a group of query heads, each a range of its own
    int window, sinks;
    float scale_log2;   // scale * log2(e): scores in base-2 units
    int out_dtype;
    bool ordered;       // the longest sequences first
};

// Two forms for up to 4 heads a KV head.  PAIRS: two blocks a step, three CTAs an
// SM, for long ranges, where a warp's time for a step is a chain of latencies that
// two blocks share; otherwise one block a step and four CTAs, for short ranges,
// where what counts is how many are under way.  us, PAIRS / not (both with TMA, on
// other lengths than above): 256 sequences x 8 of 32 to 8,192 tokens 127 / 144, 40 x 8
// of 2,048 30.6 / 35.4; 1,000 x 8 of 100 to 600 117 / 108, 256 x 8 of 30 to 130 22.5 /
// 19.0.  In between, up to 128 blocks, a call whose CTAs are more than three an SM and
// no more than four (58 to 76 sequences x 8) is one wave in the second form and two in
// the first: of equal length 28.5 / 25.5 (60 of 1,000), 29.9 / 26.4 (64 of 1,000), 55.7
// / 46.8 (64 of 2,000), 58.6 / 52.8 (76 of 2,000), fp16 46.6 / 38.2 (72 of 1,400).  (Of
// unequal length the second wave may be the short ones and hide, 26.7 / 29.7 for 60 of
// 300 to 2,000, 28.3 / 34.0 for 72, but the host does not know lengths.)  With heads of
// 64 pairs leave registers for four CTAs, and are for split ranges too (64 x 8 of 64 to
// 4,096 21.6 / 23.3, 128 x 8 of 2,000 48 / 52 in three CTAs; with heads of 128 split
// ranges take longer, 16 x 8 of 8,000 57 / 47).  More heads (NT == 2, up to 8, larger
// groups in parts) have one form: their accumulators leave registers for one block a
// step and three CTAs (two, with pairs: 81 us for 79).
template <int D, int NT, bool PAIRS>
struct QuantShape {
    static constexpr int TILE_BYTES = 16 * D;
    static constexpr int BLOCK_BYTES = 2 * TILE_BYTES;  // K then V
    static constexpr int STEP = PAIRS ? 2 : 1;          // blocks a warp takes at a time: a slot of its ring
    static constexpr int SLOT_BYTES = STEP * BLOCK_BYTES;
    static constexpr int PER_SM = (PAIRS && D == 128) || NT > 1 ? 3 : 4;
    static constexpr int SLOTS = (PER_SM == 3 ? 16 : 12) * 1024 / SLOT_BYTES;
    static constexpr int RING_BYTES = kQdWarps * SLOTS * SLOT_BYTES;
    // behind the ring: scales of 32 blocks a warp, then (m, l) of each warp and of the CTA
    static constexpr int OFF_SCALES = RING_BYTES;
    static constexpr int OFF_ML = OFF_SCALES + kQdWarps * 32 * 8;
    static constexpr int SMEM_BYTES = OFF_ML + (kQdWarps + 1) * 32 * 4;
    static_assert((kQdWarps + 1) * 4 * NT * D * 4 <= RING_BYTES, "the parts take the ring's place");
    static_assert(STEP * SLOTS <= 32, "the first loads come from one window of blocks");
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

__device__ __forceinline__ float2 ld_shared_v2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void st_shared_v2(uint32_t addr, float2 v) {
    asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(v.x), "f"(v.y) : "memory");
}

// 16 bytes to shared memory, asynchronously; the first n of them read, the others 0.
__device__ __forceinline__ void copy16(uint32_t to, const void *from, uint32_t n) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(n) : "memory");
}

__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// Until all but the last N of this thread's groups have landed.
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint2 lds64(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}

// D = A(16x32, row) * B(32x8, col) + D, e4m3 codes, fp32 accumulators.
__device__ __forceinline__ void mma_codes(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The transpose of an 8 x 8 matrix of 16-bit elements, a pair a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// A warp's part of a range.  The heads of the group go four to a tile (NT
// tiles); lane (g, t4) has head t4 of each, of tokens rho(g) and rho(g) + 8.
// (Fp16 queries' third terms have a product of their own.)
template <typename T, int D, int NT, bool PAIRS>
struct QuantPart {
    using Sh = QuantShape<D, NT, PAIRS>;
    static constexpr int STEP = Sh::STEP;
    static constexpr int KT = D / 32;        // steps of 32 dimensions
    static constexpr int MT = D / 16;        // tiles of 16 output rows
    static constexpr int NW = D / 32;        // 4-byte words of a token's codes that a lane takes of V
    static constexpr int QT = std::is_same<T, __half>::value ? 2 : 1;   // products of a query's terms
    uint32_t qb[KT][NT][QT][2];
    float acc[MT][NT][4];                    // [output rows][tile][row g value, residual, row g + 8 value, residual]
    float m_run[NT], off[NT];                // running maximum; what P subtracts
    float l_run[NT];
    float qscale[NT];                        // a head's score scale, its query's power of two taken back

    // q: G rows of D elements
    __device__ __forceinline__ void start(const T *q, int G, float scale_log2, int lane) {
        const int g = lane >> 2, t4 = lane & 3;
#pragma unroll
        for (int pn = 0; pn < NT; ++pn) {
            // column g of the tile: term g & 1 of head g / 2
            const int head = pn * 4 + (g >> 1);
            float x[D / 64][16];
            float top = 0.f;
#pragma unroll
            for (int j = 0; j < D / 64; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint4 *at = reinterpret_cast<const uint4 *>(q + head * D + 16 * (t4 + 4 * j)) + i;
                    const uint4 v = head < G ? *at : make_uint4(0u, 0u, 0u, 0u);
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 f = pair_to_f32<T>(w[e]);
                        x[j][8 * i + 2 * e] = f.x;
                        x[j][8 * i + 2 * e + 1] = f.y;
                    }
                }
            uint32_t bits = 0;
#pragma unroll
            for (int j = 0; j < D / 64; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e) bits = max(bits, __float_as_uint(x[j][e]) & 0x7fffffffu);
            bits = max(bits, __shfl_xor_sync(0xffffffffu, bits, 1));
            bits = max(bits, __shfl_xor_sync(0xffffffffu, bits, 2));
            const int e = min(max((int)(bits >> 23), 8), 254);     // exponent field of the largest
            const float f = __uint_as_float((uint32_t)(261 - e) << 23);
            // (a query that is not finite has no finite output)
            const float back = bits >= 0x7f800000u ? __uint_as_float(0x7fffffffu) : __uint_as_float((uint32_t)(e - 7) << 23);
            qscale[pn] = __shfl_sync(0xffffffffu, back, 8 * t4) * scale_log2;
#pragma unroll
            for (int j = 0; j < D / 64; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float r[4] = {x[j][4 * i] * f, x[j][4 * i + 1] * f, x[j][4 * i + 2] * f, x[j][4 * i + 3] * f};
                    uint32_t term[3];
#pragma unroll
                    for (int u = 0; u < 3; ++u) {
                        term[u] = to_e4m3x4(r[0], r[1], r[2], r[3]);
                        uint32_t lo, hi;
                        e4m3x4_to_f16x4(term[u], lo, hi);
                        const float2 a = f16x2_to_f32(lo), b = f16x2_to_f32(hi);
                        r[0] = (r[0] - a.x) * 16.f, r[1] = (r[1] - a.y) * 16.f;
                        r[2] = (r[2] - b.x) * 16.f, r[3] = (r[3] - b.y) * 16.f;
                    }
                    qb[2 * j + (i >> 1)][pn][0][i & 1] = g & 1 ? term[1] : term[0];
                    if constexpr (QT == 2) qb[2 * j + (i >> 1)][pn][1][i & 1] = g & 1 ? 0u : term[2];
                }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[mt][pn][e] = 0.f;
            m_run[pn] = -INFINITY;
            off[pn] = -7.f;
            l_run[pn] = 0.f;
        }
    }

    // STEP blocks of 16 tokens in the ring slot at `slot`, of scales sc (K, V); bit
    // t of `bits` set where token t of them is seen (all of them: ALL).
    // `release` runs once the slot has been read.
    template <bool ALL, typename F>
    __device__ __forceinline__ void attend(uint32_t slot, const float2 (&sc)[STEP], uint32_t bits, int lane, F release) {
        const int g = lane >> 2, t4 = lane & 3;
        // S^T = K Q^T
        float s[STEP][NT][QT][4];
#pragma unroll
        for (int b = 0; b < STEP; ++b)
#pragma unroll
            for (int pn = 0; pn < NT; ++pn)
#pragma unroll
                for (int u = 0; u < QT; ++u)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[b][pn][u][e] = 0.f;
        const int tok_k = token_at<D>(g);
#pragma unroll
        for (int b = 0; b < STEP; ++b)
#pragma unroll
            for (int j = 0; j < D / 64; ++j) {
                const uint4 k0 = lds128(slot + b * Sh::BLOCK_BYTES + piece_at<D>(tok_k, t4 + 4 * j));
                const uint4 k1 = lds128(slot + b * Sh::BLOCK_BYTES + piece_at<D>(tok_k + 8, t4 + 4 * j));
#pragma unroll
                for (int pn = 0; pn < NT; ++pn)
#pragma unroll
                    for (int u = 0; u < QT; ++u) {
                        mma_codes(s[b][pn][u], k0.x, k1.x, k0.y, k1.y, qb[2 * j][pn][u][0], qb[2 * j][pn][u][1]);
                        mma_codes(s[b][pn][u], k0.z, k1.z, k0.w, k1.w, qb[2 * j + 1][pn][u][0], qb[2 * j + 1][pn][u][1]);
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

        // y in place of the scores: [block][tile][token rho(g), token rho(g) + 8]
        float y[STEP][NT][2], rv[STEP];
        bool past = false;
#pragma unroll
        for (int b = 0; b < STEP; ++b) {
            const float lv = log2_approx(sc[b].y);
            rv[b] = exp2_approx(-lv);
#pragma unroll
            for (int pn = 0; pn < NT; ++pn)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float low = s[b][pn][0][2 * e + 1];
                    if constexpr (QT == 2) low = fmaf(s[b][pn][1][2 * e], 0.0625f, low);
                    y[b][pn][e] = fmaf(fmaf(low, 0.0625f, s[b][pn][0][2 * e]), qscale[pn] * sc[b].x, lv);
                    if (!ALL && !((bits >> (16 * b + tok_k + 8 * e)) & 1u)) y[b][pn][e] = -INFINITY;
                    past |= y[b][pn][e] > m_run[pn] + 8.f;
                }
        }
        // the maximum is only moved when it grows by more than 2^8
        if (__any_sync(0xffffffffu, past)) {
#pragma unroll
            for (int pn = 0; pn < NT; ++pn) {
                float mx = fmaxf(y[0][pn][0], y[0][pn][1]);
#pragma unroll
                for (int b = 1; b < STEP; ++b) mx = fmaxf(mx, fmaxf(y[b][pn][0], y[b][pn][1]));
#pragma unroll
                for (int d = 4; d < 32; d *= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                if (mx > m_run[pn] + 8.f) {
                    const float alpha = exp2_approx(m_run[pn] - mx);
                    m_run[pn] = mx;
                    off[pn] = mx - 7.f;
                    l_run[pn] *= alpha;
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[mt][pn][e] *= alpha;
                }
            }
        }
        // hidden positions may hold anything (even NaN codes): zero, so that 0 x
        // garbage cannot reach the accumulator
        if constexpr (!ALL) {
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
            // P^T fragments: tokens 0..7 and 8..15 of the block; columns value and residual of each head
            uint32_t pb[NT][2];
#pragma unroll
            for (int pn = 0; pn < NT; ++pn) {
                const float w0 = exp2_approx(y[b][pn][0] - off[pn]), w1 = exp2_approx(y[b][pn][1] - off[pn]);
                l_run[pn] = fmaf(w0 + w1, rv[b], l_run[pn]);
                uint32_t value, rest;
                pack2_split<__half>(w0, w1, value, rest);
                pb[pn][0] = transpose8(__byte_perm(value, rest, 0x5410u));
                pb[pn][1] = transpose8(__byte_perm(value, rest, 0x7632u));
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
                    for (int pn = 0; pn < NT; ++pn) mma_16816<__half>(acc[2 * i + half][pn], a, pb[pn][0], pb[pn][1]);
                }
        }
    }

    // (m, l) of the heads at ml[head], ml[16 + head]; accumulators at part[head * D + d].
    __device__ __forceinline__ void store(float *ml, float *part, int G, int lane) {
        const int g = lane >> 2, t4 = lane & 3;
#pragma unroll
        for (int pn = 0; pn < NT; ++pn) {
            const int head = pn * 4 + t4;
            float l = l_run[pn];
#pragma unroll
            for (int d = 4; d < 32; d *= 2) l += __shfl_xor_sync(0xffffffffu, l, d);
            if (g == 0) {
                ml[head] = m_run[pn];
                ml[16 + head] = l;
            }
            if (head < G)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
                    *reinterpret_cast<float2 *>(part + head * D + g * (D / 8) + 2 * mt) =
                        make_float2(acc[mt][pn][0] + acc[mt][pn][1], acc[mt][pn][2] + acc[mt][pn][3]);
        }
    }
};

constexpr int kQdMaxOrdered = 1024;

// The sequence at `place` when the longest (by visible blocks, in steps of a
// quarter octave) go first, equals in the order of the batch.  All threads of the
// CTA; `scratch` holds 1.5 KB + 16 bytes.
__device__ __forceinline__ int sequence_at(const QuantDecodeParams &p, int place, uint8_t *scratch, int tid, int threads) {
    int *count = reinterpret_cast<int *>(scratch);          // [128] sequences of each length class, longest first
    uint8_t *cls = scratch + 512;                           // [num_seqs]
    int *found = reinterpret_cast<int *>(scratch + 512 + kQdMaxOrdered);
    for (int i = tid; i < 128; i += threads) count[i] = 0;
    __syncthreads();
    for (int i = tid; i < p.num_seqs; i += threads) {
        const int blocks = Visible(p, __ldg(p.context_lens + i)).count;
        const int c = blocks > 0 ? min((int)(__float_as_uint((float)blocks) >> 21) - 4 * 127, 126) + 1 : 0;
        cls[i] = (uint8_t)(127 - c);
        atomicAdd(&count[127 - c], 1);
    }
    __syncthreads();
    if (tid < 32) {
        const int4 n = reinterpret_cast<const int4 *>(count)[tid];
        int before = n.x + n.y + n.z + n.w;
        const int mine = before;
        for (int d = 1; d < 32; d *= 2) {
            const int up = __shfl_up_sync(0xffffffffu, before, d);
            if (tid >= d) before += up;
        }
        before -= mine;
        // the lane whose classes hold the place; the class, and the place within it
        const int at = place - before;
        int c = 0, rest = at;
        if (rest >= n.x) c = 1, rest -= n.x;
        if (c == 1 && rest >= n.y) c = 2, rest -= n.y;
        if (c == 2 && rest >= n.z) c = 3, rest -= n.z;
        const uint32_t who = __ballot_sync(0xffffffffu, at >= 0 && at < mine);
        const int lane = __ffs(who) - 1;
        c = __shfl_sync(0xffffffffu, 4 * tid + c, lane);
        rest = __shfl_sync(0xffffffffu, rest, lane);
        for (int i = 0; i < p.num_seqs; i += 32) {
            const uint32_t equal = __ballot_sync(0xffffffffu, i + tid < p.num_seqs && cls[i + tid] == c);
            const int n_here = __popc(equal);
            if (rest < n_here) {
                if ((equal >> tid & 1u) && __popc(equal & ((1u << tid) - 1u)) == rest) *found = i + tid;
                break;
            }
            rest -= n_here;
        }
    }
    __syncthreads();
    const int s = *found;
    __syncthreads();
    return s;
}

template <typename T, int D, int NT, bool PAIRS>
__global__ void __launch_bounds__(kQdWarps * 32, QuantShape<D, NT, PAIRS>::PER_SM)
    quant_decode_kernel(const QuantDecodeParams p) {
    using Sh = QuantShape<D, NT, PAIRS>;
    constexpr int SLOTS = Sh::SLOTS, STEP = Sh::STEP;
    extern __shared__ __align__(128) uint8_t smem[];
    float *ml = reinterpret_cast<float *>(smem + Sh::OFF_ML);   // [warp][m 16, l 16], then the CTA's
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = (int)cluster_ctarank(), ranks = (int)cluster_nctarank();
    const int range = blockIdx.x / ranks;
    // the range: a sequence's place, a KV head, and a part of its group of query heads (parts side by side, so that a
    // second one finds K and V in L2)
    const int unit = range / p.parts, part_of = range - unit * p.parts;
    const int place = unit / p.Hkv, h = unit - place * p.Hkv;
    const int G = min(4 * NT, p.G - part_of * 4 * NT), hq0 = h * p.G + part_of * 4 * NT;

    uint8_t *wring = smem + warp * SLOTS * Sh::SLOT_BYTES;
    float2 *wscales = reinterpret_cast<float2 *>(smem + Sh::OFF_SCALES) + warp * 32;
    pdl_wait_primary();
    pdl_launch_dependents();

    // ---- the range's visible blocks, and this warp's share ----
    constexpr int WARPS = kQdWarps;
    const int s = p.ordered ? sequence_at(p, place, smem, tid, WARPS * 32) : place;
    const Visible vis(p, __ldg(p.context_lens + s));
    if (vis.bad && tid == 0 && rank == 0 && hq0 == 0) set_status(p.dev_status, PKV_DEV_BAD_CONTEXT);
    const int v_lo = (int)((int64_t)vis.count * rank / ranks), v_hi = (int)((int64_t)vis.count * (rank + 1) / ranks);
    const int n = max(0, (v_hi - v_lo - warp + WARPS - 1) / WARPS);
    auto logical = [&](int i) { return vis.logical(v_lo + warp + WARPS * i); };
    const int32_t *row = p.block_tables + (int64_t)s * p.max_blocks;
    // Lane i has the tile of this warp's block 32 k + i, k the window of 32 that
    // loads are issued from, and of the window after it; the scales of window k go
    // to shared memory when its first block is taken.
    const int no_tile = p.num_blocks * p.Hkv;   // past the end: the load fills zeros
    auto tile_of = [&](int i) {
        if (i >= n) return no_tile;
        const int blk = __ldg(row + logical(i));
        if (blk >= 0 && blk < p.num_blocks) return blk * p.Hkv + h;
        set_status(p.dev_status, PKV_DEV_BAD_BLOCK_ID);
        return no_tile;
    };
    int tile = 0, tile_next = tile_of(lane);
    float2 sc_mine;
    const int steps = (n + STEP - 1) / STEP;
    const uint32_t ring = smem_addr(wring), scales = smem_addr(wscales);
    // A tile goes to shared memory 16 bytes a lane at a time: piece 32 i + lane to
    // row 4 i + lane / 8 of 128 bytes, swizzled by its row.
    const uint32_t to_even = (lane >> 3) * 128 + (((lane & 7) ^ (lane >> 3)) << 4);
    const uint32_t to_odd = (lane >> 3) * 128 + (((lane & 7) ^ ((lane >> 3) + 4)) << 4);
    const uint8_t *kc = static_cast<const uint8_t *>(p.k_cache) + lane * 16, *vc = static_cast<const uint8_t *>(p.v_cache) + lane * 16;
    auto issue = [&](int j, int slot) {   // step j's blocks
        const int at = STEP * j & 31;
        if (at == 0) {
            tile = tile_next;
            sc_mine = tile < no_tile ? __ldg(reinterpret_cast<const float2 *>(p.scales) + tile) : make_float2(1.f, 1.f);
            tile_next = tile_of(STEP * j + 32 + lane);
        }
#pragma unroll
        for (int b = 0; b < STEP; ++b) {
            const int y = __shfl_sync(0xffffffffu, tile, at + b);
            const uint32_t n_bytes = y < no_tile ? 16 : 0;      // (no tile: zeros)
            const int64_t from = (int64_t)(y < no_tile ? y : 0) * Sh::TILE_BYTES;
            const uint32_t to = ring + slot * Sh::SLOT_BYTES + b * Sh::BLOCK_BYTES;
#pragma unroll
            for (int i = 0; i < Sh::TILE_BYTES / 512; ++i) {
                copy16(to + i * 512 + (i & 1 ? to_odd : to_even), kc + from + i * 512, n_bytes);
                copy16(to + Sh::TILE_BYTES + i * 512 + (i & 1 ? to_odd : to_even), vc + from + i * 512, n_bytes);
            }
        }
    };
    // (a group of copies a step, empty past the last one, so that the groups waited for are counted alike)
#pragma unroll
    for (int j = 0; j < SLOTS; ++j) {
        if (j < steps) issue(j, j);
        copies_commit();
    }

    QuantPart<T, D, NT, PAIRS> part_w;
    part_w.start(static_cast<const T *>(p.q) + ((int64_t)s * p.Hq + hq0) * D, G, p.scale_log2, lane);
    // entries [full_lo, full_hi) of the list are blocks that are seen whole
    const int full_lo = ((vis.w0 + 15) >> 4) - vis.skip, full_hi = min((vis.ctx >> 4) - vis.skip, v_hi);

    int slot = 0;
    for (int i = 0; i < steps; ++i) {
        if ((STEP * i & 31) == 0) {
            __syncwarp();
            st_shared_v2(scales + lane * 8, sc_mine);
        }
        copies_wait<SLOTS - 1>();
        __syncwarp();
        float2 sc[STEP];
#pragma unroll
        for (int b = 0; b < STEP; ++b) sc[b] = ld_shared_v2(scales + ((STEP * i & 31) + b) * 8);
        auto refill = [&] {
            __syncwarp();
            if (i + SLOTS < steps) issue(i + SLOTS, slot);
            copies_commit();
        };
        const int v0 = v_lo + warp + kQdWarps * STEP * i;
        if (v0 >= full_lo && v0 + kQdWarps * (STEP - 1) < full_hi) {
            part_w.template attend<true>(ring + slot * Sh::SLOT_BYTES, sc, 0u, lane, refill);
        } else {
            uint32_t bits = 0;
#pragma unroll
            for (int b = 0; b < STEP; ++b)
                if (STEP * i + b < n) bits |= vis.bits(logical(STEP * i + b), p.sinks) << (16 * b);
            part_w.template attend<false>(ring + slot * Sh::SLOT_BYTES, sc, bits, lane, refill);
        }
        if (++slot == SLOTS) slot = 0;
    }

    // ---- the warps' parts: (m, l) per head, accumulators [warp][head][d] over the ring ----
    __syncthreads();   // every warp is done with its slots
    float *part = reinterpret_cast<float *>(smem);
    const int GD = G * D;
    part_w.store(ml + warp * 32, part + warp * GD, G, lane);
    __syncthreads();
    float *comb = part + kQdWarps * GD;   // the CTA's accumulators, unnormalised
    float *cml = ml + kQdWarps * 32;
    const int64_t ob = ((int64_t)s * p.Hq + hq0) * D;
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

template <typename T, int D, int NT, bool PAIRS>
static int launch_quant_decode(const QuantDecodeParams &prm, int grid, int ranks, cudaStream_t stream) {
    constexpr int kSmem = QuantShape<D, NT, PAIRS>::SMEM_BYTES;
    static unsigned long long attr_set = 0;   // per instantiation and device
    if (!done_on_device(&attr_set)) {
        cudaError_t e = cudaFuncSetAttribute(quant_decode_kernel<T, D, NT, PAIRS>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(quant_decode_kernel<T, D, NT, PAIRS>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return cuda_fail(e);
        mark_done_on_device(&attr_set);
    }
    cudaError_t e = launch_cluster(quant_decode_kernel<T, D, NT, PAIRS>, grid, ranks, kQdWarps * 32, kSmem, stream, prm);
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? PKV_OK : cuda_fail(e);
}

// The form, the CTAs per range and the order, from the number of ranges and the
// blocks that one can have.
template <typename T, int D>
static int quant_decode(QuantDecodeParams &prm, int64_t blocks, int sms, cudaStream_t stream) {
    prm.parts = (prm.G + 7) / 8;
    const int64_t ranges = (int64_t)prm.num_seqs * prm.Hkv * prm.parts;
    auto power_below = [](int64_t n) {
        int r = 1;
        while (2 * r <= n && r < kQdMaxCluster) r *= 2;
        return r;
    };
    // CTAs per range.  A call of few CTAs is bound by a warp's chain of
    // latencies: down to a block a warp, up to a CTA per SM (8 ranges of 128 blocks:
    // 5.1 us in 128 CTAs, 16 in 8).  Otherwise a range is split where it has 96
    // blocks a CTA, while there are fewer than 12 CTAs an SM then: its length may
    // be far above the others', and an SM takes 2 MB no faster than in 45 us (24 x 8
    // of 500 to 30,000 tokens 73 us in 8 CTAs a range, 158 in one; 64 x 8 of 64 to
    // 4,096, heads of 64, 23 and 27; 16 x 8 of 8,000 45 and 52).  More CTAs than that cost more
    // than they even out (256 x 8 of 1,400: 132 us in two a range for 112).
    const int ranks = std::max(power_below(std::min<int64_t>(sms / ranges, blocks / kQdWarps)),
                               power_below(std::min<int64_t>(12 * sms / ranges, blocks / 96)));
    const int64_t ctas = ranges * ranks;
    // The longest first, where that evens out more than finding them costs a CTA
    // (256 x 8 of 32 to 8,192 tokens, other lengths than above: 147 us in the order
    // of the batch, 127; of 1,400 each 112 and 116).
    prm.ordered = ctas > 3 * sms && blocks > ctas / 13 && prm.num_seqs <= kQdMaxOrdered;
    if (prm.G > 4) return launch_quant_decode<T, D, 2, false>(prm, (int)ctas, ranks, stream);
    const bool pairs = D == 64 ? blocks > 48 * ranks
                               : ranks == 1 && blocks > 48 && !(blocks <= 128 && ctas <= 4 * sms && ctas > 3 * sms);
    if (pairs) return launch_quant_decode<T, D, 1, true>(prm, (int)ctas, ranks, stream);
    return launch_quant_decode<T, D, 1, false>(prm, (int)ctas, ranks, stream);
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
    if ((int64_t)num_seqs * num_q_heads * kQdMaxCluster >= (int64_t)1 << 31) return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PKV_OK;
    if (!out || !q || !k_cache || !v_cache || !kv_scales || !block_tables || !context_lens) return PKV_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(kv_scales, 8) ||
        !aligned(block_tables, 4) || !aligned(context_lens, 4))
        return PKV_ERR_INVALID_ARG;
    int sms = 0;
    rc = current_sm_count(&sms);
    if (rc != PKV_OK) return rc;
    QuantDecodeParams prm;
    prm.out = out;
    prm.q = q;
    prm.k_cache = k_cache;
    prm.v_cache = v_cache;
    prm.scales = kv_scales;
    prm.block_tables = block_tables;
    prm.context_lens = context_lens;
    prm.dev_status = dev_status;
    prm.num_seqs = num_seqs;
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
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dtype == PKV_DTYPE_BF16)
        return head_dim == 128 ? quant_decode<__nv_bfloat16, 128>(prm, blocks, sms, st)
                               : quant_decode<__nv_bfloat16, 64>(prm, blocks, sms, st);
    return head_dim == 128 ? quant_decode<__half, 128>(prm, blocks, sms, st)
                           : quant_decode<__half, 64>(prm, blocks, sms, st);
}
