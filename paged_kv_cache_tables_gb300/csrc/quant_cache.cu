// The cache held in 8 bits: this step's rows quantised into it
// (pkv_kv_append_e4m3), and rows of sequences read back (pkv_kv_gather_e4m3).
//
// Mathematics.  A (block, KV head)'s K tile and V tile each have one scale s; a
// stored code c stands for c s.  Of the rows that a call writes to a tile, a is
// the largest finite |x|, and
//     s' = scale(a) where the call writes offset 0, else max(s, scale(a)),
//     row x -> e4m3(x / s'),   where s' > s the tile's other rows c -> e4m3(c s / s'),
// scale(a) the least power of two with a <= 448 scale(a).
//
// What bounds them: HBM, and for few rows the chain slot, row and scale, maximum,
// store.  Append of 256 decodes (8 heads of 128, bf16) 2.0 us, 4,327 mixed rows 7.0
// us (56 % of the measured copy rate), a prompt of 16,383 rows (16 heads of 64,
// fp16) 19.8 us (75 %; 8 heads of 128 18.7, 80 %); with a warp for every (token, head,
// K or V), most of which found another one to do their work, 4.9, 16 and 78 us.
// Read back: 64 sequences of up to 8,000 tokens (742 MB) 114 us, 96 %; 32-bit rows 190
// us, 96 %; 777 rows 4.1 us.  With 16 codes and 32 bytes of output a thread, halves of whose sectors were
// stored apart, and each row's sequence searched for by itself, 192 us.
#include <cuda_runtime.h>

#include <algorithm>

#include "pkv.h"
#include "pkv_device.cuh"
#include "pkv_host.h"
#include "pkv_quant.cuh"

namespace pkv {

struct QuantAppendParams {
    const void *k, *v;
    int64_t k_stride, v_stride;   // elements from a token to the next
    const int64_t *slots;
    uint8_t *k_cache, *v_cache;
    float *scales;                // [block][head][K, V]
    int *dev_status;
    int T, num_blocks, Hkv, span;
};

template <typename T>
constexpr uint32_t kInfBits = std::is_same<T, __nv_bfloat16>::value ? 0x7f80u : 0x7c00u;

// Largest magnitudes among pairs of 16-bit values so far, with eight more.
__device__ __forceinline__ uint32_t max_pair(uint32_t top, uint4 x) {
    return __vmaxu2(__vmaxu2(__vmaxu2(top, x.x & 0x7fff7fffu), __vmaxu2(x.y & 0x7fff7fffu, x.z & 0x7fff7fffu)), x.w & 0x7fff7fffu);
}

// The same of the finite ones only: four times the instructions, for rows that
// turn out to hold others.
template <typename T>
__device__ __forceinline__ uint32_t finite_max_pair(uint32_t top, uint4 x) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t lo = w[i] & 0x7fffu, hi = (w[i] >> 16) & 0x7fffu;
        lo = lo < kInfBits<T> ? lo : 0u;
        hi = hi < kInfBits<T> ? hi : 0u;
        top = __vmaxu2(top, lo | hi << 16);
    }
    return top;
}

// The largest finite magnitude that the lanes of `group` hold in their N pieces, as bits.
template <typename T, int N>
__device__ __forceinline__ uint32_t group_max(uint32_t group, const uint4 (&x)[N]) {
    uint32_t top = 0u;
#pragma unroll
    for (int e = 0; e < N; ++e) top = max_pair(top, x[e]);
    top = __reduce_max_sync(group, max(top & 0xffffu, top >> 16));
    if (top >= kInfBits<T>) {
        top = 0u;
#pragma unroll
        for (int e = 0; e < N; ++e) top = finite_max_pair<T>(top, x[e]);
        top = __reduce_max_sync(group, max(top & 0xffffu, top >> 16));
    }
    return top;
}

// Four codes times r, as codes.
__device__ __forceinline__ uint32_t rescale4(uint32_t codes, float r) {
    uint32_t a, b;
    e4m3x4_to_f16x4(codes, a, b);
    const float2 x = f16x2_to_f32(a), y = f16x2_to_f32(b);
    return to_e4m3x4(x.x * r, x.y * r, y.x * r, y.y * r);
}

// Eight values times f as codes.
template <typename T>
__device__ __forceinline__ uint2 codes8(uint4 x, float f) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    const uint64_t f2 = f2_pack(f, f);
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 a = pair_to_f32<T>(w[i]);
        f2_unpack(f2_mul(f2_pack(a.x, a.y), f2), v[2 * i], v[2 * i + 1]);
    }
    return make_uint2(to_e4m3x4(v[0], v[1], v[2], v[3]), to_e4m3x4(v[4], v[5], v[6], v[7]));
}

// The scale of a tile from that before (none where the block starts anew) and the
// largest magnitude written, as bits.
template <typename T>
__device__ __forceinline__ float new_scale(float before, uint32_t top) {
    return fmaxf(before > 0.f ? before : 0.f, block_scale(pair_to_f32<T>(top).x));   // (a scale that is none counts as 0)
}

// A CTA takes `span` tokens (up to 16): the blocks whose first row in the call is
// one of them, with all of their rows, which stand behind one another (up to 15
// of them past the span).  A decode's block has one row: LANES lanes take it,
// with its K and V and the two scales.  A chunk's have up to 16: a warp takes a
// (block, K or V, head) tile, its rows in registers between the maximum and the
// rounding.  gridDim.y CTAs share a span.
template <typename T, int D>
__global__ void __launch_bounds__(256, 4) kv_append_e4m3_kernel(const QuantAppendParams p) {
    constexpr int LANES = D / 8;          // lanes of a row, 8 values each
    constexpr int ROWS = 32 / LANES;      // rows a warp takes at a time
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t0 = (int64_t)blockIdx.x * p.span;
    const int sub = lane / LANES, col = lane % LANES;
    const T *k = static_cast<const T *>(p.k), *v = static_cast<const T *>(p.v);
    __shared__ uint8_t singles[8][32];    // per warp: lanes of the blocks with one row
    pdl_wait_primary();
    pdl_launch_dependents();
    // lane i: the slot of token t0 + i - 1
    const int64_t at = t0 + lane - 1;
    const int64_t slot = at >= 0 && at < p.T ? __ldg(p.slots + at) : -1;
    const int64_t block = slot < 0 ? -1 : slot >> 4;
    const int my_off = (int)(slot & 15);
    const bool inside = lane >= 1 && lane <= p.span;         // (tokens past the last have no slot)
    if (inside && block >= p.num_blocks && blockIdx.y == 0 && warp == 0) set_status(p.dev_status, PKV_DEV_BAD_SLOT);
    const int64_t before = __shfl_up_sync(0xffffffffu, block, 1), after = __shfl_down_sync(0xffffffffu, block, 1);
    const uint32_t changes = __ballot_sync(0xffffffffu, block != before);
    const bool first = inside && block >= 0 && block < p.num_blocks && block != before;
    const bool alone = first && (block != after || lane == 31);
    const uint32_t ones = __ballot_sync(0xffffffffu, alone);
    uint32_t runs = __ballot_sync(0xffffffffu, first && !alone);

    // ---- blocks with one row ----
    if (ones) {
        if (alone) singles[warp][__popc(ones & ((1u << lane) - 1u))] = (uint8_t)lane;
        __syncwarp();
        const int units = __popc(ones) * p.Hkv;
        const int stride = 8 * ROWS * gridDim.y;
        for (int u0 = (blockIdx.y * 8 + warp) * ROWS; u0 < units; u0 += stride) {
            const int u = u0 + sub;
            const bool on = u < units;
            const int i = on ? singles[warp][u / p.Hkv] : 0, h = on ? u % p.Hkv : 0;
            const int64_t mine = __shfl_sync(0xffffffffu, block, i);
            const int off = __shfl_sync(0xffffffffu, my_off, i);
            if (!on) continue;   // (whole groups of LANES lanes: what follows stays inside one)
            const uint32_t group = LANES == 16 ? 0xffffu << (sub * 16) : 0xffu << (sub * 8);
            const int64_t tile = mine * p.Hkv + h;
            const uint4 xk = __ldg(reinterpret_cast<const uint4 *>(k + (t0 + i - 1) * p.k_stride + h * D) + col);
            const uint4 xv = __ldg(reinterpret_cast<const uint4 *>(v + (t0 + i - 1) * p.v_stride + h * D) + col);
            float2 *scales = reinterpret_cast<float2 *>(p.scales) + tile;
            const float2 was = *scales;
            const float2 old = off ? make_float2(was.x > 0.f ? was.x : 0.f, was.y > 0.f ? was.y : 0.f) : make_float2(0.f, 0.f);
            const uint4 ks[1] = {xk}, vs[1] = {xv};
            const float2 now = make_float2(new_scale<T>(old.x, group_max<T>(group, ks)), new_scale<T>(old.y, group_max<T>(group, vs)));
            const float2 inv = make_float2(1.f / now.x, 1.f / now.y);
            uint8_t *ck = p.k_cache + tile * 16 * D, *cv = p.v_cache + tile * 16 * D;
            *reinterpret_cast<uint2 *>(ck + off * D + col * 8) = codes8<T>(xk, inv.x);
            *reinterpret_cast<uint2 *>(cv + off * D + col * 8) = codes8<T>(xv, inv.y);
            // a scale that grows takes the other rows along
            auto others = [&](uint8_t *tile_at, float ratio) {
                for (int e = col; e < D; e += LANES) {
                    if (e / (D / 16) == off) continue;
                    uint4 *at4 = reinterpret_cast<uint4 *>(tile_at) + e;
                    const uint4 c = *at4;
                    *at4 = make_uint4(rescale4(c.x, ratio), rescale4(c.y, ratio), rescale4(c.z, ratio), rescale4(c.w, ratio));
                }
            };
            if (off && now.x != was.x) others(ck, old.x * inv.x);
            if (off && now.y != was.y) others(cv, old.y * inv.y);
            if (col == 0 && (now.x != was.x || now.y != was.y)) *scales = now;
        }
        __syncwarp();
    }

    // ---- blocks with more ----
    const int per_block = 2 * p.Hkv;
    int item = blockIdx.y * 8 + warp;                         // among those of the block at hand
    while (runs) {
        const int i = __ffs(runs) - 1;                        // the lane of the block's first token
        const uint32_t next = i < 31 ? changes >> (i + 1) : 0u;
        const int n = min(next ? __ffs(next) : 32 - i, 16);   // its rows
        const int64_t mine = __shfl_sync(0xffffffffu, block, i);
        const uint32_t written = __reduce_or_sync(0xffffffffu, lane >= i && lane < i + n ? 1u << my_off : 0u);
        for (; item < per_block; item += 8 * gridDim.y) {
            const int kv = item >= p.Hkv, h = item - kv * p.Hkv;
            const int64_t tile = mine * p.Hkv + h;
            float *scale = p.scales + tile * 2 + kv;
            const float was = *scale;
            const int64_t stride = kv ? p.v_stride : p.k_stride;
            const T *rows = (kv ? v : k) + (t0 + i - 1) * stride + h * D;
            uint4 x[16 / ROWS];
#pragma unroll
            for (int e = 0; e < 16 / ROWS; ++e) {
                const int r = e * ROWS + sub;
                x[e] = r < n ? __ldg(reinterpret_cast<const uint4 *>(rows + r * stride) + col) : make_uint4(0u, 0u, 0u, 0u);
            }
            const bool anew = written & 1u;
            const float old = !anew && was > 0.f ? was : 0.f;
            const float now = new_scale<T>(old, group_max<T>(0xffffffffu, x));
            const float inv = 1.f / now;
            uint8_t *out = (kv ? p.v_cache : p.k_cache) + tile * 16 * D;
#pragma unroll
            for (int e = 0; e < 16 / ROWS; ++e) {
                const int r = e * ROWS + sub;
                const int off = __shfl_sync(0xffffffffu, my_off, (i + r) & 31);
                if (r < n) *reinterpret_cast<uint2 *>(out + off * D + col * 8) = codes8<T>(x[e], inv);
            }
            if (!anew && now != was) {
                const float ratio = old * inv;
                for (int e = lane; e < D; e += 32) {          // 16-byte pieces of the tile
                    if (written >> (e / (D / 16)) & 1u) continue;
                    uint4 *at4 = reinterpret_cast<uint4 *>(out) + e;
                    const uint4 c = *at4;
                    *at4 = make_uint4(rescale4(c.x, ratio), rescale4(c.y, ratio), rescale4(c.z, ratio), rescale4(c.w, ratio));
                }
            }
            if (lane == 0 && now != was) *scale = now;
        }
        item -= per_block;
        runs &= runs - 1;
    }
}

struct QuantGatherParams {
    void *k, *v;
    const uint8_t *k_cache, *v_cache;
    const float *scales;
    const int32_t *block_tables, *cu_seqlens, *first;
    int *dev_status;
    int max_blocks, num_blocks, num_seqs, total, Hkv, per_cta;
};

// N codes (16 bytes of output) times s, rounded once to the output's type.
template <typename O>
__device__ __forceinline__ uint4 values(uint2 codes, float s) {
    uint32_t a, b;
    e4m3x4_to_f16x4(codes.x, a, b);
    const float2 x = f16x2_to_f32(a), y = f16x2_to_f32(b);
    if constexpr (std::is_same<O, float>::value) {
        return make_uint4(__float_as_uint(x.x * s), __float_as_uint(x.y * s), __float_as_uint(y.x * s), __float_as_uint(y.y * s));
    } else {
        e4m3x4_to_f16x4(codes.y, a, b);
        const float2 z = f16x2_to_f32(a), w = f16x2_to_f32(b);
        return make_uint4(pack2<O>(x.x * s, x.y * s), pack2<O>(y.x * s, y.y * s), pack2<O>(z.x * s, z.y * s),
                          pack2<O>(w.x * s, w.y * s));
    }
}

// A CTA takes `per_cta` rows (16 or 64): their places in the cache first, found by
// one warp, then a thread takes 16 bytes of output in one column of several rows.
template <typename O, int D>
__global__ void __launch_bounds__(256) kv_gather_e4m3_kernel(const QuantGatherParams p) {
    pdl_wait_primary();
    pdl_launch_dependents();
    __shared__ int64_t place[64];   // block * 16 + offset; -1: zeros; -2: not written
    const int64_t row0 = (int64_t)blockIdx.x * p.per_cta;
    const int n = (int)min((int64_t)p.per_cta, p.total - row0);
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        // the last s with cu[s] <= row0, 32 candidates at a time
        int lo = 0, span = p.num_seqs;
        while (span > 1) {
            const int step = (span + 31) >> 5;
            const int s = lo + lane * step;
            const bool below = lane * step < span && __ldg(p.cu_seqlens + s) <= row0;
            const uint32_t m = __ballot_sync(0xffffffffu, below);
            const int k = m ? 31 - __clz(m) : 0;
            lo += k * step;
            span = min(step, span - k * step);
        }
        for (int r = lane; r < p.per_cta; r += 32) {
            // rows of a CTA are of one sequence or a few: on from there, up to 32 steps and then by halves
            const int64_t row = row0 + r;
            int s = lo, hi = p.num_seqs;
            for (int step = 0; step < 32 && s + 1 < hi && __ldg(p.cu_seqlens + s + 1) <= row; ++step) ++s;
            while (hi - s > 1 && __ldg(p.cu_seqlens + s + 1) <= row) {
                const int mid = (s + hi) >> 1;
                if (__ldg(p.cu_seqlens + mid) <= row) s = mid; else hi = mid;
            }
            int64_t to = -2;
            if (r < n && row < __ldg(p.cu_seqlens + p.num_seqs)) {
                const int64_t in = row - __ldg(p.cu_seqlens + s);
                const int64_t pos = in + (p.first ? __ldg(p.first + s) : 0);
                to = -1;
                if (in >= 0 && pos >= 0 && pos < (int64_t)p.max_blocks * 16) {
                    const int blk = __ldg(p.block_tables + (int64_t)s * p.max_blocks + pos / 16);
                    if (blk >= 0 && blk < p.num_blocks)
                        to = (int64_t)blk * 16 + (pos & 15);
                    else
                        set_status(p.dev_status, PKV_DEV_BAD_BLOCK_ID);
                } else {
                    set_status(p.dev_status, in < 0 ? PKV_DEV_BAD_CHUNK : PKV_DEV_BAD_CONTEXT);
                }
            }
            place[r] = to;
        }
    }
    __syncthreads();
    constexpr int CODES = 16 / (int)sizeof(O);
    constexpr int PIECES = D / CODES;
    const int columns = 2 * p.Hkv * PIECES;                  // of K, then of V
    // threads beyond the columns take other rows
    const int groups = max(1, 256 / columns);
    const int group = (int)threadIdx.x / columns;
    if (columns < 256 && group >= groups) return;
    constexpr int BATCH = 8;
    for (int c = columns < 256 ? (int)threadIdx.x - group * columns : (int)threadIdx.x; c < columns; c += 256) {
        const int kv = c >= p.Hkv * PIECES;
        const int hc = c - kv * p.Hkv * PIECES;
        const int h = hc / PIECES, piece = hc - h * PIECES;
        const uint8_t *cache = (kv ? p.v_cache : p.k_cache) + piece * CODES;
        O *to = static_cast<O *>(kv ? p.v : p.k) + (row0 * p.Hkv + h) * D + piece * CODES;
        for (int r0 = columns < 256 ? group : 0; r0 < n; r0 += BATCH * groups) {
            uint2 codes[BATCH];
            float s[BATCH];
#pragma unroll
            for (int e = 0; e < BATCH; ++e) {
                const int r = r0 + e * groups;
                const int64_t at = r < n ? place[r] : -2;
                codes[e] = make_uint2(0u, 0u);
                s[e] = 0.f;
                if (at >= 0) {
                    const int64_t tile = (at >> 4) * p.Hkv + h;
                    const uint8_t *from = cache + (tile * 16 + (at & 15)) * D;
                    if constexpr (CODES == 8)
                        codes[e] = __ldg(reinterpret_cast<const uint2 *>(from));
                    else
                        codes[e].x = __ldg(reinterpret_cast<const uint32_t *>(from));
                    s[e] = __ldg(p.scales + tile * 2 + kv);
                }
            }
#pragma unroll
            for (int e = 0; e < BATCH; ++e) {
                const int r = r0 + e * groups;
                if (r < n && place[r] != -2)
                    *reinterpret_cast<uint4 *>(to + (int64_t)r * p.Hkv * D) = values<O>(codes[e], s[e]);
            }
        }
    }
}

}  // namespace pkv

extern "C" int pkv_kv_append_e4m3(const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                                  const int64_t *slot_mapping, int num_tokens, void *k_cache, void *v_cache,
                                  float *kv_scales, int num_blocks, int block_size, int num_kv_heads, int head_dim,
                                  int dtype, int *dev_status, void *stream) {
    pkv::NvtxRange nvtx_range("pkv_kv_append_e4m3");
    using namespace pkv;
    if (num_tokens < 0 || num_blocks <= 0 || num_kv_heads <= 0) return PKV_ERR_INVALID_ARG;
    if (dtype != PKV_DTYPE_F16 && dtype != PKV_DTYPE_BF16) return PKV_ERR_UNSUPPORTED;
    if (block_size != 16 || (head_dim != 64 && head_dim != 128)) return PKV_ERR_UNSUPPORTED;
    if ((int64_t)num_tokens * num_kv_heads >= (int64_t)1 << 30) return PKV_ERR_UNSUPPORTED;
    if (num_kv_heads > 1 << 16) return PKV_ERR_UNSUPPORTED;   // (offsets in a token's row are 32-bit)
    if (num_tokens == 0) return PKV_OK;
    if (!k || !v || !slot_mapping || !k_cache || !v_cache || !kv_scales) return PKV_ERR_INVALID_ARG;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(slot_mapping, 8) ||
        !aligned(kv_scales, 8) || k_stride < 0 || v_stride < 0 || k_stride % 8 != 0 || v_stride % 8 != 0)
        return PKV_ERR_INVALID_ARG;
    // Tokens a CTA, and CTAs that share them.  16 tokens, by as many CTAs as leave a
    // warp 8 KB of a block's rows (a prompt of 16,383 rows, 16 heads of 64, 20 us in
    // spans of 16 by two, 27.5 in spans of 8 by four; 6,000 rows of 32 heads of 128 25.1
    // us by eight, 30.7 by two; 16,383 of one head 5.2 by one, 6.0 by two).  Where rows
    // are few, 8 by four (us, and in spans of 16; 8 heads of 128 and 16 of 64): 256
    // decodes 2.0 and 4.4, 2.2 and 5.0; 1,000 2.9 and 4.5, 3.0 and 5.1; 4 chunks of 250
    // 3.9 and 4.8, 3.4 and 5.3; 500 decodes and a chunk of 500 4.0 and 4.5, 3.2 and 5.1; but
    // a chunk of 512 alone 3.0 and 2.5, 2.5 and 2.7, one of 1,000 3.8 and 2.6, 3.1 and
    // 2.8.  Rows of 32 heads of 128 have eight CTAs a span of 16, and gain nothing from
    // spans of 8: 256 decodes 4.5 and 4.5, a chunk of 512 5.9 and 3.1.
    const bool few = num_tokens <= 1024 && num_kv_heads * head_dim < 4096;
    const int span = few ? 8 : 16;
    const int slices = few ? 4 : std::max(1, std::min(8, num_kv_heads * head_dim / 512));
    const QuantAppendParams prm = {k, v, k_stride, v_stride, slot_mapping, static_cast<uint8_t *>(k_cache),
                                   static_cast<uint8_t *>(v_cache), kv_scales, dev_status, num_tokens, num_blocks,
                                   num_kv_heads, span};
    const dim3 grid((unsigned)((num_tokens + span - 1) / span), (unsigned)slices);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    auto launch = [&](auto kernel) { return launch_pdl(kernel, grid, dim3(256), 0, st, prm); };
    cudaError_t e;
    if (dtype == PKV_DTYPE_BF16)
        e = head_dim == 128 ? launch(kv_append_e4m3_kernel<__nv_bfloat16, 128>) : launch(kv_append_e4m3_kernel<__nv_bfloat16, 64>);
    else
        e = head_dim == 128 ? launch(kv_append_e4m3_kernel<__half, 128>) : launch(kv_append_e4m3_kernel<__half, 64>);
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? PKV_OK : cuda_fail(e);
}

extern "C" int pkv_kv_gather_e4m3(void *k, void *v, const void *k_cache, const void *v_cache, const float *kv_scales,
                                  const int32_t *block_tables, int max_blocks_per_seq, const int32_t *cu_seqlens,
                                  const int32_t *first, int num_seqs, int total, int num_blocks, int block_size,
                                  int num_kv_heads, int head_dim, int out_dtype, int *dev_status, void *stream) {
    pkv::NvtxRange nvtx_range("pkv_kv_gather_e4m3");
    using namespace pkv;
    if (num_seqs < 0 || total < 0 || num_blocks <= 0 || num_kv_heads <= 0 || max_blocks_per_seq <= 0)
        return PKV_ERR_INVALID_ARG;
    if (block_size != 16 || (head_dim != 64 && head_dim != 128)) return PKV_ERR_UNSUPPORTED;
    if (out_dtype != PKV_DTYPE_F16 && out_dtype != PKV_DTYPE_BF16 && out_dtype != PKV_DTYPE_F32) return PKV_ERR_UNSUPPORTED;
    if (num_kv_heads > 1 << 16) return PKV_ERR_UNSUPPORTED;   // (a CTA's items are counted in 32 bits)
    if (num_seqs == 0 || total == 0) return PKV_OK;
    if (!k || !v || !k_cache || !v_cache || !kv_scales || !block_tables || !cu_seqlens) return PKV_ERR_INVALID_ARG;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(kv_scales, 8) ||
        !aligned(block_tables, 4) || !aligned(cu_seqlens, 4) || !aligned(first, 4))
        return PKV_ERR_INVALID_ARG;
    int sms = 0;
    const int rc = current_sm_count(&sms);
    if (rc != PKV_OK) return rc;
    // rows a CTA: 16, or as many as give each of its threads 16 columns, where the
    // GPU is full even so (64 sequences x 8,000, one head of 64: 15.6 us with 64
    // rows, 34 with 16; eight heads of 128: 114 with 16, 120 with 64)
    const int columns = 2 * num_kv_heads * head_dim / (out_dtype == PKV_DTYPE_F32 ? 4 : 8);
    int per_cta = std::min(64, std::max(16, 16 * (256 / columns)));
    if ((int64_t)total < (int64_t)per_cta * 8 * sms) per_cta = 16;
    const QuantGatherParams prm = {k, v, static_cast<const uint8_t *>(k_cache), static_cast<const uint8_t *>(v_cache),
                                   kv_scales, block_tables, cu_seqlens, first, dev_status, max_blocks_per_seq, num_blocks,
                                   num_seqs, total, num_kv_heads, per_cta};
    const dim3 grid((unsigned)((total + (int64_t)per_cta - 1) / per_cta));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    auto launch = [&](auto wide, auto narrow) {
        return head_dim == 128 ? launch_pdl(wide, grid, dim3(256), 0, st, prm) : launch_pdl(narrow, grid, dim3(256), 0, st, prm);
    };
    cudaError_t e;
    if (out_dtype == PKV_DTYPE_BF16)
        e = launch(kv_gather_e4m3_kernel<__nv_bfloat16, 128>, kv_gather_e4m3_kernel<__nv_bfloat16, 64>);
    else if (out_dtype == PKV_DTYPE_F16)
        e = launch(kv_gather_e4m3_kernel<__half, 128>, kv_gather_e4m3_kernel<__half, 64>);
    else
        e = launch(kv_gather_e4m3_kernel<float, 128>, kv_gather_e4m3_kernel<float, 64>);
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? PKV_OK : cuda_fail(e);
}
