// The cache held in 8 bits: this step's rows quantised into it
// (pkv_kv_append_e4m3), and rows of sequences read back (pkv_kv_gather_e4m3).
//
// Mathematics.  A (block, KV head)'s K tile and V tile each have one scale s; a
// stored code c stands for c s.  Of the rows that a call writes to a tile, a is
// the largest finite |x|, and
//     s' = scale(a) where the call writes offset 0, else max(s, scale(a)),
//     row x -> e4m3(x / s'),   where s' > s the tile's other rows c -> e4m3(c s / s'),
// scale(a) the least power of two with a <= 448 scale(a).
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
    int T, num_blocks, Hkv;
};

// Largest of the finite magnitudes among eight 16-bit values, as bits.
template <typename T>
__device__ __forceinline__ uint32_t finite_max8(uint4 x) {
    constexpr uint32_t inf = std::is_same<T, __nv_bfloat16>::value ? 0x7f80u : 0x7c00u;
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = w[i] & 0x7fffu, hi = (w[i] >> 16) & 0x7fffu;
        m = max(m, max(lo < inf ? lo : 0u, hi < inf ? hi : 0u));
    }
    return m;
}

// Four codes times r, as codes.
__device__ __forceinline__ uint32_t rescale4(uint32_t codes, float r) {
    uint32_t a, b;
    e4m3x4_to_f16x4(codes, a, b);
    const float2 x = f16x2_to_f32(a), y = f16x2_to_f32(b);
    return to_e4m3x4(x.x * r, x.y * r, y.x * r, y.y * r);
}

// A warp per (token, head, K or V): that of a block's first token in the call
// takes all of its tokens, which stand behind one another; the others leave.
template <typename T, int D>
__global__ void __launch_bounds__(256) kv_append_e4m3_kernel(const QuantAppendParams p) {
    pdl_wait_primary();
    pdl_launch_dependents();
    constexpr int LANES = D / 8;          // lanes of a row, 8 values each
    constexpr int ROWS = 32 / LANES;      // rows a warp takes at a time
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (w >= (int64_t)p.T * p.Hkv * 2) return;
    const int kv = (int)(w & 1);
    const int h = (int)((w >> 1) % p.Hkv);
    const int t = (int)((w >> 1) / p.Hkv);
    // lane i: the slot of token t + i - 1
    const int64_t at = (int64_t)t + lane - 1;
    const int64_t slot = at >= 0 && at < p.T && lane < 17 ? __ldg(p.slots + at) : -1;
    const int64_t block = slot < 0 ? -1 : slot / 16;
    const int64_t mine = __shfl_sync(0xffffffffu, block, 1);
    if (mine < 0) return;
    if (mine >= p.num_blocks) {
        if (kv == 0 && h == 0 && lane == 0) set_status(p.dev_status, PKV_DEV_BAD_SLOT);
        return;
    }
    const uint32_t same = __ballot_sync(0xffffffffu, block == mine);
    if (same & 1u) return;                                   // not the first
    const int n = __ffs(~(same >> 1)) - 1;                   // tokens of the block, up to 16
    const int my_off = (int)(slot & 15);
    const uint32_t written = __reduce_or_sync(0xffffffffu, lane >= 1 && lane <= n ? 1u << my_off : 0u);

    const int64_t tile = mine * p.Hkv + h;
    float *scale = p.scales + tile * 2 + kv;
    const float was = written & 1u ? 0.f : *scale;
    const T *rows = static_cast<const T *>(kv ? p.v : p.k) + (int64_t)t * (kv ? p.v_stride : p.k_stride) + h * D;
    const int64_t stride = kv ? p.v_stride : p.k_stride;
    const int sub = lane / LANES, col = lane % LANES;
    uint4 x[16 / ROWS];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 16 / ROWS; ++i) {
        const int r = i * ROWS + sub;
        x[i] = r < n ? __ldg(reinterpret_cast<const uint4 *>(rows + r * stride) + col) : make_uint4(0u, 0u, 0u, 0u);
        top = max(top, finite_max8<T>(x[i]));
    }
    top = __reduce_max_sync(0xffffffffu, top);
    const float old = was > 0.f ? was : 0.f;                 // (a scale that is none counts as 0)
    const float now = fmaxf(old, block_scale(pair_to_f32<T>(top).x));
    const float inv = 1.f / now;
    uint8_t *out = (kv ? p.v_cache : p.k_cache) + tile * 16 * D;
#pragma unroll
    for (int i = 0; i < 16 / ROWS; ++i) {
        const int r = i * ROWS + sub;
        const int off = __shfl_sync(0xffffffffu, my_off, (r & 15) + 1);
        if (r < n) {
            const float2 a = pair_to_f32<T>(x[i].x), b = pair_to_f32<T>(x[i].y), c = pair_to_f32<T>(x[i].z),
                         d = pair_to_f32<T>(x[i].w);
            const uint2 codes = make_uint2(to_e4m3x4(a.x * inv, a.y * inv, b.x * inv, b.y * inv),
                                           to_e4m3x4(c.x * inv, c.y * inv, d.x * inv, d.y * inv));
            *reinterpret_cast<uint2 *>(out + off * D + col * 8) = codes;
        }
    }
    if (now == was) return;
    if (!(written & 1u)) {
        const float ratio = old * inv;
        for (int i = lane; i < D; i += 32) {                 // 16-byte pieces of the tile
            const int r = i / (D / 16);
            if (written >> r & 1u) continue;
            uint4 *at4 = reinterpret_cast<uint4 *>(out) + i;
            const uint4 c = *at4;
            *at4 = make_uint4(rescale4(c.x, ratio), rescale4(c.y, ratio), rescale4(c.z, ratio), rescale4(c.w, ratio));
        }
    }
    if (lane == 0) *scale = now;
}

struct QuantGatherParams {
    void *k, *v;
    const uint8_t *k_cache, *v_cache;
    const float *scales;
    const int32_t *block_tables, *cu_seqlens, *first;
    int *dev_status;
    int max_blocks, num_blocks, num_seqs, total, Hkv;
};

// Four codes times s, rounded once to the output's type.
template <typename O>
__device__ __forceinline__ void put4(O *to, uint32_t codes, float s) {
    uint32_t a, b;
    e4m3x4_to_f16x4(codes, a, b);
    const float2 x = f16x2_to_f32(a), y = f16x2_to_f32(b);
    if constexpr (std::is_same<O, float>::value)
        *reinterpret_cast<float4 *>(to) = make_float4(x.x * s, x.y * s, y.x * s, y.y * s);
    else
        *reinterpret_cast<uint2 *>(to) = make_uint2(pack2<O>(x.x * s, x.y * s), pack2<O>(y.x * s, y.y * s));
}

// A CTA takes 16 rows: their places in the cache first, then 16 codes a thread
// at a time.
template <typename O, int D>
__global__ void __launch_bounds__(256) kv_gather_e4m3_kernel(const QuantGatherParams p) {
    pdl_wait_primary();
    pdl_launch_dependents();
    __shared__ int64_t place[16];   // block * 16 + offset; -1: zeros; -2: not written
    const int64_t row0 = (int64_t)blockIdx.x * 16;
    const int n = (int)min((int64_t)16, p.total - row0);
    if (threadIdx.x < 16) {
        int64_t to = -2;
        const int64_t r = row0 + threadIdx.x;
        if (threadIdx.x < n && r < __ldg(p.cu_seqlens + p.num_seqs)) {
            int lo = 0, hi = p.num_seqs;   // the last s with cu[s] <= r
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (__ldg(p.cu_seqlens + mid) <= r) lo = mid; else hi = mid;
            }
            const int64_t in = r - __ldg(p.cu_seqlens + lo);
            const int64_t pos = in + (p.first ? __ldg(p.first + lo) : 0);
            if (in >= 0 && pos >= 0 && pos < (int64_t)p.max_blocks * 16) {
                const int blk = __ldg(p.block_tables + (int64_t)lo * p.max_blocks + pos / 16);
                const bool ok = blk >= 0 && blk < p.num_blocks;
                to = ok ? (int64_t)blk * 16 + (pos & 15) : -1;
                if (!ok) set_status(p.dev_status, PKV_DEV_BAD_BLOCK_ID);
            } else {
                to = -1;
                set_status(p.dev_status, in < 0 ? PKV_DEV_BAD_CHUNK : PKV_DEV_BAD_CONTEXT);
            }
        }
        place[threadIdx.x] = to;
    }
    __syncthreads();
    constexpr int PIECES = D / 16;
    const int per_row = p.Hkv * PIECES;
    for (int i = threadIdx.x; i < 2 * n * per_row; i += 256) {
        const int kv = i >= n * per_row;
        const int j = i - kv * n * per_row;
        const int r = j / per_row, rest = j - r * per_row;
        const int h = rest / PIECES, c = rest - h * PIECES;
        const int64_t at = place[r];
        if (at == -2) continue;
        uint4 codes = make_uint4(0u, 0u, 0u, 0u);
        float s = 0.f;
        if (at >= 0) {
            const int64_t tile = (at >> 4) * p.Hkv + h;
            codes = __ldg(reinterpret_cast<const uint4 *>((kv ? p.v_cache : p.k_cache) + (tile * 16 + (at & 15)) * D) + c);
            s = __ldg(p.scales + tile * 2 + kv);
        }
        O *to = static_cast<O *>(kv ? p.v : p.k) + ((row0 + r) * p.Hkv + h) * D + c * 16;
        put4(to, codes.x, s);
        put4(to + 4, codes.y, s);
        put4(to + 8, codes.z, s);
        put4(to + 12, codes.w, s);
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
    const int64_t warps = (int64_t)num_tokens * num_kv_heads * 2;
    if (warps >= (int64_t)1 << 31) return PKV_ERR_UNSUPPORTED;
    if (num_tokens == 0) return PKV_OK;
    if (!k || !v || !slot_mapping || !k_cache || !v_cache || !kv_scales) return PKV_ERR_INVALID_ARG;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(slot_mapping, 8) ||
        !aligned(kv_scales, 8) || k_stride < 0 || v_stride < 0 || k_stride % 8 != 0 || v_stride % 8 != 0)
        return PKV_ERR_INVALID_ARG;
    const QuantAppendParams prm = {k, v, k_stride, v_stride, slot_mapping, static_cast<uint8_t *>(k_cache),
                                   static_cast<uint8_t *>(v_cache), kv_scales, dev_status, num_tokens, num_blocks,
                                   num_kv_heads};
    const dim3 grid((unsigned)((warps + 7) / 8));
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
    const QuantGatherParams prm = {k, v, static_cast<const uint8_t *>(k_cache), static_cast<const uint8_t *>(v_cache),
                                   kv_scales, block_tables, cu_seqlens, first, dev_status, max_blocks_per_seq, num_blocks,
                                   num_seqs, total, num_kv_heads};
    const dim3 grid((unsigned)((total + (int64_t)15) / 16));
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
