// Attention over the cache held in 8 bits: decode (pkv_paged_decode_attention_e4m3)
// and chunked prefill (pkv_paged_prefill_attention_e4m3).
//
// Mathematics.  A row at position p sees position t iff t <= p and (t > p -
// window or t < sinks); its key is K_t = k_t a, its value V_t = v_t b, k and v
// codes, a and b the scales of t's block:
//     out = sum_t softmax_t(scale q . K_t) V_t.
//
// The plainest form: a warp per (row, query head), a lane per head_dim / 32
// dimensions, position by position with the running maximum and sum of the
// softmax in fp32.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "pkv.h"
#include "pkv_device.cuh"
#include "pkv_host.h"
#include "pkv_quant.cuh"

namespace pkv {

struct QuantAttentionParams {
    void *out;
    const void *q;
    const int32_t *cu_seqlens;     // NULL: a row a sequence (decode)
    const uint8_t *k_cache, *v_cache;
    const float *scales;
    const int32_t *block_tables, *context_lens;
    int *dev_status;
    int num_seqs, max_blocks, num_blocks, Hq, Hkv, G, window, sinks, total_q, max_q_len;
    float scale_log2;
    int out_dtype;
};

template <typename T, int D>
__global__ void __launch_bounds__(128) quant_attention_kernel(const QuantAttentionParams p) {
    pdl_wait_primary();
    pdl_launch_dependents();
    constexpr int N = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int hq = (int)(w % p.Hq);
    const int64_t rest = w / p.Hq;
    const int i = (int)(rest % p.max_q_len);
    const int c = (int)(rest / p.max_q_len);
    if (c >= p.num_seqs) return;
    const int q0 = p.cu_seqlens ? __ldg(p.cu_seqlens + c) : c;
    const int n = p.cu_seqlens ? __ldg(p.cu_seqlens + c + 1) - q0 : 1;
    int ctx = __ldg(p.context_lens + c);
    const int cap = p.max_blocks * 16;
    if (p.cu_seqlens) {
        const int bad = n < 0 || n > ctx || n > p.max_q_len || q0 < 0 || n > p.total_q - q0 ? PKV_DEV_BAD_CHUNK
                        : ctx > cap                                                        ? PKV_DEV_BAD_CONTEXT
                                                                                           : 0;
        if (bad && i == 0 && hq == 0 && lane == 0) set_status(p.dev_status, bad);
        if (bad || i >= n) return;
    } else if (ctx < 0 || ctx > cap) {
        if (hq == 0 && lane == 0) set_status(p.dev_status, PKV_DEV_BAD_CONTEXT);
        ctx = min(max(ctx, 0), cap);
    }
    const int64_t row = (int64_t)(q0 + i) * p.Hq + hq;
    const int h = hq / p.G;
    float q[N], o[N] = {};
    for (int e = 0; e < N; ++e) q[e] = (float)static_cast<const T *>(p.q)[row * D + lane * N + e];
    float m = -INFINITY, l = 0.f;
    const int pos = ctx - n + i, w0 = max(pos - p.window + 1, 0);
    auto step = [&](int t) {
        const int blk = __ldg(p.block_tables + (int64_t)c * p.max_blocks + t / 16);
        const bool ok = blk >= 0 && blk < p.num_blocks;
        if (!ok && lane == 0) set_status(p.dev_status, PKV_DEV_BAD_BLOCK_ID);
        const int64_t tile = (int64_t)(ok ? blk : 0) * p.Hkv + h;
        const int64_t at = (tile * 16 + t % 16) * D + lane * N;
        const float a = __ldg(p.scales + tile * 2), b = __ldg(p.scales + tile * 2 + 1);
        float x = 0.f, v[N];
        for (int e = 0; e < N; e += 2) {
            const float2 k2 = f16x2_to_f32(e4m3x2_to_f16x2(__ldg(reinterpret_cast<const uint16_t *>(p.k_cache + at + e))));
            const float2 v2 = f16x2_to_f32(e4m3x2_to_f16x2(__ldg(reinterpret_cast<const uint16_t *>(p.v_cache + at + e))));
            x += q[e] * k2.x + q[e + 1] * k2.y;
            v[e] = ok ? v2.x * b : 0.f;
            v[e + 1] = ok ? v2.y * b : 0.f;
        }
        for (int s = 16; s > 0; s >>= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
        x = ok ? x * a * p.scale_log2 : 0.f;
        const float mn = fmaxf(m, x);
        const float sub = mn == -INFINITY ? 0.f : mn;
        const float f = exp2f(m - sub), wt = exp2f(x - sub);
        l = l * f + wt;
        for (int e = 0; e < N; ++e) o[e] = o[e] * f + wt * v[e];
        m = mn;
    };
    for (int t = 0; t < min(p.sinks, w0); ++t) step(t);
    for (int t = w0; t <= pos; ++t) step(t);
    for (int e = 0; e < N; ++e) store_out<T>(p.out, p.out_dtype, row * D + lane * N + e, pos >= 0 ? o[e] / l : 0.f);
}

// What both calls refuse, and the launch.
static int quant_attention(QuantAttentionParams p, int num_seqs, int block_size, int head_dim, int window, int num_sinks,
                           float scale, int dtype, cudaStream_t stream) {
    const int64_t warps = (int64_t)num_seqs * p.max_q_len * p.Hq;
    if ((warps + 3) / 4 >= (int64_t)1 << 31) return PKV_ERR_UNSUPPORTED;
    p.num_seqs = num_seqs;
    const int64_t capacity = (int64_t)p.max_blocks * 16;
    p.window = window < capacity ? window : (int)capacity;   // no context is longer
    p.sinks = num_sinks < capacity ? num_sinks : (int)capacity;
    p.scale_log2 = scale * 1.4426950408889634f;
    const dim3 grid((unsigned)((warps + 3) / 4));
    auto launch = [&](auto kernel) { return launch_pdl(kernel, grid, dim3(128), 0, stream, p); };
    cudaError_t e;
    if (dtype == PKV_DTYPE_BF16)
        e = head_dim == 128 ? launch(quant_attention_kernel<__nv_bfloat16, 128>) : launch(quant_attention_kernel<__nv_bfloat16, 64>);
    else
        e = head_dim == 128 ? launch(quant_attention_kernel<__half, 128>) : launch(quant_attention_kernel<__half, 64>);
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
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(kv_scales, 8) ||
        !aligned(cu_seqlens, 4) || !aligned(block_tables, 4) || !aligned(context_lens, 4))
        return PKV_ERR_INVALID_ARG;
    QuantAttentionParams p = {};
    p.out = out, p.q = q, p.cu_seqlens = cu_seqlens, p.k_cache = static_cast<const uint8_t *>(k_cache);
    p.v_cache = static_cast<const uint8_t *>(v_cache), p.scales = kv_scales, p.block_tables = block_tables;
    p.context_lens = context_lens, p.dev_status = dev_status;
    p.max_blocks = max_blocks_per_seq, p.num_blocks = num_blocks, p.Hq = num_q_heads, p.Hkv = num_kv_heads;
    p.G = num_q_heads / num_kv_heads, p.total_q = total_q, p.max_q_len = max_q_len, p.out_dtype = out_dtype;
    return quant_attention(p, num_seqs, block_size, head_dim, window, num_sinks, scale, dtype, static_cast<cudaStream_t>(stream));
}
