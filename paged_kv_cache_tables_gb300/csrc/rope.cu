// Queries and keys made ready for the cache in one pass: an RMS norm of each
// head (optional), rotary positions, and on the append path the step's K and V
// rows stored in the paged cache by slot (pkv_qk_rope, pkv_qk_rope_append);
// and the rotation's frequencies (pkv_rope_frequencies, host).
//
// Mathematics.  For a head row x of head_dim d at position p:
//     y = x * rsqrt(mean(x^2) + eps) * w             (with a weight)
//     (y_i, y_j) -> m * (y_i cos a - y_j sin a, y_i sin a + y_j cos a),
//     a = p * f_k for the k-th pair of the first r dimensions,
// pairs (2k, 2k + 1) interleaved or (k, k + r/2) half.  Everything between the
// 16-bit loads and the one 16-bit store is fp32: norm, rotation and factor
// cost a single rounding.
//
// The angle.  p * f in fp32 loses whole radians at far positions, and fp64 is
// slow here.  A frequency is kept as a fraction of a turn in 64-bit fixed
// point, F = round(f / 2 pi * 2^64): p * F modulo 2^64 is p turns of it with
// the whole turns gone and an error of p * 2^-65 turns, from integer
// multiplies alone.  Its top 32 bits, as a signed number of half turns, go to
// sincospif, which needs no reduction.
//
// What bounds it: HBM, each row read and written once.  A CTA computes the
// (cos, sin) of its tokens' pairs once into shared memory for all heads (a
// thread for itself would spend more time in sincospif than its bytes take);
// a row is head_dim / 16 lanes of two 16-byte chunks each, chosen so that
// both ends of a pair are in one thread and no lane exchange is needed: lane
// l < r/16 holds pairs 8l .. 8l+7, a lane behind them 16 plain dimensions.
#include <cuda_runtime.h>

#include <cmath>

#include "pkv.h"
#include "pkv_device.cuh"
#include "pkv_host.h"

namespace pkv {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxTokens = 16;   // tokens a CTA takes at most

struct RopeParams {
    void *q_out, *k_out;
    const void *q, *k, *v;
    int64_t q_out_stride, k_out_stride, q_stride, k_stride, v_stride;   // elements between tokens
    const int32_t *positions;
    const int64_t *slot_mapping;
    const int64_t *freqs;
    const void *q_weight, *k_weight;
    void *k_cache, *v_cache;
    int *dev_status;
    int T, Hq, Hkv, rot, num_blocks, tokens_per_cta;
    int weight_f32;
    float mscale, eps;
};

template <typename T>
__device__ __forceinline__ void unpack8(const uint4 &u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (std::is_same<T, __nv_bfloat16>::value) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        } else {
            const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            f[2 * i] = v.x;
            f[2 * i + 1] = v.y;
        }
    }
}

template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]), pack2<T>(f[6], f[7]));
}

template <typename T>
__device__ __forceinline__ void load_weight8(const void *w, int f32, int at, float (&f)[8]) {
    if (f32) {
        const float4 a = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(w) + at));
        const float4 b = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(w) + at) + 1);
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    } else {
        unpack8<T>(__ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(w) + at)), f);
    }
}

// LANES = head_dim / 16 lanes hold a row; rows of a token: its query heads,
// its key heads and (APPEND) its value heads.
template <typename T, int LANES, bool INTERLEAVED, bool APPEND>
__global__ void __launch_bounds__(kRopeThreads) qk_rope_kernel(const RopeParams p) {
    extern __shared__ float4 rope_smem[];   // (cos, sin) pairs, see below
    constexpr int kRows = kRopeThreads / LANES;
    constexpr int D = LANES * 16;
    const int tid = threadIdx.x, l = tid % LANES;
    const int t0 = blockIdx.x * p.tokens_per_cta, nt = min(p.tokens_per_cta, p.T - t0);
    const int per_token = p.Hq + (APPEND ? 2 : 1) * p.Hkv;
    const int rlanes = p.rot / 16;          // lanes of a row that rotate
    const int items = nt * per_token;
    // element offsets of this lane's two chunks within a row
    const bool turns = l < rlanes;
    const int c0 = turns && !INTERLEAVED ? 8 * l : 16 * l;
    const int c1 = turns && !INTERLEAVED ? p.rot / 2 + 8 * l : 16 * l + 8;
    pdl_wait_primary();
    pdl_launch_dependents();

    auto source = [&](int t, int row) -> const T * {
        const int64_t tok = t0 + t;
        if (row < p.Hq) return static_cast<const T *>(p.q) + tok * p.q_stride + (int64_t)row * D;
        row -= p.Hq;
        if (!APPEND || row < p.Hkv) return static_cast<const T *>(p.k) + tok * p.k_stride + (int64_t)row * D;
        return static_cast<const T *>(p.v) + tok * p.v_stride + (int64_t)(row - p.Hkv) * D;
    };

    // the first row's loads are in flight while the angles are computed
    int item = tid / LANES;
    uint4 a = make_uint4(0, 0, 0, 0), b = a;
    if (item < items) {
        const T *x = source(item / per_token, item % per_token);
        a = *reinterpret_cast<const uint4 *>(x + c0);
        b = *reinterpret_cast<const uint4 *>(x + c1);
    }
    // pair 8 l + e of token t is half (e & 1) of the float4 at
    // t * rot/4 + (e / 2) * rlanes + l: a row's lanes read neighbours
    const int pairs = p.rot / 2;
    for (int i = tid; i < nt * pairs; i += kRopeThreads) {
        const int t = i / pairs, k = i % pairs;
        const uint64_t turn = (uint64_t)(int64_t)__ldg(p.positions + t0 + t) * (uint64_t)__ldg(p.freqs + k);
        float s, c;
        sincospif((float)(int32_t)(turn >> 32) * 4.656612873077393e-10f, &s, &c);   // 2^-31: half turns
        reinterpret_cast<float2 *>(rope_smem)[2 * (t * (pairs / 2) + ((k & 7) >> 1) * rlanes + (k >> 3)) + (k & 1)] =
            make_float2(p.mscale * c, p.mscale * s);
    }
    __syncthreads();

    for (; item < items; item += kRows) {
        const int t = item / per_token, row = item % per_token;
        const int64_t tok = t0 + t;
        uint4 na = make_uint4(0, 0, 0, 0), nb = na;
        if (item + kRows < items) {
            const T *x = source((item + kRows) / per_token, (item + kRows) % per_token);
            na = *reinterpret_cast<const uint4 *>(x + c0);
            nb = *reinterpret_cast<const uint4 *>(x + c1);
        }
        const bool is_q = row < p.Hq, is_v = APPEND && row >= p.Hq + p.Hkv;
        if (!is_v) {
            float x0[8], x1[8];
            unpack8<T>(a, x0);
            unpack8<T>(b, x1);
            const void *w = is_q ? p.q_weight : p.k_weight;
            if (w != nullptr) {   // the same for all lanes of a row
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) ss += x0[e] * x0[e] + x1[e] * x1[e];
                const unsigned m = LANES == 8 ? 0xffu << (tid & 24) : 0xfu << (tid & 28);
#pragma unroll
                for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(m, ss, o);
                const float inv = 1.f / sqrtf(ss * (1.f / D) + p.eps);
                float w0[8], w1[8];
                load_weight8<T>(w, p.weight_f32, c0, w0);
                load_weight8<T>(w, p.weight_f32, c1, w1);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x0[e] = x0[e] * inv * w0[e];
                    x1[e] = x1[e] * inv * w1[e];
                }
            }
            if (turns) {
                const float4 *cs = rope_smem + t * (pairs / 2) + l;
#pragma unroll
                for (int e2 = 0; e2 < 4; ++e2) {
                    const float4 f = cs[e2 * rlanes];   // cos, sin of pair 2 e2, then of pair 2 e2 + 1
                    if constexpr (INTERLEAVED) {
                        float(&x)[8] = e2 < 2 ? x0 : x1;
                        const int i = (e2 & 1) * 4;
                        const float u0 = x[i], u1 = x[i + 1], u2 = x[i + 2], u3 = x[i + 3];
                        x[i] = u0 * f.x - u1 * f.y;
                        x[i + 1] = u0 * f.y + u1 * f.x;
                        x[i + 2] = u2 * f.z - u3 * f.w;
                        x[i + 3] = u2 * f.w + u3 * f.z;
                    } else {
                        const float u0 = x0[2 * e2], u1 = x1[2 * e2], u2 = x0[2 * e2 + 1], u3 = x1[2 * e2 + 1];
                        x0[2 * e2] = u0 * f.x - u1 * f.y;
                        x1[2 * e2] = u0 * f.y + u1 * f.x;
                        x0[2 * e2 + 1] = u2 * f.z - u3 * f.w;
                        x1[2 * e2 + 1] = u2 * f.w + u3 * f.z;
                    }
                }
            }
            a = pack8<T>(x0);
            b = pack8<T>(x1);
        }
        T *dst = nullptr;
        if (is_q) {
            dst = static_cast<T *>(p.q_out) + tok * p.q_out_stride + (int64_t)row * D;
        } else if constexpr (!APPEND) {
            dst = static_cast<T *>(p.k_out) + tok * p.k_out_stride + (int64_t)(row - p.Hq) * D;
        } else {
            const int h = is_v ? row - p.Hq - p.Hkv : row - p.Hq;
            const int64_t slot = __ldg(p.slot_mapping + tok);
            const int64_t block = slot >> 4;
            if (slot >= 0 && block < p.num_blocks)
                dst = static_cast<T *>(is_v ? p.v_cache : p.k_cache) +
                      ((block * p.Hkv + h) * 16 + (slot & 15)) * (int64_t)D;
            else if (slot >= 0 && l == 0 && h == 0)
                set_status(p.dev_status, PKV_DEV_BAD_SLOT);
        }
        if (dst != nullptr) {
            *reinterpret_cast<uint4 *>(dst + c0) = a;
            *reinterpret_cast<uint4 *>(dst + c1) = b;
        }
        a = na;
        b = nb;
    }
}

// Rows of `a` and `b` (n tokens, la / lb elements each, strides sa / sb,
// addresses in bytes of 2-byte elements): whether a row of one may share
// memory with a row of the other.  Rows of one fused buffer (equal strides)
// are told apart by their place in it; other overlaps of the address ranges
// count as shared.
static bool rows_meet(const void *a, int64_t sa, int64_t la, const void *b, int64_t sb, int64_t lb, int64_t n) {
    const int64_t x = (int64_t)reinterpret_cast<uintptr_t>(a) / 2, y = (int64_t)reinterpret_cast<uintptr_t>(b) / 2;
    const int64_t xe = x + (n - 1) * sa + la, ye = y + (n - 1) * sb + lb;
    if (xe <= y || ye <= x) return false;
    if (n == 1 || sa != sb || sa <= 0) return true;
    const int64_t off = ((y - x) % sa + sa) % sa;   // b's rows start `off` elements behind a's, modulo the stride
    return !(off >= la && off + lb <= sa);
}

template <typename T, int LANES>
static cudaError_t launch_rope_t(const RopeParams &prm, bool interleaved, bool append, int grid, size_t smem,
                                 cudaStream_t stream) {
    auto go = [&](auto kernel) { return launch_pdl(kernel, dim3(grid), dim3(kRopeThreads), smem, stream, prm); };
    if (interleaved)
        return append ? go(qk_rope_kernel<T, LANES, true, true>) : go(qk_rope_kernel<T, LANES, true, false>);
    return append ? go(qk_rope_kernel<T, LANES, false, true>) : go(qk_rope_kernel<T, LANES, false, false>);
}

static int rope_checks(const RopeParams &p, int head_dim, int dtype, int weight_dtype, bool append) {
    if (p.T < 0 || p.Hq <= 0 || p.Hkv <= 0) return PKV_ERR_INVALID_ARG;
    if (dtype != PKV_DTYPE_F16 && dtype != PKV_DTYPE_BF16) return PKV_ERR_UNSUPPORTED;
    if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
    if (p.rot < 16 || p.rot > head_dim || p.rot % 16 != 0) return PKV_ERR_UNSUPPORTED;
    if ((p.q_weight || p.k_weight) && weight_dtype != dtype && weight_dtype != PKV_DTYPE_F32) return PKV_ERR_UNSUPPORTED;
    if ((int64_t)p.Hq + 2 * (int64_t)p.Hkv > (1 << 20)) return PKV_ERR_UNSUPPORTED;
    if (!std::isfinite(p.mscale)) return PKV_ERR_INVALID_ARG;
    if ((p.q_weight || p.k_weight) && !(std::isfinite(p.eps) && p.eps >= 0.f)) return PKV_ERR_INVALID_ARG;
    if (p.T == 0) return PKV_OK;
    const int64_t lq = (int64_t)p.Hq * head_dim, lk = (int64_t)p.Hkv * head_dim, T = p.T;
    if (!p.q_out || !p.q || !p.k || !p.positions || !p.freqs) return PKV_ERR_INVALID_ARG;
    if (!aligned(p.q_out, 16) || !aligned(p.q, 16) || !aligned(p.k, 16) || !aligned(p.positions, 4) ||
        !aligned(p.freqs, 8) || !aligned(p.q_weight, 16) || !aligned(p.k_weight, 16))
        return PKV_ERR_INVALID_ARG;
    if (p.q_stride % 8 || p.k_stride % 8 || p.q_out_stride % 8 || p.q_stride < 0 || p.k_stride < 0)
        return PKV_ERR_INVALID_ARG;
    if (T > 1 && p.q_out_stride < lq) return PKV_ERR_INVALID_ARG;
    auto same = [&](const void *a, int64_t sa, const void *b, int64_t sb) { return a == b && (sa == sb || T == 1); };
    // an output may replace its own input row by row; anything else it touches
    // must be apart from the rows still to be read
    if (!same(p.q_out, p.q_out_stride, p.q, p.q_stride) &&
        rows_meet(p.q_out, p.q_out_stride, lq, p.q, p.q_stride, lq, T))
        return PKV_ERR_INVALID_ARG;
    if (rows_meet(p.q_out, p.q_out_stride, lq, p.k, p.k_stride, lk, T)) return PKV_ERR_INVALID_ARG;
    if (append) {
        if (!p.v || !p.slot_mapping || !p.k_cache || !p.v_cache) return PKV_ERR_INVALID_ARG;
        if (!aligned(p.v, 16) || !aligned(p.slot_mapping, 8) || !aligned(p.k_cache, 16) || !aligned(p.v_cache, 16))
            return PKV_ERR_INVALID_ARG;
        if (p.v_stride % 8 || p.v_stride < 0) return PKV_ERR_INVALID_ARG;
        if (rows_meet(p.q_out, p.q_out_stride, lq, p.v, p.v_stride, lk, T)) return PKV_ERR_INVALID_ARG;
    } else {
        if (!p.k_out || !aligned(p.k_out, 16) || p.k_out_stride % 8) return PKV_ERR_INVALID_ARG;
        if (T > 1 && p.k_out_stride < lk) return PKV_ERR_INVALID_ARG;
        if (!same(p.k_out, p.k_out_stride, p.k, p.k_stride) &&
            rows_meet(p.k_out, p.k_out_stride, lk, p.k, p.k_stride, lk, T))
            return PKV_ERR_INVALID_ARG;
        if (rows_meet(p.k_out, p.k_out_stride, lk, p.q, p.q_stride, lq, T) ||
            rows_meet(p.k_out, p.k_out_stride, lk, p.q_out, p.q_out_stride, lq, T))
            return PKV_ERR_INVALID_ARG;
    }
    return PKV_OK;
}

static int rope_launch(RopeParams &prm, int head_dim, int interleaved, int dtype, bool append, cudaStream_t stream) {
    int sms = 0;
    int rc = current_sm_count(&sms);
    if (rc != PKV_OK) return rc;
    // tokens a CTA takes: about three rows per row of threads, but no fewer
    // than two CTAs per SM while there are tokens for them
    const int per_token = prm.Hq + (append ? 2 : 1) * prm.Hkv;
    const int rows = kRopeThreads / (head_dim / 16);
    int64_t tokens = ((int64_t)3 * rows + per_token - 1) / per_token;
    tokens = tokens < 1 ? 1 : (tokens > kRopeMaxTokens ? kRopeMaxTokens : tokens);
    while (tokens > 1 && (prm.T + tokens - 1) / tokens < 2 * sms) --tokens;
    prm.tokens_per_cta = (int)tokens;
    const int grid = (int)((prm.T + tokens - 1) / tokens);
    const size_t smem = (size_t)tokens * prm.rot / 2 * sizeof(float2);
    cudaError_t e;
    if (dtype == PKV_DTYPE_BF16)
        e = head_dim == 128 ? launch_rope_t<__nv_bfloat16, 8>(prm, interleaved, append, grid, smem, stream)
                            : launch_rope_t<__nv_bfloat16, 4>(prm, interleaved, append, grid, smem, stream);
    else
        e = head_dim == 128 ? launch_rope_t<__half, 8>(prm, interleaved, append, grid, smem, stream)
                            : launch_rope_t<__half, 4>(prm, interleaved, append, grid, smem, stream);
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? PKV_OK : cuda_fail(e);
}

}  // namespace pkv

extern "C" int pkv_qk_rope(void *q_out, int64_t q_out_stride, void *k_out, int64_t k_out_stride, const void *q,
                           int64_t q_stride, const void *k, int64_t k_stride, const int32_t *positions,
                           const int64_t *freqs, int rotary_dim, int interleaved, float mscale, const void *q_weight,
                           const void *k_weight, int weight_dtype, float eps, int num_tokens, int num_q_heads,
                           int num_kv_heads, int head_dim, int dtype, void *stream) {
    pkv::NvtxRange nvtx_range("pkv_qk_rope");
    using namespace pkv;
    RopeParams prm = {};
    prm.q_out = q_out;
    prm.k_out = k_out;
    prm.q = q;
    prm.k = k;
    prm.q_out_stride = q_out_stride;
    prm.k_out_stride = k_out_stride;
    prm.q_stride = q_stride;
    prm.k_stride = k_stride;
    prm.positions = positions;
    prm.freqs = freqs;
    prm.q_weight = q_weight;
    prm.k_weight = k_weight;
    prm.T = num_tokens;
    prm.Hq = num_q_heads;
    prm.Hkv = num_kv_heads;
    prm.rot = rotary_dim;
    prm.weight_f32 = weight_dtype == PKV_DTYPE_F32;
    prm.mscale = mscale;
    prm.eps = eps;
    int rc = rope_checks(prm, head_dim, dtype, weight_dtype, false);
    if (rc != PKV_OK || num_tokens == 0) return rc;
    return rope_launch(prm, head_dim, interleaved, dtype, false, static_cast<cudaStream_t>(stream));
}

extern "C" int pkv_qk_rope_append(void *q_out, int64_t q_out_stride, const void *q, int64_t q_stride, const void *k,
                                  int64_t k_stride, const void *v, int64_t v_stride, const int32_t *positions,
                                  const int64_t *slot_mapping, const int64_t *freqs, int rotary_dim, int interleaved,
                                  float mscale, const void *q_weight, const void *k_weight, int weight_dtype, float eps,
                                  int num_tokens, void *k_cache, void *v_cache, int num_blocks, int block_size,
                                  int num_q_heads, int num_kv_heads, int head_dim, int dtype, int *dev_status,
                                  void *stream) {
    pkv::NvtxRange nvtx_range("pkv_qk_rope_append");
    using namespace pkv;
    RopeParams prm = {};
    prm.q_out = q_out;
    prm.q = q;
    prm.k = k;
    prm.v = v;
    prm.q_out_stride = q_out_stride;
    prm.q_stride = q_stride;
    prm.k_stride = k_stride;
    prm.v_stride = v_stride;
    prm.positions = positions;
    prm.slot_mapping = slot_mapping;
    prm.freqs = freqs;
    prm.q_weight = q_weight;
    prm.k_weight = k_weight;
    prm.k_cache = k_cache;
    prm.v_cache = v_cache;
    prm.dev_status = dev_status;
    prm.T = num_tokens;
    prm.Hq = num_q_heads;
    prm.Hkv = num_kv_heads;
    prm.rot = rotary_dim;
    prm.num_blocks = num_blocks;
    prm.weight_f32 = weight_dtype == PKV_DTYPE_F32;
    prm.mscale = mscale;
    prm.eps = eps;
    if (num_blocks <= 0) return PKV_ERR_INVALID_ARG;
    if (block_size != 16) return PKV_ERR_UNSUPPORTED;
    int rc = rope_checks(prm, head_dim, dtype, weight_dtype, true);
    if (rc != PKV_OK || num_tokens == 0) return rc;
    return rope_launch(prm, head_dim, interleaved, dtype, true, static_cast<cudaStream_t>(stream));
}

// ---------------------------------------------------------------- frequencies

extern "C" int pkv_rope_frequencies(int64_t *freqs, float *mscale, int rotary_dim, double base, int scaling,
                                    double factor, double original_context, double low, double high) {
    if (!freqs || !mscale) return PKV_ERR_INVALID_ARG;
    if (rotary_dim < 16 || rotary_dim > 128 || rotary_dim % 16 != 0) return PKV_ERR_UNSUPPORTED;
    if (!(std::isfinite(base) && base > 1.0)) return PKV_ERR_INVALID_ARG;
    if (scaling < PKV_ROPE_PLAIN || scaling > PKV_ROPE_YARN) return PKV_ERR_UNSUPPORTED;
    if (scaling != PKV_ROPE_PLAIN && !(std::isfinite(factor) && factor >= 1.0)) return PKV_ERR_INVALID_ARG;
    if (scaling == PKV_ROPE_BANDS || scaling == PKV_ROPE_YARN) {
        if (!(std::isfinite(original_context) && original_context > 0.0)) return PKV_ERR_INVALID_ARG;
        if (!(std::isfinite(low) && std::isfinite(high) && low > 0.0 && high > low)) return PKV_ERR_INVALID_ARG;
    }
    constexpr double kTwoPi = 6.283185307179586476925286766559;
    const double r = rotary_dim;
    if (scaling == PKV_ROPE_NTK) base *= std::pow(factor, r / (r - 2.0));
    // the pair index at which a frequency makes `turns` turns over the original context
    auto pair_at = [&](double turns) { return r * std::log(original_context / (turns * kTwoPi)) / (2.0 * std::log(base)); };
    double first = 0.0, last = 0.0;
    if (scaling == PKV_ROPE_YARN) {
        first = std::fmax(std::floor(pair_at(high)), 0.0);
        last = std::fmin(std::ceil(pair_at(low)), r - 1.0);
    }
    *mscale = scaling == PKV_ROPE_YARN ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
    for (int i = 0; i < rotary_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / r);
        if (scaling == PKV_ROPE_LINEAR) {
            f /= factor;
        } else if (scaling == PKV_ROPE_BANDS) {
            double s = (original_context * f / kTwoPi - low) / (high - low);
            s = s < 0.0 ? 0.0 : (s > 1.0 ? 1.0 : s);
            f = s * f + (1.0 - s) * f / factor;
        } else if (scaling == PKV_ROPE_YARN) {
            double ramp = (i - first) / std::fmax(last - first, 1e-3);
            ramp = ramp < 0.0 ? 0.0 : (ramp > 1.0 ? 1.0 : ramp);
            f = f / factor * ramp + f * (1.0 - ramp);
        }
        // 0 < f <= 1: less than a sixth of a turn, so the fixed-point value
        // is below 2^62 and exact to the double's own 53 bits
        freqs[i] = (int64_t)std::llround(f / kTwoPi * 18446744073709551616.0);
    }
    return PKV_OK;
}
