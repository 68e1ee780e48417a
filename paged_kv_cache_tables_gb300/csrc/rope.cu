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
// the whole turns gone, exactly, from integer multiplies alone; what is left is p
// times F's own error, that of f in double (below 2^-52 turns, 2^-55 measured).
// The product's top 32 bits, as a signed number of half turns, go to sincospif,
// which needs no reduction.
//
// What bounds it: HBM, each row read and written once, if the instructions per
// byte stay few and enough bytes are on their way.  A row is head_dim / 16
// lanes of two 16-byte chunks each, chosen so that both ends of a pair are in
// one thread: lane l < r/16 holds pairs 8l .. 8l+7, a lane behind them 16
// plain dimensions.  A warp takes up to four groups of rows of one token and one
// kind (query, key or value heads): it issues all their loads at once, and
// while they are under way works out what the rows share, the (cos, sin) of a
// lane's eight pairs (the groups of lanes share the sincospi among them), the
// weight, the slot and the addresses.  The arithmetic is on packed pairs of
// floats.  16,383 tokens x 32 heads of 128 (268 MB in and out): 40.0 us, 99 % of
// the measured copy rate; 4,344 tokens normed, rotated and appended (107 MB): 20.5
// us, 77 %; 64 tokens: 1.6 us.  Before the loads were issued together: 50.2, 24.8
// and 1.9 us.  Measured and left: CTAs of one warp (20.0 us, but calls of many
// small rows are then bound by the launch of CTAs, about 3 a ns), key and value
// heads in one warp (21.1 us), the norms of all groups worked out first (21.2 us),
// the weights folded into cos and sin besides (23.4 us).
#include <cuda_runtime.h>

#include <cmath>

#include "pkv.h"
#include "pkv_device.cuh"
#include "pkv_host.h"

namespace pkv {

constexpr int kRopeThreads = 64;
constexpr int kRopeSteps = 4;   // groups of rows a warp takes at most

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
    int T, Hq, Hkv, rot, num_blocks;
    int q_units, k_units, units;   // warps that take a token's query heads, its key heads, and in all
    int rows_per_unit;
    int weight_f32;
    float mscale, eps;
};

// Eight 16-bit values as four packed pairs of floats, and back.
template <typename T>
__device__ __forceinline__ void unpack8(const uint4 &u, uint64_t (&f)[4]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (std::is_same<T, __nv_bfloat16>::value) {
            f[i] = f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
        } else {
            const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            f[i] = f2_pack(v.x, v.y);
        }
    }
}

template <typename T>
__device__ __forceinline__ uint4 pack8(const uint64_t (&f)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a, b;
        f2_unpack(f[i], a, b);
        w[i] = pack2<T>(a, b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T>
__device__ __forceinline__ void load_weight8(const void *w, int f32, int at, uint64_t (&f)[4]) {
    if (f32) {
        const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(w) + at);
        const float4 a = __ldg(p), b = __ldg(p + 1);
        f[0] = f2_pack(a.x, a.y), f[1] = f2_pack(a.z, a.w), f[2] = f2_pack(b.x, b.y), f[3] = f2_pack(b.z, b.w);
    } else {
        unpack8<T>(__ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(w) + at)), f);
    }
}

// LANES = head_dim / 16 lanes hold a row.
template <typename T, int LANES, bool INTERLEAVED, bool APPEND>
__global__ void __launch_bounds__(kRopeThreads) qk_rope_kernel(const RopeParams p) {
    constexpr int kGroup = 32 / LANES;   // rows a warp holds at a time
    constexpr int kShare = 8 / kGroup;   // pairs whose sincospi a lane computes for its column of lanes
    constexpr int D = LANES * 16;
    const int lane = threadIdx.x & 31, l = lane % LANES, sub = lane / LANES;
    const uint32_t unit = blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
    const uint32_t token = unit / (uint32_t)p.units;
    if (token >= (uint32_t)p.T) return;
    const int64_t tok = token;
    // the warp's rows: heads [first, first + rows) of one kind
    int first = (int)(unit - token * (uint32_t)p.units);
    const bool is_q = first < p.q_units, is_v = APPEND && first >= p.q_units + p.k_units;
    first = (first - (is_q ? 0 : (is_v ? p.q_units + p.k_units : p.q_units))) * p.rows_per_unit;
    const int rows = min(p.rows_per_unit, (is_q ? p.Hq : p.Hkv) - first);
    // element offsets of this lane's two chunks within a row
    const bool turns = l < p.rot / 16;
    const int c0 = turns && !INTERLEAVED ? 8 * l : 16 * l;
    const int c1 = turns && !INTERLEAVED ? p.rot / 2 + 8 * l : 16 * l + 8;
    const T *src = is_q   ? static_cast<const T *>(p.q) + tok * p.q_stride
                   : is_v ? static_cast<const T *>(p.v) + tok * p.v_stride
                          : static_cast<const T *>(p.k) + tok * p.k_stride;
    src += (first + sub) * D;
    pdl_wait_primary();
    pdl_launch_dependents();

    uint4 a[kRopeSteps], b[kRopeSteps];
#pragma unroll
    for (int st = 0; st < kRopeSteps; ++st) {
        if (st * kGroup + sub < rows) {
            a[st] = *reinterpret_cast<const uint4 *>(src + st * kGroup * D + c0);
            b[st] = *reinterpret_cast<const uint4 *>(src + st * kGroup * D + c1);
        } else {
            a[st] = b[st] = make_uint4(0, 0, 0, 0);
        }
    }
    // where the rows go: as they came, or (a token's heads 16 rows apart in a block) into the cache
    T *dst;
    int64_t step = D;
    if (is_q) {
        dst = static_cast<T *>(p.q_out) + tok * p.q_out_stride;
    } else if constexpr (APPEND) {
        const int64_t slot = __ldg(p.slot_mapping + tok), block = slot >> 4;
        if (slot < 0 || block >= p.num_blocks) {
            if (slot >= 0 && lane == 0) set_status(p.dev_status, PKV_DEV_BAD_SLOT);
            return;
        }
        dst = static_cast<T *>(is_v ? p.v_cache : p.k_cache) + (block * p.Hkv * 16 + (slot & 15)) * D;
        step = 16 * D;
    } else {
        dst = static_cast<T *>(p.k_out) + tok * p.k_out_stride;
    }
    dst += (first + sub) * step;

    if (!is_v) {
        // cos and sin (times mscale) of pairs 2i and 2i + 1 of this lane
        uint64_t cs[4], sn[4];
        const uint64_t pos = (uint64_t)(int64_t)__ldg(p.positions + tok);
        float c[kShare], s[kShare];
#pragma unroll
        for (int e = 0; e < kShare; ++e) {
            const uint64_t turn = turns ? pos * (uint64_t)__ldg(p.freqs + 8 * l + kShare * sub + e) : 0ull;
            sincospif((float)(int32_t)(turn >> 32) * 4.656612873077393e-10f, &s[e], &c[e]);   // 2^-31: half turns
            c[e] *= p.mscale;
            s[e] *= p.mscale;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float v[4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int from = (2 * i + e) / kShare * LANES + l;
                v[e] = __shfl_sync(0xffffffffu, c[(2 * i + e) % kShare], from);
                v[2 + e] = __shfl_sync(0xffffffffu, s[(2 * i + e) % kShare], from);
            }
            cs[i] = f2_pack(v[0], v[1]);
            sn[i] = f2_pack(v[2], v[3]);
        }
        const void *w = is_q ? p.q_weight : p.k_weight;
        uint64_t w0[4], w1[4];
        if (w != nullptr) {
            load_weight8<T>(w, p.weight_f32, c0, w0);
            load_weight8<T>(w, p.weight_f32, c1, w1);
        }
        constexpr uint64_t kMinus = 0x8000000080000000ull;   // the signs of a packed pair
#pragma unroll
        for (int st = 0; st < kRopeSteps; ++st) {
            if (st * kGroup >= rows) break;
            uint64_t x0[4], x1[4];
            unpack8<T>(a[st], x0);
            unpack8<T>(b[st], x1);
            if (w != nullptr) {
                uint64_t s2 = f2_mul(x0[0], x0[0]), s3 = f2_mul(x1[0], x1[0]);
#pragma unroll
                for (int e = 1; e < 4; ++e) {
                    s2 = f2_fma(x0[e], x0[e], s2);
                    s3 = f2_fma(x1[e], x1[e], s3);
                }
                float u, v;
                f2_unpack(f2_add(s2, s3), u, v);
                float ss = u + v;
#pragma unroll
                for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                const float inv = rsqrtf(ss * (1.f / D) + p.eps);
                const uint64_t inv2 = f2_pack(inv, inv);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x0[e] = f2_mul(f2_mul(x0[e], inv2), w0[e]);
                    x1[e] = f2_mul(f2_mul(x1[e], inv2), w1[e]);
                }
            }
            if (turns) {
                if constexpr (INTERLEAVED) {
                    // (y0, y1) -> (y0, y1) c + (-y1, y0) s
                    auto turn = [&](uint64_t y, uint64_t c2, uint64_t s2) {
                        float y0, y1;
                        f2_unpack(y, y0, y1);
                        return f2_fma(f2_pack(-y1, y0), s2, f2_mul(y, c2));
                    };
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float ca, cb, sa, sb;
                        f2_unpack(cs[e], ca, cb);
                        f2_unpack(sn[e], sa, sb);
                        uint64_t *x = e < 2 ? x0 : x1;
                        x[2 * (e & 1)] = turn(x[2 * (e & 1)], f2_pack(ca, ca), f2_pack(sa, sa));
                        x[2 * (e & 1) + 1] = turn(x[2 * (e & 1) + 1], f2_pack(cb, cb), f2_pack(sb, sb));
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint64_t y0 = x0[e], y1 = x1[e];
                        x0[e] = f2_fma(y1 ^ kMinus, sn[e], f2_mul(y0, cs[e]));
                        x1[e] = f2_fma(y1, cs[e], f2_mul(y0, sn[e]));
                    }
                }
            }
            a[st] = pack8<T>(x0);
            b[st] = pack8<T>(x1);
        }
    }
#pragma unroll
    for (int st = 0; st < kRopeSteps; ++st) {
        if (st * kGroup + sub < rows) {
            *reinterpret_cast<uint4 *>(dst + st * kGroup * step + c0) = a[st];
            *reinterpret_cast<uint4 *>(dst + st * kGroup * step + c1) = b[st];
        }
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
static cudaError_t launch_rope_t(const RopeParams &prm, bool interleaved, bool append, int grid, cudaStream_t stream) {
    auto go = [&](auto kernel) { return launch_pdl(kernel, dim3(grid), dim3(kRopeThreads), 0, stream, prm); };
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
    // groups of rows a warp takes: kRopeSteps, fewer while that leaves SMs
    // with less than 16 warps
    const int group = 32 / (head_dim / 16);
    for (int steps = kRopeSteps;; --steps) {
        prm.rows_per_unit = steps * group;
        prm.q_units = (prm.Hq + prm.rows_per_unit - 1) / prm.rows_per_unit;
        prm.k_units = (prm.Hkv + prm.rows_per_unit - 1) / prm.rows_per_unit;
        prm.units = prm.q_units + (append ? 2 : 1) * prm.k_units;
        if (steps == 1 || (int64_t)prm.T * prm.units >= 16 * sms) break;
    }
    const int64_t warps = (int64_t)prm.T * prm.units;
    if (warps > INT32_MAX) return PKV_ERR_UNSUPPORTED;
    const int grid = (int)((warps + kRopeThreads / 32 - 1) / (kRopeThreads / 32));
    cudaError_t e;
    if (dtype == PKV_DTYPE_BF16)
        e = head_dim == 128 ? launch_rope_t<__nv_bfloat16, 8>(prm, interleaved, append, grid, stream)
                            : launch_rope_t<__nv_bfloat16, 4>(prm, interleaved, append, grid, stream);
    else
        e = head_dim == 128 ? launch_rope_t<__half, 8>(prm, interleaved, append, grid, stream)
                            : launch_rope_t<__half, 4>(prm, interleaved, append, grid, stream);
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
