// pkv_norm_rope.cu -- norms of q and k per head with the rotary rotation in the same pass, alone, fused with the
// append, or fused with the quantising append of the fp8 cache.
//
// A head's row x of q or k at a token becomes
//
//     y = x / sqrt(mean(x^2) + eps) * w,   then the first rotary_dim dims of y turn in pairs,
//     z_a = m (y_a cos t_i - y_b sin t_i),   z_b = m (y_b cos t_i + y_a sin t_i),   t_i = p[axis_i] f_i:
//
// a token has a position on each of one to four axes (time, height, width of a picture's patch) and pair i
// turns by the position on its own axis.  Everything from the row to z is float32, the norm's sum too; z is
// rounded once, to fp16, or for the fp8 cache to E4M3 codes with the row scale max|z| / 448 (codes of the
// float32 z: rounding to fp16 first would round twice).  Angles are the fixed-point phases of pkv_rope.
//
// What bounds it: memory; every row is read once and written once, some 7 flops an element.
//
// A row's 16-element units lie in LANES neighbouring lanes of a warp (8 for heads of 128 dims), so that a row's
// sums are log2(LANES) shuffles and a lane keeps one unit for all the rows it meets: its eight (cos, sin) pairs
// stay in registers.  A unit is 32 bytes (two 16-byte pieces): pieces c and c + rotary_dim / 16 hold both
// halves of eight half-layout pairs, two neighbouring pieces eight interleaved pairs.  One CTA takes one token
// (and, when tokens are few, a slice of its rows): the first rows' loads are in flight while rotary_dim / 2 of
// its threads compute the angles once for all heads.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "pkv.h"
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace {

__device__ int g_norm_error;

constexpr int kNormThreads = 128;
constexpr int kNormAhead = 3;  // rows a lane keeps in flight: 48 rows of 128 dims per CTA
constexpr int kMaxHeadDim = PKV_MAX_ROPE_HEAD_DIM;

struct NormParams {
    uint4 *q_out;
    const uint4 *q, *k, *v;     // v null: no append
    uint4 *k_out;               // without a cache
    uint4 *k_cache, *v_cache;   // fp16 cache
    uint2 *k_codes, *v_codes;   // fp8 cache: eight codes each
    float *k_scale, *v_scale;
    const int64_t *slot_mapping;
    const int32_t *positions;   // [num_tokens][num_axes]
    const int32_t *axes;        // [rotary_dim / 2], or null: all on axis 0
    const int64_t *frequencies;
    const float *q_weight, *k_weight;  // null: those rows are not normalised
    int64_t q_out_stride, q_stride, k_out_stride, k_stride, v_stride;  // 16-byte pieces between tokens
    int64_t num_slots;
    int num_q_heads, num_kv_heads, head_dim, rotary_dim, block_size, num_axes;
    int interleaved;
    float magnitude, eps, inv_dim;
    int rows_per_cta;
};

__device__ __forceinline__ void unpack(const uint4 &p, float *x) {
    const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = pkv::half2_bits_to_float2(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ uint4 pack(const float *x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint2 pack_e4m3(const float *x, float s) {
    return make_uint2(pkv::quantize_e4m3x2(x[0], x[1], s) | (pkv::quantize_e4m3x2(x[2], x[3], s) << 16),
                      pkv::quantize_e4m3x2(x[4], x[5], s) | (pkv::quantize_e4m3x2(x[6], x[7], s) << 16));
}

template <int LANES, bool FP8>
__global__ void __launch_bounds__(kNormThreads) norm_rope_kernel(const __grid_constant__ NormParams P) {
    constexpr int kRows = kNormThreads / LANES;  // rows of one pass
    // (cos, sin) of pair i = 8 u + 2 j + e at float4 j * LANES + u, weights of element 4 j + e of unit u likewise:
    // a row's lanes read neighbouring float4s.
    __shared__ float4 s_cs[4 * LANES], s_weight[2][4 * LANES];
    pkv::pdl_wait_primary();  // by every thread: the next kernel may rely on it
    pkv::pdl_launch_dependents();
    const int64_t t = blockIdx.x;
    const int units = P.head_dim / 16, r16 = P.rotary_dim / 16;
    const int u = threadIdx.x % LANES;
    const bool in_row = u < units;
    const int begin = blockIdx.y * P.rows_per_cta;
    const int rows = P.num_q_heads + P.num_kv_heads + (P.v ? P.num_kv_heads : 0);
    const int end = min(rows, begin + P.rows_per_cta);

    int64_t slot = -1, cache_row = 0;
    if (P.v) {
        slot = __ldg(P.slot_mapping + t);
        if (slot >= P.num_slots) {
            if (threadIdx.x == 0 && blockIdx.y == 0) pkv::record_error(&g_norm_error, PKV_DEV_BAD_SLOT);
            slot = -1;
        }
        if (slot >= 0) {
            const int64_t block = slot / P.block_size;
            cache_row = block * P.num_kv_heads * P.block_size + (slot - block * P.block_size);
        }
    }
    // Row `row` of the token: 0 q, 1 k, 2 v.
    auto kind_of = [&](int row) { return row < P.num_q_heads ? 0 : (row < P.num_q_heads + P.num_kv_heads ? 1 : 2); };
    auto live = [&](int row) { return in_row && row < end && (kind_of(row) == 0 || !P.v || slot >= 0); };
    // The two pieces of the lane's unit, in its row.
    auto first_of = [&](int kind) { return kind < 2 && u < r16 && !P.interleaved ? u : 2 * u; };
    auto second_of = [&](int kind) { return kind < 2 && u < r16 && !P.interleaved ? u + r16 : 2 * u + 1; };
    uint4 a[kNormAhead], b[kNormAhead];
    auto fetch = [&](int base) {
#pragma unroll
        for (int i = 0; i < kNormAhead; ++i) {
            const int row = base + i * kRows;
            a[i] = b[i] = make_uint4(0, 0, 0, 0);
            if (!live(row)) continue;
            const int kind = kind_of(row);
            const uint4 *src = kind == 0   ? P.q + t * P.q_stride + static_cast<int64_t>(row) * (2 * units)
                               : kind == 1 ? P.k + t * P.k_stride + static_cast<int64_t>(row - P.num_q_heads) * (2 * units)
                                           : P.v + t * P.v_stride + static_cast<int64_t>(row - P.num_q_heads - P.num_kv_heads) * (2 * units);
            a[i] = src[first_of(kind)];
            b[i] = src[second_of(kind)];
        }
    };
    const int row0 = begin + static_cast<int>(threadIdx.x) / LANES;
    fetch(row0);

    for (int i = threadIdx.x; i < P.rotary_dim / 2; i += kNormThreads) {
        int axis = P.axes ? __ldg(P.axes + i) : 0;
        if (axis < 0 || axis >= P.num_axes) {
            pkv::record_error(&g_norm_error, PKV_DEV_BAD_AXIS);
            axis = 0;
        }
        const uint64_t pos = static_cast<uint64_t>(static_cast<int64_t>(__ldg(P.positions + t * P.num_axes + axis)));
        const uint64_t turns = pos * static_cast<uint64_t>(__ldg(P.frequencies + i)) + (1ull << 31);
        const float x = static_cast<float>(static_cast<int32_t>(turns >> 32)) * (1.f / 2147483648.f);
        float si, co;
        sincospif(x, &si, &co);
        reinterpret_cast<float2 *>(s_cs)[(((i & 7) >> 1) * LANES + (i >> 3)) * 2 + (i & 1)] = make_float2(co * P.magnitude, si * P.magnitude);
    }
    for (int i = threadIdx.x; i < P.head_dim / 2; i += kNormThreads) {  // float4 i of q's weight, then of k's
        const bool is_k = i >= P.head_dim / 4;
        const float *w = is_k ? P.k_weight : P.q_weight;
        const int f = is_k ? i - P.head_dim / 4 : i, piece = f >> 1;
        const bool split = !P.interleaved && piece < 2 * r16;  // the halves' pieces: unit piece % r16
        const int unit = split ? (piece < r16 ? piece : piece - r16) : piece >> 1;
        const int second = split ? piece >= r16 : piece & 1;
        if (w) s_weight[is_k][(2 * second + (f & 1)) * LANES + unit] = __ldg(reinterpret_cast<const float4 *>(w) + f);
    }
    __syncthreads();
    float4 cs[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) cs[j] = u < r16 ? s_cs[j * LANES + u] : make_float4(0.f, 0.f, 0.f, 0.f);

    for (int base = row0; base - row0 < end - begin; base += kNormAhead * kRows) {  // (the same passes in all lanes)
        if (base != row0) fetch(base);
#pragma unroll
        for (int i = 0; i < kNormAhead; ++i) {
            const int row = base + i * kRows, kind = kind_of(row);
            if (i > 0 && base - row0 + i * kRows >= end - begin) break;  // (in all lanes)
            float x[16];  // zeros where the lane holds nothing
            unpack(a[i], x);
            unpack(b[i], x + 8);
            const bool normed = kind == 0 ? P.q_weight != nullptr : kind == 1 && P.k_weight != nullptr;
            float2 sum = {0.f, 0.f};
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
                sum.x = fmaf(x[e], x[e], sum.x);
                sum.y = fmaf(x[e + 1], x[e + 1], sum.y);
            }
            float square = sum.x + sum.y;
#pragma unroll
            for (int d = LANES / 2; d >= 1; d >>= 1) square += __shfl_xor_sync(pkv::kFullMask, square, d);
            if (normed && in_row) {
                const float r = rsqrtf(fmaf(square, P.inv_dim, P.eps));
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 w = s_weight[kind][j * LANES + u];
                    x[4 * j] *= r * w.x;
                    x[4 * j + 1] *= r * w.y;
                    x[4 * j + 2] *= r * w.z;
                    x[4 * j + 3] *= r * w.w;
                }
            }
            if (kind < 2 && u < r16) {
                if (P.interleaved) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float c0 = x[4 * j], c1 = x[4 * j + 1], c2 = x[4 * j + 2], c3 = x[4 * j + 3];
                        x[4 * j] = c0 * cs[j].x - c1 * cs[j].y;
                        x[4 * j + 1] = c1 * cs[j].x + c0 * cs[j].y;
                        x[4 * j + 2] = c2 * cs[j].z - c3 * cs[j].w;
                        x[4 * j + 3] = c3 * cs[j].z + c2 * cs[j].w;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float a0 = x[2 * j], a1 = x[2 * j + 1], b0 = x[8 + 2 * j], b1 = x[9 + 2 * j];
                        x[2 * j] = a0 * cs[j].x - b0 * cs[j].y;
                        x[8 + 2 * j] = b0 * cs[j].x + a0 * cs[j].y;
                        x[2 * j + 1] = a1 * cs[j].z - b1 * cs[j].w;
                        x[9 + 2 * j] = b1 * cs[j].z + a1 * cs[j].w;
                    }
                }
            }
            const int first = first_of(kind), second = second_of(kind);
            if (FP8) {
                float most = 0.f;
#pragma unroll
                for (int e = 0; e < 16; ++e) most = fmaxf(most, fabsf(x[e]));
#pragma unroll
                for (int d = LANES / 2; d >= 1; d >>= 1) most = fmaxf(most, __shfl_xor_sync(pkv::kFullMask, most, d));
                if (kind != 0 && live(row)) {
                    const float s = __fdiv_rn(most, 448.f);
                    const int kvh = row - P.num_q_heads - (kind == 2 ? P.num_kv_heads : 0);
                    const int64_t to = cache_row + static_cast<int64_t>(kvh) * P.block_size;
                    uint2 *codes = (kind == 2 ? P.v_codes : P.k_codes) + to * (2 * units);
                    codes[first] = pack_e4m3(x, s);
                    codes[second] = pack_e4m3(x + 8, s);
                    if (u == 0) (kind == 2 ? P.v_scale : P.k_scale)[to] = s;
                    continue;
                }
            }
            if (!live(row)) continue;
            uint4 *dst;
            if (kind == 0) {
                dst = P.q_out + t * P.q_out_stride + static_cast<int64_t>(row) * (2 * units);
            } else {
                const int kvh = row - P.num_q_heads - (kind == 2 ? P.num_kv_heads : 0);
                dst = P.v ? (kind == 2 ? P.v_cache : P.k_cache) + (cache_row + static_cast<int64_t>(kvh) * P.block_size) * (2 * units)
                          : P.k_out + t * P.k_out_stride + static_cast<int64_t>(kvh) * (2 * units);
            }
            dst[first] = pack(x);
            dst[second] = pack(x + 8);
        }
    }
}

// Strides arrive in elements.  A row of heads must not run into the next token's.
bool stride_ok(int64_t stride, int heads, int head_dim, int num_tokens) {
    if (stride % 8 != 0) return false;
    return num_tokens <= 1 || stride >= static_cast<int64_t>(heads) * head_dim;
}

template <bool FP8>
int launch_norm_rope(NormParams p, int num_tokens, pkv_stream_t stream) {
    const int units = p.head_dim / 16;
    const int lanes = units <= 1 ? 1 : (units <= 2 ? 2 : (units <= 4 ? 4 : (units <= 8 ? 8 : 16)));
    const int pass = kNormThreads / lanes, rows = p.num_q_heads + p.num_kv_heads + (p.v ? p.num_kv_heads : 0);
    // One CTA per token; with few tokens a token's rows are cut into single passes, so that a decode step's call
    // is one round of loads on many SMs instead of three on few.
    p.rows_per_cta = num_tokens <= 304 ? pass : (rows + pass - 1) / pass * pass;
    p.inv_dim = 1.f / static_cast<float>(p.head_dim);
    const int64_t slices = (rows + p.rows_per_cta - 1) / p.rows_per_cta;
    if (slices > 65535) return PKV_ERR_UNSUPPORTED;
    auto kernel = FP8            ? norm_rope_kernel<8, FP8>
                  : lanes == 1   ? norm_rope_kernel<1, false>
                  : lanes == 2   ? norm_rope_kernel<2, false>
                  : lanes == 4   ? norm_rope_kernel<4, false>
                  : lanes == 8   ? norm_rope_kernel<8, false>
                                 : norm_rope_kernel<16, false>;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(num_tokens), static_cast<unsigned>(slices));
    cfg.blockDim = dim3(kNormThreads);
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

// What the three calls check of q, k, the positions and the norms.
int check_norm_rope(const void *q_out, int64_t q_out_stride, const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                    const int32_t *positions, const int32_t *axes, int num_axes, const int64_t *frequencies,
                    const float *q_weight, const float *k_weight, float eps, int num_tokens, int num_q_heads,
                    int num_kv_heads, int head_dim, int rotary_dim, float magnitude) {
    if (num_tokens < 0 || num_q_heads < 0 || num_kv_heads < 0 || num_q_heads + num_kv_heads == 0 || head_dim <= 0 ||
        rotary_dim <= 0 || rotary_dim > head_dim || num_axes < 1 || (num_axes > 1 && !axes))
        return PKV_ERR_INVALID_ARG;
    if (!isfinite(magnitude) || !(eps >= 0.f) || !isfinite(eps)) return PKV_ERR_INVALID_ARG;
    if (num_q_heads > 65535 || num_kv_heads > 65535 || num_axes > PKV_MAX_ROPE_AXES) return PKV_ERR_UNSUPPORTED;
    if (head_dim % 16 != 0 || rotary_dim % 16 != 0 || head_dim > kMaxHeadDim) return PKV_ERR_UNSUPPORTED;
    if (!pkv_internal::aligned16(q_weight) || !pkv_internal::aligned16(k_weight) || !pkv_internal::aligned(axes, 4))
        return PKV_ERR_INVALID_ARG;
    if (num_tokens == 0) return PKV_OK;
    if ((num_q_heads > 0 && (!q_out || !q)) || (num_kv_heads > 0 && !k) || !positions || !frequencies)
        return PKV_ERR_INVALID_ARG;
    if (!pkv_internal::aligned16(q_out) || !pkv_internal::aligned16(q) || !pkv_internal::aligned16(k) ||
        !pkv_internal::aligned(positions, 4) || !pkv_internal::aligned(frequencies, 8))
        return PKV_ERR_INVALID_ARG;
    if (!stride_ok(q_out_stride, num_q_heads, head_dim, num_tokens) || !stride_ok(q_stride, num_q_heads, head_dim, num_tokens) ||
        !stride_ok(k_stride, num_kv_heads, head_dim, num_tokens))
        return PKV_ERR_INVALID_ARG;
    return PKV_OK;
}

NormParams params_of(void *q_out, int64_t q_out_stride, const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                     const int32_t *positions, const int32_t *axes, int num_axes, const int64_t *frequencies,
                     const float *q_weight, const float *k_weight, float eps, int num_q_heads, int num_kv_heads,
                     int head_dim, int rotary_dim, int interleaved, float magnitude) {
    NormParams p{};
    p.q_out = static_cast<uint4 *>(q_out);
    p.q = static_cast<const uint4 *>(q);
    p.k = static_cast<const uint4 *>(k);
    p.positions = positions;
    p.axes = axes;
    p.num_axes = num_axes;
    p.frequencies = frequencies;
    p.q_weight = q_weight;
    p.k_weight = k_weight;
    p.eps = eps;
    p.q_out_stride = q_out_stride / 8;
    p.q_stride = q_stride / 8;
    p.k_stride = k_stride / 8;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.head_dim = head_dim;
    p.rotary_dim = rotary_dim;
    p.block_size = 1;
    p.interleaved = interleaved != 0;
    p.magnitude = magnitude;
    return p;
}

}  // namespace

extern "C" PKV_API int pkv_norm_rope(void *q_out, int64_t q_out_stride, void *k_out, int64_t k_out_stride, const void *q,
                                     int64_t q_stride, const void *k, int64_t k_stride, const int32_t *positions,
                                     const int32_t *axes, int num_axes, const int64_t *frequencies,
                                     const float *q_weight, const float *k_weight, float eps, int num_tokens,
                                     int num_q_heads, int num_kv_heads, int head_dim, int rotary_dim, int interleaved,
                                     float magnitude, pkv_stream_t stream) {
    const int st = check_norm_rope(q_out, q_out_stride, q, q_stride, k, k_stride, positions, axes, num_axes, frequencies, q_weight,
                                   k_weight, eps, num_tokens, num_q_heads, num_kv_heads, head_dim, rotary_dim, magnitude);
    if (st != PKV_OK || num_tokens == 0) return st;
    if (num_kv_heads > 0 && (!k_out || !pkv_internal::aligned16(k_out))) return PKV_ERR_INVALID_ARG;
    if (!stride_ok(k_out_stride, num_kv_heads, head_dim, num_tokens)) return PKV_ERR_INVALID_ARG;
    NormParams p = params_of(q_out, q_out_stride, q, q_stride, k, k_stride, positions, axes, num_axes, frequencies, q_weight, k_weight,
                             eps, num_q_heads, num_kv_heads, head_dim, rotary_dim, interleaved, magnitude);
    p.k_out = static_cast<uint4 *>(k_out);
    p.k_out_stride = k_out_stride / 8;
    return launch_norm_rope<false>(p, num_tokens, stream);
}

extern "C" PKV_API int pkv_norm_rope_append(void *q_out, int64_t q_out_stride, const void *q, int64_t q_stride,
                                            const void *k_new, int64_t k_stride, const void *v_new, int64_t v_stride,
                                            void *k_cache, void *v_cache, const int64_t *slot_mapping,
                                            const int32_t *positions, const int32_t *axes, int num_axes,
                                            const int64_t *frequencies, const float *q_weight, const float *k_weight,
                                            float eps, int num_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                                            int rotary_dim, int block_size, int64_t num_blocks, int interleaved,
                                            float magnitude, pkv_stream_t stream) {
    const int st = check_norm_rope(q_out, q_out_stride, q, q_stride, k_new, k_stride, positions, axes, num_axes, frequencies, q_weight,
                                   k_weight, eps, num_tokens, num_q_heads, num_kv_heads, head_dim, rotary_dim, magnitude);
    if (st != PKV_OK) return st;
    if (num_kv_heads <= 0 || block_size <= 0 || num_blocks <= 0 || !k_cache || !v_cache) return PKV_ERR_INVALID_ARG;
    if (!pkv_internal::aligned16(k_cache) || !pkv_internal::aligned16(v_cache)) return PKV_ERR_INVALID_ARG;
    if (num_tokens == 0) return PKV_OK;
    if (!v_new || !slot_mapping || !pkv_internal::aligned16(v_new) || !pkv_internal::aligned(slot_mapping, 8) ||
        !stride_ok(v_stride, num_kv_heads, head_dim, num_tokens))
        return PKV_ERR_INVALID_ARG;
    NormParams p = params_of(q_out, q_out_stride, q, q_stride, k_new, k_stride, positions, axes, num_axes, frequencies, q_weight,
                             k_weight, eps, num_q_heads, num_kv_heads, head_dim, rotary_dim, interleaved, magnitude);
    p.v = static_cast<const uint4 *>(v_new);
    p.v_stride = v_stride / 8;
    p.k_cache = static_cast<uint4 *>(k_cache);
    p.v_cache = static_cast<uint4 *>(v_cache);
    p.slot_mapping = slot_mapping;
    p.num_slots = num_blocks * block_size;
    p.block_size = block_size;
    return launch_norm_rope<false>(p, num_tokens, stream);
}

extern "C" PKV_API int pkv_norm_rope_append_fp8kv(void *q_out, int64_t q_out_stride, const void *q, int64_t q_stride,
                                                  const void *k_new, int64_t k_stride, const void *v_new,
                                                  int64_t v_stride, void *k_codes, float *k_scale, void *v_codes,
                                                  float *v_scale, const int64_t *slot_mapping, const int32_t *positions,
                                                  const int32_t *axes, int num_axes, const int64_t *frequencies,
                                                  const float *q_weight, const float *k_weight, float eps,
                                                  int num_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                                                  int rotary_dim, int block_size, int64_t num_blocks, int interleaved,
                                                  float magnitude, pkv_stream_t stream) {
    const int st = check_norm_rope(q_out, q_out_stride, q, q_stride, k_new, k_stride, positions, axes, num_axes, frequencies, q_weight,
                                   k_weight, eps, num_tokens, num_q_heads, num_kv_heads, head_dim, rotary_dim, magnitude);
    if (st != PKV_OK) return st;
    if (head_dim != PKV_HEAD_DIM) return PKV_ERR_UNSUPPORTED;
    if (num_kv_heads <= 0 || block_size <= 0 || num_blocks <= 0 || !k_codes || !k_scale || !v_codes || !v_scale) return PKV_ERR_INVALID_ARG;
    if (!pkv_internal::aligned16(k_codes) || !pkv_internal::aligned16(v_codes) || !pkv_internal::aligned(k_scale, 4) ||
        !pkv_internal::aligned(v_scale, 4))
        return PKV_ERR_INVALID_ARG;
    if (num_tokens == 0) return PKV_OK;
    if (!v_new || !slot_mapping || !pkv_internal::aligned16(v_new) || !pkv_internal::aligned(slot_mapping, 8) ||
        !stride_ok(v_stride, num_kv_heads, head_dim, num_tokens))
        return PKV_ERR_INVALID_ARG;
    NormParams p = params_of(q_out, q_out_stride, q, q_stride, k_new, k_stride, positions, axes, num_axes, frequencies, q_weight,
                             k_weight, eps, num_q_heads, num_kv_heads, head_dim, rotary_dim, interleaved, magnitude);
    p.v = static_cast<const uint4 *>(v_new);
    p.v_stride = v_stride / 8;
    p.k_codes = static_cast<uint2 *>(k_codes);
    p.v_codes = static_cast<uint2 *>(v_codes);
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.slot_mapping = slot_mapping;
    p.num_slots = num_blocks * block_size;
    p.block_size = block_size;
    return launch_norm_rope<true>(p, num_tokens, stream);
}

namespace pkv_internal {

int norm_rope_take_error(int *code) {
    int value = 0;
    if (cudaMemcpyFromSymbol(&value, g_norm_error, sizeof(int)) != cudaSuccess) return PKV_ERR_CUDA;
    if (value != 0) {
        const int zero = 0;
        if (cudaMemcpyToSymbol(g_norm_error, &zero, sizeof(int)) != cudaSuccess) return PKV_ERR_CUDA;
    }
    *code = value;
    return PKV_OK;
}

}  // namespace pkv_internal
