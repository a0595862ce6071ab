// pkv_rope.cu -- rotary positions for q and k, alone or fused with the append into the paged cache.
//
// A token at position p rotates the pairs (x_a, x_b) of the first `rotary_dim` dims of every head,
//
//     y_a = m (x_a cos t_i - x_b sin t_i),   y_b = m (x_b cos t_i + x_a sin t_i),   t_i = p f_i,
//
// pair i being dims (i, i + rotary_dim / 2) (half layout) or (2i, 2i + 1) (interleaved); the dims
// past rotary_dim pass through unchanged.  The arithmetic is float32, rounded once to fp16.
//
// The angle.  p f_i reaches 10^6 radians, where a float32 product has lost every bit of the phase and
// float64 runs at a thousandth of the float32 rate here.  The frequencies are therefore fixed-point:
// f_i / 2 pi in units of 2^-64 turns, and p x frequency in wrapping 64-bit integers is the phase
// modulo one turn, exactly.  What is rounded is the frequency: computed in float64, it is off by some 2^-53 of itself (and
// by 2^-65 turns, half a unit), so the phase by some 2^-55 p turns for the fastest pairs: 2^-24 turns at the largest
// position, 2^-35 at a million.  Its upper 32 bits, signed, are a fraction in [-1/2, 1/2)
// turns, and sincospif takes them from there.
//
// What bounds it: memory (every row is read once and written once; 3 flops an element): 8192 tokens of 48
// rows, half of each head rotated in interleaved pairs, 201 MB in 35.6 us, 5.65 TB/s, 85 % of what a plain copy
// reaches; 4099 tokens of 64 rows out of a fused projection, 134 MB in 23.3 us, 86 %.  The issue slots are half
// busy beside it.  A decode step's 16 tokens take 2.2 us (back to back in a graph).  One CTA
// takes one token (and, when tokens are few, a slice of its rows, so that the call spreads over the
// SMs): its rows' first loads are in flight while rotary_dim / 2 of its threads compute the angles
// once for all heads into shared memory.  A thread's unit is 32 bytes (two 16-byte pieces): pieces c
// and c + rotary_dim / 16 hold both halves of eight half-layout pairs, two neighbouring pieces eight
// interleaved pairs.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "pkv.h"
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace {

__device__ int g_rope_error;

constexpr int kRopeThreads = 128;
constexpr int kRopePrefetch = 3;   // units a thread keeps in flight: 384 = 48 rows of 128 dims
constexpr int kMaxHeadDim = 256;

struct RopeParams {
    uint4 *q_out;
    const uint4 *q;
    uint4 *k_out;  // rotated k rows, or null: they go to k_cache
    const uint4 *k;
    const uint4 *v;  // appended unrotated (null without a cache)
    uint4 *k_cache, *v_cache;
    const int64_t *slot_mapping;
    const int32_t *positions;
    const int64_t *frequencies;
    int64_t q_out_stride, q_stride, k_out_stride, k_stride, v_stride;  // 16-byte pieces between tokens
    int64_t num_slots;
    int num_q_heads, num_kv_heads, head_dim, rotary_dim, block_size;
    int interleaved;
    float magnitude;
    int units_per_cta;
};

// Eight rotated pairs: (a, b) the halves' pieces, or two neighbouring interleaved pieces.
__device__ __forceinline__ void rotate_unit(uint4 &x, uint4 &y, const float4 *cs, int stride, bool interleaved) {
    uint32_t a[4] = {x.x, x.y, x.z, x.w}, b[4] = {y.x, y.y, y.z, y.w};
    if (interleaved) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float4 c = cs[j * stride];  // (cos, sin) of pairs 2j and 2j + 1 of the unit
            uint32_t(&w)[4] = j < 2 ? a : b;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float2 p = pkv::half2_bits_to_float2(w[(2 * j + e) & 3]);
                const float co = e ? c.z : c.x, si = e ? c.w : c.y;
                const __half2 r = __floats2half2_rn(p.x * co - p.y * si, p.y * co + p.x * si);
                w[(2 * j + e) & 3] = *reinterpret_cast<const uint32_t *>(&r);
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float4 c = cs[j * stride];
            const float2 p = pkv::half2_bits_to_float2(a[j]), q = pkv::half2_bits_to_float2(b[j]);
            const __half2 u = __floats2half2_rn(p.x * c.x - q.x * c.y, p.y * c.z - q.y * c.w);
            const __half2 v = __floats2half2_rn(q.x * c.x + p.x * c.y, q.y * c.z + p.y * c.w);
            a[j] = *reinterpret_cast<const uint32_t *>(&u);
            b[j] = *reinterpret_cast<const uint32_t *>(&v);
        }
    }
    x = make_uint4(a[0], a[1], a[2], a[3]);
    y = make_uint4(b[0], b[1], b[2], b[3]);
}

// UNITS: units per row where known at compile time (8: heads of 128 dims, whose 8192-token append takes 35.6 us
// that way and 35.9 the other), else 0.
template <int UNITS>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams P) {
    // (cos, sin) of pair i = 8 u + 2 j + e at float4 j * (rotary / 16) + u: neighbouring units' reads
    // of one j are neighbouring float4s.
    __shared__ float4 s_cs[kMaxHeadDim / 4];
    pkv::pdl_wait_primary();  // by every thread: the next kernel may rely on it
    pkv::pdl_launch_dependents();
    const int64_t t = blockIdx.x;
    const int units_per_row = UNITS ? UNITS : P.head_dim / 16;
    const int r16 = P.rotary_dim / 16;
    const int heads = P.num_q_heads + P.num_kv_heads + (P.v ? P.num_kv_heads : 0);
    const int begin = blockIdx.y * P.units_per_cta;
    const int end = min(heads * units_per_row, begin + P.units_per_cta);

    int64_t slot = 0;
    if (P.k_cache) {
        slot = __ldg(P.slot_mapping + t);
        if (slot >= P.num_slots) {
            if (threadIdx.x == 0 && blockIdx.y == 0) pkv::record_error(&g_rope_error, PKV_DEV_BAD_SLOT);
            slot = -1;
        }
    }
    const int64_t block = P.k_cache && slot >= 0 ? slot / P.block_size : 0;
    const int64_t cache_row = P.k_cache ? block * P.num_kv_heads * P.block_size + (max(slot, static_cast<int64_t>(0)) - block * P.block_size) : 0;
    // A unit's two pieces: where they are read and written; `first` is the piece in its row.
    struct Unit {
        const uint4 *src;
        uint4 *dst;
        int u, first, second;
        bool live, rotated;
    };
    auto locate = [&](int unit) {
        Unit x{nullptr, nullptr, 0, 0, 0, false, false};
        if (unit >= end) return x;
        const int row = unit / units_per_row;
        x.u = unit - row * units_per_row;
        int kvh = row - P.num_q_heads;
        const bool is_v = kvh >= P.num_kv_heads;
        if (is_v) kvh -= P.num_kv_heads;
        x.rotated = !is_v && x.u < r16;
        x.first = x.rotated && !P.interleaved ? x.u : 2 * x.u;
        x.second = x.rotated && !P.interleaved ? x.u + r16 : 2 * x.u + 1;
        const int pieces = 2 * units_per_row;
        x.live = true;
        if (row < P.num_q_heads) {
            x.src = P.q + t * P.q_stride + static_cast<int64_t>(row) * pieces;
            x.dst = P.q_out + t * P.q_out_stride + static_cast<int64_t>(row) * pieces;
        } else {
            x.src = (is_v ? P.v + t * P.v_stride : P.k + t * P.k_stride) + static_cast<int64_t>(kvh) * pieces;
            if (P.k_cache) {
                x.live = slot >= 0;  // a padding token: its k and v go nowhere
                x.dst = (is_v ? P.v_cache : P.k_cache) + (cache_row + static_cast<int64_t>(kvh) * P.block_size) * pieces;
            } else {
                x.dst = P.k_out + t * P.k_out_stride + static_cast<int64_t>(kvh) * pieces;
            }
        }
        if (!x.rotated && x.src == x.dst) x.live = false;  // in place: nothing to do past rotary_dim
        return x;
    };
    Unit un[kRopePrefetch];
    uint4 a[kRopePrefetch], b[kRopePrefetch];
    auto fetch = [&](int base) {
#pragma unroll
        for (int i = 0; i < kRopePrefetch; ++i) {
            un[i] = locate(base + i * kRopeThreads);
            if (un[i].live) {
                a[i] = un[i].src[un[i].first];
                b[i] = un[i].src[un[i].second];
            }
        }
    };
    fetch(begin + threadIdx.x);

    const uint64_t pos = static_cast<uint64_t>(static_cast<int64_t>(__ldg(P.positions + t)));
    for (int i = threadIdx.x; i < P.rotary_dim / 2; i += kRopeThreads) {
        const uint64_t turns = pos * static_cast<uint64_t>(__ldg(P.frequencies + i)) + (1ull << 31);
        const float x = static_cast<float>(static_cast<int32_t>(turns >> 32)) * (1.f / 2147483648.f);
        float si, co;
        sincospif(x, &si, &co);
        const int u = i >> 3, j = (i & 7) >> 1;
        reinterpret_cast<float2 *>(s_cs)[(j * r16 + u) * 2 + (i & 1)] = make_float2(co * P.magnitude, si * P.magnitude);
    }
    __syncthreads();
    for (int base = begin + threadIdx.x; base < end; base += kRopePrefetch * kRopeThreads) {
        if (base != begin + static_cast<int>(threadIdx.x)) fetch(base);
#pragma unroll
        for (int i = 0; i < kRopePrefetch; ++i) {
            if (!un[i].live) continue;
            if (un[i].rotated) rotate_unit(a[i], b[i], s_cs + un[i].u, r16, P.interleaved != 0);
            un[i].dst[un[i].first] = a[i];
            un[i].dst[un[i].second] = b[i];
        }
    }
}

// Strides arrive in elements.  A row of heads must not run into the next token's.
bool stride_ok(int64_t stride, int heads, int head_dim, int num_tokens) {
    if (stride % 8 != 0) return false;
    return num_tokens <= 1 || stride >= static_cast<int64_t>(heads) * head_dim;
}

int launch_rope(RopeParams p, int num_tokens, pkv_stream_t stream) {
    const int units = (p.num_q_heads + p.num_kv_heads + (p.v ? p.num_kv_heads : 0)) * (p.head_dim / 16);
    // One CTA per token and kRopePrefetch units a thread are one pass; with few tokens a token's rows
    // are cut into slices of one unit a thread, so that a decode step's call is one round of loads on
    // many SMs instead of three on few (48 rows, in a graph: 16 tokens 2.2 us sliced and 2.6 whole, 304 tokens 2.9
    // both, 512 tokens 4.4 and 3.4).
    const int per_cta = num_tokens <= 304 ? kRopeThreads : ((units + kRopeThreads - 1) / kRopeThreads) * kRopeThreads;
    const int64_t slices = (units + per_cta - 1) / per_cta;
    if (slices > 65535) return PKV_ERR_UNSUPPORTED;
    p.units_per_cta = per_cta;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(num_tokens), static_cast<unsigned>(slices));
    cfg.blockDim = dim3(kRopeThreads);
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, p.head_dim == 128 ? rope_kernel<8> : rope_kernel<0>, p) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

int check_rope(const void *q_out, const void *q, const void *k, const int32_t *positions, const int64_t *frequencies,
               int num_tokens, int num_q_heads, int num_kv_heads, int head_dim, int rotary_dim, float magnitude) {
    if (num_tokens < 0 || num_q_heads < 0 || num_kv_heads < 0 || num_q_heads + num_kv_heads == 0 || head_dim <= 0 ||
        rotary_dim <= 0 || rotary_dim > head_dim)
        return PKV_ERR_INVALID_ARG;
    if (num_q_heads > 65535 || num_kv_heads > 65535) return PKV_ERR_UNSUPPORTED;
    if (!isfinite(magnitude)) return PKV_ERR_INVALID_ARG;
    if (head_dim % 16 != 0 || rotary_dim % 16 != 0 || head_dim > kMaxHeadDim) return PKV_ERR_UNSUPPORTED;
    if (num_tokens == 0) return PKV_OK;
    if ((num_q_heads > 0 && (!q_out || !q)) || (num_kv_heads > 0 && !k) || !positions || !frequencies)
        return PKV_ERR_INVALID_ARG;
    if (!pkv_internal::aligned16(q_out) || !pkv_internal::aligned16(q) || !pkv_internal::aligned16(k) ||
        !pkv_internal::aligned(positions, 4) || !pkv_internal::aligned(frequencies, 8))
        return PKV_ERR_INVALID_ARG;
    return PKV_OK;
}

}  // namespace

extern "C" PKV_API int pkv_rope_frequencies(int64_t *frequencies, double *magnitude, const pkv_rope_spec *spec) {
    if (!spec || (!frequencies && !magnitude)) return PKV_ERR_INVALID_ARG;
    const int d = spec->rotary_dim;
    const double base = spec->base, factor = spec->factor, ctx = spec->original_context;
    const double slow = spec->slow_turns, fast = spec->fast_turns;
    if (d <= 0 || d % 2 != 0 || !(base > 1.0) || !isfinite(base)) return PKV_ERR_INVALID_ARG;
    if (spec->method < PKV_ROPE_PLAIN || spec->method > PKV_ROPE_RAMP) return PKV_ERR_INVALID_ARG;
    if (spec->method != PKV_ROPE_PLAIN && !(factor >= 1.0 && isfinite(factor))) return PKV_ERR_INVALID_ARG;
    if (spec->method == PKV_ROPE_BASE && d <= 2) return PKV_ERR_INVALID_ARG;
    if (spec->method >= PKV_ROPE_BANDS &&
        (!(ctx > 0.0) || !isfinite(ctx) || !(slow > 0.0) || !(fast > slow) || !isfinite(fast)))
        return PKV_ERR_INVALID_ARG;
    constexpr double kTurn = 6.283185307179586476925286766559;
    if (magnitude) *magnitude = spec->method == PKV_ROPE_RAMP ? 0.1 * log(factor) + 1.0 : 1.0;
    if (!frequencies) return PKV_OK;
    double lo = 0.0, hi = 0.0;
    if (spec->method == PKV_ROPE_RAMP) {  // the pair index that makes n turns over ctx tokens
        lo = fmax(floor(d * log(ctx / (fast * kTurn)) / (2.0 * log(base))), 0.0);
        hi = fmin(ceil(d * log(ctx / (slow * kTurn)) / (2.0 * log(base))), d - 1.0);
    }
    for (int i = 0; i < d / 2; ++i) {
        double f = pow(base, -2.0 * i / d), keep = 1.0;
        if (spec->method == PKV_ROPE_LINEAR) {
            f /= factor;
        } else if (spec->method == PKV_ROPE_BASE) {
            f = pow(base * pow(factor, static_cast<double>(d) / (d - 2)), -2.0 * i / d);
        } else if (spec->method == PKV_ROPE_BANDS) {
            keep = fmin(fmax((ctx * f / kTurn - slow) / (fast - slow), 0.0), 1.0);
            f = keep * f + (1.0 - keep) * f / factor;
        } else if (spec->method == PKV_ROPE_RAMP) {
            keep = 1.0 - fmin(fmax((i - lo) / fmax(hi - lo, 1e-3), 0.0), 1.0);
            f = keep * f + (1.0 - keep) * f / factor;
        }
        frequencies[i] = static_cast<int64_t>(llrint(ldexp(f / kTurn, 64)));  // f <= 1: below 2^62
    }
    return PKV_OK;
}

extern "C" PKV_API int pkv_rope(void *q_out, int64_t q_out_stride, void *k_out, int64_t k_out_stride, const void *q,
                                int64_t q_stride, const void *k, int64_t k_stride, const int32_t *positions,
                                const int64_t *frequencies, int num_tokens, int num_q_heads, int num_kv_heads,
                                int head_dim, int rotary_dim, int interleaved, float magnitude, pkv_stream_t stream) {
    const int st = check_rope(q_out, q, k, positions, frequencies, num_tokens, num_q_heads, num_kv_heads, head_dim,
                              rotary_dim, magnitude);
    if (st != PKV_OK || num_tokens == 0) return st;
    if (num_kv_heads > 0 && (!k_out || !pkv_internal::aligned16(k_out))) return PKV_ERR_INVALID_ARG;
    if (!stride_ok(q_out_stride, num_q_heads, head_dim, num_tokens) || !stride_ok(q_stride, num_q_heads, head_dim, num_tokens) ||
        !stride_ok(k_out_stride, num_kv_heads, head_dim, num_tokens) || !stride_ok(k_stride, num_kv_heads, head_dim, num_tokens))
        return PKV_ERR_INVALID_ARG;
    RopeParams p{};
    p.q_out = static_cast<uint4 *>(q_out);
    p.q = static_cast<const uint4 *>(q);
    p.k_out = static_cast<uint4 *>(k_out);
    p.k = static_cast<const uint4 *>(k);
    p.positions = positions;
    p.frequencies = frequencies;
    p.q_out_stride = q_out_stride / 8;
    p.q_stride = q_stride / 8;
    p.k_out_stride = k_out_stride / 8;
    p.k_stride = k_stride / 8;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.head_dim = head_dim;
    p.rotary_dim = rotary_dim;
    p.block_size = 1;
    p.interleaved = interleaved != 0;
    p.magnitude = magnitude;
    return launch_rope(p, num_tokens, stream);
}

extern "C" PKV_API int pkv_rope_append(void *q_out, int64_t q_out_stride, const void *q, int64_t q_stride,
                                       const void *k_new, int64_t k_stride, const void *v_new, int64_t v_stride,
                                       void *k_cache, void *v_cache, const int64_t *slot_mapping,
                                       const int32_t *positions, const int64_t *frequencies, int num_tokens,
                                       int num_q_heads, int num_kv_heads, int head_dim, int rotary_dim,
                                       int block_size, int64_t num_blocks, int interleaved, float magnitude,
                                       pkv_stream_t stream) {
    const int st = check_rope(q_out, q, k_new, positions, frequencies, num_tokens, num_q_heads, num_kv_heads, head_dim,
                              rotary_dim, magnitude);
    if (st != PKV_OK) return st;
    if (num_kv_heads <= 0 || block_size <= 0 || num_blocks <= 0 || !k_cache || !v_cache) return PKV_ERR_INVALID_ARG;
    if (!pkv_internal::aligned16(k_cache) || !pkv_internal::aligned16(v_cache)) return PKV_ERR_INVALID_ARG;
    if (num_tokens == 0) return PKV_OK;
    if (!v_new || !slot_mapping || !pkv_internal::aligned16(v_new) || !pkv_internal::aligned(slot_mapping, 8))
        return PKV_ERR_INVALID_ARG;
    if (!stride_ok(q_out_stride, num_q_heads, head_dim, num_tokens) || !stride_ok(q_stride, num_q_heads, head_dim, num_tokens) ||
        !stride_ok(k_stride, num_kv_heads, head_dim, num_tokens) || !stride_ok(v_stride, num_kv_heads, head_dim, num_tokens))
        return PKV_ERR_INVALID_ARG;
    RopeParams p{};
    p.q_out = static_cast<uint4 *>(q_out);
    p.q = static_cast<const uint4 *>(q);
    p.k = static_cast<const uint4 *>(k_new);
    p.v = static_cast<const uint4 *>(v_new);
    p.k_cache = static_cast<uint4 *>(k_cache);
    p.v_cache = static_cast<uint4 *>(v_cache);
    p.slot_mapping = slot_mapping;
    p.positions = positions;
    p.frequencies = frequencies;
    p.q_out_stride = q_out_stride / 8;
    p.q_stride = q_stride / 8;
    p.k_stride = k_stride / 8;
    p.v_stride = v_stride / 8;
    p.num_slots = num_blocks * block_size;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.head_dim = head_dim;
    p.rotary_dim = rotary_dim;
    p.block_size = block_size;
    p.interleaved = interleaved != 0;
    p.magnitude = magnitude;
    return launch_rope(p, num_tokens, stream);
}

namespace pkv_internal {

int rope_take_error(int *code) {
    int value = 0;
    if (cudaMemcpyFromSymbol(&value, g_rope_error, sizeof(int)) != cudaSuccess) return PKV_ERR_CUDA;
    if (value != 0) {
        const int zero = 0;
        if (cudaMemcpyToSymbol(g_rope_error, &zero, sizeof(int)) != cudaSuccess) return PKV_ERR_CUDA;
    }
    *code = value;
    return PKV_OK;
}

}  // namespace pkv_internal
