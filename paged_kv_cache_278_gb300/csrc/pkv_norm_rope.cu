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
// stay in registers.  A unit is two 16-byte pieces: pieces u and u + rotary_dim / 16 hold both halves of eight half-layout
// pairs, any piece four interleaved pairs; neighbouring lanes' pieces are neighbours, so that each of a unit's two loads
// and stores is one line for the row's lanes.  The lanes compute a token's angles, one or two sincospi each, and share
// them by shuffles.
//
// A pass is 32 / LANES rows of one kind (q, k or v) of one token; up to kBatch passes of a kind are a batch.  Each warp has an even
// stretch of the call's batches and a ring of kStages batches of shared memory, which bulk copies fill ahead of it: what
// is in flight costs no registers.  Two passes are worked on at a time: with 16 warps on an SM it is the chains of
// dependent instructions that the kernel waits for, more than memory (8192 tokens of 48 rows, three axes: 37 us, 39 one
// pass at a time, 41 with a warp per batch that loads into registers, 47 with a CTA per token; 29.7 at the rate of a
// plain copy).  With few tokens a warp takes one pass straight from global memory: one round of loads on many SMs.
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
constexpr int kNormWarps = kNormThreads / 32;
constexpr int kBatch = 2;    // passes: 8 rows of 128 dims
constexpr int kStages = 3;
constexpr int kBatchBytes = kBatch * 32 * 32;  // a lane's unit is 32 bytes
constexpr int kMaxHeadDim = PKV_MAX_ROPE_HEAD_DIM;
// Up to one pass for each of the warps that 152 SMs hold of the other kernel, a warp takes one pass straight from global
// memory (48 rows a token, in a graph: 64 tokens 2.6 us so and 3.4 from the ring, 150 tokens 2.8 and 3.4, 300 tokens
// 4.0 and 3.9, 600 tokens 5.9 and 4.5).
constexpr int kFewPasses = 152 * 16;
constexpr int kNormCtas = 4;  // per SM

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
    int num_tokens, q_passes, k_passes, passes;  // of a token: passes of q rows, of k rows, of all
    int batches;                                 // of a token
};

// Two float32 in a register pair, and arithmetic on both at once, each lane rounded as the scalar form.
using Pair = uint64_t;
__device__ __forceinline__ Pair pair(float lo, float hi) {
    Pair d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ float2 halves(Pair p) {
    float2 d;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(p));
    return d;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
    Pair d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
    Pair d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ Pair twice(float x) { return pair(x, x); }

__device__ __forceinline__ void unpack(const uint4 &p, Pair (&x)[8], int from) {
    const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = pkv::half2_bits_to_float2(w[i]);
        x[from + i] = pair(f.x, f.y);
    }
}
__device__ __forceinline__ uint4 pack(const Pair (&x)[8], int from) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = halves(x[from + i]);
        const __half2 h = __floats2half2_rn(f.x, f.y);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// E4M3 codes of a row's unit for the row scale s = max|x| / 448, as pkv::quantize_e4m3x2 gives them.  The quotient is the
// IEEE one: with r the reciprocal of s rounded to nearest, x r corrected once by its remainder over s is the
// correctly rounded x / s (P. Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990) where nothing leaves the normal range, and nothing does for quotients of 2^-11 to 448 (smaller
// ones have code 0 either way) with s in [2^-90, 2^100]: other scales are brought there, with x, by a power of two.
// Three packed operations for two quotients, where the division takes some twenty.
struct Quantiser {
    Pair r, minus_s;
    bool zero;

    __device__ __forceinline__ Quantiser(float s, Pair (&x)[8]) : zero(s == 0.f) {
        if (s < 0x1p-90f || s > 0x1p100f) {
            const float k = s < 1.f ? 0x1p100f : 0x1p-60f;
            s *= k;
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = mul2(x[e], twice(k));
        }
        r = twice(__frcp_rn(s));
        minus_s = twice(s == INFINITY ? 0.f : -s);  // (of an infinite scale x r is the quotient: 0, or NaN of an infinity)
    }
    __device__ __forceinline__ uint2 codes(const Pair (&x)[8], int from) const {
        uint32_t c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const Pair q0 = mul2(x[from + i], r);
            const float2 q = halves(fma2(fma2(q0, minus_s, x[from + i]), r, q0));
            uint16_t h;
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(q.y), "f"(q.x));
            c[i] = h;
        }
        return zero ? make_uint2(0u, 0u) : make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
    }
};

__device__ __forceinline__ uint4 lds128_now(uint32_t addr) {  // ordered behind the barrier that published it
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

// One warp's view of a token at a time.  Kinds of rows: 0 q, 1 k, 2 v.
template <int LANES, bool FP8, bool INTERLEAVED>
struct RowWarp {
    static constexpr int kRows = 32 / LANES;                     // rows of one pass
    static constexpr int kShare = kRows >= 8 ? 1 : 8 / kRows;    // of a unit's eight pairs: angles a lane computes
    const NormParams &P;
    int lane, u, g, units, half0, half1;
    bool turns0, turns1;  // whether the unit's pieces are rotated (together, in the half layout)
    int64_t t, slot, next_slot, cache_row;
    // of the angles this lane computes
    int axis[kShare], next_position[kShare];
    uint64_t frequency[kShare];
    Pair co[INTERLEAVED ? 8 : 4], si[INTERLEAVED ? 8 : 4], back[INTERLEAVED ? 1 : 4];  // as rotate takes them

    __device__ __forceinline__ explicit RowWarp(const NormParams &params) : P(params), t(-1), slot(-1), next_slot(-1), cache_row(0) {
        lane = threadIdx.x & 31;
        u = lane % LANES;
        g = lane / LANES;
        units = P.head_dim / 16;
        const int r16 = P.rotary_dim / 16;
        half0 = first_piece(u, units, r16);
        half1 = second_piece(u, units, r16);
        turns0 = INTERLEAVED ? half0 < 2 * r16 : u < r16;
        turns1 = INTERLEAVED ? half1 < 2 * r16 : u < r16;
    }
    // The two pieces of unit `unit` of a q or k row.
    static __device__ __forceinline__ int first_piece(int unit, int units, int r16) { return INTERLEAVED || unit < r16 ? unit : unit + r16; }
    static __device__ __forceinline__ int second_piece(int unit, int units, int r16) { return INTERLEAVED || unit >= r16 ? unit + units : unit + r16; }
    // Angle e of this lane's share of the unit's eight: the pair it turns, or -1.
    __device__ __forceinline__ int pair_of(int e) const {
        const int j = g * kShare + e;
        if (j >= 8 || !(INTERLEAVED && j >= 4 ? turns1 : turns0)) return -1;
        return INTERLEAVED ? 4 * (j < 4 ? half0 : half1) + (j & 3) : 8 * u + j;
    }
    // The axes and frequencies of the angles this lane computes.
    __device__ __forceinline__ void load_axes() {
#pragma unroll
        for (int e = 0; e < kShare; ++e) {
            const int i = pair_of(e);
            if (i < 0) continue;
            axis[e] = P.axes ? __ldg(P.axes + i) : 0;
            if (axis[e] < 0 || axis[e] >= P.num_axes) {
                pkv::record_error(&g_norm_error, PKV_DEV_BAD_AXIS);
                axis[e] = 0;
            }
            frequency[e] = static_cast<uint64_t>(__ldg(P.frequencies + i));
        }
    }
    __device__ __forceinline__ int heads_of(int kind) const { return kind == 0 ? P.num_q_heads : P.num_kv_heads; }
    __device__ __forceinline__ const uint4 *rows_of(int kind, int64_t token) const {
        return kind == 0 ? P.q + token * P.q_stride : (kind == 1 ? P.k + token * P.k_stride : P.v + token * P.v_stride);
    }
    // The lane's two pieces of a row of this kind.
    __device__ __forceinline__ int piece0(int kind) const { return kind == 2 ? u : half0; }
    __device__ __forceinline__ int piece1(int kind) const { return kind == 2 ? u + units : half1; }

    // What begin() needs of a token, on its way.
    __device__ __forceinline__ void fetch(int64_t token) {
#pragma unroll
        for (int e = 0; e < kShare; ++e)
            if (pair_of(e) >= 0) next_position[e] = __ldg(P.positions + token * P.num_axes + axis[e]);
        if (P.v) next_slot = __ldg(P.slot_mapping + token);
    }
    // The fetched token's slot and angles.
    __device__ __forceinline__ void begin(int64_t token) {
        t = token;
        slot = next_slot;
        if (P.v && slot >= P.num_slots) {
            if (lane == 0) pkv::record_error(&g_norm_error, PKV_DEV_BAD_SLOT);
            slot = -1;
        }
        float2 own[kShare];
#pragma unroll
        for (int e = 0; e < kShare; ++e) {
            own[e] = make_float2(0.f, 0.f);
            if (pair_of(e) < 0) continue;
            const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(next_position[e])) * frequency[e] + (1ull << 31);
            const float x = static_cast<float>(static_cast<int32_t>(phase >> 32)) * (1.f / 2147483648.f);
            float s, c;
            sincospif(x, &s, &c);
            own[e] = make_float2(c * P.magnitude, s * P.magnitude);
        }
        float c[8], s[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int from = (j / kShare) * LANES + u;
            c[j] = __shfl_sync(pkv::kFullMask, own[j % kShare].x, from);
            s[j] = __shfl_sync(pkv::kFullMask, own[j % kShare].y, from);
        }
        if constexpr (INTERLEAVED) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                co[j] = twice(c[j]);
                si[j] = pair(-s[j], s[j]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                co[j] = pair(c[2 * j], c[2 * j + 1]);
                si[j] = pair(s[2 * j], s[2 * j + 1]);
                back[j] = pair(-s[2 * j], -s[2 * j + 1]);
            }
        }
        if (P.v && slot >= 0) {
            const int64_t block = slot < 0x7fffffff ? static_cast<int>(slot) / P.block_size : slot / P.block_size;
            cache_row = block * P.num_kv_heads * P.block_size + (slot - block * P.block_size);
        }
    }

    // (a, b) -> (a c - b s, b c + a s) for the unit's pairs.
    __device__ __forceinline__ void rotate(Pair (&x)[8]) const {
        if constexpr (INTERLEAVED) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 f = halves(x[j]);
                const Pair y = fma2(x[j], co[j], mul2(pair(f.y, f.x), si[j]));
                x[j] = (j < 4 ? turns0 : turns1) ? y : x[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const Pair lo = x[j], hi = x[4 + j];
                x[j] = fma2(lo, co[j], mul2(hi, back[j]));
                x[4 + j] = fma2(hi, co[j], mul2(lo, si[j]));
            }
        }
    }

    // Passes of one kind: rows head0 + g, head0 + g + kRows, ... of the token's `count` passes, N at a time for
    // their chains to overlap.  `source` gives a pass's pieces (zeros where a row or the lane's unit is none), `weights`
    // the unit's four float4s as they lie in its pieces.
    template <int KIND, int N, typename Source, typename Weights>
    __device__ __forceinline__ void run(int head0, int count, const Source &source, const Weights &weights) {
        const int heads = heads_of(KIND), pieces = 2 * units;
        const bool normed = KIND == 0 ? P.q_weight != nullptr : (KIND == 1 && P.k_weight != nullptr);
        const bool goes = u < units && (KIND == 0 || !P.v || slot >= 0);
        int head = head0 + g;
        // where the first row goes, and what lies between passes
        int64_t step = static_cast<int64_t>(kRows) * pieces, row = 0;
        uint4 *dst = nullptr;
        if (KIND == 0) {
            dst = P.q_out + t * P.q_out_stride + head * pieces;
        } else if (!P.v) {
            dst = P.k_out + t * P.k_out_stride + head * pieces;
        } else {
            row = cache_row + static_cast<int64_t>(head) * P.block_size;
            step *= P.block_size;
            if (!FP8) dst = P.k_cache + row * pieces;
        }
        uint2 *codes = FP8 && KIND > 0 ? (KIND == 1 ? P.k_codes : P.v_codes) + row * pieces : nullptr;
        float *scale = FP8 && KIND > 0 ? (KIND == 1 ? P.k_scale : P.v_scale) + row : nullptr;
        const int64_t scale_step = static_cast<int64_t>(kRows) * P.block_size;
        const int at0 = piece0(KIND), at1 = piece1(KIND);
#pragma unroll 1
        for (int i = 0; i < count; i += N, head += N * kRows) {
            uint4 raw[N][2];
            bool writes[N];
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const bool there = u < units && head + n * kRows < heads && i + n < count;
                writes[n] = goes && there;
                source(i + n, there, at0, at1, raw[n][0], raw[n][1]);
            }
            Pair x[N][8];
#pragma unroll
            for (int n = 0; n < N; ++n) {
                unpack(raw[n][0], x[n], 0);
                unpack(raw[n][1], x[n], 4);
            }
            if constexpr (KIND < 2) {
                if (normed) {
                    float square[N];
#pragma unroll
                    for (int n = 0; n < N; ++n) {
                        Pair sum = mul2(x[n][0], x[n][0]), sum1 = mul2(x[n][1], x[n][1]);
#pragma unroll
                        for (int e = 2; e < 8; e += 2) {
                            sum = fma2(x[n][e], x[n][e], sum);
                            sum1 = fma2(x[n][e + 1], x[n][e + 1], sum1);
                        }
                        const float2 p = halves(sum), q = halves(sum1);
                        square[n] = (p.x + p.y) + (q.x + q.y);
                    }
#pragma unroll
                    for (int d = LANES / 2; d >= 1; d >>= 1)
#pragma unroll
                        for (int n = 0; n < N; ++n) square[n] += __shfl_xor_sync(pkv::kFullMask, square[n], d);
#pragma unroll
                    for (int n = 0; n < N; ++n) {
                        const Pair r = twice(rsqrtf(fmaf(square[n], P.inv_dim, P.eps)));
#pragma unroll
                        for (int e = 0; e < 8; ++e) x[n][e] = mul2(x[n][e], r);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float4 f = weights(j);
#pragma unroll
                        for (int n = 0; n < N; ++n) {
                            x[n][2 * j] = mul2(x[n][2 * j], pair(f.x, f.y));
                            x[n][2 * j + 1] = mul2(x[n][2 * j + 1], pair(f.z, f.w));
                        }
                    }
                }
                if (turns0) {  // (a second piece is rotated only with the first)
#pragma unroll
                    for (int n = 0; n < N; ++n) rotate(x[n]);
                }
            }
            if constexpr (FP8 && KIND > 0) {
                float most[N];
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    most[n] = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float2 f = halves(x[n][e]);
                        most[n] = fmaxf(most[n], fmaxf(fabsf(f.x), fabsf(f.y)));
                    }
                }
#pragma unroll
                for (int d = LANES / 2; d >= 1; d >>= 1)
#pragma unroll
                    for (int n = 0; n < N; ++n) most[n] = fmaxf(most[n], __shfl_xor_sync(pkv::kFullMask, most[n], d));
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    if (writes[n]) {
                        const float s = __fdiv_rn(most[n], 448.f);
                        const Quantiser quantiser(s, x[n]);
                        codes[at0] = quantiser.codes(x[n], 0);
                        codes[at1] = quantiser.codes(x[n], 4);
                        if (u == 0) *scale = s;
                    }
                    codes += step;
                    scale += scale_step;
                }
            } else {
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    if (writes[n]) {
                        dst[at0] = pack(x[n], 0);
                        dst[at1] = pack(x[n], 4);
                    }
                    dst += step;
                }
            }
        }
    }
    // The same of v into the fp16 cache: its rows as they are.
    template <int N, typename Source>
    __device__ __forceinline__ void copy(int head0, int count, const Source &source) {
        const bool goes = u < units && slot >= 0;
        int head = head0 + g;
        const int64_t step = static_cast<int64_t>(kRows) * P.block_size * (2 * units);
        uint4 *dst = P.v_cache + (cache_row + static_cast<int64_t>(head) * P.block_size) * (2 * units) + u;
#pragma unroll 1
        for (int i = 0; i < count; i += N, head += N * kRows) {
            uint4 raw[N][2];
            bool there[N];
#pragma unroll
            for (int n = 0; n < N; ++n) {
                there[n] = u < units && head + n * kRows < P.num_kv_heads && i + n < count;
                source(i + n, there[n], u, u + units, raw[n][0], raw[n][1]);
            }
#pragma unroll
            for (int n = 0; n < N; ++n) {
                if (goes && there[n]) {
                    dst[0] = raw[n][0];
                    dst[units] = raw[n][1];
                }
                dst += step;
            }
        }
    }
    template <int N, typename Source, typename Weights>
    __device__ __forceinline__ void run_kind(int kind, int head0, int count, const Source &source, const Weights &weights) {
        if (kind == 0)
            run<0, N>(head0, count, source, weights);
        else if (kind == 1)
            run<1, N>(head0, count, source, weights);
        else if constexpr (FP8)
            run<2, N>(head0, count, source, weights);
        else
            copy<N>(head0, count, source);
    }
};

// One pass a warp, straight from global memory.
template <int LANES, bool FP8, bool INTERLEAVED>
__global__ void __launch_bounds__(kNormThreads) norm_rope_few_kernel(const __grid_constant__ NormParams P) {
    pkv::pdl_wait_primary();  // by every thread: the next kernel may rely on it
    pkv::pdl_launch_dependents();
    RowWarp<LANES, FP8, INTERLEAVED> rows(P);
    const int at = blockIdx.x * kNormWarps + threadIdx.x / 32;
    if (at >= P.num_tokens * P.passes) return;
    const int token = at / P.passes, pass = at - token * P.passes;
    const int kind = pass < P.q_passes ? 0 : (pass < P.q_passes + P.k_passes ? 1 : 2);
    const int head0 = (pass - (kind == 0 ? 0 : P.q_passes + (kind == 2 ? P.k_passes : 0))) * rows.kRows;
    uint4 a = make_uint4(0, 0, 0, 0), b = a;
    if (rows.u < rows.units && head0 + rows.g < rows.heads_of(kind)) {
        const uint4 *src = rows.rows_of(kind, token) + (head0 + rows.g) * 2 * rows.units;
        a = src[rows.piece0(kind)];
        b = src[rows.piece1(kind)];
    }
    const float4 *weight = reinterpret_cast<const float4 *>(kind == 0 ? P.q_weight : P.k_weight);
    float4 w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        w[j] = kind < 2 && weight && rows.u < rows.units ? __ldg(weight + 2 * (j < 2 ? rows.half0 : rows.half1) + (j & 1)) : make_float4(1.f, 1.f, 1.f, 1.f);
    rows.load_axes();
    rows.fetch(token);
    rows.begin(token);
    rows.template run_kind<1>(
        kind, head0, 1,
        [&](int, bool, int, int, uint4 &x, uint4 &y) {
            x = a;
            y = b;
        },
        [&](int j) { return w[j]; });
}

template <int LANES, bool FP8, bool INTERLEAVED>
__global__ void __launch_bounds__(kNormThreads, kNormCtas) norm_rope_kernel(const __grid_constant__ NormParams P) {
    __shared__ __align__(128) unsigned char s_ring[kNormWarps][kStages][kBatchBytes];
    __shared__ uint64_t s_full[kNormWarps][kStages];
    __shared__ float4 s_weight[2][4 * LANES];  // float4 j of unit u at j * LANES + u: a row's lanes read neighbouring ones
    const int warp = threadIdx.x / 32;
    const uint32_t ring = pkv::smem_addr(s_ring[warp]), full = pkv::smem_addr(s_full[warp]);
    if (threadIdx.x % 32 == 0) {
        for (int i = 0; i < kStages; ++i) pkv::mbar_init(full + 8 * i, 1);
        pkv::fence_mbar_init();
    }
    __syncwarp();
    pkv::pdl_wait_primary();
    pkv::pdl_launch_dependents();
    RowWarp<LANES, FP8, INTERLEAVED> rows(P);
    const int64_t all = static_cast<int64_t>(P.num_tokens) * P.batches, warps = static_cast<int64_t>(gridDim.x) * kNormWarps;
    const int64_t own = static_cast<int64_t>(blockIdx.x) * kNormWarps + warp;
    const int64_t first = all * own / warps;
    const int count = static_cast<int>(all * (own + 1) / warps - first);
    int64_t load_token = first / P.batches, token = load_token;
    int load_batch = static_cast<int>(first - load_token * P.batches), batch = load_batch, loaded = 0;
    const int q_batches = (P.q_passes + kBatch - 1) / kBatch, k_batches = (P.k_passes + kBatch - 1) / kBatch;
    const int row_bytes = P.head_dim * 2;
    // A token's batch: rows of one kind, from head0 on.
    auto kind_of = [&](int n) { return n < q_batches ? 0 : (n < q_batches + k_batches ? 1 : 2); };
    auto head0_of = [&](int n, int kind) { return (n - (kind == 0 ? 0 : q_batches + (kind == 2 ? k_batches : 0))) * (kBatch * rows.kRows); };
    // Fills stage loaded % kStages.
    auto load = [&]() {
        if (rows.lane == 0) {
            const int kind = kind_of(load_batch), head0 = head0_of(load_batch, kind);
            const uint32_t bar = full + 8 * (loaded % kStages);
            const uint32_t bytes = min(rows.heads_of(kind) - head0, kBatch * rows.kRows) * row_bytes;
            pkv::mbar_arrive_expect_tx(bar, bytes);
            pkv::bulk_copy_g2s(ring + (loaded % kStages) * kBatchBytes, rows.rows_of(kind, load_token) + head0 * 2 * rows.units, bytes, bar);
        }
        ++loaded;
        if (++load_batch == P.batches) {
            load_batch = 0;
            ++load_token;
        }
    };
    for (int i = 0; i < kStages && i < count; ++i) load();
    if (count > 0) {
        rows.load_axes();
        rows.fetch(token);
    }
    for (int i = threadIdx.x; i < 8 * LANES; i += kNormThreads) {
        const int kind = i / (4 * LANES), j = i / LANES % 4, unit = i % LANES;
        const float4 *w = reinterpret_cast<const float4 *>(kind == 0 ? P.q_weight : P.k_weight);
        const int piece = j < 2 ? rows.first_piece(unit, rows.units, P.rotary_dim / 16) : rows.second_piece(unit, rows.units, P.rotary_dim / 16);
        if (w && unit < rows.units) s_weight[kind][j * LANES + unit] = __ldg(w + 2 * piece + (j & 1));
    }
    __syncthreads();
    for (int n = 0; n < count; ++n) {
        if (token != rows.t) {
            rows.begin(token);
            if (token + 1 < P.num_tokens) rows.fetch(token + 1);
        }
        const int stage = n % kStages;
        if (!__all_sync(pkv::kFullMask, pkv::mbar_wait_bounded(full + 8 * stage, (n / kStages) & 1))) {
            if (rows.lane == 0) pkv::record_error(&g_norm_error, PKV_DEV_WAIT_TIMEOUT);
            for (int i = n + 1; i < loaded; ++i)  // copies in flight land before the CTA's memory goes (bounded)
                pkv::mbar_wait_bounded(full + 8 * (i % kStages), (i / kStages) & 1);
            return;
        }
        const int kind = kind_of(batch), head0 = head0_of(batch, kind);
        const int passes = min(kBatch, (rows.heads_of(kind) - head0 + rows.kRows - 1) / rows.kRows);
        rows.template run_kind<2>(
            kind, head0, passes,
            [&](int i, bool there, int at0, int at1, uint4 &x, uint4 &y) {
                const uint32_t at = ring + stage * kBatchBytes + (i * rows.kRows + rows.g) * row_bytes;
                x = there ? lds128_now(at + 16 * at0) : make_uint4(0, 0, 0, 0);
                y = there ? lds128_now(at + 16 * at1) : make_uint4(0, 0, 0, 0);
            },
            [&](int j) { return s_weight[kind & 1][j * LANES + rows.u]; });
        __syncwarp();  // every lane has read the stage
        if (loaded < count) {
            pkv::fence_proxy_async_smem();
            load();
        }
        if (++batch == P.batches) {
            batch = 0;
            ++token;
        }
    }
}

// Strides arrive in elements.  A row of heads must not run into the next token's.
bool stride_ok(int64_t stride, int heads, int head_dim, int num_tokens) {
    if (stride % 8 != 0) return false;
    return num_tokens <= 1 || stride >= static_cast<int64_t>(heads) * head_dim;
}

using NormKernel = void (*)(NormParams);
template <int LANES, bool FP8>
NormKernel kernel_of(bool few, bool interleaved) {
    if (few) return interleaved ? norm_rope_few_kernel<LANES, FP8, true> : norm_rope_few_kernel<LANES, FP8, false>;
    return interleaved ? norm_rope_kernel<LANES, FP8, true> : norm_rope_kernel<LANES, FP8, false>;
}

template <bool FP8>
int launch_norm_rope(NormParams p, int num_tokens, pkv_stream_t stream) {
    const int units = p.head_dim / 16;
    const int lanes = units <= 1 ? 1 : (units <= 2 ? 2 : (units <= 4 ? 4 : (units <= 8 ? 8 : 16)));
    const int rows = 32 / lanes;
    p.num_tokens = num_tokens;
    p.q_passes = (p.num_q_heads + rows - 1) / rows;
    p.k_passes = (p.num_kv_heads + rows - 1) / rows;
    p.passes = p.q_passes + (p.v ? 2 : 1) * p.k_passes;
    p.batches = (p.q_passes + kBatch - 1) / kBatch + (p.v ? 2 : 1) * ((p.k_passes + kBatch - 1) / kBatch);
    p.inv_dim = 1.f / static_cast<float>(p.head_dim);
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return PKV_ERR_CUDA;
    const int64_t passes = static_cast<int64_t>(num_tokens) * p.passes;
    const bool few = passes <= kFewPasses;
    const int64_t warps = few ? passes : static_cast<int64_t>(num_tokens) * p.batches;
    int64_t ctas = (warps + kNormWarps - 1) / kNormWarps;
    if (!few && ctas > static_cast<int64_t>(sms) * kNormCtas) ctas = static_cast<int64_t>(sms) * kNormCtas;
    const bool i = p.interleaved != 0;
    const NormKernel kernel = FP8          ? kernel_of<8, FP8>(few, i)
                              : lanes == 1 ? kernel_of<1, false>(few, i)
                              : lanes == 2 ? kernel_of<2, false>(few, i)
                              : lanes == 4 ? kernel_of<4, false>(few, i)
                              : lanes == 8 ? kernel_of<8, false>(few, i)
                                           : kernel_of<16, false>(few, i);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
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
