// pkv_weights.cu -- decode attention that also accumulates, per cached position, the attention it received.
//
//     out[b][hq]       = sum_t p[hq][t] V[t],   p[hq][t] = exp(scale q[hq] . K[t] - lse[hq])
//     scores[b][h][t] += sum over the group's q heads of p[hq][t]
//
// The weights need the log-sum-exp of the whole row, which is known only after every key has been
// seen.  Reading K again would add half of the step's HBM traffic; instead the attention pass leaves
// its scaled dot products (float32, log2 units, [request][kv head][token][group]) in the workspace, 4 G bytes
// per token against the 512 bytes of its K and V rows, and a second launch turns them into weights.
// At 64 requests x 2049 tokens, 8 kv heads, G = 4 they are 17 MB, which stay in the 129 MB L2.
//
//   * attention pass: one CTA per (request, kv head, 1024-token partition), four warps each with a private
//     ring of 16-token chunks (tensor copies, 128-byte swizzle), the tensor-core engine of the
//     decode kernels with one 8-byte store per lane and token pair added; contexts past one partition
//     leave a partial output each.  Bound by HBM, as the decode kernels are: 90 us for the 538 MB of 64 x 2049 tokens alone on
//     cold caches, what the plain decode kernel takes there; with the weights pass 97 us, 84 % of the copy bandwidth
//     (32768, 24577, 16385 and 8193 tokens 62 us, 82 %).
//   * weights pass: one CTA per (request, kv head, 1024 tokens): the partitions' (m, l) give the
//     group's log-sum-exps, then one exponential per (token, head) and one read-modify-write of
//     scores per token, by exactly one thread: no atomics, a fixed order.  Its CTAs of a (request, kv head) join the
//     partial outputs too, each a share of the dims: no counter has to survive from one call to the next, so any calls
//     may take turns on one workspace, whatever it held.  Bound by latency (10-12 us alone): its
//     loads are issued together, those of scores while the attention pass still runs.  The join
//     by the last partition to arrive, with a counter, took as long or longer: 97.1 us against 96.9 (64 x 2049) and 63.4
//     against 61.8 (the four contexts).
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "pkv.h"
#include "pkv_device.cuh"
#include "pkv_internal.h"

#include "pkv_engine.cuh"

namespace {

__device__ int g_weights_error;

constexpr int kPart = PKV_DEFAULT_PARTITION;
constexpr int kWeightThreads = 256;

struct WeightParams {
    DecodeParams d;  // its maps and split buffers
    float *raw;      // [B][Hkv][cap][G] scaled dot products, log2 units
    float *scores;   // [B][Hkv][capacity]
    int64_t capacity;
};

// The decode engine, leaving each chunk's scaled scores in `raw` on the way to the softmax.
template <int G>
struct TcEngineScored : TcEngine<G> {
    float *raw;  // this (request, kv head)'s [cap][G]

    __device__ __forceinline__ void qk_scored(uint32_t k_tile, int valid, int lane, unsigned char *scratch, int tok0) {
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        this->dots(s, k_tile, lane);
        const int g = lane >> 2, h0 = (lane & 3) * 2;
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] *= this->q_scale;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            if (g + 8 * r < valid && h0 < G) {
                float *at = raw + static_cast<int64_t>(tok0 + g + 8 * r) * G + h0;
                if constexpr (G == 1)
                    *at = s[2 * r];
                else
                    *reinterpret_cast<float2 *>(at) = make_float2(s[2 * r], s[2 * r + 1]);
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] = g + 8 * (e >> 1) < valid ? s[e] : -INFINITY;
        this->softmax(s, lane, scratch);
    }
};

// The request's context within its table (a longer one is recorded and cut).
__device__ __forceinline__ int context_of(const DecodeParams &P, int b, bool report) {
    const int cap = P.max_blocks_per_seq * P.block_size;
    int ctx = __ldg(P.context_lens + b);
    if (ctx > cap) {
        if (report) pkv::record_error(&g_weights_error, PKV_DEV_BAD_CONTEXT);
        ctx = cap;
    }
    return max(ctx, 0);
}

template <int G>
__global__ void __launch_bounds__(kThreads, PKV_DECODE_MIN_CTAS)
    scored_partition_kernel(const __grid_constant__ WeightParams W) {
    const DecodeParams &P = W.d;
    using L = SmemLayout<true>;
    extern __shared__ __align__(1024) unsigned char smem[];
    pkv::pdl_wait_primary();
    pkv::pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z;
    const int bs = P.block_size;
    const int ctx = context_of(P, b, part == 0 && kvh == 0 && threadIdx.x == 0);
    const int64_t head_row = static_cast<int64_t>(b) * P.num_q_heads + kvh * G;
    if (ctx == 0) {  // no cached position: zero output, nothing to accumulate
        if (part == 0)
            for (int i = threadIdx.x; i < G * kD; i += kThreads) P.out[head_row * kD + i] = __float2half_rn(0.f);
        return;
    }
    const int n_parts = (ctx + kPart - 1) / kPart;
    if (part >= n_parts) return;
    const int start = part * kPart;
    const int n_tok = min(kPart, ctx - start);
    const int n_chunks = (n_tok + kChunk - 1) / kChunk;
    const int lb0 = start / bs, n_bt = (start + n_tok - 1) / bs - lb0 + 1;

    int32_t *s_table = reinterpret_cast<int32_t *>(smem + L::table(G));
    unsigned char *scratch = smem + L::probs + warp * L::probs_per_warp(G);
    const uint32_t bar0 = pkv::smem_addr(smem + L::bars) + warp * kStages * kBarsPerStage * 8;
    const uint32_t stage0 = pkv::smem_addr(smem + L::stages) + warp * kStages * L::stage;
    // The 128-byte swizzle needs 1 KB-aligned tiles; a CTA without them stages no tokens.
    const bool smem_ok = (pkv::smem_addr(smem) & 1023) == 0;
    if (!smem_ok && threadIdx.x == 0) pkv::record_error(&g_weights_error, PKV_DEV_SMEM_MISALIGNED);
    if (lane == 0) {
#pragma unroll
        for (int s = 0; s < kStages; ++s) pkv::mbar_init(bar0 + 8 * s, 1);
        pkv::fence_mbar_init();
    }
    for (int i = threadIdx.x; i < n_bt; i += kThreads) {
        int32_t id = __ldg(P.block_tables + static_cast<int64_t>(b) * P.max_blocks_per_seq + lb0 + i);
        if (id < 0 || id >= P.num_blocks) {
            pkv::record_error(&g_weights_error, PKV_DEV_BAD_BLOCK_ID);
            id = 0;
        }
        s_table[i] = id;
    }
    TcEngineScored<G> eng;
    eng.init(P, b, kvh, lane);
    const int64_t cap = static_cast<int64_t>(P.max_blocks_per_seq) * bs;
    eng.raw = W.raw + (static_cast<int64_t>(b) * P.num_kv_heads + kvh) * cap * G;
    __syncthreads();

    const int my_chunks = smem_ok && n_chunks > warp ? (n_chunks - warp + kWarps - 1) / kWarps : 0;
    auto issue = [&](int i) {  // whole 16-row boxes: a ragged tail's extra rows stay inside the block
        if (lane != 0) return;
        const int tok0 = start + (warp + i * kWarps) * kChunk;
        const int lb = tok0 / bs;
        const int y = static_cast<int>((static_cast<int64_t>(s_table[lb - lb0]) * P.num_kv_heads + kvh) * bs + tok0 - lb * bs);
        const int st = i % kStages;
        const uint32_t dst = stage0 + st * L::stage, bar = bar0 + 8 * st;
        pkv::mbar_arrive_expect_tx(bar, 4 * kHalfTile);
        pkv::tma_load_2d(dst, &W.d.tmap_k, 0, y, bar);
        pkv::tma_load_2d(dst + kHalfTile, &W.d.tmap_k, 64, y, bar);
        pkv::tma_load_2d(dst + L::k_tile, &W.d.tmap_v, 0, y, bar);
        pkv::tma_load_2d(dst + L::k_tile + kHalfTile, &W.d.tmap_v, 64, y, bar);
    };
    int issued = 0, consumed = 0;
    for (; issued < min(my_chunks, kStages); ++issued) issue(issued);
    for (int i = 0; i < my_chunks; ++i) {
        const int st = i % kStages;
        if (!__all_sync(pkv::kFullMask, pkv::mbar_wait_bounded(bar0 + 8 * st, (i / kStages) & 1))) {
            if (lane == 0) pkv::record_error(&g_weights_error, PKV_DEV_WAIT_TIMEOUT);
            break;
        }
        consumed = i + 1;
        const int cidx = warp + i * kWarps;
        const int valid = min(kChunk, n_tok - cidx * kChunk);
        const uint32_t k_tile = stage0 + st * L::stage, v_tile = k_tile + L::k_tile;
        if (valid < kChunk) {  // the MMA reads all 16 V rows: those past the context may hold anything
            for (int x = lane; x < (kChunk - valid) * 16; x += 32)
                asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(v_tile + TcEngine<G>::swz(valid + x / 16, x % 16)),
                             "r"(0)
                             : "memory");
            __syncwarp();
        }
        eng.qk_scored(k_tile, valid, lane, scratch, start + cidx * kChunk);
        eng.pv(v_tile, valid, lane, scratch);
        __syncwarp();
        if (i + kStages < my_chunks) {
            pkv::fence_proxy_async_smem();
            issue(i + kStages);
            ++issued;
        }
    }
    // after a wait that ran out: the copies still in flight land before the buffers are reused (bounded)
    for (int i = consumed; i < issued; ++i) pkv::mbar_wait_bounded(bar0 + 8 * (i % kStages), (i / kStages) & 1);

    // ---- the four warps' states, merged in the stage buffers
    __syncthreads();
    float *c_acc = reinterpret_cast<float *>(smem);
    float *c_m = c_acc + kWarps * G * kAccStride;
    float *c_l = c_m + kWarps * G;
    float *c_f = c_l + kWarps * G;
    float *c_row = c_f + kWarps * G;
    static_assert((kWarps * G * (kAccStride + 3) + 2 * G) * 4 <= L::stage_bytes, "combine area must fit the stages");
    eng.finish(warp, lane, c_acc, c_m, c_l);
    __syncthreads();
    if (threadIdx.x < G) {
        const int hh = threadIdx.x;
        float M = -INFINITY, S = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, c_m[w * G + hh]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = exp2f(c_m[w * G + hh] - M);
            c_f[w * G + hh] = f;
            S = fmaf(c_l[w * G + hh], f, S);
        }
        c_row[hh] = M;
        c_row[G + hh] = S;
    }
    __syncthreads();
    const bool direct = n_parts == 1;
    for (int idx = threadIdx.x; idx < G * (kD / 4); idx += kThreads) {
        const int hh = idx / (kD / 4), dim = 4 * (idx % (kD / 4));
        float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float4 a = *reinterpret_cast<const float4 *>(c_acc + (w * G + hh) * kAccStride + dim);
            const float f = c_f[w * G + hh];
            o[0] = fmaf(a.x, f, o[0]);
            o[1] = fmaf(a.y, f, o[1]);
            o[2] = fmaf(a.z, f, o[2]);
            o[3] = fmaf(a.w, f, o[3]);
        }
        const float S = c_row[G + hh];
        const int64_t row = head_row + hh, prow = row * P.max_partitions + part;
        if (direct) {
            const __half2 lo = __floats2half2_rn(o[0] / S, o[1] / S), hi = __floats2half2_rn(o[2] / S, o[3] / S);
            *reinterpret_cast<uint2 *>(P.out + row * kD + dim) =
                make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
        } else {
            *reinterpret_cast<float4 *>(P.o_part + prow * kD + dim) = make_float4(o[0] / S, o[1] / S, o[2] / S, o[3] / S);
        }
        if (dim == 0) {
            P.m_part[prow] = c_row[hh] * kLn2;
            P.l_part[prow] = S;
        }
    }
}

template <int G>
__global__ void __launch_bounds__(kWeightThreads) accumulate_weights_kernel(const __grid_constant__ WeightParams W) {
    const DecodeParams &P = W.d;
    __shared__ float s_lse[G], s_top[G], s_inv[G];
    __shared__ float4 s_join[kWeightThreads];
    const int part = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z;
    const int ctx = context_of(P, b, false);
    const int start = part * kPart;
    const int end = min(ctx, start + kPart);
    const int64_t cap = static_cast<int64_t>(P.max_blocks_per_seq) * P.block_size;
    const int64_t head = static_cast<int64_t>(b) * P.num_kv_heads + kvh;
    const float *raw = W.raw + head * cap * G;
    float *scores = W.scores + head * W.capacity;
    // What scores holds: like context_lens it is not written by the attention pass, whose CTAs have all started,
    // behind their own wait for what came before; so it is read while the last of them run.
    constexpr int kPerThread = kPart / kWeightThreads;
    float before[kPerThread];
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const int t = start + i * kWeightThreads + static_cast<int>(threadIdx.x);
        before[i] = t < end ? __ldcg(scores + t) : 0.f;
    }
    pkv::pdl_wait_primary();
    pkv::pdl_launch_dependents();
    if (start >= ctx) return;
    const int n_parts = (ctx + kPart - 1) / kPart;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float s[kPerThread][G];
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const int t = min(start + i * kWeightThreads + static_cast<int>(threadIdx.x), end - 1);
        const float *at = raw + static_cast<int64_t>(t) * G;
        if constexpr (G >= 4) {
#pragma unroll
            for (int k = 0; k < G / 4; ++k) {
                const float4 v = __ldcg(reinterpret_cast<const float4 *>(at) + k);
                s[i][4 * k] = v.x;
                s[i][4 * k + 1] = v.y;
                s[i][4 * k + 2] = v.z;
                s[i][4 * k + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int k = 0; k < G; ++k) s[i][k] = __ldcg(at + k);
        }
    }
    // The partial outputs: this CTA joins `share` of the group's G x 32 pieces of four dims, n_parts threads (or as many
    // as there are, in turn) to a piece.
    const int share = (G * (kD / 4) + n_parts - 1) / n_parts, joiners = min(kWeightThreads / share, n_parts);
    const int joiner = static_cast<int>(threadIdx.x) / share, piece = part * share + static_cast<int>(threadIdx.x) % share;
    const int head_of = piece / (kD / 4);
    const int64_t head_row = static_cast<int64_t>(b) * P.num_q_heads + kvh * G;
    const int64_t part_row = (head_row + head_of) * P.max_partitions;
    const bool joins = n_parts > 1 && joiner < joiners && piece < G * (kD / 4);
    auto partial = [&](int p, float &m, float &l) {
        m = __ldcg(P.m_part + part_row + p);
        l = __ldcg(P.l_part + part_row + p);
        return __ldcg(reinterpret_cast<const float4 *>(P.o_part + (part_row + p) * kD) + piece % (kD / 4));
    };
    float m0 = 0.f, l0 = 0.f;
    float4 o0 = make_float4(0.f, 0.f, 0.f, 0.f);
    if (joins) o0 = partial(joiner, m0, l0);
    if (warp < G) {  // one warp per head: its log-sum-exp in log2 units from the partitions' (m, l)
        const int64_t row = (static_cast<int64_t>(b) * P.num_q_heads + kvh * G + warp) * P.max_partitions;
        float M = -INFINITY, S = 0.f;
        for (int p = lane; p < n_parts; p += 32) M = fmaxf(M, __ldcg(P.m_part + row + p));
#pragma unroll
        for (int sh = 16; sh >= 1; sh >>= 1) M = fmaxf(M, __shfl_xor_sync(pkv::kFullMask, M, sh));
        for (int p = lane; p < n_parts; p += 32) S += __ldcg(P.l_part + row + p) * expf(__ldcg(P.m_part + row + p) - M);
#pragma unroll
        for (int sh = 16; sh >= 1; sh >>= 1) S += __shfl_xor_sync(pkv::kFullMask, S, sh);
        if (lane == 0) {
            s_lse[warp] = fmaf(M, kLog2e, log2f(S));
            s_top[warp] = M;
            s_inv[warp] = 1.f / S;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const int t = start + i * kWeightThreads + static_cast<int>(threadIdx.x);
        float w = 0.f;
#pragma unroll
        for (int k = 0; k < G; ++k) w += pkv::exp2_approx(s[i][k] - s_lse[k]);
        if (t < end) scores[t] = before[i] + w;
    }
    if (n_parts == 1) return;  // the attention pass wrote the output
    if (joins) {
        const float top = s_top[head_of];
        float w = l0 * expf(m0 - top);
        float4 o = make_float4(w * o0.x, w * o0.y, w * o0.z, w * o0.w);
        for (int p = joiner + joiners; p < n_parts; p += joiners) {
            const float4 x = partial(p, m0, l0);
            w = l0 * expf(m0 - top);
            o.x = fmaf(w, x.x, o.x);
            o.y = fmaf(w, x.y, o.y);
            o.z = fmaf(w, x.z, o.z);
            o.w = fmaf(w, x.w, o.w);
        }
        s_join[threadIdx.x] = o;
    }
    __syncthreads();
    if (joins && joiner == 0) {
        float4 o = s_join[threadIdx.x];
        for (int j = 1; j < joiners; ++j) {
            const float4 x = s_join[j * share + threadIdx.x];
            o.x += x.x;
            o.y += x.y;
            o.z += x.z;
            o.w += x.w;
        }
        const float inv = s_inv[head_of];
        const __half2 lo = __floats2half2_rn(o.x * inv, o.y * inv), hi = __floats2half2_rn(o.z * inv, o.w * inv);
        *reinterpret_cast<uint2 *>(P.out + (head_row + head_of) * kD + 4 * (piece % (kD / 4))) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
    }
}

using pkv_internal::align256;

// Workspace: o_part | m_part | l_part | raw, each 256-byte aligned.  Every call writes what it reads.
struct WeightsLayout {
    size_t m, l, raw, total;
    int parts;
};
WeightsLayout weights_layout(int num_seqs, int num_q_heads, int64_t cap) {
    WeightsLayout w{};
    w.parts = static_cast<int>((cap + kPart - 1) / kPart);
    const size_t rows = static_cast<size_t>(num_seqs) * num_q_heads * w.parts;
    w.m = w.parts > 1 ? align256(rows * kD * sizeof(float)) : 0;
    w.l = w.m + align256(rows * sizeof(float));
    w.raw = w.l + align256(rows * sizeof(float));
    w.total = w.raw + align256(static_cast<size_t>(num_seqs) * num_q_heads * cap * sizeof(float));
    return w;
}

template <int G>
int launch_weights(const WeightParams &w, int num_seqs, cudaStream_t stream) {
    using L = SmemLayout<true>;
    auto kernel = scored_partition_kernel<G>;
    const int smem = L::total(G, kPart);
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return PKV_ERR_CUDA;
    static std::atomic<uint64_t> configured{0};  // one bit per device
    const uint64_t bit = 1ull << (dev & 63);
    if (!(configured.load(std::memory_order_acquire) & bit)) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
            return PKV_ERR_CUDA;
        configured.fetch_or(bit, std::memory_order_acq_rel);
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(w.d.max_partitions, w.d.num_kv_heads, num_seqs);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, w) != cudaSuccess) return PKV_ERR_CUDA;
    cfg.blockDim = dim3(kWeightThreads);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, accumulate_weights_kernel<G>, w) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace

extern "C" PKV_API size_t pkv_weights_workspace_size(int num_seqs, int num_q_heads, int head_dim, int max_context) {
    if (num_seqs <= 0 || num_q_heads <= 0 || head_dim != kD || max_context <= 0) return 0;
    return weights_layout(num_seqs, num_q_heads, max_context).total;
}

extern "C" PKV_API int pkv_decode_attention_weights(void *out, float *scores, int64_t score_capacity, const void *q,
                                                    const void *k_cache, const void *v_cache,
                                                    const int32_t *block_tables, const int32_t *context_lens,
                                                    int num_seqs, int max_blocks_per_seq, int num_q_heads,
                                                    int num_kv_heads, int head_dim, int block_size,
                                                    int64_t num_blocks, float scale, void *workspace,
                                                    size_t workspace_bytes, pkv_stream_t stream) {
    const int st = pkv_internal::check_decode_args(q, k_cache, v_cache, block_tables, context_lens, num_seqs,
                                                   max_blocks_per_seq, num_q_heads, num_kv_heads, head_dim, block_size,
                                                   num_blocks);
    if (st != PKV_OK) return st;
    const int64_t cap = static_cast<int64_t>(max_blocks_per_seq) * block_size;
    if (!out || !scores || !pkv_internal::aligned(out, 8) || !pkv_internal::aligned(scores, 4) || score_capacity < cap)
        return PKV_ERR_INVALID_ARG;
    if (num_seqs == 0) return PKV_OK;
    const int64_t rows = num_blocks * num_kv_heads * block_size;
    if (rows >= 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;  // box row coordinates are signed 32-bit
    const WeightsLayout lay = weights_layout(num_seqs, num_q_heads, cap);
    if (!workspace || workspace_bytes < lay.total || !pkv_internal::aligned(workspace, 256)) return PKV_ERR_WORKSPACE;
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    WeightParams w{};
    DecodeParams &p = w.d;
    p.q = static_cast<const __half *>(q);
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.out = static_cast<__half *>(out);
    p.o_part = reinterpret_cast<float *>(ws);
    p.m_part = reinterpret_cast<float *>(ws + lay.m);
    p.l_part = reinterpret_cast<float *>(ws + lay.l);
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.block_size = block_size;
    p.num_blocks = num_blocks;
    p.q_scale = scale * kLog2e;
    p.partition_size = kPart;
    p.max_partitions = lay.parts;
    w.raw = reinterpret_cast<float *>(ws + lay.raw);
    w.scores = scores;
    w.capacity = score_capacity;
    int e = pkv_internal::encode_fp16_cache_map(&p.tmap_k, k_cache, rows);
    if (e == PKV_OK) e = pkv_internal::encode_fp16_cache_map(&p.tmap_v, v_cache, rows);
    if (e != PKV_OK) return e;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    switch (num_q_heads / num_kv_heads) {
        case 1: return launch_weights<1>(w, num_seqs, s);
        case 2: return launch_weights<2>(w, num_seqs, s);
        case 4: return launch_weights<4>(w, num_seqs, s);
        case 8: return launch_weights<8>(w, num_seqs, s);
        default: return PKV_ERR_UNSUPPORTED;
    }
}

namespace pkv_internal {

int weights_take_error(int *code) {
    int value = 0;
    if (cudaMemcpyFromSymbol(&value, g_weights_error, sizeof(int)) != cudaSuccess) return PKV_ERR_CUDA;
    if (value != 0) {
        const int zero = 0;
        if (cudaMemcpyToSymbol(g_weights_error, &zero, sizeof(int)) != cudaSuccess) return PKV_ERR_CUDA;
    }
    *code = value;
    return PKV_OK;
}

}  // namespace pkv_internal
