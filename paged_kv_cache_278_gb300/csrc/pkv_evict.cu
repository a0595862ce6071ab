// pkv_evict.cu -- eviction of the least attended cached positions.
//
// For every (request b, kv head h) with more than `budget` cached positions n = context_lens[b], kept are
// the first `sinks`, the last `recent` and, of the positions between them, those with the largest
// accumulated attention weight scores[b][h][.] (ties: the lower position; a NaN counts as the smallest
// value).  The kept rows of K, V and scores move, in position order, to positions 0, 1, ... of the
// request's new block table, which may name the same blocks: kept position p_i >= i, so a row only ever
// moves towards the front.
//
// Two launches:
//   * select: one CTA per (b, h).  The border value is found by bisection on the order-preserving
//     integer image of the float bits, 32 counts of "how many keys are >= x" over keys held in
//     registers; no atomics, so the result does not depend on any order.  The kept set is then a
//     bitmap over the positions (above the border, the lowest ties, sinks, recent); prefix popcounts
//     of its words give every kept position its place.
//   * move: bound by HBM (each kept row is read once and written once).  In a block that both tables
//     name, a row's place may be the source of a row placed earlier, so rows move in order: a cluster
//     of CTAs takes a (request, kv head)'s K, or V, step by step, all its CTAs load their rows of the
//     step, meet, and store them (later sources lie behind every place of the step).  Tables with no
//     block in common need no meeting.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "pkv.h"
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace {

__device__ int g_evict_error;

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kListKeys = 2;        // undecided keys per thread once they are listed
constexpr int kMoveThreads = 256;
constexpr int kRowLanes = PKV_HEAD_DIM * 2 / 16;  // threads that move one row, 16 bytes each
constexpr int kMoveBatch = 4;                     // rows in flight per thread
constexpr int kMoveRows = kMoveThreads / kRowLanes * kMoveBatch;  // rows of a CTA's step

struct EvictParams {
    unsigned char *k_cache, *v_cache;
    int32_t *kept;      // [B][Hkv][budget]
    float *new_scores;  // [B][Hkv][capacity]
    int32_t *new_lens;
    const float *scores;
    const int32_t *block_tables, *new_tables, *context_lens;
    int64_t capacity, num_blocks;
    int max_blocks, max_new_blocks, num_kv_heads, block_size, row_bytes;
    int budget, recent, sinks;
    int cluster;  // CTAs that move one (request, kv head)'s K, or V, together
};

// Larger float <-> larger integer; NaN smallest, so that it is evicted first.
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t u = __float_as_uint(x);
    const uint32_t k = u == 0x80000000u ? 0u : u;  // -0 ties with +0
    const uint32_t o = k ^ (static_cast<uint32_t>(static_cast<int32_t>(k) >> 31) | 0x80000000u);
    return (u & 0x7fffffffu) > 0x7f800000u ? 0u : o;
}

// The request's cached positions, within its table.
__device__ __forceinline__ int cached(const EvictParams &P, int b, bool report) {
    const int cap = P.max_blocks * P.block_size;
    int n = __ldcg(P.context_lens + b);  // may alias new_lens: not through the read-only path
    if (n > cap) {
        if (report) pkv::record_error(&g_evict_error, PKV_DEV_BAD_CONTEXT);
        n = cap;
    }
    return max(n, 0);
}

// Sum over the CTA; every thread gets it.  `s` holds kSelWarps + 1 ints, alternated by the caller
// between two arrays so that one barrier per sum is enough.
__device__ __forceinline__ int block_sum(int v, int *s) {
    v = __reduce_add_sync(pkv::kFullMask, v);
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    return __reduce_add_sync(pkv::kFullMask, s[threadIdx.x & 31]);
}

// Exclusive prefix sum over the CTA's threads and the total.
__device__ __forceinline__ int block_scan(int v, int *s, int &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(pkv::kFullMask, x, d);
        if (lane >= d) x += y;
    }
    __syncthreads();
    if (lane == 31) s[warp] = x;
    __syncthreads();
    int w = s[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(pkv::kFullMask, w, d);
        if (lane >= d) w += y;
    }
    total = __shfl_sync(pkv::kFullMask, w, 31);
    const int before = __shfl_sync(pkv::kFullMask, w, (warp + 31) & 31);
    return x - v + (warp ? before : 0);
}

// KPT keys per thread live in registers (positions j * kSelThreads + thread); positions past
// KPT * kSelThreads are read again for each count.
template <int KPT>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const __grid_constant__ EvictParams P) {
    extern __shared__ uint32_t s_words[];  // [words] above the border, then kept | [words] at the border, then prefixes
    __shared__ int s_sum[2][kSelWarps];
    __shared__ uint32_t s_list[kListKeys * kSelThreads];
    __shared__ int s_listed;
    pkv::pdl_wait_primary();
    pkv::pdl_launch_dependents();
    const int h = blockIdx.x, b = blockIdx.y;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = static_cast<int64_t>(b) * P.num_kv_heads + h;
    const float *scores = P.scores + row * P.capacity;
    float *out = P.new_scores + row * P.capacity;
    int32_t *kept = P.kept + row * P.budget;
    const int n = cached(P, b, tid == 0 && h == 0);
    const int m = min(n, P.budget);

    if (n > P.budget) {
        const int first = min(P.sinks, n), last = n - P.recent;  // candidates [first, last)
        const int need = P.budget - P.sinks - P.recent;
        uint32_t key[KPT];
#pragma unroll
        for (int j = 0; j < KPT; ++j) key[j] = __float_as_uint(__ldcg(scores + min(j * kSelThreads + tid, n - 1)));  // all in flight
#pragma unroll
        for (int j = 0; j < KPT; ++j) {
            const int p = j * kSelThreads + tid;
            const uint32_t k = order_key(__uint_as_float(key[j]));
            key[j] = p >= first && p < last ? k : 0u;
        }
        // The largest border with at least `need` candidate keys >= it (keys of 0 outside the
        // candidates are never counted: every tested border is above 0).
        uint32_t border = 0;
        int flip = 0;
        if (need > 0) {
            int upper = 0, inside = last - first;  // keys above the undecided range, and in it
            int above_list = 0;                    // keys above the listed ones
            uint32_t mine[kListKeys] = {};
            bool listed = false;
            for (int bit = 31; bit >= 0; --bit) {
                const uint32_t trial = border | (1u << bit);
                int c = 0;
                if (!listed) {
#pragma unroll
                    for (int j = 0; j < KPT; ++j) c += key[j] >= trial;
                    for (int p = KPT * kSelThreads + tid; p < last; p += kSelThreads)
                        c += p >= first && order_key(__ldcg(scores + p)) >= trial;
                    c = block_sum(c, s_sum[flip]);
                } else {
#pragma unroll
                    for (int j = 0; j < kListKeys; ++j) c += mine[j] >= trial;
                    c = above_list + block_sum(c, s_sum[flip]);
                }
                flip ^= 1;
                if (c == need) {  // exactly the keys from `trial` on: none at the border itself
                    border = trial - 1;
                    break;
                }
                if (c > need) {
                    border = trial;
                    inside = c - upper;
                } else {
                    inside -= c - upper;
                    upper = c;
                }
                if (!listed && bit > 0 && inside <= kListKeys * kSelThreads) {
                    // The few undecided keys, in any order, spread over the threads: from here on a
                    // count costs a barrier, not a pass over the row.
                    if (tid == 0) s_listed = 0;
                    __syncthreads();
                    auto push = [&](uint32_t x, bool cand) {
                        const bool in = cand && x >= border && (x - border) < (1u << bit);
                        const uint32_t mask = __ballot_sync(pkv::kFullMask, in);
                        int at = 0;
                        if (lane == 0 && mask) at = atomicAdd(&s_listed, __popc(mask));
                        at = __shfl_sync(pkv::kFullMask, at, 0) + __popc(mask & ((1u << lane) - 1u));
                        if (in) s_list[at] = x;
                    };
#pragma unroll
                    for (int j = 0; j < KPT; ++j) {
                        const int p = j * kSelThreads + tid;
                        push(key[j], p >= first && p < last);
                    }
                    for (int p0 = KPT * kSelThreads; p0 < last; p0 += kSelThreads) {
                        const int p = p0 + tid;
                        const bool cand = p >= first && p < last;
                        push(cand ? order_key(__ldcg(scores + p)) : 0u, cand);
                    }
                    __syncthreads();
#pragma unroll
                    for (int j = 0; j < kListKeys; ++j) mine[j] = j * kSelThreads + tid < s_listed ? s_list[j * kSelThreads + tid] : 0u;
                    listed = true;
                    above_list = upper;
                }
            }
        } else {
            border = 0xffffffffu;  // above every key: nothing between the sinks and the recent ones
        }
        // Bitmaps of the positions above and at the border.
        const int words = (n + 31) / 32;
        uint32_t *s_above = s_words, *s_at = s_words + words;
        const int64_t rounds = (n + kSelThreads - 1) / kSelThreads;
        auto mark = [&](int j, uint32_t k) {
            const int p = j * kSelThreads + tid;
            const bool cand = p >= first && p < last, fixed = p < n && !cand;
            const uint32_t above = __ballot_sync(pkv::kFullMask, fixed || (cand && k > border));
            const uint32_t at = __ballot_sync(pkv::kFullMask, cand && need > 0 && k == border);
            const int w = j * kSelWarps + warp;
            if (lane == 0 && w < words) {
                s_above[w] = above;
                s_at[w] = at;
            }
        };
#pragma unroll
        for (int j = 0; j < KPT; ++j)
            if (j < rounds) mark(j, key[j]);
        for (int j = KPT; j < rounds; ++j) {
            const int p = j * kSelThreads + tid;
            mark(j, p < n ? order_key(__ldcg(scores + p)) : 0u);
        }
        __syncthreads();
        // Ties left to take, from the lowest position on: thread t owns `per` neighbouring words.
        const int per = (words + kSelThreads - 1) / kSelThreads;
        const int w0 = tid * per, w1 = min(words, w0 + per);
        int above = 0, at = 0;
        for (int w = w0; w < w1; ++w) {
            above += __popc(s_above[w]);
            at += __popc(s_at[w]);
        }
        int total_above = 0, total_at = 0;
        block_scan(above, s_sum[0], total_above);
        int before = block_scan(at, s_sum[1], total_at);
        int room = m - total_above - before;  // ties that may still be taken at this thread's first word
        int mine = 0;
        for (int w = w0; w < w1; ++w) {
            uint32_t ties = s_at[w];
            const int c = __popc(ties);
            if (c > room) {  // keep the lowest `room` set bits
                uint32_t keep = 0;
                for (int i = 0; i < room; ++i) {
                    const uint32_t low = ties & (0u - ties);
                    keep |= low;
                    ties ^= low;
                }
                ties = keep;
            }
            room -= c;
            s_above[w] |= ties;
            mine += __popc(s_above[w]);
        }
        int total = 0;
        int place = block_scan(mine, s_sum[0], total);
        for (int w = w0; w < w1; ++w) {
            s_at[w] = place;
            place += __popc(s_above[w]);
        }
        __syncthreads();
        // Places and scores, kRounds x kSelThreads positions at a time.  new_scores may be scores itself:
        // places lie at or before their positions, so all of a step's scores are read before any of its
        // places is written, and the next step reads behind every place written so far.
        constexpr int kRounds = 8;
        for (int64_t j0 = 0; j0 < rounds; j0 += kRounds) {
            float x[kRounds];
#pragma unroll
            for (int u = 0; u < kRounds; ++u) {
                const int w = static_cast<int>((j0 + u) * kSelWarps + warp);
                x[u] = __ldcg(scores + min(w * 32 + lane, n - 1));
            }
            if (out == scores) __syncthreads();
#pragma unroll
            for (int u = 0; u < kRounds; ++u) {
                const int w = static_cast<int>((j0 + u) * kSelWarps + warp);
                const uint32_t bits = w < words ? s_above[w] : 0u;
                if ((bits >> lane) & 1u) {
                    const int i = static_cast<int>(s_at[w]) + __popc(bits & ((1u << lane) - 1u));
                    kept[i] = w * 32 + lane;
                    out[i] = x[u];
                }
            }
        }
    } else {
        for (int p = tid; p < n; p += kSelThreads) {
            kept[p] = p;
            if (out != scores) out[p] = __ldcg(scores + p);
        }
        for (int p = n + tid; p < P.budget; p += kSelThreads) kept[p] = -1;
    }
    __syncthreads();
    for (int64_t p = m + tid; p < P.capacity; p += kSelThreads) out[p] = 0.f;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

__global__ void __launch_bounds__(kMoveThreads) move_kernel(const __grid_constant__ EvictParams P) {
    __shared__ unsigned char *s_src[2][kMoveRows], *s_dst[2][kMoveRows];
    pkv::pdl_wait_primary();
    pkv::pdl_launch_dependents();
    const int tid = threadIdx.x;
    const int rank = blockIdx.x % P.cluster, h = blockIdx.y, b = blockIdx.z;
    unsigned char *cache = static_cast<int>(blockIdx.x) < P.cluster ? P.k_cache : P.v_cache;
    const int n = cached(P, b, false);
    int m = min(n, P.budget);
    if (m > P.max_new_blocks * P.block_size) {
        if (tid == 0 && blockIdx.x == 0 && h == 0) pkv::record_error(&g_evict_error, PKV_DEV_BAD_CONTEXT);
        m = P.max_new_blocks * P.block_size;
    }
    const int32_t *kept = P.kept + (static_cast<int64_t>(b) * P.num_kv_heads + h) * P.budget;
    const int32_t *from = P.block_tables + static_cast<int64_t>(b) * P.max_blocks;
    const int32_t *to = P.new_tables + static_cast<int64_t>(b) * P.max_new_blocks;
    // Rows can only be in one another's way in blocks that both tables name (at the same index).
    bool shared = from == to;
    if (!shared) {
        const int blocks = min((m + P.block_size - 1) / P.block_size, P.max_blocks);
        bool same = false;
        for (int i = tid; i < blocks; i += kMoveThreads) same = same || __ldg(from + i) == __ldg(to + i);
        shared = __syncthreads_or(same);
    }
    auto address = [&](const int32_t *table, int p) -> unsigned char * {
        const int blk = p / P.block_size;
        const int32_t id = __ldg(table + blk);
        if (id < 0 || id >= P.num_blocks) {
            pkv::record_error(&g_evict_error, PKV_DEV_BAD_BLOCK_ID);
            return nullptr;
        }
        const int64_t r = (static_cast<int64_t>(id) * P.num_kv_heads + h) * P.block_size + (p - blk * P.block_size);
        return cache + r * P.row_bytes;
    };
    const int stride = P.cluster * kMoveRows;  // rows of the cluster's step
    const int steps = (m + stride - 1) / stride;
    auto locate = [&](int step) {  // one thread per row: where it is and where it goes (null: nowhere)
        if (tid >= kMoveRows) return;
        const int i = step * stride + rank * kMoveRows + tid;
        unsigned char *s = nullptr, *d = nullptr;
        if (i < m) {
            s = address(from, __ldg(kept + i));
            d = address(to, i);
            if (s == nullptr || s == d) d = nullptr;  // a bad block, or the row is where it belongs
        }
        s_src[step & 1][tid] = s;
        s_dst[step & 1][tid] = d;
    };
    const int row = tid / kRowLanes, byte = tid % kRowLanes * 16;
    locate(0);
    __syncthreads();
    for (int step = 0; step < steps; ++step) {
        uint4 x[kMoveBatch];
        unsigned char *dst[kMoveBatch];
#pragma unroll
        for (int u = 0; u < kMoveBatch; ++u) {
            const int i = u * (kMoveThreads / kRowLanes) + row;
            dst[u] = s_dst[step & 1][i];
            if (dst[u] != nullptr) x[u] = __ldcg(reinterpret_cast<const uint4 *>(s_src[step & 1][i] + byte));
        }
        if (step + 1 < steps) locate(step + 1);
        if (shared) {  // every row of the cluster's step has been read before any is written
            cluster_arrive();
            cluster_wait();
        }
#pragma unroll
        for (int u = 0; u < kMoveBatch; ++u)
            if (dst[u] != nullptr) *reinterpret_cast<uint4 *>(dst[u] + byte) = x[u];
        __syncthreads();  // the next step's rows are located
    }
    // new_lens may be context_lens: the other CTAs' min(n, budget) is the same from either value
    if (tid == 0 && blockIdx.x == 0 && h == 0) P.new_lens[b] = min(n, P.budget);
}

template <int KPT>
int launch_select(const EvictParams &p, int num_seqs, size_t smem, cudaStream_t stream, cudaLaunchAttribute *attr) {
    auto kernel = select_kernel<KPT>;
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
        return PKV_ERR_CUDA;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(p.num_kv_heads, num_seqs);
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace

extern "C" PKV_API int pkv_evict(void *k_cache, void *v_cache, int32_t *kept, float *new_scores, int32_t *new_lens,
                                 const float *scores, const int32_t *block_tables, const int32_t *new_tables,
                                 const int32_t *context_lens, int num_seqs, int max_blocks_per_seq,
                                 int max_new_blocks, int64_t score_capacity, int num_kv_heads, int head_dim,
                                 int block_size, int64_t num_blocks, int budget, int recent, int sinks,
                                 pkv_stream_t stream) {
    if (num_seqs < 0 || max_blocks_per_seq <= 0 || max_new_blocks <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
        block_size <= 0 || num_blocks <= 0 || budget <= 0 || recent < 0 || sinks < 0)
        return PKV_ERR_INVALID_ARG;
    if (recent > budget || sinks > budget - recent) return PKV_ERR_INVALID_ARG;
    if (head_dim != PKV_HEAD_DIM) return PKV_ERR_UNSUPPORTED;
    const int64_t cap = static_cast<int64_t>(max_blocks_per_seq) * block_size;
    if (cap > PKV_MAX_EVICT_CONTEXT || static_cast<int64_t>(max_new_blocks) * block_size > 0x7fffffffLL)
        return PKV_ERR_UNSUPPORTED;
    if (score_capacity < cap || num_blocks > 0x7fffffffLL) return PKV_ERR_INVALID_ARG;
    if (num_seqs > 65535 || num_kv_heads > 65535) return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PKV_OK;
    if (!k_cache || !v_cache || !kept || !new_scores || !new_lens || !scores || !block_tables || !new_tables || !context_lens)
        return PKV_ERR_INVALID_ARG;
    if (!pkv_internal::aligned16(k_cache) || !pkv_internal::aligned16(v_cache) || !pkv_internal::aligned(kept, 4) ||
        !pkv_internal::aligned(new_scores, 4) || !pkv_internal::aligned(new_lens, 4) || !pkv_internal::aligned(scores, 4) ||
        !pkv_internal::aligned(block_tables, 4) || !pkv_internal::aligned(new_tables, 4) ||
        !pkv_internal::aligned(context_lens, 4))
        return PKV_ERR_INVALID_ARG;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return PKV_ERR_CUDA;
    EvictParams p{};
    p.k_cache = static_cast<unsigned char *>(k_cache);
    p.v_cache = static_cast<unsigned char *>(v_cache);
    p.kept = kept;
    p.new_scores = new_scores;
    p.new_lens = new_lens;
    p.scores = scores;
    p.block_tables = block_tables;
    p.new_tables = new_tables;
    p.context_lens = context_lens;
    p.capacity = score_capacity;
    p.num_blocks = num_blocks;
    p.max_blocks = max_blocks_per_seq;
    p.max_new_blocks = max_new_blocks;
    p.num_kv_heads = num_kv_heads;
    p.block_size = block_size;
    p.row_bytes = head_dim * 2;
    p.budget = budget;
    p.recent = recent;
    p.sinks = sinks;
    // CTAs per cluster: doubled, to at most eight, while the grid has fewer than three CTAs per SM and
    // the kept rows fill a step of the larger cluster.
    p.cluster = 1;
    while (p.cluster < 8 && static_cast<int64_t>(num_seqs) * num_kv_heads * 2 * p.cluster < 3 * sms &&
           budget >= 2 * p.cluster * kMoveRows)
        p.cluster *= 2;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const size_t smem = (static_cast<size_t>(cap) + 31) / 32 * 8;
    const int64_t kpt = (cap + kSelThreads - 1) / kSelThreads;
    const int st = kpt <= 4    ? launch_select<4>(p, num_seqs, smem, s, &attr)
                   : kpt <= 16 ? launch_select<16>(p, num_seqs, smem, s, &attr)
                               : launch_select<32>(p, num_seqs, smem, s, &attr);
    if (st != PKV_OK) return st;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(2 * p.cluster, num_kv_heads, num_seqs);
    cfg.blockDim = dim3(kMoveThreads);
    cfg.stream = s;
    cudaLaunchAttribute attrs[2] = {attr, {}};
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = p.cluster;
    attrs[1].val.clusterDim.y = 1;
    attrs[1].val.clusterDim.z = 1;
    cfg.attrs = attrs;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, move_kernel, p) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

namespace pkv_internal {

int evict_take_error(int *code) {
    int value = 0;
    if (cudaMemcpyFromSymbol(&value, g_evict_error, sizeof(int)) != cudaSuccess) return PKV_ERR_CUDA;
    if (value != 0) {
        const int zero = 0;
        if (cudaMemcpyToSymbol(g_evict_error, &zero, sizeof(int)) != cudaSuccess) return PKV_ERR_CUDA;
    }
    *code = value;
    return PKV_OK;
}

}  // namespace pkv_internal
