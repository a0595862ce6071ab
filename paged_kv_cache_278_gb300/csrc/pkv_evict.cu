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
//   * select: one cluster of CTAs per (b, h), its scores in registers.  The border value is the need-th largest
//     of the order-preserving integer images of the candidates, found by four histograms (9, 8, 8, 7
//     bits) that the CTAs add up through distributed shared memory; counts do not depend on the
//     order of the atomics that made them.  The kept set is then a bitmap over the positions (above the
//     border, the lowest ties, sinks, recent); prefix popcounts of its words give every kept position
//     its place.  Bound by latency, four meetings of the cluster in a row: 20 us alone, of 42 in all, for 32 rows of
//     16385 to 32768 scores, 14 of 41 for 128 rows of 1951 to 3900.
//   * move: bound by HBM (each kept row is read once and written once): 134 MB in 23 us into new blocks, 29 us where
//     the clusters meet at every step.  In a block that both tables
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

constexpr int kSelThreads = 512;
constexpr int kBins = 512, kPasses = 4;  // digits of 9, 8, 8 and 7 bits
constexpr int kMoveThreads = 256;
constexpr int kRowLanes = PKV_HEAD_DIM * 2 / 16;  // threads that move one row, 16 bytes each
constexpr int kMoveBatch = 4;                     // rows in flight per thread (2 and 8 measured 15 and 13 % slower on 4 x 32768 -> 4096; the
                                                  // next step's rows read ahead too take 72 registers, and 16 x 3900 -> 1024 in place 50 us, not 41)
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
    int select_cluster;  // CTAs that select of one (request, kv head) together
    int cluster;         // CTAs that move one's K, or V, together
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

// Of the kept positions, those that the new table has room for.
__device__ __forceinline__ int moved(const EvictParams &P, int kept) { return min(kept, P.max_new_blocks * P.block_size); }

// Exclusive prefix sum over the CTA's threads, and the total.
template <int W>
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
    int w = lane < W ? s[lane] : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(pkv::kFullMask, w, d);
        if (lane >= d) w += y;
    }
    total = __shfl_sync(pkv::kFullMask, w, 31);
    const int before = __shfl_sync(pkv::kFullMask, w, (warp + 31) & 31);
    return x - v + (warp ? before : 0);
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// The same shared-memory address in the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t of_rank(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ int load_remote(uint32_t addr) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ int4 load_remote4(uint32_t addr) {
    int4 v;
    asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

// One cluster per (b, h), each CTA with a run of kSelThreads KPT positions: thread's are (j kSelThreads + thread) 4 + e
// of its CTA's run, e < 4, j < KPT / 4, in registers.
template <int KPT>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const __grid_constant__ EvictParams P) {
    constexpr int T = kSelThreads, W = T / 32, J = KPT / 4, kRun = T * KPT, kWords = kRun / 32;
    static_assert(kBins == T, "a thread adds up one bin");
    __shared__ __align__(16) int s_hist[kPasses][kBins];
    __shared__ uint32_t s_above[kWords], s_at[kWords];  // bitmaps: above the border, then kept; at the border, then places
    __shared__ __align__(16) int s_total[kBins];  // the cluster's histogram of a pass, from the highest bin to the lowest
    __shared__ int s_sum[2][W];
    __shared__ __align__(16) int4 s_count;  // this CTA's positions above and at the border
    __shared__ int s_bin, s_upper, s_inside;
    const int tid = threadIdx.x, lane = tid & 31;
    for (int i = tid; i < kPasses * kBins; i += T) (&s_hist[0][0])[i] = 0;
    __syncthreads();
    pkv::pdl_wait_primary();
    pkv::pdl_launch_dependents();
    const int ranks = P.select_cluster, rank = blockIdx.x % ranks;
    const int h = blockIdx.x / ranks, b = blockIdx.y;
    const int64_t row = static_cast<int64_t>(b) * P.num_kv_heads + h;
    const float *scores = P.scores + row * P.capacity;
    float *out = P.new_scores + row * P.capacity;
    int32_t *kept = P.kept + row * P.budget;
    const int n = cached(P, b, tid == 0 && blockIdx.x == 0);
    const int m = min(n, P.budget), room_for = moved(P, m);
    const int run = rank * kRun;      // the CTA's first position

    if (n > P.budget) {  // (the whole cluster)
        const int first = min(P.sinks, n), last = n - P.recent;  // candidates [first, last)
        const int need = P.budget - P.sinks - P.recent;
        float raw[KPT];
#pragma unroll
        for (int j = 0; j < J; ++j) {  // all in flight (clamped: what lies past n is never looked at); 16-byte loads measured the same
            const int p = run + (j * T + tid) * 4;
#pragma unroll
            for (int e = 0; e < 4; ++e) raw[4 * j + e] = __ldcg(scores + min(p + e, n - 1));
        }
        auto position = [&](int i) { return run + ((i / 4) * T + tid) * 4 + i % 4; };
        auto candidate = [&](int p) { return p >= first && p < last; };
        uint32_t border = 0xffffffffu;  // above every key: nothing between the sinks and the recent ones
        if (need > 0) {
            // Digit by digit: the bin of the need-th largest key among those that share the digits so far, from the
            // cluster's histograms.  Every CTA finds the same.
            border = 0;
            int left = need;  // of the keys that share the digits so far, this many are above or at the border
#pragma unroll 1
            for (int pass = 0; pass < kPasses; ++pass) {
                constexpr int kShift[kPasses] = {23, 15, 7, 0};
                const int shift = pass == 0 ? kShift[0] : pass == 1 ? kShift[1] : pass == 2 ? kShift[2] : kShift[3];
                const uint32_t digit = pass == 0 ? 0x1ffu : pass == 3 ? 0x7fu : 0xffu;
                const uint32_t known = pass == 0 ? 0u : 0xffffffffu << (shift + (pass == 3 ? 7 : 8));
#pragma unroll
                for (int i = 0; i < KPT; ++i) {
                    const uint32_t k = order_key(raw[i]);
                    if (candidate(position(i)) && ((k ^ border) & known) == 0) atomicAdd(&s_hist[pass][(k >> shift) & digit], 1);
                }
                cluster_arrive();
                cluster_wait();
                const uint32_t mine = pkv::smem_addr(&s_hist[pass][kBins - 1 - tid]);
                int c = 0;
                for (int r = 0; r < ranks; ++r) c += load_remote(of_rank(mine, r));
                s_total[tid] = c;
                __syncthreads();
                if (tid < 32) {  // one warp finds the bin: each lane sixteen neighbouring ones
                    int own[kBins / 32], sum = 0;
#pragma unroll
                    for (int i = 0; i < kBins / 32; i += 4) {
                        const int4 v = *reinterpret_cast<const int4 *>(s_total + lane * (kBins / 32) + i);
                        own[i] = v.x;
                        own[i + 1] = v.y;
                        own[i + 2] = v.z;
                        own[i + 3] = v.w;
                        sum += v.x + v.y + v.z + v.w;
                    }
                    int upper = sum;
#pragma unroll
                    for (int d = 1; d < 32; d <<= 1) {
                        const int y = __shfl_up_sync(pkv::kFullMask, upper, d);
                        if (lane >= d) upper += y;
                    }
                    upper -= sum;
                    if (upper < left && left <= upper + sum) {  // one lane
                        bool found = false;
#pragma unroll
                        for (int i = 0; i < kBins / 32; ++i) {
                            if (!found && left <= upper + own[i]) {
                                found = true;
                                s_bin = kBins - 1 - (lane * (kBins / 32) + i);
                                s_upper = upper;
                                s_inside = own[i];
                            }
                            upper += own[i];
                        }
                    }
                }
                __syncthreads();
                border |= static_cast<uint32_t>(s_bin) << shift;
                left -= s_upper;
                if (left == s_inside && border > 0) {  // the whole bin is taken: every key from its lower end on
                    border -= 1;
                    break;
                }
            }
        }
        // Bitmaps of the positions above and at the border.
        int above = 0, at = 0;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            uint32_t x = 0, y = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int p = position(4 * j + e);
                const uint32_t k = order_key(raw[4 * j + e]);
                const bool c = candidate(p);
                x |= static_cast<uint32_t>(p < n && (!c || k > border)) << e;
                y |= static_cast<uint32_t>(c && need > 0 && k == border) << e;
            }
            x <<= 4 * (lane & 7);
            y <<= 4 * (lane & 7);
#pragma unroll
            for (int d = 1; d < 8; d <<= 1) {  // eight lanes make a word
                x |= __shfl_xor_sync(pkv::kFullMask, x, d);
                y |= __shfl_xor_sync(pkv::kFullMask, y, d);
            }
            if ((lane & 7) == 0) {
                s_above[(j * T + tid) / 8] = x;
                s_at[(j * T + tid) / 8] = y;
            }
        }
        __syncthreads();
        // Thread t owns `kPer` neighbouring words.
        constexpr int kPer = (kWords + T - 1) / T;
        const int w0 = min(kWords, tid * kPer), w1 = min(kWords, w0 + kPer);
        for (int w = w0; w < w1; ++w) {
            above += __popc(s_above[w]);
            at += __popc(s_at[w]);
        }
        int total_above = 0, total_at = 0;
        const int above_before = block_scan<W>(above, s_sum[0], total_above), at_before = block_scan<W>(at, s_sum[1], total_at);
        if (tid == 0) s_count = make_int4(total_above, total_at, 0, 0);
        cluster_arrive();
        cluster_wait();
        // Ties are taken from the lowest position on: `room` of the cluster's, of which `lower` lie in earlier runs.
        int room = m, place = 0, lower = 0;
        for (int r = 0; r < ranks; ++r) {
            const int4 c = load_remote4(of_rank(pkv::smem_addr(&s_count), r));
            room -= c.x;
            if (r < rank) {
                place += c.x;
                lower += c.y;
            }
        }
        // (ties taken so far: in earlier runs, then before this thread's words)
        place += min(lower, room) + above_before + max(min(lower + at_before, room) - min(lower, room), 0);
        room -= lower + at_before;
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
            s_at[w] = place;
            place += __popc(s_above[w]);
        }
        __syncthreads();
        // Every kept position and score to its place.  (new_scores may be scores itself: every CTA has read all of its
        // scores by the cluster's last meeting.)
#pragma unroll
        for (int i = 0; i < KPT; ++i) {
            const int p = position(i), w = (p - run) / 32;
            const uint32_t bits = s_above[w];
            if ((bits >> (p & 31)) & 1u) {
                const int to = static_cast<int>(s_at[w]) + __popc(bits & ((1u << (p & 31)) - 1u));
                if (to < room_for) {
                    kept[to] = p;
                    out[to] = raw[i];
                }
            }
        }
    } else {
        for (int p = rank * T + tid; p < room_for; p += ranks * T) {
            kept[p] = p;
            if (out != scores) out[p] = __ldcg(scores + p);
        }
    }
    for (int64_t p = static_cast<int64_t>(room_for) + rank * T + tid; p < P.budget; p += ranks * T) kept[p] = -1;
    // Zeros behind the kept scores (read by every CTA, see above), shared out between the CTAs.
    for (int64_t p = static_cast<int64_t>(room_for) + rank * T + tid; p < P.capacity; p += ranks * T) out[p] = 0.f;
    cluster_arrive();  // no CTA's shared memory goes while another may read it
    cluster_wait();
}

__global__ void __launch_bounds__(kMoveThreads) move_kernel(const __grid_constant__ EvictParams P) {
    __shared__ unsigned char *s_src[2][kMoveRows], *s_dst[2][kMoveRows];
    pkv::pdl_wait_primary();
    pkv::pdl_launch_dependents();
    const int tid = threadIdx.x;
    const int rank = blockIdx.x % P.cluster, h = blockIdx.y, b = blockIdx.z;
    unsigned char *cache = static_cast<int>(blockIdx.x) < P.cluster ? P.k_cache : P.v_cache;
    const int n = cached(P, b, false);
    const int m = moved(P, min(n, P.budget));
    if (m < min(n, P.budget) && tid == 0 && blockIdx.x == 0 && h == 0) pkv::record_error(&g_evict_error, PKV_DEV_BAD_CONTEXT);
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
    // new_lens may be context_lens: the other CTAs' m is the same from either value
    if (tid == 0 && blockIdx.x == 0 && h == 0) P.new_lens[b] = m;
}

template <int KPT>
int launch_select(const EvictParams &p, int num_seqs, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(p.num_kv_heads * p.select_cluster, num_seqs);
    cfg.blockDim = dim3(kSelThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attrs[2] = {};
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = p.select_cluster;
    attrs[1].val.clusterDim.y = 1;
    attrs[1].val.clusterDim.z = 1;
    cfg.attrs = attrs;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, select_kernel<KPT>, p) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
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
    // the kept rows fill a step of the larger cluster.  (Whole call alone between flushes, 8 kv heads, all requests equally
    // long, uniform scores, into new blocks, one CTA against this rule: 4 x 32768 -> 4096 148 and 48 us, in place 215 and
    // 56; always eight against it: 64 x 2048 -> 512 76 and 72.)
    p.cluster = 1;
    while (p.cluster < 8 && static_cast<int64_t>(num_seqs) * num_kv_heads * 2 * p.cluster < 3 * sms &&
           budget >= 2 * p.cluster * kMoveRows)
        p.cluster *= 2;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // Eight CTAs to a row as long as a thread has four scores left; more than 32 a thread only past 131072.  (Timed
    // like the clusters above, one CTA against this rule: 4 x 32768 -> 4096 66 and 48 us, 1 x 32768 -> 8192 67 and 46,
    // 8 x 8192 -> 2048 43 and 41, 16 x 3900 -> 1024 41 both.)
    const int64_t runs = (cap + kSelThreads - 1) / kSelThreads;  // scores per thread of a single CTA
    p.select_cluster = runs <= 4 ? 1 : (runs <= 8 ? 2 : (runs <= 16 ? 4 : 8));
    const int64_t each = (runs + p.select_cluster - 1) / p.select_cluster;
    const int st = each <= 4    ? launch_select<4>(p, num_seqs, s)
                   : each <= 8  ? launch_select<8>(p, num_seqs, s)
                   : each <= 16 ? launch_select<16>(p, num_seqs, s)
                   : each <= 32 ? launch_select<32>(p, num_seqs, s)
                                : launch_select<64>(p, num_seqs, s);
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
