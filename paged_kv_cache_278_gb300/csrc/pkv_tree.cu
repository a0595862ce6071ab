// pkv_tree.cu -- a tree of drafted tokens around its attention: the ancestor masks and depths that go with its
// parents, and the accepted path moved together in the cache.  (The attention itself is in pkv_prompt.cu.)
//
// A request's n_b drafted tokens lie behind its context in any order that puts a node behind its parent, node i
// at position base + i (base = context_lens[b] - n_b).  A node's mask has the bit of every node it attends to.
//
// Both kernels are bound by latency.  keep_path moves a few rows per request: all of a kept row's K and V pieces
// are columns of 16 bytes, a column belongs to one thread, and the thread goes up the path with eight rows in
// flight.  Path entries ascend, so path[j] >= j: a row is read before anything is written over it.  What comes before
// the rows, the sizes, the path and its blocks, is three loads in a row, each of them all at once (with every thread
// looking up its own rows: 256 paths of 1-12 nodes 9.7 us).
#include <cuda_runtime.h>
#include <stdint.h>

#include "pkv.h"
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace {

__device__ int g_tree_error;

constexpr int kMaskThreads = 128;
constexpr int kKeepThreads = 256;
constexpr int kKeepAhead = 8;   // rows in flight per column
constexpr int kKeepRun = 128;   // path entries located at a time
constexpr int kKeepCluster = 8;  // CTAs of one request at most (portable cluster size)
constexpr int kPieces = PKV_HEAD_DIM / 8;

// One CTA per request, one thread per node: up the parents to a root.  Parents come before their children, so
// the walk ends after at most `node` steps.
__global__ void __launch_bounds__(kMaskThreads)
    tree_masks_kernel(uint32_t *mask, int32_t *depths, const int32_t *__restrict__ parents, const int32_t *__restrict__ query_start,
                      int total_q, int max_query_len, int words) {
    const int start = __ldg(query_start + blockIdx.x), n = __ldg(query_start + blockIdx.x + 1) - start;
    if (n < 0 || n > max_query_len || start < 0 || start > total_q - n) {
        if (threadIdx.x == 0) pkv::record_error(&g_tree_error, PKV_DEV_BAD_CONTEXT);
        return;
    }
    for (int i = threadIdx.x; i < n; i += kMaskThreads) {
        uint32_t *row = mask + static_cast<int64_t>(start + i) * words;
        for (int w = 0; w < words; ++w) row[w] = 0;
        int depth = -1;
        for (int at = i; at >= 0;) {
            row[at >> 5] |= 1u << (at & 31);
            ++depth;
            const int up = __ldg(parents + start + at);
            if (up >= at) {  // not a node before it: taken for a root
                pkv::record_error(&g_tree_error, PKV_DEV_BAD_PATH);
                break;
            }
            at = up;
        }
        if (depths) depths[start + i] = depth;
    }
}

struct KeepParams {
    uint4 *cache[2];  // K, V
    int32_t *new_lens;
    const int32_t *block_tables, *context_lens, *query_start, *path, *path_lens;
    int max_blocks, max_path, num_kv_heads, block_size;
    int64_t num_blocks;
};

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait;" ::: "memory"); }

// One cluster of gridDim.x CTAs per request (blockIdx.y).  A path goes through in runs of kKeepRun entries: a thread
// each finds the entries' rows, all at once, then every thread moves its columns.
__global__ void __launch_bounds__(kKeepThreads) keep_path_kernel(const __grid_constant__ KeepParams P) {
    __shared__ int64_t s_from[kKeepRun], s_to[kKeepRun];  // cache rows of kv head 0; s_from -1: nothing to move
    pkv::pdl_wait_primary();
    pkv::pdl_launch_dependents();
    const int64_t b = blockIdx.y;
    const bool teller = blockIdx.x == 0 && threadIdx.x == 0;
    const int32_t *path = P.path + b * P.max_path;
    // the first run's entries are on their way with the request's sizes
    int at = 0, before = -1;
    if (threadIdx.x < min(P.max_path, kKeepRun)) {
        at = __ldg(path + threadIdx.x);
        if (threadIdx.x > 0) before = __ldg(path + threadIdx.x - 1);
    }
    const int ctx = __ldcg(P.context_lens + b), n = __ldg(P.query_start + b + 1) - __ldg(P.query_start + b);
    const int len = __ldg(P.path_lens + b);
    const int64_t room = static_cast<int64_t>(P.max_blocks) * P.block_size;
    int error = PKV_DEV_OK;
    if (n < 0 || ctx < n || ctx > room)
        error = PKV_DEV_BAD_CONTEXT;
    else if (len < 0 || len > P.max_path || len > n)
        error = PKV_DEV_BAD_PATH;
    const int base = ctx - n;
    // the whole path is checked before anything moves
    int bad = 0;
    if (error == PKV_DEV_OK) {
        if (threadIdx.x < min(len, kKeepRun)) bad = at <= before || at >= n;
        for (int i = kKeepRun + threadIdx.x; i < len; i += kKeepThreads) {
            const int x = __ldg(path + i);
            bad |= x <= __ldg(path + i - 1) || x >= n;
        }
    }
    if (__syncthreads_or(bad)) error = PKV_DEV_BAD_PATH;
    if (error != PKV_DEV_OK && teller) pkv::record_error(&g_tree_error, error);
    cluster_arrive();  // this CTA has read context_lens[b], which new_lens may be
    if (error == PKV_DEV_OK) {
        const int32_t *table = P.block_tables + b * P.max_blocks;
        // Row of kv head 0 at a position, or -1 for a bad block.
        auto row_of = [&](int position) -> int64_t {
            const int block = position / P.block_size;
            const int32_t id = __ldg(table + block);
            if (id < 0 || id >= P.num_blocks) {
                pkv::record_error(&g_tree_error, PKV_DEV_BAD_BLOCK_ID);
                return -1;
            }
            return static_cast<int64_t>(id) * P.num_kv_heads * P.block_size + (position - block * P.block_size);
        };
        const int columns = 2 * P.num_kv_heads * kPieces;
        for (int run = 0; run < len; run += kKeepRun) {
            const int count = min(len - run, kKeepRun);
            if (run > 0) {
                __syncthreads();
                if (threadIdx.x < count) at = __ldg(path + run + threadIdx.x);
            }
            if (threadIdx.x < count) {
                const int i = run + threadIdx.x;
                int64_t from = -1, to = -1;
                if (at != i) {  // (else it is there already)
                    from = row_of(base + at);
                    to = row_of(base + i);
                }
                s_from[threadIdx.x] = to < 0 ? -1 : from;
                s_to[threadIdx.x] = to;
            }
            __syncthreads();
            for (int c = blockIdx.x * kKeepThreads + threadIdx.x; c < columns; c += gridDim.x * kKeepThreads) {
                const int head = c / kPieces % P.num_kv_heads, piece = c % kPieces;
                uint4 *const cache = P.cache[c >= columns / 2] + static_cast<int64_t>(head) * P.block_size * kPieces + piece;
                for (int i0 = 0; i0 < count; i0 += kKeepAhead) {
                    uint4 x[kKeepAhead];
#pragma unroll
                    for (int i = 0; i < kKeepAhead; ++i)
                        if (i0 + i < count && s_from[i0 + i] >= 0) x[i] = cache[s_from[i0 + i] * kPieces];
#pragma unroll
                    for (int i = 0; i < kKeepAhead; ++i)
                        if (i0 + i < count && s_from[i0 + i] >= 0) cache[s_to[i0 + i] * kPieces] = x[i];
                }
            }
        }
    }
    cluster_wait();
    if (teller && P.new_lens) P.new_lens[b] = error == PKV_DEV_OK ? base + len : ctx;
}

}  // namespace

extern "C" PKV_API int pkv_tree_masks(int32_t *mask, int32_t *depths, const int32_t *parents, const int32_t *query_start,
                                      int num_seqs, int total_q, int max_query_len, int mask_words, pkv_stream_t stream) {
    if (num_seqs < 0 || total_q < 0 || max_query_len < 0 || mask_words < 0) return PKV_ERR_INVALID_ARG;
    if (max_query_len > PKV_MAX_QUERY_LEN) return PKV_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(mask_words) * 32 < max_query_len) return PKV_ERR_INVALID_ARG;
    if (num_seqs == 0 || total_q == 0 || max_query_len == 0) return PKV_OK;
    if (!mask || !parents || !query_start || !pkv_internal::aligned(mask, 4) || !pkv_internal::aligned(depths, 4) ||
        !pkv_internal::aligned(parents, 4) || !pkv_internal::aligned(query_start, 4))
        return PKV_ERR_INVALID_ARG;
    tree_masks_kernel<<<num_seqs, kMaskThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
        reinterpret_cast<uint32_t *>(mask), depths, parents, query_start, total_q, max_query_len, mask_words);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

extern "C" PKV_API int pkv_keep_path(void *k_cache, void *v_cache, int32_t *new_lens, const int32_t *block_tables,
                                     const int32_t *context_lens, const int32_t *query_start, const int32_t *path,
                                     const int32_t *path_lens, int num_seqs, int max_blocks_per_seq, int max_path,
                                     int num_kv_heads, int head_dim, int block_size, int64_t num_blocks, pkv_stream_t stream) {
    if (num_seqs < 0 || max_blocks_per_seq <= 0 || max_path < 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 ||
        num_blocks <= 0)
        return PKV_ERR_INVALID_ARG;
    if (head_dim != PKV_HEAD_DIM || num_seqs > 65535 || num_kv_heads > 65535) return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PKV_OK;
    if (!k_cache || !v_cache || !block_tables || !context_lens || !query_start || !path_lens || (max_path > 0 && !path))
        return PKV_ERR_INVALID_ARG;
    if (!pkv_internal::aligned16(k_cache) || !pkv_internal::aligned16(v_cache) || !pkv_internal::aligned(new_lens, 4) ||
        !pkv_internal::aligned(block_tables, 4) || !pkv_internal::aligned(context_lens, 4) ||
        !pkv_internal::aligned(query_start, 4) || !pkv_internal::aligned(path, 4) || !pkv_internal::aligned(path_lens, 4))
        return PKV_ERR_INVALID_ARG;
    KeepParams p{};
    p.cache[0] = static_cast<uint4 *>(k_cache);
    p.cache[1] = static_cast<uint4 *>(v_cache);
    p.new_lens = new_lens;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.query_start = query_start;
    p.path = path;
    p.path_lens = path_lens;
    p.max_blocks = max_blocks_per_seq;
    p.max_path = max_path;
    p.num_kv_heads = num_kv_heads;
    p.block_size = block_size;
    p.num_blocks = num_blocks;
    const int columns = 2 * num_kv_heads * kPieces;
    int ctas = 1;
    while (ctas < kKeepCluster && ctas * kKeepThreads < columns) ctas *= 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), static_cast<unsigned>(num_seqs));
    cfg.blockDim = dim3(kKeepThreads);
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2]{};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(ctas);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, keep_path_kernel, p) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

namespace pkv_internal {

int tree_take_error(int *code) {
    int value = 0;
    if (cudaMemcpyFromSymbol(&value, g_tree_error, sizeof(int)) != cudaSuccess) return PKV_ERR_CUDA;
    if (value != 0) {
        const int zero = 0;
        if (cudaMemcpyToSymbol(g_tree_error, &zero, sizeof(int)) != cudaSuccess) return PKV_ERR_CUDA;
    }
    *code = value;
    return PKV_OK;
}

}  // namespace pkv_internal
