// pkv_tree.cu -- a tree of drafted tokens around its attention: the ancestor masks and depths that go with its
// parents, the accepted path moved together in the cache, and the attention itself over short contexts (long ones and
// large batches: pkv_prompt.cu).
//
// A request's n_b drafted tokens lie behind its context in any order that puts a node behind its parent, node i
// at position base + i (base = context_lens[b] - n_b).  A node's mask has the bit of every node it attends to.
//
// tree_masks and keep_path are bound by latency.  keep_path moves a few rows per request: all of a kept row's K and V pieces
// are columns of 16 bytes, a column belongs to one thread, and the thread goes up the path with eight rows in
// flight.  Path entries ascend, so path[j] >= j: a row is read before anything is written over it.  What comes before
// the rows, the sizes, the path and its blocks, is three loads in a row, each of them all at once (with every thread
// looking up its own rows: 256 paths of 1-12 nodes 9.7 us).
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "pkv.h"
#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_tree.cuh"

namespace {

__device__ int g_tree_error;

constexpr int kMaskThreads = 128;
constexpr int kKeepThreads = 256;
constexpr int kKeepAhead = 8;   // rows in flight per column
constexpr int kKeepRun = 128;   // path entries located at a time
constexpr int kKeepCluster = 8;  // CTAs of one request at most (portable cluster size)
constexpr int kPieces = PKV_HEAD_DIM / 8;

// One CTA per request, one thread per node: up the parents to a root.  Parents come before their children, so
// the walk ends after at most `node` steps.  Bound by the deepest climb, a parent's load and a mask word read and written back
// in global memory a step, and past 128 nodes by several of them in turn (in a graph: 64 trees of 16 nodes 1.9 us, 256 of 61 3.2, a
// tree of 1024 with random parents 32, a line of 1024 661; the masks and parents are 0.02 us of HBM).
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

// ---------------------------------------------------------------- attention over short contexts
// Where a call has few rows and few keys, the time of the tensor-memory kernel is its start: barriers, tensor memory,
// copies' descriptors.  Here one CTA takes 16 (token, head) rows of one kv head, its eight warps a 16-key chunk each in
// turn, everything from global memory straight into registers, and one meeting at the end.  Bound by latency: 8 nodes over
// 300 keys (32 heads, 8 kv heads) 8.9 us where the other
// kernel takes 14.6.
//
// m16n8k16 products without shared memory.  A thread holds 32 neighbouring dims of a row (64 bytes, four loads), lane % 4
// saying which 32, and gives the product's k index a meaning of its own: in step s its four k are dims 4 s .. 4 s + 3 of
// its 32, for Q and K alike.  V's 8 x 8 blocks of (key, two of a lane's dims) are transposed by movmatrix, so that an
// output tile's columns are two dims of each of the four lanes', and a lane ends up with the same 32 dims of its output rows.
// Weights, lifted by 2^7 as in the other kernel, go into the product with V as two fp16 parts, like the decode kernels': with one
// the output's error is 2.5e-4 of its norm, with two the 2.1e-4 of its own rounding, for 0.3 us (8 nodes over 300 keys 8.6 and
// 8.9; over 1000 keys 15.0 and 15.9).  Sums are float32.
constexpr int kShortWarps = 8;
constexpr int kShortThreads = 32 * kShortWarps;
constexpr int kShortSmem = kShortWarps * 16 * PKV_HEAD_DIM * 4;  // the warps' outputs
constexpr float kShortLift = 7.0f;
constexpr float kShortLn2 = 0.6931471805599453f;
// It is taken where its CTAs are no more than the SMs and the tables no longer than 1024 positions (32 heads, 8 kv heads,
// 16-token blocks, in a graph, this kernel and the other: 8 nodes over 300 keys 8.9 and 14.6 us, 61 over 300 9.0 and 20.2,
// 4 x 16 over 300 8.9 and 15.2, 8 x 16 over 300 (256 CTAs) 14.7 and 15.7, 16 x 16 over 300 27.0 and 17.1; 8 over 1000 15.9 and
// 17.5, 61 over 1000 18.3 and 23.0; 8 over 2000 26.8 and 16.5, 61 over 2000 32.1 and 22.0).  The host does not know the
// contexts: a short one behind a longer table takes the other kernel.
constexpr int kShortCtas = 152, kShortContext = 1024;

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// 32 dims of a row.
__device__ __forceinline__ void load_dims(uint32_t (&r)[16], const __half *row) {
    const uint4 *p = reinterpret_cast<const uint4 *>(row);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint4 v = __ldg(p + i);
        r[4 * i] = v.x;
        r[4 * i + 1] = v.y;
        r[4 * i + 2] = v.z;
        r[4 * i + 3] = v.w;
    }
}

// Two softmax weights (lifted by 2^7: from 0 to 2^7) as the sum of two fp16 each, packed: off by at most 2^-21 of
// the weight, or 2^-25 where that is more.  The upper part is taken at least 2^-11 of the weight and one fp16 step (2^-24)
// below it, so that from 2^-23 on (2^-30 of the row's largest) both parts are above 0: an infinity in V times each of
// them is the same infinity, where a part of 0 or below would make NaN of it.
__device__ __forceinline__ void split_weights(float w0, float w1, uint32_t &upper, uint32_t &lower) {
    constexpr float kBelow = 1.f - 0x1p-11f, kStep = 0x1p-24f;
    const float u0 = fminf(w0 * kBelow, w0 - kStep), u1 = fminf(w1 * kBelow, w1 - kStep);
    asm("cvt.rz.relu.f16x2.f32 %0, %1, %2;" : "=r"(upper) : "f"(u1), "f"(u0));
    const float2 taken = pkv::half2_bits_to_float2(upper);
    const __half2 rest = __floats2half2_rn(w0 - taken.x, w1 - taken.y);
    lower = *reinterpret_cast<const uint32_t *>(&rest);
}

__global__ void __launch_bounds__(kShortThreads, 1) tree_short_kernel(const __grid_constant__ pkv_internal::TreeCall P) {
    extern __shared__ __align__(16) float4 s_out[];  // [warp][16 rows][32 pieces], see piece_at
    __shared__ float s_m[kShortWarps][16], s_l[kShortWarps][16];
    pkv::pdl_wait_primary();
    pkv::pdl_launch_dependents();
    const int kvh = blockIdx.x, b = blockIdx.z, warp = threadIdx.x / 32, lane = threadIdx.x & 31, g = lane >> 2, quarter = lane & 3;
    const int start = __ldg(P.query_start + b), n = __ldg(P.query_start + b + 1) - start, keys = __ldg(P.context_lens + b);
    if (n < 0 || n > P.max_query_len || start < 0 || start > P.total_q - n || keys < n || keys > P.max_blocks * P.block_size) {
        if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0) pkv::record_error(&g_tree_error, PKV_DEV_BAD_CONTEXT);
        return;
    }
    const int rows = n << P.group_log2, row0 = blockIdx.y * 16, base = keys - n, group_mask = (1 << P.group_log2) - 1;
    if (row0 >= rows) return;
    // The thread's two rows (those past the last one are computed like it and not stored).
    const uint32_t *mask[2];
    uint32_t q[2][16];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int row = min(row0 + g + 8 * r, rows - 1), token = start + (row >> P.group_log2), head = (kvh << P.group_log2) + (row & group_mask);
        mask[r] = P.mask + static_cast<int64_t>(token) * P.mask_words;
        load_dims(q[r], static_cast<const __half *>(P.q) + token * P.q_stride + head * PKV_HEAD_DIM + quarter * 32);
    }
    const int32_t *table = P.block_tables + static_cast<int64_t>(b) * P.max_blocks;
    // Element of the cache at which a chunk's rows begin (this lane's dims of its first row).
    auto chunk_at = [&](int key0) -> int64_t {
        const int block = key0 / P.block_size;
        int32_t id = __ldg(table + block);
        if (id < 0 || id >= P.num_blocks) {
            if (lane == 0) pkv::record_error(&g_tree_error, PKV_DEV_BAD_BLOCK_ID);
            id = 0;
        }
        return ((static_cast<int64_t>(id) * P.num_kv_heads + kvh) * P.block_size + (key0 - block * P.block_size)) * PKV_HEAD_DIM + quarter * 32;
    };
    const __half *const k_cache = static_cast<const __half *>(P.k_cache), *const v_cache = static_cast<const __half *>(P.v_cache);
    uint32_t k[2][16], v[2][16];  // rows g and g + 8 of the chunk
    auto load = [&](uint32_t(&x)[2][16], const __half *cache, int64_t at) {
#pragma unroll
        for (int h = 0; h < 2; ++h) load_dims(x[h], cache + at + (8 * h + g) * PKV_HEAD_DIM);
    };
    float o[16][4];
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // of rows g, g + 8 over this warp's chunks (l: this thread's keys)
    int stripped = 0;
    int key0 = warp * 16;
    int64_t at = 0;
    if (key0 < keys) {
        at = chunk_at(key0);
        load(k, k_cache, at);
        load(v, v_cache, at);
    }
    for (; key0 < keys; key0 += 16 * kShortWarps) {
        const int next = key0 + 16 * kShortWarps;
        const bool more = next < keys;
        const int64_t next_at = more ? chunk_at(next) : 0;
        float s[2][4];  // keys 8 t + 2 quarter, + 1 of rows g (0, 1) and g + 8 (2, 3)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int e = 0; e < 4; ++e) s[t][e] = 0.f;
#pragma unroll
            for (int step = 0; step < 8; ++step) {
                const uint32_t a[4] = {q[0][2 * step], q[1][2 * step], q[0][2 * step + 1], q[1][2 * step + 1]};
                pkv::mma16816(s[t], a, k[t][2 * step], k[t][2 * step + 1]);
            }
        }
        if (more) load(k, k_cache, next_at);
        if (key0 + 15 >= base) {  // some rows may not see some of these keys
            const int from = key0 - base;  // the node at the chunk's first key
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint32_t seen = __funnelshift_r(pkv::tree_word(mask[r], from >> 5, n), pkv::tree_word(mask[r], (from >> 5) + 1, n), from & 31);
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (!(seen >> (8 * t + 2 * quarter + e) & 1)) s[t][2 * r + e] = -INFINITY;
            }
            // weights there can be 0, and 0 x inf is NaN: past the context zeros, infinities and NaN of a node put aside
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int key = key0 + 8 * h + g;
                if (key < base) continue;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const uint32_t bad = ((v[h][i] & 0x7c007c00u) + 0x04000400u) & 0x80008000u;  // exponent 31, per half
                    if (key >= keys) {
                        v[h][i] = 0;
                    } else if (bad) {
                        stripped = 1;
                        v[h][i] &= ~((bad >> 15) * 0xffffu);
                    }
                }
            }
        }
        uint32_t p[4], low[4];  // the weights' upper and lower parts
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float top = fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1])) * P.q_scale;
            top = fmaxf(top, __shfl_xor_sync(pkv::kFullMask, top, 1));
            top = fmaxf(top, __shfl_xor_sync(pkv::kFullMask, top, 2));
            const float m_new = fmaxf(m[r], top - kShortLift);
            const float f = m[r] == -INFINITY ? 0.f : exp2f(m[r] - m_new), ms = m_new == -INFINITY ? 0.f : m_new;
            m[r] = m_new;
            l[r] *= f;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const float w0 = pkv::exp2_approx(fmaf(s[t][2 * r], P.q_scale, -ms)), w1 = pkv::exp2_approx(fmaf(s[t][2 * r + 1], P.q_scale, -ms));
                l[r] += w0 + w1;
                split_weights(w0, w1, p[2 * t + r], low[2 * t + r]);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                o[i][2 * r] *= f;
                o[i][2 * r + 1] *= f;
            }
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint32_t v0 = transpose8x8(v[0][i]), v1 = transpose8x8(v[1][i]);
            pkv::mma16816(o[i], p, v0, v1);
            pkv::mma16816(o[i], low, v0, v1);
        }
        if (more) load(v, v_cache, next_at);
    }
    // Outputs to shared memory: piece x (four dims) of quarter y's 32 dims of row z.
    auto piece_at = [](int w, int z, int y, int x) { return (w * 16 + z) * 32 + y * 8 + (x ^ ((2 * y + z) & 7)); };
#pragma unroll
    for (int r = 0; r < 2; ++r) {
#pragma unroll
        for (int x = 0; x < 8; ++x)
            s_out[piece_at(warp, g + 8 * r, quarter, x)] = make_float4(o[2 * x][2 * r], o[2 * x][2 * r + 1], o[2 * x + 1][2 * r], o[2 * x + 1][2 * r + 1]);
        l[r] += __shfl_xor_sync(pkv::kFullMask, l[r], 1);
        l[r] += __shfl_xor_sync(pkv::kFullMask, l[r], 2);
        if (quarter == 0) {
            s_m[warp][g + 8 * r] = m[r];
            s_l[warp][g + 8 * r] = l[r];
        }
    }
    const bool fix = __syncthreads_or(stripped);
    // A thread per eight dims of a row.
    const int z = threadIdx.x >> 4, y = (threadIdx.x >> 2) & 3, x0 = 2 * (threadIdx.x & 3), row = row0 + z;
    if (row >= rows) return;
    float top = -INFINITY, total = 0.f;
#pragma unroll
    for (int w = 0; w < kShortWarps; ++w) top = fmaxf(top, s_m[w][z]);
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kShortWarps; ++w) {
        const float f = s_m[w][z] == -INFINITY ? 0.f : exp2f(s_m[w][z] - top);
        total = fmaf(s_l[w][z], f, total);
        const float4 lo = s_out[piece_at(w, z, y, x0)], hi = s_out[piece_at(w, z, y, x0 + 1)];
        const float part[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = fmaf(part[i], f, acc[i]);
    }
    const int token = start + (row >> P.group_log2), head = (kvh << P.group_log2) + (row & group_mask), dim = 32 * y + 4 * x0;
    const uint32_t *own_mask = P.mask + static_cast<int64_t>(token) * P.mask_words;
    // A row that sees nothing is zero; one whose scores are all minus infinity has no softmax: NaN (0 x inf).
    const float inv = total == 0.f && pkv::tree_blind(own_mask, base, n) ? 0.f : 1.f / total;
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] *= inv;
    if (fix) {  // every row that sees an infinity's or a NaN's key gets it whole
        for (int node = 0; node < n; ++node) {
            if (!(pkv::tree_word(own_mask, node >> 5, n) >> (node & 31) & 1)) continue;
            const int key = base + node, block = key / P.block_size;
            const int32_t id = __ldg(table + block);
            const __half *row_v = v_cache + ((static_cast<int64_t>(id < 0 || id >= P.num_blocks ? 0 : id) * P.num_kv_heads + kvh) * P.block_size +
                                             (key - block * P.block_size)) * PKV_HEAD_DIM + dim;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float value = __half2float(row_v[i]);
                if (!isfinite(value)) acc[i] += value;
            }
        }
    }
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 pair = __floats2half2_rn(acc[2 * i], acc[2 * i + 1]);
        h[i] = *reinterpret_cast<const uint32_t *>(&pair);
    }
    const int64_t out_row = static_cast<int64_t>(token) * P.num_q_heads + head;
    *reinterpret_cast<uint4 *>(static_cast<__half *>(P.out) + out_row * PKV_HEAD_DIM + dim) = make_uint4(h[0], h[1], h[2], h[3]);
    if ((threadIdx.x & 15) == 0 && P.lse != nullptr) P.lse[out_row] = (top + log2f(total)) * kShortLn2;
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

bool tree_is_short(const TreeCall &c) {
    const int64_t ctas = static_cast<int64_t>(c.num_seqs) * c.num_kv_heads * (((c.max_query_len << c.group_log2) + 15) / 16);
    return ctas <= kShortCtas && static_cast<int64_t>(c.max_blocks) * c.block_size <= kShortContext;
}

int tree_short(const TreeCall &c, pkv_stream_t stream) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return PKV_ERR_CUDA;
    static std::atomic<uint64_t> configured{0};  // one bit per device
    const uint64_t bit = 1ull << (dev & 63);
    if (!(configured.load(std::memory_order_acquire) & bit)) {
        if (cudaFuncSetAttribute(tree_short_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kShortSmem) != cudaSuccess) return PKV_ERR_CUDA;
        configured.fetch_or(bit, std::memory_order_acq_rel);
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(c.num_kv_heads), static_cast<unsigned>(((c.max_query_len << c.group_log2) + 15) / 16),
                       static_cast<unsigned>(c.num_seqs));
    cfg.blockDim = dim3(kShortThreads);
    cfg.dynamicSmemBytes = kShortSmem;
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tree_short_kernel, c) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

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
