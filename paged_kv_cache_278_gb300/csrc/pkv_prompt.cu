// pkv_prompt.cu -- causal attention of whole prompts (packed) and of chunks of new tokens over the
// paged cache, on the 5th-generation tensor cores.
//
//     out[t][hq] = softmax_s(scale q[t][hq] . K[s] : s at or before t's position) V,   lse[t][hq]
//
// Rows.  The (token, q head) rows that read one kv head are packed token by token, the group's heads
// together: with G heads a 128-row tile is 128 / G tokens, so K and V are read once per group and the
// causal border of a tile is only 128 / G tokens wide.  One CTA takes two neighbouring tiles, A and B.
//
// What bounds it: the tensor cores, 4 x 128 flops a (row, key) pair, with one exponential per pair close
// behind (128 x 128 pairs: 1024 tensor cycles, 512 or more of the special-function units).  The two tiles
// take turns: while the tensor cores run tile A's P V and next Q K^T, tile B's warps do their softmax.
// Measured: one prompt of 16384 tokens (32 heads, G = 4) 1.52 ms, 1.45 PFLOP/s, 76 % of the measured bf16 rate (the
// same MMAs without the softmax arithmetic: 1.34 ms); four chunks of 2039 to 2048 tokens that end at 8192, 6827, 5462 and 4097
// cached ones in 16-token blocks 0.53 ms, 1.3 PFLOP/s; 37 and 34 tokens that end at 32768 and 16385 in 64-token blocks
// 60 us, 3.4 TB/s of K and V; sixteen prompts of 17 to 1000 tokens 71 us: a pair there is three key tiles long, and its start, its border tile, the last P V and the epilogue
// (some 7000 cycles together) outweigh them.
//
//   TMEM (512 columns): S_A | S_B | O_A | O_B, 128 fp32 columns each.  P (fp16, two per column) replaces
//       S in place and is the A operand of P V straight from TMEM.
//       A pair whose rows fit tile A alone is run by both softmax groups: A takes the even key tiles, B the
//       odd ones, with a row state each, joined at the end (B's accumulator lies in the same TMEM lanes).
//   warps 0-3, 4-7  softmax of tile A, B: one thread per row, its 128 scores in registers; online max
//       with lazy rescaling (O is rescaled only when a score exceeds the reference max by more than
//       2^8, then by the row's own thread), row sums in fp32 of the unrounded weights.  P is rounded to
//       fp16 once, which keeps P V at the fp16 rate (the decode kernels, bound by HBM, carry a second fp16 part): beside
//       the output's own rounding, 2.0e-4 of its norm, that adds 1.5e-4 to 2.0e-4.
//       The weights are taken 2^7 too large, and so are the sums: fp16's range up to 2^15 is used, and a weight keeps its
//       11 bits down to 2^-21 of the row's largest, some of them down to 2^-32, instead of 2^-14 and 2^-25: the
//       tail behind one dominant key counts in P V as it does in the sum.
//   warp 8  issues every tcgen05.mma (one lane).
//   warps 9, 10  issue the tensor copies: Q (64 KB) once per item and the K tiles of 128 keys, and the V tiles,
//       each through a ring of two 32 KB stages.  Two warps: with 16-token blocks a tile is 16 copies of 2 KB, and
//       one warp issuing both K's and V's held the MMAs up (the four chunks 632 us against 551 then).
//
// Work items are (pair of tiles, kv head, split of the keys), dealt to one persistent CTA per SM,
// the longest first and in alternating direction, so that CTAs end together: warp 11 finds them, a few
// ahead of the others.  Calls with too few items to fill the SMs split each item's keys; partial
// results are joined by a second launch.
//
// Keys past the context are never multiplied: the last key tile's MMAs stop at its 16-key group and
// that group's unused V rows are zeroed in shared memory, whatever the cache holds there.  Infinities and NaN in V
// reach the rows that see their position and no others (clean_values).
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "pkv.h"
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace {

__device__ int g_prompt_error;

constexpr int kDim = PKV_HEAD_DIM;
constexpr int kTileRows = 128;             // query rows per tile (M) and keys per K/V tile (N)
constexpr int kSlab = kTileRows * 128;     // 128 rows x 64 fp16 dims, 128-byte swizzle
constexpr int kOperand = 2 * kSlab;        // a whole 128 x 128 fp16 operand tile
constexpr int kRing = 2;                   // stages of K, and of V
constexpr int kItems = 4;                  // work items found ahead
constexpr int kSoftmaxWarps = 8;
constexpr int kPromptThreads = 32 * (kSoftmaxWarps + 4);  // three warpgroups
constexpr int kSoftmaxRegs = 200, kOtherRegs = 88;  // launch: 384 x 168 = 64,512 registers; 256 x 200 + 128 x 88 = 62,464
constexpr int kMmaWarp = kSoftmaxWarps, kLoadWarp = kSoftmaxWarps + 1, kValueWarp = kSoftmaxWarps + 2,
              kItemWarp = kSoftmaxWarps + 3;
constexpr float kLazy = 8.0f;              // log2 units
constexpr float kLift = 7.0f;              // P is at most 2^(kLazy + kLift) = 2^15, in fp16's range
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kMaxSplits = 64;
constexpr int64_t kMaxContext = 1 << 30;  // positions and their sums with a tile's stay in 32 bits
constexpr int kPlannedSms = 152;  // the split plan, and with it the workspace, is the same on every device

struct PromptParams {
    __half *out;
    float *lse;                   // natural log, or null
    const int32_t *query_start;   // [num_seqs + 1]
    const int32_t *block_tables;  // null: K and V are packed like q
    const int32_t *context_lens;
    float *o_part, *m_part, *l_part;  // splits > 1: [total_q][Hq][splits](x 128), m in log2 units
    int num_seqs, total_q, max_query_len, max_blocks, num_q_heads, num_kv_heads, block_size;
    int64_t num_blocks;
    int group_log2, box_rows;
    int splits;       // at most; the kernels take split_count of it
    int split_tiles;  // key tiles that a split is worth
    float q_scale;                // scale * log2(e)
    const __half *v;   // V as the maps read it: [rows][128], rows v_stride elements apart where packed
    int64_t v_stride;
    CUtensorMap tmap_q, tmap_k, tmap_v;
};

// One unit of work; `kv_count` per softmax group is 0 for a group without rows or without keys here.
struct alignas(16) Item {
    int seq;        // -1: no more items
    int kvh;
    int split;      // -1: the only one, which writes the output itself
    int row0;       // q row (token) of the pair's first token
    int live[2];    // live tokens of the groups' tiles (both tile A's where the groups share it)
    int pos0;       // logical position of the first token
    int keys;       // the request's context
    int kv_first, kv_count[2];
    int shared;     // 1: the groups share tile A, taking its key tiles in turn
};
static_assert(sizeof(Item) == 48, "read as three 16-byte pieces");

struct PromptSmem {
    static constexpr int q = 0;                              // two operand tiles
    static constexpr int ring = 2 * kOperand;
    static constexpr int values = ring + kRing * kOperand;   // ring: K stages, values: V stages
    static constexpr int bars = values + kRing * kOperand;
    static constexpr int n_bars = 4 * kRing + 2 + 2 * kItems + 8 + 2 + 1;
    static constexpr int tmem_slot = bars + n_bars * 8;
    static constexpr int items = (tmem_slot + 4 + 15) / 16 * 16;
    static constexpr int state = items + kItems * static_cast<int>(sizeof(Item));  // [2 groups][128 rows] (m, l)
    static constexpr int dirty = state + 2 * kTileRows * 8;                   // [kItems] item number + 1, see clean_values
    static constexpr int staging = (dirty + kItems * 4 + 127) / 128 * 128;  // [8 warps][32 rows][128 bytes]
    static constexpr int total = staging + kSoftmaxWarps * 32 * 128;
    static_assert(total <= 227 * 1024, "a CTA's shared memory");
};

// Barriers by index.
constexpr int kBarKFull = 0, kBarKEmpty = kRing, kBarVFull = 2 * kRing, kBarVEmpty = 3 * kRing, kBarQFull = 4 * kRing, kBarQEmpty = kBarQFull + 1,
              kBarItemFull = kBarQEmpty + 1, kBarItemEmpty = kBarItemFull + kItems, kBarS = kBarItemEmpty + kItems, kBarP = kBarS + 2,
              kBarO = kBarP + 4, kBarState = kBarO + 2, kBarJoined = kBarState + 1, kBarDrain = kBarJoined + 1;

// ---- TMEM moves (one row per lane, consecutive 32-bit columns)
// The load is asynchronous: its registers may be used after tmem_landed on them.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t (&r)[64]) {
#define PKV_R8(i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
        "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
        "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];"
        : PKV_R8(0), PKV_R8(8), PKV_R8(16), PKV_R8(24), PKV_R8(32), PKV_R8(40), PKV_R8(48), PKV_R8(56)
        : "r"(taddr)
        : "memory");
#undef PKV_R8
}
// Waits for every load issued so far and ties it to these registers, so that no use moves ahead of it.
__device__ __forceinline__ void tmem_landed(uint32_t (&r)[64]) {
#define PKV_R8(i) "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]), "+r"(r[i + 6]), "+r"(r[i + 7])
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : PKV_R8(0), PKV_R8(8), PKV_R8(16), PKV_R8(24), PKV_R8(32), PKV_R8(40), PKV_R8(48), PKV_R8(56)
                 :
                 : "memory");
#undef PKV_R8
}

// (a0, a1) * (b, b) + (c, c) and (a0, a1) + (b0, b1): packed two-lane float32, each lane rounded as the scalar form.
__device__ __forceinline__ float2 fma2s(uint32_t a0, uint32_t a1, float b, float c) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rc;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %4};\n\tmov.b64 rc, {%5, %5};\n\t"
        "fma.rn.f32x2 rc, ra, rb, rc;\n\tmov.b64 {%0, %1}, rc;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "r"(a0), "r"(a1), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float2 fma2v(uint32_t a0, uint32_t a1, float b, float c0, float c1) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rc;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %4};\n\tmov.b64 rc, {%5, %6};\n\t"
        "fma.rn.f32x2 rc, ra, rb, rc;\n\tmov.b64 {%0, %1}, rc;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "r"(a0), "r"(a1), "f"(b), "f"(c0), "f"(c1));
    return d;
}
__device__ __forceinline__ void add2(float2 &d, float b0, float b1) {
    asm("{\n\t.reg .b64 ra, rb;\n\tmov.b64 ra, {%0, %1};\n\tmov.b64 rb, {%2, %3};\n\tadd.rn.f32x2 ra, ra, rb;\n\t"
        "mov.b64 {%0, %1}, ra;\n\t}"
        : "+f"(d.x), "+f"(d.y)
        : "f"(b0), "f"(b1));
}

template <int N>
__device__ __forceinline__ void grow_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void shrink_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// 16 columns into registers (waited for), and out of registers (completed by tmem_wait_st).
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
#define PKV_R8(i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : PKV_R8(0), PKV_R8(8)
        : "r"(taddr)
        : "memory");
#undef PKV_R8
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
#define PKV_R8(i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(
            taddr),
        PKV_R8(0), PKV_R8(8)
        : "memory");
#undef PKV_R8
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D[tmem] (+)= A[tmem] * B[smem]: A is 128 rows x 16 fp16, two per 32-bit column.
__device__ __forceinline__ void umma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1 : 0)
        : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Waits for phase `parity` of the barrier; false after kWaitLimitNs.  The waits here are links of the chain
// softmax -> MMA -> softmax, mostly shorter than a read of the global timer, so that is read only once
// every 256 polls.
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity) {
    uint64_t since = 0;
    for (uint32_t polls = 0;; ++polls) {
        if (pkv::mbar_try_wait(bar, parity)) return true;
        if ((polls & 255u) == 255u) {
            const uint64_t now = pkv::global_timer_ns();
            if (since == 0) since = now;
            if (now - since > pkv::kWaitLimitNs) return false;
        }
    }
}

// A value that is the same in all lanes, as the compiler can see: what the MMA warp computes from it
// stays in uniform registers, which the MMA instructions take their descriptors from.  (With the
// items' fields as loaded, a tcgen05.mma cost about 130 cycles of issue, twice its execution.)
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(pkv::kFullMask, x, 0); }
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(pkv::kFullMask, x, 0); }

// True in one lane of the (converged) warp, always the same one.
__device__ __forceinline__ bool elected() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ void tma_prefetch_3d(const void *tensor_map, int x, int y, int z) {
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global [%0, {%1, %2, %3}];" ::"l"(tensor_map), "r"(x), "r"(y), "r"(z)
                 : "memory");
}

__device__ __forceinline__ uint4 lds128v(uint32_t addr) {  // ordered behind the barrier that published it
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// The request's new tokens and context, checked; a bad one counts as no tokens.
struct Request {
    int start, tokens, keys;
};
__device__ __forceinline__ Request request_of(const PromptParams &P, int b, bool report) {
    Request r;
    r.start = __ldg(P.query_start + b);
    r.tokens = __ldg(P.query_start + b + 1) - r.start;
    const bool paged = P.block_tables != nullptr;
    r.keys = paged ? __ldg(P.context_lens + b) : r.tokens;
    bool bad = r.tokens < 0 || r.tokens > P.max_query_len || r.start < 0 || r.start > P.total_q - r.tokens;
    if (paged) bad = bad || r.keys < r.tokens || r.keys > P.max_blocks * P.block_size;
    if (bad) {
        if (report) pkv::record_error(&g_prompt_error, PKV_DEV_BAD_CONTEXT);
        r.tokens = 0;
    }
    return r;
}

// Pairs of tiles of a request whose last key tile is `tile` or a later one.
__device__ __forceinline__ int pairs_past(const Request &r, int tile, int pair_tokens) {
    const int pairs = (r.tokens + pair_tokens - 1) / pair_tokens;
    const int64_t need = static_cast<int64_t>(tile) * kTileRows + 1 - (r.keys - r.tokens);  // tokens up to the pair's end
    if (need <= 0) return pairs;
    if (r.tokens < need) return 0;
    return pairs - (static_cast<int>(need) + pair_tokens - 1) / pair_tokens + 1;
}

// The same over every request (all lanes get the sum).
__device__ __forceinline__ int pairs_from(const PromptParams &P, int tile, int pair_tokens, int lane, bool report) {
    int c = 0;
    for (int b = lane; b < P.num_seqs; b += 32) c += pairs_past(request_of(P, b, report), tile, pair_tokens);
    return __reduce_add_sync(pkv::kFullMask, c);
}

// Key tiles of the longest context.
__device__ __forceinline__ int most_tiles(const PromptParams &P, int lane) {
    int tiles = 0;
    for (int b = lane; b < P.num_seqs; b += 32) {
        const Request r = request_of(P, b, false);
        if (r.tokens > 0) tiles = max(tiles, (r.keys + kTileRows - 1) / kTileRows);
    }
    return __reduce_max_sync(pkv::kFullMask, tiles);
}

// Splits of each item's keys, from the call's actual pairs and contexts, which the host does not know; the
// same in every CTA and in the joining launch.  Two items per SM (the longer ones come first) where the
// items are fewer than half of the SMs; up to two thirds of them, three splits make two rounds of a third of the
// work; past that the rounds cost what the splits save.  (G = 4, 8 kv heads, 16-token blocks, one call alone between
// flushes, all requests equally long, whole against split: 2 x 37 tokens ending at 32768 419 and 84 us, 37 at 4096 66 and 26,
// 4 x 100 at 8192 117 and 88, 8 x 64 at 4096 70 and 66; two splits of 128 items 119 and 146.)
__device__ __forceinline__ int split_count(const PromptParams &P, int pairs, int tiles) {
    if (P.splits <= 1) return 1;
    const int items = max(pairs * P.num_kv_heads, 1);
    int s = 2 * items <= kPlannedSms ? 2 * kPlannedSms / items : (3 * items <= 2 * kPlannedSms ? 3 : 1);
    const int most = min(P.splits, tiles / P.split_tiles);
    if (most < s) s = most * items > kPlannedSms ? kPlannedSms / items : most;  // two rounds are full, or it is one
    return max(s, 1);
}

// Item `index` of the call: pairs by their last key tile, from the last to the first (the longest first), for
// each the kv heads and the splits.
__device__ Item find_item(const PromptParams &P, int64_t index, int splits, int tiles, int lane) {
    const int tile_tokens = kTileRows >> P.group_log2, pair_tokens = 2 * tile_tokens;
    Item it{};
    const int split = static_cast<int>(index % splits);
    it.split = splits > 1 ? split : -1;
    it.kvh = static_cast<int>(index / splits % P.num_kv_heads);
    const int rank = static_cast<int>(index / splits / P.num_kv_heads);
    int lo = 0, hi = tiles;  // pairs_from(lo) > rank >= pairs_from(hi) = past
    int past = 0;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        const int c = pairs_from(P, mid, pair_tokens, lane, false);
        if (c > rank) {
            lo = mid;
        } else {
            hi = mid;
            past = c;
        }
    }
    int nth = rank - past;  // which of the pairs that end in tile lo
    int seq = -1, pair = 0;
    for (int b0 = 0; b0 < P.num_seqs; b0 += 32) {
        const int b = b0 + lane;
        int here = 0, last = 0;  // pairs of request b that end in tile lo, and the last of them
        if (b < P.num_seqs) {
            const Request r = request_of(P, b, false);
            const int later = pairs_past(r, lo + 1, pair_tokens);
            here = pairs_past(r, lo, pair_tokens) - later;
            last = (r.tokens + pair_tokens - 1) / pair_tokens - later - 1;
        }
        int upto = here;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(pkv::kFullMask, upto, d);
            if (lane >= d) upto += y;
        }
        const int all = __shfl_sync(pkv::kFullMask, upto, 31);
        if (nth >= all) {
            nth -= all;
            continue;
        }
        const int who = __ffs(__ballot_sync(pkv::kFullMask, nth < upto)) - 1;
        seq = b0 + who;
        pair = __shfl_sync(pkv::kFullMask, last + (upto - here), who) - nth;
        break;
    }
    it.seq = seq;
    if (seq < 0) return it;
    const Request r = request_of(P, seq, false);
    const int t0 = pair * pair_tokens;
    it.row0 = r.start + t0;
    it.pos0 = r.keys - r.tokens + t0;
    it.keys = r.keys;
    int count[2] = {0, 0};
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        it.live[t] = min(max(r.tokens - t0 - t * tile_tokens, 0), tile_tokens);
        if (it.live[t] > 0) count[t] = (it.pos0 + t * tile_tokens + it.live[t] - 1) / kTileRows + 1;
    }
    const int all = max(count[0], count[1]);
    const int per = (all + splits - 1) / splits;
    it.kv_first = split * per;
    const int end = min(all, it.kv_first + per);
#pragma unroll
    for (int t = 0; t < 2; ++t) it.kv_count[t] = max(min(count[t], end) - it.kv_first, 0);
    it.shared = it.live[1] == 0;
    if (it.shared) {
        it.live[1] = it.live[0];
        it.kv_count[1] = it.kv_count[0] / 2;
        it.kv_count[0] -= it.kv_count[1];
    }
    return it;
}

// V rows of a tile that not every row of the item may see: weights there can be 0, and 0 x inf is NaN.  A group's
// four warps (`part` 0-3) go over the tile before its weights are delivered: rows past the context become
// zeros (whatever lies there), and infinities and NaN of cached rows too, with the item marked: its epilogue gives
// them to the rows that do see them.  Both groups may do this to one tile: the second finds zeros.
__device__ __forceinline__ void clean_values(uint32_t v, int valid, int part, int lane, volatile uint32_t *dirty, uint32_t mark) {
    // 512 bytes at a time: rows 4 (i % 8) + lane / 8 of this part, half i / 8 of the dims
    const uint32_t at0 = v + (32 * part + (lane >> 3)) * 128 + (lane & 7) * 16;
    auto bad_of = [](uint32_t w) { return ((w & 0x7c007c00u) + 0x04000400u) & 0x80008000u; };  // exponent 31, per half
    uint32_t bad = 0;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        uint4 x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = pkv::lds128(at0 + half * kSlab + i * 512);
#pragma unroll
        for (int i = 0; i < 8; ++i) bad |= bad_of(x[i].x) | bad_of(x[i].y) | bad_of(x[i].z) | bad_of(x[i].w);
    }
    if (__any_sync(pkv::kFullMask, bad != 0) || 32 * part + 32 > valid) {
#pragma unroll 1
        for (int i = 0; i < 16; ++i) {
            const int row = 32 * part + 4 * (i & 7) + (lane >> 3);
            const uint32_t at = at0 + (i >> 3) * kSlab + (i & 7) * 512;
            const uint4 x = lds128v(at);
            const uint32_t b[4] = {bad_of(x.x), bad_of(x.y), bad_of(x.z), bad_of(x.w)};
            const bool past = row >= valid;
            if (!past && (b[0] | b[1] | b[2] | b[3])) {
                *dirty = mark;
                __threadfence_block();  // whoever finds the zeros finds the mark
            }
            if (past)
                sts128(at, 0u, 0u, 0u, 0u);
            else if (b[0] | b[1] | b[2] | b[3])
                sts128(at, x.x & ~((b[0] >> 15) * 0xffffu), x.y & ~((b[1] >> 15) * 0xffffu), x.z & ~((b[2] >> 15) * 0xffffu),
                       x.w & ~((b[3] >> 15) * 0xffffu));
        }
        pkv::fence_proxy_async_smem();  // before the arrival that lets the MMA read the tile
    }
    __syncwarp();
}

// Key tiles that an item's groups go through: the same ones, or each its own.
__device__ __forceinline__ int key_tiles(bool shared, int a, int b) { return shared ? a + b : max(a, b); }

template <bool PAGED>
__global__ void __launch_bounds__(kPromptThreads, 1) prompt_kernel(const __grid_constant__ PromptParams P) {
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t base = pkv::smem_addr(smem);
    const int warp = uniform(static_cast<int>(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    const uint32_t bars = base + PromptSmem::bars;
    auto bar = [bars](int i) { return bars + 8 * i; };
    volatile Item *slots = reinterpret_cast<volatile Item *>(smem + PromptSmem::items);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + PromptSmem::tmem_slot);

    const bool aligned = (base & 1023) == 0;  // the swizzled operand tiles need it (the same in every CTA)
    if (threadIdx.x == 0) {
        for (int i = 0; i < PromptSmem::n_bars; ++i) {
            uint32_t count = 1;
            if (i >= kBarItemEmpty && i < kBarItemEmpty + kItems) count = kSoftmaxWarps + 3;
            if (i >= kBarP && i < kBarP + 4) count = 4;  // one arrival per softmax warp of the tile
            if (i == kBarState || i == kBarJoined) count = kSoftmaxWarps;
            pkv::mbar_init(bar(i), count);
        }
        pkv::fence_mbar_init();
    }
    volatile uint32_t *dirty = reinterpret_cast<volatile uint32_t *>(smem + PromptSmem::dirty);
    if (threadIdx.x < kItems) dirty[threadIdx.x] = 0;
    if (warp == kMmaWarp && aligned) pkv::tmem_alloc(pkv::smem_addr(tmem_slot), 512);
    pkv::tmem_fence_before_sync();
    __syncthreads();
    pkv::tmem_fence_after_sync();
    pkv::pdl_wait_primary();
    pkv::pdl_launch_dependents();
    if (!aligned) {
        if (threadIdx.x == 0) pkv::record_error(&g_prompt_error, PKV_DEV_SMEM_MISALIGNED);
        return;
    }
    const uint32_t tmem = uniform(*tmem_slot);
    const int glog = P.group_log2, tile_tokens = kTileRows >> glog;
    // A wait that runs out is recorded; its warp leaves its loop, and so do the others in their turn.
    auto wait = [&](int b, uint32_t phase) {
        if (__all_sync(pkv::kFullMask, wait_phase(bar(b), phase & 1))) return true;
        if (lane == 0) pkv::record_error(&g_prompt_error, PKV_DEV_WAIT_TIMEOUT);
        return false;
    };

    if (warp >= kSoftmaxWarps) {
        shrink_registers<kOtherRegs>();
        // The cache row at which this lane's box of a key tile starts (lane = 2 x box + half).
        const int boxes_per_tile = PAGED ? kTileRows / P.box_rows : 1;
        auto box_row = [&](int seq, int kvh, int keys, int tile) -> int {
            const int key = tile * kTileRows + (lane >> 1) * P.box_rows;
            if (!PAGED || lane >= 2 * boxes_per_tile || key >= keys) return 0;
            int32_t id = __ldg(P.block_tables + static_cast<int64_t>(seq) * P.max_blocks + key / P.block_size);
            if (id < 0 || id >= P.num_blocks) {
                pkv::record_error(&g_prompt_error, PKV_DEV_BAD_BLOCK_ID);
                id = 0;
            }
            return static_cast<int>((static_cast<int64_t>(id) * P.num_kv_heads + kvh) * P.block_size + key % P.block_size);
        };
        // Copies of one K or V tile into a stage (box by box where paged; packed, rows past the sequence are
        // the next one's, past the tensor zeros).
        auto copy_tile = [&](const void *map, uint32_t dst, uint32_t full, int keys, int kvh, int tile, int first_row, int row) {
            if (PAGED) {
                const int boxes = (min(kTileRows, keys - tile * kTileRows) + P.box_rows - 1) / P.box_rows;
                if (lane == 0) pkv::mbar_arrive_expect_tx(full, boxes * P.box_rows * 256);
                __syncwarp();
                if (lane < 2 * boxes)
                    pkv::tma_load_2d(dst + (lane & 1) * kSlab + (lane >> 1) * P.box_rows * 128, map, 64 * (lane & 1), row, full);
            } else if (lane == 0) {
                pkv::mbar_arrive_expect_tx(full, kOperand);
                for (int half = 0; half < 2; ++half)
                    pkv::tma_load_2d(dst + half * kSlab, map, kvh * kDim + 64 * half, first_row + tile * kTileRows, full);
            }
            __syncwarp();
        };
        if (warp == kItemWarp) {
            // ---------------------------------------------------------------- work items, up to kItems ahead
            const int pairs = pairs_from(P, 0, 2 * tile_tokens, lane, blockIdx.x == 0);
            const int tiles = most_tiles(P, lane);
            const int splits = split_count(P, pairs, tiles);
            const uint32_t n_items = static_cast<uint32_t>(pairs) * P.num_kv_heads * splits;  // (bounded by the host)
            bool ok = true;
            for (uint32_t k = 0; ok; ++k) {
                // the rounds go in alternating direction: a CTA's items are not always the longest of their round
                const uint32_t index = k * gridDim.x + ((k & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
                Item it{};
                it.seq = -1;
                if (index < n_items) it = find_item(P, index, splits, tiles, lane);
                const int slot = k % kItems;
                if (!(ok = wait(kBarItemEmpty + slot, k / kItems + 1))) break;
                if (lane == 0) {
                    volatile int *d = reinterpret_cast<volatile int *>(slots + slot);
                    const int *s = reinterpret_cast<const int *>(&it);
#pragma unroll
                    for (int i = 0; i < static_cast<int>(sizeof(Item) / 4); ++i) d[i] = s[i];
                    mbar_arrive(bar(kBarItemFull + slot));
                }
                __syncwarp();
                if (it.seq < 0) break;
            }
        } else if (warp == kLoadWarp) {
            // ---------------------------------------------------------------- Q and K
            uint32_t stage = 0, loaded = 0;  // K stages filled, items with keys (one Q each)
            bool ok = true;
            for (uint32_t k = 0; ok; ++k) {
                const int slot = k % kItems;
                if (!(ok = wait(kBarItemFull + slot, k / kItems))) break;
                Item it;
                {
                    const uint32_t at = base + PromptSmem::items + slot * sizeof(Item);
                    uint4 *d = reinterpret_cast<uint4 *>(&it);
                    d[0] = lds128v(at);
                    d[1] = lds128v(at + 16);
                    d[2] = lds128v(at + 32);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kBarItemEmpty + slot));
                if (it.seq < 0) break;
                const int n_kv = key_tiles(it.shared, it.kv_count[0], it.kv_count[1]);
                int row = box_row(it.seq, it.kvh, it.keys, it.kv_first);
                for (int j = 0; j < n_kv; ++j, ++stage) {
                    const int tile = it.kv_first + j, st = stage % kRing;
                    const int ahead = j + 1 < n_kv ? box_row(it.seq, it.kvh, it.keys, tile + 1) : 0;
                    if (!(ok = wait(kBarKEmpty + st, stage / kRing + 1))) break;
                    copy_tile(&P.tmap_k, base + PromptSmem::ring + st * kOperand, bar(kBarKFull + st), it.keys, it.kvh, tile,
                              it.row0 - it.pos0, row);
                    row = ahead;
                    if (j > 0) continue;
                    // The first K tile is under way: now Q, once the last item's Q K^T are done (it is brought near meanwhile).
                    if (lane < (it.shared ? 2 : 4))
                        tma_prefetch_3d(&P.tmap_q, 64 * (lane & 1), it.kvh << glog, it.row0 + (lane >> 1) * tile_tokens);
                    __syncwarp();
                    if (!(ok = wait(kBarQEmpty, loaded + 1))) break;
                    ++loaded;
                    if (lane == 0) {
                        const int tiles = it.shared ? 1 : 2;
                        pkv::mbar_arrive_expect_tx(bar(kBarQFull), tiles * kOperand);
                        for (int t = 0; t < tiles; ++t)
                            for (int half = 0; half < 2; ++half)
                                pkv::tma_load_3d(base + PromptSmem::q + t * kOperand + half * kSlab, &P.tmap_q, 64 * half, it.kvh << glog,
                                                 it.row0 + t * tile_tokens, bar(kBarQFull));
                    }
                    __syncwarp();
                }
            }
            if (!ok) {  // copies still in flight land before the CTA's memory goes (bounded)
                if (loaded) wait_phase(bar(kBarQFull), (loaded - 1) & 1);
                for (uint32_t s = stage > kRing ? stage - kRing : 0; s < stage; ++s)
                    wait_phase(bar(kBarKFull + s % kRing), (s / kRing) & 1);
            }
        } else if (warp == kValueWarp) {
            // ---------------------------------------------------------------- V
            uint32_t stage = 0;
            bool ok = true;
            for (uint32_t k = 0; ok; ++k) {
                const int slot = k % kItems;
                if (!(ok = wait(kBarItemFull + slot, k / kItems))) break;
                const int seq = slots[slot].seq, kvh = slots[slot].kvh, keys = slots[slot].keys, first = slots[slot].kv_first;
                const int n_kv = key_tiles(slots[slot].shared != 0, slots[slot].kv_count[0], slots[slot].kv_count[1]);
                const int first_row = slots[slot].row0 - slots[slot].pos0;
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kBarItemEmpty + slot));
                if (seq < 0) break;
                int row = n_kv > 0 ? box_row(seq, kvh, keys, first) : 0;
                for (int j = 0; j < n_kv; ++j, ++stage) {
                    const int tile = first + j, st = stage % kRing;
                    const int ahead = j + 1 < n_kv ? box_row(seq, kvh, keys, tile + 1) : 0;
                    if (!(ok = wait(kBarVEmpty + st, stage / kRing + 1))) break;
                    copy_tile(&P.tmap_v, base + PromptSmem::values + st * kOperand, bar(kBarVFull + st), keys, kvh, tile, first_row, row);
                    row = ahead;
                }
            }
            if (!ok)
                for (uint32_t s = stage > kRing ? stage - kRing : 0; s < stage; ++s)
                    wait_phase(bar(kBarVFull + s % kRing), (s / kRing) & 1);
        } else if (warp == kMmaWarp) {
            // ---------------------------------------------------------------- tensor-core issue
            constexpr uint32_t kIdescPV = pkv::umma_idesc_f16_f32(kTileRows, kDim) | (1u << 16);  // V: MN-major
            uint32_t k_stage = 0, v_stage = 0, loaded = 0, p_count[2] = {0, 0};
            bool ok = true;
            for (uint32_t k = 0; ok; ++k) {
                const int slot = k % kItems;
                if (!(ok = wait(kBarItemFull + slot, k / kItems))) break;
                const int seq = uniform(slots[slot].seq), keys = uniform(slots[slot].keys), first = uniform(slots[slot].kv_first);
                const int n[2] = {uniform(slots[slot].kv_count[0]), uniform(slots[slot].kv_count[1])};
                const bool shared = uniform(slots[slot].shared) != 0;
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kBarItemEmpty + slot));
                if (seq < 0) break;
                const int n_kv = key_tiles(shared, n[0], n[1]);
                if (n_kv == 0) continue;  // an empty split
                // 16-key groups of key tile j that hold cached keys
                auto groups_of = [&](int j) { return (min(kTileRows, keys - (first + j) * kTileRows) + 15) / 16; };
                auto qk = [&](int t, uint32_t st, int groups) {
                    if (elected()) {
                        const uint32_t q = base + PromptSmem::q + (shared ? 0 : t) * kOperand, kk = base + PromptSmem::ring + (st % kRing) * kOperand;
                        const uint32_t idesc = pkv::umma_idesc_f16_f32(kTileRows, groups * 16);
    #pragma unroll
                        for (int ks = 0; ks < kDim / 16; ++ks) {
                            const uint32_t off = (ks >> 2) * kSlab + (ks & 3) * 32;
                            pkv::umma_f16(tmem + t * kTileRows, pkv::umma_desc_k_sw128(q + off), pkv::umma_desc_k_sw128(kk + off), idesc,
                                          ks > 0);
                        }
                        pkv::umma_commit(bar(kBarS + t));
                    }
                    __syncwarp();
                };
                auto commit = [&](int b) {
                    if (elected()) pkv::umma_commit(bar(b));
                    __syncwarp();
                };
                if (!(ok = wait(kBarQFull, loaded))) break;
                ++loaded;
                // O of group t += P V of key tile j (the group's `local`-th)
                auto pv = [&](int t, uint32_t v, int groups, int local) {
                    for (int half = 0; half < 2; ++half) {  // keys 0-63 while the softmax finishes 64-127
                        if (!wait(kBarP + 2 * t + half, p_count[t])) return false;
                        pkv::tmem_fence_after_sync();
                        if (elected()) {
#pragma unroll
                            for (int g = 4 * half; g < 4 * half + 4; ++g)
                                if (g < groups)
                                    umma_f16_ta(tmem + 2 * kTileRows + t * kDim, tmem + t * kTileRows + g * 8,
                                                pkv::umma_desc_mn_sw128(v + g * 2048, kSlab, 1024), kIdescPV, local > 0 || g > 0);
                            if (half == 1 && local + 1 == n[t]) pkv::umma_commit(bar(kBarO + t));
                        }
                        __syncwarp();
                    }
                    ++p_count[t];
                    return true;
                };
                auto k_landed = [&]() { return wait(kBarKFull + k_stage % kRing, k_stage / kRing); };
                // Q K^T of the first key tile for both groups, or of the first two for one each
                const int firsts = shared ? min(2, n_kv) : 1;
                for (int x = 0; x < firsts && ok; ++x) {
                    if (!(ok = k_landed())) break;
                    pkv::tmem_fence_after_sync();
                    for (int t = 0; t < 2; ++t)
                        if (shared ? t == x : n[t] > 0) qk(t, k_stage, groups_of(x));
                    commit(kBarKEmpty + k_stage % kRing);
                    ++k_stage;
                }
                if (!ok) break;
                if (n_kv == firsts) commit(kBarQEmpty);
                for (int j = 0; j < n_kv && ok; ++j) {
                    const int k_tile = j + (shared ? 2 : 1);
                    const bool more = k_tile < n_kv;
                    if (!(ok = wait(kBarVFull + v_stage % kRing, v_stage / kRing))) break;
                    const uint32_t v = base + PromptSmem::values + (v_stage % kRing) * kOperand;
                    const int groups = groups_of(j), local = shared ? j >> 1 : j;
                    bool k_here = false;
                    for (int t = 0; t < 2; ++t) {
                        if (shared ? t != (j & 1) : j >= n[t]) continue;
                        if (!(ok = pv(t, v, groups, local))) break;
                        if (local + 1 < n[t]) {
                            if (!k_here && !(ok = k_landed())) break;
                            k_here = true;
                            qk(t, k_stage, groups_of(k_tile));
                        }
                    }
                    if (!ok) break;
                    commit(kBarVEmpty + v_stage % kRing);
                    ++v_stage;
                    if (more) {  // (some group always takes the next K tile)
                        commit(kBarKEmpty + k_stage % kRing);
                        ++k_stage;
                        if (k_tile + 1 == n_kv) commit(kBarQEmpty);  // the item's last Q K^T has been issued
                    }
                }
            }
            if (!ok) {  // MMAs in flight end before tensor memory is freed (bounded)
                if (elected()) pkv::umma_commit(bar(kBarDrain));
                __syncwarp();
                wait_phase(bar(kBarDrain), 0);
            }
        }
    } else {
        // ---------------------------------------------------------------- softmax and output of one tile
        grow_registers<kSoftmaxRegs>();
        const int t = warp >> 2;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;  // this warp's TMEM lanes
        const uint32_t t_s = tmem + lanes + t * kTileRows, t_o = tmem + lanes + 2 * kTileRows + t * kDim;
        const int r = (warp & 3) * 32 + lane, tok = r >> glog;
        const float sc = P.q_scale;
        uint32_t s_count = 0, o_count = 0, joins = 0, v_stage = 0;  // v_stage: V stages of the items so far
        float2 *s_state = reinterpret_cast<float2 *>(smem + PromptSmem::state);
        bool ok = true;
        for (uint32_t k = 0; ok; ++k) {
            const int slot = k % kItems;
            if (!(ok = wait(kBarItemFull + slot, k / kItems))) break;
            const uint4 i0 = lds128v(base + PromptSmem::items + slot * sizeof(Item)), i1 = lds128v(base + PromptSmem::items + slot * sizeof(Item) + 16),
                        i2 = lds128v(base + PromptSmem::items + slot * sizeof(Item) + 32);
            const int seq = i0.x, kvh = i0.y, split = i0.z, slot_row0 = i0.w;
            const int live = t ? i1.y : i1.x, pos0 = i1.z, first = i2.x;
            const int n = t ? i2.z : i2.y, n_of_other = t ? i2.y : i2.z;
            const bool shared = i2.w != 0;
            const int tile = shared ? 0 : t;
            const int tile_pos = pos0 + tile * tile_tokens;  // position of the tile's first token
            const int64_t q_row = static_cast<int64_t>(slot_row0) + tile * tile_tokens + tok;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kBarItemEmpty + slot));
            if (seq < 0) break;
            const int pos = tile_pos + min(tok, live - 1);  // rows past the last token: computed like it, never stored
            const int n_kv = key_tiles(shared, n, n_of_other), keys = i1.w;
            float m_ref = -INFINITY, l = 0.f;  // what weights are relative to: kLift below a score, so that they reach 2^kLift
            for (int j = 0; j < n; ++j) {
                const int key0 = (first + (shared ? 2 * j + t : j)) * kTileRows;
                // A tile that some row of the item does not see to its end is cleaned first, while S is on its way.  Its V
                // barrier may be asked for this phase only once the last one is over (its parity would pass for this
                // one's): that is so where P V of the stage's last tile precedes what this group has waited for
                // already, and for shared rows and split keys once S is there, which was issued behind it.
                const bool border = key0 + kTileRows - 1 > pos0, early = split < 0 && !shared;
                const uint32_t vs = v_stage + (shared ? 2 * j + t : j);
                const uint32_t v = base + PromptSmem::values + (vs % kRing) * kOperand;
                bool cleaned = !border;
#pragma unroll 1
                for (int step = 0; step < 2; ++step) {
                    if (step == 1) {
                        if (!(ok = wait(kBarS + t, s_count))) break;
                        ++s_count;
                    }
                    if (!cleaned && (early || step == 1)) {
                        if (!(ok = wait(kBarVFull + vs % kRing, vs / kRing))) break;
                        clean_values(v, min(kTileRows, keys - key0), warp & 3, lane, dirty + k % kItems, k + 1);
                        cleaned = true;
                    }
                }
                if (!ok) break;
                pkv::tmem_fence_after_sync();
                uint32_t s0[64], s1[64];
                tmem_ld64(t_s, s0);
                tmem_landed(s0);
                tmem_ld64(t_s + 64, s1);
                const bool masked = key0 + kTileRows - 1 > tile_pos;  // the causal border, or the context's end
                const int lim = pos - key0;
                if (masked) {
#pragma unroll
                    for (int c = 0; c < 64; ++c) s0[c] = c <= lim ? s0[c] : 0xff800000u;
                }
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < 64; c += 2)
                    mx[(c >> 1) & 3] = fmaxf(fmaxf(mx[(c >> 1) & 3], __uint_as_float(s0[c])), __uint_as_float(s0[c + 1]));
                tmem_landed(s1);
                if (masked) {
#pragma unroll
                    for (int c = 0; c < 64; ++c) s1[c] = 64 + c <= lim ? s1[c] : 0xff800000u;
                }
#pragma unroll
                for (int c = 0; c < 64; c += 2)
                    mx[(c >> 1) & 3] = fmaxf(fmaxf(mx[(c >> 1) & 3], __uint_as_float(s1[c])), __uint_as_float(s1[c + 1]));
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;
                if (__any_sync(pkv::kFullMask, top > m_ref + (kLift + kLazy))) {
                    const float m_new = top > m_ref + (kLift + kLazy) ? top - kLift : m_ref;
                    const float a = m_ref == -INFINITY ? 0.f : exp2f(m_ref - m_new);
                    const float f = m_new == m_ref ? 1.f : a;
                    l *= f;
                    m_ref = m_new;
                    if (j > 0) {  // P V of the earlier tiles has completed: S of this one was issued behind it
#pragma unroll
                        for (int c = 0; c < kDim; c += 16) {
                            uint32_t o[16];
                            tmem_ld16(t_o + c, o);
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            tmem_st16(t_o + c, o);
                        }
                    }
                }
                const float ms = m_ref == -INFINITY ? 0.f : m_ref;  // no visible key yet: weights exp2(-inf) = 0
                float2 sum[2] = {{0.f, 0.f}, {0.f, 0.f}};
                auto weights = [&](const uint32_t(&x)[64], int half) {
#pragma unroll
                    for (int q = 0; q < 64; q += 32) {
                        uint32_t p[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float2 e = fma2s(x[q + 2 * i], x[q + 2 * i + 1], sc, -ms);
                            const float p0 = pkv::exp2_approx(e.x), p1 = pkv::exp2_approx(e.y);
                            add2(sum[i & 1], p0, p1);
                            const __half2 pk = __floats2half2_rn(p0, p1);
                            p[i] = *reinterpret_cast<const uint32_t *>(&pk);
                        }
                        tmem_st16(t_s + 32 * half + q / 2, p);
                    }
                    tmem_wait_st();
                    pkv::tmem_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kBarP + 2 * t + half));
                };
                weights(s0, 0);
                weights(s1, 1);
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            }
            if (!ok) break;
            v_stage += n_kv;
            if (n > 0) {
                if (!(ok = wait(kBarO + t, o_count))) break;
                ++o_count;
                pkv::tmem_fence_after_sync();
            }
            const bool store = tok < live;
            // The row's state and the two accumulators that make it up: its own alone, or where the groups
            // share the rows both, each group finishing half of the dims.
            float m = m_ref, total = l, w_own = 1.f, w_other = 0.f;
            if (shared) {
                s_state[t * kTileRows + r] = make_float2(m_ref, l);
                pkv::tmem_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kBarState));
                if (!(ok = wait(kBarState, joins))) break;
                pkv::tmem_fence_after_sync();
                const float2 o = s_state[(t ^ 1) * kTileRows + r];
                m = fmaxf(m_ref, o.x);
                w_own = m_ref == -INFINITY ? 0.f : exp2f(m_ref - m);
                w_other = o.x == -INFINITY ? 0.f : exp2f(o.x - m);
                total = l * w_own + o.y * w_other;
            }
            const int n_other = shared ? n_of_other : 0;
            // A split may hold none of the row's keys.  A whole row sees one at least, so only scores of minus infinity make its
            // sum 0: it has no softmax, and becomes NaN here (0 x inf) and in the joining launch alike.
            const float inv = total == 0.f && split >= 0 ? 0.f : 1.f / total;
            w_own *= inv;
            w_other *= inv;
            const int64_t row = q_row * P.num_q_heads + (kvh << glog) + (r & ((1 << glog) - 1));
            if (n > 0 || n_other > 0) {
                // 128 bytes of each row at a time (64 fp16 dims, or 32 float32 ones of a partial result) through the
                // warp's own 4 KB, so that eight lanes store a whole line.  The 16-byte pieces of row x lie at piece
                // ^ (x % 8).  Lane's share of a line: piece lane % 8 of rows 4 i + lane / 8.
                const bool whole = split < 0;
                const uint32_t lines = base + PromptSmem::staging + warp * 4096, mine = lines + lane * 128;
                const uint32_t row_bytes = whole ? kDim * 2 : P.splits * kDim * 4;
                const int group_mask = (1 << glog) - 1;
                unsigned char *const dst = reinterpret_cast<unsigned char *>(whole ? static_cast<void *>(P.out) : static_cast<void *>(P.o_part)) +
                                           ((static_cast<int64_t>(slot_row0) + tile * tile_tokens) * P.num_q_heads + (kvh << glog)) * row_bytes +
                                           (whole ? 0 : split * kDim * 4) + (lane & 7) * 16;
                uint32_t offset[8];  // of the lane's rows, from the tile's first (under 2^32: 128 tokens' rows)
                bool keep[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int x = (warp & 3) * 32 + 4 * i + (lane >> 3);
                    offset[i] = ((x >> glog) * P.num_q_heads + (x & group_mask)) * row_bytes;
                    keep[i] = (x >> glog) < live;
                }
                auto store_line = [&](int line) {
                    __syncwarp();
                    uint4 v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int x = 4 * i + (lane >> 3);
                        v[i] = lds128v(lines + x * 128 + (((lane & 7) ^ (x & 7)) << 4));
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (keep[i]) *reinterpret_cast<uint4 *>(dst + offset[i] + line * 128) = v[i];
                    __syncwarp();
                };
                const int c_begin = shared ? t * (kDim / 2) : 0, c_end = shared ? c_begin + kDim / 2 : kDim;
                const uint32_t t_other = tmem + lanes + 2 * kTileRows + (t ^ 1) * kDim;
#pragma unroll 1
                for (int c = c_begin; c < c_end; c += 64) {
                    uint32_t o[64];
                    if (n > 0) {
                        tmem_ld64(t_o + c, o);
                        tmem_landed(o);
#pragma unroll
                        for (int i = 0; i < 64; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * w_own);
                    } else {
#pragma unroll
                        for (int i = 0; i < 64; ++i) o[i] = 0u;
                    }
                    if (n_other > 0) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t q[32];
                            pkv::tmem_ld32(t_other + c + 32 * h, q);
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                o[32 * h + i] = __float_as_uint(fmaf(__uint_as_float(q[i]), w_other, __uint_as_float(o[32 * h + i])));
                        }
                    }
                    if (dirty[k % kItems] == k + 1) {
                        // Infinities and NaN that were taken out of V: every row that sees their key gets them whole
                        // (an infinity times a weight above 0 is one; a weight that underflowed is taken for one above 0).
                        for (int key = max(pos0 / kTileRows, first) * kTileRows; key <= pos && key < (first + n_kv) * kTileRows; ++key) {
                            const __half *row_v;
                            if (PAGED) {
                                const int32_t id = __ldg(P.block_tables + static_cast<int64_t>(i0.x) * P.max_blocks + key / P.block_size);
                                row_v = P.v + ((static_cast<int64_t>(id < 0 || id >= P.num_blocks ? 0 : id) * P.num_kv_heads + kvh) * P.block_size +
                                               key % P.block_size) * kDim;
                            } else {
                                row_v = P.v + (slot_row0 - pos0 + static_cast<int64_t>(key)) * P.v_stride + kvh * kDim;
                            }
#pragma unroll
                            for (int i = 0; i < 64; ++i) {
                                const float x = __half2float(row_v[c + i]);
                                if (!isfinite(x)) o[i] = __float_as_uint(__uint_as_float(o[i]) + x);
                            }
                        }
                    }
                    if (whole) {
#pragma unroll
                        for (int u = 0; u < 8; ++u) {
                            uint32_t w[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const __half2 v = __floats2half2_rn(__uint_as_float(o[8 * u + 2 * i]), __uint_as_float(o[8 * u + 2 * i + 1]));
                                w[i] = *reinterpret_cast<const uint32_t *>(&v);
                            }
                            sts128(mine + ((u ^ (lane & 7)) << 4), w[0], w[1], w[2], w[3]);
                        }
                        store_line(c / 64);
                    } else {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
#pragma unroll
                            for (int u = 0; u < 8; ++u)
                                sts128(mine + ((u ^ (lane & 7)) << 4), o[32 * h + 4 * u], o[32 * h + 4 * u + 1], o[32 * h + 4 * u + 2],
                                       o[32 * h + 4 * u + 3]);
                            store_line(c / 32 + h);
                        }
                    }
                }
                pkv::tmem_fence_before_sync();  // O read before the next item's first P V (ordered by its weights' arrival)
            }
            if (store && (t == 0 || !shared)) {
                if (split >= 0) {
                    P.m_part[row * P.splits + split] = total == 0.f ? -INFINITY : m;
                    P.l_part[row * P.splits + split] = total;
                } else if (P.lse != nullptr) {
                    P.lse[row] = (m + log2f(total)) * kLn2;
                }
            }
            if (shared) {  // neither accumulator is written again before both groups have read both
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kBarJoined));
                if (!(ok = wait(kBarJoined, joins))) break;
                ++joins;
            }
        }
    }
    pkv::tmem_fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) {
        pkv::tmem_fence_after_sync();
        pkv::tmem_dealloc(tmem, 512);
    }
}

// Joins the splits of each (token, head) row: one warp per row, four dims a lane, BATCH splits' loads in flight.
// Sixteen take 120 registers, two CTAs per SM; where those hold fewer rows than there are, eight loads a lane and
// four CTAs do better (one call alone between flushes: 512 tokens ending at 8192, three splits, 90 -> 87 us in all;
// 2 x 37 tokens ending at 32768 each the other way, 89 -> 84).
constexpr int kJoinThreads = 256;
template <int BATCH>
__global__ void __launch_bounds__(kJoinThreads, BATCH == 8 ? 4 : 2) prompt_join_kernel(const __grid_constant__ PromptParams P) {
    __shared__ int s_splits;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x < 32) {
        const int n = split_count(P, pairs_from(P, 0, 2 * kTileRows >> P.group_log2, lane, false), most_tiles(P, lane));
        if (lane == 0) s_splits = n;
    }
    __syncthreads();
    const Request r = request_of(P, blockIdx.y, false);
    // So far only the call's inputs, which the attention launch (every CTA of which has started, behind its own wait
    // for what came before) does not write; its partial results from here on.
    pkv::pdl_wait_primary();
    pkv::pdl_launch_dependents();
    const int splits = s_splits;
    if (splits == 1) return;  // the outputs are there
    const int64_t rows = static_cast<int64_t>(r.tokens) * P.num_q_heads;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * (kJoinThreads / 32) + (threadIdx.x >> 5); i < rows;
         i += static_cast<int64_t>(gridDim.x) * (kJoinThreads / 32)) {
        const int64_t row = static_cast<int64_t>(r.start) * P.num_q_heads + i;
        const float *m = P.m_part + row * P.splits, *l = P.l_part + row * P.splits;
        // lane s holds splits s and s + 32: all of the row's (m, l) in one round of loads
        float ms[2], ls[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int s = lane + 32 * u;
            ms[u] = s < splits ? __ldcg(m + s) : -INFINITY;
            ls[u] = s < splits ? __ldcg(l + s) : 0.f;
        }
        float top = fmaxf(ms[0], ms[1]);
#pragma unroll
        for (int sh = 16; sh >= 1; sh >>= 1) top = fmaxf(top, __shfl_xor_sync(pkv::kFullMask, top, sh));
        float total = 0.f;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            ls[u] = ls[u] == 0.f ? 0.f : ls[u] * exp2f(ms[u] - top);  // a split without visible keys wrote no output
            total += ls[u];
        }
#pragma unroll
        for (int sh = 16; sh >= 1; sh >>= 1) total += __shfl_xor_sync(pkv::kFullMask, total, sh);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int s0 = 0; s0 < splits; s0 += BATCH) {
            float4 o[BATCH];
            float w[BATCH];
#pragma unroll
            for (int u = 0; u < BATCH; ++u) {
                const int s = s0 + u;
                w[u] = __shfl_sync(pkv::kFullMask, s < 32 ? ls[0] : ls[1], s & 31);  // (0 past the last split)
                o[u] = __ldcg(reinterpret_cast<const float4 *>(P.o_part + (row * P.splits + min(s, splits - 1)) * kDim) + lane);
            }
#pragma unroll
            for (int u = 0; u < BATCH; ++u) {
                const bool written = w[u] != 0.f;  // else the slot holds anything (selected away, so that all loads are in flight)
                acc.x = fmaf(w[u], written ? o[u].x : 0.f, acc.x);
                acc.y = fmaf(w[u], written ? o[u].y : 0.f, acc.y);
                acc.z = fmaf(w[u], written ? o[u].z : 0.f, acc.z);
                acc.w = fmaf(w[u], written ? o[u].w : 0.f, acc.w);
            }
        }
        const float inv = 1.f / total;
        const __half2 lo = __floats2half2_rn(acc.x * inv, acc.y * inv), hi = __floats2half2_rn(acc.z * inv, acc.w * inv);
        *reinterpret_cast<uint2 *>(P.out + row * kDim + 4 * lane) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
        if (lane == 0 && P.lse != nullptr) P.lse[row] = (top + log2f(total)) * kLn2;
    }
}

// ---------------------------------------------------------------- weights of a chunk's rows
// scores[b][h][s] += sum over the chunk's rows (token t at or after s, q head of kv head h) of
// exp(scale q . K[s] - lse).  The sums run over rows, so the product is taken transposed: S^T = K Q^T with the
// 128 keys of a tile as M (one TMEM lane, one thread each) and 128 packed rows as N; a thread adds up its
// key's weights over all columns in its own registers and one thread adds them to scores: no exchange,
// no atomics, a fixed order.  Bound by the exponentials, one per (row, key) pair (2 x 128 tensor flops),
// until a chunk is so small that reading K bounds it.  The last 256 and 253 tokens of 16384 and 8193 (32 heads, G = 4):
// 200 million pairs in 57 us, where the exponentials alone would take 22 and the MMAs 27: a group's chain per 128 x 128 tile,
// from S^T's arrival through its load to the sums, is some 2100 cycles, of which 1100 are arithmetic.
//   warps 0-3, 4-7  a key tile each, or the even and odd row tiles of one, with two S^T buffers of 128 TMEM columns
//   warp 8          issues the MMAs
//   warps 9, 10     issue the tensor copies of K tiles and of Q tiles, each through a ring
//   warp 11         finds the items (two neighbouring 128-key tiles of one request and kv head, or one), a few ahead
struct ChunkWeightParams {
    PromptParams p;
    const float *lse;
    float *scores;
    int64_t capacity;
};

constexpr int kKeyStages = 4, kRowRing = 2;  // three and three: 70 us where this takes 67 (2 x 256 tokens over 16384 keys each, alone)

struct ChunkWeightSmem {
    static constexpr int keys = 0;
    static constexpr int rows = kKeyStages * kOperand;
    static constexpr int lse = rows + kRowRing * kOperand;        // [8 warps][128] floats, log2 units
    static constexpr int sums = lse + kSoftmaxWarps * kTileRows * 4;  // [kItems][128] floats
    static constexpr int bars = sums + kItems * kTileRows * 4;
    static constexpr int n_bars = 2 * kKeyStages + 2 * kRowRing + 8 + 3 * kItems + 1;
    static constexpr int tmem_slot = bars + n_bars * 8;
    static constexpr int items = (tmem_slot + 4 + 15) / 16 * 16;
    static constexpr int total = items + kItems * 48;
};
constexpr int kWKeyFull = 0, kWKeyEmpty = kKeyStages, kWRowFull = 2 * kKeyStages, kWRowEmpty = kWRowFull + kRowRing,
              kWS = kWRowEmpty + kRowRing, kWSFree = kWS + 4, kWItemFull = kWSFree + 4, kWItemEmpty = kWItemFull + kItems,
              kWSum = kWItemEmpty + kItems, kWDrain = kWSum + kItems;

// Key tiles of one request and kv head, and the row tiles that see some of them.  Group g takes the row tiles from
// first[g] on: all of them for key tile `tile` + g, or where the groups share one key tile every second one.
struct alignas(16) KeyItem {
    int seq, kvh, tile, start;
    int tokens, keys, count, shared;
    int first[2];
};
static_assert(sizeof(KeyItem) == 48, "read as 16-byte pieces");

// Item `index`; `pair`: 1 for two key tiles an item, 0 for one.
__device__ KeyItem find_key_item(const PromptParams &P, uint32_t index, int pair, int lane) {
    KeyItem it{};
    it.seq = -1;
    const uint32_t heads = P.num_kv_heads;
    int rank = static_cast<int>(index / heads);
    it.kvh = static_cast<int>(index - rank * heads);
    for (int b0 = 0; b0 < P.num_seqs; b0 += 32) {
        const int b = b0 + lane;
        int tiles = 0;
        if (b < P.num_seqs) {
            const Request r = request_of(P, b, false);
            tiles = r.tokens > 0 ? ((r.keys + kTileRows - 1) / kTileRows + pair) >> pair : 0;
        }
        int upto = tiles;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(pkv::kFullMask, upto, d);
            if (lane >= d) upto += y;
        }
        const int all = __shfl_sync(pkv::kFullMask, upto, 31);
        if (rank >= all) {
            rank -= all;
            continue;
        }
        const int who = __ffs(__ballot_sync(pkv::kFullMask, rank < upto)) - 1;
        it.seq = b0 + who;
        it.tile = (rank - __shfl_sync(pkv::kFullMask, upto - tiles, who)) << pair;
        break;
    }
    if (it.seq < 0) return it;
    const Request r = request_of(P, it.seq, false);
    it.start = r.start;
    it.tokens = r.tokens;
    it.keys = r.keys;
    it.shared = pair ^ 1;
    it.count = ((r.tokens << P.group_log2) + kTileRows - 1) / kTileRows;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        const int key0 = (it.tile + (pair & g)) * kTileRows;
        const int skip = max(key0 - (r.keys - r.tokens), 0);  // tokens before the tile's first key
        const int first = (skip << P.group_log2) / kTileRows;
        it.first[g] = pair ? (key0 < r.keys ? first : it.count) : first + ((first & 1) != g);
    }
    return it;
}

__global__ void __launch_bounds__(kPromptThreads, 1) chunk_weights_kernel(const __grid_constant__ ChunkWeightParams W) {
    using L = ChunkWeightSmem;
    const PromptParams &P = W.p;
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t base = pkv::smem_addr(smem);
    const int warp = uniform(static_cast<int>(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    const uint32_t bars = base + L::bars;
    auto bar = [bars](int i) { return bars + 8 * i; };
    volatile KeyItem *slots = reinterpret_cast<volatile KeyItem *>(smem + L::items);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::tmem_slot);
    const bool aligned = (base & 1023) == 0;
    if (threadIdx.x == 0) {
        for (int i = 0; i < L::n_bars; ++i) {
            uint32_t count = 1;
            if ((i >= kWSFree && i < kWSFree + 4) || (i >= kWSum && i < kWSum + kItems)) count = 4;
            if (i >= kWItemEmpty && i < kWItemEmpty + kItems) count = kSoftmaxWarps + 3;
            pkv::mbar_init(bar(i), count);
        }
        pkv::fence_mbar_init();
    }
    if (warp == kMmaWarp && aligned) pkv::tmem_alloc(pkv::smem_addr(tmem_slot), 512);
    pkv::tmem_fence_before_sync();
    __syncthreads();
    pkv::tmem_fence_after_sync();
    pkv::pdl_wait_primary();
    pkv::pdl_launch_dependents();
    if (!aligned) {
        if (threadIdx.x == 0) pkv::record_error(&g_prompt_error, PKV_DEV_SMEM_MISALIGNED);
        return;
    }
    const uint32_t tmem = uniform(*tmem_slot);
    const int glog = P.group_log2, tile_tokens = kTileRows >> glog;
    auto wait = [&](int b, uint32_t phase) {
        if (__all_sync(pkv::kFullMask, wait_phase(bar(b), phase & 1))) return true;
        if (lane == 0) pkv::record_error(&g_prompt_error, PKV_DEV_WAIT_TIMEOUT);
        return false;
    };

    if (warp >= kSoftmaxWarps) {
        shrink_registers<kOtherRegs>();
        const int boxes_per_tile = kTileRows / P.box_rows;
        // A published item, its slot released.
        auto take = [&](uint32_t k, KeyItem &it) {
            const int slot = k % kItems;
            if (!wait(kWItemFull + slot, k / kItems)) return false;
            uint4 *d = reinterpret_cast<uint4 *>(&it);
#pragma unroll
            for (int i = 0; i < 3; ++i) d[i] = lds128v(base + L::items + slot * sizeof(KeyItem) + 16 * i);
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kWItemEmpty + slot));
            return true;
        };
        if (warp == kItemWarp) {
            // ---------------------------------------------------------------- work items, up to kItems ahead
            int tiles = 0, pairs = 0;
            for (int b = lane; b < P.num_seqs; b += 32) {
                const Request r = request_of(P, b, blockIdx.x == 0);
                const int n = r.tokens > 0 ? (r.keys + kTileRows - 1) / kTileRows : 0;
                tiles += n;
                pairs += (n + 1) / 2;
            }
            tiles = __reduce_add_sync(pkv::kFullMask, tiles);
            pairs = __reduce_add_sync(pkv::kFullMask, pairs);
            // Two key tiles an item read Q half as often; one where that leaves SMs idle.  (One call alone between flushes:
            // 2 x 256 tokens over 16384 keys each 67 us against 78, 32 tokens over 32768 29 against 34.)
            const int pair = static_cast<int64_t>(tiles) * P.num_kv_heads > gridDim.x ? 1 : 0;
            const uint32_t n_items = static_cast<uint32_t>(pair ? pairs : tiles) * P.num_kv_heads;
            bool ok = true;
            for (uint32_t k = 0; ok; ++k) {
                const uint32_t index = k * gridDim.x + blockIdx.x;
                KeyItem it{};
                it.seq = -1;
                if (index < n_items) it = find_key_item(P, index, pair, lane);
                const int slot = k % kItems;
                if (!(ok = wait(kWItemEmpty + slot, k / kItems + 1))) break;
                if (lane == 0) {
                    volatile int *d = reinterpret_cast<volatile int *>(slots + slot);
                    const int *s = reinterpret_cast<const int *>(&it);
#pragma unroll
                    for (int i = 0; i < static_cast<int>(sizeof(KeyItem) / 4); ++i) d[i] = s[i];
                    mbar_arrive(bar(kWItemFull + slot));
                }
                __syncwarp();
                if (it.seq < 0) break;
            }
        } else if (warp == kLoadWarp) {
            // ---------------------------------------------------------------- K tiles
            uint32_t loaded = 0;
            bool ok = true;
            for (uint32_t k = 0; ok; ++k) {
                KeyItem it;
                if (!(ok = take(k, it)) || it.seq < 0) break;
                const int end = it.tile + (it.shared || it.first[1] >= it.count ? 1 : 2);
                for (int tile = it.tile; tile < end; ++tile, ++loaded) {
                    const int key = tile * kTileRows + (lane >> 1) * P.box_rows;
                    int32_t id = 0;
                    if (lane < 2 * boxes_per_tile && key < it.keys)
                        id = __ldg(P.block_tables + static_cast<int64_t>(it.seq) * P.max_blocks + key / P.block_size);
                    if (id < 0 || id >= P.num_blocks) {
                        pkv::record_error(&g_prompt_error, PKV_DEV_BAD_BLOCK_ID);
                        id = 0;
                    }
                    const int64_t row = (static_cast<int64_t>(id) * P.num_kv_heads + it.kvh) * P.block_size + key % P.block_size;
                    const int ks = loaded % kKeyStages;
                    if (!(ok = wait(kWKeyEmpty + ks, loaded / kKeyStages + 1))) break;
                    const int boxes = (min(kTileRows, it.keys - tile * kTileRows) + P.box_rows - 1) / P.box_rows;
                    if (lane == 0) pkv::mbar_arrive_expect_tx(bar(kWKeyFull + ks), boxes * P.box_rows * 256);
                    __syncwarp();
                    if (lane < 2 * boxes)
                        pkv::tma_load_2d(base + L::keys + ks * kOperand + (lane & 1) * kSlab + (lane >> 1) * P.box_rows * 128, &P.tmap_k,
                                         64 * (lane & 1), static_cast<int>(row), bar(kWKeyFull + ks));
                    __syncwarp();
                }
            }
            if (!ok)  // copies still in flight land before the CTA's memory goes (bounded)
                for (uint32_t s = loaded > kKeyStages ? loaded - kKeyStages : 0; s < loaded; ++s)
                    wait_phase(bar(kWKeyFull + s % kKeyStages), (s / kKeyStages) & 1);
        } else if (warp == kValueWarp) {
            // ---------------------------------------------------------------- Q tiles
            uint32_t rows = 0;
            bool ok = true;
            for (uint32_t k = 0; ok; ++k) {
                KeyItem it;
                if (!(ok = take(k, it)) || it.seq < 0) break;
                for (int i = min(it.first[0], it.first[1]); i < it.count; ++i) {
                    const int st = rows % kRowRing;
                    if (!(ok = wait(kWRowEmpty + st, rows / kRowRing + 1))) break;
                    ++rows;
                    if (lane == 0) {
                        pkv::mbar_arrive_expect_tx(bar(kWRowFull + st), kOperand);
                        for (int half = 0; half < 2; ++half)
                            pkv::tma_load_3d(base + L::rows + st * kOperand + half * kSlab, &P.tmap_q, 64 * half, it.kvh << glog,
                                             it.start + i * tile_tokens, bar(kWRowFull + st));
                    }
                    __syncwarp();
                }
            }
            if (!ok)
                for (uint32_t s = rows > kRowRing ? rows - kRowRing : 0; s < rows; ++s)
                    wait_phase(bar(kWRowFull + s % kRowRing), (s / kRowRing) & 1);
        } else if (warp == kMmaWarp) {
            uint32_t rows = 0, tiles = 0, fills[2] = {0, 0};  // Q and K tiles taken, each group's S^T filled
            bool ok = true;
            for (uint32_t k = 0; ok; ++k) {
                const int slot = k % kItems;
                if (!(ok = wait(kWItemFull + slot, k / kItems))) break;
                const int seq = uniform(slots[slot].seq), count = uniform(slots[slot].count);
                const int first[2] = {uniform(slots[slot].first[0]), uniform(slots[slot].first[1])};
                const bool shared = uniform(slots[slot].shared) != 0;
                const int all_rows = uniform(slots[slot].tokens) << glog;
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kWItemEmpty + slot));
                if (seq < 0) break;
                const bool two = !shared && first[1] < count;  // key tiles
                if (!(ok = wait(kWKeyFull + tiles % kKeyStages, tiles / kKeyStages))) break;
                for (int i = min(first[0], first[1]); i < count && ok; ++i, ++rows) {
                    const int st = rows % kRowRing;
                    if (!(ok = wait(kWRowFull + st, rows / kRowRing))) break;
                    const uint32_t idesc = pkv::umma_idesc_f16_f32(kTileRows, (min(kTileRows, all_rows - i * kTileRows) + 15) / 16 * 16);
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        if (i < first[g] || (shared && ((i ^ first[g]) & 1))) continue;
                        const uint32_t ks = (tiles + (shared ? 0 : g)) % kKeyStages;
                        if (g == 1 && two && i == first[1] && !(ok = wait(kWKeyFull + ks, (tiles + 1) / kKeyStages))) break;
                        const int buf = 2 * g + (fills[g] & 1);
                        if (!(ok = wait(kWSFree + buf, (fills[g] >> 1) + 1))) break;
                        ++fills[g];
                        pkv::tmem_fence_after_sync();
                        if (elected()) {
                            const uint32_t a = base + L::keys + ks * kOperand, b = base + L::rows + st * kOperand;
#pragma unroll
                            for (int x = 0; x < kDim / 16; ++x) {
                                const uint32_t off = (x >> 2) * kSlab + (x & 3) * 32;
                                pkv::umma_f16(tmem + buf * kTileRows, pkv::umma_desc_k_sw128(a + off), pkv::umma_desc_k_sw128(b + off), idesc, x > 0);
                            }
                            pkv::umma_commit(bar(kWS + buf));
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                    if (elected()) {
                        pkv::umma_commit(bar(kWRowEmpty + st));
                        if (i + 1 == count) {
                            pkv::umma_commit(bar(kWKeyEmpty + tiles % kKeyStages));
                            if (two) pkv::umma_commit(bar(kWKeyEmpty + (tiles + 1) % kKeyStages));
                        }
                    }
                    __syncwarp();
                }
                tiles += two ? 2 : 1;
            }
            if (!ok) {  // MMAs in flight end before tensor memory is freed (bounded)
                if (elected()) pkv::umma_commit(bar(kWDrain));
                __syncwarp();
                wait_phase(bar(kWDrain), 0);
            }
        }
    } else {
        grow_registers<kSoftmaxRegs>();
        const int grp = warp >> 2;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const int key_lane = (warp & 3) * 32 + lane;  // this thread's key in the tile
        float4 *s_lse = reinterpret_cast<float4 *>(smem + L::lse) + warp * 32;  // this warp's own copy: no other warp waits for it
        float *s_sum = reinterpret_cast<float *>(smem + L::sums);
        const float sc = P.q_scale;
        uint32_t seen = 0;  // S^T tiles this group has read
        bool ok = true;
        for (uint32_t k = 0; ok; ++k) {
            const int slot = k % kItems;
            if (!(ok = wait(kWItemFull + slot, k / kItems))) break;
            const uint4 i0 = lds128v(base + L::items + slot * sizeof(KeyItem)), i1 = lds128v(base + L::items + slot * sizeof(KeyItem) + 16),
                        i2 = lds128v(base + L::items + slot * sizeof(KeyItem) + 32);
            const int seq = i0.x, kvh = i0.y, start = i0.w, tokens = i1.x, keys = i1.y, count = i1.z;
            const bool shared = i1.w != 0;
            const int tile = static_cast<int>(i0.z) + (shared ? 0 : grp), step = shared ? 2 : 1;
            if (seq < 0) break;
            const int key = tile * kTileRows + key_lane;
            const int rows = tokens << glog;
            float2 sum[2] = {{0.f, 0.f}, {0.f, 0.f}};
            // What scores holds, in flight through the whole item.
            float *const at = W.scores + (static_cast<int64_t>(seq) * P.num_kv_heads + kvh) * W.capacity + key;
            const bool writes = (grp == 0 || !shared) && key < keys;
            const float before = writes ? __ldcg(at) : 0.f;
            // minus the lse of four neighbouring columns of row tile i, log2 units (of one token with 4 heads or more)
            const float *const lse = W.lse + static_cast<int64_t>(start) * P.num_q_heads + (kvh << glog);
            auto column_lse = [&](int i) {
                const int c = i * kTileRows + 4 * lane;
                float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i < count && c < rows) {  // (rows is a multiple of the group: with 4 heads all four columns are live)
                    const float *p = lse + (c >> glog) * P.num_q_heads + (c & ((1 << glog) - 1));
                    if (glog >= 2) {
                        z = __ldg(reinterpret_cast<const float4 *>(p));
                    } else {
                        const int step = glog == 1 ? 1 : P.num_q_heads;  // columns c, c + 1: two heads, or two tokens
                        z.x = __ldg(p);
                        if (c + 1 < rows) z.y = __ldg(p + step);
                        if (c + 2 < rows) z.z = __ldg(p + (glog == 1 ? P.num_q_heads : 2 * step));
                        if (c + 3 < rows) z.w = __ldg(p + (glog == 1 ? P.num_q_heads + 1 : 3 * step));
                    }
                }
                return make_float4(z.x * -kLog2e, z.y * -kLog2e, z.z * -kLog2e, z.w * -kLog2e);
            };
            int i = grp ? i2.y : i2.x;
            float4 z = column_lse(i);
            for (; i < count; i += step) {
                const int buf = 2 * grp + (seen & 1);
                __syncwarp();
                s_lse[lane] = z;
                z = column_lse(i + step);
                if (!(ok = wait(kWS + buf, seen >> 1))) break;
                ++seen;
                pkv::tmem_fence_after_sync();
                uint32_t s0[64], s1[64];
                tmem_ld64(tmem + lanes + buf * kTileRows, s0);
                tmem_ld64(tmem + lanes + buf * kTileRows + 64, s1);
                tmem_landed(s0);
                tmem_landed(s1);
                pkv::tmem_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kWSFree + buf));
                const int pos0 = keys - tokens + i * tile_tokens;  // position of the tile's first row
                if (pos0 >= (tile + 1) * kTileRows - 1 && rows - i * kTileRows >= kTileRows) {
                    auto all = [&](const uint32_t(&x)[64], const float4 *lse4) {
#pragma unroll
                        for (int c = 0; c < 16; ++c) {
                            const float4 e = lse4[c];  // negated
                            const float2 a = fma2v(x[4 * c], x[4 * c + 1], sc, e.x, e.y), b = fma2v(x[4 * c + 2], x[4 * c + 3], sc, e.z, e.w);
                            add2(sum[0], pkv::exp2_approx(a.x), pkv::exp2_approx(a.y));
                            add2(sum[1], pkv::exp2_approx(b.x), pkv::exp2_approx(b.y));
                        }
                    };
                    all(s0, s_lse);
                    all(s1, s_lse + 16);
                } else {  // columns from the first token at or after the key, to the last live row
                    const int from = max(key - pos0, 0) << glog, to = rows - i * kTileRows;
                    auto some = [&](const uint32_t(&x)[64], int c0) {
#pragma unroll
                        for (int c = 0; c < 64; c += 2) {
                            const float2 e = reinterpret_cast<const float2 *>(s_lse)[(c0 + c) / 2];
                            const float2 a = fma2v(x[c], x[c + 1], sc, e.x, e.y);
                            const float w0 = pkv::exp2_approx(a.x), w1 = pkv::exp2_approx(a.y);
                            add2(sum[(c >> 1) & 1], c0 + c >= from && c0 + c < to ? w0 : 0.f,
                                 c0 + c + 1 >= from && c0 + c + 1 < to ? w1 : 0.f);
                        }
                    };
                    some(s0, 0);
                    some(s1, 64);
                }
            }
            if (!ok) break;
            const float total = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            float other = 0.f;
            if (shared) {  // the slot's sums are read before the slot's next item is published
                if (grp == 1) {
                    s_sum[slot * kTileRows + key_lane] = total;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kWSum + slot));
                } else {
                    if (!(ok = wait(kWSum + slot, k / kItems))) break;
                    other = s_sum[slot * kTileRows + key_lane];
                }
            }
            if (writes) *at = before + (total + other);
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kWItemEmpty + slot));
        }
    }
    pkv::tmem_fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) {
        pkv::tmem_fence_after_sync();
        pkv::tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------ host side

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

int encode_map(CUtensorMap *map, int rank, const void *base, const cuuint64_t *dims, const cuuint64_t *strides, const cuuint32_t *box) {
    static const EncodeTiledFn fn = [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return static_cast<EncodeTiledFn>(nullptr);
        return reinterpret_cast<EncodeTiledFn>(ptr);
    }();
    if (!fn) return PKV_ERR_CUDA;
    const cuuint32_t elem[3] = {1, 1, 1};
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank, const_cast<void *>(base), dims, strides, box, elem,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? PKV_OK : PKV_ERR_CUDA;
}

// q rows [total][Hq][128] with `stride` elements between tokens, read in (64 dims, group, 128 / group) boxes.
int encode_query(CUtensorMap *map, const void *q, int64_t stride, int total, int num_q_heads, int group) {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(kDim), static_cast<cuuint64_t>(num_q_heads), static_cast<cuuint64_t>(total)};
    const cuuint64_t strides[2] = {kDim * 2, static_cast<cuuint64_t>(stride) * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(group), static_cast<cuuint32_t>(kTileRows / group)};
    return encode_map(map, 3, q, dims, strides, box);
}

// [rows][cols] fp16 with `stride` elements between rows, read in `box_rows` x 64 boxes.
int encode_rows(CUtensorMap *map, const void *base, int64_t rows, int64_t cols, int64_t stride, int box_rows) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride) * 2};
    const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)};
    return encode_map(map, 2, base, dims, strides, box);
}


// Key tiles that a split is worth: the joining launch costs by the rows, so one per 1024 rows, two at least and
// eight at most.  (One call alone between flushes, 37 tokens x 32 heads over 1000 keys: 22.5 us with two tiles, 27 with
// four, 27.5 whole; 160 over 4096: 42 with two or four, 34 with five; 512 over 2048: 49 with four, 41 whole.)
int split_tiles(int total_q, int num_q_heads) {
    const int64_t t = static_cast<int64_t>(total_q) * num_q_heads / 1024;
    return t < 2 ? 2 : (t > 8 ? 8 : static_cast<int>(t));
}

// The most splits of each item's keys: 1 when the items, by the fewest pairs that total_q rows make, fill two
// thirds of the SMs or the contexts are short, else what gives four items per SM.
int plan_splits(int num_seqs, int total_q, int num_q_heads, int num_kv_heads, int max_context) {
    const int pair_tokens = 2 * kTileRows / (num_q_heads / num_kv_heads);
    const int64_t pairs = (static_cast<int64_t>(total_q) + pair_tokens - 1) / pair_tokens;
    const int64_t items = (pairs > num_seqs ? pairs : num_seqs) * num_kv_heads;
    if (3 * items > 2 * kPlannedSms) return 1;
    const int64_t by_keys = max_context / (split_tiles(total_q, num_q_heads) * kTileRows);
    if (by_keys < 3) return 1;
    int64_t s = 4 * kPlannedSms / (items > 0 ? items : 1);
    s = s < by_keys ? s : by_keys;
    s = s < kMaxSplits ? s : kMaxSplits;
    return s > 1 ? static_cast<int>(s) : 1;
}

using pkv_internal::align256;

size_t prompt_workspace(int total_q, int num_q_heads, int splits) {
    if (splits <= 1) return 0;
    const size_t rows = static_cast<size_t>(total_q) * num_q_heads * splits;
    return align256(rows * kDim * sizeof(float)) + 2 * align256(rows * sizeof(float));
}

bool group_ok(int num_q_heads, int num_kv_heads) {
    const int g = num_q_heads / num_kv_heads;
    return g == 1 || g == 2 || g == 4 || g == 8;
}

template <bool PAGED>
int launch_prompt(PromptParams p, int max_context, void *workspace, size_t workspace_bytes, pkv_stream_t stream) {
    p.splits = plan_splits(p.num_seqs, p.total_q, p.num_q_heads, p.num_kv_heads, max_context);
    p.split_tiles = split_tiles(p.total_q, p.num_q_heads);
    const size_t need = prompt_workspace(p.total_q, p.num_q_heads, p.splits);
    if (need) {
        if (!workspace || workspace_bytes < need || !pkv_internal::aligned(workspace, 256)) return PKV_ERR_WORKSPACE;
        const size_t rows = static_cast<size_t>(p.total_q) * p.num_q_heads * p.splits;
        unsigned char *ws = static_cast<unsigned char *>(workspace);
        p.o_part = reinterpret_cast<float *>(ws);
        p.m_part = reinterpret_cast<float *>(ws + align256(rows * kDim * sizeof(float)));
        p.l_part = reinterpret_cast<float *>(ws + align256(rows * kDim * sizeof(float)) + align256(rows * sizeof(float)));
    }
    auto kernel = prompt_kernel<PAGED>;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return PKV_ERR_CUDA;
    static std::atomic<uint64_t> configured{0};  // one bit per device
    const uint64_t bit = 1ull << (dev & 63);
    if (!(configured.load(std::memory_order_acquire) & bit)) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, PromptSmem::total) != cudaSuccess)
            return PKV_ERR_CUDA;
        configured.fetch_or(bit, std::memory_order_acq_rel);
    }
    const int pair_tokens = 2 * kTileRows >> p.group_log2;
    const int64_t most = (static_cast<int64_t>(p.total_q) / pair_tokens + p.num_seqs) * p.num_kv_heads * p.splits;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(most < sms ? most : sms));
    cfg.blockDim = dim3(kPromptThreads);
    cfg.dynamicSmemBytes = PromptSmem::total;
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, p) != cudaSuccess) return PKV_ERR_CUDA;
    if (p.splits == 1) return PKV_OK;
    const int64_t rows = static_cast<int64_t>(p.max_query_len < p.total_q ? p.max_query_len : p.total_q) * p.num_q_heads;
    const int64_t by_rows = (rows + kJoinThreads / 32 - 1) / (kJoinThreads / 32), by_sms = (4 * sms + p.num_seqs - 1) / p.num_seqs;
    const bool many = static_cast<int64_t>(p.total_q) * p.num_q_heads > 2 * sms * (kJoinThreads / 32);
    cfg.gridDim = dim3(static_cast<unsigned>(by_rows < by_sms ? by_rows : by_sms), p.num_seqs);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, many ? prompt_join_kernel<8> : prompt_join_kernel<16>, p) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

int log2_of(int g) { return g == 1 ? 0 : (g == 2 ? 1 : (g == 4 ? 2 : 3)); }

// What both forms check; PKV_OK with *done set when there is nothing to do.
int check_prompt(const float *lse, const void *q, int64_t q_stride, const int32_t *start, int num_seqs,
                 int total_q, int max_query_len, int num_q_heads, int num_kv_heads, int head_dim, float scale, bool *done) {
    *done = false;
    if (num_seqs < 0 || total_q < 0 || max_query_len < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0)
        return PKV_ERR_INVALID_ARG;
    if (num_q_heads % num_kv_heads != 0 || !(scale > 0.f) || !isfinite(scale)) return PKV_ERR_INVALID_ARG;
    if (head_dim != kDim || !group_ok(num_q_heads, num_kv_heads) || num_seqs > 65535 || num_q_heads > 65535) return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0 || total_q == 0 || max_query_len == 0) {
        *done = true;
        return PKV_OK;
    }
    if (!q || !start) return PKV_ERR_INVALID_ARG;
    if (!pkv_internal::aligned16(q) || !pkv_internal::aligned(start, 4) ||
        (lse && !pkv_internal::aligned(lse, 4)))
        return PKV_ERR_INVALID_ARG;
    if (q_stride % 8 != 0 || q_stride < static_cast<int64_t>(num_q_heads) * head_dim) return PKV_ERR_INVALID_ARG;
    return PKV_OK;
}

}  // namespace

extern "C" PKV_API size_t pkv_prefill_workspace_size(int num_seqs, int total_q, int num_q_heads, int num_kv_heads, int head_dim,
                                                     int max_context) {
    if (num_seqs <= 0 || total_q <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads != 0 ||
        head_dim != kDim || max_context <= 0 || !group_ok(num_q_heads, num_kv_heads))
        return 0;
    return prompt_workspace(total_q, num_q_heads, plan_splits(num_seqs, total_q, num_q_heads, num_kv_heads, max_context));
}

extern "C" PKV_API int pkv_prefill_attention(void *out, float *lse, const void *q, int64_t q_stride, const void *k,
                                             int64_t k_stride, const void *v, int64_t v_stride, const int32_t *seq_start,
                                             int num_seqs, int total_tokens, int max_seq_len, int num_q_heads,
                                             int num_kv_heads, int head_dim, float scale, void *workspace,
                                             size_t workspace_bytes, pkv_stream_t stream) {
    bool done = false;
    int st = check_prompt(lse, q, q_stride, seq_start, num_seqs, total_tokens, max_seq_len, num_q_heads, num_kv_heads,
                          head_dim, scale, &done);
    if (st != PKV_OK || done) return st;
    if (!out || !pkv_internal::aligned16(out)) return PKV_ERR_INVALID_ARG;
    const int64_t least = static_cast<int64_t>(num_kv_heads) * head_dim;
    if (!k || !v || !pkv_internal::aligned16(k) || !pkv_internal::aligned16(v) || k_stride % 8 != 0 || v_stride % 8 != 0 ||
        k_stride < least || v_stride < least)
        return PKV_ERR_INVALID_ARG;
    PromptParams p{};
    p.out = static_cast<__half *>(out);
    p.lse = lse;
    p.query_start = seq_start;
    p.v = static_cast<const __half *>(v);
    p.v_stride = v_stride;
    p.num_seqs = num_seqs;
    p.total_q = total_tokens;
    p.max_query_len = max_seq_len;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.group_log2 = log2_of(num_q_heads / num_kv_heads);
    p.q_scale = scale * kLog2e;
    st = encode_query(&p.tmap_q, q, q_stride, total_tokens, num_q_heads, num_q_heads / num_kv_heads);
    if (st == PKV_OK) st = encode_rows(&p.tmap_k, k, total_tokens, least, k_stride, kTileRows);
    if (st == PKV_OK) st = encode_rows(&p.tmap_v, v, total_tokens, least, v_stride, kTileRows);
    if (st != PKV_OK) return st;
    return launch_prompt<false>(p, max_seq_len, workspace, workspace_bytes, stream);
}

extern "C" PKV_API int pkv_prefill_attention_paged(void *out, float *lse, const void *q, int64_t q_stride,
                                                   const void *k_cache, const void *v_cache, const int32_t *block_tables,
                                                   const int32_t *context_lens, const int32_t *query_start, int num_seqs,
                                                   int total_q, int max_query_len, int max_blocks_per_seq, int num_q_heads,
                                                   int num_kv_heads, int head_dim, int block_size, int64_t num_blocks,
                                                   float scale, void *workspace, size_t workspace_bytes,
                                                   pkv_stream_t stream) {
    int st = pkv_internal::check_decode_args(q, k_cache, v_cache, block_tables, context_lens, num_seqs, max_blocks_per_seq,
                                             num_q_heads, num_kv_heads, head_dim, block_size, num_blocks);
    if (st != PKV_OK) return st;
    bool done = false;
    st = check_prompt(lse, q, q_stride, query_start, num_seqs, total_q, max_query_len, num_q_heads, num_kv_heads, head_dim,
                      scale, &done);
    if (st != PKV_OK || done) return st;
    if (!out || !pkv_internal::aligned16(out)) return PKV_ERR_INVALID_ARG;
    const int64_t rows = num_blocks * num_kv_heads * block_size;
    if (rows >= 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;  // box row coordinates are signed 32-bit
    if (static_cast<int64_t>(max_blocks_per_seq) * block_size > kMaxContext) return PKV_ERR_UNSUPPORTED;
    PromptParams p{};
    p.out = static_cast<__half *>(out);
    p.lse = lse;
    p.v = static_cast<const __half *>(v_cache);
    p.query_start = query_start;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.num_seqs = num_seqs;
    p.total_q = total_q;
    p.max_query_len = max_query_len;
    p.max_blocks = max_blocks_per_seq;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.block_size = block_size;
    p.num_blocks = num_blocks;
    p.group_log2 = log2_of(num_q_heads / num_kv_heads);
    p.q_scale = scale * kLog2e;
    p.box_rows = kTileRows;
    while (block_size % p.box_rows != 0) p.box_rows /= 2;  // a box never leaves its block: 16 at least
    st = encode_query(&p.tmap_q, q, q_stride, total_q, num_q_heads, num_q_heads / num_kv_heads);
    if (st == PKV_OK) st = encode_rows(&p.tmap_k, k_cache, rows, kDim, kDim, p.box_rows);
    if (st == PKV_OK) st = encode_rows(&p.tmap_v, v_cache, rows, kDim, kDim, p.box_rows);
    if (st != PKV_OK) return st;
    return launch_prompt<true>(p, static_cast<int>(static_cast<int64_t>(max_blocks_per_seq) * block_size), workspace, workspace_bytes,
                               stream);
}

extern "C" PKV_API int pkv_prefill_attention_weights(float *scores, int64_t score_capacity, const void *q, int64_t q_stride,
                                                     const float *lse, const void *k_cache, const int32_t *block_tables,
                                                     const int32_t *context_lens, const int32_t *query_start, int num_seqs,
                                                     int total_q, int max_query_len, int max_blocks_per_seq, int num_q_heads,
                                                     int num_kv_heads, int head_dim, int block_size, int64_t num_blocks,
                                                     float scale, pkv_stream_t stream) {
    int st = pkv_internal::check_decode_args(q, k_cache, k_cache, block_tables, context_lens, num_seqs, max_blocks_per_seq,
                                             num_q_heads, num_kv_heads, head_dim, block_size, num_blocks);
    if (st != PKV_OK) return st;
    bool done = false;
    st = check_prompt(lse, q, q_stride, query_start, num_seqs, total_q,
                      max_query_len, num_q_heads, num_kv_heads, head_dim, scale, &done);
    if (st != PKV_OK) return st;
    const int64_t cap = static_cast<int64_t>(max_blocks_per_seq) * block_size;
    if (!scores || !pkv_internal::aligned(scores, 4) || score_capacity < cap || (!done && !lse)) return PKV_ERR_INVALID_ARG;
    // four heads' values are read at once (whole rows of a 16-byte aligned lse begin so too)
    if (num_q_heads / num_kv_heads >= 4 && !pkv_internal::aligned16(lse)) return PKV_ERR_INVALID_ARG;
    if (done) return PKV_OK;
    const int64_t rows = num_blocks * num_kv_heads * block_size;
    if (rows >= 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;  // box row coordinates are signed 32-bit
    if (static_cast<int64_t>(max_blocks_per_seq) * block_size > kMaxContext) return PKV_ERR_UNSUPPORTED;
    ChunkWeightParams w{};
    PromptParams &p = w.p;
    p.query_start = query_start;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.num_seqs = num_seqs;
    p.total_q = total_q;
    p.max_query_len = max_query_len;
    p.max_blocks = max_blocks_per_seq;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.block_size = block_size;
    p.num_blocks = num_blocks;
    p.group_log2 = log2_of(num_q_heads / num_kv_heads);
    p.q_scale = scale * kLog2e;
    p.box_rows = kTileRows;
    while (block_size % p.box_rows != 0) p.box_rows /= 2;
    w.lse = lse;
    w.scores = scores;
    w.capacity = score_capacity;
    st = encode_query(&p.tmap_q, q, q_stride, total_q, num_q_heads, num_q_heads / num_kv_heads);
    if (st == PKV_OK) st = encode_rows(&p.tmap_k, k_cache, rows, kDim, kDim, p.box_rows);
    if (st != PKV_OK) return st;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return PKV_ERR_CUDA;
    static std::atomic<uint64_t> configured{0};  // one bit per device
    const uint64_t bit = 1ull << (dev & 63);
    if (!(configured.load(std::memory_order_acquire) & bit)) {
        if (cudaFuncSetAttribute(chunk_weights_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, ChunkWeightSmem::total) !=
            cudaSuccess)
            return PKV_ERR_CUDA;
        configured.fetch_or(bit, std::memory_order_acq_rel);
    }
    const int64_t most = (cap + kTileRows - 1) / kTileRows * num_seqs * num_kv_heads;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(most < sms ? most : sms));
    cfg.blockDim = dim3(kPromptThreads);
    cfg.dynamicSmemBytes = ChunkWeightSmem::total;
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, chunk_weights_kernel, w) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

namespace pkv_internal {

int prompt_take_error(int *code) {
    int value = 0;
    if (cudaMemcpyFromSymbol(&value, g_prompt_error, sizeof(int)) != cudaSuccess) return PKV_ERR_CUDA;
    if (value != 0) {
        const int zero = 0;
        if (cudaMemcpyToSymbol(g_prompt_error, &zero, sizeof(int)) != cudaSuccess) return PKV_ERR_CUDA;
    }
    *code = value;
    return PKV_OK;
}

}  // namespace pkv_internal
