// pkv_tree.cuh -- the masks of drafted trees as the attention kernels read them, and the call of the one for short
// contexts.
#pragma once

#include <stdint.h>

#include "pkv.h"

namespace pkv {

// Word `i` of a node's mask: all ones before the tree, nothing behind its last node.
__device__ __forceinline__ uint32_t tree_word(const uint32_t *mask, int i, int tokens) {
    if (i < 0) return 0xffffffffu;
    const int left = tokens - 32 * i;
    if (left <= 0) return 0u;
    return __ldg(mask + i) & (left >= 32 ? 0xffffffffu : (1u << left) - 1u);
}
// Whether a row of a tree sees nothing at all.
__device__ __forceinline__ bool tree_blind(const uint32_t *mask, int base, int tokens) {
    uint32_t any = base > 0;
    for (int i = 0; i * 32 < tokens; ++i) any |= tree_word(mask, i, tokens);
    return any == 0;
}

}  // namespace pkv

namespace pkv_internal {

// pkv_decode_attention_tree's checked arguments.
struct TreeCall {
    void *out;
    float *lse;
    const void *q, *k_cache, *v_cache;
    const int32_t *block_tables, *context_lens, *query_start;
    const uint32_t *mask;
    int64_t q_stride, num_blocks;
    int mask_words, num_seqs, total_q, max_query_len, max_blocks, num_q_heads, num_kv_heads, block_size, group_log2;
    float q_scale;  // scale x log2(e)
};
// Whether the call is for tree_short (else its tiles are worth the 5th-generation tensor cores' kernel), and that call.
bool tree_is_short(const TreeCall &c);
int tree_short(const TreeCall &c, pkv_stream_t stream);

}  // namespace pkv_internal
