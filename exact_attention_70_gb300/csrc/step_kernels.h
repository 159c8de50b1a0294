// step_kernels.h -- parameters and launchers of the calls around paged attention (plan, norm with rotation,
// decode behind shared prefixes).
#pragma once

#include "kernels.h"

namespace attn {

// ---- a step's pages and slots -------------------------------------------------------------------

struct PlanParams {
    const int* cache_seqlens;  // [batch] tokens held
    const int* new_lens;       // [batch] tokens to come
    int* block_table;          // [batch, max_pages]
    const int* free_pages;     // [num_free], of which the first *free_count are free
    const int* free_count;
    int* free_left;
    int* cu_seqlens_q;   // [batch + 1]
    int* seqlens_after;  // [batch]
    int* positions;      // [total_q]
    int* slot_map;       // [total_q]
    int* page_off;       // workspace [batch + 1]: new pages before a sequence's; free_count.  Null: a small step
    unsigned* status;
    int batch, total_q, page_size, max_pages, num_free, num_pages;
};

// Steps of up to so many tokens and sequences take one launch and no workspace: 2048 tokens of 16 sequences
// 5.1 us (two launches 5.4), 4096 tokens 7.1 (5.3), 64 single tokens 4.1 (5.9); a launch is about 2 us of host time.
constexpr int kPlanSmall = 2048;

cudaError_t launch_plan(const PlanParams& p, cudaStream_t stream);

// ---- norms of queries and keys with the rotation ------------------------------------------------

constexpr int kNrAxes = 3;
constexpr int kNrBwdBlocks = kGb300Sms * 2;  // blocks (partial sums of the weights' gradients) of the backward

struct NormRopeParams {
    const __nv_bfloat16* q;  // [total, Hq, d], q_stride elements between tokens
    const __nv_bfloat16* k;
    const __nv_bfloat16* v;  // append
    const void* q_weight;    // [d] or null: no norm
    const void* k_weight;
    const float* rot_cos;  // [rot_rows, rot_dim / 2]
    const float* rot_sin;
    const int* positions;  // [axes, total]
    const int* slots;      // append: [total], negative: none
    __nv_bfloat16* q_out;  // [total, Hq, d]
    __nv_bfloat16* k_out;
    __nv_bfloat16* k_cache;  // append: [cache_rows, Hkv, d]
    __nv_bfloat16* v_cache;
    const __nv_bfloat16* dq_out;  // backward: [total, Hq, d]
    const __nv_bfloat16* dk_out;
    __nv_bfloat16* dq;
    __nv_bfloat16* dk;
    float* dq_weight;
    float* dk_weight;
    float* part_w;  // [kNrBwdBlocks, d]
    unsigned* status;
    unsigned plane_axis[4];  // two bits a plane
    float eps;
    int q_stride, k_stride, v_stride, dq_stride, dk_stride;
    int weight_f32, total, Hq, Hkv, rot_dim, rot_rows, interleaved, axes, cache_rows;
    int blocks[3], par_log2[3];  // by kind of row (queries, keys, values), set by the launchers
};

cudaError_t launch_norm_rope(NormRopeParams p, int head_dim, bool append, cudaStream_t stream);
cudaError_t launch_norm_rope_bwd(NormRopeParams p, int head_dim, cudaStream_t stream);

// ---- decode behind shared prefixes -------------------------------------------------------------

// Workspace of attn_decode_kvcache_shared: [header][groups][lengths][units][items][LSE of the parts][O of the parts]
struct SharedHeader {
    int n_items[2];    // of units with many rows, and behind them in the list those of units with few
    int next_item[2];  // the claim counters of the two halves
    int n_own;         // units of the sequences' own keys
    int bad;           // lengths that do not fit: nothing is computed
    int ctas;          // CTAs that do units with many rows
    int pad[57];
};

// Query rows that walk the same keys: up to two tiles of tokens, of one sequence against its own keys or of
// a group against its prefix.  Its key blocks are cut into `pieces`, a piece's rows leave `split` parts
// (few rows: one a warp); part s of kv head h lies at part + (h pieces split + s) rows.
struct alignas(16) SharedUnit {
    int q0, ntok;          // tokens [q0, q0 + ntok) of q
    int row;               // of block_table
    int key_min, key_end;  // keys [key_min, key_end)
    int pos0;              // the key position of token q0 (prefix: beyond every key)
    int blk0, nblk;        // key blocks
    int pieces, split, part, rows;
    int prefix;    // of a sequence's unit: the first unit of its group's prefix, or -1
    int group_q0;  // and that prefix's first token
    int pad[2];
};

struct SharedParams {
    CUtensorMap tm_q;   // 3-D over q [total_q, Hq, d], box {64, g, tpt}
    CUtensorMap tm_q1;  // the same with box {64, g, 1}
    CUtensorMap tm_k;   // 3-D over the cache [num_pages * page_size, Hkv, d], box {64, 1, box_rows}
    CUtensorMap tm_v;
    CUtensorMap tm_k64;  // the same with box {64, 1, min(box_rows, 64)}
    CUtensorMap tm_v64;
    const __nv_bfloat16* q;
    __nv_bfloat16* out;
    float* lse;
    float* part_lse;  // log2
    float* part_o;    // [parts, d]
    SharedHeader* header;
    int4* groups;    // [groups] (where shared memory does not hold them)
    int2* lengths;   // [units]: key blocks and rows (likewise)
    SharedUnit* units;  // those of prefixes, and from own_base on the sequences' own
    int2* items;        // {unit, piece << 16 | kv head}
    const int* cu_q;  // null: one query a sequence
    const int* seqlens;
    const int* block_table;
    const int* group_starts;
    const int* prefix_lens;
    unsigned* status;
    int batch, n_groups, total_q, max_seqlen_q, Hq, Hkv, g, tpt;
    int many;  // some unit may have many rows, as far as the host knows (else tm_q, tm_q1 are not there)
    int page_size, box_rows, max_pages, num_pages;
    int max_units, max_items, max_parts, own_base;
    int lse_head, lse_tok;  // strides of lse
    float scale_log2;
};

// CTAs for units with many rows, at most, and pieces that the work of units with few is cut into, about: two to an SM.
constexpr int kSharedShares = kGb300Sms, kSharedSmallShares = 2 * kGb300Sms;
constexpr int kSharedSmallRows = 16;  // the rows of a unit that count as few
constexpr int kSharedSmallSplit = 4;  // parts that their pieces leave

cudaError_t launch_shared_attn(const SharedParams& p, int head_dim, int num_sms, int own_units, cudaStream_t stream);
cudaError_t configure_shared_kernels();

}  // namespace attn
