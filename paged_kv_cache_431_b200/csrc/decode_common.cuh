// decode_common.cuh -- pieces shared by the decode kernels (16-bit and quantized pools).
#pragma once

#include "common.cuh"
#include "internal.h"

namespace pkv {

constexpr int kMaxPartTiles = 256;   // partition_tokens <= 4096
constexpr float kLog2e = 1.4426950408889634f;

// L2 cache hints of the decode kernels: the K/V stream is read once (evict_first), the
// split-K partials are read back by the merge soon after (evict_last).
#ifndef PKV_L2_HINTS
#define PKV_L2_HINTS 3
#endif
constexpr bool kHintKV = (PKV_L2_HINTS & 1) != 0;
constexpr bool kHintPartials = (PKV_L2_HINTS & 2) != 0;

// Ragged form (paged_cross_attn, paged_decode_attn_groups): a grid z index is an item, a run of
// query rows that share their keys.
//   kCross   item = sequence b: rows row_starts[b] .. row_starts[b+1]-1 against its own cached
//            tokens 0 .. ctx_lens[b]-1
//   kPrefix  item = group g: rows (sequences) row_starts[g] .. against the group's prefix, by
//            the table of its first sequence
//   kSuffix  item = sequence b of the grouped batch: its one row against the tokens from its
//            group's prefix to its context's end
// A KV head's query rows of an item are (row, head of the group), row major.
enum RaggedMode { kCross = 0, kPrefix = 1, kSuffix = 2 };

struct RaggedParams {
    int mode;
    const int32_t* row_starts;    // [items + 1]; kSuffix: [groups + 1]
    const int32_t* prefix_lens;   // [groups] (kPrefix, kSuffix)
    int items;                    // row_starts has items + 1 entries
    int total_rows, max_rows;     // rows of q; rows of an item that the grid covers
    int max_tokens;               // the caller's bound of an item's keys, in whole blocks (the grid covers it)
    int max_prefix;               // kPrefix, kSuffix: tokens of a prefix that the grid covers
    int pre_part;                 // kSuffix's merge: tokens per prefix partition
    int max_group;                // kSuffix: sequences of a group that the prefix pass covered
    int beside;                   // launched to run beside the kernel before it
    void* out16;                  // [total_rows][H_q][d] of q's dtype
};

struct DecodeParams {
    const void* q;
    const int32_t* tables;
    const int32_t* ctx_lens;
    const float* k_scale;
    const float* v_scale;
    float* out;
    float* ws_o;
    float* ws_ml;
    int32_t* status;
    int W, H_q, H_kv, G, N, part_tokens, max_parts;
    int num_seqs;
    // Partitions cover tokens tok_base .. ctx-1 and write workspace slots part_base + part of
    // a row of `slots`.  Plain decode: 0, 0, max_parts.  Shared-prefix (cascade) decode:
    // tok_base = prefix length, part_base = key splits of the prefix (slots 0 .. part_base-1
    // hold the prefix's partials).
    int tok_base, part_base, slots;
    int prefix_blocks;      // cascade: table entries every sequence must share with row 0
    int window;             // sliding window: tokens a query sees (0: the whole context)
    int hgroups;            // CTAs per KV head, 16 query heads each (G > 16 takes several)
    int q_bf16;             // q dtype: 1 bf16, 0 f16
    float scale_log2;
    int hold_tile;          // test hook: this CTA-local tile's copy is never issued (-1: none)
    long long wait_cycles;  // bound of every wait on a copy (SM cycles)
    RaggedParams rg;        // ragged form only
};

// Context length of sequence b, clamped to what the table and the grid can cover (with a
// window the grid covers any context: a query reads at most window + 15 tokens' blocks).
__device__ __forceinline__ int checked_ctx(const DecodeParams& p, int b, bool report)
{
    int ctx = p.ctx_lens[b];
    const int cap = p.window ? p.W * kBlock : min(p.W * kBlock, p.tok_base + p.max_parts * p.part_tokens);
    if (ctx < p.tok_base || ctx > cap) {
        if (report) flag_status(p.status, PKV_DEV_BAD_LENGTH);
        ctx = ctx < p.tok_base ? p.tok_base : cap;
    }
    return ctx;
}

// First token the query sees: ctx - window with a sliding window, else 0.
__device__ __forceinline__ int visible_lo(const DecodeParams& p, int ctx)
{
    return (p.window > 0 && ctx > p.window) ? ctx - p.window : 0;
}

// First token of partition 0: the prefix end (cascade), or the block holding visible_lo.
__device__ __forceinline__ int seq_base(const DecodeParams& p, int ctx)
{
    return p.window > 0 ? (visible_lo(p, ctx) & ~(kBlock - 1)) : p.tok_base;
}

// Partitions of this launch that sequence b's context needs.
__device__ __forceinline__ int part_count(const DecodeParams& p, int ctx)
{
    return (ctx - seq_base(p, ctx) + p.part_tokens - 1) / p.part_tokens;
}

// Workspace slot (row = b * H_q + h) of partition `part` of this launch.
__device__ __forceinline__ size_t ws_slot(const DecodeParams& p, size_t row, int part)
{
    return row * p.slots + p.part_base + part;
}

// An item of the ragged form: query rows row0 .. row0 + rows - 1 against tokens base .. end-1 of
// the sequence whose table is row `table`; `whole` when no other keys belong to these rows.
struct RaggedItem {
    int row0, rows, table, base, end;
    bool whole;
};

// Tokens of group g's prefix: whole blocks, within the table and the grid.
__device__ __forceinline__ int group_prefix(const RaggedParams& r, int W, int g, int32_t* status, bool report)
{
    int n = r.prefix_lens[g];
    const int cap = min(W * kBlock, r.max_prefix);
    if (n < 0 || n > cap) {
        if (report) flag_status(status, PKV_DEV_BAD_LENGTH);
        n = n < 0 ? 0 : cap;
    }
    if (n % kBlock) {
        if (report) flag_status(status, PKV_DEV_BAD_PREFIX);
        n -= n % kBlock;
    }
    return n;
}

// Rows of item i, clipped to q's rows and to what the grid covers (`report` flags a clip).
__device__ __forceinline__ void item_rows(const RaggedParams& r, int i, int& row0, int& rows, int32_t* status, bool report)
{
    const int a = r.row_starts[i], b = r.row_starts[i + 1];
    row0 = max(0, min(a, r.total_rows));
    rows = max(0, min(min(b, r.total_rows) - row0, r.max_rows));
    if (report && (a != row0 || b < a || b - a != rows)) flag_status(status, PKV_DEV_BAD_LENGTH);
}

// The item whose rows hold row t, or -1 (one whole warp asks).  The 32 lanes look at 32 items at
// a time, so that a batch of hundreds is a few independent loads.
__device__ __forceinline__ int item_of_row(const RaggedParams& r, int t)
{
    const int lane = threadIdx.x & 31;
    for (int i0 = 0; i0 < r.items; i0 += 32) {
        const int i = i0 + lane;
        const bool in = i < r.items && r.row_starts[i] <= t && t < r.row_starts[i + 1];
        const unsigned hit = __ballot_sync(0xffffffffu, in);
        if (hit) return i0 + __ffs(hit) - 1;
    }
    return -1;
}

// Item b of the launch (one whole warp asks).  rows 0: nothing to do.
__device__ __forceinline__ RaggedItem ragged_item(const RaggedParams& r, const int32_t* ctx_lens, int W, int b,
                                                  int32_t* status, bool report)
{
    RaggedItem it;
    it.base = 0;
    if (r.mode == kSuffix) {
        // a sequence of no group is padding; one past max_group was not covered (and was reported)
        int g = item_of_row(r, b);
        if (g >= 0 && b - r.row_starts[g] >= r.max_group) g = -1;
        it.row0 = it.table = b;
        it.rows = g >= 0 ? 1 : 0;
        it.end = g >= 0 ? ctx_lens[b] : 0;
        it.base = g >= 0 ? group_prefix(r, W, g, status, report) : 0;
        it.whole = it.base == 0;
    } else {
        item_rows(r, b, it.row0, it.rows, status, report);
        it.whole = r.mode == kCross;
        it.table = it.whole ? b : it.row0;
        it.end = it.rows == 0 ? 0 : it.whole ? ctx_lens[b] : group_prefix(r, W, b, status, report);
    }
    const int cap = min(W * kBlock, it.base + r.max_tokens);
    if (it.end < it.base || it.end > cap) {
        if (report) flag_status(status, PKV_DEV_BAD_LENGTH);
        it.end = it.end < it.base ? it.base : cap;
    }
    return it;
}

// The suffix pass of a grouped decode is launched to run beside its prefix pass (neither needs the
// other), and the merge after it waits only for its primary, the suffix grid.  So that grid has one
// more item, whose first block does nothing but wait for the prefix grid: the suffix grid is then
// complete only after the prefix grid is, its partials visible.  True for blocks of that item.
__device__ __forceinline__ bool ragged_beside(const RaggedParams& r)
{
    if (!r.beside || blockIdx.z != gridDim.z - 1) return false;
    if ((blockIdx.x | blockIdx.y) == 0) pdl_wait_primary();
    return true;
}

// Index (in rows of H_q heads, flattened) of the item's query row n of KV head g.
__device__ __forceinline__ size_t ragged_row(const RaggedItem& it, int G, int H_q, int g, int n)
{
    return (size_t)(it.row0 + n / G) * H_q + g * G + n % G;
}

// Four floats as 16-bit values of q's dtype.
__device__ __forceinline__ uint2 pack4(float4 v, bool bf16)
{
    return bf16 ? make_uint2(pack2<true>(v.x, v.y), pack2<true>(v.z, v.w))
                : make_uint2(pack2<false>(v.x, v.y), pack2<false>(v.z, v.w));
}

// Byte address of 16-byte chunk `c` of row `t` in a tile stored as 128-byte-wide TMA
// boxes of 16 rows with the 128-byte swizzle (chunk index XOR row % 8).
__device__ __forceinline__ uint32_t swz128(uint32_t tile, int t, int c)
{
    return tile + (uint32_t)((c >> 3) * (16 * 128) + t * 128 + (((c & 7) ^ (t & 7)) << 4));
}


// CUDA-core (FP32 FMA) decode for 16-bit pools (decode_simt.cu); f2 = packed fp32x2 FMA.
bool decode_simt_supported(int d, int G, int kv_dtype);
int launch_decode_simt(const DecodeParams& p, int kv_dtype, int G, bool f2, dim3 grid, cudaStream_t s,
                       const CUtensorMap* tmk, const CUtensorMap* tmv);

// tcgen05 decode for groups of 64 or 128 query heads (decode_tc.cu).
bool decode_tc_supported(int d, int G, int kv_dtype);
int launch_decode_tc(const DecodeParams& p, int kv_dtype, const CUtensorMap* tmq, const CUtensorMap* tmk,
                     const CUtensorMap* tmv, cudaStream_t s);

// tcgen05 decode for groups of 64 query heads with the keys on the MMA's M side (decode_tc_keys.cu).
bool decode_tck_supported(int d, int G, int kv_dtype);
bool make_q_map_seq(CUtensorMap* map, const void* q, int B, int H_q, PFN_encode enc);
int launch_decode_tck(const DecodeParams& p, int kv_dtype, const CUtensorMap* tmq, const CUtensorMap* tmk,
                      const CUtensorMap* tmv, cudaStream_t s);

// tcgen05 decode for fp8 pools with 8 query heads per KV head, codes fed to kind::f8f6f4
// MMAs (decode_tc_fp8.cu).
bool decode_tc_fp8_supported(int d, int G, int kv_dtype);
int launch_decode_tc_fp8(const DecodeParams& p, const CUtensorMap* tmk, const CUtensorMap* tmv, cudaStream_t s);

// Launch the quantized-pool decode kernel (decode_quant.cu).
int launch_decode_quant(const DecodeParams& p, int kv_dtype, int d, int nht, dim3 grid, cudaStream_t s,
                        const CUtensorMap* tmk, const CUtensorMap* tmv);
// tcgen05 kernel of the ragged form, one file per pool dtype (ragged_tc.cuh).
int launch_ragged_tc_bf16(const DecodeParams& p, int d, bool pair, int items, int max_rows, const CUtensorMap* tmk,
                          const CUtensorMap* tmv, cudaStream_t s);
int launch_ragged_tc_f16(const DecodeParams& p, int d, bool pair, int items, int max_rows, const CUtensorMap* tmk,
                         const CUtensorMap* tmv, cudaStream_t s);
int launch_ragged_tc_int8(const DecodeParams& p, int d, bool pair, int items, int max_rows, const CUtensorMap* tmk,
                          const CUtensorMap* tmv, cudaStream_t s);
int launch_ragged_tc_int4(const DecodeParams& p, int d, bool pair, int items, int max_rows, const CUtensorMap* tmk,
                          const CUtensorMap* tmv, cudaStream_t s);
int launch_ragged_tc_fp8(const DecodeParams& p, int d, bool pair, int items, int max_rows, const CUtensorMap* tmk,
                         const CUtensorMap* tmv, cudaStream_t s);

// The same kernels over ragged items (decode.cu, decode_quant.cu).
int launch_decode_quant_ragged(const DecodeParams& p, int kv_dtype, int d, int nht, dim3 grid, cudaStream_t s,
                               const CUtensorMap* tmk, const CUtensorMap* tmv);

}  // namespace pkv
