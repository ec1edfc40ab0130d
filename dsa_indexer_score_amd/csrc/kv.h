// Launch interface of the paged key/value cache: append and attention.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dsai {

// The cache and the sequences in it, as the kernels read them.  Rows of d
// elements are numbered (page * heads + head) * page_size + slot.
struct KvCache {
    void *k, *v;              // [pages, heads, page, d] bf16 or e4m3
    float *k_scale, *v_scale; // [pages, heads], e4m3 only
    uint32_t pages;
    int heads;
    int page_shift;           // log2 of the tokens per page
    const int32_t *cu;        // [nseq + 1] rows of this call, packed
    const int32_t *seq_len;   // [nseq]
    const int32_t *table;     // page ids, sequence i at table + i * table_stride
    int64_t table_stride;
    int table_width;
    int nseq;
};

struct KvAppendParams {
    KvCache c;
    const uint16_t *src[3];   // k, v, q: bf16, strides in elements
    int64_t tok_stride[3], head_stride[3];
    uint16_t *q_out;
    int64_t qo_tok, qo_head;
    const float *cos, *sin;   // [rope_rows, rot / 2], or null: no rotation
    int64_t rope_rows;
    int rot, interleaved;
    int q_heads;              // 0: no queries
    int64_t N;                // new tokens
    int q_steps, q_parts;     // steps of 512 channels by a wave, waves for a token's queries
    int64_t kv_blocks;        // blocks of pages, before those of queries
};

struct KvAttendParams {
    KvCache c;
    const uint16_t *q;        // bf16, [S, q_heads, d] with strides in elements
    int64_t q_tok, q_head;
    int64_t S;
    int q_heads, group;       // query heads in all, and per key head
    float c2;                 // |softmax scale| * log2(e), or 1 where that is 0
    uint32_t q_and, q_xor;    // the scale's sign, or its being 0, on pairs of query elements
    int causal;
    uint16_t *out;            // [S, q_heads, d] bf16
    float *lse;               // [S, q_heads] or null
    // selected positions: row t's entries at idx + t * W, valid_len[t] of them
    const int32_t *idx;
    int W;
    const int32_t *valid_len;
    const int32_t *idx0;      // [nseq] or null, subtracted from the entries
    // selected positions of tile_rows neighbouring rows, as launch_kv_pick writes
    // them (or null): per slot tile_rows * W entries, for each row of the slot a bit
    // for each entry (which it has), and the number of entries
    uint32_t *pick, *pick_rows;
    int *pick_n;
    // the split: `chunk` keys a block, nsplit blocks along the keys; rows that
    // need more than one leave (o, m, l) in part_o / part_ml for the join
    int head_tile, groups;    // query heads of a key head that a block takes, blocks for all
    int tile_rows;            // query rows of a sequence that one block takes
    int64_t slot0, slots;     // row tiles of the launch, empty ones among them
    int chunk, nsplit;
    float *part_o;            // [nsplit, S, q_heads, d]
    float2 *part_ml;          // [nsplit, S, q_heads]
};

hipError_t launch_kv_append(int dtype, int d, const KvAppendParams &p, hipStream_t st);

// Blocks of a launch: units (slot, split, key head) times groups.
__host__ __device__ inline int64_t kv_units(const KvAttendParams &p) { return p.slots * p.nsplit * p.c.heads; }
inline int64_t kv_blocks(const KvAttendParams &p)
{
    return p.groups == 1 ? kv_units(p) : (kv_units(p) + 7) / 8 * 8 * p.groups;
}

// nt: 16-column tiles of query rows x heads per block (1 or 2)
hipError_t launch_kv_rows(int dtype, int d, int nt, const KvAttendParams &p, hipStream_t st);
// 256 columns per block: many query rows
hipError_t launch_kv_tiles(int dtype, int d, const KvAttendParams &p, hipStream_t st);
// The lists of p.slots times tile_rows (2 or 4) rows (W at most kKvSharedWidth)
hipError_t launch_kv_pick(const KvAttendParams &p, hipStream_t st);
hipError_t launch_kv_join(int d, const KvAttendParams &p, hipStream_t st);

constexpr int kKvSharedWidth = 4096; // entries of a row that launch_kv_pick takes
constexpr int kKvSharedRows = 4;     // rows that share a list at most
constexpr int kKvRowsCols = 32;   // columns of a launch_kv_rows block at most
constexpr int kKvTileCols = 256;  // columns of a launch_kv_tiles block

}  // namespace dsai
