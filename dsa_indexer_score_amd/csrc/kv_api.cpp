// Host side of the paged key/value cache's C ABI (include/dsa_indexer.h):
// argument checks, the split along the keys, workspace sizes and launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "dsa_indexer.h"
#include "host_common.h"
#include "kv.h"

namespace {

using dsai::aligned;
using dsai::DeviceGuard;
using dsai::fail_hip;

int64_t round_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }
int64_t div_up(int64_t x, int64_t a) { return (x + a - 1) / a; }

int log2_page(int page)
{
    for (int s = 4; s <= 7; ++s)
        if (page == 1 << s) return s;
    return -1;
}

int check_cache(const indexer_kv_cache *c)
{
    if (!c || c->device < 0 || c->heads < 1 || c->d < 1 || c->page < 1 || c->pages < 1)
        return IDX_EINVAL;
    if (c->dtype != IDX_F32 && c->dtype != IDX_BF16 && c->dtype != IDX_FP8_E4M3) return IDX_EINVAL;
    if (c->dtype == IDX_F32 || (c->d != 64 && c->d != 128) || log2_page(c->page) < 0)
        return IDX_EUNSUPPORTED;
    if (c->pages > INT32_MAX || c->heads > 65535 ||
        c->pages * c->heads >= (int64_t)UINT32_MAX / c->page)
        return IDX_EUNSUPPORTED;  // rows are numbered in 32 bits
    const bool fp8 = c->dtype == IDX_FP8_E4M3;
    if (!c->k || !c->v || !aligned(c->k, 16) || !aligned(c->v, 16)) return IDX_EINVAL;
    if (fp8 ? !c->k_scale || !c->v_scale : c->k_scale || c->v_scale) return IDX_EINVAL;
    if (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4)) return IDX_EINVAL;
    return IDX_OK;
}

// Positions, and entries of a row, that a call may count: the kernels' loops run
// up to 2^17 past the last one in 32 bits.
constexpr int64_t kMaxKeys = (int64_t(1) << 31) - (int64_t(1) << 18);

// Sizes only: what the workspace functions may look at.
int check_seq_sizes(const indexer_kv_cache *c, const indexer_kv_seqs *s, int64_t rows)
{
    if (!s || s->nseq < 0 || s->table_width < 0 || rows < 0) return IDX_EINVAL;
    if (s->nseq > 0 && s->table_stride < s->table_width) return IDX_EINVAL;
    if (rows + 2 * (int64_t)s->nseq >= INT32_MAX ||
        (int64_t)s->table_width * c->page >= kMaxKeys)
        return IDX_EUNSUPPORTED;
    return IDX_OK;
}

int check_seqs(const indexer_kv_cache *c, const indexer_kv_seqs *s, int64_t rows)
{
    const int rc = check_seq_sizes(c, s, rows);
    if (rc != IDX_OK) return rc;
    if (s->nseq > 0 && (!s->cu_q || !s->seq_len || (s->table_width > 0 && !s->table)))
        return IDX_EINVAL;
    if (!aligned(s->cu_q, 4) || !aligned(s->seq_len, 4) || !aligned(s->table, 4)) return IDX_EINVAL;
    return IDX_OK;
}

// Rows of bf16 that the kernels read (or write) 16 bytes at a time.
bool rows_ok(const indexer_kv_rows *r)
{
    return r && r->ptr && aligned(r->ptr, 16) && r->row_stride >= 0 && r->head_stride >= 0 &&
           r->row_stride % 8 == 0 && r->head_stride % 8 == 0;
}

// Rows that are written must not share memory: one stride spans the other.
bool rows_apart(const indexer_kv_rows *r, int64_t rows, int64_t heads, int64_t d)
{
    if (rows <= 1) return heads <= 1 || r->head_stride >= d;
    if (heads <= 1) return r->row_stride >= d;
    return (r->head_stride >= d && r->row_stride >= (heads - 1) * r->head_stride + d) ||
           (r->row_stride >= d && r->head_stride >= (rows - 1) * r->row_stride + d);
}

// Bytes from the first element of a rows tensor to behind its last.
uintptr_t span(const indexer_kv_rows *r, int64_t rows, int64_t heads, int64_t d)
{
    return (uintptr_t)((rows - 1) * r->row_stride + (heads - 1) * r->head_stride + d) * 2;
}

bool overlap(const void *a, uintptr_t an, const void *b, uintptr_t bn)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + bn && y < x + an;
}

dsai::KvCache kernel_cache(const indexer_kv_cache *c, const indexer_kv_seqs *s)
{
    dsai::KvCache k{};
    k.k = c->k;
    k.v = c->v;
    k.k_scale = c->k_scale;
    k.v_scale = c->v_scale;
    k.pages = (uint32_t)c->pages;
    k.heads = c->heads;
    k.page_shift = log2_page(c->page);
    k.cu = s->cu_q;
    k.seq_len = s->seq_len;
    k.table = s->table;
    k.table_stride = s->table_stride;
    k.table_width = s->table_width;
    k.nseq = s->nseq;
    return k;
}

// How a call is cut into blocks; depends on host sizes only, so that the
// workspace functions and the calls agree.
struct Plan {
    bool tiles, shared;
    int64_t pass;             // slots of a launch
    int nt, head_tile, groups, tile_rows, nsplit, chunk;
    int64_t slots, part_ml, pick_n, pick_rows, bytes;
};

constexpr int64_t kCus = 256;
// Parts of a row's keys in the row kernel (microseconds of GPU time, e4m3, d =
// 128, 8 key heads).  Two blocks for each CU where single rows are few or parts
// are long, one otherwise: 4 rows of 4,096 keys 13.5 with 512 blocks, 15.0 with
// 256, but 16 rows of 4,096 keys 35.7 with 512, 32.3 with 256; 262,144 keys, one
// row, 105 with 512, 111 with 768.  Selected keys: one (4 rows of 4,096: 13.8
// with 256, 15.1 with 512).  A join costs what some 768 keys do: 16 rows of 1,024
// keys 12.6 in one part, 14.8 in two; one row of 1,024 11.5 in one part, 9.6 in
// eight.  A part of 128 keys is one round of a block's waves (one row of 2,048
// keys: 9.3 with 16 parts, 10.5 with 8); selected keys, which take longer to look
// up, go by 256 (11.0 with 16, 10.5 with 8).  64 rows of up to 16,384 keys: 258
// with parts of 4,096, 272 with 8,192, 264 with 2,048.
constexpr int64_t kFillBlocks = 512;
constexpr int64_t kFillWaves = 4096;
constexpr int64_t kMinChunk = 128, kMinPicked = 256;
constexpr int64_t kLongChunk = 4096, kFewUnits = 64;
constexpr int64_t kJoinKeys = 768;
// Columns (query rows of a sequence x query heads of a key head) up to which a
// sequence's rows go by blocks of 32 columns, straight from memory.
constexpr int64_t kFewCols = 64;
constexpr int kTilesHeads = 64;       // query heads of a key head in a block of 256 columns
// Lists of one launch's groups of rows: 256 MB, about 26,000 rows of 2,048
// positions; more rows take several launches.
constexpr int64_t kPickBytes = int64_t(1) << 28;
// Four rows share their selections rather than two where that fills 16 columns
// that two leave empty (2,048 rows x 2,048 of 65,536, 32 / 8 heads, e4m3: 283 us
// against 412), or, with 5 to 8 heads a key head, takes 32 columns in place of 16
// and leaves several rounds of blocks (64 / 8 heads: 420 against 426, bf16 509
// against 607; 777 rows of 4 key heads, one round: 93 against 90).
constexpr int64_t kManyBlocks = 2048;
constexpr int64_t kMinTileChunk = 512;

Plan make_plan(const indexer_kv_cache *c, int64_t S, int q_heads, int nseq, int64_t max_len,
               bool selected)
{
    Plan p{};
    const int group = q_heads / c->heads;
    const int64_t rows = selected ? 1 : div_up(S, std::max(nseq, 1));  // of a sequence, on average
    p.tiles = !selected && rows * group > kFewCols;
    const int cols = p.tiles ? dsai::kKvTileCols : dsai::kKvRowsCols;
    p.head_tile = std::min(group, p.tiles ? kTilesHeads : cols);
    p.groups = (int)div_up(group, p.head_tile);
    if (p.tiles) {
        p.tile_rows = cols / p.head_tile;
    } else {
        p.nt = (int)div_up(std::min<int64_t>(rows * p.head_tile, cols), 16);
        p.tile_rows = selected ? 1 : 16 * p.nt / p.head_tile;
    }
    p.slots = selected ? S : S / p.tile_rows + nseq;
    // row tiles with rows: a sequence's last one is not full
    const int64_t units = std::max(S / p.tile_rows, std::min<int64_t>(S, nseq)) * c->heads * p.groups;
    // Neighbouring rows share what they select: where 16 columns hold a row's
    // heads and such groups of rows alone fill the GPU.
    if (selected && group <= 16 && max_len <= dsai::kKvSharedWidth && S >= 2 * (int64_t)nseq &&
        S / 2 * c->heads >= kFillBlocks && c->pages * c->page <= (int64_t)UINT32_MAX) {
        p.shared = true;
        const bool four = group <= 4 || (group <= 8 && S / 4 * c->heads >= kManyBlocks);
        p.tile_rows = four && S >= 4 * (int64_t)nseq ? 4 : 2;
        p.nt = (int)div_up(p.tile_rows * group, 16);
        p.slots = S / p.tile_rows + nseq;
        const int64_t list = p.tile_rows * max_len, bits = p.tile_rows * div_up(list, 32) * 4;
        p.pass = std::min(p.slots, std::max<int64_t>(kPickBytes / (list * 4 + bits + 4), 1));
        p.nsplit = 1;
        p.chunk = INT32_MAX;
        p.pick_n = p.pass * list * 4;
        p.pick_rows = p.pick_n + p.pass * 4;
        p.bytes = p.pick_rows + p.pass * bits;
        return p;
    }
    const int64_t keys = std::max<int64_t>(max_len, 1);
    int64_t nsplit;
    if (p.tiles) {
        // The longest block should not outlast the others: parts of at most a
        // CU's share, less where two blocks run on a CU (d = 64), with rows that
        // are a sequence's last ones and see half of themselves on average.  One
        // prompt of 4,001 tokens (d = 64, 12 / 4 heads): 120 us in one part, 79 in
        // four; 4,096 rows over 16,384 keys (d = 128, 16 / 4 heads, as many blocks
        // as CUs): 580 in one, 617 in two.
        const int64_t seen = keys - std::min(rows, keys) / 2;
        const int64_t share = std::max<int64_t>(
            units * seen / kCus * (c->d == 64 ? 3 : 5) / 4, 1);
        nsplit = std::min(div_up(keys, share), keys / kMinTileChunk);
    } else {
        // parts that fill the GPU, where they save more than the join takes; among
        // several sequences parts of at most kLongChunk keys, so that the
        // longest does not trail the others
        const int64_t fill = !selected && units <= kFewUnits ? kFillBlocks : kCus;
        nsplit = std::max(std::min(fill / units, keys / (selected ? kMinPicked : kMinChunk)),
                          std::min(kFillBlocks / units, keys / kLongChunk));
        if (nsplit > 1 && keys - keys / nsplit < kJoinKeys) nsplit = 1;
        if (!selected && nseq > 1) nsplit = std::max(nsplit, keys / kLongChunk);
    }
    nsplit = std::max<int64_t>(nsplit, 1);
    int64_t chunk = round_up(div_up(keys, nsplit), 128);
    nsplit = div_up(keys, chunk);
    if (nsplit <= 1) nsplit = 1, chunk = INT32_MAX;
    p.nsplit = (int)nsplit;
    p.chunk = (int)chunk;
    p.pass = p.slots;
    if (nsplit > 1) {
        p.part_ml = round_up(nsplit * S * q_heads * c->d * 4, 256);
        p.bytes = p.part_ml + nsplit * S * q_heads * 8;
    }
    return p;
}

int check_attend_sizes(const indexer_kv_cache *c, const indexer_kv_seqs *s, int64_t S, int q_heads)
{
    int rc = check_cache(c);
    if (rc != IDX_OK) return rc;
    rc = check_seq_sizes(c, s, S);
    if (rc != IDX_OK) return rc;
    if (q_heads < 1 || q_heads % c->heads) return IDX_EINVAL;
    if (S * (int64_t)q_heads >= INT32_MAX) return IDX_EUNSUPPORTED;
    return IDX_OK;
}

int64_t most_keys(const indexer_kv_cache *c, const indexer_kv_seqs *s, int64_t max_len)
{
    const int64_t cap = (int64_t)s->table_width * c->page;
    return max_len > 0 && max_len < cap ? max_len : cap;
}

int attend(const indexer_kv_cache *c, const indexer_kv_seqs *s, const indexer_kv_rows *q,
           int64_t S, int q_heads, float scale, int causal, int64_t max_len, const int32_t *idx,
           int W, const int32_t *valid_len, const int32_t *idx0, void *out, float *lse,
           void *workspace, size_t workspace_bytes, void *stream)
{
    int rc = check_attend_sizes(c, s, S, q_heads);
    if (rc != IDX_OK) return rc;
    rc = check_seqs(c, s, S);
    if (rc != IDX_OK) return rc;
    const double c2 = std::fabs((double)scale) * 1.4426950408889634074;
    if (!std::isfinite((float)c2)) return IDX_EINVAL;
    if (S == 0 || s->nseq == 0) return IDX_OK;  // no row belongs to a sequence
    if (idx && W >= kMaxKeys) return IDX_EUNSUPPORTED;
    if (!rows_ok(q) || !out || !aligned(out, 16) || !aligned(lse, 4)) return IDX_EINVAL;
    // blocks read rows when others have written theirs
    const uintptr_t qn = span(q, S, q_heads, c->d), ln = lse ? (uintptr_t)S * q_heads * 4 : 0;
    const uintptr_t on = (uintptr_t)S * q_heads * c->d * 2;
    if (overlap(q->ptr, qn, out, on) || (lse && overlap(q->ptr, qn, lse, ln)) ||
        (lse && overlap(out, on, lse, ln)))
        return IDX_EINVAL;
    const Plan pl = make_plan(c, S, q_heads, s->nseq, idx ? W : most_keys(c, s, max_len),
                              idx != nullptr);
    // (in double: the product of the largest sizes passes 64 bits)
    if (((double)pl.slots * pl.nsplit * c->heads + 8) * pl.groups >= INT32_MAX)
        return IDX_EUNSUPPORTED;
    if (pl.bytes > 0 && (!workspace || workspace_bytes < (size_t)pl.bytes || !aligned(workspace, 16)))
        return IDX_EWORKSPACE;

    DeviceGuard guard(c->device);
    if (guard.err != hipSuccess) return fail_hip(guard.err);
    dsai::KvAttendParams p{};
    p.c = kernel_cache(c, s);
    p.q = static_cast<const uint16_t *>(q->ptr);
    p.q_tok = q->row_stride;
    p.q_head = q->head_stride;
    p.S = S;
    p.q_heads = q_heads;
    p.group = q_heads / c->heads;
    p.c2 = (float)c2;
    p.q_and = 0xffffffffu;
    p.q_xor = scale < 0.0f ? 0x80008000u : 0;
    if (p.c2 == 0.0f) p.c2 = 1.0f, p.q_and = 0;
    p.causal = causal;
    p.out = static_cast<uint16_t *>(out);
    p.lse = lse;
    p.idx = idx;
    p.W = W;
    p.valid_len = valid_len;
    p.idx0 = idx0;
    p.head_tile = pl.head_tile;
    p.groups = pl.groups;
    p.tile_rows = pl.tile_rows;
    p.chunk = pl.chunk;
    p.nsplit = pl.nsplit;
    p.part_o = static_cast<float *>(workspace);
    p.part_ml = reinterpret_cast<float2 *>(static_cast<char *>(workspace) + pl.part_ml);
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (pl.shared) {
        p.pick = static_cast<uint32_t *>(workspace);
        p.pick_n = reinterpret_cast<int *>(static_cast<char *>(workspace) + pl.pick_n);
        p.pick_rows = reinterpret_cast<uint32_t *>(static_cast<char *>(workspace) + pl.pick_rows);
    }
    for (p.slot0 = 0; p.slot0 < pl.slots; p.slot0 += pl.pass) {
        p.slots = std::min(pl.pass, pl.slots - p.slot0);
        hipError_t e = hipSuccess;
        if (pl.shared) e = dsai::launch_kv_pick(p, st);
        if (e != hipSuccess) return fail_hip(e);
        e = pl.tiles ? dsai::launch_kv_tiles(c->dtype, c->d, p, st)
                     : dsai::launch_kv_rows(c->dtype, c->d, pl.nt, p, st);
        if (e != hipSuccess) return fail_hip(e);
    }
    if (pl.nsplit > 1) {
        const hipError_t e = dsai::launch_kv_join(c->d, p, st);
        if (e != hipSuccess) return fail_hip(e);
    }
    return IDX_OK;
}

}  // namespace

extern "C" {

int indexer_kv_append(const indexer_kv_cache *c, const indexer_kv_seqs *s,
                      const indexer_kv_rows *k, const indexer_kv_rows *v, int64_t N,
                      const float *cos, const float *sin, int64_t rope_rows, int rot,
                      int interleaved, const indexer_kv_rows *q, int q_heads,
                      const indexer_kv_rows *q_out, void *stream)
{
    int rc = check_cache(c);
    if (rc != IDX_OK) return rc;
    rc = check_seqs(c, s, N);
    if (rc != IDX_OK) return rc;
    if (interleaved != 0 && interleaved != 1) return IDX_EINVAL;
    if (!cos != !sin) return IDX_EINVAL;
    if (cos) {
        if (rot < 2 || rot > c->d || rope_rows < 1) return IDX_EINVAL;
        if (rot % 16) return IDX_EUNSUPPORTED;
        if (!aligned(cos, 16) || !aligned(sin, 16)) return IDX_EINVAL;
    }
    if (q_heads < 0 || (q_heads > 0 && (!q || !q_out))) return IDX_EINVAL;
    if (N == 0 || s->nseq == 0) return IDX_OK;
    if (!rows_ok(k) || !rows_ok(v)) return IDX_EINVAL;
    if (q_heads > 0 && (!rows_ok(q) || !rows_ok(q_out) || !rows_apart(q_out, N, q_heads, c->d)))
        return IDX_EINVAL;
    if (q_heads > 0 &&
        (q->ptr != q_out->ptr || (N > 1 && q->row_stride != q_out->row_stride) ||
         (q_heads > 1 && q->head_stride != q_out->head_stride)) &&
        overlap(q->ptr, span(q, N, q_heads, c->d), q_out->ptr, span(q_out, N, q_heads, c->d)))
        return IDX_EINVAL;  // in place is fine, anything between is not

    dsai::KvAppendParams p{};
    p.c = kernel_cache(c, s);
    const indexer_kv_rows *src[3] = {k, v, q_heads > 0 ? q : nullptr};
    for (int i = 0; i < 3; ++i) {
        if (!src[i]) continue;
        p.src[i] = static_cast<const uint16_t *>(src[i]->ptr);
        p.tok_stride[i] = src[i]->row_stride;
        p.head_stride[i] = src[i]->head_stride;
    }
    if (q_heads > 0) {
        p.q_out = static_cast<uint16_t *>(q_out->ptr);
        p.qo_tok = q_out->row_stride;
        p.qo_head = q_out->head_stride;
    }
    p.cos = cos;
    p.sin = sin;
    p.rope_rows = rope_rows;
    p.rot = cos ? rot : 0;
    p.interleaved = interleaved;
    p.q_heads = q_heads;
    p.N = N;
    // A sequence of n new tokens touches at most n / page + 2 pages; with
    // page slots numbered from cu / page + 2 i, sequence i has that many.
    p.kv_blocks = (N / c->page + 2 * (int64_t)s->nseq) * div_up(c->heads, 4) * 2;
    // A wave turns up to eight steps of 512 / d heads of a token's queries; a few
    // tokens are spread over more waves (64 tokens x 64 heads: 9.7 us by 16
    // steps in one wave, 5.4 by one step each).
    const int64_t steps = div_up(q_heads, 512 / c->d);
    p.q_steps = 8;
    while (p.q_steps > 1 && N * div_up(steps, p.q_steps) < kFillWaves) p.q_steps /= 2;
    p.q_parts = (int)std::max<int64_t>(1, div_up(steps, p.q_steps));
    if (p.kv_blocks + N * p.q_parts >= INT32_MAX) return IDX_EUNSUPPORTED;
    DeviceGuard guard(c->device);
    if (guard.err != hipSuccess) return fail_hip(guard.err);
    const hipError_t e = dsai::launch_kv_append(c->dtype, c->d, p, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? IDX_OK : fail_hip(e);
}

int indexer_kv_attend_workspace_bytes(const indexer_kv_cache *c, const indexer_kv_seqs *s,
                                      int64_t S, int q_heads, int64_t max_len, size_t *bytes)
{
    if (!bytes || max_len < 0) return IDX_EINVAL;
    const int rc = check_attend_sizes(c, s, S, q_heads);
    if (rc != IDX_OK) return rc;
    *bytes = S > 0 && s->nseq > 0
                 ? (size_t)make_plan(c, S, q_heads, s->nseq, most_keys(c, s, max_len), false).bytes
                 : 0;
    return IDX_OK;
}

int indexer_kv_attend(const indexer_kv_cache *c, const indexer_kv_seqs *s,
                      const indexer_kv_rows *q, int64_t S, int q_heads, float scale, int causal,
                      int64_t max_len, void *out, float *lse, void *workspace,
                      size_t workspace_bytes, void *stream)
{
    if (max_len < 0 || (causal != 0 && causal != 1)) return IDX_EINVAL;
    return attend(c, s, q, S, q_heads, scale, causal, max_len, nullptr, 0, nullptr, nullptr, out,
                  lse, workspace, workspace_bytes, stream);
}

int indexer_kv_attend_selected_workspace_bytes(const indexer_kv_cache *c, const indexer_kv_seqs *s,
                                               int64_t S, int q_heads, int W, size_t *bytes)
{
    if (!bytes || W < 1) return IDX_EINVAL;
    const int rc = check_attend_sizes(c, s, S, q_heads);
    if (rc != IDX_OK) return rc;
    if (W >= kMaxKeys) return IDX_EUNSUPPORTED;
    *bytes = S > 0 && s->nseq > 0 ? (size_t)make_plan(c, S, q_heads, s->nseq, W, true).bytes : 0;
    return IDX_OK;
}

int indexer_kv_attend_selected(const indexer_kv_cache *c, const indexer_kv_seqs *s,
                               const indexer_kv_rows *q, int64_t S, int q_heads, float scale,
                               const int32_t *idx, int W, const int32_t *valid_len,
                               const int32_t *idx0, void *out, float *lse, void *workspace,
                               size_t workspace_bytes, void *stream)
{
    const bool none = S == 0 || (s && s->nseq == 0);    // no rows to select for
    if (W < 1 || (!none && (!idx || !valid_len)) || !aligned(idx, 4) || !aligned(valid_len, 4) ||
        !aligned(idx0, 4))
        return IDX_EINVAL;
    return attend(c, s, q, S, q_heads, scale, 0, 0, idx, W, valid_len, idx0, out, lse, workspace,
                  workspace_bytes, stream);
}

}  // extern "C"
