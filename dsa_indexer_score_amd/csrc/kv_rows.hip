// kv_rows: attention of a few query rows over the paged cache, all of a
// sequence's keys or the positions selected for the row.
//
//   o = sum_j softmax_j(scale q . k_j) v_j,   lse = log sum_j exp(scale q . k_j)
//
// One pass over the keys with a reference m and the sum l of each row; the scores
// are kept in base 2 (scale * log2 e, times the key page's scale, is one fp32
// factor on the exact bf16 products that the matrix unit sums in fp32).  m is the
// first tile's maximum, and a later one where a lane's 8 probabilities of a tile
// add up to more than 2^13: between these no maximum is computed (452 -> 434 us
// for the selections below).
//
// A block takes the query rows of one key head (up to 32 columns: rows of a
// sequence times the head's query heads) and a range of the keys; its four
// waves take turns at tiles of 32 keys, each with a softmax state of its own,
// joined through LDS at the end.  Nothing but the list of key rows is shared in
// the loop, so there is no barrier in it: keys and values go from memory through
// registers and a part of LDS of the wave's own to the matrix unit.  Both
// products are computed transposed, S^T = K Q^T and O^T = V^T P^T:
//  - the keys are the rows of A; lane (m, g) reads 16-byte chunks of key m, and
//    the contraction takes the channels in the order in which they come;
//  - S^T leaves lane (n, g) with the scores of column n against keys 4 g + i of
//    both halves of the tile, which is the B operand of the second product when
//    the contraction takes the keys in that order: P never leaves its lane;
//  - V^T needs, for a channel, the values of those eight keys: the transposing
//    LDS reads (ds_read_b64_tr_b8, _b16) give them; codes are widened exactly to
//    bf16.
// P is rounded to bf16 for the matrix unit after it took the value page's scale
// (relative 2^-8, as the rounding of the output); l sums the unrounded
// probabilities.
//
// Blocks that share a row (more keys than one chunk) write (o, m, l) to the
// workspace and join_kernel adds them up; the order is fixed, so results repeat.
//
// Bound by memory where keys are many: 262,144 keys of 8 heads (e4m3, d = 128)
// for one row of 64 heads take 98 us with the join, 5.5 TB/s (a large copy: 4.7);
// 64 rows of up to 16,384 keys 238 us, 4.7 TB/s.  With few keys it is the chain of
// dependent loads (sequence, page, row): 5.5 us for 128 keys, 0.9 us for each 128
// more in a block.  2,048 rows with 2,048 selected positions each (64 / 8 heads)
// take 434 us, with 32 / 8 heads 283: the vector unit, which widens 256 codes of a
// position for 32 columns (there 16), is busy for 55 % of it, the matrix unit for
// 22 %, and they overlap little.
#include "kv_common.h"

namespace dsai {
namespace {

constexpr int kList = 1024;             // keys resolved to rows at a time
constexpr uint32_t kNoPage = 0xffffffffu;
constexpr float kMost = 8192.0f;        // of a lane's probabilities of a tile against the reference
constexpr int kPickThreads = 512;
constexpr int kPickBits = 1 << 17;      // positions that a row's bitmap covers at a time
constexpr int kFewParts = 16;           // parts that one wave joins
constexpr float kLn2 = 0.693147180559945309f;

template <bool HI> __device__ inline uint32_t widen2(uint32_t w)
{
    auto v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI);
    return __builtin_bit_cast(uint32_t, v);
}

// A tile of 32 keys and values on its way: read from memory with neighbouring
// lanes on neighbouring 16-byte chunks of a row (the address unit takes four
// lanes at a time and one cache line for each), then through LDS, private to
// the wave, into the operands.
template <bool FP8, int D> struct Staged {
    static constexpr int RB = FP8 ? D : 2 * D;      // bytes of a row
    static constexpr int NCH = RB / 16;             // chunks of a row
    static constexpr int RL = 64 / NCH;             // rows of a load
    static constexpr int LD = 32 / RL;              // loads of a tile
    kvu4 k[LD], v[LD];

    // Chunk c of key row r lies at place c ^ swizzle(r), so that eight lanes
    // reading one chunk of eight neighbouring rows meet in no bank.
    __device__ static int swizzle(int r) { return NCH == 4 ? (r >> 2) & 3 : r & (NCH - 1); }
    // Value rows likewise, for the 16 lanes of a transposing read: one chunk of
    // keys 4 g .. 4 g + 3 and 16 + 4 g .. (8 bits), two of four keys (16 bits).
    __device__ static int value_swizzle(int r)
    {
        return FP8 ? NCH == 8 ? (r & 3) | (r >> 2 & 4) : r >> 4 & 1 : NCH == 16 ? (r & 3) << 1 : r & 2;
    }

    // off: byte offsets of the tile's rows; kb and vb point at the lane's chunk
    __device__ void load(const char *kb, const char *vb, const uint64_t *off, int lane)
    {
#pragma unroll
        for (int x = 0; x < LD; ++x) {
            const uint64_t o = off[x * RL + lane / NCH];
            k[x] = *reinterpret_cast<const kvu4 *>(kb + o);
            v[x] = *reinterpret_cast<const kvu4 *>(vb + o);
        }
    }
    // bad: rows that are not there; their values are 0, whatever was read
    __device__ void put(kvu4 *stage, uint32_t bad, int lane) const
    {
#pragma unroll
        for (int x = 0; x < LD; ++x) {
            const int r = x * RL + lane / NCH, c = lane % NCH;
            stage[r * NCH + (c ^ swizzle(r))] = k[x];
            kvu4 y = v[x];
            if (bad && (bad >> r & 1)) y = kvu4{0, 0, 0, 0};
            stage[(32 + r) * NCH + (c ^ value_swizzle(r))] = y;
        }
    }
};

// What a lane takes of a tile of 32 keys.
template <bool FP8, int D> struct Tile {
    static constexpr int ES = FP8 ? 1 : 2;
    static constexpr int KU = D * ES / 64;          // 16-byte chunks of a key
    static constexpr int KS = D / 32;               // contraction steps of S
    static constexpr int MT = D / 16;               // 16-channel tiles of O
    using ST = Staged<FP8, D>;
    kvu4 k[2][KU];

    __device__ void get_keys(const kvu4 *stage, int m, int g)
    {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int u = 0; u < KU; ++u)
                k[t][u] = stage[(16 * t + m) * ST::NCH + ((4 * u + g) ^ ST::swizzle(16 * t + m))];
    }
    __device__ kvb8 key(int t, int step) const
    {
        if constexpr (FP8) {
            const kvu4 x = k[t][step >> 1];
            const uint32_t a = step & 1 ? x.z : x.x, b = step & 1 ? x.w : x.y;
            const uint4 w = make_uint4(widen2<false>(a), widen2<true>(a), widen2<false>(b),
                                       widen2<true>(b));
            return __builtin_bit_cast(kvb8, w);
        } else {
            return __builtin_bit_cast(kvb8, k[t][step]);
        }
    }

    // Channel 16 t + m of the lane's eight keys.  The reads transpose: of 16
    // lanes each names 8 bytes, together 8 keys x 16 codes or 4 keys x 16 bf16
    // values, and each gets one column.
    __device__ static kvb8 value(const kvu4 *stage, int t, int m, int g)
    {
        typedef __attribute__((address_space(3))) const char *Lds;
        if constexpr (FP8) {
            typedef int W2 __attribute__((ext_vector_type(2)));
            typedef __attribute__((address_space(3))) W2 *P;
            const int j = m >> 1, r = 16 * (j >> 2) + 4 * g + (j & 3);
            const kvu4 *at = stage + (32 + r) * ST::NCH + (t ^ ST::value_swizzle(r));
            const W2 w = __builtin_amdgcn_ds_read_tr8_b64_v2i32((P)((Lds)at + 8 * (m & 1)));
            const uint4 y = make_uint4(widen2<false>(w[0]), widen2<true>(w[0]), widen2<false>(w[1]),
                                       widen2<true>(w[1]));
            return __builtin_bit_cast(kvb8, y);
        } else {
            typedef short W4 __attribute__((ext_vector_type(4)));
            typedef __attribute__((address_space(3))) W4 *P;
            W4 w[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = 16 * h + 4 * g + (m >> 2), c = 2 * t + (m >> 1 & 1);
                const kvu4 *at = stage + (32 + r) * ST::NCH + (c ^ ST::value_swizzle(r));
                w[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)((Lds)at + 8 * (m & 1)));
            }
            typedef short W8 __attribute__((ext_vector_type(8)));
            const W8 y = __builtin_shufflevector(w[0], w[1], 0, 1, 2, 3, 4, 5, 6, 7);
            return __builtin_bit_cast(kvb8, y);
        }
    }
};

// What the rows of a block attend to: all of the sequence's tokens, one row's
// selected positions, or the selections of a few neighbouring rows as pick_kernel
// put them together (each position once, with the rows that have it).
enum { kAll = 0, kSelected = 1, kShared = 2 };

// Three blocks a CU where registers allow it and the keys come from the L2 (few
// rows' selections: 752 us with three against 839 with two); streaming
// all keys from memory two do better (99 against 105 us over 262,144 keys).
template <bool FP8, int D, int NT, int MODE>
__global__ __launch_bounds__(256, MODE != kAll && NT == 1 && FP8 ? 3 : 2)
void rows_kernel(KvAttendParams p)
{
    constexpr bool SEL = MODE == kSelected, ALL = MODE == kAll, SHARED = MODE == kShared;
    using TL = Tile<FP8, D>;
    using ST = typename TL::ST;
    constexpr int MT = TL::MT;
    constexpr int PITCH = D + 4;
    struct List {
        uint64_t off[kList];            // byte offsets of the keys' rows
        float ks[FP8 ? kList : 4], vs[FP8 ? kList : 4];
        uint32_t bad[kList / 32];       // which of a tile's keys are not there
        uint32_t has[SHARED ? kKvSharedRows : 1][kList / 32];  // which of them a row has
    };
    struct Join { float o[4][16][PITCH]; };
    struct Work { List list; kvu4 stage[4][64 * ST::NCH]; };
    __shared__ __align__(16) union { Work work; Join join; } smem;
    Work &sm = smem.work;
    __shared__ float sm_m[4][16 * NT], sm_l[4][16 * NT];

    const KvCache &kc = p.c;
    const int tid = threadIdx.x, wave = uniform(tid >> 6), lane = tid & 63;
    const int n = lane & 15, g = lane >> 4;

    // ---- which rows, key head, query heads and keys
    const int gsize = p.head_tile;
    const BlockAt blk = block_at(p);
    if (blk.none) return;
    const int head = blk.head, grp = blk.grp, split = blk.split;
    const int64_t slot = p.slot0 + blk.slot;

    // The selection comes while the sequence is looked up: entries of the list
    // before it is known how many count (they lie in the row all the same).
    const int e0 = split * p.chunk;
    uint32_t raw[kList / 256];           // selected positions, or picked cache slots
    uint32_t row_has = 0;                // 32 of them, bit by bit, for thread / 32's row
    const int row_words = (p.tile_rows * p.W + 31) >> 5;
    const int held = SEL ? p.W : p.tile_rows * p.W;
    const int64_t entry0 = (SEL ? slot : blk.slot) * held;
    const uint32_t *given = SEL ? reinterpret_cast<const uint32_t *>(p.idx) : p.pick;
    auto fetch = [&](int s0, int end) KV_INLINE {
#pragma unroll
        for (int k = 0; k < kList / 256; ++k) {
            const int i = s0 + tid + 256 * k;
            raw[k] = i < end ? given[entry0 + i] : 0;
        }
        if constexpr (SHARED) {
            const int r = tid >> 5, w = (s0 >> 5) + (tid & 31);
            if (r < p.tile_rows && w < row_words)
                row_has = p.pick_rows[(blk.slot * p.tile_rows + r) * row_words + w];
        }
    };
    int count = 0;
    if constexpr (SEL) count = p.valid_len[slot];
    if constexpr (SHARED) count = p.pick_n[blk.slot];
    if constexpr (!ALL) fetch(e0, held);

    const int R = SEL ? 1 : p.tile_rows;
    const Seq sq = find_seq(kc, p.S, slot, R, SEL ? 0 : 1);
    const int seq = sq.i, c0 = sq.c0;
    const int rows_in_seq = sq.c1 - sq.c0;
    const int64_t t0 = SEL ? slot - c0 : (slot - (c0 / R + (int64_t)seq)) * R;
    if (t0 < 0 || t0 >= rows_in_seq) return;
    const int ntok = (int)(rows_in_seq - t0 < R ? rows_in_seq - t0 : R);
    const int len = clamped(sq.len, (int64_t)kc.table_width << kc.page_shift);
    const int64_t row0 = c0 + t0;
    // entries: keys 0 .. entries of the sequence, or of the row's selection
    int entries, base = 0;
    if constexpr (SEL) {
        entries = clamped(count, p.W);
        base = p.idx0 ? p.idx0[seq] : 0;
    } else if constexpr (SHARED) {
        entries = count;
    } else {
        const int64_t last = p.causal ? (int64_t)len - rows_in_seq + t0 + ntok : len;
        entries = clamped(last < 0 ? 0 : (int)last, len);
    }
    if (split > 0 && e0 >= entries) return;
    const int e1 = entries - e0 < p.chunk ? entries : e0 + p.chunk;

    // ---- the columns: query rows x heads
    kvb8 q[NT][TL::KS];
    int lim[NT], has[NT];        // the column sees no entries from lim on; its row
    int minlim = 0x7fffffff;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int col = 16 * t + n, tok = col / gsize, hh = grp * gsize + col % gsize;
        const bool in = tok < ntok && hh < p.group;
        lim[t] = 0x7fffffff;
        has[t] = tok < ntok ? tok : 0;     // of no use where the block has no such row
        if constexpr (ALL) {
            if (in && p.causal) {
                const int64_t x = (int64_t)len - rows_in_seq + t0 + tok + 1;
                lim[t] = x < 0 ? 0 : (int)x;
            }
        }
        minlim = lim[t] < minlim ? lim[t] : minlim;
        const uint16_t *src = p.q + (row0 + tok) * p.q_tok +
                              (int64_t)(head * p.group + hh) * p.q_head;
#pragma unroll
        for (int s = 0; s < TL::KS; ++s) {
            // the channels that the key operand of this step holds
            const int at = FP8 ? 64 * (s >> 1) + 16 * g + 8 * (s & 1) : 32 * s + 8 * g;
            uint4 x = make_uint4(0, 0, 0, 0);
            if (in) x = *reinterpret_cast<const uint4 *>(src + at);
            x = signed_queries(x, p.q_and, p.q_xor);
            q[t][s] = __builtin_bit_cast(kvb8, x);
        }
    }
#pragma unroll
    for (int s = 1; s < 16; s <<= 1) {
        const int o = __shfl_xor(minlim, s);
        minlim = o < minlim ? o : minlim;
    }
    minlim = uniform(minlim);

    // The reference that the probabilities are taken against, once a key was seen.
    kvf4 o[NT][MT];
    float ref[NT], l[NT];
    bool seen[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        ref[t] = 0.0f;
        seen[t] = false;
        l[t] = 0.0f;
#pragma unroll
        for (int i = 0; i < MT; ++i) o[t][i] = kvf4{0, 0, 0, 0};
    }

    const char *kb = static_cast<const char *>(kc.k) + lane % ST::NCH * 16;
    const char *vb = static_cast<const char *>(kc.v) + lane % ST::NCH * 16;
    kvu4 *stage = sm.stage[wave];
    const int page_mask = (1 << kc.page_shift) - 1;
    const int32_t *table = kc.table + (int64_t)seq * kc.table_stride;

    // The staged tile of 32 keys, s0 + at .. s0 + at + 31 of the entries.
    auto process = [&](int s0, int at) KV_INLINE {
        TL cur;
        cur.get_keys(stage, n, g);
        const uint32_t bad = SHARED ? 0 : (uint32_t)uniform((int)sm.list.bad[at >> 5]);
        const bool edge = ALL && s0 + at + 32 > minlim;
        float ks[8], vs[8];
        auto factors = [&](const float *list, float (&f)[8]) KV_INLINE {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float4 a = *reinterpret_cast<const float4 *>(list + at + 16 * h + 4 * g);
                f[4 * h] = a.x; f[4 * h + 1] = a.y; f[4 * h + 2] = a.z; f[4 * h + 3] = a.w;
            }
        };
        if constexpr (FP8) factors(sm.list.ks, ks);
        uint4 pk[NT];
        kvf4 acc[NT][2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int s = 0; s < TL::KS; ++s) {
                const kvb8 a = cur.key(h, s);
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    acc[t][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        a, q[t][s], s ? acc[t][h] : kvf4{0, 0, 0, 0}, 0, 0, 0);
            }
        __builtin_amdgcn_sched_barrier(0);   // values after the scores: registers are short
        if constexpr (FP8) factors(sm.list.vs, vs);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[j] = __builtin_fmaf(acc[t][j >> 2][j & 3], FP8 ? ks[j] : p.c2, -ref[t]);
            if constexpr (SHARED) {
                const uint32_t own = sm.list.has[has[t]][at >> 5];
                if (__ballot(own != ~0u)) {
                    const uint32_t cut = ~own >> (4 * g);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {   // all ones where the row has no such key
                        const uint32_t no = __builtin_amdgcn_sbfe(cut, 16 * (j >> 2) + (j & 3), 1);
                        x[j] = __uint_as_float((__float_as_uint(x[j]) & ~no) | (0xff800000u & no));
                    }
                }
            } else if (bad || edge) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int key = 16 * (j >> 2) + 4 * g + (j & 3);
                    if ((bad >> key & 1) || (ALL && s0 + at + key >= lim[t])) x[j] = -__builtin_inff();
                }
            }
            float y[8], sum;
            auto probabilities = [&]() KV_INLINE {
                sum = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    y[j] = __builtin_amdgcn_exp2f(x[j]);
                    sum += y[j];
                }
            };
            bool again = __ballot(!seen[t]) != 0;
            if (!again) {
                probabilities();
                again = __ballot(sum > kMost) != 0;
            }
            if (again) {                 // a new reference: the maximum, if it is more
                float top = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])),
                                  fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
                top = max_over_rows(top);
                const bool some = top > -__builtin_inff();
                const float up = seen[t] ? fmaxf(top, 0.0f) : some ? top : 0.0f;
                const float a = __builtin_amdgcn_exp2f(seen[t] ? -up : 0.0f);
                ref[t] += up;
                seen[t] |= some;
                l[t] *= a;
#pragma unroll
                for (int i = 0; i < MT; ++i) o[t][i] *= a;
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] -= up;
                probabilities();
            }
            l[t] += sum;
            if constexpr (FP8) {
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] *= vs[j];
            }
            pk[t] = make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]),
                               pack_bf16(y[6], y[7]));
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const kvb8 a = TL::value(stage, i, n, g);
#pragma unroll
            for (int t = 0; t < NT; ++t)
                o[t][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    a, __builtin_bit_cast(kvb8, pk[t]), o[t][i], 0, 0, 0);
        }
    };

    for (int s0 = e0; s0 < e1; s0 += kList) {
        // ---- resolve up to kList entries to cache rows and their scales
        const int cnt = e1 - s0 < kList ? e1 - s0 : kList;
        const int padded = (cnt + 31) & ~31;
        if (s0 > e0) __syncthreads();
        int64_t pos[kList / 256];
        uint32_t id[kList / 256];
        bool there[kList / 256];
#pragma unroll
        for (int k = 0; k < kList / 256; ++k) {
            const int i = tid + 256 * k;
            there[k] = i < cnt;
            pos[k] = s0 + i;
            if constexpr (SEL) {
                pos[k] = (int64_t)(int)raw[k] - base;
                there[k] = there[k] && pos[k] >= 0 && pos[k] < len;
            }
            if constexpr (SHARED) pos[k] = raw[k];
        }
#pragma unroll
        for (int k = 0; k < kList / 256; ++k) {
            if constexpr (SHARED)
                id[k] = there[k] ? (uint32_t)(pos[k] >> kc.page_shift) : kNoPage;
            else
                id[k] = there[k] ? (uint32_t)table[pos[k] >> kc.page_shift] : kNoPage;
        }
        float ks[FP8 ? kList / 256 : 1], vs[FP8 ? kList / 256 : 1];
#pragma unroll
        for (int k = 0; k < kList / 256; ++k) {
            const int i = tid + 256 * k;
            there[k] = id[k] < kc.pages;
            const uint32_t unit = there[k] ? id[k] * (uint32_t)kc.heads + head : 0;
            const uint64_t row = ((uint64_t)unit << kc.page_shift) +
                                 (there[k] ? (int)pos[k] & page_mask : 0);
            if (i < padded) sm.list.off[i] = row * (uint64_t)(D * TL::ES);
            if constexpr (FP8) {
                ks[k] = there[k] ? kc.k_scale[unit] : 0.0f;
                vs[k] = there[k] ? kc.v_scale[unit] : 0.0f;
            }
            const uint64_t bad = __ballot(!there[k]);
            if (lane == 0) {
                sm.list.bad[i >> 5] = (uint32_t)bad;
                sm.list.bad[(i >> 5) + 1] = (uint32_t)(bad >> 32);
            }
        }
        if constexpr (SHARED)
            if (tid >> 5 < kKvSharedRows) sm.list.has[tid >> 5][tid & 31] = row_has;
        __syncthreads();

        // ---- tiles of 32 keys, in turn over the waves, the next one's loads ahead
        // (the first one's along with the scales and the next list's entries)
        ST next;
        int at = wave * 32;
        if (at < padded) next.load(kb, vb, sm.list.off + at, lane);
        if constexpr (!ALL)
            if (s0 + kList < e1) fetch(s0 + kList, e1);
        if constexpr (FP8) {
#pragma unroll
            for (int k = 0; k < kList / 256; ++k) {
                const int i = tid + 256 * k;
                if (i < padded) {
                    sm.list.ks[i] = ks[k] * p.c2;
                    sm.list.vs[i] = vs[k];
                }
            }
            __syncthreads();
        }
        for (; at < padded; at += 128) {
            next.put(stage, (uint32_t)uniform((int)sm.list.bad[at >> 5]), lane);
            if (at + 128 < padded) next.load(kb, vb, sm.list.off + at + 128, lane);
            process(s0, at);
        }
    }

    // ---- join the waves
    float f[NT], mx[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        mx[t] = seen[t] ? ref[t] : -__builtin_inff();
        l[t] += __shfl_xor(l[t], 16);
        l[t] += __shfl_xor(l[t], 32);
        if (g == 0) {
            sm_m[wave][16 * t + n] = mx[t];
            sm_l[wave][16 * t + n] = l[t];
        }
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int col = 16 * t + n;
        const float m4 = fmaxf(fmaxf(sm_m[0][col], sm_m[1][col]), fmaxf(sm_m[2][col], sm_m[3][col]));
        f[t] = mx[t] == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(mx[t] - m4);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        if (t > 0) __syncthreads();
#pragma unroll
        for (int w = 0; w < MT; ++w) {
            const kvf4 x = o[t][w] * f[t];
            *reinterpret_cast<kvf4 *>(&smem.join.o[wave][n][16 * w + 4 * g]) = x;
        }
        __syncthreads();
        // thread: column tid / 16, D / 16 channels
        constexpr int C = D / 16;
        const int cl = tid >> 4, ch = (tid & 15) * C, col = 16 * t + cl;
        const int tok = col / gsize, hh = grp * gsize + col % gsize;
        if (tok < ntok && hh < p.group) {
            float m4 = sm_m[0][col];
#pragma unroll
            for (int w = 1; w < 4; ++w) m4 = fmaxf(m4, sm_m[w][col]);
            float sum = 0.0f, y[C];
#pragma unroll
            for (int j = 0; j < C; ++j) y[j] = 0.0f;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                if (sm_m[w][col] != -__builtin_inff())
                    sum += sm_l[w][col] * __builtin_amdgcn_exp2f(sm_m[w][col] - m4);
#pragma unroll
                for (int j = 0; j < C; ++j) y[j] += smem.join.o[w][cl][ch + j];
            }
            const int64_t out = (row0 + tok) * p.q_heads + head * p.group + hh;
            // the row's own keys decide whether other blocks have a part of it
            int own = entries;
            if constexpr (ALL) {
                if (p.causal) {
                    const int64_t x = (int64_t)len - rows_in_seq + t0 + tok + 1;
                    own = x < 0 ? 0 : x < len ? (int)x : len;
                }
            }
            if (own <= p.chunk) {
                if (split == 0) {
                    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
                    for (int j = 0; j < C; j += 2)
                        *reinterpret_cast<uint32_t *>(p.out + out * D + ch + j) =
                            pack_bf16(y[j] * inv, y[j + 1] * inv);
                    if (p.lse && ch == 0)
                        p.lse[out] = sum > 0.0f ? (m4 + __builtin_amdgcn_logf(sum)) * kLn2
                                                : -__builtin_inff();
                }
            } else {
                const int64_t part = (int64_t)split * p.S * p.q_heads + out;
#pragma unroll
                for (int j = 0; j < C; j += 4)
                    *reinterpret_cast<float4 *>(p.part_o + part * D + ch + j) =
                        make_float4(y[j], y[j + 1], y[j + 2], y[j + 3]);
                if (ch == 0) p.part_ml[part] = make_float2(m4, sum);
            }
        }
    }
}

// One block joins the parts of one (row, head): D / 4 threads a part, as many
// parts at a time as T threads hold and those eight deep; each thread adds its
// parts in order and the threads of a channel are added in order.  Bound by
// latency: with 256 threads 64 parts are one round of loads (24 -> 5.9 us for 64
// rows x heads of 64 parts against one wave each), with 64 threads few parts
// keep fewer waves (4,096 rows x heads of at most 4 parts: 9.2 -> 5.5 us).
template <int D, bool SEL, int T>
__global__ __launch_bounds__(T) void join_kernel(KvAttendParams p)
{
    constexpr int TP = D / 4, NG = T / TP;
    __shared__ float sm_y[NG][D + 4];
    __shared__ float sm_m[4], sm_l[NG];
    const KvCache &kc = p.c;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int64_t unit = blockIdx.x;
    const int64_t row = unit / p.q_heads;
    const Seq sq = find_seq(kc, p.S, row, 1, 0);
    const int c0 = sq.c0, c1 = sq.c1;
    if (row < c0 || row >= c1) return;
    int own;
    if constexpr (SEL) {
        own = clamped(p.valid_len[row], p.W);
    } else {
        const int len = clamped(sq.len, (int64_t)kc.table_width << kc.page_shift);
        const int64_t x = p.causal ? (int64_t)len - (c1 - c0) + (row - c0) + 1 : len;
        own = x < 0 ? 0 : x < len ? (int)x : len;
    }
    if (own <= p.chunk) return;                     // written by its one block
    int parts = (own - 1) / p.chunk + 1;            // own + chunk may pass 32 bits
    parts = parts < p.nsplit ? parts : p.nsplit;
    const int64_t step = p.S * p.q_heads;
    float m = -__builtin_inff();
    for (int s = tid; s < parts; s += T) m = fmaxf(m, p.part_ml[s * step + unit].x);
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) m = fmaxf(m, __shfl_xor(m, x));
    if constexpr (T > 64) {
        if (lane == 0) sm_m[wave] = m;
        __syncthreads();
        m = fmaxf(fmaxf(sm_m[0], sm_m[1]), fmaxf(sm_m[2], sm_m[3]));
    }
    const int grp = tid / TP, ch = tid % TP * 4;
    float l = 0.0f, y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (m != -__builtin_inff()) {
#pragma unroll 8
        for (int s = grp; s < parts; s += NG) {
            const float2 ml = p.part_ml[s * step + unit];
            const float4 x = *reinterpret_cast<const float4 *>(p.part_o + (s * step + unit) * D + ch);
            const float w = __builtin_amdgcn_exp2f(ml.x - m);
            l += w * ml.y;
            y[0] += w * x.x;
            y[1] += w * x.y;
            y[2] += w * x.z;
            y[3] += w * x.w;
        }
    }
    *reinterpret_cast<float4 *>(&sm_y[grp][ch]) = make_float4(y[0], y[1], y[2], y[3]);
    if (ch == 0) sm_l[grp] = l;
    __syncthreads();
    if (tid >= D / 2) return;
    float sum = 0.0f, a = 0.0f, b = 0.0f;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        sum += sm_l[g];
        a += sm_y[g][2 * tid];
        b += sm_y[g][2 * tid + 1];
    }
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    *reinterpret_cast<uint32_t *>(p.out + unit * D + 2 * tid) = pack_bf16(a * inv, b * inv);
    if (p.lse && tid == 0)
        p.lse[unit] = sum > 0.0f ? (m + __builtin_amdgcn_logf(sum)) * kLn2 : -__builtin_inff();
}

// The selections of R neighbouring rows of a sequence as one list of cache slots
// (page id * page size + slot), each with the rows that have it: first what all
// of them have, then row by row what no row before has, in the rows' order.  The
// rows then share what rows_kernel reads and widens of a common position, and
// all key heads share the looking up of pages.  Which rows have a position is
// read from their bitmaps in LDS, kPickBits positions at a time; rows that name
// a position twice share nothing.  Positions out of the sequence and on pages
// that do not exist are dropped.
//
// KM: entries of a row and thread.  Bound by latency, so two blocks a CU where
// the entries leave the registers for it (512 blocks of four rows of 2,048
// positions: 25 us, with KM = 8, one block a CU, 43).
template <int R, int KM>
__global__ __launch_bounds__(kPickThreads, R * KM <= 20 ? 4 : 2)
void pick_kernel(KvAttendParams p)
{
    static_assert(KM * kPickThreads <= kPickBits / 8, "the entries' rows go where the bitmaps were");
    static_assert(KM * 4 <= 32 && R <= 4, "the rows that have a thread's entries: 4 bits each");
    typedef uint32_t Words __attribute__((ext_vector_type(R)));
    __shared__ __align__(16) Words sm_bits[kPickBits / 32 + 4];
    __shared__ int sm_cnt[R + 1][64];
    __shared__ int sm_odd[8];
    uint32_t *words = reinterpret_cast<uint32_t *>(sm_bits);
    const KvCache &kc = p.c;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int64_t slot = p.slot0 + blockIdx.x;
    const Seq sq = find_seq(kc, p.S, slot, R, 1);
    const int seq = sq.i, c0 = sq.c0, c1 = sq.c1;
    const int64_t t0 = (slot - (c0 / R + (int64_t)seq)) * R;
    if (t0 < 0 || t0 >= c1 - c0) return;
    const int len = clamped(sq.len, (int64_t)kc.table_width << kc.page_shift);
    const int64_t row0 = c0 + t0;
    const int rows = (int)(c1 - c0 - t0 < R ? c1 - c0 - t0 : R);
    const int most = len > 0 ? p.W : 0;   // no token: nothing to look up
    int cnt[R], some = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        cnt[r] = r < rows ? clamped(p.valid_len[row0 + r], most) : 0;
        some += cnt[r] > 0;
    }
    const int base = p.idx0 ? p.idx0[seq] : 0;
    const int32_t *table = kc.table + (int64_t)seq * kc.table_stride;

    int pos[R][KM];                     // -1: no such position
    uint32_t at[R][KM];                 // its cache slot
    uint32_t here[R] = {};              // bit k: entry tid + 512 k has one
    uint32_t with[R] = {};              // bits 4 k ..: the rows that have it
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int32_t *src = p.idx + (row0 + (r < rows ? r : 0)) * p.W;
        const int last = cnt[r] > 0 ? cnt[r] - 1 : 0;   // loads without branches between them
#pragma unroll
        for (int k = 0; k < KM; ++k) {
            if (kPickThreads * k >= cnt[r]) continue;
            const int i = tid + kPickThreads * k;
            pos[r][k] = src[i < last ? i : last];
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int k = 0; k < KM; ++k) {
            at[r][k] = 0xffffffffu;
            if (kPickThreads * k >= cnt[r]) {
                pos[r][k] = -1;
                continue;
            }
            const int64_t x = (int64_t)pos[r][k] - base;
            const bool in = tid + kPickThreads * k < cnt[r] && x >= 0 && x < len;
            pos[r][k] = in ? (int)x : -1;
            at[r][k] = (uint32_t)table[in ? x >> kc.page_shift : 0];
        }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int k = 0; k < KM; ++k) {
            if (at[r][k] >= kc.pages) pos[r][k] = -1;
            if (pos[r][k] >= 0) here[r] |= 1u << k;
            at[r][k] = (at[r][k] << kc.page_shift) +
                       ((uint32_t)pos[r][k] & ((1u << kc.page_shift) - 1));
        }

    bool twice = false;
    if (some > 1) {
        for (int w0 = 0; w0 < len; w0 += kPickBits) {
            if (w0 > 0) __syncthreads();
            const int bits = len - w0 < kPickBits ? len - w0 : kPickBits;
            for (int i = tid; i < (bits + 31) / 32 * R / 4 + 1; i += kPickThreads)
                reinterpret_cast<uint4 *>(sm_bits)[i] = make_uint4(0, 0, 0, 0);
            __syncthreads();
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int k = 0; k < KM; ++k) {
                    const uint32_t x = (uint32_t)(pos[r][k] - w0);
                    if (kPickThreads * k < cnt[r] && pos[r][k] >= 0 && x < (uint32_t)kPickBits)
                        twice |= atomicOr(&words[(x >> 5) * R + r], 1u << (x & 31)) >> (x & 31) & 1;
                }
            __syncthreads();
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int k = 0; k < KM; ++k) {
                    const uint32_t x = (uint32_t)(pos[r][k] - w0);
                    if (kPickThreads * k < cnt[r] && pos[r][k] >= 0 && x < (uint32_t)kPickBits) {
                        const Words w = sm_bits[x >> 5];
                        uint32_t m = 0;
#pragma unroll
                        for (int o = 0; o < R; ++o) m |= (w[o] >> (x & 31) & 1) << o;
                        with[r] |= m << (4 * k);
                    }
                }
        }
    }
    const bool any = __ballot(twice) != 0;
    if (lane == 0) sm_odd[wave] = any;
    __syncthreads();
    bool apart = some <= 1;
#pragma unroll
    for (int w = 0; w < 8; ++w) apart |= sm_odd[w] != 0;
    __syncthreads();
    const uint32_t full = (1u << rows) - 1;
    uint32_t list[R + 1] = {};          // bit k: entry tid + 512 k belongs to the list
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int k = 0; k < KM; ++k) {
            if (apart) with[r] = (with[r] & ~(15u << (4 * k))) | 1u << (4 * k + r);
            const uint32_t m = with[r] >> (4 * k) & 15;
            if ((here[r] >> k & 1) && (m & ((1u << r) - 1)) == 0)
                list[r == 0 && m == full ? 0 : r + 1] |= 1u << k;
        }
#pragma unroll
    for (int l = 0; l <= R; ++l)
#pragma unroll
        for (int k = 0; k < KM; ++k) {
            const int c = __popcll(__ballot(list[l] >> k & 1));
            if (lane == 0) sm_cnt[l][8 * k + wave] = c;
        }
    __syncthreads();
    if (wave <= R) {                    // lists' entries before those of (k, wave)
        const int c = lane < 8 * KM ? sm_cnt[wave][lane] : 0;
        int sum = c;
#pragma unroll
        for (int s = 1; s < 64; s <<= 1) {
            const int y = __shfl_up(sum, s);
            if (lane >= s) sum += y;
        }
        sm_cnt[wave][lane] = sum - c;
        if (lane == 63) sm_odd[wave] = sum;
    }
    __syncthreads();
    uint32_t *out = p.pick + (int64_t)blockIdx.x * R * p.W;
    uint8_t *rows_of = reinterpret_cast<uint8_t *>(sm_bits);   // the bitmaps are done with
    const uint64_t below = (1ull << lane) - 1;
    int first = 0;
#pragma unroll
    for (int l = 0; l <= R; ++l) {
        const int r = l == 0 ? 0 : l - 1;
#pragma unroll
        for (int k = 0; k < KM; ++k) {
            const bool mine = list[l] >> k & 1;
            const uint64_t b = __ballot(mine);
            if (mine) {
                const int to = first + sm_cnt[l][8 * k + wave] + __popcll(b & below);
                out[to] = at[r][k];
                rows_of[to] = (uint8_t)(with[r] >> (4 * k) & 15);
            }
        }
        first += sm_odd[l];
    }
    __syncthreads();
    const int row_words = (R * p.W + 31) >> 5;
    uint32_t *out_rows = p.pick_rows + (int64_t)blockIdx.x * R * row_words;
    for (int i = 64 * wave; i < first; i += kPickThreads) {
        const uint32_t m = i + lane < first ? rows_of[i + lane] : 0;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint64_t b = __ballot(m >> r & 1);
            const int w = (i >> 5) + lane;          // the last one may be past the row's words
            if (lane < 2 && w < row_words)
                out_rows[r * row_words + w] = (uint32_t)(lane ? b >> 32 : b);
        }
    }
    if (tid == 0) p.pick_n[blockIdx.x] = first;
}

template <bool FP8, int D>
hipError_t launch_rows(int nt, const KvAttendParams &p, hipStream_t st)
{
    const dim3 g((uint32_t)kv_blocks(p)), b(256);
#define ROWS(NT)                                                                  \
    case NT:                                                                      \
        if (p.pick) rows_kernel<FP8, D, NT, kShared><<<g, b, 0, st>>>(p);          \
        else if (p.idx) rows_kernel<FP8, D, NT, kSelected><<<g, b, 0, st>>>(p);   \
        else rows_kernel<FP8, D, NT, kAll><<<g, b, 0, st>>>(p);                   \
        break
    switch (nt) {
        ROWS(1);
        ROWS(2);
    default: return hipErrorInvalidValue;
    }
#undef ROWS
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_rows(int dtype, int d, int nt, const KvAttendParams &p, hipStream_t st)
{
    const bool fp8 = dtype == 2;
    if (d == 64) return fp8 ? launch_rows<true, 64>(nt, p, st) : launch_rows<false, 64>(nt, p, st);
    if (d == 128) return fp8 ? launch_rows<true, 128>(nt, p, st) : launch_rows<false, 128>(nt, p, st);
    return hipErrorInvalidValue;
}

hipError_t launch_kv_pick(const KvAttendParams &p, hipStream_t st)
{
    const dim3 g((uint32_t)p.slots);
    const bool wide = p.W > 5 * kPickThreads;
    if (p.tile_rows == 2 && wide) pick_kernel<2, 8><<<g, kPickThreads, 0, st>>>(p);
    else if (p.tile_rows == 2) pick_kernel<2, 5><<<g, kPickThreads, 0, st>>>(p);
    else if (p.tile_rows == 4 && wide) pick_kernel<4, 8><<<g, kPickThreads, 0, st>>>(p);
    else if (p.tile_rows == 4) pick_kernel<4, 5><<<g, kPickThreads, 0, st>>>(p);
    else return hipErrorInvalidValue;
    return hipGetLastError();
}

hipError_t launch_kv_join(int d, const KvAttendParams &p, hipStream_t st)
{
    const dim3 g((uint32_t)(p.S * p.q_heads));
    const bool sel = p.idx != nullptr;
    if (d != 64 && d != 128) return hipErrorInvalidValue;
#define JOIN(D, T)                                              \
    do {                                                        \
        if (sel) join_kernel<D, true, T><<<g, T, 0, st>>>(p);   \
        else join_kernel<D, false, T><<<g, T, 0, st>>>(p);      \
    } while (0)
    if (d == 64) {
        if (p.nsplit > kFewParts) JOIN(64, 256);
        else JOIN(64, 64);
    } else {
        if (p.nsplit > kFewParts) JOIN(128, 256);
        else JOIN(128, 64);
    }
#undef JOIN
    return hipGetLastError();
}

}  // namespace dsai
