// kv_tiles: attention of many query rows (prefill) over the paged cache.
//
// The products and the softmax are those of kv_rows, transposed in the same
// way: S^T = K Q^T, O^T = V^T P^T on v_mfma_f32_32x32x16_bf16, P passes from
// one to the other without leaving its lane.  Here the matrix unit is the
// bound, so keys and values are brought to bf16 once per block and shared:
//
//  - a block takes 256 columns (query rows of a sequence x query heads of a
//    key head), eight waves of 32, and walks the keys in tiles of 64;
//  - K and V^T of a tile lie in LDS as the matrix unit's operands, 16 bytes a
//    lane and 1 KB an operand, two tiles of each (64 KB at d = 128).  Positions
//    are XORed with the chunk that they hold, so that neither the writes of one
//    key's chunks nor the reads of one operand meet in a bank;
//  - waves 0-3 and 4-7 (one of each on every SIMD) run half a tile apart: while
//    one group is in its matrix phase (O of tile j, S of tile j + 1), the other
//    is in its vector phase (softmax of its tile, and bringing in the next: the
//    first group the keys, the second the values).  A barrier ends each phase.
//
// Each page of 16 or more tokens covers whole groups of 16 keys, so a key
// scale is a scalar for 8 of a lane's scores: it costs no vector operation but
// in the running maximum.  The value scale goes into the bf16 values: exact
// when it is a power of two (as append writes it), rounded to nearest even
// otherwise, like the values of a bf16 cache.  The running maximum moves only
// when a score exceeds it by more than 2^8, so that O is rarely rescaled; the
// probabilities are at most 2^8 then, in fp32 sums and bf16 operands that lose
// nothing by it.  At d = 128 the maximum is not even computed unless a lane's 32
// probabilities of a tile add up to more than 2^13 against the present one (1.98
// -> 1.87 ms for the chunk below); the scores have to be kept for that, and at d =
// 64, where four waves share a SIMD's registers, that costs more than the maximum
// (134 -> 243 us for five packed prompts).
//
// Bound by the matrix unit and the exponentials beside it, which overlap little:
// 4,096 rows behind 28,672 keys (e4m3, d = 128, 32 / 8 heads) take 1.86 to 2.02
// ms, 1.0 to 1.1 PFLOP/s (a large matrix product: 1.4); at d = 64, with twice the
// exponentials for each product, 0.55 PFLOP/s.
#include <type_traits>

#include "kv_common.h"

namespace dsai {
namespace {

typedef float kvf16 __attribute__((ext_vector_type(16)));

constexpr float kLn2 = 0.693147180559945309f;
constexpr int kTile = 64;  // keys
constexpr int kRanked = 16;     // sequences whose tiles are ranked
constexpr float kSlack = 8.0f;  // log2 of the largest probability against the running maximum
constexpr float kMost = 8192.0f;  // of a lane's probabilities of a tile against it, unless the maximum is looked for

template <bool HI> __device__ inline uint32_t widen_scaled(uint32_t w, float s)
{
    auto v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, HI);
    return __builtin_bit_cast(uint32_t, v);
}

template <bool HI> __device__ inline uint32_t widen_times(uint32_t w, float s)
{
    auto v = __builtin_amdgcn_cvt_pk_f32_fp8(w, HI);
    return pack_bf16(v[0] * s, v[1] * s);
}

__device__ inline uint32_t perm(uint32_t hi, uint32_t lo, uint32_t sel)
{
    return __builtin_amdgcn_perm(hi, lo, sel);
}

// The row tile of rank r when all sequences' tiles are put in the order of the
// keys that they see, the most first (ties: by sequence, then from its end).
// Blocks start in that order, so that the longest are not among the last; five
// packed prompts of 333 to 4,001 tokens: 141 -> 135 us.  Few sequences only:
// their tiles that see more than x keys are counted for 64 values of x at a time.
struct RowTile {
    Seq sq;
    int64_t t0;      // first row of the sequence, or -1: no tile of this rank
};

__device__ inline RowTile ranked_tile(const KvAttendParams &p, int64_t r)
{
    const KvCache &kc = p.c;
    const int lane = threadIdx.x & 63, nseq = kc.nseq, at = lane < nseq ? lane : nseq - 1;
    const uint32_t R = (uint32_t)p.tile_rows;
    const int c0 = clamped(kc.cu[at], p.S), c1 = clamped(kc.cu[at + 1], p.S);
    const int len = clamped(kc.seq_len[at], (int64_t)kc.table_width << kc.page_shift);
    const int n = c1 > c0 ? c1 - c0 : 0;
    const int tiles = (int)((n + R - 1) / R);
    // tiles of sequence i that see more than x keys
    auto above = [&](int i, int x) KV_INLINE {
        const int li = __builtin_amdgcn_readlane(len, i), ni = __builtin_amdgcn_readlane(n, i);
        const int ti = __builtin_amdgcn_readlane(tiles, i);
        if (!p.causal) return li > x ? ti : 0;
        const int y = x - (li - ni);     // a tile's last row sees li - ni + min(its end, ni)
        return x < 0 || y < 0 ? ti : y >= ni ? 0 : ti - (int)((uint32_t)y / R);
    };
    RowTile out;
    out.t0 = -1;
    int most = 0, total = 0;
    for (int i = 0; i < nseq; ++i) {
        const int li = __builtin_amdgcn_readlane(len, i);
        most = li > most ? li : most;
        total += __builtin_amdgcn_readlane(tiles, i);
    }
    if (r >= total) return out;
    int lo = 0, hi = most + 1;           // more than r tiles see at least lo keys, not so for hi
    while (hi - lo > 1) {
        const int step = (hi - lo + 63) / 64;
        const int x = lo + lane * step;
        int sum = 0;
        for (int i = 0; i < nseq; ++i) sum += above(i, x - 1);
        int cnt = __popcll(__ballot(x < hi && sum > r));
        cnt = cnt < 1 ? 1 : cnt;
        lo = uniform(lo + (cnt - 1) * step);
        hi = uniform(hi - lo < step ? hi : lo + step);
    }
    int rest = (int)r;
    for (int i = 0; i < nseq; ++i) rest -= above(i, lo);
    for (int i = 0; i < nseq; ++i) {
        const int more = above(i, lo), same = above(i, lo - 1) - more;
        if (rest >= same) {
            rest -= same;
            continue;
        }
        out.sq.i = i;
        out.sq.c0 = __builtin_amdgcn_readlane(c0, i);
        out.sq.c1 = __builtin_amdgcn_readlane(c1, i);
        out.sq.len = __builtin_amdgcn_readlane(len, i);
        out.t0 = (int64_t)(__builtin_amdgcn_readlane(tiles, i) - 1 - more - rest) * R;
        break;
    }
    return out;
}

template <bool FP8, int D>
__global__ __launch_bounds__(512, D == 64 ? 4 : 2) void tiles_kernel(KvAttendParams p)
{
    constexpr int ES = FP8 ? 1 : 2;
    constexpr int KS = D / 16;          // contraction steps of S
    constexpr int DT = D / 32;          // 32-channel tiles of O
    constexpr int KL = D * ES / 64;     // 16-byte loads of keys per thread and tile
    constexpr int KC = D * ES / 16;     // 16-byte chunks of a key in memory
    constexpr int VQ = D / 4;           // groups of four channels
    constexpr uint32_t RB = D * ES;     // bytes of a row
    constexpr bool LAZY = D == 128;
    __shared__ uint4 kf[2][2 * KS * 64];
    __shared__ uint4 vf[2][4 * DT * 64];
    __shared__ __align__(16) float sm_ks[2][4];  // factor of each 16 keys' scores; < 0: not there

    const KvCache &kc = p.c;
    const int tid = threadIdx.x, wave = uniform(tid >> 6), lane = tid & 63;
    const int n = lane & 31, g = lane >> 5;
    const int st = tid & 255;           // thread of the group

    // ---- which rows, key head, query heads and keys
    const int gsize = p.head_tile;
    const BlockAt blk = block_at(p);
    if (blk.none) return;
    const int head = blk.head, grp = blk.grp, split = blk.split;
    const int R = p.tile_rows;
    RowTile tile;
    if (kc.nseq > 1 && kc.nseq <= kRanked) {
        tile = ranked_tile(p, blk.slot);
    } else {
        const int64_t slot = p.slots - 1 - blk.slot;  // causal: a sequence's longest rows first
        tile.sq = find_seq(kc, p.S, slot, R, 1);
        tile.t0 = (slot - (tile.sq.c0 / R + (int64_t)tile.sq.i)) * R;
    }
    const Seq sq = tile.sq;
    const int64_t t0 = tile.t0;
    if (t0 < 0 || t0 >= sq.c1 - sq.c0) return;
    const int seq = sq.i, c0 = sq.c0;
    const int rows_in_seq = sq.c1 - sq.c0;
    const int ntok = (int)(rows_in_seq - t0 < R ? rows_in_seq - t0 : R);
    const int len = clamped(sq.len, (int64_t)kc.table_width << kc.page_shift);
    const int64_t row0 = c0 + t0;
    const int64_t last = p.causal ? (int64_t)len - rows_in_seq + t0 + ntok : len;
    const int entries = clamped(last < 0 ? 0 : (int)last, len);
    const int e0 = split * p.chunk;
    if (split > 0 && e0 >= entries) return;
    const int e1 = entries - e0 < p.chunk ? entries : e0 + p.chunk;
    const int ntile = (e1 - e0 + kTile - 1) / kTile;

    // ---- the lane's column
    const int col = wave * 32 + n, tok = col / gsize, hh = grp * gsize + col % gsize;
    const bool in = tok < ntok && hh < p.group;
    int own = in ? len : 0;              // keys that the column sees
    if (in && p.causal) {
        const int64_t x = (int64_t)len - rows_in_seq + t0 + tok + 1;
        own = x < 0 ? 0 : x < len ? (int)x : len;
    }
    int lo = in ? own : 0x7fffffff;      // the fewest that one of the wave's columns sees
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
        const int a = __shfl_xor(lo, s);
        lo = a < lo ? a : lo;
    }
    lo = uniform(lo);
    kvb8 q[KS];
    {
        const uint16_t *src = p.q + (row0 + tok) * p.q_tok +
                              (int64_t)(head * p.group + hh) * p.q_head;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (in) x = *reinterpret_cast<const uint4 *>(src + 32 * (s >> 1) + 16 * g + 8 * (s & 1));
            x = signed_queries(x, p.q_and, p.q_xor);
            q[s] = __builtin_bit_cast(kvb8, x);
        }
#pragma unroll
        for (int s = 0; s < KS; ++s) asm volatile("" : "+v"(q[s]));  // waited for before the loop
    }

    const char *kb = static_cast<const char *>(kc.k), *vb = static_cast<const char *>(kc.v);
    const int shift = kc.page_shift, page_mask = (1 << shift) - 1;
    const int32_t *table = kc.table + (int64_t)seq * kc.table_stride;

    // ---- bringing in a tile: page ids two tiles ahead, loads into registers one
    // ahead, then into LDS.  A wave's load covers at most 16 neighbouring keys,
    // which lie on one page, so page ids are scalars.
    uint32_t ld[8 * ES];                 // a wave brings in keys or values, never both
    int idk[KL], idg = 0;                // pages of the loads (values: idk[0]), of group `lane`
    float sc = 0.0f;                     // group `lane`'s key scale, or the values' scale
    bool gone = false;
    int left = 0;                        // values: tokens that the group of 16 holds
    const int gw = wave & 3;             // wave of the group
    const int pages_wide = kc.table_width - 1;
    auto page_at = [&](int pos) KV_INLINE {
        const int i = pos >> shift;
        return table[i < pages_wide ? i : pages_wide];
    };
    // keys: load x of thread st is chunk (st + 256 x) % KC of key (st + 256 x) / KC
    auto ids_k = [&](int tile) KV_INLINE {
        const int at = e0 + tile * kTile;
#pragma unroll
        for (int x = 0; x < KL; ++x) idk[x] = page_at(at + (64 * gw + 256 * x) / KC);
        if (gw == 0) idg = page_at(at + 16 * (lane & 3));
    };
    auto load_k = [&](int tile) KV_INLINE {
        const int at = e0 + tile * kTile;
#pragma unroll
        for (int x = 0; x < KL; ++x) {
            const int base = (64 * gw + 256 * x) / KC;           // the wave's first key
            const uint32_t id = (uint32_t)uniform(idk[x]);
            const uint32_t unit = id < kc.pages ? id * (uint32_t)kc.heads + head : 0;
            const char *row = kb + (uint64_t)((unit << shift) + ((at + base) & page_mask)) * RB;
            const uint4 w = *reinterpret_cast<const uint4 *>(row + lane * 16);
            ld[4 * x] = w.x;
            ld[4 * x + 1] = w.y;
            ld[4 * x + 2] = w.z;
            ld[4 * x + 3] = w.w;
        }
        if (gw == 0) {
            // no page, or no token: the scale may be anything
            gone = (uint32_t)idg >= kc.pages || at + 16 * (lane & 3) >= len;
            const uint32_t unit = gone ? 0 : (uint32_t)idg * (uint32_t)kc.heads + head;
            if constexpr (FP8) sc = kc.k_scale[unit];
        }
    };
    auto store_k = [&](int buf) KV_INLINE {
#pragma unroll
        for (int x = 0; x < KL; ++x) {
            const int i = st + 256 * x, key = i / KC, kt = key >> 5, m = key & 31, c = i % KC;
            const uint4 w = make_uint4(ld[4 * x], ld[4 * x + 1], ld[4 * x + 2], ld[4 * x + 3]);
            if constexpr (FP8) {         // chunk c: channels 16 c .. 16 c + 15, c = 2 u + g
                uint4 *dst = &kf[buf][(kt * KS + (c & ~1)) * 64 + 32 * (c & 1) + (m ^ c)];
                dst[0] = make_uint4(widen_scaled<false>(w.x, 1.0f), widen_scaled<true>(w.x, 1.0f),
                                    widen_scaled<false>(w.y, 1.0f), widen_scaled<true>(w.y, 1.0f));
                dst[64] = make_uint4(widen_scaled<false>(w.z, 1.0f), widen_scaled<true>(w.z, 1.0f),
                                     widen_scaled<false>(w.w, 1.0f), widen_scaled<true>(w.w, 1.0f));
            } else {                     // channels 8 c .. 8 c + 7, c = 4 u + 2 g + h
                const int u = c >> 2, gg = (c >> 1) & 1, h = c & 1;
                kf[buf][(kt * KS + 2 * u + h) * 64 + 32 * gg + (m ^ (2 * u + gg))] = w;
            }
        }
        if (st < 4) {
            // normal and so above 0: it multiplies the -inf of what is masked
            sm_ks[buf][st] = gone ? -1.0f : fmaxf(FP8 ? sc * p.c2 : p.c2, 0x1p-126f);
        }
    };
    // values: wave gw takes keys 16 gw .. 16 gw + 15, lane (dq, half): channels
    // 4 dq .. 4 dq + 3 of keys 4 half + {0 .. 3, 8 .. 11}
    const int dq = lane & 31, half = lane >> 5;
    const uint32_t v_lane = (uint32_t)(4 * half) * RB + (dq < VQ ? dq : 0) * (4 * ES);
    auto ids_v = [&](int tile) KV_INLINE { idk[0] = page_at(e0 + tile * kTile + 16 * gw); };
    auto load_v = [&](int tile) KV_INLINE {
        const int at = e0 + tile * kTile + 16 * gw;
        const uint32_t id = (uint32_t)uniform(idk[0]);
        const uint32_t unit = id < kc.pages ? id * (uint32_t)kc.heads + head : 0;
        const char *row = vb + (uint64_t)((unit << shift) + (at & page_mask)) * RB;
        left = id < kc.pages ? len - at : 0;
        if constexpr (FP8) sc = kc.v_scale[unit];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const char *at = row + v_lane + ((j & 3) + 8 * (j >> 2)) * RB;
            if constexpr (FP8) {
                ld[j] = *reinterpret_cast<const uint32_t *>(at);
            } else {
                const uint2 w = *reinterpret_cast<const uint2 *>(at);
                ld[2 * j] = w.x;
                ld[2 * j + 1] = w.y;
            }
        }
    };
    auto store_v = [&](int buf) KV_INLINE {
        if (left < 16) {                 // slots behind the last token may hold anything
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (4 * half + (j & 3) + 8 * (j >> 2) >= left)
                    for (int w = 0; w < ES; ++w) ld[ES * j + w] = 0;
            if (left <= 0) sc = 0.0f;
        }
        if (dq >= VQ) return;
        uint4 y[4];
        if constexpr (FP8) {
            uint32_t o[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t *x = ld + 4 * h;
                const uint32_t a0 = perm(x[1], x[0], 0x05010400), a1 = perm(x[1], x[0], 0x07030602);
                const uint32_t b0 = perm(x[3], x[2], 0x05010400), b1 = perm(x[3], x[2], 0x07030602);
                o[h][0] = perm(b0, a0, 0x05040100);
                o[h][1] = perm(b0, a0, 0x07060302);
                o[h][2] = perm(b1, a1, 0x05040100);
                o[h][3] = perm(b1, a1, 0x07060302);
            }
            const uint32_t bits = (uint32_t)uniform((int)__float_as_uint(sc));
            if ((bits & 0x7fffffu) == 0 && bits > 0) {
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    y[t] = make_uint4(widen_scaled<false>(o[0][t], sc), widen_scaled<true>(o[0][t], sc),
                                      widen_scaled<false>(o[1][t], sc), widen_scaled<true>(o[1][t], sc));
            } else {
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    y[t] = make_uint4(widen_times<false>(o[0][t], sc), widen_times<true>(o[0][t], sc),
                                      widen_times<false>(o[1][t], sc), widen_times<true>(o[1][t], sc));
            }
        } else {
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const uint32_t sel = t & 1 ? 0x07060302 : 0x05040100;
                uint32_t w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = ld[2 * j + (t >> 1)];
                y[t] = make_uint4(perm(w[1], w[0], sel), perm(w[3], w[2], sel),
                                  perm(w[5], w[4], sel), perm(w[7], w[6], sel));
            }
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int ch = 4 * (dq & 7) + t;    // channel within the tile of 32
            vf[buf][(gw * DT + (dq >> 3)) * 64 + 32 * half + (ch ^ ((ch >> 2) & 3))] = y[t];
        }
    };

    kvf16 o[DT], s[2];
    float mx = -__builtin_inff(), l = 0.0f;
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[i][j] = 0.0f;

    auto key_op = [&](int buf, int kt, int x) KV_INLINE {
        return __builtin_bit_cast(kvb8, kf[buf][(kt * KS + x) * 64 + 32 * g + (n ^ ((x & ~1) + g))]);
    };
    auto value_op = [&](int buf, int x, int i) KV_INLINE {
        return __builtin_bit_cast(kvb8, vf[buf][(x * DT + i) * 64 + 32 * g + (n ^ ((n >> 2) & 3))]);
    };
    uint4 pk[4];
    // operands that are read ahead of their products, and of those before the barrier
    constexpr int AHEAD = D == 64 ? 4 : 8, PRE = D == 64 ? 0 : 8;
    kvb8 pre[PRE + 1];
    kvf4 kfac = {};
    auto read_ahead = [&](int buf) KV_INLINE {
#pragma unroll
        for (int k = 0; k < PRE; ++k) pre[k] = value_op(buf, k / DT, k % DT);
    };
    auto scores = [&](int buf) KV_INLINE {
#pragma unroll
        for (int x = 0; x < KS; ++x)
#pragma unroll
            for (int kt = 0; kt < 2; ++kt)
                s[kt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(key_op(buf, kt, x), q[x],
                                                                x ? s[kt] : kvf16{}, 0, 0, 0);
        kfac = *reinterpret_cast<const kvf4 *>(sm_ks[buf]);
    };
    auto outputs = [&](int buf) KV_INLINE {
#pragma unroll
        for (int k = 0; k < 4 * DT; ++k)
            o[k % DT] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                k < PRE ? pre[k] : value_op(buf, k / DT, k % DT),
                __builtin_bit_cast(kvb8, pk[k / DT]), o[k % DT], 0, 0, 0);
    };
    auto softmax = [&](int tile) KV_INLINE {
        const int at = e0 + tile * kTile;
        float ks[4];
        int miss = 0;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int u = uniform(__float_as_int(kfac[x]));
            ks[x] = __builtin_bit_cast(float, u & 0x7fffffff);
            miss |= (u < 0) << x;
        }
        if (at + kTile > lo || miss) {
#pragma unroll
            for (int kt = 0; kt < 2; ++kt)
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int key = 32 * kt + 8 * (j >> 2) + 4 * g + (j & 3);
                    if (at + key >= own || (miss >> (key >> 4) & 1)) s[kt][j] = -__builtin_inff();
                }
        }
        auto maximum = [&]() KV_INLINE {     // factors are positive, so maxima carry over
            float top = -__builtin_inff();
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                float m = s[x >> 1][8 * (x & 1)];
#pragma unroll
                for (int j = 1; j < 8; ++j) m = fmaxf(m, s[x >> 1][8 * (x & 1) + j]);
                top = fmaxf(top, m * ks[x]);
            }
            return max_over_halves(top);
        };
        auto raise = [&](float top) KV_INLINE {
            const float m2 = fmaxf(mx, top);
            const float a = mx == m2 ? 1.0f : __builtin_amdgcn_exp2f(mx - m2);
            mx = m2;
            l *= a;
#pragma unroll
            for (int i = 0; i < DT; ++i) o[i] *= a;
        };
        float sum;
        auto probabilities = [&]() KV_INLINE {
            const float m1 = mx == -__builtin_inff() ? 0.0f : mx;
            sum = LAZY ? 0.0f : l;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                float e[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    e[j] = __builtin_amdgcn_exp2f(
                        __builtin_fmaf(s[x >> 1][8 * (x & 1) + j], ks[x], -m1));
                    sum += e[j];
                }
                pk[x] = make_uint4(pack_bf16(e[0], e[1]), pack_bf16(e[2], e[3]),
                                   pack_bf16(e[4], e[5]), pack_bf16(e[6], e[7]));
            }
        };
        if constexpr (LAZY) {
            bool again = __ballot(mx == -__builtin_inff() && own > at) != 0;  // first keys
            if (!again) {
                probabilities();
                again = __ballot(sum > kMost) != 0;
            }
            if (again) {
                raise(maximum());
                probabilities();
            }
            l += sum;
        } else {
            const float top = maximum();
            if (__ballot(top > mx + kSlack)) raise(top);   // also the first tile: mx = -inf
            probabilities();
            l = sum;
        }
        asm volatile("" : "+v"(l));          // summed here, not behind the matrix phase
    };

    // ---- tiles, the two groups a phase apart.  Phase 2 j: the first group's
    // softmax of tile j, which also writes the keys of j + 1 (read from phase
    // 2 j + 1 on; the buffer's last keys were read in phase 2 j - 2); phase
    // 2 j + 1: the second group's, which writes the values of j + 1.
    // The groups' loops are instantiated apart, so that loads in flight need no
    // moving between registers where the two would join.
    auto run = [&](auto keys) KV_INLINE {
        constexpr bool KEYS = decltype(keys)::value;
        auto ids = [&](int tile) KV_INLINE { if constexpr (KEYS) ids_k(tile); else ids_v(tile); };
        auto load = [&](int tile) KV_INLINE { if constexpr (KEYS) load_k(tile); else load_v(tile); };
        auto store = [&](int buf) KV_INLINE { if constexpr (KEYS) store_k(buf); else store_v(buf); };
        ids(0);
        load(0);
        ids(1);
        store(0);
        load(1);
        ids(2);
        __syncthreads();
        if constexpr (!KEYS) __syncthreads();
        scores(0);
        __syncthreads();
        for (int j = 0; j < ntile; ++j) {
            softmax(j);
            store((j + 1) & 1);
            load(j + 2);
            ids(j + 3);
            read_ahead(j & 1);
            __syncthreads();
            __builtin_amdgcn_s_setprio(1);
            outputs(j & 1);
            scores((j + 1) & 1);             // behind the last tile: of no use, and unused
            // an operand is read for every product, several ahead of its use
            __builtin_amdgcn_sched_group_barrier(0x100, AHEAD - PRE, 0);
#pragma unroll
            for (int x = 0; x < 4 * DT + 2 * KS - AHEAD + 1; ++x) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            }
            __builtin_amdgcn_sched_group_barrier(0x008, AHEAD - 1, 0);
            __builtin_amdgcn_s_setprio(0);
            if (KEYS || j + 1 < ntile) __syncthreads();
        }
    };
    if (ntile > 0) {
        if (wave < 4) run(std::true_type{});
        else run(std::false_type{});
    }

    // ---- rows out: a lane holds 4 channels in a row of each 8, of one column
    l += __shfl_xor(l, 32);
    if (!in) return;
    const int64_t out = (row0 + tok) * p.q_heads + head * p.group + hh;
    if (own <= p.chunk) {
        if (split > 0) return;
        const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const uint2 w = make_uint2(pack_bf16(o[i][4 * x] * inv, o[i][4 * x + 1] * inv),
                                           pack_bf16(o[i][4 * x + 2] * inv, o[i][4 * x + 3] * inv));
                *reinterpret_cast<uint2 *>(p.out + out * D + 32 * i + 8 * x + 4 * g) = w;
            }
        if (p.lse && g == 0)
            p.lse[out] = l > 0.0f ? (mx + __builtin_amdgcn_logf(l)) * kLn2 : -__builtin_inff();
    } else {
        const int64_t part = (int64_t)split * p.S * p.q_heads + out;
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x)
                *reinterpret_cast<float4 *>(p.part_o + part * D + 32 * i + 8 * x + 4 * g) =
                    make_float4(o[i][4 * x], o[i][4 * x + 1], o[i][4 * x + 2], o[i][4 * x + 3]);
        if (g == 0) p.part_ml[part] = make_float2(mx, l);
    }
}

}  // namespace

hipError_t launch_kv_tiles(int dtype, int d, const KvAttendParams &p, hipStream_t st)
{
    const dim3 g((uint32_t)kv_blocks(p)), b(512);
    const bool fp8 = dtype == 2;
    if (d == 64) {
        if (fp8) tiles_kernel<true, 64><<<g, b, 0, st>>>(p);
        else tiles_kernel<false, 64><<<g, b, 0, st>>>(p);
    } else if (d == 128) {
        if (fp8) tiles_kernel<true, 128><<<g, b, 0, st>>>(p);
        else tiles_kernel<false, 128><<<g, b, 0, st>>>(p);
    } else {
        return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace dsai
