// kv_append: new keys and values into the paged cache, keys rotated by their
// positions on the way, and the same rotation of the step's queries.
//
// A page of one key head is quantised as a whole: with amax the largest
// magnitude of the tokens it receives, its scale is the smallest power of two
// s with amax <= 448 s, or the scale it has if that is larger and the page
// holds tokens of the sequence already; those are brought to a grown scale in
// place.  Powers of two make every product code * s exact in bf16 and fp32 and
// the change of scale exact but for codes that fall below the smallest normal
// one, which are rounded to nearest even once more.
//
// One wave takes one (page, key head) of the keys or of the values: it keeps the
// page's new tokens in registers (16 KB at 64 tokens of 128), reduces their
// maximum and writes them once.  Four heads of a page make a block, which keeps
// the page's cosines and sines in LDS.  The queries of a token are one wave's.
// Bound by memory: every input is read once and every output written once,
// loads first, so that a wave has 8 to 16 KB in flight.  32,768 tokens of 32 + 8
// + 8 heads of 128: 150 us, 5.0 TB/s (a large copy: 4.7); 64 single tokens of 64
// + 8 + 8 heads: 5.4 us, three rounds of dependent loads.  The rotation
// is computed without contraction into fused multiply-adds (each product is
// rounded to fp32 and the sum again), so that a key's code does not depend on
// how the compiler pairs operations.
#include "kv_common.h"

namespace dsai {
namespace {

constexpr float kE4m3Max = 448.0f;
constexpr int kMinExp = -117, kMaxExp = 120;  // code * 2^e is a normal bf16 for every code

// The smallest power of two s with amax <= 448 s (amax finite, >= 0).
__device__ inline float pow2_scale(float amax)
{
    const uint32_t u = __float_as_uint(amax);
    // 448 = 1.75 * 2^8: the exponent goes up by one when the mantissa exceeds 1.75
    int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = e < kMinExp ? kMinExp : e > kMaxExp ? kMaxExp : e;
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

__device__ inline void unpack8(const kvu4 w, float (&f)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ inline kvu4 pack8(const float (&f)[8])
{
    return kvu4{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                pack_bf16(f[6], f[7])};
}

__device__ inline uint2 codes8(const float (&f)[8])
{
    uint32_t a = 0, b = 0;
    a = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], a, false);
    a = __builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], a, true);
    b = __builtin_amdgcn_cvt_pk_fp8_f32(f[4], f[5], b, false);
    b = __builtin_amdgcn_cvt_pk_fp8_f32(f[6], f[7], b, true);
    return make_uint2(a, b);
}

// The rotation of the 8 channels [8 c, 8 c + 8) that a lane holds of one row,
// by 8 cosines and sines (interleaved pairs: the first 4).  Lanes of one row are
// neighbours; with halves, channel i pairs with i + rot / 2, which another lane
// of the row holds (rot is a multiple of 16).  Every lane of the wave has to
// call it.
__device__ inline void turn(const KvAppendParams &p, const kvu4 x, int c, const kvf4 (&cs)[2],
                            const kvf4 (&sn)[2], float (&f)[8])
{
#pragma clang fp contract(off)
    unpack8(x, f);
    const bool on = 8 * c < p.rot;
    if (p.interleaved) {
        if (!on) return;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = f[2 * i], b = f[2 * i + 1];
            const float ac = a * cs[0][i], bs = b * sn[0][i], bc = b * cs[0][i], as = a * sn[0][i];
            f[2 * i] = ac - bs;
            f[2 * i + 1] = bc + as;
        }
        return;
    }
    const int hop = p.rot >> 4;              // lanes between the halves
    const bool first = 8 * c < (p.rot >> 1);
    const int lane = threadIdx.x & 63;
    const int from = !on ? lane : first ? lane + hop : lane - hop;
    kvu4 y;
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = __shfl(x[i], from);
    float o[8];
    unpack8(y, o);
    if (!on) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float own = f[i] * cs[i >> 2][i & 3], other = o[i] * sn[i >> 2][i & 3];
        f[i] = first ? own - other : own + other;
    }
}

// Where the lane's cosines and sines start in a row of rot / 2.
__device__ inline int turn_at(const KvAppendParams &p, int c)
{
    if (8 * c >= p.rot) return 0;
    if (p.interleaved) return 4 * c;
    return 8 * c < (p.rot >> 1) ? 8 * c : 8 * c - (p.rot >> 1);
}

// One page of up to four heads of the keys (which = 0) or the values (1).
template <bool FP8, int D, int PAGE>
__device__ inline void append_page(const KvAppendParams &p, int64_t slot, int head0, int which,
                                   float *rope)
{
    constexpr int L = D / 8, ROWS = 64 / L;                    // lanes a row, rows a step
    constexpr int NIT = PAGE / ROWS;
    const KvCache &kc = p.c;
    const int tid = threadIdx.x, lane = tid & 63, c = lane % L, r = lane / L;
    const int head = head0 + uniform(tid >> 6);
    const Seq sq = find_seq(kc, p.N, slot, PAGE, 2);
    const int c0 = sq.c0, n = sq.c1 - sq.c0;
    const int cap = kc.table_width * PAGE;                      // < 2^31, checked on the host
    const int held = clamped(sq.len, cap);
    const int64_t pg = held / PAGE + (slot - (c0 / PAGE + 2 * (int64_t)sq.i));
    // positions past the table or past the rotation's rows are not written
    int64_t end = (int64_t)held + (n > 0 ? n : 0);
    end = end < cap ? end : cap;
    if (p.cos && end > p.rope_rows) end = p.rope_rows;
    if (pg < held / PAGE || pg * PAGE >= end || held >= end) return;   // the whole block
    const uint32_t id = (uint32_t)kc.table[(int64_t)sq.i * kc.table_stride + pg];
    const int s0 = pg * PAGE > held ? 0 : held - (int)pg * PAGE;       // slots to fill
    const int s1 = (int)(end - pg * PAGE < PAGE ? end - pg * PAGE : PAGE);
    const bool mine = head < kc.heads;
    const int64_t ts = p.tok_stride[which];
    const uint16_t *src = p.src[which] + (mine ? head : 0) * p.head_stride[which] + 8 * c +
                          (c0 + (pg * PAGE - held)) * ts;              // slot 0's token
    const bool turns = which == 0 && p.cos;

    // all rows' loads first; lanes behind the last row read it again
    kvu4 x[NIT];
#pragma unroll
    for (int it = 0; it < NIT; ++it) {
        const int s = s0 + it * ROWS, at = s + r < s1 ? s + r : s1 - 1;
        if (s < s1) x[it] = *reinterpret_cast<const kvu4 *>(src + at * ts);
    }
    // the page's cosines and sines, for all its heads: the first round of loads
    // as well, before anything waits for the page id
    const int half = p.rot >> 1;
    const int total = turns ? (s1 - s0) * half : 0;
    const float *cos = p.cos + (pg * PAGE + s0) * half, *sin = p.sin + (pg * PAGE + s0) * half;
    kvf4 cs0 = {}, sn0 = {};
    if (4 * tid < total) {
        cs0 = *reinterpret_cast<const kvf4 *>(cos + 4 * tid);
        sn0 = *reinterpret_cast<const kvf4 *>(sin + 4 * tid);
    }
    if (id >= kc.pages) return;                                        // the whole block
    const int64_t unit = (int64_t)id * kc.heads + (mine ? head : 0);
    float old = 0.0f;                    // the scale of a page that holds tokens already
    if constexpr (FP8)
        if (s0 > 0) old = (which ? kc.v_scale : kc.k_scale)[unit];
    if (turns) {
        if (4 * tid < total) {
            *reinterpret_cast<kvf4 *>(rope + 4 * tid) = cs0;
            *reinterpret_cast<kvf4 *>(rope + total + 4 * tid) = sn0;
        }
        for (int k = 4 * tid + 1024; k < total; k += 1024) {
            *reinterpret_cast<kvf4 *>(rope + k) = *reinterpret_cast<const kvf4 *>(cos + k);
            *reinterpret_cast<kvf4 *>(rope + total + k) = *reinterpret_cast<const kvf4 *>(sin + k);
        }
        __syncthreads();
        rope += turn_at(p, c);
    }
    if (!mine) return;
    auto rotated = [&](int it, float (&f)[8]) KV_INLINE {
        if (!turns) {
            unpack8(x[it], f);
            return;
        }
        const int at = it * ROWS + r < s1 - s0 ? it * ROWS + r : s1 - s0 - 1;
        const kvf4 *cp = reinterpret_cast<const kvf4 *>(rope + at * half);
        const kvf4 *sp = reinterpret_cast<const kvf4 *>(rope + (s1 - s0 + at) * half);
        const kvf4 cs[2] = {cp[0], p.interleaved ? cp[0] : cp[1]};
        const kvf4 sn[2] = {sp[0], p.interleaved ? sp[0] : sp[1]};
        turn(p, x[it], c, cs, sn, f);
    };

    if constexpr (!FP8) {
        kvu4 *dst = reinterpret_cast<kvu4 *>(which ? kc.v : kc.k) + unit * PAGE * L + c;
#pragma unroll
        for (int it = 0; it < NIT; ++it) {
            const int s = s0 + it * ROWS, at = s + r;
            if (s >= s1) continue;                                     // the whole wave
            kvu4 y = x[it];
            if (turns) {
                float f[8];
                rotated(it, f);
                y = pack8(f);
            }
            if (at < s1) dst[at * L] = y;
        }
    } else {
        float f[NIT][8];
        float amax = 0.0f;
#pragma unroll
        for (int it = 0; it < NIT; ++it) {
            if (s0 + it * ROWS >= s1) continue;                        // the whole wave
            rotated(it, f[it]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                // infinities and NaN become the code NaN and do not move the scale
                const float a = __builtin_fabsf(f[it][j]);
                const bool fin = a < __builtin_inff();
                amax = fin && a > amax ? a : amax;
                if (!fin) f[it][j] = __builtin_nanf("");
            }
        }
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) amax = fmaxf(amax, __shfl_xor(amax, m));
        float *scale = (which ? kc.v_scale : kc.k_scale) + unit;
        uint2 *dst = reinterpret_cast<uint2 *>(which ? kc.v : kc.k) + unit * PAGE * L + c;
        float s = pow2_scale(amax);
        if (s0 > 0) {
            if (old >= s) {
                s = old;
            } else {                                                   // the held tokens' codes
                const float ratio = old / s;
                for (int at = r; at < s0; at += ROWS) {
                    const uint2 w = dst[at * L];
                    float g[8];
                    const uint32_t u[2] = {w.x, w.y};
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(u[j], false);
                        auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(u[j], true);
                        g[4 * j] = lo[0] * ratio;
                        g[4 * j + 1] = lo[1] * ratio;
                        g[4 * j + 2] = hi[0] * ratio;
                        g[4 * j + 3] = hi[1] * ratio;
                    }
                    dst[at * L] = codes8(g);
                }
            }
        }
        const float inv = 1.0f / s;
#pragma unroll
        for (int it = 0; it < NIT; ++it) {
            const int at = s0 + it * ROWS + r;
            if (at >= s1) continue;
            float g[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) g[j] = f[it][j] * inv;
            dst[at * L] = codes8(g);
        }
        if (lane == 0) *scale = s;
    }
}

// The queries of one token, p.q_steps steps of 64 / L heads by one wave, up to
// eight loads deep.
template <int D>
__device__ inline void rotate_queries(const KvAppendParams &p, int64_t tok, int part)
{
    constexpr int L = D / 8, HEADS = 64 / L, DEEP = 8;
    const KvCache &kc = p.c;
    const int lane = threadIdx.x & 63, c = lane % L, r = lane / L;
    const uint16_t *src = p.src[2] + tok * p.tok_stride[2] + 8 * c;
    uint16_t *dst = p.q_out + tok * p.qo_tok + 8 * c;
    const int last = p.q_heads - 1, first = part * p.q_steps * HEADS;
    const int end = first + p.q_steps * HEADS <= last ? first + p.q_steps * HEADS : last + 1;
    kvu4 x[DEEP];
    auto load = [&](int h0) KV_INLINE {  // lanes behind the last head read it again
#pragma unroll
        for (int k = 0; k < DEEP; ++k) {
            const int h = h0 + k * HEADS;
            if (h < end)
                x[k] = *reinterpret_cast<const kvu4 *>(src + (h + r < last ? h + r : last) *
                                                                 p.head_stride[2]);
        }
    };
    load(first);                         // under way while the position is looked up
    const Seq sq = find_seq(kc, p.N, tok, 1, 0);
    if (tok < sq.c0 || tok >= sq.c1) return;                           // rows of no sequence
    const int held = clamped(sq.len, (int64_t)kc.table_width << kc.page_shift);
    const int64_t pos = held + (tok - sq.c0);
    if (p.cos && pos >= p.rope_rows) return;
    kvf4 cs[2] = {}, sn[2] = {};
    if (p.cos) {
        const int64_t at = pos * (p.rot >> 1) + turn_at(p, c);
        cs[0] = *reinterpret_cast<const kvf4 *>(p.cos + at);
        sn[0] = *reinterpret_cast<const kvf4 *>(p.sin + at);
        if (!p.interleaved) {
            cs[1] = *reinterpret_cast<const kvf4 *>(p.cos + at + 4);
            sn[1] = *reinterpret_cast<const kvf4 *>(p.sin + at + 4);
        }
    }
    for (int h0 = first; h0 < end; h0 += DEEP * HEADS) {
        if (h0 > first) load(h0);
#pragma unroll
        for (int k = 0; k < DEEP; ++k) {
            const int h = h0 + k * HEADS;
            if (h >= end) continue;                                    // the whole wave
            kvu4 y = x[k];
            if (p.cos) {
                float f[8];
                turn(p, x[k], c, cs, sn, f);
                y = pack8(f);
            }
            if (h + r <= last) *reinterpret_cast<kvu4 *>(dst + (h + r) * p.qo_head) = y;
        }
    }
}

template <bool FP8, int D, int PAGE>
__global__ __launch_bounds__(256) void append_kernel(KvAppendParams p)
{
    __shared__ __align__(16) float rope[PAGE * D];
    int64_t b = blockIdx.x;
    if (b < p.kv_blocks) {
        const int quads = (p.c.heads + 3) / 4;
        const int head = (int)(b % quads) * 4;
        b /= quads;
        append_page<FP8, D, PAGE>(p, b >> 1, head, (int)(b & 1), rope);
    } else {
        const uint32_t u = (uint32_t)(b - p.kv_blocks) * 4 + uniform(threadIdx.x >> 6);
        const uint32_t tok = u / (uint32_t)p.q_parts;
        if (tok < p.N) rotate_queries<D>(p, tok, (int)(u % (uint32_t)p.q_parts));
    }
}

template <bool FP8, int D>
hipError_t launch_page(const KvAppendParams &p, hipStream_t st)
{
    const int64_t blocks = p.kv_blocks + (p.q_heads > 0 ? (p.N * p.q_parts + 3) / 4 : 0);
    const dim3 g((uint32_t)blocks), b(256);
    switch (p.c.page_shift) {
    case 4: append_kernel<FP8, D, 16><<<g, b, 0, st>>>(p); break;
    case 5: append_kernel<FP8, D, 32><<<g, b, 0, st>>>(p); break;
    case 6: append_kernel<FP8, D, 64><<<g, b, 0, st>>>(p); break;
    case 7: append_kernel<FP8, D, 128><<<g, b, 0, st>>>(p); break;
    default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(int dtype, int d, const KvAppendParams &p, hipStream_t st)
{
    const bool fp8 = dtype == 2;
    if (d == 64) return fp8 ? launch_page<true, 64>(p, st) : launch_page<false, 64>(p, st);
    if (d == 128) return fp8 ? launch_page<true, 128>(p, st) : launch_page<false, 128>(p, st);
    return hipErrorInvalidValue;
}

}  // namespace dsai
