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
// One wave takes one (page, key head) of the keys or of the values, so nothing
// is shared between waves: it keeps the page's new tokens in registers (16 KB
// at 64 tokens of 128), reduces their maximum and writes them once.  Bound by
// memory: every input is read once and every code written once.  The rotation
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

__device__ inline void unpack8(const uint4 &x, float (&f)[8])
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ inline uint4 pack8(const float (&f)[8])
{
    return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                      pack_bf16(f[6], f[7]));
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

// The rotation of the 8 channels [8 c, 8 c + 8) that a lane holds of one row.
// Lanes of one row are neighbours; with halves, channel i pairs with i +
// rot / 2, which another lane of the row holds (rot is a multiple of 16).
// Every lane of the wave has to call it.
struct Turn {
    float cs[8], sn[8];
    bool on;

    __device__ void load(const KvAppendParams &p, int64_t pos, int c)
    {
        const int half = p.rot >> 1;
        on = p.cos && 8 * c < p.rot;
        if (!on) return;
        if (p.interleaved) {
            const float4 a = *reinterpret_cast<const float4 *>(p.cos + pos * half + 4 * c);
            const float4 b = *reinterpret_cast<const float4 *>(p.sin + pos * half + 4 * c);
            cs[0] = a.x; cs[1] = a.y; cs[2] = a.z; cs[3] = a.w;
            sn[0] = b.x; sn[1] = b.y; sn[2] = b.z; sn[3] = b.w;
        } else {
            const int at = 8 * c < half ? 8 * c : 8 * c - half;
            const float4 *a = reinterpret_cast<const float4 *>(p.cos + pos * half + at);
            const float4 *b = reinterpret_cast<const float4 *>(p.sin + pos * half + at);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float4 x = a[i], y = b[i];
                cs[4 * i] = x.x; cs[4 * i + 1] = x.y; cs[4 * i + 2] = x.z; cs[4 * i + 3] = x.w;
                sn[4 * i] = y.x; sn[4 * i + 1] = y.y; sn[4 * i + 2] = y.z; sn[4 * i + 3] = y.w;
            }
        }
    }

    __device__ void apply(const KvAppendParams &p, const uint4 &x, int c, float (&f)[8]) const
    {
#pragma clang fp contract(off)
        unpack8(x, f);
        if (!p.cos) return;
        if (p.interleaved) {
            if (!on) return;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a = f[2 * i], b = f[2 * i + 1];
                const float ac = a * cs[i], bs = b * sn[i], bc = b * cs[i], as = a * sn[i];
                f[2 * i] = ac - bs;
                f[2 * i + 1] = bc + as;
            }
            return;
        }
        const int hop = p.rot >> 4;          // lanes between the halves
        const bool first = 8 * c < (p.rot >> 1);
        const int lane = threadIdx.x & 63;
        const int from = !on ? lane : first ? lane + hop : lane - hop;
        uint4 y;
        y.x = __shfl(x.x, from);
        y.y = __shfl(x.y, from);
        y.z = __shfl(x.z, from);
        y.w = __shfl(x.w, from);
        float o[8];
        unpack8(y, o);
        if (!on) return;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float own = f[i] * cs[i], other = o[i] * sn[i];
            f[i] = first ? own - other : own + other;
        }
    }
};

// One (page, head) of the keys (which = 0) or the values (which = 1).
template <bool FP8, int D, int PAGE>
__device__ inline void append_page(const KvAppendParams &p, int64_t slot, int head, int which)
{
    constexpr int L = D / 8, ROWS = 64 / L, NIT = PAGE / ROWS;  // lanes a row, rows a step
    const KvCache &kc = p.c;
    const int lane = threadIdx.x & 63, c = lane % L, r = lane / L;
    const int i = find_seq(kc.cu, kc.nseq, slot, PAGE, 2);
    const int c0 = clamped(kc.cu[i], p.N), n = clamped(kc.cu[i + 1], p.N) - c0;
    const int cap = kc.table_width * PAGE;                      // < 2^31, checked on the host
    const int held = clamped(kc.seq_len[i], cap);
    const int64_t pg = held / PAGE + (slot - (c0 / PAGE + 2 * (int64_t)i));
    // positions past the table or past the rotation's rows are not written
    int64_t end = (int64_t)held + (n > 0 ? n : 0);
    end = end < cap ? end : cap;
    if (p.cos && end > p.rope_rows) end = p.rope_rows;
    if (pg < held / PAGE || pg * PAGE >= end || held >= end) return;
    const uint32_t id = (uint32_t)kc.table[(int64_t)i * kc.table_stride + pg];
    if (id >= kc.pages) return;
    const int s0 = pg * PAGE > held ? 0 : held - (int)pg * PAGE;       // slots to fill
    const int s1 = (int)(end - pg * PAGE < PAGE ? end - pg * PAGE : PAGE);
    const int64_t unit = (int64_t)id * kc.heads + head;
    const uint16_t *src = p.src[which] + head * p.head_stride[which] + 8 * c;
    const int64_t tok0 = c0 + (pg * PAGE - held);                      // token of slot 0

    if constexpr (!FP8) {
        uint4 *dst = reinterpret_cast<uint4 *>(which ? kc.v : kc.k) + unit * PAGE * L + c;
        for (int s = s0; s < s1; s += ROWS) {
            const int at = s + r;
            const bool in = at < s1;
            uint4 x = make_uint4(0, 0, 0, 0);
            if (in) x = *reinterpret_cast<const uint4 *>(src + (tok0 + at) * p.tok_stride[which]);
            if (which == 0) {
                Turn t;
                t.load(p, pg * PAGE + (in ? at : s), c);
                float f[8];
                t.apply(p, x, c, f);
                x = pack8(f);
            }
            if (in) dst[(int64_t)at * L] = x;
        }
        return;
    } else {
        float f[NIT][8];
        float amax = 0.0f;
#pragma unroll
        for (int it = 0; it < NIT; ++it) {
            const int s = s0 + it * ROWS, at = s + r;
            if (s >= s1) continue;                                     // the whole wave
            const bool in = at < s1;
            uint4 x = make_uint4(0, 0, 0, 0);
            if (in) x = *reinterpret_cast<const uint4 *>(src + (tok0 + at) * p.tok_stride[which]);
            if (which == 0) {
                Turn t;
                t.load(p, pg * PAGE + (in ? at : s), c);
                t.apply(p, x, c, f[it]);
            } else {
                unpack8(x, f[it]);
            }
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
            const float old = *scale;
            if (old >= s) {
                s = old;
            } else {                                                   // the held tokens' codes
                const float ratio = old / s;
                for (int at = r; at < s0; at += ROWS) {
                    const uint2 w = dst[(int64_t)at * L];
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
                    dst[(int64_t)at * L] = codes8(g);
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
            dst[(int64_t)at * L] = codes8(g);
        }
        if (lane == 0) *scale = s;
    }
}

// The queries of 64 / L heads at a time of one token, all its heads by one wave.
template <int D>
__device__ inline void rotate_queries(const KvAppendParams &p, int64_t tok)
{
    constexpr int L = D / 8, HEADS = 64 / L;
    const KvCache &kc = p.c;
    const int lane = threadIdx.x & 63, c = lane % L, r = lane / L;
    const int i = find_seq(kc.cu, kc.nseq, tok, 1, 0);
    const int c0 = clamped(kc.cu[i], p.N), c1 = clamped(kc.cu[i + 1], p.N);
    if (tok < c0 || tok >= c1) return;                                 // rows of no sequence
    const int held = clamped(kc.seq_len[i], (int64_t)kc.table_width << kc.page_shift);
    const int64_t pos = held + (tok - c0);
    if (p.cos && pos >= p.rope_rows) return;
    Turn t;
    t.load(p, pos, c);
    for (int h = 0; h < p.q_heads; h += HEADS) {
        const bool in = h + r < p.q_heads;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (in)
            x = *reinterpret_cast<const uint4 *>(p.src[2] + tok * p.tok_stride[2] +
                                                 (h + r) * p.head_stride[2] + 8 * c);
        float f[8];
        t.apply(p, x, c, f);
        if (in)
            *reinterpret_cast<uint4 *>(p.q_out + tok * p.qo_tok + (h + r) * p.qo_head + 8 * c) =
                pack8(f);
    }
}

template <bool FP8, int D, int PAGE>
__global__ __launch_bounds__(256) void append_kernel(KvAppendParams p)
{
    const int64_t unit = (int64_t)blockIdx.x * 4 + uniform(threadIdx.x >> 6);
    if (unit < p.kv_units) {
        // neighbouring waves take the heads of one page: they read the same
        // rows of the rotation tables
        const int head = (int)(unit % p.c.heads);
        const int64_t u = unit / p.c.heads;
        append_page<FP8, D, PAGE>(p, u >> 1, head, (int)(u & 1));
    } else if (unit - p.kv_units < p.q_units) {
        rotate_queries<D>(p, unit - p.kv_units);
    }
}

template <bool FP8, int D>
hipError_t launch_page(const KvAppendParams &p, hipStream_t st)
{
    const int64_t blocks = (p.kv_units + p.q_units + 3) / 4;
    if (blocks == 0) return hipSuccess;
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
