// Device helpers shared by the paged cache's kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kv.h"

#define KV_INLINE __attribute__((always_inline))

namespace dsai {
namespace {

typedef __bf16 kvb8 __attribute__((ext_vector_type(8)));
typedef __bf16 kvb2 __attribute__((ext_vector_type(2)));
typedef float kvf4 __attribute__((ext_vector_type(4)));
typedef uint32_t kvu4 __attribute__((ext_vector_type(4)));

__device__ inline int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// The largest of the four lanes n, n + 16, n + 32, n + 48.
__device__ inline float max_over_rows(float x)
{
    const uint32_t u = __float_as_uint(x);
    auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const uint32_t y = __float_as_uint(fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1])));
    auto b = __builtin_amdgcn_permlane16_swap(y, y, false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

// The larger of the lanes n and n + 32.
__device__ inline float max_over_halves(float x)
{
    const uint32_t u = __float_as_uint(x);
    auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}

// What a block of an attention launch works on.  Blocks are dealt to the eight
// XCDs in turn: with eight key heads each XCD keeps to one head's keys, and the
// groups of one key head's query heads are eight blocks apart, so that the
// second finds the keys in the L2 that the first filled.
struct BlockAt {
    int head, grp, split;
    int64_t slot;
    bool none;
};

__device__ inline BlockAt block_at(const KvAttendParams &p)
{
    BlockAt r;
    uint32_t u = blockIdx.x;             // fewer than 2^31 blocks, checked on the host
    r.grp = 0;
    r.none = false;
    if (p.groups > 1) {
        const uint32_t g = (uint32_t)p.groups, b = u >> 3;
        r.grp = (int)(b % g);
        u = (b / g) * 8 + (u & 7);
        r.none = u >= (uint32_t)kv_units(p);
    }
    const uint32_t heads = (uint32_t)p.c.heads, slots = (uint32_t)p.slots;
    r.head = (int)(u % heads);
    u /= heads;
    r.split = (int)(u / slots);
    r.slot = u % slots;
    return r;
}

// Two floats to packed bf16, round to nearest even.
__device__ inline uint32_t pack_bf16(float a, float b)
{
    kvb2 v;
    v[0] = (__bf16)a;
    v[1] = (__bf16)b;
    return __builtin_bit_cast(uint32_t, v);
}

// Eight query elements with their sign turned, or cleared: a factor of the
// scores that is not positive is applied here, so that the kernels' is.
__device__ inline uint4 signed_queries(uint4 x, uint32_t keep, uint32_t flip)
{
    return make_uint4((x.x & keep) ^ flip, (x.y & keep) ^ flip, (x.z & keep) ^ flip,
                      (x.w & keep) ^ flip);
}

__device__ inline int clamped(int x, int64_t hi)
{
    return x < 0 ? 0 : (int64_t)x > hi ? (int)hi : x;
}

// A sequence of the call: rows [c0, c1) of it, clamped to [0, rows], and its
// length as given.
struct Seq {
    int i, c0, c1, len;
};

// The sequence of the largest i in [0, nseq) with max(cu[i], 0) / div + mul * i
// <= slot, by the whole wave: 64 probes a step down to 64 sequences, whose
// rows and lengths then come with one round of loads.  For an array that does
// not ascend the answer is some sequence.
__device__ inline Seq find_seq(const KvCache &kc, int64_t rows, int64_t slot, int div, int mul)
{
    const int lane = threadIdx.x & 63;
    int lo = 0, hi = kc.nseq;
    auto fits = [&](int x, int i) KV_INLINE {
        return (int64_t)((x < 0 ? 0 : x) / div) + (int64_t)mul * i <= slot;
    };
    while (hi - lo > 64) {
        const int step = (hi - lo + 63) / 64;
        const int64_t i = lo + (int64_t)lane * step;
        const bool in = i < hi;
        const int at = in ? (int)i : lo;
        int cnt = __popcll(__ballot(in && fits(kc.cu[at], at)));
        cnt = cnt < 1 ? 1 : cnt;
        lo += (cnt - 1) * step;
        if (lo >= hi) lo = hi - 1;
        hi = hi - lo < step ? hi : lo + step;
        lo = uniform(lo);
        hi = uniform(hi);
    }
    const bool in = lo + lane < hi;
    const int at = in ? lo + lane : lo;
    const int a = kc.cu[at], b = kc.cu[at + 1], n = kc.seq_len[at];
    int cnt = __popcll(__ballot(in && fits(a, at)));
    cnt = uniform(cnt < 1 ? 0 : cnt - 1);
    Seq s;
    s.i = lo + cnt;
    s.c0 = clamped(__builtin_amdgcn_readlane(a, cnt), rows);
    s.c1 = clamped(__builtin_amdgcn_readlane(b, cnt), rows);
    s.len = __builtin_amdgcn_readlane(n, cnt);
    return s;
}

}  // namespace
}  // namespace dsai
