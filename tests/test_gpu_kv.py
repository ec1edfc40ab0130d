"""The paged key/value cache on the GPU against the fp64 / token-by-token
reference in oracle/kv.py.

Codes, scales and rotated rows have to be equal bit for bit (the definition
fixes every rounding).  For attention the tolerance of an output element is

    2^-8 |o|                 its rounding to bf16
  + 2^-8 A                   the probabilities' rounding to bf16, A = sum p |v|
  + 2 e A                    scores off by e each, so p off by e, above and below
  + (n + 8) 2^-24 A          fp32 sums over n keys

with e = (d + 8) 2^-24 max_j scale sum |q| |k| + 2^-22 |lse range|: d products
summed in fp32, the factors' roundings and exp2's error; lse is off by e and its
own last steps, 2^-21 (1 + |lse|)."""
import numpy as np
import pytest
import torch

import dsa_indexer_score_amd as dsai
from oracle import kv as okv

pytestmark = pytest.mark.gpu
DEV = "cuda"


def log(*a):
    print(*a, flush=True)


class Problem:
    """A filled cache with pages in a shuffled order, NaN wherever no token lies."""

    def __init__(self, seed, dtype, heads, d, page, lens, spare=2, nan=True, pow2=False):
        g = np.random.default_rng(seed)
        self.g, self.dtype, self.heads, self.d, self.page = g, dtype, heads, d, page
        need = [-(-n // page) for n in lens]
        pages, width = sum(need) + spare, max(need + [1]) + 1
        perm = g.permutation(pages)
        self.table = np.full((len(lens), width), -1, np.int32)
        at = 0
        for i, n in enumerate(need):
            self.table[i, :n] = perm[at:at + n]
            at += n
        self.lens = np.array(lens, np.int32)
        fp8 = dtype == torch.float8_e4m3fn
        self.cache, self.scale = {}, {}
        for w in "kv":
            x = g.standard_normal((pages, heads, page, d)).astype(np.float32) * \
                np.exp(0.5 * g.standard_normal((1, heads, 1, d))).astype(np.float32)
            used = np.zeros((pages, page), bool)
            for i, n in enumerate(lens):
                for pos in range(n):
                    used[self.table[i, pos // page], pos % page] = True
            if fp8:
                s = np.stack([[okv.pow2_scale(np.abs(x[p, h]).max()) for h in range(heads)]
                              for p in range(pages)]).astype(np.float32)
                # scales need not be powers of two for attention
                s = s * np.float32(1.0 if pow2 else 1.25)
                c = okv.to_e4m3(x / s[:, :, None, None])
                if nan:
                    c = np.where(used[:, None, :, None], c, np.uint8(0x7f))
                    s = np.where(used.any(1)[:, None], s, np.float32(np.nan))
                self.cache[w], self.scale[w] = c, s
            else:
                x = torch.from_numpy(x).to(torch.bfloat16).float().numpy()
                if nan:
                    x = np.where(used[:, None, :, None], x, np.float32(np.nan))
                self.cache[w], self.scale[w] = x, None

    def gpu(self):
        fp8 = self.dtype == torch.float8_e4m3fn
        t = {}
        for w in "kv":
            x = torch.from_numpy(self.cache[w])
            t[w] = (x.view(torch.float8_e4m3fn) if fp8 else x.to(torch.bfloat16)).to(DEV)
            t[w + "s"] = torch.from_numpy(self.scale[w]).to(DEV) if fp8 else None
        return dsai.KVCache(t["k"], t["v"], k_scale=t["ks"], v_scale=t["vs"])

    def queries(self, S, q_heads):
        q = torch.from_numpy(self.g.standard_normal((S, q_heads, self.d)).astype(np.float32) * 1.5)
        return q.to(torch.bfloat16)


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def check(out, lse, ref, d, where=""):
    o, l, mag, size, keys = ref
    out, lse = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    mine = ~np.isnan(l)
    e = (d + 8) * 2.0 ** -24 * size + 2.0 ** -22 * (1 + np.where(np.isfinite(l), np.abs(l), 0) + size)
    tol = 2.0 ** -8 * np.abs(o) + mag * (2.0 ** -8 + 2 * e[..., None] +
                                         (keys[:, None, None] + 8) * 2.0 ** -24) + 1e-30
    assert np.isfinite(out[mine]).all(), where
    worst = float(np.nanmax(np.where(mine[..., None], np.abs(out - o) / tol, 0))) if out.size else 0
    assert worst <= 1, f"{where}: output off by {worst} tolerances"
    empty = mine & np.isneginf(l)
    assert (out[empty] == 0).all() and np.isneginf(lse[empty]).all(), where
    some = mine & np.isfinite(l)
    ltol = e + 2.0 ** -21 * (1 + np.abs(l))
    assert (np.abs(lse[some] - l[some]) <= ltol[some]).all(), f"{where}: lse"


FP8, BF16 = torch.float8_e4m3fn, torch.bfloat16
ATTEND = [
    # dtype, d, page, key heads, group, lens, rows per sequence, causal, padding rows
    (FP8, 128, 64, 2, 8, [1, 64, 65, 333], [1, 1, 1, 1], True, 0),
    (FP8, 64, 16, 1, 1, [17], [1], True, 0),
    (BF16, 128, 16, 2, 4, [31, 32, 33, 0, 1], [1, 1, 1, 1, 1], True, 2),
    (BF16, 64, 128, 3, 7, [129, 500], [1, 1], True, 0),
    (FP8, 128, 32, 1, 64, [200, 7], [1, 1], True, 0),          # one key head: four column tiles
    (FP8, 64, 64, 1, 100, [90], [2], True, 1),                 # more heads than a block takes
    (BF16, 128, 64, 1, 24, [70, 3], [3, 3], True, 0),
    (FP8, 128, 128, 2, 3, [40, 0, 260, 5], [5, 2, 0, 9], True, 3),   # rows that see nothing
    (FP8, 64, 32, 2, 2, [100, 45], [37, 45], True, 0),
    (BF16, 64, 16, 4, 3, [150, 64, 1], [150, 20, 1], True, 1),
    (FP8, 128, 64, 2, 4, [300, 129], [130, 129], True, 0),
    (BF16, 128, 32, 1, 16, [90], [90], True, 0),
    (FP8, 64, 16, 2, 5, [65, 9], [11, 9], False, 0),
    (BF16, 128, 64, 2, 1, [77, 130], [77, 64], False, 1),
    (FP8, 128, 64, 1, 8, [9001], [1], True, 0),                # split along the keys
    (BF16, 64, 32, 2, 4, [5000, 257, 0, 3001], [1, 1, 1, 1], True, 1),
    (FP8, 128, 16, 2, 6, [4097, 600], [3, 2], True, 0),
    (FP8, 128, 64, 1, 40, [2500, 1100], [2, 4], True, 0),
    # many rows: 256 columns a block
    (FP8, 128, 64, 1, 8, [700], [300], True, 1),
    (FP8, 64, 16, 2, 3, [1, 400, 0, 333], [1, 400, 5, 100], True, 2),
    (BF16, 128, 16, 1, 7, [777, 64], [130, 64], True, 0),
    (BF16, 64, 128, 2, 1, [1000], [600], True, 0),
    (FP8, 128, 32, 1, 100, [150], [9], True, 0),
    (FP8, 128, 128, 1, 4, [5000, 90], [70, 70], True, 3),       # split along the keys
    (BF16, 64, 32, 1, 16, [4500], [33], False, 0),
    (FP8, 64, 64, 1, 64, [200, 3000], [3, 5], True, 0),
]


def run_attend(c, nan=True, pow2=False, **kw):
    dtype, d, page, heads, group, lens, rows, causal, pad = c
    pr = Problem(hash((d, page, heads, group, len(lens), lens[0])) % 1000, dtype, heads, d, page,
                 lens, nan=nan, pow2=pow2)
    S = sum(rows) + pad
    cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    q = pr.queries(S, heads * group)
    ref = okv.attend(q.double().numpy(), cu, pr.lens, pr.table, pr.cache["k"], pr.scale["k"],
                     pr.cache["v"], pr.scale["v"], d ** -0.5, causal)
    cache = pr.gpu()
    out = torch.full((S, heads * group, d), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((S, heads * group), 7.0, device=DEV)
    cache.attend(q.to(DEV), dev(cu), dev(pr.lens), dev(pr.table), causal=causal, with_lse=True,
                 out=(out, lse), **kw)
    torch.cuda.synchronize()
    assert bool((out[S - pad:] == 7).all()) and bool((lse[S - pad:] == 7).all())
    return out, lse, ref, d


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("c", ATTEND, ids=range(len(ATTEND)))
def test_attend_matches_the_reference(c, pow2):
    log(c)
    check(*run_attend(c, pow2=pow2), where=str(c))


@pytest.mark.parametrize("scale", [0.0, -0.09])
@pytest.mark.parametrize("c", [ATTEND[5], ATTEND[18], ATTEND[20]], ids=["rows", "fp8", "bf16"])
def test_attend_with_a_factor_that_is_not_positive(c, scale):
    dtype, d, page, heads, group, lens, rows, causal, pad = c
    pr = Problem(11, dtype, heads, d, page, lens)
    cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    q = pr.queries(sum(rows), heads * group)
    ref = okv.attend(q.double().numpy(), cu, pr.lens, pr.table, pr.cache["k"], pr.scale["k"],
                     pr.cache["v"], pr.scale["v"], scale)
    out, lse = pr.gpu().attend(q.to(DEV), dev(cu), dev(pr.lens), dev(pr.table), scale=scale,
                               with_lse=True)
    check(out, lse, ref, d, str(scale))


@pytest.mark.parametrize("c", [ATTEND[0], ATTEND[14], ATTEND[15]], ids=["short", "long", "ragged"])
def test_attend_with_a_length_bound_gives_the_same(c):
    a = run_attend(c)
    b = run_attend(c, max_len=max(c[5]))
    check(*b, where="bounded")
    assert a[0].shape == b[0].shape


def test_attend_reads_strided_queries():
    pr = Problem(3, FP8, 2, 128, 32, [50, 70])
    cu = np.array([0, 4, 9], np.int32)
    wide = pr.queries(9, 20).to(DEV)
    q = wide[:, 5:13]                                          # a slice of the heads
    ref = okv.attend(q.double().cpu().numpy(), cu, pr.lens, pr.table, pr.cache["k"], pr.scale["k"],
                     pr.cache["v"], pr.scale["v"], 0.11)
    cache = pr.gpu()
    args = dev(cu), dev(pr.lens), dev(pr.table)
    out, lse = cache.attend(q, *args, scale=0.11, with_lse=True)
    check(out, lse, ref, 128)
    head_major = q.transpose(0, 1).contiguous().transpose(0, 1)
    out2, lse2 = cache.attend(head_major, *args, scale=0.11, with_lse=True)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("nseq", [130, 4500])
def test_more_sequences_than_one_round_of_probes(nseq):
    """Sequences of 0 to 40 tokens with 0 to 3 rows, some without rows at all:
    attention, selected attention and append find every row's sequence."""
    g = np.random.default_rng(nseq)
    lens = g.integers(1, 40, nseq)
    rows = np.minimum(g.integers(0, 4, nseq), lens)
    pr = Problem(nseq, FP8, 1, 64, 16, list(lens), nan=False, pow2=True)
    S = int(rows.sum())
    cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    q = pr.queries(S, 2)
    cache = pr.gpu()
    args = dev(cu), dev(pr.lens), dev(pr.table)
    ref = okv.attend(q.double().numpy(), cu, pr.lens, pr.table, pr.cache["k"], pr.scale["k"],
                     pr.cache["v"], pr.scale["v"], 0.125)
    out, lse = cache.attend(q.to(DEV), *args, with_lse=True)
    check(out, lse, ref, 64, "all")
    idx, vl = selection(g, S, 33, cu, [int(x) for x in lens])
    ref = okv.attend(q.double().numpy(), cu, pr.lens, pr.table, pr.cache["k"], pr.scale["k"],
                     pr.cache["v"], pr.scale["v"], 0.125, idx=idx, valid_len=vl)
    out, lse = cache.attend_selected(q.to(DEV), dev(idx), dev(vl), *args, with_lse=True)
    check(out, lse, ref, 64, "selected")
    # the rows' tokens again, behind what precedes them
    x = torch.from_numpy(g.standard_normal((S, 1, 64)).astype(np.float32)).to(BF16)
    held = (lens - rows).astype(np.int32)
    want, s = okv.append(pr.cache["k"], pr.scale["k"], x.float().numpy(), cu, held, pr.table)
    cache.append(x.to(DEV), x.to(DEV), dev(cu), dev(held), dev(pr.table))
    assert np.array_equal(cache.k.view(torch.uint8).cpu().numpy(), want)
    assert np.array_equal(cache.k_scale.cpu().numpy(), s)


@pytest.mark.parametrize("dtype", [FP8, BF16])
def test_rows_past_four_gigabytes(dtype):
    """Pages at the end of buffers of 2^32 bytes and more, by every path."""
    H, d, page = 2, 128, 128
    each = H * page * d * (1 if dtype == FP8 else 2)
    pages = 2 ** 32 // each + 40
    cache = dsai.KVCache.allocate(pages, H, d, page=page, dtype=dtype, device=DEV)
    assert cache.k.numel() * cache.k.element_size() > 2 ** 32
    L, n, G = 1200, 300, 4
    ids = (pages - 1 - np.random.default_rng(1).permutation(39)[:10]).astype(np.int32)[None]
    g = torch.Generator(device=DEV).manual_seed(1)
    k, v = (torch.randn((L, H, d), generator=g, device=DEV).to(BF16) for _ in range(2))
    q = torch.randn((n, H * G, d), generator=g, device=DEV).to(BF16)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    cache.append(k, v, i32(0, L), i32(0), dev(ids))
    # a small cache with the same pages
    twin = dsai.KVCache.allocate(10, H, d, page=page, dtype=dtype, device=DEV)
    low = torch.arange(10, dtype=torch.int32, device=DEV)[None]
    twin.append(k, v, i32(0, L), i32(0), low)
    at = dev(ids[0]).long()
    for w in ("k", "v"):
        a, b = getattr(cache, w), getattr(twin, w)
        filled = L // page
        assert torch.equal(a[at[:filled]].view(torch.uint8), b[:filled].view(torch.uint8))
    idx = torch.arange(0, L, 5, dtype=torch.int32, device=DEV).repeat(n, 1)
    vl = torch.full((n,), idx.shape[1], dtype=torch.int32, device=DEV)
    for rows, name in ((1, "one row"), (n, "many rows")):
        cu = i32(0, rows)
        a = cache.attend(q[:rows], cu, i32(L), dev(ids), with_lse=True)
        b = twin.attend(q[:rows], cu, i32(L), low, with_lse=True)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]), name
        a = cache.attend_selected(q[:rows], idx[:rows], vl[:rows], cu, i32(L), dev(ids), with_lse=True)
        b = twin.attend_selected(q[:rows], idx[:rows], vl[:rows], cu, i32(L), low, with_lse=True)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]), name
    check(*twin.attend(q, i32(0, n), i32(L), low, with_lse=True), okv.attend(
        q.double().cpu().numpy(), [0, n], [L], low.cpu().numpy(),
        twin.k.view(torch.uint8).cpu().numpy() if dtype == FP8 else twin.k.float().cpu().numpy(),
        None if dtype == BF16 else twin.k_scale.cpu().numpy(),
        twin.v.view(torch.uint8).cpu().numpy() if dtype == FP8 else twin.v.float().cpu().numpy(),
        None if dtype == BF16 else twin.v_scale.cpu().numpy(), d ** -0.5), d, "twin")


def test_pair_lists_of_more_than_one_launch():
    """More rows than the lists of one launch hold: the rows behind it as well."""
    S, W, L = 17001, 4096, 200
    pr = Problem(3, FP8, 1, 64, 16, [L], pow2=True)
    g = torch.Generator(device=DEV).manual_seed(4)
    idx = torch.full((S, W), -1, dtype=torch.int32, device=DEV)
    idx[:, :40] = torch.rand((S, L), generator=g, device=DEV).argsort(1)[:, :40].sort(1).values.int()
    vl = torch.randint(1, 41, (S,), generator=g, device=DEV).int()
    q = torch.randn((S, 1, 64), generator=g, device=DEV).to(BF16)
    cache = pr.gpu()
    args = dev(np.array([0, S], np.int32)), dev(pr.lens), dev(pr.table)
    assert cache.attend_selected_workspace_bytes(S, 1, 1, W) <= 2 ** 28
    out, lse = cache.attend_selected(q, idx, vl, *args, with_lse=True)
    K, _ = okv.sequence(pr.cache["k"], pr.scale["k"], pr.table[0], L)
    V, _ = okv.sequence(pr.cache["v"], pr.scale["v"], pr.table[0], L)
    at = idx[:, :40].long()
    x = (q.double() * torch.from_numpy(K[:, 0]).to(DEV)[at]).sum(2) * 64 ** -0.5
    x.masked_fill_(torch.arange(40, device=DEV) >= vl[:, None], -float("inf"))
    p, val = x.softmax(1), torch.from_numpy(V[:, 0]).to(DEV)[at]
    ref = (p[:, :, None] * val).sum(1).cpu().numpy()[:, None]
    mag = (p[:, :, None] * val.abs()).sum(1).cpu().numpy()[:, None]
    size = (q.double().abs() * torch.from_numpy(np.abs(K[:, 0])).to(DEV)[at]).sum(2).amax(1)
    check(out, lse, (ref, x.logsumexp(1).cpu().numpy()[:, None], mag,
                     size.cpu().numpy()[:, None] * 64 ** -0.5, vl.cpu().numpy()), 64, "pairs")


def test_a_table_of_no_width_holds_nothing():
    cache = dsai.KVCache.allocate(4, 1, 64, page=16, device=DEV)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    for S in (1, 200, 1100):
        q = torch.randn((S, 1, 64), device=DEV).to(BF16)
        args = i32(0, S), i32(50), torch.empty((1, 0), dtype=torch.int32, device=DEV)
        out, lse = cache.attend(q, *args, with_lse=True)
        assert bool((out == 0).all()) and bool((lse == -float("inf")).all())
        idx = torch.arange(7, dtype=torch.int32, device=DEV).repeat(S, 1)
        out, lse = cache.attend_selected(q, idx, torch.full((S,), 7, dtype=torch.int32, device=DEV),
                                         *args, with_lse=True)
        assert bool((out == 0).all()) and bool((lse == -float("inf")).all())
        before = cache.k.view(torch.uint8).clone()
        cache.append(q, q, *args)
        assert torch.equal(before, cache.k.view(torch.uint8))


def test_a_batch_without_rows():
    cache = dsai.KVCache.allocate(4, 2, 64, page=16, device=DEV)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    q = torch.empty((0, 4, 64), dtype=BF16, device=DEV)
    idx = torch.empty((0, 9), dtype=torch.int32, device=DEV)
    for args in ((i32(0), i32(), torch.empty((0, 3), dtype=torch.int32, device=DEV)),
                 (i32(0, 0), i32(5), i32(0, 1, 2)[None])):
        assert cache.attend(q, *args).shape == q.shape
        assert cache.attend_selected(q, idx, i32(), *args).shape == q.shape
        assert cache.append(q[:, :2], q[:, :2], *args, q=q).shape == q.shape


@pytest.mark.parametrize("c", [ATTEND[6], ATTEND[18], ATTEND[19]], ids=["rows", "tiles", "ragged"])
def test_factors_that_underflow_leave_masked_positions_masked(c):
    """Key scales of 2^-117 and a factor of 1e-38: every score is 0 in fp32, the
    mask still counts, and what a row sees weighs the same."""
    dtype, d, page, heads, group, lens, rows, causal, pad = c
    pr = Problem(13, FP8, heads, d, page, lens)
    pr.scale["k"] = np.where(np.isfinite(pr.scale["k"]), np.float32(2.0 ** -117), np.float32(np.nan))
    cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    q = pr.queries(sum(rows), heads * group)
    ref = okv.attend(q.double().numpy(), cu, pr.lens, pr.table, pr.cache["k"], pr.scale["k"],
                     pr.cache["v"], pr.scale["v"], 1e-38)
    out, lse = pr.gpu().attend(q.to(DEV), dev(cu), dev(pr.lens), dev(pr.table), scale=1e-38,
                               with_lse=True)
    check(out, lse, ref, d, "underflow")


@pytest.mark.parametrize("step", [1, -1], ids=["growing", "shrinking"])
@pytest.mark.parametrize("rows", [3, 300])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [FP8, BF16])
def test_scores_that_double_from_page_to_page(dtype, d, rows, step):
    """Later keys that leave the first ones' maximum far behind (up to some 2^12,
    beyond any exponent's range), and the other way round."""
    L, page = 750, 64
    pr = Problem(17, dtype, 1, d, page, [L])
    for j in range(-(-L // page)):
        f = np.float32(2.0 ** (j if step > 0 else 11 - j))
        kind = pr.scale if dtype == FP8 else pr.cache
        kind["k"][pr.table[0, j]] *= f
    cu = np.array([0, rows], np.int32)
    q = pr.queries(rows, 8)
    ref = okv.attend(q.double().numpy(), cu, pr.lens, pr.table, pr.cache["k"], pr.scale["k"],
                     pr.cache["v"], pr.scale["v"], d ** -0.5)
    out, lse = pr.gpu().attend(q.to(DEV), dev(cu), dev(pr.lens), dev(pr.table), with_lse=True)
    check(out, lse, ref, d, f"{rows} rows")


@pytest.mark.parametrize("rows,group", [(1, 1), (1, 128)], ids=["rows", "tiles"])
def test_a_sequence_of_nearly_2_31_positions(rows, group):
    """All pages but the last are page 0 (score 0, value 1), the last is page 1
    (score 16, value -1): o = (n - 128 - 128 e^16) / (n - 128 + 128 e^16).

    The sums of ones are exact (below 2^24 a lane).  e^16 comes from an exponent
    of 24 bits below 32, off by 2^-20, so by 2^-20 relative, and exp2's last
    step; the parts, at most 512, are added in fp32: 2^-15.  Together below 2^-14."""
    page, width = 128, 2 ** 31 // 128 - 2 ** 18 // 128 - 1
    n = page * width
    k = torch.zeros((2, 1, page, 64), device=DEV)
    k[1, :, :, 0] = 16
    v = torch.ones((2, 1, page, 64), device=DEV)
    v[1] = -1
    one = torch.ones((2, 1), device=DEV)
    cache = dsai.KVCache(k.to(FP8), v.to(FP8), k_scale=one, v_scale=one)
    table = torch.zeros((1, width), dtype=torch.int32, device=DEV)
    table[0, -1] = 1
    q = torch.zeros((rows, group, 64), dtype=BF16, device=DEV)
    q[:, :, 0] = 1
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    out, lse = cache.attend(q, i32(0, rows), i32(n), table, scale=1.0, with_lse=True)
    big, rest = 128 * np.exp(16.0), float(n - 128)
    o, l = (rest - big) / (rest + big), np.log(rest + big)
    assert float((out.double() - o).abs().max()) <= 2.0 ** -8 * o + 2.0 ** -13
    assert float((lse.double() - l).abs().max()) <= 2.0 ** -14 + 2.0 ** -21 * (1 + l)
    # selected positions at both ends, by one row and by pairs of rows
    for S in (1, 1024):
        idx = i32(0, 5, n - 129, n - 128, n - 1, n, -1).repeat(S, 1)
        qs = q[:1, :1].expand(S, 1, 64)
        out, lse = cache.attend_selected(qs, idx, i32(7).repeat(S), i32(0, S), i32(n), table,
                                         scale=1.0, with_lse=True)
        o, l = (3 - 2 * np.exp(16.0)) / (3 + 2 * np.exp(16.0)), np.log(3 + 2 * np.exp(16.0))
        assert float((out.double() - o).abs().max()) <= 2.0 ** -8 + 2.0 ** -13
        assert float((lse.double() - l).abs().max()) <= 2.0 ** -14 + 2.0 ** -21 * (1 + l)


@pytest.mark.parametrize("group", [4, 64])
@pytest.mark.parametrize("dtype", [FP8, BF16])
def test_pages_that_do_not_exist_are_masked(dtype, group):
    pr = Problem(5, dtype, 2, 64, 16, [100, 60, 3000])
    pr.table[0, 2] = -1
    pr.table[1, 0] = 10 ** 9
    pr.table[1, 1:4] = np.iinfo(np.int32).min
    pr.table[2, 7:150] = 77777
    cu = np.array([0, 3, 5, 6], np.int32)
    q = pr.queries(6, 2 * group)
    ref = okv.attend(q.double().numpy(), cu, pr.lens, pr.table, pr.cache["k"], pr.scale["k"],
                     pr.cache["v"], pr.scale["v"], 64 ** -0.5)
    out, lse = pr.gpu().attend(q.to(DEV), dev(cu), dev(pr.lens), dev(pr.table), with_lse=True)
    check(out, lse, ref, 64)
    assert np.isneginf(ref[1][3]).all()                        # a row that sees missing pages only


def test_lengths_beyond_the_table_and_below_zero():
    pr = Problem(6, FP8, 1, 64, 16, [48, 30])
    table = np.ascontiguousarray(pr.table[:, :3])
    cu = np.array([0, 1, 2], np.int32)
    q = pr.queries(2, 4)
    for lens in ([48, -5], [10 ** 9, 30], [np.iinfo(np.int32).max, 0]):
        lens = np.array(lens, np.int32)
        ref = okv.attend(q.double().numpy(), cu, lens, table, pr.cache["k"], pr.scale["k"],
                         pr.cache["v"], pr.scale["v"], 0.125)
        out, lse = pr.gpu().attend(q.to(DEV), dev(cu), dev(lens), dev(table), scale=0.125,
                                   with_lse=True)
        check(out, lse, ref, 64, str(lens))


SELECTED = [
    # dtype, d, page, key heads, group, lens, rows, W
    (FP8, 128, 64, 1, 64, [700, 90], [1, 1], 67),
    (FP8, 128, 64, 2, 8, [500], [9], 129),
    (BF16, 64, 32, 2, 3, [333, 1, 0], [5, 2, 2], 51),
    (BF16, 128, 16, 4, 1, [64], [33], 1),
    (FP8, 64, 128, 1, 90, [400], [2], 2051),                    # split along the row
    (FP8, 128, 16, 2, 20, [3000], [1], 2500),
    (BF16, 64, 16, 1, 40, [900, 901], [3, 4], 700),
]


PAIRS = [
    # many rows and few heads a key head: two or four neighbouring rows share their positions
    (FP8, 128, 64, 8, 8, [300], [151], 65),
    (BF16, 64, 16, 4, 5, [333, 41, 0, 200], [160, 41, 3, 101], 40),
    (FP8, 64, 32, 16, 16, [500, 90], [64, 3], 129),
    (BF16, 128, 128, 2, 3, [700], [513], 70),
    (FP8, 128, 16, 1, 1, [260, 300], [512, 515], 33),
    (BF16, 64, 32, 8, 4, [600, 0, 70], [258, 5, 2], 70),
    (FP8, 64, 16, 8, 3, [1700], [261], 1500),                    # several lists of entries
    (FP8, 128, 16, 16, 8, [400, 30], [515, 6], 37),              # four rows in 32 columns
    (BF16, 128, 64, 16, 6, [300], [700], 21),
]


def selection(g, S, W, cu, lens, idx0=None):
    idx = np.full((S, W), -1, np.int32)
    vl = np.zeros(S, np.int32)
    for i, L in enumerate(lens):
        base = 0 if idx0 is None else int(idx0[i])
        for r in range(cu[i], cu[i + 1]):
            n = int(min(L, g.integers(0, W + 1))) if r % 3 else min(L, W)
            idx[r, :n] = np.sort(g.choice(L, n, replace=False)) + base if n else []
            vl[r] = n
    return idx, vl


@pytest.mark.parametrize("c", SELECTED, ids=range(len(SELECTED)))
@pytest.mark.parametrize("offset", [False, True])
def test_selected_matches_the_reference(c, offset):
    dtype, d, page, heads, group, lens, rows, W = c
    log(c, offset)
    pr = Problem(d + W, dtype, heads, d, page, lens)
    pad = 2
    S = sum(rows) + pad
    cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    idx0 = (np.cumsum([0] + lens[:-1]) + 13).astype(np.int32) if offset else None
    idx, vl = selection(pr.g, S, W, cu, lens, idx0)
    if offset and W > 20:       # entries of no token, in any order, and one twice
        idx[0, 3], idx[0, 5], idx[0, 7] = -1, 10 ** 9, np.iinfo(np.int32).min
        idx[0, 9] = idx[0, 8]
        vl[0] = W
        vl[1] = 10 ** 6
    q = pr.queries(S, heads * group)
    ref = okv.attend(q.double().numpy(), cu, pr.lens, pr.table, pr.cache["k"], pr.scale["k"],
                     pr.cache["v"], pr.scale["v"], d ** -0.5, idx=idx, valid_len=vl, idx0=idx0)
    out = torch.full((S, heads * group, d), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((S, heads * group), 7.0, device=DEV)
    pr.gpu().attend_selected(q.to(DEV), dev(idx), dev(vl), dev(cu), dev(pr.lens), dev(pr.table),
                             idx0=None if idx0 is None else dev(idx0), with_lse=True,
                             out=(out, lse))
    torch.cuda.synchronize()
    check(out, lse, ref, d, str(c))
    assert bool((out[S - pad:] == 7).all()) and bool((lse[S - pad:] == 7).all())


@pytest.mark.parametrize("c", PAIRS, ids=range(len(PAIRS)))
def test_neighbouring_rows_that_share_positions(c):
    """Rows that drift from one to the next, some without entries, some with
    entries of no token, out of order or twice, next to ordinary ones."""
    dtype, d, page, heads, group, lens, rows, W = c
    log(c)
    pr = Problem(d + W + 1, dtype, heads, d, page, lens, pow2=True)
    pad = 3
    S = sum(rows) + pad
    cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    idx0 = (np.arange(len(lens)) * 1000 + 5).astype(np.int32)
    idx, vl = np.full((S, W), -1, np.int32), np.zeros(S, np.int32)
    for i, L in enumerate(lens):
        score = pr.g.standard_normal(L)
        for r in range(cu[i], cu[i + 1]):
            score += 0.3 * pr.g.standard_normal(L)
            n = min(W, L) if r % 5 else int(pr.g.integers(0, min(W, L) + 1))
            if r % 11 == 3:
                n = 0
            sel = np.sort(np.argsort(-score)[:n]) + idx0[i]
            if r % 7 == 2 and n > 12:
                sel[3], sel[5], sel[9] = -1, 10 ** 9, sel[8]
            if r % 7 == 4:
                sel = sel[::-1]
            idx[r, :n], vl[r] = sel, n
    pr.table[0, 1] = 10 ** 6                                     # a page that is not there
    q = pr.queries(S, heads * group)
    ref = okv.attend(q.double().numpy(), cu, pr.lens, pr.table, pr.cache["k"], pr.scale["k"],
                     pr.cache["v"], pr.scale["v"], d ** -0.5, idx=idx, valid_len=vl, idx0=idx0)
    out = torch.full((S, heads * group, d), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((S, heads * group), 7.0, device=DEV)
    cache = pr.gpu()
    args = (q.to(DEV), dev(idx), dev(vl), dev(cu), dev(pr.lens), dev(pr.table))
    assert cache.attend_selected_workspace_bytes(S, heads * group, len(lens), W) > 0
    cache.attend_selected(*args, idx0=dev(idx0), with_lse=True, out=(out, lse))
    torch.cuda.synchronize()
    check(out, lse, ref, d, str(c))
    assert bool((out[S - pad:] == 7).all()) and bool((lse[S - pad:] == 7).all())


def test_selecting_everything_is_attention():
    """Every position selected, in ascending order: attend's rows."""
    pr = Problem(9, FP8, 2, 128, 64, [300])
    cu = np.array([0, 1], np.int32)
    q = pr.queries(1, 16).to(DEV)
    cache = pr.gpu()
    args = dev(cu), dev(pr.lens), dev(pr.table)
    a = cache.attend(q, *args, with_lse=True)
    idx = torch.arange(300, dtype=torch.int32, device=DEV)[None]
    b = cache.attend_selected(q, idx, torch.tensor([300], dtype=torch.int32, device=DEV), *args,
                              with_lse=True)
    assert float((a[1] - b[1]).abs().max()) < 1e-5
    assert float((a[0].float() - b[0].float()).abs().max()) < 2 ** -7 * float(a[0].abs().max())


APPEND = [
    # dtype, d, page, heads, held, new, rot, interleaved, query heads, padding rows
    (FP8, 128, 64, 2, [0, 63, 64, 70], [1, 1, 1, 1], 128, False, 8, 0),
    (FP8, 64, 16, 3, [5, 0, 16, 31], [40, 0, 3, 17], 32, True, 5, 3),
    (BF16, 128, 32, 2, [0, 33], [70, 1], 64, False, 0, 1),
    (BF16, 64, 16, 1, [15, 2], [2, 33], 64, True, 3, 0),
    (FP8, 128, 128, 1, [100, 0], [300, 128], 96, False, 2, 0),
    (FP8, 64, 128, 2, [1, 255], [130, 2], 16, False, 9, 2),
    (FP8, 128, 16, 2, [3], [14], 0, False, 0, 0),
    (FP8, 64, 32, 1, [0] * 70, [1] * 70, 64, False, 1, 0),       # more sequences than lanes
    (FP8, 128, 32, 1, [0, 7], [90, 90], 48, True, 1, 0),
    (BF16, 128, 128, 1, [60], [200], 112, False, 17, 0),
]


@pytest.mark.parametrize("c", APPEND, ids=range(len(APPEND)))
def test_append_matches_the_reference(c):
    dtype, d, page, heads, held, new, rot, inter, q_heads, pad = c
    log(c)
    pr = Problem(d + page + len(held), dtype, heads, d, page, [h + n for h, n in zip(held, new)],
                 nan=False)
    g = pr.g
    held = np.array(held, np.int32)
    N = sum(new) + pad
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    x = {w: torch.from_numpy((g.standard_normal((N, heads, d)) * np.exp(
        2.0 * g.standard_normal((N, heads, 1)))).astype(np.float32)).to(torch.bfloat16) for w in "kv"}
    q = torch.from_numpy(g.standard_normal((N, max(q_heads, 1), d)).astype(np.float32)).to(BF16)
    cos = sin = None
    if rot:
        ang = np.arange(max(held + np.array(new)) + 5)[:, None] * 10000.0 ** (
            -np.arange(rot // 2) / (rot // 2))
        cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    ref = {}
    for w in "kv":
        turn = (cos, sin, inter) if w == "k" else ()
        ref[w] = okv.append(pr.cache[w], pr.scale[w], x[w].float().numpy(), cu, held, pr.table, *turn)
    cache = pr.gpu()
    wide = {w: torch.zeros((N, heads + 3, d), dtype=BF16, device=DEV) for w in "kv"}
    for w in "kv":                                               # rows with strides of their own
        wide[w][:, 2:2 + heads] = x[w].to(DEV)
    q_out = torch.full((N, q_heads, d), 7.0, dtype=BF16, device=DEV) if q_heads else None
    cache.append(wide["k"][:, 2:2 + heads], wide["v"][:, 2:2 + heads], dev(cu), dev(held),
                 dev(pr.table), cos=None if cos is None else dev(cos),
                 sin=None if sin is None else dev(sin), interleaved=inter,
                 q=q[:, :q_heads].contiguous().to(DEV) if q_heads else None, q_out=q_out)
    torch.cuda.synchronize()
    for w in "kv":
        got = getattr(cache, w)
        want, s = ref[w]
        if dtype == FP8:
            a, b = got.view(torch.uint8).cpu().numpy(), want
            nan = (b & 0x7f) == 0x7f
            assert ((a & 0x7f) == 0x7f)[nan].all() and (a == b)[~nan].all(), \
                f"{w}: {int(((a != b) & ~nan).sum())} codes differ"
            assert np.array_equal(getattr(cache, w + "_scale").cpu().numpy(), s), w
        else:
            assert np.array_equal(got.float().cpu().numpy(), want), w
    if q_heads:
        got = q_out.float().cpu().numpy()
        for i in range(len(held)):
            for t in range(new[i]):
                r = cu[i] + t
                y = okv.rotate(q[r, :q_heads].float().numpy(), held[i] + t, cos, sin, inter)
                assert np.array_equal(got[r], torch.from_numpy(y).to(BF16).float().numpy()), (i, t)
        assert (got[N - pad:] == 7).all()


def test_append_of_values_that_are_not_finite_and_extreme_scales():
    pr = Problem(1, FP8, 2, 64, 16, [40, 40, 40], nan=False)
    held = np.array([5, 0, 16], np.int32)
    cu = np.array([0, 3, 20, 24], np.int32)
    x = torch.from_numpy(pr.g.standard_normal((24, 2, 64)).astype(np.float32)).to(BF16)
    x[0, 0, 3], x[1, 0, 4], x[2, 1, 5] = float("inf"), float("nan"), -float("inf")
    x[3:20] = 0                                                   # a page of zeros
    x[20:24, 0] *= 1e36
    x[20:24, 1] *= 1e-36
    want, s = okv.append(pr.cache["k"], pr.scale["k"], x.float().numpy(), cu, held, pr.table)
    cache = pr.gpu()
    cache.append(x.to(DEV), x.to(DEV), dev(cu), dev(held), dev(pr.table))
    a = cache.k.view(torch.uint8).cpu().numpy()
    nan = (want & 0x7f) == 0x7f
    assert nan.sum() == 3 and ((a & 0x7f) == 0x7f)[nan].all() and (a == want)[~nan].all()
    assert np.array_equal(cache.k_scale.cpu().numpy(), s)


def test_append_past_the_table_or_the_rotation_leaves_everything_else():
    pr = Problem(2, FP8, 1, 64, 16, [60, 60], nan=False)
    table = np.ascontiguousarray(pr.table[:, :3])                 # 48 positions
    table[1, 1] = -1                                              # a page that is not there
    held, cu = np.array([40, 10], np.int32), np.array([0, 20, 40], np.int32)
    x = torch.from_numpy(pr.g.standard_normal((40, 1, 64)).astype(np.float32)).to(BF16)
    ang = np.arange(45)[:, None] * 0.1 ** np.arange(32)
    cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    want, s = okv.append(pr.cache["k"], pr.scale["k"], x.float().numpy(), cu, held, table, cos, sin)
    cache = pr.gpu()
    q_out = torch.full((40, 1, 64), 7.0, dtype=BF16, device=DEV)
    cache.append(x.to(DEV), x.to(DEV), dev(cu), dev(held), dev(table), cos=dev(cos), sin=dev(sin),
                 q=x.to(DEV), q_out=q_out)
    assert np.array_equal(cache.k.view(torch.uint8).cpu().numpy(), want)
    assert np.array_equal(cache.k_scale.cpu().numpy(), s)
    assert bool((q_out[5:20] == 7).all()) and not bool((q_out[:5] == 7).any())
    assert not bool((q_out[20:40] == 7).any(dim=2).any())


def test_tokens_one_by_one_hold_what_a_prompt_holds():
    """80 tokens appended one at a time: every held value stays within the steps
    of its page's final scale (half a step when written, half a step for each of
    the scale's growths that made it subnormal)."""
    g = np.random.default_rng(8)
    cache = dsai.KVCache.allocate(8, 2, 64, page=32, device=DEV)
    table = torch.tensor([[5, 1, 7]], dtype=torch.int32, device=DEV)
    x = torch.from_numpy((g.standard_normal((80, 2, 64)) * np.exp(
        g.standard_normal((80, 1, 1)))).astype(np.float32)).to(BF16).to(DEV)
    cu = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    for t in range(80):
        n = torch.tensor([t], dtype=torch.int32, device=DEV)
        cache.append(x[t:t + 1], x[t:t + 1], cu, n, table)
    for pg in range(3):
        n = min(32, 80 - 32 * pg)
        pid = int(table[0, pg])
        s = cache.k_scale[pid].double()
        got = cache.k[pid].float().double()[:, :n] * s[:, None, None]
        want = x[32 * pg:32 * pg + n].double().transpose(0, 1)
        step = torch.maximum(want.abs() * 2.0 ** -4, 2.0 ** -9 * s[:, None, None])
        assert bool(((got - want).abs() <= step).all())
        assert bool((s == torch.tensor([float(okv.pow2_scale(want[h].abs().max().item()))
                                        for h in range(2)], device=DEV).double()).all())


def test_queries_may_turn_in_place():
    cache = dsai.KVCache.allocate(4, 1, 128, page=16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    q = torch.randn((9, 6, 128), generator=g, device=DEV).to(BF16)
    k = torch.randn((9, 1, 128), generator=g, device=DEV).to(BF16)
    ang = torch.arange(64, device=DEV)[:, None] * 0.9 ** torch.arange(64, device=DEV)
    args = (k, k, torch.tensor([0, 9], dtype=torch.int32, device=DEV),
            torch.tensor([7], dtype=torch.int32, device=DEV),
            torch.tensor([[0, 1, 2]], dtype=torch.int32, device=DEV))
    out = cache.append(*args, cos=ang.cos(), sin=ang.sin(), q=q)
    same = cache.append(*args, cos=ang.cos(), sin=ang.sin(), q=q, q_out=q)
    assert same is q and torch.equal(out, q)


def _decode_state(seed=4, dtype=FP8, lens=(300, 5000, 64), heads=2, q_heads=16, d=128, page=64):
    pr = Problem(seed, dtype, heads, d, page, [n + 8 for n in lens], nan=False)
    pr.lens = np.array(lens, np.int32)
    return pr, pr.gpu(), pr.queries(len(lens), q_heads).to(DEV)


def test_a_decode_step_replays_from_a_graph():
    """append, attend and attend_selected captured once and replayed with new
    tokens and lengths in place, eager work in between; each replay equals the
    eager calls on a copy of the cache."""
    pr, cache, q = _decode_state()
    B, H, d = 3, 2, 128
    g = torch.Generator(device=DEV).manual_seed(3)
    x = [torch.randn((B, H, d), generator=g, device=DEV).to(BF16) for _ in range(2)]
    cu = torch.arange(B + 1, dtype=torch.int32, device=DEV)
    held = dev(pr.lens)
    after = held + 1
    table = dev(pr.table)
    ang = torch.arange(6000, device=DEV)[:, None] * 0.8 ** torch.arange(64, device=DEV)
    cos, sin = ang.cos(), ang.sin()
    idx = torch.arange(257, dtype=torch.int32, device=DEV).repeat(B, 1)
    vl = torch.tensor([257, 100, 0], dtype=torch.int32, device=DEV)
    qr = torch.empty_like(q)
    outs = [(torch.empty_like(q), torch.empty((B, 16), device=DEV)) for _ in range(2)]
    ws = [torch.empty(cache.attend_workspace_bytes(B, 16, B, table.shape[1]), dtype=torch.uint8,
                      device=DEV),
          torch.empty(cache.attend_selected_workspace_bytes(B, 16, B, 257), dtype=torch.uint8,
                      device=DEV)]
    assert ws[0].numel() > 0

    def step(c, qr, outs, ws):
        c.append(x[0], x[1], cu, held, table, cos=cos, sin=sin, q=q, q_out=qr)
        c.attend(qr, cu, after, table, with_lse=True, workspace=ws[0], out=outs[0])
        c.attend_selected(qr, idx, vl, cu, after, table, with_lse=True, workspace=ws[1], out=outs[1])

    twin = dsai.KVCache(cache.k.clone(), cache.v.clone(), k_scale=cache.k_scale.clone(),
                        v_scale=cache.v_scale.clone())
    before = {n: getattr(cache, n).clone() for n in ("k", "v", "k_scale", "v_scale")}
    step(cache, qr, outs, ws)                                  # warm up, then take it back
    torch.cuda.synchronize()
    for n, t in before.items():
        getattr(cache, n).view(torch.uint8).copy_(t.view(torch.uint8))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(cache, qr, outs, ws)
    for r in range(5):
        graph.replay()
        torch.cuda.synchronize()
        e_qr = torch.empty_like(q)
        e_out = [(torch.empty_like(q), torch.empty((B, 16), device=DEV)) for _ in range(2)]
        step(twin, e_qr, e_out, [torch.full_like(w, 0xff) for w in ws])
        torch.cuda.synchronize()
        assert torch.equal(qr, e_qr), r
        for (a, b), (c, e) in zip(outs, e_out):
            assert torch.equal(a, c) and torch.equal(b, e), r
        for n in ("k", "v", "k_scale", "v_scale"):
            assert torch.equal(getattr(cache, n).view(torch.uint8),
                               getattr(twin, n).view(torch.uint8)), (r, n)
        for t in x + [q]:
            t.copy_(torch.randn(t.shape, generator=g, device=DEV).to(BF16) * (r + 1))
        held += 1
        after += 1


def test_a_prompt_replays_from_a_graph():
    """append of a chunk, attention of its rows in parts along the keys and over
    pairs of selections, captured once and replayed on new tokens with other work
    between; two graphs with workspaces of their own."""
    H, G, d, page, held, n, W = 2, 8, 64, 16, 900, 600, 64
    width = -(-(held + n) // page)
    g = torch.Generator(device=DEV).manual_seed(8)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    table = torch.randperm(width, generator=g, device=DEV).int()[None]
    cu, before, after = i32(0, n), i32(held), i32(held + n)
    rand = lambda *s: torch.randn(s, generator=g, device=DEV).to(BF16)  # noqa: E731
    cache, twin = (dsai.KVCache.allocate(width, H, d, page=page, device=DEV) for _ in range(2))
    old = rand(held, H, d)
    for c in (cache, twin):
        c.append(old, old, i32(0, held), i32(0), table)
    k, v, q = rand(n, H, d), rand(n, H, d), rand(n, H * G, d)
    idx = torch.randint(0, held, (n, W), generator=g, device=DEV).sort(1).values.int()
    vl = torch.randint(0, W + 1, (n,), generator=g, device=DEV).int()

    def space():
        sizes = (cache.attend_workspace_bytes(n, H * G, 1, width),
                 cache.attend_selected_workspace_bytes(n, H * G, 1, W))
        assert min(sizes) > 0
        return [torch.full((s,), 0xff, dtype=torch.uint8, device=DEV) for s in sizes], \
            [(torch.empty_like(q), torch.empty((n, H * G), device=DEV)) for _ in range(2)]

    def step(c, ws, outs):
        c.append(k, v, cu, before, table)
        c.attend(q, cu, after, table, with_lse=True, workspace=ws[0], out=outs[0])
        c.attend_selected(q, idx, vl, cu, after, table, with_lse=True, workspace=ws[1], out=outs[1])

    mine = [space(), space()]
    step(cache, *mine[0])
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in mine]
    for graph, (ws, outs) in zip(graphs, mine):
        with torch.cuda.graph(graph):
            step(cache, ws, outs)
    for r in range(4):
        graphs[r % 2].replay()
        ws, outs = space()
        step(twin, ws, outs)
        torch.cuda.synchronize()
        for (a, b), (x, y) in zip(mine[r % 2][1], outs):
            assert torch.equal(a, x) and torch.equal(b, y), r
        for t in (k, v, q):
            t.copy_(rand(*t.shape))
        idx.copy_(torch.randint(0, held, (n, W), generator=g, device=DEV).sort(1).values.int())


def test_calls_run_on_the_current_stream():
    """Work on a side stream, its inputs made there behind a long queue."""
    pr, cache, q = _decode_state(seed=6)
    cu, n, table = torch.arange(4, dtype=torch.int32, device=DEV), dev(pr.lens), dev(pr.table)
    want = cache.attend(q, cu, n, table, with_lse=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        a = torch.randn((4096, 4096), device=DEV)
        for _ in range(20):
            a = a @ a * 1e-3
        late = torch.empty_like(q)
        late.copy_(q)
        got = cache.attend(late, cu, n, table, with_lse=True)
    side.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_two_streams_at_once_with_workspaces_of_their_own():
    pr, cache, q = _decode_state(seed=7)
    cu, n, table = torch.arange(4, dtype=torch.int32, device=DEV), dev(pr.lens), dev(pr.table)
    qs = [q, (q.float() * 0.5).to(BF16)]
    want = [cache.attend(x, cu, n, table, with_lse=True) for x in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    got = [None, None]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = cache.attend(qs[i], cu, n, table, with_lse=True)
    torch.cuda.synchronize()
    for w, x in zip(want, got):
        assert torch.equal(w[0], x[0]) and torch.equal(w[1], x[1])


def test_append_select_attend_in_a_run():
    """A prompt and three decode steps of one layer: the tokens go into the cache,
    the indexer selects positions (expanded pools with the tail), attention reads
    them; every step against the reference on what the cache holds."""
    H, Hq, d, page, m, topk, hi, di = 2, 8, 64, 32, 4, 32, 4, 64
    L0, steps = 203, 3
    g = torch.Generator(device=DEV).manual_seed(12)
    rnd = lambda *s: torch.randn(s, generator=g, device=DEV).to(BF16)  # noqa: E731
    cache = dsai.KVCache.allocate(12, H, d, page=page, device=DEV)
    cache.k.view(torch.uint8).fill_(0x7f)
    cache.v.view(torch.uint8).fill_(0x7f)
    table = torch.randperm(12, device=DEV).to(torch.int32)[None]
    ang = torch.arange(400, device=DEV)[:, None] * 0.7 ** torch.arange(32, device=DEV)
    cos, sin = ang.cos(), ang.sin()
    ikeys, w = rnd(400, di), torch.randn(hi, generator=g, device=DEV)
    pooled = ikeys[:400].float().view(100, m, di).mean(1).to(BF16)
    held = 0
    for n in [L0] + [1] * steps:
        cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
        before = torch.tensor([held], dtype=torch.int32, device=DEV)
        q = cache.append(rnd(n, H, d), rnd(n, H, d), cu, before, table, cos=cos, sin=sin,
                         q=rnd(n, Hq, d))
        held += n
        T = held // m
        idx, vl = dsai.score_topk(rnd(n, hi, di), w, pooled[:T].contiguous(), m=m, topk=topk,
                                  expand=True, tail=True, q_pos0=held - n)
        lens = torch.tensor([held], dtype=torch.int32, device=DEV)
        out, lse = cache.attend_selected(q, idx, vl, cu, lens, table, with_lse=True)
        ref = okv.attend(q.double().cpu().numpy(), cu.cpu().numpy(), np.array([held]),
                         table.cpu().numpy(), cache.k.view(torch.uint8).cpu().numpy(),
                         cache.k_scale.cpu().numpy(), cache.v.view(torch.uint8).cpu().numpy(),
                         cache.v_scale.cpu().numpy(), d ** -0.5, idx=idx.cpu().numpy(),
                         valid_len=vl.cpu().numpy())
        check(out, lse, ref, d, f"held {held}")
        assert int(vl[-1]) > topk - m
        full = cache.attend(q, cu, lens, table)
        assert bool(torch.isfinite(full.float()).all())


def test_packed_documents_are_selected_and_attended_by_global_indices():
    """score_topk_varlen's rows (global key indices) with idx0 = cu_k."""
    H, Hq, d, page = 1, 4, 128, 16
    g = torch.Generator(device=DEV).manual_seed(2)
    n = [70, 1, 133]
    cu = torch.tensor([0, 70, 71, 204], dtype=torch.int32, device=DEV)
    S = 204
    q, k, v = (torch.randn((S, h, d), generator=g, device=DEV).to(BF16) for h in (Hq, H, H))
    cache = dsai.KVCache.allocate(16, H, d, page=page, dtype=BF16, device=DEV)
    table = torch.full((3, 9), -1, dtype=torch.int32, device=DEV)
    ids = torch.randperm(16, device=DEV).to(torch.int32)
    at = 0
    for i, x in enumerate(n):
        c = -(-x // page)
        table[i, :c] = ids[at:at + c]
        at += c
    cache.append(k, v, cu, torch.zeros(3, dtype=torch.int32, device=DEV), table)
    iq, ik = (torch.randn(s, generator=g, device=DEV).to(BF16) for s in ((S, 4, 64), (S, 64)))
    idx, vl = dsai._handle(BF16, False, False, 0, 0, iq.device).score_topk_varlen(
        iq, torch.randn(4, generator=g, device=DEV), ik, cu, cu, topk=24)
    lens = torch.tensor(n, dtype=torch.int32, device=DEV)
    out, lse = cache.attend_selected(q, idx, vl, cu, lens, table, idx0=cu[:3].contiguous(),
                                     with_lse=True)
    ref = okv.attend(q.double().cpu().numpy(), cu.cpu().numpy(), np.array(n), table.cpu().numpy(),
                     cache.k.float().cpu().numpy(), None, cache.v.float().cpu().numpy(), None,
                     d ** -0.5, idx=idx.cpu().numpy(), valid_len=vl.cpu().numpy(),
                     idx0=cu.cpu().numpy())
    check(out, lse, ref, d, "packed")


def test_the_binding_refuses_mismatched_tensors():
    pr, cache, q = _decode_state(seed=8)
    cu, n, table = torch.arange(4, dtype=torch.int32, device=DEV), dev(pr.lens), dev(pr.table)
    kv = torch.zeros((3, 2, 128), dtype=BF16, device=DEV)
    idx, vl = torch.zeros((3, 5), dtype=torch.int32, device=DEV), torch.zeros(3, dtype=torch.int32,
                                                                             device=DEV)
    bad = [lambda: cache.attend(q.float(), cu, n, table), lambda: cache.attend(q.cpu(), cu, n, table),
           lambda: cache.attend(q[:, :15], cu, n, table), lambda: cache.attend(q[..., :64], cu, n, table),
           lambda: cache.attend(q, cu[:3], n, table), lambda: cache.attend(q, cu.long(), n, table),
           lambda: cache.attend(q, cu, n, table[:2]), lambda: cache.attend(q, cu, n, table.T),
           lambda: cache.attend(q, cu, n, table, out=(q.float(), None)),
           lambda: cache.attend(q, cu, n, table, with_lse=True, out=(q.clone(), None)),
           lambda: cache.attend(q, cu, n, table, workspace=torch.empty(16, dtype=torch.uint8, device=DEV)),
           lambda: cache.attend(q, cu, n, table, max_len=-1),
           lambda: cache.attend(q, cu, n, table, scale=float("nan")),
           lambda: cache.attend_selected(q, idx[:2], vl, cu, n, table),
           lambda: cache.attend_selected(q, idx.long(), vl, cu, n, table),
           lambda: cache.attend_selected(q, idx, vl, cu, n, table, idx0=vl[:2]),
           lambda: cache.append(kv, kv[:2], cu, n, table), lambda: cache.append(kv[:, :1], kv, cu, n, table),
           lambda: cache.append(kv, kv, cu, n, table, cos=torch.zeros((9, 32), device=DEV)),
           lambda: cache.append(kv, kv, cu, n, table, cos=torch.zeros((9, 20), device=DEV),
                                sin=torch.zeros((9, 20), device=DEV)),
           lambda: cache.append(kv, kv, cu, n, table, q_out=kv),
           lambda: cache.append(kv[..., ::2], kv, cu, n, table),
           lambda: cache.append(kv, kv, cu, n, table, q=q, q_out=q[:1].expand(3, -1, -1))]
    for i, f in enumerate(bad):
        with pytest.raises((TypeError, ValueError, RuntimeError)):
            f()
            pytest.fail(f"call {i} was accepted")
