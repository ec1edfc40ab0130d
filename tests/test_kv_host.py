"""The paged key/value cache without a GPU: refusals of the C ABI and of the
binding (nothing here reaches a device call), workspace sizes, and the
reference's own arithmetic against closed forms."""
import ctypes

import numpy as np
import pytest
import torch

from dsa_indexer_score_amd import _lib
from dsa_indexer_score_amd.kv import KVCache
from oracle import kv as okv

P = 1 << 20          # pointers that are never followed: 16-byte aligned
OUT = P + (1 << 40)
LSE = P + (1 << 41)


def cache(**kw):
    c = dict(dtype=_lib.IDX_FP8_E4M3, device=0, heads=2, d=128, page=64, pages=10, k=P, v=P,
             k_scale=P, v_scale=P)
    c.update(kw)
    return _lib.KvCache(*(c[n] for n, _ in _lib.KvCache._fields_))


def seqs(**kw):
    s = dict(cu_q=P, seq_len=P, table=P, table_stride=8, table_width=8, nseq=3)
    s.update(kw)
    return _lib.KvSeqs(*(s[n] for n, _ in _lib.KvSeqs._fields_))


def rows(ptr=P, row_stride=256, head_stride=128):
    return _lib.KvRows(ptr, row_stride, head_stride)


BAD_CACHE = [
    (dict(dtype=7), _lib.IDX_EINVAL), (dict(dtype=_lib.IDX_F32), _lib.IDX_EUNSUPPORTED),
    (dict(device=-1), _lib.IDX_EINVAL), (dict(heads=0), _lib.IDX_EINVAL),
    (dict(d=96), _lib.IDX_EUNSUPPORTED), (dict(d=0), _lib.IDX_EINVAL),
    (dict(page=8), _lib.IDX_EUNSUPPORTED), (dict(page=48), _lib.IDX_EUNSUPPORTED),
    (dict(page=256), _lib.IDX_EUNSUPPORTED), (dict(pages=0), _lib.IDX_EINVAL),
    (dict(pages=2 ** 26, heads=1), _lib.IDX_EUNSUPPORTED),      # 2^32 rows
    (dict(pages=2 ** 31), _lib.IDX_EUNSUPPORTED), (dict(k=None), _lib.IDX_EINVAL),
    (dict(v=P + 8), _lib.IDX_EINVAL), (dict(k_scale=None), _lib.IDX_EINVAL),
    (dict(dtype=_lib.IDX_BF16), _lib.IDX_EINVAL),               # scales given
    (dict(v_scale=P + 2), _lib.IDX_EINVAL),
]
BAD_SEQS = [
    (dict(nseq=-1), _lib.IDX_EINVAL), (dict(cu_q=None), _lib.IDX_EINVAL),
    (dict(seq_len=None), _lib.IDX_EINVAL), (dict(table=None), _lib.IDX_EINVAL),
    (dict(table_stride=7), _lib.IDX_EINVAL), (dict(table_width=-1), _lib.IDX_EINVAL),
    (dict(table_width=2 ** 25, table_stride=2 ** 25), _lib.IDX_EUNSUPPORTED),
    (dict(nseq=2 ** 30), _lib.IDX_EUNSUPPORTED), (dict(cu_q=P + 1), _lib.IDX_EINVAL),
]


def attend(c=None, s=None, q=None, S=5, q_heads=8, scale=0.1, causal=1, max_len=0, out=OUT,
           lse=LSE, ws=None, n=0):
    return _lib.load().indexer_kv_attend(c or cache(), s or seqs(), q or rows(), S, q_heads, scale,
                                         causal, max_len, out, lse, ws, n, None)


def selected(c=None, s=None, q=None, S=5, q_heads=8, scale=0.1, idx=P, W=9, vl=P, idx0=None,
             out=OUT, lse=LSE, ws=None, n=0):
    return _lib.load().indexer_kv_attend_selected(c or cache(), s or seqs(), q or rows(), S,
                                                  q_heads, scale, idx, W, vl, idx0, out, lse, ws,
                                                  n, None)


def append(c=None, s=None, k=None, v=None, N=5, cos=None, sin=None, rope_rows=0, rot=0,
           interleaved=0, q=None, q_heads=0, q_out=None):
    return _lib.load().indexer_kv_append(c or cache(), s or seqs(), k or rows(), v or rows(), N,
                                         cos, sin, rope_rows, rot, interleaved, q, q_heads, q_out,
                                         None)


@pytest.mark.parametrize("call", [attend, selected, append])
def test_bad_caches_and_sequences_are_refused(call):
    for kw, code in BAD_CACHE:
        assert call(c=cache(**kw)) == code, kw
    for kw, code in BAD_SEQS:
        assert call(s=seqs(**kw)) == code, kw


def test_bad_arguments_of_attend_are_refused():
    for fn in (attend, selected):
        for kw in (dict(S=-1), dict(q_heads=0), dict(q_heads=7), dict(scale=float("inf")),
                   dict(scale=float("nan")), dict(scale=3e38), dict(out=None), dict(out=P + 2), dict(lse=P + 2),
                   dict(q=rows(P + 8)), dict(q=rows(None)), dict(q=rows(row_stride=130)),
                   dict(q=rows(head_stride=-128)), dict(q=rows(row_stride=-256))):
            assert fn(**kw) == _lib.IDX_EINVAL, kw
        assert fn(S=2 ** 29) == _lib.IDX_EUNSUPPORTED
        assert fn(S=0) == 0 and fn(s=seqs(nseq=0)) == 0       # nothing to do
    empty = dict(idx=None, vl=None, q=rows(None), out=None, lse=None)
    assert selected(S=0, **empty) == 0 and selected(s=seqs(nseq=0), **empty) == 0
    assert attend(S=0, q=rows(None), out=None, lse=None) == 0
    for kw in (dict(causal=2), dict(max_len=-1)):
        assert attend(**kw) == _lib.IDX_EINVAL
    for kw in (dict(W=0), dict(idx=None), dict(vl=None), dict(idx=P + 2), dict(idx0=P + 1)):
        assert selected(**kw) == _lib.IDX_EINVAL


def test_outputs_that_overlap_the_queries_are_refused():
    """q of 5 rows, 256 elements apart, 8 heads 128 apart: 2,304 elements from first to last."""
    far = P + 2 * (4 * 256 + 7 * 128 + 128)
    for fn in (attend, selected):
        for out in (P, P + 16, far - 16, P - 2 * 5 * 8 * 128 + 16):
            assert fn(out=out) == _lib.IDX_EINVAL, out
            assert fn(lse=out if out >= P else P - 4) == _lib.IDX_EINVAL, out
        for lse in (OUT, OUT + 2 * 5 * 8 * 128 - 4, OUT - 4):
            assert fn(lse=lse) == _lib.IDX_EINVAL, lse
    ok = dict(q=rows(), q_heads=2)
    for q_out in (rows(P + 16), rows(P, 512, 128), rows(P, 256, 1280), rows(P + 2 * 4 * 256)):
        assert append(q_out=q_out, **ok) == _lib.IDX_EINVAL


def test_bad_arguments_of_append_are_refused():
    E, U = _lib.IDX_EINVAL, _lib.IDX_EUNSUPPORTED
    for kw, code in ((dict(N=-1), E), (dict(k=rows(None)), E), (dict(v=rows(P + 4)), E),
                     (dict(k=rows(row_stride=100)), E), (dict(interleaved=2), E),
                     (dict(cos=P, rope_rows=9, rot=64), E), (dict(cos=P, sin=P, rope_rows=9), E),
                     (dict(cos=P, sin=P, rope_rows=9, rot=144), E),
                     (dict(cos=P, sin=P, rope_rows=9, rot=40), U),
                     (dict(cos=P, sin=P, rope_rows=0, rot=64), E),
                     (dict(cos=P + 4, sin=P, rope_rows=9, rot=64), E), (dict(q_heads=-1), E),
                     (dict(q_heads=2), E), (dict(q_heads=2, q=rows()), E),
                     (dict(q_heads=2, q=rows(), q_out=rows(row_stride=0)), E),
                     (dict(q_heads=2, q=rows(), q_out=rows(head_stride=0)), E),
                     (dict(q_heads=4, q=rows(), q_out=rows(row_stride=256, head_stride=128)), E),
                     (dict(N=2 ** 31 - 1), U)):
        assert append(**kw) == code, kw
    assert append(N=0) == 0 and append(s=seqs(nseq=0)) == 0


def test_workspace_is_asked_for_exactly_when_rows_are_split():
    lib, n = _lib.load(), ctypes.c_size_t()
    wide = seqs(table_width=4096, table_stride=4096, nseq=1)
    size = lambda s, S, H, L: (lib.indexer_kv_attend_workspace_bytes(  # noqa: E731
        cache(), s, S, H, L, ctypes.byref(n)), n.value)
    assert size(wide, 1, 16, 256) == (0, 0)                    # one chunk
    rc, long = size(wide, 1, 16, 0)
    assert rc == 0 and long > 0
    assert size(wide, 1, 16, 4096 * 64) == (0, long) == size(wide, 1, 16, 2 ** 40)
    assert size(wide, 8192, 16, 0) == (0, 0)                   # enough rows to fill the GPU
    assert size(wide, 0, 16, 0) == (0, 0)
    # each part of a row is d + 2 floats
    assert long % (16 * (128 * 4 + 8)) == 0
    assert attend(s=wide, S=1, q_heads=16) == _lib.IDX_EWORKSPACE
    assert attend(s=wide, S=1, q_heads=16, ws=P, n=long - 1) == _lib.IDX_EWORKSPACE
    assert attend(s=wide, S=1, q_heads=16, ws=P + 8, n=long) == _lib.IDX_EWORKSPACE
    for bad in ((-1, 16, 0), (1, 15, 0), (1, 16, -1)):
        assert size(wide, *bad)[0] == _lib.IDX_EINVAL
    sel = lambda S, W: (lib.indexer_kv_attend_selected_workspace_bytes(  # noqa: E731
        cache(), wide, S, 16, W, ctypes.byref(n)), n.value)
    assert sel(1, 200) == (0, 0) and sel(4096, 5000) == (0, 0)
    # many rows: lists of 2 or 4 rows' positions (4 bytes and a bit for each row an
    # entry, a count), at most 256 MB of them at a time
    group = lambda rows: rows * 2048 * 4 + rows * rows * 2048 // 8 + 4  # noqa: E731
    assert sel(2048, 2048) == (0, (2048 // 2 + 1) * group(2))
    assert sel(4096, 2048) == (0, (4096 // 4 + 1) * group(4))
    assert sel(10 ** 6, 2048)[1] <= 2 ** 28 < sel(10 ** 6, 2048)[1] + group(4)
    rc, few = sel(1, 2048)
    assert rc == 0 and few > 0
    assert selected(s=wide, S=1, q_heads=16, W=2048) == _lib.IDX_EWORKSPACE
    assert sel(1, 0)[0] == _lib.IDX_EINVAL
    assert lib.indexer_kv_attend_workspace_bytes(cache(), wide, 1, 16, 0, None) == _lib.IDX_EINVAL


def test_positions_are_counted_in_32_bits_with_room_to_spare():
    """2^31 - 2^18 positions of a sequence, or entries of a row, are too many."""
    lib, n = _lib.load(), ctypes.c_size_t()
    for page in (16, 128):
        for width, code in ((2 ** 31 // page - 2 ** 18 // page, _lib.IDX_EUNSUPPORTED),
                            (2 ** 31 // page - 2 ** 18 // page - 1, 0)):
            s = seqs(table_width=width, table_stride=width)
            assert lib.indexer_kv_attend_workspace_bytes(cache(page=page), s, 1, 8, 0,
                                                         ctypes.byref(n)) == code
            if code:
                for call in (attend, selected, append):
                    assert call(c=cache(page=page), s=s) == code
    assert selected(W=2 ** 31 - 2 ** 18) == _lib.IDX_EUNSUPPORTED
    # blocks of a launch: the product of sequences, parts and heads passes 2^64
    many = dict(c=cache(pages=1, heads=65535, page=16), S=1, q_heads=65535, q=rows(P, 0, 128),
                lse=LSE)
    wide = 2 ** 27 - 2 ** 14 - 1
    s = seqs(nseq=2 ** 30 - 2, table_width=wide, table_stride=wide)
    assert attend(s=s, **many) == _lib.IDX_EUNSUPPORTED
    assert lib.indexer_kv_attend_selected_workspace_bytes(
        cache(), seqs(), 1, 8, 2 ** 31 - 2 ** 18, ctypes.byref(n)) == _lib.IDX_EUNSUPPORTED


def test_the_binding_refuses_tensors_that_are_not_a_cache():
    t = lambda *s, dt=torch.bfloat16: torch.zeros(s).to(dt)    # noqa: E731
    f8 = torch.float8_e4m3fn
    for kw, err in ((dict(k=t(2, 1, 16, 64), v=t(2, 1, 16, 64, dt=f8)), TypeError),
                    (dict(k=t(2, 1, 16, 64, dt=torch.float32), v=t(2, 1, 16, 64)), TypeError),
                    (dict(k=t(2, 1, 16, 64), v=t(2, 1, 16, 128)), ValueError),
                    (dict(k=t(2, 16, 64), v=t(2, 16, 64)), ValueError),
                    (dict(k=t(2, 1, 20, 64), v=t(2, 1, 20, 64)), ValueError),
                    (dict(k=t(2, 1, 16, 32), v=t(2, 1, 16, 32)), ValueError),
                    (dict(k=t(2, 1, 16, 64, dt=f8), v=t(2, 1, 16, 64, dt=f8)), ValueError),
                    (dict(k=t(2, 1, 16, 64), v=t(2, 1, 16, 64), k_scale=torch.ones(2, 1)), ValueError),
                    (dict(k=t(2, 1, 16, 64), v=t(2, 1, 16, 64)), ValueError)):   # not on a GPU
        with pytest.raises(err):
            KVCache(kw.pop("k"), kw.pop("v"), **kw)


def test_reference_scale_is_the_smallest_power_of_two():
    for x in (0.0, 1e-38, 1.0, 447.9, 448.0, 448.1, 1e30, 3.3e38):
        s = float(okv.pow2_scale(x))
        m, e = np.frexp(s)
        assert m == 0.5 and -117 <= e - 1 <= 120
        assert x <= 448 * s and (e - 1 == -117 or x > 448 * s / 2)


def test_reference_rotation_turns_pairs():
    """cos = 0, sin = 1 is a quarter turn of each pair, in both layouts."""
    x = np.arange(64, dtype=np.float32)[None]
    z, o = np.zeros((1, 16), np.float32), np.ones((1, 16), np.float32)
    y = okv.rotate(x, 0, z, o, False)
    assert np.array_equal(y[0, :16], -x[0, 16:32]) and np.array_equal(y[0, 16:32], x[0, :16])
    y = okv.rotate(x, 0, z, o, True)
    assert np.array_equal(y[0, 0:32:2], -x[0, 1:32:2]) and np.array_equal(y[0, 1:32:2], x[0, 0:32:2])
    assert np.array_equal(y[0, 32:], x[0, 32:])


def test_reference_attention_of_equal_scores_is_the_mean():
    k = np.zeros((7, 2, 64), np.float32)
    v = np.random.default_rng(0).standard_normal((7, 2, 64))
    q = np.ones((4, 64))
    out, lse, _, _ = okv.attend_row(q, k, v, 0.3)
    for h in range(4):
        assert np.allclose(out[h], v[:, h // 2].mean(0)) and np.isclose(lse[h], np.log(7))
