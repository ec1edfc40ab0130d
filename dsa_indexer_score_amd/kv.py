"""The paged key/value cache: appending tokens, and attention over all of a
sequence's tokens or over the positions that the indexer selected.

As the rest of the binding, this only checks tensors, allocates outputs and
the workspace through PyTorch and passes pointers and the current HIP stream
to the library (indexer_kv_* in include/dsa_indexer.h).
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _lib
from ._lib import IDX_BF16, IDX_FP8_E4M3

_DTYPE_CODE = {torch.bfloat16: IDX_BF16, torch.float8_e4m3fn: IDX_FP8_E4M3}
_PAGES = (16, 32, 64, 128)
_INT32, _BF16, _F32 = torch.int32, torch.bfloat16, torch.float32
_FEW_KEYS = 768

# The current stream's handle without a Stream object around it: a decode step
# makes calls that take the GPU a few microseconds, and the object costs two.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _addr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


class KVCache:
    """Keys and values in pages, [pages, heads, page, d] in bf16 or e4m3, the
    latter with fp32 scales [pages, heads] (value = code * scale); d is 64 or
    128, page 16, 32, 64 or 128.

    The tensors are the caller's: append writes into them.  Calls take the
    sequences as int32 device tensors: cu [nseq + 1] (the call's rows of
    sequence i are [cu[i], cu[i+1]); rows behind cu[nseq] are left alone),
    seq_len [nseq] and the block table [nseq, width] of page ids."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, *, k_scale: Optional[torch.Tensor] = None,
                 v_scale: Optional[torch.Tensor] = None):
        if k.dtype not in _DTYPE_CODE or v.dtype != k.dtype:
            raise TypeError("k and v must both be bfloat16 or float8_e4m3fn")
        if k.dim() != 4 or v.shape != k.shape:
            raise ValueError("k and v must be [pages, heads, page, d]")
        pages, heads, page, d = k.shape
        if d not in (64, 128) or page not in _PAGES or pages < 1 or heads < 1:
            raise ValueError(f"d must be 64 or 128 and page one of {_PAGES}; got {tuple(k.shape)}")
        fp8 = k.dtype == torch.float8_e4m3fn
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if (t is not None) != fp8:
                raise ValueError("k_scale and v_scale [pages, heads] are required exactly for "
                                 "float8_e4m3fn")
            if t is not None and (t.dtype != torch.float32 or tuple(t.shape) != (pages, heads)):
                raise ValueError(f"{name} must be float32 [pages, heads]")
        for name, t in (("k", k), ("v", v), ("k_scale", k_scale), ("v_scale", v_scale)):
            if t is not None and (t.device != k.device or not t.is_cuda or not t.is_contiguous()):
                raise ValueError(f"{name} must be contiguous on the GPU of k")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.device, self.dtype, self._gpu = k.device, k.dtype, k.get_device()
        self.pages, self.heads, self.page, self.d = pages, heads, page, d
        self._lib = _lib.load()
        self._c = _lib.KvCache(_DTYPE_CODE[k.dtype], k.device.index or 0, heads, d, page, pages,
                               _addr(k), _addr(v), _addr(k_scale), _addr(v_scale))
        self._ref = ctypes.byref(self._c)

    @classmethod
    def allocate(cls, pages: int, heads: int, d: int, *, page: int = 64,
                 dtype: torch.dtype = torch.float8_e4m3fn, device="cuda") -> "KVCache":
        """A cache of uninitialised pages (append writes every slot and scale
        that attention reads)."""
        k, v = (torch.empty((pages, heads, page, d), dtype=dtype, device=device) for _ in range(2))
        s = [torch.empty((pages, heads), dtype=torch.float32, device=device) for _ in range(2)] \
            if dtype == torch.float8_e4m3fn else [None, None]
        return cls(k, v, k_scale=s[0], v_scale=s[1])

    # ---- arguments (get_device() is -1 for tensors that are not on a GPU)
    def _seqs(self, cu, seq_len, table):
        n, gpu = seq_len.numel(), self._gpu
        if seq_len.dim() != 1 or cu.dim() != 1 or cu.numel() != n + 1 or table.dim() != 2:
            raise ValueError("cu must be [nseq + 1], seq_len [nseq] and table [nseq, width]")
        rows, width = table.shape
        stride, inner = table.stride()
        if rows != n:
            raise ValueError("cu must be [nseq + 1], seq_len [nseq] and table [nseq, width]")
        if cu.dtype is not _INT32 or seq_len.dtype is not _INT32 or table.dtype is not _INT32 or \
                cu.get_device() != gpu or seq_len.get_device() != gpu or table.get_device() != gpu:
            raise ValueError(f"cu, seq_len and table must be int32 on {self.device}")
        if not (cu.is_contiguous() and seq_len.is_contiguous()) or (inner != 1 and width > 1):
            raise ValueError("cu and seq_len must be contiguous, and table's rows")
        if n <= 1:
            stride = width
        elif stride < width:
            raise ValueError("table's rows must not overlap")
        return _lib.KvSeqs(cu.data_ptr(), seq_len.data_ptr(), table.data_ptr(), stride, width, n)

    def _rows(self, name, t, rows=None, heads=None):
        """A [rows, heads, d] bf16 tensor with strides, as the library takes it."""
        if t.dtype is not _BF16 or t.get_device() != self._gpu:
            raise TypeError(f"{name} must be bfloat16 on {self.device}")
        shape = t.shape
        if len(shape) != 3 or shape[2] != self.d or (rows is not None and shape[0] != rows) or \
                (heads is not None and shape[1] != heads):
            raise ValueError(f"{name} must be [rows, heads, {self.d}]"
                             f"{'' if rows is None else f' with {rows} rows'}"
                             f"{'' if heads is None else f' and {heads} heads'}")
        s0, s1, s2 = t.stride()
        if shape[0] <= 1:
            s0 = 0
        if shape[1] <= 1:
            s1 = 0
        p = t.data_ptr()
        if (s2 != 1 or s0 % 8 or s1 % 8 or p % 16) and t.numel():
            raise ValueError(f"{name} needs contiguous channels, 16-byte aligned rows and strides "
                             f"that are multiples of 8")
        return _lib.KvRows(p, s0, s1)

    def _attend_args(self, q, cu, seq_len, table, scale, with_lse, out):
        seqs = self._seqs(cu, seq_len, table)
        rows = self._rows("q", q)
        S, Hq, _ = q.shape
        if Hq < 1 or Hq % self.heads:
            raise ValueError(f"q's heads must be a multiple of the cache's {self.heads}")
        if out is None:
            o = torch.empty_like(q, memory_format=torch.contiguous_format)
            # (empty_strided takes the host a quarter less than empty)
            lse = torch.empty_strided((S, Hq), (Hq, 1), dtype=torch.float32,
                                      device=self.device) if with_lse else None
        else:
            o, lse = out
            if o is None or o.dtype != torch.bfloat16 or o.shape != q.shape or \
                    o.device != self.device or not o.is_contiguous() or o.data_ptr() % 16:
                raise ValueError("out must be a contiguous, 16-byte aligned bfloat16 tensor of q's "
                                 "shape on the cache's device")
            if lse is not None and (lse.dtype != torch.float32 or tuple(lse.shape) != (S, Hq) or
                                    lse.device != self.device or not lse.is_contiguous()):
                raise ValueError("out lse must be a contiguous float32 [S, q_heads] tensor")
            if with_lse and lse is None:
                raise ValueError("with_lse needs an lse tensor in out")
        scale = self.d ** -0.5 if scale is None else float(scale)
        return seqs, rows, S, Hq, o, lse, scale

    def _run(self, call, size, name, workspace, keys):
        """call(ptr, bytes) with a workspace of size() bytes.  With few keys a call
        mostly needs none: it is made without asking first (9.5 against 10.7 us for
        four short rows), and the library refuses it, before it does anything, if
        it needs one after all."""
        rc = _lib.IDX_EWORKSPACE
        if workspace is None and 0 < keys <= _FEW_KEYS:
            rc = call(None, 0)
        if rc == _lib.IDX_EWORKSPACE:
            ws = self._workspace(size(), workspace)
            rc = call(_addr(ws), 0 if ws is None else ws.numel())
        _lib.check(rc, name)

    def _workspace(self, n, workspace):
        if workspace is None:
            return torch.empty_strided((n,), (1,), dtype=torch.uint8, device=self.device) if n else None
        if workspace.dtype != torch.uint8 or workspace.dim() != 1 or \
                not workspace.is_contiguous() or workspace.device != self.device or \
                workspace.numel() < n:
            raise ValueError(f"workspace must be a contiguous uint8 tensor of at least {n} bytes "
                             f"on {self.device}")
        return workspace

    # ---- calls
    def append(self, k, v, cu, seq_len, table, *, cos=None, sin=None, interleaved: bool = False,
               q=None, q_out=None):
        """New keys and values k, v [N, heads, d] (bf16, any row and head
        strides that are multiples of 8) behind the seq_len tokens that each
        sequence holds; seq_len itself is left to the caller.  cos and sin
        (float32 [positions, rot / 2]) rotate the first rot channels of the
        keys, and of q [N, q_heads, d] into q_out (allocated if None; may be
        q).  Returns q_out, or None without q; see indexer_kv_append."""
        rk = self._rows("k", k, heads=self.heads)
        N = k.shape[0]
        rv = self._rows("v", v, rows=N, heads=self.heads)
        seqs = self._seqs(cu, seq_len, table)
        if (cos is None) != (sin is None):
            raise ValueError("cos and sin come together")
        rope_rows = rot = 0
        if cos is not None:
            shape = cos.shape
            if len(shape) != 2 or shape != sin.shape:
                raise ValueError("cos and sin must be [positions, rot / 2]")
            if cos.dtype is not _F32 or sin.dtype is not _F32 or cos.get_device() != self._gpu or \
                    sin.get_device() != self._gpu or \
                    not (cos.is_contiguous() and sin.is_contiguous()):
                raise ValueError(f"cos and sin must be contiguous float32 on {self.device}")
            rope_rows, rot = shape[0], 2 * shape[1]
            if rot % 16 or not 16 <= rot <= self.d or rope_rows < 1:
                raise ValueError(f"the rotated channels must be a multiple of 16, at most {self.d}")
        rq = ro = None
        heads = 0
        if q is not None:
            rq = self._rows("q", q, rows=N)
            heads = q.shape[1]
            if q_out is None:
                q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
                ro = _lib.KvRows(q_out.data_ptr(), heads * self.d, self.d)
            else:
                ro = self._rows("q_out", q_out, rows=N, heads=heads)
        elif q_out is not None:
            raise ValueError("q_out without q")
        rc = self._lib.indexer_kv_append(self._ref, seqs, rk, rv, N, _addr(cos), _addr(sin),
                                         rope_rows, rot, int(bool(interleaved)), rq, heads, ro,
                                         _raw_stream(self._gpu))
        _lib.check(rc, "indexer_kv_append")
        return q_out

    def attend_workspace_bytes(self, S: int, q_heads: int, nseq: int, width: int,
                               max_len: int = 0) -> int:
        n = ctypes.c_size_t()
        s = _lib.KvSeqs(None, None, None, width, width, nseq)
        _lib.check(self._lib.indexer_kv_attend_workspace_bytes(self._ref, s, S, q_heads, max_len,
                                                               ctypes.byref(n)),
                   "indexer_kv_attend_workspace_bytes")
        return n.value

    def attend(self, q, cu, seq_len, table, *, scale: Optional[float] = None, causal: bool = True,
               max_len: int = 0, with_lse: bool = False,
               workspace: Optional[torch.Tensor] = None, out=None):
        """q [S, q_heads, d] bf16 over its sequences' seq_len tokens (each
        sequence's rows are its last positions) -> out [S, q_heads, d] bf16[,
        lse [S, q_heads] fp32].  scale defaults to d ** -0.5; max_len (host
        int, 0 = unknown) bounds seq_len.  out = (out, lse or None) writes
        into the caller's tensors; see indexer_kv_attend."""
        seqs, rows, S, Hq, o, lse, scale = self._attend_args(q, cu, seq_len, table, scale, with_lse,
                                                             out)
        args = (self._ref, seqs, rows, S, Hq, scale, int(bool(causal)), max_len, o.data_ptr(),
                _addr(lse))
        stream = _raw_stream(self._gpu)
        self._run(lambda ws, n: self._lib.indexer_kv_attend(*args, ws, n, stream),
                  lambda: self.attend_workspace_bytes(S, Hq, seqs.nseq, seqs.table_width, max_len),
                  "indexer_kv_attend", workspace, max_len)
        return (o, lse) if with_lse else o

    def attend_selected_workspace_bytes(self, S: int, q_heads: int, nseq: int, W: int) -> int:
        n = ctypes.c_size_t()
        s = _lib.KvSeqs(None, None, None, 1, 1, nseq)
        _lib.check(self._lib.indexer_kv_attend_selected_workspace_bytes(
            self._ref, s, S, q_heads, W, ctypes.byref(n)),
            "indexer_kv_attend_selected_workspace_bytes")
        return n.value

    def attend_selected(self, q, idx, valid_len, cu, seq_len, table, *, idx0=None,
                        scale: Optional[float] = None, with_lse: bool = False,
                        workspace: Optional[torch.Tensor] = None, out=None):
        """q [S, q_heads, d] bf16 over the positions idx[t, :valid_len[t]]
        (int32 [S, W] and [S], as score_topk returns them) of each row's
        sequence; idx0 (int32 [nseq]) is subtracted from a sequence's entries
        (cu_k or cu_tok of score_topk_varlen).  Returns out[, lse] as attend
        does; see indexer_kv_attend_selected."""
        seqs, rows, S, Hq, o, lse, scale = self._attend_args(q, cu, seq_len, table, scale, with_lse,
                                                             out)
        if idx.dim() != 2 or idx.shape[0] != S or idx.shape[1] < 1 or tuple(valid_len.shape) != (S,):
            raise ValueError("idx must be [S, W] and valid_len [S]")
        if idx.dtype is not _INT32 or valid_len.dtype is not _INT32 or \
                idx.get_device() != self._gpu or valid_len.get_device() != self._gpu or \
                not (idx.is_contiguous() and valid_len.is_contiguous()):
            raise ValueError(f"idx and valid_len must be contiguous int32 on {self.device}")
        if idx0 is not None and (idx0.dtype is not _INT32 or idx0.get_device() != self._gpu or
                                 not idx0.is_contiguous() or tuple(idx0.shape) != (seqs.nseq,)):
            raise ValueError(f"idx0 must be contiguous int32 [nseq] on {self.device}")
        W = idx.shape[1]
        args = (self._ref, seqs, rows, S, Hq, scale, idx.data_ptr(), W, valid_len.data_ptr(),
                _addr(idx0), o.data_ptr(), _addr(lse))
        stream = _raw_stream(self._gpu)
        self._run(lambda ws, n: self._lib.indexer_kv_attend_selected(*args, ws, n, stream),
                  lambda: self.attend_selected_workspace_bytes(S, Hq, seqs.nseq, W),
                  "indexer_kv_attend_selected", workspace, W)
        return (o, lse) if with_lse else o
