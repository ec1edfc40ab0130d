"""Measured cases of the paged key/value cache: appending to it, attention over
all of it, and attention over the positions that the indexer selected.

The cache holds keys and values in pages of `page` tokens, [pages, heads,
page, d], in bf16 or in e4m3 codes with one fp32 scale (a power of two) for
each page and head; a block table names the pages of each sequence.

* append    rotates new keys by their positions and writes keys and values
            behind the tokens each sequence holds; rotates the step's queries.
* attend    softmax(scale q k^T) v of every query row over its sequence's
            cache (causal), with the log-sum-exp of each row and head.
* selected  the same over the positions in the row of an index array only,
            as the indexer writes it: ascending, then -1.

Each operator has a plain form here (elementary torch operations in fp32) and
a call of the framework (`own = True`); `exact` is a 64-bit evaluation written
apart from both.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
MIN_EXP, MAX_EXP = -117, 120    # exponents of the power-of-two scales
CACHE_TYPE = {"bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one decode step of 64 sequences: latency; some pages' scales grow
        dict(name="append_decode_64", op="append", seqs=64, new_lo=1, new_hi=1, held=8191,
             q_heads=64, heads=8, d=128, page=64, dtype="fp8", rot=128, interleaved=False),
        # the prompt of one long sequence at once: bandwidth
        dict(name="append_prefill_32768", op="append", seqs=1, new_lo=32768, new_hi=32768, held=0,
             q_heads=32, heads=8, d=128, page=64, dtype="fp8", rot=128, interleaved=False),
        # chunks of a few sequences, odd lengths, half of the head rotated
        dict(name="append_ragged_bf16", op="append", seqs=7, new_lo=61, new_hi=997, held=1501,
             q_heads=12, heads=4, d=64, page=16, dtype="bf16", rot=32, interleaved=True),
        # a handful of short conversations, one token each: latency
        dict(name="attend_decode_short_4", op="attend", seqs=4, len_lo=37, len_hi=517, rows_lo=1,
             rows_hi=1, q_heads=32, heads=8, d=128, page=64, dtype="fp8"),
        # a full decode batch, contexts from a few tokens to 16K
        dict(name="attend_decode_ragged_64", op="attend", seqs=64, len_lo=11, len_hi=16384,
             rows_lo=1, rows_hi=1, q_heads=64, heads=8, d=128, page=64, dtype="fp8"),
        # one sequence over a long context: the split along the cache
        dict(name="attend_decode_long_262144", op="attend", seqs=1, len_lo=262144, len_hi=262144,
             rows_lo=1, rows_hi=1, q_heads=64, heads=8, d=128, page=64, dtype="fp8"),
        # one chunk of a long prompt behind what the cache holds already
        dict(name="attend_prefill_chunk", op="attend", seqs=1, len_lo=32768, len_hi=32768,
             rows_lo=4096, rows_hi=4096, q_heads=32, heads=8, d=128, page=64, dtype="fp8"),
        # packed prompts of odd lengths, bf16 cache, three queries a key head
        dict(name="attend_prefill_packed_bf16", op="attend", seqs=5, len_lo=333, len_hi=4001,
             rows_lo=333, rows_hi=4001, q_heads=12, heads=4, d=64, page=16, dtype="bf16"),
        # decode over the indexer's 2,048 positions, one key head for all queries
        dict(name="selected_decode_16", op="selected", seqs=16, len=65536, rows=1, topk=2048,
             pool=1, q_heads=64, heads=1, d=128, page=64, dtype="fp8"),
        # a prefill chunk over the indexer's positions, grouped heads
        dict(name="selected_prefill_2048", op="selected", seqs=1, len=65536, rows=2048, topk=2048,
             pool=1, q_heads=64, heads=8, d=128, page=64, dtype="fp8"),
        # pools of four expanded to positions with the incomplete tail (W = 2,051), bf16
        dict(name="selected_pooled_2051", op="selected", seqs=3, len=32767, rows=259, topk=2048,
             pool=4, q_heads=32, heads=4, d=64, page=32, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "attend", "attend", "selected", "selected"))
    heads = rng.choice((1, 2, 4, 8))
    c = dict(op=op, heads=heads, q_heads=heads * rng.choice((1, 2, 3, 4, 7, 8, 16)),
             d=rng.choice((64, 128)), page=rng.choice((16, 32, 64, 128)),
             dtype=rng.choice(("fp8", "fp8", "bf16")))
    if op == "append":
        c.update(seqs=_log_int(rng, 1, 128), held=rng.randint(0, 8191),
                 rot=rng.choice((c["d"], c["d"] // 2)), interleaved=rng.random() < 0.5)
        c["new_hi"] = 1 if rng.random() < 0.4 else _log_int(rng, 2, max(2, 32768 // c["seqs"]))
        c["new_lo"] = rng.randint(1, c["new_hi"])
    elif op == "attend":
        c["seqs"] = _log_int(rng, 1, 64)
        c["len_hi"] = _log_int(rng, 64, 262144 // c["seqs"])
        c["len_lo"] = rng.randint(1, c["len_hi"])
        if rng.random() < 0.5:      # decode, or a few tokens of a draft
            c["rows_hi"] = min(c["len_lo"], rng.choice((1, 1, 1, 2, 5)))
        else:                       # prefill of no more work than the largest listed case
            c["len_hi"] = min(c["len_hi"], 32768 // c["seqs"])
            c["len_lo"] = min(c["len_lo"], c["len_hi"])
            most = 4096 // min(c["seqs"], 8) * 4096 // max(4096, c["q_heads"] * c["d"])
            c["rows_hi"] = min(c["len_lo"], _log_int(rng, 16, most))
        c["rows_lo"] = rng.randint(1, c["rows_hi"])
    else:
        c["pool"] = rng.choice((1, 1, 4))
        c["topk"] = rng.choice((64, 512, 1024, 2048))
        if rng.random() < 0.5:
            c.update(seqs=_log_int(rng, 1, 32), rows=1)
        else:
            c.update(seqs=rng.randint(1, 3), rows=_log_int(rng, 2, 600))
        c["len"] = _log_int(rng, max(c["rows"], 100), 65536)
    return c


# --------------------------------------------------------------------------
# sizes that follow from a case
# --------------------------------------------------------------------------
def _spread(n, lo, hi):
    """n whole numbers in [lo, hi], spread evenly in an uneven order, the first hi."""
    return [hi if i == 0 else lo + int((hi - lo) * ((i * 0.6180339887498949) % 1.0))
            for i in range(n)]


def _plan(case):
    """Per sequence: rows of this call, tokens held when it is made."""
    if case["op"] == "append":
        new = _spread(case["seqs"], case["new_lo"], case["new_hi"])
        held = _spread(case["seqs"], case["held"] // 3, case["held"])
        return new, held
    if case["op"] == "attend":
        return (_spread(case["seqs"], case["rows_lo"], case["rows_hi"]),
                _spread(case["seqs"], case["len_lo"], case["len_hi"]))
    return [case["rows"]] * case["seqs"], [case["len"] - 3 * i if case["len"] > case["rows"] + 3 * i
                                           else case["len"] for i in range(case["seqs"])]


def _width(case):
    return case["topk"] + (case["pool"] - 1)


def work(case):
    rows, held = _plan(case)
    S, H, Hq, d = sum(rows), case["heads"], case["q_heads"], case["d"]
    es = 1 if case["dtype"] == "fp8" else 2
    if case["op"] == "append":
        pages = sum((h + n - 1) // case["page"] - h // case["page"] + 1
                    for n, h in zip(rows, held))
        return {"bytes": S * H * d * 2 * (2 + es) + S * Hq * d * 4 + S * case["rot"] * 4
                + (pages * H * 16 if es == 1 else 0) + 4 * pages,
                "flops": S * (H + Hq) * case["rot"] * 3 + (S * H * d * 4 if es == 1 else 0)}
    io = S * Hq * (d * 4 + 4)
    if case["op"] == "attend":
        pairs = sum(n * h - n * (n - 1) // 2 for n, h in zip(rows, held))
        keys = sum(held)
    else:
        per = [[min(case["topk"] // case["pool"], (h - n + t + 1) // case["pool"]) * case["pool"]
                for t in range(n)] for n, h in zip(rows, held)]
        pairs = sum(map(sum, per))
        keys = sum(min(h, sum(p)) for h, p in zip(held, per))
        io += pairs * 4
    scales = 8 * H * -(-keys // case["page"]) if es == 1 else 0
    return {"bytes": io + keys * H * d * 2 * es + scales, "flops": 4 * pairs * Hq * d}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _pow2_scale(amax):
    """The smallest power of two s with amax <= 448 s (exponent clamped)."""
    m, e = torch.frexp(amax / E4M3_MAX)                 # amax / 448 = m 2^e, m in [0.5, 1)
    e = torch.where(m == 0.5, e - 1, e)
    e = torch.where(amax > 0, e, torch.full_like(e, MIN_EXP)).clamp(MIN_EXP, MAX_EXP)
    return torch.ldexp(torch.ones_like(amax), e)


def _filled_cache(case, pages, g, dev):
    """Pages of plausible keys or values: per-channel gains, quantised per page and head."""
    H, d, page = case["heads"], case["d"], case["page"]
    gain = torch.exp(0.5 * torch.randn((1, H, 1, d), generator=g, device=dev))
    x = torch.randn((pages, H, page, d), generator=g, device=dev) * gain
    if case["dtype"] == "bf16":
        return x.to(torch.bfloat16), None
    s = _pow2_scale(x.abs().amax(dim=(2, 3)))
    return (x / s[:, :, None, None]).to(torch.float8_e4m3fn), s


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    rows, held = _plan(case)
    H, Hq, d, page = case["heads"], case["q_heads"], case["d"], case["page"]
    S, B = sum(rows), len(rows)
    total = [h + n for n, h in zip(rows, held)] if case["op"] == "append" else held
    need = [-(-t // page) for t in total]
    pages, width = sum(need) + 3, max(need)
    perm = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    col = torch.arange(width, device=dev)[None, :]
    n_pages = torch.tensor(need, device=dev)[:, None]
    first = torch.tensor([sum(need[:i]) for i in range(B)], device=dev)[:, None]
    table = torch.where(col < n_pages, perm[(first + col).clamp(max=pages - 1)],
                        torch.full((), -1, dtype=torch.int32, device=dev)).contiguous()
    st = dict(case=dict(case), scale=d ** -0.5, table=table,
              cu=torch.tensor([sum(rows[:i]) for i in range(B + 1)], dtype=torch.int32, device=dev),
              seq_len=torch.tensor(held, dtype=torch.int32, device=dev), max_rows=max(rows),
              max_len=max(held))
    st["k"], st["k_scale"] = _filled_cache(case, pages, g, dev)
    st["v"], st["v_scale"] = _filled_cache(case, pages, g, dev)
    st["q"] = (torch.randn((S, Hq, d), generator=g, device=dev) * 1.5).to(torch.bfloat16)
    if case["op"] == "append":
        for name in ("k_new", "v_new"):
            x = torch.randn((S, H, d), generator=g, device=dev)
            gain = torch.exp(0.5 * torch.randn((S, 1, 1), generator=g, device=dev))
            st[name] = (x * gain).to(torch.bfloat16)
        half = case["rot"] // 2
        ang = torch.arange(width * page, device=dev, dtype=torch.float64)[:, None] * \
            10000.0 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)
        st["cos"], st["sin"] = ang.cos().float(), ang.sin().float()
    if case["op"] == "selected":
        st["idx"], st["valid_len"] = _selection(case, rows, held, g, dev)
    if own:
        import dsa_indexer_score_amd as dsai
        st["cache"] = dsai.KVCache(st["k"], st["v"], k_scale=st["k_scale"], v_scale=st["v_scale"])
    return st


def _selection(case, rows, held, g, dev):
    """Index rows as the indexer writes them.  Neighbouring rows share about three
    quarters of their positions and drift apart over some hundred rows."""
    m, W, ksel = case["pool"], _width(case), case["topk"] // case["pool"]
    idx = torch.full((sum(rows), W), -1, dtype=torch.int32, device=dev)
    vl = torch.zeros((sum(rows),), dtype=torch.int32, device=dev)
    r0 = 0
    for n, h in zip(rows, held):
        T = h // m
        a, b = (torch.randn((1, max(T, 1)), generator=g, device=dev) for _ in range(2))
        for t0 in range(0, n, 512):
            t = torch.arange(t0, min(n, t0 + 512), device=dev)
            p = h - n + t                                          # position of the row
            P = ((p + 1) // m).clamp(max=T)                        # pools it sees
            x = torch.cos(t * 0.003)[:, None] * a + torch.sin(t * 0.003)[:, None] * b
            x = x + 0.25 * torch.randn(x.shape, generator=g, device=dev)
            x.masked_fill_(torch.arange(x.shape[1], device=dev)[None, :] >= P[:, None],
                           -math.inf)
            kk = min(ksel, x.shape[1])
            top = x.topk(kk, dim=1)
            key = torch.where(torch.isinf(top.values), torch.full_like(top.indices, T + 1),
                              top.indices).sort(dim=1).values
            pos = (key[:, :, None] * m + torch.arange(m, device=dev)).reshape(len(t), -1)
            cnt = P.clamp(max=kk) * m
            out = torch.full((len(t), W), -1, dtype=torch.int64, device=dev)
            out[:, :pos.shape[1]] = torch.where(
                torch.arange(pos.shape[1], device=dev)[None, :] < cnt[:, None], pos,
                torch.full_like(pos, -1))
            if m > 1:                                              # the incomplete pool
                tail = p + 1 - P * m
                j = torch.arange(m - 1, device=dev)[None, :]
                at = torch.where(j < tail[:, None], cnt[:, None] + j, torch.full_like(j, W))
                wide = torch.cat([out, out[:, :1]], dim=1)
                wide.scatter_(1, at, P[:, None] * m + j)
                out, cnt = wide[:, :W], cnt + tail
            idx[r0 + t0:r0 + t0 + len(t)] = out.to(torch.int32)
            vl[r0 + t0:r0 + t0 + len(t)] = cnt.to(torch.int32)
        r0 += n
    return idx, vl


# --------------------------------------------------------------------------
# the calls
# --------------------------------------------------------------------------
def run(st):
    op = st["case"]["op"]
    if own:
        c = st["cache"]
        if op == "append":
            q = c.append(st["k_new"], st["v_new"], st["cu"], st["seq_len"], st["table"],
                         cos=st["cos"], sin=st["sin"], interleaved=st["case"]["interleaved"],
                         q=st["q"])
            return _cache_outputs(st, q)
        if op == "attend":
            out, lse = c.attend(st["q"], st["cu"], st["seq_len"], st["table"], scale=st["scale"],
                                max_len=st["max_len"], with_lse=True)
        else:
            out, lse = c.attend_selected(st["q"], st["idx"], st["valid_len"], st["cu"],
                                         st["seq_len"], st["table"], scale=st["scale"],
                                         with_lse=True)
        return {"out": out, "lse": lse}
    if op == "append":
        return _plain_append(st)
    return _plain_attend(st) if op == "attend" else _plain_selected(st)


def _cache_outputs(st, q):
    out = {"q": q, "k": st["k"], "v": st["v"]}
    if st["k_scale"] is not None:
        out.update(k_scale=st["k_scale"], v_scale=st["v_scale"])
    return out


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------
def _rows_of(st):
    """Sequence and offset within it of each row."""
    S = st["q"].shape[0]
    row = torch.arange(S, device=st["q"].device)
    seq = torch.searchsorted(st["cu"].long(), row, right=True) - 1
    return seq, row - st["cu"].long()[seq]


def _rotated(x, pos, st):
    """x [N, heads, d] in fp32 with its first `rot` channels rotated by pos."""
    rot, half = st["case"]["rot"], st["case"]["rot"] // 2
    x = x.float()
    c, s = st["cos"][pos][:, None, :], st["sin"][pos][:, None, :]
    if st["case"]["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * c - b * s, b * c + a * s], dim=-1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:rot]
        y = torch.cat([a * c - b * s, b * c + a * s], dim=-1)
    return torch.cat([y, x[..., rot:]], dim=-1)


def _plain_append(st):
    page = st["case"]["page"]
    seq, t = _rows_of(st)
    held = st["seq_len"].long()
    pos = held[seq] + t
    pid = st["table"].long()[seq, pos // page]
    new_k = _rotated(st["k_new"], pos, st)
    new_v = st["v_new"].float()
    q = _rotated(st["q"], pos, st).to(torch.bfloat16)
    _plain_write(st, "k", new_k, pid, pos % page)
    _plain_write(st, "v", new_v, pid, pos % page)
    return _cache_outputs(st, q)


def _plain_write(st, which, x, pid, slot):
    cache, scale, page = st[which], st[which + "_scale"], st["case"]["page"]
    if scale is None:
        cache[pid, :, slot] = x.to(torch.bfloat16)
        return
    held, n = st["seq_len"].long(), st["cu"].long().diff()
    # what each page needs, and what the tokens it holds already were scaled by
    need = torch.zeros_like(scale).scatter_reduce(
        0, pid[:, None].expand(-1, scale.shape[1]), x.abs().amax(dim=2), "amax")
    touched = torch.zeros(scale.shape[0], dtype=torch.bool, device=scale.device)
    touched[pid] = True
    part = st["table"].long().gather(
        1, (held // page).clamp(max=st["table"].shape[1] - 1)[:, None])[:, 0].clamp(min=0)
    keeps = (held % page > 0) & (n > 0)
    old = torch.zeros_like(scale)
    old[part] = torch.where(keeps[:, None], scale[part], old[part])
    new = torch.where(touched[:, None], torch.maximum(old, _pow2_scale(need)), scale)
    # the held tokens of a page that is partly full, at the page's new scale
    codes = cache.view(torch.uint8)[part].view(torch.float8_e4m3fn)
    moved = (codes.float() * (old[part] / new[part])[:, :, None, None]).to(torch.float8_e4m3fn)
    is_held = (torch.arange(page, device=scale.device)[None, :] < (held % page)[:, None]) & \
        keeps[:, None]
    cache.view(torch.uint8)[part] = torch.where(is_held[:, None, :, None], moved.view(torch.uint8),
                                                codes.view(torch.uint8))
    cache.view(torch.uint8)[pid, :, slot] = \
        (x / new[pid][:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    scale.copy_(new)


def _sequences(st, which):
    """[B, heads, width * page, d] in fp32: each sequence's keys or values in order."""
    cache, scale = st[which], st[which + "_scale"]
    t = st["table"].long().clamp(min=0)
    if scale is None:
        x = cache[t].float()
    else:
        x = cache.view(torch.uint8)[t].view(torch.float8_e4m3fn).float() * scale[t][..., None, None]
    B, n, H, page, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(B, H, n * page, d)


def _softmax_rows(scores):
    """(unnormalised probabilities, their sum, log-sum-exp) of the last axis; -inf is masked."""
    m = scores.amax(dim=-1, keepdim=True)
    p = torch.exp(scores - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    z = p.sum(dim=-1, keepdim=True)
    return p, z, (m + torch.log(z))[..., 0]


def _plain_attend(st):
    c = st["case"]
    seq, t = _rows_of(st)
    B, n, H, G, d = st["seq_len"].shape[0], st["max_rows"], c["heads"], \
        c["q_heads"] // c["heads"], c["d"]
    dev = st["q"].device
    q = torch.zeros((B, n, H, G, d), device=dev)
    q[seq, t] = st["q"].float().reshape(-1, H, G, d)
    q = q.permute(0, 2, 1, 3, 4).reshape(B, H, n * G, d)
    k = _sequences(st, "k")
    scores = torch.matmul(q, k.transpose(2, 3)) * st["scale"]
    del k
    held, cnt = st["seq_len"].long(), st["cu"].long().diff()
    last = held[:, None] - cnt[:, None] + torch.arange(n, device=dev)     # row's own position
    last = torch.minimum(last, held[:, None] - 1)
    sees = torch.arange(scores.shape[3], device=dev) <= last[:, :, None]
    scores.view(B, H, n, G, -1).masked_fill_(~sees[:, None, :, None, :], -math.inf)
    p, z, lse = _softmax_rows(scores)
    del scores
    v = torch.where((torch.arange(p.shape[3], device=dev) < held[:, None])[:, None, :, None],
                    _sequences(st, "v"), torch.zeros((), device=dev))
    out = (torch.matmul(p, v) / z).view(B, H, n, G, d).permute(0, 2, 1, 3, 4)[seq, t]
    lse = lse.view(B, H, n, G).permute(0, 2, 1, 3)[seq, t]
    return {"out": out.reshape(-1, H * G, d).to(torch.bfloat16), "lse": lse.reshape(-1, H * G)}


def _gathered(st, which, pid, slot):
    """[S, heads, W, d] in fp32: the rows' selected keys or values."""
    cache, scale = st[which], st[which + "_scale"]
    if scale is None:
        x = cache[pid, :, slot].float()
    else:
        x = cache.view(torch.uint8)[pid, :, slot].view(torch.float8_e4m3fn).float() * \
            scale[pid][..., None]
    return x.transpose(1, 2)


def _plain_selected(st):
    c = st["case"]
    seq, _ = _rows_of(st)
    S, H, G, d = seq.shape[0], c["heads"], c["q_heads"] // c["heads"], c["d"]
    idx = st["idx"].long()
    sees = (torch.arange(idx.shape[1], device=idx.device) < st["valid_len"][:, None]) & (idx >= 0)
    pos = idx.clamp(min=0)
    pid = st["table"].long()[seq[:, None], pos // c["page"]].clamp(min=0)
    q = st["q"].float().view(S, H, G, d)
    scores = torch.matmul(q, _gathered(st, "k", pid, pos % c["page"]).transpose(2, 3)) * st["scale"]
    scores.masked_fill_(~sees[:, None, None, :], -math.inf)
    p, z, lse = _softmax_rows(scores)
    out = torch.matmul(p, _gathered(st, "v", pid, pos % c["page"])) / z
    return {"out": out.reshape(S, H * G, d).to(torch.bfloat16), "lse": lse.reshape(S, H * G)}


# --------------------------------------------------------------------------
# 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    rows, held = _plan(case)
    return _exact_append(st, rows, held) if case["op"] == "append" else \
        _exact_attention(st, rows, held)


def _exact_pages(st, which, i, n):
    """[heads, n, d] in fp64: the first n tokens of sequence i."""
    page = st["case"]["page"]
    ids = st["table"][i, :-(-n // page)].long()
    if st[which + "_scale"] is None:
        x = st[which][ids].double()
    else:
        x = st[which].view(torch.uint8)[ids].view(torch.float8_e4m3fn).double() * \
            st[which + "_scale"][ids].double()[:, :, None, None]
    return x.transpose(0, 1).flatten(1, 2)[:, :n]


def _exact_attention(st, rows, held):
    c = st["case"]
    H, G, d = c["heads"], c["q_heads"] // c["heads"], c["d"]
    S = sum(rows)
    out = torch.zeros((S, H, G, d), dtype=torch.float64, device=st["q"].device)
    lse = torch.full((S, H, G), -math.inf, dtype=torch.float64, device=st["q"].device)
    r0 = 0
    for i, (n, h) in enumerate(zip(rows, held)):
        K, V = _exact_pages(st, "k", i, h), _exact_pages(st, "v", i, h)
        step = 256 if c["op"] == "attend" else 32
        for t0 in range(0, n, step):
            t = torch.arange(t0, min(n, t0 + step), device=out.device)
            at = slice(r0 + t0, r0 + t0 + len(t))
            for j in range(H):
                q = st["q"][at].double().view(len(t), H, G, d)[:, j]
                if c["op"] == "attend":
                    x = torch.matmul(q.reshape(-1, d), K[j].T).view(len(t), G, h) * st["scale"]
                    keep = torch.arange(h, device=x.device) <= (h - n + t)[:, None]
                else:
                    sel, cnt = st["idx"][at].long(), st["valid_len"][at]
                    keep = torch.arange(sel.shape[1], device=sel.device) < cnt[:, None]
                    sel = torch.where(keep, sel, torch.zeros_like(sel))
                    x = torch.matmul(q, K[j][sel].transpose(1, 2)) * st["scale"]
                x = torch.where(keep[:, None, :], x, torch.full_like(x, -math.inf))
                lse[at, j] = torch.logsumexp(x, dim=-1)
                w = torch.softmax(x, dim=-1)
                if c["op"] == "attend":
                    out[at, j] = torch.matmul(w.reshape(-1, h), V[j]).view(len(t), G, d)
                else:
                    out[at, j] = torch.matmul(w, V[j][sel])
        r0 += n
    return {"out": out.view(S, H * G, d), "lse": lse.view(S, H * G)}


def _exact_append(st, rows, held):
    c = st["case"]
    page, rot = c["page"], c["rot"]
    res = {w: st[w].to(torch.float64) if c["dtype"] == "bf16" else st[w].float().double()
           for w in ("k", "v")}
    scale = {w: None if st[w + "_scale"] is None else st[w + "_scale"].double() for w in ("k", "v")}
    qs, r0 = [], 0
    for i, (n, h) in enumerate(zip(rows, held)):
        pos = torch.arange(h, h + n, device=st["q"].device)
        cos, sin = st["cos"][pos].double()[:, None], st["sin"][pos].double()[:, None]

        def turn(x):
            x = x.double().clone()
            first = slice(0, rot, 2) if c["interleaved"] else slice(0, rot // 2)
            second = slice(1, rot, 2) if c["interleaved"] else slice(rot // 2, rot)
            a, b = x[..., first].clone(), x[..., second].clone()
            x[..., first], x[..., second] = a * cos - b * sin, a * sin + b * cos
            return x

        qs.append(turn(st["q"][r0:r0 + n]))
        new = {"k": turn(st["k_new"][r0:r0 + n]), "v": st["v_new"][r0:r0 + n].double()}
        for w, x in new.items():
            # the touched pages, filled up to whole pages: [pages, heads, page, d]
            b0, b1 = h // page, (h + n - 1) // page + 1
            ids = st["table"][i, b0:b1].long()
            whole = torch.zeros(((b1 - b0) * page,) + x.shape[1:], dtype=torch.float64,
                                device=x.device)
            whole[h - b0 * page:h - b0 * page + n] = x
            whole = whole.view(b1 - b0, page, *x.shape[1:]).transpose(1, 2)
            mine = torch.zeros((b1 - b0) * page, dtype=torch.bool, device=x.device)
            mine[h - b0 * page:h - b0 * page + n] = True
            mine = mine.view(b1 - b0, 1, page, 1)
            before = torch.zeros_like(mine)
            before[0, 0, :h - b0 * page] = True
            if scale[w] is None:
                res[w][ids] = torch.where(mine, whole, res[w][ids])
                continue
            top = whole.abs().amax(dim=(2, 3))
            s = torch.exp2(torch.ceil(torch.log2(top / E4M3_MAX)).clamp(MIN_EXP, MAX_EXP))
            was = scale[w][ids]
            if h > b0 * page:
                s[0] = torch.maximum(s[0], was[0])
            res[w][ids] = torch.where(mine, whole / s[:, :, None, None], torch.where(
                before, res[w][ids] * (was / s)[:, :, None, None], res[w][ids]))
            scale[w][ids] = s
        r0 += n
    out = {"q": torch.cat(qs), "k": res["k"], "v": res["v"]}
    if scale["k"] is not None:
        out.update(k_scale=scale["k"], v_scale=scale["v"])
    return out
