"""Plain reference of the paged key/value cache: numpy and torch on the CPU,
token by token, in the arithmetic of the operators' definitions.

append works on copies in fp32, product by product, because the codes and
scales it has to give are those of the definition, not of real numbers;
attention is computed in fp64 and comes with what bounds the kernel's error.
"""
import numpy as np
import torch

E4M3_MAX = 448.0


def to_e4m3(x):
    """fp32 array -> e4m3 bytes, rounded to nearest even (NaN and inf: NaN)."""
    x = np.asarray(x, np.float32).copy()
    x[~np.isfinite(x)] = np.nan
    return torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def from_e4m3(b):
    b = np.ascontiguousarray(b)
    return torch.from_numpy(b).view(torch.float8_e4m3fn).float().numpy()


def pow2_scale(amax):
    """The smallest power of two s, 2^-117 <= s <= 2^120, with amax <= 448 s."""
    e = -117
    while e < 120 and float(amax) > E4M3_MAX * 2.0 ** e:
        e += 1
    return np.float32(2.0 ** e)


def rotate(x, pos, cos, sin, interleaved):
    """x [..., d] fp32, one token's heads, each product and sum rounded to fp32."""
    if cos is None:
        return x.astype(np.float32)
    y = x.astype(np.float32).copy()
    half = cos.shape[1]
    first = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    second = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    a, b = y[..., first].copy(), y[..., second].copy()
    c, s = cos[pos].astype(np.float32), sin[pos].astype(np.float32)
    y[..., first] = a * c - b * s
    y[..., second] = b * c + a * s
    return y


def append(cache, scale, x, cu, seq_len, table, cos=None, sin=None, interleaved=False):
    """cache [pages, heads, page, d]: float32 values (bf16 caches) or uint8 codes
    with scale [pages, heads]; x [N, heads, d] fp32.  Returns new (cache, scale)."""
    cache, scale = cache.copy(), None if scale is None else scale.copy()
    page = cache.shape[2]
    cap = table.shape[1] * page
    for i in range(len(seq_len)):
        held = min(max(int(seq_len[i]), 0), cap)
        new = {}                                     # page number -> [(slot, values)]
        for t in range(int(cu[i + 1]) - int(cu[i])):
            pos = held + t
            if pos >= cap or (cos is not None and pos >= cos.shape[0]):
                break
            y = rotate(x[cu[i] + t], pos, cos, sin, interleaved)
            new.setdefault(pos // page, []).append((pos % page, y))
        for pg, toks in new.items():
            pid = int(table[i, pg])
            if not 0 <= pid < cache.shape[0]:
                continue
            if scale is None:
                for slot, y in toks:
                    cache[pid, :, slot] = torch.from_numpy(y).to(torch.bfloat16).float().numpy()
                continue
            keep = max(0, held - pg * page)          # tokens of the sequence in the page already
            for h in range(cache.shape[1]):
                vals = np.stack([y[h] for _, y in toks])
                mag = np.abs(vals[np.isfinite(vals)])
                s = pow2_scale(mag.max() if mag.size else 0.0)
                if keep and scale[pid, h] >= s:
                    s = scale[pid, h]
                elif keep:
                    ratio = np.float32(scale[pid, h]) / s
                    cache[pid, h, :keep] = to_e4m3(from_e4m3(cache[pid, h, :keep]) * ratio)
                inv = np.float32(1.0) / s
                for slot, y in toks:
                    cache[pid, h, slot] = to_e4m3(y[h] * inv)
                scale[pid, h] = s
    return cache, scale


def sequence(cache, scale, table_row, n):
    """[n, heads, d] fp64 values of a sequence's first n tokens, and which of them
    lie on a page that exists."""
    pages, heads, page, d = cache.shape
    out = np.zeros((n, heads, d))
    there = np.zeros(n, bool)
    for pos in range(0, n, page):
        pid = int(table_row[pos // page])
        if not 0 <= pid < pages:
            continue
        m = min(page, n - pos)
        x = from_e4m3(cache[pid]).astype(np.float64) * scale[pid].astype(np.float64)[:, None, None] \
            if scale is not None else cache[pid].astype(np.float64)
        out[pos:pos + m] = x[:, :m].transpose(1, 0, 2)
        there[pos:pos + m] = True
    return out, there


def attend_row(q, k, v, scale):
    """q [Hq, d], k and v [n, heads, d] of the tokens that the row sees (fp64).
    Returns out [Hq, d], lse [Hq], sum of p |v| [Hq, d], and scale sum |q| |k| at
    its largest [Hq] (what the rounding of a score is relative to)."""
    Hq, d = q.shape
    n, heads, _ = k.shape
    G = Hq // heads
    out, mag = np.zeros((Hq, d)), np.zeros((Hq, d))
    lse, size = np.full(Hq, -np.inf), np.zeros(Hq)
    if n == 0:
        return out, lse, mag, size
    for j in range(heads):
        qj = q[j * G:(j + 1) * G]
        s = scale * (qj @ k[:, j].T)
        m = s.max(axis=1, keepdims=True)
        p = np.exp(s - m)
        z = p.sum(axis=1, keepdims=True)
        at = slice(j * G, (j + 1) * G)
        out[at], mag[at] = (p / z) @ v[:, j], (p / z) @ np.abs(v[:, j])
        lse[at] = (m + np.log(z))[:, 0]
        size[at] = abs(scale) * (np.abs(qj) @ np.abs(k[:, j]).T).max(axis=1)
    return out, lse, mag, size


def attend(q, cu, seq_len, table, k, k_scale, v, v_scale, scale, causal=True, idx=None,
           valid_len=None, idx0=None):
    """All rows of packed sequences; rows of no sequence come back as NaN."""
    S, Hq, d = q.shape
    out, mag = np.full((S, Hq, d), np.nan), np.zeros((S, Hq, d))
    lse, size = np.full((S, Hq), np.nan), np.zeros((S, Hq))
    keys = np.zeros(S, np.int64)
    cap = table.shape[1] * k.shape[2]
    for i in range(len(seq_len)):
        L = min(max(int(seq_len[i]), 0), cap)
        K, there = sequence(k, k_scale, table[i], L)
        V, _ = sequence(v, v_scale, table[i], L)
        n = int(cu[i + 1]) - int(cu[i])
        for t in range(n):
            row = int(cu[i]) + t
            if idx is None:
                sees = np.arange(min(max(L - n + t + 1, 0), L) if causal else L)
            else:
                e = idx[row, :min(max(int(valid_len[row]), 0), idx.shape[1])].astype(np.int64)
                e = e - (0 if idx0 is None else int(idx0[i]))
                sees = e[(e >= 0) & (e < L)]
            sees = sees[there[sees]] if len(sees) else sees.astype(np.int64)
            out[row], lse[row], mag[row], size[row] = attend_row(q[row], K[sees], V[sees], scale)
            keys[row] = len(sees)
    return out, lse, mag, size, keys
