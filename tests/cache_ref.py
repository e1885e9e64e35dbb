"""Plain 64-bit forms of the cache-side operators, for the tests: dequantised
rows, attention, block means and scores, selection and step tables.  Written
from the definitions in include/mla_query.h; shares no code with the library."""

import math

import numpy as np
import torch

ROW_BYTES = {0: 576, 1: 656, 2: 352, 3: 576}


def float_codes(exp_bits, man_bits, bias, nan=()):
    """Values of every code of a small float format (sign on top)."""
    out = []
    for c in range(1 << (exp_bits + man_bits)):
        e, m = c >> man_bits, c % (1 << man_bits)
        frac = m / (1 << man_bits)
        out.append(math.nan if c in nan else
                   frac * 2.0 ** (1 - bias) if e == 0 else (1 + frac) * 2.0 ** (e - bias))
    return np.array(out + [-v for v in out])


E4M3 = float_codes(4, 3, 7, nan=(127,))
E2M1 = float_codes(2, 1, 1)


def rows64(raw, layout, row_scale=None):
    """FP64 keys [n, 576] of raw cache rows [n, row bytes] (numpy uint8)."""
    raw = np.asarray(raw)
    if layout in (0, 3):
        return E4M3[raw] * np.asarray(row_scale, dtype=np.float64).reshape(-1, 1)
    out = np.empty((len(raw), 576))
    if layout == 1:
        s = np.ascontiguousarray(raw[:, 512:528]).view(np.float32).astype(np.float64)
        out[:, :512] = E4M3[raw[:, :512]] * np.repeat(s, 128, axis=1)
        pe = np.ascontiguousarray(raw[:, 528:]).view(np.uint16).astype(np.uint32) << 16
        out[:, 512:] = pe.view(np.float32)
        return out
    for k in range(256):
        out[:, 2 * k] = E2M1[raw[:, k] & 15]
        out[:, 2 * k + 1] = E2M1[raw[:, k] >> 4]
    for s in range(32):
        out[:, 16 * s:16 * s + 16] *= E4M3[raw[:, 256 + 8 * (s % 4) + s // 4]][:, None]
    out[:, 512:] = E4M3[raw[:, 288:]]
    return out


def make_cache(rng, pages, page, layout):
    """A cache of finite random rows and its k_scale (numpy): latents near N(0, 1)."""
    n = pages * page
    raw = np.zeros((n, ROW_BYTES[layout]), dtype=np.uint8)
    scale = np.array([0.05], dtype=np.float32)
    if layout == 3:
        scale = rng.uniform(0.01, 0.2, size=pages).astype(np.float32)

    def e4m3(shape, lo, hi):
        # codes of magnitudes up to 2^hi: exponent fields lo..hi, any mantissa and sign
        e = rng.integers(lo + 7, hi + 8, size=shape)
        return (rng.integers(0, 2, shape) << 7 | e << 3 | rng.integers(0, 8, shape)).astype(np.uint8)

    if layout in (0, 3):
        raw[:] = e4m3(raw.shape, -2, 4)
    elif layout == 1:
        raw[:, :512] = e4m3((n, 512), 1, 7)
        s = np.exp2(rng.integers(-9, -6, size=(n, 4))).astype(np.float32)
        raw[:, 512:528] = s.view(np.uint8).reshape(n, 16)
        pe = torch.from_numpy(rng.standard_normal((n, 64), dtype=np.float32)).to(torch.bfloat16)
        raw[:, 528:] = pe.view(torch.uint8).numpy().reshape(n, 128)
    else:
        raw[:, :256] = rng.integers(0, 256, (n, 256))
        raw[:, 256:288] = (rng.integers(4, 7, (n, 32)) << 3 | rng.integers(0, 8, (n, 32)))
        raw[:, 288:] = e4m3((n, 64), -4, 0)
    return raw.reshape(pages, page, -1), scale


def make_table(rng, lens, page, pages, width=None):
    """A block table over pages handed out in random order, -1 behind each request's last."""
    need = [-(-int(n) // page) for n in lens]
    assert sum(need) <= pages
    order, at = rng.permutation(pages), 0
    bt = np.full((len(lens), width or max(1, max(need))), -1, dtype=np.int32)
    for r, k in enumerate(need):
        bt[r, :k] = order[at:at + k]
        at += k
    return bt


def positions(lens_t, page, width, pages, table_row, blocks=None):
    """(page, offset) pairs that a token looks at, in order; `blocks`: its selected ones."""
    out = []
    js = range(width) if blocks is None else blocks
    for j in js:
        if j < 0 or j >= width:
            continue
        for off in range(page):
            if j * page + off < lens_t and 0 <= table_row[j] < pages:
                out.append((int(table_row[j]), off))
    return out


def attend64(q, keys, scale):
    """(out [H, 512], lse [H], weight mass A [H, 512] = sum p |c|, logit slack) of one
    token; q [H, 576], keys [n, 576] in FP64."""
    heads = len(q)
    if len(keys) == 0:
        z = np.zeros((heads, 512))
        return z, np.full(heads, -np.inf), z, np.zeros(heads)
    x = (q @ keys.T) * scale
    m = x.max(1, keepdims=True)
    p = np.exp(x - m)
    tot = p.sum(1, keepdims=True)
    p /= tot
    # a bound of sum |q_c k_c| over the keys: what the FP32 accumulation can be off by is
    # 576 roundings of at most half a step of it
    mag = (np.abs(q) @ np.abs(keys).T).max(1) * scale
    return p @ keys[:, :512], (m + np.log(tot))[:, 0], p @ np.abs(keys[:, :512]), mag


def select_ref(scores, n, first, last, k):
    """The selected blocks of one token, ascending."""
    s = [float(v) for v in scores[:n]]
    s = [-math.inf if math.isnan(v) else v for v in s]
    for j in range(n):
        if j < first or j >= n - last:
            s[j] = math.inf
    order = sorted(range(n), key=lambda j: (-s[j], j))
    return sorted(order[:min(k, n)])


def tables_ref(new, lens, table, stack, count, page, max_tokens):
    """One step of the tables, request after request (lists and numpy copies)."""
    lens, table, stack = list(map(int, lens)), table.copy(), stack.copy()
    width, rows = table.shape[1], len(lens)
    refused = False
    out = list(lens)
    sound = [0 <= n and -(-n // page) <= width for n in lens]
    for r in range(rows):
        if not sound[r]:
            refused = True
        elif new[r] < 0:
            for j in range(-(-lens[r] // page)):
                stack[count] = table[r, j]
                count += 1
            out[r] = 0
    slots, rows_of, len_of, cu, stop = [], [], [], [0], False
    for r in range(rows):
        k = int(new[r])
        if sound[r] and k > 0:
            have, need = -(-lens[r] // page), -(-(lens[r] + k) // page)
            if need > width:
                refused = True
            elif stop or need - have > count or len(slots) + k > max_tokens:
                stop = refused = True
            else:
                for j in range(have, need):
                    count -= 1
                    table[r, j] = stack[count]
                for i in range(k):
                    p = lens[r] + i
                    slots.append(int(table[r, p // page]) * page + p % page)
                    rows_of.append(r)
                    len_of.append(p + 1)
                out[r] = lens[r] + k
        cu.append(len(slots))
    pad = max_tokens - len(slots)
    return dict(lens=out, table=table, stack=stack, count=count, slots=slots + [-1] * pad,
                token_row=rows_of + [-1] * pad, token_len=len_of + [0] * pad, cu=cu, refused=refused)
