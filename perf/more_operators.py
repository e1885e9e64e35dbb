"""The prompt's side of a latent-attention layer: what is measured, in plain torch form.

Four operators around a prompt and the paged latent KV cache that it fills:

* ``rope``    rotary positions with one or several axes (time, height, width) of query rows;
* ``store``   cache rows of many tokens written in one of the 8- and 4-bit layouts (norm, rotation and
              quantisation in one pass), and what was written read back;
* ``read``    the cached rows of ragged requests read back as BF16 rows, one request after another;
* ``attend``  attention of packed documents over expanded keys: causal, with a two-way prefix, capped
              scores or a bias by distance.

``run`` computes them with elementary torch operations in 32 bits, or, with ``own`` set, through the
package's entry points.
"""

import math

import torch

own = False

LATENT, ROPE, ROW = 512, 64, 576
NOPE, VALUE = 128, 128
QK = NOPE + ROPE
# cache layouts: the package's numbers, bytes of one token's row
LAYOUTS = {"e4m3": 0, "ds": 1, "nvfp4": 2, "e4m3_page": 3}
ROW_BYTES = {"e4m3": 576, "ds": 656, "nvfp4": 352, "e4m3_page": 576}
SOFTMAX_SCALE = QK ** -0.5
EPS = 1e-6
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
# which axis turns each of the 32 pairs: time for the slow ones, height and width for the rest
SECTIONS = (8, 12, 12)


def listed():
    return [
        # the queries of a full decode batch: latency alone
        dict(name="rope_b64_h128_rows", op="rope", tokens=64, heads=128, axes=1, interleaved=True, rows=True, far=65536),
        # a prompt of text and images: three axes, the halves of a head as pairs
        dict(name="rope_8191_h16_axes3", op="rope", tokens=8191, heads=16, axes=3, interleaved=False, rows=False,
             far=1000000),
        # what a decode step of 64 requests appends, kept normalised by its caller
        dict(name="store_64_ds", op="store", requests=64, shortest=1, longest=1, before=4000, page=64, layout="ds",
             norm=False, axes=0, fused=True, pad=0),
        # chunks of eight prompts: norm, rotation and quantisation
        dict(name="store_16k_e4m3_norm_rope", op="store", requests=8, shortest=2000, longest=2048, before=1000, page=64,
             layout="e4m3", norm=True, axes=1, fused=True, pad=5),
        # the cached context of one short request
        dict(name="read_1x700_ds", op="read", requests=1, shortest=700, longest=700, page=64, layout="ds", skip=0),
        # the contexts of eight long requests, a scale for each page
        dict(name="read_8x16k_e4m3_page", op="read", requests=8, shortest=9001, longest=16384, page=64,
             layout="e4m3_page", skip=0),
        # one short prompt at 16 local heads (tensor parallel over many ranks)
        dict(name="attend_1x512_h16", op="attend", docs=1, shortest=512, longest=512, context=0, heads=16, causal=True,
             prefix=0, cap=0.0, bias=False, pad=0),
        # one long prompt
        dict(name="attend_1x8192_h16", op="attend", docs=1, shortest=8192, longest=8192, context=0, heads=16, causal=True,
             prefix=0, cap=0.0, bias=False, pad=0),
        # a packed batch of short documents, scores capped
        dict(name="attend_24x1000_h64_cap", op="attend", docs=24, shortest=100, longest=1000, context=0, heads=64,
             causal=True, prefix=0, cap=30.0, bias=False, pad=0),
        # prompts whose first part looks both ways, biased by distance, two padded tokens behind the last
        dict(name="attend_4x2000_h40_prefix_bias", op="attend", docs=4, shortest=1001, longest=2000, context=0, heads=40,
             causal=True, prefix=700, cap=0.0, bias=True, pad=2),
        # a chunk of a prompt behind what its request has in the cache, scores capped
        dict(name="attend_2x300_on_16k_h16_cap", op="attend", docs=2, shortest=300, longest=300, context=16000, heads=16,
             causal=True, prefix=0, cap=50.0, bias=False, pad=0),
        # one token over a long context
        dict(name="attend_1_on_64k_h16", op="attend", docs=1, shortest=1, longest=1, context=65535, heads=16, causal=True,
             prefix=0, cap=0.0, bias=False, pad=0),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["rope", "store", "store", "read", "attend", "attend", "attend", "attend"])
    if op == "rope":
        heads = rng.choice([1, 3, 8, 16, 24, 64, 127, 128])
        return dict(op=op, tokens=_log(rng, 1, 131072 // heads), heads=heads, axes=rng.choice([1, 1, 2, 3]),
                    interleaved=rng.choice([True, False]), rows=rng.choice([True, False]), far=_log(rng, 100, 1 << 30))
    page, layout = rng.choice([1, 7, 16, 32, 48, 64, 64, 64, 100, 128]), rng.choice(sorted(LAYOUTS))
    requests = _log(rng, 1, 64)
    if op == "store":
        longest = _log(rng, 1, 16384 // requests if layout != "nvfp4" else max(1, 2048 // requests))
        return dict(op=op, requests=requests, shortest=rng.randint(max(1, longest // 4), longest), longest=longest,
                    before=rng.choice([0, rng.randint(1, 5000)]), page=page, layout=layout,
                    norm=rng.choice([True, True, False]), axes=rng.choice([0, 1, 1, 3]),
                    fused=rng.choice([True, False]), pad=rng.choice([0, 0, 3]))
    if op == "read":
        longest = _log(rng, 1, min(65536, 131072 // requests))
        return dict(op=op, requests=requests, shortest=rng.randint(max(1, longest // 8), longest), longest=longest,
                    page=page, layout=layout, skip=rng.choice([0, 0, rng.randint(0, longest)]))
    heads, docs = rng.choice([1, 3, 8, 16, 16, 24, 40, 64, 128]), _log(rng, 1, 64)
    room = (1 << 30) // (docs * heads)  # scores of a document and head
    longest = _log(rng, 1, min(8192, math.isqrt(room), (1 << 22) // (docs * heads)))
    context = rng.choice([0, 0, 1, -1])
    if context > 0:
        context = _log(rng, 1, max(1, min(room // longest, (1 << 22) // (docs * heads)) - longest))
    elif context < 0:
        context = -rng.randint(0, longest)
    return dict(op=op, docs=docs, shortest=rng.randint(max(1, longest // 4), longest), longest=longest, context=context,
                heads=heads, causal=rng.choice([True, True, True, False]), prefix=rng.choice([0, 0, rng.randint(1, longest)]),
                cap=rng.choice([0.0, 0.0, 20.0, 50.0]), bias=rng.choice([False, False, True]), pad=rng.choice([0, 0, 3]))


# ---------------------------------------------------------------- inputs


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _host(seed):
    return torch.Generator().manual_seed(int(seed))


def _normal(shape, g, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def _lengths(case, n, h):
    """Ragged lengths, spread evenly between the case's shortest and longest, in random order."""
    t = torch.arange(n) / max(1, n - 1)
    return (case["longest"] - ((case["longest"] - case["shortest"]) * t).long())[torch.randperm(n, generator=h)]


def _inv_freq():
    """Radians a position for each of the 32 pairs, in 64 bits."""
    return 10000.0 ** (-torch.arange(0, ROPE, 2, dtype=torch.float64) / ROPE)


def _axis(axes):
    """The axis of each pair."""
    a = torch.arange(len(SECTIONS)).repeat_interleave(torch.tensor(SECTIONS))
    return a.clamp_max(axes - 1).to(torch.int32)


def _positions(axes, tokens, far, h):
    """Positions [axes, tokens]: time runs on from a random start, the other axes lie within a picture."""
    start = int(torch.randint(0, max(1, far - tokens), (1,), generator=h))
    time = torch.arange(start, start + tokens)
    rest = torch.randint(0, 200, (axes - 1, tokens), generator=h)
    return torch.cat([time[None], rest]).to(torch.int32)


def _paged(lens, page, h):
    """Block table of requests with these lengths over pages handed out in random order, and the number of pages."""
    need = (lens + page - 1) // page
    pages = int(need.sum()) + 3
    at = need.cumsum(0) - need
    j = torch.arange(int(need.max()))
    order = torch.randperm(pages, generator=h).to(torch.int32)
    table = torch.where(j < need[:, None], order[(at[:, None] + j).clamp_max(pages - 1)], -1)
    return table.to(torch.int32), pages


def _cache(layout, pages, page, g):
    """A cache [pages, page, row bytes] of normalised latents and rope keys, and its scales."""
    n, dev = pages * page, "cuda"
    x = torch.randn((n, ROW), generator=g, device=dev)
    lat, pe = x[:, :LATENT], x[:, LATENT:]
    code = lambda v: v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)  # noqa: E731
    scale = torch.full((1,), 0.05, device=dev)
    if layout == "e4m3":
        rows = code(x / scale)
    elif layout == "e4m3_page":
        scale = torch.exp2(torch.rand(pages, generator=g, device=dev) * 3.0 - 6.0)
        rows = code(x / scale.repeat_interleave(page)[:, None])
    elif layout == "ds":
        s = (lat.abs().view(n, 4, 128).amax(2) / 448.0).clamp_min(1e-4).log2().ceil().exp2()
        rows = torch.cat([code(lat.view(n, 4, 128) / s[..., None]).view(n, LATENT), s.view(torch.uint8).view(n, 16),
                          pe.to(torch.bfloat16).contiguous().view(torch.uint8).view(n, 128)], 1)
    else:
        s = code((lat.abs().view(n, 32, 16).amax(2) / 6.0).clamp_min(2.0 ** -9))
        nib = torch.randint(0, 256, (n, 256), generator=g, device=dev, dtype=torch.uint8)
        place = torch.arange(32, device=dev)
        scales = torch.empty_like(s)
        scales[:, 8 * (place % 4) + place // 4] = s
        rows = torch.cat([nib, scales, code(pe)], 1)
    return rows.view(pages, page, -1), scale


def prepare(case, seed):
    g, h, dev = _gen(seed), _host(seed), "cuda"
    op, s = case["op"], dict(case=case)
    if op == "rope":
        n, heads, axes = case["tokens"], case["heads"], case["axes"]
        x = _normal((n, heads, ROW if case["rows"] else ROPE), g, 0.78)
        pos = _positions(axes, n, case["far"], h)
        s.update(x=x[..., -ROPE:], pos=(pos if axes > 1 else pos[0]).to(dev), inv_freq=_inv_freq(), axis=_axis(axes),
                 out=torch.empty((n, heads, ROPE), dtype=torch.bfloat16, device=dev))
    elif op in ("store", "read"):
        new = _lengths(case, case["requests"], h)
        before = torch.full_like(new, case["before"]) if op == "store" else (new - 1).clamp_max(case["skip"])
        lens = before + new if op == "store" else new
        table, pages = _paged(lens, case["page"], h)
        count = lens - before  # the rows that are read
        cu = torch.cat([torch.zeros(1, dtype=torch.long), count.cumsum(0)])
        total = int(cu[-1])
        s.update(table=table.to(dev), first=before.to(torch.int32).to(dev), cu=cu.to(torch.int32).to(dev), pages=pages,
                 back=torch.zeros((total, ROW), dtype=torch.bfloat16, device=dev))
        if op == "read":
            s["cache"], s["scale"] = _cache(case["layout"], pages, case["page"], g)
            return _with_handles(s)
        req = torch.arange(case["requests"]).repeat_interleave(count)
        pos = before[req] + torch.arange(total) - cu[req]
        slots = table[req, pos // case["page"]].long() * case["page"] + pos % case["page"]
        pad = case["pad"]
        n = total + pad
        slots = torch.cat([slots, torch.full((pad,), -1)])
        pos = torch.cat([pos, torch.zeros(pad, dtype=torch.long)]).to(torch.int32)
        if case["axes"] > 1:
            pos = torch.cat([pos[None], torch.randint(0, 200, (case["axes"] - 1, n), generator=h).to(torch.int32)])
        wide = _normal((n, 2112 if case["fused"] else ROW), g)
        rows = wide[:, -ROW:]  # a fused q_a | kv_c | k_pe row, or a row of its own
        scale = torch.full((1,), 0.05, device=dev)
        if case["layout"] == "e4m3_page":
            scale = torch.exp2(torch.rand(pages, generator=g, device=dev) * 3.0 - 6.0)
        s.update(kv_c=rows[:, :LATENT], k_pe=rows[:, LATENT:], slots=slots.to(dev), pos=pos.to(dev), scale=scale, n=n,
                 total=total, gamma=(1.0 + 0.1 * torch.randn(LATENT, generator=g, device=dev)).to(torch.bfloat16),
                 inv_freq=_inv_freq(), axis=_axis(max(1, case["axes"])),
                 cache=torch.zeros((pages, case["page"], ROW_BYTES[case["layout"]]), dtype=torch.uint8, device=dev),
                 rows=torch.empty((n, ROW), dtype=torch.bfloat16, device=dev))
    else:
        heads = case["heads"]
        nq = _lengths(case, case["docs"], h)
        nk = (nq + case["context"]).clamp_min(0)
        zero = torch.zeros(1, dtype=torch.long)
        cu_q, cu_k = torch.cat([zero, nq.cumsum(0)]), torch.cat([zero, nk.cumsum(0)])
        tq, tk = int(cu_q[-1]) + case["pad"], max(1, int(cu_k[-1]))
        q = _normal((tq, heads, QK), g, 1.5)
        kv = _normal((tk, heads, NOPE + VALUE), g)  # a latent row's keys and values, head after head
        s.update(q=q, kv=kv, k_pe=_normal((tk, ROPE), g), cu_q=cu_q.to(torch.int32).to(dev),
                 cu_k=cu_k.to(torch.int32).to(dev), prefix=None, slopes=None,
                 out=torch.zeros((tq, heads, VALUE), dtype=torch.bfloat16, device=dev),
                 lse=torch.zeros((tq, heads), device=dev))
        if case["prefix"]:
            s["prefix"] = torch.randint(0, case["prefix"] + 1, (case["docs"],), generator=h).to(torch.int32).to(dev)
        if case["bias"]:  # what a position further away costs, head by head
            s["slopes"] = torch.exp2(-8.0 * torch.arange(1, heads + 1, device=dev) / heads)
    return _with_handles(s)


def _with_handles(s):
    """What a program makes once and keeps: the rotation's frequencies, the attention's workspace."""
    if own:
        from mla_query_projection_gb300 import runner as R

        if "inv_freq" in s:
            s["rotary"] = R.Rotary(s["inv_freq"], s["axis"], interleaved=s["case"].get("interleaved", True))
        if s["case"]["op"] == "attend":
            s["attn"] = R.PromptAttention(s["case"]["heads"])
    return s


# ---------------------------------------------------------------- the framework's calls


def _own(s):
    from mla_query_projection_gb300 import runner as R

    c = s["case"]
    if c["op"] == "rope":
        s["rotary"].apply(s["x"], s["pos"], out=s["out"])
        return {"out": s["out"]}
    if c["op"] == "attend":
        q, kv = s["q"], s["kv"]
        s["attn"].attend(q[..., :NOPE], q[..., NOPE:], kv[..., :NOPE], s["k_pe"], kv[..., NOPE:], s["cu_q"], SOFTMAX_SCALE,
                         cu_k=s["cu_k"], causal=c["causal"], prefix=s["prefix"], softcap=c["cap"], slopes=s["slopes"],
                         out=s["out"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    layout = LAYOUTS[c["layout"]]
    if c["op"] == "store":
        R.cache_write(s["kv_c"], s["k_pe"], s["slots"], s["cache"], layout, k_scale=s["scale"],
                      gamma=s["gamma"] if c["norm"] else None, eps=EPS, rotary=s["rotary"] if c["axes"] else None,
                      positions=s["pos"] if c["axes"] else None, rows=s["rows"])
    R.cache_read(s["cache"], layout, s["scale"], s["table"], s["cu"], s["back"], first=s["first"])
    return {"rows": s["rows"], "back": s["back"]} if c["op"] == "store" else {"rows": s["back"]}


# ---------------------------------------------------------------- the plain forms


def _rotate(x, pos, inv_freq, axis, interleaved):
    """x [tokens, heads, 64] in 32 bits, turned; the angles come from 64 bits."""
    pos = pos if pos.dim() == 2 else pos[None]
    angle = pos.double()[axis.long().to(x.device)].T * inv_freq.to(x.device)  # [tokens, 32]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    x = x.unflatten(-1, (32, 2)) if interleaved else x.unflatten(-1, (2, 32)).transpose(-1, -2)
    y = torch.stack([x[..., 0] * cos - x[..., 1] * sin, x[..., 1] * cos + x[..., 0] * sin], -1)
    return y.flatten(-2) if interleaved else y.transpose(-1, -2).flatten(-2)


def _plain_rope(s):
    y = _rotate(s["x"].float(), s["pos"], s["inv_freq"], s["axis"], s["case"]["interleaved"])
    return {"out": y.to(torch.bfloat16)}


def _held8(x):
    """x as an E4M3 code holds it, in 32 bits."""
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).float()


def _held4(x):
    """x as an E2M1 code holds it: to the nearest, of two as near to the even code."""
    a = x.abs()
    at = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)).long()
    return torch.tensor(E2M1, device=x.device)[at] * torch.where(x < 0, -1.0, 1.0)


def _held(n, pe, layout, scale):
    """The values [tokens, 576] that a cache row holds of a normalised row and its rope part."""
    if layout in ("e4m3", "e4m3_page"):
        return _held8(torch.cat([n, pe], 1) / scale) * scale
    if layout == "ds":
        t = n.unflatten(1, (4, 128))
        s = (t.abs().amax(2, keepdim=True) / 448.0).clamp_min(1e-4).log2().ceil().exp2()
        return torch.cat([(_held8(t / s) * s).flatten(1), pe], 1)
    t = n.unflatten(1, (32, 16))
    s = _held8((t.abs().amax(2, keepdim=True) / 6.0).clamp_min(2.0 ** -9))
    return torch.cat([(_held4(t * (1.0 / s)) * s).flatten(1), _held8(pe)], 1)


def _plain_store(s):
    c, bf = s["case"], torch.bfloat16
    x, pe = s["kv_c"].float(), s["k_pe"]
    if c["norm"]:
        rr = torch.rsqrt((x * x).sum(1, keepdim=True) / LATENT + EPS)
        x = (x * rr * s["gamma"].float()).to(bf).float()
    if c["axes"]:
        pe = _rotate(pe.float()[:, None], s["pos"], s["inv_freq"], s["axis"], True)[:, 0].to(bf)
    m = s["total"]
    scale = s["scale"][(s["slots"][:m] // c["page"])][:, None] if c["layout"] == "e4m3_page" else s["scale"]
    back = _held(x[:m], pe[:m].float(), c["layout"], scale)
    return {"rows": torch.cat([x.to(bf), pe], 1), "back": back.to(bf)}


def _plain_read(s):
    c = s["case"]
    page, total = c["page"], s["back"].shape[0]
    at = torch.arange(total, device="cuda")
    req = torch.searchsorted(s["cu"][1:].contiguous(), at.int(), right=True)
    pos = s["first"][req].long() + at - s["cu"][req]
    blk = s["table"][req, pos // page].long()
    raw = s["cache"].view(-1, s["cache"].shape[2])[blk * page + pos % page]
    f8 = lambda r: r.contiguous().view(torch.float8_e4m3fn).float()  # noqa: E731
    if c["layout"] in ("e4m3", "e4m3_page"):
        x = f8(raw) * (s["scale"][blk][:, None] if c["layout"] == "e4m3_page" else s["scale"])
    elif c["layout"] == "ds":
        t = raw[:, LATENT:528].contiguous().view(torch.float32)
        lat = (f8(raw[:, :LATENT]).unflatten(1, (4, 128)) * t[..., None]).flatten(1)
        x = torch.cat([lat, raw[:, 528:].contiguous().view(torch.bfloat16).float()], 1)
    else:
        val = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
        by = raw[:, :256].int()
        j = torch.arange(32, device="cuda")
        code = f8(raw[:, 256 + 8 * (j % 4) + j // 4])
        lat = (torch.stack([val[by & 15], val[by >> 4]], 2).flatten(1).unflatten(1, (32, 16)) * code[..., None]).flatten(1)
        x = torch.cat([lat, f8(raw[:, 288:])], 1)
    return {"rows": x.to(torch.bfloat16)}


def _plain_attend(s):
    """All documents beside one another, each padded to the longest."""
    c, dev = s["case"], "cuda"
    cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
    nq, nk = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
    i = torch.arange(c["longest"], device=dev)
    j = torch.arange(max(1, c["longest"] + c["context"]), device=dev)
    row = (cu_q[:-1, None] + i).clamp_max(s["q"].shape[0] - 1)
    key = (cu_k[:-1, None] + j).clamp_max(s["kv"].shape[0] - 1)
    have = i < nq[:, None]
    q = s["q"][row].transpose(1, 2).float()  # [docs, heads, nq, 192]
    kv = s["kv"][key].transpose(1, 2).float()
    pe = s["k_pe"][key].float()[:, None].expand(-1, c["heads"], -1, -1)
    x = torch.matmul(q, torch.cat([kv[..., :NOPE], pe], -1).transpose(2, 3)) * SOFTMAX_SCALE
    if c["cap"]:
        x = torch.tanh(x / c["cap"]) * c["cap"]
    place = i[None, :, None] + (nk - nq)[:, None, None]  # each query's own position among the keys
    far = (place - j).abs()
    if s["slopes"] is not None:
        x = x - s["slopes"][:, None, None] * far[:, None].float()
    seen = (j < nk[:, None])[:, None].expand(-1, len(i), -1)
    if c["causal"]:
        both = s["prefix"].long()[:, None, None] if s["prefix"] is not None else 0
        seen = seen & ((j <= place) | (j < both))
    x = torch.where(seen[:, None], x, -math.inf)
    m = x.amax(3, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(3, keepdim=True)
    o = torch.matmul(p, kv[..., NOPE:]) / torch.where(total == 0.0, 1.0, total)
    out, lse = s["out"].clone(), s["lse"].clone()
    out[row[have]] = o.transpose(1, 2)[have].to(torch.bfloat16)
    lse[row[have]] = (m + torch.log(total)).squeeze(3).transpose(1, 2)[have]
    return {"out": out, "lse": lse}


PLAIN = {"rope": _plain_rope, "store": _plain_store, "read": _plain_read, "attend": _plain_attend}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- in 64 bits


def _codes64(bits_exp, bits_man, bias, nan):
    """Values of all codes of a small float format, sign bit on top, from its definition."""
    v = []
    for c in range(1 << (bits_exp + bits_man)):
        e, m = c >> bits_man, (c & ((1 << bits_man) - 1)) / (1 << bits_man)
        v.append(math.nan if c in nan else m * 2.0 ** (1 - bias) if e == 0 else (1 + m) * 2.0 ** (e - bias))
    return torch.tensor(v + [-x for x in v], dtype=torch.float64, device="cuda")


def _nearest64(x, values):
    """x to the nearest of a format's non-negative values, with its sign; of two as near to the even code."""
    mid = (values[1:] + values[:-1]) / 2
    a = x.abs()
    low = torch.bucketize(a, mid)  # the lower one where a lies on a middle
    tie = (low < len(mid)) & (a == mid[low.clamp_max(len(mid) - 1)]) & (low % 2 == 1)
    return values[low + tie.long()] * torch.sign(x)


def _turned64(x, pos, interleaved, axes):
    y = torch.empty_like(x)
    section = [0] * SECTIONS[0] + [1] * SECTIONS[1] + [2] * SECTIONS[2]
    for p in range(32):
        w = pos.reshape(-1, x.shape[0])[min(section[p], axes - 1)].double() * 10000.0 ** (-2 * p / ROPE)
        a, b = (2 * p, 2 * p + 1) if interleaved else (p, p + 32)
        co, si = torch.cos(w)[:, None], torch.sin(w)[:, None]
        y[..., a] = x[..., a] * co - x[..., b] * si
        y[..., b] = x[..., a] * si + x[..., b] * co
    return y


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op == "rope":
        return {"out": _turned64(s["x"].double(), s["pos"], case["interleaved"], case["axes"])}
    e4, e2 = _codes64(4, 3, 7, (127,)), _codes64(2, 1, 1, ())
    if op == "store":
        n, pe = s["kv_c"].double(), s["k_pe"].double()
        if case["norm"]:
            n = n / torch.sqrt(n.square().mean(1, keepdim=True) + EPS) * s["gamma"].double()
        if case["axes"]:
            pe = _turned64(pe[:, None], s["pos"], True, case["axes"])[:, 0]
        rows = torch.cat([n, pe], 1)
        # what is quantised is the row as it is handed on, in BF16
        lat, rope = rows.to(torch.bfloat16).double()[:s["total"]].split([LATENT, ROPE], 1)
        if case["layout"] in ("e4m3", "e4m3_page"):
            sc = s["scale"].double()
            if case["layout"] == "e4m3_page":
                sc = sc[s["slots"][:s["total"]] // case["page"]][:, None]
            back = _nearest64(torch.cat([lat, rope], 1) / sc, e4[:127]) * sc
        elif case["layout"] == "ds":
            t = lat.view(-1, 4, 128)
            sc = torch.exp2(torch.ceil(torch.log2((t.abs().amax(2, keepdim=True) / 448.0).clamp_min(1e-4))))
            back = torch.cat([(_nearest64(t / sc, e4[:127]) * sc).flatten(1), rope], 1)
        else:
            t = lat.view(-1, 32, 16)
            sc = _nearest64((t.abs().amax(2, keepdim=True) / 6.0).clamp_min(2.0 ** -9), e4[:127])
            back = torch.cat([(_nearest64(t / sc, e2[:8]) * sc).flatten(1), _nearest64(rope, e4[:127])], 1)
        return {"rows": rows, "back": back}
    if op == "read":
        out = torch.empty(s["back"].shape, dtype=torch.float64, device="cuda")
        cu, page = s["cu"].tolist(), case["page"]
        flat = s["cache"].view(-1, s["cache"].shape[2])
        for r, first in enumerate(s["first"].tolist()):
            pos = torch.arange(first, first + cu[r + 1] - cu[r], device="cuda")
            blk = s["table"][r].long()[torch.div(pos, page, rounding_mode="floor")]
            raw, o = flat[blk * page + pos % page], out[cu[r]:cu[r + 1]]
            if case["layout"] == "e4m3":
                o[:] = e4[raw.long()] * s["scale"].double()
            elif case["layout"] == "e4m3_page":
                o[:] = e4[raw.long()] * s["scale"].double()[blk][:, None]
            elif case["layout"] == "ds":
                t = raw[:, 512:528].contiguous().view(torch.float32).double().repeat_interleave(128, 1)
                o[:, :512] = e4[raw[:, :512].long()] * t
                o[:, 512:] = raw[:, 528:].contiguous().view(torch.bfloat16).double()
            else:
                by = raw[:, :256].long()
                o[:, 0:512:2], o[:, 1:512:2] = e2[by % 16], e2[by // 16]
                for b in range(32):
                    o[:, 16 * b:16 * b + 16] *= e4[raw[:, 256 + 8 * (b % 4) + b // 4].long()][:, None]
                o[:, 512:] = e4[raw[:, 288:].long()]
        return {"rows": out}
    out, lse = s["out"].double(), s["lse"].double()
    cu_q, cu_k, heads = s["cu_q"].tolist(), s["cu_k"].tolist(), case["heads"]
    for d in range(case["docs"]):
        q0, q1, k0, k1 = cu_q[d], cu_q[d + 1], cu_k[d], cu_k[d + 1]
        nq, nk = q1 - q0, k1 - k0
        place = torch.arange(nq, device="cuda")[:, None] + nk - nq
        j = torch.arange(nk, device="cuda")
        hidden = torch.zeros((nq, nk), dtype=torch.bool, device="cuda")
        if case["causal"]:
            hidden = j > place
            if s["prefix"] is not None:
                hidden &= j >= int(s["prefix"][d])
        step = max(1, (1 << 27) // max(1, nq * nk))
        for h in range(0, heads, step):
            q = s["q"][q0:q1, h:h + step].double().transpose(0, 1)
            kv = s["kv"][k0:k1, h:h + step].double().transpose(0, 1)
            x = q[..., :NOPE] @ kv[..., :NOPE].transpose(1, 2) + q[..., NOPE:] @ s["k_pe"][k0:k1].double().T
            x = x / math.sqrt(QK)
            if case["cap"]:
                x = case["cap"] * torch.tanh(x / case["cap"])
            if s["slopes"] is not None:
                x -= s["slopes"][h:h + step].double()[:, None, None] * (place - j).abs()
            x.masked_fill_(hidden, -math.inf)
            z = torch.logsumexp(x, 2)
            w = torch.exp(x - torch.where(torch.isinf(z), 0.0, z)[..., None])
            out[q0:q1, h:h + step] = (w @ kv[..., NOPE:]).transpose(0, 1)
            lse[q0:q1, h:h + step] = z.transpose(0, 1)
    return {"out": out, "lse": lse}


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    op = case["op"]
    if op == "rope":
        n = case["tokens"] * case["heads"]
        return {"bytes": 4.0 * n * ROPE + 4.0 * case["tokens"] * case["axes"], "flops": 3.0 * n * ROPE}
    if op == "attend":
        # the expected number of scores, the documents' lengths taken alike
        nq = (case["longest"] if case["docs"] == 1 else (case["shortest"] + case["longest"]) / 2)
        nk = max(0.0, nq + case["context"])
        pairs = nq * nk
        if case["causal"]:
            low = max(0.0, nk - nq + 1)
            rows = nk - low + 1 if nk > 0 else 0.0
            pairs = rows * (low + nk) / 2
            if case["prefix"]:  # keys behind a query that a prefix of half the longest one still shows
                p = min(case["prefix"] / 2, nk)
                hidden = max(0.0, p - low)
                pairs += hidden * hidden / 2
        n = case["docs"] * case["heads"]
        seen = nk * n * (NOPE + VALUE) * 2 + nk * case["docs"] * ROPE * 2
        return {"bytes": seen + nq * n * ((QK + VALUE) * 2 + 4), "flops": 2.0 * pairs * n * (QK + VALUE)}
    n = case["requests"] * (case["longest"] if case["requests"] == 1 else (case["shortest"] + case["longest"]) / 2)
    if op == "read":
        n = max(case["requests"] * 1.0, n - case["requests"] * case["skip"])
        return {"bytes": n * (ROW_BYTES[case["layout"]] + ROW * 2), "flops": n * ROW}
    # the row as it came, as it is handed on, in the cache, and read back
    held = ROW_BYTES[case["layout"]]
    return {"bytes": n * (3 * ROW * 2 + 2 * held + 8) + case["pad"] * 2.0 * ROW * 2, "flops": n * ROW * 8}
