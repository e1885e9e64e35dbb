"""The decode step's cache-side operators: what is measured, in plain torch form.

Five operators around the paged latent KV cache that the decode step writes:

* ``tables``  block tables, slot map and causal lengths from request lengths;
* ``attend``  latent attention over the paged 8-bit (or 4-bit) cache, over the
  whole context or over a list of selected blocks;
* ``mean``    the mean key of every block touched by new tokens;
* ``score``   a cheap score of every block for every query;
* ``select``  the best-scored blocks of every query.

``run`` computes them with elementary torch operations in 32 bits, or, with
``own`` set, through the package's entry points.
"""

import math

import torch

own = False

LATENT, ROPE, ROW = 512, 64, 576
# cache layouts: bytes of one token's row
LAYOUTS = {"e4m3": 0, "ds": 1, "nvfp4": 2, "e4m3_page": 3}
ROW_BYTES = {"e4m3": 576, "ds": 656, "nvfp4": 352, "e4m3_page": 576}
SOFTMAX_SCALE = 192.0 ** -0.5  # 128 nope + 64 rope columns of a head
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one short request at 16 local heads (tensor parallel over many ranks): latency alone
        dict(name="attend_b1_h16_512_e4m3", op="attend", rows=1, nq=1, pad=0, heads=16, page=64, pages=8,
             shortest=512, longest=512, layout="e4m3", q="bf16", blocks=0),
        # one request whose context fills a 1024-page cache: the latency of a long context
        dict(name="attend_b1_h64_64k_e4m3", op="attend", rows=1, nq=1, pad=0, heads=64, page=64, pages=1024,
             shortest=65536, longest=65536, layout="e4m3", q="bf16", blocks=0),
        # a full serving batch over 4096 pages, ragged, two padded tokens of a captured batch
        dict(name="attend_b62_h128_4k_ds", op="attend", rows=62, nq=1, pad=2, heads=128, page=64, pages=4096,
             shortest=700, longest=4096, layout="ds", q="bf16", blocks=0),
        # eight long requests, FP8 queries, a scale for each page; 32 selected blocks of up to 256
        dict(name="attend_b8_h128_sparse32_e4m3_page", op="attend", rows=8, nq=1, pad=0, heads=128, page=64,
             pages=2048, shortest=9001, longest=16384, layout="e4m3_page", q="e4m3", blocks=32),
        # a decode step of 64 requests: one new token each, a page now and then, some finished
        dict(name="tables_r64_decode", op="tables", rows=64, page=64, pages=4096, blocks=64, longest_new=1,
             fill=0.8, release=4, tokens=64),
        # a step with chunked prefill: up to 256 requests appending up to 256 tokens each
        dict(name="tables_r256_prefill", op="tables", rows=256, page=64, pages=4096, blocks=64, longest_new=256,
             fill=0.3, release=16, tokens=32768),
        # the decode step's own pages: one touched page for each of 64 requests
        dict(name="mean_r64_decode_ds", op="mean", rows=64, page=64, pages=4096, shortest=700, longest=4096,
             new=1, layout="ds"),
        # eight prompts just written: all of their pages
        dict(name="mean_r8_prefill_e4m3", op="mean", rows=8, page=64, pages=2048, shortest=9001, longest=16384,
             new=0, layout="e4m3"),
        # one query over the 1024 blocks of a long request
        dict(name="score_b1_h64_1024", op="score", rows=1, heads=64, page=64, pages=1024, shortest=65536,
             longest=65536, q="bf16"),
        # a serving batch at 128 heads, 64 to 256 blocks a request
        dict(name="score_b64_h128_256", op="score", rows=64, heads=128, page=64, pages=16384, shortest=4096,
             longest=16384, q="bf16"),
        # one query's 1024 blocks down to 32
        dict(name="select_b1_1024_k32", op="select", rows=1, blocks=1024, k=32, first=1, last=2),
        # the largest batch, 4096 blocks each, 128 kept
        dict(name="select_b256_4096_k128", op="select", rows=256, blocks=4096, k=128, first=1, last=4),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "attend", "tables", "mean", "score", "select"])
    page = rng.choice([1, 7, 16, 32, 48, 64, 64, 64, 100, 128])
    if op == "select":
        n = _log(rng, 1, 8192)
        return dict(op=op, rows=_log(rng, 1, 256), blocks=n, k=_log(rng, 1, min(n + 3, 512)),
                    first=rng.randint(0, 2), last=rng.randint(0, 4))
    rows = _log(rng, 1, 64)
    if op == "tables":
        rows = _log(rng, 1, 1000)
        return dict(op=op, rows=rows, page=page, pages=max(1, _log(rng, 1, 64) * rows), blocks=_log(rng, 4, 200),
                    longest_new=_log(rng, 1, 400), fill=rng.uniform(0.05, 0.95), release=rng.randint(0, rows // 3),
                    tokens=_log(rng, 1, 400 * rows))
    nq = rng.choice([1, 1, 1, 2, 4]) if op == "attend" and rows <= 16 else 1
    longest = _log(rng, 1, min(65536, 140000 // (rows * nq)))  # cached tokens in all: 140000
    shortest = rng.randint(max(1, longest // 8), longest)
    pages = rows * -(-longest // page) + rng.randint(0, 40)
    if op == "mean":
        return dict(op=op, rows=rows, page=page, pages=pages, shortest=shortest, longest=longest,
                    new=rng.choice([0, 1, 1, 5, 130]), layout=rng.choice(sorted(LAYOUTS)))
    heads = rng.choice([1, 3, 8, 16, 24, 32, 40, 64, 64, 96, 127, 128, 128])
    q = rng.choice(["bf16", "bf16", "e4m3"])
    if op == "score":
        return dict(op=op, rows=rows, heads=heads, page=page, pages=pages, shortest=shortest, longest=longest, q=q)
    blocks = rng.choice([0, 0, _log(rng, 1, 64)])
    if blocks:
        blocks = min(blocks, max(1, 4096 // page))
    return dict(op=op, rows=rows, nq=nq, pad=rng.choice([0, 0, 3]), heads=heads, page=page,
                pages=pages, shortest=shortest, longest=longest, layout=rng.choice(sorted(LAYOUTS)), q=q,
                blocks=blocks)


# ---------------------------------------------------------------- inputs


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _host(seed):
    return torch.Generator().manual_seed(int(seed))


def _e4m3(x):
    """OCP E4M3 codes of x, saturating."""
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _cache(layout, pages, page, g):
    """A cache [pages, page, row bytes] of normalised latents and rope keys as the decode step writes them,
    and its scales."""
    n, dev = pages * page, "cuda"
    rows = torch.empty((n, ROW_BYTES[layout]), dtype=torch.uint8, device=dev)
    scale = torch.full((1,), 0.05, device=dev)
    if layout == "e4m3_page":
        scale = torch.exp2(torch.rand(pages, generator=g, device=dev) * 3.0 - 6.0)
    for a in range(0, n, 1 << 16):
        b = min(n, a + (1 << 16))
        x = torch.randn((b - a, ROW), generator=g, device=dev)
        lat, pe = x[:, :LATENT], x[:, LATENT:]
        if layout == "e4m3":
            rows[a:b] = _e4m3(x / scale)
        elif layout == "e4m3_page":
            rows[a:b] = _e4m3(x / scale[torch.arange(a, b, device=dev) // page, None])
        elif layout == "ds":
            s = (lat.abs().view(-1, 4, 128).amax(2) / 448.0).clamp_min(1e-4).log2().ceil().exp2()
            rows[a:b, :LATENT] = _e4m3(lat.view(-1, 4, 128) / s[..., None]).view(-1, LATENT)
            rows[a:b, LATENT:528] = s.view(torch.uint8).view(-1, 16)
            rows[a:b, 528:] = pe.to(torch.bfloat16).view(torch.uint8).view(-1, 128)
        else:
            code = _e4m3((lat.abs().view(-1, 32, 16).amax(2) / 6.0).clamp_min(2.0 ** -9))
            y = lat.view(-1, 32, 16) / code.view(torch.float8_e4m3fn).float()[..., None]
            mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=dev)
            nib = (torch.bucketize(y.abs(), mid) + 8 * (y < 0)).view(-1, LATENT).to(torch.uint8)
            rows[a:b, :256] = nib[:, ::2] | (nib[:, 1::2] << 4)
            s = torch.arange(32, device=dev)
            rows[a:b, 256 + 8 * (s % 4) + s // 4] = code.view(-1, 32)
            rows[a:b, 288:] = _e4m3(pe)
    return rows.view(pages, page, -1), scale


def _lengths(case, h):
    """Ragged lengths between the case's shortest and longest; the first request is the longest."""
    n = torch.randint(case["shortest"], case["longest"] + 1, (case["rows"],), generator=h)
    n[0] = case["longest"]
    room, total = case["pages"], 0
    for i in range(len(n)):  # no more than the cache holds
        left = room - total - (len(n) - 1 - i)
        n[i] = min(int(n[i]), max(1, left) * case["page"])
        total += -(-int(n[i]) // case["page"])
    return n.to(torch.int32)


def _table(lens, page, pages, h):
    """Block tables of requests with these lengths over pages handed out in random order; -1 behind the last."""
    need = (lens + page - 1) // page
    width = int(need.max())
    bt = torch.full((len(lens), width), -1, dtype=torch.int32)
    order, at = torch.randperm(pages, generator=h).to(torch.int32), 0
    for i, k in enumerate(need.tolist()):
        bt[i, :k] = order[at:at + k]
        at += k
    return bt


def _queries(tokens, heads, kind, g):
    """Latent and rope queries with the spread that the projections give them; codes and their scale for 8 bits."""
    ql = (torch.randn((tokens, heads, LATENT), generator=g, device="cuda") * 0.44).to(torch.bfloat16)
    qp = (torch.randn((tokens, heads, ROPE), generator=g, device="cuda") * 0.78).to(torch.bfloat16)
    if kind == "bf16":
        return ql, qp, None
    inv = torch.full((1,), 32.0, device="cuda")
    return _e4m3(ql.float() * inv), _e4m3(qp.float() * inv), inv


def prepare(case, seed):
    g, h, dev = _gen(seed), _host(seed), "cuda"
    op, s = case["op"], dict(case=case)
    if op == "tables":
        rows, page, blocks = case["rows"], case["page"], case["blocks"]
        lens = (torch.rand(rows, generator=h) * case["fill"] * blocks * page).to(torch.int32)
        cap, used = max(1, int(case["pages"] * 0.9)), 0
        for i in range(rows):  # no more than the cache holds
            lens[i] = min(int(lens[i]), (cap - used) * page)
            used += -(-int(lens[i]) // page)
        new = torch.randint(0 if case["longest_new"] > 1 else 1, case["longest_new"] + 1, (rows,), generator=h).to(torch.int32)
        if case["release"]:
            new[torch.randperm(rows, generator=h)[:case["release"]]] = -1
        bt = torch.full((rows, blocks), -1, dtype=torch.int32)
        order, at = torch.randperm(case["pages"], generator=h).to(torch.int32), 0
        for i, k in enumerate(((lens + page - 1) // page).tolist()):
            bt[i, :k] = order[at:at + k]
            at += k
        stack = torch.full((case["pages"],), -1, dtype=torch.int32)
        stack[:case["pages"] - at] = order[at:]
        s.update(lens=lens.to(dev), new=new.to(dev), table=bt.to(dev), stack=stack.to(dev),
                 count=torch.tensor([case["pages"] - at], dtype=torch.int32, device=dev))
        t = case["tokens"]
        s.update(lens_out=torch.empty_like(s["lens"]), count_out=torch.empty_like(s["count"]),
                 cu=torch.empty(rows + 1, dtype=torch.int32, device=dev),
                 slots=torch.empty(t, dtype=torch.int64, device=dev),
                 token_row=torch.empty(t, dtype=torch.int32, device=dev),
                 token_len=torch.empty(t, dtype=torch.int32, device=dev),
                 flags=torch.zeros(1, dtype=torch.int32, device=dev))
        return s
    if op == "select":
        sc = torch.randn((case["rows"], case["blocks"]), generator=g, device=dev) * 12.0
        n = torch.randint((case["blocks"] + 1) // 2, case["blocks"] + 1, (case["rows"],), generator=h)
        n[0] = case["blocks"]
        s.update(scores=sc, lens=n.to(torch.int32).to(dev),
                 sel=torch.empty((case["rows"], case["k"]), dtype=torch.int32, device=dev),
                 count=torch.empty(case["rows"], dtype=torch.int32, device=dev))
        return s
    lens = _lengths(case, h)
    table = _table(lens, case["page"], case["pages"], h)
    if op == "mean":
        cache, scale = _cache(case["layout"], case["pages"], case["page"], g)
        before = (lens - case["new"]).clamp_min(0) if case["new"] else torch.zeros_like(lens)
        s.update(cache=cache, scale=scale, table=table.to(dev), lens_to=lens.to(dev), lens_from=before.to(dev),
                 mean=torch.zeros((case["pages"], ROW), dtype=torch.bfloat16, device=dev),
                 flags=torch.zeros(1, dtype=torch.int32, device=dev))
        return s
    if op == "score":
        ql, qp, inv = _queries(case["rows"], case["heads"], case["q"], g)
        mean = (torch.randn((case["pages"], ROW), generator=g, device=dev) * case["page"] ** -0.5).to(torch.bfloat16)
        s.update(q_latent=ql, q_pe=qp, inv=inv, mean=mean, table=table.to(dev), lens=lens.to(dev),
                 scores=torch.empty((case["rows"], table.shape[1]), device=dev),
                 flags=torch.zeros(1, dtype=torch.int32, device=dev))
        return s
    # attend: nq query tokens a request (the last ones of its context), then padded tokens
    nq, page = case["nq"], case["page"]
    tokens = case["rows"] * nq + case["pad"]
    row = torch.full((tokens,), -1, dtype=torch.int32)
    tlen = torch.zeros(tokens, dtype=torch.int32)
    row[:case["rows"] * nq] = torch.arange(case["rows"], dtype=torch.int32).repeat_interleave(nq)
    back = torch.arange(nq - 1, -1, -1, dtype=torch.int32).repeat(case["rows"])
    tlen[:case["rows"] * nq] = (lens.repeat_interleave(nq) - back).clamp_min(0)
    cache, scale = _cache(case["layout"], case["pages"], page, g)
    flat = cache.view(-1, cache.shape[2])
    for i, n in enumerate(lens.tolist()):  # what lies behind a request's last token is never read as a value
        if n % page:
            p = int(table[i, n // page])
            flat[p * page + n % page:(p + 1) * page] = 0x7F
    ql, qp, inv = _queries(tokens, case["heads"], case["q"], g)
    s.update(cache=cache, scale=scale, table=table.to(dev), token_row=row.to(dev), lens=tlen.to(dev),
             q_latent=ql, q_pe=qp, inv=inv,
             out=torch.empty((tokens, case["heads"], LATENT), dtype=torch.bfloat16, device=dev),
             lse=torch.empty((tokens, case["heads"]), device=dev))
    if case["blocks"]:
        k = case["blocks"]
        sel, cnt = torch.full((tokens, k), -1, dtype=torch.int32), torch.zeros(tokens, dtype=torch.int32)
        for t, n in enumerate(tlen.tolist()):
            nb = -(-n // page)
            c = min(k, nb)
            if c:  # the block of the newest token, and others
                pick = torch.cat([torch.randperm(nb - 1, generator=h)[:c - 1], torch.tensor([nb - 1])]).sort().values
                sel[t, :c] = pick.to(torch.int32)
            cnt[t] = c
        s.update(sel=sel.to(dev), sel_count=cnt.to(dev))
    if own:
        from mla_query_projection_gb300.runner import PagedAttention

        s["attn"] = PagedAttention(tokens, case["heads"])
    return s


# ---------------------------------------------------------------- the framework's calls


def _own(s):
    from mla_query_projection_gb300 import runner as R

    c = s["case"]
    if c["op"] == "tables":
        R.tables_step(s["new"], s["lens"], s["table"], s["stack"], s["count"], c["page"], s["lens_out"], s["count_out"],
                      s["slots"], s["token_row"], s["token_len"], s["cu"], s["flags"])
    elif c["op"] == "mean":
        R.blocks_mean(s["cache"], LAYOUTS[c["layout"]], s["scale"], s["table"], s["lens_from"], s["lens_to"], s["mean"],
                      s["flags"])
    elif c["op"] == "score":
        R.blocks_score(s["q_latent"], s["q_pe"], s["mean"], c["page"], s["table"], s["lens"], s["scores"],
                       q_scale_inv=s["inv"], flags=s["flags"])
    elif c["op"] == "select":
        R.blocks_select(s["scores"], s["lens"], 1, c["first"], c["last"], s["sel"], s["count"])
    else:
        s["attn"].decode(s["q_latent"], s["q_pe"], s["cache"], LAYOUTS[c["layout"]], s["table"], s["lens"], SOFTMAX_SCALE,
                         k_scale=s["scale"], q_scale_inv=s["inv"], token_row=s["token_row"], sel=s.get("sel"),
                         sel_count=s.get("sel_count"), out=s["out"], lse=s["lse"])


# ---------------------------------------------------------------- the plain forms


def _dequant(raw, layout, scale):
    """FP32 keys [..., 576] of raw rows [..., row bytes]; scale broadcasts over the rows."""
    if layout in ("e4m3", "e4m3_page"):
        return raw.view(torch.float8_e4m3fn).float() * scale
    if layout == "ds":
        t = raw[..., LATENT:528].contiguous().view(torch.float32)
        lat = raw[..., :LATENT].contiguous().view(torch.float8_e4m3fn).float()
        lat = (lat.unflatten(-1, (4, 128)) * t[..., None]).flatten(-2)
        return torch.cat([lat, raw[..., 528:].contiguous().view(torch.bfloat16).float()], -1)
    val = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=raw.device)
    by = raw[..., :256].int()
    lat = torch.stack([val[by & 15], val[by >> 4]], -1).flatten(-2)
    at = torch.arange(32, device=raw.device)
    code = raw[..., 256 + 8 * (at % 4) + at // 4].contiguous().view(torch.float8_e4m3fn).float()
    lat = (lat.unflatten(-1, (32, 16)) * code[..., None]).flatten(-2)
    return torch.cat([lat, raw[..., 288:].contiguous().view(torch.float8_e4m3fn).float()], -1)


def _query(s):
    if s["inv"] is None:
        return torch.cat([s["q_latent"], s["q_pe"]], -1).float()
    q = torch.cat([s["q_latent"], s["q_pe"]], -1).view(torch.float8_e4m3fn)
    return q.float() / s["inv"]


def _positions(s):
    """Logical positions [tokens, n] that each query looks at, and which of them count."""
    c, dev = s["case"], "cuda"
    page = c["page"]
    if c["blocks"]:
        off = torch.arange(page, device=dev)
        pos = (s["sel"][:, :, None].long() * page + off).flatten(1)
        listed_ = torch.arange(s["sel"].shape[1], device=dev) < s["sel_count"][:, None]
        ok = listed_.repeat_interleave(page, 1) & (pos >= 0) & (pos < s["lens"][:, None])
    else:
        pos = torch.arange(c["longest"], device=dev).expand(len(s["lens"]), -1)
        ok = pos < s["lens"][:, None]
    return pos, ok


def _plain_attend(s):
    c = s["case"]
    page = c["page"]
    pos, ok = _positions(s)
    at = torch.where(ok, pos, 0)
    blk = s["table"].long()[s["token_row"].long().clamp_min(0)[:, None], at // page]
    blk = torch.where(ok, blk, 0)
    raw = s["cache"].view(-1, s["cache"].shape[2])[blk * page + at % page]
    scale = s["scale"][blk][..., None] if c["layout"] == "e4m3_page" else s["scale"]
    k = torch.where(ok[..., None], _dequant(raw, c["layout"], scale), 0.0)
    x = torch.bmm(_query(s), k.transpose(1, 2)) * SOFTMAX_SCALE
    x = torch.where(ok[:, None], x, -math.inf)
    m = x.amax(2, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(2, keepdim=True)
    o = torch.bmm(p, k[..., :LATENT]) / torch.where(total == 0.0, 1.0, total)
    return {"out": o.to(torch.bfloat16), "lse": (m + torch.log(total)).squeeze(2)}


def _plain_tables(s):
    """Requests in row order: releases give their pages back, then appends take pages from the top of the stack. A
    request that its row cannot hold is left as it is; from the first that finds no pages or no room on, so are all."""
    c, dev = s["case"], "cuda"
    page, lens, new = c["page"], s["lens"].long(), s["new"].long()
    rows, width = s["table"].shape
    have = (lens + page - 1) // page
    freed = torch.where(new < 0, have, 0)
    stack, count = s["stack"].clone(), s["count"].long()
    give = freed.cumsum(0) - freed
    j = torch.arange(width, device=dev)
    back = (j < freed[:, None])
    stack[(count + give[:, None] + j)[back]] = s["table"][back]
    avail = count + freed.sum()
    wants = (new > 0) & ((lens + new + page - 1) // page <= width)
    take = torch.where(wants, (lens + new + page - 1) // page - have, 0)
    toks = torch.where(wants, new, 0)
    fits = wants & (take.cumsum(0) <= avail) & (toks.cumsum(0) <= c["tokens"])
    take, toks = torch.where(fits, take, 0), torch.where(fits, toks, 0)
    first = take.cumsum(0) - take
    k = j - have[:, None]
    put = (k >= 0) & (k < take[:, None])
    table = s["table"].clone()
    table[put] = stack[(avail - 1 - first[:, None] - k)[put]]
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), toks.cumsum(0)])
    t = torch.arange(c["tokens"], device=dev)
    row = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    ok = t < cu[-1]
    row = torch.where(ok, row, 0)
    pos = torch.where(ok, lens[row] + t - cu[row], 0)
    slot = torch.where(ok, table[row, pos // page].long() * page + pos % page, -1)
    i32 = torch.int32
    return {"lens": torch.where(new < 0, 0, lens + toks).to(i32), "table": table, "stack": stack,
            "count": (avail - take.sum()).to(i32), "cu": cu.to(i32), "slots": slot,
            "token_row": torch.where(ok, row, -1).to(i32), "token_len": torch.where(ok, pos + 1, 0).to(i32)}


def _plain_mean(s):
    c = s["case"]
    page = c["page"]
    j = torch.arange(s["table"].shape[1], device="cuda")
    hit = (j >= s["lens_from"][:, None] // page) & (j * page < s["lens_to"][:, None])
    filled = (s["lens_to"][:, None] - j * page).clamp(0, page)[hit]
    p = s["table"][hit].long()
    scale = s["scale"][p][:, None, None] if c["layout"] == "e4m3_page" else s["scale"]
    x = _dequant(s["cache"][p], c["layout"], scale)
    x = torch.where((torch.arange(page, device="cuda") < filled[:, None])[..., None], x, 0.0)
    mean = s["mean"].clone()
    mean[p] = (x.sum(1) / filled[:, None]).to(torch.bfloat16)
    return {"mean": mean}


def _plain_score(s):
    page = s["case"]["page"]
    j = torch.arange(s["table"].shape[1], device="cuda")
    ok = j * page < s["lens"][:, None]
    k = s["mean"][torch.where(ok, s["table"], 0).long()].float()
    x = torch.bmm(_query(s), k.transpose(1, 2)).amax(1)
    return {"scores": torch.where(ok, x, -math.inf)}


def _plain_select(s):
    c = s["case"]
    j = torch.arange(c["blocks"], device="cuda")
    n = s["lens"][:, None]
    key = torch.where(s["scores"].isnan(), -math.inf, s["scores"])
    key = torch.where((j < c["first"]) | (j >= n - c["last"]), math.inf, key)
    place = torch.where(j < n, key, -math.inf).sort(dim=1, descending=True, stable=True).indices
    place = torch.cat([place, place.new_full((c["rows"], max(0, c["k"] - c["blocks"])), c["blocks"])], 1)[:, :c["k"]]
    kept = torch.where(place < n, place, 1 << 30)
    kept = torch.where(torch.arange(c["k"], device="cuda") < n.clamp_max(c["k"]), kept, 1 << 30).sort(1).values
    count = n.clamp_max(c["k"]).squeeze(1)
    return {"sel": torch.where(kept < (1 << 30), kept, -1).to(torch.int32), "count": count.to(torch.int32)}


OUTPUTS = {
    "attend": {"out": "out", "lse": "lse"},
    "tables": {"lens": "lens_out", "table": "table", "stack": "stack", "count": "count_out", "cu": "cu",
               "slots": "slots", "token_row": "token_row", "token_len": "token_len"},
    "mean": {"mean": "mean"},
    "score": {"scores": "scores"},
    "select": {"sel": "sel", "count": "count"},
}
PLAIN = {"attend": _plain_attend, "tables": _plain_tables, "mean": _plain_mean, "score": _plain_score,
         "select": _plain_select}


def run(state):
    if own:
        _own(state)
        return {k: state[v] for k, v in OUTPUTS[state["case"]["op"]].items()}
    return PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- in 64 bits


def _codes64(bits_exp, bits_man, bias, nan):
    """Values of all codes of a small float format, sign bit on top, from its definition."""
    n = 1 << (bits_exp + bits_man)
    v = []
    for c in range(n):
        e, m = c >> bits_man, c & ((1 << bits_man) - 1)
        x = (m / (1 << bits_man)) * 2.0 ** (1 - bias) if e == 0 else (1 + m / (1 << bits_man)) * 2.0 ** (e - bias)
        v.append(math.nan if c in nan else x)
    return torch.tensor(v + [-x for x in v], dtype=torch.float64, device="cuda")


def _rows64(raw, layout, scale):
    e4 = _codes64(4, 3, 7, (127,))
    if layout.startswith("e4m3"):
        return e4[raw.long()] * scale
    if layout == "ds":
        t = raw[:, 512:528].contiguous().view(torch.float32).double().repeat_interleave(128, 1)
        return torch.cat([e4[raw[:, :512].long()] * t, raw[:, 528:].contiguous().view(torch.bfloat16).double()], 1)
    e2 = _codes64(2, 1, 1, ())
    by = raw[:, :256].long()
    lat = torch.empty((len(raw), 512), dtype=torch.float64, device="cuda")
    lat[:, 0::2], lat[:, 1::2] = e2[by % 16], e2[by // 16]
    for b in range(32):
        lat[:, 16 * b:16 * b + 16] *= e4[raw[:, 256 + 8 * (b % 4) + b // 4].long()][:, None]
    return torch.cat([lat, e4[raw[:, 288:].long()]], 1)


def _queries64(s, t):
    if s["inv"] is None:
        return torch.cat([s["q_latent"][t].double(), s["q_pe"][t].double()], 1)
    return _codes64(4, 3, 7, (127,))[torch.cat([s["q_latent"][t], s["q_pe"][t]], 1).long()] / s["inv"].double()


def exact(case, seed):
    op, page = case["op"], case.get("page", 1)
    if op in ("tables", "select"):
        return None  # whole numbers
    s = prepare(case, seed)
    table = s["table"].tolist()
    if op == "mean":
        mean = s["mean"].double()
        for r, (a, b) in enumerate(zip(s["lens_from"].tolist(), s["lens_to"].tolist())):
            js = [j for j in range(a // page, -(-b // page))]
            if not js:
                continue
            p = torch.tensor([table[r][j] for j in js], device="cuda")
            raw = s["cache"][p].view(len(js) * page, -1)
            sc = s["scale"].double()
            sc = sc[p].repeat_interleave(page)[:, None] if case["layout"] == "e4m3_page" else sc
            x = _rows64(raw, case["layout"], sc).view(len(js), page, ROW)
            n = torch.tensor([min(page, b - j * page) for j in js], device="cuda")
            x = x.masked_fill((torch.arange(page, device="cuda") >= n[:, None])[..., None], 0.0)
            mean[p] = x.sum(1) / n[:, None].double()
        return {"mean": mean}
    if op == "score":
        out = torch.full(s["scores"].shape, -math.inf, dtype=torch.float64, device="cuda")
        for r, n in enumerate(s["lens"].tolist()):
            nb = -(-n // page)
            k = s["mean"][s["table"][r, :nb].long()].double()
            out[r, :nb] = (_queries64(s, r) @ k.T).max(0).values
        return {"scores": out}
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    flat = s["cache"].view(-1, s["cache"].shape[2])
    for t, (r, n) in enumerate(zip(s["token_row"].tolist(), s["lens"].tolist())):
        if n == 0:
            continue
        if case["blocks"]:
            js = s["sel"][t, :int(s["sel_count"][t])].tolist()
        else:
            js = range(-(-n // page))
        pos = torch.cat([torch.arange(j * page, min(n, (j + 1) * page)) for j in js]).cuda()
        blk = s["table"][r].long()[pos // page]
        sc = s["scale"].double()
        sc = sc[blk][:, None] if case["layout"] == "e4m3_page" else sc
        k = _rows64(flat[blk * page + pos % page], case["layout"], sc)
        x = _queries64(s, t) @ k.T * SOFTMAX_SCALE
        lse[t] = torch.logsumexp(x, 1)
        out[t] = torch.exp(x - lse[t][:, None]) @ k[:, :512]
    return {"out": out, "lse": lse}


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    op = case["op"]
    if op == "tables":
        # lengths, new counts, the free list's ends; the tokens' slots, rows and lengths
        return {"bytes": 4.0 * 4 * case["rows"] + 16.0 * case["tokens"], "flops": 0.0}
    if op == "select":
        return {"bytes": 4.0 * case["rows"] * (case["blocks"] * 0.75 + case["k"]), "flops": 0.0}
    page, mean_len = case["page"], (case["shortest"] + case["longest"]) / 2
    if case["rows"] == 1:
        mean_len = case["longest"]
    blocks = math.ceil(mean_len / page)
    if op == "mean":
        touched = math.ceil(case["new"] / page) if case["new"] else blocks
        tokens = case["rows"] * (min(mean_len, case["new"] + page / 2) if case["new"] else mean_len)
        return {"bytes": tokens * ROW_BYTES[case["layout"]] + case["rows"] * touched * ROW * 2.0,
                "flops": tokens * ROW}
    qb = 2 if case["q"] == "bf16" else 1
    if op == "score":
        return {"bytes": case["rows"] * (blocks * (ROW * 2.0 + 4) + case["heads"] * ROW * qb),
                "flops": 2.0 * case["rows"] * blocks * case["heads"] * ROW}
    seen = min(mean_len, case["blocks"] * page) if case["blocks"] else mean_len
    read = case["rows"] * seen * ROW_BYTES[case["layout"]] * (case["nq"] if case["blocks"] else 1)
    tokens = case["rows"] * case["nq"]
    return {"bytes": read + tokens * case["heads"] * (ROW * qb + LATENT * 2 + 4.0),
            "flops": 2.0 * tokens * seen * case["heads"] * (ROW + LATENT)}
