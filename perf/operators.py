"""Cases, plain forms and 64-bit results of the paged 8-bit cache operators.

The paged cache holds projected keys and values in e4m3 with one power-of-two
scale for each page and KV head:

  k_pages [n_pages, Hkv, d_store, page]  projected keys, dimension-major inside a page
  v_pages [n_pages, Hkv, page, 128]      values, token-major
  k_scale, v_scale [n_pages, Hkv] f32    stored code * scale is the value
  block_table [B, max_pages] int32       page of every run of `page` tokens of a sequence

Operators:

  append  rotate new keys by their position, project them (k~ = rope(k) P), quantise keys and values
          into the pages; an open page whose scale has to grow is re-coded
  decode  one query token for each sequence: rotate, project, keep the k largest dimensions of each
          head, attend over the pages
  gather  pages back into a contiguous cache (what chunked prefill reads)
"""
import math
import random

import torch

own = False

D = 128
S_MIN_EXP = -60            # smallest scale a page is given: 2^-60
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one new token of one sequence: what every step of a lone chat pays, latency counts
        {"name": "append_one_token", "op": "append", "batch": 1, "tokens": 1, "hkv": 8, "page": 64, "d_store": 128,
         "dtype": "bf16", "rot": 128, "interleaved": False, "start": 1000},
        # one decode step of a full serving batch over truncated keys
        {"name": "append_decode_256", "op": "append", "batch": 256, "tokens": 256, "hkv": 8, "page": 64,
         "d_store": 96, "dtype": "bf16", "rot": 128, "interleaved": False, "start": 8192},
        # three ragged prompts that start inside a page, f32, half of the dimensions rotated in pairs
        {"name": "append_prompt_f32", "op": "append", "batch": 3, "tokens": 701, "hkv": 4, "page": 32,
         "d_store": 100, "dtype": "f32", "rot": 64, "interleaved": True, "start": 333},
        # long prompts of eight sequences packed into one call
        {"name": "append_prompts_16384", "op": "append", "batch": 8, "tokens": 16384, "hkv": 8, "page": 128,
         "d_store": 128, "dtype": "bf16", "rot": 128, "interleaved": False, "start": 512},
        # the smallest attention call: one sequence, one KV head, f32 in and out
        {"name": "decode_f32_1024", "op": "decode", "batch": 1, "hq": 4, "hkv": 1, "len": 1024, "ragged": False,
         "page": 64, "d_store": 128, "k": 96, "dtype": "f32", "rot": 128, "interleaved": False},
        # the decode shape of the benchmark: 8 sequences of 8192 tokens
        {"name": "decode_8x8192", "op": "decode", "batch": 8, "hq": 32, "hkv": 8, "len": 8192, "ragged": False,
         "page": 64, "d_store": 128, "k": 96, "dtype": "bf16", "rot": 128, "interleaved": False},
        # one long context, split over the whole machine
        {"name": "decode_1x131072", "op": "decode", "batch": 1, "hq": 32, "hkv": 8, "len": 131072, "ragged": False,
         "page": 128, "d_store": 128, "k": 96, "dtype": "bf16", "rot": 128, "interleaved": False},
        # a ragged batch over truncated keys, a slot of the batch idle, odd lengths that end inside pages
        {"name": "decode_ragged_m96", "op": "decode", "batch": 32, "hq": 32, "hkv": 8, "len": 2047, "ragged": True,
         "page": 32, "d_store": 96, "k": 64, "dtype": "bf16", "rot": 128, "interleaved": False},
        # one query head for each KV head and few dimensions: most key rows are never read
        {"name": "decode_mha_k32", "op": "decode", "batch": 16, "hq": 16, "hkv": 16, "len": 4096, "ragged": True,
         "page": 128, "d_store": 128, "k": 32, "dtype": "bf16", "rot": 64, "interleaved": True},
        # the largest: a ragged batch of long contexts, eight query heads for each KV head
        {"name": "decode_32x32768_g8", "op": "decode", "batch": 32, "hq": 64, "hkv": 8, "len": 32768, "ragged": True,
         "page": 128, "d_store": 128, "k": 64, "dtype": "bf16", "rot": 128, "interleaved": False},
        # the history of one sequence before a prompt chunk
        {"name": "gather_1x4096", "op": "gather", "batch": 1, "hkv": 8, "len": 4096, "ragged": False, "page": 64,
         "d_store": 128, "dtype": "bf16"},
        # a ragged batch out of small pages, truncated keys
        {"name": "gather_16x16384", "op": "gather", "batch": 16, "hkv": 8, "len": 16384, "ragged": True, "page": 16,
         "d_store": 96, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    """A whole number in [lo, hi], spread evenly over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append", "decode", "decode", "decode", "gather"])
    page = rng.choice([16, 32, 64, 128])
    d_store = rng.choice([128, 128, 96, 64, 100, 48])
    hkv = rng.choice([1, 2, 4, 8, 8, 16])
    rot, interleaved = rng.choice([(128, False), (128, True), (64, False), (32, True), (0, False)])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "append":
        batch = _log_int(rng, 1, 256)
        if rng.random() < 0.4:
            tokens = batch                                     # one token for each sequence
        else:
            tokens = max(batch, _log_int(rng, 1, 131072 // hkv))
        return {"op": op, "batch": batch, "tokens": tokens, "hkv": hkv, "page": page, "d_store": d_store,
                "dtype": dtype, "rot": rot, "interleaved": interleaved, "start": _log_int(rng, 1, 16384)}
    ragged = rng.random() < 0.6
    if op == "decode":
        g = rng.choice([1, 2, 4, 4, 8, 3, 7])
        length = _log_int(rng, 1, 131072)
        batch = _log_int(rng, 1, max(1, min(256, 3600000 // (length * hkv))))
        return {"op": op, "batch": batch, "hq": g * hkv, "hkv": hkv, "len": length, "ragged": ragged, "page": page,
                "d_store": d_store, "k": rng.randint(1, d_store), "dtype": dtype, "rot": rot,
                "interleaved": interleaved}
    length = _log_int(rng, 1, 32768)
    batch = _log_int(rng, 1, max(1, min(64, 700000 // (length * hkv))))
    return {"op": op, "batch": batch, "hkv": hkv, "len": length, "ragged": ragged, "page": page, "d_store": d_store,
            "dtype": dtype}


# ------------------------------------------------------------------ what a case's batch looks like

def _lengths(case):
    """Cached tokens of every sequence: the longest first; a ragged batch of four or more has an idle slot."""
    b, top = case["batch"], case["len"]
    if not case["ragged"]:
        return [top] * b
    r = random.Random("%d %d %d" % (b, top, case["hkv"]))
    lens = [top] + [r.randint(1, top) for _ in range(b - 1)]
    if b >= 4:
        lens[b // 2] = 0
    return lens


def _runs(case):
    """(start, new tokens) of every sequence of an append; with more tokens than sequences the runs are ragged
    and, in a batch of four or more, one sequence gets none."""
    b, n = case["batch"], case["tokens"]
    r = random.Random("%d %d %d" % (b, n, case["start"]))
    start = [case["start"]] + [r.randint(0, case["start"]) for _ in range(b - 1)]
    if n == b:
        return start, [1] * b
    alive = [i for i in range(b) if b < 4 or i != b // 2]
    w = [r.uniform(0.2, 1.0) for _ in alive]
    cuts = [int(n * sum(w[:i + 1]) / sum(w)) for i in range(len(alive))]
    cuts[-1] = n
    new = [0] * b
    for i, s in enumerate(alive):
        new[s] = cuts[i] - (cuts[i - 1] if i else 0)
    return start, new


def _spread(m):
    """Standard deviation of the projected dimensions: a decaying spectrum over a noise floor."""
    j = torch.arange(D, dtype=torch.float64)
    return (torch.exp(-j / 32) + 0.0025).sqrt()[:m]


_UNIONS = {}


def _union(k, m, g):
    """Expected number of key dimensions that a group of g heads keeps between them."""
    if (k, m, g) not in _UNIONS:
        gen = torch.Generator().manual_seed(0)
        z = (torch.randn(256, g, m, generator=gen, dtype=torch.float64) * _spread(m)).abs()
        keep = torch.zeros(256, g, m, dtype=torch.bool).scatter_(2, z.topk(k, dim=2).indices, True)
        _UNIONS[(k, m, g)] = float(keep.any(1).sum(1).double().mean())
    return _UNIONS[(k, m, g)]


def work(case):
    h, m, size = case["hkv"], case["d_store"], 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "append":
        n = case["tokens"]
        # new keys and values in, codes out, the projection once, a row of the rotation table for each token
        by = n * h * (2 * D * size + m + D) + h * D * m * 4 + n * case["rot"] * 4
        return {"bytes": by, "flops": 2.0 * n * h * D * m + 3.0 * n * h * case["rot"]}
    total = sum(_lengths(case))
    if case["op"] == "gather":
        return {"bytes": total * h * (m + D) * (1 + size), "flops": 0}
    hq, k = case["hq"], case["k"]
    by = total * h * (_union(k, m, hq // h) + D) + 2 * case["batch"] * hq * D * size + h * D * m * 4
    return {"bytes": by, "flops": 2.0 * total * hq * (k + D) + 2.0 * case["batch"] * hq * D * m}


# ------------------------------------------------------------------ inputs

def _table(n_pos, rot):
    """cos | sin of every position's angles, [n_pos, rot] f32 (angles in 64 bits: far positions)."""
    inv = 500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(n_pos, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


def _turn(x, cos, sin, rot, interleaved, back=False):
    """x [..., 128] with its first `rot` dimensions rotated by angles whose cos and sin are [..., rot / 2]."""
    if not rot:
        return x
    if back:
        sin = -sin
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
    return y


def _pow2_scale(amax):
    """The smallest power of two s with amax <= 448 s, at least 2^S_MIN_EXP."""
    mant, ex = torch.frexp(amax.float())
    e = ex - 9 + (mant > 0.875).int()
    e = torch.where(amax > 0, e, torch.full_like(e, S_MIN_EXP)).clamp(min=S_MIN_EXP)
    return torch.ldexp(torch.ones_like(amax, dtype=torch.float32), e)


def _codes(x):
    """f32 -> e4m3 codes (nearest even, saturating) as bytes."""
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _fill_pages(n_pages, h, rows, cols, dim_axis, gen):
    """Random page contents: codes [n_pages, h, rows, cols] and scales; `dim_axis` says which axis has the
    decaying spectrum of projected keys (None: values, all alike)."""
    codes = torch.empty(n_pages, h, rows, cols, dtype=torch.uint8, device="cuda")
    scale = torch.empty(n_pages, h, dtype=torch.float32, device="cuda")
    step = max(1, (1 << 27) // (h * rows * cols))
    sd = None if dim_axis is None else _spread(rows).float().cuda()[:, None]
    for i in range(0, n_pages, step):
        n = min(step, n_pages - i)
        x = torch.randn(n, h, rows, cols, device="cuda", generator=gen)
        if sd is not None:
            x *= sd
        x *= torch.exp(0.3 * torch.randn(n, h, 1, 1, device="cuda", generator=gen))   # pages differ in size
        s = _pow2_scale(x.abs().amax((2, 3)))
        codes[i:i + n] = _codes(x / s[:, :, None, None])
        scale[i:i + n] = s
    return codes, scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    b, h, m, page, dt = case["batch"], case["hkv"], case["d_store"], case["page"], DTYPES[case["dtype"]]
    st = {"case": case}
    if case["op"] == "append":
        start, new = _runs(case)
        ends = [s + n for s, n in zip(start, new)]
        own_pages = [(e + page - 1) // page - s // page if n else 0 for s, n, e in zip(start, new, ends)]
        n_pages = 1 + sum(own_pages)                       # page 0: a shared prefix, never appended to
        width = max(1, max((e + page - 1) // page for e in ends))
        # the pages each run touches are its own, in shuffled order; the ones before them are the shared prefix
        order = (torch.randperm(n_pages - 1, generator=gen, device="cuda") + 1).cpu().tolist()
        rows = []
        for s, n, p in zip(start, new, own_pages):
            row = [0] * width
            if n:
                row[s // page:s // page + p] = order[:p]
                order = order[p:]
            rows.append(row)
        st["table"] = torch.tensor(rows, dtype=torch.int32, device="cuda")
        st["start"] = torch.tensor(start, dtype=torch.int32, device="cuda")
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        st["cu"] = None if case["tokens"] == b else torch.tensor(cu, dtype=torch.int32, device="cuda")
        n_pos = width * page
    else:
        lens = _lengths(case)
        need = [(n + page - 1) // page for n in lens]
        n_pages, width = max(1, sum(need)), max(1, max(need))
        order = torch.randperm(n_pages, generator=gen, device="cuda")
        table = torch.full((b, width), -1, dtype=torch.int64, device="cuda")     # entries past a length are unset
        mask = torch.arange(width, device="cuda")[None, :] < torch.tensor(need, device="cuda")[:, None]
        table[mask] = order[:sum(need)]
        st["table"] = table.int()
        st["len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        n_pos = max(1, max(lens))
    st["k_pages"], st["k_scale"] = _fill_pages(n_pages, h, m, page, 0, gen)
    st["v_pages"], st["v_scale"] = _fill_pages(n_pages, h, page, D, None, gen)
    if case["op"] != "gather":
        rot, inter = case["rot"], case["interleaved"]
        st["table_rope"] = _table(n_pos, rot) if rot else None
        r = torch.linalg.qr(torch.randn(h, D, D, device="cuda", generator=gen, dtype=torch.float64))[0]
        st["P"] = r.float().contiguous()
        sd = _spread(D).cuda()
        heads, n = (case["hq"], b) if case["op"] == "decode" else (h, case["tokens"])
        # rows whose projections have the decaying spectrum once they are rotated to their position
        z = torch.randn(n, heads, D, device="cuda", generator=gen, dtype=torch.float64) * sd
        x = torch.einsum("nhgd,hed->nhge", z.view(n, h, heads // h, D), r).reshape(n, heads, D)
        if case["op"] == "decode":
            x = 3.0 * x
            pos = (st["len"].long() - 1).clamp(min=0)
        else:
            pos = _positions(st)[1]
        if rot:
            cs = st["table_rope"].double()[pos][:, None, :]
            x = _turn(x, cs[..., :rot // 2], cs[..., rot // 2:], rot, inter, back=True)
        st["x"] = x.to(dt)
        if case["op"] == "append":
            v = torch.randn(n, heads, D, device="cuda", generator=gen)
            st["v"] = (v * torch.exp(0.3 * torch.randn(n, 1, 1, device="cuda", generator=gen))).to(dt)
    if case["op"] == "gather":
        st["cap"] = max(16, -(-case["len"] // 16) * 16)
    if own:
        import sparse_dimension_attention_b200 as aq
        st["cache"] = aq.AquaPagedCache.from_buffers(st["k_pages"], st["v_pages"], st["k_scale"], st["v_scale"],
                                                     st["table"])
        if case["op"] != "gather":
            st["rope"] = aq.AquaRope(st["table_rope"], interleaved=case["interleaved"]) if case["rot"] else None
        if case["op"] == "decode":
            hq = case["hq"]
            st["ws"] = torch.empty(aq.aqua_paged_decode_workspace_size(st["cache"].desc, hq), dtype=torch.uint8,
                                   device="cuda")
            st["out"] = torch.empty(b, hq, D, dtype=dt, device="cuda")
            st["lse"] = torch.empty(b, hq, dtype=torch.float32, device="cuda")
            st["sel"] = torch.empty(b, hq, case["k"], dtype=torch.int32, device="cuda")
        if case["op"] == "gather":
            st["dst"] = aq.AquaCache(b, h, st["cap"], d_store=m, dtype=dt)
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    op = st["case"]["op"]
    if own:
        return {"append": _own_append, "decode": _own_decode, "gather": _own_gather}[op](st)
    return {"append": _plain_append, "decode": _plain_decode, "gather": _plain_gather}[op](st)


def _own_append(st):
    import sparse_dimension_attention_b200 as aq
    c = st["cache"]
    aq.aqua_paged_append(c.desc, st["x"], st["v"], st["start"], st["P"], cu_new=st["cu"], rope=st["rope"])
    return {"k": c.k_pages.view(torch.float8_e4m3fn), "v": c.v_pages.view(torch.float8_e4m3fn),
            "k_scale": c.k_scale, "v_scale": c.v_scale}


def _own_decode(st):
    import sparse_dimension_attention_b200 as aq
    case = st["case"]
    aq.aqua_paged_decode_attn(st["cache"].desc, st["x"], st["len"], st["P"], case["hq"], case["k"], st["out"],
                              st["ws"], rope=st["rope"], sel_out=st["sel"], lse_out=st["lse"])
    return {"out": st["out"], "lse": st["lse"], "sel": st["sel"]}


def _own_gather(st):
    import sparse_dimension_attention_b200 as aq
    dst = st["dst"]
    aq.aqua_paged_gather(st["cache"].desc, st["len"], dst.desc, st["case"]["len"])
    return {"k": dst.k_proj, "v": dst.v, "len": dst.len}


def _positions(st):
    """Sequence and position of every new token of an append."""
    start = st["start"].long()
    n, b = st["case"]["tokens"], st["case"]["batch"]
    tok = torch.arange(n, device="cuda")
    if st["cu"] is None:
        return tok, start
    cu = st["cu"].long()
    seq = torch.searchsorted(cu[1:].contiguous(), tok, right=True).clamp(max=b - 1)
    return seq, start[seq] + tok - cu[seq]


def _plain_append(st):
    case = st["case"]
    h, m, page = case["hkv"], case["d_store"], case["page"]
    seq, pos = _positions(st)
    pid, slot = st["table"].long()[seq, pos // page], pos % page
    k = st["x"].float()
    if case["rot"]:
        cs = st["table_rope"][pos][:, None, :]
        k = _turn(k, cs[..., :case["rot"] // 2], cs[..., case["rot"] // 2:], case["rot"], case["interleaved"])
    k = torch.einsum("nhd,hde->nhe", k, st["P"][:, :, :m])
    v = st["v"].float()
    # the page that each sequence's run starts in, when it holds tokens already
    start = st["start"].long()
    first = st["table"].long().gather(1, (start // page).clamp(max=st["table"].shape[1] - 1)[:, None])[:, 0]
    count = torch.zeros_like(start).index_add_(0, seq, torch.ones_like(seq))
    fill = torch.where(count > 0, start % page, torch.zeros_like(start))
    heads = torch.arange(h, device="cuda")[None, :]
    for name, x, by_dim in (("k", k, True), ("v", v, False)):
        pages, scale = st[name + "_pages"], st[name + "_scale"]
        size = torch.where(x.isfinite(), x.abs(), torch.zeros_like(x)).amax(-1)            # [n, h]
        amax = torch.zeros_like(scale).index_reduce_(0, pid, size, "amax")
        fresh = torch.zeros_like(scale[:, 0], dtype=torch.bool)
        fresh[pid] = True
        new = torch.where(fresh[:, None], _pow2_scale(amax), scale)                        # untouched pages keep theirs
        held = torch.zeros_like(fresh).index_put_((first,), fill > 0, accumulate=True)     # pages with tokens in them
        new = torch.where(held[:, None], torch.maximum(new, scale), new)
        # re-code what the open pages hold
        ratio = (scale / new)[first]
        old = pages[first]
        again = _codes(old.view(torch.float8_e4m3fn).float() * ratio[:, :, None, None])
        inside = torch.arange(page, device="cuda")[None, :] < fill[:, None]
        inside = inside[:, None, None, :] if by_dim else inside[:, None, :, None]
        pages[first] = torch.where(inside, again, old)
        scale.copy_(new)
        # the new tokens
        c = _codes(x / new[pid][:, :, None])
        if by_dim:
            pages[pid[:, None], heads, :, slot[:, None]] = c
        else:
            pages[pid[:, None], heads, slot[:, None]] = c
    return {"k": st["k_pages"].view(torch.float8_e4m3fn), "v": st["v_pages"].view(torch.float8_e4m3fn),
            "k_scale": st["k_scale"], "v_scale": st["v_scale"]}


def _plain_read(st):
    """K~ [B, h, m, T] and V [B, h, T, 128] in f32 from the pages; T: whole pages up to the longest sequence."""
    case = st["case"]
    b, h, m, page = case["batch"], case["hkv"], case["d_store"], case["page"]
    t = st["table"].long().clamp(min=0)
    k = st["k_pages"][t].view(torch.float8_e4m3fn).float() * st["k_scale"][t][..., None, None]
    k = k.permute(0, 2, 3, 1, 4).reshape(b, h, m, -1)
    v = st["v_pages"][t].view(torch.float8_e4m3fn).float() * st["v_scale"][t][..., None, None]
    return k, v.permute(0, 2, 1, 3, 4).reshape(b, h, -1, D)


def _plain_decode(st):
    case = st["case"]
    b, hq, h, m, kk = case["batch"], case["hq"], case["hkv"], case["d_store"], case["k"]
    g, dt = hq // h, DTYPES[case["dtype"]]
    lens = st["len"].long()
    # 64 bits up to the projected query: which of two nearly equal dimensions is kept decides the scores
    q = st["x"].double()
    if case["rot"]:
        cs = st["table_rope"].double()[(lens - 1).clamp(min=0)][:, None, :]
        q = _turn(q, cs[..., :case["rot"] // 2], cs[..., case["rot"] // 2:], case["rot"], case["interleaved"])
    q = torch.einsum("bhgd,hde->bhge", q.view(b, h, g, D), st["P"].double()).float()
    order = q[..., :m].abs().sort(dim=-1, descending=True, stable=True).indices[..., :kk]
    sel = order.sort(dim=-1).values
    qm = torch.zeros_like(q[..., :m]).scatter_(-1, sel, q.gather(-1, sel))
    keys, vals = _plain_read(st)
    s = torch.matmul(qm, keys) * (1.0 / math.sqrt(D))                                # [b, h, g, T]
    seen = torch.arange(s.shape[-1], device="cuda")[None, :] < lens[:, None]
    s = s.masked_fill(~seen[:, None, None, :], -math.inf)
    top = s.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, vals.masked_fill(~seen[:, None, :, None], 0.0)) / total
    out = torch.where(total > 0, out, torch.zeros_like(out))
    lse = torch.where(total > 0, top + torch.log(total), torch.full_like(total, -math.inf))
    return {"out": out.reshape(b, hq, D).to(dt), "lse": lse.reshape(b, hq), "sel": sel.reshape(b, hq, kk).int()}


def _plain_gather(st):
    case, cap, dt = st["case"], st["cap"], DTYPES[st["case"]["dtype"]]
    k, v = _plain_read(st)
    seen = torch.arange(cap, device="cuda")[None, :] < st["len"].long()[:, None]
    grow = cap - k.shape[-1]
    k, v = torch.nn.functional.pad(k, (0, grow)), torch.nn.functional.pad(v, (0, 0, 0, grow))
    return {"k": torch.where(seen[:, None, None, :], k, torch.zeros_like(k)).to(dt),
            "v": torch.where(seen[:, None, :, None], v, torch.zeros_like(v)).to(dt), "len": st["len"].clone()}


# ------------------------------------------------------------------ 64 bits, from the definition

def _e4m3_value(x):
    """The nearest e4m3 number of each f64 (ties to even, saturating at 448), as f64."""
    ex = torch.frexp(x.abs().clamp(min=2.0 ** -6))[1] - 1                 # floor(log2 |x|), normals from 2^-6
    step = torch.ldexp(torch.ones_like(x), ex - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _e4m3_decode(code):
    """Bytes -> the f64 they stand for, from the format: sign, four exponent bits (bias 7), three of mantissa."""
    c = code.long()
    e, f = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e > 0, torch.ldexp(1.0 + f / 8, e - 7), f * 2.0 ** -9)
    return torch.where(c >= 128, -mag, mag)


def _exact_rows(x, pos, table, rot, interleaved):
    """Rows [n, heads, 128] in f64 times the block rotation of their positions, written as complex products."""
    x = x.double()
    if not rot:
        return x
    w = torch.complex(table.double()[pos][:, :rot // 2], table.double()[pos][:, rot // 2:])[:, None, :]
    if interleaved:
        z = torch.complex(x[..., 0:rot:2].contiguous(), x[..., 1:rot:2].contiguous()) * w
        head = torch.view_as_real(z).reshape(*x.shape[:-1], rot)
    else:
        z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * w
        head = torch.cat([z.real, z.imag], -1)
    return torch.cat([head, x[..., rot:]], -1)


def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _exact_append, "decode": _exact_decode, "gather": _exact_gather}[case["op"]](st)


def _exact_append(st):
    case = st["case"]
    h, m, page = case["hkv"], case["d_store"], case["page"]
    start, new = _runs(case)
    table = st["table"].tolist()
    out = {n: _e4m3_decode(st[n + "_pages"]) for n in ("k", "v")}
    scales = {n: st[n + "_scale"].double() for n in ("k", "v")}
    at = 0
    for b, (s, n) in enumerate(zip(start, new)):
        if n:
            pos = torch.arange(s, s + n, device="cuda")
            rows = _exact_rows(st["x"][at:at + n], pos, st["table_rope"], case["rot"], case["interleaved"])
            both = {"k": torch.stack([rows[:, i] @ st["P"][i, :, :m].double() for i in range(h)]),      # [h, n, m]
                    "v": st["v"][at:at + n].double().transpose(0, 1)}
            done = 0
            while done < n:
                p, lo = table[b][(s + done) // page], (s + done) % page
                cnt = min(page - lo, n - done)
                for name, rows_of in both.items():
                    x = rows_of[:, done:done + cnt]                                      # [h, cnt, dims]
                    big = x.abs().amax((1, 2))
                    e = torch.ceil(torch.log2(big / 448))
                    e = torch.where(448 * 2.0 ** (e - 1) >= big, e - 1, e)               # log2 rounds: put e right
                    e = torch.where(448 * 2.0 ** e < big, e + 1, e).clamp(min=S_MIN_EXP)
                    sc = torch.where(big > 0, 2.0 ** e, torch.full_like(e, 2.0 ** S_MIN_EXP))
                    blk = out[name][p] if name == "v" else out[name][p].transpose(1, 2)  # [h, page, dims]
                    if lo:
                        was = scales[name][p]
                        sc = torch.maximum(sc, was)
                        blk[:, :lo] = _e4m3_value(blk[:, :lo] * (was / sc)[:, None, None])
                    blk[:, lo:lo + cnt] = _e4m3_value(x / sc[:, None, None])
                    scales[name][p] = sc
                done += cnt
        at += n
    return {"k": out["k"], "v": out["v"], "k_scale": scales["k"], "v_scale": scales["v"]}


def _exact_sequence(st, b, n):
    """K~ [h, m, n] and V [h, n, 128] of sequence b in f64."""
    t = st["table"][b, :-(-n // st["case"]["page"])].long()
    k = _e4m3_decode(st["k_pages"][t]) * st["k_scale"][t].double()[:, :, None, None]
    v = _e4m3_decode(st["v_pages"][t]) * st["v_scale"][t].double()[:, :, None, None]
    return torch.cat(list(k), -1)[..., :n], torch.cat(list(v), 1)[:, :n]


def _exact_decode(st):
    case = st["case"]
    b, hq, h, m, kk = case["batch"], case["hq"], case["hkv"], case["d_store"], case["k"]
    out = torch.zeros(b, hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((b, hq), -math.inf, dtype=torch.float64, device="cuda")
    lens = _lengths(case)
    pos = torch.tensor([max(n - 1, 0) for n in lens], device="cuda")
    q = _exact_rows(st["x"], pos, st["table_rope"], case["rot"], case["interleaved"])
    for i, n in enumerate(lens):
        if not n:
            continue
        k, v = _exact_sequence(st, i, n)
        for head in range(h):
            rows = slice(head * (hq // h), (head + 1) * (hq // h))
            qt = (q[i, rows] @ st["P"][head].double())[:, :m]
            # dimension i is kept when fewer than k others are larger, or equal and before it
            a = qt.abs()
            ahead = (a[:, None, :] > a[:, :, None]) | ((a[:, None, :] == a[:, :, None]) &
                                                      torch.ones(m, m, device="cuda").tril(-1).bool()[None])
            s = (qt * (ahead.sum(-1) < kk)) @ k[head] / math.sqrt(D)
            lse[i, rows] = torch.logsumexp(s, -1)
            out[i, rows] = torch.exp(s - lse[i, rows][:, None]) @ v[head]
    return {"out": out, "lse": lse, "sel": None}


def _exact_gather(st):
    case, cap = st["case"], st["cap"]
    b, h, m = case["batch"], case["hkv"], case["d_store"]
    k = torch.zeros(b, h, m, cap, dtype=torch.float64, device="cuda")
    v = torch.zeros(b, h, cap, D, dtype=torch.float64, device="cuda")
    for i, n in enumerate(_lengths(case)):
        if n:
            k[i, :, :, :n], v[i, :, :n] = _exact_sequence(st, i, n)
    return {"k": k, "v": v, "len": None}
