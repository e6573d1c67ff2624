"""Measured cases of the operators around the S3D8 linears of a decoder layer.

Four operators that a text decoder runs between its quantised linears:

  attention  one new token per sequence over a paged key/value cache
  append     rotary embedding of q and k, and the new keys and values into the cache's pages
  pages      copying, extending, forking, freeing and compacting the pages of a cache of many layers
  norm       the residual update behind a block (post-norm, gate, scale) with the pre-norm of the
             next block, forward (bf16 or int8 activations) and backward

With ``own`` false, ``run`` computes them with elementary torch operations in 32 bits; with ``own``
true it makes the library calls.  Sizes are those of the Llama-3.2-11B text decoder (hidden size
4096, MLP size 14336, 4096 / 1024 wide q and k/v projections = 32 / 8 heads of 128, 40 layers) and
generic ones around them.
"""
import math

import torch

own = False

LAYERS = 40


def _attn(name, batch, longest, shortest, **more):
    c = {"op": "attention", "name": name, "batch": batch, "longest": longest, "shortest": shortest,
         "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 16, "cache": "bf16", "window": 0,
         "head_major": True}
    return {**c, **more}


def _append(name, tokens, **more):
    c = {"op": "append", "name": name, "tokens": tokens, "q_heads": 32, "kv_heads": 8, "dim": 128,
         "rotary": 128, "page": 16, "cache": "bf16", "interleaved": False, "head_major": True}
    return {**c, **more}


def _pages(name, what, **more):
    c = {"op": "pages", "name": name, "what": what, "layers": LAYERS, "pages": 1024, "page": 16,
         "kv_heads": 8, "dim": 128, "rows": 64, "width": 64, "longest": 200, "count": 16,
         "head_major": True}
    return {**c, **more}


def _norm(name, tokens, hidden, **more):
    c = {"op": "norm", "name": name, "tokens": tokens, "hidden": hidden, "direction": "forward",
         "post": True, "gate": "none", "alpha": 1.0, "int8": False}
    return {**c, **more}


def listed():
    return [
        # one user, a short chat turn just begun: nothing but latency
        _attn("attention: 1 sequence of 19 tokens", 1, 19, 19),
        # a serving batch in mid-flight: every length from one token to some thousands, an idle slot
        _attn("attention: 64 sequences of 0 to 8191 tokens", 64, 8191, 0),
        # long documents, large pages, the token-major layout
        _attn("attention: 8 sequences of 90001 to 131072 tokens", 8, 131072, 90001, page=64,
              head_major=False),
        # the cache in 8 bits, sliding window over part of it
        _attn("attention: 48 sequences of 1 to 30011 tokens in int8", 48, 30011, 1, cache="int8",
              page=32, window=16384),
        # a decode step of a serving batch
        _append("append: 61 new tokens", 61),
        # a prefill of several prompts
        _append("append: 16384 tokens", 16384),
        # a prefill into an 8-bit cache
        _append("append: 4099 tokens in int8", 4099, cache="int8", page=32),
        # parallel sampling: 16 continuations forked from running sequences
        _pages("pages: fork 16 sequences", "fork"),
        # handing memory back: every other page of the pool is free
        _pages("pages: compact a half-empty pool", "compact", count=250),
        # one token between two linears of the decoder, codes out for the next linear
        _norm("norm: 1 token to int8", 1, 4096, post=False, int8=True),
        # training, gated block (cross-attention layers) with norms on both sides
        _norm("norm: backward of 8192 tokens, gated", 8192, 4096, direction="backward", gate="scalar"),
        # training forward, odd token count, channel gate
        _norm("norm: 16383 tokens, channel gate", 16383, 4096, gate="channel", alpha=0.22),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["attention", "attention", "attention", "append", "append", "pages", "norm", "norm"])
    if kind == "attention":
        while True:
            kv = rng.choice([1, 2, 4, 8, 8])
            q = kv * rng.choice([1, 2, 4, 4, 7, 8, 16])
            dim = rng.choice([64, 80, 128, 128, 128, 256])
            batch, longest = _log(rng, 1, 256), _log(rng, 1, 131072)
            cache = rng.choice(["bf16", "bf16", "int8"])
            if batch * longest * kv * dim <= 8 * 131072 * 8 * 128 // 2 and q <= 128:
                break
        return {"op": "attention", "batch": batch, "longest": longest,
                "shortest": rng.choice([0, 1, longest // 2, longest]), "q_heads": q, "kv_heads": kv,
                "dim": dim, "page": rng.choice([1, 8, 16, 16, 24, 32, 64, 128]), "cache": cache,
                "window": rng.choice([0, 0, 0, 1, 129, 4096]), "head_major": rng.random() < 0.5}
    if kind == "append":
        kv = rng.choice([1, 2, 4, 8, 8])
        dim = rng.choice([64, 80, 128, 128, 256])
        return {"op": "append", "tokens": _log(rng, 1, 12288), "q_heads": kv * rng.choice([1, 3, 4, 4]),
                "kv_heads": kv, "dim": dim, "rotary": rng.choice([dim, dim, dim // 2, 16]),
                "page": rng.choice([1, 8, 16, 16, 24, 64]), "cache": rng.choice(["bf16", "bf16", "int8"]),
                "interleaved": rng.random() < 0.3, "head_major": rng.random() < 0.5}
    if kind == "pages":
        rows = _log(rng, 2, 64)
        what = rng.choice(["copy", "extend", "fork", "fork", "free", "compact"])
        longest = _log(rng, 1, 200)
        return {"op": "pages", "what": what, "layers": rng.choice([1, 2, 7, 20, 40]), "pages": 1024,
                "page": rng.choice([8, 16, 16, 24]), "kv_heads": rng.choice([1, 2, 8]),
                "dim": rng.choice([64, 128]), "rows": rows, "width": 64, "longest": longest,
                "count": _log(rng, 1, 250) if what in ("compact", "copy") else rng.randint(1, rows // 2),
                "head_major": rng.random() < 0.5}
    while True:
        tokens, hidden = _log(rng, 1, 16384), 16 * _log(rng, 4, 1024)
        if tokens * hidden <= 16383 * 4096 // 2:
            break
    return {"op": "norm", "tokens": tokens, "hidden": hidden,
            "direction": rng.choice(["forward", "forward", "backward"]), "post": rng.random() < 0.6,
            "gate": rng.choice(["none", "scalar", "channel"]), "alpha": rng.choice([1.0, 1.0, 0.22, 2.5]),
            "int8": rng.random() < 0.3}


# ---- sizes that follow from a case ------------------------------------------


def _spread(count, lo, hi):
    """`count` lengths from lo to hi, both among them, in an order that mixes them."""
    if count == 1:
        return [hi]
    return [lo + ((i * 7919) % count) * (hi - lo) // (count - 1) if math.gcd(7919, count) == 1 else
            lo + i * (hi - lo) // (count - 1) for i in range(count)]


def _lens(c):
    if c["op"] == "pages":
        return _spread(c["rows"], 1, c["longest"])
    return _spread(c["batch"], c["shortest"], c["longest"])


def _seen(c):
    """Cache tokens that the attention of a case has to read."""
    w = c["window"]
    return sum(min(n, w) if w else n for n in _lens(c))


def _token_bytes(c):
    """Bytes of one token's key and value in all heads of one layer."""
    per_head = 2 * c["dim"] if c.get("cache", "bf16") == "bf16" else c["dim"] + 4
    return 2 * c["kv_heads"] * per_head


def work(c):
    if c["op"] == "attention":
        seen, qo = _seen(c), c["batch"] * c["q_heads"] * c["dim"] * 2
        table = sum(-(-n // c["page"]) for n in _lens(c)) * 4
        return {"bytes": seen * _token_bytes(c) + 2 * qo + table + 4 * c["batch"],
                "flops": 4 * seen * c["q_heads"] * c["dim"]}
    if c["op"] == "append":
        t, d = c["tokens"], c["dim"]
        q, kv = t * c["q_heads"] * d * 2, 2 * t * c["kv_heads"] * d * 2
        return {"bytes": 2 * q + kv + t * _token_bytes(c) + t * (4 * c["rotary"] + 8),
                "flops": 3 * t * (c["q_heads"] + c["kv_heads"]) * c["rotary"]}
    if c["op"] == "pages":
        meta = 4 * (c["rows"] * c["width"] + c["rows"] + c["pages"])
        if c["what"] in ("copy", "compact"):
            moved = c["count"] * c["page"]
        elif c["what"] == "fork":
            moved = sum(n % c["page"] for n in _lens(c)[:c["count"]])
        else:
            moved = 0
        return {"bytes": 2 * moved * c["layers"] * _token_bytes(c) + meta, "flops": 0}
    n, d = c["tokens"] * c["hidden"], c["hidden"]
    if c["direction"] == "backward":
        return {"bytes": 12 * n + 2 * d + 4 * d, "flops": 30 * n}
    return {"bytes": 6 * n + (n + 4 * c["tokens"] if c["int8"] else 2 * n) + 2 * d, "flops": 12 * n}


# ---- inputs -----------------------------------------------------------------


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, shape, dtype=torch.bfloat16, std=1.0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)


def _cache(g, lead, pages, page, heads, dim, head_major, dtype="bf16"):
    """A cache [*lead, pages, page, heads, dim] in the asked memory order, holding earlier tokens;
    int8 codes come with fp32 scales [*lead, pages, page, heads]."""
    shape = (*lead, pages, heads, page, dim) if head_major else (*lead, pages, page, heads, dim)
    n = len(lead)
    turn = (lambda t: t.transpose(n + 1, n + 2)) if head_major else (lambda t: t)
    if dtype == "bf16":
        return turn(_normal(g, shape)), None
    codes = torch.randint(-127, 128, shape, dtype=torch.int8, device="cuda", generator=g)
    scale = torch.empty(shape[:-1], device="cuda").uniform_(0.01, 0.03, generator=g)
    return turn(codes), turn(scale)


def _tables(g, c, lens, width):
    """A block table [rows, width]: each row's pages scattered over the cache, -1 behind them."""
    used = [-(-n // c["page"]) for n in lens]
    order = torch.randperm(c["pages"], device="cuda", generator=g).to(torch.int32)
    at = torch.tensor([sum(used[:i]) for i in range(len(used))], device="cuda")
    col = torch.arange(width, device="cuda")
    got = order[(at[:, None] + col).clamp(max=c["pages"] - 1)]
    have = torch.tensor(used, device="cuda")
    return torch.where(col < have[:, None], got, -1).to(torch.int32).contiguous()


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    s = {"case": c}
    if c["op"] == "attention":
        lens = _lens(c)
        c["pages"] = max(1, sum(-(-n // c["page"]) for n in lens))
        width = max(1, -(-max(lens) // c["page"]))
        s["q"] = _normal(g, (c["batch"], c["q_heads"], c["dim"]))
        for x in "kv":
            s[x], s[x + "_scale"] = _cache(g, (), c["pages"], c["page"], c["kv_heads"], c["dim"],
                                           c["head_major"], c["cache"])
        s["table"] = _tables(g, c, lens, width)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((c["batch"], c["q_heads"]), device="cuda")
    elif c["op"] == "append":
        t, d = c["tokens"], c["dim"]
        rows = max(1, min(64, t // 64)) if t > 512 else t       # a prefill, or a decode step
        each = -(-t // rows)
        before = 0 if t > 512 else 37
        width = -(-(each + before) // c["page"])
        c["pages"] = rows * width
        s["q"] = _normal(g, (t, c["q_heads"], d))
        s["new_k"], s["new_v"] = (_normal(g, (t, c["kv_heads"], d)) for _ in "kv")
        for x in "kv":
            s[x], s[x + "_scale"] = _cache(g, (), c["pages"], c["page"], c["kv_heads"], d,
                                           c["head_major"], c["cache"])
        s["table"] = torch.randperm(c["pages"], device="cuda", generator=g).to(torch.int32).view(rows, width)
        i = torch.arange(t, device="cuda")
        s["rows"] = (i // each).to(torch.int32)
        s["positions"] = (i % each + before).to(torch.int32)
        freq = 500000.0 ** (-torch.arange(0, c["rotary"], 2, device="cuda") / c["rotary"])
        angle = torch.arange(each + before, device="cuda")[:, None] * freq
        s["cos"], s["sin"] = angle.cos(), angle.sin()
        s["q_out"] = torch.empty_like(s["q"])
        if c["cache"] == "int8":
            s["values"] = [torch.empty(s[x].shape, dtype=torch.bfloat16, device="cuda") for x in "kv"]
    elif c["op"] == "pages":
        lens = _lens(c)
        lead = (c["layers"],)
        for x in "kv":
            s[x], _ = _cache(g, lead, c["pages"], c["page"], c["kv_heads"], c["dim"], c["head_major"])
        # table, lens and reference counts in one buffer, so that one copy sets them back
        r, w = c["rows"], c["width"]
        s["meta0"] = torch.empty(r * w + r + c["pages"], dtype=torch.int32, device="cuda")
        table, n, refs = _views(c, s["meta0"])
        count = c["count"]
        if c["what"] in ("extend", "fork", "free"):
            table.copy_(_tables(g, c, lens, w))
            n.copy_(torch.tensor(lens, dtype=torch.int32))
            refs.zero_()
            refs[table[table >= 0].long()] = 1
            if r > 1 and c["what"] != "fork":       # two rows share their first page
                refs[table[1, 0].long()] = 0
                table[1, 0] = table[0, 0]
                refs[table[0, 0].long()] = 2
            who = torch.arange(r, dtype=torch.int32, device="cuda")
            if c["what"] == "fork":     # rows behind the parents take the children
                s["parents"] = who[:count].contiguous()
                s["children"] = who[count:2 * count].contiguous()
                old = table[count:2 * count].flatten().long()
                refs[old[old >= 0]] = 0
                table[count:2 * count] = -1
                n[count:2 * count] = 0
            else:
                s["seqs"] = who[:count].contiguous()
                s["add"] = torch.randint(1, 40, (count,), dtype=torch.int32, device="cuda", generator=g)
        else:
            # half of the pool is live; `count` of its pages lie in the upper half
            live, most = c["pages"] // 2, c["pages"]
            low = torch.randperm(live, device="cuda", generator=g)
            high = torch.randperm(most - live, device="cuda", generator=g)[:count] + live
            have = torch.cat([low[count:], high])
            refs.zero_()
            refs[have] = 1
            have = have[torch.randperm(live, device="cuda", generator=g)].to(torch.int32)
            used = min(r * w, live)
            table.fill_(-1)
            table.view(-1)[:used] = have[:used]
            n.fill_(w * c["page"])
            s["src"], s["dst"] = high.to(torch.int32), low[:count].to(torch.int32)
        s["meta"] = s["meta0"].clone()
    else:
        t, d = c["tokens"], c["hidden"]
        s["h"], s["y"] = _normal(g, (t, d)), _normal(g, (t, d), std=0.5)
        s["w_pre"] = _normal(g, (d,), std=0.1).add_(1.0)
        s["w_post"] = _normal(g, (d,), std=0.1).add_(1.0) if c["post"] else None
        s["gate"] = {"none": None, "scalar": _normal(g, (1,)), "channel": _normal(g, (d,))}[c["gate"]]
        if c["direction"] == "backward":
            s["dh"], s["dx"] = _normal(g, (t, d)), _normal(g, (t, d))
        elif c["int8"]:
            s["values"] = torch.empty((t, d), dtype=torch.bfloat16, device="cuda")
    if own:
        s.update(_handles(s))
    return s


def _views(c, meta):
    r, w = c["rows"], c["width"]
    return meta[:r * w].view(r, w), meta[r * w:r * w + r], meta[r * w + r:]


def _handles(s):
    """The library's handles and workspaces that a program keeps between its calls."""
    import s3d8_a8_linear_gb300 as s3d8
    c = s["case"]
    if c["op"] == "attention":
        cache = s3d8.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        return {"kv": cache, "space": s3d8.paged_attention_workspace(cache, c["batch"], c["q_heads"])}
    if c["op"] == "append":
        return {"kv": s3d8.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])}
    if c["op"] == "pages":
        pool = s3d8.KVPool([s3d8.KVCache(s["k"][i], s["v"][i]) for i in range(c["layers"])])
        return {"pool": pool, "space": s3d8.pages_workspace(pool, c["rows"])}
    if c["direction"] == "backward":
        return {"space": s3d8.residual_norm_backward_workspace(c["tokens"], c["hidden"])}
    return {}


# ---- one pass ---------------------------------------------------------------


def run(s):
    c = s["case"]
    return {"attention": _run_attention, "append": _run_append, "pages": _run_pages,
            "norm": _run_norm}[c["op"]](s, c)


def _run_attention(s, c):
    if own:
        import s3d8_a8_linear_gb300 as s3d8
        s3d8.paged_attention(s["q"], s["kv"], s["table"], s["lens"], window=c["window"], out=s["out"],
                             lse=s["lse"], workspace=s["space"])
        return {"out": s["out"], "lse": s["lse"]}
    b, hq, d = s["q"].shape
    hk = c["kv_heads"]
    at = s["table"].clamp(min=0).long()
    n = at.shape[1] * c["page"]
    pos = torch.arange(n, device="cuda")
    lens = s["lens"].long()[:, None]
    seen = pos < lens
    if c["window"]:
        seen &= pos >= lens - c["window"]
    k, v = s["k"][at].reshape(b, n, hk, d).float(), s["v"][at].reshape(b, n, hk, d).float()
    if c["cache"] == "int8":
        k *= s["k_scale"][at].reshape(b, n, hk, 1)
        v *= s["v_scale"][at].reshape(b, n, hk, 1)
    v.masked_fill_(~seen[:, :, None, None], 0.0)
    q = s["q"].float().view(b, hk, hq // hk, d) * (1.0 / math.sqrt(d))
    score = torch.einsum("bhgd,bnhd->bhgn", q, k).masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = (score - top.clamp(min=-3e38)).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.einsum("bhgn,bnhd->bhgd", p, v) / total.clamp(min=1e-38)
    lse = top + total.log()
    return {"out": out.view(b, hq, d).to(torch.bfloat16), "lse": lse.view(b, hq)}


def _run_append(s, c):
    if own:
        import s3d8_a8_linear_gb300 as s3d8
        s3d8.rope_append(s["q"], s["new_k"], s["new_v"], s["cos"], s["sin"], s["positions"], s["kv"],
                         s["table"], rows=s["rows"], q_out=s["q_out"], interleaved=c["interleaved"])
        q = s["q_out"]
    else:
        at, pos = s["positions"].long(), s["rows"].long()
        page, slot = s["table"][pos, at // c["page"]].long(), at % c["page"]
        q = _rotate(s, c, s["q"], at).to(torch.bfloat16)
        k, v = _rotate(s, c, s["new_k"], at), s["new_v"].float()
        if c["cache"] == "int8":
            k, s["k_scale"][page, slot] = _codes(k)
            v, s["v_scale"][page, slot] = _codes(v)
        s["k"][page, slot] = k.to(s["k"].dtype)
        s["v"][page, slot] = v.to(s["v"].dtype)
    if c["cache"] == "int8":
        torch.mul(s["k"], s["k_scale"][..., None], out=s["values"][0])
        torch.mul(s["v"], s["v_scale"][..., None], out=s["values"][1])
        return {"q": q, "k": s["values"][0], "v": s["values"][1]}
    return {"q": q, "k": s["k"], "v": s["v"]}


def _rotate(s, c, x, at):
    x, r = x.float(), c["rotary"]
    cos, sin = s["cos"][at][:, None], s["sin"][at][:, None]
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if c["interleaved"] else (x[..., :r // 2], x[..., r // 2:r])
    turned = (a * cos - b * sin, b * cos + a * sin)
    turned = torch.stack(turned, -1).flatten(-2) if c["interleaved"] else torch.cat(turned, -1)
    return torch.cat((turned, x[..., r:]), -1)


def _codes(x):
    """int8 codes (as floats) and scales of the last axis: absmax / 127, nearest even."""
    scale = x.abs().amax(-1) / torch.full((), 127.0, device="cuda")
    q = (x / scale.masked_fill(scale == 0, 1.0)[..., None]).round_().clamp_(-127, 127)
    return q, scale


def _run_pages(s, c):
    s["meta"].copy_(s["meta0"])      # the tables as they were: a pass can be made again
    table, lens, refs = _views(c, s["meta"])
    out = {"k": s["k"], "v": s["v"], "table": table, "lens": lens, "refs": refs}
    what = c["what"]
    if own:
        import s3d8_a8_linear_gb300 as s3d8
        if what == "copy":
            s3d8.copy_pages(s["pool"], s["src"], s["dst"])
        elif what == "extend":
            out["got"] = s3d8.extend_pages(table, lens, refs, s["seqs"], s["add"], c["page"], workspace=s["space"])
        elif what == "fork":
            out["got"] = s3d8.fork_pages(s["pool"], table, lens, refs, s["parents"], s["children"], workspace=s["space"])
        elif what == "free":
            s3d8.free_pages(table, lens, refs, s["seqs"])
        else:
            out["live"] = s3d8.compact_pages(s["pool"], table, refs, workspace=s["space"])
        return out
    if what == "copy":
        s["k"][:, s["dst"].long()] = s["k"][:, s["src"].long()]
        s["v"][:, s["dst"].long()] = s["v"][:, s["src"].long()]
    elif what == "extend":
        out["got"] = _extend(s, c, table, lens, refs)
    elif what == "fork":
        out["got"] = _fork(s, c, table, lens, refs)
    elif what == "free":
        rows = table[s["seqs"].long()]
        refs.scatter_add_(0, rows.clamp(min=0).flatten().long(), -(rows >= 0).flatten().int())
        table[s["seqs"].long()] = -1
        lens[s["seqs"].long()] = 0
    else:
        out["live"] = _compact(s, c, table, refs)
    return out


def _lowest_free(refs):
    """Free page ids in ascending order (live ones behind them), and how many are free."""
    live = refs != 0
    return torch.argsort(live, stable=True), (~live).sum()


def _extend(s, c, table, lens, refs):
    rows, col = s["seqs"].long(), torch.arange(c["width"], device="cuda")
    have = (lens[rows] + (c["page"] - 1)) // c["page"]
    want = (lens[rows] + s["add"] + (c["page"] - 1)) // c["page"]
    fits = want <= c["width"]
    need = torch.where(fits, want - have, 0)
    begin = need.cumsum(0) - need
    ids, free = _lowest_free(refs)
    ok = fits & ((need == 0) | (begin + need <= free))
    new = (col >= have[:, None]) & (col < want[:, None]) & ok[:, None]
    page = ids[(begin[:, None] + col - have[:, None]).clamp(0, c["pages"] - 1)]
    table[rows] = torch.where(new, page.int(), table[rows])
    refs.scatter_add_(0, page.flatten(), new.flatten().int())
    lens[rows] += torch.where(ok, s["add"], 0)
    return ok.int()


def _fork(s, c, table, lens, refs):
    parents, children = s["parents"].long(), s["children"].long()
    n, col = lens[parents], torch.arange(c["width"], device="cuda")
    full, part = n // c["page"], n % c["page"]
    need = part > 0
    rank = need.cumsum(0) - 1
    ids, free = _lowest_free(refs)
    ok = ~need | (rank < free)
    new = ids[rank.clamp(0)]
    rows = table[parents]
    last = rows.gather(1, full.clamp(max=c["width"] - 1)[:, None].long())[:, 0].clamp(min=0).long()
    shared = (col < full[:, None]) & ok[:, None]
    fresh = need & ok
    child = torch.where(shared, rows, -1)
    table[children] = torch.where((col == full[:, None]) & fresh[:, None], new[:, None].int(), child)
    lens[children] = torch.where(ok, n, 0)
    refs.scatter_add_(0, rows.clamp(min=0).flatten().long(), shared.flatten().int())
    refs.scatter_add_(0, new, fresh.int())
    to = torch.where(fresh, new, rows[:, 0].clamp(min=0).long())     # a live page keeps what it has
    some = ((torch.arange(c["page"], device="cuda") < part[:, None]) & fresh[:, None])[:, :, None, None]
    s["k"][:, to] = torch.where(some, s["k"][:, last], s["k"][:, to])
    s["v"][:, to] = torch.where(some, s["v"][:, last], s["v"][:, to])
    return ok.int()


def _compact(s, c, table, refs):
    ids = torch.arange(c["pages"], device="cuda")
    live = refs != 0
    count = live.sum()
    hole, mover = ~live & (ids < count), live & (ids >= count)
    holes, movers = hole.nonzero()[:, 0], mover.nonzero()[:, 0]     # as many of either
    to = ids.scatter(0, movers, holes)                              # new id of each page
    s["k"][:, holes] = s["k"][:, movers]
    s["v"][:, holes] = s["v"][:, movers]
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()].int(), table))
    refs[holes] = refs[movers]
    refs[movers] = 0
    return count.int().view(1)


def _run_norm(s, c):
    more = {"w_post": s["w_post"], "gate": s["gate"], "alpha": c["alpha"], "tanh_gate": c["gate"] == "scalar"}
    eps = 1e-5
    if own:
        import s3d8_a8_linear_gb300 as s3d8
        if c["direction"] == "backward":
            return s3d8.residual_norm_backward(s["dh"], s["dx"], s["h"], s["y"], w_pre=s["w_pre"], eps=eps,
                                               workspace=s["space"], **more)
        if c["int8"]:
            h, codes, scale = s3d8.residual_norm_quant(s["h"], s["y"], w_pre=s["w_pre"], eps=eps, **more)
            return {"h": h, "x": torch.mul(codes, scale[:, None], out=s["values"])}
        h, x = s3d8.residual_norm(s["h"], s["y"], w_pre=s["w_pre"], eps=eps, **more)
        return {"h": h, "x": x}
    y, wp = s["y"].float(), s["w_pre"].float()
    r_post = (y.square().mean(-1, keepdim=True) + eps).rsqrt() if c["post"] else None
    u = y * r_post * s["w_post"].float() if c["post"] else y
    g = s["gate"].float() if s["gate"] is not None else torch.ones(1, device="cuda")
    slope = 1.0 - g.tanh().square() if more["tanh_gate"] else torch.ones_like(g)
    gain = c["alpha"] * (g.tanh() if more["tanh_gate"] else g)
    if c["direction"] == "backward":
        h, dx = s["h"].float(), s["dx"].float()      # h: the stream behind the update, as stored
        r = (h.square().mean(-1, keepdim=True) + eps).rsqrt()
        a = dx * wp
        gh = s["dh"].float() + r * a - h * (r.pow(3) * (a * h).mean(-1, keepdim=True))
        du = gh * gain
        grads = {"dh": gh.to(torch.bfloat16), "dw_pre": (dx * h * r).sum(0)}
        if c["post"]:
            b = du * s["w_post"].float()
            dy = r_post * b - y * (r_post.pow(3) * (b * y).mean(-1, keepdim=True))
            grads["dw_post"] = (du * y * r_post).sum(0)
        else:
            dy = du
        grads["dy"] = dy.to(torch.bfloat16)
        if s["gate"] is not None:
            dg = (gh * u).sum(0)
            grads["dgate"] = c["alpha"] * slope * (dg.sum(0, keepdim=True) if c["gate"] == "scalar" else dg)
        return grads
    h = (s["h"].float() + gain * u).to(torch.bfloat16)
    hf = h.float()
    x = (hf * (hf.square().mean(-1, keepdim=True) + eps).rsqrt() * wp).to(torch.bfloat16)
    if c["int8"]:
        codes, scale = _codes(x.float())
        return {"h": h, "x": torch.mul(codes, scale[:, None], out=s["values"])}
    return {"h": h, "x": x}


# ---- the definitions in 64 bits ---------------------------------------------


def exact(case, seed):
    if case["op"] == "pages":
        return None         # nothing is computed but whole numbers and copies
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] != "attention":
        return _exact_append(s, c) if c["op"] == "append" else _exact_norm(s, c)
    hq, d, hk = c["q_heads"], c["dim"], c["kv_heads"]
    out = torch.zeros((c["batch"], hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((c["batch"], hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lens(c)):
        first = max(0, n - c["window"]) if c["window"] else 0
        if n == 0:
            continue
        pos = torch.arange(first, n, device="cuda")
        page, slot = s["table"][b].long()[pos // c["page"]], pos % c["page"]
        for h in range(hk):
            k, v = s["k"][page, slot, h].double(), s["v"][page, slot, h].double()
            if c["cache"] == "int8":
                k *= s["k_scale"][page, slot, h].double()[:, None]
                v *= s["v_scale"][page, slot, h].double()[:, None]
            heads = slice(h * (hq // hk), (h + 1) * (hq // hk))
            score = s["q"][b, heads].double() @ k.T / math.sqrt(d)
            lse[b, heads] = torch.logsumexp(score, -1)
            out[b, heads] = torch.exp(score - lse[b, heads, None]) @ v
    return {"out": out, "lse": lse}


def _exact_append(s, c):
    r, pos = c["rotary"], s["positions"].long()
    angle = torch.complex(s["cos"].double(), s["sin"].double())[pos][:, None]

    def turn(x):
        x = x.double().clone()
        if c["interleaved"]:
            z = torch.complex(x[..., 0:r:2].clone(), x[..., 1:r:2].clone()) * angle
            x[..., 0:r:2], x[..., 1:r:2] = z.real, z.imag
        else:
            z = torch.complex(x[..., :r // 2].clone(), x[..., r // 2:r].clone()) * angle
            x[..., :r // 2], x[..., r // 2:r] = z.real, z.imag
        return x

    def store(cache, scale, new):
        old = cache.double() if scale is None else cache.double() * scale.double()[..., None]
        if scale is not None:
            step = new.abs().amax(-1, keepdim=True) / 127
            new = torch.where(step > 0, (new / step).round() * step, 0.0)
        old[s["table"].long()[s["rows"].long(), pos // c["page"]], pos % c["page"]] = new
        return old

    return {"q": turn(s["q"]), "k": store(s["k"], s["k_scale"], turn(s["new_k"])),
            "v": store(s["v"], s["v_scale"], s["new_v"].double())}


def _exact_norm(s, c):
    eps, d = 1e-5, c["hidden"]
    y, wp = s["y"].double(), s["w_pre"].double()
    wo = s["w_post"].double() if c["post"] else torch.ones(d, dtype=torch.float64, device="cuda")
    inv = torch.rsqrt((y * y).sum(-1, keepdim=True) / d + eps) if c["post"] else torch.ones_like(y[:, :1])
    unit = y * inv
    raw = s["gate"].double() if s["gate"] is not None else torch.ones(1, dtype=torch.float64, device="cuda")
    tanh = c["gate"] == "scalar"
    gain = c["alpha"] * (torch.tanh(raw) if tanh else raw)
    if c["direction"] == "forward":
        h = (s["h"].double() + gain * wo * unit)
        kept = h.to(torch.bfloat16).double()        # the stream is held in bf16, and normalised as held
        x = kept * torch.rsqrt((kept * kept).sum(-1, keepdim=True) / d + eps) * wp
        if c["int8"]:
            x = x.to(torch.bfloat16).double()
            step = x.abs().amax(-1, keepdim=True) / 127
            x = torch.where(step > 0, (x / step).round() * step, 0.0)
        return {"h": h, "x": x}
    h, dx = s["h"].double(), s["dx"].double()
    inv_h = torch.rsqrt((h * h).sum(-1, keepdim=True) / d + eps)
    hat = h * inv_h
    a = dx * wp
    total = s["dh"].double() + inv_h * (a - hat * (a * hat).sum(-1, keepdim=True) / d)
    du = total * gain
    b = du * wo
    dy = inv * (b - unit * (b * unit).sum(-1, keepdim=True) / d) if c["post"] else du
    got = {"dh": total, "dw_pre": (dx * hat).sum(0), "dy": dy}
    if c["post"]:
        got["dw_post"] = (du * unit).sum(0)
    if s["gate"] is not None:
        dg = (total * wo * unit).sum(0)
        slope = 1 / torch.cosh(raw) ** 2 if tanh else torch.ones_like(raw)
        got["dgate"] = c["alpha"] * slope * (dg.sum().view(1) if c["gate"] == "scalar" else dg)
    return got
