"""Measured cases of a vision decoder's operators around its S3D8 linears.

  cross   attention of text tokens to the encoder's states of their images, each token over a
          span of them: prompts, single tokens, and a training step with its gradients
  rope    the norm of each query and key head with the rotation in the same pass: into the paged
          cache, as tensors, and the gradients
  sample  the next token of each sequence from the head's logits and given random numbers:
          temperature, top-k, top-p, min-p

With ``own`` false, ``run`` computes them with elementary torch operations (32 bits; 64 for the
sums of a whole vocabulary, which decide on tokens); with ``own`` true it makes the library calls.
Sizes are those of the Llama-3.2-11B text decoder (32 / 8 heads of 128, a vocabulary of 128256)
with images of 1601 states a tile, and generic ones around them.
"""
import math

import torch

own = False

VOCAB = 128256
EPS = 1e-5


def _cross(name, batch, tokens, states, **more):
    c = {"op": "cross", "name": name, "batch": batch, "tokens": tokens, "states": states, "images": 1,
         "shortest": states, "blind": 0, "q_heads": 32, "kv_heads": 8, "dim": 128, "train": False}
    return {**c, **more}


def _rope(name, what, tokens, **more):
    c = {"op": "rope", "name": name, "what": what, "tokens": tokens, "q_heads": 32, "kv_heads": 8,
         "dim": 128, "rotary": 128, "page": 16, "cache": "bf16", "interleaved": False}
    return {**c, **more}


def _sample(name, rows, **more):
    c = {"op": "sample", "name": name, "rows": rows, "vocab": VOCAB, "limits": "all", "spread": 3.0,
         "banned": 0.0}
    return {**c, **more}


def listed():
    return [
        # one user's next token, one image tile: nothing but latency
        _cross("cross: 1 token, 1601 states", 1, 1, 1601),
        # a serving batch: every sequence its own images, some smaller, one without any
        _cross("cross: 48 tokens, 48 x 6404 states", 48, 1, 6404, shortest=0),
        # four prompts with an image of four tiles each, an odd length, text in front of the image
        _cross("cross: 4 x 2047 tokens, 4 x 6404 states", 4, 2047, 6404, blind=5),
        # a training step of long documents, two images one after the other in each
        _cross("cross: train 2 x 2048 tokens, 2 x 6404 states", 2, 2048, 6404, images=2, train=True),
        # a training step of a small model: short texts, narrow heads, ragged images
        _cross("cross: train 5 x 333 tokens, 5 x 1601 states", 5, 333, 1601, shortest=700, blind=3,
               q_heads=16, kv_heads=16, dim=80, train=True),
        # a decode step of a serving batch
        _rope("rope: append 61 tokens", "append", 61),
        # a prefill of several prompts
        _rope("rope: append 16384 tokens", "append", 16384),
        # the keys of four prompts' images, which have no position
        _rope("rope: norm 25616 x 8 heads", "forward", 25616, q_heads=8, kv_heads=0, rotary=0),
        # a training step's gradients
        _rope("rope: backward of 8191 tokens", "backward", 8191),
        # one user's next token
        _sample("sample: 1 row", 1),
        # a serving batch, every row with limits of its own, some words banned
        _sample("sample: 64 rows, mixed", 64, limits="mixed", banned=0.2),
        # many continuations of one prompt, from the whole vocabulary
        _sample("sample: 509 rows, temperature", 509, limits="none"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["cross", "cross", "cross", "rope", "rope", "sample", "sample"])
    if kind == "cross":
        while True:
            train = rng.random() < 0.4
            batch, tokens, states = _log(rng, 1, 64), _log(rng, 1, 4096), _log(rng, 1, 16384)
            kv = rng.choice([1, 2, 4, 8, 8, 16])
            q, dim = kv * rng.choice([1, 1, 2, 4, 4, 5, 8]), rng.choice([16, 64, 64, 80, 96, 128, 128])
            if rng.random() < 0.3:
                tokens = 1
            pairs = batch * tokens * states * q
            if pairs * max(dim, 64) <= 4 * 2047 * 6404 * 4096 // (7 if train else 2) and q <= 64 \
                    and batch * states * kv * dim <= 48 * 6404 * 1024:
                break
        images = min(tokens, states, rng.choice([1, 1, 2, 3]))
        return {"op": "cross", "batch": batch, "tokens": tokens, "states": states, "images": images,
                "shortest": rng.choice([0, 1, states // 2, states, states]) // images,
                "blind": rng.choice([0, 0, min(3, tokens // 2)]),
                "q_heads": q, "kv_heads": kv, "dim": dim, "train": train}
    if kind == "rope":
        kv, dim = rng.choice([1, 2, 4, 8, 8]), rng.choice([64, 80, 128, 128, 256])
        what = rng.choice(["append", "append", "forward", "backward"])
        rotary = rng.choice([dim, dim, dim // 2, 16] + ([0] if what != "append" else []))
        return {"op": "rope", "what": what, "tokens": _log(rng, 1, 12288),
                "q_heads": kv * rng.choice([1, 3, 4, 4]), "kv_heads": kv, "dim": dim, "rotary": rotary,
                "page": rng.choice([1, 8, 16, 16, 24, 64]), "cache": rng.choice(["bf16", "bf16", "int8"]),
                "interleaved": rng.random() < 0.3}
    while True:
        rows, vocab = _log(rng, 1, 512), _log(rng, 8, 262144)
        if rows * vocab <= 509 * VOCAB:
            break
    return {"op": "sample", "rows": rows, "vocab": vocab, "limits": rng.choice(["all", "mixed", "none"]),
            "spread": rng.choice([0.5, 2.0, 3.0, 8.0]), "banned": rng.choice([0.0, 0.0, 0.3])}


# ---- sizes that follow from a case ------------------------------------------


def _visible(c):
    """Per sequence and image, how many of its states are real (an image fills its share of the
    sequence's states, or less)."""
    share, n = c["states"] // c["images"], c["batch"] * c["images"]
    low = min(c["shortest"], share)
    return [share - i * (share - low) // max(1, n - 1) for i in range(n)]


def _image_of(c):
    """For each token of a sequence, the image that it looks at; -1 for the first `blind` ones."""
    return [-1 if t < c["blind"] else t * c["images"] // c["tokens"] for t in range(c["tokens"])]


def work(c):
    if c["op"] == "cross":
        seen, at = _visible(c), _image_of(c)
        lookers = [at.count(i) for i in range(c["images"])]
        pairs = sum(n * lookers[i % c["images"]] for i, n in enumerate(seen))
        used = sum(n for i, n in enumerate(seen) if lookers[i % c["images"]])
        rows = c["batch"] * c["tokens"]
        q, kv = 2 * rows * c["q_heads"] * c["dim"], 4 * used * c["kv_heads"] * c["dim"]
        if c["train"]:      # q, dout -> out, dq; k, v -> dk, dv
            return {"bytes": 4 * q + 2 * kv + 8 * rows, "flops": 14 * pairs * c["q_heads"] * c["dim"]}
        return {"bytes": 2 * q + kv + 8 * rows + 4 * rows * c["q_heads"],
                "flops": 4 * pairs * c["q_heads"] * c["dim"]}
    if c["op"] == "rope":
        keyed = c["tokens"] * (c["q_heads"] + c["kv_heads"]) * c["dim"]
        angles = c["tokens"] * (4 * c["rotary"] + 4)
        if c["what"] == "append":
            v = c["tokens"] * c["kv_heads"] * c["dim"]
            stored = 2 * 2 * v if c["cache"] == "bf16" else 2 * (v + 4 * v // c["dim"])
            return {"bytes": 2 * keyed + 2 * v + 2 * (keyed - v) + stored + angles + 4 * c["tokens"],
                    "flops": 7 * keyed}
        if c["what"] == "forward":
            return {"bytes": 4 * keyed + angles, "flops": 7 * keyed}
        return {"bytes": 6 * keyed + angles, "flops": 14 * keyed}
    n = c["rows"] * c["vocab"]
    return {"bytes": 2 * n + 24 * c["rows"], "flops": 4 * n}


# ---- inputs -----------------------------------------------------------------


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, shape, std=1.0):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, std, generator=g)


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    s = {"case": c}
    {"cross": _prepare_cross, "rope": _prepare_rope, "sample": _prepare_sample}[c["op"]](s, c, g)
    return s


def _prepare_cross(s, c, g):
    b, n, m, d = c["batch"], c["tokens"], c["states"], c["dim"]
    s["q"] = _normal(g, (b * n, c["q_heads"], d))
    # keys and values side by side, as one projection of the states gives them
    both = _normal(g, (b * m, 2 * c["kv_heads"], d))
    s["k"], s["v"] = both[:, :c["kv_heads"]], both[:, c["kv_heads"]:]
    if c["train"]:
        s["dout"] = _normal(g, (b * n, c["q_heads"], d))
    share = m // c["images"]
    at = torch.tensor(_image_of(c), device="cuda").expand(b, n)
    real = torch.tensor(_visible(c), device="cuda").view(b, c["images"])
    first = torch.arange(b, device="cuda")[:, None] * m + at.clamp(min=0) * share
    last = first + torch.where(at < 0, 0, real.gather(1, at.clamp(min=0)))
    s["spans"] = torch.stack((first, last), -1).view(b * n, 2).to(torch.int32)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((b * n, c["q_heads"]), device="cuda")
    if own:
        import s3d8_a8_linear_gb300 as s3d8
        size = (b * n, b * m, c["q_heads"], c["kv_heads"], d)
        s["space"] = s3d8.cross_attention_workspace(*size)
        if c["train"]:
            s["back"] = s3d8.cross_attention_backward_workspace(*size)


def _prepare_rope(s, c, g):
    t, d, hq, hk = c["tokens"], c["dim"], c["q_heads"], c["kv_heads"]
    append = c["what"] == "append"
    # what one projection gives: queries, keys (and values) of a token side by side
    fused = _normal(g, (t, hq + (2 if append else 1) * hk, d))
    s["q"], s["new_k"] = fused[:, :hq], fused[:, hq:hq + hk]
    s["q_norm"], s["k_norm"] = (_normal(g, (d,), 0.1).add_(1.0) for _ in "qk")
    rows = max(1, min(64, t // 64)) if t > 512 else t       # a prefill, or a decode step
    each = -(-t // rows)
    before = 0 if t > 512 else 37
    i = torch.arange(t, device="cuda")
    s["positions"] = (i % each + before).to(torch.int32)
    if c["rotary"]:
        freq = 500000.0 ** (-torch.arange(0, c["rotary"], 2, device="cuda").double() / c["rotary"])
        angle = torch.arange(each + before, device="cuda")[:, None] * freq
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
    else:
        s["cos"] = s["sin"] = None
    if append:
        s["new_v"] = fused[:, hq + hk:]
        width = -(-(each + before) // c["page"])
        pages = rows * width
        shape = (pages, hk, c["page"], d)
        s["k"], s["k_scale"] = _cache(g, shape, c["cache"])
        s["v"], s["v_scale"] = _cache(g, shape, c["cache"])
        s["table"] = torch.randperm(pages, device="cuda", generator=g).to(torch.int32).view(rows, width)
        s["rows"] = (i // each).to(torch.int32)
        s["q_out"] = torch.empty((t, hq, d), dtype=torch.bfloat16, device="cuda")
        if c["cache"] == "int8":
            s["values"] = [torch.empty(s["k"].shape, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
        if own:
            import s3d8_a8_linear_gb300 as s3d8
            s["kv"] = s3d8.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    elif c["what"] == "backward":
        s["dq"], s["dk"] = _normal(g, (t, hq, d)), _normal(g, (t, hk, d))
        if own:
            import s3d8_a8_linear_gb300 as s3d8
            s["space"] = s3d8.norm_rope_backward_workspace(t, hq, hk, d)


def _cache(g, shape, kind):
    """One side of a cache that holds earlier tokens, and its scales."""
    if kind == "bf16":
        return _normal(g, shape).transpose(1, 2), None
    codes = torch.randint(-127, 128, shape, dtype=torch.int8, device="cuda", generator=g)
    return codes.transpose(1, 2), torch.empty(shape[:3], device="cuda").uniform_(0.01, 0.03, generator=g).transpose(1, 2)


def _prepare_sample(s, c, g):
    n, v = c["rows"], c["vocab"]
    # a head's logits: most tokens in a wide bulk, a few well above it
    x = torch.empty((n, v), device="cuda").normal_(0.0, 1.0, generator=g)
    x = c["spread"] * (x + 0.15 * x.square() * x.sign())
    if c["banned"]:
        x.masked_fill_(torch.rand((n, v), device="cuda", generator=g) < c["banned"], -math.inf)
    s["logits"] = x.to(torch.bfloat16)
    s["u"] = torch.rand((n,), device="cuda", generator=g)
    i = torch.arange(n, device="cuda")
    s["temperature"] = 0.6 + 0.05 * (i % 13).float()
    s["top_k"] = s["top_p"] = s["min_p"] = None
    if c["limits"] == "all":
        s["top_k"] = (20 + i % 50).to(torch.int32)
        s["top_p"] = 0.9 + 0.01 * (i % 8).float()
        s["min_p"] = 0.01 + 0.01 * (i % 5).float()
    elif c["limits"] == "mixed":        # each row one limit, several, none, or the largest logit
        s["temperature"] = torch.where(i % 7 == 6, 0.0, s["temperature"])
        s["top_k"] = torch.where(i % 3 == 0, 1 + (i * 37) % 1000, 0).to(torch.int32)
        s["top_p"] = torch.where(i % 4 < 2, 0.5 + 0.45 * s["u"].roll(1), 1.0)
        s["min_p"] = torch.where(i % 5 == 1, 0.05, 0.0)
    s["logprob"] = torch.empty((n,), device="cuda")


# ---- one pass ---------------------------------------------------------------


def run(s):
    c = s["case"]
    return {"cross": _run_cross, "rope": _run_rope, "sample": _run_sample}[c["op"]](s, c)


def _run_cross(s, c):
    if own:
        import s3d8_a8_linear_gb300 as s3d8
        s3d8.cross_attention(s["q"], s["k"], s["v"], s["spans"], out=s["out"], lse=s["lse"], workspace=s["space"])
        if not c["train"]:
            return {"out": s["out"], "lse": s["lse"]}
        g = s3d8.cross_attention_backward(s["dout"], s["q"], s["k"], s["v"], s["out"], s["lse"], s["spans"],
                                          workspace=s["back"])
        return {"out": s["out"], "dq": g["dq"], "dk": g["dk"], "dv": g["dv"]}
    b, n, m, d, hk = c["batch"], c["tokens"], c["states"], c["dim"], c["kv_heads"]
    group, scale = c["q_heads"] // hk, 1.0 / math.sqrt(c["dim"])

    def rows(x):    # [b, hk, tokens x group, d]: the query heads of a key/value head follow their token
        return x.float().view(b, n, hk, group, d).permute(0, 2, 1, 3, 4).reshape(b, hk, n * group, d)

    def back(x):
        return x.view(b, hk, n, group, d).permute(0, 2, 1, 3, 4).reshape(b * n, hk * group, d).to(torch.bfloat16)

    def keyed(x):
        return x.float().view(b, m, hk, d).transpose(1, 2)

    q, k, v = rows(s["q"]), keyed(s["k"]), keyed(s["v"])
    spans = s["spans"].view(b, n, 1, 2) - torch.arange(b, device="cuda").view(b, 1, 1, 1) * m
    at = torch.arange(m, device="cuda")
    seen = (at >= spans[..., :1]) & (at < spans[..., 1:])                       # [b, n, 1, m]
    seen = seen.expand(b, n, group, m).reshape(b, 1, n * group, m)
    p = torch.matmul(q, k.transpose(-1, -2)).mul_(scale).masked_fill_(~seen, -math.inf)
    top = p.amax(-1, keepdim=True)
    p.sub_(top.clamp(min=-3e38)).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (top + total.log()).view(b, hk, n, group).transpose(1, 2).reshape(b * n, hk * group)
    p.div_(total.clamp(min=1e-38))
    out = torch.matmul(p, v)
    if not c["train"]:
        return {"out": back(out), "lse": lse}
    dout = rows(s["dout"])
    dv = torch.matmul(p.transpose(-1, -2), dout)
    delta = (dout * out).sum(-1, keepdim=True)
    ds = torch.matmul(dout, v.transpose(-1, -2)).sub_(delta).mul_(p).mul_(scale)
    dq, dk = torch.matmul(ds, k), torch.matmul(ds.transpose(-1, -2), q)
    flat = [x.transpose(1, 2).reshape(b * m, hk, d).to(torch.bfloat16) for x in (dk, dv)]
    return {"out": back(out), "dq": back(dq), "dk": flat[0], "dv": flat[1]}


def _turn(s, c, x, back=False):
    r = c["rotary"]
    if not r:
        return x
    at = s["positions"].long()
    cos, sin = s["cos"][at][:, None], s["sin"][at][:, None]
    if back:
        sin = -sin
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if c["interleaved"] else (x[..., :r // 2], x[..., r // 2:r])
    turned = (a * cos - b * sin, b * cos + a * sin)
    turned = torch.stack(turned, -1).flatten(-2) if c["interleaved"] else torch.cat(turned, -1)
    return torch.cat((turned, x[..., r:]), -1)


def _normed(s, c, x, w):
    x = x.float()
    return _turn(s, c, x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * w.float())


def _normed_back(s, c, dz, x, w):
    x, dy = x.float(), _turn(s, c, dz.float(), back=True)
    unit = x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    a = dy * w.float()
    dx = (a - unit * (a * unit).mean(-1, keepdim=True)) * (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    return dx.to(torch.bfloat16), (dy * unit).sum((0, 1))


def _codes(x):
    """int8 codes (as floats) and scales of the last axis: absmax / 127, nearest even."""
    scale = x.abs().amax(-1) / torch.full((), 127.0, device="cuda")
    q = (x / scale.masked_fill(scale == 0, 1.0)[..., None]).round_().clamp_(-127, 127)
    return q, scale


def _run_rope(s, c):
    at = {"positions": s["positions"], "interleaved": c["interleaved"], "eps": EPS}
    if c["what"] == "append":
        return _run_append(s, c)
    some_k = c["kv_heads"] > 0
    if c["what"] == "forward":
        if own:
            import s3d8_a8_linear_gb300 as s3d8
            q, k = s3d8.norm_rope(s["q"], s["new_k"] if some_k else None, s["q_norm"],
                                  s["k_norm"] if some_k else None, s["cos"], s["sin"], **at)
            return {"q": q, "k": k} if some_k else {"q": q}
        got = {"q": _normed(s, c, s["q"], s["q_norm"]).to(torch.bfloat16)}
        if some_k:
            got["k"] = _normed(s, c, s["new_k"], s["k_norm"]).to(torch.bfloat16)
        return got
    if own:
        import s3d8_a8_linear_gb300 as s3d8
        return s3d8.norm_rope_backward(s["dq"], s["dk"], s["q"], s["new_k"], s["q_norm"], s["k_norm"], s["cos"],
                                       s["sin"], workspace=s["space"], **at)
    dq, dwq = _normed_back(s, c, s["dq"], s["q"], s["q_norm"])
    dk, dwk = _normed_back(s, c, s["dk"], s["new_k"], s["k_norm"])
    return {"dq": dq, "dk": dk, "dq_norm": dwq, "dk_norm": dwk}


def _run_append(s, c):
    if own:
        import s3d8_a8_linear_gb300 as s3d8
        q = s3d8.rope_append(s["q"], s["new_k"], s["new_v"], s["cos"], s["sin"], s["positions"], s["kv"], s["table"],
                             rows=s["rows"], q_out=s["q_out"], interleaved=c["interleaved"], q_norm=s["q_norm"],
                             k_norm=s["k_norm"], eps=EPS)
    else:
        at = s["positions"].long()
        page, slot = s["table"][s["rows"].long(), at // c["page"]].long(), at % c["page"]
        q = _normed(s, c, s["q"], s["q_norm"]).to(torch.bfloat16)
        k, v = _normed(s, c, s["new_k"], s["k_norm"]), s["new_v"].float()
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


def _run_sample(s, c):
    if own:
        import s3d8_a8_linear_gb300 as s3d8
        tokens = s3d8.sample(s["logits"], s["u"], s["temperature"], s["top_k"], s["top_p"], s["min_p"],
                             logprob=s["logprob"])
        return {"tokens": tokens, "logprob": s["logprob"]}
    n, v = s["logits"].shape
    x, order = torch.sort(s["logits"].float(), dim=-1, descending=True, stable=True)
    temp = s["temperature"].double()[:, None]
    hot = temp > 0
    w = ((x.double() - x[:, :1].double()) / torch.where(hot, temp, 1.0)).exp()
    w = torch.where(hot | (torch.arange(v, device="cuda") == 0), w, 0.0)        # cold: the first alone
    mass = w.cumsum(-1)
    last = torch.full((n, 1), v, device="cuda")
    if s["top_k"] is not None:
        k = s["top_k"].long()[:, None]
        last = torch.where(k > 0, k.clamp(max=v), last)
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        some = (mass < p * mass.gather(1, last - 1)).sum(-1, keepdim=True) + 1
        last = torch.where(p < 1, torch.minimum(some, last), last)
    if s["min_p"] is not None:
        last = torch.minimum(last, (w >= s["min_p"].double()[:, None]).sum(-1, keepdim=True).clamp(min=1))
    kept = mass.gather(1, last - 1)
    rank = torch.minimum((mass <= s["u"].double()[:, None] * kept).sum(-1, keepdim=True), last - 1)
    return {"tokens": order.gather(1, rank)[:, 0].int(), "logprob": (w.gather(1, rank) / kept).log().float()[:, 0]}


# ---- the definitions in 64 bits ---------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "rope":
        return _exact_rope(s, c)
    if c["op"] == "sample":
        got = {"tokens": torch.empty(c["rows"], dtype=torch.int32, device="cuda"),
               "logprob": torch.zeros(c["rows"], dtype=torch.float64, device="cuda")}
        for b in range(c["rows"]):
            _exact_row(s, b, got)
        return got
    got = {"out": torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")}
    if c["train"]:
        got["dq"] = torch.zeros_like(got["out"])
        got["dk"] = torch.zeros(s["k"].shape, dtype=torch.float64, device="cuda")
        got["dv"] = torch.zeros_like(got["dk"])
    else:
        got["lse"] = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    for b in range(c["batch"]):
        for h in range(c["q_heads"]):
            _exact_head(s, c, b, h, got)
    return got


def _exact_head(s, c, b, h, got):
    """One query head of one sequence."""
    t, e = slice(b * c["tokens"], (b + 1) * c["tokens"]), slice(b * c["states"], (b + 1) * c["states"])
    where, g = s["spans"].long()[t], h // (c["q_heads"] // c["kv_heads"])
    j = torch.arange(e.start, e.stop, device="cuda")
    hidden = (j < where[:, :1]) | (j >= where[:, 1:])
    blind = hidden.all(-1, keepdim=True)
    with torch.enable_grad():
        q, k, v = (x.double().requires_grad_(c["train"]) for x in (s["q"][t, h], s["k"][e, g], s["v"][e, g]))
        score = (q @ k.T / math.sqrt(c["dim"])).masked_fill(hidden, -math.inf)
        o = torch.softmax(score.masked_fill(blind, 0.0), -1).masked_fill(blind, 0.0) @ v
        if c["train"]:
            dq, dk, dv = torch.autograd.grad(o, (q, k, v), s["dout"][t, h].double())
            got["dq"][t, h] = dq
            got["dk"][e, g] += dk
            got["dv"][e, g] += dv
        else:
            got["lse"][t, h] = torch.logsumexp(score, -1)
    got["out"][t, h] = o.detach()


def _exact_rope(s, c):
    r, pos = c["rotary"], s["positions"].long()

    def turn(x):
        if not r:
            return x
        angle = torch.complex(s["cos"].double(), s["sin"].double())[pos][:, None]
        if c["interleaved"]:
            z = torch.view_as_complex(x[..., :r].unflatten(-1, (r // 2, 2)).contiguous()) * angle
            done = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(x[..., :r // 2], x[..., r // 2:r]) * angle
            done = torch.cat((z.real, z.imag), -1)
        return torch.cat((done, x[..., r:]), -1)

    def whole(x, w):
        return turn(x * w / torch.sqrt((x * x).sum(-1, keepdim=True) / c["dim"] + EPS))

    q, k = s["q"].double(), s["new_k"].double()
    wq, wk = s["q_norm"].double(), s["k_norm"].double()
    if c["what"] == "forward":
        return {"q": whole(q, wq), "k": whole(k, wk)} if c["kv_heads"] else {"q": whole(q, wq)}
    if c["what"] == "backward":
        with torch.enable_grad():
            leaves = [x.requires_grad_() for x in (q, k, wq, wk)]
            grads = torch.autograd.grad((whole(q, wq), whole(k, wk)), leaves, (s["dq"].double(), s["dk"].double()))
        return dict(zip(("dq", "dk", "dq_norm", "dk_norm"), grads))

    def store(cache, scale, new):
        old = cache.double() if scale is None else cache.double() * scale.double()[..., None]
        if scale is not None:
            step = new.abs().amax(-1, keepdim=True) / 127
            new = torch.where(step > 0, (new / step).round() * step, 0.0)
        old[s["table"].long()[s["rows"].long(), pos // c["page"]], pos % c["page"]] = new
        return old

    return {"q": whole(q, wq), "k": store(s["k"], s["k_scale"], whole(k, wk)),
            "v": store(s["v"], s["v_scale"], s["new_v"].double())}


def _exact_row(s, b, got):
    """One row, as probabilities: which ranks stay, and where u falls among them."""
    x = s["logits"][b].double()
    if not s["temperature"][b] > 0:
        got["tokens"][b] = (x == x.max()).nonzero()[0, 0]
        return
    p = torch.softmax(x / s["temperature"][b].double(), 0)
    order = torch.argsort(-x, stable=True)
    p = p[order]
    if s["top_k"] is not None and s["top_k"][b] > 0:
        p = p[:s["top_k"][b]]
    stays = torch.ones_like(p, dtype=torch.bool)
    if s["top_p"] is not None and s["top_p"][b] < 1:
        stays &= p.cumsum(0) - p < s["top_p"][b].double() * p.sum()
    if s["min_p"] is not None:
        stays &= p >= s["min_p"][b].double() * p[0]
    p = p[stays] / p[stays].sum()
    rank = torch.searchsorted(p.cumsum(0), s["u"][b].double(), right=True).clamp(max=p.numel() - 1)
    got["tokens"][b], got["logprob"][b] = order[rank], p[rank].log()
