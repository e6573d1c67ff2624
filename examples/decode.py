"""A small text decoder served with S3D8 linears and a paged key/value cache.

Random weights of the given sizes are cast to S3D8; prompts are read and continued
greedily, one token per sequence and step.  Each step runs, per layer: q, k and v
linears, rotary append into the cache, attention of the new token, the output
linear, the residual update fused with the MLP's norm and its int8 codes, gate, up
and down linears, and the residual update fused with the next layer's norm.  The
attention blocks are gated (through tanh), as cross-attention blocks of vision
decoders are.  Half way, every sequence is forked into two continuations, the first
ones are released, and the cache is compacted.

With --images, every second layer attends to the states of its sequence's image instead of
the text: their keys (each head normed) and values are made once, and forked sequences share
them.  --head-norms norms the heads of the other layers in front of their rotation.  With
--temperature the next tokens are drawn, from the --top-k first ones and the share --top-p.

    python examples/decode.py [--layers 4] [--steps 32] [--int8-cache] [--images 1601] ...
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import s3d8_a8_linear_gb300 as s3d8  # noqa: E402

BF = torch.bfloat16


def _linear(gen, n, k):
    """An S3D8 matrix [n, k]: packed bytes, table, channel scales."""
    w = (torch.randn((n, k), generator=gen, device="cuda") * k ** -0.5).to(BF)
    draws = torch.randint(-2 ** 31, 2 ** 31 - 1, (32,), dtype=torch.int32, device="cuda", generator=gen)
    _, table = s3d8.fit_centroids(w, draws, iters=4)
    packed, scale = s3d8.encode(w, table)
    return dict(packed=packed, centroids=table, chan_scale=scale, N=n)


class Decoder:
    def __init__(self, layers=2, hidden=512, heads=8, kv_heads=2, dim=64, mlp=1024, vocab=1000, seed=0,
                 images=False, head_norms=False):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        norm = lambda: (1 + 0.1 * torch.randn(hidden, generator=gen, device="cuda")).to(BF)  # noqa: E731
        self.embed = torch.randn((vocab, hidden), generator=gen, device="cuda").to(BF)
        self.layers = [dict(q=_linear(gen, heads * dim, hidden), k=_linear(gen, kv_heads * dim, hidden),
                            v=_linear(gen, kv_heads * dim, hidden), o=_linear(gen, hidden, heads * dim),
                            gate=_linear(gen, mlp, hidden), up=_linear(gen, mlp, hidden),
                            down=_linear(gen, hidden, mlp), attn_norm=norm(), mlp_norm=norm(),
                            attn_gate=torch.randn(1, generator=gen, device="cuda").add_(1).to(BF))
                       for _ in range(layers)]
        self.final_norm, self.head = norm(), _linear(gen, vocab, hidden)
        self.crossing = [bool(images) and i % 2 == 1 for i in range(layers)]     # layers that attend to an image
        for w, crosses in zip(self.layers, self.crossing):
            for name in ("q_norm", "k_norm"):
                w[name] = (1 + 0.1 * torch.randn(dim, generator=gen, device="cuda")).to(BF) \
                    if crosses or head_norms else None

    def look(self, states, ops=s3d8):
        """Keys and values of image states [S, hidden] for each layer that attends to them."""
        x = s3d8.quantize_act(states)
        made = []
        for w in (w for w, crosses in zip(self.layers, self.crossing) if crosses):
            k, v = (t.view(states.shape[0], -1, self.dim) for t in _project(x, w["k"], w["v"]))
            made.append((ops.norm_rope(k, q_norm=w["k_norm"])[0], v))
        return made

    def angles(self, length):
        freq = 10000.0 ** (-torch.arange(0, self.dim, 2, device="cuda") / self.dim)
        a = torch.arange(length, device="cuda")[:, None] * freq
        return a.cos(), a.sin()


def _project(x, *weights):
    """Several linears of one input (codes and scales); one launch for few tokens."""
    xq, xs = x
    if xq.shape[0] <= 4:
        return s3d8.linear_batch([dict(xq=xq, xscale=xs, **w) for w in weights], xq.shape[0])
    return [s3d8.linear(w["packed"], w["centroids"], w["chan_scale"], xq, xs, w["N"]) for w in weights]


def step(model, tokens, positions, rows, pool, table, lens, cos, sin, ops=s3d8, workspace=None, images=(), spans=None):
    """Logits of one new token per sequence, whose keys and values go to `positions`
    of the block table's `rows`; `lens` counts the tokens with the new one.  `images`:
    what look() made; `spans`: each token's states of them."""
    h = model.embed[tokens]
    n, norms = h.shape[0], [w["attn_norm"] for w in model.layers[1:]] + [model.final_norm]
    _, *x = ops.residual_norm_quant(h, w_pre=model.layers[0]["attn_norm"])
    caches, images = iter(pool.caches), iter(images)
    for w, crosses, next_norm in zip(model.layers, model.crossing, norms):
        if crosses:
            (q,) = _project(x, w["q"])
            q, _ = ops.norm_rope(q.view(n, -1, model.dim), q_norm=w["q_norm"])
            a = ops.cross_attention(q, *next(images), spans)
        else:
            q, k, v = _project(x, w["q"], w["k"], w["v"])
            q, k, v = (t.view(n, -1, model.dim) for t in (q, k, v))
            cache, normed = next(caches), {} if w["q_norm"] is None else dict(q_norm=w["q_norm"], k_norm=w["k_norm"])
            q = ops.rope_append(q, k, v, cos, sin, positions, cache, table, rows=rows, **normed)
            a = ops.paged_attention(q, cache, table[rows.long()], lens, workspace=workspace)
        (o,) = _project(s3d8.quantize_act(a.view(n, -1)), w["o"])
        h, *x = ops.residual_norm_quant(h, o, gate=w["attn_gate"], tanh_gate=True, w_pre=w["mlp_norm"])
        gate, up = _project(x, w["gate"], w["up"])
        act = (torch.nn.functional.silu(gate.float()) * up.float()).to(BF)
        (down,) = _project(s3d8.quantize_act(act), w["down"])
        h, *x = ops.residual_norm_quant(h, down, w_pre=next_norm)
    (logits,) = _project(x, model.head)
    return logits


class Server:
    """Sequences in rows of one block table over the caches of all layers that have one."""

    def __init__(self, model, pages=256, page=16, rows=16, width=16, dtype=BF):
        self.model, self.page = model, page
        self.pool = s3d8.KVPool([s3d8.KVCache.empty(pages, page, model.kv_heads, model.dim, dtype)
                                 for crosses in model.crossing if not crosses])
        self.images, self.spans = (), torch.zeros((rows, 2), dtype=torch.int32, device="cuda")
        self.table = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
        self.space = s3d8.pages_workspace(self.pool, rows)
        self.attention = s3d8.paged_attention_workspace(self.pool.caches[0], rows, model.heads)
        self.cos, self.sin = model.angles(width * page)

    def show(self, states, rows, spans, ops=s3d8):
        """The states [S, hidden] of all images, and the ones that each row's sequence sees."""
        self.images = self.model.look(states, ops)
        self.spans[rows.long()] = spans

    def feed(self, rows, tokens, ops=s3d8):
        """One more token in each row (int32); the logits behind them."""
        one = torch.ones_like(rows)
        got = s3d8.extend_pages(self.table, self.lens, self.refs, rows, one, self.page, workspace=self.space)
        lens = self.lens[rows.long()]
        # a sequence that found no page waits: a padding token, of an empty sequence
        positions = torch.where(got > 0, lens - 1, -1)
        return step(self.model, tokens, positions, rows, self.pool, self.table, torch.where(got > 0, lens, 0),
                    self.cos, self.sin, ops, self.attention, self.images, self.spans[rows.long()])

    def fork(self, parents, children):
        self.spans[children.long()] = self.spans[parents.long()]
        return s3d8.fork_pages(self.pool, self.table, self.lens, self.refs, parents, children, workspace=self.space)

    def free(self, rows):
        s3d8.free_pages(self.table, self.lens, self.refs, rows)

    def compact(self):
        return s3d8.compact_pages(self.pool, self.table, self.refs, workspace=self.space)


def serve(model, prompts, steps, dtype=BF, compact=True, ops=s3d8, states=None, spans=None, limits=None, seed=0, **sizes):
    """Read prompts [n, length], continue each for `steps` tokens; half way the
    sequences move to forked rows.  `states` [S, hidden] and `spans` [n, 2]: the images.
    `limits`: temperature, top_k, ... of sample(), [n] each; None takes the likeliest token.
    Returns the tokens and the last logits."""
    n = prompts.shape[0]
    server = Server(model, rows=2 * n, dtype=dtype, **sizes)
    rows = torch.arange(n, dtype=torch.int32, device="cuda")
    if states is not None:
        server.show(states, rows, spans, ops)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    for t in range(prompts.shape[1]):
        logits = server.feed(rows, prompts[:, t], ops)
    out = []
    for i in range(steps):
        if i == steps // 2:
            children = rows + n
            server.fork(rows, children)
            server.free(rows)
            if compact:
                server.compact()
            rows = children
        if limits is None:
            out.append(logits.float().argmax(-1))
        else:
            out.append(ops.sample(logits, torch.rand(n, generator=gen, device="cuda"), **limits).long())
        logits = server.feed(rows, out[-1], ops)
    return torch.stack(out, 1), logits


def main():
    p = argparse.ArgumentParser()
    for name, value in (("layers", 4), ("hidden", 4096), ("heads", 32), ("kv-heads", 8), ("dim", 128),
                        ("mlp", 14336), ("vocab", 32000), ("sequences", 4), ("prompt", 32), ("steps", 32)):
        p.add_argument("--" + name, type=int, default=value)
    p.add_argument("--int8-cache", action="store_true")
    p.add_argument("--images", type=int, default=0, metavar="STATES", help="one image of so many states a sequence")
    p.add_argument("--head-norms", action="store_true")
    p.add_argument("--temperature", type=float)
    p.add_argument("--top-k", type=int, default=0)
    p.add_argument("--top-p", type=float, default=1.0)
    a = p.parse_args()
    s3d8.load(build_if_missing=True)
    model = Decoder(a.layers, a.hidden, a.heads, a.kv_heads, a.dim, a.mlp, a.vocab,
                    images=a.images > 0, head_norms=a.head_norms)
    gen = torch.Generator(device="cuda").manual_seed(1)
    prompts = torch.randint(0, a.vocab, (a.sequences, a.prompt), device="cuda", generator=gen)
    dtype = torch.int8 if a.int8_cache else BF
    width = -(-(a.prompt + a.steps) // 16)
    more = dict(width=width)
    if a.images:
        first = torch.arange(a.sequences, dtype=torch.int32, device="cuda") * a.images
        more.update(states=torch.randn((a.sequences * a.images, a.hidden), generator=gen, device="cuda").to(BF),
                    spans=torch.stack((first, first + a.images), -1))
    if a.temperature is not None:
        each = lambda x, t: torch.full((a.sequences,), x, dtype=t, device="cuda")  # noqa: E731
        more["limits"] = dict(temperature=each(a.temperature, torch.float32), top_k=each(a.top_k, torch.int32),
                              top_p=each(a.top_p, torch.float32))
    serve(model, prompts, a.steps, dtype, **more)
    torch.cuda.synchronize()
    begin = time.perf_counter()
    tokens, _ = serve(model, prompts, a.steps, dtype, **more)
    torch.cuda.synchronize()
    took = time.perf_counter() - begin
    if s3d8.device_status() != 0:
        raise SystemExit("a kernel reported an error")
    print(f"{a.sequences} sequences, {a.prompt} + {a.steps} tokens, {a.layers} layers: "
          f"{took / (a.prompt + a.steps) * 1e3:.3f} ms a step; first continuation {tokens[0, :8].tolist()}")


if __name__ == "__main__":
    main()
