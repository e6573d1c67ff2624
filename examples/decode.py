"""A small text decoder served with S3D8 linears and a paged key/value cache.

Random weights of the given sizes are cast to S3D8; prompts are read and continued
greedily, one token per sequence and step.  Each step runs, per layer: q, k and v
linears, rotary append into the cache, attention of the new token, the output
linear, the residual update fused with the MLP's norm and its int8 codes, gate, up
and down linears, and the residual update fused with the next layer's norm.  The
attention blocks are gated (through tanh), as cross-attention blocks of vision
decoders are.  Half way, every sequence is forked into two continuations, the first
ones are released, and the cache is compacted.

    python examples/decode.py [--layers 4] [--steps 32] [--int8-cache] ...
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
    def __init__(self, layers=2, hidden=512, heads=8, kv_heads=2, dim=64, mlp=1024, vocab=1000, seed=0):
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


def step(model, tokens, positions, rows, pool, table, lens, cos, sin, ops=s3d8, workspace=None):
    """Logits of one new token per sequence, whose keys and values go to `positions`
    of the block table's `rows`; `lens` counts the tokens with the new one."""
    h = model.embed[tokens]
    n, norms = h.shape[0], [w["attn_norm"] for w in model.layers[1:]] + [model.final_norm]
    _, *x = ops.residual_norm_quant(h, w_pre=model.layers[0]["attn_norm"])
    for w, cache, next_norm in zip(model.layers, pool.caches, norms):
        q, k, v = _project(x, w["q"], w["k"], w["v"])
        q, k, v = (t.view(n, -1, model.dim) for t in (q, k, v))
        q = ops.rope_append(q, k, v, cos, sin, positions, cache, table, rows=rows)
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
    """Sequences in rows of one block table over the caches of all layers."""

    def __init__(self, model, pages=256, page=16, rows=16, width=16, dtype=BF):
        self.model, self.page = model, page
        self.pool = s3d8.KVPool([s3d8.KVCache.empty(pages, page, model.kv_heads, model.dim, dtype)
                                 for _ in model.layers])
        self.table = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
        self.space = s3d8.pages_workspace(self.pool, rows)
        self.attention = s3d8.paged_attention_workspace(self.pool.caches[0], rows, model.heads)
        self.cos, self.sin = model.angles(width * page)

    def feed(self, rows, tokens, ops=s3d8):
        """One more token in each row (int32); the logits behind them."""
        one = torch.ones_like(rows)
        got = s3d8.extend_pages(self.table, self.lens, self.refs, rows, one, self.page, workspace=self.space)
        lens = self.lens[rows.long()]
        # a sequence that found no page waits: a padding token, of an empty sequence
        positions = torch.where(got > 0, lens - 1, -1)
        return step(self.model, tokens, positions, rows, self.pool, self.table, torch.where(got > 0, lens, 0),
                    self.cos, self.sin, ops, self.attention)

    def fork(self, parents, children):
        return s3d8.fork_pages(self.pool, self.table, self.lens, self.refs, parents, children, workspace=self.space)

    def free(self, rows):
        s3d8.free_pages(self.table, self.lens, self.refs, rows)

    def compact(self):
        return s3d8.compact_pages(self.pool, self.table, self.refs, workspace=self.space)


def serve(model, prompts, steps, dtype=BF, compact=True, ops=s3d8, **sizes):
    """Read prompts [n, length], continue each for `steps` tokens; half way the
    sequences move to forked rows.  Returns the tokens and the last logits."""
    n = prompts.shape[0]
    server = Server(model, rows=2 * n, dtype=dtype, **sizes)
    rows = torch.arange(n, dtype=torch.int32, device="cuda")
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
        out.append(logits.float().argmax(-1))
        logits = server.feed(rows, out[-1], ops)
    return torch.stack(out, 1), logits


def main():
    p = argparse.ArgumentParser()
    for name, value in (("layers", 4), ("hidden", 4096), ("heads", 32), ("kv-heads", 8), ("dim", 128),
                        ("mlp", 14336), ("vocab", 32000), ("sequences", 4), ("prompt", 32), ("steps", 32)):
        p.add_argument("--" + name, type=int, default=value)
    p.add_argument("--int8-cache", action="store_true")
    a = p.parse_args()
    s3d8.load(build_if_missing=True)
    model = Decoder(a.layers, a.hidden, a.heads, a.kv_heads, a.dim, a.mlp, a.vocab)
    gen = torch.Generator(device="cuda").manual_seed(1)
    prompts = torch.randint(0, a.vocab, (a.sequences, a.prompt), device="cuda", generator=gen)
    dtype = torch.int8 if a.int8_cache else BF
    width = -(-(a.prompt + a.steps) // 16)
    serve(model, prompts, a.steps, dtype, width=width)
    torch.cuda.synchronize()
    begin = time.perf_counter()
    tokens, _ = serve(model, prompts, a.steps, dtype, width=width)
    torch.cuda.synchronize()
    took = time.perf_counter() - begin
    if s3d8.device_status() != 0:
        raise SystemExit("a kernel reported an error")
    print(f"{a.sequences} sequences, {a.prompt} + {a.steps} tokens, {a.layers} layers: "
          f"{took / (a.prompt + a.steps) * 1e3:.3f} ms a step; first continuation {tokens[0, :8].tolist()}")


if __name__ == "__main__":
    main()
