"""The vision decoder's operators as they are used: a serving run through the example
(states looked at once, normed heads, cross attention, drawn tokens, forks) against plain
operators, a training step through three operators against the same in 64 bits, and runs
that are captured, on other streams and side by side.

Serving: the plain operators differ from the kernels in the order of fp32 sums, so a bf16
value may round the other way (2^-8) and an int8 code may move by one step (1/127 of a row's
maximum); with four layers the logits agree to 5% of their norm.  Drawn tokens are compared
on the kernels' own logits.

Training: each operator rounds its outputs to bf16 (2^-8 of a value, forward and backward),
and the weights of the attention once more; a gradient passes at most eight such roundings
(residual, two products of the attention with their rounded operands, norm), each 2^-9 on
average over a tensor's norm: 8 * 2^-9 = 2^-6 bounds their sum.
"""
import importlib.util
import os
import threading

import numpy as np
import pytest
import torch

import s3d8_a8_linear_gb300 as s3d8
from test_gpu_decode_example import PlainOps

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    s3d8.load(build_if_missing=True)
    torch.cuda.set_device(0)
    spec = importlib.util.spec_from_file_location("decode_example", os.path.join(ROOT, "examples", "decode.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    yield module
    assert s3d8.device_status() == 0


def _normed(x, w):
    f = x.float()
    return f * (f.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * w.float()


class PlainVision(PlainOps):
    @staticmethod
    def norm_rope(x, q_norm):
        return _normed(x, q_norm).to(BF), None

    @staticmethod
    def rope_append(q, k, v, cos, sin, positions, cache, table, rows, q_norm=None, k_norm=None):
        if q_norm is not None:
            q, k = _normed(q, q_norm), _normed(k, k_norm)
        return PlainOps.rope_append(q, k, v, cos, sin, positions, cache, table, rows)

    @staticmethod
    def cross_attention(q, k, v, spans):
        out = torch.zeros_like(q)
        for t, (a, b) in enumerate(spans.tolist()):
            if a >= b:
                continue
            keys, values = (x[a:b].float().repeat_interleave(q.shape[1] // x.shape[1], 1) for x in (k, v))
            p = torch.softmax(torch.einsum("hd,nhd->hn", q[t].float(), keys) * q.shape[2] ** -0.5, -1)
            out[t] = torch.einsum("hn,nhd->hd", p, values)
        return out


def _images(sequences, gen, hidden=512):
    """Ragged images, one behind the other; the last sequence has none."""
    sizes = [100 + 77 * i for i in range(sequences)]
    ends = np.cumsum(sizes)
    spans = torch.tensor([[e - n, e] for n, e in zip(sizes, ends)], dtype=torch.int32, device="cuda")
    spans[-1] = 0
    return torch.randn((int(ends[-1]), hidden), generator=gen, device="cuda").to(BF), spans


@pytest.mark.parametrize("dtype", [BF, torch.int8])
@pytest.mark.parametrize("sequences", [1, 3, 7])
def test_example_with_images_against_plain_operators(example, sequences, dtype):
    model = example.Decoder(layers=4, seed=sequences, images=True, head_norms=True)
    gen = torch.Generator(device="cuda").manual_seed(5)
    prompts = torch.randint(0, 1000, (sequences, 9), device="cuda", generator=gen)
    states, spans = _images(sequences + 1, gen)
    spans = spans[-sequences:].contiguous()
    rows = torch.arange(sequences, dtype=torch.int32, device="cuda")
    servers = [example.Server(model, rows=2 * sequences, dtype=dtype) for _ in range(2)]
    for s, ops in zip(servers, (s3d8, PlainVision)):
        s.show(states, rows, spans, ops)
    for t in range(prompts.shape[1]):
        if t == 5:              # forked sequences see their parents' images
            for s in servers:
                s.fork(rows, rows + sequences)
                s.free(rows)
            rows = rows + sequences
        got, want = (s.feed(rows, prompts[:, t], ops).float() for s, ops in zip(servers, (s3d8, PlainVision)))
        assert float((got - want).norm() / want.norm()) < 0.05, t


def test_drawn_continuations(example):
    """Tokens drawn inside serve() are those of the definition on the logits there, and
    compaction changes nothing."""
    model = example.Decoder(layers=2, images=True)
    gen = torch.Generator(device="cuda").manual_seed(6)
    n = 5
    prompts = torch.randint(0, 1000, (n, 4), device="cuda", generator=gen)
    states, spans = _images(n, gen)
    limits = dict(temperature=torch.tensor([0.0, 0.5, 1.0, 1.5, 0.8], device="cuda"),
                  top_k=torch.tensor([0, 40, 0, 7, 1], dtype=torch.int32, device="cuda"),
                  top_p=torch.tensor([1.0, 0.9, 0.6, 1.0, 1.0], device="cuda"))
    drawn = []

    class Recorded:
        def __getattr__(self, name):
            return getattr(s3d8, name)

        @staticmethod
        def sample(logits, u, **more):
            drawn.append((logits.clone(), u.clone(), s3d8.sample(logits, u, **more)))
            return drawn[-1][2]

    more = dict(states=states, spans=spans, limits=limits, page=8)
    moved = example.serve(model, prompts, 12, ops=Recorded(), **more)
    stayed = example.serve(model, prompts, 12, compact=False, **more)
    assert all(torch.equal(a, b) for a, b in zip(moved, stayed))
    from test_gpu_sample import _one
    assert len(drawn) == 12
    for i, (logits, u, tokens) in enumerate(drawn):
        assert torch.equal(moved[0][:, i], tokens.long())
        x = logits.float().cpu().numpy().astype(np.float64)
        for b in range(n):
            want, _ = _one(x[b], float(u[b]), float(limits["temperature"][b]), int(limits["top_k"][b]), float(limits["top_p"][b]))
            assert int(tokens[b]) == want, (i, b)
    assert bool((moved[0][4] == torch.stack([d[0][4].float().argmax() for d in drawn])).all())


# ---- a training step --------------------------------------------------------


def _problem(T, S, heads, kv_heads, dim, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def leaf(*shape, mean=0.0, scale=1.0):
        return (mean + scale * torch.randn(shape, generator=gen, device="cuda")).to(BF).requires_grad_()

    hidden = heads * dim
    p = dict(h=leaf(T, hidden), q=leaf(T, heads, dim), k=leaf(S, kv_heads, dim), v=leaf(S, kv_heads, dim),
             q_norm=leaf(dim, mean=1.0, scale=0.1), k_norm=leaf(dim, mean=1.0, scale=0.1), gate=leaf(1),
             w=leaf(hidden, mean=1.0, scale=0.1))
    lo = torch.arange(T, device="cuda") * 2 // T * (S // 2)
    spans = torch.stack((lo, lo + S // 2), -1).int()
    spans[:3] = 0               # text in front of the first image
    dh, dx = (torch.randn((T, hidden), generator=gen, device="cuda").to(BF) for _ in range(2))
    return p, spans, dh, dx


def _step(p, spans):
    q, _ = s3d8.NormRope.apply(p["q"], None, p["q_norm"])
    k, _ = s3d8.NormRope.apply(p["k"], None, p["k_norm"])
    a = s3d8.CrossAttention.apply(q, k, p["v"], spans)
    return s3d8.ResidualNorm.apply(p["h"], a.view(p["h"].shape), None, p["gate"], p["w"], 1.0, 1e-5, True)


def _plain_step(p, spans):
    def norm(x, w):
        return x * (x.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * w

    q, k = norm(p["q"], p["q_norm"]), norm(p["k"], p["k_norm"])
    group = q.shape[1] // k.shape[1]
    j = torch.arange(k.shape[0], device="cuda")
    seen = (j >= spans[:, :1]) & (j < spans[:, 1:])
    s = torch.einsum("thd,shd->hts", q, k.repeat_interleave(group, 1)) * q.shape[2] ** -0.5
    some = seen.any(-1)
    w = torch.softmax(torch.where(seen | ~some[:, None], s, -torch.inf), -1) * some[:, None]
    a = torch.einsum("hts,shd->thd", w, p["v"].repeat_interleave(group, 1))
    h = p["h"] + p["gate"].tanh() * a.reshape(p["h"].shape)
    return h, norm(h, p["w"])


@pytest.mark.parametrize("T,S,heads,kv_heads,dim", [(37, 150, 4, 4, 64), (300, 514, 8, 2, 128), (129, 1601, 4, 1, 80)])
def test_a_training_step(example, T, S, heads, kv_heads, dim):
    p, spans, dh, dx = _problem(T, S, heads, kv_heads, dim)
    h, x = _step(p, spans)
    got = torch.autograd.grad((h, x), list(p.values()), (dh, dx))
    exact = {n: t.detach().double().requires_grad_() for n, t in p.items()}
    H, X = _plain_step(exact, spans)
    want = torch.autograd.grad((H, X), list(exact.values()), (dh.double(), dx.double()))
    for n, a, b in zip(("h", "x", *p), (h, x, *got), (H, X, *want)):
        a, b = a.detach().double(), b.detach()
        if n == "gate":         # one number, a sum of T * hidden products of random signs
            size = float((dh.double().norm() + dx.double().norm()) * 2)
            assert abs(float(a - b)) <= 2.0 ** -6 * size, n
            continue
        assert float((a - b).norm() / b.norm()) <= 2.0 ** -6, n


# ---- captured, on other streams, side by side -------------------------------


def _run(p, spans, limits, spaces):
    """What a decode step does with the operators, into tensors of its own."""
    q, _ = s3d8.norm_rope(p["q"], q_norm=p["q_norm"])
    a = s3d8.cross_attention(q, p["k"], p["v"], spans, workspace=spaces[0])
    tokens = s3d8.sample(a.view(a.shape[0], -1), limits["u"], limits["temperature"])
    g = s3d8.cross_attention_backward(a, q, p["k"], p["v"], a, torch.zeros(a.shape[:2], device="cuda"), spans,
                                      workspace=spaces[1])
    b = s3d8.norm_rope_backward(g["dq"], None, p["q"], q_norm=p["q_norm"])
    return a, tokens, g["dk"], g["dv"], b["dq"], b["dq_norm"]


def _inputs(seed):
    p, spans, _, _ = _problem(70, 700, 8, 2, 128, seed)
    p = {n: t.detach() for n, t in p.items()}
    gen = torch.Generator(device="cuda").manual_seed(seed)
    limits = dict(u=torch.rand(70, generator=gen, device="cuda"), temperature=torch.full((70,), 0.7, device="cuda"))
    size = (70, 700, 8, 2, 128)
    return p, spans, limits, (s3d8.cross_attention_workspace(*size), s3d8.cross_attention_backward_workspace(*size))


def test_captured_and_replayed(example):
    mine, other = _inputs(1), _inputs(2)
    want = [[t.clone() for t in _run(*i)] for i in (mine, other)]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        _run(*mine)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        got = _run(*mine)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    for a, b in zip((*mine[0].values(), mine[1], *mine[2].values()), (*other[0].values(), other[1], *other[2].values())):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[1]))


def test_side_by_side(example):
    """Two streams, and two threads of them: each has its inputs and workspaces."""
    inputs = [_inputs(3), _inputs(4)]
    want = [[t.clone() for t in _run(*i)] for i in inputs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in inputs]
    got = [[], []]

    def work(i):
        with torch.cuda.stream(streams[i]):
            for _ in range(10):
                got[i].append(_run(*inputs[i]))

    for i in range(2):
        work(i)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in range(2):
        assert len(got[i]) == 20
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))


def test_backward_captured(example):
    """The gradients of a step captured on another stream, replayed for other inputs.  (No
    eager graph of the same leaves may be alive: autograd would join its stream to the
    captured one.)"""
    (p, spans, dh, dx), (other, _, dh2, dx2) = (_problem(64, 256, 4, 2, 64, seed) for seed in (5, 6))
    leaves = list(p.values())
    want = [torch.autograd.grad(_step(i, spans), list(i.values()), d) for i, d in ((p, (dh, dx)), (other, (dh2, dx2)))]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        torch.autograd.grad(_step(p, spans), leaves, (dh, dx))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        got = torch.autograd.grad(_step(p, spans), leaves, (dh, dx))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    with torch.no_grad():
        for n, t in p.items():
            t.copy_(other[n])
        dh.copy_(dh2), dx.copy_(dx2)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[1]))
