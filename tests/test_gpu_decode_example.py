"""The serving example end to end: the same decoder with its norms, rotary append and
attention replaced by plain ones on dense tensors, and the invariance of its results
under compaction.

The plain operators differ from the kernels in the order of fp32 sums, so a bf16
value may round the other way (2^-8) and an int8 code may move by one step (1/127 of
a row's maximum); with two layers the logits agree to 5% of their norm.
"""
import importlib.util
import os

import pytest
import torch

import s3d8_a8_linear_gb300 as s3d8

pytestmark = pytest.mark.gpu

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


class PlainOps:
    """The operators of a decode step with elementary operations, token by token."""

    @staticmethod
    def residual_norm_quant(h, y=None, gate=None, w_pre=None, tanh_gate=False):
        h = h if y is None else (h.float() + (1.0 if gate is None else gate.float().tanh()) * y.float()).to(torch.bfloat16)
        f = h.float()
        x = (f * (f.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * w_pre.float()).to(torch.bfloat16)
        return h, *s3d8.quantize_act(x)

    @staticmethod
    def rope_append(q, k, v, cos, sin, positions, cache, table, rows):
        at = positions.long()
        c, s = cos[at][:, None], sin[at][:, None]

        def turn(x):
            a, b = x.float().chunk(2, -1)
            return torch.cat((a * c - b * s, b * c + a * s), -1)

        page = table[rows.long(), at // cache.page_size].long()
        for store, scale, new in ((cache.k, cache.k_scale, turn(k)), (cache.v, cache.v_scale, v.float())):
            if scale is not None:
                step = new.abs().amax(-1) / 127
                scale[page, at % cache.page_size] = step
                new = (new / step[..., None]).round()
            store[page, at % cache.page_size] = new.to(store.dtype)
        return turn(q).to(torch.bfloat16)

    @staticmethod
    def paged_attention(q, cache, table, lens, workspace=None):
        out = torch.empty_like(q)
        for b in range(q.shape[0]):
            pos = torch.arange(int(lens[b]), device=q.device)
            at = table[b].long()[pos // cache.page_size], pos % cache.page_size
            k, v = cache.k[at].float(), cache.v[at].float()
            if cache.k_scale is not None:
                k, v = k * cache.k_scale[at][..., None], v * cache.v_scale[at][..., None]
            groups = q.shape[1] // k.shape[1]
            k, v = (t.repeat_interleave(groups, 1) for t in (k, v))
            p = torch.softmax(torch.einsum("hd,nhd->hn", q[b].float(), k) * q.shape[2] ** -0.5, -1)
            out[b] = torch.einsum("hn,nhd->hd", p, v)
        return out


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.int8])
@pytest.mark.parametrize("sequences", [1, 3, 7])
def test_example_against_plain_operators(example, sequences, dtype):
    model = example.Decoder(layers=2, seed=sequences)
    gen = torch.Generator(device="cuda").manual_seed(5)
    prompts = torch.randint(0, 1000, (sequences, 21), device="cuda", generator=gen)
    rows = torch.arange(sequences, dtype=torch.int32, device="cuda")
    servers = [example.Server(model, rows=sequences, dtype=dtype) for _ in range(2)]
    for t in range(prompts.shape[1]):      # the same tokens for both: a sampled one could differ by a near-tie
        got, want = (s.feed(rows, prompts[:, t], ops).float() for s, ops in zip(servers, (s3d8, PlainOps)))
        assert float((got - want).norm() / want.norm()) < 0.05, t


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.int8])
def test_compaction_changes_nothing(example, dtype):
    model = example.Decoder(layers=2)
    gen = torch.Generator(device="cuda").manual_seed(6)
    prompts = torch.randint(0, 1000, (5, 40), device="cuda", generator=gen)
    moved = example.serve(model, prompts, 30, dtype, page=8)
    stayed = example.serve(model, prompts, 30, dtype, page=8, compact=False)
    assert all(torch.equal(a, b) for a, b in zip(moved, stayed))


def test_sequences_without_pages_wait(example):
    """Six pages for four sequences: those that find none get an empty step, and the
    others' results do not change."""
    model = example.Decoder(layers=2)
    rows = torch.arange(4, dtype=torch.int32, device="cuda")
    tokens = torch.tensor([1, 2, 3, 4], device="cuda")
    small = example.Server(model, pages=6, page=4, rows=4, width=4)
    large = example.Server(model, pages=64, page=4, rows=4, width=4)
    for i in range(6):
        a, b = small.feed(rows, tokens), large.feed(rows, tokens)
        fed = 4 if i < 4 else 2
        assert small.lens.tolist() == [i + 1] * fed + [4] * (4 - fed)
        assert torch.equal(a[:fed], b[:fed])
    small.free(rows[:2].contiguous())
    assert int((small.refs != 0).sum()) == 2
