"""The calls between two linears in CUDA graphs, on two streams and from two threads at
once, each with a workspace of its own; and scores that are not finite."""
import threading

import pytest
import torch

import s3d8_a8_linear_gb300 as s3d8
from gpu_util import dev
from test_gpu_kv_cache import BF, I32, _cache, _fill, _i32, _lib, _parts, _pool, _rand  # noqa: F401

pytestmark = pytest.mark.gpu


def _graph(call):
    """`call` once as it is (first calls set kernels up), then captured."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    return graph, got


@pytest.mark.parametrize("int8", [False, True])
def test_a_decode_step_in_a_graph(int8):
    """Append, attention and norm captured once and replayed with other tokens and lengths, with
    kept workspaces and with ones allocated in the graph."""
    g = torch.Generator().manual_seed(1)
    lens0 = [700, 3, 0, 40, 9001]
    B, width = len(lens0), 600
    cache = _cache(900, 16, 2, 128, int8, "head")
    table, _ = _fill(cache, g, lens0, width, 16)
    spare = iter(sorted(set(range(900)) - set(table.flatten().tolist())))
    for b, n in enumerate(lens0):          # room for three more tokens
        for col in (n // 16, n // 16 + 1):
            if table[b, col] < 0:
                table[b, col] = next(spare)
    q, k, v, h = _rand(g, B, 8, 128), _rand(g, B, 2, 128), _rand(g, B, 2, 128), _rand(g, B, 1024)
    w = _rand(g, 1024)
    angle = torch.rand((10000, 64), generator=g) * 6
    cos, sin = angle.cos().to(dev()), angle.sin().to(dev())
    lens = _i32(lens0)
    pos = lens.clone()
    kept = s3d8.paged_attention_workspace(cache, B, 8)

    def step(ws):
        turned = s3d8.rope_append(q, k, v, cos, sin, pos, cache, table)
        a = s3d8.paged_attention(turned, cache, table, lens, workspace=ws)
        return turned, a, *s3d8.residual_norm_quant(h, a.view(B, -1), w_pre=w)

    for ws in (kept, None):
        lens.copy_(_i32([n + 1 for n in lens0]))
        pos.copy_(_i32(lens0))
        graph, got = _graph(lambda: step(ws))
        for more in range(3):
            for t in (q, k, v, h):
                t.copy_(_rand(g, *t.shape))
            pos.copy_(_i32([n + more for n in lens0]))
            lens.copy_(pos + 1)
            graph.replay()
            mine = [t.clone() for t in got]
            for one, want in zip(mine, step(kept)):
                assert torch.equal(one, want)


def test_page_calls_and_gradients_in_graphs():
    pool = _pool(2, 40, 8, 2, 64, False, "head", 1)
    rows, width = 6, 5
    first = (torch.full((rows, width), -1, dtype=I32, device=dev()), torch.zeros(rows, dtype=I32, device=dev()),
             torch.zeros(40, dtype=I32, device=dev()))
    table, lens, refs = (t.clone() for t in first)
    space = s3d8.pages_workspace(pool, rows)
    contents = [t.clone() for t in _parts(pool)]
    grown, parents, children, old = _i32([4, 1]), _i32([1, 4]), _i32([0, 2]), _i32([1])

    def life():
        for t, was in zip((table, lens, refs), first):
            t.copy_(was)
        for t, was in zip(_parts(pool), contents):
            t.copy_(was)
        a = s3d8.extend_pages(table, lens, refs, grown, _i32_graph, 8, workspace=space)
        b = s3d8.fork_pages(pool, table, lens, refs, parents, children, workspace=space)
        s3d8.free_pages(table, lens, refs, old)
        return a, b, s3d8.compact_pages(pool, table, refs, workspace=space)

    _i32_graph = _i32([19, 30])
    graph, got = _graph(life)
    for add in ([19, 30], [8, 16], [1, 40]):
        _i32_graph.copy_(_i32(add))
        graph.replay()
        mine = [t.clone() for t in (*got, table, lens, refs, *_parts(pool))]
        for one, want in zip(mine, (*life(), table, lens, refs, *_parts(pool))):
            assert torch.equal(one, want)

    g = torch.Generator().manual_seed(3)
    h, y, dh, dx = (_rand(g, 300, 2048) for _ in range(4))
    w = _rand(g, 2048)
    keep = s3d8.residual_norm_backward_workspace(300, 2048)
    graph, got = _graph(lambda: s3d8.residual_norm_backward(dh, dx, h, y, w, w_pre=w, workspace=keep))
    for t in (h, y, dh, dx):
        t.copy_(_rand(g, *t.shape))
    graph.replay()
    mine = {k: t.clone() for k, t in got.items()}
    for k, want in s3d8.residual_norm_backward(dh, dx, h, y, w, w_pre=w).items():
        assert torch.equal(mine[k], want), k


@pytest.mark.parametrize("threads", [False, True])
def test_two_streams_with_workspaces_of_their_own(threads):
    """Calls of unlike lengths on two streams, queued turn by turn or by two threads."""
    g = torch.Generator().manual_seed(8)
    lens = ([30000, 5, 900], [77, 12000] * 8)
    work = []
    for n in lens:
        cache = _cache(sum(-(-x // 16) for x in n) + 1, 16, 4, 128, len(work) == 1, "head")
        table, _ = _fill(cache, g, n, max(n) // 16 + 1, 16)
        q = _rand(g, len(n), 16, 128)
        space = s3d8.paged_attention_workspace(cache, len(n), 16)
        space.fill_(171)
        want = s3d8.paged_attention(q, cache, table, _i32(n))
        work.append((cache, table, q, _i32(n), space, want, torch.cuda.Stream(), []))
    torch.cuda.synchronize()

    def call(w):
        with torch.cuda.stream(w[6]):
            w[7].append(s3d8.paged_attention(w[2], w[0], w[1], w[3], workspace=w[4]))

    if threads:
        both = [threading.Thread(target=lambda w=w: [call(w) for _ in range(30)]) for w in work]
        for t in both:
            t.start()
        for t in both:
            t.join()
    else:
        for _ in range(30):
            for w in work:
                call(w)
    torch.cuda.synchronize()
    for w in work:
        assert len(w[7]) == 30 and all(torch.equal(out, w[5]) for out in w[7])


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("n", [40, 9000])
def test_scores_that_are_not_finite(n, int8):
    """As the definition has it: a score of +inf or NaN makes its query's row NaN, one of -inf among
    finite ones is a weight of 0, and nothing but scores of -inf gives zeros and lse = -inf."""
    g = torch.Generator().manual_seed(n)
    cache = _cache(n // 16 + 2, 16, 1, 64, int8, "head")
    table, _ = _fill(cache, g, [n], n // 16 + 1, 16)
    page, slot = table[0, 1].long(), 5                    # token 21
    q = _rand(g, 1, 4, 64)
    q[0, :, 0] = torch.tensor([1.0, -1.0, 1.0, -1.0], device=dev()).to(BF)
    at = cache.k_scale if int8 else cache.k
    if int8:
        cache.k[page, slot, 0] = 0
        cache.k[page, slot, 0, 0] = 127
        at[page, slot, 0] = float("inf")                  # scores 127 inf and -127 inf
    else:
        at[page, slot, 0] = 0
        at[page, slot, 0, 0] = float("inf")
        q[0, :, 1:] = q[0, :, 1:].abs()                   # 0 times them stays 0
    lse = torch.empty((1, 4), device=dev())
    out = s3d8.paged_attention(q, cache, table, _i32([n]), lse=lse)
    assert bool(torch.isnan(out[0, ::2]).all()) and bool(torch.isnan(lse[0, ::2]).all())
    assert bool(torch.isfinite(out[0, 1::2]).all()) and bool(torch.isfinite(lse[0, 1::2]).all())
    cache.k[..., 0] = 127 if int8 else float("inf")       # every token's score is +inf or -inf
    if int8:
        cache.k[..., 1:] = 0
        at.fill_(float("inf"))
    out = s3d8.paged_attention(q, cache, table, _i32([n]), lse=lse)
    assert bool(torch.isnan(out[0, ::2]).all()) and bool(torch.isnan(lse[0, ::2]).all())
    assert bool((out[0, 1::2] == 0).all()) and bool((lse[0, 1::2] == -float("inf")).all())
