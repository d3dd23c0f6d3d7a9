"""Inputs that the kernel before rewrites in place, at batch sizes whose decode gives long contexts and the last ones to
clusters and the others to one CTA each: every call reads what was written just before it."""
import pytest
import torch

from tests import _gpu
from tests.test_gpu_cache_ops import Step, gen, pool16, randn, rows_pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("S,Hkv,long", [(100, 8, 3), (100, 8, 0), (128, 5, 2), (230, 4, 40), (31, 32, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_decode_rows_after_its_inputs_are_rewritten(S, Hkv, long, D):
    pa = _gpu.lib()
    g = gen(S + long + D)
    bs, Hq, NB, maxB = 16, 2 * Hkv, 300, 130
    k, v, ks, vs = (t.cuda() for t in rows_pool(g, NB, Hkv, bs, D))
    sets = []
    for _ in range(3):
        lens = torch.randint(0, 60, (S,), generator=g)
        lens[torch.randperm(S, generator=g)[:long]] = 2040
        bt = torch.randint(0, NB, (S, maxB), generator=g)
        sets.append([t.cuda() for t in (randn(g, S, Hq, D).bfloat16(), bt.to(torch.int32), lens.to(torch.int32))])
    scale = 0.1
    want = []
    for q, bt, cl in sets:
        out = torch.full_like(q, float("nan"))
        pa.decode_rows(out, q, k, v, ks, vs, bt, cl, scale)
        torch.cuda.synchronize()
        want.append(out)
    q, bt, cl = (torch.empty_like(t) for t in sets[0])
    outs = [torch.full_like(q, float("nan")) for _ in range(30)]
    for i, out in enumerate(outs):
        for t, new in zip((q, bt, cl), sets[i % 3]):
            t.copy_(new)
        pa.decode_rows(out, q, k, v, ks, vs, bt, cl, scale)
    assert all(torch.equal(out, want[i % 3]) for i, out in enumerate(outs))
    # from a graph, whose replays rewrite them
    graph, i = torch.cuda.CUDAGraph(), torch.zeros(1, dtype=torch.int64, device="cuda")
    stacks = [torch.stack(x) for x in zip(*sets)]
    out = torch.full_like(q, float("nan"))
    with torch.cuda.graph(graph):
        for t, stack in zip((q, bt, cl), stacks):
            t.copy_(stack.index_select(0, i)[0])
        pa.decode_rows(out, q, k, v, ks, vs, bt, cl, scale)
    for n in (2, 0, 1, 1, 2):
        i.fill_(n)
        graph.replay()
        assert torch.equal(out, want[n])
    assert pa.get_device_error() == 0


@pytest.mark.parametrize("S,Hkv,Hq,D", [(64, 8, 32, 128), (160, 3, 3, 64), (62, 8, 16, 64)])
def test_decode_selected_after_its_tables_are_rewritten(S, Hkv, Hq, D):
    """The selection itself is the kernel before."""
    pa = _gpu.lib()
    g = gen(S + D)
    bs, n, NB, L = 16, 40, 200, 16 * 120
    k, v = (pool16(g, NB, Hkv, bs, D, "bf16", "bf16").cuda() for _ in range(2))
    bt = torch.randint(0, NB, (S, L // bs), generator=g).to(torch.int32).cuda()
    cl = torch.full((S,), L, dtype=torch.int32).cuda()
    sets = [(randn(g, S, Hkv, L // bs).cuda(), randn(g, S, Hq, D).bfloat16().cuda()) for _ in range(3)]
    tables, lens = torch.zeros((S, Hkv, n), dtype=torch.int32).cuda(), torch.zeros((S, Hkv), dtype=torch.int32).cuda()
    q = torch.empty_like(sets[0][1])

    def step(i, out, wait):
        q.copy_(sets[i][1])
        pa.select_blocks(tables, lens, sets[i][0], bt, cl, bs)
        if wait:
            torch.cuda.synchronize()
        pa.decode_selected(out, q, k, v, tables, lens, 0.1)
        return out

    want = [step(i, torch.empty_like(q), True) for i in range(3)]
    outs = [step(i % 3, torch.full_like(q, float("nan")), False) for i in range(30)]
    assert all(torch.equal(out, want[i % 3]) for i, out in enumerate(outs))
    assert pa.get_device_error() == 0


def test_the_step_of_a_batch_that_takes_clusters_at_its_end():
    """All the operators of a decode step one after another, 480 contexts of chosen blocks, against the same with a
    wait after each."""
    pa = _gpu.lib()
    lens = [int(x) for x in torch.randint(1, 1500, (240,), generator=gen(5))]
    a, b = Step(pa, gen(7), lens, n=40, P=0), Step(pa, gen(7), lens, n=40, P=0)

    class Waiting:
        def __getattr__(self, name):
            def call(*args, **kwargs):
                getattr(pa, name)(*args, **kwargs)
                torch.cuda.synchronize()
            return call

    b.pa = Waiting()
    for seed in range(5):
        new = randn(gen(seed), *a.qkv.shape).bfloat16().cuda()
        a.qkv.copy_(new)
        b.qkv.copy_(new)
        a.run()
        b.run()
        for x in ("out", "q_out", "k", "v", "bounds", "scores", "tables", "lens"):
            assert torch.equal(getattr(a, x), getattr(b, x)), x
    assert pa.get_device_error() == 0
