"""Calls of one kernel with different shared-memory sizes from two host threads at once: none is refused, and each
gives what it gives alone."""
import threading

import pytest
import torch

from tests import _gpu
from tests import _ref64 as R
from tests.test_gpu_cache_ops import gen, randn

pytestmark = pytest.mark.gpu


def run_together(works, times):
    """Each of `works` is called `times` times on a stream and in a thread of its own; their exceptions are raised."""
    errors, start = [], threading.Barrier(len(works))
    streams = [torch.cuda.Stream() for _ in works]
    torch.cuda.synchronize()

    def loop(work, stream):
        try:
            with torch.cuda.stream(stream):
                start.wait()
                for _ in range(times):
                    work()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=loop, args=a) for a in zip(works, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    if errors:
        raise errors[0]


def test_selections_of_many_blocks():
    pa = _gpu.lib()
    g = gen(1)
    bs, n, calls = 8, 40, []
    for blocks in (17000, 50000):  # keys in shared memory: 68 KB and 200 KB
        scores = randn(g, 1, 1, blocks)
        bt = torch.arange(blocks, dtype=torch.int32)[None]
        tables, lens = torch.zeros((1, 1, n), dtype=torch.int32).cuda(), torch.zeros((1, 1), dtype=torch.int32).cuda()
        args = (tables, lens, scores.cuda(), bt.cuda(), torch.tensor([blocks * bs], dtype=torch.int32).cuda(), bs, 1, 1)
        calls.append((args, R.select(scores[0, 0], blocks * bs, bs, n, 1, 1)))
    run_together([lambda a=a: pa.select_blocks(*a) for a, _ in calls], 3000)
    for (tables, *_), want in calls:
        assert tables[0, 0].tolist() == want
    assert pa.get_device_error() == 0


@pytest.mark.parametrize("Hq,qlen", [(8, 1), (64, 1), (64, 4)])
def test_one_pass_and_split_decodes(Hq, qlen):
    """The split variant takes more shared memory than the one-pass variant of the same kernel."""
    pa = _gpu.lib()
    g = gen(Hq)
    Hkv, D, bs, L = 2, 128, 16, 700
    k, v = (randn(g, 50, Hkv, bs, D).bfloat16().cuda() for _ in range(2))
    bt = torch.randperm(50, generator=g)[:44].to(torch.int32)[None].cuda()
    cl = torch.tensor([L], dtype=torch.int32).cuda()
    shape = (1, Hq, D) if qlen == 1 else (1, qlen, Hq, D)
    q = randn(g, *shape).bfloat16().cuda()
    once, split = torch.empty_like(q), torch.empty_like(q)
    ws = torch.empty(pa.decode_multi_split_workspace_size(1, qlen, Hq, D, L, 64), dtype=torch.uint8, device="cuda")
    args = (q, k, v, bt, cl, 0.1)
    if qlen == 1:
        works = [lambda: pa.decode(once, *args), lambda: pa.decode_split(split, *args, 1.0, L, 64, ws)]
    else:
        works = [lambda: pa.decode_multi(once, *args), lambda: pa.decode_multi_split(split, *args, 1.0, L, 64, ws)]
    for w in works:
        w()
    want = [once.clone(), split.clone()]
    run_together(works, 2000)
    assert torch.equal(once, want[0]) and torch.equal(split, want[1])
    assert pa.get_device_error() == 0


def test_one_pass_and_split_decodes_over_row_scaled_caches():
    pa = _gpu.lib()
    g = gen(4)
    Hkv, Hq, D, bs, L = 2, 8, 128, 16, 700
    k, v = (randn(g, 50, Hkv, bs, D).to(R.E4M3).cuda() for _ in range(2))
    ks, vs = (torch.rand((50, Hkv, bs), generator=g).cuda() for _ in range(2))
    bt = torch.randperm(50, generator=g)[:44].to(torch.int32)[None].cuda()
    cl = torch.tensor([L], dtype=torch.int32).cuda()
    q = randn(g, 1, Hq, D).bfloat16().cuda()
    once, split = torch.empty_like(q), torch.empty_like(q)
    ws = torch.empty(pa.decode_multi_split_workspace_size(1, 1, Hq, D, L, 64), dtype=torch.uint8, device="cuda")
    works = [lambda: pa.decode_rows(once, q, k, v, ks, vs, bt, cl, 0.1),
             lambda: pa.decode_rows(split, q, k, v, ks, vs, bt, cl, 0.1, L, 64, ws)]
    for w in works:
        w()
    want = [once.clone(), split.clone()]
    run_together(works, 2000)
    assert torch.equal(once, want[0]) and torch.equal(split, want[1])
    assert pa.get_device_error() == 0
