"""A host thread whose first CUDA call is one of the library's: it works as in any other thread."""
import threading

import pytest
import torch

from tests import _gpu
from tests.test_gpu_cache_ops import gen, randn

pytestmark = pytest.mark.gpu


def in_new_thread(work):
    errors = []

    def run():
        try:
            work()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    t = threading.Thread(target=run)
    t.start()
    t.join()
    if errors:
        raise errors[0]


@pytest.mark.parametrize("name", ["decode", "decode_split", "decode_multi", "decode_wide", "prefill", "decode_rows",
                                  "decode_selected", "cache_and_decode"])
def test_the_first_call_of_a_thread(name):
    pa = _gpu.lib()
    g = gen(1)
    Hkv, Hq, D, bs, L = 2, 64 if name == "decode_wide" else 8, 128, 16, 300
    k, v = (randn(g, 30, Hkv, bs, D).bfloat16().cuda() for _ in range(2))
    k8, v8 = (torch.randint(0, 100, (30, Hkv, bs, D), generator=g, dtype=torch.uint8).cuda() for _ in range(2))
    ks, vs = (torch.rand((30, Hkv, bs), generator=g).cuda() for _ in range(2))
    bt, cl = torch.arange(20, dtype=torch.int32)[None].cuda(), torch.tensor([L], dtype=torch.int32).cuda()
    q = randn(g, 1, *([3] if name in ("decode_multi", "prefill") else []), Hq, D).bfloat16().cuda()
    out, ws = torch.empty_like(q), torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    key, slot = randn(g, 1, Hkv, D).bfloat16().cuda(), torch.tensor([int(L - 1)]).cuda()
    lens = torch.full((1, Hkv), L, dtype=torch.int32).cuda()
    tables = bt[:, None].expand(-1, Hkv, -1).contiguous()
    calls = {"decode": lambda: pa.decode(out, q, k, v, bt, cl, 0.1),
             "decode_wide": lambda: pa.decode(out, q, k, v, bt, cl, 0.1),
             "decode_split": lambda: pa.decode_split(out, q, k, v, bt, cl, 0.1, 1.0, L, 64, ws),
             "decode_multi": lambda: pa.decode_multi(out, q, k, v, bt, cl, 0.1),
             "prefill": lambda: pa.prefill(out, q, k, v, bt, cl, 0.1),
             "decode_rows": lambda: pa.decode_rows(out, q, k8, v8, ks, vs, bt, cl, 0.1),
             "decode_selected": lambda: pa.decode_selected(out, q, k, v, tables, lens, 0.1),
             "cache_and_decode": lambda: pa.cache_and_decode(out, q, key, key, slot, k, v, bt, cl, 0.1)}
    calls[name]()
    want = out.clone()
    out.fill_(float("nan"))
    torch.cuda.synchronize()
    in_new_thread(calls[name])
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert pa.get_device_error() == 0
