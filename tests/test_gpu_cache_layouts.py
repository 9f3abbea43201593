"""Cache pools whose rows lie on 2-, 4- and 8-byte boundaries: each call gives
what it gives on a pool with contiguous pages."""
import pytest
import torch

import speculative_decoding_verification_88_b200 as sv
from speculative_decoding_verification_88_b200 import build as svbuild

from test_gpu_cache import T, bits, check_attention, make, paths, trees

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    svbuild.build()


@pytest.fixture
def dev():
    return torch.device("cuda:0")


def moved(cache, first, step):
    """The same pool with `first` bytes before it and rows a multiple of 16
    bytes and `step` bytes apart."""
    es = cache.k.element_size()
    made = []
    for t in (cache.k, cache.v):
        pages, page, H, D = t.shape
        row = (-(-D * es // 16) * 16 + step) // es
        room = torch.empty(first // es + pages * page * H * row, dtype=torch.uint8 if es == 1 else t.dtype, device="cuda")
        x = room[first // es:].view(pages, page, H, row)[..., :D]
        x.copy_(t.view(torch.uint8) if es == 1 else t)
        made.append(x.view(t.dtype))
    return sv.KVCache(*made, *(None if s is None else s.clone() for s in (cache.k_scale, cache.v_scale)))


def same(a, b):
    for x, y in ((a.k, b.k), (a.v, b.v), (a.k_scale, b.k_scale), (a.v_scale, b.v_scale)):
        assert x is None or torch.equal(bits(x.view(torch.uint8) if x.dtype == T["e4m3"] else x),
                                        bits(y.view(torch.uint8) if y.dtype == T["e4m3"] else y))


@pytest.mark.parametrize("kv", ["bf16", "fp32", "e4m3"])
@pytest.mark.parametrize("D", [128, 80, 72])
@pytest.mark.parametrize("first,step", [(0, 8), (8, 0), (8, 8), (0, 4), (4, 0), (16, 16)])
def test_calls_on_pools_of_any_alignment(dev, kv, D, first, step):
    lens, N, page, H = [70, 9], 6, 16, 2
    cache, table, clen = make(lens, N, page, H, D, T[kv], seed=D)
    other = moved(cache, first, step)
    same(cache, other)
    src = T["bf16"] if kv == "e4m3" else T[kv]
    k, v, q = (torch.randn(2, N, h, D, device=dev).to(src) for h in (H, H, 4))
    parent = trees(2, N, 3)
    rope = sv.rotary_frequencies(D // 16 * 16, device=dev)
    got = [sv.cache_write(c, table, clen, k, v, parent=parent, rope=rope, q=q) for c in (cache, other)]
    assert torch.equal(bits(got[0]), bits(got[1]))
    same(cache, other)
    if kv != "fp32":
        check_attention(got[1], other, table, clen, parent)
    path, acc = paths(2, N, 1)
    for c in (cache, other):
        sv.cache_commit(c, table, clen, {"accepted_len": acc, "path": path})
    same(cache, other)
    offs = torch.tensor([0, 76, 91], dtype=torch.int32, device=dev)
    for to in ("bf16", "fp16", "fp32"):
        a, b = (sv.cache_read(c, table, offs, 91, T[to]) for c in (cache, other))
        assert torch.equal(bits(a["k"]), bits(b["k"])) and torch.equal(bits(a["v"]), bits(b["v"]))
