"""The commit's new lengths in one of its inputs."""
import pytest
import torch

import speculative_decoding_verification_88_b200 as sv
from speculative_decoding_verification_88_b200 import build as svbuild

from test_gpu_cache import T, bits, paths

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    svbuild.build()


@pytest.fixture
def dev():
    return torch.device("cuda:0")


@pytest.mark.parametrize("into", ["cache_len", "accepted_len"])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("B,N,layers", [(1, 64, 64), (3, 26, 24), (40, 8, 2), (5, 1, 1)])
def test_new_lengths_in_an_input(dev, into, kv, B, N, layers):
    """Many blocks work on a sequence; none reads a length that another has
    written, and rows and lengths are those of a call with a tensor of its own."""
    page, H, D = 16, 8, 128
    per = -(-(60 + N) // page)
    pools = []
    for _ in range(2):
        g = torch.Generator("cuda").manual_seed(B)
        c = sv.KVCache.empty(B * per, page, H, D, T[kv], layers=layers)
        for t in (c.k, c.v, c.k_scale, c.v_scale):
            if t is not None:
                raw = t.view(torch.uint8) if kv == "e4m3" and t.dim() == 5 else t
                raw.copy_(torch.randint(0, 100, t.shape, device=dev, generator=g))
        pools.append(c)
    table = torch.randperm(B * per).int().view(B, per).to(dev)
    lens = torch.randint(0, 60, (B,), dtype=torch.int32, device=dev)
    path, acc = paths(B, N, 7)
    want = sv.cache_commit(pools[0], table, lens, {"accepted_len": acc, "path": path})
    for _ in range(20):
        a, b = lens.clone(), acc.clone()
        to = a if into == "cache_len" else b
        other = sv.KVCache(*(None if t is None else t.clone() for t in (pools[1].k, pools[1].v, pools[1].k_scale, pools[1].v_scale)))
        got = sv.cache_commit(other, table, a, {"accepted_len": b, "path": path}, new_len=to)
        assert got is to and torch.equal(got, want)
        for x, y in zip((other.k, other.v, other.k_scale, other.v_scale), (pools[0].k, pools[0].v, pools[0].k_scale, pools[0].v_scale)):
            if x is not None:
                x, y = (t.view(torch.uint8) if kv == "e4m3" and t.dim() == 5 else t for t in (x, y))
                assert torch.equal(bits(x), bits(y))
