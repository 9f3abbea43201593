"""Rotary positions and the cache write at head sizes that fill no whole block,
and at positions as far as 2^31."""
import math
from fractions import Fraction

import pytest
import torch

import cache_ref as ref
import speculative_decoding_verification_88_b200 as sv
from speculative_decoding_verification_88_b200 import build as svbuild

from test_gpu_cache import T, bits, check_write, close, empty_pool, expect_write, rotation_bound, snapshot

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    svbuild.build()


@pytest.fixture
def dev():
    return torch.device("cuda:0")


@pytest.mark.parametrize("D,H", [(416, 128), (320, 256), (384, 192), (208, 571), (512, 1024), (2, 1024), (240, 1023),
                                 (336, 37), (272, 15)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rotary_of_heads_that_do_not_divide_a_block(dev, D, H, dtype):
    g = torch.Generator().manual_seed(D)
    x = torch.randn(3, H, D, generator=g).to(T[dtype]).to(dev)
    pos = torch.tensor([0, 7, 1000], dtype=torch.int32)
    rd = D // 2 // 2 * 2 if H % 2 else D
    rope = sv.rotary_frequencies(max(rd, 2), device=dev)
    want = ref.rotate(x, pos, rope.inv_freq)
    close(sv.rotary(x, pos.to(dev), rope), want, rotation_bound(x, want, 2 * rope.inv_freq.numel(), T[dtype], 1.0, False),
          "rotary")


@pytest.mark.parametrize("D,H,Hq", [(208, 85, 401), (208, 285, 1), (240, 100, 55), (176, 17, 300)])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_cache_write_of_heads_that_do_not_divide_a_block(dev, D, H, Hq, kv):
    g = torch.Generator().manual_seed(H)
    cache = empty_pool(3, 16, H, D, T[kv])
    table = torch.tensor([[2, 0]], dtype=torch.int32, device=dev)
    clen = torch.tensor([14], dtype=torch.int32, device=dev)
    k, v = (torch.randn(1, 4, H, D, generator=g).to(torch.bfloat16).to(dev) for _ in range(2))
    q = torch.randn(1, 4, Hq, D, generator=g).to(torch.bfloat16).to(dev)
    rope = sv.rotary_frequencies(D, device=dev)
    before = snapshot(cache)
    got = sv.cache_write(cache, table, clen, k, v, rope=rope, q=q)
    check_write(cache, before, expect_write(cache, table, [14], k, v, None, None, rope), k, rope)
    pos = torch.arange(14, 18, dtype=torch.int32)[None]
    want = ref.rotate(q, pos, rope.inv_freq)
    close(got, want, rotation_bound(q, want, D, T["bf16"], 1.0, False), "q")
    assert torch.equal(bits(got), bits(sv.rotary(q, pos.to(dev), rope)))
