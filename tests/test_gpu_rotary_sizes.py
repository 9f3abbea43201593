"""Rotary positions and the cache write at head sizes that fill no whole block,
and at positions as far as 2^31."""
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


PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")
FAR = [2 ** 31 - 1, 2 ** 31 - 2, -2 ** 31, 2 ** 30 + 12345, 1000000007, -123456789, 65537, 1]


def exact_angles(pos, inv_freq):
    """position * frequency less whole turns, from exact arithmetic, in 64 bits."""
    out = []
    for t in pos:
        row = []
        for f in inv_freq.tolist():
            a = int(t) * Fraction(f)
            row.append(float(a - 2 * PI * round(a / (2 * PI))))
        out.append(row)
    return torch.tensor(out, dtype=torch.float64)


def turn(x, angle, interleaved):
    """x [T, H, D] in 64 bits, its first pairs turned by angle [T, rd / 2]."""
    y = x.double().cpu().clone()
    rd = 2 * angle.shape[-1]
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    first = slice(0, rd, 2) if interleaved else slice(0, rd // 2)
    second = slice(1, rd, 2) if interleaved else slice(rd // 2, rd)
    a, b = y[..., first].clone(), y[..., second].clone()
    y[..., first], y[..., second] = a * c - b * s, b * c + a * s
    return y


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("base", [1.5, 10000.0, 500000.0])
def test_rotary_at_far_positions(dev, interleaved, dtype, base):
    """The same bound as at near positions: what the reduction leaves is exact."""
    D, rd = 64, 48
    x = torch.randn(len(FAR), 3, D, generator=torch.Generator().manual_seed(1)).to(T[dtype])
    rope = sv.rotary_frequencies(rd, base, interleaved=interleaved, device=dev)
    want = turn(x, exact_angles(FAR, rope.inv_freq), interleaved)
    got = sv.rotary(x.to(dev), torch.tensor(FAR, dtype=torch.int32, device=dev), rope)
    close(got, want, rotation_bound(x, want, rd, T[dtype], 1.0, interleaved), "rotary")


@pytest.mark.parametrize("D,rd", [(64, 64), (128, 64), (66, 22)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_codes_at_far_positions(dev, D, rd, interleaved):
    """8-bit rows of the last positions there are hold the codes and scales of
    exact arithmetic."""
    N, H, page = 24, 4, 4096
    pages = 2 ** 31 // page
    length = 2 ** 31 - N
    cache = empty_pool(2, page, H, D, T["e4m3"])
    table = torch.full((1, pages), -1, dtype=torch.int32, device=dev)
    table[0, pages - 1] = 1
    clen = torch.tensor([length], dtype=torch.int32, device=dev)
    g = torch.Generator().manual_seed(D)
    k, v = (torch.randn(1, N, H, D, generator=g).to(torch.bfloat16).to(dev) for _ in range(2))
    rope = sv.rotary_frequencies(rd, interleaved=interleaved, device=dev)
    y = turn(k[0], exact_angles(range(length, length + N), rope.inv_freq), interleaved)
    place = length % page
    before = snapshot(cache)
    sv.cache_write(cache, table, clen, k, v, rope=rope)
    rows = [(1, place + j, 0, j, y[j], v[0, j].double().cpu()) for j in range(N)]
    check_write(cache, before, rows, k, rope)
