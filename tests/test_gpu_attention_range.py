"""Tree attention where weights, scales and queries span a wide range: a token
that takes most of a row's weight before a long flat context, rows of V far
larger than the others, small elements of a query beside large ones, lengths
past the capacity."""
import math

import pytest
import torch

import speculative_decoding_verification_88_b200 as sv
from speculative_decoding_verification_88_b200 import build as svbuild

from test_gpu_cache import T, empty_pool, fill, make
from test_gpu_cache_use import attention64, heads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    svbuild.build()


@pytest.fixture
def dev():
    return torch.device("cuda:0")


def within(got, want, wabs, floor, score, n, dtype, what):
    """The output's own rounding; the weights' (u of the queries' type, and the
    part `floor` of the sum of |v| that the smallest weights may be off by);
    twice the scores' error in the exponent and the exponential's 2^-21; 32-bit
    sums over n tokens; half a step of the smallest 16-bit floats."""
    u = torch.finfo(dtype).eps / 2
    tol = u * want.abs() + (u + 2 * (score + 2.0 ** -21) + n * 2.0 ** -23) * (1 + 2 * u) * wabs + floor
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25
    over = ((got.double() - want).abs() / tol).max().item()
    assert over <= 1, f"{what}: {over:.3g} times its bound"


def one_sequence(n, N, D, dtype, k, v, page=64):
    """A pool that holds rows k, v [n + N, 1, D] of one sequence."""
    pages = -(-(n + N) // page)
    cache = empty_pool(pages, page, 1, D, dtype)
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(n)).int()[None]
    fill(cache, table, 0, range(n + N), k, v)
    return cache, table.cuda(), torch.tensor([n], dtype=torch.int32, device="cuda")


def score_error(q, cache):
    """A score's: head_dim + 16 roundings of 32 bits (truncating sums); 8-bit
    pools: each element of q within 2^-17 of the row's largest."""
    D = q.shape[-1]
    k = cache.k.float().nan_to_num()
    err = 0.0
    if cache.k_scale is not None:
        k = k * cache.k_scale.nan_to_num().transpose(1, 2)[..., None]
        err = 2.0 ** -17 * q.float().abs().max().item() * k.abs().sum(-1).max().item()
    most = q.float().norm(dim=-1).max().item() * k.norm(dim=-1).max().item()  # of the sums of |q k|
    return D ** -0.5 * (err + most * (D + 16) * 2.0 ** -23)


def chain(N):
    return (torch.arange(N, dtype=torch.int32) - 1).clamp(min=0)[None].cuda()


def sink(n, N, G, D, qt, kv, gap, size, spread, seed):
    """A first token whose weight is 2^gap of each other one's."""
    g = torch.Generator().manual_seed(seed)
    sign = torch.randn(D, generator=g).sign()
    k = 0.02 * torch.randn(n + N, 1, D, generator=g)
    k[0] = sign * (gap * math.log(2) / D ** 0.5)  # scores D^-1/2 sign . k
    v = spread * (1 + 0.3 * torch.randn(n + N, 1, D, generator=g))
    v[0] = size * torch.randn(D, generator=g)
    cache, table, clen = one_sequence(n, N, D, T[kv], k, v)
    q = sign.expand(1, N, G, D).to(T[qt]).cuda().contiguous()
    return cache, table, clen, q, score_error(q, cache)


@pytest.mark.parametrize("qt", ["bf16", "fp16"])
@pytest.mark.parametrize("G,N", [(4, 5), (8, 1), (12, 4), (26, 4), (50, 4), (8, 64)])
@pytest.mark.parametrize("n,gap,size", [(4000, 12.4, 0.1), (4000, 16.5, 0.0), (32000, 14.0, 0.1), (32000, 15.5, 0.05),
                                        (32000, 17.3, 0.0)])
def test_a_token_that_stands_out_over_8_bit_pools(dev, qt, G, N, n, gap, size):
    """The many small weights behind it keep the bits of the queries' type: as
    8-bit terms the smallest step is 2^-16 and the largest weight at least 2^13
    times half the largest scale, so a weight is off by less than 2^-28 of the
    largest beside its relative rounding."""
    D = 128 if G != 12 else 64
    cache, table, clen, q, score = sink(n, N, G, D, qt, "e4m3", gap, size, 1.0, n + G)
    want, wabs = attention64(q, cache, table, clen, chain(N))
    got = sv.tree_attention(q, cache, table, clen)["out"]
    floor = n * 2.0 ** -28 * 448.0 * cache.v_scale.nan_to_num().max().item()
    within(got, want, wabs, floor, score, n, T[qt], "out")


@pytest.mark.parametrize("G,N", [(4, 5), (26, 4), (8, 64)])
@pytest.mark.parametrize("gap", [12.3, 19.7, 25.2])
def test_a_token_that_stands_out_over_16_bit_floats(dev, G, N, gap):
    """The largest weight is near 2^7, so the smallest step, 2^-24, is 2^-31 of it."""
    n, D = 4000, 128
    cache, table, clen, q, score = sink(n, N, G, D, "fp16", "fp16", gap, 0.0, 100.0, G)
    want, wabs = attention64(q, cache, table, clen, chain(N))
    got = sv.tree_attention(q, cache, table, clen)["out"]
    within(got, want, wabs, n * 2.0 ** -32 * 300.0, score, n, T["fp16"], "out")


@pytest.mark.parametrize("qt", ["bf16", "fp16"])
@pytest.mark.parametrize("G", [1, 2, 7, 10, 20, 40])
@pytest.mark.parametrize("n", [100, 126, 130, 1000])
@pytest.mark.parametrize("size", [2.0 ** 20, 2.0 ** 60, 448.0 * 2.0 ** 118])
def test_a_large_sibling_does_not_coarsen_others_weights(dev, qt, G, n, size):
    """V's rows of nodes that a node does not see have no part in its result,
    however large: the bound is that of what it sees."""
    N, D = 6, 64
    parent = torch.tensor([[0, 0, 0, 1, 2, 2]], dtype=torch.int32, device=dev)
    cache, table, clen = make([n], N, 16, 2, D, T["e4m3"], seed=n)
    for j in (1, 4):
        fill(cache, table, 0, [n + j], torch.full((1, 2, D), 0.5), torch.full((1, 2, D), size))
    q = heads(1, N, 2 * G, D, T[qt], 1)
    got = sv.tree_attention(q, cache, table, clen, parent)["out"]
    want, wabs = attention64(q, cache, table, clen, parent)
    for j in (0, 2, 5):  # (what they see is below 8)
        within(got[:, j], want[:, j], wabs[:, j], n * 2.0 ** -28 * 8.0, score_error(q, cache), n, T[qt], f"node {j}")


@pytest.mark.parametrize("G,N", [(4, 2), (100, 1), (8, 64)])
@pytest.mark.parametrize("power", [-85, -30, 40, 114])
def test_scales_of_v_far_from_one(dev, G, N, power):
    """Results scale with V: rows of 2^power times the size give 2^power times the sums."""
    n, D = 700, 64
    g = torch.Generator().manual_seed(G)
    k, v = (torch.randn(n + N, 1, D, generator=g) for _ in range(2))
    cache, table, clen = one_sequence(n, N, D, T["e4m3"], k, v)
    cache.v_scale.mul_(2.0 ** power)
    q = heads(1, N, G, D, T["bf16"], 2)
    want, wabs = attention64(q, cache, table, clen, chain(N))
    got = sv.tree_attention(q, cache, table, clen)["out"]
    shrink = 2.0 ** -power
    within(got.double() * shrink, want * shrink, wabs * shrink, n * 2.0 ** -28 * 8.0, score_error(q, cache), n, T["bf16"],
           "out")


@pytest.mark.parametrize("qt", ["bf16", "fp16"])
@pytest.mark.parametrize("G", [1, 3, 50, 100, 200])
def test_small_elements_of_queries_over_8_bit_pools(dev, qt, G):
    """Each element of q enters within 2^-17 of its row's largest one: here 127
    that lie between two of the smallest codes, beside one of 2^7."""
    D, N = 128, 1
    k = torch.ones(1, 1, D)
    k[..., 0] = 0.0
    cache, table, clen = one_sequence(0, N, D, T["e4m3"], k, torch.ones(1, 1, D))
    q = torch.full((1, 1, G, D), 2.0 ** -7 * (1 + 1 / 8 + 15 / 128))
    q[..., 0] = 2.0 ** 7
    scale = 4.0
    got = sv.tree_attention(q.to(T[qt]).to(dev), cache, table, clen, scale=scale, lse=True)["lse"].double().cpu()
    row = cache.k.float()[table[0, 0].item(), 0, 0].double().cpu() * cache.k_scale[table[0, 0].item(), 0, 0].double().cpu()
    want = scale * (q.double() @ row)
    most = scale * (q.double().abs() @ row.abs())
    tol = scale * 2.0 ** -17 * 2.0 ** 7 * row.abs().sum() + most * (D + 16) * 2.0 ** -23 + 2.0 ** -20 * (1 + want.abs())
    assert ((got - want).abs() <= tol).all(), f"{((got - want).abs() / tol).max():.3g} times the bound"


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("page,D,layout", [(16, 64, "hnd"), (16, 256, "hnd"), (12, 66, "padded")])
@pytest.mark.parametrize("length", [2 ** 30, 2 ** 31 - 1])
def test_lengths_past_the_capacity(dev, kv, page, D, layout, length):
    """They attend to what has a place, and no loop runs past it."""
    cache, table, clen = make([96], 0, page, 2, D, T[kv], layout)
    table = table[:, :96 // page].contiguous()
    q = heads(1, 3, 4, D, T["bf16"], 1)
    ws = sv.Workspace(dev, 256)
    clen.fill_(96)
    want = sv.tree_attention(q, cache, table, clen, lse=True, workspace=ws)
    assert ws.device_status() == sv.SV_FLAG_CAPACITY
    clen.fill_(length)
    got = sv.tree_attention(q, cache, table, clen, lse=True, workspace=ws)
    assert ws.device_status() == sv.SV_FLAG_CAPACITY
    assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])
    assert torch.isfinite(got["out"]).all()


@pytest.mark.parametrize("G,N", [(4, 2), (12, 4), (100, 1), (8, 64)])
@pytest.mark.parametrize("n", [250, 1000, 30000])
@pytest.mark.parametrize("small,large", [(-85, 60), (-40, 90), (-85, 105)])
def test_scales_of_v_far_from_one_another(dev, G, N, n, small, large):
    """Tokens whose V is next to nothing beside others' still count in the sum of
    the weights: every second 128 tokens are 2^(large - small) times the size."""
    D = 64
    g = torch.Generator().manual_seed(n)
    k, v = (torch.randn(n + N, 1, D, generator=g) for _ in range(2))
    cache, table, clen = one_sequence(n, N, D, T["e4m3"], k, v)
    power = torch.where(torch.arange(n + N) // 128 % 2 == 0, small, large).double()
    page = table[0].long()[torch.arange(n + N, device=dev) // cache.page_size]
    cache.v_scale[page, 0, torch.arange(n + N, device=dev) % cache.page_size] *= (2.0 ** power).float().to(dev)
    q = heads(1, N, G, D, T["bf16"], 2)
    want, wabs = attention64(q, cache, table, clen, chain(N))
    got = sv.tree_attention(q, cache, table, clen, lse=True)
    within(got["out"].double() * 2.0 ** -large, want * 2.0 ** -large, wabs * 2.0 ** -large, n * 2.0 ** -28 * 8.0,
           score_error(q, cache), n, T["bf16"], "out")
    # the sum alone does not depend on V at all
    cache.v_scale.nan_to_num_().fill_(1.0)
    alone = sv.tree_attention(q, cache, table, clen, lse=True)["lse"]
    # each within twice the exponential's and the sums' roundings of 32 bits
    assert (got["lse"] - alone).abs().max().item() <= 2 * (2.0 ** -20 * (1 + alone.abs().max().item()) + n * 2.0 ** -23)
