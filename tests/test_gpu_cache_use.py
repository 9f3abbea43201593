"""Cache-side calls as programs may make them: large and ragged batches, two
calls at once, other streams, captured graphs, shared and repeated indices,
empty batches, queries and rows that are not finite.  Results are compared
with 64-bit forms, or bit for bit with the same call made alone.
"""
import math

import pytest
import torch

import speculative_decoding_verification_88_b200 as sv
from speculative_decoding_verification_88_b200 import build as svbuild

from test_gpu_cache import T, bits, check_attention, check_write, empty_pool, expect_write, fill, make, snapshot, trees

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    svbuild.build()


@pytest.fixture
def dev():
    return torch.device("cuda:0")


def launches(fn):
    lib = sv.load_library()
    n = lib.spec_verify_kernel_launches()
    fn()
    return lib.spec_verify_kernel_launches() - n


def heads(B, N, H, D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(B, N, H, D, generator=g).to(dtype).cuda()


# --------------------------------------------------------- batches and splits

@pytest.mark.parametrize("qt,kv", [("bf16", "bf16"), ("fp16", "e4m3")])
@pytest.mark.parametrize("B,Hkv,G,N", [(300, 1, 2, 2), (297, 2, 1, 1), (520, 1, 1, 3)])
def test_attention_of_many_short_sequences(dev, qt, kv, B, Hkv, G, N):
    """More sequences than the split's threads, lengths 0 to 140, some all padding."""
    lens = [(37 * b) % 141 for b in range(B)]
    cache, table, clen = make(lens, N, 16, Hkv, 64, T[kv], seed=B)
    count = torch.tensor([(b % 4 + 1) * N // 4 if b % 3 else N for b in range(B)], dtype=torch.int32, device=dev)
    check_attention(heads(B, N, Hkv * G, 64, T[qt], 1), cache, table, clen, trees(B, N, 2), count)


@pytest.mark.parametrize("qt,kv", [("bf16", "bf16"), ("fp16", "e4m3")])
@pytest.mark.parametrize("lens,N,Hkv,G,D,page", [
    ([130, 3], 2, 2, 2, 8, 16), ([130, 3], 2, 3, 1, 24, 8), ([70], 3, 2, 2, 120, 16), ([70], 3, 1, 2, 1, 16),
    ([70], 3, 2, 1, 3, 5), ([20], 2, 1, 3, 255, 16), ([300], 2, 1, 512, 32, 16), ([100], 64, 1, 16, 64, 16),
    ([40], 1, 1, 1024, 16, 32), ([700], 2, 1, 2, 64, 4096), ([5 * (b % 3) for b in range(2000)], 1, 1, 1, 16, 16)])
def test_attention_of_unusual_sizes(dev, qt, kv, lens, N, Hkv, G, D, page):
    """The smallest, largest and odd heads, groups, pages and batches."""
    cache, table, clen = make(lens, N, page, Hkv, D, T[kv], seed=D)
    check_attention(heads(len(lens), N, Hkv * G, D, T[qt], 1), cache, table, clen, trees(len(lens), N, 2))


@pytest.mark.parametrize("qt,kv", [("bf16", "bf16"), ("bf16", "e4m3"), ("fp16", "e4m3")])
def test_attention_of_one_long_sequence_next_to_short_ones(dev, qt, kv):
    """One sequence over all blocks, others of one tile before and behind it."""
    lens = [3, 60000, 0, 127]
    cache, table, clen = make(lens, 3, 64, 1, 64, T[kv], seed=5)
    check_attention(heads(4, 3, 3, 64, T[qt], 6), cache, table, clen)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("tiles", [147, 148, 149, 591, 592, 593])
def test_attention_where_the_split_changes(dev, kv, tiles):
    """Tiles (128 tokens each) around one and four for each of 148 blocks."""
    cache, table, clen = make([tiles * 128 - 1], 1, 128, 1, 16, T[kv], seed=tiles)
    check_attention(heads(1, 1, 2, 16, T["bf16"], tiles), cache, table, clen)


@pytest.mark.parametrize("qt,kv", [("fp16", "e4m3"), ("bf16", "e4m3"), ("fp16", "fp16")])
@pytest.mark.parametrize("page", [8, 24])
def test_attention_with_the_least_shared_memory(dev, qt, kv, page):
    """Two row tiles and the smallest boxes: the fewest ring entries."""
    cache, table, clen = make([700, 0, 33], 64, page, 1, 128, T[kv], seed=page)
    check_attention(heads(3, 64, 4, 128, T[qt], 3), cache, table, clen, trees(3, 64, 4))


def attention64(q, cache, table, clen, parent):
    """The formula in 64 bits on the GPU, a sequence at a time: out, and the sums of w |v|."""
    B, N, Hq, D = q.shape
    H, page = cache.num_heads, cache.page_size
    out = torch.zeros(B, N, Hq, D, dtype=torch.float64, device=q.device)
    wabs = torch.zeros_like(out)
    k8, v8 = (x.view(torch.uint8) if cache.k_scale is not None else x for x in (cache.k, cache.v))
    for b in range(B):
        L = int(clen[b])
        t = torch.arange(L + N, device=q.device)
        pg, pl = table[b].long()[t // page], t % page
        rows = []
        for x, sc in ((k8, cache.k_scale), (v8, cache.v_scale)):
            r = x[pg, pl]
            r = r.double() if sc is None else r.view(T["e4m3"]).double() * sc.transpose(1, 2)[pg, pl].double()[..., None]
            rows.append(r.permute(1, 0, 2))  # [H, tokens, D]
        see = torch.zeros(N, L + N, dtype=torch.bool)
        see[:, :L] = True
        up = parent[b].tolist()
        for i in range(N):
            j = i
            see[i, L + j] = True
            while j > 0:
                j = up[j]
                see[i, L + j] = True
        qb = q[b].double().view(N, H, Hq // H, D).permute(1, 2, 0, 3)  # [H, G, N, D]
        s = qb @ rows[0][:, None].transpose(-1, -2) * D ** -0.5
        w = torch.softmax(s.masked_fill(~see.to(q.device), -math.inf), -1)
        out[b] = (w @ rows[1][:, None]).permute(2, 0, 1, 3).reshape(N, Hq, D)
        wabs[b] = (w @ rows[1][:, None].abs()).permute(2, 0, 1, 3).reshape(N, Hq, D)
    return out, wabs


@pytest.mark.parametrize("qt,kv,B,N,Hkv,G,D,page", [
    ("bf16", "bf16", 64, 26, 8, 4, 128, 64), ("fp16", "fp16", 48, 5, 8, 4, 128, 16),
    ("bf16", "e4m3", 96, 26, 8, 4, 128, 64), ("fp16", "e4m3", 64, 9, 8, 8, 64, 32),
    ("bf16", "bf16", 24, 40, 8, 8, 128, 64), ("bf16", "bf16", 200, 4, 8, 1, 64, 128),
    ("fp16", "e4m3", 16, 40, 8, 8, 128, 16), ("bf16", "e4m3", 16, 64, 8, 4, 64, 8),
    ("bf16", "e4m3", 40, 5, 8, 8, 128, 128), ("bf16", "e4m3", 64, 3, 8, 2, 96, 16),
    ("fp16", "fp16", 100, 13, 4, 8, 80, 32)])
def test_attention_of_batches_that_wait_for_memory(dev, qt, kv, B, N, Hkv, G, D, page):
    """Every block walks several sequences, and the products wait for the tiles:
    each tile's wait has to be for that very tile.  The bound as in
    check_attention, with scores of at most 60 (|q k| of 128 unit elements
    over sqrt(128), four standard deviations a factor)."""
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, 4000, (B,), generator=g).tolist()
    need = [-(-(n + N) // page) for n in lens]
    order = torch.randperm(sum(need), generator=g).int()
    table = torch.full((B, max(need)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    cache, table = empty_pool(sum(need), page, Hkv, D, T[kv]), table.to(dev)
    clen = torch.tensor(lens, dtype=torch.int32, device=dev)
    gg = torch.Generator("cuda").manual_seed(B)
    zero = torch.zeros(1, dtype=torch.int32, device=dev)
    for b, n in enumerate(lens):
        k, v = (torch.randn(1, n + N, Hkv, D, device=dev, generator=gg).to(T[qt]) for _ in range(2))
        sv.cache_write(cache, table[b:b + 1], zero, k, v)
    q = torch.randn(B, N, Hkv * G, D, device=dev, generator=gg).to(T[qt])
    parent = trees(B, N, B)
    runs = [sv.tree_attention(q, cache, table, clen, parent)["out"] for _ in range(12)]
    want, wabs = attention64(q, cache, table, clen, parent)
    u = torch.finfo(T[qt]).eps / 2
    score = 60 * (D + 16) * 2.0 ** -23
    tiny = 4100 * 2.0 ** -25 * 16  # weights below the 16-bit float's or the last term's range, |v| < 8
    tol = u * want.abs() + (u + 2 * (score + 2.0 ** -21) + 4100 * 2.0 ** -23) * (1 + 2 * u) * wabs + tiny * (qt == "fp16" or kv == "e4m3")
    over = ((runs[0].double() - want).abs() - tol).amax(dim=(1, 3)).flatten()
    assert not (over > 0).any() and not torch.isnan(runs[0]).any(), f"{int((over > 0).sum())} of {over.numel()} (sequence, head)s off"
    for r in runs[1:]:
        assert torch.equal(r, runs[0])


# ------------------------------------------------------------ views and values

@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_attention_of_broadcast_and_transposed_queries_and_tables(dev, kv):
    cache, table, clen = make([200], 5, 16, 2, 64, T[kv])
    clen = clen.repeat(3)
    one = heads(1, 5, 4, 64, T["bf16"], 1)
    want = sv.tree_attention(one.repeat(3, 1, 1, 1), cache, table.repeat(3, 1), clen)["out"]
    assert torch.equal(want, sv.tree_attention(one.expand(3, 5, 4, 64), cache, table.expand(3, -1), clen)["out"])
    turned = one.repeat(3, 1, 1, 1).transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(want, sv.tree_attention(turned, cache, table.repeat(3, 1), clen)["out"])
    same = heads(1, 1, 1, 64, T["bf16"], 2)
    want = sv.tree_attention(same.repeat(3, 5, 4, 1), cache, table.repeat(3, 1), clen)["out"]
    assert torch.equal(want, sv.tree_attention(same.expand(3, 5, 4, 64), cache, table.repeat(3, 1), clen)["out"])


@pytest.mark.parametrize("qt,kv", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3"), ("fp16", "e4m3")])
@pytest.mark.parametrize("page,D,layout,L", [(16, 64, "hnd", 300), (16, 128, "nhd", 40), (12, 66, "padded", 50)])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_attention_of_queries_that_are_not_finite(dev, qt, kv, page, D, layout, L, bad):
    """Their own rows are NaN (the keys have both signs), all others as without them."""
    cache, table, clen = make([L], 4, page, 2, D, T[kv], layout)
    q = heads(1, 4, 6, D, T[qt], 1)
    clean = sv.tree_attention(q, cache, table, clen, lse=True)
    q[0, 1, 2, 7] = bad
    q[0, 3, 5] = bad
    got = sv.tree_attention(q, cache, table, clen, lse=True)
    odd = torch.zeros(1, 4, 6, dtype=torch.bool, device=dev)
    odd[0, 1, 2] = odd[0, 3, 5] = True
    assert torch.isnan(got["out"][odd]).all()
    assert torch.equal(got["out"][~odd], clean["out"][~odd]) and torch.equal(got["lse"][~odd], clean["lse"][~odd])


@pytest.mark.parametrize("qt,kv", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3"), ("fp16", "e4m3")])
@pytest.mark.parametrize("G", [1, 2, 10, 20])
def test_attention_past_the_largest_values(dev, qt, kv, G):
    """A masked place's weight is zero, not merely small: the largest finite
    values behind it (an 8-bit row's scale 2^118) do not show."""
    lens, N, D = [100, 126, 130], 6, 64
    cache, table, clen = make(lens, N, 16, 2, D, T[kv])
    parent = torch.tensor([[0, 0, 0, 1, 2, 2]] * 3, dtype=torch.int32, device=dev)
    q = heads(3, N, 2 * G, D, T[qt], 1)
    clean = sv.tree_attention(q, cache, table, clen, parent)["out"]
    for b, n in enumerate(lens):
        for j in (1, 4):
            top = torch.finfo(T[qt]).max if kv != "e4m3" else 448.0 * 2.0 ** 118
            pos = [n + j]
            fill(cache, table, b, pos, torch.full((1, 2, D), 0.5), torch.full((1, 2, D), top))
    got = sv.tree_attention(q, cache, table, clen, parent)["out"]
    for j in (0, 2, 5):  # their paths do not meet nodes 1 and 4
        if kv == "e4m3":  # (the tile's weights share a factor that follows V's scales)
            assert torch.isfinite(got[:, j]).all()
        else:
            assert torch.equal(got[:, j], clean[:, j])


@pytest.mark.parametrize("qt,kv", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3"), ("fp16", "e4m3")])
@pytest.mark.parametrize("G", [2, 10, 26, 75])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_whose_maximum_grows(dev, qt, kv, G, D):
    """Every tile raises some rows' maximum, with few rows and many: what has
    been summed is scaled down each time, and not while it is being added to."""
    n, N = 1500, 4
    cache, table, clen = make([n], N, 16, 1, D, T[kv], seed=G)
    g = torch.Generator().manual_seed(G)
    sign = torch.randn(1, 1, D, generator=g).sign()
    ramp = torch.linspace(0.1, 30, n + N)[:, None, None] * sign
    fill(cache, table, 0, range(n + N), ramp * torch.ones(n + N, 1, D), torch.randn(n + N, 1, D, generator=g) * 3)
    size = torch.rand(1, N, G, 1, generator=g) * 1.5
    q = (sign[None] * size + 0.01 * torch.randn(1, N, G, D, generator=g)).to(T[qt]).to(dev)
    got = check_attention(q, cache, table, clen)
    for _ in range(10):
        assert torch.equal(got["out"], sv.tree_attention(q, cache, table, clen)["out"])


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("page,D,layout", [(16, 64, "hnd"), (12, 66, "padded")])
def test_attention_to_nothing_but_bad_pages(dev, kv, page, D, layout):
    """Zeros and -inf, not NaN, where no page of a row is valid."""
    cache, table, clen = make([200, 100], 3, page, 1, D, T[kv], layout)
    q = heads(2, 3, 2, D, T["bf16"], 1)
    want = sv.tree_attention(q, cache, table, clen, lse=True)
    table[0] = -1
    got = sv.tree_attention(q, cache, table, clen, lse=True)
    assert (got["out"][0] == 0).all() and (got["lse"][0] == -math.inf).all()
    assert torch.equal(got["out"][1], want["out"][1]) and torch.equal(got["lse"][1], want["lse"][1])


def test_two_sequences_that_share_their_context(dev):
    """The same pages in two rows of the table, as shared prefixes have them."""
    cache, table, clen = make([128, 128], 4, 16, 2, 64, T["bf16"])
    alone = table.clone()
    table[1, :8] = table[0, :8]
    q = heads(1, 4, 4, 64, T["bf16"], 1).repeat(2, 1, 1, 1)
    got = sv.tree_attention(q, cache, table, clen)["out"]
    assert torch.equal(got[0], sv.tree_attention(q, cache, alone, clen)["out"][0])
    offs = torch.tensor([0, 128, 256], dtype=torch.int32, device=dev)
    rows = sv.cache_read(cache, table, offs, 256)
    assert torch.equal(rows["k"][:128], rows["k"][128:])


def test_commit_of_a_path_that_names_one_node_twice(dev):
    """Each row receives what the named row held before the call."""
    cache, table, clen = make([20], 8, 16, 2, 64, T["bf16"])
    offs = torch.tensor([0, 28], dtype=torch.int32, device=dev)
    was = sv.cache_read(cache, table, offs, 28)
    path = torch.tensor([[0, 5, 5, 3, 7, 7, 7, 7]], dtype=torch.int32, device=dev)
    acc = torch.tensor([7], dtype=torch.int32, device=dev)
    new = sv.cache_commit(cache, table, clen, {"accepted_len": acc, "path": path})
    now = sv.cache_read(cache, table, offs, 28)
    assert new.tolist() == [28]
    at = list(range(20)) + [20 + j for j in (0, 5, 5, 3, 7, 7, 7, 7)]
    assert torch.equal(now["k"], was["k"][at]) and torch.equal(now["v"], was["v"][at])


@pytest.mark.parametrize("src", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rd,layout", [(128, 128, "hnd"), (96, 32, "nhd"), (66, 22, "padded")])
def test_turned_rows_at_the_ends_of_their_type(dev, src, interleaved, D, rd, layout):
    """Codes and scales of turned 8-bit rows are those of exact arithmetic: rows
    up to the type's largest value (whose sums pass it), tiny and zero ones, one
    element alone, values that are 448ths of one another, both zeros; a row with
    an infinity or a NaN has a NaN scale and leaves its neighbours alone."""
    H, N = 2, 12
    cache, table, clen = make([9], N, 16, H, D, T["e4m3"], layout)
    top = torch.finfo(T[src]).max
    g = torch.Generator().manual_seed(D)
    k = torch.randn(1, N, H, D, generator=g).double()
    k[0, 0] *= top / k[0, 0].abs().amax()
    k[0, 1] = top * torch.randn(H, D, generator=g).sign()
    k[0, 2] = top / 3
    k[0, 3] *= torch.finfo(T[src]).tiny
    k[0, 4] = 0.0
    k[0, 5] = -0.0
    k[0, 6] = 0.0
    k[0, 6, 0, D // 2 - 1], k[0, 6, 1, 0] = 3.0, -5.0
    k[0, 7, 0, 3], k[0, 7, 1, D - 1] = math.inf, math.nan
    k[0, 8] = torch.arange(D) * 0.75 * 2.0 ** -4 + 0.75 * 17
    k[0, 8, :, 0] = 448 * 0.75
    k[0, 9] = (torch.arange(D) - D // 2) * 2.0 ** -9
    k[0, 10] *= 1e-42
    k = k.to(T[src]).to(dev)
    rope = sv.rotary_frequencies(rd, interleaved=interleaved, device=dev)
    for turn in (rope, None):
        before = snapshot(cache)
        sv.cache_write(cache, table, clen, k, k, rope=turn)
        check_write(cache, before, expect_write(cache, table, [9], k, k, None, None, turn), k, turn)


# ------------------------------------------------------ empty and tiny batches

def test_empty_batches_do_nothing(dev):
    cache, table, clen = make([5], 2, 16, 2, 64, T["bf16"])
    before = bits(cache.k), bits(cache.v)
    none_t, none_l = table[:0], clen[:0]

    def calls():
        for B, N in ((0, 3), (1, 0)):
            t, ln = (none_t, none_l) if B == 0 else (table, clen)
            k = torch.zeros(B, N, 2, 64, dtype=torch.bfloat16, device=dev)
            sv.cache_write(cache, t, ln, k, k)
        q = torch.zeros(0, 3, 4, 64, dtype=torch.bfloat16, device=dev)
        assert sv.tree_attention(q, cache, none_t, none_l)["out"].shape == q.shape
        offs = torch.zeros(2, dtype=torch.int32, device=dev)
        assert sv.cache_read(cache, table, offs, 0)["k"].shape == (0, 2, 64)
        assert sv.cache_commit(cache, none_t, none_l, {"accepted_len": none_l}).shape == (0,)
        x = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device=dev)
        pos = torch.zeros(0, dtype=torch.int32, device=dev)
        assert sv.rotary(x, pos, sv.rotary_frequencies(64, device=dev)).shape == x.shape

    assert launches(calls) == 0
    assert torch.equal(bits(cache.k), before[0]) and torch.equal(bits(cache.v), before[1])


def test_launch_counts(dev):
    """As documented, for both forms of attention and of the commit."""
    rope = sv.rotary_frequencies(64, device=dev)
    for page, layout, L, grids in ((16, "hnd", 900, 2), (128, "hnd", 20, 1), (12, "padded", 900, 1)):
        cache, table, clen = make([L], 3, page, 1, 64, T["bf16"], layout)
        if page == 128:
            table = table[:, :1].contiguous()
        q = heads(1, 3, 2, 64, T["bf16"], 1)
        assert launches(lambda: sv.tree_attention(q, cache, table, clen)) == grids
        k = heads(1, 3, 1, 64, T["bf16"], 2)
        assert launches(lambda: sv.cache_write(cache, table, clen, k, k, rope=rope, q=q)) == 1
        pos = torch.zeros(1, 3, dtype=torch.int32, device=dev)
        assert launches(lambda: sv.rotary(q, pos, rope)) == 1
        res = {"accepted_len": torch.ones_like(clen), "path": torch.tensor([[0, 2, -1]], dtype=torch.int32, device=dev)}
        assert launches(lambda: sv.cache_commit(cache, table, clen, res)) == 1
        assert launches(lambda: sv.cache_commit(cache, table, clen, res, new_len=clen)) == 2
        offs = torch.tensor([0, 10], dtype=torch.int32, device=dev)
        assert launches(lambda: sv.cache_read(cache, table, offs, 10)) == 1


# ------------------------------------------------------------ at the same time

@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_calls_at_once_on_two_streams_of_one_cache(dev, kv):
    """Readers of one pool on two streams, and a writer of other pages of it."""
    cache, table, clen = make([900, 2000, 40], 8, 16, 2, 128, T[kv])
    qs = [heads(3, 8, 8, 128, T["bf16"], s) for s in (1, 2)]
    parents = [trees(3, 8, s) for s in (3, 4)]
    want = [sv.tree_attention(q, cache, table, clen, p)["out"] for q, p in zip(qs, parents)]
    offs = torch.tensor([0, 900, 2900, 2940], dtype=torch.int32, device=dev)
    rows = sv.cache_read(cache, table, offs, 2940)
    spare = empty_pool(8, 16, 2, 128, T[kv])
    own = torch.arange(8, dtype=torch.int32, device=dev)[None].contiguous()
    k = heads(1, 100, 2, 128, T["bf16"], 9)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got[i].append(sv.tree_attention(qs[i], cache, table, clen, parents[i])["out"])
        with torch.cuda.stream(streams[2]):
            sv.cache_write(spare, own, torch.zeros_like(clen[:1]), k, k)
            back = sv.cache_read(cache, table, offs, 2940)
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(x, want[i]) for x in got[i])
    assert torch.equal(back["k"], rows["k"]) and torch.equal(back["v"], rows["v"])


def test_flags_of_calls_without_a_workspace(dev):
    """They reach the device's own word, from eager calls on any stream and from
    a graph replayed after workspaces have come, grown and gone."""
    cache, table, clen = make([40, 40], 2, 16, 2, 64, T["bf16"])
    table[1, 0] = 10 ** 6
    q = heads(2, 2, 4, 64, T["bf16"], 1)
    sv.cache_device_status()
    want = sv.tree_attention(q, cache, table, clen)["out"]
    assert sv.cache_device_status(clear=False) == sv.SV_FLAG_INVALID_PAGE
    assert sv.cache_device_status() == sv.SV_FLAG_INVALID_PAGE and sv.cache_device_status() == 0
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    sv.tree_attention(q, cache, table, clen, stream=other)
    assert sv.cache_device_status(stream=other) == sv.SV_FLAG_INVALID_PAGE
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = sv.tree_attention(q, cache, table, clen)["out"]
    assert sv.cache_device_status() == 0
    for n in (1 << 10, 1 << 20, 1 << 24):
        sv.default_workspace(dev).ensure(n)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and sv.cache_device_status() == sv.SV_FLAG_INVALID_PAGE


def test_captured_step_replayed_on_new_contents(dev):
    """One captured step, replayed while lengths, tables and trees change in
    place, gives what eager calls give on the same contents."""
    B, N = 3, 6
    cache, table, clen = make([30, 0, 200], 64, 16, 2, 64, T["e4m3"])
    rope = sv.rotary_frequencies(64, device=dev)
    parent = trees(B, N, 1)
    q, k, v = (heads(B, N, h, 64, T["bf16"], h) for h in (4, 2, 2))
    path = torch.zeros(B, N, dtype=torch.int32, device=dev)
    acc = torch.zeros(B, dtype=torch.int32, device=dev)

    def step(c, lens):
        turned = sv.cache_write(c, table, lens, k, v, parent=parent, rope=rope, q=q)
        out = sv.tree_attention(turned, c, table, lens, parent)["out"]
        return out, sv.cache_commit(c, table, lens, {"accepted_len": acc, "path": path}, new_len=lens)

    twin = sv.KVCache(*(x.clone() for x in (cache.k, cache.v, cache.k_scale, cache.v_scale)))
    lens = clen.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = step(cache, clen)
    for s in range(5):
        parent.copy_(trees(B, N, 10 + s))
        path.copy_(torch.tensor([[0, 1, 3, -1, -1, -1], [0, 2, 4, 5, -1, -1], [0, -1, -1, -1, -1, -1]], dtype=torch.int32))
        acc.copy_(torch.tensor([2, 3, 0], dtype=torch.int32))
        q.add_(0.25)
        graph.replay()
        want, _ = step(twin, lens)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(clen, lens)
        assert torch.equal(bits(cache.k_scale), bits(twin.k_scale))
        assert torch.equal(bits(cache.k.view(torch.uint8)), bits(twin.k.view(torch.uint8)))


def test_results_in_the_callers_tensors(dev):
    """Preallocated results are used and are all that is written."""
    cache, table, clen = make([100, 7], 3, 16, 2, 64, T["bf16"])
    q = heads(2, 3, 4, 64, T["bf16"], 1)
    want = sv.tree_attention(q, cache, table, clen, lse=True)
    room = torch.full((4, 3, 4, 64), 7.0, dtype=torch.bfloat16, device=dev)
    res = sv.tree_attention(q, cache, table, clen, lse=True, out={"out": room[1:3], "lse": torch.empty(2, 3, 4, device=dev)})
    assert res["out"].data_ptr() == room[1].data_ptr()
    assert torch.equal(room[1:3], want["out"]) and torch.equal(res["lse"], want["lse"])
    assert (room[0] == 7).all() and (room[3] == 7).all()
    odd = torch.full((2 * 3 * 4 * 64 + 9,), 7.0, dtype=torch.bfloat16, device=dev)
    sv.tree_attention(q, cache, table, clen, out={"out": odd[1:-8].view(2, 3, 4, 64)})  # on 2-byte boundaries only
    # another kernel: both round the result (2^-8 of it each) and one its weights
    # (2^-8 of the sum of w |v|); neither exceeds the largest |v|
    top = torch.nan_to_num(cache.v.float(), 0.0).abs().max().item()
    assert (odd[1:-8].view(2, 3, 4, 64).float() - want["out"].float()).abs().max() <= 3 * 2.0 ** -8 * top + 2.0 ** -12
    assert odd[0] == 7 and (odd[-8:] == 7).all()


def test_layers_of_one_pool(dev):
    """Each layer's calls work on that layer alone; a commit moves all."""
    layers, N = 3, 4
    cache = empty_pool(6, 16, 2, 64, T["e4m3"], layers=layers)
    table = torch.tensor([[4, 0, 3]], dtype=torch.int32, device=dev)
    clen = torch.tensor([30], dtype=torch.int32, device=dev)
    zero = torch.zeros_like(clen)
    rows = [heads(1, 34, 2, 64, T["bf16"], s) for s in range(layers)]
    for i, x in enumerate(rows):
        sv.cache_write(cache.layer(i), table, zero, x, x * 2)
    offs = torch.tensor([0, 34], dtype=torch.int32, device=dev)
    was = [sv.cache_read(cache.layer(i), table, offs, 34) for i in range(layers)]
    q = heads(1, N, 4, 64, T["bf16"], 9)
    for i in range(layers):
        alone = empty_pool(6, 16, 2, 64, T["e4m3"])
        sv.cache_write(alone, table, zero, rows[i], rows[i] * 2)
        assert torch.equal(sv.tree_attention(q, cache.layer(i), table, clen)["out"],
                           sv.tree_attention(q, alone, table, clen)["out"])
    path = torch.tensor([[0, 2, 3, -1]], dtype=torch.int32, device=dev)
    sv.cache_commit(cache, table, clen, {"accepted_len": zero + 2, "path": path})
    at = list(range(31)) + [32, 33, 33]
    for i in range(layers):
        now = sv.cache_read(cache.layer(i), table, offs, 34)
        assert torch.equal(now["k"], was[i]["k"][at]) and torch.equal(now["v"], was[i]["v"][at])


def test_refusals_of_the_python_calls(dev):
    """Tensors of another type, shape, device or layout are refused before any launch."""
    cache, table, clen = make([40], 3, 16, 2, 64, T["bf16"])
    q, k = heads(1, 3, 4, 64, T["bf16"], 1), heads(1, 3, 2, 64, T["bf16"], 2)
    rope = sv.rotary_frequencies(64, device=dev)
    offs = torch.tensor([0, 10], dtype=torch.int32, device=dev)
    acc = torch.zeros_like(clen)
    pos = torch.zeros(1, 3, dtype=torch.int32, device=dev)
    wide = torch.zeros(1, 3, 4, 128, dtype=torch.bfloat16, device=dev)[..., ::2]
    coded = empty_pool(4, 16, 2, 64, T["e4m3"])
    bad = [
        lambda: sv.tree_attention(q.cpu(), cache, table, clen),
        lambda: sv.tree_attention(q.float(), cache, table, clen),
        lambda: sv.tree_attention(q.half(), cache, table, clen),
        lambda: sv.tree_attention(q[..., :32].contiguous(), cache, table, clen),
        lambda: sv.tree_attention(q[:, :, :3].contiguous(), cache, table, clen),
        lambda: sv.tree_attention(wide, cache, table, clen),
        lambda: sv.tree_attention(q, cache, table.long(), clen),
        lambda: sv.tree_attention(q, cache, table.cpu(), clen),
        lambda: sv.tree_attention(q, cache, table[0], clen),
        lambda: sv.tree_attention(q, cache, table.repeat(2, 1), clen),
        lambda: sv.tree_attention(q, cache, table, clen.long()),
        lambda: sv.tree_attention(q, cache, table, clen, pos[:, :2]),
        lambda: sv.tree_attention(q, cache, table, clen, scale=math.inf),
        lambda: sv.tree_attention(q, cache, table, clen, out={"out": torch.empty(1, 3, 4, 64, dtype=torch.bfloat16)}),
        lambda: sv.tree_attention(q, cache, table, clen, out={"out": torch.empty_like(q).float()}),
        lambda: sv.tree_attention(heads(1, 65, 4, 64, T["bf16"], 1), cache, table, clen),
        lambda: sv.tree_attention(q[:, :0], cache, table, clen),
        lambda: sv.cache_write(cache, table, clen, k, k.half()),
        lambda: sv.cache_write(cache, table, clen, k.half(), k.half()),
        lambda: sv.cache_write(cache, table, clen, k, k[:, :2]),
        lambda: sv.cache_write(cache, table, clen, q, q),
        lambda: sv.cache_write(cache, table, clen, k, k, q=q),
        lambda: sv.cache_write(cache, table, clen, k, k, q=q.half(), rope=rope),
        lambda: sv.cache_write(cache, table, clen, k, k, rope=sv.rotary_frequencies(128, device=dev)),
        lambda: sv.cache_write(cache, table, clen, k, k, count=clen[0]),
        lambda: sv.cache_read(cache, table, offs, 10, torch.float8_e4m3fn),
        lambda: sv.cache_read(cache, table, offs.long(), 10),
        lambda: sv.cache_read(cache, table, offs, 10, start=offs),
        lambda: sv.cache_read(cache, table, offs, 10, out={"k": torch.empty(10, 2, 64, dtype=torch.bfloat16)}),
        lambda: sv.cache_commit(cache, table, clen, {"accepted_len": acc.long()}),
        lambda: sv.cache_commit(cache, table, clen, {"accepted_len": acc, "path": pos[0]}),
        lambda: sv.cache_commit(cache, table, clen, {"accepted_len": acc, "path": pos}, new_len=clen.long()),
        lambda: sv.rotary(q, pos.long(), rope),
        lambda: sv.rotary(q, pos[0], rope),
        lambda: sv.rotary(coded.k[:1, :3], pos[:, :2], rope),
        lambda: sv.rotary(q, pos, sv.rotary_frequencies(128, device=dev)),
        lambda: sv.rotary(q, pos, rope, out=q.float()),
        lambda: sv.rotary(wide, pos, rope),
        lambda: sv.Rotary(rope.inv_freq.float()),
        lambda: sv.Rotary(rope.inv_freq.cpu()),
        lambda: sv.rotary_frequencies(63, device=dev),
        lambda: sv.KVCache(coded.k, coded.v),
        lambda: sv.KVCache(cache.k, cache.v, coded.k_scale, coded.v_scale),
        lambda: sv.KVCache(cache.k, cache.v.contiguous()[:1]),
        lambda: sv.KVCache(cache.k.cpu(), cache.v.cpu()),
        lambda: cache.layer(0),
    ]

    def all_of_them():
        for i, call in enumerate(bad):
            with pytest.raises((TypeError, ValueError, RuntimeError)):
                call()
                pytest.fail(f"call {i} was not refused")

    assert launches(all_of_them) == 0
