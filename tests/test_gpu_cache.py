"""Cache-side operators on the GPU against plain 64-bit forms.

Every pool place that holds no token of a sequence is NaN (values, codes and
scales), so a read of one shows in the results.  Bounds: u(t) = eps(t)/2 is
the largest relative error of one rounding to t.
"""
import math

import pytest
import torch

import cache_ref as ref
import speculative_decoding_verification_88_b200 as sv
from speculative_decoding_verification_88_b200 import build as svbuild

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}
U32 = 2.0 ** -24


def u(dtype):
    return torch.finfo(dtype).eps / 2


@pytest.fixture(scope="module", autouse=True)
def built():
    svbuild.build()


@pytest.fixture
def dev():
    return torch.device("cuda:0")


def bits(t):
    """A tensor's memory as integers (compares NaNs too)."""
    return t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()]).cpu()


def empty_pool(pages, page, H, D, dtype, layout="hnd", layers=None):
    """A NaN-filled pool in one of three layouts."""
    lead = () if layers is None else (layers,)
    coded = dtype == torch.float8_e4m3fn
    store = torch.uint8 if coded else dtype
    made = []
    for _ in range(2):
        if layout == "hnd":
            t = torch.empty((*lead, pages, H, page, D), dtype=store, device="cuda").transpose(-3, -2)
        elif layout == "nhd":
            t = torch.empty((*lead, pages, page, H, D), dtype=store, device="cuda")
        else:  # rows padded by an odd number of elements: nothing is 16-byte aligned
            t = torch.empty((*lead, pages, page, H, D + 3), dtype=store, device="cuda")[..., :D]
        t.fill_(0x7F) if coded else t.fill_(math.nan)
        made.append(t.view(dtype) if coded and layout == "hnd" else t)
    if coded and layout != "hnd":
        made = [t.view(torch.float8_e4m3fn) for t in made]
    if coded:
        made += [torch.full((*lead, pages, H, page), math.nan, device="cuda") for _ in range(2)]
    return sv.KVCache(*made)


def fill(cache, table, b, positions, k, v):
    """Put rows k, v [n, H, D] at a sequence's positions."""
    for x, sc, y in ((cache.k, cache.k_scale, k), (cache.v, cache.v_scale, v)):
        pos = torch.tensor(list(positions), dtype=torch.long)
        if not len(pos):
            continue
        pg = table[b].cpu().long()[pos // cache.page_size].cuda()
        pl = (pos % cache.page_size).cuda()
        if sc is None:
            x[pg, pl] = y.to(x.dtype).cuda()
        else:
            code, scale = ref.code_rows(y.double())
            x.view(torch.uint8)[pg, pl] = code.float().to(torch.float8_e4m3fn).view(torch.uint8).cuda()
            sc.transpose(1, 2)[pg, pl] = scale.cuda()


def make(lens, N, page, H, D, dtype, layout="hnd", seed=0, extra_pages=2, spread=1.0):
    """A pool that holds lens[b] + N tokens of each sequence on shuffled pages."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-(max(0, n) + N) // page) for n in lens]
    order = torch.randperm(sum(need) + extra_pages, generator=g).tolist()
    table = torch.full((len(lens), max(1, max(need)) + 1), -7, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    cache = empty_pool(sum(need) + extra_pages, page, H, D, dtype, layout)
    for b, n in enumerate(lens):
        n = max(0, n) + N
        k, v = (torch.randn(n, H, D, generator=g) * spread for _ in range(2))
        fill(cache, table, b, range(n), k, v)
    return cache, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")


def trees(B, N, seed, bad=()):
    g = torch.Generator().manual_seed(seed)
    p = torch.zeros(B, N, dtype=torch.int32)
    for j in range(1, N):
        p[:, j] = torch.randint(0, j, (B,), generator=g).int()
    for b, j, value in bad:
        p[b, j] = value
    return p.cuda()


def close(got, want, tol, what):
    got = got.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what + ": NaN places"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), what + ": infinities"
    fine = torch.isfinite(want)
    over = (got - want).abs()[fine] - tol.expand_as(want)[fine]
    assert not over.numel() or over.max() <= 0, f"{what}: {over.max():.3g} over its bound"


# ------------------------------------------------------------------ rotary

def rotation_bound(x, want, rd, dtype, magnitude, interleaved):
    """The angle in half turns is rounded to 32 bits (pi 2^-24 in radians), cos
    and sin are within 2 units (CUDA's stated sincospi error), two products, a
    sum and the factor round once each; then one rounding to the type."""
    a = x.double().cpu().abs()
    pair = torch.zeros_like(a)
    if interleaved:
        s = a[..., 0:rd:2] + a[..., 1:rd:2]
        pair[..., 0:rd:2] = pair[..., 1:rd:2] = s
    else:
        s = a[..., :rd // 2] + a[..., rd // 2:rd]
        pair[..., :rd // 2] = pair[..., rd // 2:rd] = s
    one = pair * abs(magnitude) * (math.pi + 2 * 2 + 4) * U32
    return one * (1 + u(dtype)) + (u(dtype) if dtype != torch.float32 else 0.0) * want.abs() + 2.0 ** -40


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T_,H,D,rd", [(1, 1, 2, 2), (5, 32, 128, 128), (33, 3, 128, 64), (7, 5, 80, 32),
                                       (4, 2, 66, 22), (3, 2, 512, 512), (700, 7, 96, 48), (9, 1, 64, 2)])
def test_rotary(dev, dtype, interleaved, T_, H, D, rd):
    g = torch.Generator().manual_seed(T_ + D)
    x = torch.randn(T_, H, D, generator=g).to(T[dtype]).to(dev)
    pos = torch.randint(-5, 2 ** 31 - 1, (T_,), generator=g).int()
    pos[0] = 0
    rope = sv.rotary_frequencies(rd, 500000.0, scaling="yarn", factor=4.0, original_len=4096.0,
                                 interleaved=interleaved, device=dev)
    for inverse in (False, True):
        want = ref.rotate(x, pos, rope.inv_freq, interleaved, rope.magnitude, inverse)
        # the angle itself, position * f, is one 64-bit product on both sides
        far = (pos.double().abs()[:, None, None] * 2.0 ** -52).expand_as(want) * x.double().cpu().abs().amax(-1, True) * 4
        got = sv.rotary(x, pos.to(dev), rope, inverse=inverse)
        close(got, want, rotation_bound(x, want, rd, T[dtype], rope.magnitude, interleaved) + far, "rotary")
        assert torch.equal(bits(got[..., rd:]), bits(x[..., rd:]))
    y = x.clone()
    assert sv.rotary(y, pos.to(dev), rope, out=y) is y
    assert torch.equal(bits(y), bits(sv.rotary(x, pos.to(dev), rope)))


def test_rotary_strided_batch_and_transpose(dev):
    """[B, N, H, D] views of a fused projection; inverse is the transpose (the
    gradient): <R x, y> = <x, R' y>, and differences give the same."""
    B, N, H, D = 3, 4, 5, 64
    fused = torch.randn(B, N, 3 * H, D, device=dev)
    x = fused[:, :, H:2 * H]
    pos = torch.randint(0, 10000, (B, N), dtype=torch.int32, device=dev)
    rope = sv.rotary_frequencies(32, device=dev)
    got = sv.rotary(x, pos, rope)
    assert torch.equal(got, sv.rotary(x.contiguous(), pos, rope))
    y = torch.randn_like(got)
    back = sv.rotary(y, pos, rope, inverse=True)
    left, right = (got.double() * y.double()).sum(), (x.double() * back.double()).sum()
    # both sums of n products, each value within 10 * 2^-24 of the two members of its pair
    bound = 2 * 10 * U32 * 2 * (x.double().abs().sum() * y.double().abs().max()).item()
    assert abs((left - right).item()) <= bound
    for at in ((0, 0, 0, 0), (2, 3, 4, 31), (1, 2, 3, 40)):
        h = 0.5
        up, down = x.contiguous().clone(), x.contiguous().clone()
        up[at] += h
        down[at] -= h
        # the map is linear: the difference quotient is the gradient up to rounding
        d = ((sv.rotary(up, pos, rope).double() - sv.rotary(down, pos, rope).double()) * y.double()).sum() / (2 * h)
        size = (x[at[:3]].abs().max().item() + h) * y[at[:3]].abs().max().item()
        assert abs((d - back[at].double()).item()) <= 2 * 2 * 2 * 10 * U32 * size * 2 / h
    assert sv.rotary(x[:0], pos[:0], rope).shape == (0, N, H, D)


# ------------------------------------------------------------- cache write

def expect_write(cache, table, lens, k, v, parent, count, rope):
    """What the pool should hold: K and V values of every written place in 64 bits."""
    B, N = k.shape[:2]
    pages = cache.k.shape[0]
    rows = []
    for b in range(B):
        d = ref.depths(None if parent is None else parent[b].tolist(), N)
        n = N if count is None else max(0, min(N, int(count[b])))
        for j in range(n):
            L = max(0, int(lens[b]))
            t = L + j
            if t // cache.page_size >= table.shape[1]:
                continue
            pg = int(table[b, t // cache.page_size])
            if not 0 <= pg < pages:
                continue
            y = k[b, j].double().cpu()
            if rope is not None:
                y = ref.rotate(k[b, j][None], torch.tensor([L + d[j]]), rope.inv_freq, rope.interleaved,
                               rope.magnitude)[0]
            rows.append((pg, t % cache.page_size, b, j, y, v[b, j].double().cpu()))
    return rows


def check_write(cache, before, rows, k, rope):
    pool_type = cache.k.dtype
    touched = torch.zeros(cache.k.shape[:2], dtype=torch.bool)
    for pg, pl, b, j, y, z in rows:
        assert not touched[pg, pl]
        touched[pg, pl] = True
    now = [t.clone() for t in (cache.k, cache.v)]
    scales = None if cache.k_scale is None else [t.transpose(1, 2).cpu() for t in (cache.k_scale, cache.v_scale)]
    host = [t.cpu() if pool_type != torch.float8_e4m3fn else t.view(torch.uint8).cpu().view(pool_type) for t in now]
    for pg, pl, b, j, y, z in rows:
        for i, w in ((0, y), (1, z)):
            got = host[i][pg, pl].double()
            if scales is not None:
                code, scale = ref.code_rows(w)
                fine = torch.isfinite(scale)
                assert torch.equal(scales[i][pg, pl][fine], scale[fine]), "scale"
                assert torch.isnan(scales[i][pg, pl][~fine]).all()
                assert torch.equal(got[fine], code[fine]), "codes"
            elif i == 1 or rope is None:
                assert torch.equal(bits(host[i][pg, pl]), bits(w.to(pool_type)))
            else:
                x = k[b, j]
                tol = rotation_bound(x, w, 2 * rope.inv_freq.numel(), pool_type, rope.magnitude, rope.interleaved)
                close(got, w, tol, "k")
    # the places of no written token are as they were
    for t, old in zip((cache.k, cache.v), before[:2]):
        t = t.view(torch.uint8) if pool_type == torch.float8_e4m3fn else t
        keep = ~touched
        assert torch.equal(bits(t)[keep], bits(old)[keep])
    if scales is not None:
        for t, old in zip(scales, before[2:]):
            assert torch.equal(bits(t)[~touched], bits(old.transpose(1, 2))[~touched])


def snapshot(cache):
    s = [t.view(torch.uint8).clone() if t.dtype == torch.float8_e4m3fn else t.clone() for t in (cache.k, cache.v)]
    if cache.k_scale is not None:
        s += [cache.k_scale.clone(), cache.v_scale.clone()]
    return s


WRITES = [
    # lens, N, page, H, D, rd, layout
    ([0], 1, 16, 1, 64, 64, "hnd"),
    ([500], 5, 16, 8, 128, 128, "hnd"),
    ([0, 15, 16, 17, 100], 26, 16, 2, 128, 64, "nhd"),
    ([3, 130, 63], 64, 64, 3, 80, 32, "hnd"),
    ([7, 9], 5, 12, 2, 66, 22, "padded"),
    ([1, 2, 300], 9, 1, 2, 256, 256, "nhd"),
    ([5, -3], 200, 32, 2, 96, 96, "hnd"),
]


@pytest.mark.parametrize("src,pool", [("bf16", "bf16"), ("fp16", "fp16"), ("fp32", "fp32"), ("bf16", "e4m3"),
                                      ("fp16", "e4m3"), ("fp32", "e4m3")])
@pytest.mark.parametrize("case", range(len(WRITES)))
def test_cache_write(dev, src, pool, case):
    lens, N, page, H, D, rd, layout = WRITES[case]
    B = len(lens)
    g = torch.Generator().manual_seed(case)
    cache, table, clen = make(lens, N, page, H, D, T[pool], layout, seed=case)
    empty = empty_pool(cache.k.shape[0], page, H, D, T[pool], layout)
    k, v = (torch.randn(B, N, H, D, generator=g).to(T[src]).to(dev) for _ in range(2))
    v[0, 0, 0] = 0.0  # an all-zero row
    q = torch.randn(B, N, 2 * H, D, generator=g).to(T[src]).to(dev)
    parent = trees(B, N, case) if N <= 64 and case % 2 else None
    for interleaved, turn in ((False, True), (True, True), (False, False)):
        rope = sv.rotary_frequencies(rd, interleaved=interleaved, device=dev) if turn else None
        before = snapshot(empty)
        got = sv.cache_write(empty, table, clen, k, v, parent=parent, rope=rope, q=q if turn else None)
        check_write(empty, before, expect_write(empty, table, lens, k, v, parent, None, rope), k, rope)
        if turn:
            d = torch.tensor([ref.depths(None if parent is None else parent[b].tolist(), N) for b in range(B)])
            pos = torch.tensor(lens).clamp(min=0)[:, None] + d
            want = ref.rotate(q, pos, rope.inv_freq, interleaved)
            close(got, want, rotation_bound(q, want, rd, T[src], 1.0, interleaved), "q")
            assert torch.equal(bits(got), bits(sv.rotary(q, pos.int().to(dev), rope)))


def test_cache_write_values_that_break_rows(dev):
    """Infinities and NaN give their row a NaN scale and leave the others alone;
    tiny, huge and tied values round as exact arithmetic says."""
    H, D, N = 4, 64, 6
    cache, table, clen = make([10], N, 16, H, D, T["e4m3"])
    k = torch.randn(1, N, H, D)
    k[0, 0, 0, 3], k[0, 1, 1, 5], k[0, 1, 2, 0] = math.inf, math.nan, -math.inf
    k[0, 2] *= 1e-42  # subnormal rows, some of whose scales underflow
    k[0, 3] *= 3e38 / k[0, 3].abs().amax()
    # ties between codes: amax 448 * 3 / 4 makes the scale exactly 3/4
    k[0, 4] = torch.arange(D)[None] * 0.75 * 2.0 ** -4 + 0.75 * 17
    k[0, 4, :, 0] = 448 * 0.75
    k[0, 5] = (torch.arange(D) - 32)[None] * 2.0 ** -9  # the smallest codes
    k[0, 5, :, 0] = 448.0
    before = snapshot(cache)
    k = k.to(dev)
    sv.cache_write(cache, table, clen, k, k)
    check_write(cache, before, expect_write(cache, table, [10], k, k, None, None, None), k, None)


def test_cache_write_counts_bad_pages_and_capacity(dev):
    lens, N, page, H, D = [4, 40, 20, 0], 20, 16, 2, 64
    cache, table, clen = make(lens, N, page, H, D, T["bf16"], extra_pages=3)
    table = table[:, :4].clone().contiguous()  # 64 places: the last tree of sequence 1 still fits
    pages = cache.k.shape[0]
    table[0, 1] = pages      # outside the pool
    table[2, 1] = -1
    clen[3] = 50             # 50 + 20 > 64: six tokens have no place
    table[3] = torch.tensor([pages - 1, pages - 2, pages - 3, table[3, 0].item()])
    lens = clen.tolist()
    count = torch.tensor([20, 7, 30, 100], dtype=torch.int32, device=dev)
    parent = trees(4, N, 3, bad=[(0, 5, 5), (1, 2, -1), (2, 19, 40)])
    rope = sv.rotary_frequencies(64, device=dev)
    for kv in ("bf16", "e4m3"):
        c = empty_pool(pages, page, H, D, T[kv])
        k, v = (torch.randn(4, N, H, D, device=dev, dtype=torch.bfloat16) for _ in range(2))
        q = torch.randn(4, N, 4, D, device=dev, dtype=torch.bfloat16)
        q_out = torch.full_like(q, 7.0)
        ws = sv.Workspace(dev, 256)
        before = snapshot(c)
        sv.cache_write(c, table, clen, k, v, parent=parent, count=count, rope=rope, q=q, q_out=q_out, workspace=ws)
        check_write(c, before, expect_write(c, table, lens, k, v, parent, count, rope), k, rope)
        assert (q_out[1, 7:] == 7.0).all() and not (q_out[1, :7] == 7.0).all(-1).any()
        assert ws.device_status() == sv.SV_FLAG_INVALID_PAGE | sv.SV_FLAG_CAPACITY | sv.SV_FLAG_INVALID_TREE
        none = torch.zeros(4, dtype=torch.int32, device=dev) - 2
        before = snapshot(c)
        sv.cache_write(c, table, clen, k, v, count=none, workspace=ws)
        check_write(c, before, [], k, None)
        assert ws.device_status() == 0


# --------------------------------------------------------------- read-back

@pytest.mark.parametrize("pool,to", [("bf16", "bf16"), ("fp16", "fp32"), ("fp32", "bf16"), ("e4m3", "bf16"),
                                     ("e4m3", "fp16"), ("e4m3", "fp32")])
@pytest.mark.parametrize("lens,page,H,D,layout", [([5], 16, 1, 64, "hnd"), ([0, 1, 40, 0, 17], 16, 2, 128, "nhd"),
                                                  ([200, 33], 64, 3, 80, "hnd"), ([7, 30], 12, 2, 66, "padded"),
                                                  ([0, 0], 8, 1, 32, "hnd")])
def test_cache_read(dev, pool, to, lens, page, H, D, layout):
    cache, table, clen = make(lens, 0, page, H, D, T[pool], layout, seed=sum(lens))
    start = [n // 3 for n in lens]
    first = 3  # rows before the first sequence and behind the last stay as they were
    offs = [first]
    for n, s in zip(lens, start):
        offs.append(offs[-1] + n - s)
    total = offs[-1] + 4
    out = {x: torch.full((total, H, D), 7.0, dtype=T[to], device=dev) for x in ("k", "v")}
    got = sv.cache_read(cache, table, torch.tensor(offs, dtype=torch.int32, device=dev), total, T[to],
                        start=torch.tensor(start, dtype=torch.int32, device=dev), out=out)
    for i, x in enumerate(("k", "v")):
        assert got[x] is out[x]
        for b, n in enumerate(lens):
            want = ref.pool_rows(cache, table[b].tolist(), range(start[b], n))[i]
            # code times scale rounds once to 32 bits, then once to the type
            tol = (u(T[to]) + (U32 if pool == "e4m3" else 0)) * (1 + U32) * want.abs() + \
                (2.0 ** -25 if to == "fp16" else 0.0)
            close(got[x][offs[b]:offs[b + 1]], want, tol, x)
        assert (got[x][:first] == 7.0).all() and (got[x][offs[-1]:] == 7.0).all()


def test_cache_read_without_a_place_gives_zeros(dev):
    cache, table, clen = make([40, 40], 0, 16, 2, 64, T["bf16"])
    table[0, 1] = 10 ** 6
    ws = sv.Workspace(dev, 256)
    offs = torch.tensor([0, 40, 40 + 70], dtype=torch.int32, device=dev)
    table = table[:, :4].contiguous()  # 64 places
    table[1, 3] = table[0, 0]
    got = sv.cache_read(cache, table, offs, 110, workspace=ws)
    assert ws.device_status() == sv.SV_FLAG_INVALID_PAGE | sv.SV_FLAG_CAPACITY
    assert (got["k"][16:32] == 0).all() and (got["v"][40 + 64:] == 0).all()
    assert torch.equal(got["k"][:16], cache.k[table[0, 0].long()])


# ------------------------------------------------------------------ commit

def paths(B, N, seed):
    g = torch.Generator().manual_seed(seed)
    path = torch.full((B, N), -1, dtype=torch.int32)
    acc = torch.zeros(B, dtype=torch.int32)
    for b in range(B):
        n = int(torch.randint(0, N, (1,), generator=g)) if b else N - 1
        pick = torch.randperm(N - 1, generator=g)[:n].sort().values + 1
        path[b, 0] = 0
        path[b, 1:n + 1] = pick.int()
        acc[b] = n
    return path.cuda(), acc.cuda()


@pytest.mark.parametrize("pool", ["bf16", "e4m3", "fp32"])
@pytest.mark.parametrize("lens,N,page,H,D,layout,layers", [
    ([9], 1, 16, 1, 64, "hnd", None), ([0, 5, 31, 32], 26, 16, 2, 128, "hnd", 3),
    ([100, 3], 64, 12, 3, 66, "padded", 2), ([17] * 9, 8, 64, 4, 80, "nhd", None)])
def test_cache_commit(dev, pool, lens, N, page, H, D, layout, layers):
    B = len(lens)
    _, table, clen = make(lens, N, page, H, D, T["bf16"])
    cache = empty_pool(int(table.max()) + 3, page, H, D, T[pool], layout, layers)
    g = torch.Generator("cuda").manual_seed(1)
    for t in (cache.k, cache.v):
        if pool == "e4m3":
            t.view(torch.uint8).copy_(torch.randint(0, 127, t.shape, device=dev, generator=g).byte())
        else:
            t.copy_(torch.randn(t.shape, device=dev, generator=g))
    for t in (cache.k_scale, cache.v_scale):
        if t is not None:
            t.copy_(torch.rand(t.shape, device=dev, generator=g))
    path, acc = paths(B, N, 5)
    want = [t if layers else t[None] for t in snapshot(cache)]
    old = [t.clone() for t in want]
    for b in range(B):
        for j in range(1, int(acc[b]) + 1):
            src, dst = lens[b] + int(path[b, j]), lens[b] + j
            sp, dp = int(table[b, src // page]), int(table[b, dst // page])
            for i, t in enumerate(want):
                if i < 2:
                    t[:, dp, dst % page] = old[i][:, sp, src % page]
                else:
                    t[:, dp, :, dst % page] = old[i][:, sp, :, src % page]
    result = {"accepted_len": acc, "path": path}
    ws = sv.Workspace(dev, 256)
    new = sv.cache_commit(cache, table, clen, result, workspace=ws)
    assert new.tolist() == [n + int(a) + 1 for n, a in zip(lens, acc)]
    assert clen.tolist() == lens
    now = snapshot(cache)
    for t, w in zip(now, want):
        assert torch.equal(bits(t if layers else t[None]), bits(w))
    # a chain moves nothing, and the lengths may be updated in place
    acc2 = torch.zeros_like(acc) + 3
    sv.cache_commit(cache, table, new, {"accepted_len": acc2}, new_len=new, workspace=ws)
    cap = table.shape[1] * page
    assert new.tolist() == [min(cap, n + int(a) + 1 + 4) for n, a in zip(lens, acc)]
    for t, w in zip(snapshot(cache), now):
        assert torch.equal(bits(t), bits(w))


def test_cache_commit_in_place_lengths_and_bad_entries(dev):
    lens, N, page = [8, 8, 100], 6, 16
    cache, table, clen = make(lens, N, page, 2, 64, T["bf16"])
    table = table[:, :7].contiguous()  # 112 places
    table[1, 0] = -5  # positions 8..15 of sequence 1 have no page
    path = torch.tensor([[0, 2, 1, 99, 5, -1], [0, 3, 4, 5, -1, -1], [0, 2, 3, 5, -1, -1]], dtype=torch.int32,
                        device=dev)
    acc = torch.tensor([4, 3, 9], dtype=torch.int32, device=dev)  # 9 > N - 1 reads as 5
    before = snapshot(cache)
    ws = sv.Workspace(dev, 256)
    got = sv.cache_commit(cache, table, clen, {"accepted_len": acc, "path": path}, new_len=clen, workspace=ws)
    assert got is clen and clen.tolist() == [13, 12, 106]
    assert ws.device_status() == sv.SV_FLAG_INVALID_TREE | sv.SV_FLAG_INVALID_PAGE
    k = before[0]
    at = lambda t, b, p: t[int(table[b, p // page]), p % page]  # noqa: E731
    assert torch.equal(at(cache.k, 0, 9), at(k, 0, 10))      # 2 -> 1
    assert torch.equal(at(cache.k, 0, 10), at(k, 0, 10))     # 1 < 2: not moved
    assert torch.equal(at(cache.k, 0, 11), at(k, 0, 11))     # 99: not moved
    assert torch.equal(at(cache.k, 0, 12), at(k, 0, 13))     # 5 -> 4
    assert torch.equal(bits(cache.k[-5 % cache.k.shape[0]]), bits(k[-5 % cache.k.shape[0]]))
    assert torch.equal(at(cache.k, 2, 101), at(k, 2, 102)) and torch.equal(at(cache.k, 2, 103), at(k, 2, 105))
    # a sequence that runs past the capacity stops there
    clen.fill_(110)
    sv.cache_commit(cache, table, clen, {"accepted_len": acc}, new_len=clen, workspace=ws)
    assert clen.tolist() == [112, 112, 112] and ws.device_status() == sv.SV_FLAG_CAPACITY


# --------------------------------------------------------------- attention

def check_attention(q, cache, table, clen, parent=None, count=None, scale=None, workspace=None):
    """The bound, term by term: the output's own rounding; the weights' rounding
    (u of the queries' type, plus 2^-25 of the largest weight where a 16-bit
    float is subnormal); twice the scores' error in the
    exponent (head_dim + 16 roundings of 32 bits with truncating adds, and the
    exponential's 2^-21); 32-bit sums over the tokens."""
    got = sv.tree_attention(q, cache, table, clen, parent, count=count, scale=scale, lse=True, workspace=workspace)
    torch.cuda.synchronize()
    want, lse, wabs, smax = ref.attention(q.cpu(), cache, table.cpu(), clen.tolist(),
                                          None if parent is None else parent.cpu(),
                                          None if count is None else count.tolist(), scale)
    D, n = q.shape[-1], max(1, int(clen.max())) + q.shape[1]
    coded = cache.k.dtype == torch.float8_e4m3fn
    # 8-bit pools: a weight in [2^e, 2^(e+1)) enters as terms of 4 significant
    # bits.  The first leaves a remainder below 2^(e-3), which the second rounds
    # with a step of at most 2^(e-7): half of that is 2^-8 of the weight, u of
    # bfloat16.  Of the second's remainder, below 2^(e-7), a third (for 16-bit
    # floats) leaves half a step of 2^(e-11): 2^-12, under u of float16.
    uw = u(q.dtype)
    score = smax * (D + 16) * 2.0 ** -23
    if coded:
        # q's terms: its row is scaled so that the largest element lies in [2^7, 2^8),
        # and the smallest codes are 2^-9 apart, so an element is off by at most 2^-10,
        # 2^-17 of the largest, and a score by that times the sum of |k|.
        k = torch.nan_to_num(cache.k.float()) * torch.nan_to_num(cache.k_scale).transpose(1, 2)[..., None]
        score = score + abs(D ** -0.5 if scale is None else scale) * 2.0 ** -17 * \
            q.double().cpu().abs().amax(-1) * k.abs().sum(-1).max().item()
    tiny = 0.0
    if coded or q.dtype == torch.float16:
        top = 448.0 * torch.nan_to_num(cache.v_scale).max().item() * 2 if coded else \
            torch.nan_to_num(cache.v.float(), 0, 0, 0).abs().max().item()
        tiny = n * 2.0 ** -25 * top
    tol = u(q.dtype) * want.abs() + (uw + 2 * (score + 2.0 ** -21) + n * 2.0 ** -23)[..., None] * \
        (1 + 2 * uw) * wabs + tiny + (2.0 ** -25 if q.dtype == torch.float16 else 0.0)
    close(got["out"], want, torch.nan_to_num(tol), "out")
    close(got["lse"], lse, torch.nan_to_num(score + n * 2.0 ** -23 + 2.0 ** -20 * (1 + lse.abs()), posinf=0.0), "lse")
    return got


ATTENTION = [
    # lens, N, page, Hkv, G, D, layout, tree
    ([0], 1, 16, 1, 1, 64, "hnd", False),
    ([0, 1, 2], 3, 16, 2, 2, 64, "hnd", True),
    ([500], 5, 16, 8, 4, 64, "hnd", False),
    ([122, 123, 124, 127, 128, 129], 5, 16, 1, 4, 128, "nhd", False),
    ([63, 64, 65, 200], 64, 64, 2, 1, 128, "hnd", True),
    ([300, 0, 77], 64, 32, 1, 8, 128, "hnd", True),
    ([1000], 64, 128, 2, 3, 64, "hnd", False),
    ([40, 700], 37, 8, 2, 5, 80, "nhd", True),
    ([250], 9, 256, 2, 16, 96, "hnd", True),
    ([90, 31], 26, 48, 1, 7, 112, "hnd", True),
    ([77, 5], 6, 12, 2, 2, 66, "padded", True),
    ([50], 4, 1, 1, 3, 40, "nhd", False),
    ([150, 20], 8, 16, 1, 2, 256, "hnd", True),
    ([4100, 15], 7, 64, 1, 2, 128, "hnd", False),
    ([200], 2, 16, 1, 64, 128, "hnd", False),
    ([33], 3, 24, 1, 100, 32, "hnd", False),
    ([260], 1, 16, 3, 1, 16, "hnd", False),
]


@pytest.mark.parametrize("qt,kv", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3"), ("fp16", "e4m3")])
@pytest.mark.parametrize("case", range(len(ATTENTION)))
def test_tree_attention(dev, qt, kv, case):
    lens, N, page, Hkv, G, D, layout, tree = ATTENTION[case]
    cache, table, clen = make(lens, N, page, Hkv, D, T[kv], layout, seed=case)
    g = torch.Generator().manual_seed(case)
    q = torch.randn(len(lens), N, Hkv * G, D, generator=g).to(T[qt]).to(dev)
    check_attention(q, cache, table, clen, trees(len(lens), N, case) if tree else None)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("page,D,layout", [(16, 128, "hnd"), (12, 72, "padded")])
def test_tree_attention_padding_bad_trees_pages_and_capacity(dev, kv, page, D, layout):
    lens, N = [150, 20, 0, 40, 30, 9], 12
    cache, table, clen = make(lens, N, page, 2, D, T[kv], layout)
    parent = trees(6, N, 2, bad=[(0, 1, 1), (0, 6, -1), (1, 4, 77), (5, 3, -2)])
    count = torch.tensor([12, 7, 0, -4, 50, 1], dtype=torch.int32, device=dev)
    table[0, 2] = cache.k.shape[0] + 3  # a page of the context is missing
    q = torch.randn(6, N, 6, D, device=dev).to(torch.bfloat16)
    ws = sv.Workspace(dev, 256)
    got = check_attention(q, cache, table, clen, parent, count, workspace=ws)
    assert ws.device_status() == sv.SV_FLAG_INVALID_PAGE | sv.SV_FLAG_INVALID_TREE
    for b, n in enumerate((12, 7, 0, 0, 12, 1)):
        assert (got["out"][b, n:] == 0).all() and (got["lse"][b, n:] == -math.inf).all()
    # the last tokens of the tree have no place
    short = table[:, :-(-150 // page)].contiguous()
    check_attention(q, cache, short, clen, None, None, workspace=ws)
    assert ws.device_status() & sv.SV_FLAG_CAPACITY
    # every page is missing: rows see nothing
    gone = torch.full_like(table, -1)
    got = sv.tree_attention(q, cache, gone, clen, parent, lse=True, workspace=ws)
    assert (got["out"] == 0).all() and (got["lse"] == -math.inf).all()


@pytest.mark.parametrize("qt,kv", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3")])
def test_tree_attention_ignores_what_masked_places_hold(dev, qt, kv):
    """A node's infinities and NaN reach its own descendants only."""
    lens, N, D = [100, 126, 130], 6, 64
    cache, table, clen = make(lens, N, 16, 2, D, T[kv])
    parent = torch.tensor([[0, 0, 0, 1, 2, 2]] * 3, dtype=torch.int32, device=dev)
    q = torch.randn(3, N, 4, D, device=dev).to(T[qt])
    clean = check_attention(q, cache, table, clen, parent)
    for b, n in enumerate(lens):
        for j, kk, vv in ((1, 0.5, math.inf), (4, math.nan, math.nan)):
            k, v = torch.full((1, 2, D), 0.5), torch.full((1, 2, D), 0.25)
            if kk != kk:
                k[0, 0, 3] = kk
            v[0, 0, 5] = vv
            fill(cache, table, b, [n + j], k, v)
    got = check_attention(q, cache, table, clen, parent)
    for j in (0, 2, 5):  # their paths do not meet nodes 1 and 4
        assert torch.equal(got["out"][:, j], clean["out"][:, j])
    # the context's reach everyone
    fill(cache, table, 1, [3], torch.full((1, 2, D), 0.5), torch.full((1, 2, D), math.nan))
    got = sv.tree_attention(q, cache, table, clen, parent)["out"]
    assert torch.isnan(got[1]).all() and torch.isfinite(got[0, 0]).all()


@pytest.mark.parametrize("qt,kv", [("bf16", "bf16"), ("fp16", "e4m3")])
def test_tree_attention_extreme_scores(dev, qt, kv):
    """Scores whose maximum grows along the cache, huge ones, a zero scale, a
    negative scale, and queries at the ends of their type's range."""
    lens, N, D = [600], 4, 64
    cache, table, clen = make(lens, N, 16, 1, D, T[kv], spread=0.1)
    g = torch.Generator().manual_seed(9)
    ramp = torch.linspace(0.1, 30, 604)[:, None, None] * torch.randn(1, 1, D, generator=g).sign()
    fill(cache, table, 0, range(604), ramp * torch.ones(604, 1, D), torch.randn(604, 1, D, generator=g) * 3)
    base = ramp[-1:, :, :].sign()[None].expand(1, N, 2, D)
    for size in (1.0, 0.01, -1.0, 100.0):
        q = (base * size + 0.01 * torch.randn(1, N, 2, D, generator=g)).to(T[qt]).to(dev)
        check_attention(q, cache, table, clen)
    check_attention(q, cache, table, clen, scale=0.0)
    check_attention(q, cache, table, clen, scale=-0.01)
    top = torch.finfo(T[qt]).max
    q = torch.randn(1, N, 2, D, generator=g)
    check_attention((q * (top / 16 if qt == "fp16" else 1e30)).to(T[qt]).to(dev), cache, table, clen,
                    scale=1e-6 if qt == "fp16" else 1e-31)
    check_attention((q * torch.finfo(T[qt]).tiny).to(T[qt]).to(dev), cache, table, clen, scale=1.0)


def test_tree_attention_scales_far_apart(dev):
    """8-bit rows whose scales differ by many orders of magnitude."""
    lens, N, D = [300, 30], 5, 128
    cache, table, clen = make(lens, N, 16, 1, D, T["e4m3"])
    g = torch.Generator().manual_seed(3)
    for b, n in enumerate(lens):
        size = 10.0 ** torch.linspace(-12, 3, n + N)[torch.randperm(n + N, generator=g)]
        fill(cache, table, b, range(n + N), torch.randn(n + N, 1, D, generator=g),
             torch.randn(n + N, 1, D, generator=g) * size[:, None, None])
    q = torch.randn(2, N, 4, D, generator=g).to(torch.bfloat16).to(dev)
    check_attention(q, cache, table, clen)


def test_tree_attention_is_the_same_every_time(dev):
    """No result depends on the order in which blocks finish."""
    cache, table, clen = make([3000, 17, 900], 26, 16, 2, 128, T["bf16"])
    q = torch.randn(3, 26, 8, 128, device=dev).to(torch.bfloat16)
    parent = trees(3, 26, 1)
    first = sv.tree_attention(q, cache, table, clen, parent)["out"]
    for _ in range(20):
        assert torch.equal(first, sv.tree_attention(q, cache, table, clen, parent)["out"])


def test_tree_attention_strided_queries(dev):
    cache, table, clen = make([70, 200], 4, 16, 2, 64, T["bf16"])
    fused = torch.randn(2, 4, 12, 64, device=dev).to(torch.bfloat16)
    q = fused[:, :, 2:8]
    want = sv.tree_attention(q.contiguous(), cache, table, clen)["out"]
    assert torch.equal(want, sv.tree_attention(q, cache, table, clen)["out"])
    odd = torch.empty(2 * 4 * 6 * 64 + 1, dtype=torch.bfloat16, device=dev)[1:].view(2, 4, 6, 64)
    odd.copy_(q)  # rows on 2-byte boundaries only
    assert torch.equal(want, sv.tree_attention(odd, cache, table, clen)["out"])


def test_tree_attention_far_in_a_large_pool(dev):
    """Pool offsets past 2^31 elements and past 2^32 bytes."""
    page, H, D = 64, 8, 128
    pages = 2 ** 31 // (page * H * D) + 40
    k = torch.zeros(pages, H, page, D, dtype=torch.bfloat16, device=dev).transpose(1, 2)
    v = torch.zeros(pages, H, page, D, dtype=torch.bfloat16, device=dev).transpose(1, 2)
    cache = sv.KVCache(k, v)
    table = torch.arange(pages - 5, pages, dtype=torch.int32, device=dev)[None].contiguous()
    clen = torch.tensor([200], dtype=torch.int32, device=dev)
    x, y = (torch.randn(1, 205, H, D, device=dev).to(torch.bfloat16) for _ in range(2))
    zero = torch.zeros_like(clen)
    sv.cache_write(cache, table, zero, x, y)
    small = sv.KVCache(k[-5:].clone(), v[-5:].clone())
    near = torch.arange(5, dtype=torch.int32, device=dev)[None].contiguous()
    q = torch.randn(1, 5, 16, D, device=dev).to(torch.bfloat16)
    a = sv.tree_attention(q, cache, table, clen)["out"]
    assert torch.equal(a, sv.tree_attention(q, small, near, clen)["out"])
    offs = torch.tensor([0, 205], dtype=torch.int32, device=dev)
    got = sv.cache_read(cache, table, offs, 205)
    assert torch.equal(got["k"], x[0]) and torch.equal(got["v"], y[0])
    path = torch.tensor([[0, 3, 4, -1, -1]], dtype=torch.int32, device=dev)
    new = sv.cache_commit(cache, table, clen, {"accepted_len": zero + 2, "path": path})
    got = sv.cache_read(cache, table, offs, 205)
    assert new.tolist() == [203]
    assert torch.equal(got["k"][201], x[0, 203]) and torch.equal(got["v"][202], y[0, 204])


# ------------------------------------------------------- streams and graphs

def test_other_stream_and_captured_graphs(dev):
    """A call on another stream, and two captured graphs replayed on two
    streams at once, give what eager calls give."""
    sets = []
    for seed in (1, 2):
        cache, table, clen = make([700, 90], 6, 16, 2, 128, T["e4m3"], seed=seed)
        g = torch.Generator().manual_seed(seed)
        q, k, v = (torch.randn(2, 6, h, 128, generator=g).to(torch.bfloat16).to(dev) for h in (8, 2, 2))
        sets.append((cache, table, clen, q, k, v, trees(2, 6, seed)))
    rope = sv.rotary_frequencies(128, device=dev)

    def step(s, **kw):
        cache, table, clen, q, k, v, parent = s
        turned = sv.cache_write(cache, table, clen, k, v, parent=parent, rope=rope, q=q, **kw)
        return sv.tree_attention(turned, cache, table, clen, parent, **kw)["out"]

    want = [step(s).clone() for s in sets]
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    got = step(sets[0], stream=other)
    torch.cuda.synchronize()
    assert torch.equal(got, want[0])
    with torch.cuda.stream(other):
        got = step(sets[1])
    torch.cuda.synchronize()
    assert torch.equal(got, want[1])
    graphs, outs = [], []
    for s in sets:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(step(s))
        graphs.append(gr)
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(50):
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


# -------------------------------------------------- a step with all of them

@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_decoding_steps_with_all_of_them(dev, kv):
    """Three verify steps of a one-layer model: write, attention, logits,
    tree verify, cache and token commits.  After each, the cache holds what a
    chain write of the committed tokens alone holds, bit for bit."""
    B, N, Hkv, G, D, V, page = 4, 10, 2, 4, 64, 50, 16
    g = torch.Generator("cuda").manual_seed(0)
    emb = torch.randn(V, Hkv * G * D, device=dev, generator=g)
    wk, wv = (torch.randn(V, Hkv, D, device=dev, generator=g).to(torch.bfloat16) for _ in range(2))
    head = torch.randn(Hkv * G * D, V, device=dev, generator=g)
    rope = sv.rotary_frequencies(D, device=dev)
    cache, plain = (sv.KVCache.empty(B * 4, page, Hkv, D, T[kv]) for _ in range(2))
    table = torch.arange(B * 4, dtype=torch.int32, device=dev).view(B, 4)
    clen = torch.zeros(B, dtype=torch.int32, device=dev)
    seq = torch.ones(B, dtype=torch.int32, device=dev)
    buf = torch.zeros(B, 64, dtype=torch.int32, device=dev)
    buf[:, 0] = torch.arange(B)
    nxt = buf[:, 0].clone()
    for s in range(3):
        parent = trees(B, N, s)
        tok = torch.randint(0, V, (B, N), device=dev, dtype=torch.int32, generator=g)
        tok[:, 0] = nxt
        for it in range(2):  # a second pass after the drafts are set to the argmax of their parents
            q = emb[tok.long()].view(B, N, Hkv * G, D).to(torch.bfloat16)
            turned = sv.cache_write(cache, table, clen, wk[tok.long()], wv[tok.long()], parent=parent, rope=rope, q=q)
            out = sv.tree_attention(turned, cache, table, clen, parent)["out"]
            logits = (out.float().view(B, N, -1) @ head).contiguous()
            if it == 0:
                best = logits.argmax(-1).int()
                for b in range(B):
                    tok[b, 1:4] = best[b, parent[b, 1:4].long()]
        res = sv.tree_greedy(logits, parent, tok)
        clen = sv.cache_commit(cache, table, clen, res)
        sv.commit(res, seq, buf, next_input=nxt)
        assert torch.equal(clen + 1, seq)
        n = int(clen.max())
        toks = buf[:, :n].long()
        sv.cache_write(plain, table, torch.zeros_like(clen), wk[toks], wv[toks], count=clen, rope=rope)
        offs = torch.zeros(B + 1, dtype=torch.int32, device=dev)
        offs[1:] = clen.cumsum(0)
        a, c = (sv.cache_read(x, table, offs, int(offs[-1])) for x in (cache, plain))
        assert torch.equal(a["k"], c["k"]) and torch.equal(a["v"], c["v"])
    assert int(clen.max()) > 3  # some drafts were accepted
