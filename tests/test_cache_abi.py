"""Cache-side calls without a GPU: what the host refuses, and the rotary
frequencies against their formulas."""
import ctypes
import math

import pytest
import torch

import speculative_decoding_verification_88_b200 as sv
from speculative_decoding_verification_88_b200 import build as svbuild

OK, INVALID, MISALIGNED, WORKSPACE = 0, 1, 2, 3

# Host memory stands in for device memory: every call below is refused, or
# has nothing to do, before any CUDA call.
BUF = (ctypes.c_uint8 * 4096)()
A = (ctypes.addressof(BUF) + 255) // 256 * 256


@pytest.fixture(scope="module")
def lib():
    svbuild.build()
    return sv.load_library()


def cache(**kw):
    f = dict(k=A, v=A, k_scale=None, v_scale=None, dtype=sv.SV_BF16, num_pages=4, page_size=16,
             num_heads=2, head_dim=64, page_stride=2048, token_stride=128, head_stride=64,
             num_layers=1, layer_stride=0, scale_layer_stride=0)
    f.update(kw)
    return sv._Cache(*f.values())


def rope(**kw):
    f = dict(inv_freq=A, rotary_dim=64, interleaved=0, magnitude=1.0)
    f.update(kw)
    return sv._Rotary(*f.values())


ROWS = sv._Rows(A, 512, 128, 64)

# what every cache call refuses in the pool and the table
BAD_CACHES = [dict(k=None), dict(v=None), dict(dtype=7), dict(num_pages=0), dict(page_size=0),
              dict(num_heads=0), dict(num_heads=1025), dict(head_dim=0), dict(head_dim=257),
              dict(num_layers=0), dict(page_stride=-1), dict(token_stride=-1),
              dict(head_stride=-1), dict(layer_stride=-1), dict(k_scale=A), dict(v_scale=A),
              dict(dtype=sv.SV_E4M3), dict(dtype=sv.SV_E4M3, k_scale=A)]


def call(lib, name, **kw):
    a = CALLS[name].copy()
    a.update(kw)
    return getattr(lib, "spec_verify_" + name)(*a.values())


CALLS = {
    "rotary": dict(x=A, dtype=1, xt=128, xh=64, pos=A, rope=rope(), inv=0, T=3, H=2, D=64, out=A,
                   ot=128, oh=64, st=None),
    "cache_write": dict(c=cache(), table=A, ts=4, mp=4, lens=A, par=None, cnt=None, k=ROWS, v=ROWS,
                        dtype=1, B=2, N=3, rope=rope(), q=ROWS, Hq=4, qo=A, ws=None, st=None),
    "cache_read": dict(c=cache(), table=A, ts=4, mp=4, offs=A, start=None, B=2, total=5, ko=A, vo=A,
                       dtype=1, ws=None, st=None),
    "tree_attention": dict(q=ROWS, dtype=1, c=cache(), table=A, ts=4, mp=4, lens=A, par=A, cnt=None,
                           B=2, N=3, Hq=4, scale=0.125, out=A, lse=None, ws=None, scratch=A,
                           sb=1 << 40, st=None),
    "cache_commit": dict(c=cache(), table=A, ts=4, mp=4, lens=A, acc=A, path=A, B=2, N=3, new=A,
                         ws=None, st=None),
}


@pytest.mark.parametrize("name", ["cache_write", "cache_read", "tree_attention", "cache_commit"])
def test_bad_pools_and_tables_are_refused(lib, name):
    for bad in BAD_CACHES:
        assert call(lib, name, c=cache(**bad)) == INVALID, bad
    assert call(lib, name, c=None) == INVALID
    assert call(lib, name, table=None) == INVALID
    assert call(lib, name, ts=-1) == INVALID
    assert call(lib, name, mp=0) == INVALID
    assert call(lib, name, B=-1) == INVALID
    assert call(lib, name, B=65536) == INVALID
    assert call(lib, name, B=0, c=None, table=None) == OK
    assert call(lib, name, c=cache(k=A + 1)) == MISALIGNED
    assert call(lib, name, table=A + 2) == MISALIGNED
    assert call(lib, name, ws=A + 4) == MISALIGNED


def test_rotary_refusals(lib):
    for bad in (dict(dtype=3), dict(dtype=-1), dict(T=-1), dict(T=1 << 31), dict(H=0), dict(H=1025),
                dict(D=1), dict(D=513), dict(xt=-1), dict(oh=-1), dict(x=None), dict(out=None),
                dict(pos=None), dict(rope=None), dict(rope=rope(inv_freq=None)),
                dict(rope=rope(rotary_dim=0)), dict(rope=rope(rotary_dim=63)),
                dict(rope=rope(rotary_dim=66)), dict(rope=rope(magnitude=math.inf))):
        assert call(lib, "rotary", **bad) == INVALID, bad
    for bad in (dict(x=A + 1), dict(out=A + 1), dict(pos=A + 2), dict(rope=rope(inv_freq=A + 4))):
        assert call(lib, "rotary", **bad) == MISALIGNED, bad
    assert call(lib, "rotary", T=0, x=None) == OK


def test_cache_write_refusals(lib):
    null = sv._Rows(None, 0, 0, 0)
    back = sv._Rows(A, -1, 0, 0)
    for bad in (dict(dtype=3), dict(dtype=0), dict(dtype=2), dict(N=-1), dict(par=A, N=65),
                dict(lens=None), dict(k=None), dict(v=None), dict(k=null), dict(v=back),
                dict(rope=None), dict(q=null), dict(qo=None), dict(Hq=0),
                dict(rope=rope(rotary_dim=128))):
        assert call(lib, "cache_write", **bad) == INVALID, bad
    odd = sv._Rows(A + 1, 512, 128, 64)
    for bad in (dict(k=odd), dict(v=odd), dict(q=odd), dict(qo=A + 1), dict(lens=A + 2),
                dict(par=A + 1), dict(cnt=A + 3)):
        assert call(lib, "cache_write", **bad) == MISALIGNED, bad
    assert call(lib, "cache_write", N=0, k=None) == OK


def test_cache_read_refusals(lib):
    for bad in (dict(dtype=3), dict(total=-1), dict(total=1 << 31), dict(offs=None), dict(ko=None),
                dict(vo=None)):
        assert call(lib, "cache_read", **bad) == INVALID, bad
    for bad in (dict(offs=A + 1), dict(start=A + 2), dict(ko=A + 1), dict(vo=A + 1)):
        assert call(lib, "cache_read", **bad) == MISALIGNED, bad
    assert call(lib, "cache_read", total=0, offs=None) == OK


def test_tree_attention_refusals(lib):
    for bad in (dict(dtype=0), dict(dtype=3), dict(dtype=2), dict(N=0), dict(N=65), dict(Hq=0),
                dict(Hq=3), dict(Hq=1026), dict(scale=math.nan), dict(scale=math.inf), dict(q=None),
                dict(lens=None), dict(out=None), dict(scratch=None),
                dict(q=sv._Rows(A, 0, -1, 0)), dict(c=cache(dtype=sv.SV_F32))):
        assert call(lib, "tree_attention", **bad) == INVALID, bad
    for bad in (dict(out=A + 1), dict(lse=A + 2), dict(par=A + 2), dict(lens=A + 1), dict(cnt=A + 2),
                dict(scratch=A + 8), dict(q=sv._Rows(A + 1, 512, 128, 64))):
        assert call(lib, "tree_attention", **bad) == MISALIGNED, bad
    assert call(lib, "tree_attention", sb=0) == WORKSPACE


def test_tree_attention_scratch_size_limits(lib):
    size = lib.spec_verify_tree_attention_scratch_size
    assert size(4, 26, 32, 8, 128) > 0
    assert size(0, 1, 1, 1, 64) > 0
    for bad in ((-1, 1, 1, 1, 64), (65536, 1, 1, 1, 64), (1, 0, 1, 1, 64), (1, 65, 1, 1, 64),
                (1, 1, 3, 2, 64), (1, 1, 1, 0, 64), (1, 1, 1, 1, 0), (1, 1, 1, 1, 257)):
        assert size(*bad) == 0, bad


def test_status_refusals(lib):
    assert lib.spec_verify_cache_read_device_status(None, 0, None) == INVALID


def test_cache_commit_refusals(lib):
    for bad in (dict(N=0), dict(N=65), dict(lens=None), dict(acc=None), dict(new=None)):
        assert call(lib, "cache_commit", **bad) == INVALID, bad
    for bad in (dict(lens=A + 1), dict(acc=A + 2), dict(path=A + 2), dict(new=A + 1)):
        assert call(lib, "cache_commit", **bad) == MISALIGNED, bad


def frequencies(lib, rd, base=10000.0, kind=0, factor=1.0, L=0.0, low=1.0, high=4.0):
    out = (ctypes.c_double * max(1, rd // 2))()
    mag = ctypes.c_float(-1)
    rc = lib.spec_verify_rotary_frequencies(ctypes.addressof(out), ctypes.addressof(mag), rd, base,
                                            kind, factor, L, low, high)
    return rc, list(out), mag.value


@pytest.mark.parametrize("rd,base", [(2, 10000.0), (64, 10000.0), (128, 500000.0), (512, 2.0)])
def test_rotary_frequencies_plain_and_linear(lib, rd, base):
    want = [base ** (-2 * i / rd) for i in range(rd // 2)]
    # pow and one division, each within a few 2^-53
    rc, got, mag = frequencies(lib, rd, base)
    assert rc == OK and mag == 1.0
    assert got == pytest.approx(want, rel=1e-15)
    rc, got, mag = frequencies(lib, rd, base, 1, 8.0)
    assert rc == OK and mag == 1.0
    assert got == pytest.approx([f / 8 for f in want], rel=1e-15)


def test_rotary_frequencies_bands(lib):
    rd, base, factor, L, low, high = 128, 500000.0, 8.0, 8192.0, 1.0, 4.0
    _, got, mag = frequencies(lib, rd, base, 2, factor, L, low, high)
    assert mag == 1.0
    kinds = set()
    for i, g in enumerate(got):
        f = base ** (-2 * i / rd)
        w = 2 * math.pi / f
        if L / w > high:
            want, kind = f, "keep"
        elif L / w < low:
            want, kind = f / factor, "scaled"
        else:
            s = (L / w - low) / (high - low)
            want, kind = (1 - s) * f / factor + s * f, "between"
        kinds.add(kind)
        assert g == pytest.approx(want, rel=1e-14)
    assert kinds == {"keep", "scaled", "between"}


def test_rotary_frequencies_yarn(lib):
    rd, base, factor, L, slow, fast = 128, 10000.0, 16.0, 4096.0, 1.0, 32.0
    _, got, mag = frequencies(lib, rd, base, 3, factor, L, slow, fast)
    assert mag == pytest.approx(0.1 * math.log(factor) + 1, rel=2.0 ** -23)
    turns = lambda r: rd * math.log(L / (r * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
    lo, hi = max(0, math.floor(turns(fast))), min(rd - 1, math.ceil(turns(slow)))
    for i, g in enumerate(got):
        f = base ** (-2 * i / rd)
        ramp = min(1.0, max(0.0, (i - lo) / (hi - lo)))
        assert g == pytest.approx(f * (1 - ramp) + f / factor * ramp, rel=1e-14)
    assert got[0] == 1.0 and got[-1] < 10000.0 ** (-126 / 128) * 1.0001 / 16


def test_rotary_frequency_refusals(lib):
    for bad in (dict(rd=0), dict(rd=3), dict(rd=514), dict(rd=64, base=1.0), dict(rd=64, base=math.nan),
                dict(rd=64, kind=4), dict(rd=64, kind=-1), dict(rd=64, kind=1, factor=0.5),
                dict(rd=64, kind=2, factor=2.0, L=0.0), dict(rd=64, kind=2, factor=2.0, L=10.0, low=4.0),
                dict(rd=64, kind=3, factor=2.0, L=10.0, low=0.0)):
        assert frequencies(lib, **bad)[0] == INVALID, bad
    with pytest.raises(sv.SpecVerifyError):
        sv.rotary_frequencies(63, device="cpu")
    with pytest.raises(ValueError):
        sv.rotary_frequencies(64, scaling="other", device="cpu")


def test_bindings_refuse_cpu_tensors():
    t = torch.zeros(2, 16, 2, 64)
    with pytest.raises(TypeError):
        sv.KVCache(t, t)
    with pytest.raises(TypeError):
        sv.Rotary(torch.zeros(32, dtype=torch.float64))
    with pytest.raises(TypeError):
        sv.rotary(t, torch.zeros(2, 16, dtype=torch.int32), None)


def test_cache_commit_refuses_overlapping_lengths(lib):
    """new_len may be cache_len or accepted_len, and overlaps nothing otherwise."""
    apart = dict(lens=A, acc=A + 64, path=A + 128, new=A + 256)
    for bad in (dict(new=A + 4), dict(new=A - 4), dict(new=A + 60), dict(new=A + 68), dict(new=A + 128),
                dict(new=A + 128 + 4 * 5)):
        assert call(lib, "cache_commit", **{**apart, **bad}) == INVALID, bad
    assert call(lib, "cache_commit", **{**apart, "new": A + 4, "path": None}) == INVALID


def test_a_workspace_of_another_device_is_refused():
    """Kernels write their flags there: only memory of the call's device will do."""
    class Elsewhere:
        buf = torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError):
        sv._status(Elsewhere, torch.device("cuda:0"), None)
    assert sv._status(Elsewhere, torch.device("cpu"), None) == Elsewhere.buf.data_ptr()
    assert sv._status(None, torch.device("cuda:0"), None) is None
