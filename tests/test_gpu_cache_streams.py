"""Cache-side calls given a stream that is not the current one: what the call
itself allocates and clears belongs to that stream."""
import pytest
import torch

import speculative_decoding_verification_88_b200 as sv
from speculative_decoding_verification_88_b200 import build as svbuild

from test_gpu_cache import T, make, trees
from test_gpu_cache_use import heads

pytestmark = pytest.mark.gpu

BUSY = 200_000_000  # clock cycles: 0.1 s, against the microseconds of the calls


@pytest.fixture(scope="module", autouse=True)
def built():
    svbuild.build()


@pytest.fixture
def dev():
    return torch.device("cuda:0")


def test_padded_write_on_another_stream_keeps_its_queries(dev):
    cache, table, clen = make([20, 3], 6, 16, 2, 64, T["bf16"])
    q, k, v = (heads(2, 6, h, 64, T["bf16"], h) for h in (4, 2, 2))
    count = torch.tensor([6, 2], dtype=torch.int32, device=dev)
    rope = sv.rotary_frequencies(64, device=dev)
    want = sv.cache_write(cache, table, clen, k, v, count=count, rope=rope, q=q)
    assert (want[1, 2:] == 0).all()
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)  # on the current stream, which the call is not given
    got = sv.cache_write(cache, table, clen, k, v, count=count, rope=rope, q=q, stream=other)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("call", ["rotary", "read", "attention", "commit", "write", "workspace"])
def test_results_on_another_stream_take_no_memory_that_is_still_read(dev, call):
    """A block that the current stream has yet to read is not handed out on
    another one, for a result, for scratch or for a new workspace."""
    cache, table, clen = make([60, 40], 6, 16, 2, 64, T["bf16"])
    q, k, v = (heads(2, 6, h, 64, T["bf16"], h) for h in (4, 2, 2))
    rope = sv.rotary_frequencies(64, device=dev)
    pos = torch.arange(12, dtype=torch.int32, device=dev).view(2, 6)
    offs = torch.tensor([0, 60, 100], dtype=torch.int32, device=dev)
    path = torch.tensor([[0, 2, 4, -1, -1, -1]] * 2, dtype=torch.int32, device=dev)
    result = {"accepted_len": torch.full_like(clen, 2), "path": path}
    parent = trees(2, 6, 1)
    ws = sv.Workspace(dev, 256)

    def run(**kw):
        if call == "rotary":
            return [sv.rotary(q, pos, rope, **kw)]
        if call == "read":
            return list(sv.cache_read(cache, table, offs, 100, workspace=ws, **kw).values())
        if call == "attention":
            return list(sv.tree_attention(q, cache, table, clen, parent, lse=True, workspace=ws, **kw).values())
        if call == "commit":
            return [sv.cache_commit(cache, table, clen, result, workspace=ws, **kw)]
        if call == "workspace":  # made by the call
            return list(sv.cache_read(cache, table, offs, 100, workspace=sv.Workspace(dev), **kw).values())
        return [sv.cache_write(cache, table, clen, k, v, rope=rope, q=q, workspace=ws, **kw)]

    want = run()
    sizes = [t.numel() * t.element_size() for t in want]
    if call == "attention":
        sizes.append(sv.load_library().spec_verify_tree_attention_scratch_size(2, 6, 4, 2, 64))
    if call == "workspace":
        sizes.append(256)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    held = [torch.full((n,), 7, dtype=torch.uint8, device=dev) for n in sizes for _ in range(4)]
    kept = [torch.zeros_like(t) for t in held]
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    for t, c in zip(held, kept):
        c.copy_(t)  # waits behind the sleep
    del held, t
    got = run(stream=other)
    torch.cuda.synchronize()
    assert all((c == 7).all() for c in kept), "written over before the current stream had read it"
    if call != "commit":  # (the path has moved rows once more)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    else:
        assert torch.equal(got[0], want[0])


def test_results_of_another_stream_may_be_dropped_while_read(dev):
    """A result used on the current stream, after a wait, and dropped there is
    not handed out again on the call's stream before that use is over."""
    q = heads(2, 6, 4, 64, T["bf16"], 1)
    rope = sv.rotary_frequencies(64, device=dev)
    pos = torch.arange(12, dtype=torch.int32, device=dev).view(2, 6)
    want = sv.rotary(q, pos, rope)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = sv.rotary(q, pos, rope, stream=other)
    torch.cuda.current_stream().wait_stream(other)
    kept = torch.zeros_like(want)
    torch.cuda._sleep(BUSY)
    kept.copy_(got)
    del got
    more = [sv.rotary(q * 2, pos, rope, stream=other) for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(kept, want) and len(more) == 4


def test_a_captured_step_with_a_second_stream(dev):
    """A graph whose calls run on a stream forked from the captured one, replayed
    on new contents, gives what eager calls give."""
    B, N = 2, 6
    cache, table, clen = make([90, 17], 64, 16, 2, 64, T["e4m3"])
    twin = sv.KVCache(*(x.clone() for x in (cache.k, cache.v, cache.k_scale, cache.v_scale)))
    q, k, v = (heads(B, N, h, 64, T["bf16"], h) for h in (4, 2, 2))
    count = torch.tensor([6, 3], dtype=torch.int32, device=dev)
    parent = trees(B, N, 1)
    rope = sv.rotary_frequencies(64, device=dev)
    other = torch.cuda.Stream()

    def step(c, stream):
        turned = sv.cache_write(c, table, clen, k, v, parent=parent, count=count, rope=rope, q=q, stream=stream)
        got = sv.tree_attention(turned, c, table, clen, parent, count=count, lse=True, stream=stream)
        return turned, got["out"], got["lse"]

    step(twin, None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        other.wait_stream(torch.cuda.current_stream())
        outs = step(cache, other)
        torch.cuda.current_stream().wait_stream(other)
        total = outs[1].float().sum()
    for s in range(4):
        q.copy_(heads(B, N, 4, 64, T["bf16"], 10 + s))
        k.copy_(heads(B, N, 2, 64, T["bf16"], 20 + s))
        count.copy_(torch.tensor([s + 1, 6 - s], dtype=torch.int32))
        graph.replay()
        want = step(twin, None)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        assert torch.equal(total, want[1].float().sum())


def test_a_workspace_that_grows_while_two_streams_use_it(dev):
    """The buffer that a larger one replaces is not handed out before both the
    given and the current stream are done with it."""
    other = torch.cuda.Stream()
    ws = sv.Workspace(dev)
    ws.ensure(4096, other)
    torch.cuda.synchronize()
    old = ws.buf.data_ptr()
    ws.buf.fill_(7)
    kept = torch.zeros_like(ws.buf)
    torch.cuda._sleep(BUSY)
    kept.copy_(ws.buf)
    ws.ensure(1 << 16, other)
    with torch.cuda.stream(other):
        more = [torch.zeros(4096, dtype=torch.uint8, device=dev) for _ in range(4)]
    torch.cuda.synchronize()
    assert (kept == 7).all() and old not in [t.data_ptr() for t in more]
