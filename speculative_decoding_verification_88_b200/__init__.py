"""speculative_decoding_verification_88_b200 -- verify-and-accept for
speculative decoding on B200 (sm_100a).

A thin ctypes binding over ``libspecverify.so`` (C ABI in
``include/spec_verify.h``).  PyTorch is used only for device memory and
streams: every step of the verify path runs in the library's CUDA kernels.
There is no CPU fallback; calls raise if the library or a CUDA device is
missing.

    import speculative_decoding_verification_88_b200 as sv
    r = sv.stochastic(target, draft, draft_tokens, temperature=0.7, seed=1)
    r["accepted_len"], r["out_tokens"]
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

from .build import LIB_PATH

SV_F32, SV_BF16, SV_F16, SV_E4M3 = 0, 1, 2, 3
SV_FLAG_INVALID_TOKEN, SV_FLAG_RESIDUAL_FALLBACK, SV_FLAG_TIMEOUT = 1, 2, 4
SV_FLAG_INVALID_ROW, SV_FLAG_CAPACITY, SV_FLAG_INVALID_TREE = 8, 16, 32
SV_FLAG_BOUNDS = 64  # raised by the bounds-checked build only
SV_FLAG_INVALID_PAGE = 128

# Entry points declared in include/spec_verify.h.
EXPORTS = (
    "spec_verify_workspace_size", "spec_verify_status_string", "spec_verify_workspace_init",
    "spec_verify_read_device_status", "spec_verify_stochastic", "spec_verify_greedy",
    "spec_verify_multi_candidate", "spec_verify_multi_candidate_rows", "spec_verify_commit",
    "spec_verify_tree_workspace_size", "spec_verify_tree_greedy", "spec_verify_threshold",
    "spec_verify_philox4x32_10", "spec_verify_greedy_noalloc",
    "spec_verify_greedy_noalloc_read_device_status",
    "spec_verify_tree_stochastic_workspace_size", "spec_verify_tree_stochastic",
    "spec_verify_kernel_launches",
    "spec_verify_rotary_frequencies", "spec_verify_rotary", "spec_verify_cache_write",
    "spec_verify_cache_read", "spec_verify_tree_attention_scratch_size",
    "spec_verify_tree_attention", "spec_verify_cache_commit",
    "spec_verify_cache_read_device_status",
)

_lib = None
_lock = threading.Lock()


class _Cache(ctypes.Structure):  # sv_kv_cache
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("dtype", ctypes.c_int), ("num_pages", ctypes.c_int),
                ("page_size", ctypes.c_int), ("num_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("page_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("num_layers", ctypes.c_int), ("layer_stride", ctypes.c_int64),
                ("scale_layer_stride", ctypes.c_int64)]


class _Rows(ctypes.Structure):  # sv_rows
    _fields_ = [("data", ctypes.c_void_p), ("stride_b", ctypes.c_int64),
                ("stride_n", ctypes.c_int64), ("stride_h", ctypes.c_int64)]


class _Rotary(ctypes.Structure):  # sv_rotary
    _fields_ = [("inv_freq", ctypes.c_void_p), ("rotary_dim", ctypes.c_int),
                ("interleaved", ctypes.c_int), ("magnitude", ctypes.c_float)]


class SpecVerifyError(RuntimeError):
    pass


def library_path() -> str:
    return LIB_PATH


def load_library(path: str | None = None):
    """Load libspecverify.so (raises if it has not been built).  `path` loads
    another build of the same library (the bounds-checked one) and returns it
    without making it the default."""
    global _lib
    if path is None and _lib is not None:
        return _lib
    with _lock:
        if path is None and _lib is not None:
            return _lib
        target = path or LIB_PATH
        if not os.path.exists(target):
            raise SpecVerifyError(
                f"{target} is missing: build it with "
                "`python -m speculative_decoding_verification_88_b200.build`")
        lib = ctypes.CDLL(target)
        P, I, I64, U32, U64, SZ, F = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64,
                                      ctypes.c_uint32, ctypes.c_uint64, ctypes.c_size_t,
                                      ctypes.c_float)
        lib.spec_verify_workspace_size.argtypes = [I, I, I, I]
        lib.spec_verify_workspace_size.restype = SZ
        lib.spec_verify_status_string.argtypes = [I]
        lib.spec_verify_status_string.restype = ctypes.c_char_p
        lib.spec_verify_workspace_init.argtypes = [P, SZ, P]
        lib.spec_verify_workspace_init.restype = I
        lib.spec_verify_read_device_status.argtypes = [P, ctypes.POINTER(U32), I, P]
        lib.spec_verify_read_device_status.restype = I
        lib.spec_verify_stochastic.argtypes = [
            P, I, I64, I64, P, I, I64, I64, P, I, I, I, F, U64, U32, P, P, P, P, SZ, P]
        lib.spec_verify_stochastic.restype = I
        lib.spec_verify_greedy.argtypes = [P, I, I64, I64, P, I, I, I, P, P, P, SZ, P]
        lib.spec_verify_greedy.restype = I
        lib.spec_verify_multi_candidate.argtypes = [
            P, I, I64, I64, I64, P, I, I, I, I, P, P, P, P, SZ, P]
        lib.spec_verify_multi_candidate.restype = I
        lib.spec_verify_multi_candidate_rows.argtypes = [
            P, I, I64, I64, P, P, I, I, I, I, I, P, P, P, P, SZ, P]
        lib.spec_verify_multi_candidate_rows.restype = I
        lib.spec_verify_commit.argtypes = [P, P, I, I, P, P, I64, I, P, P, P]
        lib.spec_verify_commit.restype = I
        lib.spec_verify_tree_workspace_size.argtypes = [I, I, I]
        lib.spec_verify_tree_workspace_size.restype = SZ
        lib.spec_verify_tree_greedy.argtypes = [P, I, I64, I64, P, P, I, I, I, P, P, P, P, SZ, P]
        lib.spec_verify_tree_greedy.restype = I
        lib.spec_verify_threshold.argtypes = [P, I, I64, I64, P, I, I, I, F, F, P, P, P, SZ, P]
        lib.spec_verify_threshold.restype = I
        lib.spec_verify_tree_stochastic_workspace_size.argtypes = [I, I, I]
        lib.spec_verify_tree_stochastic_workspace_size.restype = SZ
        lib.spec_verify_tree_stochastic.argtypes = [
            P, I, I64, I64, P, P, I, I, I, F, U64, U32, P, P, P, P, SZ, P]
        lib.spec_verify_tree_stochastic.restype = I
        lib.spec_verify_philox4x32_10.argtypes = [P, I64, U64, P, P]
        lib.spec_verify_philox4x32_10.restype = I
        lib.spec_verify_greedy_noalloc.argtypes = [P, I, I64, I64, P, I, I, I, P, P, P]
        lib.spec_verify_greedy_noalloc.restype = I
        lib.spec_verify_greedy_noalloc_read_device_status.argtypes = [ctypes.POINTER(U32), I, P]
        lib.spec_verify_greedy_noalloc_read_device_status.restype = I
        C, R, X, D = (ctypes.POINTER(_Cache), ctypes.POINTER(_Rows), ctypes.POINTER(_Rotary),
                      ctypes.c_double)
        lib.spec_verify_rotary_frequencies.argtypes = [P, P, I, D, I, D, D, D, D]
        lib.spec_verify_rotary_frequencies.restype = I
        lib.spec_verify_rotary.argtypes = [P, I, I64, I64, P, X, I, I64, I, I, P, I64, I64, P]
        lib.spec_verify_rotary.restype = I
        lib.spec_verify_cache_write.argtypes = [C, P, I64, I, P, P, P, R, R, I, I, I, X, R, I, P,
                                                P, P]
        lib.spec_verify_cache_write.restype = I
        lib.spec_verify_cache_read.argtypes = [C, P, I64, I, P, P, I, I64, P, P, I, P, P]
        lib.spec_verify_cache_read.restype = I
        lib.spec_verify_tree_attention_scratch_size.argtypes = [I, I, I, I, I]
        lib.spec_verify_tree_attention_scratch_size.restype = SZ
        lib.spec_verify_tree_attention.argtypes = [R, I, C, P, I64, I, P, P, P, I, I, I, F, P, P,
                                                   P, P, SZ, P]
        lib.spec_verify_tree_attention.restype = I
        lib.spec_verify_cache_commit.argtypes = [C, P, I64, I, P, P, P, I, I, P, P, P]
        lib.spec_verify_cache_commit.restype = I
        lib.spec_verify_cache_read_device_status.argtypes = [ctypes.POINTER(U32), I, P]
        lib.spec_verify_cache_read_device_status.restype = I
        lib.spec_verify_kernel_launches.argtypes = []
        lib.spec_verify_kernel_launches.restype = U64
        if path is None:
            _lib = lib
        return lib


def status_string(code: int) -> str:
    return load_library().spec_verify_status_string(int(code)).decode()


def _check(code: int, what: str):
    if code != 0:
        raise SpecVerifyError(f"{what}: {status_string(code)}")


def launch_count() -> int:
    """Kernels the library has launched in this process so far (its own
    count; a launch captured into a CUDA graph counts once, at capture)."""
    return int(load_library().spec_verify_kernel_launches())


def workspace_size(B: int, G: int, k: int, V: int) -> int:
    return int(load_library().spec_verify_workspace_size(B, G, k, V))


class Workspace:
    """A zero-initialised device workspace, grown on demand (one per stream)."""

    def __init__(self, device=None, nbytes: int = 0):
        self.device = torch.device(device if device is not None else "cuda")
        self.buf = None
        self.ensure(nbytes)

    @property
    def nbytes(self) -> int:
        return 0 if self.buf is None else self.buf.numel()

    def ensure(self, nbytes: int, stream=None):
        if nbytes <= self.nbytes:
            return self
        self.buf = _new((max(nbytes, 256),), torch.uint8, self.device, stream)
        _check(load_library().spec_verify_workspace_init(
            self.buf.data_ptr(), self.buf.numel(), _stream_ptr(stream, self.device)),
            "spec_verify_workspace_init")
        return self

    def reset(self, stream=None):
        if self.buf is not None:
            _check(load_library().spec_verify_workspace_init(
                self.buf.data_ptr(), self.buf.numel(), _stream_ptr(stream, self.device)),
                "spec_verify_workspace_init")

    def device_status(self, clear: bool = True, stream=None) -> int:
        """Sticky SV_FLAG_* bits of the device (synchronises the stream)."""
        v = ctypes.c_uint32(0)
        _check(load_library().spec_verify_read_device_status(
            self.buf.data_ptr(), ctypes.byref(v), int(clear), _stream_ptr(stream, self.device)),
            "spec_verify_read_device_status")
        return int(v.value)


_default_ws: dict = {}


def default_workspace(device) -> Workspace:
    key = (torch.device(device), torch.cuda.current_stream(device).cuda_stream)
    ws = _default_ws.get(key)
    if ws is None:
        ws = _default_ws[key] = Workspace(device)
    return ws


def _stream_ptr(stream, device):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return SV_F32
    if t.dtype == torch.bfloat16:
        return SV_BF16
    raise TypeError(f"logits must be float32 or bfloat16, got {t.dtype}")


def _logits(t: torch.Tensor, ndim: int, name: str):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dim() != ndim:
        raise ValueError(f"{name} must be {ndim}-d, got shape {tuple(t.shape)}")
    if t.numel() > 0 and t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the vocabulary axis must be contiguous")
    return _dtype_code(t), t.stride()


def _tokens(t: torch.Tensor, shape, device, name: str) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or t.device != device or t.dtype != torch.int32:
        raise TypeError(f"{name} must be an int32 tensor on {device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.contiguous()


def _out(out, key, shape, dtype, device):
    if out is not None and key in out:
        t = out[key]
        if tuple(t.shape) != tuple(shape) or t.dtype != dtype or not t.is_contiguous():
            raise ValueError(f"out[{key!r}] must be a contiguous {dtype} tensor {tuple(shape)}")
        return t
    return torch.empty(shape, dtype=dtype, device=device)


def stochastic(target: torch.Tensor, draft: torch.Tensor, draft_tokens: torch.Tensor,
               temperature: float, seed: int, seq_offset: int = 0, *, probs: bool = False,
               out: dict | None = None, workspace: Workspace | None = None,
               stream=None) -> dict:
    """Stochastic verify: target [B,k+1,V], draft [B,k,V], draft_tokens [B,k].

    Returns accepted_len [B], out_tokens [B,k+1] (and probs [B,k,2] when
    asked), all on the device; nothing is synchronised.
    """
    lib = load_library()
    tc, (tsb, tsp, _) = _logits(target, 3, "target")
    dc, (dsb, dsp, _) = _logits(draft, 3, "draft")
    B, kp1, V = target.shape
    k = kp1 - 1
    if tuple(draft.shape) != (B, k, V) or draft.device != target.device:
        raise ValueError("draft must be [B, k, V] on the target's device")
    dev = target.device
    tok = _tokens(draft_tokens, (B, k), dev, "draft_tokens")
    res = {"accepted_len": _out(out, "accepted_len", (B,), torch.int32, dev),
           "out_tokens": _out(out, "out_tokens", (B, k + 1), torch.int32, dev)}
    if probs:
        res["probs"] = _out(out, "probs", (B, k, 2), torch.float32, dev)
    ws = workspace or default_workspace(dev)
    ws.ensure(workspace_size(B, 1, k, V), stream)
    with torch.cuda.device(dev):
        code = lib.spec_verify_stochastic(
            target.data_ptr(), tc, tsb, tsp, draft.data_ptr(), dc, dsb, dsp, tok.data_ptr(),
            B, k, V, float(temperature), int(seed) & (2**64 - 1), int(seq_offset) & 0xFFFFFFFF,
            res["accepted_len"].data_ptr(), res["out_tokens"].data_ptr(),
            res["probs"].data_ptr() if probs else None, ws.buf.data_ptr(), ws.nbytes,
            _stream_ptr(stream, dev))
    _check(code, "spec_verify_stochastic")
    return res


def greedy(target: torch.Tensor, draft_tokens: torch.Tensor, *, out: dict | None = None,
           workspace: Workspace | None = None, stream=None) -> dict:
    """Greedy verify: target [B,k+1,V], draft_tokens [B,k]."""
    lib = load_library()
    tc, (tsb, tsp, _) = _logits(target, 3, "target")
    B, kp1, V = target.shape
    k = kp1 - 1
    dev = target.device
    tok = _tokens(draft_tokens, (B, k), dev, "draft_tokens")
    res = {"accepted_len": _out(out, "accepted_len", (B,), torch.int32, dev),
           "out_tokens": _out(out, "out_tokens", (B, k + 1), torch.int32, dev)}
    ws = workspace or default_workspace(dev)
    ws.ensure(workspace_size(B, 1, k, V), stream)
    with torch.cuda.device(dev):
        code = lib.spec_verify_greedy(
            target.data_ptr(), tc, tsb, tsp, tok.data_ptr(), B, k, V,
            res["accepted_len"].data_ptr(), res["out_tokens"].data_ptr(), ws.buf.data_ptr(),
            ws.nbytes, _stream_ptr(stream, dev))
    _check(code, "spec_verify_greedy")
    return res


def multi_candidate(target: torch.Tensor, cand_tokens: torch.Tensor, *, out: dict | None = None,
                    workspace: Workspace | None = None, stream=None) -> dict:
    """Multi-candidate verify: target [B,G,k+1,V], cand_tokens [B,G,k]."""
    lib = load_library()
    tc, (tsb, tsg, tsp, _) = _logits(target, 4, "target")
    B, G, kp1, V = target.shape
    k = kp1 - 1
    dev = target.device
    tok = _tokens(cand_tokens, (B, G, k), dev, "cand_tokens")
    res = {"best_candidate": _out(out, "best_candidate", (B,), torch.int32, dev),
           "accepted_len": _out(out, "accepted_len", (B,), torch.int32, dev),
           "out_tokens": _out(out, "out_tokens", (B, k + 1), torch.int32, dev)}
    ws = workspace or default_workspace(dev)
    ws.ensure(workspace_size(B, G, k, V), stream)
    with torch.cuda.device(dev):
        code = lib.spec_verify_multi_candidate(
            target.data_ptr(), tc, tsb, tsg, tsp, tok.data_ptr(), B, G, k, V,
            res["best_candidate"].data_ptr(), res["accepted_len"].data_ptr(),
            res["out_tokens"].data_ptr(), ws.buf.data_ptr(), ws.nbytes, _stream_ptr(stream, dev))
    _check(code, "spec_verify_multi_candidate")
    return res


def multi_candidate_rows(rows: torch.Tensor, row_of: torch.Tensor, cand_tokens: torch.Tensor, *,
                         out: dict | None = None, workspace: Workspace | None = None,
                         stream=None) -> dict:
    """Multi-candidate verify on deduplicated rows: rows [B,R,V], row_of
    [B,G,k+1] (int32, the row of each (b, g, i)), cand_tokens [B,G,k].  Same
    results as multi_candidate on rows gathered to [B,G,k+1,V]."""
    lib = load_library()
    tc, (tsb, tsr, _) = _logits(rows, 3, "rows")
    B, R, V = rows.shape
    if row_of.dim() != 3 or row_of.shape[0] != B:
        raise ValueError(f"row_of must be [B, G, k+1], got {tuple(row_of.shape)}")
    G, kp1 = int(row_of.shape[1]), int(row_of.shape[2])
    k = kp1 - 1
    dev = rows.device
    rmap = _tokens(row_of, (B, G, kp1), dev, "row_of")
    tok = _tokens(cand_tokens, (B, G, k), dev, "cand_tokens")
    res = {"best_candidate": _out(out, "best_candidate", (B,), torch.int32, dev),
           "accepted_len": _out(out, "accepted_len", (B,), torch.int32, dev),
           "out_tokens": _out(out, "out_tokens", (B, k + 1), torch.int32, dev)}
    ws = workspace or default_workspace(dev)
    ws.ensure(workspace_size(B, G, k, V), stream)
    with torch.cuda.device(dev):
        code = lib.spec_verify_multi_candidate_rows(
            rows.data_ptr(), tc, tsb, tsr, rmap.data_ptr(), tok.data_ptr(), B, G, k, R, V,
            res["best_candidate"].data_ptr(), res["accepted_len"].data_ptr(),
            res["out_tokens"].data_ptr(), ws.buf.data_ptr(), ws.nbytes, _stream_ptr(stream, dev))
    _check(code, "spec_verify_multi_candidate_rows")
    return res


def threshold(target: torch.Tensor, draft_tokens: torch.Tensor, temperature: float,
              threshold: float, *, out: dict | None = None, workspace: Workspace | None = None,
              stream=None) -> dict:
    """Threshold acceptance: target [B,k+1,V], draft_tokens [B,k]; accept the
    longest prefix whose probability under softmax(target/T) is at least
    `threshold`, then the argmax of the next row."""
    lib = load_library()
    tc, (tsb, tsp, _) = _logits(target, 3, "target")
    B, kp1, V = target.shape
    k = kp1 - 1
    dev = target.device
    tok = _tokens(draft_tokens, (B, k), dev, "draft_tokens")
    res = {"accepted_len": _out(out, "accepted_len", (B,), torch.int32, dev),
           "out_tokens": _out(out, "out_tokens", (B, k + 1), torch.int32, dev)}
    ws = workspace or default_workspace(dev)
    ws.ensure(workspace_size(B, 1, k, V), stream)
    with torch.cuda.device(dev):
        code = lib.spec_verify_threshold(
            target.data_ptr(), tc, tsb, tsp, tok.data_ptr(), B, k, V, float(temperature),
            float(threshold), res["accepted_len"].data_ptr(), res["out_tokens"].data_ptr(),
            ws.buf.data_ptr(), ws.nbytes, _stream_ptr(stream, dev))
    _check(code, "spec_verify_threshold")
    return res


def tree_workspace_size(B: int, N: int, V: int) -> int:
    return int(load_library().spec_verify_tree_workspace_size(B, N, V))


def tree_greedy(node_logits: torch.Tensor, parent: torch.Tensor, tokens: torch.Tensor, *,
                out: dict | None = None, workspace: Workspace | None = None,
                stream=None) -> dict:
    """Greedy verify of a draft token tree: node_logits [B,N,V] (row j = the
    target after the path to node j), parent [B,N] and tokens [B,N] int32.
    Returns accepted_len [B], path [B,N] and out_tokens [B,N]."""
    lib = load_library()
    tc, (tsb, tsn, _) = _logits(node_logits, 3, "node_logits")
    B, N, V = node_logits.shape
    dev = node_logits.device
    par = _tokens(parent, (B, N), dev, "parent")
    tok = _tokens(tokens, (B, N), dev, "tokens")
    res = {"accepted_len": _out(out, "accepted_len", (B,), torch.int32, dev),
           "path": _out(out, "path", (B, N), torch.int32, dev),
           "out_tokens": _out(out, "out_tokens", (B, N), torch.int32, dev)}
    ws = workspace or default_workspace(dev)
    ws.ensure(tree_workspace_size(B, N, V), stream)
    with torch.cuda.device(dev):
        code = lib.spec_verify_tree_greedy(
            node_logits.data_ptr(), tc, tsb, tsn, par.data_ptr(), tok.data_ptr(), B, N, V,
            res["accepted_len"].data_ptr(), res["path"].data_ptr(), res["out_tokens"].data_ptr(),
            ws.buf.data_ptr(), ws.nbytes, _stream_ptr(stream, dev))
    _check(code, "spec_verify_tree_greedy")
    return res


def tree_stochastic_workspace_size(B: int, N: int, V: int) -> int:
    return int(load_library().spec_verify_tree_stochastic_workspace_size(B, N, V))


def tree_stochastic(node_logits: torch.Tensor, parent: torch.Tensor, tokens: torch.Tensor,
                    temperature: float, seed: int, seq_offset: int = 0, *,
                    out: dict | None = None, workspace: Workspace | None = None,
                    stream=None) -> dict:
    """Stochastic verify of a draft token tree whose siblings are Top-K
    candidates: node_logits [B,N,V], parent [B,N] and tokens [B,N] int32 as
    for tree_greedy.  Returns accepted_len [B], path [B,N] and out_tokens
    [B,N] (the accepted tokens, the drawn token, then -1)."""
    lib = load_library()
    tc, (tsb, tsn, _) = _logits(node_logits, 3, "node_logits")
    B, N, V = node_logits.shape
    dev = node_logits.device
    par = _tokens(parent, (B, N), dev, "parent")
    tok = _tokens(tokens, (B, N), dev, "tokens")
    res = {"accepted_len": _out(out, "accepted_len", (B,), torch.int32, dev),
           "path": _out(out, "path", (B, N), torch.int32, dev),
           "out_tokens": _out(out, "out_tokens", (B, N), torch.int32, dev)}
    ws = workspace or default_workspace(dev)
    ws.ensure(tree_stochastic_workspace_size(B, N, V), stream)
    with torch.cuda.device(dev):
        code = lib.spec_verify_tree_stochastic(
            node_logits.data_ptr(), tc, tsb, tsn, par.data_ptr(), tok.data_ptr(), B, N, V,
            float(temperature), int(seed) & (2**64 - 1), int(seq_offset) & 0xFFFFFFFF,
            res["accepted_len"].data_ptr(), res["path"].data_ptr(), res["out_tokens"].data_ptr(),
            ws.buf.data_ptr(), ws.nbytes, _stream_ptr(stream, dev))
    _check(code, "spec_verify_tree_stochastic")
    return res


def commit(result: dict, seq_len: torch.Tensor, token_buf: torch.Tensor, *,
           next_input: torch.Tensor | None = None, workspace: Workspace | None = None,
           stream=None) -> None:
    """Device-side commit after a verify call: append each sequence's n + 1
    committed tokens (result["out_tokens"][b, :n+1], n = result["accepted_len"][b])
    to token_buf[b, seq_len[b]:], advance seq_len and write the next step's
    input token, all on the GPU (no host synchronisation).  token_buf is an
    int32 [B, capacity] tensor whose rows may be strided; tokens past capacity
    are dropped and flagged (SV_FLAG_CAPACITY) in `workspace` if given."""
    lib = load_library()
    acc, out = result["accepted_len"], result["out_tokens"]
    dev = acc.device
    B = int(acc.shape[0])
    k = int(out.shape[1]) - 1
    acc = _tokens(acc, (B,), dev, "accepted_len")
    out = _tokens(out, (B, k + 1), dev, "out_tokens")
    if (not isinstance(seq_len, torch.Tensor) or seq_len.dtype != torch.int32 or
            seq_len.device != dev or tuple(seq_len.shape) != (B,) or not seq_len.is_contiguous()):
        raise ValueError("seq_len must be a contiguous int32 [B] tensor on the verify device")
    if (token_buf.dtype != torch.int32 or token_buf.device != dev or token_buf.dim() != 2 or
            token_buf.shape[0] != B or (token_buf.shape[1] > 1 and token_buf.stride(1) != 1)):
        raise ValueError("token_buf must be an int32 [B, capacity] tensor with contiguous rows")
    if next_input is not None and (next_input.dtype != torch.int32 or next_input.device != dev or
                                   tuple(next_input.shape) != (B,) or
                                   not next_input.is_contiguous()):
        raise ValueError("next_input must be a contiguous int32 [B] tensor")
    cap = int(token_buf.shape[1])
    stride = int(token_buf.stride(0)) if B > 1 else cap
    with torch.cuda.device(dev):
        code = lib.spec_verify_commit(
            acc.data_ptr(), out.data_ptr(), B, k, seq_len.data_ptr(), token_buf.data_ptr(),
            max(stride, cap), cap, next_input.data_ptr() if next_input is not None else None,
            workspace.buf.data_ptr() if workspace is not None and workspace.buf is not None
            else None, _stream_ptr(stream, dev))
    _check(code, "spec_verify_commit")


def greedy_noalloc(target: torch.Tensor, draft_tokens: torch.Tensor, *,
                   out: dict | None = None, stream=None) -> dict:
    """Greedy verify that allocates no device memory inside the library.

    For callers that cannot allocate on the verify path (an external
    allocator or pool owns the device, or the call runs where an allocation
    may block or fail): the library uses its own fixed 2 MiB device array
    instead of a workspace.  Pass preallocated `out` tensors to keep this
    wrapper free of allocations as well.  Calls share that array, so order
    them on one stream; the first call on a device should come before any
    stream capture.
    """
    lib = load_library()
    tc, (tsb, tsp, _) = _logits(target, 3, "target")
    B, kp1, V = target.shape
    k = kp1 - 1
    dev = target.device
    tok = _tokens(draft_tokens, (B, k), dev, "draft_tokens")
    res = {"accepted_len": _out(out, "accepted_len", (B,), torch.int32, dev),
           "out_tokens": _out(out, "out_tokens", (B, k + 1), torch.int32, dev)}
    with torch.cuda.device(dev):
        code = lib.spec_verify_greedy_noalloc(
            target.data_ptr(), tc, tsb, tsp, tok.data_ptr(), B, k, V,
            res["accepted_len"].data_ptr(), res["out_tokens"].data_ptr(), _stream_ptr(stream, dev))
    _check(code, "spec_verify_greedy_noalloc")
    return res


def greedy_noalloc_device_status(clear: bool = True, device=None, stream=None) -> int:
    """Sticky SV_FLAG_* bits raised on the device by greedy_noalloc calls on
    `device` (synchronises the stream; allocates nothing)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else \
        torch.device(device)
    v = ctypes.c_uint32(0)
    with torch.cuda.device(dev):
        _check(load_library().spec_verify_greedy_noalloc_read_device_status(
            ctypes.byref(v), int(clear), _stream_ptr(stream, dev)),
            "spec_verify_greedy_noalloc_read_device_status")
    return int(v.value)


def philox4x32_10(counters: torch.Tensor, seed: int, stream=None) -> torch.Tensor:
    """Device Philox4x32-10 of each counter row ([n,4] int32 bit patterns)."""
    lib = load_library()
    if counters.dtype != torch.int32 or counters.dim() != 2 or counters.shape[1] != 4:
        raise TypeError("counters must be an int32 tensor [n, 4] (uint32 bit patterns)")
    c = counters.contiguous()
    out = torch.empty_like(c)
    with torch.cuda.device(c.device):
        code = lib.spec_verify_philox4x32_10(c.data_ptr(), c.shape[0], int(seed) & (2**64 - 1),
                                              out.data_ptr(), _stream_ptr(stream, c.device))
    _check(code, "spec_verify_philox4x32_10")
    return out


# ---------------------------------------------------------------- cache side

_TYPES = {torch.float32: SV_F32, torch.bfloat16: SV_BF16, torch.float16: SV_F16,
          torch.float8_e4m3fn: SV_E4M3}
_ROPE = {"none": 0, "linear": 1, "bands": 2, "yarn": 3}


# The calls below may run many times a step for a few microseconds of work, so
# their checks are kept to plain attribute tests, and the stream and device are
# looked up without making objects.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _launch(fn, what, device, stream, args):
    """Call an entry point, whose last argument is the stream, with `device` current."""
    st = _raw_stream(device.index) if stream is None else stream.cuda_stream
    if _current_device() == device.index:
        code = fn(*args, st)
    else:
        with torch.cuda.device(device):
            code = fn(*args, st)
    if code != 0:
        _check(code, what)


def _new(shape, dtype, device, stream, zero=False):
    """A new tensor of the call's stream.  With `stream`, its memory must come
    from there too: a block of the current stream may still be read by what that
    stream has yet to do.  The current one may use the result and drop it."""
    make = torch.zeros if zero else torch.empty
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        made = make(shape, dtype=dtype, device=device)
    made.record_stream(torch.cuda.current_stream(device))
    return made


def _result(out, key, shape, dtype, device, stream):
    """_out, refusing a caller's tensor on another device."""
    if out is None or key not in out:
        return _new(shape, dtype, device, stream)
    made = _out(out, key, shape, dtype, device)
    if made.device != device:
        raise ValueError(f"out[{key!r}] must be on {device}")
    if stream is not None:
        made.record_stream(stream)
    return made


def _like(t, stream):
    """A new contiguous tensor of t's shape and type."""
    if stream is None and t.is_contiguous():
        return torch.empty_like(t)
    return _new(t.shape, t.dtype, t.device, stream)


def _ints(t, shape, device, name):
    if (not isinstance(t, torch.Tensor) or t.dtype is not torch.int32 or t.shape != shape or
            t.device != device or not t.is_contiguous()):
        raise TypeError(f"{name} must be a contiguous int32 tensor {tuple(shape)} on {device}")
    return t.data_ptr()


def _rows(t, heads, dim, name, like=None):
    """Code and descriptor of a [B, N, heads, dim] tensor (`like`: another one)."""
    code = _TYPES.get(t.dtype) if isinstance(t, torch.Tensor) else None
    if code is None or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor of a floating type")
    shape = t.shape
    if len(shape) != 4 or (heads is not None and shape[2] != heads) or shape[3] != dim:
        raise ValueError(f"{name} must be [B, N, {'H' if heads is None else heads}, {dim}], "
                         f"got {tuple(shape)}")
    if like is not None and (t.dtype is not like.dtype or shape[0] != like.shape[0] or
                             shape[1] != like.shape[1] or t.device != like.device):
        raise ValueError(f"{name} must match k's type, device, B and N")
    sb, sn, sh, sd = t.stride()
    if sd != 1 and dim > 1 and t.numel() > 0:
        raise ValueError(f"{name}: the last axis must be contiguous")
    return code, _Rows(t.data_ptr(), sb, sn, sh)


class KVCache:
    """A paged cache pool: k and v [pages, page_size, heads, head_dim] (or
    [layers, pages, ...]) of one floating type with any strides but a contiguous
    last axis, the same for both; float8_e4m3fn pools come with float32 scales
    [pages, heads, page_size] (or [layers, ...]).  Page tables are passed to the
    calls.  cache_commit moves rows in all layers; the other calls use layer 0
    (`layer(i)` is another one's pool).  `KVCache.empty` allocates one with each head's page contiguous."""

    __slots__ = ("k", "v", "k_scale", "v_scale", "device", "page_size", "num_heads", "head_dim",
                 "layers", "_c")

    def __init__(self, k, v, k_scale=None, v_scale=None):
        if k.dtype not in _TYPES or not k.is_cuda or k.dim() not in (4, 5):
            raise TypeError("k must be a CUDA tensor [(layers,) pages, page_size, heads, head_dim] "
                            "of float32, bfloat16, float16 or float8_e4m3fn")
        stride = k.stride()
        if v.dtype != k.dtype or v.device != k.device or v.shape != k.shape or v.stride() != stride:
            raise ValueError("v must have k's type, device, shape and strides")
        *layers, pages, page_size, heads, dim = k.shape
        if stride[-1] != 1 and dim > 1:
            raise ValueError("the pool's last axis must be contiguous")
        coded = k.dtype == torch.float8_e4m3fn
        if coded != (k_scale is not None) or coded != (v_scale is not None):
            raise ValueError("float8_e4m3fn pools, and only they, have k_scale and v_scale")
        if coded:
            want = (*layers, pages, heads, page_size)
            for s in (k_scale, v_scale):
                if (s.dtype != torch.float32 or s.device != k.device or tuple(s.shape) != want or
                        s.stride()[-3:] != (heads * page_size, page_size, 1)):
                    raise ValueError(f"scales must be float32 {want}, contiguous but for layers")
            if layers and k_scale.stride(0) != v_scale.stride(0):
                raise ValueError("k_scale and v_scale must have the same strides")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.device, self.page_size, self.num_heads, self.head_dim = k.device, page_size, heads, dim
        self.layers = layers[0] if layers else 1
        self._c = _Cache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr() if coded else None,
                         v_scale.data_ptr() if coded else None, _TYPES[k.dtype], pages, page_size,
                         heads, dim, stride[-4], stride[-3], stride[-2], self.layers,
                         stride[0] if layers else 0,
                         k_scale.stride(0) if layers and coded else 0)

    @classmethod
    def empty(cls, num_pages, page_size, num_heads, head_dim, dtype=torch.bfloat16, device="cuda",
              layers=None):
        """A pool of zeros whose layout is [(layers,) pages, heads, page_size, head_dim]."""
        lead = () if layers is None else (layers,)
        shape = (*lead, num_pages, num_heads, page_size)
        made = []
        for _ in range(2):
            t = torch.zeros((*shape, head_dim), device=device,
                            dtype=torch.uint8 if dtype == torch.float8_e4m3fn else dtype)
            made.append(t.view(dtype).transpose(-3, -2))
        if dtype == torch.float8_e4m3fn:
            made += [torch.zeros(shape, dtype=torch.float32, device=device) for _ in range(2)]
        return cls(*made)

    def layer(self, i):
        """Layer i's pool (shares memory)."""
        if self.k.dim() == 4:
            raise ValueError("this pool has one layer")
        return KVCache(self.k[i], self.v[i], None if self.k_scale is None else self.k_scale[i],
                       None if self.v_scale is None else self.v_scale[i])


class Rotary:
    """Rotary positions: float64 frequencies [rotary_dim / 2] on the device, the
    pair layout and the factor on cos and sin (see rotary_frequencies)."""

    __slots__ = ("inv_freq", "interleaved", "magnitude", "_c")

    def __init__(self, inv_freq, interleaved=False, magnitude=1.0):
        if (inv_freq.dtype != torch.float64 or not inv_freq.is_cuda or inv_freq.dim() != 1 or
                not inv_freq.is_contiguous()):
            raise TypeError("inv_freq must be a contiguous float64 CUDA tensor [rotary_dim / 2]")
        self.inv_freq, self.interleaved, self.magnitude = inv_freq, interleaved, magnitude
        self._c = _Rotary(inv_freq.data_ptr(), 2 * inv_freq.shape[0], int(interleaved), magnitude)


def rotary_frequencies(rotary_dim: int, base: float = 10000.0, *, scaling: str = "none",
                       factor: float = 1.0, original_len: float = 0.0, low: float = 1.0,
                       high: float = 0.0, interleaved: bool = False, device="cuda") -> Rotary:
    """Rotary frequencies base^(-2i/rotary_dim) on `device`, scaled for long
    contexts: "none", "linear" (all / factor), "bands" (by wavelength; low and
    high bound original_len / wavelength) or "yarn" (a ramp over the pairs that
    turn between `high` and `low` times over original_len).  `high` defaults to
    4 for "bands" and 32 for "yarn"."""
    if scaling not in _ROPE:
        raise ValueError(f"scaling must be one of {sorted(_ROPE)}, got {scaling!r}")
    if high == 0.0:
        high = 32.0 if scaling == "yarn" else 4.0
    host = (ctypes.c_double * max(1, rotary_dim // 2))()
    mag = ctypes.c_float(1.0)
    _check(load_library().spec_verify_rotary_frequencies(
        ctypes.addressof(host), ctypes.addressof(mag), rotary_dim, base, _ROPE[scaling], factor,
        original_len, low, high), "spec_verify_rotary_frequencies")
    return Rotary(torch.tensor(list(host), dtype=torch.float64, device=device), interleaved,
                  float(mag.value))


def rotary(x: torch.Tensor, positions: torch.Tensor, rope: Rotary, *, inverse: bool = False,
           out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Rotary positions: x [T, H, D] or [B, N, H, D] (float32, bfloat16 or
    float16; last axis contiguous), positions [T] or [B, N] int32.  `inverse`
    turns back (the transposed map, hence the gradient).  `out` may be x."""
    lib = load_library()
    code = _TYPES.get(x.dtype) if isinstance(x, torch.Tensor) else None
    if code is None or code == SV_E4M3 or not x.is_cuda:
        raise TypeError("x must be a CUDA tensor of float32, bfloat16 or float16")
    shape, dev = x.shape, x.device
    if len(shape) == 4:
        B, N, H, D = shape
        lead, T = (B, N), B * N
    elif len(shape) == 3:
        T, H, D = shape
        lead = (T,)
    else:
        raise ValueError(f"x must be [T, H, D] or [B, N, H, D], got shape {tuple(shape)}")
    pos = _ints(positions, lead, dev, "positions")
    if rope.inv_freq.device != dev:
        raise ValueError("the rotary frequencies must be on x's device")
    if out is None:
        out = _like(x, stream)
        to = (H * D, D)
    elif out.dtype != x.dtype or out.device != dev or out.shape != shape:
        raise ValueError("out must have x's type, device and shape")
    else:
        to = _token_strides(out, "out")
    if x.numel() == 0:
        return out
    _launch(lib.spec_verify_rotary, "spec_verify_rotary", dev, stream,
            (x.data_ptr(), code, *_token_strides(x, "x"), pos, rope._c, int(inverse), T, H, D,
             out.data_ptr(), *to))
    return out


def _token_strides(t, name):
    """Strides of tokens and heads of a [T, H, D] or [B, N, H, D] tensor."""
    s = t.stride()
    if s[-1] != 1 and t.numel() > 0:
        raise ValueError(f"{name}: the last axis must be contiguous")
    if len(s) == 3:
        return s[0], s[1]
    B, N = t.shape[:2]
    if B > 1 and N > 1 and s[0] != N * s[1]:
        raise ValueError(f"{name}: tokens must be evenly spaced over B and N")
    return (s[1] if N > 1 else s[0]), s[2]


def _table(page_table, B, device):
    t = page_table
    shape, stride = (t.shape, t.stride()) if isinstance(t, torch.Tensor) else ((), ())
    if (len(shape) != 2 or t.dtype is not torch.int32 or shape[0] != B or t.device != device or
            (stride[1] != 1 and shape[1] > 1)):
        raise TypeError(f"page_table must be int32 [{B}, max_pages] on {device}, rows contiguous")
    return t.data_ptr(), stride[0], shape[1]


def _status(workspace, device, stream):
    """Where a call reports its flags: the workspace, or the device's own word (None)."""
    if workspace is None:
        return None
    if workspace.buf is None:
        workspace.ensure(256, stream)
    if workspace.buf.device != device:
        raise ValueError(f"the workspace must be on {device}")
    return workspace.buf.data_ptr()


def cache_device_status(clear: bool = True, device=None, stream=None) -> int:
    """Sticky SV_FLAG_* bits raised on `device` by the cache-side calls that were
    given no workspace (synchronises the stream)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else \
        torch.device(device)
    v = ctypes.c_uint32(0)
    with torch.cuda.device(dev):
        _check(load_library().spec_verify_cache_read_device_status(
            ctypes.byref(v), int(clear), _stream_ptr(stream, dev)),
            "spec_verify_cache_read_device_status")
    return int(v.value)


def cache_write(cache: KVCache, page_table: torch.Tensor, cache_len: torch.Tensor,
                k: torch.Tensor, v: torch.Tensor, *, parent: torch.Tensor | None = None,
                count: torch.Tensor | None = None, rope: Rotary | None = None,
                q: torch.Tensor | None = None, q_out: torch.Tensor | None = None,
                workspace: Workspace | None = None, stream=None) -> torch.Tensor | None:
    """Write k and v [B, N, heads, head_dim] of N new tokens a sequence at
    positions cache_len[b] + j of the paged cache, K turned by `rope` to
    position cache_len[b] + depth (in the tree `parent` [B, N], else j), in 8
    bits if the pool is float8_e4m3fn.  `q` [B, N, Hq, head_dim] is turned in
    the same launch and returned.  Only the first count[b] tokens are written."""
    lib = load_library()
    code_t, kr = _rows(k, cache.num_heads, cache.head_dim, "k")
    _, vr = _rows(v, cache.num_heads, cache.head_dim, "v", k)
    B, N = k.shape[:2]
    dev = cache.device
    if k.device != dev:
        raise ValueError("k and v must be on the cache's device")
    if rope is not None and rope.inv_freq.device != dev:
        raise ValueError("the rotary frequencies must be on the cache's device")
    lens = _ints(cache_len, (B,), dev, "cache_len")
    par = None if parent is None else _ints(parent, (B, N), dev, "parent")
    cnt = None if count is None else _ints(count, (B,), dev, "count")
    table, tstride, pages = _table(page_table, B, dev)
    qr, Hq, qo = None, 0, None
    if q is not None:
        if rope is None:
            raise ValueError("q is turned by rope: pass both")
        _, qr = _rows(q, None, cache.head_dim, "q", k)
        Hq = q.shape[2]
        if q_out is None:
            # (padding rows are left as they were)
            q_out = _like(q, stream) if cnt is None else _new(q.shape, q.dtype, dev, stream, True)
        elif (q_out.shape != q.shape or q_out.dtype != q.dtype or q_out.device != dev or
              not q_out.is_contiguous()):
            raise ValueError("q_out must be a contiguous tensor like q")
        qo = q_out.data_ptr()
    _launch(lib.spec_verify_cache_write, "spec_verify_cache_write", dev, stream,
            (cache._c, table, tstride, pages, lens, par, cnt, kr, vr, code_t, B, N,
             None if rope is None else rope._c, qr, Hq, qo, _status(workspace, dev, stream)))
    return q_out


def cache_read(cache: KVCache, page_table: torch.Tensor, offsets: torch.Tensor, total: int,
               dtype: torch.dtype = torch.bfloat16, *, start: torch.Tensor | None = None,
               out: dict | None = None, workspace: Workspace | None = None, stream=None) -> dict:
    """Cached rows as packed k and v [total, heads, head_dim] of `dtype`: row r
    of offsets[b] <= r < offsets[b+1] is sequence b's token at position
    start[b] + r - offsets[b].  Other rows are left as they were (unset, unless
    `out` brings the tensors)."""
    lib = load_library()
    dev = cache.device
    B = int(offsets.shape[0]) - 1
    if B < 0 or dtype not in _TYPES or dtype == torch.float8_e4m3fn:
        raise ValueError("offsets must be [B + 1] and dtype float32, bfloat16 or float16")
    offs = _ints(offsets, (B + 1,), dev, "offsets")
    st0 = None if start is None else _ints(start, (B,), dev, "start")
    table, tstride, pages = _table(page_table, B, dev)
    shape = (int(total), cache.num_heads, cache.head_dim)
    res = {x: _result(out, x, shape, dtype, dev, stream) for x in ("k", "v")}
    if total == 0:
        return res
    _launch(lib.spec_verify_cache_read, "spec_verify_cache_read", dev, stream,
            (cache._c, table, tstride, pages, offs, st0, B, int(total), res["k"].data_ptr(),
             res["v"].data_ptr(), _TYPES[dtype], _status(workspace, dev, stream)))
    return res


@functools.lru_cache(maxsize=256)
def _scratch_bytes(*sizes):
    return load_library().spec_verify_tree_attention_scratch_size(*sizes)


def tree_attention(q: torch.Tensor, cache: KVCache, page_table: torch.Tensor,
                   cache_len: torch.Tensor, parent: torch.Tensor | None = None, *,
                   count: torch.Tensor | None = None, scale: float | None = None,
                   lse: bool = False, out: dict | None = None,
                   workspace: Workspace | None = None, stream=None) -> dict:
    """Attention of drafted tokens over the cache that holds them
    (cache_write): q [B, N, Hq, head_dim] bfloat16 or float16, node i of the
    tree `parent` [B, N] (None: a chain) sees cache_len[b] context tokens, its
    ancestors and itself; Hq a multiple of the cache's heads; scale defaults to
    head_dim ** -0.5.  Returns out [B, N, Hq, head_dim] (and lse [B, N, Hq])."""
    lib = load_library()
    code_t, qr = _rows(q, None, cache.head_dim, "q")
    B, N, Hq, D = q.shape
    dev = cache.device
    if q.device != dev:
        raise ValueError("q must be on the cache's device")
    lens = _ints(cache_len, (B,), dev, "cache_len")
    par = None if parent is None else _ints(parent, (B, N), dev, "parent")
    cnt = None if count is None else _ints(count, (B,), dev, "count")
    table, tstride, pages = _table(page_table, B, dev)
    if out is None:
        res = {"out": _like(q, stream)}
    else:
        res = {"out": _result(out, "out", (B, N, Hq, D), q.dtype, dev, stream)}
    if lse:
        res["lse"] = _result(out, "lse", (B, N, Hq), torch.float32, dev, stream)
    if scale is None:
        scale = D ** -0.5
    need = _scratch_bytes(B, N, Hq, cache.num_heads, D)
    scratch = _new((need or 16,), torch.uint8, dev, stream)
    _launch(lib.spec_verify_tree_attention, "spec_verify_tree_attention", dev, stream,
            (qr, code_t, cache._c, table, tstride, pages, lens, par, cnt, B, N, Hq, float(scale),
             res["out"].data_ptr(), res["lse"].data_ptr() if lse else None,
             _status(workspace, dev, stream), scratch.data_ptr(), scratch.shape[0]))
    return res


def cache_commit(cache: KVCache, page_table: torch.Tensor, cache_len: torch.Tensor, result: dict,
                 *, new_len: torch.Tensor | None = None, workspace: Workspace | None = None,
                 stream=None) -> torch.Tensor:
    """After a verify call: move the accepted path's cache rows, in all layers
    of the pool, from positions cache_len[b] + path[b, j] to cache_len[b] + j,
    and return the new lengths cache_len + accepted_len + 1 (in `new_len`,
    which may be cache_len or the result's accepted_len).  `result` is what tree_greedy or tree_stochastic
    returned; results without a path (a chain) only advance the lengths."""
    lib = load_library()
    acc, path = result["accepted_len"], result.get("path")
    dev = cache.device
    B = int(acc.shape[0])
    lens = _ints(cache_len, (B,), dev, "cache_len")
    accepted = _ints(acc, (B,), dev, "accepted_len")
    if path is not None:
        N = int(path.shape[1]) if path.dim() == 2 else -1
        path = _ints(path, (B, N), dev, "path")
    else:
        N = int(result["out_tokens"].shape[1]) if "out_tokens" in result else 64
    table, tstride, pages = _table(page_table, B, dev)
    if new_len is None:
        new_len = _new((B,), torch.int32, dev, stream)
    _launch(lib.spec_verify_cache_commit, "spec_verify_cache_commit", dev, stream,
            (cache._c, table, tstride, pages, lens, accepted, path, B, N,
             _ints(new_len, (B,), dev, "new_len"), _status(workspace, dev, stream)))
    return new_len
