"""The cache-side operators of a speculative decoding step, as measured cases.

Five operators stand around the verify-and-accept calls: rotary positions, the
paged cache's write (plain or 8-bit), its read-back, attention of drafted
tokens (a chain or a tree) over the cache, and the move of an accepted path's
cache rows into place.  `run` computes one of them, in elementary torch
operations or, where `own` is set, through the package's entry points.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32,
          "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one user's chain of four drafts and the last token, short context: latency
        dict(name="attn_one_user", op="attn", B=1, N=5, lo=480, hi=520, Hkv=8, G=4, D=64, page=16,
             q="fp16", kv="fp16", tree=False, lens=1),
        # the batch of the stochastic tree benchmark (64 trees of 26 nodes) over mixed contexts
        dict(name="attn_tree_batch", op="attn", B=64, N=26, lo=700, hi=4096, Hkv=8, G=4, D=128,
             page=64, q="bf16", kv="bf16", tree=True, lens=2),
        # two long documents, 8-bit cache, a chain of four drafts
        dict(name="attn_long_e4m3", op="attn", B=2, N=5, lo=120000, hi=131000, Hkv=8, G=8, D=128,
             page=128, q="bf16", kv="e4m3", tree=False, lens=3),
        # the widest trees (64 nodes) of a model with eight query heads a cache head
        dict(name="attn_wide_tree", op="attn", B=8, N=64, lo=2500, hi=5000, Hkv=8, G=8, D=128,
             page=32, q="bf16", kv="bf16", tree=True, lens=4),
        # rotary of one user's queries
        dict(name="rotary_one_user", op="rotary", T=5, H=32, D=128, rd=128, t="bf16",
             interleaved=False, base=10000.0, far=4000),
        # a long prompt's queries and keys, part of the head, interleaved pairs
        dict(name="rotary_prompt", op="rotary", T=16000, H=40, D=128, rd=64, t="bf16",
             interleaved=True, base=500000.0, far=1000000),
        # the cache write of one user's step
        dict(name="write_one_user", op="write", B=1, N=5, lo=480, hi=520, Hkv=8, G=4, D=128, rd=128,
             page=16, q="bf16", kv="bf16", tree=False, interleaved=False, lens=5),
        # prompt chunks of eight users into an 8-bit cache
        dict(name="write_prompt_e4m3", op="write", B=8, N=1000, lo=0, hi=900, Hkv=8, G=4, D=128,
             rd=128, page=64, q="bf16", kv="e4m3", tree=False, interleaved=False, lens=6),
        # two short sequences read back
        dict(name="read_two_users", op="read", B=2, lo=100, hi=200, Hkv=8, D=128, page=16, kv="e4m3",
             to="bf16", lens=7),
        # a batch's contexts read back from the 8-bit cache
        dict(name="read_batch", op="read", B=32, lo=500, hi=4096, Hkv=8, D=128, page=64, kv="e4m3",
             to="bf16", lens=8),
        # one user's accepted path, one layer
        dict(name="commit_one_user", op="commit", B=1, N=26, L=1, lo=20, hi=60, Hkv=8, D=128, page=16,
             kv="bf16", depth=5, lens=9),
        # the tree batch's accepted paths in all layers of a model
        dict(name="commit_batch", op="commit", B=64, N=26, L=32, lo=20, hi=60, Hkv=8, D=128, page=16,
             kv="bf16", depth=8, lens=10),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "rotary", "write", "read", "commit"])
    lens = rng.randrange(1 << 20)
    page = rng.choice([16, 32, 64, 128])
    if op == "rotary":
        D = rng.choice([64, 80, 96, 128])
        H = rng.randint(1, 40)
        T = _log(rng, 1, min(16000, 80_000_000 // (H * D)))
        return dict(op=op, T=T, H=H, D=D, rd=rng.choice([D, D // 2 // 16 * 16 or 32]),
                    t=rng.choice(["bf16", "fp16", "fp32"]) if T * H * D < 40_000_000 else "bf16",
                    interleaved=rng.random() < 0.5, base=rng.choice([10000.0, 500000.0]),
                    far=_log(rng, 10000, 1000000))
    if op == "commit":
        L, B = _log(rng, 1, 32), _log(rng, 1, 64)
        return dict(op=op, B=B, N=rng.randint(1, 64 if L * B < 800 else 26), L=L, lo=0, hi=_log(rng, 1, 60),
                    Hkv=rng.choice([1, 2, 4, 8]), D=rng.choice([64, 128]), page=16,
                    kv=rng.choice(["bf16", "e4m3"]), depth=rng.randint(1, 8), lens=lens)
    Hkv, D = rng.choice([1, 2, 4, 8]), rng.choice([64, 80, 96, 128, 128])
    if op == "read":
        B = _log(rng, 1, 32)
        hi = _log(rng, 1, 4096)
        return dict(op=op, B=B, lo=rng.randint(0, hi), hi=hi, Hkv=Hkv, D=D, page=page,
                    kv=rng.choice(["e4m3", "bf16"]), to=rng.choice(["bf16", "fp16"]), lens=lens)
    G = rng.choice([1, 2, 4, 8])
    q = rng.choice(["bf16", "fp16"])
    if op == "write":
        B = _log(rng, 1, 64)
        N = _log(rng, 1, max(1, 8000 // B))
        return dict(op=op, B=B, N=N, lo=0, hi=_log(rng, 1, 900), Hkv=Hkv, G=min(G, 4), D=D,
                    rd=rng.choice([D, D // 2 // 16 * 16 or 32]), page=page, q=q,
                    kv=rng.choice([q, "e4m3"]), tree=N <= 64 and rng.random() < 0.5,
                    interleaved=rng.random() < 0.5, lens=lens)
    N = _log(rng, 1, 64)
    B = _log(rng, 1, 64)
    # at most the tree batch's cached tokens, and the wide tree's scores
    most = min(120000, 120000 // B, 16_000_000 // (B * N * G))
    hi = _log(rng, 1, max(1, most))
    return dict(op="attn", B=B, N=N, lo=rng.randint(hi // 8, hi), hi=hi, Hkv=Hkv, G=G, D=D, page=page,
                q=q, kv=rng.choice([q, "e4m3"]), tree=rng.random() < 0.6, lens=lens)


def _lengths(case):
    r = random.Random(case["lens"])
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]


def _accepted(case):
    r = random.Random(case["lens"] + 1)
    return [r.randint(0, min(case["depth"], case["N"] - 1)) for _ in range(case["B"])]


def _paths(case):
    """Root-to-node paths: node 0, then increasing node numbers."""
    r = random.Random(case["lens"] + 2)
    return [[0] + sorted(r.sample(range(1, case["N"]), n)) for n in _accepted(case)]


def work(case):
    op = case["op"]
    if op == "rotary":
        n = case["T"] * case["H"]
        return {"bytes": 2 * n * case["D"] * BYTES[case["t"]] + 4 * case["T"] + 4 * case["rd"],
                "flops": 3 * n * case["rd"]}
    row = case["Hkv"] * (case["D"] * BYTES[case["kv"]] + (4 if case["kv"] == "e4m3" else 0))
    if op == "read":
        t = sum(_lengths(case))
        return {"bytes": 2 * t * (row + case["Hkv"] * case["D"] * BYTES[case["to"]]) + 4 * (t // case["page"]) + 64,
                "flops": 2 * t * case["Hkv"] * case["D"]}
    if op == "commit":
        moved = sum(sum(1 for j, x in enumerate(p) if x != j) for p in _paths(case))
        return {"bytes": 2 * 2 * case["L"] * moved * row + 4 * case["B"] * (case["N"] + 3), "flops": 0}
    tokens = case["B"] * case["N"]
    q = case["Hkv"] * case["G"] * case["D"] * BYTES[case["q"]]
    if op == "write":
        kv_in = 2 * case["Hkv"] * case["D"] * BYTES[case["q"]]
        return {"bytes": tokens * (2 * q + kv_in + 2 * row),
                "flops": tokens * (3 * case["rd"] * case["Hkv"] * (case["G"] + 1) + 4 * case["Hkv"] * case["D"])}
    t = sum(_lengths(case)) + tokens
    pairs = sum((n + case["N"] / 2) for n in _lengths(case)) * case["N"]
    return {"bytes": 2 * t * row + 2 * tokens * q + 4 * (t // case["page"]),
            "flops": 4 * pairs * case["Hkv"] * case["G"] * case["D"]}


# ----------------------------------------------------------------- inputs

def _quantise(x):
    """Codes and scales of rows of x (one scale for each row of the last axis)."""
    x = x.float()
    scale = x.abs().amax(-1) / E4M3_MAX
    safe = torch.where(scale > 0, scale, torch.ones_like(scale))
    code = (x / safe[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return code, scale


def _pages(case, lengths, extra, gen):
    """A page table [B, M] over shuffled pages; entries that no token needs are -1."""
    need = [-(-(n + extra) // case["page"]) for n in lengths]
    total = max(1, sum(need))
    order = torch.randperm(total, generator=gen).tolist()
    table = torch.full((len(need), max(1, max(need))), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    return table.cuda(), total


def _pool(case, total, g, layers=None):
    """A cache pool [.., pages, heads, page, D], keys and values of a model's size."""
    shape = (total, case["Hkv"], case["page"], case["D"])
    kv, got = DTYPES[case["kv"]], {}
    for name, spread in (("k", 1.0), ("v", 0.7)):
        parts, scales = [], []
        for _ in range(layers or 1):
            x = torch.randn(shape, device="cuda", generator=g) * spread
            if case["kv"] == "e4m3":
                code, scale = _quantise(x)
                parts.append(code)
                scales.append(scale)
            else:
                parts.append(x.to(kv))
        pool = torch.stack([p.view(torch.uint8) if case["kv"] == "e4m3" else p for p in parts])
        pool = pool.view(torch.float8_e4m3fn) if case["kv"] == "e4m3" else pool
        got[name] = (pool if layers else pool[0]).transpose(-3, -2)  # [.., pages, page, heads, D]
        got[name + "_scale"] = None
        if scales:
            got[name + "_scale"] = torch.stack(scales) if layers else scales[0]
    return got


def _trees(case, gen):
    """Random parents [B, N]: node j hangs below any node before it, near ones more often."""
    B, N = case["B"], case["N"]
    u = torch.rand(B, N, generator=gen)
    j = torch.arange(N)
    parent = torch.minimum((u.sqrt() * j).long(), (j - 1).clamp(min=0))
    return parent.int().cuda()


def _frequencies(rd, base):
    return (base ** (-torch.arange(0, rd, 2, dtype=torch.float64) / rd)).cuda()


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    gen = torch.Generator().manual_seed(seed)
    op = case["op"]
    s = {"case": case}
    if op == "rotary":
        t = DTYPES[case["t"]]
        s["x"] = torch.randn(case["T"], case["H"], case["D"], device="cuda", generator=g).to(t)
        start = int(torch.randint(0, case["far"], (1,), generator=gen))
        s["positions"] = torch.arange(start, start + case["T"], dtype=torch.int32).cuda()
        s["inv_freq"] = _frequencies(case["rd"], case["base"])
        return s
    lengths = _lengths(case)
    s["cache_len"] = torch.tensor(lengths, dtype=torch.int32).cuda()
    if op == "read":
        s["table"], total = _pages(case, lengths, 0, gen)
        s.update(_pool(case, total, g))
        off = [0]
        for n in lengths:
            off.append(off[-1] + n)
        s["offsets"] = torch.tensor(off, dtype=torch.int32).cuda()
        s["total"] = off[-1]
        return s
    N = case["N"]
    s["table"], total = _pages(case, lengths, N, gen)
    if op == "commit":
        s.update(_pool(case, total, g, layers=case["L"]))
        path = torch.full((case["B"], N), -1, dtype=torch.int32)
        for b, p in enumerate(_paths(case)):
            path[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
        s["path"] = path.cuda()
        s["accepted_len"] = torch.tensor(_accepted(case), dtype=torch.int32).cuda()
        return s
    s.update(_pool(case, total, g))
    s["parent"] = _trees(case, gen) if case["tree"] else None
    qt = DTYPES[case["q"]]
    s["q"] = torch.randn(case["B"], N, case["Hkv"] * case["G"], case["D"], device="cuda", generator=g).to(qt)
    if op == "write":
        s["new_k"], s["new_v"] = (torch.randn(case["B"], N, case["Hkv"], case["D"], device="cuda",
                                              generator=g).to(qt) for _ in range(2))
        s["inv_freq"] = _frequencies(case["rd"], 10000.0)
    return s


# ------------------------------------------------------------ plain forms

def _rotate(x, positions, inv_freq, interleaved):
    """x [.., H, D] in 32 bits, rotated; positions [..]."""
    angle = positions.double()[..., None] * inv_freq
    c, s = angle.cos().float()[..., None, :], angle.sin().float()[..., None, :]
    rd = 2 * inv_freq.numel()
    x = x.float()
    part = x[..., :rd]
    if interleaved:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = part[..., :rd // 2], part[..., rd // 2:]
        turned = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((turned, x[..., rd:]), -1)


def _ancestors(parent, N):
    """[B or 1, N, N]: whether node i sees node j (its ancestors and itself)."""
    if parent is None:
        return torch.ones(1, N, N, dtype=torch.bool, device="cuda").tril()
    node = torch.arange(N, device="cuda")
    step = (parent[..., None] == node) & (node[:, None] > 0)
    see = (step | torch.eye(N, dtype=torch.bool, device="cuda")).float()
    for _ in range(6):  # paths of up to 64 steps
        see = (see @ see).clamp(max=1.0)
    return see > 0


def _slots(table, position, page):
    """Page and place in it of each sequence's positions [B, n]."""
    at = table.gather(1, (position // page).long().clamp(max=table.shape[1] - 1)).long()
    return at, (position % page).long()


def _plain_write(s):
    case, (B, N) = s["case"], s["q"].shape[:2]
    node = torch.arange(N, device="cuda", dtype=torch.int32)
    depth = node[None] if s["parent"] is None else _ancestors(s["parent"], N).sum(-1) - 1
    position = s["cache_len"][:, None] + depth
    q = _rotate(s["q"], position, s["inv_freq"], case["interleaved"]).to(s["q"].dtype)
    k = _rotate(s["new_k"], position, s["inv_freq"], case["interleaved"])
    page, place = _slots(s["table"], s["cache_len"][:, None] + node, case["page"])
    for name, x in (("k", k), ("v", s["new_v"])):
        if case["kv"] == "e4m3":
            code, scale = _quantise(x)
            s[name].view(torch.uint8)[page, place] = code.view(torch.uint8)
            s[name + "_scale"].transpose(1, 2)[page, place] = scale
        else:
            s[name][page, place] = x.to(s[name].dtype)
    return q


def _rows(s, name, page, place):
    x = s[name].view(torch.uint8)[page, place].view(torch.float8_e4m3fn) if s[name + "_scale"] is not None \
        else s[name][page, place]
    x = x.float()
    return x if s[name + "_scale"] is None else x * s[name + "_scale"].transpose(1, 2)[page, place][..., None]


def _plain_read(s):
    case, total = s["case"], s["total"]
    n = s["offsets"].diff()
    b = torch.repeat_interleave(torch.arange(case["B"], device="cuda"), n, output_size=total)
    position = torch.arange(total, device="cuda") - s["offsets"][:-1].long()[b]
    page, place = s["table"][b, position // case["page"]].long(), position % case["page"]
    to = DTYPES[case["to"]]
    return {"k": _rows(s, "k", page, place).to(to), "v": _rows(s, "v", page, place).to(to)}


def _plain_commit(s):
    case = s["case"]
    j = torch.arange(case["N"], device="cuda", dtype=torch.int32)[None]
    on = j <= s["accepted_len"][:, None]
    base = s["cache_len"][:, None]
    sp, so = _slots(s["table"], base + torch.where(on, s["path"], 0), case["page"])
    dp, do = _slots(s["table"], base + torch.where(on, j, 0), case["page"])
    for name in ("k", "v"):
        x = s[name].view(torch.uint8) if s[name + "_scale"] is not None else s[name]
        x[:, dp, do] = x[:, sp, so]
        if s[name + "_scale"] is not None:
            y = s[name + "_scale"].transpose(2, 3)
            y[:, dp, do] = y[:, sp, so]
    return s["cache_len"] + s["accepted_len"] + 1


def _plain_attention(s):
    case, (B, N, H, D) = s["case"], s["q"].shape
    page, T = case["page"], s["table"].shape[1] * case["page"]
    position = torch.arange(T, device="cuda", dtype=torch.int32)[None].expand(B, T)
    at, place = _slots(s["table"], position, page)
    at = at.clamp(min=0)
    k, v = _rows(s, "k", at, place), _rows(s, "v", at, place)  # [B, T, Hkv, D]
    q = s["q"].float().reshape(B, N, case["Hkv"], case["G"], D).permute(0, 2, 3, 1, 4)
    score = q.reshape(B, case["Hkv"], case["G"] * N, D) @ k.permute(0, 2, 3, 1)
    score = score.reshape(B, case["Hkv"], case["G"], N, T) * D ** -0.5
    node = (position - s["cache_len"][:, None])[:, None]  # [B, 1, T]
    see = _ancestors(s["parent"], N).expand(B, N, N)
    see = see.gather(2, node.clamp(0, N - 1).long().expand(B, N, T)) & (node < N) | (node < 0)
    score = score.masked_fill(~see[:, None, None], -math.inf)
    p = (score - score.amax(-1, keepdim=True)).exp()
    p = p / p.sum(-1, keepdim=True)
    out = p.reshape(B, case["Hkv"], case["G"] * N, T) @ v.permute(0, 2, 1, 3)
    out = out.reshape(B, case["Hkv"], case["G"], N, D).permute(0, 3, 1, 2, 4).reshape(B, N, H, D)
    return out.to(s["q"].dtype)


def _cached(s):
    names = ("k", "v") if s["k_scale"] is None else ("k", "v", "k_scale", "v_scale")
    return {n: s[n] for n in names}


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if own:
        import speculative_decoding_verification_88_b200 as sv

        if op == "rotary":
            return sv.rotary(s["x"], s["positions"], sv.Rotary(s["inv_freq"], interleaved=case["interleaved"]))
        cache = sv.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        if op == "attn":
            return sv.tree_attention(s["q"], cache, s["table"], s["cache_len"], s["parent"])["out"]
        if op == "read":
            return sv.cache_read(cache, s["table"], s["offsets"], s["total"], DTYPES[case["to"]])
        if op == "write":
            q = sv.cache_write(cache, s["table"], s["cache_len"], s["new_k"], s["new_v"], parent=s["parent"],
                               rope=sv.Rotary(s["inv_freq"], interleaved=case["interleaved"]), q=s["q"])
            return {"q": q, **_cached(s)}
        new_len = sv.cache_commit(cache, s["table"], s["cache_len"],
                                  {"accepted_len": s["accepted_len"], "path": s["path"]})
        return {"len": new_len, **_cached(s)}
    if op == "rotary":
        return _rotate(s["x"], s["positions"], s["inv_freq"], case["interleaved"]).to(s["x"].dtype)
    if op == "attn":
        return _plain_attention(s)
    if op == "read":
        return _plain_read(s)
    if op == "write":
        return {"q": _plain_write(s), **_cached(s)}
    return {"len": _plain_commit(s), **_cached(s)}


# ---------------------------------------------------------------- 64 bits

def _exact_rotation(x, position, inv_freq, interleaved):
    """Each pair as a complex number times exp(i position f)."""
    rd = 2 * inv_freq.numel()
    y = x.double().clone()
    first = slice(0, rd, 2) if interleaved else slice(0, rd // 2)
    second = slice(1, rd, 2) if interleaved else slice(rd // 2, rd)
    z = torch.complex(y[..., first], y[..., second])
    angle = torch.einsum("...,f->...f", position.double(), inv_freq)[..., None, :]
    z = z * torch.polar(torch.ones_like(angle), angle)
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_code(y):
    """Scales in 32 bits, as they are held; codes to the nearest of the 8-bit values, ties to even."""
    scale = (y.abs().amax(-1) / E4M3_MAX).float()
    r = (y / torch.where(scale > 0, scale, 1.0).double()[..., None]).clamp(-E4M3_MAX, E4M3_MAX)
    step = torch.exp2(torch.floor(torch.log2(r.abs().clamp(min=2.0 ** -6))) - 3)  # spacing at r
    return torch.round(r / step) * step, scale.double()


def _values(s, name):
    x = s[name].view(torch.uint8).view(torch.float8_e4m3fn).double() if s[name + "_scale"] is not None \
        else s[name].double()
    return x if s[name + "_scale"] is None else x * s[name + "_scale"].double().transpose(-2, -1)[..., None]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rotary":
        return _exact_rotation(s["x"], s["positions"], s["inv_freq"], case["interleaved"])
    lengths, table = _lengths(case), s["table"].tolist()
    if op == "read":
        got = {}
        for name in ("k", "v"):
            x = _values(s, name)
            got[name] = torch.cat([x[table[b][:-(-n // case["page"])]].flatten(0, 1)[:n]
                                   for b, n in enumerate(lengths)] or [x[:0, 0]])
        return got
    if op == "commit":  # moves: no arithmetic, compared with the plain form's own values
        return None
    B, N, page = case["B"], case["N"], case["page"]
    parent = [[j - 1 for j in range(N)]] * B if s["parent"] is None else s["parent"].tolist()
    up = []  # the nodes that each node sees
    for b in range(B):
        rows = [[0]]
        for j in range(1, N):
            rows.append(rows[parent[b][j]] + [j])
        up.append(rows)
    if op == "write":
        depth = torch.tensor([[len(r) - 1 for r in rows] for rows in up], device="cuda")
        position = s["cache_len"][:, None] + depth
        out = {"q": _exact_rotation(s["q"], position, s["inv_freq"], case["interleaved"])}
        new = {"k": _exact_rotation(s["new_k"], position, s["inv_freq"], case["interleaved"]),
               "v": s["new_v"].double()}
        at = torch.tensor([[table[b][(n + j) // page] * page + (n + j) % page for j in range(N)]
                           for b, n in enumerate(lengths)], device="cuda").flatten()
        for name, y in new.items():
            pool = s[name].double()
            if case["kv"] == "e4m3":
                y, scale = _exact_code(y)
                held = s[name + "_scale"].double().transpose(1, 2).contiguous()
                held.flatten(0, 1)[at] = scale.flatten(0, 1)
                out[name + "_scale"] = held.transpose(1, 2)
            pool = pool.contiguous()
            pool.flatten(0, 1)[at] = y.flatten(0, 1)
            out[name] = pool
        return out
    Hkv, G, D = case["Hkv"], case["G"], case["D"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    # fetched by sequence, so that a long cache is never held whole in 64 bits
    for b, n in enumerate(lengths):
        pages = table[b][:-(-(n + N) // page)]
        part = {**s, **{x: s[x].view(torch.uint8)[pages].view(torch.float8_e4m3fn) if s[x + "_scale"] is not None
                        else s[x][pages] for x in ("k", "v")}}
        for x in ("k_scale", "v_scale"):
            part[x] = None if s[x] is None else s[x][pages]
        k, v = (_values(part, x).flatten(0, 1)[:n + N] for x in ("k", "v"))
        hidden = torch.ones(N, N, dtype=torch.bool)
        for i, r in enumerate(up[b]):
            hidden[i, r] = False
        hidden = hidden.cuda()
        for h in range(Hkv):
            q = s["q"][b, :, h * G:(h + 1) * G].double()  # [N, G, D]
            score = torch.tensordot(q, k[:, h], dims=([2], [1])) / math.sqrt(D)
            score[:, :, n:].masked_fill_(hidden[:, None], -math.inf)
            weight = torch.exp(score - torch.logsumexp(score, -1, keepdim=True))
            out[b, :, h * G:(h + 1) * G] = torch.tensordot(weight, v[:, h], dims=([2], [0]))
    return out
