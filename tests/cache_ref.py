"""Plain 64-bit forms of the cache-side operators, one sequence at a time."""
import math

import torch

E4M3_MAX = 448.0


def rotate(x, pos, inv_freq, interleaved=False, magnitude=1.0, inverse=False):
    """x [..., H, D], pos [...]: the rotation in 64 bits."""
    y = x.double().cpu().clone()
    f = inv_freq.double().cpu()
    rd = 2 * f.numel()
    ang = pos.cpu().double()[..., None] * f
    c, s = (ang.cos() * magnitude)[..., None, :], (ang.sin() * magnitude)[..., None, :]
    if inverse:
        s = -s
    if interleaved:
        a, b = y[..., 0:rd:2].clone(), y[..., 1:rd:2].clone()
        y[..., 0:rd:2], y[..., 1:rd:2] = a * c - b * s, b * c + a * s
    else:
        a, b = y[..., :rd // 2].clone(), y[..., rd // 2:rd].clone()
        y[..., :rd // 2], y[..., rd // 2:rd] = a * c - b * s, b * c + a * s
    return y


def code_rows(y):
    """e4m3 values (as doubles) and float scales of rows of y, from exact arithmetic."""
    scale = (y.abs().amax(-1) / E4M3_MAX).float()
    r = y / torch.where(scale > 0, scale, torch.ones_like(scale)).double()[..., None]
    r = r.clamp(-E4M3_MAX, E4M3_MAX)
    step = torch.exp2(torch.floor(torch.log2(r.abs().clamp(min=2.0 ** -6))) - 3)
    code = torch.round(r / step) * step  # torch rounds halves to even
    bad = ~torch.isfinite(y).all(-1)
    scale[bad] = math.nan
    return code, scale


def ancestors(parent, N, count=None):
    """For each node its sorted ancestors and itself, or [] when it sees nothing."""
    n = N if count is None else max(0, min(N, count))
    rows = []
    for j in range(N):
        if j >= n:
            rows.append([])
        elif j == 0:
            rows.append([0])
        else:
            p = j - 1 if parent is None else int(parent[j])
            rows.append(rows[p] + [j] if 0 <= p < j and rows[p] else [])
    return rows


def depths(parent, N):
    """Depth of each node as the cache write counts it (an invalid parent: a root)."""
    d = []
    for j in range(N):
        p = j - 1 if parent is None else int(parent[j])
        d.append(d[p] + 1 if j > 0 and 0 <= p < j else 0)
    return d


def pool_rows(cache, table_row, positions):
    """K and V of a sequence's positions as doubles [n, H, D] on the CPU, and
    which positions have a place."""
    pages = cache.k.shape[-4]
    ok = []
    for t in positions:
        i = t // cache.page_size
        ok.append(i < len(table_row) and 0 <= table_row[i] < pages)
    got = []
    for x, sc in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        x = (x.view(torch.uint8).cpu().view(x.dtype) if sc is not None else x.cpu())
        sc = None if sc is None else sc.cpu()
        rows = []
        for t, good in zip(positions, ok):
            pg, pl = (table_row[t // cache.page_size], t % cache.page_size) if good else (0, 0)
            r = x[pg, pl].double()
            rows.append(r if sc is None else r * sc[pg, :, pl].double()[:, None])
        got.append(torch.stack(rows) if rows else torch.zeros(0, cache.num_heads, cache.head_dim).double())
    return got[0], got[1], ok


def attention(q, cache, table, cache_len, parent=None, count=None, scale=None):
    """out, lse and the terms of an error bound: for each output the sum of
    w |v| and, for each row, the largest scale * sum |q k| over what it sees."""
    B, N, Hq, D = q.shape
    G = Hq // cache.num_heads
    scale = D ** -0.5 if scale is None else scale
    q = q.double().cpu()
    out = torch.zeros(B, N, Hq, D, dtype=torch.float64)
    lse = torch.full((B, N, Hq), -math.inf, dtype=torch.float64)
    wabs = torch.zeros_like(out)
    smax = torch.zeros(B, N, Hq, dtype=torch.float64)
    for b in range(B):
        L = max(0, int(cache_len[b]))
        row = table[b].tolist()
        rows = ancestors(None if parent is None else parent[b].tolist(), N,
                         None if count is None else int(count[b]))
        K, V, ok = pool_rows(cache, row, range(L + N))
        for i in range(N):
            see = [t for t in range(L) if ok[t]] + [L + j for j in rows[i] if ok[L + j]]
            if not rows[i] or not see:
                continue
            k, v = K[see], V[see]
            for h in range(Hq):
                s = scale * (k[:, h // G] @ q[b, i, h])
                lse[b, i, h] = torch.logsumexp(s, 0)
                if lse[b, i, h] == -math.inf:
                    continue
                w = torch.exp(s - lse[b, i, h])
                out[b, i, h] = w @ v[:, h // G]
                wabs[b, i, h] = w @ v[:, h // G].abs()
                smax[b, i, h] = abs(scale) * (k[:, h // G].abs() @ q[b, i, h].abs()).max()
    return out, lse, wabs, smax
