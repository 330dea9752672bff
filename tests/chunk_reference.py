"""The operators of a prompt chunk in 64 bits, written out plainly in torch.

Test infrastructure: device-agnostic float64 forms of mla_rope_axes,
mla_append_tokens, mla_chunk_attn and mla_linear.  They share no code with the
kernels; test_chunk_reference_cpu.py pins them against the fp64 oracle and
against library routines.
"""
import math

import torch


def rope_axes(x, pos, sections, base, inverse=False):
    """x [n, heads, d_r]; pos [axes, n]; pair i, in the run of axis a, turns by
    pos[a] * base^(-2i / d_r)."""
    x = x.double()
    d_r = x.shape[-1]
    out = torch.empty_like(x)
    i = 0
    for a, count in enumerate(sections):
        for _ in range(count):
            ang = pos[a].double() * base ** (-2.0 * i / d_r)
            c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
            if inverse:
                s = -s
            x0, x1 = x[..., 2 * i], x[..., 2 * i + 1]
            out[..., 2 * i] = x0 * c - x1 * s
            out[..., 2 * i + 1] = x0 * s + x1 * c
            i += 1
    assert 2 * i == d_r
    return out


def new_rows(kv, d_c, pos, sections, base, norm_weight=None, norm_eps=0.0):
    """The cache rows of raw rows kv [n, d_c + d_r], unrounded."""
    kv = kv.double()
    c = kv[:, :d_c]
    if norm_weight is not None:
        c = c / torch.sqrt((c * c).mean(1, keepdim=True) + norm_eps) * norm_weight.double()
    k = rope_axes(kv[:, None, d_c:], pos, sections, base)[:, 0]
    return torch.cat([c, k], 1)


def owners(tok_start, n):
    """Sequence of each token, -1 outside every range."""
    out = [-1] * n
    ts = [int(v) for v in tok_start]
    for b in range(len(ts) - 1):
        for t in range(ts[b], ts[b + 1]):
            out[t] = b
    return out


def slots(tok_start, row0, block_table, n):
    """Flat cache row of each token, -1 outside every range."""
    out = []
    bt = block_table.tolist()
    for t, b in enumerate(owners(tok_start, n)):
        if b < 0:
            out.append(-1)
        else:
            r = int(row0[b]) + t - int(tok_start[b])
            out.append(bt[b][r // 64] * 64 + r % 64)
    return out


def attended(b, cache, block_table, segs, deltas, d_c, base):
    """Rows [R, d_c + d_r] of sequence b with their rotary keys moved to the
    request positions, and those positions."""
    rows, kpos = [], []
    for lo, hi, ver, pos0 in segs[b].tolist():
        if hi <= lo:
            continue
        r = torch.arange(lo, hi, device=cache.device)
        x = cache[block_table[b].long()[r // 64], r % 64].double()
        p = torch.full((1, hi - lo), float(deltas[ver]), dtype=torch.float64, device=cache.device)
        k = x[:, d_c:]
        if deltas[ver]:
            k = rope_axes(k[:, None], p, [k.shape[1] // 2], base)[:, 0]
        rows.append(torch.cat([x[:, :d_c], k], 1))
        kpos.append(pos0 + r - lo)
    if not rows:
        w = cache.shape[-1]
        return cache.new_zeros((0, w), dtype=torch.float64), torch.zeros(0, dtype=torch.int64, device=cache.device)
    return torch.cat(rows), torch.cat(kpos)


def chunk_attn(q, tok_start, q_pos, w_uk, w_uv, cache, block_table, segs, deltas, scale, base,
               heads=None):
    """v [n, H, d_v], lse [n, H] and what scales the error bounds: spread [n, H, d_v] = sum_t a_t
    |V_t|, lat [n, H, d_v] = |W_UV| |sum_t a_t c_t| and key [n, H] = max_t sum_i |q_i K_ti| over the
    seen rows' content.  Rows of tokens outside every range are NaN.  A masked row has no part in
    anything.  ``heads`` limits the work to some heads (the others stay NaN)."""
    n, H, _ = q.shape
    d_c, d_n, d_v = w_uk.shape[2], w_uk.shape[1], w_uv.shape[1]
    nan = dict(dtype=torch.float64, device=q.device)
    v, spread, lat = (torch.full((n, H, d_v), math.nan, **nan) for _ in range(3))
    lse, key = torch.full((n, H), math.nan, **nan), torch.zeros((n, H), **nan)
    ts = [int(t) for t in tok_start]
    for b in range(len(ts) - 1):
        if ts[b + 1] <= ts[b]:
            continue
        mine = slice(ts[b], ts[b + 1])
        rows, kpos = attended(b, cache, block_table, segs, deltas, d_c, base)
        see = kpos[None, :] <= q_pos[mine].long()[:, None]
        any_row = see.any(0)
        rows, see = rows[any_row], see[:, any_row]     # rows that nobody sees are not read
        for h in (range(H) if heads is None else heads):
            K = rows[:, :d_c] @ w_uk[h].double().T
            V = rows[:, :d_c] @ w_uv[h].double().T
            qh = q[mine, h].double()
            s = scale * (qh[:, :d_n] @ K.T + qh[:, d_n:] @ rows[:, d_c:].T)
            s = torch.where(see, s, torch.full_like(s, -math.inf))
            l = torch.logsumexp(s, 1) if s.shape[1] else torch.full((s.shape[0],), -math.inf, **nan)
            a = torch.where(see, torch.exp(s - torch.where(torch.isinf(l), 0.0, l)[:, None]), 0.0)
            # a weight of zero times a value that is not finite: only seen rows count
            num = lambda x: torch.nan_to_num(x, nan=0.0, posinf=0.0, neginf=0.0)
            vals = [a @ num(V), a @ num(V).abs(),
                    (a @ num(rows[:, :d_c])).abs() @ w_uv[h].double().abs().T]
            if rows.shape[0]:
                size = qh[:, :d_n].abs() @ num(K).abs().T
                key[mine, h] = torch.where(see, size, 0.0).amax(1)
            broken = (see & ~torch.isfinite(rows).all(1)[None, :]).any(1)
            for x in vals:
                x[broken] = math.nan
            l[broken] = math.nan
            v[mine, h], spread[mine, h], lat[mine, h], lse[mine, h] = (*vals, l)
    return v, lse, dict(spread=spread, lat=lat, key=key)


def linear(x, w, bias=None, act="none", residual=None):
    y = x.double() @ w.double().T
    if bias is not None:
        y = y + bias.double()
    if act == "silu":
        y = y / (1 + torch.exp(-y))
    elif act == "gelu":
        y = 0.5 * y * (1 + torch.erf(y / math.sqrt(2.0)))
    return y if residual is None else y + residual.double()
