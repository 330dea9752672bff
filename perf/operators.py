"""The operators of a prompt chunk over the paged latent cache, as cases to be measured.

A serving step that takes a chunk of new tokens per sequence rotates the
queries' rotary part (``rope``), writes the new tokens into the paged latent
cache (``append``), attends every new token to its sequence's cached rows
(``chunk``) and applies the output projection with the residual (``linear``).
``run`` computes each either in its plain form, from elementary torch
operations in 32 bits (64 for angles and for what decides a 4- or 2-bit code),
or, when the module's ``own`` is true, by the calls of the package's binding.
"""
import math

import torch

own = False

PAGE = 64
DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
# the latent attention dimensions of the package's configurations, by storage type
DIMS = {"bf16": dict(d_c=512, d_r=64, d_n=128, d_v=128), "f32": dict(d_c=32, d_r=16, d_n=16, d_v=16)}
BASE = 10000.0
FAR = 2 ** 31 - 1


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a decode step's rotary queries: 16 sequences, one new token each; latency
        dict(name="rope_decode", op="rope", dtype="bf16", H=128, n_tok=16, axes=1, inverse=False, far=4096),
        # a video prompt: time, height and width positions, an odd number of tokens
        dict(name="rope_video", op="rope", dtype="bf16", H=64, n_tok=4099, axes=3, inverse=False, far=32768),
        # 64 sequences each append the one token they just made
        dict(name="append_decode", op="append", dtype="bf16", B=64, n_tok=64, tail=0, axes=1, norm=True,
             bits_c=0, past=2000, ragged=False),
        # a long prompt enters the cache: raw latents normalised on the way, three position axes
        dict(name="append_prompt", op="append", dtype="bf16", B=2, n_tok=8192, tail=0, axes=3, norm=True,
             bits_c=0, past=100, ragged=True),
        # ragged chunks of five sequences into an INT4 cache, padded batch
        dict(name="append_int4", op="append", dtype="bf16", B=5, n_tok=1531, tail=21, axes=1, norm=True,
             bits_c=4, past=300, ragged=True),
        # the single-token form: 16 sequences of about 4K cached rows, one new token each
        dict(name="chunk_tokens", op="chunk", dtype="bf16", H=128, B=16, n_tok=16, tail=0, past=4080,
             doc=0, ragged=False),
        # four ragged chunks behind a relocated document, 64 heads, padded batch
        dict(name="chunk_ragged", op="chunk", dtype="bf16", H=64, B=4, n_tok=1333, tail=11, past=1900,
             doc=1000, ragged=True),
        # one long chunk over a long cache, every head: the largest work
        dict(name="chunk_long", op="chunk", dtype="bf16", H=128, B=1, n_tok=2048, tail=0, past=8192,
             doc=0, ragged=False),
        # the fp32 configuration's small dimensions
        dict(name="chunk_f32", op="chunk", dtype="f32", H=8, B=3, n_tok=75, tail=2, past=256, doc=0,
             ragged=True),
        # output projection of 16 decoded tokens onto the residual: the weights are the time
        dict(name="linear_tokens", op="linear", dtype="bf16", M=16, N=7168, K=16384, bias=False, act="none",
             residual=True),
        # the same of a prompt chunk
        dict(name="linear_prompt", op="linear", dtype="bf16", M=4096, N=7168, K=16384, bias=False, act="none",
             residual=True),
        # odd sizes, strides that are no multiple of a tile, bias and activation
        dict(name="linear_odd", op="linear", dtype="bf16", M=333, N=2056, K=1000, bias=True, act="silu",
             residual=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "chunk", "chunk", "linear"])
    dtype = "f32" if rng.random() < 0.15 else "bf16"
    if op == "rope":
        return dict(op=op, dtype=dtype, H=rng.choice([1, 8, 32, 64, 128]), n_tok=_log(rng, 1, 8192),
                    axes=rng.choice([1, 2, 3]), inverse=rng.random() < 0.5, far=_log(rng, 16, 1 << 20))
    if op == "append":
        B = _log(rng, 1, 64)
        return dict(op=op, dtype=dtype, B=B, n_tok=max(B, _log(rng, 1, 8192)), tail=rng.choice([0, 0, 1, 37]),
                    axes=rng.choice([1, 2, 3]), norm=rng.random() < 0.7, bits_c=rng.choice([0, 0, 2, 4]),
                    past=_log(rng, 1, 2000), ragged=rng.random() < 0.7)
    if op == "linear":
        if dtype == "f32":
            return dict(op=op, dtype=dtype, M=_log(rng, 1, 256), N=_log(rng, 1, 1024), K=_log(rng, 1, 1024),
                        bias=rng.random() < 0.5, act=rng.choice(["none", "silu", "gelu"]),
                        residual=rng.random() < 0.5)
        return dict(op=op, dtype=dtype, M=_log(rng, 1, 4096), N=8 * _log(rng, 8, 896), K=8 * _log(rng, 8, 2048),
                    bias=rng.random() < 0.5, act=rng.choice(["none", "silu", "gelu"]),
                    residual=rng.random() < 0.5)
    if dtype == "f32":
        B = rng.choice([1, 2, 3, 5])
        return dict(op=op, dtype=dtype, H=8, B=B, n_tok=max(B, _log(rng, 1, 128)), tail=rng.choice([0, 3]),
                    past=_log(rng, 1, 400), doc=rng.choice([0, 100]), ragged=rng.random() < 0.7)
    H, B = rng.choice([8, 32, 64, 128]), _log(rng, 1, 12)
    n_tok, past = max(B, _log(rng, 1, 2048)), _log(rng, 1, 8192)
    while B * H * n_tok * (past + n_tok) > 128 * 2048 * 10240 or B * H * (past + n_tok) > 3 * 128 * 10240:
        past, B = max(1, past // 2), max(1, B // 2)
    doc = rng.choice([0, 0, 64, 700])
    return dict(op=op, dtype=dtype, H=H, B=B, n_tok=n_tok, tail=rng.choice([0, 0, 5]), past=past,
                doc=doc if doc < past else 0, ragged=rng.random() < 0.7)


# ------------------------------------------------------------------ inputs
def _lens(case):
    """New tokens of each sequence (their sum is n_tok): even, or in the ratio 1 : 2 : .. : B."""
    B, n = case["B"], case["n_tok"]
    w = [b + 1 if case["ragged"] else 1 for b in range(B)]
    cut = [1 * b + (n - B) * sum(w[:b]) // sum(w) for b in range(B + 1)]
    return [cut[b + 1] - cut[b] for b in range(B)]


def _past(case):
    """Cached rows of each sequence before the chunk."""
    return [max(1, case["past"] - 37 * b) if case["ragged"] else case["past"] for b in range(case["B"])]


def _sections(axes, d_r):
    """Rotary pairs of each position axis: all, halves, or a quarter and three eighths twice."""
    half = d_r // 2
    return {1: [half], 2: [half // 2, half - half // 2], 3: [half // 4, half * 3 // 8, half - half // 4 - half * 3 // 8]}[axes]


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device=DEV)


def _offsets(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _pages(g, rows):
    """A block table of pages in random order, unused entries at one spare page; (table, pages of the pool)."""
    need = [-(-r // PAGE) for r in rows]
    total = sum(need)
    perm = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    at = torch.arange(max(need), device=DEV)[None, :]
    first, n = _ints(_offsets(need)[:-1], torch.int64)[:, None], _ints(need, torch.int64)[:, None]
    return torch.where(at < n, perm[(first + at).clamp(max=total - 1)], total).to(torch.int32), total + 1


def prepare(case, seed):
    g, dt = _gen(seed), DTYPES[case["dtype"]]
    s = dict(case=case)
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        s["x"], s["w"] = _normal(g, (M, K), dt), _normal(g, (N, K), dt, 1 / math.sqrt(K))
        s["bias"] = _normal(g, (N,), torch.float32) if case["bias"] else None
        s["residual"] = _normal(g, (M, N), dt) if case["residual"] else None
        s["out"] = torch.zeros((M, N), dtype=dt, device=DEV)
        return s
    d = DIMS[case["dtype"]]
    s["dims"] = dict(d, H=case.get("H", 8), d_model=7168 if case["dtype"] == "bf16" else 128)
    if case["op"] == "rope":
        H, n = case["H"], case["n_tok"]
        s["q"] = _normal(g, (n, H, d["d_n"] + d["d_r"]), dt)
        # neighbouring tokens have neighbouring positions; the last one is the farthest
        s["pos"] = (case["far"] - n + torch.arange(n, device=DEV)[None, :] //
                    _ints([1, 16, 1], torch.int64)[:case["axes"], None]).to(torch.int32).contiguous()
        s["sections"] = _sections(case["axes"], d["d_r"])
        s["out"] = torch.zeros_like(s["q"])
        return s
    lens, past = _lens(case), _past(case)
    starts = _offsets(lens)
    s["tok_start"], s["total"] = _ints(starts), starts[-1]
    n_all = starts[-1] + case["tail"]
    rows = [p + n for p, n in zip(past, lens)]
    if case["op"] == "append":
        s["block_table"], n_pages = _pages(g, rows)
        s["row0"] = _ints(past)
        s["kv"] = _normal(g, (n_all, d["d_c"] + d["d_r"]), dt, 1.5)
        s["norm_weight"] = 1 + 0.1 * torch.randn(d["d_c"], generator=g, device=DEV) if case["norm"] else None
        step = torch.arange(n_all, device=DEV)[None, :] // _ints([1, 16, 1], torch.int64)[:case["axes"], None]
        s["pos"] = (step + case["past"]).to(torch.int32).contiguous()
        s["sections"] = _sections(case["axes"], d["d_r"])
        if case["bits_c"]:
            size = 1.0 if case["norm"] else 1.5
            low = 0.35 if case["bits_c"] == 4 else 0.9
            s["scale_c"] = size * (low + 0.1 * torch.rand(d["d_c"], generator=g, device=DEV))
            s["scale_r"] = 0.5 + 0.1 * torch.rand(d["d_r"], generator=g, device=DEV)
            width = (d["d_c"] * case["bits_c"] + d["d_r"] * 4) // 8
            s["cache"] = torch.randint(0, 256, (n_pages, PAGE, width), generator=g, device=DEV, dtype=torch.uint8)
        else:
            s["cache"] = _normal(g, (n_pages, PAGE, d["d_c"] + d["d_r"]), dt)
        return s
    H, B = case["H"], case["B"]
    # segments: rows before the document, then (with a document) rows cached at positions from 0
    doc = case["doc"]
    segs, held = [], []
    for r in rows:
        pre = (r - doc) // PAGE * PAGE if doc and r > doc + PAGE else 0
        segs.append([[0, r, 0, 0], [0, 0, 0, 0]] if not pre else [[0, pre, 0, 0], [pre, r, 1, pre]])
        held.append(r)
    s["segs"] = _ints(segs)
    s["deltas"] = [0, 512] if doc else [0]
    s["block_table"], n_pages = _pages(g, held)
    s["max_rows"] = sum(-(-r // PAGE) * PAGE for r in held) + (PAGE * B if doc else 0)
    s["cache"] = _normal(g, (n_pages, PAGE, d["d_c"] + d["d_r"]), dt)
    s["cache"][-1] = float("nan")   # the spare page is never read
    s["q"] = _normal(g, (n_all, H, d["d_n"] + d["d_r"]), dt)
    pos = [p + i for p, n in zip(past, lens) for i in range(n)] + [0] * case["tail"]
    s["q_pos"] = _ints(pos)
    s["w_uk"] = _normal(g, (H, d["d_n"], d["d_c"]), dt, 1 / math.sqrt(d["d_c"]))
    s["w_uv"] = _normal(g, (H, d["d_v"], d["d_c"]), dt, 1 / math.sqrt(d["d_c"]))
    s["most"] = max(lens)
    s["v"] = torch.zeros((n_all, H, d["d_v"]), dtype=dt, device=DEV)
    return s


# ------------------------------------------------------------------ the package's calls
def _own(s):
    from head_latent_attention_02_b200 import mla
    case = s["case"]
    if case["op"] == "linear":
        if "ws" not in s:
            size = mla.linear_workspace_size(s["x"], s["w"])
            s["ws"] = torch.empty(max(size, 256), dtype=torch.uint8, device=DEV)
        mla.linear(s["x"], s["w"], s["out"], bias=s["bias"], act=case["act"], residual=s["residual"],
                   workspace=s["ws"])
        return s["out"]
    d = s["dims"]
    if "call_dims" not in s:
        s["call_dims"] = mla.Dims(d["H"], d["d_c"], d["d_r"], d["d_n"], d["d_v"], d["d_model"], PAGE,
                                  mla.MLA_BF16 if case["dtype"] == "bf16" else mla.MLA_F32,
                                  1 / math.sqrt(d["d_n"] + d["d_r"]), BASE)
    dims = s["call_dims"]
    if case["op"] == "rope":
        # the rotary part of the projected queries, as the slice it is
        mla.rope_axes(dims, s["q"][..., d["d_n"]:], s["pos"], s["sections"], s["out"][..., d["d_n"]:],
                      inverse=case["inverse"])
        return s["out"][..., d["d_n"]:]
    if case["op"] == "append":
        bits = (case["bits_c"], 4) if case["bits_c"] else None
        mla.append_tokens(dims, s["kv"], s["tok_start"], s["row0"], s["pos"], s["sections"], s["cache"],
                          s["block_table"], norm_weight=s["norm_weight"], norm_eps=1e-6, bits=bits,
                          scale_c=s.get("scale_c"), scale_r=s.get("scale_r"))
        if not bits:
            return s["cache"]
        packed = s["cache"].view(-1, s["cache"].shape[-1])
        if "rows" not in s:
            s["rows"] = torch.empty((packed.shape[0], d["d_c"] + d["d_r"]), dtype=DTYPES[case["dtype"]], device=DEV)
        mla.dequant_rows(dims, case["bits_c"], 4, packed, s["scale_c"], s["scale_r"], s["rows"])
        return s["rows"]
    if "ws" not in s:
        size = mla.chunk_workspace_size(dims, case["B"], s["q"].shape[0], len(s["deltas"]),
                                        s["block_table"].shape[1], s["segs"].shape[1], s["max_rows"])
        s["ws"] = torch.empty(size, dtype=torch.uint8, device=DEV)
    mla.chunk_attn(dims, s["q"], s["tok_start"], s["q_pos"], s["w_uk"], s["w_uv"], s["cache"],
                   s["block_table"], s["segs"], s["deltas"], s["max_rows"], s["v"], s["ws"])
    return s["v"]


# ------------------------------------------------------------------ plain forms
def _act(y, act):
    if act == "silu":
        return y * torch.sigmoid(y)
    return 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5))) if act == "gelu" else y


def _turn(angles, x):
    """Rotates the adjacent pairs of x's last axis by the angles."""
    c, n = torch.cos(angles).to(x.dtype), torch.sin(angles).to(x.dtype)
    x0, x1 = x[..., 0::2], x[..., 1::2]
    return torch.stack([x0 * c - x1 * n, x0 * n + x1 * c], -1).flatten(-2)


def _theta(d_r):
    return BASE ** (-torch.arange(0, d_r, 2, device=DEV, dtype=torch.float64) / d_r)


def _axis_angles(pos, sections, d_r):
    """[tokens, d_r / 2]: pair i turns by its axis' position times its frequency, in 64 bits."""
    axis = torch.repeat_interleave(torch.arange(len(sections), device=DEV), _ints(sections, torch.int64),
                                   output_size=d_r // 2)
    return pos[axis].T.double() * _theta(d_r)


def _owner(starts, n):
    """The sequence of each of the first n tokens, and the token's place in it."""
    t = torch.arange(n, device=DEV)
    b = torch.searchsorted(starts[1:].long(), t, right=True)
    return b, t - starts.long()[b]


def _plain_append(s):
    case, d, n = s["case"], s["dims"], s["total"]
    wide = torch.float64 if case["bits_c"] else torch.float32
    kv, dt = s["kv"][:n].to(wide), DTYPES[case["dtype"]]
    c, k = kv[:, :d["d_c"]], kv[:, d["d_c"]:]
    if s["norm_weight"] is not None:
        c = c / torch.sqrt((c * c).mean(-1, keepdim=True) + 1e-6) * s["norm_weight"].to(wide)
    k = _turn(_axis_angles(s["pos"][:, :n], s["sections"], d["d_r"]), k)
    new = torch.cat([c, k], -1).float().to(dt)
    b, i = _owner(s["tok_start"], n)
    row = s["row0"].long()[b] + i
    slot = s["block_table"].long()[b, row // PAGE] * PAGE + row % PAGE
    flat = s["cache"].view(-1, s["cache"].shape[-1])
    if not case["bits_c"]:
        flat[slot] = new
        return s["cache"]
    scale = torch.cat([s["scale_c"], s["scale_r"]])
    code = torch.round(new.float() / scale)
    bits_c, dc = case["bits_c"], d["d_c"]
    low = 2 ** (bits_c - 1)
    cc, cr = code[:, :dc].clamp(-low, low - 1), code[:, dc:].clamp(-8, 7)
    per = 8 // bits_c
    up = 2 ** (bits_c * torch.arange(per, device=DEV))
    by_c = ((cc.long() % (2 * low)).view(n, -1, per) * up).sum(-1)
    by_r = ((cr.long() % 16).view(n, -1, 2) * _ints([1, 16], torch.int64)).sum(-1)
    flat[slot] = torch.cat([by_c, by_r], -1).to(torch.uint8)
    # the values the codes stand for
    w = dc * bits_c // 8
    f_c = (flat[:, :w, None].long() // up % (2 * low)).flatten(1)
    f_r = (flat[:, w:, None].long() // _ints([1, 16], torch.int64) % 16).flatten(1)
    signed = torch.cat([(f_c + low) % (2 * low) - low, (f_r + 8) % 16 - 8], -1)
    return (signed.float() * scale).to(dt)


def _rows_of(s):
    """The pages' rows [B, rows, width] in 32 bits, rows outside every segment zero, with their positions
    (far beyond every query where there is none) and relocation versions."""
    table, segs = s["block_table"].long(), s["segs"].long()
    B, R = table.shape[0], table.shape[1] * PAGE
    r = torch.arange(R, device=DEV)[None, None, :]
    inside = (r >= segs[:, :, 0:1]) & (r < segs[:, :, 1:2])
    kpos = torch.where(inside, segs[:, :, 3:4] + r - segs[:, :, 0:1], FAR).amin(1)
    ver = torch.where(inside, segs[:, :, 2:3], 0).amax(1)
    rows = s["cache"][table].view(B, R, -1).float()
    return torch.where(inside.any(1)[..., None], rows, 0.0), kpos, ver


def _plain_chunk(s):
    case, d, n = s["case"], s["dims"], s["total"]
    scale = 1 / math.sqrt(d["d_n"] + d["d_r"])
    rows, kpos, ver = _rows_of(s)
    c, k_r = rows[..., :d["d_c"]], rows[..., d["d_c"]:]
    if len(s["deltas"]) > 1:
        # relocated rows: their keys were turned for positions delta before the ones they have here
        k_r = _turn(_ints(s["deltas"], torch.float64)[ver][..., None] * _theta(d["d_r"]), k_r)
    b, i = _owner(s["tok_start"], n)
    q = torch.zeros((case["B"], s["most"]) + s["q"].shape[1:], device=DEV)
    q_pos = torch.full((case["B"], s["most"]), -1, dtype=torch.int64, device=DEV)
    q[b, i], q_pos[b, i] = s["q"][:n].float(), s["q_pos"][:n].long()
    w_uk, w_uv = s["w_uk"].float(), s["w_uv"].float()
    few = s["most"] < 171   # below it the absorbed form is less work than expanding the rows
    q_n, q_r = q[..., :d["d_n"]], q[..., d["d_n"]:]
    scores = torch.einsum("bqhr,blr->bhql", q_r, k_r)
    if few:
        scores += torch.einsum("bqhc,blc->bhql", torch.einsum("bqhn,hnc->bqhc", q_n, w_uk), c)
    else:
        scores += torch.einsum("bqhn,bhln->bhql", q_n, torch.einsum("blc,hnc->bhln", c, w_uk))
    scores.mul_(scale).masked_fill_(kpos[:, None, None, :] > q_pos[:, None, :, None], -math.inf)
    top = scores.amax(-1, keepdim=True).clamp(min=-1e30)
    p = scores.sub_(top).exp_()
    p /= p.sum(-1, keepdim=True).clamp(min=1e-30)
    if few:
        v = torch.einsum("bqhc,hdc->bqhd", torch.einsum("bhql,blc->bqhc", p, c), w_uv)
    else:
        v = torch.einsum("bhql,bhld->bqhd", p, torch.einsum("blc,hdc->bhld", c, w_uv))
    s["v"][:n] = v[b, i].to(s["v"].dtype)
    return s["v"]


def run(state):
    if own:
        return _own(state)
    s, case = state, state["case"]
    if case["op"] == "linear":
        y = s["x"].float() @ s["w"].float().T
        if s["bias"] is not None:
            y = y + s["bias"]
        y = _act(y, case["act"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return y.to(s["out"].dtype)
    if case["op"] == "rope":
        d = s["dims"]
        angles = _axis_angles(s["pos"], s["sections"], d["d_r"])[:, None, :]
        return _turn(-angles if case["inverse"] else angles, s["q"][..., d["d_n"]:].float()).to(s["q"].dtype)
    return _plain_append(s) if case["op"] == "append" else _plain_chunk(s)


# ------------------------------------------------------------------ floors
def _visible(case):
    """(query, row) pairs that attend, rows held, for each sequence."""
    out = []
    for past, n in zip(_past(case), _lens(case)):
        out.append((n * past + n * (n + 1) // 2, past + n, n))
    return out


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": e * (M * K + N * K + M * N * (2 if case["residual"] else 1)) + (4 * N if case["bias"] else 0),
                "flops": 2 * M * N * K}
    d = DIMS[case["dtype"]]
    if case["op"] == "rope":
        values = case["n_tok"] * case["H"] * d["d_r"]
        return {"bytes": 2 * e * values + 4 * case["axes"] * case["n_tok"], "flops": 3 * values}
    if case["op"] == "append":
        n, width = case["n_tok"], d["d_c"] + d["d_r"]
        held = (d["d_c"] * case["bits_c"] + d["d_r"] * 4) // 8 if case["bits_c"] else e * width
        work_bytes = n * (e * width + held + 4 * case["axes"])
        if case["bits_c"]:   # the whole pool is read back as the values it stands for
            pool = (sum(-(-(p + m) // PAGE) for p, m in zip(_past(case), _lens(case))) + 1) * PAGE
            work_bytes += pool * (held + e * width)
        return {"bytes": work_bytes, "flops": n * (4 * d["d_c"] + 3 * d["d_r"])}
    H, width = case["H"], d["d_c"] + d["d_r"]
    flops = 0
    for pairs, rows, n in _visible(case):
        expanded = 2 * pairs * (d["d_n"] + d["d_r"] + d["d_v"]) + 2 * rows * d["d_c"] * (d["d_n"] + d["d_v"])
        absorbed = 2 * pairs * (2 * d["d_c"] + d["d_r"]) + 2 * n * d["d_c"] * (d["d_n"] + d["d_v"])
        flops += H * min(expanded, absorbed)
    rows, n = sum(v[1] for v in _visible(case)), case["n_tok"]
    return {"bytes": e * (rows * width + n * H * (d["d_n"] + d["d_r"] + d["d_v"]) + H * d["d_c"] * (d["d_n"] + d["d_v"])),
            "flops": flops}


# ------------------------------------------------------------------ 64-bit definitions
def _exact_linear(s, case):
    y = s["x"].double().matmul(s["w"].double().t())
    if s["bias"] is not None:
        y += s["bias"].double()
    if case["act"] == "silu":
        y = y / (1 + torch.exp(-y))
    elif case["act"] == "gelu":
        y = y * torch.special.ndtr(y)
    return y + s["residual"].double() if s["residual"] is not None else y


def _spin(x, angles):
    """Pairs as complex numbers, turned by exp(i angle)."""
    z = torch.view_as_complex(x.double().unflatten(-1, (-1, 2)).contiguous())
    return torch.view_as_real(z * torch.polar(torch.ones_like(angles), angles)).flatten(-2)


def _pair_angles(s, n, d_r):
    first, cols = 0, []
    for a, count in enumerate(s["sections"]):
        freq = torch.exp(-math.log(BASE) * 2 / d_r * torch.arange(first, first + count, device=DEV, dtype=torch.float64))
        cols.append(s["pos"][a, :n].double()[:, None] * freq)
        first += count
    return torch.cat(cols, 1)


def _exact_append(s, case):
    d, n = s["dims"], s["total"]
    x = s["kv"][:n].double()
    c = x[:, :d["d_c"]]
    if s["norm_weight"] is not None:
        c = c * torch.rsqrt(c.square().mean(1, keepdim=True) + 1e-6) * s["norm_weight"].double()
    rows = torch.cat([c, _spin(x[:, d["d_c"]:], _pair_angles(s, n, d["d_r"]))], 1)
    starts, firsts = s["tok_start"].tolist(), s["row0"].tolist()
    table = s["block_table"].tolist()
    where = [table[b][(firsts[b] + i) // PAGE] * PAGE + (firsts[b] + i) % PAGE
             for b in range(case["B"]) for i in range(starts[b + 1] - starts[b])]
    flat = s["cache"].reshape(-1, s["cache"].shape[-1])
    if not case["bits_c"]:
        out = flat.double()
        out[_ints(where, torch.int64)] = rows
        return out.view(s["cache"].shape)
    scale = torch.cat([s["scale_c"], s["scale_r"]])
    bits = [case["bits_c"]] * d["d_c"] + [4] * d["d_r"]
    edge = 2.0 ** (_ints(bits, torch.float64) - 1)
    stored = rows.float().to(DTYPES[case["dtype"]]).float()   # a row is rounded to the storage type first
    code = torch.round(stored / scale).double()
    code = torch.minimum(torch.maximum(code, -edge), edge - 1)
    at = torch.tensor(_offsets(bits)[:-1], device=DEV)
    field = (flat.long()[:, at // 8] >> (at % 8)) & (2 * edge.long() - 1)
    out = torch.where(field >= edge.long(), field - 2 * edge.long(), field).double()
    out[_ints(where, torch.int64)] = code
    return (out.float() * scale).to(DTYPES[case["dtype"]]).double()


def _exact_chunk(s, case):
    d, scale = s["dims"], 1 / math.sqrt(s["dims"]["d_n"] + s["dims"]["d_r"])
    out = s["v"].double()
    starts = s["tok_start"].tolist()
    theta = torch.exp(-math.log(BASE) * 2 / d["d_r"] * torch.arange(d["d_r"] // 2, device=DEV, dtype=torch.float64))
    for b, segments in enumerate(s["segs"].tolist()):
        rows, pos = [], []
        for lo, hi, version, base in segments:
            if hi <= lo:
                continue
            at = torch.arange(lo, hi, device=DEV)
            x = s["cache"][s["block_table"][b].long()[at // PAGE], at % PAGE].double()
            turned = _spin(x[:, d["d_c"]:], (s["deltas"][version] * theta).expand(hi - lo, -1).contiguous())
            rows.append(torch.cat([x[:, :d["d_c"]], turned], 1))
            pos.append(base + at - lo)
        rows, pos = torch.cat(rows), torch.cat(pos)
        mine = slice(starts[b], starts[b + 1])
        q = s["q"][mine].double()
        hidden = pos[None, :] > s["q_pos"][mine].long()[:, None]
        for h in range(case["H"]):
            key = torch.cat([rows[:, :d["d_c"]] @ s["w_uk"][h].double().t(), rows[:, d["d_c"]:]], 1)
            weight = torch.softmax((q[:, h] @ key.t() * scale).masked_fill(hidden, -math.inf), -1)
            out[mine, h] = weight @ (rows[:, :d["d_c"]] @ s["w_uv"][h].double().t())
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        return _exact_linear(s, case)
    if case["op"] == "rope":
        angles = _pair_angles(s, case["n_tok"], s["dims"]["d_r"])
        return _spin(s["q"][..., s["dims"]["d_n"]:], (-angles if case["inverse"] else angles)[:, None, :].expand(-1, case["H"], -1).contiguous())
    return _exact_append(s, case) if case["op"] == "append" else _exact_chunk(s, case)
