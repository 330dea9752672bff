"""mla_chunk_attn against its 64-bit form, and a run of the four chunk operators.

Bounds for bf16.  S_t = scale * sum q_i K_i with K rounded to bf16 (expanded
route) or q absorbed and rounded (absorbed route): off by at most
d = scale * sum |q_i| |K_i| 2^-8 over the content part, so a weight is off by a
factor within exp(2 d).  Each weight and each value row is rounded once (2^-8
each; the absorbed route rounds the weights and the weighted latent instead, the
latter seen through W_UV), and the result once: every value lies within
(exp(2 d) (1 + 2^-8)^2 - 1) sum_t a_t |V_t| + 2^-8 |v| plus, for the absorbed
route, 2^-8 |W_UV| |o_lat| (1e-6: the fp32 sums).  That is the worst case; over
independent roundings the L2 error is at most about sqrt(4) 2^-8 / sqrt(3) =
4.5e-3, below the bar of 1e-2 that the decode tests use, as is the error of
lse (d over independent roundings of 128 products).  fp32: the decode tests'
bar, 1e-5.
"""
import math

import numpy as np
import pytest
import torch

from head_latent_attention_02_b200 import mla, runner
from tests import chunk_reference as R

pytestmark = pytest.mark.gpu
BASE = 10000.0
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from head_latent_attention_02_b200 import build
    build.build()
    mla.lib()
    assert mla.get_status() == 0


def _i32(v):
    return torch.as_tensor(np.asarray(v, np.int32), device="cuda")


class Case:
    """Sequences of cached rows with new tokens at their ends, pages in random
    order, NaN in every row that no segment holds and in a spare page."""

    def __init__(self, kind, H, lens, past, doc=0, tail=0, d=None, seed=0, base_page=0, n_pages=None,
                 deltas=(0, 512)):
        d = d or (dict(d_c=512, d_r=64, d_n=128, d_v=128) if kind == "bf16"
                  else dict(d_c=32, d_r=16, d_n=16, d_v=16))
        self.kind, self.H, self.B, self.d = kind, H, len(lens), d
        dt = BF if kind == "bf16" else torch.float32
        g = torch.Generator(device="cuda").manual_seed(seed + H + sum(lens))
        rn = lambda *s: torch.randn(*s, device="cuda", generator=g)
        self.scale = 1 / math.sqrt(d["d_n"] + d["d_r"])
        self.dims = mla.Dims(H, d["d_c"], d["d_r"], d["d_n"], d["d_v"], 256, 64,
                             mla.MLA_BF16 if kind == "bf16" else mla.MLA_F32, self.scale, BASE)
        starts = np.concatenate([[0], np.cumsum(lens)])
        self.n, self.total = int(starts[-1]) + tail, int(starts[-1])
        rows = [p + n for p, n in zip(past, lens)]
        segs = []
        for r in rows:
            pre = (r - doc) // 64 * 64 if doc and r > doc + 64 else 0
            segs.append([[0, r, 0, 0], [0, 0, 0, 0]] if not pre else [[0, pre, 0, 0], [pre, r, 1, pre]])
        need = [-(-r // 64) for r in rows]
        used = sum(need)
        n_pages = n_pages or used + 1
        perm = base_page + torch.randperm(used, generator=g, device="cuda").cpu().numpy()
        bt = np.full((self.B, max(need + [1])), n_pages - 1, np.int32)
        at = 0
        for b, k in enumerate(need):
            bt[b, :k] = perm[at:at + k]
            at += k
        self.cache = (torch.empty(n_pages, 64, d["d_c"] + d["d_r"], device="cuda", dtype=dt) if base_page else
                      torch.full((n_pages, 64, d["d_c"] + d["d_r"]), math.nan, device="cuda", dtype=dt))
        for b, r in enumerate(rows):
            if r:
                t = torch.arange(r, device="cuda")
                pg = _i32(bt[b]).long()[t // 64]
                self.cache[pg, t % 64] = rn(r, d["d_c"] + d["d_r"]).to(dt)
        self.q = rn(self.n, H, d["d_n"] + d["d_r"]).to(dt)
        self.w_uk = (rn(H, d["d_n"], d["d_c"]) / math.sqrt(d["d_c"])).to(dt)
        self.w_uv = (rn(H, d["d_v"], d["d_c"]) / math.sqrt(d["d_c"])).to(dt)
        self.ts, self.segs, self.bt = _i32(starts), _i32(segs), _i32(bt)
        pos = np.zeros(self.n, np.int32)
        for b in range(self.B):
            pos[starts[b]:starts[b + 1]] = past[b] + np.arange(lens[b])
        self.q_pos = _i32(pos)
        self.deltas = list(deltas) if doc else [0]
        self.max_rows = sum(need) * 64 + (64 * self.B if doc else 0)
        self.v = torch.full((self.n, H, d["d_v"]), 7.0, device="cuda", dtype=dt)
        self.lse = torch.full((self.n, H), 7.0, device="cuda")

    def workspace(self, fill=0xff):
        size = mla.chunk_workspace_size(self.dims, self.B, self.n, len(self.deltas), self.bt.shape[1],
                                        self.segs.shape[1], self.max_rows)
        assert size > 0
        return torch.full((size,), fill, dtype=torch.uint8, device="cuda")    # NaN bits

    def run(self, ws=None, lse=True, stream=None):
        mla.chunk_attn(self.dims, self.q, self.ts, self.q_pos, self.w_uk, self.w_uv, self.cache, self.bt,
                       self.segs, self.deltas, self.max_rows, self.v, self.workspace() if ws is None else ws,
                       lse=self.lse if lse else None, stream=stream)
        return self

    def reference(self, heads=None):
        return R.chunk_attn(self.q, self.ts, self.q_pos, self.w_uk, self.w_uv, self.cache, self.bt, self.segs,
                            self.deltas, self.scale, BASE, heads)

    def check(self, status=0, heads=None):
        torch.cuda.synchronize()
        assert mla.get_status() == status
        v, lse, by = self.reference(heads)
        hs = list(range(self.H)) if heads is None else heads
        got, want = self.v[:self.total][:, hs].double(), v[:self.total][:, hs]
        gl, wl = self.lse[:self.total][:, hs].double(), lse[:self.total][:, hs]
        spread, lat, key = (by[k][:self.total][:, hs] for k in ("spread", "lat", "key"))
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert (self.v[self.total:] == 7).all() and (self.lse[self.total:] == 7).all()
        inf = torch.isinf(wl)
        assert torch.equal(torch.isinf(gl), inf) and (gl[inf] < 0).all()
        fine = ~torch.isnan(want)
        if self.kind == "bf16":
            step = 2.0 ** -8
            factor = torch.exp(2 * self.scale * key * step)[..., None] * (1 + step) ** 2 - 1
            tol = factor * spread + step * lat * (1 + factor) + step * want.abs() + 1e-6
            rel, dl = 1e-2, 1e-2
        else:
            tol = torch.full_like(want, 1e-5)
            rel, dl = 1e-5, 1e-5
        assert ((got - want).abs() <= tol)[fine].all()
        if fine.any():
            assert (got - want)[fine].norm() <= rel * want[fine].norm() + 1e-30
        keep = torch.isfinite(wl)
        assert (gl - wl)[keep].abs().le(dl).all()


SMALL = [
    ([1], [0], 0, 0), ([1] * 6, [0, 1, 63, 64, 65, 300], 0, 0), ([3, 0, 17, 1], [5, 9, 126, 700], 0, 4),
    ([40, 2], [100, 900], 100, 1), ([0, 0], [64, 3], 0, 2),
]


@pytest.mark.parametrize("lens,past,doc,tail", SMALL)
@pytest.mark.parametrize("H", [1, 5, 128])
def test_few_tokens(lens, past, doc, tail, H):
    Case("bf16", H, lens, past, doc, tail).run().check()


@pytest.mark.parametrize("lens,past,doc,tail", SMALL + [([200, 64], [10, 333], 64, 3)])
@pytest.mark.parametrize("d", [None, dict(d_c=40, d_r=6, d_n=7, d_v=9), dict(d_c=300, d_r=32, d_n=24, d_v=136)])
def test_fp32(lens, past, doc, tail, d):
    Case("f32", 3, lens, past, doc, tail, d=d).run().check()


@pytest.mark.parametrize("d", [dict(d_c=64, d_r=16, d_n=24, d_v=40), dict(d_c=512, d_r=64, d_n=64, d_v=96)])
def test_bf16_other_widths(d):
    Case("bf16", 3, [40, 2, 1], [100, 900, 0], 100, 1, d=d).run().check()


@pytest.mark.parametrize("kind,d", [("bf16", dict(d_c=42, d_r=6, d_n=9, d_v=7)), ("bf16", dict(d_c=600, d_r=8, d_n=8, d_v=8)),
                                    ("f32", dict(d_c=4, d_r=4, d_n=1, d_v=1)), ("f32", dict(d_c=516, d_r=2, d_n=3, d_v=2))])
def test_generic_widths(kind, d):
    """Rows of whole and of broken groups of four elements, narrow and wide ones."""
    Case(kind, 2, [40, 2, 1], [200, 300, 0], 100, 1, d=d).run().check()


LARGE = [
    ([256], [0], 0, 0), ([512], [128], 0, 0), ([513], [1], 0, 0), ([700], [63], 0, 5), ([1100], [1000], 0, 0),
    ([300, 0, 333, 290], [64, 700, 129, 5], 0, 7), ([400, 600], [700, 1500], 500, 0), ([257], [4000], 0, 0),
]


@pytest.mark.parametrize("lens,past,doc,tail", LARGE)
@pytest.mark.parametrize("H", [1, 8])
def test_chunks(lens, past, doc, tail, H):
    c = Case("bf16", H, lens, past, doc, tail)
    if lens != [257]:            # with few heads its long context goes to the absorbed route
        assert c.workspace().numel() > c.max_rows * H * 512        # the expanded route
    c.run().check()


def test_a_chunk_over_a_long_context():
    c = Case("bf16", 64, [257], [4000])
    assert c.workspace().numel() > c.max_rows * 64 * 512
    c.run().check(heads=[0, 17, 63])


def test_every_head_of_a_wide_layer():
    Case("bf16", 128, [290, 600], [500, 130]).run().check(heads=[0, 1, 63, 127])


@pytest.mark.parametrize("size", [2.0 ** -12, 2.0 ** -3, 2.0 ** 9, 2.0 ** 14, 2.0 ** 60])
def test_values_of_every_size(size):
    """Values are held as halves between limits on their size and as bfloat16 outside them."""
    c = Case("bf16", 4, [300, 280], [100, 300])
    c.w_uv.mul_(size)
    c.run()
    torch.cuda.synchronize()
    assert mla.get_status() == 0
    v, _, _ = c.reference()
    off = (c.v.double() - v).norm() / v.norm()
    # K (about 0.8 of a rounding in the scores), the result, and weights and values in bfloat16
    assert off <= (2.3e-3 if 0.125 <= size <= 512 else 4.5e-3)
    # the last row, seen by one token alone, far larger than all others
    c.cache[int(c.bt[0, 399 // 64]), 399 % 64, :512] = 2.0 ** 40
    c.run()
    torch.cuda.synchronize()
    assert torch.isfinite(c.v.float()).all() or size > 2.0 ** 50
    others = [t for t in range(580) if t != 299]
    assert (c.v[others].double() - v[others]).norm() <= 4.5e-3 * v[others].norm()


def test_heads_in_groups():
    """More than 1 GiB of keys and values: the heads run in several passes."""
    c = Case("bf16", 128, [512], [17000])
    rows = -(-c.max_rows // 64) * 64
    assert c.workspace(0).numel() < rows * 128 * 512
    c.run().check(heads=[0, 62, 63, 64, 65, 127])


def test_negative_and_far_relocation():
    for deltas in [(0, -3000), (7, 100000)]:
        Case("bf16", 4, [300], [400], 200, deltas=deltas).run().check()
        Case("bf16", 4, [3], [400], 200, deltas=deltas).run().check()
        Case("f32", 4, [3], [400], 200, deltas=deltas).run().check()


@pytest.mark.parametrize("kind,lens", [("bf16", [3, 2]), ("bf16", [300, 280]), ("f32", [30, 4])])
def test_tokens_that_see_nothing(kind, lens):
    c = Case(kind, 4, lens, [100, 10])
    c.q_pos[1] = -1
    c.q_pos[lens[0]:] = -5
    c.run().check()
    assert (c.v[1] == 0).all() and torch.isinf(c.lse[1]).all()
    assert (c.v[lens[0]:] == 0).all()
    # positions out of order, and one that sees everything
    c.q_pos[0], c.q_pos[1] = 2 ** 31 - 1, 50
    c.run().check()


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("kind,lens", [("bf16", [300]), ("bf16", [700, 290]), ("f32", [20]), ("bf16", [3, 2]),
                                       ("bf16", [40])])
def test_what_a_masked_row_holds_does_not_matter(kind, lens, bad):
    """Rows behind a token: the last cached row is seen by the last token alone, and only it."""
    c = Case(kind, 4, lens, [100] * len(lens))
    last = 100 + lens[0] - 1
    page = int(c.bt[0, last // 64])
    for col in (0, 511 if kind == "bf16" else 31):
        keep = c.cache[page, last % 64, col].clone()
        c.cache[page, last % 64, col] = bad
        c.run()
        torch.cuda.synchronize()
        assert mla.get_status() == 0
        v, _, _ = c.reference()
        at = lens[0] - 1
        assert torch.isnan(c.v[at]).all()
        others = [t for t in range(c.total) if t != at]
        assert torch.isfinite(c.v[others]).all()
        assert (c.v[others].double() - v[others]).norm() <= 1e-2 * v[others].norm()
        c.cache[page, last % 64, col] = keep
    c.run().check()


@pytest.mark.parametrize("kind,lens", [("bf16", [3, 2, 4]), ("bf16", [300, 280, 290]), ("f32", [30, 4, 9])])
def test_invalid_sequences_get_nan_and_leave_the_others(kind, lens):
    past = [100, 200, 300]
    ref = Case(kind, 4, lens, past).run()
    torch.cuda.synchronize()
    assert mla.get_status() == 0
    a, b = lens[0], lens[0] + lens[1]
    breaks = {
        "page": lambda c: c.bt.__setitem__((1, 1), c.cache.shape[0]),
        "negative page": lambda c: c.bt.__setitem__((1, 0), -1),
        "row_begin": lambda c: c.segs.__setitem__((1, 0, 0), 3),
        "row_end": lambda c: c.segs.__setitem__((1, 0, 1), 1 << 20),
        "version": lambda c: c.segs.__setitem__((1, 0, 2), 1),
    }
    for name, f in breaks.items():
        c = Case(kind, 4, lens, past)
        f(c)
        c.run()
        torch.cuda.synchronize()
        assert mla.get_status() == 6, name
        assert mla.get_status() == 0
        assert torch.isnan(c.v[a:b]).all() and torch.isnan(c.lse[a:b]).all(), name
        assert torch.equal(c.v[:a], ref.v[:a]) and torch.equal(c.v[b:], ref.v[b:]), name
    # token ranges out of order or past the tokens: left out, nothing written there
    for at, val in ((1, a + lens[1] + 50), (2, -1), (3, c.n + 1)):
        c = Case(kind, 4, lens, past)
        c.ts[at] = val
        c.run()
        torch.cuda.synchronize()
        assert mla.get_status() == 6
        out = torch.isfinite(c.v)
        assert out.all()


def test_more_rows_than_announced():
    c = Case("bf16", 4, [300, 300], [100, 5000])
    c.max_rows = 64 * 8
    c.run()
    torch.cuda.synchronize()
    assert mla.get_status() == 6
    assert torch.isnan(c.v[300:]).all() and torch.isfinite(c.v[:300]).all()


def test_offsets_beyond_32_bits():
    """A cache of more than 2^31 elements, the sequence in its last pages."""
    pages = 60000
    assert pages * 64 * 576 > 2 ** 31
    for lens in ([300], [2, 1]):
        c = Case("bf16", 2, lens, [200] * len(lens), base_page=pages - 40, n_pages=pages)
        c.run().check()
        del c
    torch.cuda.empty_cache()


def test_same_bits_every_time_on_any_workspace():
    for lens in ([600, 300], [3, 5]):
        c = Case("bf16", 8, lens, [700, 90])
        c.run()
        v = c.v.clone()
        for fill in (0, 0x7f):
            c.v.fill_(7)
            c.run(c.workspace(fill))
            assert torch.equal(c.v, v)
        c.v.fill_(7)
        c.run(lse=False)
        assert torch.equal(c.v, v)


@pytest.mark.parametrize("H,lens,past", [(128, [4] * 32, 64), (128, [6, 1] * 10, 130), (64, [8] * 16, 1024)])
def test_many_short_sequences_again_and_again(H, lens, past):
    """Runs of a CTA pair that change sequences every few pages."""
    c = Case("bf16", H, lens, [past] * len(lens))
    ws = c.workspace()
    c.run(ws)
    torch.cuda.synchronize()
    v = c.v.clone()
    for _ in range(10):
        for _ in range(30):
            c.run(ws)
        torch.cuda.synchronize()
        assert mla.get_status() == 0
        assert torch.equal(c.v, v)
    c.check(heads=[0, H - 1])


def test_streams_and_replayed_graphs():
    cs = [Case("bf16", 8, [600], [500], seed=1), Case("bf16", 8, [600], [500], seed=2)]
    streams = [torch.cuda.Stream() for _ in cs]
    wss = [c.workspace() for c in cs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for c, s, ws in zip(cs, streams, wss):
            c.run(ws, stream=s)
    for c in cs:
        c.check()
    # two graphs over one workspace, replayed in order; inputs changed in between
    graphs = []
    for c in cs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=streams[0]):
            c.run(wss[0])
        graphs.append(g)
    gen = torch.Generator(device="cuda").manual_seed(3)
    for c in cs:
        c.q.normal_(generator=gen)
        c.q_pos.sub_(17)
    for _ in range(2):
        for g in graphs:
            g.replay()
    for c in cs:
        c.check()


def test_workspace_is_asked_for():
    for kind, lens in (("bf16", [300]), ("bf16", [2]), ("f32", [3])):
        c = Case(kind, 4, lens, [100])
        need = c.workspace().numel()
        with pytest.raises(mla.MLAError) as e:
            c.run(torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
        assert e.value.code == 3
        with pytest.raises(mla.MLAError) as e:
            c.run(torch.empty(need + 16, dtype=torch.uint8, device="cuda")[16:])
        assert e.value.code == 1
        assert (c.v == 7).all()


@pytest.mark.parametrize("kind,lens,past,sections", [
    ("bf16", [300, 0, 420], [64, 9, 700], [8, 12, 12]), ("bf16", [1, 1, 2], [300, 64, 0], [32]),
    ("f32", [20, 3, 1], [70, 0, 200], [4, 4]),
])
def test_a_layer_over_two_chunks(kind, lens, past, sections):
    """runner.run_chunk twice, the second chunk attending the first one's rows: rotation, append
    with RMSNorm, attention and projection onto the residual, against the same steps in 64 bits
    (each step's reference starts from the stored result of the step before)."""
    H, axes = 4, len(sections)
    c = Case(kind, H, lens, past, tail=3)
    dt, d = c.q.dtype, c.d
    d_model = 200
    g = torch.Generator(device="cuda").manual_seed(11)
    rn = lambda *s: torch.randn(*s, device="cuda", generator=g)
    w_o = (rn(d_model, H * d["d_v"]) / 16).to(dt)
    norm = 1 + 0.1 * rn(d["d_c"])
    pos = torch.randint(0, 5000, (axes, c.n), device="cuda", generator=g, dtype=torch.int32)
    p = runner.chunk_problem(c.dims, c.w_uk, c.w_uv, w_o, c.cache, c.bt, c.segs, c.deltas, c.max_rows, c.ts,
                             _i32(past), c.q_pos, pos, sections, norm_weight=norm)
    half = 2.0 ** -8 if kind == "bf16" else 2.0 ** -24
    for step in range(2):
        q, kv, res = rn(c.n, H, d["d_n"] + d["d_r"]).to(dt), (2 * rn(c.n, d["d_c"] + d["d_r"])).to(dt), rn(c.n, d_model).to(dt)
        raw = q.clone()
        out = runner.run_chunk(p, q, kv, residual=res)
        torch.cuda.synchronize()
        assert mla.get_status() == 0
        rot = R.rope_axes(raw[..., d["d_n"]:], pos, sections, BASE)
        assert (q[..., d["d_n"]:].double() - rot).norm() <= half * rot.norm() + 1e-6
        assert torch.equal(q[..., :d["d_n"]], raw[..., :d["d_n"]])
        want = R.new_rows(kv, d["d_c"], pos, sections, BASE, norm, 1e-6)
        slot = [s for s in R.slots(c.ts, past, c.bt, c.n)]
        live = [t for t, s in enumerate(slot) if s >= 0]
        got = c.cache.view(-1, c.cache.shape[-1])[[slot[t] for t in live]].double()
        assert (got - want[live]).norm() <= (half + 2.0 ** -20) * want[live].norm()
        c.q, c.v = q, p.v
        v, _, _ = c.reference()
        bar = 1e-2 if kind == "bf16" else 1e-5
        assert (p.v[live].double() - v[live]).norm() <= bar * v[live].norm()
        ref = R.linear(p.v.view(c.n, -1), w_o, residual=res)
        assert (out.double() - ref).norm() <= (half + 2.0 ** -20) * ref.norm()
        assert torch.equal(out[c.total:], res[c.total:])       # padded tokens keep the residual
        # the next chunk: the same tokens again, one chunk further (segments grow)
        if step == 0:
            grown = [p0 + 2 * n for p0, n in zip(past, lens)]
            need = [-(-r // 64) for r in grown]
            bt = np.full((len(lens), max(need)), 0, np.int32)
            first = c.cache.shape[0]
            extra = sum(need)
            cache = torch.full((first + extra, 64, c.cache.shape[-1]), math.nan, device="cuda", dtype=dt)
            cache[:first] = c.cache
            old = c.bt.cpu().numpy()
            nxt = first
            for b, k in enumerate(need):
                have = -(-(past[b] + lens[b]) // 64)
                bt[b, :have] = old[b, :have]
                for i in range(have, k):
                    bt[b, i], nxt = nxt, nxt + 1
            past = [p0 + n for p0, n in zip(past, lens)]
            c.cache, c.bt, c.max_rows = cache, _i32(bt), sum(need) * 64
            c.segs = _i32([[[0, r, 0, 0], [0, 0, 0, 0]] for r in grown])
            for b in range(len(lens)):
                c.q_pos[int(c.ts[b]):int(c.ts[b + 1])] += lens[b]
            pos += 5
            p = runner.chunk_problem(c.dims, c.w_uk, c.w_uv, w_o, c.cache, c.bt, c.segs, c.deltas, c.max_rows,
                                     c.ts, _i32(past), c.q_pos, pos, sections, norm_weight=norm)


@pytest.mark.parametrize("side", [False, True])
def test_a_padded_batch_after_a_full_one(side):
    """The same problem with fewer live tokens: those left out project zeros, not the values that the
    batch before left in their rows."""
    c = Case("f32", 2, [20, 12], [70, 3])
    g = torch.Generator(device="cuda").manual_seed(5)
    rn = lambda *s: torch.randn(*s, device="cuda", generator=g)
    p = runner.chunk_problem(c.dims, c.w_uk, c.w_uv, rn(48, 2 * c.d["d_v"]), c.cache, c.bt, c.segs, c.deltas,
                             c.max_rows, c.ts, _i32([70, 3]), c.q_pos, c.q_pos[None].clone(), [8])
    stream = torch.cuda.Stream() if side else None
    for live in (32, 24):
        c.ts[2] = live
        q, kv, res = rn(c.n, 2, 32), rn(c.n, 48), rn(c.n, 48)
        torch.cuda.synchronize()
        out = runner.run_chunk(p, q, kv, residual=res, stream=stream)
        torch.cuda.synchronize()
        assert mla.get_status() == 0
        assert torch.equal(out[live:], res[live:])
        assert not torch.equal(out[live - 1], res[live - 1])


@pytest.mark.parametrize("d_n,d_v", [(8, 1), (128, 7), (16, 64), (128, 72), (24, 130), (128, 136), (8, 264)])
@pytest.mark.parametrize("lens,past", [([1], [5000]), ([17, 0, 1, 16], [0, 9, 64, 700])])
def test_few_tokens_of_any_value_width(d_n, d_v, lens, past):
    """Value widths that end inside a group of eight, of 64 and of 128 channels; one long sequence
    split over every pair of SMs."""
    Case("bf16", 3, lens, past, tail=2, d=dict(d_c=512, d_r=64, d_n=d_n, d_v=d_v)).run().check()


@pytest.mark.parametrize("lens,past,doc", [([5] * 60, [300] * 60, 0), ([7, 0, 9] * 18, [90, 64, 500] * 18, 128),
                                           ([37] * 8, [1000] * 8, 0)])
def test_more_few_tokens_than_one_pass_takes(lens, past, doc):
    """The absorbed route in passes of 256 tokens of 128 heads, cut inside sequences."""
    c = Case("bf16", 128, lens, past, doc, tail=2)
    assert c.total > 256
    assert c.workspace().numel() < c.max_rows * 128 * 512 + 2 ** 28
    c.run().check(heads=[0, 63, 127])


def test_thousands_of_sequences():
    """Shares are kept for the sequences of one pass, not for all; 700 sequences of a token each."""
    dims = mla.Dims(128, 512, 64, 128, 128, 256, 64, mla.MLA_BF16, 0.07, BASE)
    assert 0 < mla.chunk_workspace_size(dims, 4096, 4096, 1, 64, 1, 4096 * 64) < 2 ** 28
    Case("bf16", 128, [1, 0, 1, 1] * 175, [3, 64, 70, 0] * 175).run().check(heads=[0, 127])


def _off(c, v, rows=slice(None), heads=slice(None), channels=slice(None)):
    """Relative L2 error of a part of the result."""
    want = v[rows][:, heads][:, :, channels]
    return float((c.v[rows][:, heads][:, :, channels].double() - want).norm() / want.norm())


def test_values_far_below_the_largest_keep_their_precision():
    """A sequence, a head, a channel and the rows that a token sees, each 2^-20 of the others: every
    one is held to the bar of roundings to bf16 (4.5e-3, the module's docstring) by its own size."""
    c = Case("bf16", 4, [300, 280, 300], [100, 300, 256])
    small = 2.0 ** -20
    rows = [400, 580, 556]
    at = lambda b, t: (_i32(c.bt[b].cpu().numpy()).long()[t // 64], t % 64)
    t = torch.arange(rows[1], device="cuda")
    c.cache[(*at(1, t), slice(0, 512))] *= small               # a sequence
    t = torch.arange(128, device="cuda")
    c.cache[(*at(2, t), slice(0, 512))] *= small               # the first rows of another
    c.w_uv[1] *= small                                         # a head
    c.w_uv[2, 77] *= small                                     # a channel
    c.q_pos[580:600] = 127                                     # tokens that see the small rows alone
    c.run().check()
    v, _, _ = c.reference()
    parts = {"others": dict(rows=slice(0, 300), heads=[0, 3]), "sequence": dict(rows=slice(300, 580), heads=[0, 3]),
             "rows": dict(rows=slice(580, 600), heads=[0, 3]), "head": dict(rows=slice(0, 300), heads=[1]),
             "head and sequence": dict(rows=slice(300, 580), heads=[1]),
             "channel": dict(rows=slice(0, 300), heads=[2], channels=[77])}
    for name, part in parts.items():
        assert _off(c, v, **part) <= 4.5e-3, name
    # what the small ones lose in halves is not lost: the others keep theirs
    assert _off(c, v, **parts["others"]) <= 2.3e-3


@pytest.mark.parametrize("size", [2.0 ** 40, 2.0 ** -40, math.inf])
def test_neighbours_do_not_change_a_sequence(size):
    """Latents of another sequence, of any size: the same bits."""
    c = Case("bf16", 4, [300, 280], [100, 300])
    c.run()
    v, lse = c.v.clone(), c.lse.clone()
    t = torch.arange(580, device="cuda")
    c.cache[c.bt[1].long()[t // 64], t % 64, :512] *= size
    c.run()
    torch.cuda.synchronize()
    assert mla.get_status() == 0
    assert torch.equal(c.v[:300], v[:300]) and torch.equal(c.lse[:300], lse[:300])


@pytest.mark.parametrize("up,values", [(58, 0), (70, 0), (-70, 0), (58, 118), (70, 118), (58, -60), (70, -50),
                                       (-70, -110)])
def test_latents_and_values_near_the_ends_of_their_range(up, values):
    """Latents 2^up, keys of order one, values 2^values: the result stays finite and as near.  Squared
    norms of latents of 2^70 are infinite in 32 bits, those of 2^-70 vanish."""
    c = Case("bf16", 2, [300], [200])
    c.cache[..., :512] *= 2.0 ** up
    c.w_uk.mul_(2.0 ** -up)
    c.w_uv.mul_(2.0 ** (values - up))
    c.run()
    torch.cuda.synchronize()
    assert mla.get_status() == 0
    v, lse, _ = c.reference()
    assert torch.isfinite(c.v).all()
    assert _off(c, v) <= 4.5e-3
    assert (c.lse.double() - lse).abs().max() <= 1e-2
