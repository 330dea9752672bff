"""mla_rope_axes and mla_append_tokens against their 64-bit forms.

Bounds (half a step of the storage type is eps / 2 of the value: bf16 2^-8,
fp32 2^-24):
  rotation, bf16   2^-8 |y| for the rounding; sine and cosine are float, off by
                   at most 2^-22 each, and the two products and their sum round
                   to 2^-24: below 2^-20 (|x0| + |x1|) together
  rotation, fp32   2^-24 |y| for the one rounding; the double arithmetic before
                   it is off by 2^-50 (|x0| + |x1|) at positions below 2^20
                   (the angle itself is a rounded product)
  normalised       the float sum of 512 squares is 16 additions a lane and 5
  latent           between lanes, then a division, a square root and two products:
                   below 32 roundings of 2^-24, on top of the storage rounding
  codes            exact: what decides them is computed in double on both sides
"""
import numpy as np
import pytest
import torch

from head_latent_attention_02_b200 import mla
from tests import chunk_reference as R

pytestmark = pytest.mark.gpu
BASE = 10000.0
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
DT = {"bf16": (torch.bfloat16, mla.MLA_BF16), "f32": (torch.float32, mla.MLA_F32)}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from head_latent_attention_02_b200 import build
    build.build()
    mla.lib()
    assert mla.get_status() == 0


def _dims(kind, d_c=512, d_r=64, H=8):
    return mla.Dims(H, d_c, d_r, 128, 128, 256, 64, DT[kind][1], 0.1, BASE)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _pair_size(x):
    """|x0| + |x1| of the pair each element belongs to."""
    a = x.double().abs().unflatten(-1, (-1, 2)).sum(-1, keepdim=True)
    return a.expand(*a.shape[:-1], 2).flatten(-2)


def _check_turned(got, x, want, dt):
    slack = 2.0 ** -20 if dt == torch.bfloat16 else 2.0 ** -50
    tol = HALF[dt] * want.abs() + slack * _pair_size(x)
    assert (got.double() - want).abs().le(tol).all()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("n,H,d_r,sections", [
    (1, 1, 64, [32]), (1, 128, 64, [8, 12, 12]), (3, 5, 64, [0, 32]), (17, 16, 6, [1, 1, 1]),
    (16, 128, 128, [64]), (600, 64, 64, [8, 12, 12]), (700, 3, 64, [16, 16]), (513, 1, 16, [4, 2, 1, 1]),
    (1030, 7, 40, [20]),
])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope(kind, n, H, d_r, sections, inverse):
    dt = DT[kind][0]
    g = _gen(n + H + d_r)
    x = torch.randn(n, H, d_r, device="cuda", generator=g).to(dt)
    pos = torch.randint(-500, 100000, (len(sections), n), device="cuda", generator=g, dtype=torch.int32)
    out = torch.full_like(x, float("nan"))
    mla.rope_axes(_dims(kind, d_r=d_r), x, pos, sections, out, inverse=inverse)
    assert mla.get_status() == 0
    _check_turned(out, x, R.rope_axes(x, pos, sections, BASE, inverse), dt)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_rope_of_slices_in_place_and_unaligned(kind):
    dt = DT[kind][0]
    d = _dims(kind)
    pos = torch.arange(40, device="cuda", dtype=torch.int32)[None]
    for n, off, width in [(40, 128, 192), (40, 1, 65), (40, 3, 200)]:
        q = torch.randn(n, 6, width, device="cuda", generator=_gen(off)).to(dt)
        keep = q.clone()
        x = q[..., off:off + 64]
        want = R.rope_axes(keep[..., off:off + 64], pos, [32], BASE)
        mla.rope_axes(d, x, pos, [32], x)
        _check_turned(x, keep[..., off:off + 64], want, dt)
        keep[..., off:off + 64] = q[..., off:off + 64]
        assert torch.equal(q, keep)          # nothing beside the slice changed
    # heads outside tokens, and one vector broadcast over the heads
    x = torch.randn(5, 40, 64, device="cuda", generator=_gen(9)).to(dt).transpose(0, 1)
    out = torch.empty_like(x)
    mla.rope_axes(d, x, pos, [32], out)
    _check_turned(out, x, R.rope_axes(x, pos, [32], BASE), dt)
    one = torch.randn(40, 1, 64, device="cuda", generator=_gen(10)).to(dt).expand(40, 5, 64)
    out = torch.empty(40, 5, 64, device="cuda", dtype=dt)
    mla.rope_axes(d, one, pos, [32], out)
    _check_turned(out, one, R.rope_axes(one, pos, [32], BASE), dt)


def test_rope_far_positions():
    """Positions up to the end of int32: the angle's product rounds to 2^-53 of
    2^31 radians, 2^-22, in both sides' arithmetic."""
    x = torch.randn(4, 2, 64, device="cuda", generator=_gen(1)).bfloat16()
    pos = torch.tensor([[2 ** 31 - 1, -2 ** 31, 2 ** 30 + 7, 0]], device="cuda", dtype=torch.int32)
    out = torch.empty_like(x)
    mla.rope_axes(_dims("bf16"), x, pos, [32], out)
    want = R.rope_axes(x, pos, [32], BASE)
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -20 + 2.0 ** -21) * _pair_size(x)
    assert (out.double() - want).abs().le(tol).all()


def test_rope_inverse_is_the_gradient():
    """Against the formula (above) and against differences of the kernel itself, in fp32."""
    d = _dims("f32", d_r=16)
    g = _gen(4)
    x, grad = (torch.randn(3, 2, 16, device="cuda", generator=g) for _ in range(2))
    pos = torch.tensor([[1, 70, 9], [4, 5, 60]], device="cuda", dtype=torch.int32)
    back, up, dn = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    mla.rope_axes(d, grad, pos, [3, 5], back, inverse=True)
    step = 2.0 ** -3            # the operator is linear: the step only has to be exact
    for idx in [(0, 0, 0), (1, 1, 7), (2, 0, 15)]:
        e = torch.zeros_like(x)
        e[idx] = step
        mla.rope_axes(d, x + e, pos, [3, 5], up)
        mla.rope_axes(d, x - e, pos, [3, 5], dn)
        diff = ((up - dn).double() * grad.double()).sum() / (2 * step)
        # four values of |y| < 8 round to 2^-24 each, divided by the step
        assert abs(float(diff - back[idx])) < 4 * 8 * 4 * 2.0 ** -24 / step


def _ragged(lens, tail, past, g):
    starts = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    need = [-(-(p + n) // 64) for p, n in zip(past, lens)]
    n_pages = sum(need) + 2
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32).cpu()
    bt = torch.full((len(lens), max(need + [1])), n_pages + 5, dtype=torch.int32)   # unused: out of range
    at = 0
    for b, k in enumerate(need):
        bt[b, :k] = perm[at:at + k]
        at += k
    i32 = lambda a: torch.as_tensor(np.asarray(a, np.int32), device="cuda")
    return i32(starts), i32(past), bt.cuda(), n_pages, int(starts[-1]) + tail


CASES = [([1], 0, [0]), ([1] * 40, 0, list(range(0, 400, 10))), ([5, 0, 130, 1], 9, [60, 3, 63, 64]),
         ([0, 0], 4, [5, 6]), ([700], 0, [31])]


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("lens,tail,past", CASES)
@pytest.mark.parametrize("norm,axes,d_c,d_r", [
    (True, 1, 512, 64), (False, 3, 512, 64), (True, 2, 40, 6), (True, 1, 1100, 128), (False, 1, 13, 2)])
def test_append(kind, lens, tail, past, norm, axes, d_c, d_r):
    dt = DT[kind][0]
    g = _gen(len(lens) + d_c)
    ts, row0, bt, n_pages, n = _ragged(lens, tail, past, g)
    wide = d_c + d_r + (8 if d_c == 512 else 3)          # a stride beyond the row, unaligned for odd widths
    kv = (1.5 * torch.randn(n, wide, device="cuda", generator=g)).to(dt)[:, :d_c + d_r]
    half = d_r // 2
    sections = {1: [half], 2: [half // 2, half - half // 2], 3: [8, 12, 12]}[axes]
    pos = torch.randint(0, 40000, (axes, n), device="cuda", generator=g, dtype=torch.int32)
    w = (1 + 0.1 * torch.randn(d_c, device="cuda", generator=g)) if norm else None
    cache = torch.full((n_pages, 64, d_c + d_r), float("nan"), dtype=dt, device="cuda")
    mla.append_tokens(_dims(kind, d_c, d_r), kv, ts, row0, pos, sections, cache, bt, norm_weight=w, norm_eps=1e-6)
    assert mla.get_status() == 0
    want = R.new_rows(kv, d_c, pos, sections, BASE, w, 1e-6)
    slot = R.slots(ts, row0, bt, n)
    flat = cache.view(-1, d_c + d_r)
    written = [s for s in slot if s >= 0]
    untouched = torch.ones(flat.shape[0], dtype=torch.bool, device="cuda")
    untouched[written] = False
    assert torch.isnan(flat[untouched]).all()
    live = [t for t, s in enumerate(slot) if s >= 0]
    if not live:
        return
    got, ref = flat[written], want[live]
    lat = HALF[dt] * ref[:, :d_c].abs() * (1 + 2.0 ** -8) + (2.0 ** -19 * ref[:, :d_c].abs() if norm else 0)
    if norm:
        assert (got[:, :d_c].double() - ref[:, :d_c]).abs().le(lat).all()
    else:
        assert torch.equal(got[:, :d_c], kv[live][:, :d_c])        # copied bit for bit
    _check_turned(got[:, d_c:], kv[live][:, d_c:], ref[:, d_c:], dt)


@pytest.mark.parametrize("kind,d_c,d_r", [("bf16", 512, 64), ("f32", 32, 16), ("bf16", 1056, 64)])
@pytest.mark.parametrize("bits_c", [4, 2])
@pytest.mark.parametrize("lens,tail,past", CASES[1:3])
def test_append_codes_are_exact(kind, d_c, d_r, bits_c, lens, tail, past):
    dt = DT[kind][0]
    g = _gen(bits_c + d_c)
    ts, row0, bt, n_pages, n = _ragged(lens, tail, past, g)
    d = _dims(kind, d_c, d_r)
    kv = (1.5 * torch.randn(n, d_c + d_r, device="cuda", generator=g)).to(dt)
    kv[0, :4] = torch.tensor([float("inf"), -float("inf"), 3e38, 0.0])       # saturate
    w = None
    pos = torch.randint(0, 40000, (1, n), device="cuda", generator=g, dtype=torch.int32)
    sc = 0.3 + 0.2 * torch.rand(d_c, device="cuda", generator=g)
    sr = 0.4 + 0.2 * torch.rand(d_r, device="cuda", generator=g)
    width = (d_c * bits_c + d_r * 4) // 8
    for w in (None, 1 + 0.1 * torch.randn(d_c, device="cuda", generator=g)):
        x = kv.clone()
        if w is not None:
            x[0, :4] = 1.0           # an infinite row has no norm
        pool = torch.randint(0, 256, (n_pages, 64, width), device="cuda", generator=g, dtype=torch.uint8)
        before = pool.clone().view(-1, width)
        mla.append_tokens(d, x, ts, row0, pos, [d_r // 2], pool, bt, norm_weight=w, norm_eps=1e-6,
                          bits=(bits_c, 4), scale_c=sc, scale_r=sr)
        assert mla.get_status() == 0
        rows = R.new_rows(x, d_c, pos, [d_r // 2], BASE, w, 1e-6).float().to(dt)
        packed = torch.empty(n, width, dtype=torch.uint8, device="cuda")
        mla.pack_rows(d, bits_c, 4, rows, sc, sr, packed)
        slot = R.slots(ts, row0, bt, n)
        for t, s in enumerate(slot):
            if s >= 0:
                before[s] = packed[t]
        assert torch.equal(pool.view(-1, width), before)


def test_append_reports_and_skips_bad_entries():
    d = _dims("f32", 32, 16)
    kv = torch.randn(6, 48, device="cuda")
    pos = torch.zeros(1, 6, device="cuda", dtype=torch.int32)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    cases = [
        # sequence 1's page id is out of range, sequence 2's row lies past the table
        (i32([0, 2, 4, 6]), i32([3, 0, 128]), i32([[1, 0], [-3, 0], [2, 2]]), {(1, 3): 0, (1, 4): 1}),
        (i32([0, 2, 4, 6]), i32([-1, 2 ** 31 - 1, 5]), i32([[1, 0], [0, 0], [2, 2]]),
         {(1, 0): 1, (2, 5): 4, (2, 6): 5}),                         # negative row; row overflow
        (i32([0, 4, 2, 6]), i32([0, 10, 20]), i32([[0, 0], [1, 1], [2, 2]]), None),   # starts out of order
        (i32([3, 4, 5, 5]), i32([0, 0, 0]), i32([[0, 0], [1, 1], [2, 2]]), {(0, 0): 3, (1, 0): 4}),
    ]
    for k, (ts, row0, bt, want) in enumerate(cases):
        cache = torch.full((3, 64, 48), float("nan"), device="cuda")
        mla.append_tokens(d, kv, ts, row0, pos, [8], cache, bt)
        assert mla.get_status() == 6
        assert mla.get_status() == 0
        if want is not None:
            got = {(int(p), int(s)) for p, s in (~torch.isnan(cache).any(-1)).nonzero()}
            assert got == set(want), k
            for (p, s), t in want.items():
                assert torch.equal(cache[p, s], kv[t])               # position zero: the raw row


def test_append_on_another_stream_and_replayed():
    d = _dims("bf16")
    g = _gen(3)
    ts, row0, bt, n_pages, n = _ragged([3, 70], 0, [10, 20], g)
    kv = torch.randn(n, 576, device="cuda", generator=g).bfloat16()
    pos = torch.zeros(1, n, device="cuda", dtype=torch.int32)
    cache = torch.zeros(n_pages, 64, 576, device="cuda").bfloat16()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        mla.append_tokens(d, kv, ts, row0, pos, [32], cache, bt)
        mla.rope_axes(d, kv[:, None, 512:], pos, [32], kv[:, None, 512:])
    kv.normal_(generator=g)
    pos += 1000
    want = kv.clone()
    graph.replay()
    torch.cuda.synchronize()
    slot = R.slots(ts, row0, bt, n)
    got = cache.view(-1, 576)[slot]
    assert torch.equal(got[:, :512], want[:, :512])
    assert torch.equal(got[:, 512:], kv[:, 512:])    # the same rotation, in the cache and in place
    # another stream than the current one
    other = torch.empty_like(cache)
    s.wait_stream(torch.cuda.current_stream())
    mla.append_tokens(d, want, ts, row0, pos, [32], other, bt, stream=s)
    s.synchronize()
    assert torch.equal(other.view(-1, 576)[slot], got)
