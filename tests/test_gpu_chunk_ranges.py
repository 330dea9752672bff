"""Who owns a token when tok_start is out of order, alike in every route of mla_chunk_attn: a sequence
whose range is not [lo, hi) with 0 <= lo <= hi <= n_tok, or starts before an earlier start, is left out."""
import pytest
import torch

from head_latent_attention_02_b200 import mla, runner
from tests import chunk_reference as R
from tests.test_gpu_chunk import Case, _i32, _lib  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu
KINDS = {"generic": ("f32", None), "generic, bf16": ("bf16", dict(d_c=64, d_r=16, d_n=24, d_v=40)),
         "expanded": ("bf16", None), "absorbed": ("bf16", dict(d_c=512, d_r=64, d_n=64, d_v=96))}


def owned(ts, n):
    """The ranges that hold, by the rule above: {sequence: (first token, last + 1)}."""
    return {b: (ts[b], ts[b + 1]) for b in range(len(ts) - 1)
            if 0 <= ts[b] < ts[b + 1] <= n and ts[b] >= max(ts[:b + 1])}


STARTS = [
    ([0, 10, 5, 20], 20, {0: (0, 10)}),                   # the last range begins inside the first one
    ([0, 50, 10, 30], 60, {0: (0, 50)}),
    ([30, 10, 20, 40], 40, {}),
    ([0, 4, 4, 2, 9], 12, {0: (0, 4)}),
    ([-3, 5, 9], 12, {1: (5, 9)}),
    ([0, 5, 99], 12, {0: (0, 5)}),
    ([0, 3, 2, 7, 12], 12, {0: (0, 3), 3: (7, 12)}),      # behind every start again
]


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("ts,n,want", STARTS)
def test_token_ranges_out_of_order(kind, ts, n, want):
    assert owned(ts, n) == want
    k, d = KINDS[kind]
    B = len(ts) - 1
    c = Case(k, 3, [n] + [0] * (B - 1), [70 + 30 * b for b in range(B)], d=d)
    c.q_pos.fill_(1000)                                    # every row is seen
    c.ts = _i32(ts)
    c.run()
    torch.cuda.synchronize()
    assert mla.get_status() == 6
    assert mla.get_status() == 0
    free = torch.ones(n, dtype=torch.bool, device="cuda")
    for b, (lo, hi) in want.items():
        v, lse, _ = R.chunk_attn(c.q, [lo, hi], c.q_pos, c.w_uk, c.w_uv, c.cache, c.bt[b:b + 1],
                                 c.segs[b:b + 1], c.deltas, c.scale, 10000.0)
        bar = 1e-5 if k == "f32" else 1e-2
        assert (c.v[lo:hi].double() - v[lo:hi]).norm() <= bar * v[lo:hi].norm()
        assert (c.lse[lo:hi].double() - lse[lo:hi]).abs().max() <= bar
        free[lo:hi] = False
    assert (c.v[free] == 7).all() and (c.lse[free] == 7).all()


@pytest.mark.parametrize("kind", list(KINDS))
def test_an_invalid_table_of_a_sequence_without_tokens(kind):
    """It records BAD_INDEX, and changes nothing else."""
    k, d = KINDS[kind]
    c = Case(k, 3, [9, 0, 5], [70, 200, 64], d=d).run()
    c.check()
    v = c.v.clone()
    c.segs[1, 0, 1] = 1 << 20
    c.run()
    torch.cuda.synchronize()
    assert mla.get_status() == 6
    assert torch.equal(c.v, v)


@pytest.mark.parametrize("kind", list(KINDS))
def test_more_rows_than_announced_in_every_route(kind):
    """The sequences up to max_rows are attended, those past it get NaN."""
    k, d = KINDS[kind]
    c = Case(k, 3, [9, 4, 5, 6], [70, 200, 5000, 40], d=d)
    full = c.run()
    torch.cuda.synchronize()
    assert mla.get_status() == 0
    v = full.v.clone()
    c.max_rows = 64 * 6                     # two pages and four; 79 and one more do not fit
    c.v.fill_(7)
    c.run()
    torch.cuda.synchronize()
    assert mla.get_status() == 6
    assert mla.get_status() == 0
    bar = 1e-5 if k == "f32" else 1e-2      # another bound may take another route
    assert (c.v[:13].double() - v[:13].double()).norm() <= bar * v[:13].double().norm()
    assert torch.isnan(c.v[13:]).all() and torch.isnan(c.lse[13:]).all()


@pytest.mark.parametrize("kind", list(KINDS))
def test_tables_of_more_pages_than_32_bits_count(kind):
    """70 sequences, all but the first of 2^25 - 1 pages each, a table of 2^31 entries: past max_rows."""
    k, d = KINDS[kind]
    B, wide = 70, 2 ** 25 - 1
    c = Case(k, 2, [2] * B, [100] + [3] * (B - 1), d=d).run()
    c.check()
    v = c.v.clone()
    bt = torch.zeros(B, wide, dtype=torch.int32, device="cuda")
    bt[:, :c.bt.shape[1]] = c.bt
    c.bt = bt
    c.segs[1:, 0, 1] = wide * 64
    c.run()
    torch.cuda.synchronize()
    assert mla.get_status() == 6
    bar = 1e-5 if k == "f32" else 1e-2
    assert (c.v[:2].double() - v[:2].double()).norm() <= bar * v[:2].double().norm()
    assert torch.isnan(c.v[2:]).all() and torch.isnan(c.lse[2:]).all()
    c.bt = bt = None
    torch.cuda.empty_cache()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("B,n", [(2, 0), (0, 0), (0, 3)])
def test_a_layer_without_tokens_or_sequences(kind, B, n):
    """run_chunk on an empty step: nothing appended, every row (padding) keeps the residual."""
    c = Case(kind, 2, [1, 1], [70, 3])
    dt, d = c.q.dtype, c.d
    new = lambda *s: torch.randn(*s, device="cuda").to(dt)
    empty = torch.zeros(n, dtype=torch.int32, device="cuda")
    p = runner.chunk_problem(c.dims, c.w_uk, c.w_uv, new(48, 2 * d["d_v"]), c.cache, c.bt[:B], c.segs[:B],
                             c.deltas, c.max_rows, torch.zeros(B + 1, dtype=torch.int32, device="cuda"),
                             _i32([70, 3])[:B], empty, empty[None].clone(), [d["d_r"] // 2])
    before = c.cache.clone()
    q, kv, res = new(n, 2, d["d_n"] + d["d_r"]), new(n, d["d_c"] + d["d_r"]), new(n, 48)
    out = runner.run_chunk(p, q, kv, residual=res)
    torch.cuda.synchronize()
    assert mla.get_status() == 0
    assert out.shape == (n, 48) and torch.equal(out, res)
    assert torch.equal(c.cache.view(torch.uint8), before.view(torch.uint8))


def test_a_refused_layer_call_changes_nothing():
    """A query, latent rows or residual that a later step would refuse: q is not rotated, nothing appended."""
    c = Case("f32", 2, [5, 4], [70, 3])
    p = runner.chunk_problem(c.dims, c.w_uk, c.w_uv, torch.randn(48, 32, device="cuda"), c.cache, c.bt, c.segs,
                             c.deltas, c.max_rows, c.ts, _i32([70, 3]), c.q_pos, c.q_pos[None].clone(), [8])
    new = lambda *s: torch.randn(*s, device="cuda")
    wide = new(9, 2, 40)
    good = (new(9, 2, 32), new(9, 48), new(9, 48))
    cache = c.cache.clone()
    for bad in ((wide[..., :32], good[1], good[2]), (good[0], new(8, 48), good[2]), (good[0], good[1], new(9, 47)),
                (good[0], good[1].double(), good[2]), (good[0], good[1], good[2].bfloat16()),
                (good[0], good[1], torch.randn(9, 48)), (good[0], good[1], new(1, 48).expand(9, 48)),
                (good[0], new(1, 48).expand(9, 48), good[2])):
        q = bad[0].clone()
        with pytest.raises(ValueError):
            runner.run_chunk(p, bad[0], bad[1], residual=bad[2])
        torch.cuda.synchronize()
        assert torch.equal(bad[0], q)
        assert torch.equal(c.cache.view(torch.uint8), cache.view(torch.uint8))
    runner.run_chunk(p, *good[:2], residual=good[2])
    assert mla.get_status() == 0
