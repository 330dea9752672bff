"""The choice between the routes of mla_chunk_attn, and the error bar that the absorbed route is held to."""
import math

import pytest
import torch

from head_latent_attention_02_b200 import build as B
from head_latent_attention_02_b200 import mla
from tests import chunk_routes

LOW_PARTS_BAR = 2.5e-3


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    mla.lib()


def _dims(**kw):
    d = dict(H=128, d_c=512, d_r=64, d_n=128, d_v=128, d_model=7168, page_size=64, dtype=mla.MLA_BF16,
             scale=1 / 192 ** 0.5, rope_base=10000.0)
    d.update(kw)
    return mla.Dims(**d)


@pytest.mark.parametrize("H,seqs,rows,below,above", [
    (16, 1, 4096, 120, 300), (64, 4, 2048, 55, 110), (128, 16, 1024, 40, 85), (128, 1, 16384, 95, 190),
])
def test_few_tokens_are_absorbed_and_many_expanded(H, seqs, rows, below, above):
    """Tokens a sequence well below and well above the crossing, sequences of equal length."""
    for n, want in ((1, False), (below, False), (above, True)):
        if seqs * rows * H * 512 >= 2 ** 30:
            size = mla.chunk_workspace_size(_dims(H=H), seqs, n * seqs, 1, rows // 64, 1, seqs * rows)
            assert (size > 2 ** 29) == want          # heads in groups; the absorbed route stays far below
        else:
            assert chunk_routes.expanded(_dims(H=H), seqs, n * seqs, 1, rows // 64, 1, seqs * rows) == want


def test_other_widths_have_neither():
    for kw in (dict(dtype=mla.MLA_F32, d_c=32, d_r=16), dict(d_n=12), dict(d_c=256)):
        assert mla.chunk_workspace_size(_dims(**kw), 1, 4, 1, 4, 1, 256) == 256


def _absorbed(weights_low, latents_low, seed=0):
    """Relative L2 error of the absorbed route's roundings alone (its sums in 64 bits), for unit-normal
    data: queries absorbed and rounded, softmax weights and weighted latents in one or two bf16 parts."""
    g = torch.Generator().manual_seed(seed)
    H, n, rows = 8, 8, 700
    rnd = lambda x: x.to(torch.bfloat16).double()
    rn = lambda *s: rnd(torch.randn(*s, generator=g, dtype=torch.float64))
    w_uk, w_uv = rnd(rn(H, 128, 512) / 512 ** 0.5), rnd(rn(H, 128, 512) / 512 ** 0.5)
    c, k_r, q = rn(rows, 512), rn(rows, 64), rn(n, H, 192)
    two = lambda x, low: rnd(x) + (rnd(x - rnd(x)) if low else 0.0)

    def run(exact):
        q_abs = torch.einsum("nhk,hkc->nhc", q[..., :128], w_uk)
        s = (q_abs if exact else rnd(q_abs)) @ c.T + q[..., 128:] @ k_r.T
        s = s / 192 ** 0.5
        p = torch.exp(s - s.amax(-1, keepdim=True))
        total = p.sum(-1, keepdim=True)
        o = (p if exact else two(p, weights_low)) @ c / total
        v = torch.einsum("nhc,hdc->nhd", o if exact else two(o, latents_low), w_uv)
        return v if exact else rnd(v)

    want = run(True)
    return float((run(False) - want).norm() / want.norm())


def test_the_absorbed_route_s_bar_tells_a_lost_low_part():
    """The result's rounding and the absorbed query's are about 1.66e-3 and 1.36e-3 of the result,
    2.15e-3 together; a latent without its low part adds 1.66e-3 to that, a weight a little less (the
    largest one of a row is 1 and has none): 2.6e-3 to 2.8e-3."""
    assert _absorbed(True, True) < LOW_PARTS_BAR - 2e-4
    assert _absorbed(False, True) > LOW_PARTS_BAR
    assert _absorbed(True, False) > LOW_PARTS_BAR
