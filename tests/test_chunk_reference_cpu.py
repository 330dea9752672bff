"""Pins of tests/chunk_reference.py: against the fp64 oracle, complex numbers,
finite differences and torch's library routines."""
import math

import numpy as np
import torch

from head_latent_attention_02_b200.workloads import Workload, make_inputs
from oracle import mla_oracle as O
from tests import chunk_reference as R


def test_equal_axes_are_the_one_axis_rotation():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(5, 2, 16, generator=g, dtype=torch.float64)
    pos = torch.tensor([3, 0, 77, -5, 1000])
    want = np.stack([[O.rope_rotate(x[t, h].numpy(), int(pos[t]), 10000.0) for h in range(2)]
                     for t in range(5)])
    for sections in ([8], [3, 5], [2, 0, 6], [1, 3, 4]):
        got = R.rope_axes(x, pos.repeat(len(sections), 1), sections, 10000.0)
        assert np.abs(got.numpy() - want).max() < 1e-12


def test_axes_turn_their_own_pairs_as_complex_numbers():
    g = torch.Generator().manual_seed(2)
    x = torch.randn(4, 1, 12, generator=g, dtype=torch.float64)
    pos = torch.tensor([[1, 2, 3, 4], [50, 60, 70, 80], [-7, 0, 7, 14]])
    sections = [1, 2, 3]
    got = R.rope_axes(x, pos, sections, 500.0)
    axis = [0, 1, 1, 2, 2, 2]
    for t in range(4):
        for i in range(6):
            z = complex(x[t, 0, 2 * i], x[t, 0, 2 * i + 1])
            w = z * np.exp(1j * float(pos[axis[i], t]) * 500.0 ** (-i / 6))
            assert abs(complex(got[t, 0, 2 * i], got[t, 0, 2 * i + 1]) - w) < 1e-12


def test_inverse_undoes_and_is_the_gradient():
    g = torch.Generator().manual_seed(3)
    x = torch.randn(3, 2, 8, generator=g, dtype=torch.float64)
    grad = torch.randn(3, 2, 8, generator=g, dtype=torch.float64)
    pos = torch.tensor([[1, 5, 9], [2, 4, 8]])
    turned = R.rope_axes(x, pos, [1, 3], 10000.0)
    assert (R.rope_axes(turned, pos, [1, 3], 10000.0, inverse=True) - x).abs().max() < 1e-13
    back = R.rope_axes(grad, pos, [1, 3], 10000.0, inverse=True)
    eps = 1e-6
    for idx in [(0, 0, 0), (1, 1, 5), (2, 0, 7)]:
        d = torch.zeros_like(x)
        d[idx] = eps
        up = (grad * R.rope_axes(x + d, pos, [1, 3], 10000.0)).sum()
        dn = (grad * R.rope_axes(x - d, pos, [1, 3], 10000.0)).sum()
        assert abs(float((up - dn) / (2 * eps) - back[idx])) < 1e-8


def test_new_rows_match_the_oracle_writer_and_rms_norm():
    g = torch.Generator().manual_seed(4)
    kv = torch.randn(6, 32 + 8, generator=g, dtype=torch.float64)
    pos = torch.arange(6)[None]
    plain = R.new_rows(kv, 32, pos, [4], 10000.0)
    want = O.cache_rows(kv[:, :32].numpy(), kv[:, 32:].numpy(), pos[0].numpy(), 10000.0)
    assert np.abs(plain.numpy() - want).max() < 1e-12
    w = 1 + 0.1 * torch.randn(32, generator=g, dtype=torch.float64)
    normed = R.new_rows(kv, 32, pos, [4], 10000.0, w, 1e-5)
    lib = torch.nn.functional.rms_norm(kv[:, :32], (32,), w, 1e-5)
    assert (normed[:, :32] - lib).abs().max() < 1e-12
    assert torch.equal(normed[:, 32:], plain[:, 32:])


def test_one_token_per_sequence_is_the_oracle_decode():
    wl = Workload("cr", "f32", B=3, H=4, d_c=32, d_r=16, d_n=16, d_v=16, d_model=64,
                  lengths=[70, 1, 130], scattered=True)
    inp = make_inputs(wl, seed=5, poison=True)
    o_ref, l_ref = O.decode(inp, form="direct")[:2]
    v_ref, _ = O.out_proj(o_ref, inp.w_uv, inp.w_o)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a))
    q_pos = t(inp.q_pos)
    q_rot = R.rope_axes(t(inp.q_rope), q_pos[None], [8], wl.rope_base)
    q = torch.cat([t(inp.q_nope).double(), q_rot], -1)
    v, lse, _ = R.chunk_attn(q, [0, 1, 2, 3], q_pos, t(inp.w_uk), t(inp.w_uv), t(inp.pool),
                             t(inp.block_table), t(inp.segs), [0], wl.scale, wl.rope_base)
    assert np.abs(lse.numpy() - l_ref).max() < 1e-9
    assert np.abs(v.numpy() - v_ref.reshape(v.shape)).max() < 1e-9


def test_causal_chunk_matches_sdpa_and_hides_masked_rows():
    g = torch.Generator().manual_seed(6)
    H, d_c, d_r, d_n, d_v, past, n = 2, 24, 8, 12, 10, 90, 7
    cache = torch.full((4, 64, d_c + d_r), math.nan, dtype=torch.float64)
    bt = torch.tensor([[2, 0]], dtype=torch.int32)
    rows = torch.randn(past + n, d_c + d_r, generator=g, dtype=torch.float64)
    cache[2], cache[0, :past + n - 64] = rows[:64], rows[64:]
    q = torch.randn(n, H, d_n + d_r, generator=g, dtype=torch.float64)
    w_uk = torch.randn(H, d_n, d_c, generator=g, dtype=torch.float64)
    w_uv = torch.randn(H, d_v, d_c, generator=g, dtype=torch.float64)
    segs = torch.tensor([[[0, past + n, 0, 0]]], dtype=torch.int32)
    q_pos = torch.arange(past, past + n)
    args = (q, [0, n], q_pos, w_uk, w_uv, cache, bt, segs, [0], 0.3, 10000.0)
    v, lse, _ = R.chunk_attn(*args)
    k = torch.cat([torch.einsum("tc,hnc->htn", rows[:, :d_c], w_uk),
                   rows[None, :, d_c:].expand(H, -1, -1)], -1)
    vv = torch.einsum("tc,hdc->htd", rows[:, :d_c], w_uv)
    mask = torch.arange(past + n)[None] <= q_pos[:, None]
    want = torch.nn.functional.scaled_dot_product_attention(q.transpose(0, 1), k, vv, mask, scale=0.3)
    assert (v - want.transpose(0, 1)).abs().max() < 1e-11
    # the last row is seen by the last token only
    cache[0, past + n - 1 - 64] = math.inf
    w, _, _ = R.chunk_attn(*args)
    assert torch.equal(w[:-1], v[:-1]) and torch.isnan(w[-1]).all()


def test_linear_matches_library_activations():
    g = torch.Generator().manual_seed(7)
    x, w = torch.randn(3, 5, generator=g, dtype=torch.float64), torch.randn(4, 5, generator=g, dtype=torch.float64)
    b, r = torch.randn(4, generator=g, dtype=torch.float64), torch.randn(3, 4, generator=g, dtype=torch.float64)
    y = torch.nn.functional.linear(x, w, b)
    F = torch.nn.functional
    assert (R.linear(x, w, b, "none", r) - (y + r)).abs().max() < 1e-13
    assert (R.linear(x, w, b, "silu", r) - (F.silu(y) + r)).abs().max() < 1e-13
    assert (R.linear(x, w, b, "gelu") - F.gelu(y)).abs().max() < 1e-13
