"""mla_append_tokens with tok_start out of order: the owners are those of mla_chunk_attn."""
import pytest
import torch

from head_latent_attention_02_b200 import mla
from tests.test_gpu_chunk_ranges import STARTS, owned
from tests.test_gpu_tokens import _dims, _lib  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu
MORE = [
    ([0, 5, 3, 50], 50, {0: (0, 5)}),                              # prefix of starts, not the largest last
    ([0, 50, 30, 60], 60, {0: (0, 50)}),
    (list(range(0, 80, 2)) + [7, 79, 90], 90, {**{b: (2 * b, 2 * b + 2) for b in range(39)}, 41: (79, 90)}),
    ([60] + [0] * 40 + [70], 70, {}),                              # the break lies in another batch of 32
    ([0] * 40 + [4, 2, 9], 9, {39: (0, 4)}),
]


@pytest.mark.parametrize("ts,n,want", STARTS + MORE)
def test_token_ranges_out_of_order(ts, n, want):
    assert owned(ts, n) == want
    B = len(ts) - 1
    d = _dims("f32", 32, 16)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    kv = torch.randn(n, 48, device="cuda")
    bt = torch.arange(2 * B, device="cuda", dtype=torch.int32).view(B, 2)
    cache = torch.full((2 * B, 64, 48), float("nan"), device="cuda")
    row0 = [b % 50 for b in range(B)]
    mla.append_tokens(d, kv, i32(ts), i32(row0), torch.zeros(1, n, dtype=torch.int32, device="cuda"), [8], cache,
                      bt)
    assert mla.get_status() == 6
    assert mla.get_status() == 0
    ref = torch.full_like(cache, float("nan")).view(B, 128, 48)
    for b, (lo, hi) in want.items():
        ref[b, row0[b]:row0[b] + hi - lo] = kv[lo:hi]
    assert torch.equal(torch.nan_to_num(cache.view(B, 128, 48), nan=99.0), torch.nan_to_num(ref, nan=99.0))


@pytest.mark.parametrize("ts,n", [([0, 4, 4, 9], 9), ([0, 4, 4, 9], 12), ([0] * 70, 3), (list(range(70)), 69)])
def test_ordered_ranges_report_nothing(ts, n):
    B = len(ts) - 1
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    cache = torch.zeros(2 * B, 64, 48, device="cuda")
    bt = torch.arange(2 * B, device="cuda", dtype=torch.int32).view(B, 2)
    mla.append_tokens(_dims("f32", 32, 16), torch.randn(n, 48, device="cuda"), i32(ts), i32([0] * B),
                      torch.zeros(1, n, dtype=torch.int32, device="cuda"), [8], cache, bt)
    assert mla.get_status() == 0
