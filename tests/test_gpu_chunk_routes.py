"""The routes that mla_chunk_attn takes on a device for the sizes of test_gpu_chunk.py; its tests of
masks, bad values, invalid sequences, streams and graphs on the absorbed route (few tokens over a short
context take the expanded one); and the absorbed route's error against 64 bits."""
import math

import pytest
import torch

from head_latent_attention_02_b200 import mla
from tests import chunk_routes
from tests import test_gpu_chunk as T
from tests.test_chunk_routes_cpu import LOW_PARTS_BAR
from tests.test_gpu_chunk import _lib  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu
# rows of 512 + 64 under heads that are not 128 wide: always the absorbed route
NARROW = dict(d_c=512, d_r=64, d_n=64, d_v=96)


def _expanded(c):
    return chunk_routes.expanded(c.dims, c.B, c.n, len(c.deltas), c.bt.shape[1], c.segs.shape[1], c.max_rows)


@pytest.mark.parametrize("H,absorbed", [(1, [[1100], [400, 600], [257]]), (8, [[257]]), (16, [])])
def test_routes_of_chunks(H, absorbed):
    for lens, past, doc, tail in T.LARGE:
        assert _expanded(T.Case("bf16", H, lens, past, doc, tail)) == (lens not in absorbed), lens


def test_routes_of_long_contexts_passes_and_groups():
    assert _expanded(T.Case("bf16", 64, [257], [4000]))
    assert _expanded(T.Case("bf16", 128, [290, 600], [500, 130]))
    # passes of 256 tokens of 128 heads
    for lens, past, doc in [([5] * 60, [300] * 60, 0), ([7, 0, 9] * 18, [90, 64, 500] * 18, 128),
                            ([37] * 8, [1000] * 8, 0)]:
        c = T.Case("bf16", 128, lens, past, doc, tail=2)
        assert c.total > 256 and not _expanded(c)
    # groups of heads: less than all keys and values, more than the absorbed route ever asks for
    dims = T.Case("bf16", 128, [1], [1]).dims
    rows = 17536
    size = mla.chunk_workspace_size(dims, 1, 512, 1, rows // 64, 2, rows)
    assert rows * 128 * 512 / 2 <= size < rows * 128 * 512


@pytest.fixture
def narrow(monkeypatch):
    """Every bf16 case of test_gpu_chunk.py on the absorbed route."""
    class Narrow(T.Case):
        def __init__(self, kind, *args, d=None, **kw):
            super().__init__(kind, *args, d=d or (NARROW if kind == "bf16" else None), **kw)

        def run(self, *args, **kw):
            assert self.kind != "bf16" or not _expanded(self)
            return super().run(*args, **kw)

    monkeypatch.setattr(T, "Case", Narrow)


@pytest.mark.parametrize("lens,past,doc,tail", T.SMALL + [([300, 0, 33, 29], [64, 700, 129, 5], 64, 7)])
@pytest.mark.parametrize("H", [1, 5, 128])
def test_absorbed_tokens(narrow, lens, past, doc, tail, H):
    T.Case("bf16", H, lens, past, doc, tail).run().check()


@pytest.mark.parametrize("lens", [[3, 2], [40, 30]])
def test_absorbed_tokens_that_see_nothing(narrow, lens):
    T.test_tokens_that_see_nothing("bf16", lens)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("lens", [[3, 2], [40], [300, 20]])
def test_absorbed_masked_rows(narrow, lens, bad):
    T.test_what_a_masked_row_holds_does_not_matter("bf16", lens, bad)


@pytest.mark.parametrize("lens", [[3, 2, 4], [100, 90, 30]])
def test_absorbed_invalid_sequences(narrow, lens):
    T.test_invalid_sequences_get_nan_and_leave_the_others("bf16", lens)


def test_absorbed_rows_beyond_the_announced(narrow):
    T.test_more_rows_than_announced()


def test_absorbed_relocation_and_far_pages(narrow):
    T.test_negative_and_far_relocation()
    T.test_offsets_beyond_32_bits()


def test_absorbed_bits_streams_and_graphs(narrow):
    T.test_same_bits_every_time_on_any_workspace()
    T.test_streams_and_replayed_graphs()
    T.test_many_short_sequences_again_and_again(64, [8] * 16, 1024)


@pytest.mark.parametrize("size", [2.0 ** 40, 2.0 ** -40, math.inf])
def test_absorbed_neighbours(narrow, size):
    T.test_neighbours_do_not_change_a_sequence(size)


@pytest.mark.parametrize("lens,past", [([1] * 8, [690] * 8), ([3, 9, 30], [2000, 300, 700])])
def test_the_absorbed_route_keeps_both_parts(lens, past):
    for d in (None, NARROW):
        c = T.Case("bf16", 16, lens, past, d=d)
        if d is None and _expanded(c):
            continue
        c.run()
        torch.cuda.synchronize()
        assert mla.get_status() == 0
        v, _, _ = c.reference()
        assert (c.v.double() - v).norm() <= LOW_PARTS_BAR * v.norm()
