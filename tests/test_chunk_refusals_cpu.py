"""More refusals of the prompt-chunk entry points, on the CPU: none of the fake pointers is ever used."""
import numpy as np
import pytest

from head_latent_attention_02_b200 import mla
from tests.test_chunk_abi_cpu import FAKE, INVALID, L, _append, _chunk, _linear, _rope  # noqa: F401  (L: the fixture)


@pytest.mark.parametrize("name", ["ts", "row0", "pos", "bt", "norm"])
def test_append_refuses_misaligned_arrays(L, name):
    assert _append(L, **{name: FAKE + 2}) == INVALID


@pytest.mark.parametrize("name", ["sc", "sr"])
def test_append_refuses_misaligned_scales(L, name):
    assert _append(L, **{**dict(bc=4, br=4, sc=FAKE, sr=FAKE), name: FAKE + 2}) == INVALID


@pytest.mark.parametrize("name", ["ts", "q_pos", "bt", "segs"])
@pytest.mark.parametrize("off", [1, 2])
def test_chunk_refuses_misaligned_arrays(L, name, off):
    assert _chunk(L, **{name: FAKE + off}) == INVALID


def test_in_place_with_other_strides_is_refused(L):
    assert _rope(L, xt=0) == INVALID                    # x and out are the same pointer
    assert _rope(L, xh=0) == INVALID
    assert _rope(L, xt=8 * 64 + 64) == INVALID
    assert _rope(L, ot=16 * 64, oh=128) == INVALID
    assert _linear(L, res=FAKE, rs=16) == INVALID
    assert _linear(L, res=FAKE, rs=8, os=9) == INVALID


@pytest.mark.parametrize("values", [[0, 2 ** 31], [-2 ** 31 - 1], [2 ** 32 + 5], [0.5], [8, 2 ** 40, 8]])
def test_binding_refuses_integers_that_32_bits_do_not_hold(values):
    """Relocation offsets and sections: wrapped, they would be other ones."""
    with pytest.raises(ValueError, match="32-bit"):
        mla._ints(values)


def test_binding_takes_integers_of_any_kind():
    assert list(mla._ints([2 ** 31 - 1, -2 ** 31, np.int64(7), 8.0])) == [2 ** 31 - 1, -2 ** 31, 7, 8]
