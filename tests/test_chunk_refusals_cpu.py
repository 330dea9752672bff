"""More refusals of the prompt-chunk entry points, on the CPU: none of the fake pointers is ever used."""
import pytest

from tests.test_chunk_abi_cpu import FAKE, INVALID, L, _append, _chunk  # noqa: F401  (L: the fixture)


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
