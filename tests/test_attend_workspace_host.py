"""Workspaces of lean_paged_attention, no GPU needed: their sizes, which callers may
keep, are those of before caches in 8 bits."""
import pytest

from block_quantized_weight_dot_gb300 import build as lib_build


@pytest.fixture(scope="module")
def lean():
    lib_build.build()
    from block_quantized_weight_dot_gb300 import lean as L
    return L


@pytest.mark.parametrize("hq,hkv,dim", [(15, 5, 64), (8, 2, 64), (16, 2, 128), (12, 1, 64), (32, 2, 128), (6, 2, 256), (40, 4, 256),
                                        (2, 1, 16), (9, 1, 80), (9, 3, 136)])
def test_sizes_are_kept(lean, hq, hkv, dim):
    """2048 bytes; for 160 blocks ten parts (rows of dim + 4 floats) and eight folds (of dim + 8) of a group's heads."""
    h, d = (16 if hq // hkv > 8 else 8), (64 if dim <= 64 else 128 if dim <= 128 else 256)
    for seqs in (1, 384, 100000):
        assert lean.lean_paged_attention_workspace_bytes(seqs, hq, hkv, dim) == 2048 + 160 * 4 * h * (10 * (d + 4) + 8 * (d + 8))
