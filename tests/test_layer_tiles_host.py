"""Which kernel a product with its epilogue runs (no GPU needed): the sizes that the GPU tests mean for a tile reach it."""
import pytest

L = pytest.importorskip("fp8_block_scaled_pf8_amd._lib", reason="libpf8.so not built (run __graft_entry__.build())")

from tests.test_gpu_fprop_act_tiles import CASES, FIRST  # noqa: E402


@pytest.mark.parametrize("tile,gated,m,n,k", CASES)
def test_sizes_reach_their_tile(tile, gated, m, n, k):
    assert L.pf8_fprop_act_tile(m, n, k, int(gated)) == tile[0] * 65536 + tile[1]


def test_every_tile_is_among_them():
    assert {c[:2] for c in FIRST} == {(t, g) for t in ((64, 64), (128, 128), (256, 128), (256, 256)) for g in (False, True)}


def test_few_tokens_and_refusals():
    f = L.pf8_fprop_act_tile
    assert {f(m, 2048, 6144, 0) for m in (1, 2, 16)} == {16 * 65536 + 16}
    assert f(33, 2048, 6144, 0) == 32 * 65536 + 16 and f(257, 1024, 128, 1) == 64 * 65536 + 16
    for bad in ((0, 16, 128, 0), (1, 0, 128, 0), (1, 16, 0, 0), (1, 16, 100, 0), (1, 192, 128, 1), (1, 128, 128, 2),
                (1 << 31, 16, 128, 0), (-1, 16, 128, 0)):
        assert f(*bad) == 0
