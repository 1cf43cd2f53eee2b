"""The shapes that the products are tested at reach every tile and every cut of the rule by which
moe_mx_linear chooses."""
import pytest

from linear_rule import FEW, MANY, Rule


def test_the_rule_is_read():
    r = Rule()
    assert r.few > 0 and len(r.tiles) == 4 and r.smallest not in [t[:2] for t in r.tiles]
    assert r.tile(r.few, 4096) is None and r.tile(r.few + 1, 1) == r.smallest


def test_every_tile_has_a_shape():
    r = Rule()
    assert set(MANY) == {t[:2] for t in r.tiles} | {r.smallest}


@pytest.mark.parametrize("tile", MANY, ids=lambda t: f"{t[0]}x{t[1]}")
def test_shapes_reach_their_tile(tile):
    T, N, K = MANY[tile]
    assert Rule().tile(T, N) == tile
    assert T % tile[0] and N % tile[1] and K // 128 >= 5


@pytest.mark.parametrize("cut", FEW, ids=lambda c: "{} steps, {} passes, {}".format(*c))
def test_shapes_of_few_rows_reach_their_cut(cut):
    assert Rule().cut(*FEW[cut]) == cut
