"""Small weights over e4m3 caches: rows that give one slot most of their weight
and thousands of slots the rest keep that rest's share (to the bound of
kv_bounds.py, which allows nothing absolutely), in narrow, wide and pair items, whole and
cut into parts."""
import pytest

from kv_bounds import Sink

pytestmark = pytest.mark.gpu

# 24, 100 and 200 rows of a key head
SHAPES = {"narrow": 6, "wide": 25, "pair": 50}


@pytest.mark.parametrize("spread", [0.0, 1.0])
@pytest.mark.parametrize("share", [0.3, 0.6, 0.9])
@pytest.mark.parametrize("slots", [2000, 8000, 32000])
@pytest.mark.parametrize("shape", list(SHAPES))
def test_small_weights(shape, slots, share, spread):
    """In a batch of as many sequences as there are groups, so that no item is cut."""
    Sink(slots, share, spread, SHAPES[shape], 304, seed=slots).check()


@pytest.mark.parametrize("shape", list(SHAPES))
def test_small_weights_in_parts(shape):
    Sink(20000, 0.8, 0.5, SHAPES[shape], 1, seed=1).check()
    Sink(5000, 0.8, 0.0, SHAPES[shape], 17, D=64, page=16, seed=2).check()
