"""BlockManager.take with counts that no manager has, or that an int32 does not hold."""
import pytest

from libbuild import build_and_import

pkv = build_and_import()


@pytest.mark.parametrize("n", [7, 2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 1, 10 ** 30])
def test_more_than_there_are(n):
    bm = pkv.BlockManager(6, 4)
    with pytest.raises(pkv.PkvError) as e:
        bm.take(n)
    assert e.value.status == pkv.ERR_NO_BLOCKS and bm.num_free == 6


@pytest.mark.parametrize("n", [-1, -5])
def test_fewer_than_none(n):
    bm = pkv.BlockManager(6, 4)
    with pytest.raises(pkv.PkvError) as e:
        bm.take(n)
    assert e.value.status == pkv.ERR_INVALID_ARG and bm.num_free == 6
