"""The page calls where sequences have no room for pages, pools have none, or there are no sequences."""
import pytest

from test_gpu_kv_pages import Pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n_pages", [0, 10])
def test_tables_without_pages(n_pages):
    """Lengths, reference counts and the number of copies are written whole all the same."""
    p = Pool(n_pages, 3, 0, 16, apart=2)
    p.compact(n_pages)
    p.compact(12)
    p.compact(12, more=3)
    p.release([0, -1, 5], window=4)
    p.fork([-1, 0, -1])
    _, status = p.extend([0, 0, 0])
    assert status == 0
    _, status = p.extend([0, 1, 0])
    assert status == 0x10


def test_no_pages_in_the_pool():
    p = Pool(0, 3, 4, 16)
    _, status = p.extend([0, 1, 0])
    assert status == 0x20
    p.compact(0)
    p.compact(7, more=1)


def test_no_sequences():
    p = Pool(9, 0, 4, 16)
    p.extend([])
    p.compact(9)
    p.release()
