"""tq_kv_attn at the edges of what its arguments allow: pages that are not
there, weights far apart, the launch plans of each shape."""
import numpy as np
import pytest

from gpu_util import say
from test_gpu_kv_attn import _check, _inputs, _run

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# rows and lengths that the kernels for 16, 32 and 128 rows take
LENS = [[(1, 700)], [(50, 900)], [(1040, 2000)], [(1040, 1200), (300, 400), (1, 1)]]


@pytest.mark.parametrize("i", range(len(LENS)))
def test_missing_pages_beside_a_page_that_was_never_written(i):
    """Holes in the middle of a context, while page 0 of the pool, which no
    sequence holds, has whatever scales its memory had: the same output bits
    as with ordinary ones there."""
    lens = LENS[i]
    say(f"attention with holes and an unwritten page 0, {lens}")
    d = _inputs(np.random.default_rng(400 + i), 4, 2, 128, lens)
    table = d["table"]
    if (table == 0).any():  # page 0's place goes to a page that nobody holds
        table[table == 0] = next(p for p in range(len(d["ks"])) if not (table == p).any())
    table[0, 3], table[0, 7], table[0, 8] = -1, 1 << 20, -9
    clean = _run(d)
    _check(d, clean)
    for ks, vs in ((np.inf, np.inf), (2.0 ** -6, np.inf), (np.inf, 2.0 ** -6), (2.0 ** -6, 2.0 ** 122), (2.0 ** 100, 2.0 ** 127),
                   (np.nan, np.nan), (2.0 ** -6, np.nan), (-1.0, 2.0 ** 122), (0.0, 0.0), (2.0 ** -6, 2.0 ** -126)):
        d["ks"][0], d["vs"][0] = ks, vs
        assert np.array_equal(_run(d).view(np.uint16), clean.view(np.uint16)), (ks, vs)
