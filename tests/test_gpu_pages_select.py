"""Page choice where the queries are extreme."""
import pytest

import pages_ref as R
from test_gpu_pages import Filled, _np

pytestmark = pytest.mark.gpu


def chosen(f, q, keep=4):
    import torch
    sel = torch.full((q.shape[0], f.Hkv, keep), 99, dtype=torch.int32, device="cuda")
    f.pool.select(0, q, sel, keep_first=0, keep_last=0)
    f.pool.check()
    return sel.tolist()


@pytest.mark.parametrize("exp", [-90, -99, -101, -110, -121, -122, -124, 60, 110])
def test_the_choice_does_not_depend_on_the_queries_size(exp):
    """Whole queries of at most 7 bits times a power of two (bf16 holds them all, down to 2^-133): the pages are those of
    the same queries without it."""
    import torch
    f = Filled([700, 330], page_size=16, n_pages=80, max_pages_per_seq=50)
    whole = torch.tensor(f.rng.integers(-90, 91, size=(2, 8, 128)), dtype=torch.float64)
    want = [[R.choose(_np(whole[r, 4 * h:4 * h + 4]), [R.summary(f.hk[r][j * 16:j * 16 + 16, h]) for j in range(-(-f.lens[r] // 16))],
                      -(-f.lens[r] // 16), 4, 0, 0) for h in range(2)] for r in range(2)]
    q = (whole * 2.0 ** exp).to(torch.bfloat16)
    assert torch.equal(q.double(), whole * 2.0 ** exp)
    assert chosen(f, q.cuda()) == want


def test_the_smallest_queries():
    """One channel at bf16's smallest number, 2^-133, with either sign."""
    import torch
    f = Filled([700], page_size=16, n_pages=50, max_pages_per_seq=50)
    for sign in (1.0, -1.0):
        for at in (5, 77):
            q = torch.zeros(1, 8, 128, dtype=torch.float64)
            q[:, :, at] = sign
            want = [R.choose(_np(q[0, 4 * h:4 * h + 4]), [R.summary(f.hk[0][j * 16:j * 16 + 16, h]) for j in range(44)], 44, 4, 0, 0)
                    for h in range(2)]
            tiny = (q * 2.0 ** -133).to(torch.bfloat16)
            assert float(tiny.abs().max()) > 0
            assert chosen(f, tiny.cuda())[0] == want
