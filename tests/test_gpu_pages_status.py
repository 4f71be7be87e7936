"""What the paged cache's calls latch on the device, and how it is reported."""
import pytest

from test_gpu_pages import Filled, _i32

pytestmark = pytest.mark.gpu


def names(pool):
    """What repeated checks report, until there is nothing more."""
    from quantized_decode_attention_gb300 import DQError
    got = []
    while len(got) < 10:
        try:
            pool.check()
            return got
        except DQError as e:
            got.append(e.name)
    return got


def test_check_reports_everything_that_was_latched():
    """A resize that finds no pages and an append of a value that is not finite in one step: two reports, then none."""
    import torch
    f = Filled([40, 0], n_pages=4)
    f.pool.resize(_i32([1]), _i32([700]))
    f.pool.resize(_i32([0]), _i32([41]))
    x = torch.ones(1, 2, 128, dtype=torch.bfloat16, device="cuda")
    x[0, 1, 7] = float("nan")
    f.pool.append(0, x, x, rows=_i32([0]))
    assert names(f.pool) == ["DQ_ENOMEM", "DQ_ENONFINITE"]


def test_check_names_each_bit_once_the_gravest_first():
    f = Filled([40])
    status = f.pool.tensors["status"].view(-1)[:4].view(dtype=_i32([0]).dtype)
    status[0] = 1 | 2 | 64 | 128 | 256 | 512
    assert names(f.pool) == ["DQ_ETIMEOUT", "DQ_ENOMEM", "DQ_EINVAL", "DQ_EINVAL", "DQ_EINVAL", "DQ_ENONFINITE"]
    assert int(status[0]) == 0

