"""What the paged cache's calls latch on the device, and how it is reported."""
import pytest

import pages_ref as R
from test_gpu_pages import Filled, _cu, _i32, _np

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


@pytest.mark.parametrize("rows, counts", [([0, 1, 0], [1, 1, 1]), ([1, 0, 0], [2, 1, 70]), ([0] * 130 + [1], [0] * 128 + [3, 2, 2])])
def test_append_refuses_a_row_that_is_named_twice(rows, counts):
    """Its pages and summaries stay as they are; the other row's token is written."""
    import torch
    f = Filled([200, 100], n_pages=20)
    p = f.pool
    before = [p.tensors[n].clone() for n in ("pages", "summary")]
    n, at = sum(counts), sum(counts[:rows.index(1)])
    x = torch.randn(n, 2, 128, device="cuda").to(torch.bfloat16)
    p.append(0, x, x, rows=_i32(rows), cu=None if counts == [1] * 3 else _cu(counts), max_new=max(counts))
    assert names(p) == ["DQ_EINVAL"]
    own = p.tensors["table"][0, :4].tolist()
    for t, b in zip((p.tensors[n] for n in ("pages", "summary")), before):
        assert torch.equal(t.view(20, -1)[own], b.view(20, -1)[own])
    new = counts[rows.index(1)]
    k, v = (torch.empty(new, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    p.read(0, k, v, rows=_i32([1]), cu=_cu([new]), max_new=new)
    p.check()
    want = torch.tensor(R.quantise(_np(x[at:at + new]), 0)[2]).to(torch.bfloat16)
    assert torch.equal(k.cpu(), want) and torch.equal(v.cpu(), want)


def test_append_takes_a_row_that_is_named_again_without_tokens():
    import torch
    f = Filled([200, 100], n_pages=20)
    x = torch.randn(3, 2, 128, device="cuda").to(torch.bfloat16)
    f.pool.append(0, x, x, rows=_i32([0, 1, 0, -1, -1]), cu=_cu([2, 1, 0, 0, 0]), max_new=2)
    k, v = torch.empty_like(x), torch.empty_like(x)
    f.pool.read(0, k, v, cu=_cu([2, 1]), max_new=2)
    f.pool.check()
    assert torch.equal(k.cpu(), torch.tensor(R.quantise(_np(x), 0)[2]).to(torch.bfloat16)) and torch.equal(k, v)


def test_a_new_handle_is_ready_on_every_stream():
    """Memory that held something else, a long fill of the current stream, and the first call at once on another stream."""
    import torch
    f = Filled([2500, 1900, 40], n_pages=128, max_pages_per_seq=50)
    q = f.queries([1, 1, 1])
    want = f.attend(q, [1, 1, 1])
    out, lse = torch.empty_like(q), torch.empty(3, 8, device="cuda")
    side, size = torch.cuda.Stream(), f.pool.tensors["workspace"].numel()
    x = torch.zeros(1 << 28, device="cuda")
    for _ in range(3):
        used = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        del used
        for _ in range(20):
            x.add_(1.0)
        two = f.pool.share()
        two.attention(0, q, out, lse=lse, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        del two
    f.pool.check()


def test_a_handle_made_while_a_graph_is_captured():
    import torch
    f = Filled([2500, 1900, 40], n_pages=128, max_pages_per_seq=50)
    q = f.queries([1, 1, 1])
    want = f.attend(q, [1, 1, 1])[0]
    out = torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        two = f.pool.share()
        two.attention(0, q, out)
    for _ in range(3):
        out.zero_()
        g.replay()
        assert torch.equal(out, want)
    f.pool.check()
