"""Cross attention over the paged cache against plain numpy in 64 bits."""
import numpy as np
import pytest

import pages_ref as R
from test_gpu_pages import Filled, _cu, _i32, _np

pytestmark = pytest.mark.gpu


class Encoded(Filled):
    """Rows whose tokens are an encoder's states."""

    def expect(self, q, counts, rows=None, chosen=None, scale=None):
        """As attention's: every query is the only, newest token of a call of its own."""
        rows = list(range(len(counts))) if rows is None else rows
        return Filled.expect(self, q, [1] * sum(counts), [r for r, n in zip(rows, counts) for _ in range(n)], None, scale)

    def attend(self, q, counts, rows=None, sel=None, scale=None, stream=None, pool=None):
        import torch
        out = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
        lse = torch.full(q.shape[:2], float("nan"), device="cuda")
        one = all(n == 1 for n in counts)
        (pool or self.pool).cross(self.layer, q, out, rows=None if rows is None else _i32(rows), cu=None if one else _cu(counts),
                                  max_new=max(counts), lse=lse, sm_scale=scale, stream=stream)
        return out, lse


@pytest.mark.parametrize("d, G, P, dtype", [(64, 1, 64, "f16"), (128, 4, 16, "bf16"), (64, 16, 32, "bf16"), (128, 8, 128, "f16"),
                                            (128, 1, 32, "bf16"), (64, 3, 16, "f16")])
def test_one_to_a_few_queries(d, G, P, dtype):
    """More queries than states, states that end inside tiles and pages, none, padding rows, a row named twice."""
    lens = [1, 0, 3, 15, 16, P, P + 1, 4 * P + 5, 129, 250]
    f = Encoded(lens, seed=d + G, n_kv_heads=2, n_q_heads=2 * G, head_dim=d, page_size=P, dtype=dtype, n_pages=100, max_pages_per_seq=20)
    f.verify(f.queries([1] * len(lens)), [1] * len(lens))
    rows, counts = [3, -1, 0, 9, 9, 2, 8, 1, 7, 4, 6, 5], [2, 1, 4, 1, 3, 5, 2, 3, 0, 1, 2, 4]
    f.verify(f.queries(counts, amp=3.0), counts, rows)


@pytest.mark.parametrize("d, G, P, dtype", [(64, 1, 16, "bf16"), (128, 4, 64, "f16"), (64, 7, 128, "f16"), (128, 16, 32, "bf16")])
def test_many_queries(d, G, P, dtype):
    """Blocks of query rows over fewer and more states than queries, in one call with single ones and empty rows."""
    lens = [40, 700, 1, 0, 128, 129, 300]
    f = Encoded(lens, seed=G, n_kv_heads=2, n_q_heads=2 * G, head_dim=d, page_size=P, dtype=dtype, n_pages=120, max_pages_per_seq=45)
    counts = [150, 90, 70, 33, 1, 0, 64]
    f.verify(f.queries(counts), counts)
    more = [70 if G == 1 else 33, 1, 0, 2, 1, 3, 1, 1, 0, 1, 1, 1, 2, 1]  # few on average: they have a launch of their own
    f.verify(f.queries(more), more, [1, 0, 6, 2, 5, 3, 4, 6, 1, 1, 0, 5, 6, 2])
    f.verify(f.queries([300]), [300], [1])
    f.verify(f.queries([65]), [65], [2])
    f.verify(f.queries([40, 66]), [40, 66], [1, 1])


def test_negative_and_zero_scales():
    f = Encoded([333, 70], page_size=64)
    for n in (1, 3, 40):
        for s in (-0.1, 0.0):
            f.verify(f.queries([n, n + 1]), [n, n + 1], scale=s)


def test_very_many_rows():
    rng = np.random.default_rng(8)
    lens = [int(x) for x in rng.integers(0, 90, 500)]
    f = Encoded(lens, n_pages=1500, max_pages_per_seq=6, page_size=32, n_kv_heads=1, n_q_heads=2, head_dim=64)
    for most in (2, 5, 40):
        counts = [int(x) for x in rng.integers(0, most, 500)]
        f.verify(f.queries(counts), counts)


def test_the_last_token_sees_what_attention_shows_it():
    """One query a row: cross attention and attention are the same call, bit for bit."""
    import torch
    f = Encoded([500, 33, 0, 64], n_pages=64)
    q = f.queries([1] * 4)
    a, b = f.attend(q, [1] * 4), Filled.attend(f, q, [1] * 4)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_what_is_out_of_range_is_latched():
    import torch
    from quantized_decode_attention_gb300 import DQError
    f = Encoded([40, 70], page_size=64)
    q = f.queries([2, 2])
    out = torch.empty_like(q)
    for rows, cu, most in (([0, 2], [0, 2, 4], 2), ([0, 1], [0, 2, 5], 4), ([0, 1], [0, 3, 2], 4), ([0, 1], [0, 1, 4], 2)):
        f.pool.cross(0, q, out, rows=_i32(rows), cu=_i32(cu), max_new=most)
        with pytest.raises(DQError, match="out of range"):
            f.pool.check()
    for call in (lambda: f.pool.cross(0, q.float(), out), lambda: f.pool.cross(0, q, out[:1]), lambda: f.pool.cross(0, q, out, rows=_i32([0])),
                 lambda: f.pool.cross(0, q, out, lse=torch.empty(2, 8, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    f.pool.check()


def test_rows_behind_the_last_are_left_alone():
    """Outputs and lse of tokens that no row of the call has stay as they were."""
    import torch
    f = Encoded([40, 300], n_pages=20)
    for counts in ([2, 1], [3, 50]):
        q = f.queries(counts + [7])
        out, lse = torch.full_like(q, 9.0), torch.full(q.shape[:2], 9.0, device="cuda")
        f.pool.cross(0, q, out, rows=_i32([0, 1]), cu=_cu(counts), max_new=max(counts), lse=lse)
        f.pool.check()
        n = sum(counts)
        assert (out[n:] == 9).all() and (lse[n:] == 9).all()
        want, _, tol, _ = f.expect(q[:n], counts)
        assert (np.abs(_np(out[:n]) - want) <= tol).all()


@pytest.mark.parametrize("counts", [[1, 1], [4, 5], [70, 40]])
def test_captured_with_states_that_change(counts):
    """A decoder's step in a graph; its encoder's rows are replaced by shorter ones between replays, on another stream."""
    import torch
    f = Encoded([900, 70], n_pages=40, max_pages_per_seq=16)
    q = f.queries(counts)
    out, cu = torch.empty_like(q), _cu(counts)
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        f.pool.cross(0, q, out, cu=cu, max_new=max(counts))
    for lens in ([900, 70], [33, 0], [0, 64]):
        f.pool.resize(None, _i32(lens))
        f.lens = lens
        f.hk, f.hv = [h[:n] for h, n in zip(f.hk, lens)], [h[:n] for h, n in zip(f.hv, lens)]
        if lens == [0, 64]:
            break  # (row 1 was emptied: its new page holds nothing of use)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        f.pool.check()
        want, _, tol, _ = f.expect(q, counts)
        assert (np.abs(_np(out) - want) <= tol).all()


def test_single_queries_beside_many():
    """One row brings many queries and the others few: those of few have the kernel for few, and the bits that a call of theirs
    alone gives (32 states are one step of it, whatever share they are in; max_new 5 as a bound takes the same tile)."""
    import torch
    f = Encoded([1 + 2 * i % 32 for i in range(16)] + [300], n_q_heads=8, n_pages=64)
    counts = [1 + i % 3 for i in range(16)] + [300]
    n = sum(counts[:16])
    q = f.queries(counts)
    out, lse = f.attend(q, counts)
    alone, lse_alone = torch.empty_like(q[:n]), torch.empty_like(lse[:n])
    f.pool.cross(0, q[:n], alone, cu=_cu(counts[:16]), max_new=5, lse=lse_alone)
    f.pool.check()
    assert torch.equal(lse[:n], lse_alone) and torch.equal(out[:n], alone)
    want, _, tol, _ = f.expect(q, counts)
    assert (np.abs(_np(out) - want) <= tol).all()
