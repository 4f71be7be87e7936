"""The paged cache's kernel for many query rows where its running maximum moves, where its inputs are
extreme, and run again on the same inputs; against plain numpy in 64 bits (pages_ref)."""
import numpy as np
import pytest

import pages_ref as R
from test_gpu_pages import Filled, _cu, _dt, _i32, _np, _pool

pytestmark = pytest.mark.gpu

NEW = 40  # new tokens: with 4 query heads a KV head, one full tile of 128 query rows and a part of another


def rising(steps, n, dtype, d, H=2, G=4, seed=0):
    """A row of n tokens whose logits rise by `rise` at each (token, rise) of `steps` for queries along a sign pattern,
    and whose values shrink by as much, so that the outputs weigh old and new tokens alike; those queries, queries
    against the pattern (falling logits) and random ones in one warp."""
    import torch
    rng = np.random.default_rng(seed)
    z = np.zeros(n)
    for at, rise in steps:
        z[at:] += rise
    sign = rng.choice([-1.0, 1.0], size=(H, d))
    k = (0.05 + z[:, None, None] / np.sqrt(d)) * sign
    v = rng.normal(size=(n, H, d)) * np.clip(1000 * np.exp(-z), 2.0 ** -6, 1000)[:, None, None]
    f = Filled.__new__(Filled)
    f.pool = _pool(dtype=dtype, max_seqs=1, n_kv_heads=H, n_q_heads=H * G, head_dim=d, page_size=32, n_pages=n // 32 + 1,
                   max_pages_per_seq=n // 32 + 1)
    f.dtype, f.layer, f.lens, f.rng, f.Hkv, f.G, f.d, f.P = dtype, 0, [n], rng, H, G, d, 32
    k, v = (torch.tensor(x).to(_dt(dtype)) for x in (k, v))
    f.pool.resize(None, _i32([n]))
    f.pool.append(0, k.cuda(), v.cuda(), cu=_cu([n]), max_new=n)
    f.hk, f.hv = [R.quantise(_np(k), 0)[2]], [R.quantise(_np(v), 0)[2]]
    q = rng.normal(size=(NEW, H * G, d))
    for h in range(H * G):
        if h % 4 < 3:
            q[:, h] = sign[h // G] * (-1.0 if h % 4 == 2 else 1.0)
    return f, torch.tensor(q).to(_dt(dtype)).cuda()


def close(f, q, counts):
    """Within the bound of Filled.expect and what raising a maximum adds to it: a weight is rounded up to 3 more times
    (a tile's weights follow each later raise in the tile: 3 2^-11 of the weight), each of its 4 roundings is off by
    2^-25 at least where the weight is below binary16's normal range (2^-32 of the largest weight, which is held as
    2^7 or more), and a raise's factor, off by 2^-22, stands in the sum and the accumulator alike but moves the
    logarithm of the sum: 2^-22 for each 32 tokens."""
    out, lse = f.attend(q, counts)
    f.pool.check()
    want, wl, tol, ltol = f.expect(q, counts)
    at = 0
    for r, n in enumerate(counts):
        for h in range(f.Hkv * f.G):
            big = np.abs(f.hv[r][:, h // f.G])
            seen = np.arange(f.lens[r])[None, :] <= (f.lens[r] - n + np.arange(n))[:, None]
            a, _ = R.attend(_np(q)[at:at + n, h], f.hk[r][:, h // f.G], big, seen, f.d ** -0.5)
            tol[at:at + n, h] += 3 * 2.0 ** -11 * a + 4 * 2.0 ** -32 * big.sum(0)
        ltol[at:at + n] += 2.0 ** -22 * (f.lens[r] / 32 + 1)
        at += n
    err = np.abs(_np(out) - want)
    assert (err <= tol).all(), (float((err / tol).max()), float(err.max()))
    assert (np.abs(_np(lse) - wl) <= ltol).all(), float((np.abs(_np(lse) - wl) / ltol).max())


@pytest.mark.parametrize("dtype, d", [("f16", 128), ("bf16", 64)])
@pytest.mark.parametrize("steps, n", [
    ([(160, 5.8), (224, 5.8)], 290),                        # twice within a tile, weights of the tile before it
    ([(128, 5.8), (256, 5.8)], 390),                        # where tiles begin
    ([(224, 6.5)], 260),                                    # the last 32 tokens of a tile
    ([(32 * i, 3.0) for i in range(1, 10)], 330),           # every 32 tokens
    ([(900, 5.8), (1210, 5.8), (2400, 6.0)], 2700),         # units that CTAs share
])
def test_maxima_that_rise_along_the_row(steps, n, dtype, d):
    f, q = rising(steps, n, dtype, d, seed=n)
    close(f, q, [NEW])


@pytest.mark.parametrize("counts", [[40, 33, 150], [600, 1, 9]])
def test_many_tokens_are_the_same_every_time(counts):
    import torch
    f = Filled([1000, 700, 333], n_pages=64, max_pages_per_seq=20)
    q = f.queries(counts)
    a = [f.attend(q, counts) for _ in range(6)]
    f.pool.check()
    for x in a[1:]:
        assert torch.equal(x[0], a[0][0]) and torch.equal(x[1], a[0][1])


@pytest.mark.parametrize("dtype, amp", [("bf16", 2.0 ** 40), ("bf16", 2.0 ** -60), ("f16", 2.0 ** 13), ("f16", 2.0 ** -14)])
def test_many_tokens_of_very_large_and_very_small_queries(dtype, amp):
    f = Filled([170, 200], dtype=dtype)
    f.verify(f.queries([NEW, NEW], amp=amp), [NEW, NEW], scale=0.1 / amp)


def test_many_tokens_where_one_key_takes_all_and_where_all_are_equal():
    import torch
    f = Filled([350, 150], wide=False)
    q = f.queries([NEW, NEW])
    q[:NEW] = (torch.tensor(f.hk[0][177]).repeat_interleave(4, 0) * 8).to(q.dtype).cuda()
    q[NEW:] = 0.0
    close(f, q, [NEW, NEW])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_query_that_is_not_finite_stays_in_its_row_among_many(bad):
    import torch
    f = Filled([350])
    q = f.queries([NEW])
    want, _, tol, _ = f.expect(q, [NEW])
    q[7, 3, 5] = bad
    out, lse = f.attend(q, [NEW])
    assert torch.isnan(out[7, 3]).all() and torch.isnan(lse[7, 3])
    err = np.abs(_np(out) - want)
    err[7, 3] = 0
    assert (err <= tol).all()


def test_many_tokens_of_strided_queries_and_exponents():
    import torch
    f = Filled([190, 133], k_exp=3, v_exp=-6, page_size=32, dtype="f16")
    w = torch.empty(2 * NEW, 3, 8, 128, dtype=torch.float16, device="cuda")
    w[:, 1] = f.queries([NEW, NEW])
    f.verify(w[:, 1], [NEW, NEW])
    f.verify(w.permute(2, 0, 1, 3)[:, :, 1].transpose(0, 1), [NEW, NEW])
