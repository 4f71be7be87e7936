"""Cross and shared attention, weighing and eviction at the ends of their ranges."""
import numpy as np
import pytest

import pages_ref as R
from test_gpu_pages import Filled, _cu, _i32, _np, _pool
from test_gpu_pages_cross import Encoded
from test_gpu_pages_scores import Pool2, Weighed, chosen
from test_gpu_pages_shared import Forked

pytestmark = pytest.mark.gpu


def test_shared_of_1024_rows_in_groups_of_all_sizes():
    """Groups of none, one and many rows, rows in no group, one and several tokens a row."""
    rng = np.random.default_rng(2)
    sizes, groups = [], []
    while sum(sizes) < 900:
        sizes.append(int(rng.choice([1, 2, 3, 9, 33, 70])))
        groups.append((int(rng.integers(0, 130)), [None if rng.random() < 0.05 else int(x) for x in rng.integers(1, 40, sizes[-1])]))
    f = Forked(groups, n_pages=6000, page_size=16, max_pages_per_seq=12, n_kv_heads=1, n_q_heads=2, head_dim=64)
    n = len(f.lens)
    assert n <= 1024
    f.verify(f.queries([1] * n), [1] * n)
    counts = [max(1, min(x, int(y))) for x, y in zip(f.lens, rng.integers(0, 9, n))]
    f.verify(f.queries(counts), counts)
    f.bounds = [5, 5] + f.bounds[2:-3] + [f.bounds[-4]] * 2  # an empty group at either end, rows outside
    f.verify(f.queries([1] * n), [1] * n)


@pytest.mark.parametrize("rows, n", [(1, 1), (3, 1), (2, 70)])
def test_shared_where_nothing_or_everything_is_small(rows, n):
    """One row, groups of a row each, one page in common."""
    f = Forked([(16, [n] * rows)], n_pages=60, page_size=16, max_pages_per_seq=12, n_q_heads=4)
    counts = [n] * rows
    f.verify(f.queries(counts), counts)
    f.bounds = list(range(rows + 1))
    assert f.plan(counts, None, f.bounds)[:, 0].tolist() == [0] * rows
    f.verify(f.queries(counts), counts)


def test_many_heads():
    """128 KV heads, and 16 query heads a KV head."""
    f = Encoded([70, 5], n_kv_heads=128, n_q_heads=128, head_dim=64, n_pages=8)
    f.verify(f.queries([2, 40]), [2, 40])
    g = Forked([(128, [3, 9, 1])], n_kv_heads=64, n_q_heads=128, head_dim=64, n_pages=12)
    g.verify(g.queries([1, 2, 1]), [1, 2, 1])
    w = Weighed([70, 5], n_kv_heads=128, n_q_heads=128, head_dim=64, n_pages=8)
    w.verify_weights([2, 1])
    w.verify_weights([60, 5])


def test_weights_of_queries_below_the_normal_range():
    """fp16 queries whose values are subnormal, with a scale that makes the softmax an ordinary one."""
    f = Weighed([70, 200], dtype="f16")
    for n in (1, 20):
        f.verify_weights([n, n], amp=2.0 ** -14, scale=0.1 * 2.0 ** 14)


def test_a_mixed_batch_is_weighed_by_both_kernels():
    f = Weighed([400, 900, 0, 33, 700, 64, 1300], n_pages=80, max_pages_per_seq=24)
    f.verify_weights([150, 1, 1, 33, 2, 9, 64])
    f.verify_weights([64, 33, 150, 1, 9, 1, 1], [5, 3, 0, -1, 4, 2, 6])


def test_1024_pairs_are_evicted():
    rng = np.random.default_rng(6)
    n = 500
    lens = [int(x) for x in rng.integers(0, 40, n)]
    f = Pool2(lens, n, L=2, H=1, d=64, P=16, n_pages=3300, M=3, seed=6)
    keep = [int(rng.integers(0, x + 1)) for x in lens]
    dst = [int(x) for x in n + rng.permutation(n)]
    f.resize(dst, keep)
    f.verify(list(range(n)) + [-1] * 24, dst + [3] * 24, 0, 0)
    f.pool.check()


def test_evict_of_more_scores_than_shared_memory_holds():
    """60000 tokens, 49152 of whose scores are held on chip; equal scores across that border."""
    import torch
    n, keep = 60000, 20000
    p = _pool(n_pages=1700, page_size=64, n_kv_heads=1, n_q_heads=1, head_dim=64, max_seqs=2, max_pages_per_seq=960)
    p.resize(_i32([0, 1]), _i32([n, keep]))
    g = torch.Generator("cuda").manual_seed(1)
    k, v = (torch.randn(n, 1, 64, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    p.append(0, k, v, rows=_i32([0]), cu=_i32([0, n]), max_new=n)
    for step in (0.001, 0.5, 100.0):
        s = torch.zeros(1, 2, 1, n + 1, device="cuda")
        s[0, 0, 0, :n] = torch.round(torch.randn(n, generator=g, device="cuda") / step) * step
        before = s[0, 0, 0, :n].cpu().numpy()
        p.evict(s, _i32([0]), _i32([1]), keep_first=4, keep_last=100)
        p.check()
        fixed = np.r_[0:4, n - 100:n]
        order = np.argsort(-before[4:n - 100], kind="stable")[:keep - 104] + 4
        pick = np.sort(np.r_[fixed, order])
        assert np.array_equal(s[0, 1, 0, :keep].cpu().numpy(), before[pick])
        ka, va = (torch.empty(keep, 1, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        kb, vb = (torch.empty(n, 1, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        p.read(0, ka, va, rows=_i32([1]), cu=_i32([0, keep]), max_new=keep)
        p.read(0, kb, vb, rows=_i32([0]), cu=_i32([0, n]), max_new=n)
        at = torch.tensor(pick, device="cuda")
        assert torch.equal(ka, kb[at]) and torch.equal(va, vb[at])


def test_beyond_four_gigabytes_of_pages():
    """Pages whose bytes lie past 2^32: all four operators."""
    import torch
    N, P = 32000, 128
    p = _pool(n_pages=N, page_size=P, n_kv_heads=8, n_q_heads=32, max_seqs=4, max_pages_per_seq=5)
    assert p.tensors["pages"].numel() > 1 << 32
    p.tensors["refs"][:N - 14] = 1  # what is free lies at the end
    rng = np.random.default_rng(4)
    k, v = (torch.tensor(rng.normal(size=(420, 8, 128))).to(torch.bfloat16).cuda() for _ in range(2))
    p.resize(_i32([0]), _i32([400]))
    p.append(0, k[:400], v[:400], rows=_i32([0]), cu=_i32([0, 400]), max_new=400)
    p.fork(_i32([0, 0]), _i32([1, 2]))
    p.resize(_i32([1, 2]), _i32([410, 410]))
    for r in (1, 2):
        p.append(0, k[390 + 10 * r:400 + 10 * r], v[390 + 10 * r:400 + 10 * r], rows=_i32([r]), cu=_i32([0, 10]), max_new=10)
    p.check()
    hk, hv = R.quantise(_np(k), 0)[2], R.quantise(_np(v), 0)[2]
    f = Forked.__new__(Forked)
    f.pool, f.layer, f.dtype, f.Hkv, f.G, f.d, f.P, f.rng = p, 0, "bf16", 8, 4, 128, P, rng
    f.lens, f.bounds = [400, 410, 410, 0], [0, 2]
    f.hk = [hk[:400], hk[:410], np.concatenate([hk[:400], hk[410:]])]
    f.hv = [hv[:400], hv[:410], np.concatenate([hv[:400], hv[410:]])]
    for counts in ([1, 1], [9, 3], [10, 10]):
        assert f.plan(counts, [1, 2], [0, 2])[:, 0].tolist() == [384] * 2
        f.verify(f.queries(counts), counts, [1, 2])
    e = Encoded.__new__(Encoded)
    e.__dict__.update(f.__dict__)
    e.verify(e.queries([3, 50]), [3, 50], [1, 2])
    w = Weighed.__new__(Weighed)
    w.__dict__.update(f.__dict__)
    w.attend = lambda q, c, rows=None, sel=None, scale=None: Filled.attend(w, q, c, rows, sel, scale)
    for counts in ([1, 1], [10, 300]):
        w.verify_weights(counts, [1, 2], cap=420)
    p.resize(_i32([3]), _i32([200]))
    s = torch.rand(1, 4, 8, 410, device="cuda")
    before = _np(s)
    p.evict(s, _i32([2]), _i32([3]), keep_last=10)
    p.check()
    ka, va = (torch.empty(200, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    p.read(0, ka, va, rows=_i32([3]), cu=_i32([0, 200]), max_new=200)
    for h in range(8):
        pick = chosen(before[0, 2, h], 410, 200, 0, 10)
        assert (_np(ka[:, h]) == f.hk[2][pick, h]).all() and (_np(va[:, h]) == f.hv[2][pick, h]).all()


def test_calls_on_another_device_are_refused_and_streams_are_taken_as_numbers():
    import torch
    f = Forked([(200, [30, 22])], n_pages=40, n_q_heads=4)
    s = torch.cuda.Stream()
    q = f.queries([1, 1])
    out, plan, scratch = torch.empty_like(q), torch.empty(2, 2, dtype=torch.int32, device="cuda"), f.pool.shared_scratch(2)
    torch.cuda.synchronize()
    f.pool.common(plan, always=True, stream=s.cuda_stream)
    f.pool.shared(0, q, out, plan, scratch, stream=s.cuda_stream)
    f.pool.check(s.cuda_stream)
    want, _, tol, _ = f.expect(q, [1, 1])
    assert (np.abs(_np(out) - want) <= tol).all()
    for call in (lambda: f.pool.cross(0, q, out.cpu()), lambda: f.pool.common(plan.cpu()), lambda: f.pool.weigh(0, q, torch.empty(2, 4), torch.empty(1)),
                 lambda: f.pool.evict(torch.zeros(1, 3, 2, 9), _i32([0]), _i32([1]))):
        with pytest.raises(ValueError):
            call()
