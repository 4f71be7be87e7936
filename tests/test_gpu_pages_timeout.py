"""A bounded wait of the paged cache's attention that runs out.

dq_pages_test_expire_wait is an attention call whose barriers wait for an arrival that
nobody makes, with a limit of 2 ms: the kernels go through their (finite) work without
it, the status says that the outputs are not valid, and the calls after it are right
again.  No fault and no hang is involved."""
import pytest

from test_gpu_pages import Filled, _cu

pytestmark = pytest.mark.gpu

LIMIT = 2_000_000  # ns


def expire(pool, q, counts):
    import torch
    from quantized_decode_attention_gb300 import pages
    out = torch.empty_like(q)
    one = all(n == 1 for n in counts)
    cu = None if one else _cu(counts)
    torch.cuda.synchronize()
    st = pages._load().dq_pages_test_expire_wait(pool._c, pool._b, 0, q.data_ptr(), q.stride(0), q.stride(1), out.data_ptr(),
                                                 None if one else cu.data_ptr(), len(counts), q.shape[0], max(counts), LIMIT,
                                                 torch.cuda.current_stream().cuda_stream)
    assert st == 0, pages._load().dq_last_error()
    torch.cuda.synchronize()


def recovers(f, counts, handles, expired):
    """Every handle's calls are what they were before the expired one; the timeout is reported once."""
    import torch
    from quantized_decode_attention_gb300 import DQError
    q = f.queries(counts)
    want = f.attend(q, counts)
    f.pool.check()
    expire(expired, q, counts)
    with pytest.raises(DQError) as e:
        handles[0].check()
    assert e.value.name == "DQ_ETIMEOUT", str(e.value)
    handles[-1].check()  # reported once
    for _ in range(3):
        for h in handles:
            got = f.attend(q, counts, pool=h)
            h.check()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("d, counts", [(128, [600, 40]), (64, [40, 333])])
def test_many_tokens_recover(d, counts):
    """Two tiles, whole units and units that CTAs share, over stages that are used again and again."""
    f = Filled([1500, 700], n_pages=64, max_pages_per_seq=24, head_dim=d)
    recovers(f, counts, [f.pool], f.pool)


@pytest.mark.parametrize("d, P, counts", [(128, 64, [1, 1, 1, 1]), (64, 16, [1, 1, 1, 1]), (128, 128, [4, 1, 2, 3]), (64, 32, [4, 4, 3, 1])])
def test_few_tokens_recover_on_every_handle(d, P, counts):
    """The workspace of the call that gave up is the second handle's, the status both handles'.  Units that CTAs share,
    units of one warp, and an empty row."""
    f = Filled([2500, 1900, 40, 0], n_pages=5000 // P, max_pages_per_seq=2600 // P + 2, page_size=P, head_dim=d)
    two = f.pool.share()
    recovers(f, counts, [f.pool, two], two)
    recovers(f, counts, [two, f.pool], f.pool)


def test_a_mixed_batch_recovers():
    f = Filled([2500, 1900, 40], n_pages=128, max_pages_per_seq=50)
    two = f.pool.share()
    recovers(f, [200, 1, 4], [f.pool, two], two)


# ---- cross and shared attention, weights ---------------------------------------------------------------
def timed_out(pool, other, name, *args):
    """The call of dq_pages_test_expire_<name>; its timeout is reported once, by whichever handle asks first."""
    import torch
    from quantized_decode_attention_gb300 import DQError, pages
    torch.cuda.synchronize()
    L = pages._load()
    assert getattr(L, "dq_pages_test_expire_" + name)(pool._c, pool._b, 0, *args, LIMIT, torch.cuda.current_stream().cuda_stream) == 0, L.dq_last_error()
    torch.cuda.synchronize()
    with pytest.raises(DQError) as e:
        other.check()
    assert e.value.name == "DQ_ETIMEOUT", str(e.value)
    pool.check()


def same_again(f, want, call):
    import torch
    for _ in range(3):
        for x, y in zip(call(), want):
            assert torch.equal(x, y)
        f.pool.check()


@pytest.mark.parametrize("d, P, lens, counts", [
    (128, 64, [1500, 700], [600, 40]), (64, 16, [900, 300], [40, 500]), (128, 64, [2500, 1900, 40, 0], [1, 1, 1, 1]),
    (64, 32, [2500, 1900, 40], [4, 3, 1]), (128, 128, [2500, 1900, 40], [1, 3, 200])])
def test_cross_attention_recovers(d, P, lens, counts):
    import torch
    from test_gpu_pages_cross import Encoded
    f = Encoded(lens, n_pages=sum(lens) // P + 8, max_pages_per_seq=max(lens) // P + 2, page_size=P, head_dim=d)
    two, q = f.pool.share(), f.queries(counts)
    want = f.attend(q, counts)
    cu = None if all(n == 1 for n in counts) else _cu(counts)
    out = torch.empty_like(q)
    for a, b in ((f.pool, two), (two, f.pool)):
        timed_out(a, b, "cross", q.data_ptr(), q.stride(0), q.stride(1), out.data_ptr(), None if cu is None else cu.data_ptr(), len(counts),
                  q.shape[0], max(counts))
        for h in (a, b):
            same_again(f, want, lambda: f.attend(q, counts, pool=h))


@pytest.mark.parametrize("d, P, groups, counts", [
    (128, 64, [(1000, [9, 30, 70, 5]), (500, [7, 90])], [1] * 6),               # few query rows in both launches
    (64, 16, [(700, [9, 30, None]), (400, [7, 90])], [2, 1, 1, 3, 2]),
    (128, 64, [(2000, [5 + i for i in range(40)])], [1] * 40),                  # few in the rows' own, many in the common one
    (128, 32, [(1500, [200, 150]), (600, [80, 120])], [150, 100, 60, 90]),      # many in both
    (128, 64, [(1500, [300, 9]), (256, [4, 1]), (320, [2, 2]), (128, [1, 1]), (640, [9, 8])], [250, 1, 1, 1, 2, 1, 1, 1, 1, 2])])  # each, in both
def test_shared_attention_recovers(d, P, groups, counts):
    """The wait runs out in the launch over the rows' own pages and in the one over the common ones, which begins beside it."""
    import torch
    from test_gpu_pages import _i32
    from test_gpu_pages_shared import Forked
    f = Forked(groups, n_pages=sum(m + sum((x or 0) + 2 * P for x in c) for m, c in groups) // P + 12, max_pages_per_seq=40 * 64 // P, page_size=P, head_dim=d)
    two, q = f.pool.share(), f.queries(counts)
    want = f.attend(q, counts)
    cu = None if all(n == 1 for n in counts) else _cu(counts)
    out, plan, scratch, b = torch.empty_like(q), f.plan(counts, None, f.bounds), f.pool.shared_scratch(sum(counts)), _i32(f.bounds)
    assert (plan[:, 0] > 0).any()
    per = max(sum(counts[x:y]) for x, y in zip(f.bounds, f.bounds[1:]))
    for a, o in ((f.pool, two), (two, f.pool)):
        timed_out(a, o, "shared", q.data_ptr(), q.stride(0), q.stride(1), out.data_ptr(), None if cu is None else cu.data_ptr(), len(counts),
                  q.shape[0], max(counts), b.data_ptr(), len(groups), per, plan.data_ptr(), scratch.data_ptr())
        for h in (a, o):
            same_again(f, want, lambda: f.attend(q, counts, pool=h))


@pytest.mark.parametrize("d, dtype, counts", [(128, "bf16", [300, 60, 17]), (64, "f16", [40, 333, 70]), (128, "f16", [1, 250, 3])])
def test_weights_recover(d, dtype, counts):
    """Whole units and units that CTAs share; in the last case with a launch for few beside it, which waits for nothing."""
    import torch
    from test_gpu_pages_scores import Weighed
    f = Weighed([2600, 900, 300], n_pages=80, max_pages_per_seq=45, head_dim=d, dtype=dtype)
    two, q, cu = f.pool.share(), f.queries(counts), _cu(counts)
    _, lse = f.attend(q, counts)
    start, s = f.scores(), f.scores()

    def weigh(pool):
        s.copy_(start)
        pool.weigh(0, q, lse, s, cu=cu, max_new=max(counts))
        return [s.clone()]

    want = weigh(f.pool)
    for a, o in ((f.pool, two), (two, f.pool)):
        timed_out(a, o, "weigh", q.data_ptr(), q.stride(0), q.stride(1), lse.data_ptr(), s.data_ptr(), s.shape[-1], cu.data_ptr(), len(counts),
                  q.shape[0], max(counts))
        for h in (a, o):
            same_again(f, want, lambda: weigh(h))


def test_weights_of_few_wait_for_nothing():
    import torch
    from quantized_decode_attention_gb300 import pages
    from test_gpu_pages_scores import Weighed
    f = Weighed([300, 77])
    q = f.queries([1, 1])
    _, lse = f.attend(q, [1, 1])
    a, b = f.scores(value=0.0), f.scores(value=0.0)
    st = pages._load().dq_pages_test_expire_weigh(f.pool._c, f.pool._b, 0, q.data_ptr(), q.stride(0), q.stride(1), lse.data_ptr(), a.data_ptr(),
                                                  a.shape[-1], None, 2, 2, 1, LIMIT, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    f.pool.weigh(0, q, lse, b, sm_scale=1.0)
    f.pool.check()
    assert torch.equal(a, b)
