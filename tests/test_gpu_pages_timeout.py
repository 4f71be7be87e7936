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
