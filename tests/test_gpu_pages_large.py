"""The paged cache at the ends of its ranges: the largest pool and row table, the most heads, pages chosen among the most;
against plain numpy in 64 bits (pages_ref)."""
import numpy as np
import pytest

import pages_ref as R
from test_gpu_pages import Filled, _i32, _np, _pool, _same

pytestmark = pytest.mark.gpu


def test_lengths_and_compaction_of_the_largest_pool():
    """2^20 pages, nearly all held: the free ones lie anywhere, the live ones that move at the end."""
    import torch
    from quantized_decode_attention_gb300 import DQError
    N, P, S, M = 1 << 20, 16, 6, 3000
    rng = np.random.default_rng(3)
    pool = _pool(page_size=P, n_pages=N, max_seqs=S, max_pages_per_seq=M, n_kv_heads=1, n_q_heads=1, head_dim=64)
    m = R.Model(N, P, S, M)
    m.refs = [int(x) for x in rng.random(N) < 0.995]  # held by rows that are not in this table
    pool.tensors["refs"].copy_(torch.tensor(m.refs, dtype=torch.int32))
    pool.tensors["pages"].random_(0, 256, generator=torch.Generator("cuda").manual_seed(1))
    bytes_of = lambda: pool.tensors["pages"].view(N, -1)
    assert N - sum(m.refs) > 1024
    for lens in ([1500 * P + 1, 3, 0, 2000 * P, 17, P], [9, 700 * P, 1200 * P + 5, 2000 * P, 0, 1300 * P], [M * P] * 6):
        fine = m.resize(range(S), lens)
        pool.resize(None, _i32(lens))
        if fine:
            pool.check()
        else:
            with pytest.raises(DQError, match="DQ_ENOMEM"):
                pool.check()
        _same(pool, m)
    assert not fine
    want = bytes_of().clone()
    m.compact()
    pool.compact()
    pool.check()
    _same(pool, m)
    assert m.copies
    a, b = (torch.tensor(x, device="cuda") for x in zip(*m.copies))
    want[b] = want[a]
    assert torch.equal(bytes_of(), want)


def test_the_most_heads():
    f = Filled([70, 5, 0], n_kv_heads=128, n_q_heads=256, head_dim=64, page_size=32, n_pages=8, max_pages_per_seq=4)
    for counts in ([1, 1, 1], [3, 2, 1], [40, 3, 20]):
        f.verify(f.queries(counts), counts)


def test_the_most_query_heads_a_kv_head():
    f = Filled([150, 33], n_kv_heads=32, n_q_heads=512, head_dim=128, page_size=16, n_pages=16, max_pages_per_seq=12)
    for counts in ([1, 1], [2, 1], [17, 5]):
        f.verify(f.queries(counts), counts)


@pytest.mark.parametrize("keep, first, last", [(512, 3, 2), (1, 0, 0), (37, 0, 0)])
def test_a_choice_among_the_most_pages(keep, first, last):
    import torch
    n, H, d = 16384, 2, 64
    rng = np.random.default_rng(keep)
    pool = _pool(n_pages=n, page_size=16, n_kv_heads=H, n_q_heads=2 * H, head_dim=d, max_seqs=1, max_pages_per_seq=n)
    raw = rng.integers(-127, 128, size=(n, H, 2, d)).astype(np.int8)
    raw.sort(axis=2)
    raw = raw[:, :, ::-1]  # largest, smallest
    e = rng.integers(-6, 4, size=(n, H)).astype(np.int32)
    img = np.zeros((n, H, 2 * d + 16), dtype=np.uint8)
    img[:, :, :2 * d] = raw.reshape(n, H, 2 * d).view(np.uint8)
    img[:, :, 2 * d:2 * d + 4] = e[..., None].view(np.uint8)
    pool.tensors["summary"].copy_(torch.tensor(img.reshape(-1)))
    pool.resize(None, _i32([16 * n - 5]))
    table = pool.tensors["table"][0].cpu().numpy()
    q = torch.tensor(rng.normal(size=(1, 2 * H, d))).to(torch.bfloat16).cuda()
    sel = torch.empty(1, H, keep, dtype=torch.int32, device="cuda")
    pool.select(0, q, sel, keep_first=first, keep_last=last)
    pool.check()
    for h in range(H):
        sums = [(raw[table[j], h, 0], raw[table[j], h, 1], int(e[table[j], h])) for j in range(n)]
        assert sel[0, h].tolist() == R.choose(_np(q[0, 2 * h:2 * h + 2]), sums, n, keep, first, last)
