"""Attention of rows that begin with the same pages, against plain numpy in 64 bits."""
import numpy as np
import pytest

import pages_ref as R
from test_gpu_pages import Filled, _cu, _i32, _np, _pool

pytestmark = pytest.mark.gpu


class Forked(Filled):
    """groups: (tokens of the parent, [tokens that each child has beside them]): rows are the children, in order."""

    def __init__(self, groups, seed=0, layer=0, dtype="bf16", **kw):
        import torch
        from test_gpu_pages import _dt
        n = sum(len(c) for _, c in groups)
        self.dtype, self.layer, self.rng = dtype, layer, np.random.default_rng(seed)
        self.pool = _pool(dtype=dtype, max_seqs=n + len(groups), **kw)
        c = self.pool.cfg
        self.Hkv, self.G, self.d, self.P = c.n_kv_heads, c.n_q_heads // c.n_kv_heads, c.head_dim, c.page_size
        rnd = lambda m: torch.tensor(self.rng.normal(size=(m, self.Hkv, self.d)) * 1.5).to(_dt(dtype))
        self.pool.tensors["pages"].fill_(0xFF)
        self.lens, self.hk, self.hv, self.bounds, k_all = [], [], [], [0], []
        parents = list(range(n, n + len(groups)))
        held = []
        for p, (m, _) in zip(parents, groups):
            k, v = rnd(m), rnd(m)
            held.append((k, v))
            self.pool.resize(_i32([p]), _i32([m]))
            if m:
                self.pool.append(layer, k.cuda(), v.cuda(), rows=_i32([p]), cu=_i32([0, m]), max_new=m)
        for (m, children), (k, v), p in zip(groups, held, parents):
            first = self.bounds[-1]
            rows = list(range(first, first + len(children)))
            self.bounds.append(first + len(children))
            self.pool.fork(_i32([p] * len(rows)), _i32(rows))
            self.pool.resize(_i32([p]), _i32([0]))
            for r, more in zip(rows, children):
                if more is None:  # a place that nobody has
                    self.pool.resize(_i32([r]), _i32([0]))
                    self.lens.append(0)
                    self.hk.append(np.zeros((0, self.Hkv, self.d)))
                    self.hv.append(np.zeros((0, self.Hkv, self.d)))
                    continue
                a, b = rnd(more), rnd(more)
                self.pool.resize(_i32([r]), _i32([m + more]))
                if more:
                    self.pool.append(layer, a.cuda(), b.cuda(), rows=_i32([r]), cu=_i32([0, more]), max_new=more)
                self.lens.append(m + more)
                self.hk.append(R.quantise(_np(torch.cat([k, a])), c.k_exp)[2])
                self.hv.append(R.quantise(_np(torch.cat([v, b])), c.v_exp)[2])
        self.pool.check()
        self.parents = [m for m, _ in groups]

    def expect(self, q, counts, rows=None, chosen=None, scale=None):
        """As attention's, and two small things that its bound leaves out.  (a) The stored output is the computed one, o + e,
        rounded by at most eps |o + e| <= eps |o| + eps |e|, where |e| <= tol: eps tol more.  (b) A weight is a binary16 number
        in units in which the largest is at least 2^7, so that one below the normal range, 2^-14, is off by up to 2^-25, which is
        2^-32 of the sum: 2^-32 sum |v| more (seen where one key outweighs the rest and its value in a channel is 0)."""
        import torch
        from test_gpu_pages import _dt
        out, lse, tol, ltol = Filled.expect(self, q, counts, rows, chosen, scale)
        at = 0
        for i, n in enumerate(counts):
            r = i if rows is None else rows[i]
            if r >= 0:
                tol[at:at + n] += 2.0 ** -32 * np.abs(self.hv[r]).sum(0).repeat(self.G, 0)
            at += n
        return out, lse, tol * (1 + torch.finfo(_dt(self.dtype)).eps / 2), ltol

    always = True

    def plan(self, counts, rows=None, bounds=None):
        """What common() found, as a list of (tokens, row)."""
        import torch
        n = len(counts)
        plan = torch.full((n, 2), 77, dtype=torch.int32, device="cuda")
        one = all(x == 1 for x in counts)
        self.pool.common(plan, groups=None if bounds is None else _i32(bounds), rows=None if rows is None else _i32(rows),
                         cu=None if one else _cu(counts), always=self.always)
        return plan

    def attend(self, q, counts, rows=None, sel=None, scale=None, stream=None, pool=None):
        import torch
        out = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
        lse = torch.full(q.shape[:2], float("nan"), device="cuda")
        one = all(n == 1 for n in counts)
        b = self.bounds
        plan = self.plan(counts, rows, b)
        scratch = self.pool.shared_scratch(sum(counts))
        scratch.fill_(0xFF)
        per = max(sum(counts[x:y]) for x, y in zip(b, b[1:]))
        (pool or self.pool).shared(self.layer, q, out, plan, scratch, groups=_i32(b), max_group=max(1, per), rows=None if rows is None else _i32(rows),
                                   cu=None if one else _cu(counts), max_new=max(counts), lse=lse, sm_scale=scale, stream=stream)
        return out, lse


@pytest.mark.parametrize("d, G, P, dtype", [(128, 4, 64, "bf16"), (64, 1, 16, "f16"), (128, 8, 16, "f16"), (64, 5, 128, "bf16"),
                                            (128, 16, 32, "bf16"), (128, 1, 128, "f16")])
def test_single_tokens(d, G, P, dtype):
    """Groups of one row to many, parents that end inside a page, on its border and before the first; empty places."""
    groups = [(5 * P + 3, [1, 40, None, 2 * P, 7]), (3 * P, [1, 1, 5]), (P - 1, [1, 2, 3]), (2 * P + 1, [9]), (7 * P, [1] * 9 + [None]),
              (0, [5, 17]), (4 * P, [None, None])]
    f = Forked(groups, seed=d + G, n_kv_heads=2, n_q_heads=2 * G, head_dim=d, page_size=P, dtype=dtype, n_pages=200, max_pages_per_seq=12)
    n = len(f.lens)
    plan = f.plan([1] * n, None, f.bounds).tolist()
    for g, (m, children) in enumerate(groups):
        there = [x for x in children if x is not None]
        want = m // P * P if len(there) > 1 else 0
        for i in range(f.bounds[g], f.bounds[g + 1]):
            assert plan[i][0] == want, (g, i, plan[i])
            assert want == 0 or f.bounds[g] <= plan[i][1] < f.bounds[g + 1]
    f.verify(f.queries([1] * n), [1] * n)
    f.verify(f.queries([1] * n, amp=4.0), [1] * n, scale=0.3)


@pytest.mark.parametrize("d, G, P, dtype", [(128, 4, 64, "f16"), (64, 2, 16, "bf16"), (128, 16, 32, "f16"), (64, 7, 128, "f16")])
def test_several_tokens(d, G, P, dtype):
    """Ragged new tokens: none, a few, more than a tile of query rows, and more than the row has beside its parent (less is
    common then)."""
    groups = [(6 * P, [9, 80, 70]), (4 * P + 2, [200, 150, 3, 5]), (3 * P, [2, None, 4, 90, 1]), (5 * P, [33, 40])]
    f = Forked(groups, seed=G, n_kv_heads=2, n_q_heads=2 * G, head_dim=d, page_size=P, dtype=dtype, n_pages=200, max_pages_per_seq=24)
    for counts in ([3, 2, 1, 5, 0, 3, 2, 1, 1, 4, 7, 1, 2, 2], [9, 80, 70, 130, 1, 2, 5, 2, 3, 1, 90, 1, 40, 30],
                   [2, 80 + P, 1, 150, 150, 3, 5, 2, 1, 1, 0, 1, 33, 34]):
        f.verify(f.queries(counts), counts)


def test_common_only_where_it_pays():
    """Left to itself, common() takes much that many rows share and leaves little that few do: its estimate is far from its
    limit of 20 us on both sides (4 KV heads of 128, 144 bytes each of a key and value: 63 x 4 x 4096 x 144 / 5e6 us = 30, twice
    for two groups; 2 x 4 x 640 x 144 / 5e6 = 0.15)."""
    f = Forked([(4096, [1 + i % 5 for i in range(64)]), (640, [3, 9, 1])], n_kv_heads=4, n_q_heads=8, n_pages=300, max_pages_per_seq=70)
    n = [1] * 67
    assert f.plan(n, None, f.bounds)[:, 0].tolist() == [4096] * 64 + [640] * 3
    f.always = False
    assert f.plan(n, None, f.bounds)[:, 0].tolist() == [4096] * 64 + [0] * 3
    f.verify(f.queries(n), n)
    n = [1 + i % 5 for i in range(64)] + [2, 9, 1]
    assert f.plan(n, None, f.bounds)[:, 0].tolist() == [4096] * 64 + [0] * 3
    f.verify(f.queries(n), n)


def test_a_big_group_over_a_long_beginning():
    """One group of 70 rows: whole tiles of query rows, and parts of units in many CTAs."""
    f = Forked([(3000, [1 + i % 9 for i in range(70)])], n_pages=400, max_pages_per_seq=60)
    f.verify(f.queries([1] * 70), [1] * 70)
    counts = [1 + i % 9 for i in range(70)]
    f.verify(f.queries(counts), counts)


@pytest.mark.parametrize("counts", [[1] * 4, [3] * 4, [1, 2, 9, 20]])
def test_permuted_rows_and_rows_that_share_nothing(counts):
    """A group's rows in any order, named twice, padding among them; a stranger in the group: nothing is common."""
    f = Forked([(200, [30, 22, 41, 50])], n_pages=40, n_q_heads=4)
    f.bounds = [0, 4]
    for rows in ([2, 0, 3, 1], [1, 1, 1, 0], [-1, 2, -3, 3], [2, -1, -1, -1], [-1] * 4):
        f.verify(f.queries(counts), counts, rows)
    g = Forked([(200, [30, 22]), (200, [41, 50])], n_pages=40, n_q_heads=4)
    g.bounds = [0, 4]
    assert g.plan(counts, None, [0, 4])[:, 0].tolist() == [0] * 4
    g.verify(g.queries(counts), counts)
    g.bounds = [1, 3]  # rows of the call that are in no group
    assert g.plan(counts, None, [1, 3])[:, 0].tolist() == [0] * 4
    g.verify(g.queries(counts), counts)


def test_one_group_of_all_is_the_default():
    import torch
    f = Forked([(640, [5, 9, 13])], n_pages=40, max_pages_per_seq=14)
    q = f.queries([1] * 3)
    plan, out, scratch = f.plan([1] * 3), torch.empty_like(q), f.pool.shared_scratch(3)
    assert plan[:, 0].tolist() == [640] * 3
    f.pool.shared(0, q, out, plan, scratch)
    f.pool.check()
    want, _, tol, _ = f.expect(q, [1] * 3)
    assert (np.abs(_np(out) - want) <= tol).all()


def test_a_fork_of_a_fork_shares_the_whole_of_it():
    """Children of a child: a group of them has more in common than one with their uncle."""
    f = Forked([(256, [70, 1])], n_pages=40, page_size=64, n_q_heads=4)
    p = f.pool
    p.resize(_i32([1]), _i32([0]))
    p.fork(_i32([0]), _i32([1]))  # row 1: a second holder of row 0's 326 tokens
    f.lens[1], f.hk[1], f.hv[1] = f.lens[0], f.hk[0], f.hv[0]
    assert f.plan([1, 1]).tolist() == [[320, 0]] * 2  # (whole pages that the newest token sees all of)
    f.verify(f.queries([1, 1]), [1, 1])
    p.resize(_i32([1]), _i32([320]))  # on a page's border: the last page is not before the newest token
    f.lens[1] = 320
    f.hk[1], f.hv[1] = f.hk[0][:320], f.hv[0][:320]
    assert f.plan([1, 1])[:, 0].tolist() == [256] * 2
    f.verify(f.queries([1, 1]), [1, 1])
    assert f.plan([2, 70])[:, 0].tolist() == [192] * 2


def test_what_is_out_of_range_is_latched():
    import torch
    from quantized_decode_attention_gb300 import DQError
    f = Forked([(200, [30, 22]), (200, [41, 50])], n_pages=40)
    q = f.queries([1] * 4)
    out, scratch = torch.empty_like(q), f.pool.shared_scratch(4)
    plan = f.plan([1] * 4, None, f.bounds)
    f.pool.check()

    def bad(**kw):
        a = dict(plan=plan, groups=_i32(f.bounds), max_group=2)
        a.update(kw)
        f.pool.shared(0, q, out, a["plan"], scratch, groups=a["groups"], max_group=a["max_group"])
        with pytest.raises(DQError, match="out of range"):
            f.pool.check()

    for groups in ([0, 2, 5], [0, 3, 2], [-1, 2, 4]):
        bad(groups=_i32(groups))
        f.pool.common(plan.clone(), groups=_i32(groups))
        with pytest.raises(DQError, match="out of range"):
            f.pool.check()
    bad(max_group=1)
    for at, x in ((0, -64), (0, 63), (0, 64 * 12 + 64), (1, 99), (1, -1), (0, 1 << 30)):
        p = plan.clone()
        p[:, at] = x
        bad(plan=p)
    for call in (lambda: f.pool.shared(0, q, out, plan[:3], scratch), lambda: f.pool.shared(0, q, out, plan, scratch[:-4]),
                 lambda: f.pool.shared(0, q, out, plan.long(), scratch), lambda: f.pool.common(plan, rows=_i32([0])),
                 lambda: f.pool.common(plan, cu=_i32([0, 1])), lambda: f.pool.shared(0, q, out, plan, scratch.cpu())):
        with pytest.raises(ValueError):
            call()
    f.pool.check()


def test_the_same_every_time_and_in_graphs_on_two_streams():
    """Two handles, scratches and captured graphs over the same rows at the same time; replays after a row was shortened
    follow the plan that they capture."""
    import torch
    f = Forked([(2000, [30, 22, 5, 9, 1, 1, 60, 8])], n_pages=64, max_pages_per_seq=40)
    n = 8
    q = [f.queries([1] * n) for _ in range(2)]
    want = [f.attend(x, [1] * n) for x in q]
    for x, w in zip(q, want):
        again = f.attend(x, [1] * n)
        assert torch.equal(again[0], w[0]) and torch.equal(again[1], w[1])
    handles, s, graphs, outs, keep = [f.pool, f.pool.share()], [torch.cuda.Stream(), torch.cuda.Stream()], [], [], []
    for i in range(2):
        o, plan, scratch = torch.empty_like(q[i]), torch.empty(n, 2, dtype=torch.int32, device="cuda"), f.pool.shared_scratch(n)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s[i]):
            handles[i].common(plan, always=True)
            for _ in range(3):
                handles[i].shared(0, q[i], o, plan, scratch)
        graphs.append(g)
        outs.append(o)
        keep.append((plan, scratch))
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(s[i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(outs[i], want[i][0])
    f.pool.resize(_i32([1, 2]), _i32([700, 0]))
    f.lens[1], f.lens[2] = 700, 0
    for held in (f.hk, f.hv):
        held[1], held[2] = held[1][:700], held[2][:0]
    torch.cuda.synchronize()
    graphs[0].replay()
    torch.cuda.synchronize()
    f.pool.check()
    exp, _, tol, _ = f.expect(q[0], [1] * n)
    assert (np.abs(_np(outs[0]) - exp) <= tol).all()


@pytest.mark.parametrize("n", [1, 3])
def test_a_captured_plan_that_stops_to_pay(n):
    """A replay after a row was shortened to little: what is left in common is no longer worth it, and the launches that the graph
    holds attend without it (2^12 tokens, 63 x 4 x 4096 x 144 / 5e6 us = 30 saved; then 64 tokens, 0.5; the limit is 20)."""
    import torch
    f = Forked([(4096, [n + i % 5 for i in range(64)])], n_kv_heads=4, n_q_heads=4, n_pages=300, max_pages_per_seq=70)
    counts = [n] * 64
    q = f.queries(counts)
    out, plan, scratch = torch.empty_like(q), torch.empty(64, 2, dtype=torch.int32, device="cuda"), f.pool.shared_scratch(64 * n)
    cu = None if n == 1 else _cu(counts)
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        f.pool.common(plan, cu=cu)
        f.pool.shared(0, q, out, plan, scratch, cu=cu, max_new=n)
    for tokens in (4096, 64):
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        f.pool.check()
        assert plan[:, 0].tolist() == [tokens if tokens > 64 else 0] * 64
        want, _, tol, _ = f.expect(q, counts)
        assert (np.abs(_np(out) - want) <= tol).all()
        f.pool.resize(_i32([5]), _i32([100]))
        f.lens[5] = 100
        f.hk[5], f.hv[5] = f.hk[5][:100], f.hv[5][:100]


def test_tokens_of_no_row_are_left_alone():
    import torch
    f = Forked([(640, [5, 9, 13])], n_pages=40, max_pages_per_seq=14)
    for counts in ([1, 2, 1], [3, 40, 9]):
        n = sum(counts)
        q = f.queries(counts + [5])
        out, lse = torch.full_like(q, 9.0), torch.full(q.shape[:2], 9.0, device="cuda")
        plan = f.plan(counts)
        f.pool.shared(0, q, out, plan, f.pool.shared_scratch(n + 5), cu=_cu(counts), max_new=max(counts), lse=lse)
        f.pool.check()
        assert (out[n:] == 9).all() and (lse[n:] == 9).all() and torch.isfinite(out[:n]).all()


@pytest.mark.parametrize("counts", [[1, 0, 1, 1, 0], [2, 0, 3, 1, 0], [40, 0, 9, 70, 0], [0, 0, 1, 300, 0]])
def test_short_rows_that_bring_nothing(counts):
    """Rows of the group that hold less than the others have in common, and bring nothing: they do not count, and they are in
    order.  One of them is of the same beginning, one a stranger; each is at the group's front, middle and end once."""
    f = Forked([(320, [60, None, 9, 300]), (70, [30])], n_pages=60, page_size=32, max_pages_per_seq=24)
    f.bounds = [0, 5]
    f.pool.fork(_i32([0]), _i32([1]))
    f.pool.resize(_i32([1]), _i32([100]))
    f.lens[1], f.hk[1], f.hv[1] = 100, f.hk[0][:100], f.hv[0][:100]
    for rows in (None, [1, 4, 0, 3, 2], [2, 4, 0, 1, 3]):
        c = counts if rows is None else [counts[r] for r in rows]
        there = [r for r, n in enumerate(counts) if n]
        want = min([320] + [(f.lens[r] - counts[r]) // 32 * 32 for r in there])
        assert f.plan(c, rows, [0, 5])[:, 0].tolist() == [want] * 5
        f.pool.check()
        f.verify(f.queries(c), c, rows)


def test_nothing_in_common_is_attention():
    """Where the plan is empty the rows' own pages are all there is, and the launch over them has the whole card, as attention's has:
    the same shares, and so the same bits."""
    import torch
    f = Filled([2040, 2048, 1990, 2041, 2015, 2000, 2048, 1985], n_kv_heads=4, n_q_heads=16, n_pages=300, max_pages_per_seq=33)
    n = [1] * 8
    q = f.queries(n)
    want = f.attend(q, n)
    out, lse, plan = torch.empty_like(q), torch.empty_like(want[1]), torch.empty(8, 2, dtype=torch.int32, device="cuda")
    f.pool.common(plan, always=True)
    assert plan[:, 0].tolist() == [0] * 8
    f.pool.shared(0, q, out, plan, f.pool.shared_scratch(8), lse=lse)
    f.pool.check()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_few_tokens_beside_a_chunk_are_attention():
    """Rows with few new tokens beside one with many: each goes to the kernel that its number asks for, as in attention, so that with
    nothing in common the bits are attention's."""
    import torch
    f = Filled([300, 77, 150, 512, 64, 700], n_q_heads=8, n_pages=64)
    counts = [1, 2, 1, 1, 3, 500]
    q = f.queries(counts)
    want = f.attend(q, counts)
    out, lse, plan = torch.empty_like(q), torch.empty_like(want[1]), torch.empty(6, 2, dtype=torch.int32, device="cuda")
    f.pool.common(plan, cu=_cu(counts), always=True)
    f.pool.shared(0, q, out, plan, f.pool.shared_scratch(sum(counts)), cu=_cu(counts), max_new=500, lse=lse)
    f.pool.check()
    assert torch.equal(lse, want[1]) and torch.equal(out, want[0])


def test_groups_with_few_tokens_beside_one_with_many():
    """Groups of which one brings a chunk: the common pages of each by the kernel that its number of query rows asks for."""
    f = Forked([(640, [9, 30]), (256, [5, 1, 2]), (1024, [400, 20]), (320, [1, 1])], n_q_heads=8, n_pages=100, max_pages_per_seq=24)
    counts = [1, 2, 1, 1, 1, 390, 2, 1, 1]
    f.verify(f.queries(counts), counts)


def test_many_groups_with_few_tokens_beside_one_with_many():
    """The same with more groups, so that those of few have a launch over their common pages; a group without a row that brings
    anything, and one of a single row."""
    f = Forked([(256, [5, 1]), (640, [9, 30, 2]), (320, [400, 20]), (128, [1, 1]), (200, [3]), (512, [7, 1, 60]), (384, [None, 2])], n_q_heads=8,
               n_pages=120, max_pages_per_seq=24)
    counts = [1, 1, 2, 1, 1, 390, 1, 0, 0, 1, 2, 1, 3, 1, 1]
    f.verify(f.queries(counts), counts)


def test_savings_of_unlike_groups_add_up():
    """The launch over common pages costs the call once: groups that would not pay for it alone, however many groups the call has,
    are taken beside one that does.  Reading once saves, at 4 KV heads of 128, 63 x 4 x 4096 x 144 / 5e6 us = 30 for the first group,
    11 x 4 x 2048 x 144 / 5e6 = 2.6 for the second, and 0.15 for the third, which is less than a group's own place in the launch takes (1.5)."""
    f = Forked([(4096, [1 + i % 5 for i in range(64)]), (2048, [1 + i % 3 for i in range(12)]), (640, [3, 9, 1]), (640, [2])], n_kv_heads=4,
               n_q_heads=8, n_pages=400, max_pages_per_seq=70)
    f.always = False
    n = [1] * 80
    assert f.plan(n, None, f.bounds)[:, 0].tolist() == [4096] * 64 + [2048] * 12 + [0] * 4
    f.verify(f.queries(n), n)
    assert f.plan([1] * 16, list(range(64, 80)), [0, 12, 15, 16])[:, 0].tolist() == [0] * 16  # (2.6 and 0.15, of 20)
    f.pool.check()


def test_groups_of_one_row_save_nothing():
    """One pair behind 2048 tokens saves 8 x 2048 x 144 / 5e6 us = 0.5 of the 20 that the launch costs, beside 62 rows in groups of
    their own as it does alone."""
    f = Forked([(2048, [1, 2])] + [(60 + i, [1]) for i in range(62)], n_kv_heads=8, n_q_heads=8, n_pages=160, max_pages_per_seq=34)
    f.always = False
    n = [1] * 64
    assert f.plan(n, None, f.bounds)[:, 0].tolist() == [0] * 64
    f.always = True
    assert f.plan(n, None, f.bounds)[:, 0].tolist() == [2048] * 2 + [0] * 62
    f.verify(f.queries(n), n)


def test_many_small_savings_and_groups_out_of_order():
    """Twenty groups that save 1.2 us each pay for the launch together (2 x 8 x 2560 x 144 / 5e6; 23.6 in all), of which none is
    worth its place beside others; with half of them nothing is taken.  Groups out of order are reported, whatever is beside them."""
    from quantized_decode_attention_gb300 import DQError
    f = Forked([(2560, [1, 2, 3])] * 20, n_kv_heads=8, n_q_heads=8, n_pages=900, max_pages_per_seq=42)
    f.always = False
    n = [1] * 60
    assert f.plan(n, None, f.bounds)[:, 0].tolist() == [2560] * 60
    f.verify(f.queries(n), n)
    assert f.plan([1] * 30, None, f.bounds[:11])[:, 0].tolist() == [0] * 30
    f.pool.check()
    for b in ([0, 3, 2, 6], [0, 40, 61], [-1, 3, 60]):
        f.plan(n, None, b)
        with pytest.raises(DQError, match="out of range"):
            f.pool.check()


def test_a_captured_choice_among_groups():
    """The choice among groups in a graph, beside the attention that follows it: a replay after rows of the group that pays were
    shortened takes nothing, one after they are empty the same."""
    import torch
    f = Forked([(4096, [1 + i % 5 for i in range(64)]), (2048, [1 + i % 3 for i in range(12)])], n_kv_heads=4, n_q_heads=4, n_pages=400,
               max_pages_per_seq=70)
    n = [1] * 76
    q = f.queries(n)
    out, plan, scratch, b = torch.empty_like(q), torch.empty(76, 2, dtype=torch.int32, device="cuda"), f.pool.shared_scratch(76), _i32(f.bounds)
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        for _ in range(2):
            f.pool.common(plan, groups=b)
            f.pool.shared(0, q, out, plan, scratch, groups=b, max_group=64)
    for length, want in ((None, [4096] * 64 + [2048] * 12), (100, [0] * 76), (0, [0] * 76)):
        if length is not None:
            f.pool.resize(_i32(range(60)), _i32([length] * 60))
            for r in range(60):
                f.lens[r], f.hk[r], f.hv[r] = length, f.hk[r][:length], f.hv[r][:length]
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        f.pool.check()
        assert plan[:, 0].tolist() == want
        exp, _, tol, _ = f.expect(q, n)
        assert (np.abs(_np(out) - exp) <= tol).all()
