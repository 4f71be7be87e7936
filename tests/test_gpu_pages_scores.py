"""Scores by attention weight, and eviction by them, against plain numpy."""
import numpy as np
import pytest

import pages_ref as R
from test_gpu_pages import Filled, _cu, _dt, _i32, _np, _pool, _same
from test_gpu_pages_status import names

pytestmark = pytest.mark.gpu


# ---- weigh -----------------------------------------------------------------------------------------
class Weighed(Filled):
    def scores(self, cap=None, value=None):
        import torch
        cap = cap or max(self.lens) + 5
        if value is not None:
            return torch.full((len(self.lens), self.Hkv, cap), value, device="cuda")
        return torch.tensor(self.rng.random((len(self.lens), self.Hkv, cap)), dtype=torch.float32, device="cuda")

    def verify_weights(self, counts, rows=None, scale=None, amp=1.0, cap=None, lse=None):
        """The bound of a score: every weight is off by its logit's error (as attention's: 2^-18 sum|q k| and 2^-38 max|q| sum|k|
        for the product, 2^-20 for the exponential), by lse's product with log2 e (2^-23 |lse|) and by the rounding of the
        difference in log2 units (2^-23 |z - lse|, on top of z's own 2^-23 |z|); a sum of N positive terms by N 2^-24."""
        import torch
        scale = self.d ** -0.5 if scale is None else scale
        q = self.queries(counts, amp=amp)
        if lse is None:
            _, lse = self.attend(q, counts, rows, None, scale)
        s = self.scores(cap)
        before = _np(s)
        one = all(n == 1 for n in counts)
        self.pool.weigh(self.layer, q, lse, s, rows=None if rows is None else _i32(rows), cu=None if one else _cu(counts),
                        max_new=max(counts), sm_scale=scale)
        self.pool.check()
        want, tol = before.copy(), np.zeros(before.shape)
        at = 0
        qn, ln = _np(q), _np(lse)
        for i, n in enumerate(counts):
            r = i if rows is None else rows[i]
            L = 0 if r < 0 else self.lens[r]
            for h in range(self.Hkv if L and n else 0):
                k = self.hk[r][:, h]
                got, err = np.zeros(L), np.zeros(L)
                for g in range(self.G):
                    x, l = qn[at:at + n, h * self.G + g], ln[at:at + n, h * self.G + g]
                    seen = (np.arange(L)[None, :] <= (L - n + np.arange(n))[:, None]) & np.isfinite(l)[:, None]
                    l = np.where(np.isfinite(l), l, 0)[:, None]
                    z = x @ k.T * scale
                    w = np.where(seen, np.exp(np.where(seen, z - l, 0)), 0)
                    d = abs(scale) * (2.0 ** -18 * (np.abs(x) @ np.abs(k).T) + 2.0 ** -38 * np.abs(x).max(1)[:, None] * np.abs(k).sum(1)[None, :])
                    got += w.sum(0)
                    err += (w * (d + 2.0 ** -20 + 2.0 ** -23 * (np.abs(l) + np.abs(z - l) + np.abs(z)))).sum(0)
                old = np.where(np.arange(L) < L - n, before[r, h, :L], 0)
                want[r, h, :L] = old + got
                tol[r, h, :L] = err + got * (n * self.G + 2) * 2.0 ** -24 + (old + got) * 2.0 ** -24
            at += n
        err = np.abs(_np(s) - want)
        assert (err <= tol).all(), (float((err - tol).max()), float(err.max()))


@pytest.mark.parametrize("d, G, P, dtype", [(128, 4, 64, "bf16"), (64, 1, 16, "f16"), (128, 8, 32, "f16"), (64, 5, 128, "bf16"),
                                            (128, 16, 128, "bf16"), (64, 16, 16, "f16"), (128, 1, 16, "bf16"), (128, 3, 64, "f16")])
def test_weights_of_single_tokens(d, G, P, dtype):
    """Lengths from nothing to many pages, ends inside tiles and pages, padding and permuted rows, an odd capacity."""
    lens = [1, 0, 15, 16, 17, P - 1, P, P + 1, 5 * P + 7, 129, 300]
    f = Weighed(lens, seed=d + G, n_kv_heads=2, n_q_heads=2 * G, head_dim=d, page_size=P, dtype=dtype, n_pages=100, max_pages_per_seq=24)
    f.verify_weights([1] * 11, [3, 8, -1, 0, 10, 1, 7, 2, 9, 4, 6], cap=5 * P + 301)
    f.verify_weights([1] * len(lens), scale=0.3, amp=2.0)


@pytest.mark.parametrize("d, G, P, dtype", [(128, 4, 64, "bf16"), (64, 2, 16, "f16"), (128, 8, 128, "f16"), (128, 1, 32, "bf16"),
                                            (64, 7, 64, "bf16"), (128, 16, 16, "f16")])
def test_weights_of_several_tokens(d, G, P, dtype):
    """Ragged new tokens, causal at the end; rows with none, and a row with more queries than it has tokens."""
    lens = [200, 3, 64, 130, 0, 77, 257]
    f = Weighed(lens, seed=G, n_kv_heads=2, n_q_heads=2 * G, head_dim=d, page_size=P, dtype=dtype, n_pages=100, max_pages_per_seq=24)
    f.verify_weights([5, 3, 64, 0, 2, 80, 131])
    f.verify_weights([2, 1, 3, 1, 1, 2, 4], amp=2.0)
    f.verify_weights([200, 3, 64, 130, 1, 77, 257], scale=-0.05)
    f.verify_weights([33, 0, 0, 40], [6, 0, 1, 3])
    f.verify_weights([1, 2, 0, 1, 0, 1, max(60, 48 // G + 1)])  # G 1 and 2: few on average, with a launch of their own


def test_weights_of_long_rows():
    f = Weighed([2600, 1500], n_pages=80, max_pages_per_seq=45)
    for counts in ([1, 1], [7, 8], [60, 64], [300, 17]):
        f.verify_weights(counts)


def test_weights_of_very_many_rows():
    rng = np.random.default_rng(8)
    lens = [int(x) for x in rng.integers(0, 90, 700)]
    f = Weighed(lens, n_pages=2200, max_pages_per_seq=6, page_size=32, n_kv_heads=1, n_q_heads=2, head_dim=64)
    for most in (2, 4, 60):
        f.verify_weights([int(x) for x in rng.integers(0, most, 700)])


@pytest.mark.parametrize("dtype, amp", [("bf16", 2.0 ** 40), ("bf16", 2.0 ** -60), ("f16", 2.0 ** 13)])
def test_weights_of_very_large_and_very_small_queries(dtype, amp):
    f = Weighed([70, 200], dtype=dtype)
    f.verify_weights([1, 1], amp=amp, scale=0.1 / amp)
    f.verify_weights([20, 19], amp=amp, scale=0.1 / amp)


@pytest.mark.parametrize("n", [1, 30])
def test_queries_that_see_nothing_add_nothing(n):
    """lse of -inf, as attention gives it to them."""
    import torch
    f = Weighed([50, 70])
    f.verify_weights([n, n], lse=torch.full((2 * n, 8), -float("inf"), device="cuda"))


@pytest.mark.parametrize("n", [1, 70])
def test_a_row_too_long_or_named_twice_is_left_alone(n):
    import torch
    f = Weighed([100, 90, 110], n_pages=20)
    q = f.queries([n] * 3)
    _, lse = f.attend(q, [n] * 3)
    for cap, rows, done in ((95, [0, 1, 2], [1]), (120, [0, 2, 0], [2]), (120, [1, 1, 1], [])):
        s = f.scores(cap)
        before = s.clone()
        f.pool.weigh(0, q, lse, s, rows=_i32(rows), cu=_cu([n] * 3), max_new=n)
        assert names(f.pool) == ["DQ_EINVAL"]
        for r in range(3):
            assert torch.equal(s[r], before[r]) != (r in done)
    with pytest.raises(ValueError):
        f.pool.weigh(0, q, lse, s[:2])
    with pytest.raises(ValueError):
        f.pool.weigh(0, q, lse.half(), s)
    with pytest.raises(ValueError):
        f.pool.weigh(0, q, lse, s.transpose(0, 1))


def test_weights_beyond_four_gigabytes_of_scores():
    """Scores of a row that lie past 2^32 bytes."""
    import torch
    f = Weighed([5, 40], n_kv_heads=2, max_pages_per_seq=12)
    cap = 1 << 22
    p = _pool(max_seqs=140, n_pages=8, max_pages_per_seq=4)
    p.resize(_i32([139]), _i32([40]))
    k = f.k[1].cuda()
    p.append(0, k, f.v[1].cuda(), rows=_i32([139]), cu=_i32([0, 40]), max_new=40)
    s = torch.zeros(140, 2, cap, device="cuda")
    small = f.scores(value=0.0)
    for n in (1, 40):
        q = f.queries([n])
        out, lse = torch.empty_like(q), torch.empty(n, 8, device="cuda")
        cu = _i32([0, n])
        f.pool.attention(0, q, out, rows=_i32([1]), cu=cu, max_new=n, lse=lse)
        f.pool.weigh(0, q, lse, small, rows=_i32([1]), cu=cu, max_new=n)
        p.weigh(0, q, lse, s, rows=_i32([139]), cu=cu, max_new=n)
        f.pool.check()
        p.check()
        assert torch.equal(s[139, :, :45], small[1]) and float(small[1].sum()) > 1


def test_weights_are_the_same_every_time():
    import torch
    f = Weighed([1000, 700, 1], n_pages=64, max_pages_per_seq=20)
    for counts in ([1, 1, 1], [130, 60, 1]):
        q = f.queries(counts)
        _, lse = f.attend(q, counts)
        got = []
        for _ in range(3):
            s = f.scores(value=0.0)
            f.pool.weigh(0, q, lse, s, cu=_cu(counts), max_new=max(counts))
            got.append(s)
        assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


# ---- evict -----------------------------------------------------------------------------------------
def chosen(score, n, keep, first, last):
    """Positions that stay, ascending."""
    if keep == n:
        return list(range(n))
    fixed = [j for j in range(n) if j < first or j >= n - last]
    rest = [j for j in range(n) if first <= j < n - last]
    key = lambda j: (-(-np.inf if np.isnan(score[j]) else score[j]), np.isnan(score[j]), j)
    return sorted(fixed + sorted(rest, key=key)[:keep - len(fixed)])


class Pool2:
    """A pool of L layers whose first rows hold random tokens, all its bytes in numpy."""

    def __init__(self, lens, more, L=2, H=2, d=128, P=64, seed=0, n_pages=120, M=24, cap=None, dtype="bf16", k_exp=0):
        import torch
        self.rng = np.random.default_rng(seed)
        self.lens, self.L, self.H, self.d, self.P, self.N = lens, L, H, d, P, n_pages
        R_ = len(lens) + more
        self.pool = _pool(n_layers=L, n_pages=n_pages, page_size=P, n_kv_heads=H, n_q_heads=H, head_dim=d, max_seqs=R_, max_pages_per_seq=M,
                          dtype=dtype, k_exp=k_exp)
        self.m = R.Model(n_pages, P, R_, M)
        gen = torch.Generator("cuda").manual_seed(seed)
        for n in ("pages", "summary"):
            self.pool.tensors[n].random_(0, 256, generator=gen)
        self.resize(range(len(lens)), lens)
        self.codes = []  # [layer][row]: codes and scales of keys and values, held keys in units of 2^k_exp
        for layer in range(L):
            n = sum(lens)
            k, v = (torch.tensor(self.rng.normal(size=(n, H, d)) * np.exp(self.rng.normal(size=(n, 1, 1)))).to(_dt(dtype)) for _ in range(2))
            if n:
                self.pool.append(layer, k.cuda(), v.cuda(), rows=_i32(range(len(lens))), cu=_cu(lens), max_new=max(lens))
            at, rows = 0, []
            for x in lens:
                kc, ks, kh = R.quantise(_np(k[at:at + x]), k_exp)
                vc, vs, _ = R.quantise(_np(v[at:at + x]), 0)
                rows.append((kc, ks, vc, vs, kh * 2.0 ** -k_exp))
                at += x
            self.codes.append(rows)
        self.pool.check()
        self.cap = cap or max(lens) + 3
        self.scores = torch.tensor(np.round(self.rng.normal(size=(L, R_, H, self.cap)), 2), dtype=torch.float32, device="cuda")  # (many are equal)

    def resize(self, rows, lens):
        assert self.m.resize(list(rows), list(lens))
        self.pool.resize(_i32(rows), _i32(lens))

    def image(self):
        t = self.pool.tensors
        return (t["pages"].cpu().numpy().reshape(self.L, self.N, self.H, -1).copy(),
                t["summary"].cpu().numpy().reshape(self.L, self.N, self.H, -1).copy(), self.scores.cpu().numpy().copy())

    def verify(self, src, dst, first, last, done=None):
        """Every byte of the pool, every summary and every score after evict(); `done`: the pairs that are carried out."""
        pages, sums, scores = self.image()
        self.pool.evict(self.scores, _i32(src), _i32(dst), keep_first=first, keep_last=last)
        for i, (s, t) in enumerate(zip(src, dst)):
            if s < 0 or t < 0 or (done is not None and i not in done):
                continue
            n, keep = self.lens[s], self.m.length[t]
            for layer in range(self.L):
                kc, ks, vc, vs, held = self.codes[layer][s]
                for h in range(self.H):
                    pick = chosen(scores[layer, s, h], n, keep, first, last)
                    scores[layer, t, h, :keep] = scores[layer, s, h, pick]
                    for u, j in enumerate(pick):
                        R.put_token(pages[layer, self.m.table[t][u // self.P], h], self.P, self.d, u % self.P, kc[j, h], ks[j, h], vc[j, h], vs[j, h])
                    for o, page in enumerate(self.m.table[t]):
                        hi, lo, e = R.summary(held[pick[o * self.P:(o + 1) * self.P], h])
                        b = sums[layer, page, h]
                        b[:self.d], b[self.d:2 * self.d] = hi.view(np.uint8), lo.view(np.uint8)
                        b[2 * self.d:2 * self.d + 4] = np.array([e], dtype=np.int32).view(np.uint8)
        got = self.image()
        assert (got[0] == pages).all() and (got[1] == sums).all() and np.array_equal(got[2], scores, equal_nan=True)
        _same(self.pool, self.m)


@pytest.mark.parametrize("d, P, first, last", [(128, 64, 4, 16), (64, 16, 0, 0), (128, 16, 1, 7), (64, 128, 3, 40), (128, 32, 0, 9), (128, 128, 5, 0),
                                               (64, 32, 0, 1)])
def test_evict_keeps_the_highest_scores(d, P, first, last):
    """Ragged rows to a few, some, all but one and all of their tokens, to nothing, through permuted lists with padding."""
    lens = [3 * P + 5, 200, 1, 0, 2 * P, 77, 300]
    f = Pool2(lens, 9, d=d, P=P, seed=P + d, n_pages=200, k_exp=2 if d == 64 else 0)
    keep = [max(first + last, P + 3), 199, 1, 0, max(first + last, 2 * P - 9), 77, max(first + last, 41)]
    src, dst = [6, 0, 3, -1, 2, 1, 5, 4, 0], [8, 7, 15, 9, 10, 11, 12, 13, -2]
    pairs = [(s, t) for s, t in zip(src, dst) if s >= 0 and t >= 0]
    f.resize([t for _, t in pairs], [keep[s] for s, _ in pairs])
    f.verify(src, dst, first, last)
    f.pool.check()


def test_evict_of_equal_and_odd_scores():
    """All equal, NaN, infinities, both zeros, subnormal and negative ones."""
    import torch
    f = Pool2([500] * 6, 6, L=1, n_pages=200, seed=3)
    s = f.scores
    s[0, 0] = 1.0
    s[0, 1, :, ::3] = float("nan")
    s[0, 2, :, ::2] = -float("inf")
    s[0, 2, :, 5::7] = float("inf")
    s[0, 3] = 0.0
    s[0, 3, :, ::2] = -0.0
    s[0, 4] *= 1e-40
    s[0, 5] = float("nan")
    f.resize(range(6, 12), [100, 400, 260, 77, 130, 40])
    f.verify(list(range(6)), list(range(6, 12)), 2, 3)
    f.pool.check()


def test_evict_of_long_rows():
    f = Pool2([9000, 4100], 2, L=1, H=1, d=64, P=16, n_pages=1400, M=600, seed=5)
    f.resize([2, 3], [2500, 4099])
    f.verify([0, 1], [2, 3], 4, 64)
    f.pool.check()


def test_evict_of_rows_that_share_pages():
    """Sources that hold the same pages, one source for two rows; a destination that another row holds too is not written."""
    f = Pool2([300], 6, seed=7)
    f.m.fork([0], [1])
    f.pool.fork(_i32([0]), _i32([1]))
    f.lens.append(300)
    for c in f.codes:
        c.append(c[0])
    f.resize([2, 3, 4], [100, 200, 64])
    f.verify([1, 0, 1], [2, 3, 4], 1, 5)
    f.pool.check()
    f.m.fork([2], [5])
    f.pool.fork(_i32([2]), _i32([5]))
    f.pool.check()
    pages, sums, _ = f.image()
    f.pool.evict(f.scores, _i32([0]), _i32([5]))
    assert names(f.pool) == ["DQ_EINVAL"]
    got = f.image()
    assert (got[0] == pages).all() and (got[1] == sums).all()


def test_evict_refuses_on_the_device():
    """More tokens than there are, rows out of range, named twice, source and destination at once, fewer than are kept anyway, a
    row longer than the scores: nothing is written for the pair, the others are carried out."""
    f = Pool2([300, 200, 120], 5, n_pages=60, cap=250, seed=9)
    f.resize([3, 4, 5, 6], [100, 90, 130, 20])
    for src, dst, first, last, done in (([1, 2], [3, 5], 0, 0, [0]), ([8, 1], [4, 3], 0, 0, [1]), ([1, 2], [3, 99], 0, 0, [0]),
                                        ([1, 2, 1], [3, 4, 3], 0, 0, [1]), ([1, 4], [4, 3], 0, 0, []), ([1, 1], [6, 3], 15, 6, [1]),
                                        ([0, 2], [3, 4], 0, 0, [1]), ([1, 1], [1, 4], 0, 0, [1])):
        if done == []:
            before = f.image()
            f.pool.evict(f.scores, _i32(src), _i32(dst), keep_first=first, keep_last=last)

            got = f.image()
            assert all(np.array_equal(a, b) for a, b in zip(before, got))
        else:
            f.verify(src, dst, first, last, done)
        assert names(f.pool) == ["DQ_EINVAL"], (src, dst)
    for call in (lambda: f.pool.evict(f.scores[0], _i32([1]), _i32([3])), lambda: f.pool.evict(f.scores, _i32([1]), _i32([3, 4])),
                 lambda: f.pool.evict(f.scores.double(), _i32([1]), _i32([3])), lambda: f.pool.evict(f.scores[:, :4], _i32([1]), _i32([3]))):
        with pytest.raises(ValueError):
            call()


# ---- together --------------------------------------------------------------------------------------------
@pytest.mark.parametrize("captured", [False, True])
def test_a_conversation_at_a_budget(captured):
    """A prompt, decode steps of two layers that weigh what they attend to (called, or captured once and replayed), and an
    eviction into a second row and back whenever the budget is passed; the kept tokens are followed in numpy."""
    import torch
    P, H, G, d, L, budget, most = 16, 2, 4, 128, 2, 40, 48
    pool = _pool(page_size=P, n_pages=40, n_layers=L, n_kv_heads=H, n_q_heads=H * G, head_dim=d, max_seqs=4, max_pages_per_seq=5)
    rng = np.random.default_rng(3)
    rnd = lambda *s: torch.tensor(rng.normal(size=s)).to(torch.bfloat16).cuda()
    held = [[[np.zeros((0, d)), np.zeros((0, d))] for _ in range(H)] for _ in range(L)]  # [layer][head]: keys, values in order
    weight = [[np.zeros(0) for _ in range(H)] for _ in range(L)]
    scores = torch.full((L, 4, H, most + 3), 7.0, device="cuda")

    def add(layer, k, v):
        for h in range(H):
            for x, y in ((0, k), (1, v)):
                held[layer][h][x] = np.concatenate([held[layer][h][x], R.quantise(_np(y[:, h]), 0)[2]])

    def follow(layer, q, out, n):
        x = _np(q)
        for h in range(H):
            k, v = held[layer][h]
            seen = np.arange(len(k))[None, :] <= (len(k) - n + np.arange(n))[:, None]
            w = np.zeros(len(k))
            for g in range(G):
                y = x[:, h * G + g]
                o, l = R.attend(y, k, v, seen, d ** -0.5)
                assert np.abs(_np(out[:, h * G + g]) - o).max() <= 2.0 ** -8 * np.abs(o).max() + 2.0 ** -9 * np.abs(v).max()
                w += np.where(seen, np.exp(y @ k.T * d ** -0.5 - l[:, None]), 0).sum(0)
            weight[layer][h] = np.concatenate([weight[layer][h], np.zeros(n)]) + w

    row, spare, n = 1, 3, 30
    q, k, v = ([rnd(n, x, d) for _ in range(L)] for x in (H * G, H, H))
    pool.resize(_i32([row]), _i32([n]))
    cu = _i32([0, n])
    for layer in range(L):
        pool.append(layer, k[layer], v[layer], rows=_i32([row]), cu=cu, max_new=n)
        out, lse = torch.empty_like(q[layer]), torch.empty(n, H * G, device="cuda")
        pool.attention(layer, q[layer], out, rows=_i32([row]), cu=cu, max_new=n, lse=lse)
        pool.weigh(layer, q[layer], lse, scores[layer], rows=_i32([row]), cu=cu, max_new=n)
        add(layer, k[layer], v[layer])
        follow(layer, q[layer], out, n)
    rt, lens = _i32([row]), _i32([0])
    q1, k1, v1 = ([torch.zeros(1, x, d, dtype=torch.bfloat16, device="cuda") for _ in range(L)] for x in (H * G, H, H))
    out1, lse1 = [torch.zeros_like(x) for x in q1], [torch.zeros(1, H * G, device="cuda") for _ in range(L)]

    def step():
        pool.resize(rt, lens)
        for layer in range(L):
            pool.append(layer, k1[layer], v1[layer], rows=rt)
            pool.attention(layer, q1[layer], out1[layer], rows=rt, lse=lse1[layer])
            pool.weigh(layer, q1[layer], lse1[layer], scores[layer], rows=rt)

    graph, evictions = None, 0
    for t in range(40):
        n += 1
        rt.fill_(row)
        lens.fill_(n)
        for layer in range(L):
            for x in (q1[layer], k1[layer], v1[layer]):
                x.copy_(rnd(*x.shape))
        if captured and t == 1:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        if graph is not None:
            graph.replay()
        else:
            step()
        pool.check()
        for layer in range(L):
            add(layer, k1[layer], v1[layer])
            follow(layer, q1[layer], out1[layer], 1)
            for h in range(H):
                got = _np(scores[layer, row, h, :n])
                assert np.abs(got - weight[layer][h]).max() <= 1e-5 * weight[layer][h].max()
        if n < most:
            continue
        evictions += 1
        pool.resize(_i32([spare]), _i32([budget]))
        pool.evict(scores, _i32([row]), _i32([spare]), keep_first=2, keep_last=8)
        pool.resize(_i32([row]), _i32([0]))
        pool.check()
        for layer in range(L):
            for h in range(H):
                pick = chosen(_np(scores[layer, row, h, :n]), n, budget, 2, 8)
                weight[layer][h] = weight[layer][h][pick]
                held[layer][h] = [x[pick] for x in held[layer][h]]
        row, spare, n = spare, row, budget
        assert int(pool.tensors["refs"].sum()) == -(-budget // P)
    assert evictions == 3


def test_weigh_evict_and_select_on_other_streams():
    """Calls on a stream of their own, ordered by events; the evicted row's summaries serve select."""
    import torch
    f = Pool2([600], 1, L=1, P=16, M=40, n_pages=80, seed=1)
    p, s = f.pool, torch.cuda.Stream()
    f.resize([1], [200])
    torch.cuda.synchronize()
    q = torch.randn(1, 2, 128, device="cuda").to(torch.bfloat16)
    out, lse = torch.empty_like(q), torch.empty(1, 2, device="cuda")
    sel = torch.empty(1, 2, 4, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    p.attention(0, q, out, rows=_i32([0]), lse=lse, stream=s)
    p.weigh(0, q, lse, f.scores[0], rows=_i32([0]), stream=s)
    s.synchronize()
    scores = f.scores.cpu().numpy()
    p.evict(f.scores, _i32([0]), _i32([1]), keep_first=1, keep_last=1, stream=s)
    p.select(0, q, sel, rows=_i32([1]), stream=s)
    p.check(s)
    for h in range(2):
        pick = chosen(scores[0, 0, h], 600, 200, 1, 1)
        held = f.codes[0][0][4][pick, h]
        sums = [R.summary(held[j * 16:(j + 1) * 16]) for j in range(13)]
        assert sel[0, h].tolist() == R.choose(_np(q[0, h:h + 1]), sums, 13, 4, 1, 1)


def test_weights_of_single_tokens_beside_a_chunk():
    """One row brings a chunk and the others a token: theirs are weighed by the kernel for few, every score by one thread in an order
    of its own, and so with the bits of a call without the chunk."""
    import torch
    f = Weighed([300 - 7 * i for i in range(16)] + [300], n_pages=100)
    counts = [1] * 16 + [200]
    f.verify_weights(counts)
    q = f.queries(counts)
    _, lse = f.attend(q, counts)
    a, b = f.scores(value=0.5), f.scores(value=0.5)
    f.pool.weigh(0, q, lse, a, cu=_cu(counts), max_new=200)
    f.pool.weigh(0, q[:16], lse[:16].contiguous(), b)
    f.pool.check()
    assert torch.equal(a[:16], b[:16])


def test_a_destination_that_another_row_holds_is_reported_as_such():
    from quantized_decode_attention_gb300 import DQError
    f = Pool2([100], 3, seed=3)
    f.resize([1], [64])
    f.pool.fork(_i32([1]), _i32([2]))
    f.pool.check()
    f.pool.evict(f.scores, _i32([0]), _i32([2]))
    with pytest.raises(DQError, match="eviction met a page that several rows hold"):
        f.pool.check()
    f.pool.check()
