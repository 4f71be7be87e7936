"""The paged 4-bit cache on the GPU against plain numpy in 64 bits (pages_ref)."""
import math

import numpy as np
import pytest

import pages_ref as R

pytestmark = pytest.mark.gpu


def _pool(**kw):
    from quantized_decode_attention_gb300 import PagePool, make_pages_config
    a = dict(n_layers=1, n_pages=64, page_size=64, n_kv_heads=2, n_q_heads=8, head_dim=128, max_seqs=8, max_pages_per_seq=12)
    a.update(kw)
    return PagePool.allocate(make_pages_config(**a))


def _dt(name):
    import torch
    return {"bf16": torch.bfloat16, "f16": torch.float16}[name]


def _i32(x):
    import torch
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def _np(t):
    return t.detach().cpu().double().numpy()


def _cu(counts):
    return _i32(np.concatenate([[0], np.cumsum(counts)]))


class Filled:
    """A pool whose rows hold random tokens, and the same in numpy: k[r], v[r] [len, Hkv, d] as held."""

    def __init__(self, lens, seed=0, layer=0, wide=True, dtype="bf16", step=None, **kw):
        import torch
        self.dtype = dtype
        self.pool = _pool(dtype=dtype, max_seqs=len(lens), **kw)
        c = self.pool.cfg
        self.layer, self.lens, self.rng = layer, list(lens), np.random.default_rng(seed)
        self.Hkv, self.G, self.d, self.P = c.n_kv_heads, c.n_q_heads // c.n_kv_heads, c.head_dim, c.page_size
        mean = self.rng.normal(size=(self.Hkv, self.d)) * 1.4
        amp = np.where(self.rng.random((self.Hkv, self.d)) < 0.03, 10.0, 1.0) if wide else 1.0
        self.k, self.v = [], []
        for n in lens:
            k = torch.tensor((self.rng.normal(size=(n, self.Hkv, self.d)) + mean) * amp).to(_dt(dtype))
            v = torch.tensor(self.rng.normal(size=(n, self.Hkv, self.d))).to(_dt(dtype))
            self.k.append(k)
            self.v.append(v)
        self.pool.tensors["pages"].fill_(0xFF)  # scales of tokens that are not there are NaN
        self.pool.resize(None, _i32(lens))
        if sum(lens):
            self.pool.append(layer, torch.cat(self.k).cuda(), torch.cat(self.v).cuda(), cu=_cu(lens), max_new=max(lens))
        self.pool.check()
        self.hk = [R.quantise(_np(x), c.k_exp)[2] for x in self.k]
        self.hv = [R.quantise(_np(x), c.v_exp)[2] for x in self.v]

    def queries(self, counts, amp=1.0):
        import torch
        return torch.tensor(self.rng.normal(size=(sum(counts), self.Hkv * self.G, self.d)) * amp).to(_dt(self.dtype)).cuda()

    def expect(self, q, counts, rows=None, chosen=None, scale=None):
        """out, lse in 64 bits, and a bound on the error of each output.

        The bound: the stored output is rounded once (eps / 2 of its type, plus half of
        the smallest fp16 step); a weight is rounded to 11 bits (2^-11 of it); a logit is
        off by delta, which moves weights by delta and, through their sum, the result by
        twice that: delta = 2^-18 sum|q k| (fp32 sums of d products, truncated) plus
        2^-38 max|q| sum|k| (queries scaled to binary16) plus 2^-20 (the exponential)."""
        import torch
        scale = self.d ** -0.5 if scale is None else scale
        q = _np(q)
        out, lse, tol, ltol = np.zeros(q.shape), np.full(q.shape[:2], -np.inf), np.zeros(q.shape), np.zeros(q.shape[:2])
        eps = torch.finfo(_dt(self.dtype)).eps / 2
        at = 0
        for i, n in enumerate(counts):
            r = i if rows is None else rows[i]
            L = 0 if r < 0 else self.lens[r]
            for h in range(self.Hkv * self.G if L else 0):
                hk = h // self.G
                k, v = self.hk[r][:, hk], self.hv[r][:, hk]
                seen = np.arange(L)[None, :] <= (L - n + np.arange(n))[:, None]
                if chosen is not None:
                    seen = seen & np.isin(np.arange(L) // self.P, chosen[i][hk])[None, :]
                qq = q[at:at + n, h]
                o, l = R.attend(qq, k, v, seen, scale)
                a, _ = R.attend(qq, k, np.abs(v), seen, scale)
                big = np.where(seen, np.abs(qq) @ np.abs(k).T, 0).max(1)
                wide = np.where(seen, np.abs(k).sum(1)[None, :], 0).max(1) * np.abs(qq).max(1)
                delta = abs(scale) * (2.0 ** -18 * big + 2.0 ** -38 * wide) + 2.0 ** -20
                out[at:at + n, h], lse[at:at + n, h] = o, l
                tol[at:at + n, h] = eps * np.abs(o) + (2.0 ** -11 + 2 * delta[:, None]) * a + 2.0 ** -25
                ltol[at:at + n, h] = 2 * delta + 2.0 ** -22 * np.abs(np.where(np.isfinite(l), l, 0))
            at += n
        return out, lse, tol, ltol

    def attend(self, q, counts, rows=None, sel=None, scale=None, stream=None, pool=None):
        import torch
        out = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
        lse = torch.full(q.shape[:2], float("nan"), device="cuda")
        one = all(n == 1 for n in counts)
        (pool or self.pool).attention(self.layer, q, out, rows=None if rows is None else _i32(rows), cu=None if one else _cu(counts),
                                      max_new=max(counts), lse=lse, sel=sel, sm_scale=scale, stream=stream)
        return out, lse

    def verify(self, q, counts, rows=None, chosen=None, scale=None, sel=None):
        out, lse = self.attend(q, counts, rows, sel, scale)
        self.pool.check()
        want, wl, tol, ltol = self.expect(q, counts, rows, chosen, scale)
        err = np.abs(_np(out) - want)
        assert (err <= tol).all(), (float((err - tol).max()), float(err.max()))
        gl = _np(lse)
        assert (np.isneginf(gl) == np.isneginf(wl)).all()
        fin = np.isfinite(wl)
        assert (np.abs(gl[fin] - wl[fin]) <= ltol[fin]).all(), float((np.abs(gl[fin] - wl[fin]) - ltol[fin]).max())


# ---- quantise and read back ----------------------------------------------------------------------
@pytest.mark.parametrize("d, P, dtype, k_exp, v_exp", [
    (128, 64, "bf16", 0, 0), (64, 16, "f16", 0, -3), (128, 128, "f16", 2, 0), (64, 32, "bf16", -5, 4), (128, 16, "bf16", 0, 0),
    (64, 128, "bf16", 0, 0), (128, 32, "f16", 0, 0)])
def test_append_writes_the_formula_bit_for_bit(d, P, dtype, k_exp, v_exp):
    """Three appends of ragged lengths (none, one, across pages) to permuted rows: every byte of every page, those of
    tokens that are not there left as they were, every summary, and the read back."""
    import torch
    rng = np.random.default_rng(P + d)
    R_, M, N, H = 5, 6, 40, 2
    pool = _pool(page_size=P, head_dim=d, n_pages=N, n_kv_heads=H, n_q_heads=H, max_seqs=R_, max_pages_per_seq=M, dtype=dtype,
                 k_exp=k_exp, v_exp=v_exp, n_layers=2)
    m = R.Model(N, P, R_, M)
    pool.tensors["pages"].random_(0, 256, generator=torch.Generator("cuda").manual_seed(3))
    img = pool.tensors["pages"].cpu().numpy().reshape(2, N, H, -1).copy()
    held = [np.zeros((0, H, d)) for _ in range(R_)]
    sums = {}
    for counts in ([1, P + 3, 0, 2 * P, 5], [1, 1, 3, 1, P], [P, 0, 1, 2, 1]):
        rows = list(rng.permutation(R_))
        new = [counts[r] for r in rows]
        lens = [m.length[r] + counts[r] for r in rows]
        assert m.resize(rows, lens)
        pool.resize(_i32(rows), _i32(lens))
        n = sum(new)
        # strided views of a wider projection, a zero block, a block of zeros and signs, large and tiny blocks
        wide = torch.tensor(rng.normal(size=(n, 3 * H * d + 8)) * np.exp(rng.normal(size=(n, 1)) * 2)).to(_dt(dtype)).cuda()
        k, v = wide[:, 8:8 + H * d].view(n, H, d), wide[:, 8 + 2 * H * d:].view(n, H, d)
        k[0, 0, :16] = 0.0
        v[0, 1, 16:32] = -0.0
        v[n - 1, 0, :16] *= 3e-5
        k[n - 1, 1, 16:32] = 3000.0 if k_exp <= 0 else 60000.0
        pool.append(1, k, v, rows=_i32(rows), cu=_cu(new), max_new=max(new))
        ko, vo = torch.empty(n, H, d, dtype=_dt(dtype), device="cuda"), torch.empty(n, H, d, dtype=_dt(dtype), device="cuda")
        pool.read(1, ko, vo, rows=_i32(rows), cu=_cu(new), max_new=max(new))
        pool.check()
        kc, ks, kh = R.quantise(_np(k), k_exp)
        vc, vs, vh = R.quantise(_np(v), v_exp)
        assert torch.equal(ko.cpu(), torch.tensor(kh).to(_dt(dtype))) and torch.equal(vo.cpu(), torch.tensor(vh).to(_dt(dtype)))
        at = 0
        for r, c, L in zip(rows, new, lens):
            held[r] = np.concatenate([held[r], kh[at:at + c]])
            for i in range(c):
                t = L - c + i
                for h in range(H):
                    R.put_token(img[1, m.table[r][t // P], h], P, d, t % P, kc[at + i, h], ks[at + i, h], vc[at + i, h], vs[at + i, h])
            for j in range((L - c) // P, m.pages(L)) if c else []:
                for h in range(H):
                    sums[m.table[r][j], h] = R.summary(held[r][j * P:(j + 1) * P, h] * 2.0 ** -k_exp)
            at += c
        assert (pool.tensors["pages"].cpu().numpy().reshape(img.shape) == img).all()
    got = pool.tensors["summary"].cpu().numpy().reshape(2, N, H, 2 * d + 16)
    for (p, h), (hi, lo, e) in sums.items():
        s = got[1, p, h]
        assert (s[:d].view(np.int8) == hi).all() and (s[d:2 * d].view(np.int8) == lo).all() and s[2 * d:2 * d + 4].view(np.int32)[0] == e
    assert (got[0] == 0).all() and (got[1, [p for p in range(N) if (p, 0) not in sums]] == 0).all()


def test_ties_and_borders_of_the_rounding():
    """Every border between two codes and its neighbours, and scales on the borders of e4m3."""
    import torch
    rows = []
    for s in (1.0, 1.125, 1.875, 0.0625, 2.0 ** -9, 448.0):
        base = [6.0 * s]
        for b in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
            base += [b * s, -b * s]
        rows.append(base + [0.0])
        f = torch.tensor(base + [0.0], dtype=torch.bfloat16).double()
        for up in (1, -1):
            w = (f.to(torch.bfloat16).view(torch.int16) + up).view(torch.bfloat16).double()
            w[0] = 6.0 * s
            w[-1] = 0.0
            rows.append(w.tolist())
    for top in (6 * 1.0625, 6 * 1.1875, 6 * 17.0, 6 * 2.0 ** -10, 6 * 1.5 * 2.0 ** -9, 6 * 2.5 * 2.0 ** -9, 2784.0, 3e38, 1e-30):
        rows.append([top, -top / 2] + [top / 3] * 14)
    n = len(rows)
    x = torch.tensor(rows, dtype=torch.float64).to(torch.bfloat16).repeat(1, 4).view(n, 1, 64).cuda()
    pool = _pool(head_dim=64, n_kv_heads=1, n_q_heads=1, max_seqs=1)
    pool.resize(None, _i32([n]))
    pool.append(0, x, -x, cu=_i32([0, n]), max_new=n)
    ko, vo = torch.empty_like(x), torch.empty_like(x)
    pool.read(0, ko, vo, cu=_i32([0, n]), max_new=n)
    pool.check()
    want = R.quantise(_np(x), 0)[2]
    assert (_np(ko) == want).all() and (_np(vo) == -want).all()


def test_append_latches_what_is_not_finite_and_what_is_shared():
    import torch
    from quantized_decode_attention_gb300 import DQError
    f = Filled([40, 0, 0], page_size=64)
    for bad in (float("nan"), float("inf")):
        f.pool.resize(_i32([1]), _i32([3]))
        x = torch.ones(3, 2, 128, dtype=torch.bfloat16, device="cuda")
        x[1, 1, 5] = bad
        f.pool.append(0, torch.ones_like(x), x, rows=_i32([1]), cu=_i32([0, 3]), max_new=3)
        with pytest.raises(DQError, match="DQ_ENONFINITE"):
            f.pool.check()
        out = torch.empty(1, 8, 128, dtype=torch.bfloat16, device="cuda")
        f.pool.attention(0, torch.ones_like(out), out, rows=_i32([1]))
        f.pool.check()
        assert torch.isfinite(out).all()
    before = f.pool.tensors["pages"].clone()
    f.pool.fork(_i32([0]), _i32([2]))
    x = torch.ones(1, 2, 128, dtype=torch.bfloat16, device="cuda")
    f.pool.append(0, x, x, rows=_i32([2]))  # position 39 of a page that rows 0 and 2 hold
    with pytest.raises(DQError, match="several rows"):
        f.pool.check()
    assert torch.equal(before, f.pool.tensors["pages"])


def test_calls_with_rows_and_counts_out_of_range_touch_nothing():
    import torch
    from quantized_decode_attention_gb300 import DQError
    f = Filled([40, 70], page_size=64)
    before = [t.clone() for t in f.pool.tensors.values()]
    x = torch.ones(4, 2, 128, dtype=torch.bfloat16, device="cuda")
    q = torch.ones(4, 8, 128, dtype=torch.bfloat16, device="cuda")
    for rows, cu, most in (([0, 2], [0, 2, 4], 2), ([0, 1 << 30], [0, 2, 4], 2), ([0, 1], [0, 2, 5], 4), ([0, 1], [0, 3, 2], 4),
                           ([0, 1], [-1, 2, 4], 4)):
        rows, cu = _i32(rows), _i32(cu)
        out = torch.full_like(q, 7.0)
        ko, vo = torch.full_like(x, 7.0), torch.full_like(x, 7.0)
        f.pool.attention(0, q, out, rows=rows, cu=cu, max_new=most)
        with pytest.raises(DQError, match="out of range"):
            f.pool.check()
        f.pool.read(0, ko, vo, rows=rows, cu=cu, max_new=most)
        with pytest.raises(DQError, match="out of range"):
            f.pool.check()
    f.pool.append(0, x, x, rows=_i32([5, -1]), cu=_i32([0, 2, 4]), max_new=2)
    with pytest.raises(DQError, match="out of range"):
        f.pool.check()
    f.pool.append(0, x, x, rows=_i32([0, 1]), cu=_i32([0, 0, 4]), max_new=3)  # four tokens where three were promised
    with pytest.raises(DQError, match="out of range"):
        f.pool.check()
    f.pool.tensors["table"][0, 0] = 1000  # a table that names no page
    out = torch.empty(1, 8, 128, dtype=torch.bfloat16, device="cuda")
    f.pool.attention(0, q[:1], out, rows=_i32([0]))
    with pytest.raises(DQError, match="no page"):
        f.pool.check()
    f.pool.tensors["table"][0, 0] = before[2][0, 0]
    for t, b in zip(f.pool.tensors.values(), before):
        if t is not f.pool.tensors["workspace"]:
            assert torch.equal(t, b)


# ---- attention ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("d, G, P, dtype", [(128, 4, 64, "bf16"), (64, 1, 16, "f16"), (128, 8, 32, "f16"), (64, 5, 128, "bf16"),
                                            (128, 16, 128, "bf16"), (64, 16, 64, "f16"), (128, 1, 16, "bf16"), (128, 3, 64, "f16")])
def test_attention_of_single_tokens(d, G, P, dtype):
    """Lengths from nothing to many pages, ends inside tiles and pages, padding and permuted rows."""
    lens = [1, 0, 15, 16, 17, P - 1, P, P + 1, 5 * P + 7, 129, 300]
    f = Filled(lens, seed=d + G, n_kv_heads=2, n_q_heads=2 * G, head_dim=d, page_size=P, dtype=dtype, n_pages=100, max_pages_per_seq=24)
    rows = [3, 8, -1, 0, 10, 1, 7, 2, 9, 4, 6, 5, -7]
    f.verify(f.queries([1] * len(rows)), [1] * len(rows), rows)
    f.verify(f.queries([1] * len(lens), amp=4.0), [1] * len(lens), scale=0.3)


@pytest.mark.parametrize("d, G, P, dtype", [(128, 4, 64, "bf16"), (64, 2, 16, "f16"), (128, 8, 128, "f16"), (128, 1, 32, "bf16"),
                                            (64, 7, 64, "bf16"), (128, 16, 64, "f16")])
def test_attention_of_several_tokens(d, G, P, dtype):
    """Ragged new tokens, causal at the end; rows with none, and a row with more queries than it has tokens."""
    lens = [200, 3, 64, 130, 0, 77, 257]
    counts = [5, 3, 64, 0, 2, 80, 131]
    f = Filled(lens, seed=G, n_kv_heads=2, n_q_heads=2 * G, head_dim=d, page_size=P, dtype=dtype, n_pages=100, max_pages_per_seq=24)
    f.verify(f.queries(counts), counts)
    few = [2, 1, 3, 1, 1, 2, 4]
    f.verify(f.queries(few, amp=3.0), few)


def test_attention_of_a_long_row_and_many_short_ones():
    f = Filled([4099] + [9] * 40, n_pages=320, max_pages_per_seq=70, page_size=64)
    f.verify(f.queries([1] * 41), [1] * 41)
    counts = [33] + [2] * 40
    f.verify(f.queries(counts), counts)


def test_attention_of_very_many_rows():
    """1024 rows of all lengths, single tokens and ragged few and many."""
    rng = np.random.default_rng(8)
    lens = [int(x) for x in rng.integers(0, 90, 1024)]
    f = Filled(lens, n_pages=3000, max_pages_per_seq=6, page_size=32, n_kv_heads=1, n_q_heads=2, head_dim=64)
    f.verify(f.queries([1] * 1024), [1] * 1024)
    counts = [int(x) for x in rng.integers(0, 4, 1024)]
    f.verify(f.queries(counts), counts)
    counts = [int(x) for x in rng.integers(0, 30, 1024)]
    f.verify(f.queries(counts), counts)


@pytest.mark.parametrize("G, d", [(4, 128), (1, 64), (16, 64)])
def test_attention_of_a_mixed_batch(G, d):
    """Prompts' chunks, a few tokens and single tokens in one call, empty and padding rows among them."""
    lens = [400, 900, 0, 33, 700, 64, 0, 1300]
    f = Filled(lens, n_pages=80, max_pages_per_seq=24, n_kv_heads=2, n_q_heads=2 * G, head_dim=d)
    counts = [150, 1, 40, 33, 2, 9, 1, 1]
    f.verify(f.queries(counts), counts)
    rows = [7, -1, 1, 6, 0, 4, -3, 3]
    f.verify(f.queries(counts), counts, rows)
    f.verify(f.queries([70]), [70], [1])
    f.verify(f.queries([2]), [2], [7])


def test_attention_of_negative_and_zero_scales():
    f = Filled([333, 150], page_size=64)
    for n in (1, 2, 40):
        for s in (-0.1, 0.0):
            f.verify(f.queries([n, n]), [n, n], scale=s)


def test_attention_of_strided_queries_and_exponents():
    import torch
    f = Filled([90, 33], k_exp=3, v_exp=-6, page_size=32, dtype="f16")
    wide = f.queries([1, 1, 1])[:2]
    w = torch.empty(2, 3, 8, 128, dtype=torch.float16, device="cuda")
    w[:, 1] = wide
    f.verify(w[:, 1], [1, 1])
    f.verify(w.permute(2, 0, 1, 3)[:, :, 1].transpose(0, 1), [1, 1])


@pytest.mark.parametrize("dtype, amp", [("bf16", 2.0 ** 40), ("bf16", 2.0 ** -60), ("f16", 2.0 ** 13), ("f16", 2.0 ** -14)])
def test_attention_of_very_large_and_very_small_queries(dtype, amp):
    """sm_scale takes the queries' size out again, so that the softmax stays an ordinary one."""
    f = Filled([70, 200], dtype=dtype)
    f.verify(f.queries([1, 1], amp=amp), [1, 1], scale=0.1 / amp)


def test_attention_where_one_key_takes_all_and_where_all_are_equal():
    import torch
    f = Filled([150, 150], wide=False)
    q = f.queries([1, 1])
    q[0] = (torch.tensor(f.hk[0][77]).repeat_interleave(4, 0) * 8).to(q.dtype).cuda()
    q[1] = 0.0
    f.verify(q, [1, 1])


def test_attention_of_a_query_that_is_not_finite_stays_in_its_row():
    import torch
    f = Filled([150, 90])
    q = f.queries([1, 1])
    q[0, 3, 5] = float("nan")
    out, lse = f.attend(q, [1, 1])
    assert torch.isnan(out[0, 3]).all() and torch.isnan(lse[0, 3])
    want, _, tol, _ = f.expect(q[1:], [1], rows=[1])
    assert (np.abs(_np(out[1:]) - want) <= tol).all()


def test_attention_is_the_same_every_time():
    import torch
    f = Filled([1000, 700, 1], n_pages=64, max_pages_per_seq=20)
    q = f.queries([1, 1, 1])
    a = [f.attend(q, [1, 1, 1]) for _ in range(5)]
    for x in a[1:]:
        assert torch.equal(x[0], a[0][0]) and torch.equal(x[1], a[0][1])


# ---- chosen pages ------------------------------------------------------------------------------------
@pytest.mark.parametrize("d, G, P, dtype, keep, first, last", [
    (128, 4, 16, "bf16", 5, 1, 1), (64, 1, 16, "f16", 3, 0, 0), (128, 16, 32, "bf16", 9, 2, 3), (64, 8, 64, "f16", 2, 1, 1),
    (128, 7, 128, "f16", 3, 0, 1), (128, 2, 16, "bf16", 1, 0, 0)])
def test_select_and_attend(d, G, P, dtype, keep, first, last):
    import torch
    lens = [20 * P + 3, 1, 0, keep * P, keep * P + 1, 11 * P, 2 * P + 5]
    f = Filled(lens, seed=keep, n_kv_heads=2, n_q_heads=2 * G, head_dim=d, page_size=P, dtype=dtype, n_pages=80, max_pages_per_seq=24)
    rows = [4, 0, -1, 2, 6, 1, 3, 5]
    q = f.queries([1] * len(rows))
    sel = torch.full((len(rows), 2, keep), 99, dtype=torch.int32, device="cuda")
    f.pool.select(0, q, sel, rows=_i32(rows), keep_first=first, keep_last=last)
    f.pool.check()
    got = sel.cpu().numpy()
    want = []
    for i, r in enumerate(rows):
        want.append([])
        for h in range(2):
            n = 0 if r < 0 else -(-lens[r] // P)
            sums = [R.summary(f.hk[r][j * P:(j + 1) * P, h]) for j in range(n)]
            c = R.choose(_np(q[i, h * G:(h + 1) * G]), sums, n, keep, first, last)
            want[-1].append(c)
            assert list(got[i, h]) == c + [-1] * (keep - len(c)), (i, h)
    f.verify(q, [1] * len(rows), rows, chosen=want, sel=sel)


def test_select_takes_the_lower_page_where_scores_are_equal():
    import torch
    f = Filled([0], n_kv_heads=1, n_q_heads=1, page_size=16, n_pages=700, max_pages_per_seq=600)
    f.pool.resize(None, _i32([16 * 600]))
    x = torch.ones(16 * 600, 1, 128, dtype=torch.bfloat16, device="cuda")
    x[16 * 400:16 * 402] = 2.0
    f.pool.append(0, x, x, cu=_i32([0, 16 * 600]), max_new=16 * 600)
    sel = torch.empty(1, 1, 40, dtype=torch.int32, device="cuda")
    f.pool.select(0, x[:1], sel, keep_first=0, keep_last=2)
    f.pool.check()
    assert sel.flatten().tolist() == list(range(36)) + [400, 401, 598, 599]
    f.pool.select(0, torch.zeros_like(x[:1]), sel, keep_first=0, keep_last=0)
    assert sel.flatten().tolist() == list(range(40))
    f.pool.select(0, torch.full_like(x[:1], float("inf")), sel, keep_first=0, keep_last=0)
    f.pool.check()
    assert sel.flatten().tolist() == list(range(40))


def test_the_score_bounds_every_key_of_the_page():
    """Q+ . largest + Q- . smallest >= sum_h q_h . k for every held key, with the summaries that append wrote."""
    f = Filled([1000], page_size=32, n_pages=40, max_pages_per_seq=32)
    q = _np(f.queries([1]))[0].reshape(2, 4, 128)
    s = f.pool.tensors["summary"].cpu().numpy().reshape(40, 2, 272)
    t = f.pool.tensors["table"][0].tolist()
    for h in range(2):
        hi, lo = np.maximum(q[h], 0).sum(0), np.minimum(q[h], 0).sum(0)
        for j in range(32):
            b = s[t[j], h]
            u = 2.0 ** b[256:260].view(np.int32)[0]
            bound = (hi @ b[:128].view(np.int8) + lo @ b[128:256].view(np.int8)) * u
            assert (f.hk[0][j * 32:(j + 1) * 32, h] @ q[h].sum(0) <= bound + 1e-9).all()


def test_attention_ignores_chosen_pages_that_are_not_there():
    import torch
    f = Filled([100, 20], page_size=16, n_pages=20, max_pages_per_seq=9)
    sel = torch.tensor([[[0, -1, 6, 7, 8, 500], [-1] * 6], [[1, 2, 3, -5, -1, -1], [0, -1, -1, -1, -1, -1]]], dtype=torch.int32, device="cuda")
    f.verify(f.queries([1, 1]), [1, 1], chosen=[[[0, 6], []], [[1], [0]]], sel=sel)


# ---- lengths, forks, compaction -------------------------------------------------------------------------
def _same(pool, m):
    t = np.full((m.R, m.M), -1)
    for r, p in enumerate(m.table):
        t[r, :len(p)] = p
    assert (pool.tensors["table"].cpu().numpy().reshape(m.R, m.M) == t).all()
    assert pool.tensors["seq_len"].tolist() == m.length
    assert pool.tensors["refs"].tolist() == m.refs


@pytest.mark.parametrize("seed, P, N, R_, M, L", [(1, 16, 40, 9, 12, 1), (2, 64, 25, 17, 5, 3), (3, 32, 3000, 40, 70, 2), (4, 128, 7, 5, 3, 1)])
def test_random_lengths_forks_and_compactions(seed, P, N, R_, M, L):
    """Tables, counts, lengths and the bytes of copied and moved pages after every call, refusals among them."""
    import torch
    from quantized_decode_attention_gb300 import DQError
    rng = np.random.default_rng(seed)
    pool = _pool(page_size=P, n_pages=N, max_seqs=R_, max_pages_per_seq=M, n_layers=L, n_kv_heads=1, n_q_heads=1, head_dim=64)
    gen = torch.Generator("cuda").manual_seed(seed)
    m = R.Model(N, P, R_, M)
    for name in ("pages", "summary"):
        pool.tensors[name].random_(0, 256, generator=gen)
    view = lambda n: pool.tensors[n].view(L, N, -1)
    refused = 0
    for step in range(60):
        want = {n: view(n).clone() for n in ("pages", "summary")}
        what = rng.choice(["resize", "resize", "fork", "compact"])
        m.copies = []
        if what == "resize":
            k = int(rng.integers(1, R_ + 1))
            rows = [int(x) for x in rng.permutation(R_)[:k]]
            lens = [int(rng.choice([0, m.length[r], min(M * P, m.length[r] + 1), rng.integers(0, M * P + 1), rng.integers(0, 2 * P)])) for r in rows]
            if rng.random() < 0.15:
                i = int(rng.integers(0, k))
                rows[i], lens[i] = [(-1, lens[i]), (R_, 3), (rows[0], 1), (rows[i], M * P + 1), (rows[i], -1)][int(rng.integers(0, 5))]
            fine = m.resize(rows, lens)
            pool.resize(None if rows == list(range(k)) else _i32(rows), _i32(lens))
        elif what == "fork":
            k = int(rng.integers(1, R_))
            empty = [r for r in range(R_) if m.length[r] == 0]
            dst = [int(x) for x in rng.permutation(empty)[:k]] or [0]
            some = [r for r in range(R_) if m.length[r]] or [0]
            src = [int(rng.choice(some)) for _ in dst]
            if rng.random() < 0.2:
                i = int(rng.integers(0, len(dst)))
                src[i], dst[i] = [(-1, dst[i]), (R_, dst[i]), (src[i], src[i]), (dst[0], dst[i]), (src[i], -3)][int(rng.integers(0, 5))]
            fine = m.fork(src, dst)
            pool.fork(_i32(src), _i32(dst))
        else:
            fine = m.compact()
            pool.compact()
        if fine:
            pool.check()
        else:
            refused += 1
            with pytest.raises(DQError, match="DQ_ENOMEM|DQ_EINVAL"):
                pool.check()
        _same(pool, m)
        for n, w in want.items():
            for a, b in m.copies if fine else []:
                w[:, b] = w[:, a].clone()
            assert torch.equal(view(n), w), (step, what, n)
    assert refused


def test_a_full_list_of_rows():
    import torch
    pool = _pool(page_size=16, n_pages=5000, max_seqs=1024, max_pages_per_seq=4, n_kv_heads=1, n_q_heads=1, head_dim=64)
    m = R.Model(5000, 16, 1024, 4)
    rng = np.random.default_rng(5)
    for _ in range(3):
        lens = [int(x) for x in rng.integers(0, 65, 1024)]
        assert m.resize(range(1024), lens)
        pool.resize(None, _i32(lens))
        pool.check()
        _same(pool, m)
        m.compact()
        pool.compact()
        _same(pool, m)
    keep = [r for r in range(512) if m.length[r]]
    m.resize(range(512, 1024), [0] * 512)
    pool.resize(_i32(range(512, 1024)), torch.zeros(512, dtype=torch.int32, device="cuda"))
    assert m.fork(keep, [512 + r for r in keep])
    pool.fork(_i32(keep), _i32([512 + r for r in keep]))
    pool.check()
    _same(pool, m)


def test_pages_beyond_four_gigabytes():
    """Pages numbered so that their bytes lie past 2^32: append, copy on write, move, choice and both attentions."""
    import torch
    N, P = 32000, 128
    f = Filled.__new__(Filled)
    pool = _pool(n_pages=N, page_size=P, n_kv_heads=8, n_q_heads=32, max_seqs=3, max_pages_per_seq=4)
    assert pool.tensors["pages"].numel() > 1 << 32
    pool.tensors["refs"][:N - 12] = 1  # what is free lies at the end
    rng = np.random.default_rng(4)
    lens = [300, 130]
    pool.resize(_i32([0, 1]), _i32(lens))
    k, v = (torch.tensor(rng.normal(size=(430, 8, 128))).to(torch.bfloat16).cuda() for _ in range(2))
    pool.append(0, k, v, cu=_cu(lens), max_new=300)
    pool.fork(_i32([1]), _i32([2]))
    pool.resize(_i32([2]), _i32([131]))  # a copy of row 1's second page
    pool.append(0, k[:1], v[:1], rows=_i32([2]))
    pool.check()
    assert int(pool.tensors["table"][:, 0].min()) >= N - 12
    hk, hv = R.quantise(_np(k), 0)[2], R.quantise(_np(v), 0)[2]
    f.pool, f.layer, f.dtype, f.Hkv, f.G, f.d, f.P, f.rng = pool, 0, "bf16", 8, 4, 128, P, rng
    f.lens = [300, 130, 131]
    f.hk = [hk[:300], hk[300:], np.concatenate([hk[300:], hk[:1]])]
    f.hv = [hv[:300], hv[300:], np.concatenate([hv[300:], hv[:1]])]
    q = f.queries([1, 1, 1])
    f.verify(q, [1, 1, 1])
    counts = [40, 9, 12]
    f.verify(f.queries(counts), counts)
    sel = torch.empty(3, 8, 2, dtype=torch.int32, device="cuda")
    pool.select(0, q, sel)
    want = [[R.choose(_np(q[r, h * 4:h * 4 + 4]), [R.summary(f.hk[r][j * P:(j + 1) * P, h]) for j in range(-(-f.lens[r] // P))],
                      -(-f.lens[r] // P), 2, 1, 1) for h in range(8)] for r in range(3)]
    assert [[[x for x in y if x >= 0] for y in z] for z in sel.tolist()] == want
    f.verify(q, [1, 1, 1], chosen=want, sel=sel)
    pool.tensors["refs"][:5] = 0
    pool.compact()  # the highest pages move below
    pool.check()
    low = pool.tensors["table"][pool.tensors["table"] >= 0]
    assert low[low < 5].unique().tolist() == [0, 1, 2, 3, 4]  # five of the six pages found room (one is in two rows)
    f.verify(q, [1, 1, 1])


# ---- together --------------------------------------------------------------------------------------------
@pytest.mark.parametrize("captured", [False, True])
def test_a_beam_search_as_a_program_runs_it(captured):
    """Prompts, forks into beams, decode steps (resize, append, select, attention) of two layers, beams that end, a
    compaction in between; the steps captured once into a graph and replayed, or called."""
    import torch
    P, H, G, d, L = 16, 2, 4, 128, 2
    pool = _pool(page_size=P, n_pages=60, n_layers=L, n_kv_heads=H, n_q_heads=H * G, head_dim=d, max_seqs=8, max_pages_per_seq=10)
    m = R.Model(60, P, 8, 10)
    rng = np.random.default_rng(11)
    rnd = lambda *s: torch.tensor(rng.normal(size=s)).to(torch.bfloat16).cuda()
    held = [[[np.zeros((0, H, d)), np.zeros((0, H, d))] for _ in range(8)] for _ in range(L)]

    def add(layer, r, k, v):
        a = held[layer][r]
        held[layer][r] = [np.concatenate([a[0], R.quantise(_np(k), 0)[2]]), np.concatenate([a[1], R.quantise(_np(v), 0)[2]])]

    prompts = [37, 50]
    m.resize([0, 1], prompts)
    pool.resize(None, _i32(prompts))
    for layer in range(L):
        k, v = rnd(87, H, d), rnd(87, H, d)
        pool.append(layer, k, v, cu=_cu(prompts), max_new=50)
        add(layer, 0, k[:37], v[:37])
        add(layer, 1, k[37:], v[37:])
    src, dst = [0, 0, 1, 1], [2, 3, 4, 5]
    m.fork(src, dst)
    pool.fork(_i32(src), _i32(dst))
    for layer in range(L):
        for s, t in zip(src, dst):
            held[layer][t] = list(held[layer][s])
    rows, keep = [2, 3, 4, 5, 0, -1], 3
    rt, lens = _i32(rows), torch.zeros(6, dtype=torch.int32, device="cuda")
    q = [torch.zeros(6, H * G, d, dtype=torch.bfloat16, device="cuda") for _ in range(L)]
    kn, vn = ([torch.zeros(6, H, d, dtype=torch.bfloat16, device="cuda") for _ in range(L)] for _ in range(2))
    full, part = ([torch.zeros_like(x) for x in q] for _ in range(2))
    sel = [torch.zeros(6, H, keep, dtype=torch.int32, device="cuda") for _ in range(L)]

    def step():
        pool.resize(rt, lens)
        for layer in range(L):
            pool.append(layer, kn[layer], vn[layer], rows=rt)
            pool.attention(layer, q[layer], full[layer], rows=rt)
            pool.select(layer, q[layer], sel[layer], rows=rt)
            pool.attention(layer, q[layer], part[layer], rows=rt, sel=sel[layer])

    graph = None
    for t in range(20):
        if t == 9:  # the fork's source ends, and the pool is put together
            m.resize([1], [0])
            pool.resize(_i32([1]), _i32([0]))
            m.compact()
            pool.compact()
        now = [m.length[r] + 1 if r >= 0 else 0 for r in rows]
        assert m.resize(rows, now)
        lens.copy_(_i32(now))
        for layer in range(L):
            for x in (q[layer], kn[layer], vn[layer]):
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
        _same(pool, m)
        for layer in range(L):
            for i, r in enumerate(rows):
                if r >= 0:
                    add(layer, r, kn[layer][i:i + 1], vn[layer][i:i + 1])
            if t % 6 and t != 9:
                continue
            f = Filled.__new__(Filled)
            f.dtype, f.Hkv, f.G, f.d, f.P, f.lens = "bf16", H, G, d, P, m.length
            f.hk, f.hv = [x[0] for x in held[layer]], [x[1] for x in held[layer]]
            chosen = []
            for i, r in enumerate(rows):
                n = m.pages(m.length[r]) if r >= 0 else 0
                chosen.append([R.choose(_np(q[layer][i, h * G:(h + 1) * G]), [R.summary(f.hk[r][j * P:(j + 1) * P, h]) for j in range(n)],
                                        n, keep, 1, 1) for h in range(H)])
            for got, c in ((full, None), (part, chosen)):
                want, _, tol, _ = f.expect(q[layer], [1] * 6, rows, chosen=c)
                assert (np.abs(_np(got[layer]) - want) <= tol).all(), (t, layer, c is None)


def test_two_graphs_with_a_workspace_each():
    """Two captured steps that replay at the same time on two streams, and one whose lengths change between replays."""
    import torch
    f = Filled([2500, 1900, 40], n_pages=128, max_pages_per_seq=50)
    q = [f.queries([1, 1, 1]) for _ in range(2)]
    long = f.queries([30, 20, 25])
    want, want_long = [f.attend(x, [1, 1, 1])[0] for x in q], f.attend(long, [30, 20, 25])[0]
    handles, s, graphs, outs = [f.pool, f.pool.share()], [torch.cuda.Stream(), torch.cuda.Stream()], [], []
    cu = _cu([30, 20, 25])
    for i in range(2):
        o, ol = torch.empty_like(q[i]), torch.empty_like(long)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s[i]):
            for _ in range(3):
                handles[i].attention(0, q[i], o)
                handles[i].attention(0, long, ol, cu=cu, max_new=30)
        graphs.append(g)
        outs.append((o, ol))
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(s[i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(outs[i][0], want[i]) and torch.equal(outs[i][1], want_long)
    f.pool.resize(_i32([0, 1]), _i32([700, 0]))  # shorter, and empty: the captured call follows
    f.lens[0], f.lens[1] = 700, 0
    for held in (f.hk, f.hv):
        held[0], held[1] = held[0][:700], held[1][:0]
    graphs[0].replay()
    torch.cuda.synchronize()
    f.pool.check()
    exp, _, tol, _ = f.expect(q[0], [1, 1, 1])
    assert (np.abs(_np(outs[0][0]) - exp) <= tol).all()


def test_two_handles_on_two_streams():
    """share() gives a workspace of its own: two attentions over the same sequences at the same time."""
    import torch
    f = Filled([3000, 2000, 1500], n_pages=128, max_pages_per_seq=50)
    q = [f.queries([1, 1, 1]) for _ in range(2)]
    want = [f.attend(x, [1, 1, 1])[0] for x in q]
    two, s = f.pool.share(), [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [f.attend(q[i], [1, 1, 1], stream=s[i], pool=(f.pool, two)[i])[0] for i in range(2)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_second_layer_is_its_own():
    import torch
    f = Filled([70, 33], layer=1, n_layers=3)
    f.verify(f.queries([1, 1]), [1, 1])
    assert bool((f.pool.tensors["pages"].view(3, -1)[[0, 2]] == 0xFF).all())


def test_binding_refuses_wrong_tensors():
    import torch
    f = Filled([40, 20])
    p, q = f.pool, f.queries([1, 1])
    out = torch.empty_like(q)
    k = torch.zeros(2, 2, 128, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: p.attention(0, q.float(), out), lambda: p.attention(0, q.cpu(), out), lambda: p.attention(0, q[:1], out),
                 lambda: p.attention(0, q, out.transpose(0, 1).contiguous().transpose(0, 1)), lambda: p.attention(0, q[:, :4], out[:, :4]),
                 lambda: p.attention(0, q, out, lse=torch.empty(2, 8, dtype=torch.float16, device="cuda")),
                 lambda: p.attention(0, q, out, rows=torch.zeros(2, dtype=torch.int64, device="cuda")),
                 lambda: p.attention(0, q, out, rows=_i32([0])), lambda: p.append(0, k, k[:1]), lambda: p.append(0, k.half(), k),
                 lambda: p.append(0, k.transpose(1, 2), k), lambda: p.read(0, k, k[:, :1]), lambda: p.resize(None, torch.zeros(2, device="cuda")),
                 lambda: p.select(0, q, torch.zeros(1, 2, 4, dtype=torch.int32, device="cuda")), lambda: p.fork(_i32([0]), _i32([0, 1]))):
        with pytest.raises(ValueError):
            call()
    p.check()
