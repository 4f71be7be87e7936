"""ctypes binding of the paged 4-bit cache (include/dq_pages.h): argument checks and
marshalling only.  Every operator runs in the CUDA library on the current stream;
nothing here allocates device memory after a PagePool is made, copies to the host or
synchronizes (PagePool.check() excepted), so a whole decode step can be captured."""
from __future__ import annotations

import ctypes as C

from ._lib import DTYPES, _raise, load

P, I, LL = C.c_void_p, C.c_int, C.c_longlong


class PagesConfig(C.Structure):
    _fields_ = [(n, I) for n in ("n_layers", "n_pages", "page_size", "n_kv_heads", "n_q_heads", "head_dim", "max_seqs",
                                 "max_pages_per_seq", "dtype", "k_exp", "v_exp")]


PAGES_BUFFER_NAMES = ["pages", "summary", "table", "seq_len", "refs", "status", "workspace"]


class PagesBuffers(C.Structure):
    _fields_ = [(n, P) for n in PAGES_BUFFER_NAMES]


_ready = None


def _load():
    global _ready
    if _ready is None:
        L = load()
        cfg, buf = C.POINTER(PagesConfig), C.POINTER(PagesBuffers)
        L.dq_pages_sizes.argtypes = [cfg, C.POINTER(C.c_size_t)]
        L.dq_pages_resize.argtypes = [cfg, buf, P, P, I, P]
        L.dq_pages_fork.argtypes = [cfg, buf, P, P, I, P]
        L.dq_pages_compact.argtypes = [cfg, buf, P]
        L.dq_pages_append.argtypes = [cfg, buf, I, P, P, LL, LL, LL, LL, P, P, I, I, I, P]
        L.dq_pages_read.argtypes = [cfg, buf, I, P, P, P, P, I, I, I, P]
        L.dq_pages_attention.argtypes = [cfg, buf, I, P, LL, LL, P, P, P, P, I, I, I, P, I, C.c_float, P]
        L.dq_pages_select.argtypes = [cfg, buf, I, P, LL, LL, P, I, P, I, I, I, P]
        L.dq_pages_cross.argtypes = [cfg, buf, I, P, LL, LL, P, P, P, P, I, I, I, C.c_float, P]
        L.dq_pages_common.argtypes = [cfg, buf, P, P, I, P, I, I, P, P]
        L.dq_pages_shared_bytes.argtypes = [cfg, I, C.POINTER(C.c_size_t)]
        L.dq_pages_shared.argtypes = [cfg, buf, I, P, LL, LL, P, P, P, P, I, I, I, P, I, I, P, P, C.c_float, P]
        L.dq_pages_weigh.argtypes = [cfg, buf, I, P, LL, LL, P, P, I, P, P, I, I, I, C.c_float, P]
        L.dq_pages_evict.argtypes = [cfg, buf, P, I, P, P, I, I, I, P]
        L.dq_pages_check.argtypes = [buf, P]
        L.dq_pages_test_expire_wait.argtypes = [cfg, buf, I, P, LL, LL, P, P, I, I, I, C.c_ulonglong, P]
        L.dq_pages_test_expire_cross.argtypes = L.dq_pages_test_expire_wait.argtypes
        L.dq_pages_test_expire_shared.argtypes = [cfg, buf, I, P, LL, LL, P, P, I, I, I, P, I, I, P, P, C.c_ulonglong, P]
        L.dq_pages_test_expire_weigh.argtypes = [cfg, buf, I, P, LL, LL, P, P, I, P, I, I, I, C.c_ulonglong, P]
        for f in ("sizes", "resize", "fork", "compact", "append", "read", "attention", "cross", "common", "shared_bytes", "shared",
                  "select", "weigh", "evict", "check", "test_expire_wait", "test_expire_cross", "test_expire_shared", "test_expire_weigh"):
            getattr(L, "dq_pages_" + f).restype = C.c_int
        _ready = L
    return _ready


def make_pages_config(*, n_layers=1, n_pages, page_size=64, n_kv_heads, n_q_heads, head_dim, max_seqs, max_pages_per_seq,
                      dtype="bf16", k_exp=0, v_exp=0) -> PagesConfig:
    return PagesConfig(n_layers, n_pages, page_size, n_kv_heads, n_q_heads, head_dim, max_seqs, max_pages_per_seq,
                       DTYPES[dtype], k_exp, v_exp)


def pages_sizes(cfg: PagesConfig) -> dict:
    arr = (C.c_size_t * len(PAGES_BUFFER_NAMES))()
    _raise(_load().dq_pages_sizes(C.byref(cfg), arr))
    return dict(zip(PAGES_BUFFER_NAMES, list(arr)))


class PagePool:
    """Pages, tables and counts of many sequences, and the operators over them.

    The buffers are torch tensors (any dtype and shape with the bytes that pages_sizes()
    names): ``PagePool.allocate(cfg)`` makes them all; the constructor takes the caller's
    and makes status and workspace where none are given.  ``share()`` gives a second
    handle on the same sequences with a workspace of its own, for calls that may run at
    the same time as this handle's (another stream, another captured graph); a handle
    is kept until its calls have run.  Making one waits for the current stream, so that
    the first call may be on any other (not while a graph is captured: there, the fill is
    part of the graph).

    rows, cu, max_new as in dq_pages.h: int32 device tensors naming the call's table rows
    (None: 0, 1, ...) and where each row's new tokens begin (None: one token each);
    max_new bounds the new tokens of one row.
    """

    def __init__(self, cfg: PagesConfig, *, pages, summary, table, seq_len, refs, status=None, workspace=None):
        import torch
        self.cfg = PagesConfig.from_buffer_copy(cfg)
        self._dtype = torch.float16 if cfg.dtype == DTYPES["f16"] else torch.bfloat16
        self.device = pages.device
        sizes = pages_sizes(cfg)
        given = dict(pages=pages, summary=summary, table=table, seq_len=seq_len, refs=refs, status=status, workspace=workspace)
        for n in ("status", "workspace"):
            if given[n] is None:
                given[n] = torch.zeros(sizes[n], dtype=torch.uint8, device=self.device)
        for n, t in given.items():
            if t.device != self.device or not t.is_cuda:
                raise ValueError(f"{n} is on {t.device}: the pool's buffers are on one CUDA device")
            if not t.is_contiguous() or t.numel() * t.element_size() < sizes[n]:
                raise ValueError(f"{n}: {sizes[n]} contiguous bytes are needed")
        for n in ("table", "seq_len", "refs"):
            if given[n].dtype != torch.int32:
                raise ValueError(f"{n} must be int32")
        self.tensors = given
        self._bufs = PagesBuffers(*[given[n].data_ptr() for n in PAGES_BUFFER_NAMES])
        self._c, self._b = C.byref(self.cfg), C.byref(self._bufs)
        self._index, self._hkv, self._hq, self._d = self.device.index, cfg.n_kv_heads, cfg.n_q_heads, cfg.head_dim
        self._scale = cfg.head_dim ** -0.5
        L = _load()
        self._f = {n: getattr(L, "dq_pages_" + n) for n in ("resize", "fork", "compact", "append", "read", "attention", "cross",
                                                            "common", "shared", "select", "weigh", "evict")}
        self._int32, self._float32 = torch.int32, torch.float32
        self._current_device, self._raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
        self._torch = torch
        # what was filled on the current stream (here, by allocate()) is there for a call on any other
        with torch.cuda.device(self._index):
            if not torch.cuda.is_current_stream_capturing():
                torch.cuda.current_stream().synchronize()

    @classmethod
    def allocate(cls, cfg: PagesConfig, device="cuda") -> "PagePool":
        """A pool of empty rows and free pages."""
        import torch
        device, sizes = torch.device(device), pages_sizes(cfg)
        if device.type == "cuda" and device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        i32 = dict(dtype=torch.int32, device=device)
        return cls(cfg, pages=torch.zeros(sizes["pages"], dtype=torch.uint8, device=device),
                   summary=torch.zeros(sizes["summary"], dtype=torch.uint8, device=device),
                   table=torch.full((cfg.max_seqs, cfg.max_pages_per_seq), -1, **i32),
                   seq_len=torch.zeros(cfg.max_seqs, **i32), refs=torch.zeros(cfg.n_pages, **i32))

    def share(self) -> "PagePool":
        t = self.tensors
        return PagePool(self.cfg, **{n: t[n] for n in ("pages", "summary", "table", "seq_len", "refs", "status")})

    # ---- marshalling ----
    def _call(self, name, stream, *args):
        """The library call with this pool's device current and on `stream` (default: the current one)."""
        if stream is None:
            s = self._raw_stream(self._index)
        else:
            s = stream if isinstance(stream, int) else stream.cuda_stream
        if self._current_device() == self._index:
            st = self._f[name](self._c, self._b, *args, s)
        else:
            with self._torch.cuda.device(self._index):
                st = self._f[name](self._c, self._b, *args, s)
        if st:
            _raise(st)

    def _ints(self, t, name, n=None):
        if t is None:
            return None
        if t.dtype is not self._int32 or t.get_device() != self._index or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous int32 tensor on {self.device}")
        if n is not None and t.numel() != n:
            raise ValueError(f"{name} has {t.numel()} values: {n} are wanted")
        return t.data_ptr()

    def _tokens(self, t, name, heads, n=None):
        """(pointer, n_tok, token stride, head stride) of a [n_tok, heads, head_dim] tensor with contiguous channels."""
        if t.dtype is not self._dtype or t.get_device() != self._index:
            raise ValueError(f"{name} must be {self._dtype} on {self.device}")
        shape, stride = t.shape, t.stride()
        if len(shape) != 3 or shape[1] != heads or shape[2] != self._d or (n is not None and shape[0] != n):
            raise ValueError(f"{name} must be [{'n_tok' if n is None else n}, {heads}, {self._d}] (got {tuple(shape)})")
        if stride[2] != 1:
            raise ValueError(f"{name}: channels must be contiguous")
        return t.data_ptr(), shape[0], stride[0], stride[1]

    def _whole(self, t, name):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")

    def _rows(self, rows, cu, n_tok, max_new):
        """(rows, cu, n_rows, n_tok, max_new) of a call with n_tok new tokens."""
        if cu is None:
            return self._ints(rows, "rows", n_tok), None, n_tok, n_tok, 1 if max_new is None else max_new
        n_rows = cu.numel() - 1
        return self._ints(rows, "rows", n_rows), self._ints(cu, "cu"), n_rows, n_tok, n_tok if max_new is None else max_new

    def _lse(self, lse, n):
        if lse.dtype is not self._float32 or lse.get_device() != self._index or not lse.is_contiguous() or lse.numel() != n * self._hq:
            raise ValueError(f"lse must be contiguous fp32 [{n}, {self._hq}] on {self.device}")
        return lse.data_ptr()

    def _scores(self, scores, *lead):
        """(pointer, cap) of scores [*lead, max_seqs, n_kv_heads, cap]."""
        if scores.dtype is not self._float32 or scores.get_device() != self._index or not scores.is_contiguous():
            raise ValueError(f"scores must be contiguous fp32 on {self.device}")
        want = (*lead, self.cfg.max_seqs, self._hkv)
        if tuple(scores.shape[:-1]) != want:
            raise ValueError(f"scores must be {[*want, 'cap']} (got {tuple(scores.shape)})")
        return scores.data_ptr(), scores.shape[-1]

    def _groups(self, groups, plan, n_rows):
        """(groups, n_groups, plan) of a call with n_rows rows."""
        return self._ints(groups, "groups"), 1 if groups is None else groups.numel() - 1, self._ints(plan, "plan", 2 * n_rows)

    # ---- operators ----
    def resize(self, rows, lens, stream=None):
        """Set rows' lengths (int32 [n]; rows None: 0, 1, ...): frees, copies shared last pages on write, grows.
        Length 0 frees a row."""
        n = lens.numel()
        self._call("resize", stream, self._ints(rows, "rows", n), self._ints(lens, "lens"), n)

    def fork(self, src, dst, stream=None):
        """Empty rows dst[i] become second holders of rows src[i]'s pages."""
        self._call("fork", stream, self._ints(src, "src"), self._ints(dst, "dst", src.numel()), src.numel())

    def compact(self, stream=None):
        """Move live pages down until they are the pool's lowest."""
        self._call("compact", stream)

    def append(self, layer, k, v, rows=None, cu=None, max_new=None, stream=None):
        """Quantise the rows' newest tokens (k, v: [n_tok, n_kv_heads, head_dim]) into their pages; `rows` names a row
        with new tokens once."""
        kp, n, kt, kh = self._tokens(k, "k", self._hkv)
        vp, _, vt, vh = self._tokens(v, "v", self._hkv, n)
        self._call("append", stream, layer, kp, vp, kt, kh, vt, vh, *self._rows(rows, cu, n, max_new))

    def read(self, layer, k_out, v_out, rows=None, cu=None, max_new=None, stream=None):
        """The rows' newest tokens as the cache holds them, into contiguous k_out and v_out."""
        kp, n, _, _ = self._tokens(k_out, "k_out", self._hkv)
        vp = self._tokens(v_out, "v_out", self._hkv, n)[0]
        self._whole(k_out, "k_out")
        self._whole(v_out, "v_out")
        self._call("read", stream, layer, kp, vp, *self._rows(rows, cu, n, max_new))

    def attention(self, layer, q, out, rows=None, cu=None, max_new=None, lse=None, sel=None, sm_scale=None, stream=None):
        """Attention of the rows' newest tokens (q, out: [n_tok, n_q_heads, head_dim]) over their pages, or over the
        pages sel [n_rows, n_kv_heads, n_sel] names; lse: optional fp32 [n_tok, n_q_heads]."""
        qp, n, qt, qh = self._tokens(q, "q", self._hq)
        op = self._tokens(out, "out", self._hq, n)[0]
        self._whole(out, "out")
        sp = None
        n_sel = 0
        lp = None if lse is None else self._lse(lse, n)
        r = self._rows(rows, cu, n, max_new)
        if sel is not None:
            n_sel = sel.shape[-1]
            sp = self._ints(sel, "sel", r[2] * self._hkv * n_sel)
        self._call("attention", stream, layer, qp, qt, qh, op, lp, *r, sp, n_sel, self._scale if sm_scale is None else sm_scale)

    def cross(self, layer, q, out, rows=None, cu=None, max_new=None, lse=None, sm_scale=None, stream=None):
        """Cross attention: queries that are not the row's tokens (q, out: [n_tok, n_q_heads, head_dim]; cu and max_new
        count them; None: one for each row) over all that their rows hold; lse: optional fp32 [n_tok, n_q_heads]."""
        qp, n, qt, qh = self._tokens(q, "q", self._hq)
        op = self._tokens(out, "out", self._hq, n)[0]
        self._whole(out, "out")
        self._call("cross", stream, layer, qp, qt, qh, op, None if lse is None else self._lse(lse, n), *self._rows(rows, cu, n, max_new),
                   self._scale if sm_scale is None else sm_scale)

    def common(self, plan, groups=None, rows=None, cu=None, always=False, stream=None):
        """What the rows of each group have in common (whole leading pages that all of them hold and all their new tokens
        see), into plan int32 [n_rows, 2] for shared(), in every layer.  groups: int32 [n_groups + 1], where each group's
        rows begin among the call's (None: one group of all).  Where reading it once would cost more time than it saves,
        nothing is taken to be common, unless always is set."""
        n = plan.shape[0]
        g, n_groups, pp = self._groups(groups, plan, n)
        self._call("common", stream, self._ints(rows, "rows", n), None if cu is None else self._ints(cu, "cu", n + 1), n, g, n_groups, int(always), pp)

    def shared_scratch(self, n_tok):
        """The buffer that shared() takes for calls of up to n_tok tokens."""
        n = C.c_size_t()
        _raise(_load().dq_pages_shared_bytes(self._c, n_tok, C.byref(n)))
        return self._torch.empty(n.value, dtype=self._torch.uint8, device=self.device)

    def shared(self, layer, q, out, plan, scratch, groups=None, max_group=None, rows=None, cu=None, max_new=None, lse=None,
               sm_scale=None, stream=None):
        """attention() of rows whose groups begin with the same pages: what plan (of common(), the same groups, rows and
        cu) says that a group has in common is read once for all its queries.  max_group: a bound on one group's new
        tokens; scratch: of shared_scratch()."""
        qp, n, qt, qh = self._tokens(q, "q", self._hq)
        op = self._tokens(out, "out", self._hq, n)[0]
        self._whole(out, "out")
        self._whole(scratch, "scratch")
        if scratch.get_device() != self._index or scratch.numel() * scratch.element_size() < n * self._hq * (self._d + 2) * 4:
            raise ValueError(f"scratch: the buffer that shared_scratch({n}) gives is needed")
        r = self._rows(rows, cu, n, max_new)
        g, n_groups, pp = self._groups(groups, plan, r[2])
        self._call("shared", stream, layer, qp, qt, qh, op, None if lse is None else self._lse(lse, n), *r, g, n_groups,
                   n if max_group is None else max_group, pp, scratch.data_ptr(), self._scale if sm_scale is None else sm_scale)

    def weigh(self, layer, q, lse, scores, rows=None, cu=None, max_new=None, sm_scale=None, stream=None):
        """The attention weight that the rows' newest tokens (q: [n_tok, n_q_heads, head_dim], with the lse of their
        attention) give to each held token, summed over them and a KV head's query heads: set for the newest tokens
        themselves, added for those before.  scores: fp32 [max_seqs, n_kv_heads, cap], by table row."""
        qp, n, qt, qh = self._tokens(q, "q", self._hq)
        self._call("weigh", stream, layer, qp, qt, qh, self._lse(lse, n), *self._scores(scores), *self._rows(rows, cu, n, max_new),
                   self._scale if sm_scale is None else sm_scale)

    def evict(self, scores, src, dst, keep_first=0, keep_last=0, stream=None):
        """Rows dst (int32 [n], resized to the number of tokens that are to stay) receive, in every layer and KV head, the
        first keep_first and the last keep_last tokens of rows src and those with the highest scores (fp32 [n_layers,
        max_seqs, n_kv_heads, cap]) between them, in order, with their scores.  Rows src stay as they are."""
        n = src.numel()
        self._call("evict", stream, *self._scores(scores, self.cfg.n_layers), self._ints(src, "src"), self._ints(dst, "dst", n), n,
                   keep_first, keep_last)

    def select(self, layer, q, sel, rows=None, keep_first=1, keep_last=1, stream=None):
        """The pages that score highest for each row's one query token (q: [n_rows, n_q_heads, head_dim]) and KV head,
        into sel int32 [n_rows, n_kv_heads, n_sel], ascending, -1 behind them."""
        qp, n, qt, qh = self._tokens(q, "q", self._hq)
        n_sel = sel.shape[-1]
        self._call("select", stream, layer, qp, qt, qh, self._ints(rows, "rows", n), n,
                   self._ints(sel, "sel", n * self._hkv * n_sel), n_sel, keep_first, keep_last)

    def check(self, stream=None):
        """Synchronize and raise the gravest of what earlier calls latched on the device; the rest is left for the next
        check()."""
        cuda = self._torch.cuda
        with cuda.device(self.device.index):
            s = cuda.current_stream() if stream is None else stream
            _raise(_load().dq_pages_check(self._b, s if isinstance(s, int) else s.cuda_stream))
