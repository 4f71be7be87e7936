"""The paged cache's C ABI and binding without a GPU: exported entry points, buffer
sizes, and every refusal that the host makes before it enqueues anything."""
import ctypes as C
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EINVAL, EALIGN, EUNSUPPORTED = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    from quantized_decode_attention_gb300 import build, pages
    build.build()
    return pages._load()


def cfg(**kw):
    from quantized_decode_attention_gb300 import make_pages_config
    a = dict(n_layers=2, n_pages=40, page_size=64, n_kv_heads=8, n_q_heads=32, head_dim=128, max_seqs=6, max_pages_per_seq=9)
    a.update(kw)
    return make_pages_config(**a)


def bufs(**kw):
    from quantized_decode_attention_gb300 import pages
    b = pages.PagesBuffers(*[0x10000 * (i + 1) for i in range(7)])
    for n, x in kw.items():
        setattr(b, n, x)
    return b


def test_every_declared_symbol_is_exported(lib):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "dq_pages.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(dq_\w+)\s*\(", src))
    assert {"dq_pages_attention", "dq_pages_append", "dq_pages_select", "dq_pages_resize", "dq_pages_check"} <= names
    for n in names:
        assert hasattr(lib, n), n


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_sizes(lib, P, d):
    from quantized_decode_attention_gb300 import pages_sizes
    s = pages_sizes(cfg(page_size=P, head_dim=d))
    assert s["pages"] == 2 * 40 * 8 * P * d * 2 * 9 // 16
    assert s["summary"] == 2 * 40 * 8 * (2 * d + 16)
    assert s["table"] == 6 * 9 * 4 and s["seq_len"] == 24 and s["refs"] == 160 and s["status"] == 16
    assert all(x % 4 == 0 for x in s.values())


@pytest.mark.parametrize("bad, want", [
    (dict(n_layers=0), EINVAL), (dict(n_pages=0), EINVAL), (dict(n_pages=(1 << 20) + 1), EINVAL),
    (dict(page_size=48), EUNSUPPORTED), (dict(page_size=8), EUNSUPPORTED), (dict(head_dim=96), EUNSUPPORTED),
    (dict(n_kv_heads=0), EINVAL), (dict(n_kv_heads=129, n_q_heads=129), EINVAL), (dict(n_q_heads=33), EINVAL),
    (dict(n_q_heads=0), EINVAL), (dict(n_kv_heads=1, n_q_heads=17), EUNSUPPORTED), (dict(max_seqs=0), EINVAL),
    (dict(max_seqs=1025), EINVAL), (dict(max_pages_per_seq=0), EINVAL), (dict(max_pages_per_seq=65537), EINVAL),
    (dict(max_pages_per_seq=65536, page_size=128), EINVAL), (dict(dtype="f32"), EUNSUPPORTED),
    (dict(k_exp=17), EINVAL), (dict(v_exp=-17), EINVAL)])
def test_refused_configs(lib, bad, want):
    from quantized_decode_attention_gb300 import DQError, pages_sizes
    with pytest.raises(DQError) as e:
        pages_sizes(cfg(**bad))
    assert e.value.status == want


def refused(lib, name, want, c=None, b=None, args=()):
    c, b = c or cfg(), b or bufs()
    assert getattr(lib, name)(C.byref(c), C.byref(b), *args) == want, lib.dq_last_error()
    assert lib.dq_last_error()


Q = 0x900000
APPEND = (0, Q, Q, 1024, 128, 1024, 128, None, None, 2, 2, 1, None)
READ = (0, Q, Q, None, None, 2, 2, 1, None)
ATTEND = (0, Q, 4096, 128, Q, None, None, None, 2, 2, 1, None, 0, 0.1, None)
SELECT = (0, Q, 4096, 128, None, 2, Q, 4, 1, 1, None)


def with_(args, **at):
    a = list(args)
    for i, x in at.items():
        a[int(i[1:])] = x
    return tuple(a)


@pytest.mark.parametrize("name, args", [("dq_pages_append", APPEND), ("dq_pages_read", READ), ("dq_pages_attention", ATTEND),
                                        ("dq_pages_select", SELECT), ("dq_pages_resize", (None, Q, 2, None)),
                                        ("dq_pages_fork", (Q, Q, 2, None)), ("dq_pages_compact", (None,))])
def test_refused_pools(lib, name, args):
    for n in ("pages", "summary", "table", "seq_len", "refs", "status"):
        refused(lib, name, EINVAL, b=bufs(**{n: None}), args=args)
        refused(lib, name, EALIGN, b=bufs(**{n: 0x10008}), args=args)
    refused(lib, name, EUNSUPPORTED, c=cfg(page_size=20), args=args)
    assert getattr(lib, name)(None, C.byref(bufs()), *args) == EINVAL
    assert getattr(lib, name)(C.byref(cfg()), None, *args) == EINVAL


@pytest.mark.parametrize("name, args, want", [
    ("dq_pages_append", with_(APPEND, _0=-1), EINVAL), ("dq_pages_append", with_(APPEND, _0=2), EINVAL),
    ("dq_pages_append", with_(APPEND, _1=None), EINVAL), ("dq_pages_append", with_(APPEND, _2=None), EINVAL),
    ("dq_pages_append", with_(APPEND, _1=Q + 2), EALIGN), ("dq_pages_append", with_(APPEND, _3=1028), EALIGN),
    ("dq_pages_append", with_(APPEND, _6=4), EALIGN), ("dq_pages_append", with_(APPEND, _7=Q + 2), EALIGN),
    ("dq_pages_append", with_(APPEND, _9=0), EINVAL), ("dq_pages_append", with_(APPEND, _9=1025), EINVAL),
    ("dq_pages_append", with_(APPEND, _9=7, _10=7), EINVAL),       # rows NULL and more of them than the table has
    ("dq_pages_append", with_(APPEND, _10=3), EINVAL),             # cu NULL: one token for each row
    ("dq_pages_append", with_(APPEND, _11=2), EINVAL), ("dq_pages_append", with_(APPEND, _11=0), EINVAL),
    ("dq_pages_append", with_(APPEND, _10=0), EINVAL),
    ("dq_pages_read", with_(READ, _1=None), EINVAL), ("dq_pages_read", with_(READ, _2=Q + 8), EALIGN),
    ("dq_pages_read", with_(READ, _0=5), EINVAL),
    ("dq_pages_attention", with_(ATTEND, _1=None), EINVAL), ("dq_pages_attention", with_(ATTEND, _4=None), EINVAL),
    ("dq_pages_attention", with_(ATTEND, _4=Q + 4), EALIGN), ("dq_pages_attention", with_(ATTEND, _3=100), EALIGN),
    ("dq_pages_attention", with_(ATTEND, _5=Q + 1), EALIGN), ("dq_pages_attention", with_(ATTEND, _13=float("nan")), EINVAL),
    ("dq_pages_attention", with_(ATTEND, _11=Q, _12=0), EINVAL), ("dq_pages_attention", with_(ATTEND, _11=Q, _12=513), EINVAL),
    ("dq_pages_attention", with_(ATTEND, _7=Q, _11=Q, _12=4), EUNSUPPORTED),  # chosen pages with several tokens
    ("dq_pages_attention", with_(ATTEND, _0=-1), EINVAL),
    ("dq_pages_select", with_(SELECT, _1=None), EINVAL), ("dq_pages_select", with_(SELECT, _6=None), EINVAL),
    ("dq_pages_select", with_(SELECT, _7=0), EINVAL), ("dq_pages_select", with_(SELECT, _7=513), EINVAL),
    ("dq_pages_select", with_(SELECT, _8=-1), EINVAL), ("dq_pages_select", with_(SELECT, _8=3, _9=2), EINVAL),
    ("dq_pages_select", with_(SELECT, _6=Q + 2), EALIGN),
    ("dq_pages_resize", (None, None, 2, None), EINVAL), ("dq_pages_resize", (None, Q, 0, None), EINVAL),
    ("dq_pages_resize", (None, Q, 7, None), EINVAL), ("dq_pages_resize", (Q, Q, 1025, None), EINVAL),
    ("dq_pages_resize", (Q + 1, Q, 2, None), EALIGN),
    ("dq_pages_fork", (None, Q, 2, None), EINVAL), ("dq_pages_fork", (Q, Q, 0, None), EINVAL),
    ("dq_pages_fork", (Q, Q + 2, 2, None), EALIGN)])
def test_refused_calls(lib, name, args, want):
    refused(lib, name, want, args=args)


def test_refused_calls_without_a_workspace(lib):
    for name, args in (("dq_pages_attention", ATTEND), ("dq_pages_resize", (None, Q, 2, None)),
                       ("dq_pages_compact", (None,))):
        refused(lib, name, EINVAL, b=bufs(workspace=None), args=args)


def test_select_refuses_very_long_tables(lib):
    refused(lib, "dq_pages_select", EUNSUPPORTED, c=cfg(max_pages_per_seq=16385, page_size=16), args=SELECT)


def test_check_refuses_null(lib):
    assert lib.dq_pages_check(None, None) == EINVAL


def test_pool_refuses_host_tensors(lib):
    import torch
    from quantized_decode_attention_gb300 import PagePool, pages_sizes
    c = cfg()
    s = pages_sizes(c)
    t = {n: torch.zeros(s[n] // 4, dtype=torch.int32) for n in ("pages", "summary", "table", "seq_len", "refs")}
    with pytest.raises(ValueError, match="CUDA"):
        PagePool(c, **t)
