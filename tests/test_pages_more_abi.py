"""Cross and shared attention, weighing and eviction without a GPU: every refusal that the host and the binding make."""
import ctypes as C

import pytest

from test_pages_abi import EALIGN, EINVAL, EUNSUPPORTED, Q, bufs, cfg, lib, refused, with_  # noqa: F401

CROSS = (0, Q, 4096, 128, Q, None, None, None, 2, 2, 1, 0.1, None)
COMMON = (None, None, 2, None, 1, 0, Q, None)
SHARED = (0, Q, 4096, 128, Q, None, None, None, 2, 2, 1, None, 1, 2, Q, Q, 0.1, None)
WEIGH = (0, Q, 4096, 128, Q, Q, 64, None, None, 2, 2, 1, 0.1, None)
EVICT = (Q, 64, Q, Q, 2, 1, 1, None)


@pytest.mark.parametrize("name, args", [("dq_pages_cross", CROSS), ("dq_pages_common", COMMON), ("dq_pages_shared", SHARED),
                                        ("dq_pages_weigh", WEIGH), ("dq_pages_evict", EVICT)])
def test_refused_pools(lib, name, args):  # noqa: F811
    for n in ("pages", "summary", "table", "seq_len", "refs", "status"):
        refused(lib, name, EINVAL, b=bufs(**{n: None}), args=args)
        refused(lib, name, EALIGN, b=bufs(**{n: 0x10008}), args=args)
    refused(lib, name, EUNSUPPORTED, c=cfg(page_size=20), args=args)
    assert getattr(lib, name)(None, C.byref(bufs()), *args) == EINVAL
    assert getattr(lib, name)(C.byref(cfg()), None, *args) == EINVAL


@pytest.mark.parametrize("name, args, want", [
    ("dq_pages_cross", with_(CROSS, _0=-1), EINVAL), ("dq_pages_cross", with_(CROSS, _0=2), EINVAL),
    ("dq_pages_cross", with_(CROSS, _1=None), EINVAL), ("dq_pages_cross", with_(CROSS, _4=None), EINVAL),
    ("dq_pages_cross", with_(CROSS, _1=Q + 2), EALIGN), ("dq_pages_cross", with_(CROSS, _3=100), EALIGN),
    ("dq_pages_cross", with_(CROSS, _5=Q + 2), EALIGN), ("dq_pages_cross", with_(CROSS, _8=0), EINVAL),
    ("dq_pages_cross", with_(CROSS, _8=1025, _9=1025), EINVAL), ("dq_pages_cross", with_(CROSS, _8=7, _9=7), EINVAL),
    ("dq_pages_cross", with_(CROSS, _9=3), EINVAL), ("dq_pages_cross", with_(CROSS, _10=3), EINVAL),
    ("dq_pages_cross", with_(CROSS, _11=float("inf")), EINVAL),
    ("dq_pages_common", with_(COMMON, _2=0), EINVAL), ("dq_pages_common", with_(COMMON, _2=7), EINVAL),
    ("dq_pages_common", with_(COMMON, _4=0), EINVAL), ("dq_pages_common", with_(COMMON, _4=2), EINVAL),       # two groups, and no groups
    ("dq_pages_common", with_(COMMON, _3=Q, _4=3), EINVAL), ("dq_pages_common", with_(COMMON, _3=Q + 2), EALIGN),
    ("dq_pages_common", with_(COMMON, _6=None), EINVAL), ("dq_pages_common", with_(COMMON, _6=Q + 4), EALIGN),
    ("dq_pages_common", with_(COMMON, _1=Q + 1), EALIGN), ("dq_pages_common", with_(COMMON, _0=Q + 1), EALIGN),
    ("dq_pages_shared", with_(SHARED, _0=-1), EINVAL), ("dq_pages_shared", with_(SHARED, _1=None), EINVAL),
    ("dq_pages_shared", with_(SHARED, _2=4100), EALIGN), ("dq_pages_shared", with_(SHARED, _4=Q + 8), EALIGN),
    ("dq_pages_shared", with_(SHARED, _12=2), EINVAL), ("dq_pages_shared", with_(SHARED, _11=Q + 1), EALIGN),
    ("dq_pages_shared", with_(SHARED, _13=0), EINVAL), ("dq_pages_shared", with_(SHARED, _13=3), EINVAL),
    ("dq_pages_shared", with_(SHARED, _14=None), EINVAL), ("dq_pages_shared", with_(SHARED, _14=Q + 4), EALIGN),
    ("dq_pages_shared", with_(SHARED, _15=None), EINVAL), ("dq_pages_shared", with_(SHARED, _15=Q + 8), EALIGN),
    ("dq_pages_shared", with_(SHARED, _16=float("nan")), EINVAL),
    ("dq_pages_weigh", with_(WEIGH, _0=2), EINVAL), ("dq_pages_weigh", with_(WEIGH, _1=None), EINVAL),
    ("dq_pages_weigh", with_(WEIGH, _4=None), EINVAL), ("dq_pages_weigh", with_(WEIGH, _5=None), EINVAL),
    ("dq_pages_weigh", with_(WEIGH, _1=Q + 8), EALIGN), ("dq_pages_weigh", with_(WEIGH, _2=4097), EALIGN),
    ("dq_pages_weigh", with_(WEIGH, _4=Q + 2), EALIGN), ("dq_pages_weigh", with_(WEIGH, _5=Q + 1), EALIGN),
    ("dq_pages_weigh", with_(WEIGH, _6=0), EINVAL), ("dq_pages_weigh", with_(WEIGH, _6=(1 << 22) + 1), EINVAL),
    ("dq_pages_weigh", with_(WEIGH, _10=3), EINVAL), ("dq_pages_weigh", with_(WEIGH, _12=float("nan")), EINVAL),
    ("dq_pages_evict", with_(EVICT, _0=None), EINVAL), ("dq_pages_evict", with_(EVICT, _0=Q + 2), EALIGN),
    ("dq_pages_evict", with_(EVICT, _1=0), EINVAL), ("dq_pages_evict", with_(EVICT, _2=None), EINVAL),
    ("dq_pages_evict", with_(EVICT, _3=None), EINVAL), ("dq_pages_evict", with_(EVICT, _3=Q + 1), EALIGN),
    ("dq_pages_evict", with_(EVICT, _4=0), EINVAL), ("dq_pages_evict", with_(EVICT, _4=1025), EINVAL),
    ("dq_pages_evict", with_(EVICT, _5=-1), EINVAL), ("dq_pages_evict", with_(EVICT, _6=(1 << 22) + 1), EINVAL)])
def test_refused_calls(lib, name, args, want):  # noqa: F811
    refused(lib, name, want, args=args)


def test_refused_calls_without_a_workspace(lib):  # noqa: F811
    for name, args in (("dq_pages_cross", CROSS), ("dq_pages_shared", SHARED)):
        refused(lib, name, EINVAL, b=bufs(workspace=None), args=args)


@pytest.mark.parametrize("d, hq", [(64, 8), (128, 32)])
def test_shared_bytes(lib, d, hq):  # noqa: F811
    n, c = C.c_size_t(), cfg(head_dim=d, n_kv_heads=8, n_q_heads=hq)
    assert lib.dq_pages_shared_bytes(C.byref(c), 5, C.byref(n)) == 0 and n.value == 5 * hq * (d + 2) * 4
    for bad in (0, -1, (1 << 24) + 1):
        assert lib.dq_pages_shared_bytes(C.byref(c), bad, C.byref(n)) == EINVAL
    assert lib.dq_pages_shared_bytes(None, 5, C.byref(n)) == EINVAL and lib.dq_pages_shared_bytes(C.byref(c), 5, None) == EINVAL
    assert lib.dq_pages_shared_bytes(C.byref(cfg(head_dim=96)), 5, C.byref(n)) == EUNSUPPORTED


def test_refused_calls_whose_waits_run_out(lib):  # noqa: F811
    cross = (0, Q, 4096, 128, Q, None, 2, 2, 1, 1000, None)
    shared = (0, Q, 4096, 128, Q, None, 2, 2, 1, None, 1, 2, Q, Q, 1000, None)
    weigh = (0, Q, 4096, 128, Q, Q, 64, None, 2, 2, 1, 1000, None)
    for name, args in (("cross", cross), ("shared", shared), ("weigh", weigh)):
        name = "dq_pages_test_expire_" + name
        refused(lib, name, EINVAL, args=with_(args, _0=2))
        refused(lib, name, EINVAL, args=with_(args, _1=None))
        refused(lib, name, EALIGN, args=with_(args, _1=Q + 8))
        refused(lib, name, EINVAL, b=bufs(workspace=None), args=args)
    refused(lib, "dq_pages_test_expire_shared", EINVAL, args=with_(shared, _13=None))
    refused(lib, "dq_pages_test_expire_weigh", EINVAL, args=with_(weigh, _6=0))
