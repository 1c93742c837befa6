"""What the serving entry points refuse, through the C ABI, without a GPU:
every check runs before anything is enqueued."""
import ctypes

import pytest

ARG, UNSUPPORTED = 1, 2
P = 1 << 20  # an aligned non-null pointer that nothing dereferences


class Cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "ks", "vs")] + [("pages", ctypes.c_int64), ("heads", ctypes.c_int),
                                                                        ("page", ctypes.c_int), ("dim", ctypes.c_int)]


class Batch(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("table", "first", "length")] + [("batch", ctypes.c_int), ("max_pages", ctypes.c_int)]


class Rope(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("rows", ctypes.c_int64), ("dim", ctypes.c_int), ("adjacent", ctypes.c_int)]


CACHE = dict(k=P, v=P, ks=P, vs=P, pages=10, heads=2, page=16, dim=64)
BATCH = dict(table=P, first=P, length=P, batch=2, max_pages=4)
ROPE = dict(table=P, rows=64, dim=64, adjacent=0)


@pytest.fixture(scope="module")
def lib(built_lib):
    L = ctypes.CDLL(built_lib)
    L.qmm_last_error.restype = ctypes.c_char_p
    L.qmm_logprobs_workspace_bytes.restype = ctypes.c_size_t
    L.qmm_kv_attention_workspace_bytes.restype = ctypes.c_size_t
    return L


def ref(s):
    return None if s is None else ctypes.byref(s)


def append(lib, cache=CACHE, batch=BATCH, rope=ROPE, xt=0, K=P, ks=128, V=P, vs=128, T=3):
    i64, vp = ctypes.c_int64, ctypes.c_void_p
    return lib.qmm_kv_append(ref(cache and Cache(**cache)), ref(batch and Batch(**batch)), ref(rope and Rope(**rope)), xt, vp(K), i64(ks),
                             vp(V), i64(vs), i64(T), vp(None))


def attention(lib, cache=CACHE, batch=BATCH, rope=ROPE, qt=0, Q=P, qs=256, T=3, heads=4, scale=1.0, causal=1, window=0, max_q=1, max_kv=9,
              out=P, lse=P, ws=P, ws_bytes=0):
    i64, vp = ctypes.c_int64, ctypes.c_void_p
    return lib.qmm_kv_attention(ref(cache and Cache(**cache)), ref(batch and Batch(**batch)), ref(rope and Rope(**rope)), qt, vp(Q), i64(qs),
                                i64(T), heads, ctypes.c_float(scale), causal, i64(window), i64(max_q), i64(max_kv), vp(out), vp(lse), vp(ws),
                                ctypes.c_size_t(ws_bytes), vp(None))


SHARED = [(ARG, dict(cache=None)), (ARG, dict(batch=None)), (ARG, dict(cache=CACHE | dict(k=None))), (ARG, dict(cache=CACHE | dict(v=P + 8))),
          (ARG, dict(cache=CACHE | dict(ks=P + 2))), (ARG, dict(cache=CACHE | dict(pages=0))), (ARG, dict(cache=CACHE | dict(heads=0))),
          (UNSUPPORTED, dict(cache=CACHE | dict(page=48))), (UNSUPPORTED, dict(cache=CACHE | dict(dim=80))), (ARG, dict(cache=CACHE | dict(page=0))),
          (ARG, dict(batch=BATCH | dict(batch=-1))), (ARG, dict(batch=BATCH | dict(table=None))), (ARG, dict(batch=BATCH | dict(first=P + 2))),
          (ARG, dict(batch=BATCH | dict(max_pages=0))), (ARG, dict(batch=BATCH | dict(max_pages=1 << 28))), (ARG, dict(T=-1)),
          (ARG, dict(rope=ROPE | dict(table=None))), (ARG, dict(rope=ROPE | dict(table=P + 4))), (ARG, dict(rope=ROPE | dict(dim=12))),
          (ARG, dict(rope=ROPE | dict(dim=128))), (ARG, dict(rope=ROPE | dict(rows=63)))]


@pytest.mark.parametrize("status,args", SHARED + [
    (ARG, dict(xt=3)), (ARG, dict(K=None)), (ARG, dict(V=P + 4)), (ARG, dict(ks=127)), (ARG, dict(ks=130)), (ARG, dict(xt=1, vs=132))])
def test_append_refuses(lib, status, args):
    assert append(lib, **args) == status
    assert lib.qmm_last_error()


@pytest.mark.parametrize("status,args", SHARED + [
    (ARG, dict(qt=-1)), (ARG, dict(Q=None)), (ARG, dict(qs=255)), (ARG, dict(heads=3)), (ARG, dict(heads=0)), (ARG, dict(scale=0.0)),
    (ARG, dict(scale=float("nan"))), (ARG, dict(scale=float("inf"))), (ARG, dict(window=-1)), (ARG, dict(window=4, causal=0)),
    (ARG, dict(max_q=-1)), (ARG, dict(out=None)), (ARG, dict(out=P + 8)), (ARG, dict(lse=P + 2)), (ARG, dict(heads=2 * 257, qs=2 * 257 * 64))])
def test_attention_refuses(lib, status, args):
    assert attention(lib, **args) == status
    assert lib.qmm_last_error()


def test_nothing_to_do(lib):
    assert append(lib, T=0) == 0 and append(lib, batch=BATCH | dict(batch=0), K=None) == 0
    assert attention(lib, T=0) == 0 and attention(lib, batch=BATCH | dict(batch=0), Q=None) == 0


def test_read_refuses(lib):
    i64, vp = ctypes.c_int64, ctypes.c_void_p
    f = lambda cache=CACHE, pages=P, n=1, xt=0, K=P, V=P: lib.qmm_kv_read(ref(Cache(**cache)), vp(pages), i64(n), xt, vp(K), vp(V), vp(None))  # noqa: E731
    assert f(n=-1) == ARG and f(pages=None) == ARG and f(K=None) == ARG and f(V=P + 8) == ARG and f(xt=7) == ARG
    assert f(cache=CACHE | dict(dim=100)) == UNSUPPORTED
    assert f(n=0, pages=None) == 0


@pytest.mark.parametrize("status,args", [
    (ARG, dict(xt=5)), (ARG, dict(M=-1)), (ARG, dict(V=0)), (ARG, dict(top=-1)), (ARG, dict(V=10, top=11)), (UNSUPPORTED, dict(top=33)),
    (UNSUPPORTED, dict(V=(1 << 20) + 1, stride=1 << 21)), (ARG, dict(X=None)), (ARG, dict(X=P + 2)), (ARG, dict(stride=99)), (ARG, dict(given=None)),
    (ARG, dict(top=2, ids=None)), (ARG, dict(top=2, logp=None)), (ARG, dict(lse=P + 1)), (ARG, dict(G=-1))])
def test_logprobs_refuses(lib, status, args):
    a = dict(xt=0, X=P, stride=100, M=2, V=100, given=P, G=1, top=0, lse=P, entropy=P, glp=P, ids=P, logp=P) | args
    i64, vp = ctypes.c_int64, ctypes.c_void_p
    assert lib.qmm_logprobs(a["xt"], vp(a["X"]), i64(a["stride"]), i64(a["M"]), i64(a["V"]), vp(a["given"]), a["G"], a["top"], vp(a["lse"]),
                            vp(a["entropy"]), vp(a["glp"]), vp(a["ids"]), vp(a["logp"]), vp(None), ctypes.c_size_t(0), vp(None)) == status
    assert lib.qmm_last_error()


def test_workspace_sizes(lib):
    i64 = ctypes.c_int64
    ws = lambda M, V, top: lib.qmm_logprobs_workspace_bytes(i64(M), i64(V), top)  # noqa: E731
    assert ws(0, 100, 1) == 0 and ws(4, 0, 0) == 0 and ws(4, 100, 33) == 0 and ws(4, (1 << 20) + 1, 0) == 0
    assert ws(64, 131073, 5) >= 64 * 5 * 8 and ws(64, 131073, 0) > 0
    at = lambda cache, b, h, T, mq, mk: lib.qmm_kv_attention_workspace_bytes(ref(Cache(**cache)), b, h, i64(T), i64(mq), i64(mk))  # noqa: E731
    assert at(CACHE | dict(dim=100), 1, 4, 1, 1, 10) == 0 and at(CACHE, 1, 3, 1, 1, 10) == 0 and at(CACHE, 0, 4, 1, 1, 10) == 0
    assert at(CACHE, 1, 4, 1, 1, 100000) > 0 and at(CACHE, 1, 4, 1, 1, 64) == 0


@pytest.mark.parametrize("batch,q_heads,max_q", [(1, 4, 1), (1, 32, 1), (3, 8, 1), (7, 16, 200), (64, 4, 1), (2, 4, 90)])
def test_workspace_holds_a_shorter_cache(lib, batch, q_heads, max_q):
    """A window makes a call split like one of a shorter cache: the size for a cache is no less than for any shorter one."""
    i64, most = ctypes.c_int64, 0
    for kv in list(range(64, 6000, 32)) + list(range(6000, 140000, 992)):
        need = lib.qmm_kv_attention_workspace_bytes(ref(Cache(**CACHE)), batch, q_heads, i64(batch * max_q), i64(max_q), i64(kv))
        assert need >= most, kv
        most = need
