"""What the window-and-sink, shared-prefix and eviction calls refuse, before anything is
launched: no GPU, and no address below is ever read."""
import ctypes

import pytest
import torch

import hierarchical_chunk_sparse_b200 as hils
from hierarchical_chunk_sparse_b200 import build as hbuild

X = 0x100000  # aligned, never dereferenced: every call below fails its host checks first
INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 1, 2, 3, 4
B, H, HK, D, LQ, N = 2, 4, 2, 128, 10, 300


@pytest.fixture(scope="module")
def lib():
    hbuild.build()
    return hils.load_library()


def T(ptr=X, sb=1 << 20, sh=1 << 16, st=D):
    return hils._CTensor(ptr, sb, sh, st)


def params(**kw):
    c = hils.Params(B=B, H=H, d=D, K=0, W=64, dtype=torch.bfloat16, H_kv=HK).c()
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def bytes_of(lib, p, call, rows, other):
    return lib.hils_workspace_bytes(ctypes.byref(p), call, rows, other)


BIG = 1 << 40  # more workspace than any call needs

# each call with valid arguments (in order, by name); a test changes one of them
CALLS = {
    "hils_sink_prefill": dict(p=None, A=4, Q=T(), Lq=LQ, K=T(), V=T(), N=N, O=T(), lse=X, ws=X, nws=BIG, stream=None),
    "hils_sink_prefill_backward": dict(p=None, A=4, Q=T(), K=T(), V=T(), N=N, O=T(), lse=X, dO=T(), dQ=T(), dK=T(), dV=T(),
                                       ws=X, nws=BIG, stream=None),
    "hils_sink_weights": dict(p=None, A=4, Q=T(), Lq=LQ, K=T(), N=N, lse=X, acc=X, acc_out=X, T=N, ws=X, nws=BIG, stream=None),
    "hils_sink_decode": dict(p=None, A=4, Q=T(), Kc=T(), Vc=T(), T=N, cache_len=X, O=T(), lse=X, acc=None, acc_out=None, ws=X,
                             nws=BIG, stream=None),
    "hils_prefix_decode": dict(p=None, Q=T(), Kp=T(), Vp=T(), P=N, Kc=T(), Vc=T(), T=20, cache_len=X, O=T(), lse=X, ws=X,
                               nws=BIG, stream=None),
    "hils_cache_evict": dict(p=None, A=4, budget=100, K=T(X), V=T(2 * X), T=N, acc=3 * X, cache_len=4 * X, Kout=T(1 << 34),
                             Vout=T(1 << 35), acc_out=1 << 36, idx=1 << 37, len_out=4 * X, ws=X, nws=BIG, stream=None),
}
SIZES = {"hils_sink_prefill": (hils.HILS_CALL_SINK_PREFILL, LQ, 4), "hils_sink_prefill_backward": (hils.HILS_CALL_SINK_BACKWARD, N, 4),
         "hils_sink_weights": (hils.HILS_CALL_SINK_WEIGHTS, N, 4), "hils_sink_decode": (hils.HILS_CALL_SINK_DECODE, N, 4),
         "hils_prefix_decode": (hils.HILS_CALL_PREFIX_DECODE, 20, N), "hils_cache_evict": (hils.HILS_CALL_CACHE_EVICT, N, 100)}


def call(lib, name, p=None, **change):
    a = dict(CALLS[name])
    a["p"] = p or params()
    assert set(change) <= set(a), change
    a.update(change)
    return getattr(lib, name)(ctypes.byref(a.pop("p")), *a.values())


VIEWS = [(n, k) for n, a in CALLS.items() for k, v in a.items() if isinstance(v, hils._CTensor)]


@pytest.mark.parametrize("name,view", VIEWS)
def test_views(lib, name, view):
    assert call(lib, name, **{view: T(None)}) == INVALID
    assert call(lib, name, **{view: T(X + 8)}) == ALIGNMENT
    assert call(lib, name, **{view: T(sh=D + 4)}) == ALIGNMENT
    assert call(lib, name, **{view: T(st=D + 1)}) == ALIGNMENT


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("change,code", [
    (dict(B=-1), INVALID), (dict(W=-1), INVALID), (dict(scale=float("inf")), INVALID), (dict(H_kv=3), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(dtype=5), UNSUPPORTED), (dict(H=32, H_kv=2), UNSUPPORTED), (dict(flags=8), UNSUPPORTED),
    (dict(S=32), UNSUPPORTED),
])
def test_params(lib, name, change, code):
    assert call(lib, name, p=params(**change)) == code
    assert bytes_of(lib, params(**change), *SIZES[name]) == 0
    assert getattr(lib, name)(None, *list(CALLS[name].values())[1:]) == INVALID


@pytest.mark.parametrize("name", CALLS)
def test_workspace(lib, name):
    need = bytes_of(lib, params(), *SIZES[name])
    assert need >= 256
    assert call(lib, name, ws=None) == WORKSPACE
    assert call(lib, name, nws=255) == WORKSPACE
    assert call(lib, name, ws=X + 4) == ALIGNMENT


@pytest.mark.parametrize("name,change,code", [
    ("hils_sink_prefill", dict(A=-1), INVALID), ("hils_sink_prefill", dict(Lq=-1), INVALID),
    ("hils_sink_prefill", dict(N=LQ - 1), INVALID), ("hils_sink_prefill", dict(Lq=1 << 30, N=1 << 30), INVALID),
    ("hils_sink_prefill", dict(lse=X + 2), ALIGNMENT),
    ("hils_sink_prefill_backward", dict(A=-1), INVALID), ("hils_sink_prefill_backward", dict(N=-1), INVALID),
    ("hils_sink_prefill_backward", dict(lse=None), INVALID), ("hils_sink_prefill_backward", dict(lse=X + 1), ALIGNMENT),
    ("hils_sink_weights", dict(N=LQ - 1), INVALID), ("hils_sink_weights", dict(T=N - 1), INVALID),
    ("hils_sink_weights", dict(lse=None), INVALID), ("hils_sink_weights", dict(acc=None), INVALID),
    ("hils_sink_weights", dict(acc_out=None), INVALID), ("hils_sink_weights", dict(acc=X + 2), ALIGNMENT),
    ("hils_sink_decode", dict(T=-1), INVALID), ("hils_sink_decode", dict(A=-5), INVALID),
    ("hils_sink_decode", dict(cache_len=None), INVALID), ("hils_sink_decode", dict(cache_len=X + 1), ALIGNMENT),
    ("hils_sink_decode", dict(acc=X), INVALID), ("hils_sink_decode", dict(acc_out=X), INVALID),
    ("hils_sink_decode", dict(acc=X + 2, acc_out=X), ALIGNMENT),
    ("hils_prefix_decode", dict(P=-1), INVALID), ("hils_prefix_decode", dict(T=-1), INVALID),
    ("hils_prefix_decode", dict(cache_len=None), INVALID),
    ("hils_cache_evict", dict(budget=-1), INVALID), ("hils_cache_evict", dict(budget=67), INVALID),  # A + W = 68
    ("hils_cache_evict", dict(A=-1), INVALID), ("hils_cache_evict", dict(T=-1), INVALID),
    ("hils_cache_evict", dict(acc=None), INVALID), ("hils_cache_evict", dict(cache_len=None), INVALID),
    ("hils_cache_evict", dict(acc_out=None), INVALID), ("hils_cache_evict", dict(idx=None), INVALID),
    ("hils_cache_evict", dict(len_out=None), INVALID), ("hils_cache_evict", dict(idx=(1 << 37) + 2), ALIGNMENT),
    # outputs over what is read
    ("hils_cache_evict", dict(Kout=T(X)), INVALID), ("hils_cache_evict", dict(Vout=T(2 * X + 4096)), INVALID),
    ("hils_cache_evict", dict(Kout=T(2 * X)), INVALID), ("hils_cache_evict", dict(acc_out=3 * X), INVALID),
])
def test_arguments(lib, name, change, code):
    assert call(lib, name, **change) == code


def test_nothing_to_do_is_no_error(lib):
    """No rows: success without a launch (and without a workspace)."""
    none = T(None)
    for name in CALLS:
        assert call(lib, name, p=params(B=0), ws=None) == 0
    assert call(lib, "hils_sink_prefill", Lq=0, Q=none, O=none, ws=None) == 0
    assert call(lib, "hils_sink_weights", Lq=0, Q=none, lse=None, acc=None, acc_out=None, ws=None) == 0


def test_workspace_sizes_grow_with_the_call(lib):
    """The size for N tokens serves every shorter call."""
    for c, rows in ((hils.HILS_CALL_SINK_WEIGHTS, (1, 64, 1000, 8192)), (hils.HILS_CALL_SINK_BACKWARD, (1, 300, 8192)),
                    (hils.HILS_CALL_SINK_DECODE, (1, 500, 100000)), (hils.HILS_CALL_PREFIX_DECODE, (0, 64, 4096))):
        sizes = [bytes_of(lib, params(), c, r, 4) for r in rows]
        assert sizes == sorted(sizes) and sizes[0] >= 256
    assert bytes_of(lib, params(), hils.HILS_CALL_SINK_DECODE_ACC, 5000, 4) > bytes_of(lib, params(), hils.HILS_CALL_SINK_DECODE, 5000, 4)
    assert bytes_of(lib, params(), 99, 10, 10) == 0


# ------------------------------------------------------------------ the binding's own checks


def _z(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refuses_wrong_tensors(lib):
    p = hils.Params(B=B, H=H, d=D, K=0, W=64, dtype=torch.bfloat16, H_kv=HK)
    q, kv = _z(B, H, LQ, D), _z(B, HK, N, D)
    with pytest.raises(ValueError, match="CUDA tensor"):
        hils.hils_sink_prefill(p, 4, q, kv, kv, q)
    with pytest.raises(ValueError, match="V has shape"):
        hils._sink_call("hils_sink_prefill", p, (("V", _z(B, HK, N + 1, D), (B, HK, N, D)),), (), None, None)
    with pytest.raises(ValueError, match="O has dtype"):
        hils._sink_call("hils_sink_prefill", p, (("O", q.float(), tuple(q.shape)),), (), None, None)
    with pytest.raises(ValueError, match=r"\[B, H, T, d\]"):
        hils.hils_sink_prefill(p, 4, q[0], kv, kv, q)
    with pytest.raises(ValueError, match=r"\[B, H, T, d\]"):
        hils.hils_cache_evict(p, 0, 64, None, kv, None, None, kv, kv, None, None, None)
    with pytest.raises(ValueError, match="lse has dtype"):
        hils._sink_call("x", p, (), (("lse", _z(B, H, LQ), (B, H, LQ), torch.float32),), None, None)


@pytest.mark.parametrize("call", (hils.HILS_CALL_SINK_WEIGHTS, hils.HILS_CALL_SINK_DECODE, hils.HILS_CALL_SINK_DECODE_ACC,
                                  hils.HILS_CALL_PREFIX_DECODE, hils.HILS_CALL_CACHE_EVICT))
def test_workspaces_of_large_caches_and_of_none(lib, call):
    """More than 2^31 cached tokens over all heads (the calls' rows are their queries), and a
    batch without heads."""
    p = params(B=256, H=64, H_kv=8)
    assert bytes_of(lib, p, call, 1 << 18, 16) >= 256
    for dt in (hils.HILS_F32, hils.HILS_BF16):
        assert bytes_of(lib, params(H=0, dtype=dt), call, 1 << 18, 16) >= 0
        assert bytes_of(lib, params(B=0, dtype=dt), call, 1 << 18, 16) >= 0
    assert bytes_of(lib, p, call, -1, 16) == 0


@pytest.mark.parametrize("name", [n for n in CALLS if n != "hils_cache_evict"])
def test_no_heads_is_no_error(lib, name):
    """Nor does a batch without heads launch anything (an eviction still writes len_out)."""
    assert call(lib, name, p=params(H=0)) == 0


@pytest.mark.parametrize("name,change", [("hils_sink_prefill", dict(N=2**31 - 1)), ("hils_sink_weights", dict(N=2**31 - 1, T=2**31 - 1)),
                                         ("hils_sink_decode", dict(T=2**31 - 1)), ("hils_prefix_decode", dict(P=2**30, T=2**30)),
                                         ("hils_cache_evict", dict(T=2**31 - 1))])
def test_more_tokens_than_positions_count(lib, name, change):
    assert call(lib, name, **change) == UNSUPPORTED


@pytest.mark.parametrize("name,view,rows", [("hils_sink_prefill", "O", LQ), ("hils_sink_prefill_backward", "dQ", N),
                                            ("hils_sink_prefill_backward", "dK", N), ("hils_sink_prefill_backward", "dV", N),
                                            ("hils_sink_decode", "O", 1), ("hils_prefix_decode", "O", 1),
                                            ("hils_cache_evict", "Kout", 100), ("hils_cache_evict", "Vout", 100)])
def test_written_views_are_not_broadcast(lib, name, view, rows):
    ptr = CALLS[name][view].ptr
    for zero in ("sb", "sh") + (("st",) if rows > 1 else ()):
        assert call(lib, name, **{view: T(ptr, **{zero: 0})}) == INVALID
