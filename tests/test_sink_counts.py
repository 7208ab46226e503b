"""Counts that a C int cannot hold are refused by the binding: ctypes would keep their lower 32
bits, and a window of 2^32 tokens would be one of none. No GPU."""
import pytest
import torch

import hierarchical_chunk_sparse_b200 as hils
from hierarchical_chunk_sparse_b200 import build as hbuild

BF = torch.bfloat16


def params(**kw):
    return hils.Params(**(dict(B=1, H=2, d=64, K=0, W=8, dtype=BF, H_kv=1) | kw))


@pytest.mark.parametrize("name", ["B", "H", "d", "S", "K", "W", "H_kv"])
@pytest.mark.parametrize("value", [2 ** 31, 2 ** 32, 2 ** 32 + 64, 2 ** 63, -2 ** 31 - 1, -2 ** 32])
def test_parameters(name, value):
    with pytest.raises(ValueError, match="beyond 32 bits"):
        params(**{name: value}).c()


def test_the_largest_window_is_kept():
    assert params(W=2 ** 31 - 1).c().W == 2 ** 31 - 1


@pytest.mark.parametrize("A", [2 ** 31, 2 ** 32, 2 ** 32 + 4, -2 ** 32 + 4])
def test_sinks(A):
    p, q, kv, f = params(), torch.zeros(1, 2, 5, 64, dtype=BF), torch.zeros(1, 1, 9, 64, dtype=BF), torch.zeros(1, 2, 5)
    n, acc, idx = torch.zeros(1, dtype=torch.int32), torch.zeros(1, 1, 9), torch.zeros(1, 1, 8, dtype=torch.int32)
    for call in (lambda: hils.hils_sink_prefill(p, A, q, kv, kv, q), lambda: hils.hils_sink_weights(p, A, q, kv, f, acc),
                 lambda: hils.hils_sink_prefill_backward(p, A, q, kv, kv, q, f, q, q, kv, kv),
                 lambda: hils.hils_sink_decode(p, A, q[:, :, :1], kv, kv, n, q[:, :, :1]),
                 lambda: hils.hils_cache_evict(p, A, 8, kv, kv, acc, n, kv[:, :, :8], kv[:, :, :8], acc[..., :8], idx, n)):
        with pytest.raises(ValueError, match="A = .*beyond 32 bits"):
            call()


@pytest.mark.parametrize("rows,other", [(2 ** 32 + 16, 4), (16, 2 ** 32 + 4)])
def test_workspace_sizes(rows, other):
    hbuild.build()
    with pytest.raises(ValueError, match="beyond 32 bits"):
        hils.hils_workspace_bytes(params(), hils.HILS_CALL_SINK_DECODE, rows, other)
