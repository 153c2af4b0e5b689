"""Calls on a side stream allocate from that stream's pool: a block of the caller's pool may be in use by kernels still
queued on the caller's stream.  Shown without a GPU: the library and the binding are replaced, and every
allocation is noted with the stream that was current."""
import contextlib
import types

import pytest
import torch

from learned_sparse_kv_b200 import build as lbuild
from learned_sparse_kv_b200 import lsa

B, K = 2, 4


class FakeStream:
    cuda_stream, device = 1234, torch.device("cpu")


@pytest.fixture(scope="module", autouse=True)
def built():
    lbuild.build()


@pytest.fixture
def calls(monkeypatch):
    """(kind, was the side stream current?) of every allocation and launch."""
    seen, now = [], []

    @contextlib.contextmanager
    def on(stream):
        now.append(stream)
        yield
        now.pop()

    class Lib:
        def __getattr__(self, name):
            if name.endswith("workspace_size"):
                return lambda *a: 512
            return lambda *a: seen.append((name, bool(now))) or 0

    class Native:
        def __getattr__(self, name):
            return lambda *a: seen.append((name, bool(now)))

    real = torch.empty
    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(cuda_stream=0))
    monkeypatch.setattr(torch, "empty", lambda *a, **k: seen.append(("empty", bool(now))) or real(*a, **k))
    monkeypatch.setattr(lsa, "_lib", Lib())
    monkeypatch.setattr(lsa, "_native", Native())
    monkeypatch.setattr(lsa, "_dev", lambda t, *a: t)
    return seen


def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def ints(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


CALLS = {
    "nmi_select": lambda L, **k: L.nmi_select(bf(B, 2, 8), bf(B, 2), bf(8, 8), ints(B + 1), 4, K, **k),
    "nmi_select_union": lambda L, **k: L.nmi_select_union([bf(B, 2, 8)], [bf(B, 2)], [bf(8, 8)], ints(B + 1), 4, K, **k),
    "query_encoder": lambda L, **k: L.query_encoder(bf(B, 16), bf(8, 16), bf(16, 8), bf(2, 16), 2, 8, **k),
    "select_baseline": lambda L, **k: L.select_baseline(0, ints(B), 4, K, **k),
    "topk": lambda L, **k: L.topk(bf(B, 2, 8), bf(B, 2), bf(4, 64, 8), ints(B, 4), ints(B, K), ints(B), ints(B), K, **k),
    "append_topk": lambda L, **k: L.append_topk(bf(B, 16), bf(B, 8), bf(4, 64, 16), ints(B), bf(B, 2, 8), bf(B, 2),
                                                bf(4, 64, 8), ints(B, 4), ints(B, K), ints(B), ints(B), K, **k),
    "topk_from_scores": lambda L, **k: L.topk_from_scores(torch.zeros(8), torch.zeros(B + 1, dtype=torch.int64), 8, K, **k),
    "sparse_decode": lambda L, **k: L.sparse_decode(bf(B, 2, 64), bf(4, 64, 64), bf(4, 64, 64), ints(B, 4), ints(B, K),
                                                    ints(B), ints(B), ints(B), 64, 64, 1.0, **k),
    "merge_attention": lambda L, **k: L.merge_attention(torch.zeros(2, B, 2, 64), torch.zeros(2, B, 2), **k),
    "plan_residency": lambda L, **k: L.plan_residency(ints(4), ints(4), ints(K), ints(1), 0, 4, 4, ints(4), ints(4),
                                                      ints(1), **k),
    "label_vote": lambda L, **k: L.label_vote(torch.zeros(2, 2, 4), 0.6, 1, 0, **k),
    "build_tables": lambda L, **k: L.build_tables(ints(B, 4), ints(B), ints(B), 8, 4, **k),
    "qk_norm_rope": lambda L, **k: L.qk_norm_rope(bf(1, 1, 64), None, ints(1), torch.zeros(32), **k),
    "read_q4": lambda L, **k: L.read_q4(torch.zeros(1, 1, 2304, dtype=torch.uint8), torch.zeros(4, dtype=torch.int64), **k),
    "sparse_decode_q4": lambda L, **k: L.sparse_decode_q4(bf(B, 2, 64), torch.zeros(4, 1, 2304, dtype=torch.uint8), None,
                                                          ints(B, 4), None, None, ints(B), ints(B), 64, 64, 1.0, **k),
}


@pytest.mark.parametrize("name", CALLS)
def test_allocations_and_launch_on_the_given_stream(calls, name):
    CALLS[name](lsa)
    assert calls and not any(side for _, side in calls)
    calls.clear()
    CALLS[name](lsa, stream=FakeStream())
    assert calls and all(side for _, side in calls), calls
