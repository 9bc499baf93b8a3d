"""Edges of the many-token operators' calls that show without a GPU: what an
empty call needs, launches that do not fit, and where the binding allocates."""
import contextlib

import pytest

import sparse_matrix_vector_amd as S

OK, VALUE, OVERFLOW, UNSUPPORTED = 0, 1, 4, 5
P = 4096                                     # a pointer that is aligned and never followed


def test_no_tokens_need_no_workspace():
    L = S.lib()
    for r in (1, 16, 128):
        assert L.lora_apply(0, 64, 32, 3, r, None, None, P, P, 0, None, P, None, 0, None, 64, None, 32, None, 2, 32,
                            None, 0, None) == OK


def test_macko_plan_is_allocated_on_the_stream_that_fills_it(monkeypatch):
    """A block of the current stream's pool could still be in use by that stream's earlier work."""
    torch = pytest.importorskip("torch")
    from sparse_matrix_vector_amd import tokens
    inside, seen = [], []

    @contextlib.contextmanager
    def scope(stream, device):
        inside.append(stream)
        yield
        inside.pop()

    def empty(*a, **k):
        seen.append(("alloc", list(inside)))
        return torch.zeros(*a, **{**k, "device": "cpu"})

    monkeypatch.setattr(tokens, "_stream_scope", scope)
    monkeypatch.setattr(tokens, "macko_spmm_plan", lambda *a: seen.append(("fill", a[5])))
    monkeypatch.setattr(tokens.torch, "empty", empty)
    side = object()
    S.MackoMatrix(3, 64, torch.zeros(4, dtype=torch.int32), None, None, stream=side)
    assert seen == [("alloc", [side]), ("fill", side)]
    seen.clear()
    S.MackoMatrix(3, 64, torch.zeros(4, dtype=torch.int32), None, None)
    assert seen == [("alloc", [None]), ("fill", None)]          # the current stream
