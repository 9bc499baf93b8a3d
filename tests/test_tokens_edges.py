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


def test_launches_of_2_to_the_32_threads_are_refused():
    """A grid holds fewer than 2^32 threads: 2^24 workgroups of 256 do not fit."""
    L = S.lib()
    # 4 tokens' pieces per workgroup: 2^22 tokens of 16 (combine) or 2^23 of 8 (gather) pieces
    assert L.route_combine(1 << 22, 1, 8192, 0, P, None, P, 8192, P, 8192, None) == OVERFLOW
    assert L.route_gather(1 << 23, 1, 16384, 1, P, None, P, 16384, P, 16384, None) == OVERFLOW
    assert L.route_combine_grad(1 << 24, 1, 8, 2, P, 8, P, 8, P, None, P, 8, P, None) == OVERFLOW
    # 262145 tiles of 64 pieces of 512 columns
    n, n_out = 1 << 22, 32768
    tiles = S.route_tile_count(n, 1)
    assert L.lora_apply(n, 8, n_out, 1, 8, None, None, P, P, 0, P, P, P, tiles, P, 8, None, 0, P, 2, n_out, P,
                        S.lora_workspace_size(n, 8), None) == OVERFLOW
    # 512 groups of 64 row blocks and 512 token tiles
    assert L.macko_spmm(512, 4096, 256, 4, P, P, P, P, P, 131072, 1.0, P, 256, 0.0, P, 2, 4096, None, 0, None) == OVERFLOW
