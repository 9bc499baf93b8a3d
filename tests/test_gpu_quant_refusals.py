"""Arguments that are no tensors, or no weights, in the calls of 4-bit weights, expert
layers and embeddings, are refused."""
import pytest

torch = pytest.importorskip("torch")
S = pytest.importorskip("sparse_matrix_vector_amd")

pytestmark = pytest.mark.gpu

OTHERS = ([1, 2, 3, 4], 7, "keys", object())


def _calls():
    """{name: (function, its arguments, those that are tensors or weights, those that may be None)}."""
    half = lambda *n: torch.zeros(*n, dtype=torch.float16, device="cuda")  # noqa: E731
    ints = lambda *n: torch.zeros(*n, dtype=torch.int32, device="cuda")  # noqa: E731
    ws = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda")  # noqa: E731
    gu, dn = S.Q4Matrix.quantize(half(2, 80, 72)), S.Q4Matrix.quantize(half(2, 72, 40))
    one = S.Q4Matrix.quantize(half(80, 72))
    codes, scales = ints(80, 16), half(80, 1)
    return {
        "quantize": (S.q4_quantize, dict(w=half(80, 72), codes=codes, scales=scales, zeros=None), ("w", "codes", "scales", "zeros"),
                     ("zeros",)),
        "tiles": (S.q4_tiles, dict(n_rows=80, n_cols=72, codes=codes, scales=scales, zeros=None, tiles=ws(S.q4_tiles_size(80, 72))),
                  ("codes", "scales", "zeros", "tiles"), ("zeros", "tiles")),
        "Q4Matrix": (S.Q4Matrix, dict(n_rows=80, n_cols=72, codes=codes, scales=scales, zeros=None), ("codes", "scales", "zeros"),
                     ("zeros",)),
        "Q4Matrix.quantize": (S.Q4Matrix.quantize, dict(w=half(80, 72)), ("w",), ()),
        "matmul": (S.q4_matmul, dict(n_rows=80, n_cols=72, tiles=one.tiles, alpha=1.0, x=half(4, 72), beta=0.0, y=half(4, 80),
                                     workspace=ws(16)), ("tiles", "x", "y", "workspace"), ("workspace", "tiles")),
        "apply": (one.apply, dict(x=half(4, 72), y=half(4, 80), workspace=ws(16)), ("x", "y", "workspace"), ("workspace",)),
        "moe": (S.moe_apply, dict(keys=ints(4, 2), weights=torch.zeros(4, 2, device="cuda"), gate_up=gu, down=dn, x=half(4, 72),
                                  y=half(4, 72), workspace=ws(S.moe_workspace_size(4, 2, 72, 40))),
                ("keys", "weights", "gate_up", "down", "x", "y", "workspace"), ("weights", "workspace")),
        "lookup": (S.embed_lookup, dict(ids=ints(4), table=half(9, 16), y=half(4, 16)), ("ids", "table", "y"), ()),
        "grad": (S.embed_grad, dict(ids=ints(4), dy=half(4, 16), dtable=torch.zeros(9, 16, device="cuda"),
                                    workspace=ws(S.embed_grad_workspace_size(4, 9, 16))), ("ids", "dy", "dtable", "workspace"),
                 ("workspace",)),
    }


@pytest.mark.parametrize("name", ["quantize", "tiles", "Q4Matrix", "Q4Matrix.quantize", "matmul", "apply", "moe", "lookup", "grad"])
def test_arguments_that_are_no_tensors(name):
    call, args, tensors, optional = _calls()[name]
    call(**args)
    for arg in tensors:
        for bad in OTHERS:
            with pytest.raises(TypeError):
                call(**{**args, arg: bad})
        if arg not in optional:                              # as elsewhere, "is required" where only the pointer is asked for
            with pytest.raises((TypeError, ValueError)):
                call(**{**args, arg: None})
