"""The MACKO product of many tokens with workspaces of other sizes than its own:
a larger batch's, room for x alone, none."""
import pytest

torch = pytest.importorskip("torch")
S = pytest.importorskip("sparse_matrix_vector_amd")

import op_refs as R  # noqa: E402
from test_gpu_macko_spmm import _matrix, _weight, _x  # noqa: E402

pytestmark = pytest.mark.gpu

# rows, columns, groups, batches whose own workspaces are larger than that of the last one
BATCHES = [(1024, 1024, 1, [1000, 700, 40, 5, 1, 1026]), (512, 4096, 1, [500, 256, 33, 17, 501]), (512, 1024, 4, [512, 300, 64, 513])]


def _check(m, dense, x, y, off, what):
    for g in range(m.n_groups):
        a, b = (0, x.shape[0]) if off is None else off[g:g + 2]
        ref, bound = R.spmm(dense[g * m.n_rows:(g + 1) * m.n_rows], x[a:b], 1.0, 0.0, None, y.dtype)
        R.check(y[a:b], ref, bound, what)


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("shape", BATCHES)
def test_a_larger_batchs_workspace_serves_smaller_ones(shape, i8):
    rows, cols, groups, batches = shape
    w = _weight(groups * rows, cols, "0.8", 4, 5, i8)
    m = _matrix(w, rows, cols, 4, groups)
    last = max(batches)
    size = S.macko_spmm_workspace_size(groups, rows, cols, last)
    assert max(S.macko_spmm_workspace_size(groups, rows, cols, n) for n in batches) > size
    buf = torch.full((size + 256,), 77, dtype=torch.uint8, device="cuda")
    xb = _x(last, cols + 1, 6)
    for n in batches:
        off = None if groups == 1 else [0, n // 3, n // 3, n - n // 4, n]
        dev_off = None if off is None else torch.tensor(off, dtype=torch.int32, device="cuda")
        for x in (xb[:n, :cols].contiguous(), xb[:n, 1:]):              # as it is, and copied first
            outs = []
            # its own workspace, the last batch's, and the least of all
            for ws in (m.workspace(n), buf[:size], buf[:n * cols * 2] if x.stride(0) != cols else None):
                y = torch.full((n, rows), float("nan"), device="cuda")
                args = (rows, cols, m.mrow_ptr, m.codes, m.vals) + ((m.row_scale,) if i8 else ())
                (S.macko_spmm_i8 if i8 else S.macko_spmm)(*args, m.plan, 1.0, x, 0.0, y, ws, dev_off)
                _check(m, w[4], x, y, off, f"{shape} {n}")
                outs.append(y)
            assert torch.equal(outs[0], m.apply(x, torch.empty_like(y), tok_offsets=dev_off))
        assert (buf[size:] == 77).all()


def test_plan_of_a_side_stream_has_memory_of_that_stream():
    rows, cols = 40, 300
    w = _weight(rows, cols, "0.5", 4, 3)
    m = _matrix(w, rows, cols, 4)
    size = m.plan.numel()
    x = _x(9, cols, 1)
    want = m.apply(x, torch.empty(9, rows, device="cuda"))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        freed = torch.empty(size, dtype=torch.uint8, device="cuda")
        block = freed.data_ptr()
        del freed
        other = S.MackoMatrix(rows, cols, m.mrow_ptr, m.codes, m.vals, stream=stream)
        assert other.plan.data_ptr() != block
        side.synchronize()
        assert torch.equal(other.apply(x, torch.empty(9, rows, device="cuda")), want)
