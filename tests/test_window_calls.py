"""The window, differential and 8-bit calls from the caller's side: sizes and arguments, no GPU needed."""
import pytest
import torch

from spatial_sparse_attention_ssa_b200 import ssa

PLAN = ssa.WinPlanC(16, 16, 131072, 2800, 8)


@pytest.mark.parametrize("ops", [(ssa.OP_WINDOW_BACKWARD, ssa.OP_WINDOW_BACKWARD_TENSORS),
                                 (ssa.OP_DIFF_BACKWARD, ssa.OP_DIFF_BACKWARD_TENSORS)])
def test_workspace_of_calls_without_checkpoints_holds_no_copies(ops):
    """131072 tokens, 32/2 heads of 64: the bf16 copies of Q, K, V are 604 MB, the rest is below 100 MB."""
    lib = ssa.lib()
    for dtype in (ssa.DTYPE_BF16, ssa.DTYPE_F32):
        p = ssa.WindowParams(32, 2, 64, dtype, 0.0)
        full, tensors = (lib.ssa_window_workspace_size(op, p, PLAN) for op in ops)
        # arrays start on 256 bytes, empty ones too
        assert abs(full - tensors - (2 * 131072 * 64 * (32 + 2 + 2) if dtype == ssa.DTYPE_BF16 else 0)) < 3 * 512
        assert 0 < tensors < 100 << 20
    assert lib.ssa_window_workspace_size(ops[1], ssa.WindowParams(32, 3, 64, 0, 0.0), PLAN) == 0


def test_params_made_as_a_struct_and_changed_later():
    """The type that the binding checks is the one that the library reads."""
    e = lambda *s, dt=torch.bfloat16: torch.empty(*s, dtype=dt)  # noqa: E731
    plan = ssa.WindowPlan(e(10, 2, dt=torch.int32), e(4, 4, dt=torch.int32), 10, 3, 4)
    q, k = e(10, 4, 32), e(10, 2, 32)
    for p in (ssa.WindowParams(4, 2, 32, ssa.DTYPE_F32, 0.0), ssa.make_window_params(4, 2, 32, torch.bfloat16)):
        p.dtype = ssa.DTYPE_BF16
        with pytest.raises(ValueError, match="CUDA"):        # types and shapes are right
            ssa.ssa_window_forward(p, plan, q, k, k)
        p.dtype = ssa.DTYPE_F32
        with pytest.raises(ValueError, match="q must be"):
            ssa.ssa_window_forward(p, plan, q, k, k)
        with pytest.raises(ValueError, match="dout must be"):
            ssa.ssa_window_backward(p, plan, q.float(), k.float(), k.float(), q)
        p.dtype = 7
        with pytest.raises(ValueError, match="dtype"):
            ssa.ssa_window_forward(p, plan, q, k, k)


def test_partitions_whose_arrays_have_other_sizes_are_refused():
    e = lambda *s, dt=torch.int32: torch.empty(*s, dtype=dt)  # noqa: E731
    bins = lambda **kw: ssa.Bins(**dict(dict(id=e(10), perm=e(10), ptr=e(11), cu=e(2), key=e(10, 3), count=4), **kw))  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        ssa.ssa_window_plan(e(10, 3), bins(), 4)
    with pytest.raises(ValueError, match="win.id"):
        ssa.ssa_window_plan(e(10, 3), bins(id=e(9)), 4)
    with pytest.raises(ValueError, match="win.perm"):
        ssa.ssa_window_plan(e(10, 3), bins(perm=e(10, dt=torch.int64)), 4)
    with pytest.raises(ValueError, match="win.ptr"):
        ssa.ssa_window_plan(e(10, 3), bins(ptr=e(4)), 4)
    with pytest.raises(ValueError, match="coords"):
        ssa.ssa_window_plan(e(11, 3), bins(), 4)
