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


N, HQ, HKV, D = 100, 4, 2, 32
Q, KV = N * HQ * D * 2, N * HKV * D * 2
AT = 1 << 30          # no call gets far enough to read there: there is no device, or the call is refused
A = {x: AT + i * (1 << 20) for i, x in enumerate(("q", "k", "v", "out", "lse", "dout", "dq", "dk", "dv", "lam", "dlam", "ws"))}
REFUSED = 1


def _fwd(op, **kw):
    a, p, plan = dict(A, **kw), ssa.WindowParams(HQ, HKV, D, ssa.DTYPE_BF16, 0.0), ssa.WinPlanC(16, 16, N, 10, 0)
    if op == "window":
        return ssa.lib().ssa_window_forward(p, plan, None, a["q"], a["k"], a["v"], a["out"], a["lse"], None)
    return ssa.lib().ssa_diff_forward(p, plan, a["lam"], 0.5, a["q"], a["k"], a["v"], a["out"], None)


def _bwd(op, codes=False, **kw):
    a, p, plan = dict(A, **kw), ssa.WindowParams(HQ, HKV, D, ssa.DTYPE_BF16, 0.0), ssa.WinPlanC(16, 16, N, 10, 0)
    a8 = (ssa.Act8C * 3)(*((a[x], 16) for x in "qkv")) if codes else None
    tail = (a["q"], a["k"], a["v"], a8, a["dout"], a["dq"], a["dk"], a["dv"])
    if op == "window":
        return ssa.lib().ssa_window_backward(p, plan, None, *tail, None, a["ws"], 1 << 30, None)
    return ssa.lib().ssa_diff_backward(p, plan, a["lam"], 0.5, *tail, a["dlam"], a["ws"], 1 << 30, None)


@pytest.mark.skipif(torch.cuda.is_available(), reason="the calls that pass would read the addresses")
@pytest.mark.parametrize("op", ["window", "diff"])
def test_outputs_that_overlap_are_refused(op):
    assert _fwd(op) != REFUSED and _bwd(op) != REFUSED and _bwd(op, codes=True) != REFUSED
    assert _fwd(op, out=A["q"]) != REFUSED and _bwd(op, dk=A["k"], dv=A["v"]) != REFUSED
    for x in ("k", "v"):
        assert _fwd(op, out=A[x]) == REFUSED and _fwd(op, out=A[x] + KV - 16) == REFUSED
        assert _fwd(op, out=A[x] - Q + 16) == REFUSED and _fwd(op, out=A[x] + KV) != REFUSED
    assert _fwd(op, out=A["q"] + 16) == REFUSED
    for x in ("q", "k", "v", "dout"):
        assert _bwd(op, dq=A[x]) == REFUSED and _bwd(op, codes=True, dq=A[x]) == REFUSED
    for x in ("dk", "dv"):
        assert _bwd(op, **{x: A["dout"]}) == REFUSED and _bwd(op, **{x: A["dq"] + Q - 16}) == REFUSED
        assert _bwd(op, **{x: A["q"]}) == REFUSED and _bwd(op, codes=True, **{x: A[x[1]]}) == REFUSED
    assert _bwd(op, dk=A["v"]) == REFUSED and _bwd(op, dv=A["dk"]) == REFUSED and _bwd(op, dk=A["k"] + 16) == REFUSED
    if op == "window":
        assert _fwd(op, lse=A["out"]) == REFUSED and _fwd(op, lse=A["q"]) == REFUSED
    else:
        assert _bwd(op, dlam=A["lam"]) == REFUSED
