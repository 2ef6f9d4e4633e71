"""The window oracle pinned on CPU: torch attention, autograd, differences, brute force; and
the argument checks of the window calls that need no GPU."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import window_oracle as WO
from spatial_sparse_attention_ssa_b200 import ssa

RNG = np.random.default_rng


def _problem(seed, n=23, hq=4, hkv=2, d=8, m=3, count=4):
    r = RNG(seed)
    coords = r.integers(0, 3 * m, (n, 3))
    ids = r.integers(0, count, n)
    q, dout = r.standard_normal((2, n, hq, d))
    k, v = r.standard_normal((2, n, hkv, d))
    return coords, ids, q, k, v, dout


def _torch_window(ids, count, q, k, v, scale, off=None, table=None):
    n, hq, d = q.shape
    g = hq // k.shape[1]
    same = torch.from_numpy(np.asarray(ids)[:, None] == np.asarray(ids)[None])
    kk, vv = (x.repeat_interleave(g, 1) for x in (k, v))
    s = torch.einsum("ihd,jhd->hij", q, kk) * scale
    if table is not None:
        s = s + table[:, off]
    p = torch.softmax(s.masked_fill(~same, float("-inf")), -1)
    return torch.einsum("hij,jhd->ihd", p, vv), p


@pytest.mark.parametrize("bias", [False, True])
def test_window_against_dense_attention_and_autograd(bias):
    m = 3
    coords, ids, q, k, v, dout = _problem(1, m=m)
    table = RNG(2).standard_normal((4, 27)) if bias else None
    axis = np.array([0, 0, 1, 2, 2])
    bucket = ((axis[:, None, None] * 3 + axis[None, :, None]) * 3 + axis[None, None, :]).reshape(-1)
    r = WO.window(ids, 4, q, k, v, dout, 0.4, coords, m, table, bucket if bias else None)
    t = [torch.tensor(x, requires_grad=True) for x in (q, k, v)]
    tab = torch.tensor(table, requires_grad=True) if bias else None
    cm = coords % m
    o3 = cm[:, None] - cm[None] + m - 1
    off = torch.from_numpy(bucket[(o3[..., 0] * 5 + o3[..., 1]) * 5 + o3[..., 2]])
    out, _ = _torch_window(ids, 4, *t, 0.4, off, tab)
    np.testing.assert_allclose(r["out"][0], out.detach().numpy(), atol=1e-12)
    out.backward(torch.from_numpy(dout))
    for name, x in zip(("dq", "dk", "dv"), t):
        np.testing.assert_allclose(r[name][0], x.grad.numpy(), atol=1e-12)
    if bias:
        np.testing.assert_allclose(r["dbias"][0], tab.grad.numpy(), atol=1e-12)


def test_window_gradients_against_differences():
    m = 3
    coords, ids, q, k, v, dout = _problem(3, n=9, count=2, m=m)
    table = RNG(4).standard_normal((4, 125))
    f = lambda **kw: float((WO.window(ids, 2, *(kw.get(x, y) for x, y in (("q", q), ("k", k), ("v", v))), dout, 0.5,  # noqa: E731
                                      coords, m, kw.get("table", table))["out"][0] * dout).sum())
    r = WO.window(ids, 2, q, k, v, dout, 0.5, coords, m, table)
    h, rng = 1e-5, RNG(5)
    for name, x, grad in (("q", q, "dq"), ("k", k, "dk"), ("v", v, "dv"), ("table", table, "dbias")):
        step = rng.standard_normal(x.shape)
        num = (f(**{name: x + h * step}) - f(**{name: x - h * step})) / (2 * h)
        assert abs(num - float((r[grad][0] * step).sum())) < 1e-7, name


def test_barred_rows_give_zeros():
    """A bias of minus infinity in every bucket of a row: zeros, lse minus infinity, no gradient."""
    m = 2
    coords = np.array([[0, 0, 0], [1, 1, 1], [0, 1, 0]])
    q = k = v = dout = RNG(0).standard_normal((3, 1, 4))
    r = WO.window(np.zeros(3, int), 1, q, k, v, dout, 1.0, coords, m, np.full((1, 27), -np.inf))
    for name in ("out", "dq", "dk", "dv", "dbias"):
        assert np.all(r[name][0] == 0), name
    assert np.all(np.isneginf(r["lse"][0]))


def test_diff_against_autograd_and_differences():
    _, ids, q, k, v, dout = _problem(7, hq=8, hkv=4)
    lam = 0.3 * RNG(8).standard_normal((4, 4, 8))
    r = WO.diff(ids, 4, q, k, v, dout, 0.3, lam, 0.6)
    t = [torch.tensor(x, requires_grad=True) for x in (q, k, v, lam)]
    n = q.shape[0]
    vv = t[2].reshape(n, 2, 16)
    o1, _ = _torch_window(ids, 4, t[0][:, 0::2], t[1][:, 0::2], vv, 0.3)
    o2, _ = _torch_window(ids, 4, t[0][:, 1::2], t[1][:, 1::2], vv, 0.3)
    lamv = torch.exp((t[3][0] * t[3][1]).sum(-1)) - torch.exp((t[3][2] * t[3][3]).sum(-1)) + 0.6
    out = (o1 - lamv[None, :, None] * o2).reshape(q.shape)
    np.testing.assert_allclose(r["out"][0], out.detach().numpy(), atol=1e-12)
    out.backward(torch.from_numpy(dout))
    for name, x in zip(("dq", "dk", "dv", "dlam"), t):
        np.testing.assert_allclose(r[name][0], x.grad.numpy(), atol=1e-12)
    f = lambda x: float((WO.diff(ids, 4, q, k, v, dout, 0.3, x, 0.6)["out"][0] * dout).sum())  # noqa: E731
    step, h = RNG(9).standard_normal(lam.shape), 1e-5
    assert abs((f(lam + h * step) - f(lam - h * step)) / (2 * h) - float((r["dlam"][0] * step).sum())) < 1e-7


def test_act8_is_the_nearest_code_of_the_smallest_step():
    x = RNG(11).standard_normal((40, 32)) * 10.0 ** RNG(12).uniform(-6, 6, (40, 1))
    x[3] = 0
    x[4, :] = 127.0
    x[5, :] = 127.0001
    codes, scale = WO.act8(x)
    assert scale[3] == 1 and scale[4] == 1 and scale[5] == 2
    for i in range(40):
        if i == 3:
            continue
        top = np.abs(x[i]).max()
        assert 127 * scale[i] >= top > 127 * scale[i] / 2 and np.log2(scale[i]) % 1 == 0
        assert np.all(np.abs(codes[i] * scale[i] - x[i]) <= scale[i] / 2)
    # every value is exact in bf16: 7 bits times a power of two
    val = torch.from_numpy(codes * scale[:, None]).to(torch.float32)
    assert torch.equal(val.to(torch.bfloat16).float(), val)


def test_log_buckets():
    bucket, nb = ssa.window_log_buckets(8, device="cpu")
    assert nb == 343 and bucket.shape == (15 ** 3,) and bucket.dtype == torch.int32
    name = lambda o: 0 if o == 0 else int(np.sign(o)) * (int(np.log2(abs(o))) + 1)  # noqa: E731
    seen = {}
    for i in range(15):
        for j in range(15):
            for k in range(15):
                key = tuple(name(x - 7) for x in (i, j, k))
                assert seen.setdefault(key, int(bucket[(i * 15 + j) * 15 + k])) == int(bucket[(i * 15 + j) * 15 + k])
    assert sorted(seen.values()) == list(range(343))
    assert ssa.window_log_buckets(1, device="cpu")[1] == 1


# ---------------------------------------------------------------------------
# refusals on the host
# ---------------------------------------------------------------------------


def _ok():
    return dict(p=ssa.WindowParams(32, 2, 64, ssa.DTYPE_BF16, 0.0), plan=ssa.WinPlanC(16, 16, 100, 10, 8),
                bias=ssa.WindowBiasC(16, None, 15 ** 3), q=16, k=16, v=16, out=16)


def _forward(**kw):
    a = dict(_ok(), **kw)
    return ssa.lib().ssa_window_forward(a["p"], a["plan"], a["bias"], a["q"], a["k"], a["v"], a["out"], None, None)


def _backward(**kw):
    a = dict(_ok(), act8=None, dout=16, dq=16, dk=16, dv=16, dbias=16, ws=256, ws_bytes=16)
    a.update(kw)
    return ssa.lib().ssa_window_backward(a["p"], a["plan"], a["bias"], a["q"], a["k"], a["v"], a["act8"], a["dout"],
                                         a["dq"], a["dk"], a["dv"], a["dbias"], a["ws"], a["ws_bytes"], None)


P = ssa.WindowParams
BAD_PARAMS = [(P(0, 1, 64, 0, 0.0), 1), (P(32, 0, 64, 0, 0.0), 1), (P(32, 3, 64, 0, 0.0), 1), (P(32, 2, 48, 0, 0.0), 2),
              (P(32, 2, 64, 2, 0.0), 1), (P(32, 2, 64, 0, -1.0), 1), (P(32, 2, 64, 0, float("nan")), 1),
              (P(32, 2, 64, 0, float("inf")), 1), (P(1 << 17, 2, 64, 0, 0.0), 2), (None, 1)]
L = ssa.WinPlanC
BAD_PLANS = [L(16, 16, -1, 10, 8), L(16, 16, 100, 0, 8), L(16, 16, 100, 101, 8), L(None, 16, 100, 10, 8),
             L(16, None, 100, 10, 8), L(8, 16, 100, 10, 8), L(16, 24, 100, 10, 8), L(16, 16, 100, 10, 17),
             L(16, 16, 100, 10, -1), L(16, 16, (1 << 31) - 1, 10, 8), None]


@pytest.mark.parametrize("p,code", BAD_PARAMS)
def test_window_calls_refuse_bad_heads(p, code):
    assert _forward(p=p) == code and _backward(p=p) == code
    assert ssa.lib().ssa_window_workspace_size(ssa.OP_WINDOW_BACKWARD, p, _ok()["plan"]) == 0


@pytest.mark.parametrize("i", range(len(BAD_PLANS)))
def test_window_calls_refuse_bad_plans(i):
    assert _forward(plan=BAD_PLANS[i]) == 1 and _backward(plan=BAD_PLANS[i]) == 1


def test_window_calls_refuse_bad_arguments():
    B = ssa.WindowBiasC
    for bias in (B(None, None, 15 ** 3), B(16, None, 343), B(16, None, 0), B(16, 16, 0)):
        assert _forward(bias=bias) == 1 and _backward(bias=bias) == 1
    assert _forward(plan=L(16, 16, 100, 10, 0)) == 1      # a bias needs a plan with codes
    for x in ("q", "k", "v", "out"):
        assert _forward(**{x: None}) == 1 and _forward(**{x: 8}) == 1
    for x in ("q", "k", "v", "dout", "dq", "dk", "dv"):
        assert _backward(**{x: None}) == 1 and _backward(**{x: 8}) == 1
    assert _backward(ws=None) == 1 and _backward(ws=128) == 1
    assert _backward() == 3                               # 16 bytes of workspace
    assert _backward(bias=None) == 1                      # dbias without a bias
    A = ssa.Act8C
    for bad in ((None, 16), (16, None), (8, 16)):
        assert _backward(act8=(A * 3)((16, 16), bad, (16, 16))) == 1
    assert _forward(plan=L(None, None, 0, 0, 8)) == 0     # nothing to do


def test_diff_calls_refuse_bad_arguments():
    lib, ok = ssa.lib(), _ok()

    def fwd(p=ok["p"], plan=ok["plan"], lam=16, init=0.5, q=16):
        return lib.ssa_diff_forward(p, plan, lam, init, q, 16, 16, 16, None)

    def bwd(p=ok["p"], lam=16, init=0.5, dlam=16, ws=256, n=16):
        return lib.ssa_diff_backward(p, ok["plan"], lam, init, 16, 16, 16, None, 16, 16, 16, 16, dlam, ws, n, None)
    for p, code in BAD_PARAMS + [(P(32, 1, 64, 0, 0.0), 1), (P(3, 3, 64, 0, 0.0), 1), (P(32, 2, 128, 0, 0.0), 2)]:
        assert fwd(p=p) == code and bwd(p=p) == code
    for plan in BAD_PLANS:
        assert fwd(plan=plan) == 1
    assert fwd(lam=None) == 1 and fwd(init=float("nan")) == 1 and fwd(q=None) == 1 and fwd(q=8) == 1
    assert bwd(lam=None) == 1 and bwd(init=float("inf")) == 1 and bwd(dlam=None) == 1 and bwd(ws=1) == 1 and bwd() == 3
    assert fwd(plan=L(None, None, 0, 0, 0)) == 0


def test_plan_and_act8_refuse_bad_arguments():
    lib = ssa.lib()
    part = ssa.Partition(16, 16, 16, 16, 16, 10)

    def plan(coords=16, n=100, m=8, win=part, pl=None):
        return lib.ssa_window_plan(coords, n, m, win, pl or L(16, 16, 0, 0, 0), None)
    assert plan(n=-1) == 1 and plan(m=0) == 1 and plan(m=17) == 2 and plan(win=None) == 1
    assert plan(n=5) == 1                                 # more cells than tokens
    assert plan(win=ssa.Partition(16, 16, 16, 16, 16, 0)) == 1
    assert plan(pl=L(None, 16, 0, 0, 0)) == 1 and plan(pl=L(16, 8, 0, 0, 0)) == 1
    out = L(None, None, 7, 7, 7)
    assert plan(n=0, win=ssa.Partition(None, None, 16, 16, None, 0), pl=out) == 0 and (out.n, out.count, out.m) == (0, 0, 8)
    for fn in (lib.ssa_act8_pack, lib.ssa_act8_unpack):
        assert fn(2, 10, 64, 16, 16, 16, None) == 1 and fn(0, -1, 64, 16, 16, 16, None) == 1
        assert fn(0, 10, 48, 16, 16, 16, None) == 2 and fn(0, 10, 256, 16, 16, 16, None) == 2
        assert fn(0, 10, 64, None, 16, 16, None) == 1 and fn(0, 10, 64, 16, None, 16, None) == 1
        assert fn(0, 0, 64, None, None, None, None) == 0
    assert lib.ssa_act8_pack(0, 10, 64, 8, 16, 16, None) == 1 and lib.ssa_act8_pack(0, 10, 64, 16, 8, 16, None) == 1


def test_workspace_sizes():
    lib, ok = ssa.lib(), _ok()
    n = lib.ssa_window_workspace_size(ssa.OP_WINDOW_BACKWARD, ok["p"], ok["plan"])
    assert n >= 2 * 4 * 32 * 100 + 4 * 32 * 15 ** 3
    assert 2 * 4 * 32 * 100 <= lib.ssa_window_workspace_size(ssa.OP_DIFF_BACKWARD, ok["p"], ok["plan"]) < n
    assert lib.ssa_window_workspace_size(ssa.OP_FORWARD, ok["p"], ok["plan"]) == 0


def test_binding_refuses_shapes_types_and_devices():
    """Found before any call of the library."""
    e = lambda *s, dt=torch.bfloat16: torch.empty(*s, dtype=dt)  # noqa: E731
    p = ssa.make_window_params(4, 2, 32, torch.bfloat16)
    plan = ssa.WindowPlan(e(10, 2, dt=torch.int32), e(3, 4, dt=torch.int32), 10, 3, 4)
    q, k = e(10, 4, 32), e(10, 2, 32)
    with pytest.raises(ValueError):
        ssa.make_window_params(4, 2, 32, torch.float16)
    with pytest.raises(ValueError, match="k must be"):
        ssa.ssa_window_forward(p, plan, q, q, k)
    with pytest.raises(ValueError, match="q must be"):
        ssa.ssa_window_forward(p, plan, q.float(), k, k)
    with pytest.raises(ValueError, match="bias.table"):
        ssa.ssa_window_forward(p, plan, q, k, k, bias=ssa.WindowBias(e(3, 343, dt=torch.float32)))
    with pytest.raises(ValueError, match="bias.bucket"):
        ssa.ssa_window_forward(p, plan, q, k, k, bias=ssa.WindowBias(e(4, 9, dt=torch.float32), e(9, dt=torch.int32)))
    with pytest.raises(ValueError, match="CUDA"):
        ssa.ssa_window_forward(p, plan, q, k, k)
    with pytest.raises(ValueError, match="dout must be"):
        ssa.ssa_window_backward(p, plan, q, k, k, k)
    with pytest.raises(ValueError, match="dbias without"):
        ssa.ssa_window_backward(p, plan, q, k, k, q, dbias=e(1, dt=torch.float32))
    with pytest.raises(ValueError, match="lam must be"):
        ssa.ssa_diff_forward(p, plan, q, k, k, e(4, 4, 32, dt=torch.float32), 0.5)
    with pytest.raises(ValueError, match="codes"):
        a = ssa.Act8(e(10, 4, 32), e(10, 4, dt=torch.float32))
        ssa.ssa_window_backward(p, plan, a, a, a, q)
    with pytest.raises(ValueError):
        ssa.ssa_act8_pack(q.to(torch.float16))
    with pytest.raises(ValueError):
        ssa.ssa_act8_unpack(ssa.Act8(q, e(10, 4, dt=torch.float32)), torch.float32)
