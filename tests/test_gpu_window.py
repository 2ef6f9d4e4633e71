"""Attention inside the cells on the GPU against the fp64 oracle: window attention with a learned
relative position bias, differential attention, 8-bit checkpoints and the backward from them.

Tolerances are the oracle's per-element bounds (oracle/window_oracle.py): storage roundings of
the softmax weights, of dS and of the results (bf16: 2^-8 each, fp32 results 2^-24), fp32
roundings of scores, exponentials and sums.  TINY covers products that fall under the smallest
normal fp32 number (ex2.approx flushes them to zero).
"""
import numpy as np
import pytest
import torch

from oracle import window_oracle as WO
from spatial_sparse_attention_ssa_b200 import ssa

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 0.0}
U_OUT = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TINY = 1e-30


def shell(seed, n, seqs=1, r=10):
    """Voxels of spheres' surfaces, n per sequence at most, int32 [N, 3] and cu."""
    rng = np.random.default_rng(seed)
    out, cu = [], [0]
    for _ in range(seqs):
        u = rng.standard_normal((6 * n + 20, 3))
        x = np.floor(u / np.linalg.norm(u, axis=1, keepdims=True) * r + 1.3 * r + 1).astype(np.int32)
        x = np.unique(x, axis=0)
        x = x[np.sort(rng.permutation(len(x))[:n])]
        out.append(x)
        cu.append(cu[-1] + len(x))
    return np.concatenate(out), np.array(cu, np.int32)


def dense(seed, n, side):
    rng = np.random.default_rng(seed)
    key = np.sort(rng.permutation(side ** 3)[:n])
    return np.stack([key // side ** 2, key // side % side, key % side], 1).astype(np.int32), np.array([0, n], np.int32)


class Problem:
    def __init__(self, coords, cu, m, hq, hkv, d, dtype, seed=0, bias=None, std=1.0):
        rng = np.random.default_rng(seed)
        self.m, self.hq, self.hkv, self.d, self.dtype = m, hq, hkv, d, dtype
        n = len(coords)
        self.np_coords = coords
        self.coords = torch.from_numpy(np.ascontiguousarray(coords)).cuda()
        self.cu = torch.from_numpy(cu).cuda()
        _, self.win = ssa.ssa_bin(self.coords, self.cu, 1024, m, m)
        f = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(dtype).cuda()  # noqa: E731
        self.q, self.dout = std * f(n, hq, d), f(n, hq, d)
        self.k, self.v = f(n, hkv, d), f(n, hkv, d)
        self.lam = torch.from_numpy((0.2 * rng.standard_normal((4, max(hq // 2, 1), d))).astype(np.float32)).cuda()
        self.p = ssa.make_window_params(hq, hkv, d, dtype)
        self.bias = None
        if bias == "offset":
            self.bias = ssa.WindowBias(torch.from_numpy(rng.standard_normal((hq, (2 * m - 1) ** 3)).astype(np.float32)).cuda())
        elif bias == "log":
            bucket, nb = ssa.window_log_buckets(m)
            self.bias = ssa.WindowBias(torch.from_numpy(rng.standard_normal((hq, nb)).astype(np.float32)).cuda(), bucket)
        self.plan = ssa.ssa_window_plan(self.coords if m <= ssa.WINDOW_MAX_EDGE else None, self.win, m)

    def np64(self, x):
        return x.double().cpu().numpy()

    def ref_window(self, q=None, k=None, v=None, ids=None):
        b = self.bias
        return WO.window(self.win.id.cpu().numpy() if ids is None else ids, self.win.count,
                         *(self.np64(x) for x in (self.q if q is None else q, self.k if k is None else k,
                                                  self.v if v is None else v, self.dout)),
                         1 / np.sqrt(self.d), self.np_coords, self.m, self.np64(b.table) if b else None,
                         b.bucket.cpu().numpy() if b and b.bucket is not None else None,
                         u=U[self.dtype], u_out=U_OUT[self.dtype])

    def ref_diff(self, q=None, k=None, v=None):
        return WO.diff(self.win.id.cpu().numpy(), self.win.count,
                       *(self.np64(x) for x in (self.q if q is None else q, self.k if k is None else k,
                                                self.v if v is None else v, self.dout)),
                       1 / np.sqrt(self.d), self.np64(self.lam), 0.5, u=U[self.dtype], u_out=U_OUT[self.dtype])


def check(got, ref, name):
    value, bound = ref[name]
    g = got.double().cpu().numpy()
    assert g.shape == value.shape, name
    inf = ~np.isfinite(value)
    assert np.array_equal(g[inf], value[inf]), name
    err = np.abs(g[~inf] - value[~inf])
    over = err - (bound[~inf] + TINY)
    assert not over.size or over.max() <= 0, "%s: off by %g where %g is allowed (largest error %g)" % (
        name, err[over.argmax()], bound[~inf][over.argmax()], err.max())


def run_window(pr, q=None, k=None, v=None):
    q, k, v = pr.q if q is None else q, pr.k if k is None else k, pr.v if v is None else v
    lse = torch.empty(pr.plan.n, pr.hq, device="cuda")
    out = ssa.ssa_window_forward(pr.p, pr.plan, q, k, v, bias=pr.bias, lse=lse)
    dq, dk, dv, db = ssa.ssa_window_backward(pr.p, pr.plan, q, k, v, pr.dout, bias=pr.bias)
    assert ssa.device_status() == 0
    return dict(out=out, lse=lse, dq=dq, dk=dk, dv=dv, **({"dbias": db} if pr.bias else {}))


def run_diff(pr, q=None, k=None, v=None):
    q, k, v = pr.q if q is None else q, pr.k if k is None else k, pr.v if v is None else v
    out = ssa.ssa_diff_forward(pr.p, pr.plan, q, k, v, pr.lam, 0.5)
    dq, dk, dv, dl = ssa.ssa_diff_backward(pr.p, pr.plan, q, k, v, pr.lam, 0.5, pr.dout)
    assert ssa.device_status() == 0
    return dict(out=out, dq=dq, dk=dk, dv=dv, dlam=dl)


def check_all(got, ref):
    for name in ref:
        if name in got:
            check(got[name], ref, name)


# ---------------------------------------------------------------------------
# the plan
# ---------------------------------------------------------------------------


def test_plan_rows_tiles_and_flags():
    coords, cu = shell(1, 300, seqs=3, r=9)
    coords[7] = coords[6]  # one voxel twice
    pr = Problem(coords, cu, 5, 2, 1, 32, torch.float32)
    perm, ptr, cid = (x.cpu().numpy() for x in (pr.win.perm, pr.win.ptr, pr.win.id))
    rows, tiles = pr.plan.rows.cpu().numpy(), pr.plan.tiles.cpu().numpy()
    assert np.array_equal(rows[:, 0], perm)
    c = coords[perm] % 5
    assert np.array_equal(rows[:, 1], (c[:, 0] * 9 + c[:, 1]) * 9 + c[:, 2])
    assert tiles[-1].tolist() == [2, 0, 0, 0]     # the most tokens of a voxel
    tiles = tiles[:-1]
    live = tiles[(tiles[:, 1] & 65535) > 0]
    covered = np.concatenate([np.arange(t[0], t[0] + (t[1] & 65535)) for t in live])
    assert np.array_equal(np.sort(covered), np.arange(len(coords)))
    for t in live:
        cell = cid[perm[t[0]]]
        assert (t[2], t[3]) == (ptr[cell], ptr[cell + 1]) and (t[0] - t[2]) % 16 == 0
        assert bool(t[1] & 65536) == (cell == cid[7])
    assert np.all(tiles[(tiles[:, 1] & 65535) == 0] == 0)


def test_plan_of_arrays_that_do_not_fit_is_reported():
    coords, cu = shell(2, 100)
    pr = Problem(coords, cu, 4, 2, 1, 32, torch.float32)
    bad = ssa.Bins(pr.win.id.clone(), pr.win.perm.clone(), pr.win.ptr.clone(), pr.win.cu, pr.win.key, pr.win.count)
    bad.perm[5] = 1 << 30
    bad.id[3] = -7
    bad.ptr[2] = 1 << 29
    ssa.ssa_window_plan(pr.coords, bad, 4)
    assert ssa.STATUS_NAMES[ssa.device_status()] == "SSA_ERR_INVALID_ARG"
    assert ssa.device_status() == 0


# ---------------------------------------------------------------------------
# window attention
# ---------------------------------------------------------------------------

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hq,hkv,d,m,bias", [
    (1, 1, 32, 4, None), (4, 2, 32, 4, "offset"), (6, 2, 64, 8, "offset"), (16, 1, 64, 5, "log"), (3, 3, 128, 8, "log"),
    (2, 1, 128, 1, "offset"), (2, 2, 32, 16, "offset"), (8, 4, 64, 10, None), (2, 1, 64, 13, "log"), (5, 1, 32, 2, "log"),
    (4, 2, 64, 12, "offset"), (2, 1, 64, 16, "log"), (2, 1, 128, 12, "offset"), (2, 2, 128, 16, "offset"),
    (3, 1, 128, 13, "log"), (4, 1, 32, 14, "offset"), (12, 2, 64, 9, "offset"), (64, 64, 32, 3, "log"),
])
def test_window_forward_backward(hq, hkv, d, m, bias, dtype):
    coords, cu = shell(3, 350, seqs=2, r=9)
    pr = Problem(coords, cu, m, hq, hkv, d, DT[dtype], seed=4, bias=bias)
    check_all(run_window(pr), pr.ref_window())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,side,m", [(430, 8, 8), (65, 8, 8), (64, 8, 8), (17, 8, 8), (700, 9, 16), (1, 1, 1), (129, 7, 7)])
def test_window_dense_cells(n, side, m, dtype):
    """One cell of n tokens (a few more cells where side > m): more than one chunk of keys, chunk
    and tile edges."""
    coords, cu = dense(5, n, side)
    pr = Problem(coords, cu, m, 4, 2, 64, DT[dtype], seed=6, bias="offset")
    check_all(run_window(pr), pr.ref_window())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_cell_larger_than_any_bias_window(dtype):
    """A plan without codes: windows that cover the grid, no bias; scores with a large spread."""
    coords, cu = shell(6, 900, seqs=2, r=14)
    pr = Problem(coords, cu, 1024, 2, 1, 64, DT[dtype], seed=7, std=8.0)
    assert pr.win.count == 2 and pr.plan.m == 0
    check_all(run_window(pr), pr.ref_window())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,times,m", [(200, 3, 6), (3, 90, 2), (40, 7, 14)])
def test_voxels_that_hold_several_tokens(n, times, m, dtype):
    coords, cu = shell(8, n, r=8)
    coords = np.repeat(coords, times, 0)
    pr = Problem(coords, np.array([0, len(coords)], np.int32), m, 4, 2, 32, DT[dtype], seed=9, bias="offset")
    a, b = run_window(pr), run_window(pr)
    check_all(a, pr.ref_window())
    assert all(torch.equal(a[x], b[x]) for x in a)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("op", ["window", "diff"])
def test_lone_tokens(op, dtype):
    """Cells of one token: p is exactly 1, so dq and dk are exactly 0 and out = v (1 - lambda)."""
    n = 37
    coords = np.stack([np.arange(n) * 9, np.zeros(n), np.arange(n) % 3], 1).astype(np.int32)
    pr = Problem(coords, np.array([0, 20, n], np.int32), 4, 4, 2, 64, DT[dtype], seed=10, bias="offset")
    r = run_window(pr) if op == "window" else run_diff(pr)
    assert float(r["dq"].abs().max()) == 0 and float(r["dk"].abs().max()) == 0
    if op == "window":
        assert float(r["dbias"].abs().max()) == 0
        assert torch.equal(r["out"], pr.v.repeat_interleave(2, 1))
    check_all(r, pr.ref_window() if op == "window" else pr.ref_diff())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_barred_buckets(dtype):
    """Minus infinity in buckets: their keys count for nothing; rows with nothing left (the
    offset 0 and all others barred) give zeros; the fp32 type's lowest value bars as well."""
    coords, cu = shell(11, 300, r=9)
    pr = Problem(coords, cu, 5, 4, 2, 64, DT[dtype], seed=12, bias="offset")
    t = pr.bias.table
    t[0, ::2] = float("-inf")
    t[1] = float("-inf")
    t[2, 5:300] = torch.finfo(torch.float32).min
    r, ref = run_window(pr), pr.ref_window()
    assert float(r["out"][:, 1].abs().max()) == 0 and bool(torch.isneginf(r["lse"][:, 1]).all())
    assert float(r["dbias"][1].abs().max()) == 0 and float(r["dq"][:, 1].abs().max()) == 0
    check_all(r, ref)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_scores_far_below_zero_after_a_barred_start(dtype):
    """A cell whose first keys are barred and whose others have a bias of -300: the sums start at the
    first key that counts, wherever it stands."""
    coords, cu = dense(19, 480, 8)
    pr = Problem(coords, cu, 8, 2, 1, 64, DT[dtype], seed=20, bias="offset")
    t = pr.bias.table.view(2, 15, 15, 15)
    t -= 300.0
    t[0, 3:] = float("-inf")       # queries far along x see no key of their own or earlier layers
    t[1, :12] = float("-inf")
    r, ref = run_window(pr), pr.ref_window()
    assert bool(torch.isfinite(r["out"]).all()) and bool(torch.isfinite(r["dbias"]).all())
    check_all(r, ref)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_buckets_outside_the_table_have_no_bias(dtype):
    coords, cu = shell(13, 200, r=8)
    pr = Problem(coords, cu, 4, 2, 1, 32, DT[dtype], seed=14, bias="log")
    pr.bias.bucket[::3] = -1
    pr.bias.bucket[1::7] = pr.bias.table.shape[1]
    pr.bias.bucket[2::11] = -(1 << 31)
    check_all(run_window(pr), pr.ref_window())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("op", ["window", "diff"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_what_is_not_finite_stays_in_its_cell(op, bad, dtype):
    coords, cu = shell(15, 250, seqs=2, r=8)
    pr = Problem(coords, cu, 5, 4, 2, 32, DT[dtype], seed=16, bias="offset")
    run = run_window if op == "window" else run_diff
    clean = run(pr)
    tok = 11
    for x in (pr.q, pr.k, pr.v, pr.dout):
        x[tok] = bad
    dirty = run(pr)
    other = pr.win.id != pr.win.id[tok]
    for x in ("out", "dq", "dk", "dv"):
        assert torch.equal(clean[x][other], dirty[x][other]), x
    assert not bool(torch.isfinite(dirty["out"][tok]).all())
    assert not bool(torch.isfinite(dirty["dq"][tok]).any()) and not bool(torch.isfinite(dirty["dk"][tok]).any())


def test_bias_gradient_of_many_rows_keeps_fp32_precision():
    """A full cube of 262144 tokens and 32 heads: many rows add to one CTA's table.  Relative error of
    two heads' dbias in the 2-norm.  Per dS, roundings as random numbers of their largest sizes: ex2
    2^-22; score, lse2 and their difference, all below 8 in units of log2, 2^-22 ln 2 each; together
    2^-22 (1 + 2.1), over sqrt 3 for the root mean square: 4.3e-7.  dP is a sum of two tensor core steps
    that may cut off rather than round: 2 x 2^-23.  Together below 7e-7, which the sums' own unit must
    not add to.  (A unit that only bounds the rows by the CTA's slots is 8.6e-7 off by itself.)"""
    side, m, hq, hkv, d = 64, 4, 32, 2, 32
    n, w = side ** 3, side // m
    key = np.arange(n)
    coords = np.stack([key // side ** 2, key // side % side, key % side], 1).astype(np.int32)
    coords, cu = torch.from_numpy(coords).cuda(), torch.tensor([0, n], dtype=torch.int32, device="cuda")
    _, win = ssa.ssa_bin(coords, cu, 1024, m, m)
    gen = torch.Generator(device="cuda").manual_seed(5)
    f = lambda h: torch.randn(n, h, d, generator=gen, device="cuda").bfloat16()  # noqa: E731
    q, k, v, dout = f(hq), f(hkv), f(hkv), f(hq)
    table = 0.5 * torch.randn(hq, (2 * m - 1) ** 3, generator=gen, device="cuda")
    p = ssa.make_window_params(hq, hkv, d, torch.bfloat16)
    got = ssa.ssa_window_backward(p, ssa.ssa_window_plan(coords, win, m), q, k, v, dout, bias=ssa.WindowBias(table))[3]
    x = torch.cartesian_prod(*[torch.arange(m, device="cuda")] * 3)
    x = x[:, None] - x[None] + m - 1
    off = (x[..., 0] * (2 * m - 1) + x[..., 1]) * (2 * m - 1) + x[..., 2]
    cells = lambda t, h: (t[:, h].reshape(w, m, w, m, w, m, d).permute(0, 2, 4, 1, 3, 5, 6)  # noqa: E731
                          .reshape(w ** 3, m ** 3, d).double())
    for h in (0, 29):
        g = h // (hq // hkv)
        s = cells(q, h) @ cells(k, g).transpose(1, 2) / np.sqrt(d) + table[h].double()[off]
        s = torch.softmax(s, -1)
        dp = cells(dout, h) @ cells(v, g).transpose(1, 2)
        ds = s * (dp - (s * dp).sum(-1, keepdim=True))
        ref = torch.zeros((2 * m - 1) ** 3, dtype=torch.float64, device="cuda")
        ref.index_add_(0, off.reshape(-1), ds.sum(0).reshape(-1))
        assert float((got[h].double() - ref).norm() / ref.norm()) < 7e-7


def test_bias_and_values_move_the_output_as_the_gradient_says():
    """The gradients against differences of the operator itself (fp32): one direction each."""
    coords, cu = shell(17, 300, r=9)
    pr = Problem(coords, cu, 6, 4, 2, 32, torch.float32, seed=18, bias="log")
    r = run_window(pr)
    gen = torch.Generator(device="cuda").manual_seed(1)
    for name, x in (("dq", pr.q), ("dk", pr.k), ("dv", pr.v), ("dbias", pr.bias.table)):
        step = torch.randn(x.shape, generator=gen, device="cuda")
        keep, vals = x.clone(), []
        for h in (1e-2, -1e-2):
            x.copy_(keep + h * step)
            vals.append(float((ssa.ssa_window_forward(pr.p, pr.plan, pr.q, pr.k, pr.v, bias=pr.bias).double()
                               * pr.dout.double()).sum()))
        x.copy_(keep)
        slope, said = (vals[0] - vals[1]) / 2e-2, float((r[name].double() * step.double()).sum())
        # a central difference of step h is off by h^2 / 6 of the third derivative, which for sums
        # of ~4e4 terms of order one with random signs is some hundreds: 1e-4 / 6 * 1e3 < 0.02,
        # plus the outputs' fp32 noise sqrt(4e4) 1e-6 / 1e-2 = 0.02
        assert abs(slope - said) < 0.1 + 1e-3 * abs(said), (name, slope, said)


# ---------------------------------------------------------------------------
# differential attention
# ---------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hq,hkv,d,m", [(2, 2, 32, 4), (8, 4, 64, 8), (12, 4, 32, 5), (32, 2, 64, 4), (4, 2, 32, 20)])
def test_diff_forward_backward(hq, hkv, d, m, dtype):
    coords, cu = shell(21, 300, seqs=2, r=9)
    pr = Problem(coords, cu, m, hq, hkv, d, DT[dtype], seed=22)
    check_all(run_diff(pr), pr.ref_diff())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,side,m,d", [(430, 8, 8, 64), (65, 8, 8, 32), (64, 8, 8, 64), (33, 8, 8, 64), (1, 1, 1, 32), (129, 7, 7, 32)])
def test_diff_dense_cells(n, side, m, d, dtype):
    coords, cu = dense(23, n, side)
    pr = Problem(coords, cu, m, 4, 2, d, DT[dtype], seed=24)
    check_all(run_diff(pr), pr.ref_diff())


# ---------------------------------------------------------------------------
# 8-bit checkpoints
# ---------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("rows", [1, 5, 33, 1000])
def test_act8_codes_scales_and_values(rows, d, dtype):
    rng = np.random.default_rng(31)
    x = rng.standard_normal((rows, d)) * 10.0 ** rng.uniform(-30, 30, (rows, 1))
    special = [np.zeros(d), np.full(d, 127.0), np.full(d, 127.5), np.r_[128.0, np.full(d - 1, 0.5)],
               np.full(d, 3.38e38), np.full(d, 1e-38), np.full(d, 1e-41), np.r_[np.inf, np.ones(d - 1)],
               np.r_[np.ones(d - 1), np.nan], np.r_[64.0, np.arange(1, d) / 2.0 % 60], np.full(d, -127.0)]
    for i, s in enumerate(special[:rows - 1] if rows < 20 else special):
        x[(7 * i) % rows] = s
    t = torch.from_numpy(x.astype(np.float32)).to(DT[dtype])
    held = ssa.ssa_act8_pack(t.cuda())
    codes, scale = WO.act8(t.double().numpy())
    ok = np.isfinite(scale)
    assert np.array_equal(held.codes.cpu().numpy(), codes)
    assert np.array_equal(held.scale.cpu().double().numpy()[ok], scale[ok])
    assert bool(torch.isnan(held.scale.cpu()[torch.from_numpy(~ok)]).all())
    for out in (torch.bfloat16, torch.float32):
        val = ssa.ssa_act8_unpack(held, out).double().cpu().numpy()
        want = codes * scale[:, None]
        # values under the smallest normal number may come back as zero or as themselves
        tiny = np.abs(want) < 2.0 ** -126
        assert np.array_equal(val[ok[:, None] & ~tiny], want[ok[:, None] & ~tiny])
        assert np.all(np.abs(val[ok[:, None] & tiny]) < 2.0 ** -126)
        assert np.all(np.isnan(val[~ok]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("op", ["window", "diff"])
@pytest.mark.parametrize("hq,hkv,d,n", [(4, 2, 32, 250), (8, 2, 64, 400), (2, 2, 128, 250)])
def test_backward_from_checkpoints_is_the_backward_at_their_values(hq, hkv, d, n, op, dtype):
    if op == "diff" and d == 128:
        d = 64
    coords, cu = shell(33, n, seqs=2, r=7)
    pr = Problem(coords, cu, 8, hq, hkv, d, DT[dtype], seed=34, bias="offset")
    held = [ssa.ssa_act8_pack(x) for x in (pr.q, pr.k, pr.v)]
    vals = [ssa.ssa_act8_unpack(x, DT[dtype]) for x in held]
    if op == "window":
        got = ssa.ssa_window_backward(pr.p, pr.plan, *held, pr.dout, bias=pr.bias)
        want = ssa.ssa_window_backward(pr.p, pr.plan, *vals, pr.dout, bias=pr.bias)
        ref, names = pr.ref_window(*vals), ("dq", "dk", "dv", "dbias")
    else:
        got = ssa.ssa_diff_backward(pr.p, pr.plan, *held, pr.lam, 0.5, pr.dout)
        want = ssa.ssa_diff_backward(pr.p, pr.plan, *vals, pr.lam, 0.5, pr.dout)
        ref, names = pr.ref_diff(*vals), ("dq", "dk", "dv", "dlam")
    for name, a, b in zip(names, got, want):
        assert torch.equal(a, b), name
        check(a, ref, name)


def test_a_checkpoint_of_a_bad_row_shows_in_its_cell_only():
    coords, cu = shell(35, 250, r=8)
    pr = Problem(coords, cu, 5, 4, 2, 32, torch.bfloat16, seed=36, bias="offset")
    held = [ssa.ssa_act8_pack(x) for x in (pr.q, pr.k, pr.v)]
    clean = ssa.ssa_window_backward(pr.p, pr.plan, *held, pr.dout, bias=pr.bias)
    pr.k[9, 0, 3] = float("inf")
    held[1] = ssa.ssa_act8_pack(pr.k)
    dirty = ssa.ssa_window_backward(pr.p, pr.plan, *held, pr.dout, bias=pr.bias)
    other = pr.win.id != pr.win.id[9]
    for a, b in zip(clean[:3], dirty[:3]):
        assert torch.equal(a[other], b[other])
    assert bool(torch.isnan(dirty[0][9, 0]).all())


# ---------------------------------------------------------------------------
# how they are called
# ---------------------------------------------------------------------------


def test_a_training_step_of_two_layers_from_checkpoints():
    """The operators as they are used together: one plan, a window layer and a differential
    layer whose input is the first one's output; Q, K, V kept in 8 bits; backward through both."""
    coords, cu = shell(41, 350, seqs=2, r=9)
    pr = Problem(coords, cu, 6, 4, 2, 32, torch.float32, seed=42, bias="log")
    held = [ssa.ssa_act8_pack(x) for x in (pr.q, pr.k, pr.v)]
    q, k, v = (ssa.ssa_act8_unpack(x, torch.float32) for x in held)
    o1 = ssa.ssa_window_forward(pr.p, pr.plan, q, k, v, bias=pr.bias)
    o2 = ssa.ssa_diff_forward(pr.p, pr.plan, o1, k, v, pr.lam, 0.5)
    g2 = ssa.ssa_diff_backward(pr.p, pr.plan, o1, k, v, pr.lam, 0.5, pr.dout)
    g1 = ssa.ssa_window_backward(pr.p, pr.plan, *held, g2[0], bias=pr.bias)
    # the same by automatic differentiation of a dense form in 64 bits
    ids = pr.win.id.cpu()
    same = ids[:, None] == ids[None]
    t = [x.double().cpu().requires_grad_() for x in (q, k, v, pr.bias.table, pr.lam)]
    c = torch.from_numpy(coords).long() % 6
    o3 = c[:, None] - c[None] + 5
    off = pr.bias.bucket.cpu().long()[(o3[..., 0] * 11 + o3[..., 1]) * 11 + o3[..., 2]]

    def maps(a, b, extra=0.0):
        s = torch.einsum("ihd,jhd->hij", a, b) / np.sqrt(32) + extra
        return torch.softmax(s.masked_fill(~same, float("-inf")), -1)
    rep = lambda x: x.repeat_interleave(2, 1)  # noqa: E731
    y1 = torch.einsum("hij,jhd->ihd", maps(t[0], rep(t[1]), t[3][:, off]), rep(t[2]))
    lam = torch.exp((t[4][0] * t[4][1]).sum(-1)) - torch.exp((t[4][2] * t[4][3]).sum(-1)) + 0.5
    kp = t[1].repeat(1, 2, 1)  # both query pairs read key pair 0
    z = maps(y1, kp)
    w = z[0::2] - lam[:, None, None] * z[1::2]
    y2 = torch.einsum("hij,je->ihe", w, t[2].reshape(-1, 64)).reshape(o2.shape)
    (y2 * pr.dout.double().cpu()).sum().backward()
    # fp32 all along: relative roundings of 2^-24 through two layers of sums of up to ~100 terms of
    # either sign: 1e-5 of the largest entry leaves a factor of ten
    for got, want in ((o2, y2.detach()), (g1[0], t[0].grad), (g1[1] + g2[1], t[1].grad), (g1[2] + g2[2], t[2].grad),
                      (g1[3], t[3].grad), (g2[3], t[4].grad)):
        err = float((got.double().cpu() - want).abs().max())
        assert err <= 1e-5 * float(want.abs().max()), err


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("op", ["window", "diff"])
def test_same_bits_every_time_on_any_stream_and_from_a_graph(op, dtype):
    coords, cu = shell(43, 400, seqs=2, r=9)
    pr = Problem(coords, cu, 6, 8, 2, 64, DT[dtype], seed=44, bias="offset")
    run = run_window if op == "window" else run_diff
    first = run(pr)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = run(pr)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(first[x], second[x]) for x in first)

    def step():
        if op == "window":
            return (ssa.ssa_window_forward(pr.p, pr.plan, pr.q, pr.k, pr.v, bias=pr.bias),
                    *ssa.ssa_window_backward(pr.p, pr.plan, pr.q, pr.k, pr.v, pr.dout, bias=pr.bias))
        return (ssa.ssa_diff_forward(pr.p, pr.plan, pr.q, pr.k, pr.v, pr.lam, 0.5),
                *ssa.ssa_diff_backward(pr.p, pr.plan, pr.q, pr.k, pr.v, pr.lam, 0.5, pr.dout))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        held = step()
    pr.q.neg_()          # new values in the captured buffers
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(held, step()):
        assert torch.equal(a, b)


def test_given_buffers_are_filled_and_nothing_beside_them():
    coords, cu = shell(45, 200, r=8)
    pr = Problem(coords, cu, 4, 4, 2, 32, torch.bfloat16, seed=46, bias="log")
    n = pr.plan.n
    want = run_window(pr)
    room = {x: torch.full((n + 16, h, 32), 7.0, dtype=torch.bfloat16, device="cuda")
            for x, h in (("out", 4), ("dq", 4), ("dk", 2), ("dv", 2))}
    db = torch.full((6, pr.bias.table.shape[1]), 7.0, device="cuda")
    ssa.ssa_window_forward(pr.p, pr.plan, pr.q, pr.k, pr.v, bias=pr.bias, out=room["out"][8:n + 8])
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    ssa.ssa_window_backward(pr.p, pr.plan, pr.q, pr.k, pr.v, pr.dout, bias=pr.bias,
                            grads=tuple(room[x][8:n + 8] for x in ("dq", "dk", "dv")), dbias=db[1:5], workspace=ws)
    for x, t in room.items():
        assert torch.equal(t[8:n + 8], want[x]) and bool((t[:8] == 7).all()) and bool((t[n + 8:] == 7).all())
    assert torch.equal(db[1:5], want["dbias"]) and bool((db[0] == 7).all()) and bool((db[5] == 7).all())


def test_workspaces_and_checkpoints_where_they_do_not_belong_are_refused():
    coords, cu = shell(51, 200)
    pr = Problem(coords, cu, 4, 2, 1, 32, torch.bfloat16, seed=52)
    held = [ssa.ssa_act8_pack(x) for x in (pr.q, pr.k, pr.v)]
    with pytest.raises(ValueError, match="Act8"):
        ssa.ssa_window_forward(pr.p, pr.plan, *held)
    with pytest.raises(ValueError, match="Act8"):
        ssa.ssa_window_backward(pr.p, pr.plan, held[0], pr.k, pr.v, pr.dout)
    need = pr.plan.workspace_size(ssa.OP_WINDOW_BACKWARD, pr.p)
    with pytest.raises(ValueError, match="uint8"):
        ssa.ssa_window_backward(pr.p, pr.plan, pr.q, pr.k, pr.v, pr.dout,
                                workspace=torch.empty(need, dtype=torch.float32, device="cuda"))
    with pytest.raises(ValueError, match="CUDA"):
        ssa.ssa_window_backward(pr.p, pr.plan, pr.q, pr.k, pr.v, pr.dout, workspace=torch.empty(need, dtype=torch.uint8))


def test_two_calls_at_once_on_two_streams():
    """Two backward passes of different sizes that overlap give what each gives alone."""
    prs = []
    for seed, n, m, hq in ((61, 900, 6, 8), (62, 2500, 8, 4)):
        coords, cu = shell(seed, n, r=20)
        prs.append(Problem(coords, cu, m, hq, 2, 64, torch.bfloat16, seed=seed, bias="offset"))
    alone = [run_window(pr) for pr in prs]
    streams = [torch.cuda.Stream() for _ in prs]
    torch.cuda.synchronize()
    for _ in range(5):
        both = []
        for pr, st in zip(prs, streams):
            with torch.cuda.stream(st):
                both.append(run_window(pr))
        torch.cuda.synchronize()
        for a, b in zip(alone, both):
            assert all(torch.equal(a[x], b[x]) for x in a)


@pytest.mark.parametrize("dtype,hkv", [("bf16", 64), ("f32", 4)])
def test_places_past_32_bits(dtype, hkv):
    """A full cube of 274625 tokens with 64 heads of 128: elements past 2^31 in q (and, in bf16, k
    and v).  The last cell against fp64 for the first and the last head; bounds of one storage
    rounding of P or dS and of the result (bf16 2 x 2^-8 of the row sums' magnitudes; fp32 1e-5 for
    sums of up to 128 fp32 products, 2^-24 each)."""
    side, m, hq, d, dt = 65, 5, 64, 128, DT[dtype]
    n = side ** 3
    key = torch.arange(n, device="cuda")
    coords = torch.stack([key // side ** 2, key // side % side, key % side], 1).to(torch.int32)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    _, win = ssa.ssa_bin(coords, cu, 1024, m, m)
    plan = ssa.ssa_window_plan(coords, win, m)
    assert n * hq * d > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(7)
    f = lambda h: torch.randn(n, h, d, generator=gen, dtype=dt, device="cuda")  # noqa: E731
    q, k, v, dout = f(hq), f(hkv), f(hkv), f(hq)
    p = ssa.make_window_params(hq, hkv, d, dt)
    out = ssa.ssa_window_forward(p, plan, q, k, v)
    dq, dk, dv, _ = ssa.ssa_window_backward(p, plan, q, k, v, dout)
    last = (coords >= side - m).all(1).nonzero()[:, 0]
    g = hq // hkv
    tol = 2 * 2.0 ** -8 if dtype == "bf16" else 1e-5

    def near(got, ref, mag):
        assert bool(((got.double() - ref).abs() <= tol * mag + 1e-30).all())
    for hk in (0, hkv - 1):
        kk, vv = k[last, hk].double(), v[last, hk].double()
        rdk, rdv, mdk, mdv = (torch.zeros_like(kk) for _ in range(4))
        for h in range(hk * g, hk * g + g):
            qq, do = q[last, h].double(), dout[last, h].double()
            s = torch.softmax(qq @ kk.T / np.sqrt(d), -1)
            dp = do @ vv.T
            dd = (s * dp).sum(-1, keepdim=True)
            ds = s * (dp - dd)
            mds = s * (dp.abs() + (s * dp.abs()).sum(-1, keepdim=True))
            near(out[last, h], s @ vv, s @ vv.abs())
            near(dq[last, h], ds @ kk / np.sqrt(d), mds @ kk.abs() / np.sqrt(d))
            rdk += ds.T @ qq / np.sqrt(d)
            mdk += mds.T @ qq.abs() / np.sqrt(d)
            rdv += s.T @ do
            mdv += s.T @ do.abs()
        near(dk[last, hk], rdk, mdk)
        near(dv[last, hk], rdv, mdv)


def test_no_tokens():
    z = lambda *s, dt=torch.float32: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
    win = ssa.Bins.empty(0, 1, "cuda")
    plan = ssa.ssa_window_plan(z(0, 3, dt=torch.int32), win, 4)
    p = ssa.make_window_params(4, 2, 32, torch.float32)
    q, k = z(0, 4, 32), z(0, 2, 32)
    bias = ssa.WindowBias(torch.ones(4, 343, device="cuda"))
    assert ssa.ssa_window_forward(p, plan, q, k, k, bias=bias).shape == (0, 4, 32)
    assert float(ssa.ssa_window_backward(p, plan, q, k, k, q, bias=bias)[3].abs().max()) == 0
    lam = torch.ones(4, 2, 32, device="cuda")
    assert float(ssa.ssa_diff_backward(p, plan, q, k, k, lam, 0.5, q)[3].abs().max()) == 0
    assert ssa.ssa_act8_pack(q).codes.shape == (0, 4, 32)


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs a second device")
def test_tensors_on_another_device_than_the_current_one():
    coords, cu = shell(47, 100)
    with torch.cuda.device(1):
        pr = Problem(coords, cu, 4, 2, 1, 32, torch.float32, seed=48, bias="offset")
        want = run_window(pr)
    got = run_window(pr)
    assert all(torch.equal(want[x], got[x]) for x in want)
