"""Attention inside the cells at the limits of its numbers."""
import threading

import numpy as np
import pytest
import torch

from spatial_sparse_attention_ssa_b200 import ssa
from test_gpu_window import DT, Problem, check_all, dense, run_diff, run_window, shell

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shift", [120, -95])
@pytest.mark.parametrize("m", [5, 14])
def test_bias_gradient_scales_with_the_size_of_dp(m, shift):
    """dout and v times powers of two: dP, D and dS are the same numbers times a power of two (the
    largest |dP| here is near 2^125 and 2^-90), so dbias is, bit for bit."""
    coords, cu = shell(71, 300, r=9)
    pr = Problem(coords, cu, m, 4, 2, 32, torch.bfloat16, seed=72, bias="offset")
    want = run_window(pr)["dbias"].double() * 2.0 ** shift
    pr.dout *= 2.0 ** (shift // 2)
    pr.v *= 2.0 ** (shift - shift // 2)
    got = run_window(pr)["dbias"]
    assert bool(torch.isfinite(got).all())
    assert torch.equal(got.double(), want)


def dbias64(pr, h):
    """One head's dbias in fp64, cell by cell, and the root of the sum of all dS^2."""
    e, g = 2 * pr.m - 1, h // (pr.hq // pr.hkv)
    ref, power = torch.zeros(e ** 3, dtype=torch.float64, device="cuda"), 0.0
    ptr = pr.win.ptr[:pr.win.count + 1].tolist()
    for a, b in zip(ptr[:-1], ptr[1:]):
        tok = pr.win.perm[a:b].long()
        x = pr.coords[tok].long() % pr.m
        code = (x[:, 0] * e + x[:, 1]) * e + x[:, 2]
        k, v = pr.k[tok, g].double(), pr.v[tok, g].double()
        for i in range(0, b - a, 1000):
            t = tok[i:i + 1000]
            off = code[i:i + 1000, None] - code[None] + (pr.m - 1) * (e * e + e + 1)
            p = torch.softmax(pr.q[t, h].double() @ k.T / np.sqrt(pr.d) + pr.bias.table[h].double()[off], -1)
            dp = pr.dout[t, h].double() @ v.T
            ds = p * (dp - (p * dp).sum(-1, keepdim=True))
            ref.index_add_(0, off.reshape(-1), ds.reshape(-1))
            power += float((ds * ds).sum())
    return ref, power ** 0.5


@pytest.mark.parametrize("crowd,hq,hkv,m", [(2000, 128, 2, 4), (5000, 128, 2, 4), (20000, 4, 2, 4), (700, 128, 2, 13), (4097, 2, 1, 3)])
def test_bias_gradient_of_a_crowded_voxel_keeps_fp32_precision(crowd, hq, hkv, m):
    """One voxel with thousands of tokens beside ordinary cells.  Error of dbias in the 2-norm against
    that of all dS (a crowded voxel's own offsets nearly cancel).  Per dS, as random numbers: exponential
    2^-22, score, lse2 and their difference 2^-22 ln 2 each below 8 and twice that below 16 (lse2 of
    20000 keys), over sqrt 3: 7e-7; dP 2 x 2^-23.  Per row: the sums of up to n / 4 terms per lane are off by
    2^-25 sqrt(n / 12), 1.2e-6, common to a row, whose dS sum to zero but for the offsets that the crowd does
    not hold.  Together below 3e-6, which the fixed point must not add to."""
    coords, cu = shell(73, 600, r=9)
    coords = np.concatenate([coords, np.repeat(coords[100:101], crowd, 0)])
    coords = coords[np.random.default_rng(74).permutation(len(coords))]
    pr = Problem(coords, np.array([0, len(coords)], np.int32), m, hq, hkv, 32, torch.bfloat16, seed=75, bias="offset")
    got = ssa.ssa_window_backward(pr.p, pr.plan, pr.q, pr.k, pr.v, pr.dout, bias=pr.bias)[3]
    again = ssa.ssa_window_backward(pr.p, pr.plan, pr.q, pr.k, pr.v, pr.dout, bias=pr.bias)[3]
    assert torch.equal(got, again) and ssa.device_status() == 0
    for h in (0, hq - 1):
        ref, power = dbias64(pr, h)
        assert float((got[h].double() - ref).norm()) < 3e-6 * power


def test_bias_gradient_of_many_heads_keeps_fp32_precision():
    """512 heads leave a head one CTA, which adds the dS of all of its 125000 rows.  The tolerance is that of
    the test of many rows in test_gpu_window.py: below 7e-7 by the arithmetic of one dS, cells of 125."""
    coords, cu = dense(76, 50 ** 3, 50)
    pr = Problem(coords, cu, 5, 2, 2, 32, torch.bfloat16, seed=77)
    gen = torch.Generator(device="cuda").manual_seed(78)
    f = lambda *x: torch.randn(*x, generator=gen, device="cuda")  # noqa: E731
    pr.hq, pr.p = 512, ssa.make_window_params(512, 2, 32, torch.bfloat16)
    pr.q, pr.dout = (f(50 ** 3, 512, 32).bfloat16() for _ in range(2))
    pr.bias = ssa.WindowBias(0.5 * f(512, 729))
    got = ssa.ssa_window_backward(pr.p, pr.plan, pr.q, pr.k, pr.v, pr.dout, bias=pr.bias)[3]
    for h in (0, 300):
        ref, _ = dbias64(pr, h)
        assert float((got[h].double() - ref).norm() / ref.norm()) < 7e-7


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m", [3, 13])
def test_plan_counts_the_tokens_of_a_voxel_per_cell(m, dtype):
    """Cells with one, two and thirty tokens in a voxel side by side: the plan's counts, and results."""
    coords, _ = shell(78, 250, r=8)
    coords = np.concatenate([coords, coords[:40], np.repeat(coords[200:201], 29, 0)])
    pr = Problem(coords, np.array([0, len(coords)], np.int32), m, 2, 1, 32, DT[dtype], seed=79, bias="offset")
    ids = pr.win.id.cpu().numpy()
    tiles = pr.plan.tiles.cpu().numpy()[:-1]
    perm = pr.win.perm.cpu().numpy()
    for t in tiles[(tiles[:, 1] & 65535) > 0]:
        c = coords[ids == ids[perm[t[0]]]]
        most = int(np.unique(c, axis=0, return_counts=True)[1].max())
        assert t[1] >> 17 == (most if most > 1 else 0) and (t[1] >> 16 & 1) == (most > 1)
    check_all(run_window(pr), pr.ref_window())


@pytest.mark.parametrize("dtype,d", [("f32", 32), ("bf16", 64)])
def test_host_threads_with_plans_of_different_sizes(dtype, d):
    """Calls that overlap on the host, of plans that need different shared memory, give what each gives
    alone."""
    prs = []
    for seed, m, hkv in ((81, 3, 4), (82, 12, 2), (83, 6, 4), (84, 12, 1)):
        coords, cu = shell(seed, 300, r=9)
        prs.append(Problem(coords, cu, m, 4, hkv, d, DT[dtype], seed=seed, bias="offset"))
    alone = [run_window(pr) for pr in prs]
    torch.cuda.synchronize()
    failed = []

    def work(pr, want):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                grads = tuple(torch.empty_like(want[n]) for n in ("dq", "dk", "dv"))
                db, out = torch.empty_like(want["dbias"]), torch.empty_like(want["out"])
                ws = torch.empty(pr.plan.workspace_size(ssa.OP_WINDOW_BACKWARD, pr.p), dtype=torch.uint8, device="cuda")
                for _ in range(3000):
                    ssa.ssa_window_forward(pr.p, pr.plan, pr.q, pr.k, pr.v, bias=pr.bias, out=out)
                    ssa.ssa_window_backward(pr.p, pr.plan, pr.q, pr.k, pr.v, pr.dout, bias=pr.bias, grads=grads,
                                            dbias=db, workspace=ws)
                torch.cuda.current_stream().synchronize()
                for x, n in zip((out, *grads, db), ("out", "dq", "dk", "dv", "dbias")):
                    assert torch.equal(x, want[n]), n
        except Exception as e:  # noqa: BLE001
            failed.append(e)
    threads = [threading.Thread(target=work, args=a) for a in zip(prs, alone)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("op", ["window", "bias", "diff"])
@pytest.mark.parametrize("d", [32, 64])
def test_a_row_whose_scores_all_overflow_is_nan(d, op, dtype):
    """One infinite component of q makes every score of a row minus infinity: a softmax of NaN, not a row
    with nothing left.  Lone tokens, and a cell of 70 where every key is negative there."""
    n = 80
    coords = np.stack([np.arange(n) * 9, np.zeros(n), np.zeros(n)], 1).astype(np.int32)
    coords[10:] = dense(91, 70, 8)[0] + np.array([8 * 100, 0, 0])
    pr = Problem(coords, np.array([0, n], np.int32), 8, 4, 2, d, DT[dtype], seed=92, bias="offset" if op == "bias" else None)
    run = run_diff if op == "diff" else run_window
    pr.k[..., 3] = -pr.k[..., 3].abs() - 0.1
    clean = run(pr)
    for tok in (4, 30):
        pr.q[tok, :, 3] = float("inf")
    dirty = run(pr)
    other = (pr.win.id != pr.win.id[4]) & (pr.win.id != pr.win.id[30])
    for x in ("out", "dq", "dk", "dv"):
        assert torch.equal(clean[x][other], dirty[x][other]), x
        for tok in (4, 30):
            assert bool(torch.isnan(dirty[x][tok]).all()), x
    rest = torch.arange(n, device="cuda") >= 10
    rest[30] = False
    assert torch.equal(clean["out"][rest], dirty["out"][rest])       # other rows of the cell: their own scores
    if op == "bias" and dtype == "bf16":
        assert bool(torch.isnan(dirty["dbias"]).all())
    if op != "diff":
        assert bool(torch.isnan(dirty["lse"][[4, 30]]).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_what_the_bias_bars_stays_barred_beside_scores_that_overflow(dtype):
    """Barred keys count for nothing: a row with all keys barred gives zeros, and a row whose one key that
    is left overflows gives NaN."""
    coords, cu = dense(93, 100, 5)
    pr = Problem(coords, cu, 5, 2, 2, 32, DT[dtype], seed=94, bias="offset")
    pr.k[..., 3] = -pr.k[..., 3].abs() - 0.1
    pr.bias.table[0] = float("-inf")
    pr.bias.table[1] = float("-inf")
    pr.bias.table[1, 364] = 0.5            # the offset 0: every token sees itself alone
    clean = run_window(pr)
    assert float(clean["out"][:, 0].abs().max()) == 0 and torch.equal(clean["out"][:, 1], pr.v[:, 1])
    pr.q[7, 1, 3] = float("inf")
    dirty = run_window(pr)
    assert bool(torch.isnan(dirty["out"][7, 1]).all()) and bool(torch.isnan(dirty["lse"][7, 1]))
    keep = torch.arange(100, device="cuda") != 7
    assert torch.equal(dirty["out"][:, 0], clean["out"][:, 0]) and torch.equal(dirty["out"][keep], clean["out"][keep])
    assert float(dirty["dq"][:, 0].abs().max()) == 0 and bool(torch.isnan(dirty["dq"][7, 1]).any())
    assert bool(torch.isneginf(dirty["lse"][:, 0]).all())
    assert float(dirty["dbias"][0].abs().max()) == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("far", [-1e9, -65504.0, -2000.0, 3e6])
def test_weights_of_a_row_sum_to_one_however_far_its_scores(far, dtype):
    """A large number on every key of a row, as a mask of -1e9 is: the backward's weights are those of the
    forward and sum to one.  dv of a cell with dout of ones is the sum of all its rows' weights: the number
    of rows.  bf16: a step's half of 2^-8 each for the weights and for dv; fp32: two exponentials 2^-22."""
    coords, cu = dense(95, 40, 4)
    pr = Problem(coords, cu, 4, 2, 1, 32, DT[dtype], seed=96, bias="offset")
    pr.bias.table[:] = far
    pr.dout[:] = 1.0
    r = run_window(pr)
    total = r["dv"].double().sum(0) / 80
    tol = 2.1 * 2.0 ** -8 if dtype == "bf16" else 1e-6
    assert float((total - 1).abs().max()) < tol, total
    # dout of ones times v of one: dP is the same for every key, so dS is zero but for roundings of dP - D
    pr.v[:] = 1.0
    r = run_window(pr)
    for x in ("dq", "dk", "dbias"):
        assert float(r[x].double().abs().max()) < 32 * 80 * 2.0 ** -18, x


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m,crowd", [(4, 0), (4, 3000), (14, 0)])
def test_gradients_do_not_see_a_bias_that_all_keys_share(m, crowd, dtype):
    """q of zeros, so every score is the bias: with -1e9 everywhere the weights, and so all gradients, are
    those with 0 everywhere.  lse2 and its rest against lse2 alone: an exponential of 2^-22 more and a
    rounding of log2 of the sum, 12 at most, 2^-21 ln 2: below 1e-6 of each weight; bf16 weights and results
    may round to the other side, 2^-7 of a weight each."""
    coords, cu = shell(97, 300, r=9)
    if crowd:
        coords = np.concatenate([coords, np.repeat(coords[100:101], crowd, 0)])
        cu = np.array([0, len(coords)], np.int32)
    pr = Problem(coords, cu, m, 4, 2, 32, DT[dtype], seed=98, bias="offset")
    pr.q[:] = 0
    pr.bias.table[:] = 0
    want = run_window(pr)
    pr.bias.table[:] = -1e9
    got = run_window(pr)
    for x in ("out", "dq", "dk", "dv", "dbias"):
        near = float((got[x].double() - want[x].double()).norm())
        tol = 2.0 ** -7 if dtype == "bf16" and x != "dbias" else 1e-5
        assert near <= tol * float(want[x].double().norm()), x


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("op", ["window", "diff"])
@pytest.mark.parametrize("size", [2.0 ** 6, 2.0 ** 12])
def test_weights_of_rows_with_large_equal_scores(size, op, dtype):
    """No bias, q and k the same large vector everywhere: equal scores up to 10^8, weights 1 / n, so dv of dout of
    ones is the number of maps that read a value head, the second ones times -lambda."""
    coords, cu = dense(99, 40, 4)
    pr = Problem(coords, cu, 4, 4, 2, 32, DT[dtype], seed=100)
    pr.q[:], pr.k[:], pr.dout[:] = size, size, 1.0
    pr.lam[:] = 0
    r = run_window(pr) if op == "window" else run_diff(pr)
    # a key's weights over 40 rows sum to 1 in a map; window: 2 query heads read a key head; differential:
    # 2 output heads read the one value head, lambda is its initial value, 0.5
    want = 2.0 if op == "window" else 1.0
    tol = 2.1 * 2.0 ** -8 if dtype == "bf16" else 1e-6
    if op == "diff" and dtype == "bf16":
        tol *= 3                                    # the maps' weights are rounded each: (1 + 0.5) / (1 - 0.5)
    assert float((r["dv"].double() / want - 1).abs().max()) < tol


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_what_is_not_finite_shows_beside_rows_far_from_zero(bad, dtype):
    coords, cu = shell(101, 250, r=8)
    pr = Problem(coords, cu, 5, 4, 2, 32, DT[dtype], seed=102, bias="offset")
    pr.bias.table[:] = -1e9
    clean = run_window(pr)
    for x in (pr.q, pr.k, pr.v, pr.dout):
        x[11] = bad
    dirty = run_window(pr)
    cell = pr.win.id == pr.win.id[11]
    for x in ("out", "dq", "dk", "dv"):
        assert torch.equal(clean[x][~cell], dirty[x][~cell]), x
        assert not bool(torch.isfinite(dirty[x][11]).any()), x
        assert x == "out" or not bool(torch.isfinite(dirty[x][cell]).any()), x


@pytest.mark.parametrize("op", ["window", "diff"])
def test_a_workspace_for_tensors_serves_a_call_with_tensors(op):
    """Nothing is allocated beside what the caller gives; from checkpoints the same workspace is too small."""
    coords, cu = shell(103, 300, r=9)
    pr = Problem(coords, cu, 6, 4, 2, 64, torch.bfloat16, seed=104, bias="offset")
    window = op == "window"
    need = pr.plan.workspace_size(ssa.OP_WINDOW_BACKWARD_TENSORS if window else ssa.OP_DIFF_BACKWARD_TENSORS, pr.p)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    grads = tuple(torch.empty_like(x) for x in (pr.q, pr.k, pr.v))
    last = torch.empty_like(pr.bias.table if window else pr.lam)

    def call(q, k, v):
        if window:
            return ssa.ssa_window_backward(pr.p, pr.plan, q, k, v, pr.dout, bias=pr.bias, grads=grads, dbias=last,
                                           workspace=ws)
        return ssa.ssa_diff_backward(pr.p, pr.plan, q, k, v, pr.lam, 0.5, pr.dout, grads=grads, dlam=last, workspace=ws)
    want = run_window(pr) if window else run_diff(pr)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    got = call(pr.q, pr.k, pr.v)
    torch.cuda.synchronize()
    assert torch.cuda.max_memory_allocated() == before
    for x, y in zip(got, ("dq", "dk", "dv", "dbias" if window else "dlam")):
        assert torch.equal(x, want[y]), y
    held = [ssa.ssa_act8_pack(x) for x in (pr.q, pr.k, pr.v)]
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    call(*held)
    assert torch.cuda.max_memory_allocated() > before


def test_plans_whose_arrays_have_other_sizes_are_refused():
    coords, cu = shell(105, 200)
    pr = Problem(coords, cu, 4, 2, 1, 32, torch.float32, seed=106)
    ok = pr.plan
    for bad, what in ((ssa.WindowPlan(ok.rows, ok.tiles[:-1].contiguous(), ok.n, ok.count, ok.m), "tiles"),
                      (ssa.WindowPlan(ok.rows.long(), ok.tiles, ok.n, ok.count, ok.m), "rows"),
                      (ssa.WindowPlan(ok.rows, ok.tiles, ok.n, ok.count + 1, ok.m), "tiles"),
                      (ssa.WindowPlan(ok.rows.cpu(), ok.tiles, ok.n, ok.count, ok.m), "CUDA")):
        for call in (lambda: ssa.ssa_window_forward(pr.p, bad, pr.q, pr.k, pr.v),
                     lambda: ssa.ssa_window_backward(pr.p, bad, pr.q, pr.k, pr.v, pr.dout)):
            with pytest.raises(ValueError, match=what):
                call()
    with pytest.raises(AttributeError):          # the library would go on reading the old array
        ok.tiles = ok.tiles.clone()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("op", ["window", "diff"])
def test_results_in_the_place_of_what_they_replace(op, dtype):
    """out = q, dk = k, dv = v: the same bits."""
    coords, cu = dense(107, 420, 8)
    pr = Problem(coords, cu, 8, 4, 2, 64, DT[dtype], seed=108, bias="offset" if op == "window" else None)
    want = (run_window if op == "window" else run_diff)(pr)
    q, k, v, dq = pr.q.clone(), pr.k.clone(), pr.v.clone(), torch.empty_like(pr.q)
    if op == "window":
        ssa.ssa_window_backward(pr.p, pr.plan, pr.q, k, v, pr.dout, bias=pr.bias, grads=(dq, k, v))
        ssa.ssa_window_forward(pr.p, pr.plan, q, pr.k, pr.v, bias=pr.bias, out=q)
    else:
        ssa.ssa_diff_backward(pr.p, pr.plan, pr.q, k, v, pr.lam, 0.5, pr.dout, grads=(dq, k, v))
        ssa.ssa_diff_forward(pr.p, pr.plan, q, pr.k, pr.v, pr.lam, 0.5, out=q)
    for x, y in ((q, "out"), (dq, "dq"), (k, "dk"), (v, "dv")):
        assert torch.equal(x, want[y]), y
    with pytest.raises(ssa.SSAError, match="INVALID_ARG"):
        ssa.ssa_window_backward(pr.p, pr.plan, q, pr.k, pr.v, pr.dout, grads=(q, k, v))


@pytest.mark.parametrize("n,side,m,hq,hkv", [(500, 8, 6, 5, 1), (32, 4, 5, 16, 2), (111, 6, 12, 3, 3)])
def test_bias_gradient_of_few_rows_in_a_fine_unit(n, side, m, hq, hkv):
    """Sharp softmaxes: offsets whose dS are all small keep their bounds and the roundings of the fixed point.
    A CTA of few rows has a unit of 2^-41 of the largest |dP|, below 2^6 here: 2^-35.  At most n adds per
    offset, independent and uniform within half a unit: six times the root of n / 12 units."""
    coords, cu = dense(109, n, side)
    pr = Problem(coords, cu, m, hq, hkv, 64, torch.bfloat16, seed=110, bias="offset", std=4.0)
    got, (value, bound) = run_window(pr)["dbias"], pr.ref_window()["dbias"]
    err = np.abs(got.double().cpu().numpy() - value)
    assert np.all(err <= bound + 6 * (n / 12) ** 0.5 * 2.0 ** -35)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m,crowd,far", [(5, 0, 0.0), (14, 0, 0.0), (4, 3000, 0.0), (5, 0, -1e9), (14, 0, -1e9)])
def test_a_bias_that_is_not_trained(m, crowd, far, dtype):
    """Without the bias gradient the others are the same bits."""
    coords, cu = shell(111, 300, r=9)
    if crowd:
        coords = np.concatenate([coords, np.repeat(coords[100:101], crowd, 0)])
        cu = np.array([0, len(coords)], np.int32)
    pr = Problem(coords, cu, m, 4, 2, 32, DT[dtype], seed=112, bias="offset")
    pr.bias.table += far
    want = run_window(pr)
    *got, none = ssa.ssa_window_backward(pr.p, pr.plan, pr.q, pr.k, pr.v, pr.dout, bias=pr.bias, dbias=False)
    assert none is None and ssa.device_status() == 0
    for x, y in zip(got, ("dq", "dk", "dv")):
        assert torch.equal(x, want[y]), y


def test_bias_gradient_of_a_lone_crowded_item_after_64_bit_sums_only():
    """512 heads, so one CTA to two heads: its first batch holds only a cell for the 64-bit sums, the next
    begins with a cell of two voxels of 2000 equal tokens each.  Equal dS leave equal remainders, whose sums
    are as large as their bound.  Two kinds of rows and of keys, so the oracle's bounds in closed form."""
    coords = np.concatenate([np.tile([[0, 0, 0]], (5000, 1)), np.tile([[4, 0, 0]], (2000, 1)),
                             np.tile([[5, 0, 0]], (2000, 1))]).astype(np.int32)
    pr = Problem(coords, np.array([0, 9000], np.int32), 4, 2, 2, 32, torch.bfloat16, seed=113)
    gen = torch.Generator(device="cuda").manual_seed(114)
    f = lambda *x: torch.randn(*x, generator=gen, device="cuda")  # noqa: E731
    pr.hq, pr.p = 512, ssa.make_window_params(512, 2, 32, torch.bfloat16)
    pr.q, pr.dout = (f(9000, 512, 32).bfloat16() for _ in range(2))
    for x in (pr.q, pr.dout, pr.k, pr.v):
        x[5000:7000], x[7000:] = x[5000].clone(), x[7000].clone()
    pr.bias = ssa.WindowBias(0.5 * f(512, 343))
    got = ssa.ssa_window_backward(pr.p, pr.plan, pr.q, pr.k, pr.v, pr.dout, bias=pr.bias)[3].double().cpu()
    off, eps, kind = torch.tensor([[171, 122], [220, 171]]), 2.0 ** -24, [5000, 7000]   # one voxel along x: 49
    for h in range(0, 512, 7):
        q, k, v, do = (x[kind, y].double().cpu() for x, y in ((pr.q, h), (pr.k, h // 256), (pr.v, h // 256), (pr.dout, h)))
        t = pr.bias.table[h].double().cpu()[off]
        p = torch.softmax(q @ k.T / np.sqrt(32) + t, 1)          # of all 2000 keys of a kind
        dp, mag = do @ v.T, do.abs() @ v.abs().T
        D = (p * dp).sum(1, keepdim=True)
        ep = 2 * 36 * eps * (q.abs() @ k.abs().T / np.sqrt(32) + t.abs()).amax(1, keepdim=True) + 2.0 ** -20
        eD = (p * (dp.abs() * (ep + 4000 * eps) + 36 * eps * mag)).sum(1, keepdim=True)
        ds = p * (dp - D)
        err = p * ((dp - D).abs() * (ep + 4 * eps) + 36 * eps * mag + eD) + ds.abs() * 4000 * eps
        for a, b in ((0, 1), (1, 0)):
            assert abs(float(got[h, off[a, b]] - 2000 * ds[a, b])) <= 2000 * float(err[a, b]), (h, a)
