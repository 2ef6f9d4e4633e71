"""Cases of the window operators: attention inside the cells of a voxel partition with a
learned relative position bias, differential attention inside the cells, and 8-bit
checkpoints of Q, K, V with the backward pass that reads them.

A case fixes the sizes; `prepare` draws voxel sets and tensors from a seed, `run` is one
pass through an operator (its plain form in elementary torch operations, or with `own`
the library's kernels), `exact` the same from the definition in 64 bits.

Formulas.  Token i of a window w has the coordinate c_i; head h of the queries reads
key head h // (hq // hkv).

  window   s_ij = scale <q_i, k_j> + b[h, bucket(c_i - c_j)],  p_i = softmax_j(s_ij) over
           the tokens j of i's window,  o_i = sum_j p_ij v_j; the gradients of sum(dout o)
           with respect to q, k, v and b.
  diff     head pairs (2h, 2h+1) of q and of k are two maps a1, a2 (softmax as above, no
           bias) over one value head of width 2 d:  o_i = sum_j (a1_ij - lam_h a2_ij) v_j,
           lam_h = exp(<l[0,h], l[1,h]>) - exp(<l[2,h], l[3,h]>) + lam_init; the gradients
           with respect to q, k, v and l.
  act8     a row x [d] is held as whole numbers n in [-127, 127] and a power of two s, the
           smallest with |x| <= 127 s:  n = round(x / s), ties to even, value n s.  The
           window backward reads such rows in place of q, k, v and is exact at the values
           they hold.
"""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
LAM_INIT = 0.5


def _case(name, op, mode, n, seqs, hq, hkv, d, m, dtype, shape="shell", bias="offset"):
    c = {"op": op, "mode": mode, "n": n, "seqs": seqs, "hq": hq, "hkv": hkv, "d": d, "m": m, "dtype": dtype,
         "shape": shape, "bias": bias}
    return dict(c, name=name) if name else c


def listed():
    return [
        # the small fp32 voxel set of the first configuration (2048 tokens, windows of edge 4): latency
        _case("window fwd 2k f32", "window", "fwd", 2048, 1, 2, 1, 32, 4, "f32"),
        # the benchmark's surface shell in inference: one large bf16 shape
        _case("window fwd 131k", "window", "fwd", 131072, 1, 32, 2, 64, 8, "bf16"),
        # the same in training, forward and backward with the gradient of the bias
        _case("window train 131k", "window", "train", 131072, 1, 32, 2, 64, 8, "bf16"),
        # a ragged batch of four shapes in training, offsets in logarithmic buckets
        _case("window train 4 shapes", "window", "train", 100003, 4, 16, 2, 64, 8, "bf16", "shell", "log"),
        # a filled volume: windows of several hundred tokens, head dim 128
        _case("window train dense", "window", "train", 24576, 1, 16, 2, 128, 8, "bf16", "dense"),
        # fp32 training of a small model, odd sizes, several shapes
        _case("window train f32", "window", "train", 20011, 3, 8, 2, 32, 6, "f32"),
        # differential attention of a small voxel set: latency
        _case("diff fwd 2k", "diff", "fwd", 2048, 1, 8, 4, 32, 4, "bf16"),
        # differential attention of the benchmark's shell in training
        _case("diff train 131k", "diff", "train", 131072, 1, 32, 2, 64, 8, "bf16"),
        # fp32 differential attention of an odd batch in training
        _case("diff train f32", "diff", "train", 9001, 3, 8, 2, 32, 5, "f32"),
        # Q, K, V of the benchmark's shell into 8 bits and back
        _case("act8 round trip 131k", "act8", "pack", 131072, 1, 32, 2, 64, 8, "bf16"),
        # the backward of the benchmark's shell from 8-bit checkpoints
        _case("act8 window bwd 131k", "act8", "bwd", 131072, 1, 32, 2, 64, 8, "bf16"),
        # the same for a small odd batch
        _case("act8 window bwd 5k", "act8", "bwd", 5003, 2, 16, 4, 32, 5, "bf16", "shell", "log"),
    ]


def draw(rng):
    op, mode = rng.choice([("window", "fwd"), ("window", "train"), ("diff", "fwd"), ("diff", "train"),
                           ("act8", "pack"), ("act8", "bwd")])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    d = rng.choice([32, 64] if op == "diff" else [32, 64, 128])
    hkv = rng.choice([2, 4] if op == "diff" else [1, 2, 4])
    g = rng.choice([1, 2, 3, 4, 8, 16])
    while hkv * g * d > 2048:
        g = max(1, g // 2)
    shape = rng.choice(["shell", "shell", "dense"])
    m = rng.randint(2, 8 if shape == "dense" else 10)
    top = (8192 if dtype == "f32" else 24576) if shape == "dense" else 20011 if dtype == "f32" else 131072 if m <= 8 else 65536
    n = int(round(math.exp(rng.uniform(0.0, math.log(top)))))
    return _case(None, op, mode, max(1, min(n, top)), min(rng.randint(1, 5), max(1, n // 2)), hkv * g, hkv, d,
                 m, dtype, shape, rng.choice(["offset", "log"]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _sizes(n, s):
    """n tokens over s sequences of unequal lengths (the last ones shorter)."""
    w = [1.0 / (1 + i) for i in range(s)]
    c = [max(1, int(n * x / sum(w))) for x in w]
    c[0] += n - sum(c)
    return c


def _voxels(c, gen):
    """int32 coordinates [n, 3] in raster order within each sequence, offsets [s + 1]: the
    voxels of an ellipsoid's surface, or of a filled cube, a random part of them kept."""
    out = []
    sizes = _sizes(c["n"], c["seqs"])
    for n in sizes:
        if c["shape"] == "dense":
            side = max(1, math.ceil((n / 0.7) ** (1 / 3)))
            key = torch.arange(side ** 3, device=DEVICE)
            key = ((key // (side * side)) * 2048 + key // side % side) * 2048 + key % side
        else:
            r = math.sqrt(n / (4 * math.pi)) + 1.0
            u = torch.randn(4 * n + 64, 3, generator=gen, device=DEVICE)
            u = u / u.norm(dim=1, keepdim=True).clamp_min(1e-6)
            axes = r * (0.85 + 0.3 * torch.rand(3, generator=gen, device=DEVICE))
            x = (u * axes + 1.2 * r + 1.0).floor().long()
            key = torch.unique((x[:, 0] * 2048 + x[:, 1]) * 2048 + x[:, 2])
        pick = torch.randperm(key.numel(), generator=gen, device=DEVICE)
        pick = pick[torch.arange(n, device=DEVICE) % key.numel()]
        key = torch.sort(key[pick])[0]
        out.append(torch.stack([key // (2048 * 2048), key // 2048 % 2048, key % 2048], 1))
    cu = np.concatenate([[0], np.cumsum(sizes)])
    return torch.cat(out).to(torch.int32), torch.from_numpy(cu.astype(np.int32)).to(DEVICE)


def _cells(coords, cu, m):
    """perm (tokens sorted by window) and ptr (a window's range of perm)."""
    seq = torch.searchsorted(cu[1:].long(), torch.arange(coords.shape[0], device=coords.device), right=True)
    c = coords.long() // m
    key = ((seq * 2048 + c[:, 0]) * 2048 + c[:, 1]) * 2048 + c[:, 2]
    _, inv, cnt = torch.unique(key, return_inverse=True, return_counts=True)
    perm = torch.argsort(inv, stable=True)
    ptr = torch.cat([torch.zeros(1, dtype=torch.long, device=coords.device), cnt.cumsum(0)])
    return perm, ptr


def _buckets(m, kind):
    """Bucket of each of the (2m-1)^3 offsets, int32, and their number: every offset its own,
    or per axis the signed power of two that holds it."""
    e = 2 * m - 1
    if kind == "offset":
        return torch.arange(e ** 3, dtype=torch.int32, device=DEVICE), e ** 3
    a = torch.arange(e, device=DEVICE) - (m - 1)
    mag = torch.where(a == 0, 0, torch.floor(torch.log2(a.abs().clamp_min(1).double())).long() + 1)
    top = int(mag.max())
    axis = mag * a.sign() + top
    k = 2 * top + 1
    b = (axis[:, None, None] * k + axis[None, :, None]) * k + axis[None, None, :]
    return b.reshape(-1).to(torch.int32), k ** 3


def _dtype(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def _make(c, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(1000003 * int(seed) + 17)
    coords, cu = _voxels(c, gen)
    n, hq, hkv, d = c["n"], c["hq"], c["hkv"], c["d"]
    f = lambda *s: torch.randn(*s, generator=gen, device=DEVICE)  # noqa: E731
    t = {"coords": coords, "cu": cu}
    for name, h in (("q", hq), ("k", hkv), ("v", hkv), ("dout", hq)):
        t[name] = f(n, h, d).to(_dtype(c))
    if c["op"] == "diff":
        t["lam"] = 0.1 * f(4, hq // 2, d)
    else:
        t["bucket"], nb = _buckets(c["m"], c["bias"])
        t["bias"] = 0.5 * f(hq, nb)
    return t


def prepare(case, seed):
    c = case
    t = _make(c, seed)
    perm, ptr = _cells(t["coords"], t["cu"], c["m"])
    n, cnt = c["n"], ptr[1:] - ptr[:-1]
    longest = int(cnt.max())
    col = torch.arange(longest, device=DEVICE)
    t["live"] = col[None] < cnt[:, None]                                         # [windows, longest]
    t["slot"] = perm[(ptr[:-1, None] + col[None]).clamp_max(n - 1)]              # token of each slot
    if c["op"] != "diff":
        x = (t["coords"].long() % c["m"])
        e = 2 * c["m"] - 1
        t["code"] = (x[:, 0] * e + x[:, 1]) * e + x[:, 2]
    if c["op"] == "act8" and c["mode"] == "bwd":
        t["held"] = {name: _pack(t[name]) for name in "qkv"}
    t["case"] = c
    if own:
        from spatial_sparse_attention_ssa_b200 import ssa
        _, win = ssa.ssa_bin(t["coords"], t["cu"], 2048, c["m"], c["m"])
        t["plan"] = ssa.ssa_window_plan(t["coords"], win, c["m"])
        t["p"] = ssa.make_window_params(c["hq"], c["hkv"], c["d"], _dtype(c))
        if c["op"] == "act8" and c["mode"] == "bwd":
            t["act8"] = tuple(ssa.Act8(*t["held"][name]) for name in "qkv")
        if c["bias"] == "offset":
            t["bucket"] = None
    return t


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------


def _pack(x):
    """Whole numbers int8 [.., d] and the power-of-two step of each row, fp32 [..]."""
    top = x.float().abs().amax(-1)
    mant, expo = torch.frexp(top)
    # 127 s >= top: s = 2^(expo - 7) holds mantissas up to 127/128, else the next power
    expo = expo - 7 + (mant > 127.0 / 128.0).int()
    s = torch.where(top > 0, torch.ldexp(torch.ones_like(top), expo), torch.ones_like(top))
    s = s.clamp_min(2.0 ** -126)
    return torch.round(x.float() / s[..., None]).to(torch.int8), s


def _unpack(held, dtype):
    return (held[0].float() * held[1][..., None]).to(dtype)


def _slots(x, s):
    """[n, h, w] -> fp32 [windows, h, longest, w], zeros where a window has no token."""
    return (x.float()[s["slot"]] * s["live"][..., None, None]).transpose(1, 2).contiguous()


def _tokens(x, s, dtype):
    """[windows, h, longest, w] -> [n, h, w]: each slot's row back at its token."""
    c = s["case"]
    out = torch.empty(c["n"], x.shape[1], x.shape[3], dtype=dtype, device=x.device)
    out[s["slot"][s["live"]]] = x.transpose(1, 2)[s["live"]].to(dtype)
    return out


def _softmax(q, k, bias, s):
    """Probabilities [windows, hq, longest, longest] of q against k (key heads already repeated)."""
    x = q @ k.transpose(2, 3) / math.sqrt(s["case"]["d"])
    if bias is not None:
        x = x + bias
    x = torch.where(s["live"][:, None, None, :], x, float("-inf"))
    x = torch.exp(x - x.amax(-1, keepdim=True))
    return x / x.sum(-1, keepdim=True) * s["live"][:, None, :, None]


def _offsets(s):
    """Bucket of each pair of slots [windows, longest, longest]."""
    m = s["case"]["m"]
    e = 2 * m - 1
    code = s["code"][s["slot"]]
    off = code[:, :, None] - code[:, None, :] + (m - 1) * (e * e + e + 1)
    # slots without a token repeat another window's token: any bucket will do, nothing is added there
    return s["bucket"].long()[off.clamp(0, e ** 3 - 1)] if s["bucket"] is not None else off.clamp(0, e ** 3 - 1)


def _rep(x, g):
    return x.repeat_interleave(g, dim=1)


def _fold(x, g):
    """Sum of the query heads that share a key head."""
    return x.reshape(x.shape[0], -1, g, *x.shape[2:]).sum(2)


def _window_plain(s, q, k, v, want_out, want_grad):
    c = s["case"]
    g, dt = c["hq"] // c["hkv"], _dtype(c)
    off = _offsets(s)
    qs, ks, vs = _slots(q, s), _rep(_slots(k, s), g), _rep(_slots(v, s), g)
    p = _softmax(qs, ks, s["bias"][:, off].transpose(0, 1), s)
    r = {}
    if want_out:
        r["out"] = _tokens(p @ vs, s, dt)
    if want_grad:
        do = _slots(s["dout"], s)
        ds = do @ vs.transpose(2, 3)
        r["dv"] = _tokens(_fold(p.transpose(2, 3) @ do, g), s, dt)
        ds = p * (ds - (p * ds).sum(-1, keepdim=True))
        del p
        r["dq"] = _tokens(ds @ ks / math.sqrt(c["d"]), s, dt)
        r["dk"] = _tokens(_fold(ds.transpose(2, 3) @ qs, g) / math.sqrt(c["d"]), s, dt)
        db = torch.zeros(s["bias"].shape, dtype=torch.float64, device=DEVICE)
        db.index_add_(1, off.reshape(-1), ds.transpose(0, 1).reshape(c["hq"], -1).double())
        r["dbias"] = db.float()
    return r


def _lam(s):
    x = s["lam"]
    return torch.exp((x[0] * x[1]).sum(-1)), torch.exp((x[2] * x[3]).sum(-1))


def _diff_plain(s, want_grad):
    c = s["case"]
    g, dt, n, d = c["hq"] // c["hkv"], _dtype(c), c["n"], c["d"]
    hd = c["hq"] // 2
    e1, e2 = _lam(s)
    lam = (e1 - e2 + LAM_INIT)[None, :, None, None]
    qs, ks = _slots(s["q"], s), _slots(s["k"], s)
    q1, q2, k1, k2 = qs[:, 0::2], qs[:, 1::2], _rep(ks[:, 0::2], g), _rep(ks[:, 1::2], g)
    vs = _rep(_slots(s["v"].reshape(n, -1, 2 * d), s), g)
    a1, a2 = _softmax(q1, k1, None, s), _softmax(q2, k2, None, s)
    p = a1 - lam * a2
    r = {"out": _tokens(p @ vs, s, dt).reshape(n, c["hq"], d)}
    if want_grad:
        do = _slots(s["dout"].reshape(n, hd, 2 * d), s)
        dp = do @ vs.transpose(2, 3)
        r["dv"] = _tokens(_fold(p.transpose(2, 3) @ do, g), s, dt).reshape(n, c["hkv"], d)
        del p
        r1, r2 = (a1 * dp).sum(-1, keepdim=True), (a2 * dp).sum(-1, keepdim=True)
        d1, d2 = a1 * (dp - r1) / math.sqrt(d), -lam * a2 * (dp - r2) / math.sqrt(d)
        r["dq"] = _tokens(torch.stack([d1 @ k1, d2 @ k2], 2).flatten(1, 2), s, dt)
        x = torch.stack([_fold(d1.transpose(2, 3) @ q1, g), _fold(d2.transpose(2, 3) @ q2, g)], 2)
        r["dk"] = _tokens(x.flatten(1, 2), s, dt)
        dl = -(r2[..., 0].double().sum((0, 2))).float()
        x = s["lam"]
        y1, y2 = (dl * e1)[:, None], (-dl * e2)[:, None]
        r["dlam"] = torch.stack([y1 * x[1], y1 * x[0], y2 * x[3], y2 * x[2]])
    return r


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------


def run(state):
    s, c = state, state["case"]
    if not own:
        if c["op"] == "window":
            return _window_plain(s, s["q"], s["k"], s["v"], True, c["mode"] == "train")
        if c["op"] == "diff":
            return _diff_plain(s, c["mode"] == "train")
        if c["mode"] == "pack":
            held = {x: _pack(s[x]) for x in "qkv"}
            return {x: _unpack(held[x], _dtype(c)) for x in "qkv"}
        return _window_plain(s, *(_unpack(s["held"][x], torch.float32) for x in "qkv"), False, True)
    from spatial_sparse_attention_ssa_b200 import ssa
    p, plan = s["p"], s["plan"]
    if c["op"] == "window":
        bias = ssa.WindowBias(s["bias"], s["bucket"])
        r = {"out": ssa.ssa_window_forward(p, plan, s["q"], s["k"], s["v"], bias=bias)}
        if c["mode"] == "train":
            r["dq"], r["dk"], r["dv"], r["dbias"] = ssa.ssa_window_backward(p, plan, s["q"], s["k"], s["v"],
                                                                            s["dout"], bias=bias)
        return r
    if c["op"] == "diff":
        r = {"out": ssa.ssa_diff_forward(p, plan, s["q"], s["k"], s["v"], s["lam"], LAM_INIT)}
        if c["mode"] == "train":
            r["dq"], r["dk"], r["dv"], r["dlam"] = ssa.ssa_diff_backward(p, plan, s["q"], s["k"], s["v"], s["lam"],
                                                                         LAM_INIT, s["dout"])
        return r
    if c["mode"] == "pack":
        held = {x: ssa.ssa_act8_pack(s[x]) for x in "qkv"}
        return {x: ssa.ssa_act8_unpack(held[x], _dtype(c)) for x in "qkv"}
    q, k, v = s["act8"]
    bias = ssa.WindowBias(s["bias"], s["bucket"])
    r = {}
    r["dq"], r["dk"], r["dv"], r["dbias"] = ssa.ssa_window_backward(p, plan, q, k, v, s["dout"], bias=bias)
    return r


def work(case):
    """One pass: each input read once, each output written once; 2 flops per product of the
    contractions (scores and values forward, five of them backward) over the pairs of tokens
    of a window, counted on the voxel set of seed 0."""
    c = case
    n, hq, hkv, d = c["n"], c["hq"], c["hkv"], c["d"]
    w = 2 if c["dtype"] == "bf16" else 4
    rows_q, rows_k = n * hq * d, n * hkv * d
    if c["op"] == "act8" and c["mode"] == "pack":
        held = (rows_q + 2 * rows_k) + 4 * n * (hq + 2 * hkv)
        return {"bytes": 2 * (w * (rows_q + 2 * rows_k) + held), "flops": 0}
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(17)
    coords, cu = _voxels(c, gen)
    _, ptr = _cells(coords, cu, c["m"])
    pairs = float(((ptr[1:] - ptr[:-1]).double() ** 2).sum())
    table = 4 * hq * _buckets(c["m"], c["bias"])[1] if c["op"] != "diff" else 4 * 2 * hq * d
    plan = 8 * n
    fwd = w * (2 * rows_q + 2 * rows_k) + table + plan
    bwd = w * (2 * rows_q + 2 * rows_k) + w * (rows_q + 2 * rows_k) + 2 * table + plan
    if c["op"] == "act8":
        bwd += (1 - w) * (rows_q + 2 * rows_k) + 4 * n * (hq + 2 * hkv)
        return {"bytes": bwd, "flops": 10.0 * d * hq * pairs}
    if c["mode"] == "fwd":
        return {"bytes": fwd, "flops": 4.0 * d * hq * pairs}
    return {"bytes": fwd + bwd, "flops": 14.0 * d * hq * pairs}


# ---------------------------------------------------------------------------
# the definition in 64 bits, window by window, gradients by differentiation
# ---------------------------------------------------------------------------


def _round8(x):
    """Values of x [.., d] at 8 bits, from the definition: the smallest power of two s with
    |x| <= 127 s, n = the nearest whole number to x / s, ties to even."""
    x = x.double()
    top = x.abs().amax(-1, keepdim=True)
    s = torch.exp2(torch.ceil(torch.log2(torch.where(top > 0, top / 127.0, torch.ones_like(top)))))
    s = torch.where(127.0 * s / 2 >= top, s / 2, s)     # against the logarithm's own rounding
    s = torch.where(127.0 * s < top, s * 2, s)
    s = torch.where(top > 0, s, torch.ones_like(s)).clamp_min(2.0 ** -126)
    return torch.round(x / s) * s


def exact(case, seed):
    c = case
    t = _make(c, seed)
    if c["op"] == "act8" and c["mode"] == "pack":
        return {x: _round8(t[x]) for x in "qkv"}
    n, hq, hkv, d, m = c["n"], c["hq"], c["hkv"], c["d"], c["m"]
    g = hq // hkv
    grad = c["mode"] != "fwd"
    perm, ptr = _cells(t["coords"], t["cu"], m)
    edges = ptr.tolist()
    if len(edges) > 25000:
        return None
    src = {x: (_round8(t[x]) if c["op"] == "act8" else t[x].double()) for x in "qkv"}
    out = torch.empty(n, hq, d, dtype=torch.float64, device=DEVICE)
    gr = {x: torch.empty_like(src[x]) for x in "qkv"}
    par = (t["lam"] if c["op"] == "diff" else t["bias"]).double()
    dpar = torch.zeros_like(par)
    e = 2 * m - 1
    for a, b in zip(edges[:-1], edges[1:]):
        i = perm[a:b]
        q, k, v = (src[x][i].requires_grad_(grad) for x in "qkv")
        if c["op"] == "diff":
            w = par.clone().requires_grad_(grad)
            lam = torch.exp((w[0] * w[1]).sum(-1)) - torch.exp((w[2] * w[3]).sum(-1)) + LAM_INIT
            kk = k.reshape(b - a, hkv // 2, 1, 2, d).expand(-1, -1, g, -1, -1).reshape(b - a, hq, d)
            vv = v.reshape(b - a, hkv // 2, 1, 2 * d).expand(-1, -1, g, -1).reshape(b - a, hq // 2, 2 * d)
            z = torch.softmax(torch.einsum("ihd,jhd->hij", q, kk) / math.sqrt(d), -1)
            z = z[0::2] - lam[:, None, None] * z[1::2]
            o = torch.einsum("hij,jhe->ihe", z, vv).reshape(b - a, hq, d)
        else:
            x = t["coords"][i].long()
            off = x[:, None] - x[None] + (m - 1)
            off = t["bucket"].long()[(off[..., 0] * e + off[..., 1]) * e + off[..., 2]]
            w = par[:, off].requires_grad_(grad)
            kk, vv = (y[:, :, None].expand(-1, -1, g, -1).reshape(b - a, hq, d) for y in (k, v))
            z = torch.softmax(torch.einsum("ihd,jhd->hij", q, kk) / math.sqrt(d) + w, -1)
            o = torch.einsum("hij,jhd->ihd", z, vv)
        out[i] = o.detach()
        if grad:
            gq, gk, gv, gw = torch.autograd.grad((o * t["dout"][i].double()).sum(), (q, k, v, w))
            gr["q"][i], gr["k"][i], gr["v"][i] = gq, gk, gv
            if c["op"] == "diff":
                dpar += gw
            else:
                dpar.index_add_(1, off.reshape(-1), gw.reshape(hq, -1))
    r = {} if c["op"] == "act8" else {"out": out}
    if grad:
        r |= {"dq": gr["q"], "dk": gr["k"], "dv": gr["v"], "dlam" if c["op"] == "diff" else "dbias": dpar}
    return r
