"""Head norms with the position rotation, their gradients and the paged append against the
fp64 oracle (GPU, through the C ABI).

Tolerances. One fp32 rounding is u = 2^-24 relative. A normed row takes a sum of squares
(chains of at most 16 products a lane and 5 shuffles: < 24 u, halved by the root), a
division, a root and two products with the weight (< 6 u): < 18 u relative to the row's
values. A pair's rotation adds the angle's rounding (u half turns = pi u rad), cos and sin
within 2 units in the last place (4 u) and three roundings, all relative to the pair's
length: < 11 u. So |error| <= 32 u len(pair), with len the length of the pair that the
value belongs to, plus half a step of the result's type. Gradients: twice such factors, on
rstd (|w| + |n| mean |w n|): 64 u. dgamma: sums over at most 64 rows a lane, 5 shuffles
and the tiles, then fp64: (64 + 32) u of the sum of magnitudes, and a result's rounding."""
import numpy as np
import pytest
import torch

from oracle import dark_oracle as O

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module")
def D(cuda_ok):
    from random_feature_linear_b200 import dark
    return dark


def _t(rng, *shape, dtype=torch.float32, dev="cuda"):
    return torch.from_numpy(rng.standard_normal(shape)).to(dev).to(dtype)


def _np(t):
    return t.double().cpu().numpy()


def _pair_length(x, dims, inter):
    """For every value the length of its pair (its magnitude where it is not rotated)."""
    out = np.abs(x)
    if dims:
        ia, ib = O._pair_index(dims, inter)
        n = np.hypot(x[..., ia], x[..., ib])
        out[..., ia], out[..., ib] = n, n
    return out


def _heads(rng, B, L, counts, d, dtype, packed):
    if not packed:
        return [_t(rng, B, h, L, d, dtype=dtype) for h in counts]
    x = _t(rng, B, L, sum(counts) + 1, d, dtype=dtype).permute(0, 2, 1, 3)
    return list(torch.split(x[:, :-1], counts, dim=1))


BF, F = torch.bfloat16, torch.float32
# dtype, B, H, Hk, L, d, rot, interleaved, weight, packed, positions, base
CASES = {
    "one-token": (BF, 1, 1, 1, 1, 64, 64, False, "shared", False, "table", 1e4),
    "decode": (BF, 64, 8, 8, 1, 64, 64, False, "shared", False, "table", 1e4),
    "large-heads": (BF, 2, 8, 4, 100, 256, 256, False, "per_head", True, "table", 1e4),
    "partial-interleaved": (BF, 2, 4, 2, 67, 128, 64, True, "per_head", True, "table", 1e4),
    "odd-heads": (BF, 3, 3, 1, 37, 96, 48, False, "shared", False, "pos0", 5e5),
    "odd-sizes": (BF, 3, 5, 2, 37, 20, 6, True, "shared", True, "pos0", 1e4),
    "smallest": (BF, 2, 2, 1, 5, 4, 4, False, "shared", False, "table", 1e4),
    "no-rotation": (BF, 2, 4, 2, 33, 64, 0, False, "shared", False, None, 1e4),
    "no-weight": (BF, 2, 4, 2, 33, 64, 64, False, None, True, "table", 1e4),
    "queries-only": (BF, 2, 4, 0, 70, 80, 40, True, "shared", False, "table", 1e4),
    "f32": (F, 2, 4, 2, 67, 64, 64, False, "per_head", True, "table", 1e4),
    "f32-d256": (F, 1, 3, 3, 21, 256, 128, True, "shared", False, "pos0", 1e4),
    "f32-odd": (F, 2, 3, 2, 21, 44, 22, False, "per_head", False, "far", 1e4),
    "f32-d252": (F, 1, 2, 1, 19, 252, 250, True, "shared", True, "table", 1e4),
    "many-heads": (BF, 1, 40, 17, 9, 32, 32, False, "per_head", False, "table", 1e4),
    "many-tokens": (BF, 3, 2, 1, 5000, 32, 16, False, "shared", False, "table", 1e4),
    "far": (BF, 1, 2, 2, 40, 64, 64, False, "shared", False, "far", 1e4),
}


def _inputs(D, name):
    dtype, B, H, Hk, L, d, rot, inter, weight, packed, how, base = CASES[name]
    rng = np.random.default_rng(sum(map(ord, name)))
    counts = [H, Hk] if Hk else [H]
    q, *k = _heads(rng, B, L, counts, d, dtype, packed)
    # rows of very different sizes: the norm has to follow them
    q.mul_(torch.from_numpy(4.0 ** rng.integers(-4, 4, (B, 1, L, 1))).cuda())
    n = lambda heads: heads if weight == "per_head" else 1
    gam = [None if weight is None else 1.0 + 0.2 * _t(rng, n(h), d) for h in counts]
    pos0, pos = 0, None
    places = np.broadcast_to(np.arange(L), (B, L))
    if how == "table":
        places = rng.integers(0, 200000, (B, L))
        pos = torch.from_numpy(places.astype(np.int32)).cuda()
    elif how in ("pos0", "far"):
        pos0 = 1 << 30 if how == "far" else 777       # (fp64's own angle is good to 2^-22 there)
        places = pos0 + places
    rope = D.dark_rope_init(rot, base, 1.0, inter) if rot else None
    return dict(q=q, k=k[0] if k else None, gq=gam[0], gk=gam[1] if Hk else None, rope=rope,
                pos=pos, pos0=pos0, places=places, rng=rng, dtype=dtype, B=B, H=H, Hk=Hk, L=L, d=d,
                rot=rot, inter=inter, base=base, packed=packed)


def _close(got, ref, tol, dtype):
    lim = tol + (np.abs(ref) + tol) * HALF_STEP[dtype]
    assert np.all(np.isfinite(got))
    worst = (np.abs(got - ref) / np.maximum(lim, 1e-300)).max()
    assert worst <= 1.0, worst


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("name", list(CASES))
def test_forward(D, cuda_ok, name, in_place):
    i = _inputs(D, name)
    xs = [i["q"], i["k"]]
    want = []
    for x, g in zip(xs, (i["gq"], i["gk"])):
        if x is None:
            continue
        x = _np(x)
        ref = O.norm_rope(x, None if g is None else _np(g), 1e-5, i["places"], i["rot"], i["base"],
                          1.0, i["inter"])
        # the oracle's own angle at far places: position * 2^-53
        drift = float(np.max(np.abs(i["places"]))) * 2.0 ** -52
        want.append((ref, (32 * U + drift) * _pair_length(ref, i["rot"], i["inter"])))
    outs = xs if in_place else [None if x is None else torch.full(x.shape, float("nan"),
                                                                  dtype=x.dtype, device="cuda")
                                for x in xs]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    D.dark_qk_norm_rope_fwd(i["q"], i["k"], outs[0], outs[1], gamma_q=i["gq"], gamma_k=i["gk"],
                            eps=1e-5, rope=i["rope"], positions=i["pos"], pos0=i["pos0"],
                            dev_status=status)
    assert status.item() == 0
    for o, (ref, tol) in zip([o for o in outs if o is not None], want):
        _close(_np(o), ref, tol, i["dtype"])


@pytest.mark.parametrize("name", list(CASES))
def test_backward(D, cuda_ok, name):
    i = _inputs(D, name)
    rng, dtype, rot, inter = i["rng"], i["dtype"], i["rot"], i["inter"]
    counts = [i["H"], i["Hk"]] if i["Hk"] else [i["H"]]
    dys = _heads(rng, i["B"], i["L"], counts, i["d"], dtype, not i["packed"])
    dxs = [torch.full_like(t, float("nan")) for t in
           _heads(rng, i["B"], i["L"], counts, i["d"], dtype, i["packed"])]
    gammas = [i["gq"], i["gk"]][:len(counts)]
    dgs = [None if g is None else torch.full_like(g, float("nan")) for g in gammas]
    ws = D.alloc_qk_norm_rope_bwd_workspace(i["B"], i["H"], i["Hk"], i["L"], i["d"], "cuda")
    ws.fill_(0xff)                                    # no initial contents are promised
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    two = lambda x: (list(x) + [None])[:2]
    call = lambda: D.dark_qk_norm_rope_bwd(
        i["q"], i["k"], *two(dys), *two(dxs), gamma_q=i["gq"], gamma_k=i["gk"],
        dgamma_q=two(dgs)[0], dgamma_k=two(dgs)[1], eps=1e-5, rope=i["rope"], positions=i["pos"],
        pos0=i["pos0"], ws=ws, dev_status=status)
    call()
    assert status.item() == 0
    drift = float(np.max(np.abs(i["places"]))) * 2.0 ** -52
    for x, g, dy, dx, dg in zip([i["q"], i["k"]], gammas, dys, dxs, dgs):
        x, dy, gn = _np(x), _np(dy), None if g is None else _np(g)
        ref, rdg = O.norm_rope_backward(x, gn, 1e-5, i["places"], dy, rot, i["base"], 1.0, inter)
        wl = _pair_length(dy, rot, inter)
        if g is None:
            _close(_np(dx), ref, (64 * U + drift) * wl, dtype)
            continue
        w = wl * np.abs(gn)[None, :, None, :]
        rstd = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-5)
        n = np.abs(x) * rstd
        _close(_np(dx), ref, (64 * U + drift) * rstd * (w + n * (w * n).mean(-1, keepdims=True)),
               dtype)
        mag = (wl * n).sum(axis=(0, 2))
        if len(gn) == 1:
            mag = mag.sum(0, keepdims=True)
        _close(_np(dg), rdg.reshape(gn.shape), (96 * U + drift) * mag, torch.float32)
    # the same call again gives the same bits: no order of atomics in any sum
    before = [t.clone() for t in dxs + [g for g in dgs if g is not None]]
    call()
    for a, b in zip(before, dxs + [g for g in dgs if g is not None]):
        assert torch.equal(a, b)


@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("dtype,H,Hk,d", [(BF, 7, 1, 256), (BF, 12, 4, 64), (F, 2, 1, 128)])
def test_weight_gradients_of_many_tokens(D, cuda_ok, dtype, H, Hk, d, per_head):
    """Spans of 511 tokens a CTA and more, up to 511 rows a lane, against fp64 sums on the GPU. A
    lane's chain, 5 shuffles and 8 warps: below (511 + 13 + 80) u of the magnitudes' sum, with
    32 u and more of it for the rows' own values, as above."""
    L = 296 * 510 + 77
    g = torch.Generator("cuda").manual_seed(2)
    t = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.float32)
    q, dq, k, dk = (t(1, h, L, d).to(dtype) for h in (H, H, Hk, Hk))
    gq, gk = (1 + 0.2 * t(h if per_head else 1, d) for h in (H, Hk))
    outs = [torch.empty_like(x) for x in (q, k, gq, gk)]
    rope = D.dark_rope_init(d)
    ws = D.alloc_qk_norm_rope_bwd_workspace(1, H, Hk, L, d, "cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    D.dark_qk_norm_rope_bwd(q, k, dq, dk, outs[0], outs[1], gamma_q=gq, gamma_k=gk,
                            dgamma_q=outs[2], dgamma_k=outs[3], rope=rope, eps=1e-5, ws=ws,
                            dev_status=status)
    assert status.item() == 0
    pos = torch.arange(L, device="cuda", dtype=torch.float64)
    ang = pos[:, None] * 1e4 ** (-2.0 * torch.arange(d // 2, device="cuda", dtype=torch.float64) / d)
    c, s = ang.cos(), ang.sin()
    for x, dy, dg in ((q, dq, outs[2]), (k, dk, outs[3])):
        sums, mags = [], []
        for h in range(x.shape[1]):
            v, y = x[0, h].double(), dy[0, h].double()
            n = v * (v.square().mean(-1, keepdim=True) + 1e-5).rsqrt()
            a, b = y[:, :d // 2], y[:, d // 2:]
            u = torch.cat([a * c + b * s, b * c - a * s], 1)
            size = torch.hypot(a, b).repeat(1, 2)
            sums.append((u * n).sum(0))
            mags.append((size * n.abs()).sum(0))
        ref, mag = torch.stack(sums), torch.stack(mags)
        if not per_head:
            ref, mag = ref.sum(0, keepdim=True), mag.sum(0, keepdim=True)
        tol = (511 + 13 + 80) * U * mag + ref.abs() * U
        worst = ((dg.double() - ref).abs() / tol).max().item()
        assert worst <= 1.0, worst


def test_backward_in_place_and_broadcast_cotangent(D, cuda_ok):
    rng = np.random.default_rng(5)
    q = _t(rng, 2, 3, 40, 64, dtype=BF)
    dy = _t(rng, 2, 1, 1, 64, dtype=BF).expand(2, 3, 40, 64)       # strides of 0
    gamma = 1 + 0.1 * _t(rng, 1, 64)
    rope = D.dark_rope_init(64)
    ws = D.alloc_qk_norm_rope_bwd_workspace(2, 3, 0, 40, 64, "cuda")
    a, ga = torch.empty_like(q), torch.empty_like(gamma)
    D.dark_qk_norm_rope_bwd(q, None, dy, None, a, None, gamma_q=gamma, dgamma_q=ga, rope=rope, ws=ws)
    b, gb = dy.contiguous(), torch.empty_like(gamma)
    D.dark_qk_norm_rope_bwd(q, None, b, None, b, None, gamma_q=gamma, dgamma_q=gb, rope=rope, ws=ws)
    assert torch.equal(a, b) and torch.equal(ga, gb)
    with pytest.raises(D.DarkError):                  # a result that overlaps itself
        D.dark_qk_norm_rope_bwd(q, None, q, None, dy, None, gamma_q=gamma, dgamma_q=gb, rope=rope,
                                ws=ws)


def test_backward_into_the_inputs(D, cuda_ok):
    """dq and dk in the memory of q and k."""
    rng = np.random.default_rng(15)
    q, dq = (_t(rng, 2, 8, 400, 64, dtype=BF) for _ in range(2))
    k, dk = (_t(rng, 2, 3, 400, 64, dtype=BF) for _ in range(2))
    g, rope = [1 + 0.1 * _t(rng, n, 64) for n in (8, 1)], D.dark_rope_init(64)
    ws = D.alloc_qk_norm_rope_bwd_workspace(2, 8, 3, 400, 64, "cuda")
    res = []
    for x, y in ((torch.empty_like(q), torch.empty_like(k)), (q, k)):
        dg = [torch.empty_like(t) for t in g]
        D.dark_qk_norm_rope_bwd(q, k, dq, dk, x, y, gamma_q=g[0], gamma_k=g[1], dgamma_q=dg[0],
                                dgamma_k=dg[1], rope=rope, ws=ws)
        res.append([x, y] + dg)
    for a, b in zip(*res):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("shift", [1, 2, 4])
def test_misaligned_rows(D, cuda_ok, dtype, shift):
    """Views whose rows begin at any element give the aligned views' bits."""
    rng = np.random.default_rng(11)
    B, H, L, d = 2, 3, 9, 64
    gamma, rope = 1 + 0.1 * _t(rng, 1, d), D.dark_rope_init(d)

    def off(t):
        wide = torch.zeros(*t.shape[:3], d + 8, dtype=dtype, device="cuda")
        v = wide[..., shift:shift + d]
        v.copy_(t)
        return v
    q, dy = (_t(rng, B, H, L, d, dtype=dtype) for _ in range(2))
    ws = D.alloc_qk_norm_rope_bwd_workspace(B, H, 0, L, d, "cuda")
    res = []
    for f in (lambda t: t.clone(), off):
        x, g, y, dx = f(q), f(dy), f(torch.zeros_like(q)), f(torch.zeros_like(q))
        dg = torch.empty_like(gamma)
        D.dark_qk_norm_rope_fwd(x, None, y, None, gamma_q=gamma, rope=rope, pos0=3)
        D.dark_qk_norm_rope_bwd(x, None, g, None, dx, None, gamma_q=gamma, dgamma_q=dg, rope=rope,
                                pos0=3, ws=ws)
        kp, vp = (torch.zeros(2, H, 16, d, dtype=dtype, device="cuda") for _ in range(2))
        D.dark_kv_append(D.kv_cache(kp, vp), x, g,
                         torch.arange(2, dtype=torch.int32, device="cuda")[:, None].contiguous(),
                         torch.zeros(2, dtype=torch.int32, device="cuda"), gamma_k=gamma, rope=rope)
        res.append([y, dx, dg, kp, vp])
    half = 2 * HALF_STEP[dtype]                       # one step: other units, other sums' order
    for a, b in zip(*res):
        torch.testing.assert_close(a, b, rtol=half, atol=32 * U * 8)
    assert torch.equal(res[0][4], res[1][4])


def test_rows_around_the_result_stay(D, cuda_ok):
    """Results in a packed projection leave the values beside them alone."""
    rng = np.random.default_rng(6)
    packed = _t(rng, 2, 17, 6, 32, dtype=BF)
    keep = packed.clone()
    x = packed.permute(0, 2, 1, 3)
    D.dark_qk_norm_rope_fwd(x[:, :3], x[:, 3:4], x[:, :3], x[:, 3:4],
                            gamma_q=torch.ones(32, device="cuda"), rope=D.dark_rope_init(32))
    assert torch.equal(packed[:, :, 4:], keep[:, :, 4:])
    assert not torch.equal(packed[:, :, :4], keep[:, :, :4])


@pytest.mark.parametrize("bad", ["inf", "nan", "huge"])
def test_non_finite_rows_are_reported(D, cuda_ok, bad):
    q = torch.ones(1, 2, 5, 64, device="cuda")
    q[0, 1, 3, 7] = {"inf": float("inf"), "nan": float("nan"), "huge": 3e38}[bad]
    out = torch.empty_like(q)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = torch.ones(1, 64, device="cuda")
    D.dark_qk_norm_rope_fwd(q, None, out, None, gamma_q=g, rope=D.dark_rope_init(64),
                            dev_status=status)
    assert status.item() == D.DARK_ERR_NUMERIC
    rest = torch.ones(2, 5, dtype=torch.bool)
    rest[1, 3] = False
    assert torch.isfinite(out[0][rest.cuda()]).all()


def test_zero_rows(D, cuda_ok):
    """A row of zeros stays zero; its gradient is the cotangent over sqrt(eps)."""
    q = torch.zeros(1, 1, 3, 64, device="cuda")
    g = torch.ones(1, 64, device="cuda")
    out, dq, dg = torch.empty_like(q), torch.empty_like(q), torch.empty_like(g)
    D.dark_qk_norm_rope_fwd(q, None, out, None, gamma_q=g, eps=1e-4)
    assert not out.any()
    ws = D.alloc_qk_norm_rope_bwd_workspace(1, 1, 0, 3, 64, "cuda")
    D.dark_qk_norm_rope_bwd(q, None, torch.ones_like(q), None, dq, None, gamma_q=g, dgamma_q=dg,
                            eps=1e-4, ws=ws)
    torch.testing.assert_close(dq, torch.full_like(dq, 100.0), rtol=1e-6, atol=0)
    assert not dg.any()


@pytest.mark.parametrize("dtype", [BF, F])
def test_captured_calls_replay(D, cuda_ok, dtype):
    """Norm, gradient and append captured into one graph, replayed on new contents."""
    rng = np.random.default_rng(7)
    B, H, L, d, page = 3, 4, 20, 64, 16
    q, k, v, dq, dk = (_t(rng, B, H, L, d, dtype=dtype) for _ in range(5))
    gamma = 1 + 0.1 * _t(rng, H, d)
    rope = D.dark_rope_init(d)
    new = lambda t: torch.full_like(t, float("nan"))
    outs = [new(q), new(k), new(q), new(k), new(gamma), new(gamma)]
    table = torch.arange(B * 3, dtype=torch.int32, device="cuda").reshape(B, 3)
    lens = torch.tensor([0, 5, 17], dtype=torch.int32, device="cuda")
    kp, vp = (torch.zeros(B * 3, H, page, d, dtype=dtype, device="cuda") for _ in range(2))
    cache = D.kv_cache(kp, vp)
    ws = D.alloc_qk_norm_rope_bwd_workspace(B, H, H, L, d, "cuda")

    def step():
        D.dark_qk_norm_rope_fwd(q, k, outs[0], outs[1], gamma_q=gamma, gamma_k=gamma, rope=rope)
        D.dark_qk_norm_rope_bwd(q, k, dq, dk, outs[2], outs[3], gamma_q=gamma, gamma_k=gamma,
                                dgamma_q=outs[4], dgamma_k=outs[5], rope=rope, ws=ws)
        D.dark_kv_append(cache, k, v, table, lens, gamma_k=gamma, rope=rope)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in (q, k, v, dq, dk):
        t.copy_(_t(rng, B, H, L, d, dtype=dtype))
    lens.add_(2)
    step()
    want = [t.clone() for t in outs + [kp, vp]]
    for t in outs + [kp, vp]:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        assert torch.equal(a, b)
    for b in range(B):                                # places that this append writes
        for j in range(int(lens[b]), int(lens[b]) + L):
            p = int(table[b, j // page])
            assert torch.equal(kp[p, :, j % page], want[6][p, :, j % page])
            assert torch.equal(vp[p, :, j % page], want[7][p, :, j % page])


# ----------------------------------------------------------------- append --

# dtype, B, Hk, T, d, rot, interleaved, weight, page, have (per sequence), new, packed
APPENDS = {
    "one-token": (BF, 1, 1, 1, 64, 64, False, None, 16, [0], None, False),
    "decode": (BF, 5, 8, 1, 64, 64, False, "shared", 64, [0, 63, 64, 65, 200], None, False),
    "ragged": (BF, 4, 2, 50, 128, 64, True, "per_head", 32, [0, 31, 5, 100], [50, 0, -3, 17], True),
    "longer-than-T": (BF, 2, 2, 9, 64, 64, False, None, 24, [3, 30], [99, 9], True),
    "odd-pages": (BF, 3, 3, 41, 40, 20, False, None, 7, [0, 6, 20], [41, 40, 1], False),
    "f32": (F, 3, 3, 33, 40, 20, False, "shared", 24, [1, 2, 3], [33, 20, 7], True),
    "f32-plain": (F, 2, 1, 33, 256, 0, False, None, 128, [120, 0], None, False),
    "page-of-one": (BF, 2, 2, 5, 20, 20, True, "shared", 1, [0, 3], None, False),
}


@pytest.mark.parametrize("name", list(APPENDS))
def test_append(D, cuda_ok, name):
    dtype, B, Hk, T, d, rot, inter, weight, page, have, new, packed = APPENDS[name]
    rng = np.random.default_rng(sum(map(ord, name)))
    k, v = _heads(rng, B, T, [Hk, Hk], d, dtype, packed)
    per = -(-(max(have) + T) // page)
    n = B * per + 2
    table = rng.permutation(n)[:B * per].reshape(B, per).astype(np.int32)
    kp, vp = (_t(rng, n, Hk, page, d, dtype=dtype) for _ in range(2))
    gamma = None if weight is None else 1 + 0.2 * _t(rng, Hk if weight == "per_head" else 1, d)
    places = np.array(have)[:, None] + np.arange(T) + 1000
    keys = O.norm_rope(_np(k), None if gamma is None else _np(gamma), 1e-5, places, rot,
                       interleaved=inter)
    rk, rv = O.kv_append(_np(kp), _np(vp), keys, _np(v), table, have, new)
    wrote = O.kv_append(np.zeros(kp.shape), np.zeros(vp.shape), np.ones(k.shape), np.ones(v.shape),
                        table, have, new)[0] != 0
    len_k = O.kv_append(np.zeros(kp.shape), np.zeros(vp.shape), _pair_length(keys, rot, inter),
                        np.zeros(v.shape), table, have, new)[0]
    before = kp.clone()
    i32 = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    if new is not None:                               # tokens that stay out are not read
        for b in range(B):
            k[b, :, max(0, new[b]):] = float("nan")
            v[b, :, max(0, new[b]):] = float("nan")
    D.dark_kv_append(D.kv_cache(kp, vp), k, v, i32(table), i32(have), new_lens=i32(new),
                     gamma_k=gamma, eps=1e-5, rope=D.dark_rope_init(rot, 1e4, 1.0, inter), pos0=1000,
                     dev_status=status)
    assert status.item() == 0
    np.testing.assert_array_equal(_np(vp), rv)
    assert torch.equal(kp[~torch.from_numpy(wrote).cuda()], before[~torch.from_numpy(wrote).cuda()])
    if rot == 0 and gamma is None:
        np.testing.assert_array_equal(_np(kp), rk)
    else:
        got = _np(kp)
        _close(got[wrote], rk[wrote], 32 * U * len_k[wrote], dtype)


def test_append_takes_positions(D, cuda_ok):
    rng = np.random.default_rng(8)
    k, v = (_t(rng, 2, 2, 3, 64) for _ in range(2))
    pos = rng.integers(0, 5000, (2, 3)).astype(np.int32)
    kp, vp = (torch.zeros(4, 2, 16, 64, device="cuda") for _ in range(2))
    table = torch.tensor([[2], [0]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([4, 0], dtype=torch.int32, device="cuda")
    D.dark_kv_append(D.kv_cache(kp, vp), k, v, table, lens, rope=D.dark_rope_init(64),
                     positions=torch.from_numpy(pos).cuda())
    ref = O.rotate(_np(k), pos, 64)
    for b, (p, at) in enumerate([(2, 4), (0, 0)]):
        _close(_np(kp[p, :, at:at + 3]), ref[b], 32 * U * _pair_length(ref[b], 64, False), F)


def test_append_reports_places_without_a_page(D, cuda_ok):
    rng = np.random.default_rng(9)
    k, v = (_t(rng, 4, 1, 4, 64, dtype=BF) for _ in range(2))
    kp, vp = (torch.zeros(8, 1, 4, 64, dtype=BF, device="cuda") for _ in range(2))
    # a page number past the cache, a negative one, a negative length, a list that ends
    table = torch.tensor([[8, 1], [-1, 2], [3, 4], [5, 6]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([2, 0, -2, 6], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    D.dark_kv_append(D.kv_cache(kp, vp), k, v, table, lens, dev_status=status)
    assert status.item() == D.DARK_ERR_INVALID_ARG
    want = torch.zeros_like(vp)
    want[1, 0, :2] = v[0, 0, 2:]
    want[6, 0, 2:] = v[3, 0, :2]
    assert torch.equal(vp, want)
    # the same lists with lengths that fit: nothing to report
    status.zero_()
    D.dark_kv_append(D.kv_cache(kp, vp), k, v, table.clamp(0, 7), lens.clamp(0, 4), dev_status=status)
    assert status.item() == 0
