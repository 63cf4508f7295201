"""Cases of the serving and training operators around the exact learned-kernel mode.

Three operators, each with a plain form (elementary torch operations in fp32, angles in
fp64) and the library's own calls:

* per-head RMS norms of queries and keys with the position rotation in the same pass, and
  the backward pass of both (``norm_rope``, ``norm_rope_grad``);
* appending keys and values to a paged cache, keys normed and rotated on the way
  (``append``);
* exact-mode attention of a batch over that cache, where all sequences share one long
  prefix (``attend``): out = softmax(q^T Sigma k / sqrt(d)) v with Sigma = M^T M.

Formulas, for a head row x of d values at position p (gamma, eps, base given):
    y = x * gamma / sqrt(mean(x^2) + eps)              (without gamma: y = x)
    (a, b) -> (a cos t - b sin t, a sin t + b cos t),  t = p * base^(-2 i / rot)
for the i-th pair of the first `rot` values, pairs (i, i + rot/2) or (2i, 2i + 1).
"""
import math

import torch

own = False

EPS = 1e-6
BASE = 10000.0


# ------------------------------------------------------------------- cases --

def _norm_rope(op, name=None, **kw):
    c = {"op": op, "dtype": "bf16", "B": 1, "H": 8, "Hk": 8, "L": 1, "d": 64, "rot": 64,
         "interleaved": False, "gamma": "shared", "packed": False, "pos0": 0}
    c.update(kw)
    return c if name is None else dict(c, name=name)


def _append(name=None, **kw):
    c = {"op": "append", "dtype": "bf16", "B": 1, "Hk": 8, "T": 1, "d": 64, "rot": 64,
         "interleaved": False, "gamma": "none", "page": 64, "have": 0, "ragged": False,
         "packed": False, "pos0": 0}
    c.update(kw)
    return c if name is None else dict(c, name=name)


def _attend(name=None, **kw):
    c = {"op": "attend", "dtype": "bf16", "B": 1, "H": 8, "Hk": 8, "T": 1, "d": 64, "r": 64,
         "page": 64, "prefix": 0, "own_max": 64, "causal": False}
    c.update(kw)
    return c if name is None else dict(c, name=name)


def listed():
    return [
        # one new token of 64 sequences: a decode step's queries and keys (latency)
        _norm_rope("norm_rope", "norm-rope decode B64 d64", B=64, pos0=4096),
        # a training or prefill pass over the large-head shape (bandwidth)
        _norm_rope("norm_rope", "norm-rope B4 L8192 d256", B=4, L=8192, d=256, rot=256),
        # its gradient at the causal block's shape, queries and keys in a packed projection
        _norm_rope("norm_rope_grad", "norm-rope grad B2 L2048 d64", B=2, L=2048, packed=True),
        # gradient over a long sequence: grouped keys, partial interleaved rotation, a
        # weight for every head
        _norm_rope("norm_rope_grad", "norm-rope grad L16384 d128", H=16, Hk=4, L=16384, d=128,
                   rot=64, interleaved=True, gamma="per_head"),
        # one new token of 64 sequences into the cache (latency)
        _append("append decode B64 d64", B=64, have=1024, pos0=4096),
        # a batch of prompts of different lengths, keys normed on the way (bandwidth)
        _append("append prefill B4 T8192 d256", B=4, T=8192, d=256, rot=256, gamma="shared",
                ragged=True),
        # fp32, odd sizes: small pages that end inside a prompt, partial rotation
        _append("append fp32 T777 d40", dtype="f32", B=3, Hk=3, T=777, d=40, rot=20, page=24,
                have=100, ragged=True, packed=True),
        # a few sequences over a short system prompt (latency)
        _attend("attend B4 prefix512 d64", B=4, prefix=512, page=16),
        # the streaming-decode batch over a 4096-token prefix
        _attend("attend B64 prefix4096 d64", B=64, prefix=4096, own_max=1024),
        # large heads, a longer prefix and longer sequences
        _attend("attend B32 prefix8192 d256", B=32, d=256, r=256, prefix=8192, own_max=2048),
        # grouped heads, four drafted tokens for each sequence over a long shared document
        _attend("attend B64 T4 prefix32768 d128", B=64, H=32, T=4, d=128, r=128, page=128,
                prefix=32768, own_max=512, causal=True),
        # fp32, odd sizes: low-rank geometry, small pages, lengths that end inside them
        _attend("attend fp32 prefix1000 d40", dtype="f32", B=3, H=6, Hk=2, T=3, d=40, r=24,
                page=24, prefix=1000, own_max=777, causal=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_grad", "append", "attend", "attend"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    d = rng.choice([32, 40, 64, 64, 80, 96, 128, 128, 256])
    Hk = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 1, 2, 4])
    B = _log(rng, 1, 64)
    if op == "attend":
        own_max = _log(rng, 1, 4096)
        prefix = rng.choice([0, _log(rng, 16, 32768)])
        T = rng.choice([1, 1, 2, 3, 4, 8])
        # no more work than the largest listed case
        while B * group * Hk * T * (prefix + own_max) * d > 64 * 32 * 4 * 32768 * 128 // 4:
            B, own_max = max(1, B // 2), max(1, own_max // 2)
        return _attend(dtype=dtype, B=B, H=Hk * group, Hk=Hk, T=T, d=d,
                       r=rng.choice([d, max(4, d // 2), 24]), page=rng.choice([16, 32, 64, 128, 24]),
                       prefix=prefix, own_max=own_max, causal=rng.random() < 0.5)
    rot = rng.choice([d, d, d // 2])
    inter, packed, pos0 = rng.random() < 0.4, rng.random() < 0.5, _log(rng, 1, 200000)
    tokens = _log(rng, 1, 65536)
    if op == "append":
        T = max(1, tokens // B)
        while B * T * Hk * d > 4 * 8192 * 8 * 256:
            T //= 2
        return _append(dtype=dtype, B=B, Hk=Hk, T=T, d=d, rot=rot, interleaved=inter,
                       gamma=rng.choice(["none", "shared", "per_head"]),
                       page=rng.choice([16, 32, 64, 128, 24]), have=_log(rng, 1, 2048),
                       ragged=rng.random() < 0.5, packed=packed, pos0=pos0)
    L = max(1, tokens // B)
    while B * L * Hk * (group + 1) * d > 4 * 8192 * 16 * 256:
        L //= 2
    return _norm_rope(op, dtype=dtype, B=B, H=Hk * group, Hk=Hk, L=L, d=d, rot=rot,
                      interleaved=inter, packed=packed, pos0=pos0,
                      gamma=rng.choice(["shared", "shared", "per_head"]))


def _own_lengths(case):
    """Tokens of every sequence after the prefix: from a few to own_max, evenly spread."""
    B, most, least = case["B"], case["own_max"], case["T"] if case["causal"] else 1
    most = max(most, least)
    if B == 1:
        return [most]
    return [least + (most - least) * i // (B - 1) for i in range(B)]


def _new_lengths(case):
    """New tokens of every sequence in an append: all T, or from about T/2 to T."""
    B, T = case["B"], case["T"]
    if not case["ragged"]:
        return [T] * B
    return [max(1, T - (T // 2) * i // B) for i in range(B)]


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    d = case["d"]
    if case["op"] in ("norm_rope", "norm_rope_grad"):
        n = case["B"] * case["L"] * (case["H"] + case["Hk"]) * d
        if case["op"] == "norm_rope":
            return {"bytes": 2 * n * e, "flops": 8 * n}
        return {"bytes": 3 * n * e, "flops": 16 * n}
    if case["op"] == "append":
        n = sum(_new_lengths(case)) * case["Hk"] * d
        return {"bytes": 4 * n * e, "flops": 8 * n}
    own_sum = sum(_own_lengths(case))
    rows = case["H"] * case["T"]
    keys = case["prefix"] + own_sum
    io = 2 * case["B"] * rows * d
    return {"bytes": (2 * keys * case["Hk"] * d + io) * e,
            "flops": 4 * rows * d * (case["B"] * case["prefix"] + own_sum)
            + 4 * case["B"] * rows * case["r"] * d}


# ------------------------------------------------------------------ inputs --

def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _normal(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _heads(g, B, L, counts, d, dtype, packed):
    """One tensor [B][H][L][d] for each head count: views of one packed projection output
    [B][L][sum of counts][d], or dense tensors of their own."""
    if not packed:
        return [_normal(g, B, h, L, d, dtype=dtype) for h in counts]
    x = _normal(g, B, L, sum(counts), d, dtype=dtype).permute(0, 2, 1, 3)
    return list(torch.split(x, counts, dim=1))


def _weight(g, case, heads):
    if case["gamma"] == "none":
        return None
    return 1.0 + 0.2 * _normal(g, heads if case["gamma"] == "per_head" else 1, case["d"])


def _tables(g, B, per_row, shared, spare):
    """Page tables over a cache in random page order: [B][per_row] and [shared]."""
    n = B * per_row + shared + spare
    order = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
    return n, order[:B * per_row].reshape(B, per_row).contiguous(), \
        order[B * per_row:B * per_row + shared].contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, d, B = _dtype(case), case["d"], case["B"]
    s = {"case": case}
    if case["op"] in ("norm_rope", "norm_rope_grad"):
        H, Hk, L = case["H"], case["Hk"], case["L"]
        # a fused projection also holds the values, which this operator leaves alone
        s["q"], s["k"] = _heads(g, B, L, [H, Hk, Hk] if case["packed"] else [H, Hk], d, dt,
                                case["packed"])[:2]
        s["gq"], s["gk"] = _weight(g, case, H), _weight(g, case, Hk)
        # positions of a batch whose sequences have come differently far
        start = torch.randint(0, 1000, (B, 1), generator=g, device="cuda")
        s["pos"] = (case["pos0"] + start + torch.arange(L, device="cuda")).to(torch.int32)
        if case["op"] == "norm_rope":
            s["qo"] = torch.empty(B, H, L, d, dtype=dt, device="cuda")
            s["ko"] = torch.empty(B, Hk, L, d, dtype=dt, device="cuda")
        else:
            s["dqo"], s["dko"] = _heads(g, B, L, [H, Hk], d, dt, False)
            s["dq"], s["dk"] = _heads(g, B, L, [H, Hk, Hk] if case["packed"] else [H, Hk], d, dt,
                                      case["packed"])[:2]
            s["dgq"], s["dgk"] = torch.empty_like(s["gq"]), torch.empty_like(s["gk"])
    elif case["op"] == "append":
        Hk, T, page, have = case["Hk"], case["T"], case["page"], case["have"]
        s["k"], s["v"] = _heads(g, B, T, [Hk, Hk], d, dt, case["packed"])
        s["gk"] = _weight(g, case, Hk)
        lens = torch.randint(0, have + 1, (B,), generator=g, device="cuda")
        s["lens"] = lens.to(torch.int32)
        s["new"] = torch.tensor(_new_lengths(case), dtype=torch.int32, device="cuda") \
            if case["ragged"] else None
        pages, s["table"], _ = _tables(g, B, -(-(have + T) // page), 0, 3)
        s["kp"] = _normal(g, pages, Hk, page, d, dtype=dt)
        s["vp"] = _normal(g, pages, Hk, page, d, dtype=dt)
    else:
        H, Hk, T, page, r = case["H"], case["Hk"], case["T"], case["page"], case["r"]
        s["q"] = _normal(g, B, H, T, d, dtype=dt)
        lens = torch.tensor(_own_lengths(case), dtype=torch.int32, device="cuda")
        s["lens"] = lens[torch.randperm(B, generator=g, device="cuda")].contiguous()
        shared = -(-case["prefix"] // page)
        pages, s["table"], s["shared"] = _tables(g, B, -(-max(_own_lengths(case)) // page),
                                                 shared, 3)
        s["kp"] = _normal(g, pages, Hk, page, d, dtype=dt)
        s["vp"] = _normal(g, pages, Hk, page, d, dtype=dt)
        # the learned geometry: near the identity at full rank, Gaussian at low rank
        s["geom"] = torch.eye(d, device="cuda") + 0.05 * _normal(g, H, d, d) if r == d \
            else _normal(g, H, r, d) / math.sqrt(r)
        s["out"] = torch.empty_like(s["q"])
    if own:
        _handles(s)
    return s


def _handles(s):
    """What a program of the library keeps: the rotation, the cache and projection handles
    and the workspaces."""
    from random_feature_linear_b200 import dark as D
    case = s["case"]
    dtype = D.DARK_BF16 if case["dtype"] == "bf16" else D.DARK_F32
    if case["op"] != "attend":
        s["rope"] = D.dark_rope_init(case["rot"], BASE, 1.0, case["interleaved"])
    if case["op"] == "norm_rope_grad":
        s["ws"] = D.alloc_qk_norm_rope_bwd_workspace(case["B"], case["H"], case["Hk"], case["L"],
                                                     case["d"], "cuda")
    if case["op"] in ("append", "attend"):
        s["cache"] = D.kv_cache(s["kp"], s["vp"])
    if case["op"] == "attend":
        # the exact mode does not use the random features: one feature is enough
        omega = torch.zeros(1, 1, case["r"], device="cuda")
        s["proj"], s["wbuf"] = D.dark_make_projection(omega, s["geom"], case["H"], dtype)
        s["ws"] = D.alloc_cache_attention_workspace(
            s["proj"], s["cache"], case["B"], case["H"], case["T"], case["prefix"],
            s["table"].shape[1], "cuda")


# -------------------------------------------------------------- plain forms --

def _angles(case, pos):
    """cos and sin of every pair, [..., rot/2] for positions [...]: products in fp64."""
    i = torch.arange(case["rot"] // 2, dtype=torch.float64, device="cuda")
    t = pos.double()[..., None] * BASE ** (-2.0 * i / case["rot"])
    return t.cos().float(), t.sin().float()


def _turn(case, x, cos, sin):
    """Rotates the first `rot` values of x by the angles (cos, sin)."""
    rot = case["rot"]
    if case["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)
    return torch.cat((y, x[..., rot:]), dim=-1)


def _rstd(x):
    return torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS)


def _normed(x, gamma):
    """x [B][H][L][d] in fp32, normed with gamma [1 or H][d]; untouched without gamma."""
    return x if gamma is None else x * _rstd(x) * gamma[:, None, :]


def _plain_norm_rope(s):
    case = s["case"]
    cos, sin = _angles(case, s["pos"])
    outs = []
    for x, gamma, o in ((s["q"], s["gq"], s["qo"]), (s["k"], s["gk"], s["ko"])):
        o.copy_(_turn(case, _normed(x.float(), gamma), cos[:, None], sin[:, None]))
        outs.append(o)
    return outs


def _plain_norm_rope_grad(s):
    case = s["case"]
    cos, sin = _angles(case, s["pos"])
    outs = []
    for x, gamma, dy, dx, dgamma in ((s["q"], s["gq"], s["dqo"], s["dq"], s["dgq"]),
                                     (s["k"], s["gk"], s["dko"], s["dk"], s["dgk"])):
        x = x.float()
        # the rotation's transpose turns by the opposite angle
        u = _turn(case, dy.float(), cos[:, None], -sin[:, None])
        rstd = _rstd(x)
        n = x * rstd
        w = u * gamma[:, None, :]
        dx.copy_(rstd * (w - n * (w * n).mean(dim=-1, keepdim=True)))
        # long sums over tokens (and, for a shared weight, heads) in fp64
        dg = (u * n).sum(dim=2, dtype=torch.float64).sum(dim=0)
        dgamma.copy_(dg if gamma.shape[0] > 1 else dg.sum(dim=0, keepdim=True))
        outs += [dx, dgamma]
    return outs


def _plain_append(s):
    case = s["case"]
    T, page = case["T"], case["page"]
    t = torch.arange(T, device="cuda")
    at = s["lens"].long()[:, None] + t                      # [B][T]: place in the sequence
    cos, sin = _angles(case, case["pos0"] + at)
    k = _turn(case, _normed(s["k"].float(), s["gk"]), cos[:, None], sin[:, None])
    keep = torch.ones_like(at, dtype=torch.bool) if s["new"] is None else t < s["new"][:, None]
    pages = torch.gather(s["table"].long(), 1, torch.where(keep, at // page, 0))
    pages, rows = pages[keep], (at % page)[keep]
    s["kp"][pages, :, rows] = k.transpose(1, 2)[keep].to(s["kp"].dtype)
    s["vp"][pages, :, rows] = s["v"].transpose(1, 2)[keep]
    return [s["kp"], s["vp"]]


def _plain_attend(s):
    case = s["case"]
    B, H, Hk, T, d, P = (case[n] for n in ("B", "H", "Hk", "T", "d", "prefix"))
    G = H // Hk
    geom = s["geom"]
    # q^T Sigma k / sqrt(d) = (M^T M q / sqrt(d)) . k
    y = torch.matmul(torch.matmul(s["q"].float(), geom.transpose(1, 2)), geom) / math.sqrt(d)
    y = y.reshape(B, Hk, G * T, d)

    def own_rows(pool):                                     # [B][Hk][S][d]
        x = pool[s["table"].long()].float()
        return x.permute(0, 2, 1, 3, 4).flatten(2, 3)

    def shared_rows(pool):                                  # [Hk][P][d]
        x = pool[s["shared"].long()].float()
        return x.permute(1, 0, 2, 3).flatten(1, 2)[:, :P]

    k, v = own_rows(s["kp"]), own_rows(s["vp"])
    S = k.shape[2]
    scores = torch.matmul(y, k.transpose(2, 3)).reshape(B, Hk, G, T, S)
    j = torch.arange(S, device="cuda")
    last = s["lens"].long()[:, None].expand(B, T)           # keys that each query sees
    if case["causal"]:
        last = last - T + 1 + torch.arange(T, device="cuda")
    scores = scores.masked_fill(j >= last[:, None, None, :, None], -math.inf)
    scores = scores.reshape(B, Hk, G * T, S)
    if P:
        ks, vs = shared_rows(s["kp"]), shared_rows(s["vp"])
        rows = y.transpose(0, 1).reshape(Hk, B * G * T, d)
        pre = torch.matmul(rows, ks.transpose(1, 2)).reshape(Hk, B, G * T, P).transpose(0, 1)
        scores = torch.cat((pre, scores), dim=-1)
    top = scores.amax(dim=-1, keepdim=True)
    p = torch.exp(scores - top)
    den = p.sum(dim=-1, keepdim=True)
    num = torch.matmul(p[..., P:], v)
    if P:
        pre = p[..., :P].transpose(0, 1).reshape(Hk, B * G * T, P)
        num = num + torch.matmul(pre, vs).reshape(Hk, B, G * T, d).transpose(0, 1)
    s["out"].copy_((num / den).reshape(B, H, T, d))
    return s["out"]


# ---------------------------------------------------------------------- run --

def _own_run(s):
    from random_feature_linear_b200 import dark as D
    case = s["case"]
    if case["op"] == "norm_rope":
        D.dark_qk_norm_rope_fwd(s["q"], s["k"], s["qo"], s["ko"], gamma_q=s["gq"],
                                gamma_k=s["gk"], eps=EPS, rope=s["rope"], positions=s["pos"])
        return [s["qo"], s["ko"]]
    if case["op"] == "norm_rope_grad":
        D.dark_qk_norm_rope_bwd(s["q"], s["k"], s["dqo"], s["dko"], s["dq"], s["dk"],
                                gamma_q=s["gq"], gamma_k=s["gk"], dgamma_q=s["dgq"],
                                dgamma_k=s["dgk"], eps=EPS, rope=s["rope"],
                                positions=s["pos"], ws=s["ws"])
        return [s["dq"], s["dgq"], s["dk"], s["dgk"]]
    if case["op"] == "append":
        D.dark_kv_append(s["cache"], s["k"], s["v"], s["table"], s["lens"], new_lens=s["new"],
                         gamma_k=s["gk"], eps=EPS, rope=s["rope"], pos0=case["pos0"])
        return [s["kp"], s["vp"]]
    D.dark_cache_attention_fwd(s["proj"], s["cache"], s["q"], s["out"], s["table"], s["lens"],
                               prefix_pages=s["shared"] if case["prefix"] else None,
                               prefix_len=case["prefix"],
                               flags=D.DARK_CAUSAL if case["causal"] else 0, ws=s["ws"])
    return s["out"]


def run(state):
    if own:
        return _own_run(state)
    return {"norm_rope": _plain_norm_rope, "norm_rope_grad": _plain_norm_rope_grad,
            "append": _plain_append, "attend": _plain_attend}[state["case"]["op"]](state)


# -------------------------------------------------------------------- exact --

def _exact_matrix(case, pos):
    """Rotation of the first rot values as complex factors [..., rot/2] in fp64."""
    i = torch.arange(0, case["rot"], 2, dtype=torch.float64, device="cuda")
    return torch.polar(torch.ones((), dtype=torch.float64, device="cuda").expand(*pos.shape, i.numel()),
                       pos.double().unsqueeze(-1) * torch.exp(-math.log(BASE) * i / case["rot"]))


def _exact_pairs(case, x):
    """The first rot values of x as complex pairs."""
    half = case["rot"] // 2
    z = x[..., :case["rot"]]
    if case["interleaved"]:
        return torch.view_as_complex(z.reshape(*z.shape[:-1], half, 2).contiguous())
    return torch.complex(z[..., :half].contiguous(), z[..., half:].contiguous())


def _exact_flat(case, z, rest):
    """The inverse of _exact_pairs, with the unrotated values behind."""
    y = torch.view_as_real(z)
    y = y.flatten(-2) if case["interleaved"] else y.transpose(-1, -2).flatten(-2)
    return torch.cat((y, rest), dim=-1)


def _exact_forward(case, x, gamma, factors):
    x = x.double()
    if gamma is not None:
        x = gamma.double().unsqueeze(1) * x / (x.pow(2).sum(-1, keepdim=True) / case["d"] + EPS).sqrt()
    return _exact_flat(case, _exact_pairs(case, x) * factors, x[..., case["rot"]:])


def _exact_backward(case, x, gamma, dy, factors):
    x, dy, gamma = x.double(), dy.double(), gamma.double()
    u = _exact_flat(case, _exact_pairs(case, dy) * factors.conj(), dy[..., case["rot"]:])
    # y = gamma x / s, s = sqrt(x.x / d + eps): dx = gamma u / s - x (gamma u . x) / (d s^3)
    s = (x.pow(2).sum(-1, keepdim=True) / case["d"] + EPS).sqrt()
    w = u * gamma.unsqueeze(1)
    dx = w / s - x * (w * x).sum(-1, keepdim=True) / (case["d"] * s ** 3)
    dg = torch.einsum("bhld,bhld->hd", u, x / s)
    return dx, dg if gamma.shape[0] > 1 else dg.sum(0, keepdim=True)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm_rope", "norm_rope_grad"):
        outs = []
        f = _exact_matrix(case, s["pos"]).unsqueeze(1)
        for n in ("q", "k"):
            if case["op"] == "norm_rope":
                outs.append(_exact_forward(case, s[n], s["g" + n], f))
            else:
                outs += list(_exact_backward(case, s[n], s["g" + n], s["d" + n + "o"], f))
        return outs
    if case["op"] == "append":
        kp, vp = s["kp"].double(), s["vp"].double()
        lens, new, page = s["lens"].tolist(), _new_lengths(case), case["page"]
        for b, (have, count) in enumerate(zip(lens, new)):
            at = torch.arange(have, have + count, device="cuda")
            f = _exact_matrix(case, at + case["pos0"])
            k = _exact_forward(case, s["k"][b, :, :count], s["gk"], f)
            for first in range(have // page, (have + count - 1) // page + 1):
                lo, hi = max(have, first * page), min(have + count, (first + 1) * page)
                p = int(s["table"][b, first])
                kp[p, :, lo - first * page:hi - first * page] = k[:, lo - have:hi - have]
                vp[p, :, lo - first * page:hi - first * page] = \
                    s["v"][b, :, lo - have:hi - have].double()
        return [kp, vp]
    B, H, Hk, T, P, d, page = (case[n] for n in ("B", "H", "Hk", "T", "prefix", "d", "page"))
    out = torch.zeros(B, H, T, d, dtype=torch.float64, device="cuda")
    lens = s["lens"].tolist()
    shared = s["shared"].long()
    geom = s["geom"].double() / d ** 0.25

    def rows(pool, h, pages, count):
        return pool[pages, h].reshape(-1, d)[:count].double()

    for h in range(Hk):
        pk, pv = rows(s["kp"], h, shared, P), rows(s["vp"], h, shared, P)
        heads = slice(h * (H // Hk), (h + 1) * (H // Hk))
        # u = M q~ and w = M k~, scores u . w (the geometry differs from head to head)
        for b in range(B):
            own_pages = s["table"][b, :-(-lens[b] // page)].long()
            k = torch.cat((pk, rows(s["kp"], h, own_pages, lens[b])))
            v = torch.cat((pv, rows(s["vp"], h, own_pages, lens[b])))
            m = geom[heads]
            u = torch.einsum("grd,gtd->gtr", m, s["q"][b, heads].double())
            score = torch.einsum("gtr,grd->gtd", u, m) @ k.T
            if case["causal"]:
                key = torch.arange(len(k), device="cuda")
                last = P + lens[b] - T + torch.arange(T, device="cuda")
                score = score.where(key <= last[:, None], -math.inf)
            out[b, heads] = torch.softmax(score, dim=-1) @ v
    return out
