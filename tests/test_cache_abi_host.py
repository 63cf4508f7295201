"""Host-side refusals of the head-norm, cache-append and cache-attention calls: everything
here is refused before anything is enqueued, so no GPU is needed."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def D():
    from random_feature_linear_b200 import build
    build.build()
    from random_feature_linear_b200 import dark
    return dark


S3 = ctypes.c_int64 * 3
P = 0x10000000                      # 256-byte aligned addresses that nothing reads
Q, K, QO, KO, G, WS = (P + i * 0x1000000 for i in range(6))


def test_rope_init(D):
    r = D.dark_rope_init(8, 100.0, 2.0, True)
    assert (r.dims, r.interleaved) == (8, 1)
    for i in range(4):
        turns = 2.0 * 100.0 ** (-2.0 * i / 8) / (2 * 3.141592653589793) % 1.0
        assert abs(r.turns[i] / 2.0 ** 64 - turns) < 1e-15
    assert D.dark_rope_init(0).dims == 0
    # a negative scale turns the other way: the turns are a complement
    f, b = D.dark_rope_init(4, 50.0, 1.0), D.dark_rope_init(4, 50.0, -1.0)
    assert abs((f.turns[1] + b.turns[1]) - 2 ** 64) <= 2
    for bad in [(7,), (-2,), (258,), (8, 0.0), (8, -1.0), (8, float("inf")),
                (8, 10.0, float("nan"))]:
        with pytest.raises(D.DarkError) as ei:
            D.dark_rope_init(*bad)
        assert ei.value.status == D.DARK_ERR_INVALID_ARG
    assert D._lib.dark_rope_init(None, 8, 10.0, 1.0, 0) == D.DARK_ERR_INVALID_ARG


def _fwd(D, **kw):
    a = dict(q=Q, qs=None, k=K, ks=None, qo=QO, qos=None, ko=KO, kos=None, gq=G, hgq=1, gk=G,
             hgk=1, eps=1e-6, rope=D.dark_rope_init(64), pos=None, pos0=0, B=2, H=4, Hk=2, L=8,
             d=64, dt=D.DARK_BF16, st=None, stream=None)
    a.update(kw)
    return D._lib.dark_qk_norm_rope_fwd(*a.values())


def _bwd(D, **kw):
    n = D.dark_qk_norm_rope_bwd_workspace_bytes(2, 4, 2, 8, 64)
    a = dict(q=Q, qs=None, k=K, ks=None, gqo=P + 0x8000000, gqs=None, gko=P + 0x9000000, gks=None,
             dq=QO, dqs=None, dk=KO, dks=None, gq=G, hgq=1, gk=G, hgk=1, dgq=P + 0xa000000,
             dgk=P + 0xb000000, eps=1e-6, rope=D.dark_rope_init(64), pos=None, pos0=0, B=2, H=4,
             Hk=2, L=8, d=64, dt=D.DARK_BF16, ws=WS, n=n, st=None, stream=None)
    a.update(kw)
    return D._lib.dark_qk_norm_rope_bwd(*a.values())


BAD_ROWS = [dict(q=None), dict(k=None), dict(q=Q + 1), dict(B=0), dict(H=0), dict(Hk=-1),
            dict(L=0), dict(d=0), dict(dt=7), dict(hgq=3), dict(hgk=4), dict(eps=0.0),
            dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(pos=P + 2),
            dict(gq=G + 2), dict(qs=S3(-1, 64, 64))]
FAR_ROWS = [dict(d=260), dict(d=66), dict(B=1 << 16, L=1 << 15), dict(H=65535, hgq=1)]


@pytest.mark.parametrize("kw", BAD_ROWS + [
    dict(qo=None), dict(ko=None), dict(ko=QO), dict(qos=S3(0, 512, 64)), dict(kos=S3(1024, 512, 0)),
    dict(qo=Q, qos=S3(2048, 64, 256))])
def test_norm_rope_refuses(D, kw):
    assert _fwd(D, **kw) == D.DARK_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", FAR_ROWS)
def test_norm_rope_unsupported(D, kw):
    if kw.get("d") == 260:
        kw = dict(kw, rope=None)
    assert _fwd(D, **kw) == D.DARK_ERR_UNSUPPORTED
    assert _bwd(D, **kw) == D.DARK_ERR_UNSUPPORTED


def test_norm_rope_refuses_a_rotation_wider_than_the_row(D):
    assert _fwd(D, d=32) == D.DARK_ERR_INVALID_ARG
    r = D.dark_rope_init(64)
    r.dims = 300
    assert _fwd(D, rope=r) == D.DARK_ERR_INVALID_ARG
    r.dims = 63
    assert _fwd(D, rope=r) == D.DARK_ERR_INVALID_ARG
    r.dims, r.interleaved = 64, 2
    assert _fwd(D, rope=r) == D.DARK_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", BAD_ROWS + [
    dict(gqo=None), dict(gko=None), dict(dq=None), dict(dk=None), dict(dk=QO), dict(ws=None),
    dict(ws=WS + 16), dict(n=256), dict(dgq=None), dict(dgk=None), dict(gk=None),
    dict(dgk=P + 0xa000000), dict(dqs=S3(0, 512, 64)), dict(dq=P + 0x8000000,
                                                           dqs=S3(2048, 64, 256))])
def test_norm_rope_bwd_refuses(D, kw):
    assert _bwd(D, **kw) == D.DARK_ERR_INVALID_ARG


def test_norm_rope_refuses_results_in_the_other_input(D):
    """The other tensor's heads are still to be read when a warp stores its first results."""
    assert _fwd(D, qo=K) == D.DARK_ERR_INVALID_ARG
    assert _fwd(D, ko=Q) == D.DARK_ERR_INVALID_ARG
    for kw in [dict(dq=K), dict(dq=P + 0x9000000), dict(dk=Q), dict(dk=P + 0x8000000)]:
        assert _bwd(D, **kw) == D.DARK_ERR_INVALID_ARG
    # the forward's own input, with other strides
    assert _bwd(D, dq=Q, dqs=S3(2048, 64, 256)) == D.DARK_ERR_INVALID_ARG
    assert _bwd(D, dk=K, dks=S3(1024, 64, 128)) == D.DARK_ERR_INVALID_ARG


def test_norm_rope_bwd_refuses_a_gradient_without_its_tensor(D):
    kw = dict(k=None, gko=None, dk=None, Hk=0, n=1 << 30)
    assert _bwd(D, **kw) == D.DARK_ERR_INVALID_ARG
    assert _bwd(D, gk=None, **kw) == D.DARK_ERR_INVALID_ARG


def test_norm_rope_bwd_workspace_query(D):
    f = D.dark_qk_norm_rope_bwd_workspace_bytes
    assert f(1, 1, 0, 1, 4) > 0 and f(2, 4, 2, 8, 64) % 256 == 0
    for bad in [(0, 4, 2, 8, 64), (2, 0, 2, 8, 64), (2, 4, -1, 8, 64), (2, 4, 2, 0, 64),
                (2, 4, 2, 8, 66), (2, 4, 2, 8, 512), (1 << 16, 4, 2, 1 << 15, 64)]:
        assert f(*bad) == 0


def _cache(D, **kw):
    a = dict(k=P, v=P + 0x8000000, pages=10, heads=2, page_size=16, d=64, dtype=D.DARK_BF16)
    a.update(kw)
    return D.dark_kv_cache(*a.values())


def _append(D, cache=None, **kw):
    a = dict(k=Q, ks=None, v=K, vs=None, B=2, T=3, table=G, max_pages=4, lens=WS, new=None, gk=None,
             hgk=1, eps=1e-6, rope=None, pos=None, pos0=0, st=None, stream=None)
    a.update(kw)
    return D._lib.dark_kv_append(_cache(D) if cache is None else cache, *a.values())


BAD_CACHES = [dict(k=None), dict(v=None), dict(v=P), dict(k=P + 8), dict(pages=0), dict(heads=0),
              dict(page_size=0), dict(d=0), dict(dtype=5)]


@pytest.mark.parametrize("kw", BAD_CACHES)
def test_cache_handles_are_checked(D, kw):
    assert _append(D, _cache(D, **kw)) == D.DARK_ERR_INVALID_ARG
    assert _attend(D, _cache(D, **kw)) == D.DARK_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(k=None), dict(v=None), dict(B=0), dict(T=0), dict(table=None),
                                dict(table=G + 2), dict(max_pages=0), dict(lens=None),
                                dict(lens=WS + 1), dict(new=WS + 2), dict(pos=P + 1),
                                dict(ks=S3(-8, 64, 64)), dict(gk=G, hgk=3), dict(gk=G, eps=0.0),
                                dict(k=Q + 1)])
def test_append_refuses(D, kw):
    assert _append(D, **kw) == D.DARK_ERR_INVALID_ARG


def test_append_unsupported(D):
    assert _append(D, _cache(D, d=66)) == D.DARK_ERR_UNSUPPORTED
    assert _append(D, _cache(D, d=260)) == D.DARK_ERR_UNSUPPORTED
    assert _append(D, max_pages=(1 << 26) + 1) == D.DARK_ERR_UNSUPPORTED
    assert _append(D, B=1 << 16, T=1 << 15) == D.DARK_ERR_UNSUPPORTED
    assert _append(D, rope=D.dark_rope_init(128)) == D.DARK_ERR_INVALID_ARG
    assert D._lib.dark_kv_append(None, *([None] * 4), 1, 1, None, 1, None, None, None, 1, 1.0,
                                 None, None, 0, None, None) == D.DARK_ERR_INVALID_ARG


def _proj(D, **kw):
    a = dict(heads=4, m=1, r=64, d=64, dtype=D.DARK_BF16, generation=1, w=P + 0xc000000)
    a.update(kw)
    return D.dark_projection(*a.values())


def _attend(D, cache=None, proj=None, **kw):
    cache, proj = cache or _cache(D), proj or _proj(D)
    a = dict(q=Q, qs=None, out=QO, os=None, B=2, H=4, T=3, pre=K, plen=20, table=G, max_pages=4,
             lens=WS, flags=0, ws=P + 0xd000000, n=1 << 40, st=None, stream=None)
    a.update(kw)
    return D._lib.dark_cache_attention_fwd(proj, cache, *a.values())


@pytest.mark.parametrize("kw", [dict(q=None), dict(out=None), dict(B=0), dict(H=0), dict(T=0),
                                dict(H=3), dict(pre=None), dict(plen=-1), dict(table=None),
                                dict(max_pages=0), dict(lens=None), dict(flags=2), dict(flags=8),
                                dict(ws=None), dict(ws=P + 0xd000010), dict(n=1024), dict(q=Q + 1),
                                dict(out=QO + 1), dict(table=G + 1), dict(lens=WS + 2),
                                dict(pre=K + 1), dict(os=S3(768, 0, 64)), dict(qs=S3(-1, 0, 64)),
                                dict(H=8)])
def test_attention_refuses(D, kw):
    assert _attend(D, **kw) == D.DARK_ERR_INVALID_ARG


def test_attention_refuses_other_projections(D):
    for kw in [dict(heads=2), dict(d=32), dict(dtype=D.DARK_F32), dict(w=None), dict(w=P + 8),
               dict(m=0), dict(r=0)]:
        assert _attend(D, proj=_proj(D, **kw)) == D.DARK_ERR_INVALID_ARG
    assert D._lib.dark_cache_attention_fwd(None, _cache(D), *([None] * 4), 1, 4, 1, None, 0, None,
                                           1, None, 0, None, 0, None, None) == D.DARK_ERR_INVALID_ARG


def test_attention_unsupported(D):
    assert _attend(D, proj=_proj(D, r=300)) == D.DARK_ERR_UNSUPPORTED
    assert _attend(D, proj=_proj(D, m=2000)) == D.DARK_ERR_UNSUPPORTED
    assert _attend(D, plen=(1 << 30) + 1) == D.DARK_ERR_UNSUPPORTED
    assert _attend(D, max_pages=(1 << 26) + 1) == D.DARK_ERR_UNSUPPORTED
    assert _attend(D, B=1 << 18, T=8) == D.DARK_ERR_UNSUPPORTED
    assert _attend(D, _cache(D, heads=4096), proj=_proj(D, heads=1), B=1 << 13, H=4096, T=1) \
        == D.DARK_ERR_UNSUPPORTED


def test_attention_workspace_query(D):
    f = D.dark_cache_attention_workspace_bytes
    n = f(_proj(D), _cache(D), 2, 4, 3, 20, 4)
    assert n > 0 and n % 256 == 0
    assert f(_proj(D), _cache(D), 2, 3, 3, 20, 4) == 0
    assert f(_proj(D, d=32), _cache(D), 2, 4, 3, 20, 4) == 0
    # the workspace follows the queries and the GPU, not the cache
    assert f(_proj(D), _cache(D), 2, 4, 3, 1 << 20, 4096) < (1 << 26)


@pytest.mark.parametrize("d,heads,H,dtype", [(64, 8, 8, "BF16"), (128, 8, 32, "BF16"),
                                             (256, 2, 8, "BF16"), (40, 2, 6, "F32"),
                                             (36, 1, 8, "BF16")])
def test_attention_workspace_of_the_largest_call_is_enough(D, d, heads, H, dtype):
    """The query never falls as sequences, queries a sequence or prefix tokens are added."""
    dt = getattr(D, "DARK_" + dtype)
    proj, cache = _proj(D, heads=1, d=d, dtype=dt), _cache(D, heads=heads, d=d, dtype=dt)
    f = lambda B, T, prefix: D.dark_cache_attention_workspace_bytes(proj, cache, B, H, T, prefix, 64)
    Bs, Ts, prefixes = list(range(1, 66)) + [127, 128, 129, 500], [1, 2, 3, 8, 9, 70], \
        [0, 1, 63, 64, 65, 255, 256, 257, 4096, 4097, 32768]
    for T in Ts:
        for prefix in prefixes:
            sizes = [f(B, T, prefix) for B in Bs]
            assert sizes == sorted(sizes), (T, prefix)
    for B in Bs:
        for sizes in [[f(B, T, 4096) for T in Ts], [f(B, 1, prefix) for prefix in prefixes]]:
            assert sizes == sorted(sizes), B


def test_binding_checks_tensors(D):
    q, k = torch.zeros(2, 4, 8, 64), torch.zeros(2, 2, 8, 64)
    ok = dict(gamma_q=torch.ones(64), eps=1e-6)
    bad = [
        lambda: D.dark_qk_norm_rope_fwd(q, k, q, k[..., :32]),
        lambda: D.dark_qk_norm_rope_fwd(q, None, q, k),
        lambda: D.dark_qk_norm_rope_fwd(q, k, k, k),
        lambda: D.dark_qk_norm_rope_fwd(q.half(), None, q.half(), None),
        lambda: D.dark_qk_norm_rope_fwd(q, k.bfloat16(), q, k),
        lambda: D.dark_qk_norm_rope_fwd(q.transpose(2, 3), None, q.transpose(2, 3), None),
        lambda: D.dark_qk_norm_rope_fwd(q, k, q, k, gamma_q=torch.ones(3, 64)),
        lambda: D.dark_qk_norm_rope_fwd(q, k, q, k, gamma_q=torch.ones(64).double()),
        lambda: D.dark_qk_norm_rope_fwd(q, k, q, k, positions=torch.zeros(2, 8), **ok),
        lambda: D.dark_qk_norm_rope_fwd(q, k, q, k, positions=torch.zeros(8, dtype=torch.int32)),
        lambda: D.dark_qk_norm_rope_bwd(q, k, q, k, q, None),
        lambda: D.dark_qk_norm_rope_bwd(q, k, q, k, q, q),
        lambda: D.dark_qk_norm_rope_bwd(q, k, q, k, q, k, gamma_q=torch.ones(1, 64),
                                        dgamma_q=torch.ones(4, 64)),
        lambda: D.kv_cache(k, k[:1]),
        lambda: D.kv_cache(k.transpose(1, 2), k.transpose(1, 2)),
        lambda: D.kv_cache(k.half(), k.half()),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            raise AssertionError(i)
    c = D.kv_cache(torch.zeros(9, 2, 16, 64), torch.zeros(9, 2, 16, 64))
    assert (c.pages, c.heads, c.page_size, c.d, c.dtype) == (9, 2, 16, 64, D.DARK_F32)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    bad = [
        lambda: D.dark_kv_append(c, q, q, i32(2, 3), i32(2)),                # heads
        lambda: D.dark_kv_append(c, k.bfloat16(), k.bfloat16(), i32(2, 3), i32(2)),
        lambda: D.dark_kv_append(c, k, k, i32(3, 3), i32(2)),
        lambda: D.dark_kv_append(c, k, k, i32(2, 3).long(), i32(2)),
        lambda: D.dark_kv_append(c, k, k, i32(2, 3), i32(2), new_lens=i32(3)),
        lambda: D.dark_kv_append(c, k, k, i32(2, 3), i32(2), positions=i32(2, 3)),
        lambda: D.dark_cache_attention_fwd(_proj(D), c, q, q[:, :2], i32(2, 3), i32(2)),
        lambda: D.dark_cache_attention_fwd(_proj(D), c, q, q, i32(2, 3), i32(3)),
        lambda: D.dark_cache_attention_fwd(_proj(D), c, q, q, i32(2, 3), i32(2),
                                           prefix_pages=i32(1), prefix_len=17),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            raise AssertionError(i)
