"""Exact-mode attention over the paged cache against the fp64 oracle (GPU, through the C ABI).

Tolerances. The oracle gets the geometry as the projection buffer stores it (fp32, or fp16
for bf16 calls), so what is left are the kernel's own roundings. u = 2^-24, z the scores in
nats, p the softmax weights, y = M^T M q / sqrt(d) the query after the geometry.
 * fp32: a score is a chain of at most r + 2 d + 16 roundings of magnitudes A_j = |M|^T |M| |q|
   |k_j| / sqrt(d), so |dz| <= delta = (r + 2 d + 16) u max_j A_j; exponentials and their sums
   (chains of at most 4096 terms) add (4096 + 64) u. out moves by at most
   (2 delta + 2 delta^2 + 4160 u) sum_j p_j |v_j|.
 * bf16: the same, plus queries and weights that may be rounded to bf16 (half step
   h = 2^-8, of independent values). Weights: a sum of independent errors of at most
   h p_j |v_j| each stays below 6 h sqrt(sum_j (p_j v_j)^2) but for 2e-8 of all values
   (Hoeffding). Queries: out moves by sum_i dy_i Cov_p(k_i, v) to first order,
   below 6 h sqrt(sum_i (y_i Cov_i)^2) alike, and by 2 max_j |dy . k_j|^2 sum p |v| to second,
   with |dy . k_j| <= 6 h sqrt(sum_i (y_i k_ji)^2).
 * half a step of the result's type."""
import numpy as np
import pytest
import torch

from oracle import dark_oracle as O

pytestmark = pytest.mark.gpu
U, H8 = 2.0 ** -24, 2.0 ** -8
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def D(cuda_ok):
    from random_feature_linear_b200 import dark
    return dark


def _np(t):
    return t.double().cpu().numpy()


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Call:
    """One call's tensors: pools in random page order, rows behind every length NaN."""

    def __init__(self, D, dtype=BF, B=2, H=4, Hk=2, T=1, d=64, r=64, page=16, prefix=0,
                 lens=(40, 17), causal=False, shared_geom=False, seed=1, q_scale=1.0, spare_pages=0,
                 packed=False):
        rng = np.random.default_rng(seed)
        tensor = lambda *s: torch.from_numpy(rng.standard_normal(s)).cuda().to(dtype)
        self.D, self.B, self.H, self.T, self.d, self.dtype = D, B, H, T, d, dtype
        self.lens, self.prefix, self.page, self.causal = list(lens), prefix, page, causal
        per = max(1, -(-max(lens) // page)) + spare_pages
        shared = -(-prefix // page)
        n = B * per + shared + 2
        order = rng.permutation(n)
        self.table, self.shared = order[:B * per].reshape(B, per), order[B * per:B * per + shared]
        self.kp, self.vp = tensor(n, Hk, page, d), tensor(n, Hk, page, d)
        live = torch.zeros(n, page, dtype=torch.bool)
        for pages, count in [(self.shared, prefix)] + list(zip(self.table, lens)):
            for j in range(max(0, count)):
                live[pages[j // page], j % page] = True
        dead = ~live.cuda()[:, None, :, None].expand_as(self.kp)
        self.kp[dead], self.vp[dead] = float("nan"), float("inf")
        hg = 1 if shared_geom else H
        geom = np.eye(r, d) + 0.05 * rng.standard_normal((hg, r, d)) if r == d \
            else rng.standard_normal((hg, r, d)) / np.sqrt(r)
        self.geom = torch.from_numpy(geom).float().cuda()
        if packed:                                     # a packed projection, [B][T][H][d] results
            self.q = (q_scale * tensor(B, T, H + 2, d)).permute(0, 2, 1, 3)[:, 1:H + 1]
            self.out = torch.full((B, T, H, d), float("nan"), dtype=dtype,
                                  device="cuda").permute(0, 2, 1, 3)
        else:
            self.q = q_scale * tensor(B, H, T, d)
            self.out = torch.full_like(self.q, float("nan"))
        omega = torch.zeros(1, 1, r, device="cuda")
        self.proj, self.wbuf = D.dark_make_projection(
            omega, self.geom, H, D.DARK_BF16 if dtype == BF else D.DARK_F32)
        self.cache = D.kv_cache(self.kp, self.vp)
        self.ws = D.alloc_cache_attention_workspace(self.proj, self.cache, B, H, T, prefix,
                                                    self.table.shape[1], "cuda")
        self.ws.fill_(0xff)                            # no initial contents are promised
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.d_table, self.d_lens, self.d_shared = _i32(self.table), _i32(lens), _i32(self.shared)

    def run(self, out=None, ws=None, stream=None):
        self.D.dark_cache_attention_fwd(
            self.proj, self.cache, self.q, self.out if out is None else out, self.d_table,
            self.d_lens, prefix_pages=self.d_shared if self.prefix else None,
            prefix_len=self.prefix, flags=self.D.DARK_CAUSAL if self.causal else 0,
            ws=self.ws if ws is None else ws, dev_status=self.status, stream=stream)
        return self.out if out is None else out

    def stored_geom(self):
        """M [heads][r][d] as the projection buffer holds it."""
        p = self.proj
        w = self.wbuf.view(torch.float16 if self.dtype == BF else torch.float32)
        w = _np(w[:p.heads * (p.m + p.r) * p.d]).reshape(p.heads, p.m + p.r, p.d)[:, p.m:]
        return w / (p.d ** -0.25 * np.sqrt(np.log2(np.e) / 2))

    def tolerance(self, ref):
        """The bounds above for every output value."""
        geom, q, kp, vp = self.stored_geom(), _np(self.q), _np(self.kp), _np(self.vp)
        tol = np.zeros(ref.shape)
        G = self.H // kp.shape[1]
        for b in range(self.B):
            n = max(0, min(self.lens[b], self.table.shape[1] * self.page))
            for h in range(self.H):
                k, v = (np.concatenate([O.cache_rows(x, p, c, h // G) for p, c in
                                        ((self.shared, self.prefix), (self.table[b], n)) if c]
                                       or [np.zeros((0, self.d))]) for x in (kp, vp))
                m = O._head(geom, h)
                y = q[b, h] @ m.T @ m / np.sqrt(self.d)
                ya = np.abs(q[b, h]) @ np.abs(m).T @ np.abs(m) / np.sqrt(self.d)
                for t in range(self.T):
                    see = self.prefix + (n - self.T + t + 1 if self.causal else n)
                    if see <= 0 or (self.causal and n - self.T + t < 0):
                        continue
                    kk, vv = k[:see], v[:see]
                    z = kk @ y[t]
                    p = np.exp(z - z.max())
                    p /= p.sum()
                    pv = p @ np.abs(vv)
                    delta = (self.proj.r + 2 * self.d + 16) * U * (np.abs(kk) @ ya[t]).max()
                    e = (2 * delta + 2 * delta ** 2 + 4160 * U) * pv
                    if self.dtype == BF:
                        cov = (kk * p[:, None]).T @ vv - np.outer(p @ kk, p @ vv)
                        e += 6 * H8 * np.sqrt((p ** 2) @ (vv ** 2))
                        e += 6 * H8 * np.sqrt((y[t] ** 2) @ (cov ** 2))
                        dz = 6 * H8 * np.sqrt((kk ** 2) @ (y[t] ** 2)).max()
                        e += 2 * dz ** 2 * pv
                    tol[b, h, t] = e
        half = H8 if self.dtype == BF else U
        return tol + (np.abs(ref) + tol) * half

    def check(self, got=None):
        assert self.status.item() == 0
        n = [max(0, min(x, self.table.shape[1] * self.page)) for x in self.lens]
        ref = O.cache_attention(_np(self.q), _np(self.kp), _np(self.vp), self.stored_geom(),
                                self.table, n, self.shared, self.prefix, self.causal)
        got = _np(self.out if got is None else got)
        assert np.all(np.isfinite(got))
        tol = self.tolerance(ref)
        assert np.all(got[tol == 0] == 0)              # rows that see nothing
        worst = (np.abs(got - ref) / np.maximum(tol, 1e-300)).max()
        assert worst <= 1.0, worst


CASES = {
    "one-key": dict(B=1, H=1, Hk=1, lens=(1,)),
    "one-key-fp32": dict(dtype=F, B=1, H=1, Hk=1, lens=(1,)),
    "no-keys": dict(lens=(0, 0)),
    "some-without-keys": dict(B=4, lens=(0, 3, 0, 70)),
    "prefix-only": dict(lens=(0, 0), prefix=130),
    "prefix": dict(lens=(40, 17), prefix=77),
    "prefix-of-one": dict(lens=(1, 2), prefix=1),
    "decode-batch": dict(B=9, H=8, Hk=8, page=64, prefix=700, lens=tuple(range(1, 1000, 111))),
    "grouped": dict(B=3, H=8, Hk=2, T=4, d=128, r=128, page=32, prefix=333, lens=(300, 4, 77)),
    "grouped-causal": dict(B=3, H=8, Hk=2, T=4, d=128, r=128, page=32, prefix=333,
                           lens=(300, 4, 77), causal=True),
    "causal-padding": dict(B=4, T=5, lens=(0, 2, 5, 90), causal=True),
    "causal-padding-prefix": dict(B=4, T=5, lens=(0, 2, 5, 90), causal=True, prefix=50),
    "causal-prompt": dict(B=2, H=2, Hk=1, T=70, page=24, lens=(70, 201), causal=True, prefix=100),
    "d256": dict(B=2, H=2, Hk=2, d=256, r=256, page=64, prefix=500, lens=(300, 129)),
    "d256-many-rows": dict(B=12, H=4, Hk=2, T=2, d=256, r=64, page=64, prefix=300,
                           lens=tuple(range(5, 125, 10)), causal=True),
    "d96": dict(d=96, r=48, prefix=200, lens=(129, 64)),
    "d80-page24": dict(d=80, r=80, page=24, prefix=200, lens=(129, 64), T=3, causal=True),
    "d40": dict(d=40, r=24, page=24, prefix=100, lens=(129, 64), T=2),
    "d36-simt": dict(d=36, r=36, page=24, prefix=100, lens=(129, 64), T=2),
    "d32": dict(d=32, r=32, H=3, Hk=3, prefix=65, lens=(64, 65)),
    "page-of-one": dict(page=1, prefix=33, lens=(20, 31)),
    "page-7": dict(page=7, prefix=33, lens=(20, 131), T=2, causal=True),
    "shared-geometry": dict(shared_geom=True, prefix=64, lens=(40, 17)),
    "packed": dict(packed=True, T=3, prefix=64, lens=(40, 17), causal=True),
    "many-sequences": dict(B=700, H=1, Hk=1, d=32, r=32, page=16, prefix=20,
                           lens=tuple((7 * i) % 41 for i in range(700))),
    "many-sequences-fp32": dict(dtype=F, B=700, H=1, Hk=1, d=32, r=32, page=16,
                                lens=tuple((7 * i) % 41 for i in range(700))),
    "unequal": dict(B=6, lens=(1, 2500, 3, 64, 128, 7), page=32),
    "spare-pages": dict(spare_pages=5, prefix=30, lens=(40, 17)),
    "large-scores": dict(q_scale=12.0, prefix=200, lens=(100, 37)),
    "small-scores": dict(q_scale=0.0, prefix=200, lens=(100, 37)),
    "many-rows": dict(B=20, H=8, Hk=1, T=2, d=64, page=16, prefix=600,
                      lens=tuple(range(2, 102, 5)), causal=True),
    "many-rows-d128": dict(B=33, H=8, Hk=2, T=1, d=128, r=64, page=64, prefix=1000,
                           lens=tuple(range(0, 99, 3))),
    "many-rows-odd-pages": dict(B=40, H=4, Hk=1, T=3, d=128, r=128, page=20, prefix=777,
                                lens=tuple(range(3, 43))),
    "many-rows-d80": dict(B=50, H=4, Hk=1, T=1, d=80, r=80, page=24, prefix=421,
                          lens=tuple(range(50))),
    "many-rows-d256": dict(B=20, H=8, Hk=2, T=2, d=256, r=64, page=48, prefix=700,
                           lens=tuple(range(0, 60, 3))),
    "many-rows-d40": dict(B=30, H=4, Hk=1, T=2, d=40, r=40, page=24, prefix=300,
                          lens=tuple(range(30))),
    "many-rows-large-scores": dict(B=20, H=8, Hk=1, T=2, d=64, page=16, prefix=1300,
                                   q_scale=12.0, lens=tuple(range(2, 102, 5))),
    "many-rows-page-of-one": dict(B=17, H=4, Hk=1, page=1, d=128, r=64, prefix=300,
                                  lens=tuple(range(17))),
    # a prefix that a CTA's warps share: up to 32 rows, more of them, with d 256
    "shared-32": dict(B=3, H=10, Hk=1, d=64, page=64, prefix=500, lens=(5, 0, 90)),
    "shared-48-d128": dict(B=6, H=8, Hk=1, d=128, r=64, page=16, prefix=200,
                           lens=(5, 0, 90, 1, 31, 32)),
    "shared-70-d256": dict(B=7, H=10, Hk=1, d=256, r=32, page=128, prefix=333,
                           lens=(5, 0, 90, 1, 31, 32, 128)),
    "shared-40-odd": dict(B=5, H=8, Hk=1, d=96, r=96, page=7, prefix=101, lens=(5, 0, 9, 1, 31)),
    # nine to sixteen rows of a sequence, and more, over its own keys
    "rows-12": dict(B=2, H=6, Hk=2, T=4, d=64, page=16, lens=(100, 3), causal=True),
    "rows-40-d256": dict(B=2, H=4, Hk=1, T=10, d=256, r=64, page=16, lens=(100, 7), causal=True),
    "rows-20-odd": dict(B=2, H=4, Hk=1, T=5, d=128, page=20, r=64, lens=(101, 3), causal=True),
    "fp32": dict(dtype=F, B=3, H=6, Hk=2, T=3, d=40, r=24, page=24, prefix=100, lens=(77, 3, 30),
                 causal=True),
    "fp32-many-rows": dict(dtype=F, B=10, H=8, Hk=2, T=2, d=64, page=16, prefix=200,
                           lens=tuple(range(0, 100, 10)), causal=True),
    "fp32-d256": dict(dtype=F, d=256, r=100, page=10, prefix=50, lens=(77, 3)),
    "fp32-padding": dict(dtype=F, B=4, T=5, lens=(0, 2, 5, 90), causal=True, prefix=50),
}


@pytest.mark.parametrize("name", list(CASES))
def test_matches_oracle(D, cuda_ok, name):
    c = Call(D, **CASES[name], seed=sum(map(ord, name)))
    c.run()
    c.check()


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("B", [1, 40])
def test_a_large_score_selects_its_key(D, cuda_ok, dtype, B):
    """Queries that point at one key each, far above all others, return its value."""
    rng = np.random.default_rng(3)
    d, page, prefix, n = 64, 16, 90, 50
    c = Call(D, dtype=dtype, B=B, H=4, Hk=2, d=d, page=page, prefix=prefix, lens=(n,) * B)
    c.geom.copy_(torch.eye(d))
    c.proj, c.wbuf = D.dark_make_projection(torch.zeros(1, 1, d, device="cuda"), c.geom, 4,
                                            c.proj.dtype)
    # keys of +-1: the one pointed at scores 12 * 64 / 8 = 96, the others 12 N(0, 1)
    c.kp.copy_(torch.from_numpy(rng.choice([-1.0, 1.0], c.kp.shape)))
    c.vp.copy_(torch.from_numpy(rng.standard_normal(c.vp.shape)))
    want = torch.empty_like(c.out)
    for b in range(B):
        for h in range(4):
            j = int(rng.integers(0, prefix + n))
            pages, at = (c.shared, j) if j < prefix else (c.table[b], j - prefix)
            p = pages[at // page]
            c.q[b, h, 0] = 12 * c.kp[p, h // 2, at % page]
            want[b, h, 0] = c.vp[p, h // 2, at % page]
    c.run()
    # the others' weight is below 140 e^-40; the value itself is rounded once more
    torch.testing.assert_close(c.out, want, rtol=2.0 ** -7, atol=1e-4)


@pytest.mark.parametrize("d,page", [(64, 64), (128, 24), (256, 128)])
def test_long_prefix(D, cuda_ok, d, page):
    """Many tiles a range: against fp64 products on the GPU, root mean square error. The
    roundings of the query, the weights and the result are each at most 2^-8 relative and
    independent: together below sqrt(3) 2^-8 of the root mean square output, with the
    queries' and weights' part growing no faster than the output's own sum."""
    B, H, T, prefix = 64, 8, 8, 20011
    c = Call(D, B=B, H=H, Hk=1, T=T, d=d, r=d, page=page, prefix=prefix, lens=(9,) * B, causal=True)
    c.run()
    assert c.status.item() == 0
    k, v = (x[c.d_shared.long()].double().permute(1, 0, 2, 3).reshape(-1, d)[:prefix]
            for x in (c.kp, c.vp))
    m = torch.from_numpy(c.stored_geom()).cuda()
    for b in range(0, B, 13):
        own = c.d_table[b].long()
        kk, vv = (torch.cat([p, x[own].double().permute(1, 0, 2, 3).reshape(-1, d)[:9]])
                  for p, x in ((k, c.kp), (v, c.vp)))
        y = torch.einsum("hri,hrj,hti->htj", m, m, c.q[b].double()) / d ** 0.5
        z = y @ kk.T
        last = prefix + 9 - T + torch.arange(T, device="cuda")
        z = z.where(torch.arange(len(kk), device="cuda") <= last[:, None], -torch.inf)
        ref = torch.softmax(z, dim=-1) @ vv
        err = (c.out[b].double() - ref).pow(2).mean().sqrt() / ref.pow(2).mean().sqrt()
        assert err <= 3 ** 0.5 * H8


@pytest.mark.parametrize("scale", [12.0, 40.0])
def test_references_follow_rising_scores(D, cuda_ok, scale):
    """Several tiles a range, and a key late in the prefix far above all before it: its weight
    passes those against the first scores by up to 2^400."""
    rng = np.random.default_rng(5)
    d, page, prefix = 64, 64, 60000
    c = Call(D, B=40, H=4, Hk=2, d=d, page=page, prefix=prefix, lens=(5,) * 40)
    c.geom.copy_(torch.eye(d))
    c.proj, c.wbuf = D.dark_make_projection(torch.zeros(1, 1, d, device="cuda"), c.geom, 4,
                                            c.proj.dtype)
    g = torch.Generator(device="cuda").manual_seed(3)
    c.kp.copy_(torch.randint(0, 2, c.kp.shape, generator=g, device="cuda") * 2 - 1)
    c.vp.copy_(torch.randn(c.vp.shape, generator=g, device="cuda"))
    want = torch.empty_like(c.out)
    for b in range(40):
        for h in range(4):
            j = int(rng.integers(0, prefix))
            p = c.shared[j // page]
            c.q[b, h, 0] = scale * c.kp[p, h // 2, j % page]
            want[b, h, 0] = c.vp[p, h // 2, j % page]
    c.run()
    assert c.status.item() == 0
    # scores: scale * 64 / 8 at the key, scale N(0, 1) elsewhere (below scale 5.2 of 60000 keys
    # but for 1e-2 of all queries: 33 e^-33 of the weight at scale 12)
    torch.testing.assert_close(c.out, want, rtol=2.0 ** -7, atol=1e-4)


@pytest.mark.parametrize("dtype,d", [(BF, 64), (BF, 256), (BF, 36), (F, 64)])
@pytest.mark.parametrize("what", ["nan", "inf"])
def test_hidden_values_stay_hidden(D, cuda_ok, dtype, d, what):
    """Causal: keys and values that only later queries see do not reach earlier ones."""
    for T, lens in [(3, (21, 3)), (20, (40, 20))]:
        kw = dict(dtype=dtype, T=T, d=d, r=d, lens=lens, causal=True, prefix=20, seed=4)
        ref = Call(D, **kw)
        ref.run()
        c = Call(D, **kw)
        for b in range(2):
            last = lens[b] - 1
            p = c.table[b][last // c.page]
            c.kp[p, :, last % c.page] = float(what)
            c.vp[p, :, last % c.page] = float(what)
        c.run()
        assert c.status.item() == D.DARK_ERR_NUMERIC
        assert not torch.isfinite(c.out[:, :, T - 1]).any()
        e = 2.0 ** -22 if dtype == F else 2.0 ** -7
        torch.testing.assert_close(c.out[:, :, :T - 1], ref.out[:, :, :T - 1], rtol=e, atol=e * 0.1)


@pytest.mark.parametrize("dtype", [BF, F])
def test_bad_lists_are_reported(D, cuda_ok, dtype):
    kw = dict(dtype=dtype, B=3, prefix=20, lens=(20, 30, 40), page=16)
    ref = Call(D, **kw)
    ref.run()
    for bad in (10 ** 6, -1):
        c = Call(D, **kw)
        c.d_table[1, 0] = bad
        c.run()
        assert c.status.item() == D.DARK_ERR_INVALID_ARG
        assert torch.equal(c.out[0], ref.out[0]) and torch.equal(c.out[2], ref.out[2])
    # a length past the list is taken as the list's, a negative one as 0
    c = Call(D, **dict(kw, lens=(20, -5, 48)))
    c.d_lens[2] = 49
    c.run()
    assert c.status.item() == D.DARK_ERR_INVALID_ARG
    c.status.zero_()
    c.check()


# few rows, a prefix that warps share, tcgen05 with tensor copies and with odd pages, fp32
@pytest.mark.parametrize("dtype,B,d,page", [(BF, 2, 64, 16), (BF, 6, 64, 16), (BF, 20, 64, 16),
                                            (BF, 20, 128, 64), (BF, 20, 64, 20), (BF, 20, 256, 16),
                                            (F, 3, 64, 16), (F, 20, 40, 24)])
@pytest.mark.parametrize("at", [0, 11, -1])
def test_bad_prefix_pages_are_reported(D, cuda_ok, dtype, B, d, page, at):
    """A page number outside the cache in the shared list is not followed, and the next call with
    a right list is right."""
    kw = dict(dtype=dtype, B=B, H=4, Hk=1, d=d, r=32, page=page, prefix=777,
              lens=tuple(i % 40 for i in range(B)))
    c = Call(D, **kw)
    good = c.d_shared.clone()
    for bad in (10 ** 6, -1, c.cache.pages, -2 ** 31, 2 ** 31 - 1):
        c.d_shared.copy_(good)
        c.d_shared[at] = bad
        c.run()
        assert c.status.item() == D.DARK_ERR_INVALID_ARG
        c.status.zero_()
    c.d_shared.copy_(good)
    c.run()
    c.check()


@pytest.mark.parametrize("dtype", [BF, F])
def test_lists_may_share_pages(D, cuda_ok, dtype):
    """Sequences with the same pages, and a prefix that is also a sequence's own."""
    c = Call(D, dtype=dtype, B=3, T=2, prefix=64, lens=(40, 40, 40), page=16)
    c.table[1] = c.table[0]
    c.table[2] = c.shared[:3]
    c.kp.nan_to_num_(0.5), c.vp.nan_to_num_(0.5, posinf=0.25)
    c.d_table.copy_(_i32(c.table))
    c.run()
    c.check()
    q = c.q.clone()
    q[1] = q[0]
    c.q = q
    c.run()
    assert torch.equal(c.out[0], c.out[1])


def test_queries_past_fp16_are_reported(D, cuda_ok):
    c = Call(D, prefix=20)
    c.q[1, 2, 0, 5] = 1e5
    c.run()
    assert c.status.item() == D.DARK_ERR_NUMERIC
    rest = torch.ones(2, 4, dtype=torch.bool)
    rest[1, 2] = False
    assert torch.isfinite(c.out[rest.cuda()]).all()


@pytest.mark.parametrize("B,prefix,d", [(2, 20, 64), (20, 600, 64), (20, 600, 128), (2, 20, 256)])
@pytest.mark.parametrize("rows", [1, 40])
def test_geometry_products_past_fp16(D, cuda_ok, B, prefix, d, rows):
    """M q passes 65504 where q and y = M^T M q / sqrt(d) do not: rows of 0.05 against queries of
    6e4 (d 0.05 6e4 = 1.9e5 and more). One row of M alone, or several between rows of zeros."""
    c = Call(D, B=B, H=8, Hk=2, T=2, d=d, r=48, prefix=prefix, lens=tuple(range(2, 2 + 2 * B, 2)))
    c.geom.zero_()
    c.geom[:, 47 if rows == 1 else slice(3, 48, 7)] = 0.05
    c.proj, c.wbuf = D.dark_make_projection(torch.zeros(1, 1, 48, device="cuda"), c.geom, 8,
                                            c.proj.dtype)
    sign = torch.randint(0, 2, c.q.shape[:3], device="cuda",
                         generator=torch.Generator("cuda").manual_seed(1)) * 2 - 1
    c.q.copy_(6e4 * sign[..., None])
    c.kp *= 2.0 ** -10                                 # scores of about 6 and more
    c.run()
    c.check()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("powers", [(-12, 0, 3, 3), (3, 0, -12, -12), (-40, -2, 1, 3), (-3, 2, -6, 3)])
def test_geometries_of_rising_rows(D, cuda_ok, d, powers):
    """M q of 256 rows that grow or shrink along them, by powers of two a quarter: a warp meets
    several of them, and rows far below (or of zeros) first."""
    c = Call(D, B=3, H=4, Hk=2, T=2, d=d, r=256, prefix=40, lens=(30, 2, 77), q_scale=0.5)
    scale = torch.tensor(powers, device="cuda").repeat_interleave(64).double()
    c.geom.mul_((2.0 ** scale).float()[:, None])
    c.proj, c.wbuf = D.dark_make_projection(torch.zeros(1, 1, 256, device="cuda"), c.geom, 4,
                                            c.proj.dtype)
    c.run()
    c.check()


@pytest.mark.parametrize("dtype,B,T", [(BF, 2, 2), (BF, 2, 4), (BF, 8, 2), (F, 2, 2)])
def test_small_geometries_keep_their_bits(D, cuda_ok, dtype, B, T):
    """M = 2^-12 against keys of 2^24 gives the bits of M = 1: powers of two alone (c_m M stays a
    normal fp16 number; M q, about 2^-13, does not lose its low bits)."""
    outs = []
    for e in (0, 12):
        c = Call(D, dtype=dtype, B=B, H=8, Hk=2, T=T, prefix=200, lens=tuple(range(T, T + 2 * B, 2)))
        c.geom.copy_(torch.eye(64) * 2.0 ** -e)
        c.proj, c.wbuf = D.dark_make_projection(torch.zeros(1, 1, 64, device="cuda"), c.geom, 8,
                                                c.proj.dtype)
        c.kp *= 2.0 ** (2 * e)
        c.run()
        assert c.status.item() == 0
        outs.append(c.out)
    assert torch.equal(*outs)


@pytest.mark.parametrize("page", [16, 20])
@pytest.mark.parametrize("j", [3, 599])
@pytest.mark.parametrize("big", [1e5, -1e5])
def test_prefix_keys_past_fp16_are_reported(D, cuda_ok, page, j, big):
    """A key of one key head in a whole tile, or in the tile that ends inside a page; heads
    that read the other key head keep their results."""
    kw = dict(B=20, H=8, Hk=2, T=2, page=page, prefix=600, lens=tuple(range(2, 42, 2)))
    ref = Call(D, **kw)
    ref.run()
    assert ref.status.item() == 0
    c = Call(D, **kw)
    c.kp[c.shared[j // page], 1, j % page, 7] = big
    c.run()
    assert c.status.item() == D.DARK_ERR_NUMERIC
    assert torch.equal(c.out[:, :4], ref.out[:, :4])


def test_queries_past_fp16_after_the_geometry_are_reported(D, cuda_ok):
    c = Call(D, B=20, H=8, Hk=2, T=2, page=16, prefix=600, lens=tuple(range(2, 42, 2)))
    c.geom.copy_(4 * torch.eye(64))
    c.proj, c.wbuf = D.dark_make_projection(torch.zeros(1, 1, 64, device="cuda"), c.geom, 8,
                                            c.proj.dtype)
    ref = c.run().clone()
    assert c.status.item() == 0
    c.q[3, 2, 1, 5] = 6e4                              # times 16 / 8
    c.run()
    assert c.status.item() == D.DARK_ERR_NUMERIC
    rest = torch.ones(20, 8, 2, dtype=torch.bool)
    rest[3, 2, 1] = False
    assert torch.equal(c.out[rest.cuda()], ref[rest.cuda()])


@pytest.mark.parametrize("dtype,B,prefix", [(BF, 4, 50), (BF, 20, 600), (F, 4, 50)])
@pytest.mark.parametrize("what", [6e4, "inf", "nan"])
def test_padding_queries_may_hold_anything(D, cuda_ok, dtype, B, prefix, what):
    lens = (0, 2, 4, 90) * (B // 4)
    c = Call(D, dtype=dtype, B=B, H=8, Hk=2, T=5, lens=lens, causal=True, prefix=prefix)
    c.geom.fill_(1.0)                                  # 6e4 becomes 64 * 6e4 / 8
    c.proj, c.wbuf = D.dark_make_projection(torch.zeros(1, 1, 64, device="cuda"), c.geom, 8,
                                            c.proj.dtype)
    want = c.run().clone()
    assert c.status.item() == 0
    pad = torch.tensor([[n - 5 + t < 0 for t in range(5)] for n in lens], device="cuda")
    c.q[pad[:, None].expand(B, 8, 5)] = 0.0
    c.q[..., 5][pad[:, None].expand(B, 8, 5)] = float(what)
    c.run()
    assert c.status.item() == 0
    assert torch.equal(c.out, want)
    assert not c.out[pad[:, None].expand(B, 8, 5)].any()


@pytest.mark.parametrize("dtype", [BF, F])
def test_calls_repeat_to_the_bit_and_share_no_state(D, cuda_ok, dtype):
    """Again, in a replayed graph on another stream, and two calls at once."""
    a = Call(D, dtype=dtype, B=9, H=8, T=2, prefix=300, lens=tuple(range(0, 90, 10)), causal=True)
    b = Call(D, dtype=dtype, B=9, H=8, T=2, prefix=200, lens=tuple(range(9, 99, 10)), seed=2)
    want_a, want_b = a.run().clone(), b.run().clone()
    assert torch.equal(a.run(), want_a)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for c, s in ((a, s1), (b, s2)):
        c.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(c.graph, stream=s):
            c.run()
        c.out.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(s1):
            a.graph.replay()
        with torch.cuda.stream(s2):
            b.graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a.out, want_a) and torch.equal(b.out, want_b)
    # a replay follows new lengths
    a.lens = [x + 2 for x in a.lens]
    a.d_lens.copy_(_i32(a.lens).clamp(max=a.table.shape[1] * a.page))
    a.lens = a.d_lens.tolist()
    a.kp.nan_to_num_(0.5), a.vp.nan_to_num_(0.5, posinf=0.25)
    torch.cuda.synchronize()
    a.graph.replay()
    torch.cuda.synchronize()
    a.check()


def test_a_workspace_serves_smaller_batches(D, cuda_ok):
    """Sequences leave a batch one by one; its workspace stays."""
    kw = dict(H=8, Hk=8, page=64, prefix=1000)
    ws = None
    for B in (64, 63, 33, 17, 8, 1):
        c = Call(D, B=B, lens=tuple(3 * i for i in range(B)), **kw)
        ws = c.ws if ws is None else ws
        c.run(ws=ws)
        c.check()


@pytest.mark.parametrize("dtype,B,prefix", [(BF, 2, 50), (BF, 20, 600), (F, 20, 50)])
def test_results_in_the_queries(D, cuda_ok, dtype, B, prefix):
    """out in the memory of q, with other strides as well."""
    c = Call(D, dtype=dtype, B=B, H=8, Hk=2, T=3, prefix=prefix, lens=tuple(range(B)), causal=True)
    want = c.run().clone()
    q = c.q
    for out in (lambda t: t, lambda t: t.view(B, 3, 8, 64).permute(0, 2, 1, 3)):
        c.q = q.clone()
        assert torch.equal(c.run(out=out(c.q)), want)
    assert c.status.item() == 0


def test_large_cache_offsets(D, cuda_ok):
    """Pages whose values lie past 2^32 elements of the pool."""
    d, page, Hk = 256, 128, 8
    n = (1 << 32) // (d * page * Hk) + 4
    kp = torch.zeros(n, Hk, page, d, dtype=BF, device="cuda")
    vp = torch.zeros(n, Hk, page, d, dtype=BF, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    small = [torch.randn(3, Hk, page, d, generator=g, device="cuda").to(BF) for _ in range(2)]
    far = torch.tensor([n - 1, n - 3, n - 2], dtype=torch.int32, device="cuda")
    q = torch.randn(1, Hk, 1, d, generator=g, device="cuda").to(BF)
    proj, wbuf = D.dark_make_projection(torch.zeros(1, 1, d, device="cuda"),
                                        torch.eye(d, device="cuda")[None], Hk, D.DARK_BF16)
    outs = []
    for k, v, pages in ((small[0], small[1], torch.arange(3, dtype=torch.int32, device="cuda")),
                        (kp, vp, far)):
        cache, out = D.kv_cache(k, v), torch.empty_like(q)
        if k is kp:                                    # through the append, to the same places
            cat = [x.permute(1, 0, 2, 3).reshape(1, Hk, 3 * page, d).contiguous() for x in small]
            D.dark_kv_append(cache, *cat, far[None], torch.zeros(1, dtype=torch.int32, device="cuda"))
        ws = D.alloc_cache_attention_workspace(proj, cache, 1, Hk, 1, page, 2, "cuda")
        D.dark_cache_attention_fwd(proj, cache, q, out, pages[None, 1:].contiguous(),
                                   torch.tensor([200], dtype=torch.int32, device="cuda"),
                                   prefix_pages=pages[:1], prefix_len=page, ws=ws)
        outs.append(out)
    assert torch.equal(*outs)


@pytest.mark.parametrize("dtype", [BF, F])
def test_decoding_with_the_cache_is_causal_attention(D, cuda_ok, dtype):
    """The operators together: a prompt's queries and keys normed and rotated, the prompt
    appended, then tokens one by one and a few at a time; every output is the row of the
    exact mode's causal self-attention over the whole sequence."""
    B, H, L, d, page, prompt = 2, 4, 61, 64, 16, 40
    rng = np.random.default_rng(12)
    x = [torch.from_numpy(rng.standard_normal((B, H, L, d))).cuda().to(dtype) for _ in range(3)]
    code = D.DARK_BF16 if dtype == BF else D.DARK_F32
    gam = [1 + 0.1 * torch.from_numpy(rng.standard_normal((1, d))).float().cuda() for _ in range(2)]
    geom = torch.from_numpy(np.eye(d) + 0.05 * rng.standard_normal((H, d, d))).float().cuda()
    proj, wbuf = D.dark_make_projection(torch.zeros(1, 1, d, device="cuda"), geom, H, code)
    rope = D.dark_rope_init(d)
    q, k = torch.empty_like(x[0]), torch.empty_like(x[1])
    D.dark_qk_norm_rope_fwd(x[0], x[1], q, k, gamma_q=gam[0], gamma_k=gam[1], rope=rope, pos0=0)
    want = O.exact_attention(_np(q), _np(k), _np(x[2]), _np(geom), causal=True)

    per = -(-L // page)
    table = _i32(rng.permutation(B * per).reshape(B, per))
    kp, vp = (torch.zeros(B * per, H, page, d, dtype=dtype, device="cuda") for _ in range(2))
    cache = D.kv_cache(kp, vp)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    got = torch.empty_like(q)
    at = 0
    for T in [prompt, 1, 1, 1, 3, 8, 7]:
        new = slice(at, at + T)
        D.dark_kv_append(cache, x[1][:, :, new], x[2][:, :, new], table, lens, gamma_k=gam[1],
                         rope=rope)
        lens += T
        qs = torch.empty(B, H, T, d, dtype=dtype, device="cuda")
        D.dark_qk_norm_rope_fwd(x[0][:, :, new], None, qs, None, gamma_q=gam[0], rope=rope, pos0=at)
        assert torch.equal(qs, q[:, :, new])
        ws = D.alloc_cache_attention_workspace(proj, cache, B, H, T, 0, per, "cuda")
        D.dark_cache_attention_fwd(proj, cache, qs, got[:, :, new], table, lens,
                                   flags=D.DARK_CAUSAL, ws=ws)
        at += T
    assert at == L
    err = np.abs(_np(got) - want)
    # the library's tolerances for the exact mode: fp32 1e-4 of the head's largest, bf16 2e-2
    if dtype == F:
        assert (err.max(axis=(2, 3)) / np.abs(want).max(axis=(2, 3))).max() <= 1e-4
    else:
        assert err.max() <= 2e-2


def test_a_wait_that_runs_out_is_reported(D, cuda_ok):
    """The tcgen05 kernel's waits are bounded: the testing stall ends in a status, and the
    next call is right again."""
    c = Call(D, B=20, H=8, Hk=1, T=2, prefix=600, lens=tuple(range(2, 42, 2)))
    D.dark_set_test_stall_cycles(20000)
    try:
        c.run()
        torch.cuda.synchronize()
    finally:
        D.dark_set_test_stall_cycles(0)
    assert c.status.item() == D.DARK_ERR_TIMEOUT
    c.status.zero_()
    c.run()
    c.check()
