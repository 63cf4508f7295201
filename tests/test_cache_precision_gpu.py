"""The cache attention's number formats, path by path (GPU, through the C ABI): queries after the
geometry as hi + lo in bf16 (16 bits) or, over long prefixes of many rows, in fp16 (11 bits);
weights as hi + lo where 8 rows are taken at once, else in bf16; fp32 throughout for fp32. The
inputs and bounds are those of cache_precision.py, which its CPU tests show to fail for
queries, or weights, in one bf16."""
import numpy as np
import pytest
import torch

from cache_precision import Inputs, round_to

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32
HL, B16, H16 = "bf16x2", "bf16", "fp16"


@pytest.fixture(scope="module")
def D(cuda_ok):
    from random_feature_linear_b200 import dark
    return dark


# type, B, H, Hk, T, d, keys, page, where the keys are, formats of queries and weights
PATHS = {
    "own-8-rows": (BF, 3, 8, 2, 2, 64, 300, 16, "own", HL, HL),
    "own-8-rows-d128": (BF, 3, 8, 2, 2, 128, 300, 24, "own", HL, HL),
    "own-8-rows-d256": (BF, 2, 8, 4, 1, 256, 200, 64, "own", HL, HL),
    "own-16-rows": (BF, 2, 8, 2, 4, 128, 300, 16, "own", HL, B16),
    "own-40-rows": (BF, 2, 8, 2, 10, 64, 300, 7, "own", HL, B16),
    "own-40-rows-d256": (BF, 2, 8, 2, 10, 256, 200, 16, "own", HL, HL),
    "prefix-few-rows": (BF, 1, 8, 2, 2, 64, 500, 16, "prefix", HL, HL),
    "prefix-16-rows": (BF, 1, 8, 2, 4, 64, 500, 16, "prefix", HL, B16),
    "prefix-32-rows": (BF, 4, 8, 2, 2, 64, 500, 16, "prefix", HL, HL),
    "prefix-32-rows-d128": (BF, 4, 8, 2, 2, 128, 500, 24, "prefix", HL, HL),
    "prefix-48-rows": (BF, 6, 8, 2, 2, 64, 500, 16, "prefix", HL, B16),
    "prefix-48-rows-d128": (BF, 6, 8, 2, 2, 128, 333, 16, "prefix", HL, B16),
    "prefix-80-rows-d256": (BF, 10, 8, 2, 2, 256, 300, 16, "prefix", HL, HL),
    "prefix-128-rows": (BF, 16, 8, 2, 2, 64, 600, 16, "prefix", H16, B16),
    "prefix-128-rows-d128": (BF, 16, 8, 2, 2, 128, 640, 64, "prefix", H16, B16),
    "prefix-320-rows": (BF, 40, 8, 2, 2, 64, 600, 20, "prefix", H16, B16),
    "fp32": (F, 3, 8, 2, 2, 64, 300, 16, "own", "fp32", "fp32"),
    "fp32-prefix": (F, 16, 8, 2, 2, 64, 300, 16, "prefix", "fp32", "fp32"),
    "d36": (BF, 3, 8, 2, 2, 36, 300, 16, "own", "fp32", "fp32"),
}


@pytest.mark.parametrize("kind", ["queries", "weights"])
@pytest.mark.parametrize("name", list(PATHS))
def test_formats(D, cuda_ok, name, kind):
    dtype, B, H, Hk, T, d, n, page, where, y_fmt, p_fmt = PATHS[name]
    rng = np.random.default_rng(sum(map(ord, name + kind)))
    x = Inputs(kind, rng, B, H, Hk, T, d, n)
    per = -(-n // page)
    order = rng.permutation(per + 3)[:per]
    pools = []
    for rows in (x.k, x.v):
        pool = np.full((per + 3, Hk, page, d), np.nan)
        for j in range(n):
            pool[order[j // page], :, j % page] = rows[:, j]
        pools.append(torch.from_numpy(pool).cuda().to(dtype))
        assert np.array_equal(np.nan_to_num(pools[-1].double().cpu().numpy()),
                              np.nan_to_num(round_to(pool, "fp32" if dtype == F else "bf16")))
    eye = torch.eye(d, device="cuda")
    geom = torch.from_numpy(x.c).float().cuda()[:, None, None] * eye
    proj, wbuf = D.dark_make_projection(torch.zeros(1, 1, d, device="cuda"), geom, H,
                                        D.DARK_F32 if dtype == F else D.DARK_BF16)
    w = wbuf.view(torch.float32 if dtype == F else torch.float16)[:H * (1 + d) * d]
    w = w.reshape(H, 1 + d, d)[:, 1, 0].double().cpu().numpy()
    cache = D.kv_cache(*pools)
    q = torch.from_numpy(x.q).cuda().to(dtype)
    out = torch.full_like(q, float("nan"))
    pages = torch.from_numpy(order.astype(np.int32)).cuda()
    own = where == "own"
    ws = D.alloc_cache_attention_workspace(proj, cache, B, H, T, 0 if own else n, per, "cuda")
    ws.fill_(0xff)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    D.dark_cache_attention_fwd(
        proj, cache, q, out, pages.expand(B, per).contiguous(),
        torch.full((B,), n if own else 0, dtype=torch.int32, device="cuda"),
        prefix_pages=None if own else pages, prefix_len=0 if own else n, ws=ws, dev_status=status)
    assert status.item() == 0
    bound = x.bound(w, y_fmt, p_fmt, "fp32" if dtype == F else "bf16", d)
    worst = (np.abs(out.double().cpu().numpy() - x.result(w)) / bound).max()
    assert worst <= 1.0, worst
