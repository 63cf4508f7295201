"""Inputs of the cache attention whose result shows how queries and weights are rounded, with
their exact results and error bounds (numpy; used by the CPU and the GPU tests).

Queries are multiples s q0 of one direction a key head, the geometry c_h times the identity, so
that y = kappa s q0 with kappa the only factor that is no short number. Most keys are -q0: their
scores lie hundreds below and their weights vanish.

 * "queries": pairs of keys +-delta, delta = q0_j e_i - q0_i e_j, with values of opposite sign.
   Their exact scores are 0 and the result is 0. A rounding of y by relative errors up to h moves
   a score by at most 2 h S, S = kappa s |q0_i q0_j| (the largest pair's), and the result, a mean
   of tanh of such errors, by no more.
 * "weights": a key 0 and a key -tau q0, whose scores differ by D, with values v_c and -1: columns
   with v_c near e^-D cancel, so that roundings of the weights are not hidden by the result's. Rounding
   the weights by h moves the result by at most h sum p |v|; D is off by at most D times the
   queries' error."""
import numpy as np

U = 2.0 ** -24


def round_to(x, fmt):
    """x (fp64) in a format: fp64 (none), fp32, fp16, bf16, or bf16x2 (hi + lo in bf16)."""
    x = np.asarray(x, np.float64)
    if fmt == "fp64":
        return x
    if fmt == "fp16":
        return x.astype(np.float16).astype(np.float64)
    if fmt == "fp32":
        return x.astype(np.float32).astype(np.float64)
    if fmt == "bf16x2":
        hi = round_to(x, "bf16")
        return hi + round_to(x - hi, "bf16")
    m, e = np.frexp(x)                                 # bf16: 8 bits, ties to even
    return np.ldexp(np.rint(m * 256.0), e - 8)


# largest relative error of a rounding
STEP = {"fp64": 0.0, "fp32": U, "fp16": 2.0 ** -11, "bf16": 2.0 ** -8, "bf16x2": 2.0 ** -16}


class Inputs:
    """kind: "queries" or "weights"; n visible keys, all shared by the sequences."""

    def __init__(self, kind, rng, B, H, Hk, T, d, n, weight=1.0):
        self.kind, self.B, self.H, self.Hk, self.T, self.d, self.n = kind, B, H, Hk, T, d, n
        self.c = rng.uniform(3.0, 5.0, H)              # geometry of query head h: c[h] I
        q0 = round_to(rng.uniform(4.0, 8.0, (Hk, d)) * rng.choice([-1.0, 1.0], (Hk, d)), "bf16")
        self.s = rng.choice([0.5, 1.0, 2.0], (B, H, T))
        self.q = self.s[..., None] * np.repeat(q0, H // Hk, 0)[None, :, None, :]
        self.q0 = q0
        self.k = np.repeat(-q0[:, None], n, 1)
        self.v = round_to(rng.standard_normal((Hk, n, d)), "bf16")
        self.at = [rng.permutation(n) for _ in range(Hk)]
        self.pairs = []
        for x in range(Hk):
            if kind == "queries":
                used = []
                for a, b in self.at[x][:6].reshape(3, 2):
                    i, j = rng.choice(d, 2, replace=False)
                    delta = np.zeros(d)
                    delta[i], delta[j] = q0[x, j], -q0[x, i]
                    self.k[x, a], self.k[x, b] = delta, -delta
                    self.v[x, a] = rng.choice([-1.0, 1.0], d)
                    self.v[x, b] = -self.v[x, a]
                    used.append(abs(q0[x, i] * q0[x, j]))
                self.pairs.append(max(used))
            else:
                a, b = self.at[x][:2]
                tau = 2.0 / (16.0 / d ** 0.5 * (q0[x] ** 2).sum())       # D about 2 at c = 4, s = 1
                self.k[x, a], self.k[x, b] = 0.0, round_to(-tau * q0[x], "bf16")
                self.v[x, a] = round_to(np.exp(-np.linspace(0.3, 6.0, d)), "bf16")
                self.v[x, b] = -1.0

    def kappa(self, w):
        """y = kappa q, from the stored rows w [H] of the geometry (c_m c, as rounded)."""
        return 2.0 * np.log(2.0) * w ** 2

    def stored(self, fmt):
        """c_m c in the projection's type."""
        return round_to(self.c * self.d ** -0.25 * np.sqrt(0.5 / np.log(2.0)), fmt)

    def result(self, w, y_fmt="fp64", p_fmt="fp64"):
        """[B][H][T][d] with y (in the kernels' base-2 units) and the weights rounded."""
        y = round_to(2.0 * (w ** 2)[None, :, None, None] * self.q, y_fmt)
        k, v = (np.repeat(x, self.H // self.Hk, 0) for x in (self.k, self.v))
        z = np.einsum("bhtd,hnd->bhtn", y, k)
        p = np.exp2(z - z.max(-1, keepdims=True))
        return np.einsum("bhtn,hnd->bhtd", round_to(p, p_fmt), v) / p.sum(-1, keepdims=True)

    def bound(self, w, y_fmt, p_fmt, out_fmt, r):
        """Limits of |result - exact| with y in y_fmt and weights in p_fmt; r rows of the geometry."""
        kap = self.kappa(w)[None, :, None] * self.s
        G = self.H // self.Hk
        exact = self.result(w)
        chain = (r + 2 * self.d + 16) * U
        # M q and the second product keep 22 bits of what they are given
        hq = STEP[y_fmt] + chain + 2.0 ** -21
        if self.kind == "queries":
            tol = 2 * hq * kap * np.repeat(self.pairs, G)[None, :, None] + STEP[p_fmt] + 64 * U
            tol = np.broadcast_to(tol[..., None], exact.shape)
        else:
            k = np.repeat(np.stack([self.k[x, self.at[x][1]] for x in range(self.Hk)]), G, 0)
            D = -np.einsum("bhtd,hd->bht", kap[..., None] / self.s[..., None] * self.q, k)[..., None]
            va = np.repeat(np.stack([self.v[x, self.at[x][0]] for x in range(self.Hk)]), G, 0)[None, :, None]
            pb = 1.0 / (1.0 + np.exp(D))
            tol = pb * (1 - pb) * (va + 1) * D * hq * 1.01 + \
                (STEP[p_fmt] + 64 * U) * (pb + (1 - pb) * np.abs(va))
        return tol + (np.abs(exact) + tol) * STEP[out_fmt]
