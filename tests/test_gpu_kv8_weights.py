"""The softmax weights of the attention over the 8-bit cache where they, or the rows
of V, differ by many powers of two: what a key adds is held to its own size, not
to the largest weight's or the largest V's.

Tolerance.  Scores, sums and the output's rounding as in test_gpu_attention.py and
test_gpu_kv8.py.  A bf16 call's weight w of a key, times the key's power of two P and
scaled so that the row's largest w P lies above 2^6 (2^7 rounded to a whole power,
and growing past it only), is rounded to f16: 2^-11 of it, or 2^-25 at least.  Two
e5m2 numbers take 3 of the 11 bits at least each, and the third, times 2^5, is rounded
to 3 bits of what is left: 2^-9 of the weight, or half of 2^-16 2^-5 = 2^-22 at least.
So a weight is off by at most (2^-9 + 2^-11) of itself, or by (2^-22 + 2^-25) 2^-6
of the row's largest w P; times codes of up to 448."""
import numpy as np
import pytest
import torch

import oracle as O
from test_gpu_kv8 import Case8, quantised

pytestmark = pytest.mark.gpu

# one half, two halves, two tiles of rows; pages of boxes, of fours, of any size
TENSOR = [(2, 16), (8, 16), (20, 16), (4, 12), (8, 5)]


class Sharp(Case8):
    """Scores along one direction, chosen for each entry (natural units, at the first
    query's size; the others' are up to four times as flat), and V's sizes."""

    def __init__(self, lens, score, size, D=64, **kw):
        super().__init__(lens, D=D, **kw)
        rng = np.random.default_rng(11)
        rows = self.S * self.H * self.G
        q = rng.normal(size=(self.B, self.S, self.H * self.G, D)) * 0.05
        q[..., 0] = 8.0 / (1.0 + 3.0 * (np.arange(rows).reshape(self.S, -1) % 5) / 4.0)
        self.q = torch.from_numpy(q).to(self.dtype)
        x = self.cache.numpy().copy()
        for b, n in enumerate(lens):
            for e in range(n + self.S):
                shared = e < self.shared
                blk = (self.stable if shared else self.table[b])[e // self.bs]
                k, v = x[0, 0, blk, e % self.bs], x[0, 1, blk, e % self.bs]
                if not shared or b == 0:
                    k *= 0.02
                    k[:, 0] = score(e, n) / (8.0 * self.score["scale"])
                    v *= size(e, n)
        self.codes, self.scales = quantised(x)
        self.stands_for()

    def check_weights(self, r):
        out, lse = r.out.double().cpu().numpy(), r.lse.double().cpu().numpy()
        bf16 = self.dtype == torch.bfloat16
        for b in range(self.B):
            ref, k, _ = Case8.__mro__[1].oracle(self, b)
            e, n = self.score_error(b, k), len(k)
            sc = np.swapaxes(self.scales, -1, -2)[0, 1]
            power = 2.0 ** (O.entries(sc[..., None], self.table[b], self.bs, n)[..., 0] - 127)   # [n, H]
            if self.shared:
                power[:self.shared] = 2.0 ** (O.entries(sc[..., None], self.stable, self.bs, self.shared)[..., 0] - 127)
            most = np.stack([(ref.p[h] * power[:, h // self.G]).max(-1) for h in range(self.H * self.G)], -1)  # [S, Hq]
            step = n * 448 * (2.0 ** -22 + 2.0 ** -25) * 2.0 ** -6 * most[..., None] if bf16 else 0.0
            half = 2.0 ** -8 if bf16 else 2.0 ** -24
            tol = (2 * e + (2.0 ** -9 + 2.0 ** -11 if bf16 else 0) + (n + 16) * 2.0 ** -24) * ref.mass + step + half * np.abs(ref.out)
            far = np.abs(out[b] - ref.out)
            assert (far <= tol).all(), (b, (far / tol).max(), np.argwhere(far > tol)[:4])
            assert (np.abs(lse[b] - ref.lse) <= e + (n + 16) * 2.0 ** -24 + 2.0 ** -22 * np.abs(ref.lse)).all()


def place(where, n):
    return {"newest": n - 3, "middle": n // 2, "oldest": 2}[where]


@pytest.mark.parametrize("where", ["newest", "middle", "oldest"])
@pytest.mark.parametrize("G,bs", TENSOR)
def test_an_entry_with_most_of_the_weight_and_little_v(G, bs, where):
    """An entry that holds nearly all of the weight, with no V, little V or V as the
    others': what the others add together is not lost beside it."""
    for n, depth in ((300, 9.0), (2048, 12.0), (2048, 16.0), (9000, 15.0)):
        for v in (0.0, 2.0 ** -12, 1.0):
            def score(e, m):
                return 0.0 if e == place(where, n) else -depth - (e * 7 % 13) / 13.0

            c = Sharp([n], score, lambda e, m: v if e == place(where, n) else 1.0, S=3, H=1, G=G, bs=bs, seed=n)
            c.check_weights(c.run())


@pytest.mark.parametrize("where", ["newest", "middle", "oldest"])
@pytest.mark.parametrize("G,bs", TENSOR)
def test_a_large_v_of_little_weight(G, bs, where):
    """A V row far larger than the others, of a weight that leaves it nothing: the
    others' weights, the heavy and the many light ones, are held as without it."""
    for n, power, light in ((700, 8, 60.0), (2500, 10, 60.0), (2500, 16, 60.0), (2500, 40, 90.0)):
        def score(e, m):
            if e == place(where, n):
                return -light
            return 0.0 if e == n - 70 else -10.0 - (e * 7 % 13) / 13.0

        c = Sharp([n], score, lambda e, m: 2.0 ** power if e == place(where, n) else 1.0, S=3, H=1, G=G, bs=bs, seed=n)
        c.check_weights(c.run())


@pytest.mark.parametrize("G,bs", TENSOR)
def test_products_that_grow_and_shrink(G, bs):
    """V's sizes and the weights moving against each other along the keys, both ways,
    over far more powers of two than an e5m2 number has."""
    for a, b in ((0.02, 0.0), (-0.02, 0.0), (0.03, -0.04), (-0.03, 0.05), (0.0, 0.06), (0.0, -0.06)):
        c = Sharp([1500, 40], lambda e, m: a * e - 20.0, lambda e, m: 2.0 ** (b * (e - 700)), S=3, H=2, G=G, bs=bs, seed=5)
        c.check_weights(c.run())


@pytest.mark.parametrize("G,bs", TENSOR)
def test_light_weights_of_a_shared_prefix(G, bs):
    """The heavy entry among a request's own, the many light ones shared, and the other way round."""
    for heavy in (1400, 5):
        c = Sharp([1300, 1450, 1333], lambda e, m: 0.0 if e in (heavy, m) else -13.0, lambda e, m: 0.0 if e in (heavy, m) else 1.0,
                  S=2, H=1, G=G, bs=bs, seed=6, shared=1291)
        c.check_weights(c.run())


def test_scores_far_from_zero():
    """Scores whose own steps are larger than a power of two: the references are the
    scores', the products' powers stay exact."""
    for size in (2.0 ** 12, 2.0 ** 20, 2.0 ** 30):
        c = Sharp([600], lambda e, m: -16.0 * (e % 5), lambda e, m: 2.0 ** (e % 9 - 4), S=3, H=1, G=4, seed=8)
        c.q = (c.q.float() * size).to(c.q.dtype)
        c.q[..., 1:] = 0
        c.check_weights(c.run())
