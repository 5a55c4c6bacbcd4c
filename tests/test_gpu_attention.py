"""GPU parity of the attention over the paged cache, the entry weights and the
eviction with the float64 oracle, through the C ABI.

Tolerances.  A score's error is at most E = 2^-24 ((D + 4) |scale| sum|q||k| + 8
cap + 4 |x|): the products' float32 sum, the cap (1 - 2 / (1 + e): rounding of
three operations and two hardware functions of 2 ulp, times the cap) and the
bias.  A weight p moves by at most 2E relative (its own score and the
softmax's sum), by 2^-8 more where it is rounded to bf16; n sums of float32 add
n 2^-24.  So |out - ref| <= (2E + 2^-8 [bf16] + (n + 16) 2^-24) sum p|v| + half a
step of the output's type (2^-8 or 2^-24) |ref|, and |lse - ref| <= E + (n + 16)
2^-24 + 2^-22 |ref| (log2, its scaling, and the running reference)."""
import math

import numpy as np
import pytest
import torch

import oracle as O
from speculative_decoding_verification_37_gb300 import _lib as L
from speculative_decoding_verification_37_gb300 import api

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


class Case:
    """A batch with its tensors on the GPU and its oracle's arrays."""

    def __init__(self, lens, S=5, H=2, G=2, D=64, bs=16, dtype="bf16", layers=1, layer=0, tree=False, inplace=False,
                 gaps=False, window=0, docs=None, cap=0.0, slopes=False, shared=0, seed=0, spare=0, extra_blocks=0):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.lens, self.S, self.H, self.G, self.D, self.bs = list(lens), S, H, G, D, bs
        self.B, self.dtype, self.layer, self.layers = len(lens), DT[dtype], layer, layers
        self.shared, self.inplace = shared, inplace
        cap_len = max(lens) + (S if inplace else 0) + spare
        self.max_blocks = max(1, -(-cap_len // bs))
        need = [-(-(n + S + spare) // bs) for n in lens]
        nb = sum(need) + extra_blocks + -(-shared // bs)
        perm = rng.permutation(nb)
        table = np.zeros((self.B, self.max_blocks), np.int32)
        at = 0
        for b, k in enumerate(need):
            k = min(k, self.max_blocks)
            table[b, :k] = perm[at:at + k]
            at += k
        self.stable = None
        if shared:
            self.stable = perm[at:at + -(-shared // bs)].astype(np.int32)
        self.table = table
        self.nb = nb
        self.cache = torch.randn((layers, 2, nb, bs, H, D), generator=g).to(self.dtype)
        self.temp = None if inplace else torch.randn((self.B, layers, 2, S, H, D), generator=g).to(self.dtype)
        self.q = (1.5 * torch.randn((self.B, S, H * G, D), generator=g)).to(self.dtype)
        width = self.max_blocks * bs
        text = np.array(lens, np.int64)
        self.key_pos = None
        if gaps:
            self.key_pos = np.cumsum(rng.integers(1, 4, (self.B, width)), 1).astype(np.int32)
            text = np.array([self.key_pos[b, n - 1] + 1 if n else 0 for b, n in enumerate(lens)])
        self.mask = None
        depth = np.tile(np.arange(S), (self.B, 1))
        if tree:
            W = (S + 31) // 32
            self.mask = np.zeros((self.B, S, W), np.uint32)
            self.parent = np.full((self.B, S), -1)
            depth[:] = 0
            for b in range(self.B):
                for i in range(S):
                    if i:
                        p = self.parent[b, i] = int(rng.integers(0, i))
                        depth[b, i] = depth[b, p] + 1
                        self.mask[b, i] = self.mask[b, p]
                    self.mask[b, i, i // 32] |= np.uint32(1 << (i % 32))
        self.pos = (text[:, None] + depth).astype(np.int32) if tree or gaps else None
        self.first = None if docs is None else np.array([int(t * docs) for t in text], np.int32)
        self.slopes = (2.0 ** -(1 + np.arange(H * G) % 6)).astype(np.float32) if slopes else None
        self.score = dict(scale=1.0 / math.sqrt(D), softcap=cap)
        self.window = window

    # -- oracle ------------------------------------------------------------
    def planes(self):
        return self.cache[self.layer, 0].float().numpy(), self.cache[self.layer, 1].float().numpy()

    def row_keys(self, b):
        n, P = self.lens[b], self.shared
        kc, vc = self.planes()
        total = n + (self.S if self.inplace else 0)
        k, v = (O.entries(x, self.table[b], self.bs, total) for x in (kc, vc))
        if P:
            k[:P], v[:P] = (O.entries(x, self.stable, self.bs, P) for x in (kc, vc))
        if not self.inplace:
            t = self.temp[b, self.layer].double().numpy()
            k, v = np.concatenate([k, t[0]]), np.concatenate([v, t[1]])
        qp = self.pos[b] if self.pos is not None else np.arange(n, n + self.S)
        kp = np.concatenate([self.key_pos[b, :n] if self.key_pos is not None else np.arange(n), qp])
        return k, v, qp, kp

    def masked(self, b, qp, kp):
        n = self.lens[b]
        off = O.hidden(qp, kp, first_pos=None if self.first is None else self.first[b], window=self.window)
        off[:, n:] |= O.candidate_mask(self.S, None if self.mask is None else self.mask[b])
        return off

    def oracle(self, b):
        k, v, qp, kp = self.row_keys(b)
        off = self.masked(b, qp, kp)
        return O.attend(self.q[b].double().numpy(), k, v, qp, kp, off, slopes=self.slopes, **self.score), k, off

    # -- GPU ---------------------------------------------------------------
    def args(self):
        d = lambda x: None if x is None else (x if torch.is_tensor(x) else torch.from_numpy(  # noqa: E731
            np.ascontiguousarray(x).view(np.int32) if x.dtype == np.uint32 else np.ascontiguousarray(x))).cuda()
        a = dict(block_size=self.bs, layer=self.layer, temp_kv=d(self.temp), tree_mask=d(self.mask), pos=d(self.pos),
                 key_pos=d(self.key_pos), first_pos=d(self.first), slopes=d(self.slopes), window=self.window, **self.score)
        if self.shared:
            a.update(shared_table=d(self.stable), shared_len=self.shared)
        return [self.q.cuda(), self.cache.cuda(), d(self.table), d(np.array(self.lens, np.int32))], a

    def run(self, **over):
        pos, a = self.args()
        a.update(over)
        r = api.verify_attention(*pos, **a)
        torch.cuda.synchronize()
        return r

    def score_error(self, b, k):
        """E of the module's note, the largest over the request's pairs."""
        aq = np.abs(self.q[b].double().numpy())
        dots = max(float((aq[:, h] @ np.abs(k[:, h // self.G]).T).max()) for h in range(self.H * self.G)) if len(k) else 0.0
        reach = 0.0 if self.slopes is None else 4 * 40.0     # a farther key's weight is below 2^-57
        return 2.0 ** -24 * ((self.D + 4) * abs(self.score["scale"]) * dots + 8 * self.score["softcap"] + reach)

    def check(self, r, rows=None):
        out, lse = r.out.double().cpu().numpy(), r.lse.double().cpu().numpy()
        half = 2.0 ** -8 if self.dtype == torch.bfloat16 else 2.0 ** -24
        for b in range(self.B) if rows is None else rows:
            ref, k, off = self.oracle(b)
            e, n = self.score_error(b, k), len(k) + self.shared
            tol = (2 * e + (2.0 ** -8 if half > 1e-4 else 0) + (n + 16) * 2.0 ** -24) * ref.mass + half * np.abs(ref.out)
            bad = np.abs(out[b] - ref.out) > tol + 1e-30
            assert not bad.any() and np.isfinite(out[b]).all(), (b, np.argwhere(bad)[:4], np.abs(out[b] - ref.out).max())
            seen = np.isfinite(ref.lse)
            assert np.array_equal(np.isneginf(lse[b]), ~seen), b
            assert not out[b][~seen].any(), b
            far = np.abs(lse[b][seen] - ref.lse[seen])
            assert (far <= e + (n + 16) * 2.0 ** -24 + 2.0 ** -22 * np.abs(ref.lse[seen])).all(), (b, far.max())


SHAPES = [
    dict(lens=[1], S=1, H=1, G=1, D=64),
    dict(lens=[0, 0], S=1, H=1, G=1, D=64),                            # nothing cached: the candidate alone
    dict(lens=[0, 1, 31, 32, 33, 63, 64, 65, 127, 129, 300], S=5, H=2, G=2, D=64),
    dict(lens=[100, 7], S=13, H=2, G=4, D=128, tree=True),
    dict(lens=[257, 64], S=3, H=1, G=7, D=128, bs=1),
    dict(lens=[90, 200, 13], S=2, H=3, G=1, D=72, bs=5),
    dict(lens=[500], S=8, H=4, G=8, D=128, bs=48),                     # 64 rows a head
    dict(lens=[70, 130], S=20, H=2, G=4, D=128, tree=True),            # 80 rows
    dict(lens=[40, 77], S=70, H=1, G=2, D=64, tree=True, inplace=True),  # 140 rows, three mask words
    dict(lens=[33, 90], S=4, H=2, G=3, D=256, bs=64),
    dict(lens=[60, 10], S=3, H=2, G=2, D=8),
    dict(lens=[129, 130], S=33, H=1, G=1, D=160, inplace=True),
    dict(lens=[3000], S=2, H=2, G=2, D=128),                           # keys split over blocks
    dict(lens=[300, 40], S=12, H=2, G=8, D=128, tree=True),            # 96 rows
    dict(lens=[500, 9], S=40, H=1, G=4, D=64, tree=True),              # 160 rows: two row tiles
    dict(lens=[20], S=300, H=1, G=1, D=64, tree=True),                 # a wide tree, ten mask words
    dict(lens=[131, 5], S=300, H=1, G=1, D=64, inplace=True, bs=8),
    dict(lens=[200, 60], S=7, H=2, G=2, D=64, bs=128), dict(lens=[90], S=4, H=1, G=2, D=128, bs=24),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_shapes(i, dtype):
    c = Case(dtype=dtype, seed=i, **SHAPES[i])
    c.check(c.run())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kw", [
    dict(cap=5.0), dict(slopes=True), dict(window=40), dict(window=1), dict(docs=0.5), dict(docs=1.0),
    dict(gaps=True, window=50, slopes=True), dict(gaps=True, docs=0.7, cap=2.0),
    dict(tree=True, window=2, docs=0.99), dict(cap=30.0, slopes=True, window=100, docs=0.3, tree=True, gaps=True),
    dict(inplace=True, window=7), dict(inplace=True, tree=True, gaps=True, slopes=True),
    dict(layers=3, layer=2, spare=40),
])
def test_scores_and_masks(kw, dtype):
    c = Case([5, 64, 200, 131, 0 if not kw.get("gaps") else 1], S=6, H=2, G=3, D=64, dtype=dtype, seed=3, **kw)
    c.check(c.run())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kw", [
    dict(shared=64), dict(shared=50), dict(shared=1), dict(shared=600, D=128, G=4), dict(shared=130, inplace=True),
    dict(shared=90, tree=True, cap=4.0, slopes=True), dict(shared=200, window=60), dict(shared=200, docs=0.9),
    dict(shared=256, G=8, S=9, lens=[256] * 20),                       # nothing of one's own but the candidates
    dict(shared=77, bs=7, D=72),
    # more than 128 queries a head: two query tiles
    dict(shared=300, G=8, S=6, lens=[300, 333, 310, 301, 450, 512], window=200),
    dict(shared=300, G=8, S=6, lens=[300, 333, 310, 301, 450, 512], docs=0.8, cap=5.0, slopes=True, D=128),
    dict(shared=700, G=4, S=9, lens=[700 + 7 * i for i in range(17)], tree=True, cap=30.0, D=128),
    dict(shared=129, G=16, S=10, lens=[129, 140], slopes=True, inplace=True),
])
def test_shared_prefix(kw, dtype):
    kw = dict(kw)
    lens = kw.pop("lens", [kw["shared"] + n for n in (0, 1, 15, 100, 33)])
    args = dict(S=4, H=2, G=2, D=64)
    args.update(kw)
    c = Case(lens, dtype=dtype, seed=5, **args)
    c.check(c.run())


def test_shared_prefix_equals_reading_it_per_request():
    """The same entries, once through every request's own table: the same up
    to the arithmetic's own tolerance (both are checked against the oracle)."""
    c = Case([300, 290, 512], S=5, H=2, G=4, D=128, shared=256, seed=8)
    c.check(c.run())
    whole = c.shared // c.bs
    c.table[:, :whole] = c.stable[:whole]
    c.shared = 0
    c.check(c.run())


# every kernel: 32, 64 and 128 rows on tcgen05, the warp instructions, the CUDA cores
KERNELS = [("bf16", 2, 16), ("bf16", 8, 16), ("bf16", 16, 16), ("bf16", 2, 5), ("bf16", 8, 5), ("f32", 2, 16)]


@pytest.mark.parametrize("dtype,G,bs", KERNELS)
def test_masked_places_may_hold_anything(dtype, G, bs):
    """NaN and infinities past the length, before the document, outside the
    window and in other branches do not show; visible ones stay in their rows."""
    kw = dict(S=6, H=2, G=G, D=64, bs=bs, tree=True, docs=0.5, window=30, dtype=dtype, seed=9, spare=30)
    c = Case([70, 100], **kw)
    clean = c.run()
    c.check(clean)
    for bad in (float("nan"), float("inf"), -float("inf")):
        dirty = Case([70, 100], **kw)
        dirty.parent = c.parent
        for b, n in enumerate(c.lens):
            lo = max(int(c.first[b]), n - 29)            # the first position that candidate 0 sees
            for e in list(range(0, lo)) + list(range(n, c.max_blocks * c.bs)):
                if e // c.bs < c.max_blocks and (e < n or e // c.bs < -(-(n + 36) // c.bs)):
                    dirty.cache[0, :, c.table[b, e // c.bs], e % c.bs] = bad
            dirty.temp[b, 0, :, 5] = bad                 # node 5: the last one, nobody's ancestor
        r = dirty.run()
        assert torch.equal(r.out[:, :5], clean.out[:, :5]) and torch.equal(r.lse[:, :5], clean.lse[:, :5])
        assert not torch.isfinite(r.out[:, 5]).all()


@pytest.mark.parametrize("dtype,G,bs", KERNELS)
def test_masked_value_in_a_tile_other_rows_see(dtype, G, bs):
    """A non-finite V that one branch sees must not reach the others."""
    c = Case([40], S=3, H=1, G=G, D=64, bs=bs, tree=True, dtype=dtype, seed=1)
    c.mask[0, :, 0] = [1, 0b11, 0b101]
    c.pos[0] = [40, 41, 41]
    clean = c.run()
    c.temp[0, 0, 1, 1, 0, 5] = float("nan")
    r = c.run()
    assert torch.equal(r.out[0, [0, 2]], clean.out[0, [0, 2]])
    assert torch.isnan(r.out[0, 1, :, 5]).all() and torch.equal(r.lse, clean.lse)


def test_masked_value_of_the_shared_prefix():
    """The same where two query tiles share the keys: an entry that only some
    requests' documents reach."""
    c = Case([140, 150, 160], S=8, H=1, G=8, D=64, shared=130, docs=0.0, seed=14)
    c.first = np.array([0, 60, 100], np.int32)
    clean = c.run()
    c.check(clean)
    e = 80                                                # request 2 does not see it
    c.cache[0, 1, c.stable[e // c.bs], e % c.bs] = float("inf")
    r = c.run()
    assert torch.equal(r.out[2], clean.out[2]) and torch.equal(r.lse, clean.lse)
    assert not torch.isfinite(r.out[:2]).any(-1).all()


@pytest.mark.parametrize("dtype,G,bs", KERNELS)
def test_rows_that_see_nothing(dtype, G, bs):
    c = Case([50, 0, 20], S=3, H=2, G=G, D=64, bs=bs, tree=True, dtype=dtype, seed=2)
    c.mask[:, 1] = 0                                     # candidate 1 sees no candidate
    c.first = np.array([49, 0, 99], np.int32)            # request 2: the document starts past everything
    r = c.run()
    c.check(r)
    assert torch.isneginf(r.lse[1, 1]).all() and torch.isneginf(r.lse[2]).all()


@pytest.mark.parametrize("dtype,G,bs", KERNELS)
def test_scales(dtype, G, bs):
    """Negative and zero scales."""
    for scale in (-0.2, 0.0):
        c = Case([70, 30], S=4, H=2, G=G, D=64, bs=bs, dtype=dtype, seed=15)
        c.score["scale"] = scale
        c.check(c.run())


@pytest.mark.parametrize("bs", [16, 4])
@pytest.mark.parametrize("D,G,S", [(8, 2, 5), (24, 8, 6), (40, 16, 5), (56, 3, 3), (72, 2, 5), (80, 8, 6), (96, 16, 5),
                                   (104, 4, 3), (112, 16, 9), (120, 1, 1)])
def test_head_sizes(D, G, S, bs):
    """Heads that fill their tiles' columns in part: nothing of the next head's
    columns shows, whatever they hold."""
    kw = dict(S=S, H=2, G=G, D=D, bs=bs, tree=True, cap=20.0, slopes=True, docs=0.2, seed=D)
    c = Case([300, 40, 129, 512], **kw)
    clean = c.run()
    c.check(clean)
    dirty = Case([300, 40, 129, 512], **kw)
    dirty.cache[..., 1, :] = float("nan")
    dirty.temp[..., 1, :] = float("inf")
    r = dirty.run()
    assert torch.equal(r.out[:, :, :G], clean.out[:, :, :G]) and torch.equal(r.lse[:, :, :G], clean.lse[:, :, :G])


@pytest.mark.parametrize("kw", [
    dict(D=96, shared=700, G=8, S=9, lens=[700 + 7 * i for i in range(17)], tree=True, cap=30.0),
    dict(D=72, shared=90, G=2, S=5, lens=[90, 200, 333]), dict(D=40, shared=400, G=16, S=9, lens=[500, 400, 401]),
    dict(D=96, S=12, G=8, lens=[2000, 1500, 900], docs=0.4), dict(D=112, S=1, G=4, lens=[3000, 5, 700], inplace=True, gaps=True, window=900),
    dict(D=80, S=40, G=4, lens=[900, 100], tree=True)])
def test_head_sizes_of_long_and_shared_keys(kw):
    kw = dict(kw)
    c = Case(kw.pop("lens"), H=2, seed=3, **kw)
    c.check(c.run())


def test_growing_maxima():
    """Scores that rise along the keys, so that every tile brings a new maximum."""
    for G, D in ((2, 64), (8, 128), (16, 64)):
        c = Case([1500], S=6, H=1, G=G, D=D, seed=16)
        ramp = torch.linspace(0, 12, 1500)
        u = torch.nn.functional.normalize(torch.randn(D, generator=torch.Generator().manual_seed(0)), dim=0)
        for e in range(1500):
            c.cache[0, 0, c.table[0, e // 16], e % 16, 0] += (ramp[e] * u).to(c.dtype)
        c.q += (6 * u).to(c.dtype)
        c.check(c.run())


def test_empty_batch():
    c = Case([5], S=3, H=1, G=2, D=64)
    (q, cache, table, lens), a = c.args()
    r = api.verify_attention(q[:0], cache, table[:0], lens[:0], block_size=c.bs)
    assert r.out.shape == (0, 3, 2, 64) and r.lse.shape == (0, 3, 2)
    w, kp = torch.zeros((0, 16), device="cuda"), torch.zeros((0, 16), dtype=torch.int32, device="cuda")
    api.attention_weights(q[:0], r.lse, cache, table[:0], lens[:0], lens[:0], w, block_size=c.bs)
    api.evict_kv(cache, table[:0], lens[:0], w, kp, block_size=c.bs, budget=4)
    torch.cuda.synchronize()


def test_strides_and_views():
    """q as a slice of a fused projection, in other dimension orders."""
    c = Case([33, 100], S=5, H=2, G=2, D=64, seed=4)
    want = c.run()
    pos, a = c.args()
    q = pos[0]
    fused = torch.full((2, 5, 8, 64), float("nan"), dtype=q.dtype, device="cuda")
    fused[:, :, 2:6] = q
    heads_first = q.permute(2, 0, 1, 3).contiguous().permute(1, 2, 0, 3)
    for view in (fused[:, :, 2:6], heads_first):
        got = api.verify_attention(view, *pos[1:], **a)
        assert torch.equal(got.out, want.out) and torch.equal(got.lse, want.lse)


def test_bad_requests_are_flagged():
    c = Case([60, 61, 62, 63], S=2, H=1, G=2, D=64, seed=6)
    pos, a = c.args()
    lens = torch.tensor([60, -1, 2000, 63], dtype=torch.int32, device="cuda")
    table = pos[2].clone()
    table[3, 1] = c.nb                                    # entries 16..31 of request 3
    flags = torch.zeros(4, dtype=torch.int32, device="cuda")
    ws = api.workspace(L.SPEC_WS_ATTENTION, 4, 2 * 2, 64, "cuda")
    assert L.spec_get_status(ws) == 0
    r = api.verify_attention(pos[0], pos[1], table, lens, flags=flags, ws=ws, **a)
    assert L.spec_get_status(ws) == L.SPEC_FLAG_BAD_INPUT and L.spec_get_status(ws) == 0
    assert flags.tolist() == [0, 1, 1, 1]
    assert not r.out[1:3].any() and torch.isneginf(r.lse[1:3]).all()
    c.check(r, rows=[0])
    # the bad block's entries are left out: as if they were masked
    k, v, qp, kp = c.row_keys(3)
    off = c.masked(3, qp, kp)
    off[:, 16:32] = True
    ref = O.attend(c.q[3].double().numpy(), k, v, qp, kp, off, **c.score)
    assert np.abs(r.lse[3].cpu().numpy() - ref.lse).max() < 1e-5
    # below a shared prefix
    c = Case([60, 61], S=2, H=1, G=2, D=64, seed=6, shared=48)
    pos, a = c.args()
    flags = torch.zeros(2, dtype=torch.int32, device="cuda")
    r = api.verify_attention(*pos[:3], torch.tensor([60, 47], dtype=torch.int32, device="cuda"), flags=flags, **a)
    assert flags.tolist() == [0, 1] and not r.out[1].any()
    c.check(r, rows=[0])
    a["shared_table"][1] = -1
    r = api.verify_attention(*pos, flags=flags.zero_(), **a)
    assert flags.tolist() == [1, 1]


def test_repeats_graphs_and_streams_agree():
    """The same call again, on another stream, captured and replayed, and after
    a call of another shape on the same workspace: the same bits."""
    c = Case([3000, 17, 900], S=5, H=2, G=4, D=128, seed=7, shared=16)
    pos, a = c.args()
    want = api.verify_attention(*pos, **a)
    other = Case([10, 20, 30], S=5, H=2, G=4, D=128, seed=8, shared=8)
    other.check(other.run())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        r = api.verify_attention(*pos, **a)
        r2 = api.verify_attention(*pos, stream=s, **a)
    torch.cuda.synchronize()
    for x in (r, r2):
        assert torch.equal(x.out, want.out) and torch.equal(x.lse, want.lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cap = api.verify_attention(*pos, **a)
    cap.out.zero_()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(cap.out, want.out) and torch.equal(cap.lse, want.lse)
    # lengths are read on the device: a replay follows them
    pos[3][1] = 16
    g.replay()
    torch.cuda.synchronize()
    c.lens[1] = 16
    c.check(cap)


def test_captured_before_any_eager_call():
    """The first call of its sizes under capture: two graphs and the eager
    calls between them do not share an unzeroed workspace."""
    c = Case([2000, 33, 900], S=4, H=2, G=4, D=128, seed=23)
    pos, a = c.args()
    want = api.verify_attention(*pos, **a)
    torch.cuda.synchronize()
    api.clear_workspaces()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, api.verify_attention(*pos, **a)))
    eager = api.verify_attention(*pos, **a)
    for g, r in graphs:
        g.replay()
        g.replay()
    torch.cuda.synchronize()
    for r in (eager, graphs[0][1], graphs[1][1]):
        assert torch.equal(r.out, want.out) and torch.equal(r.lse, want.lse)


def test_another_stream_with_a_new_workspace():
    """The workspace's first use on a side stream: zeroed there, before the call."""
    c = Case([700, 40], S=3, H=2, G=2, D=64, seed=21)
    pos, a = c.args()
    want = api.verify_attention(*pos, **a)
    torch.cuda.synchronize()
    for how in (lambda s: s, lambda s: s.cuda_stream):
        api.clear_workspaces()
        s = torch.cuda.Stream()
        busy = torch.empty(1 << 28, device="cuda")
        for _ in range(20):
            busy.fill_(1.0)                               # the current stream is late
        r = api.verify_attention(*pos, stream=how(s), **a)
        s.synchronize()
        assert torch.equal(r.out, want.out) and torch.equal(r.lse, want.lse)
        torch.cuda.synchronize()


def test_offsets_past_32_bits():
    """Blocks at the end of a cache of more than 2^32 elements."""
    H, D, bs, S = 8, 128, 16, 2
    nb = (1 << 32) // (bs * H * D) + 64
    cache = torch.empty((1, 2, nb, bs, H, D), dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([[nb - 1, 3, nb - 7]], dtype=torch.int32, device="cuda")
    g = torch.Generator("cuda").manual_seed(0)
    small = torch.randn((1, 2, 3, bs, H, D), generator=g, device="cuda", dtype=torch.bfloat16)
    cache[:, :, ids[0].long()] = small
    q = torch.randn((1, S, H, D), generator=g, device="cuda", dtype=torch.bfloat16)
    temp = torch.randn((1, 1, 2, S, H, D), generator=g, device="cuda", dtype=torch.bfloat16)
    lens = torch.tensor([40], dtype=torch.int32, device="cuda")
    a = api.verify_attention(q, cache, ids, lens, block_size=bs, temp_kv=temp)
    b = api.verify_attention(q, small, torch.arange(3, dtype=torch.int32, device="cuda")[None], lens, block_size=bs,
                             temp_kv=temp)
    assert torch.equal(a.out, b.out) and torch.equal(a.lse, b.lse)


def test_many_requests_ragged():
    """More requests than threads of a block, most of them tiny."""
    rng = np.random.default_rng(1)
    lens = rng.integers(0, 50, 700)
    lens[123] = 2000
    c = Case(lens.tolist(), S=1, H=2, G=2, D=64, seed=10)
    c.check(c.run(), rows=[0, 1, 122, 123, 124, 350, 511, 512, 699])


@pytest.mark.parametrize("D,G,S,H", [(64, 2, 3, 4), (128, 1, 2, 8), (128, 4, 5, 8), (128, 4, 13, 8), (256, 1, 9, 4), (128, 8, 12, 8), (64, 4, 40, 8),
                                     (256, 2, 10, 4), (256, 4, 11, 2), (72, 8, 5, 8)])
def test_many_tiles_per_block(D, G, S, H):
    """Long items, several to a block: the ring of stages goes round often."""
    c = Case([2500, 1900, 2000, 2501, 2300, 2048, 2049, 2200] * 3, S=S, H=H, G=G, D=D, seed=D + G)
    r = c.run()
    c.check(r, rows=[0, 11, 23])
    again = c.run()
    assert torch.equal(r.out, again.out) and torch.equal(r.lse, again.lse)


@pytest.mark.parametrize("D,G,S,H", [(64, 2, 3, 4), (128, 4, 5, 3), (128, 8, 9, 2), (256, 3, 2, 2), (72, 1, 1, 5), (200, 8, 6, 1)])
def test_many_tiles_per_block_f32(D, G, S, H):
    """The same in float32: 16 and 32 rows a block, several row tiles, long items."""
    c = Case([2500, 700, 2000, 33], S=S, H=H, G=G, D=D, seed=D + G, dtype="f32", docs=0.1, slopes=True)
    r = c.run()
    c.check(r)
    again = c.run()
    assert torch.equal(r.out, again.out) and torch.equal(r.lse, again.lse)


# ---------------------------------------------------------------------------
# entry weights
# ---------------------------------------------------------------------------
def weights_case(kw, seed, dtype):
    """A batch whose last entries are committed candidates."""
    kw = dict(kw)
    S = kw.pop("S", 5)
    lens = kw.pop("lens", [5, 64, 200, 131])
    c = Case(lens, S=S, inplace=True, dtype=dtype, seed=seed, **{**dict(H=2, G=2, D=64), **kw})
    rng = np.random.default_rng(seed + 100)
    n_slots = np.array([min(n, int(x)) for n, x in zip(lens, rng.integers(0, S + 1, len(lens)))], np.int32)
    slots = np.full((c.B, S + 2), -5, np.int32)
    pos = np.zeros((c.B, S), np.int32)
    lse = rng.uniform(3, 6, (c.B, S, c.H * c.G)).astype(np.float32)
    for b, n in enumerate(n_slots):
        slots[b, :n] = np.sort(rng.permutation(S)[:n])
        start = lens[b] - n if c.key_pos is None else (c.key_pos[b, lens[b] - n - 1] + 1 if lens[b] > n else 0)
        pos[b, slots[b, :n]] = start + np.arange(n)
    return c, n_slots, slots, pos, lse


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kw", [
    dict(), dict(G=7, D=128, S=13, lens=[300, 40, 13, 64, 65]), dict(cap=5.0, slopes=True), dict(window=30),
    dict(docs=0.5), dict(gaps=True, window=60, slopes=True), dict(D=72, bs=5, H=3), dict(D=256, G=1),
    dict(S=1, G=1, lens=[1, 2, 0, 70]), dict(D=8, H=1), dict(layers=2, layer=1), dict(S=40, G=4, lens=[100, 39]),
    dict(D=160, bs=64),
])
@pytest.mark.parametrize("start", [0, 20])
def test_entry_weights(kw, dtype, start):
    c, n_slots, slots, pos, lse = weights_case(kw, 11, dtype)
    lse[0, :, 0] = -np.inf                                # a candidate head that saw nothing adds nothing
    width = c.max_blocks * c.bs
    rng = np.random.default_rng(0)
    w0 = np.zeros((c.B, width + 3), np.float32)
    for b, n in enumerate(c.lens):
        w0[b, :n - n_slots[b]] = rng.uniform(0, 2, n - n_slots[b])
    (q, cache, table, lens), a = c.args()
    for k in ("temp_kv", "tree_mask"):
        a.pop(k)
    kp0 = None if c.key_pos is None else a["key_pos"].clone()
    weight = torch.from_numpy(w0).cuda()
    a.update(pos=torch.from_numpy(pos).cuda(), slots=torch.from_numpy(slots).cuda())
    api.attention_weights(q, torch.from_numpy(lse).cuda(), cache, table, lens, torch.from_numpy(n_slots).cuda(), weight,
                          shared_len=start, **a)
    torch.cuda.synchronize()
    got = weight.double().cpu().numpy()
    for b, n in enumerate(c.lens):
        m = int(n_slots[b])
        sl = slots[b, :m]
        k = O.entries(c.planes()[0], table[b].tolist(), c.bs, n)
        kp = (c.key_pos[b, :n] if c.key_pos is not None else np.arange(n)).copy()
        kp[n - m:] = pos[b, sl]
        gain = O.entry_weights(c.q[b, sl].double().numpy(), lse[b, sl].astype(np.float64), k, pos[b, sl], kp, m,
                               first_pos=None if c.first is None else c.first[b], window=c.window, start=start,
                               slopes=c.slopes, **c.score)
        # a term moves by its score's error and by lse's rounding to log2 units (2^-24 * 2 |lse|), the
        # exponential's 2 ulp; the float32 sum of m*Hq terms and the old weight
        rel = 2 * c.score_error(b, k) + (m * c.H * c.G + 32) * 2.0 ** -24
        tol = rel * gain + 2.0 ** -23 * (w0[b, :n] + gain)
        assert (np.abs(got[b, :n] - w0[b, :n] - gain) <= tol + 1e-30).all(), (b, np.abs(got[b, :n] - w0[b, :n] - gain).max())
        assert not got[b, n:].any() and np.array_equal(got[b, :min(start, n)], w0[b, :min(start, n)])
        if kp0 is not None:
            want = kp0[b].cpu().numpy().copy()
            want[n - m:n] = pos[b, sl]
            lo = max(start, n - m)                        # entries of a shared prefix are not touched
            assert np.array_equal(a["key_pos"][b].cpu().numpy()[lo:n], want[lo:n])


@pytest.mark.parametrize("kw", [
    dict(H=3, D=128, G=4, lens=[700, 129, 128, 127]), dict(H=1, G=8, S=9, lens=[1000, 5, 0, 260]),
    dict(H=20, S=6, lens=[300, 50]), dict(H=8, G=8, D=128, S=12, lens=[400, 260], cap=20.0),
    dict(H=32, G=1, D=128, S=3, lens=[200, 17]), dict(bs=128, D=128, lens=[300, 128, 1]), dict(bs=8, lens=[131, 8, 9]),
    dict(G=3, S=7, D=128, lens=[520, 90], cap=9.0, slopes=True), dict(G=5, S=11, lens=[600, 300], slopes=True, window=200),
    dict(H=8, G=4, D=128, S=8, lens=[1500, 1100, 30, 2000] * 12, cap=30.0, slopes=True),
    dict(H=5, G=2, S=4, lens=list(range(90, 500, 7)), gaps=True, docs=0.3), dict(H=2, G=64, D=128, S=5, lens=[300, 40]),
    dict(H=128, G=1, D=128, S=3, lens=[70, 7]), dict(H=65, G=3, D=256, S=2, lens=[40]),
    dict(H=2, G=4, D=96, lens=[700, 129, 64]), dict(H=3, G=4, D=72, S=9, lens=[400, 30], cap=9.0), dict(H=2, G=8, D=40, S=9, lens=[300, 129]),
])
def test_entry_weights_of_many_tiles(kw):
    """Odd heads, several passes over the queries, one row past a multiple of the
    columns, long and many requests."""
    test_entry_weights(kw, "bf16", 0)


@pytest.mark.parametrize("kw", [
    dict(H=3, D=128, G=4, lens=[700, 129, 33, 31]), dict(H=1, G=8, S=9, lens=[1000, 5, 0, 260]), dict(H=4, D=256, G=5, S=7, lens=[400, 90]),
    dict(H=8, G=4, S=8, lens=[500, 900, 30] * 9, cap=30.0, slopes=True), dict(H=5, G=2, D=100, S=4, bs=7, lens=[300, 77, 410], gaps=True, docs=0.3)])
def test_entry_weights_of_many_tiles_f32(kw):
    """Odd heads (the last one's buffer), several blocks, rows past a multiple of
    the queries staged at a time."""
    test_entry_weights(kw, "f32", 0)


@pytest.mark.parametrize("bs", [16, 5])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_entry_weights_of_candidates_without_keys(bs, dtype):
    """A candidate whose lse is -inf adds nothing, whatever K holds."""
    c, n_slots, slots, pos, lse = weights_case(dict(D=64, bs=bs, lens=[300, 200, 40]), 5, dtype)
    n_slots[:] = 2
    slots[:, :2] = [0, 1]
    lse[:] = -np.inf
    (q, cache, table, lens), a = c.args()
    for k in ("temp_kv", "tree_mask"):
        a.pop(k)
    cache.fill_(float("nan"))
    weight = torch.rand((c.B, c.max_blocks * bs), device="cuda")
    want = weight.clone()
    a.update(pos=torch.from_numpy(pos).cuda(), slots=torch.from_numpy(slots).cuda())
    api.attention_weights(q, torch.from_numpy(lse).cuda(), cache, table, lens, torch.from_numpy(n_slots).cuda(), weight, **a)
    torch.cuda.synchronize()
    assert torch.equal(weight, want)


def test_entry_weights_without_slots_or_positions():
    """The chain's defaults: candidate j is slot j at its own entry."""
    c = Case([40, 9], S=4, H=1, G=2, D=64, inplace=True, seed=12)
    (q, cache, table, lens), a = c.args()
    n = torch.tensor([3, 4], dtype=torch.int32, device="cuda")
    lse = torch.full((2, 4, 2), 4.0, device="cuda")
    w = torch.zeros((2, c.max_blocks * c.bs), device="cuda")
    api.attention_weights(q, lse, cache, table, lens, n, w, block_size=c.bs)
    for b in range(2):
        m = int(n[b])
        k = O.entries(c.planes()[0], c.table[b], c.bs, c.lens[b])
        qp = np.arange(c.lens[b] - m, c.lens[b])
        gain = O.entry_weights(c.q[b, :m].double().numpy(), np.full((m, 2), 4.0), k, qp, np.arange(c.lens[b]), m, **c.score)
        assert np.allclose(w[b, :c.lens[b]].cpu().numpy(), gain, rtol=1e-4, atol=0)


def test_entry_weights_bad_requests():
    c = Case([40, 41, 42, 43, 44], S=3, H=1, G=2, D=64, inplace=True, seed=13)
    (q, cache, table, lens), a = c.args()
    lse = torch.full((5, 3, 2), 4.0, device="cuda")
    n = torch.tensor([2, 4, 2, 2, 2], dtype=torch.int32, device="cuda")
    slots = torch.tensor([[0, 1, 9], [0, 1, 2], [0, 3, 0], [0, 1, 0], [0, 2, 0]], dtype=torch.int32, device="cuda")
    lens = lens.clone()
    lens[3] = -4
    table = table.clone()
    table[4, 0] = -1
    w = torch.zeros((5, c.max_blocks * c.bs), device="cuda")
    flags = torch.zeros(5, dtype=torch.int32, device="cuda")
    api.attention_weights(q, lse, cache, table, lens, n, w, block_size=c.bs, slots=slots, flags=flags)
    torch.cuda.synchronize()
    assert flags.tolist() == [0, 1, 1, 1, 1]
    assert w[0].any() and not w[1:4].any()
    assert not w[4, :c.bs].any() and w[4, c.bs:44].all()


# ---------------------------------------------------------------------------
# eviction
# ---------------------------------------------------------------------------
def evict_case(lens, budget, *, layers=2, H=2, D=8, bs=4, seed=0, dtype=torch.bfloat16, spare=5, ties=False, order=None):
    rng = np.random.default_rng(seed)
    B = len(lens)
    mb = max(1, -(-(max(lens) + spare) // bs))
    nb = B * mb + 3
    table = rng.permutation(nb)[:B * mb].reshape(B, mb).astype(np.int32)
    bits = torch.from_numpy(rng.integers(0, 256, (layers, 2, nb, bs, H, D * dtype.itemsize), dtype=np.uint8))
    width = mb * bs + 2
    w = np.zeros((B, width), np.float32)
    pos = np.zeros((B, width), np.int32)
    for b, n in enumerate(lens):
        w[b, :n] = rng.integers(0, 5, n) if ties else rng.exponential(1, n)
        p = np.sort(rng.permutation(3 * n + 1)[:n])
        pos[b, :n] = rng.permutation(p) if order == "mixed" else p
    return table, bits, w, pos, nb


def run_evict(table, bits, w, pos, lens, dtype, bs, **kw):
    cache = bits.cuda().view(dtype)
    t = dict(table=torch.from_numpy(table).cuda(), len=torch.tensor(lens, dtype=torch.int32, device="cuda"),
             w=torch.from_numpy(w).cuda(), pos=torch.from_numpy(pos).cuda(),
             blocks=torch.full((len(lens),), -7, dtype=torch.int32, device="cuda"),
             flags=torch.zeros(len(lens), dtype=torch.int32, device="cuda"))
    api.evict_kv(cache, t["table"], t["len"], t["w"], t["pos"], block_size=bs, blocks_in_use=t["blocks"],
                 flags=t["flags"], **kw)
    torch.cuda.synchronize()
    return cache.view(torch.uint8).cpu().numpy(), {k: v.cpu().numpy() for k, v in t.items()}


def check_evict(lens, budget, seed=0, sink=0, recent=0, bs=4, dtype=torch.bfloat16, **kw):
    table, bits, w, pos, nb = evict_case(lens, budget, bs=bs, seed=seed, dtype=dtype, **kw)
    cache, t = run_evict(table, bits, w, pos, lens, dtype, bs, budget=budget, sink=sink, recent=recent)
    want, ww, wp = bits.numpy().copy(), w.copy(), pos.copy()
    moved = 0
    for b, n in enumerate(lens):
        e = O.evict(w[b], pos[b], n, budget=budget, sink=sink, recent=recent)
        assert t["flags"][b] == 0 and t["len"][b] == e.length and t["blocks"][b] == -(-e.length // bs)
        for f, to in e.moves:
            want[:, :, table[b, to // bs], to % bs] = bits.numpy()[:, :, table[b, f // bs], f % bs]
            ww[b, to], wp[b, to] = w[b, f], pos[b, f]
        ww[b, e.length:] = 0
        wp[b, e.length:] = 0
        moved += len(e.moves)
    assert np.array_equal(cache, want) and np.array_equal(t["w"], ww) and np.array_equal(t["pos"], wp)
    return moved


@pytest.mark.parametrize("kw", [
    dict(lens=[30], budget=20), dict(lens=[0, 1, 19, 20, 21, 40, 64], budget=20, sink=2, recent=5),
    dict(lens=[50, 33], budget=1), dict(lens=[50, 51], budget=50, sink=25, recent=25),
    dict(lens=[90, 70, 41], budget=40, ties=True, order="mixed", sink=3, recent=9),
    dict(lens=[3000, 1024, 1025, 2047], budget=1000, ties=True, sink=4, recent=100, order="mixed"),
    dict(lens=[60, 31], budget=30, layers=1, H=1, D=8, bs=1), dict(lens=[60, 31], budget=30, bs=7, dtype=torch.float32),
    dict(lens=[60, 31], budget=30, D=16, dtype=torch.float8_e4m3fn),
    dict(lens=[45, 20], budget=16, layers=9, H=8, D=128, bs=16),
    dict(lens=[40], budget=16, layers=2, H=64, D=256, bs=4),            # a unit of 32 KiB: two pieces
    dict(lens=[5000], budget=4999), dict(lens=[70] * 40, budget=33, recent=33),
    dict(lens=[60000, 50000, 49152, 49153], budget=49000, layers=1, H=1, D=8, bs=64, ties=True, sink=2, recent=300),
])
def test_evict(kw):
    assert check_evict(**{**kw, "lens": list(kw["lens"])}) >= 0


@pytest.mark.parametrize("seed", range(6))
def test_evict_random(seed):
    rng = np.random.default_rng(seed)
    budget = int(rng.integers(1, 200))
    lens = rng.integers(0, 2 * budget + 3, 9).tolist()
    check_evict(lens, budget, seed=seed, sink=int(rng.integers(0, budget // 2 + 1)),
                recent=int(rng.integers(0, budget // 2 + 1)), ties=bool(seed % 2), order="mixed" if seed > 2 else None)


def test_evict_special_weights():
    """-0 ties with 0, infinities order, negative weights are light."""
    lens, bs = [10], 4
    table, bits, w, pos, nb = evict_case(lens, 5, bs=bs, seed=1)
    w[0, :10] = [-0.0, 0.0, np.inf, -np.inf, -1.0, 1e-40, 0.0, 3.0, -0.0, 2.0]
    cache, t = run_evict(table, bits, w, pos, lens, torch.bfloat16, bs, budget=5)
    # inf, 3, 2, 1e-40, then the first of the zeros
    assert sorted(t["pos"][0, :5].tolist()) == sorted(pos[0, [2, 7, 9, 5, 0]].tolist())


def test_evict_bad_requests_stay_as_they_are():
    lens, bs = [30, 31, 32, 33, 34, 35], 4
    table, bits, w, pos, nb = evict_case(lens, 20, bs=bs, seed=2)
    w[1, 7] = np.nan
    pos[2, 3] = -1
    table[3, 5] = nb
    pos[4, :34] = 6                                       # all of them the newest
    given = [30, 31, 32, 33, 34, 1000]
    cache, t = run_evict(table, bits, w, pos, given, torch.bfloat16, bs, budget=20, recent=3)
    assert t["flags"].tolist() == [0, 1, 1, 1, 1, 1] and t["len"].tolist() == [20] + given[1:]
    assert np.array_equal(t["w"][1:], w[1:], equal_nan=True) and np.array_equal(t["pos"][1:], pos[1:])
    want = bits.numpy()
    for b in range(1, 6):
        for j in table[b]:
            if j < nb:
                assert np.array_equal(cache[:, :, j], want[:, :, j])
    assert t["blocks"].tolist() == [5, 8, 8, 9, 9, -7]


def test_evict_again_and_in_a_graph():
    """Two evictions in a row with shrinking budgets, captured and replayed."""
    lens, bs = [60, 75], 4
    table, bits, w, pos, nb = evict_case(lens, 40, bs=bs, seed=3, order="mixed")
    base = [torch.from_numpy(x).cuda() for x in (table, w, pos)]
    n0 = torch.tensor(lens, dtype=torch.int32, device="cuda")
    cache0 = bits.cuda().view(torch.bfloat16)

    def once(cache, n, w, p):
        api.evict_kv(cache, base[0], n, w, p, block_size=bs, budget=50, sink=1, recent=7)
        api.evict_kv(cache, base[0], n, w, p, block_size=bs, budget=31, sink=1, recent=7)

    plain = [cache0.clone(), n0.clone(), base[1].clone(), base[2].clone()]
    once(*plain)
    held = [cache0.clone(), n0.clone(), base[1].clone(), base[2].clone()]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        once(*held)
    for _ in range(2):
        for h, s in zip(held, (cache0, n0, base[1], base[2])):
            h.copy_(s)
        g.replay()
    torch.cuda.synchronize()
    for x, y in zip(plain, held):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert plain[1].tolist() == [31, 31]


# ---------------------------------------------------------------------------
# the operators together
# ---------------------------------------------------------------------------
def test_rounds_of_tree_decoding_with_eviction():
    """Rounds as a user's loop makes them: tree masks and positions, the
    attention of two layers, the walk, the commit, the weights, the eviction;
    a shadow copy of every request's entries follows the oracle."""
    rng = np.random.default_rng(0)
    B, Ly, H, G, D, bs, N, budget, V = 3, 2, 2, 2, 64, 4, 5, 24, 50
    S, mb = N + 1, 10
    g = torch.Generator("cuda").manual_seed(1)
    cache = torch.zeros((Ly, 2, B * mb, bs, H, D), dtype=torch.bfloat16, device="cuda")
    table = torch.from_numpy(rng.permutation(B * mb).reshape(B, mb).astype(np.int32)).cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    lens, text = torch.zeros(B, **i32), torch.zeros(B, **i32)
    weight, key_pos = torch.zeros((B, mb * bs), device="cuda"), torch.zeros((B, mb * bs), **i32)
    shadow = [[] for _ in range(B)]          # (position, weight, K/V [Ly, 2, H, D]) of every entry, in cache order
    kw = dict(block_size=bs, softcap=20.0, slopes=torch.full((H * G,), 0.05, device="cuda"))
    okw = dict(scale=D ** -0.5, softcap=20.0, slopes=[0.05] * (H * G))
    evicted = 0
    for rnd in range(14):
        par = np.array([[0, 0, 1, 1, 3]] * B, np.int32)
        tok = rng.integers(0, V, (B, N)).astype(np.int32)
        tree = [torch.from_numpy(x).cuda() for x in (tok, par)]
        rows = torch.from_numpy(np.tile(np.arange(S, dtype=np.int32), (B, 1))).cuda()
        # the mask and positions depend on the node arrays only: one-logit rows give them before the forward
        shape = api.verify_tree(torch.zeros((B * S, 1), device="cuda"), torch.zeros_like(tree[0]), tree[1], rows, text, R=S)
        q = [torch.randn((B, S, H * G, D), generator=g, device="cuda").bfloat16() for _ in range(Ly)]
        temp = torch.randn((B, Ly, 2, S, H, D), generator=g, device="cuda").bfloat16()
        att = [api.verify_attention(q[l], cache, table, lens, layer=l, temp_kv=temp, tree_mask=shape.tree_mask,
                                    pos=shape.pos, key_pos=key_pos, **kw) for l in range(Ly)]
        logits = rng.standard_normal((B * S, V)).astype(np.float32)
        for b in range(B):                    # the walk follows node 1 most rounds, then node 4, then node 5
            for node, child in ((0, 1), (1, 4), (4, 5))[:int(rng.integers(0, 4))]:
                logits[b * S + node, tok[b, child - 1]] = 9.0
        won = api.verify_tree(torch.from_numpy(logits).cuda(), tree[0], tree[1], rows, text, R=S)
        api.commit_kv(temp, cache, table, won.n_commit, lens, block_size=bs, slots=won.commit_slots)
        for l in range(Ly):
            api.attention_weights(q[l], att[l].lse, cache, table, lens, won.n_commit, weight, layer=l,
                                  slots=won.commit_slots, pos=shape.pos, key_pos=key_pos, **kw)
        text += won.n_commit
        torch.cuda.synchronize()
        for b in range(B):
            n, sl = int(won.n_commit[b]), won.commit_slots[b].tolist()
            e = shadow[b]
            qp = shape.pos[b].cpu().numpy()
            for l in range(Ly):
                t = temp[b, l].double().cpu().numpy()
                k = np.concatenate([np.array([x[2][l, 0] for x in e]).reshape(-1, H, D), t[0]])
                v = np.concatenate([np.array([x[2][l, 1] for x in e]).reshape(-1, H, D), t[1]])
                kp = np.array([x[0] for x in e] + qp.tolist())
                off = np.concatenate([np.zeros((S, len(e)), bool),
                                      O.candidate_mask(S, shape.tree_mask[b].cpu().numpy().view(np.uint32))], 1)
                ref = O.attend(q[l][b].double().cpu().numpy(), k, v, qp, kp, off, **okw)
                assert np.abs(att[l].lse[b].cpu().numpy() - ref.lse).max() < 1e-4
                assert (np.abs(att[l].out[b].double().cpu().numpy() - ref.out) <= 2.0 ** -7 * ref.mass + 1e-6).all()
                kept = sl[:n]
                gain = ref.p[:, kept].sum((0, 1))
                e = [(x[0], x[1] + gain[i], x[2]) for i, x in enumerate(e)]
                new = gain[len(e) + np.array(kept)]
                fresh = new if l == 0 else fresh + new
            shadow[b] = e + [(int(qp[s]), fresh[j], temp[b, :, :, s].double().cpu().numpy()) for j, s in enumerate(kept)]
            w = weight[b, :len(shadow[b])].cpu().numpy()
            assert np.allclose(w, [x[1] for x in shadow[b]], rtol=1e-3), (rnd, b)
            assert key_pos[b, :len(w)].tolist() == [x[0] for x in shadow[b]]
            shadow[b] = [(x[0], float(w[i]), x[2]) for i, x in enumerate(shadow[b])]
        api.evict_kv(cache, table, lens, weight, key_pos, block_size=bs, budget=budget, sink=2, recent=8)
        torch.cuda.synchronize()
        for b in range(B):
            e = O.evict([x[1] for x in shadow[b]], [x[0] for x in shadow[b]], len(shadow[b]), budget=budget, sink=2, recent=8)
            for f, to in e.moves:
                shadow[b][to] = shadow[b][f]
            shadow[b] = shadow[b][:e.length]
            evicted += len(e.moves)
            assert int(lens[b]) == e.length
            assert key_pos[b, :e.length].tolist() == [x[0] for x in shadow[b]] and not key_pos[b, e.length:].any()
            got = cache[:, :, table[b].long()].flatten(2, 3)[:, :, :e.length].double().cpu().numpy()
            want = np.array([x[2] for x in shadow[b]]).transpose(1, 2, 0, 3, 4)
            assert np.array_equal(got, want), (rnd, b)
    assert evicted > 0 and int(text.min()) > budget


# every kernel of the entry weights: tcgen05, the warp instructions, the CUDA cores in both types
WEIGHT_KERNELS = [("bf16", dict(D=64)), ("bf16", dict(D=128, G=4)), ("bf16", dict(D=64, bs=5)), ("bf16", dict(D=160)),
                  ("bf16", dict(H=65, G=3, D=256)), ("f32", dict(D=72, bs=5))]


@pytest.mark.parametrize("dtype,kw", WEIGHT_KERNELS)
def test_entry_weights_positions_below_a_shared_prefix(dtype, kw):
    """Every committed candidate's entry gets its position, also where it lies
    among the shared entries, whose weights stay as they are; a skipped
    request's positions stay too."""
    P, S, n = 40, 3, 3
    lens = [P, P + 1, P + n, P + 20, P - 2, n, 200, P, P + 1]
    c = Case(lens, S=S, inplace=True, dtype=dtype, seed=31, **{**dict(H=2, G=2), **kw})
    (q, cache, table, dl), _ = c.args()
    width = c.max_blocks * c.bs
    rng = np.random.default_rng(7)
    n_slots = np.array([n] * 7 + [2, n], np.int32)
    slots = np.tile(np.arange(S, dtype=np.int32), (c.B, 1))
    slots[8, 1] = S                                       # bad: the request is skipped
    pos = (1000 + rng.permutation(c.B * S).reshape(c.B, S)).astype(np.int32)
    kp0 = rng.integers(0, 900, (c.B, width)).astype(np.int32)
    w0 = rng.uniform(0, 2, (c.B, width)).astype(np.float32)
    lse = rng.uniform(3, 6, (c.B, S, c.H * c.G)).astype(np.float32)
    d = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    key_pos, weight, flags = d(kp0.copy()), d(w0.copy()), torch.zeros(c.B, dtype=torch.int32, device="cuda")
    api.attention_weights(q, d(lse), cache, table, dl, d(n_slots), weight, block_size=c.bs, slots=d(slots), pos=d(pos),
                          key_pos=key_pos, shared_len=P, flags=flags, **c.score)
    torch.cuda.synchronize()
    assert flags.tolist() == [0] * 8 + [1]
    kp, w = kp0.copy(), w0.astype(np.float64)
    for b, length in enumerate(lens[:8]):
        m = int(n_slots[b])
        kp[b, length - m:length] = pos[b, :m]
        k = O.entries(c.planes()[0], c.table[b].tolist(), c.bs, length)
        gain = O.entry_weights(c.q[b, :m].double().numpy(), lse[b, :m].astype(np.float64), k, pos[b, :m], kp[b, :length], m,
                               start=P, **c.score)
        tol = (2 * c.score_error(b, k) + (m * c.H * c.G + 32) * 2.0 ** -24) * gain + 2.0 ** -23 * (w0[b, :length] + gain)
        w[b, :length] += gain
        assert (np.abs(weight[b, :length].double().cpu().numpy() - w[b, :length]) <= tol + 1e-30).all(), b
        assert np.array_equal(weight[b, :min(P, length)].cpu().numpy(), w0[b, :min(P, length)])
    assert np.array_equal(key_pos.cpu().numpy(), kp)


# items split over blocks, on every kernel: tcgen05 with 32, 64 and 128 rows, the warp instructions, the CUDA cores
@pytest.mark.parametrize("dtype,G,bs", KERNELS)
@pytest.mark.parametrize("what", ["query", "tile", "newest", "light"])
def test_nan_of_split_items_shows(what, dtype, G, bs):
    """A NaN that a row sees reaches its result however its keys are split: in
    the query, in all the keys that one block sees, in the newest keys alone
    behind whole tiles, in a key whose block's weights underflow."""
    c = Case([2560, 40], S=5, H=2, G=G, D=64, bs=bs, dtype=dtype, seed=17, slopes=what == "light")
    if c.slopes is not None:
        c.slopes[:] = 1.0
    clean = c.run()
    c.check(clean)
    nan, rows = float("nan"), torch.ones((2, 5, 2 * G), dtype=torch.bool)
    rows[1] = rows[:, :, G:] = False                      # request 0, cached head 0 (the tile, the newest, the light one)
    if what == "query":
        c.q[0, 2] = nan
        rows[:] = False
        rows[0, 2] = True
    elif what == "newest":
        c.temp[0, 0, 0, :, 0] = nan
    else:
        for e in range(1280, 1408) if what == "tile" else (5,):
            c.cache[0, 0, c.table[0, e // bs], e % bs, 0] = nan
    r = c.run()
    out, lse, rows = r.out.float(), r.lse, rows.cuda()
    assert torch.isnan(out[rows]).all() and torch.isnan(lse[rows]).all()
    assert torch.equal(r.out[~rows], clean.out[~rows]) and torch.equal(lse[~rows], clean.lse[~rows])


@pytest.mark.parametrize("dtype,bs", [("bf16", 16), ("bf16", 5), ("f32", 16)])
@pytest.mark.parametrize("G,S", [(2, 2), (8, 6)])
def test_nan_of_a_split_shared_prefix_shows(G, S, dtype, bs):
    """The same in the pass over a shared prefix, up to 64 and more rows."""
    c = Case([1300, 1333, 1500, 1281], S=S, H=2, G=G, D=64, bs=bs, dtype=dtype, seed=18, shared=1280)
    clean = c.run()
    c.check(clean)
    for e in range(256, 512):
        c.cache[0, 0, c.stable[e // bs], e % bs, 0] = float("nan")
    r = c.run()
    assert torch.isnan(r.out[:, :, :G].float()).all() and torch.isnan(r.lse[:, :, :G]).all()
    assert torch.equal(r.out[:, :, G:], clean.out[:, :, G:]) and torch.equal(r.lse[:, :, G:], clean.lse[:, :, G:])


@pytest.mark.parametrize("dtype,G,bs", KERNELS)
def test_infinite_scores(dtype, G, bs):
    """An infinite score is the cap where there is one (the same as a huge score's);
    without one it weighs nothing at -inf and makes its row NaN at +inf."""
    for cap in (5.0, 0.0):
        c = Case([300, 33], S=5, H=1, G=G, D=64, bs=bs, dtype=dtype, seed=22, cap=cap)
        row = c.cache[0, 0, c.table[0, 200 // bs], 200 % bs, 0]
        row.zero_()
        got = []
        for x in (1e30, float("inf")):
            row[7] = x
            got.append(c.run())
        huge, inf = got
        nan = torch.zeros(inf.lse.shape, dtype=torch.bool, device="cuda")
        if cap == 0.0:
            nan[0] = c.q[0, :, :, 7].cuda() > 0
        assert torch.isnan(inf.lse[nan]).all() and torch.isnan(inf.out[nan].float()).all()
        assert torch.equal(inf.out[~nan], huge.out[~nan]) and torch.equal(inf.lse[~nan], huge.lse[~nan])


# kernels that leave partial results: joined by the last block (32, 64 rows), by a second kernel, the others
AT_ONCE = [dict(G=4), dict(G=8), dict(G=16), dict(G=16, shared=640), dict(G=4, bs=5), dict(G=4, dtype="f32"),
           dict(G=4, shared=640, bs=5)]


def at_once(n, *calls):
    """Every call n times, each on a stream of its own, all streams at once: its results."""
    streams = [torch.cuda.Stream() for _ in calls]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[] for _ in calls]
    for _ in range(n):
        for s, call, to in zip(streams, calls, got):
            with torch.cuda.stream(s):
                to.append(call())
    torch.cuda.synchronize()
    return got


@pytest.mark.parametrize("kw", AT_ONCE)
def test_attention_on_two_streams_at_once(kw):
    """Calls of the same sizes with other inputs, in flight together, by the
    current stream and by stream=."""
    cases = [Case([4000, 900, 1100], S=5, H=2, D=64, seed=s, **kw) for s in (40, 41)]
    args = [c.args() for c in cases]
    want = [api.verify_attention(*pos, **a) for pos, a in args]
    for c, r in zip(cases, want):
        c.check(r, rows=[0])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in args]
    calls = [lambda pos=pos, a=a: api.verify_attention(*pos, **a) for pos, a in args]
    calls += [lambda pos=pos, a=a, s=s: api.verify_attention(*pos, stream=s, **a) for (pos, a), s in zip(args, streams)]
    for results, ref in zip(at_once(25, *calls), want * 2):
        for r in results:
            assert torch.equal(r.out, ref.out) and torch.equal(r.lse, ref.lse)


@pytest.mark.parametrize("kw", AT_ONCE[1:4])
def test_graphs_beside_eager_calls(kw):
    """Two graphs captured on one stream after an eager call there, replayed on two
    others while that stream goes on."""
    cases = [Case([4000, 900, 1100], S=5, H=2, D=64, seed=s, **kw) for s in (42, 43, 44)]
    args = [c.args() for c in cases]
    want = [api.verify_attention(*pos, **a) for pos, a in args]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs = []
    for pos, a in args[:2]:
        with torch.cuda.stream(s):
            api.verify_attention(*pos, **a)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            graphs.append((g, api.verify_attention(*pos, **a)))
    torch.cuda.synchronize()
    eager = at_once(25, graphs[0][0].replay, graphs[1][0].replay,
                    lambda: api.verify_attention(*args[2][0], stream=s, **args[2][1]))[2]
    for r, ref in [(graphs[0][1], want[0]), (graphs[1][1], want[1])] + [(r, want[2]) for r in eager]:
        assert torch.equal(r.out, ref.out) and torch.equal(r.lse, ref.lse)


def test_evictions_on_two_streams_at_once():
    """The lists of moves of two batches of the same sizes."""
    lens, bs = [900, 1200, 1000, 700], 16
    batches = [evict_case(lens, 600, layers=4, D=64, bs=bs, seed=s, order="mixed") for s in (50, 51)]
    given, calls = [], []
    for table, bits, w, pos, nb in batches:
        t = [torch.from_numpy(x).cuda() for x in (table, w, pos)]
        n, cache = torch.tensor(lens, dtype=torch.int32, device="cuda"), bits.cuda().view(torch.bfloat16)

        def once(t=t, n=n, cache=cache):
            held = [cache.clone(), n.clone(), t[1].clone(), t[2].clone()]
            api.evict_kv(held[0], t[0], *held[1:], block_size=bs, budget=600, sink=4, recent=50)
            return held
        given.append(once())
        torch.cuda.synchronize()
        calls.append(once)
    for results, want in zip(at_once(25, *calls), given):
        for held in results:
            for x, y in zip(held, want):
                assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_calls_of_other_sizes_on_one_workspace():
    """A stream's calls of growing and shrinking sizes, heads and kinds share
    its workspace, and their results do not change."""
    api.clear_workspaces()
    cases = [Case([700, 40], S=3, H=2, G=2, D=64, seed=60), Case([2000, 900, 5], S=9, H=2, G=16, D=128, seed=61),
             Case([1500, 800], S=6, H=2, G=8, D=96, seed=62, shared=700), Case([333], S=2, H=1, G=3, D=200, seed=63),
             Case([900, 700, 701, 800], S=8, H=2, G=8, D=128, seed=64, shared=690), Case([2100, 60], S=5, H=2, G=4, D=256, dtype="f32", seed=65)]
    args = [c.args() for c in cases]
    for order in (range(6), range(5, -1, -1)):
        results = [(cases[i], api.verify_attention(*args[i][0], **args[i][1])) for i in order]
        for c, r in results:
            c.check(r)
    assert len({w.data_ptr() for k, w in api._WORKSPACES.items() if k[2] in api._PER_STREAM}) == 2


@pytest.mark.parametrize("dtype,bs", [("bf16", 16), ("bf16", 64), ("bf16", 5), ("f32", 16)])
@pytest.mark.parametrize("G", [2, 8, 16])
def test_a_request_without_entries_of_its_own_reads_none(G, dtype, bs):
    """Requests that end where the shared prefix does, inside a page, and one
    whose document begins past its entries: the table's id of that page is not
    read, and nothing is flagged."""
    c = Case([50, 50, 70], S=6, H=2, G=G, D=64, bs=bs, dtype=dtype, seed=19, shared=50)
    c.check(c.run())
    pos, a = c.args()
    pos[2][:2, 50 // bs] = -1
    pos[2][1, 50 // bs] = c.nb
    flags = torch.zeros(3, dtype=torch.int32, device="cuda")
    r = api.verify_attention(*pos, flags=flags, **a)
    assert flags.tolist() == [0, 0, 0]
    c.check(r)
    c = Case([50, 70], S=6, H=2, G=G, D=64, bs=bs, dtype=dtype, seed=20)
    c.first = np.array([50, 0], np.int32)
    pos, a = c.args()
    pos[2][0] = -1
    flags = torch.zeros(2, dtype=torch.int32, device="cuda")
    r = api.verify_attention(*pos, flags=flags, **a)
    assert flags.tolist() == [0, 0]
    c.check(r)
