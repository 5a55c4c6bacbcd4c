"""The CUDA-core kernel of the 8-bit cache's attention for bf16 queries: heads above
128, and caches with more entries than the tensor kernels' row numbers reach.

Its arithmetic is f32, so a weight is not rounded: |out - ref| is within (2E + (n + 16)
2^-24) sum p|v| and half a step of bf16, 2^-8 |ref|, with E of test_gpu_attention.py."""
import numpy as np
import pytest
import torch

import oracle as O
from speculative_decoding_verification_37_gb300 import api
from test_gpu_attention import Case
from test_gpu_kv8 import Case8, i32, quantised

pytestmark = pytest.mark.gpu

WIDE = [(2, 160, 16), (8, 256, 16), (4, 192, 5)]           # 16 and 32 queries a block, odd pages


class Wide(Case8):
    """Without the terms that only the tensor kernels' roundings add."""

    def score_error(self, b, k):
        return Case.score_error(self, b, k)

    def check(self, r, rows=None):
        for b in range(self.B) if rows is None else rows:
            ref, k, _ = Case.oracle(self, b)
            e, n = self.score_error(b, k), len(k) + self.shared
            out, lse = r.out[b].double().cpu().numpy(), r.lse[b].double().cpu().numpy()
            tol = (2 * e + (n + 16) * 2.0 ** -24) * ref.mass + 2.0 ** -8 * np.abs(ref.out)
            assert (np.abs(out - ref.out) <= tol + 1e-30).all(), (b, np.abs(out - ref.out).max())
            seen = np.isfinite(ref.lse)
            assert np.array_equal(np.isneginf(lse), ~seen) and not out[~seen].any()
            far = np.abs(lse[seen] - ref.lse[seen])
            assert (far <= e + (n + 16) * 2.0 ** -24 + 2.0 ** -22 * np.abs(ref.lse[seen])).all()


@pytest.mark.parametrize("kw", [dict(), dict(cap=5.0), dict(slopes=True, window=40), dict(tree=True, docs=0.5, gaps=True),
                                dict(spread=30.0, cap=3.0), dict(shared=130), dict(lens=[3000], S=2)])
@pytest.mark.parametrize("G,D,bs", WIDE)
def test_scores_and_masks(G, D, bs, kw):
    kw = dict(kw)
    lens = kw.pop("lens", [200, 131, 700] if "shared" not in kw else [130, 145, 300])
    args = dict(dict(S=6), **kw)
    c = Wide(lens, H=2, G=G, D=D, bs=bs, seed=3, **args)
    c.check(c.run())


@pytest.mark.parametrize("G,D,bs", WIDE)
def test_masked_places_may_hold_anything(G, D, bs):
    """NaN codes and exponents of 255 and 254 before the document, in another branch
    and past the candidates do not show."""
    kw = dict(S=6, H=2, G=G, D=D, bs=bs, tree=True, docs=0.5, seed=9, spare=30)
    c = Wide([70, 300], **kw)
    clean = c.run()
    c.check(clean)
    for code, scale in ((0x7f, None), (None, 255), (0xff, 254), (None, 254)):
        dirty = Wide([70, 300], **kw)
        for b, n in enumerate(c.lens):
            for e in list(range(int(c.first[b]))) + [n + 5] + list(range(n + 6, n + 30)):  # node 5: nobody's ancestor
                blk, off = c.table[b, e // bs], e % bs
                if code is not None:
                    dirty.codes[0, :, blk, off] = code
                if scale is not None:
                    dirty.scales[0, :, blk, :, off] = scale
        r = dirty.run()
        assert torch.equal(r.out[:, :5], clean.out[:, :5]) and torch.equal(r.lse[:, :5], clean.lse[:, :5])


@pytest.mark.parametrize("G,D,bs", WIDE)
def test_queries_that_are_not_finite(G, D, bs):
    c = Wide([40, 400], S=3, H=2, G=G, D=D, bs=bs, seed=1)
    clean = c.run()
    hit = torch.zeros(clean.lse.shape, dtype=torch.bool)
    hit[0, 1, 0] = hit[1, 2, 1] = True
    for x in (float("nan"), float("inf"), -float("inf")):
        c.q[0, 1, 0, 3], c.q[1, 2, 1, D - 1] = x, x
        r = c.run()
        assert not torch.isfinite(r.out[hit]).any()
        assert torch.equal(r.out[~hit], clean.out[~hit]) and torch.equal(r.lse[~hit], clean.lse[~hit])


@pytest.mark.parametrize("G,D,bs", WIDE)
def test_rows_that_see_nothing(G, D, bs):
    c = Wide([50, 0, 20], S=3, H=2, G=G, D=D, bs=bs, tree=True, seed=2)
    c.mask[:, 1] = 0                                     # candidate 1 sees no candidate
    c.first = np.array([49, 0, 99], np.int32)            # request 2: the document starts past everything
    r = c.run()
    c.check(r)
    assert torch.isneginf(r.lse[1, 1]).all() and torch.isneginf(r.lse[2]).all()


@pytest.mark.parametrize("G,D,bs", WIDE)
def test_scales_and_growing_maxima(G, D, bs):
    for scale, size, shift in ((-0.2, 1.0, 0), (0.0, 1.0, 0), (2.0 ** -63, 2.0 ** 60, 0), (2.0 ** -43, 1.0, 40), (0.1, 0.0, 0)):
        c = Wide([70, 300], S=4, H=2, G=G, D=D, bs=bs, seed=15)
        c.score["scale"] = scale
        c.q = (c.q.float() * size).to(c.q.dtype)
        c.scales = (c.scales.astype(np.int64) + shift).astype(np.uint8)
        c.stands_for()
        c.check(c.run())
    c = Wide([900], S=4, H=1, G=G, D=D, bs=bs, seed=16)
    u = torch.nn.functional.normalize(torch.randn(D, generator=torch.Generator().manual_seed(0)), dim=0)
    c.q[0] = (u * 40).to(c.q.dtype)
    x = c.cache.clone()
    for e in range(900):
        x[0, 0, c.table[0, e // bs], e % bs, 0] = u.double() * e / 50
    c.codes, c.scales = quantised(x.numpy())
    c.stands_for()
    c.check(c.run())


def test_more_entries_than_row_numbers():
    """2^30 entries a layer (37 GB): bf16 heads up to 128 go to the CUDA cores there; both
    of the kernel's forms, written, read by the attention and read back at both ends."""
    H, D, bs, nb, n, S = 1, 16, 64, 1 << 24, 130, 4
    cache = api.QuantKV(torch.empty((1, 2, nb, bs, H, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),
                        torch.empty((1, 2, nb, H, bs), dtype=torch.uint8, device="cuda"))
    g = torch.Generator().manual_seed(0)
    x = torch.randn((2, 1, n + S, H, D), generator=g).bfloat16()
    k, v = (O.kv8_values(*O.kv8_quantise(x[i, 0].double().numpy())) for i in (0, 1))
    off = np.zeros((S, n + S), bool)
    off[:, n:] = O.candidate_mask(S)
    for ids in ([[nb - 1, nb - 7, nb - 3]], [[0, nb - 1, 1]]):
        table = i32(ids)
        api.write_kv_q8(x[0].cuda(), x[1].cuda(), cache, table, i32([0]), block_size=bs)
        for G in (2, 8):
            q = torch.randn((1, S, H * G, D), generator=g).bfloat16()
            r = api.verify_attention_q8(q.cuda(), cache, table, i32([n]), block_size=bs)
            ref = O.attend(q[0].double().numpy(), k, v, np.arange(n, n + S), np.arange(n + S), off, scale=D ** -0.5)
            dots = np.abs(q[0].double().numpy()).reshape(-1, D) @ np.abs(k[:, 0]).T
            e = 2.0 ** -24 * (D + 4) * D ** -0.5 * dots.max()
            tol = (2 * e + (n + S + 16) * 2.0 ** -24) * ref.mass + 2.0 ** -8 * np.abs(ref.out)
            assert (np.abs(r.out[0].double().cpu().numpy() - ref.out) <= tol).all()
            assert (np.abs(r.lse[0].double().cpu().numpy() - ref.lse) <= e + (n + S + 16) * 2.0 ** -24 + 2.0 ** -22 * np.abs(ref.lse)).all()
        back = api.read_kv_q8(cache, table, n_max=n + S, block_size=bs, dtype=torch.float32)
        assert np.array_equal(back.k[0].double().cpu().numpy(), k) and np.array_equal(back.v[0].double().cpu().numpy(), v)
    del cache
    torch.cuda.empty_cache()
