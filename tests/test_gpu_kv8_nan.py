"""The 8-bit cache's attention: a V row that stands for NaN shows in the rows that see
it and in no others, whatever its weight, on every kernel and however keys are split."""
import pytest
import torch

from test_gpu_kv8_weights import Sharp

pytestmark = pytest.mark.gpu

# one half, two halves, more row tiles; pages of boxes, of fours, of any size; the CUDA cores
KERNELS = [("bf16", 2, 16, 64), ("bf16", 8, 16, 64), ("bf16", 16, 16, 128), ("bf16", 2, 5, 64), ("bf16", 4, 12, 64),
           ("f32", 2, 16, 64), ("f32", 8, 16, 128), ("bf16", 2, 16, 160), ("bf16", 8, 16, 256)]


def spoil(c, which, e, what):
    """Entry e of request `which` (None: of the shared prefix), cached head 0."""
    blk, off = (c.stable if which is None else c.table[which])[e // c.bs], e % c.bs
    if what == "code":
        c.codes[0, 1, blk, off, 0, 5] = 0xff
    else:
        c.scales[0, 1, blk, 0, off] = 255


def check(c, clean, hit, what):
    """`hit`: rows [B, S, Hq] that see the NaN."""
    r = c.run()
    assert torch.isnan(r.out[hit][:, 5] if what == "code" else r.out[hit]).all()
    assert torch.equal(r.out[~hit], clean.out[~hit]) and torch.equal(r.lse, clean.lse)


@pytest.mark.parametrize("what", ["code", "scale"])
@pytest.mark.parametrize("dtype,G,bs,D", KERNELS)
def test_a_nan_v_of_no_weight_shows(dtype, G, bs, D, what):
    """An entry whose score is 300 below the others', in a tile that every row sees
    whole, in one that masks keys too, in a block of its own kind (2,600 entries)."""
    for n, first in ((300, 0), (300, 3), (2600, 0), (2600, 3)):
        c = Sharp([n, 40], lambda e, m: -300.0 if e < 140 and m == n else 0.0, lambda e, m: 1.0, S=3, H=2, G=G, bs=bs, D=D,
                  dtype=dtype, seed=n, docs=0.0)
        c.first[0] = first
        clean = c.run()
        assert torch.isfinite(clean.out).all()
        spoil(c, 0, 5, what)
        hit = torch.zeros(clean.lse.shape, dtype=torch.bool, device="cuda")
        hit[0, :, :G] = True
        check(c, clean, hit, what)


@pytest.mark.parametrize("what", ["code", "scale"])
@pytest.mark.parametrize("dtype,G,bs,D", KERNELS)
def test_a_nan_v_of_no_weight_shows_in_the_rows_that_see_it_alone(dtype, G, bs, D, what):
    """Such an entry outside some rows' windows."""
    c = Sharp([300], lambda e, m: -300.0 if e < 140 else 0.0, lambda e, m: 1.0, S=5, H=2, G=G, bs=bs, D=D, dtype=dtype, seed=1,
              window=200)
    clean = c.run()
    e = 300 + 2 - 200 + 1                                # the first that candidate 2 sees, hidden from 3 and 4
    spoil(c, 0, e, what)
    hit = torch.zeros(clean.lse.shape, dtype=torch.bool, device="cuda")
    hit[0, :3, :G] = True
    check(c, clean, hit, what)


@pytest.mark.parametrize("what", ["code", "scale"])
@pytest.mark.parametrize("heavy", ["own", "shared"])
@pytest.mark.parametrize("dtype,G,bs,D", KERNELS)
def test_a_nan_v_of_no_weight_shows_beside_a_shared_prefix(dtype, G, bs, D, heavy, what):
    """In the part, the prefix or a request's own keys, that the other one leaves no weight."""
    P = 400
    c = Sharp([P + 30, P + 200], lambda e, m: 0.0 if (e >= P) == (heavy == "own") else -300.0, lambda e, m: 1.0, S=3, H=2, G=G,
              bs=bs, D=D, dtype=dtype, seed=2, shared=P)
    clean = c.run()
    hit = torch.zeros(clean.lse.shape, dtype=torch.bool, device="cuda")
    if heavy == "own":
        spoil(c, None, 17, what)
        hit[:, :, :G] = True
    else:
        spoil(c, 1, P + 9, what)
        hit[1, :, :G] = True
    check(c, clean, hit, what)
