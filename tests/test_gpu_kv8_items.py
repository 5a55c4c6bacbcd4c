"""The attention over the 8-bit cache where an item's keys lie in many blocks, and
where its tiles' notes, copies and partial results go round their buffers often."""
import pytest
import torch

from speculative_decoding_verification_37_gb300 import _lib as L
from test_gpu_kv8 import Case8

pytestmark = pytest.mark.gpu


# tiles of 128 keys, at most one a part: 9, 16, 17 and 33 parts an item
@pytest.mark.parametrize("n", [1100, 2040, 2100, 4190])
@pytest.mark.parametrize("G,bs", [(2, 16), (8, 16), (2, 5), (8, 12)])
def test_items_of_many_parts(n, G, bs):
    """A small batch's items split over more parts than are joined at a time (8): the
    oracle's results, and the same bits every time."""
    c = Case8([n], S=4, H=2, G=G, D=128, bs=bs, seed=n)
    want = c.run()
    c.check(want)
    for _ in range(10):
        r = c.run()
        assert torch.equal(r.out, want.out) and torch.equal(r.lse, want.lse)


@pytest.mark.parametrize("G,bs", [(2, 16), (8, 16), (8, 5)])
def test_a_shared_prefix_of_many_parts(G, bs):
    c = Case8([2311, 2304, 2400], S=2, H=1, G=G, D=64, bs=bs, seed=3, shared=2304)
    want = c.run()
    c.check(want)
    for _ in range(10):
        r = c.run()
        assert torch.equal(r.out, want.out) and torch.equal(r.lse, want.lse)


@pytest.mark.parametrize("bs", [5, 12])
@pytest.mark.parametrize("G", [2, 8])
def test_notes_of_tiles_copied_row_by_row(G, bs):
    """Pages that no box takes, many short items a block: every tile has exponents,
    bad blocks and a first mark of its own, in turns of a few buffers."""
    lens = [1 + (37 * i) % 260 for i in range(150)]
    c = Case8(lens, S=4, H=8, G=G, D=64, bs=bs, seed=31, spread=6.0)
    want = c.run()
    c.check(want, rows=range(0, 150, 7))
    for _ in range(5):
        r = c.run()
        assert torch.equal(r.out, want.out) and torch.equal(r.lse, want.lse)
    # the same requests without their bad blocks' entries
    for b in range(0, 150, 3):
        c.table[b, 0] = c.nb
    ws = L.new_workspace(L.SPEC_WS_ATTENTION, 150, 4 * 8 * G, 64)    # (its status word stays set)
    r = c.run(ws=ws)
    assert L.spec_get_status(ws) == L.SPEC_FLAG_BAD_INPUT
    alone = [b for b in range(150) if b % 3]
    assert torch.equal(r.out[alone], want.out[alone]) and torch.equal(r.lse[alone], want.lse[alone])
    few = [b for b in range(0, 150, 3) if c.lens[b] > bs]
    assert torch.isfinite(r.out).all() and not torch.equal(r.out[few], want.out[few])
