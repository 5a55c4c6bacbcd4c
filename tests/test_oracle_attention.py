"""Pins of the attention, entry-weight and eviction oracle (CPU): hand cases,
identities and properties that a dropped term, a wrong sign or a swapped
operand breaks."""
import math

import numpy as np
import pytest
from scipy.special import logsumexp, softmax

import oracle as O


def rnd(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape)


def test_two_keys_by_hand():
    # scores ln 3 and 0 (one query head of size 1): weights 3/4 and 1/4
    q = np.array([[[1.0]]])
    k = np.array([[[math.log(3.0)]], [[0.0]]])
    v = np.array([[[8.0]], [[4.0]]])
    a = O.attend(q, k, v, [1], [0, 1], np.zeros((1, 2), bool), scale=1.0)
    assert a.out[0, 0, 0] == pytest.approx(7.0) and a.lse[0, 0] == pytest.approx(math.log(4.0))
    # a bias of ln 3 per unit of distance takes the farther key's advantage
    a = O.attend(q, k, v, [1], [0, 1], np.zeros((1, 2), bool), scale=1.0, slopes=[math.log(3.0)])
    assert a.out[0, 0, 0] == pytest.approx(6.0)
    # a cap of c turns ln 3 into c tanh(ln 3 / c)
    a = O.attend(q, k, v, [1], [0, 1], np.zeros((1, 2), bool), scale=1.0, softcap=0.5)
    assert a.lse[0, 0] == pytest.approx(math.log(1 + math.exp(0.5 * math.tanh(2 * math.log(3.0)))))
    # nothing visible
    a = O.attend(q, k, v, [1], [0, 1], np.ones((1, 2), bool), scale=1.0)
    assert a.out[0, 0, 0] == 0 and a.lse[0, 0] == -np.inf


def test_grouped_heads_agree_with_scipy():
    q, k, v = rnd(0, 3, 6, 8), rnd(1, 11, 2, 8), rnd(2, 11, 2, 8)
    off = O.hidden(range(11, 14), range(11), window=9)
    assert off.sum() == 3 + 4 + 5 and not off[:, 5:].any()
    a = O.attend(q, k, v, range(11, 14), range(11), off, scale=0.3)
    for h in range(6):
        for i in range(3):
            x = np.where(off[i], -np.inf, 0.3 * k[:, h // 3] @ q[i, h])
            assert np.allclose(a.out[i, h], softmax(x) @ v[:, h // 3], atol=1e-12)
            assert a.lse[i, h] == pytest.approx(logsumexp(x))


def test_masks_by_position_and_tree():
    assert O.hidden([5], range(6), first_pos=2).tolist() == [[True, True, False, False, False, False]]
    assert O.hidden([5], [9, 0, 4, 3], window=2).tolist() == [[False, True, False, True]]
    assert (~O.candidate_mask(3)).tolist() == [[1, 0, 0], [1, 1, 0], [1, 1, 1]]
    # Table 10-17's shape: a root, two children, a child of the second
    words = [[1], [0b11], [0b101], [0b1101]]
    assert (~O.candidate_mask(4, words)).astype(int).tolist() == [[1, 0, 0, 0], [1, 1, 0, 0], [1, 0, 1, 0], [1, 0, 1, 1]]
    assert not O.candidate_mask(40, [[0, 1 << 7]] * 40)[0, 39] and O.candidate_mask(40, [[0, 1 << 7]] * 40)[0, 7]


def test_entry_weights_are_the_softmax_columns():
    """All candidates of a chain committed: every entry gains its column of
    the attention's weights, n * Hq in all."""
    S, Hq, n = 4, 4, 4
    q, k, v = rnd(3, S, Hq, 8), rnd(4, 13, 2, 8), rnd(5, 13, 2, 8)
    qp, kp = np.arange(9, 13), np.arange(13)
    off = np.concatenate([np.zeros((S, 9), bool), O.candidate_mask(S)], 1)
    kw = dict(scale=0.4, softcap=3.0, slopes=[0.1, 0.2, 0.3, 0.4])
    a = O.attend(q, k, v, qp, kp, off, **kw)
    g = O.entry_weights(q, a.lse, k, qp, kp, n, **kw)
    assert np.allclose(g, a.p.sum((0, 1)), atol=1e-12) and g.sum() == pytest.approx(n * Hq)
    # a rejected candidate leaves nothing and is no key
    keep = [0, 1, 3]
    seen = off.copy()
    seen[3, 9 + 2] = True          # node 3 hangs off node 1: node 2 is no ancestor
    a = O.attend(q, k, v, qp, kp, seen, **kw)
    kk = np.delete(k, 9 + 2, 0)
    g = O.entry_weights(q[keep], a.lse[keep], kk, qp[keep], np.delete(kp, 11), 3, **kw)
    assert g.sum() == pytest.approx(3 * Hq)
    assert np.allclose(g, np.delete(a.p[:, keep].sum((0, 1)), 11), atol=1e-12)


def test_eviction_by_hand():
    w = [9, 1, 5, 5, 2, 7, 0, 3]
    e = O.evict(w, range(8), 8, budget=5, sink=1, recent=2)
    # kept: 0 (sink), 6 and 7 (newest), then 5 (7.0), then 2 (5.0, before 3)
    assert e.kept == [0, 2, 5, 6, 7] and e.moves == [(5, 1), (6, 3), (7, 4)] and e.length == 5
    assert O.evict(w, range(8), 8, budget=8).moves == []
    assert O.evict([1, math.nan, 2], range(3), 3, budget=2) is None
    assert O.evict([1, 1, 2], [0, -1, 2], 3, budget=2) is None
    assert O.evict([1, 1, 2], [4, 4, 4], 3, budget=2, recent=1) is None


@pytest.mark.parametrize("seed", range(20))
def test_eviction_properties(seed):
    rng = np.random.default_rng(seed)
    n = int(rng.integers(2, 60))
    w = rng.integers(0, 8, n).astype(float)               # many ties
    pos = rng.permutation(3 * n)[:n]
    budget = int(rng.integers(1, n + 2))
    sink, recent = int(rng.integers(0, budget // 2 + 1)), int(rng.integers(0, budget // 2 + 1))
    e = O.evict(w, pos, n, budget=budget, sink=sink, recent=recent)
    assert len(e.kept) == min(n, budget) == e.length
    if n <= budget:
        return
    out = [c for c in range(n) if c not in e.kept]
    safe = {c for c in range(n) if pos[c] < sink or pos[c] > pos.max() - recent}
    assert safe <= set(e.kept)
    free = [c for c in e.kept if c not in safe]
    # no entry left out is heavier, or as heavy and earlier, than one kept for its weight
    assert all(w[o] < w[c] or (w[o] == w[c] and o > c) for o in out for c in free)
    # after the moves entries 0..budget-1 hold exactly the kept ones, each once
    held = {c: c for c in e.kept if c < budget}
    for a, b in e.moves:
        assert a >= budget > b and b not in held
        held[b] = a
    assert sorted(held) == list(range(budget)) and sorted(held.values()) == e.kept
