"""GPU parity of the 8-bit paged cache with the float64 oracle: writing, reading
back and committing bit for bit, the attention within a derived tolerance.

Tolerance of the attention.  As in test_gpu_attention.py, with the values that
the codes stand for as K and V (powers of two and codes enter exactly), and one
term more: the tensor kernels take a query as the sum of two e4m3 numbers after
scaling its largest element into (224, 448].  The second number's steps are 2^-9
at least, half of that over 224 is 2^-17.8 of the largest element; what its first
three bits leave of a bf16 value is otherwise exact.  So a score's error grows by
at most |scale| 2^-17 max|q| sum|k|.  The weights, times V's powers of two, are
rounded to f16 (2^-11 of each) and held as three e5m2 numbers: each of the first two
takes at least 3 of the 11 bits, the third is rounded to 3 (2^-9 of the weight at most),
together below the 2^-8 of a bf16 rounding that Case.check allows.  e5m2's steps end
at 2^-16; a weight of 1 at the row's largest power is at 2^7, so half a step is 2^-24 of
the largest power, for a key, with codes up to 448 and 448 powers at most twice the
largest |v| that the row sees, over a sum of weights that is at least 1."""
import math

import numpy as np
import pytest
import torch

import oracle as O
from speculative_decoding_verification_37_gb300 import _lib as L
from speculative_decoding_verification_37_gb300 import api
from test_gpu_attention import Case

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()  # noqa: E731


def quantised(x):
    """(codes, scale) arrays of a plain cache [..., bs, H, D], in the 8-bit cache's layout."""
    codes, scale = O.kv8_quantise(x)
    return codes, np.ascontiguousarray(np.swapaxes(scale, -1, -2))


def on_gpu(codes, scale):
    return api.QuantKV(torch.from_numpy(codes).view(torch.float8_e4m3fn).cuda(), torch.from_numpy(scale).cuda())


def off_gpu(cache):
    return cache.codes.view(torch.uint8).cpu().numpy(), cache.scale.cpu().numpy()


def random_cache(rng, L_, nb, bs, H, D):
    """Any bytes, NaN codes and all exponents among them."""
    return (rng.integers(0, 256, (L_, 2, nb, bs, H, D)).astype(np.uint8),
            rng.integers(0, 256, (L_, 2, nb, H, bs)).astype(np.uint8))


def tables(rng, lens, bs, spare=0):
    need = [-(-max(n, 1) // bs) for n in lens]
    mb, nb = max(need), sum(need) + spare
    perm, table, at = rng.permutation(nb), np.zeros((len(lens), max(need)), np.int32), 0
    for b, k in enumerate(need):
        table[b, :k] = perm[at:at + k]
        at += k
    return table, nb, mb


# ---------------------------------------------------------------------------
# writing
# ---------------------------------------------------------------------------
def special_rows(x):
    """Rows where rounding and exponents turn: zeros, borders, halfway points, ranges' ends."""
    D = x.shape[-1]
    flat = x.view(-1, D)
    rows = [torch.zeros(D), -torch.zeros(D), torch.full((D,), 448.0), torch.full((D,), 449.0), torch.full((D,), 450.0),
            torch.full((D,), 224.0), torch.full((D,), 1e30), torch.full((D,), -3e38), torch.full((D,), 1e-37),
            torch.full((D,), 1e-39), torch.full((D,), 2.0 ** -133),
            torch.tensor([float("nan")] + [1.0] * (D - 1)), torch.tensor([1.0] * (D - 1) + [float("inf")]),
            torch.tensor([float("-inf")] * D), torch.tensor([448.0] + [(8 + i % 8 + 0.5) * 2.0 ** (i % 13 - 10) for i in range(D - 1)]),
            torch.tensor([1e6] + [1e-6] * (D - 1))]
    for i, r in enumerate(rows[:len(flat)]):
        flat[(i * 7) % len(flat) if len(flat) % 7 else i] = r.to(x.dtype)
    return x


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kw", [
    dict(B=1, S=1, H=1, D=16, bs=1), dict(B=3, S=5, H=2, D=128), dict(B=2, S=40, H=3, D=64, bs=5, L=2),
    dict(B=2, S=17, H=40, D=32, bs=8), dict(B=4, S=33, H=1, D=80, bs=48, packed=True), dict(B=2, S=16, H=2, D=256, bs=16),
    dict(B=1, S=70, H=65, D=16, bs=3), dict(B=2, S=20, H=8, D=128, bs=64, packed=True, L=3), dict(B=2, S=31, H=4, D=160),
    dict(B=2, S=9, H=5, D=112, bs=7)])
def test_write(kw, dtype):
    kw = dict(dict(bs=16, L=1, packed=False), **kw)
    B, S, H, D, bs, Ly = (kw[k] for k in ("B", "S", "H", "D", "bs", "L"))
    rng, g = np.random.default_rng(S), torch.Generator().manual_seed(S)
    lens = [int(rng.integers(0, 40)) for _ in range(B)]
    new = [S] + [int(rng.integers(0, S + 1)) for _ in range(B - 2)] + ([0] if B > 1 else [])
    table, nb, _ = tables(rng, [n + S for n in lens], bs, spare=2)
    if kw["packed"]:
        qkv = (torch.randn((B, S, 3, H, D), generator=g) * 3).to(DT[dtype])
        k, v = special_rows(qkv[:, :, 1].contiguous()), qkv[:, :, 2].contiguous()
        qkv[:, :, 1], qkv[:, :, 2] = k, v
        dev = qkv.cuda()
        dk, dv = dev[:, :, 1], dev[:, :, 2]
    else:
        k, v = (special_rows((torch.randn((B, S, H, D), generator=g) * 3).to(DT[dtype])) for _ in range(2))
        dk, dv = k.cuda(), v.cuda()
    codes, scale = random_cache(rng, Ly, nb, bs, H, D)
    cache, flags = on_gpu(codes, scale), torch.zeros(B, dtype=torch.int32, device="cuda")
    for ragged in (True, False):
        count = new if ragged else [S] * B
        api.write_kv_q8(dk, dv, cache, i32(table), i32(lens), block_size=bs, layer=Ly - 1,
                        n_new=i32(count) if ragged else None, flags=flags)
        torch.cuda.synchronize()
        for b in range(B):
            for i, x in enumerate((k, v)):
                c, s = O.kv8_quantise(x[b, :count[b]].double().numpy())
                for e in range(count[b]):
                    blk, off = table[b, (lens[b] + e) // bs], (lens[b] + e) % bs
                    codes[Ly - 1, i, blk, off], scale[Ly - 1, i, blk, :, off] = c[e], s[e]
        got = off_gpu(cache)
        # (a zero's sign is the input's in both)
        assert np.array_equal(got[1], scale) and np.array_equal(got[0], codes)
    assert not flags.any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kw", [dict(B=80, S=70, H=1, D=128, bs=16), dict(B=160, S=3, H=3, D=64, bs=8),
                                dict(B=9, S=1100, H=2, D=16, bs=48), dict(B=3, S=3300, H=1, D=144, bs=1)])
def test_many_entries_written_and_read_back(kw, dtype):
    """Enough blocks for the wide ones; the same numbers as in one request after the other."""
    B, S, H, D, bs = (kw[k] for k in ("B", "S", "H", "D", "bs"))
    rng, g = np.random.default_rng(S), torch.Generator().manual_seed(S)
    k, v = (special_rows((torch.randn((B, S, H, D), generator=g) * 3).to(DT[dtype])) for _ in range(2))
    lens = rng.integers(0, 20, B).tolist()
    count = [S, 0, 1] + rng.integers(0, S + 1, B - 3).tolist()
    table, nb, _ = tables(rng, [n + S for n in lens], bs)
    codes, scale = random_cache(rng, 1, nb, bs, H, D)
    cache = on_gpu(codes, scale)
    api.write_kv_q8(k.cuda(), v.cuda(), cache, i32(table), i32(lens), block_size=bs, n_new=i32(count))
    r = api.read_kv_q8(cache, i32(table), i32(lens), i32(count), n_max=S, block_size=bs, dtype=torch.float32)
    for i, (x, back) in enumerate(((k, r.k), (v, r.v))):
        for b in range(B):
            c, s = O.kv8_quantise(x[b, :count[b]].double().numpy())
            at = lens[b] + np.arange(count[b])
            blk, off = table[b, at // bs], at % bs
            codes[0, i, blk, off], scale[0, i, blk, :, off] = c, s
            want = torch.from_numpy(np.concatenate([O.kv8_values(c, s), np.zeros((S - count[b], H, D))])).float()
            assert torch.equal(back[b].cpu().nan_to_num(nan=7.0, posinf=8.0, neginf=9.0), want.nan_to_num(nan=7.0, posinf=8.0, neginf=9.0))
    got = off_gpu(cache)
    assert np.array_equal(got[1], scale) and np.array_equal(got[0], codes)


def test_write_bad_requests():
    rng = np.random.default_rng(0)
    codes, scale = random_cache(rng, 1, 6, 4, 2, 64)
    cache, x = on_gpu(codes, scale), torch.randn((5, 3, 2, 64), device="cuda")
    table = i32([[0, 1], [2, 3], [4, 6], [-1, 5], [0, 1]])
    flags, ws = torch.zeros(5, dtype=torch.int32, device="cuda"), L.new_workspace(L.SPEC_WS_KV8, 5, 0, 0)
    #            negative, past the table, a bad block in part, a bad block, too many
    api.write_kv_q8(x, x, cache, table, i32([-1, 6, 2, 0, 0]), block_size=4, n_new=i32([3, 3, 3, 3, 4]), flags=flags, ws=ws)
    torch.cuda.synchronize()
    assert flags.tolist() == [L.SPEC_FLAG_BAD_INPUT] * 5 and L.spec_get_status(ws) == L.SPEC_FLAG_BAD_INPUT
    c, s = O.kv8_quantise(x[2].double().cpu().numpy())
    for i in (0, 1):
        for e in (0, 1):
            codes[0, i, 4, 2 + e], scale[0, i, 4, :, 2 + e] = c[e], s[e]
    got = off_gpu(cache)
    assert np.array_equal(got[0], codes) and np.array_equal(got[1], scale)
    assert not ws.any()


# ---------------------------------------------------------------------------
# reading back
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kw", [
    dict(B=1, n=1, H=1, D=16, bs=1), dict(B=3, n=40, H=2, D=128, bs=16), dict(B=2, n=37, H=3, D=64, bs=5, L=2),
    dict(B=2, n=18, H=40, D=32, bs=8), dict(B=5, n=33, H=1, D=80, bs=48), dict(B=2, n=16, H=2, D=256, bs=16),
    dict(B=2, n=50, H=65, D=16, bs=3)])
def test_read(kw, dtype):
    kw = dict(dict(L=1), **kw)
    B, n, H, D, bs, Ly = (kw[k] for k in ("B", "n", "H", "D", "bs", "L"))
    rng = np.random.default_rng(n)
    start = [int(rng.integers(0, 30)) for _ in range(B)]
    count = [n] + [int(rng.integers(0, n + 1)) for _ in range(B - 2)] + ([0] if B > 1 else [])
    table, nb, _ = tables(rng, [s + n for s in start], bs)
    codes, scale = random_cache(rng, Ly, nb, bs, H, D)
    cache = on_gpu(codes, scale)
    for ragged in (True, False):
        got = api.read_kv_q8(cache, i32(table), i32(start) if ragged else None, i32(count) if ragged else None, n_max=n,
                             block_size=bs, layer=Ly - 1, dtype=DT[dtype])
        for i, x in enumerate((got.k, got.v)):
            want = np.zeros((B, n, H, D))
            for b in range(B):
                for e in range(count[b] if ragged else n):
                    at = (start[b] if ragged else 0) + e
                    blk, off = table[b, at // bs], at % bs
                    want[b, e] = O.kv8_values(codes[Ly - 1, i, blk, off], scale[Ly - 1, i, blk, :, off])
            want = torch.from_numpy(want).float().to(DT[dtype])   # 448 * 2^127 is infinite in float32
            assert x.dtype == DT[dtype] and torch.equal(torch.isnan(x).cpu(), torch.isnan(want))
            assert torch.equal(x.cpu().nan_to_num(nan=7.0), want.nan_to_num(nan=7.0))


def test_read_bad_requests():
    rng = np.random.default_rng(1)
    codes, scale = random_cache(rng, 1, 6, 4, 2, 64)
    scale[:] = 127
    codes[codes & 127 == 127] = 0
    flags, ws = torch.zeros(5, dtype=torch.int32, device="cuda"), L.new_workspace(L.SPEC_WS_KV8, 5, 0, 0)
    table = np.array([[0, 1], [2, 3], [4, 6], [3, 5], [0, 1]])
    r = api.read_kv_q8(on_gpu(codes, scale), i32(table), i32([-1, 6, 2, 0, 0]), i32([3, 3, 3, 3, -1]), n_max=3, block_size=4,
                       dtype=torch.float32, flags=flags, ws=ws)
    torch.cuda.synchronize()
    bad = L.SPEC_FLAG_BAD_INPUT
    assert flags.tolist() == [bad, bad, bad, 0, bad] and L.spec_get_status(ws) == bad
    want = np.zeros((5, 3, 2, 64))
    want[2, :2] = O.kv8_values(codes[0, 0, 4, 2:4], np.swapaxes(scale[0, 0, 4, :, 2:4], 0, 1))
    want[3] = O.kv8_values(codes[0, 0, 3, :3], np.swapaxes(scale[0, 0, 3, :, :3], 0, 1))
    assert np.array_equal(r.k.double().cpu().numpy(), want)


def test_what_was_written_reads_back_within_half_a_step():
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((2, 50, 4, 128), generator=g, device="cuda") * torch.exp(3 * torch.randn((2, 50, 4, 1), generator=g, device="cuda"))
    cache, table = api.quant_kv(1, 8, 16, 4, 128), i32(np.arange(8).reshape(2, 4))
    api.write_kv_q8(x, -x, cache, table, i32([0, 0]), block_size=16)
    r = api.read_kv_q8(cache, table, n_max=50, block_size=16, dtype=torch.float32)
    assert torch.equal(r.v, -r.k)
    power = torch.exp2(torch.floor(torch.log2(x.abs().amax(-1, keepdim=True) / 224)))
    assert ((r.k - x).abs() <= torch.maximum(2.0 ** -4 * x.abs(), 2.0 ** -10 * 2 * power)).all()


# ---------------------------------------------------------------------------
# committing a tree's path
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("kw", [
    dict(lens=[0], S=1, H=1, D=16, bs=1), dict(lens=[5, 17, 0, 64], S=13, H=2, D=64, bs=16, L=3),
    dict(lens=[3, 9], S=40, H=3, D=80, bs=5), dict(lens=[100, 1], S=300, H=1, D=128, bs=16, L=2),
    dict(lens=[7] * 9, S=8, H=40, D=32, bs=8, L=5), dict(lens=[11, 30], S=1024, H=1, D=16, bs=64)])
def test_commit(kw):
    kw = dict(dict(L=1), **kw)
    lens, S, H, D, bs, Ly = (kw[k] for k in ("lens", "S", "H", "D", "bs", "L"))
    B, rng = len(lens), np.random.default_rng(S)
    table, nb, _ = tables(rng, [n + S for n in lens], bs)
    codes, scale = random_cache(rng, Ly, nb, bs, H, D)
    cache, cl = on_gpu(codes, scale), i32(lens)
    n = [min(S, int(rng.integers(0, S + 1)) if b else S // 2 + 1) for b in range(B)]
    path = [sorted(rng.choice(S, n[b], replace=False).tolist()) for b in range(B)]
    slots = np.full((B, S + 3), -1)
    for b in range(B):
        slots[b, :n[b]] = path[b]
    blocks, flags = torch.full((B,), -1, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    api.commit_kv_q8(cache, i32(table), i32(slots), i32(n), cl, block_size=bs, S=S, blocks_in_use=blocks, flags=flags)
    want = [O.kv8_commit(codes, scale, table[b], bs, lens[b], path[b], S) for b in range(B)]
    got = off_gpu(cache)
    assert np.array_equal(got[0], codes) and np.array_equal(got[1], scale) and not flags.any()
    assert cl.tolist() == want and blocks.tolist() == [-(-x // bs) for x in want]
    # the first n stay where they are
    api.commit_kv_q8(cache, i32(table), None, i32([0] * B), cl, block_size=bs, S=S)
    assert cl.tolist() == want and np.array_equal(off_gpu(cache)[0], codes)


def test_commit_bad_requests_stay_as_they_are():
    rng = np.random.default_rng(4)
    lens = [6, 6, 6, 6, -1, 14, 12, 6, 6]
    slots = np.array([[0, 2, 3], [0, 0, 3], [2, 1, 3], [0, 8, 9], [0, 1, 2], [0, 1, 2], [0, 1, 7], [0, 2, 3], [0, 2, 3]])
    n = [3, 3, 3, 3, 3, 3, 3, 9, 3]
    table = rng.permutation(36).reshape(9, 4).astype(np.int32)
    table[8, 2] = 36                                     # holds candidates 2 and 3
    codes, scale = random_cache(rng, 2, 36, 4, 1, 64)
    cache, cl = on_gpu(codes, scale), i32(lens)
    blocks, flags = torch.full((9,), -1, dtype=torch.int32, device="cuda"), torch.zeros(9, dtype=torch.int32, device="cuda")
    ws = L.new_workspace(L.SPEC_WS_KV8, 9, 0, 0)
    padded = np.concatenate([slots, np.zeros((9, 5), np.int64)], 1)
    api.commit_kv_q8(cache, i32(table), i32(padded), i32(n), cl, block_size=4, blocks_in_use=blocks, flags=flags, ws=ws)
    torch.cuda.synchronize()
    assert O.kv8_commit(codes, scale, table[0], 4, 6, [0, 2, 3], 8) == 9
    for b in range(1, 9):
        assert O.kv8_commit(codes, scale, table[b], 4, lens[b], padded[b, :n[b]].tolist(), 8) is None
    bad = L.SPEC_FLAG_BAD_INPUT
    assert flags.tolist() == [0] + [bad] * 8 and L.spec_get_status(ws) == bad and not ws.any()
    assert cl.tolist() == [9] + lens[1:] and blocks.tolist() == [3] + [-1] * 8
    assert np.array_equal(off_gpu(cache)[0], codes) and np.array_equal(off_gpu(cache)[1], scale)


def test_calls_on_two_streams_and_in_graphs():
    """Two layers written, committed and read at once, eagerly and in a graph each,
    give what one call after the other gives."""
    B, S, H, D, bs = 6, 13, 4, 64, 16
    rng, g = np.random.default_rng(8), torch.Generator(device="cuda").manual_seed(8)
    lens = rng.integers(0, 60, B).tolist()
    table, nb, _ = tables(rng, [n + S for n in lens], bs)
    table, slots = i32(table), i32([[0, 2, 5] + [-1] * 10] * B)
    x = [torch.randn((2, B, S, H, D), generator=g, device="cuda") for _ in range(2)]
    caches = [api.quant_kv(2, nb, bs, H, D) for _ in range(2)]
    starts = [i32(lens) for _ in range(2)]

    def round_(i, stream=None):
        kw = dict(block_size=bs, stream=stream)
        for layer in (0, 1):
            api.write_kv_q8(x[i][0], x[i][1], caches[i], table, starts[i], layer=layer, **kw)
        api.commit_kv_q8(caches[i], table, slots, i32([3] * B) if stream is None else n3, starts[i], **kw)
        return api.read_kv_q8(caches[i], table, n_max=60, layer=1, **kw)

    n3 = i32([3] * B)
    want = []
    for i in (0, 1):
        r = round_(i)
        want.append((off_gpu(caches[i]), r.k.clone(), r.v.clone(), starts[i].tolist()))

    def reset():
        for i in (0, 1):
            caches[i].codes.view(torch.uint8).zero_()
            caches[i].scale.zero_()
            starts[i].copy_(i32(lens))

    def check(i, r):
        got = off_gpu(caches[i])
        assert np.array_equal(got[0], want[i][0][0]) and np.array_equal(got[1], want[i][0][1])
        assert torch.equal(r.k, want[i][1]) and torch.equal(r.v, want[i][2]) and starts[i].tolist() == want[i][3]

    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        reset()
        torch.cuda.synchronize()
        r = [round_(i, streams[i]) for i in (0, 1)]
        torch.cuda.synchronize()
        for i in (0, 1):
            check(i, r[i])
    graphs, held = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for i in (0, 1):
        with torch.cuda.graph(graphs[i], stream=streams[i]):
            held.append(round_(i, streams[i]))
    for _ in range(3):
        reset()
        torch.cuda.synchronize()
        for i in (0, 1):
            with torch.cuda.stream(streams[1 - i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        for i in (0, 1):
            check(i, held[i])


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
class Case8(Case):
    """A Case whose cache is an 8-bit one; `cache` holds what it stands for."""

    def __init__(self, lens, spread=0.0, **kw):
        super().__init__(lens, inplace=True, **kw)
        x = self.cache.double().numpy()
        if spread:                                       # rows of very different sizes
            rng = np.random.default_rng(7)
            x = x * 2.0 ** rng.uniform(-spread, 0, x.shape[:-1] + (1,))
        self.codes, self.scales = quantised(x)
        self.stands_for()

    def stands_for(self):
        self.cache = torch.from_numpy(O.kv8_values(self.codes, np.swapaxes(self.scales, -1, -2)))

    def planes(self):
        return self.cache[self.layer, 0].numpy(), self.cache[self.layer, 1].numpy()

    def run(self, **over):
        pos, a = self.args()
        a.pop("temp_kv")
        a.update(over)
        r = api.verify_attention_q8(pos[0], on_gpu(self.codes, self.scales), *pos[2:], **a)
        torch.cuda.synchronize()
        return r

    def score_error(self, b, k):
        e = super().score_error(b, k)
        if self.dtype == torch.bfloat16 and len(k):
            q = np.abs(self.q[b].double().numpy()).max()
            e += abs(self.score["scale"]) * 2.0 ** -17 * q * float(np.abs(k).sum(-1).max())
        return e

    def check(self, r, rows=None):
        """As Case.check, with the weights' smallest steps."""
        self.steps = 0.0
        if self.dtype == torch.bfloat16:
            v = self.planes()[1]
            self.steps = 2.0 ** -24 * 2 * float(np.nanmax(np.abs(v)))
        super().check(r, rows)

    def oracle(self, b):
        ref, k, off = super().oracle(b)
        # (Case.check's tolerance is at least 2^-8 of the mass: the steps go there)
        ref.mass = ref.mass + 2.0 ** 8 * (len(k) + self.shared) * getattr(self, "steps", 0.0)
        return ref, k, off


SHAPES = [
    dict(lens=[1], S=1, H=1, G=1, D=64),
    dict(lens=[0, 0], S=1, H=1, G=1, D=64),                            # nothing cached: the candidate alone
    dict(lens=[0, 1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 300], S=5, H=2, G=2, D=64),
    dict(lens=[100, 7], S=13, H=2, G=4, D=128, tree=True),
    dict(lens=[257, 64], S=3, H=1, G=7, D=128, bs=1),
    dict(lens=[90, 200, 13], S=2, H=3, G=1, D=80, bs=5),
    dict(lens=[500], S=8, H=4, G=8, D=128, bs=48),                     # 64 rows a head
    dict(lens=[70, 130], S=20, H=2, G=4, D=128, tree=True),            # 80 rows
    dict(lens=[40, 77], S=70, H=1, G=2, D=64, tree=True),              # 140 rows, three mask words
    dict(lens=[33, 90], S=4, H=2, G=3, D=256, bs=64),
    dict(lens=[60, 10], S=3, H=2, G=2, D=16),
    dict(lens=[129, 130], S=33, H=1, G=1, D=160),
    dict(lens=[3000], S=2, H=2, G=2, D=128),                           # keys split over blocks
    dict(lens=[3000, 20], S=1, H=2, G=8, D=128, bs=32),
    dict(lens=[300, 40], S=12, H=2, G=8, D=128, tree=True),            # 96 rows
    dict(lens=[500, 9], S=40, H=1, G=4, D=64, tree=True),              # 160 rows: two row tiles
    dict(lens=[20], S=300, H=1, G=1, D=64, tree=True),                 # a wide tree, ten mask words
    dict(lens=[131, 5], S=300, H=1, G=1, D=64, bs=8),
    dict(lens=[200, 60], S=7, H=2, G=2, D=64, bs=128), dict(lens=[90], S=4, H=1, G=2, D=128, bs=24),
    dict(lens=[77, 300], S=4, H=2, G=2, D=32), dict(lens=[77, 300], S=4, H=2, G=2, D=48), dict(lens=[77, 300], S=4, H=3, G=2, D=96),
    dict(lens=[77, 300, 1], S=5, H=3, G=4, D=80, bs=4), dict(lens=[600, 300], S=1, H=2, G=4, D=128, bs=12),
    dict(lens=[900, 5, 131], S=7, H=2, G=8, D=48, bs=20, tree=True), dict(lens=[1500, 1], S=3, H=2, G=2, D=16, bs=1),
    dict(lens=[77, 300], S=9, H=3, G=4, D=112, bs=8), dict(lens=[2000, 33], S=9, H=3, G=4, D=80),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_shapes(i, dtype):
    c = Case8(dtype=dtype, seed=i, **SHAPES[i])
    c.check(c.run())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kw", [
    dict(cap=5.0), dict(slopes=True), dict(window=40), dict(window=1), dict(docs=0.5), dict(docs=1.0),
    dict(gaps=True, window=50, slopes=True), dict(gaps=True, docs=0.7, cap=2.0),
    dict(tree=True, window=2, docs=0.99), dict(cap=30.0, slopes=True, window=100, docs=0.3, tree=True, gaps=True),
    dict(window=7), dict(tree=True, gaps=True, slopes=True), dict(layers=3, layer=2, spare=40), dict(spread=12.0),
    dict(spread=40.0, cap=3.0), dict(cap=1024.0), dict(cap=1000.0, slopes=True, gaps=True)])
def test_scores_and_masks(kw, dtype):
    for G in (3, 9, 20):                                 # 18, 54 and 120 rows
        c = Case8([5, 64, 200, 131, 0 if not kw.get("gaps") else 1, 700], S=6, H=2, G=G, D=64, dtype=dtype, seed=3, **kw)
        c.check(c.run())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kw", [
    dict(shared=64), dict(shared=50), dict(shared=1), dict(shared=600, D=128, G=4), dict(shared=130),
    dict(shared=90, tree=True, cap=4.0, slopes=True), dict(shared=200, window=60), dict(shared=200, docs=0.9),
    dict(shared=256, G=8, S=9, lens=[256] * 20),                       # nothing of one's own but the candidates
    dict(shared=77, bs=7, D=80), dict(shared=300, G=8, S=6, lens=[300, 333, 310, 301, 450, 512], window=200),
    dict(shared=700, G=4, S=9, lens=[700 + 7 * i for i in range(17)], tree=True, cap=30.0, D=128),
    dict(shared=129, G=16, S=10, lens=[129, 140], slopes=True)])
def test_shared_prefix(kw, dtype):
    kw = dict(kw)
    lens = kw.pop("lens", [kw["shared"] + n for n in (0, 1, 15, 100, 33)])
    args = dict(S=4, H=2, G=2, D=64)
    args.update(kw)
    c = Case8(lens, dtype=dtype, seed=5, **args)
    c.check(c.run())


# one half, two halves, more row tiles; pages of whole boxes, of fours, of any size; the CUDA cores
KERNELS = [("bf16", 2, 16), ("bf16", 8, 16), ("bf16", 16, 16), ("bf16", 2, 5), ("bf16", 4, 12), ("f32", 8, 16)]


@pytest.mark.parametrize("dtype,G,bs", KERNELS)
def test_masked_places_may_hold_anything(dtype, G, bs):
    """NaN codes and exponents past the length, before the document, outside the
    window and in other branches do not show; visible ones do, in their rows."""
    kw = dict(S=6, H=2, G=G, D=64, bs=bs, tree=True, docs=0.5, window=30, dtype=dtype, seed=9, spare=30)
    c = Case8([70, 100], **kw)
    clean = c.run()
    c.check(clean)
    for what in ("code", "scale", "both"):
        dirty = Case8([70, 100], **kw)
        for b, n in enumerate(c.lens):
            lo = max(int(c.first[b]), n - 29)            # the first position that candidate 0 sees
            for e in list(range(0, lo)) + [n + 5] + list(range(n + 6, c.max_blocks * c.bs)):  # node 5: nobody's ancestor
                if e // c.bs < c.max_blocks and (e < n or e // c.bs < -(-(n + 36) // c.bs)):
                    if what != "scale":
                        dirty.codes[0, :, c.table[b, e // c.bs], e % c.bs] = 0x7f
                    if what != "code":
                        dirty.scales[0, :, c.table[b, e // c.bs], :, e % c.bs] = 255
        r = dirty.run()
        assert torch.equal(r.out[:, :5], clean.out[:, :5]) and torch.equal(r.lse[:, :5], clean.lse[:, :5])
        assert torch.isnan(r.out[:, 5]).all() and torch.isnan(r.lse[:, 5]).all()


@pytest.mark.parametrize("dtype,G,bs", KERNELS)
def test_a_nan_v_shows_in_the_rows_that_see_it(dtype, G, bs):
    for what in ("code", "scale"):
        c = Case8([40, 400], S=3, H=1, G=G, D=64, bs=bs, tree=True, dtype=dtype, seed=1)
        c.mask[:, :, 0] = [1, 0b11, 0b101]
        c.pos[:] = np.array(c.lens)[:, None] + [0, 1, 1]
        clean = c.run()
        for b, n in enumerate(c.lens):
            blk, off = c.table[b, (n + 1) // bs], (n + 1) % bs           # candidate 1's entry
            if what == "code":
                c.codes[0, 1, blk, off, 0, 5] = 0xff
            else:
                c.scales[0, 1, blk, 0, off] = 255
        r = c.run()
        assert torch.equal(r.out[:, [0, 2]], clean.out[:, [0, 2]]) and torch.equal(r.lse, clean.lse)
        assert torch.isnan(r.out[:, 1, :, 5]).all()
        # an entry that everybody sees
        c.scales[0, 1, c.table[1, 200 // bs], 0, 200 % bs] = 255
        r = c.run()
        assert torch.isnan(r.out[1]).all() and torch.equal(r.lse, clean.lse) and torch.equal(r.out[0, 0], clean.out[0, 0])


@pytest.mark.parametrize("dtype,G,bs", KERNELS)
def test_hidden_rows_of_the_largest_powers(dtype, G, bs):
    """Entries whose exponent is 254, before the document and in other branches,
    change nothing for the rows that do not see them."""
    kw = dict(S=6, H=2, G=G, D=64, bs=bs, tree=True, docs=0.5, dtype=dtype, seed=9)
    clean, c = Case8([70, 300], **kw), Case8([70, 300], **kw)
    want = clean.run()
    for b, n in enumerate(c.lens):
        for e in list(range(int(c.first[b]))) + [n + 5]:
            c.scales[0, :, c.table[b, e // bs], :, e % bs] = 254
    r = c.run()
    # (scores of at most a few units rounded once more; the weights' roundings differ)
    assert (r.lse[:, :5] - want.lse[:, :5]).abs().max() <= 2.0 ** -18
    tol = 2.0 ** -7 if dtype == "bf16" else 2.0 ** -20
    assert (r.out[:, :5].float() - want.out[:, :5].float()).abs().max() <= tol * float(clean.cache[0, 1].abs().max())


@pytest.mark.parametrize("dtype,G,bs", KERNELS)
def test_queries_that_are_not_finite(dtype, G, bs):
    c = Case8([40, 400], S=3, H=2, G=G, D=64, bs=bs, dtype=dtype, seed=1)
    clean = c.run()
    c.q[0, 1, 0, 3], c.q[1, 2, 1, 60] = float("nan"), float("nan")
    r = c.run()
    hit = torch.zeros(clean.lse.shape, dtype=torch.bool)
    hit[0, 1, 0] = hit[1, 2, 1] = True
    assert torch.isnan(r.lse[hit]).all() and torch.isnan(r.out[hit]).all()
    assert torch.equal(r.out[~hit], clean.out[~hit]) and torch.equal(r.lse[~hit], clean.lse[~hit])
    if dtype == "bf16":
        c.q[0, 1, 0, 3], c.q[1, 2, 1, 60] = float("inf"), -float("inf")
        r = c.run()
        assert not torch.isfinite(r.out[hit]).any() and torch.equal(r.out[~hit], clean.out[~hit])


@pytest.mark.parametrize("dtype,G,bs", KERNELS)
def test_rows_that_see_nothing(dtype, G, bs):
    c = Case8([50, 0, 20], S=3, H=2, G=G, D=64, bs=bs, tree=True, dtype=dtype, seed=2)
    c.mask[:, 1] = 0                                     # candidate 1 sees no candidate
    c.first = np.array([49, 0, 99], np.int32)            # request 2: the document starts past everything
    r = c.run()
    c.check(r)
    assert torch.isneginf(r.lse[1, 1]).all() and torch.isneginf(r.lse[2]).all()


@pytest.mark.parametrize("dtype,G,bs", KERNELS)
def test_scales(dtype, G, bs):
    """Negative and zero scales; queries and keys of any size."""
    for scale, size, shift in ((-0.2, 1.0, 0), (0.0, 1.0, 0), (2.0 ** -63, 2.0 ** 60, 0), (2.0 ** 37, 2.0 ** -40, 0),
                               (2.0 ** -43, 1.0, 40), (2.0 ** 57, 1.0, -60), (0.1, 0.0, 0)):
        c = Case8([70, 300], S=4, H=2, G=G, D=64, bs=bs, dtype=dtype, seed=15)
        c.score["scale"] = scale
        c.q = (c.q.float() * size).to(c.q.dtype)
        c.scales = (c.scales.astype(np.int64) + shift).astype(np.uint8)
        c.stands_for()
        c.check(c.run())


@pytest.mark.parametrize("bs", [16, 5])
@pytest.mark.parametrize("D,G,S", [(16, 2, 5), (32, 8, 6), (48, 16, 5), (80, 2, 5), (96, 16, 5), (112, 8, 6), (128, 4, 3)])
def test_head_sizes(D, G, S, bs):
    """Heads that fill their tiles' columns in part: nothing of the next head's shows."""
    kw = dict(S=S, H=2, G=G, D=D, bs=bs, tree=True, cap=20.0, slopes=True, docs=0.2, seed=D)
    c = Case8([300, 40, 129, 512], **kw)
    clean = c.run()
    c.check(clean)
    c.codes[..., 1, :] = 0x7f
    c.scales[..., 1, :] = 255
    r = c.run()
    assert torch.equal(r.out[:, :, :G], clean.out[:, :, :G]) and torch.equal(r.lse[:, :, :G], clean.lse[:, :, :G])
    assert torch.isnan(r.out[:, :, G:]).all()


@pytest.mark.parametrize("dtype,G,bs", KERNELS)
def test_growing_maxima(dtype, G, bs):
    """Scores that rise along the keys, so that every tile brings a new maximum."""
    c = Case8([1500], S=4, H=1, G=G, D=64, bs=bs, dtype=dtype, seed=16)
    u = torch.nn.functional.normalize(torch.randn(64, generator=torch.Generator().manual_seed(0)), dim=0)
    c.q[0] = (u * 40).to(c.q.dtype)
    x = c.cache.clone()
    for e in range(1500):
        x[0, 0, c.table[0, e // bs], e % bs, 0] = u.double() * e / 50
    c.codes, c.scales = quantised(x.numpy())
    c.stands_for()
    c.check(c.run())


def test_empty_batch():
    cache, empty = api.quant_kv(1, 4, 16, 2, 64), torch.zeros(0, dtype=torch.int32, device="cuda")
    table, x = torch.zeros((0, 3), dtype=torch.int32, device="cuda"), torch.zeros((0, 2, 2, 64), dtype=torch.bfloat16, device="cuda")
    api.write_kv_q8(x, x, cache, table, empty, block_size=16)
    assert api.verify_attention_q8(x, cache, table, empty, block_size=16).out.shape == (0, 2, 2, 64)
    api.commit_kv_q8(cache, table, None, empty, empty, block_size=16, S=2)
    assert api.read_kv_q8(cache, table, n_max=3, block_size=16).k.shape == (0, 3, 2, 64)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strides_and_views(dtype):
    c = Case8([90, 33], S=5, H=2, G=3, D=64, dtype=dtype, seed=4)
    want = c.run()
    pos, a = c.args()
    a.pop("temp_kv")
    B, S, Hq, D = c.q.shape
    cache = on_gpu(c.codes, c.scales)
    wide = torch.zeros((B, S, 3 * Hq, D), dtype=c.q.dtype, device="cuda")
    wide[:, :, Hq:2 * Hq] = pos[0]
    for q in (wide[:, :, Hq:2 * Hq], pos[0].permute(2, 0, 1, 3).contiguous().permute(1, 2, 0, 3)):
        r = api.verify_attention_q8(q, cache, *pos[2:], **a)
        assert torch.equal(r.out, want.out) and torch.equal(r.lse, want.lse)


def test_bad_requests_are_flagged():
    for dtype, bs in (("bf16", 16), ("bf16", 5), ("f32", 16)):
        c = Case8([40, 60, 80, 100], S=3, H=2, G=2, D=64, bs=bs, dtype=dtype, seed=6)
        clean = c.run()
        c.lens[0], c.lens[2] = -1, c.max_blocks * bs - 2
        c.table[1, 0], c.table[3, 1] = c.nb, -5
        flags, ws = torch.zeros(4, dtype=torch.int32, device="cuda"), L.new_workspace(L.SPEC_WS_ATTENTION, 4, 12, 64)
        r = c.run(flags=flags, ws=ws)
        bad = L.SPEC_FLAG_BAD_INPUT
        assert flags.tolist() == [bad] * 4 and L.spec_get_status(ws) == bad
        assert not r.out[[0, 2]].any() and torch.isneginf(r.lse[[0, 2]]).all()
        # the others without the entries of their bad blocks
        c.lens = [40, 60, 80, 100]
        for b, j in ((1, 0), (3, 1)):
            ref, k, off = _without(c, b, range(j * bs, j * bs + bs))
            n = len(k)
            half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
            tol = (2 * c.score_error(b, k) + (2.0 ** -8 if dtype == "bf16" else 0) + (n + 16) * 2.0 ** -24) * ref.mass + half * np.abs(ref.out)
            assert (np.abs(r.out[b].double().cpu().numpy() - ref.out) <= tol).all()
        assert torch.isfinite(clean.out).all()


def _without(c, b, gone):
    kept = c.table.copy()
    c.table = np.where((c.table < 0) | (c.table >= c.nb), 0, c.table)
    k, v, qp, kp = c.row_keys(b)
    off = c.masked(b, qp, kp)
    off[:, list(gone)] = True
    c.table = kept
    return O.attend(c.q[b].double().numpy(), k, v, qp, kp, off, slopes=c.slopes, **c.score), k, off


@pytest.mark.parametrize("bs", [16, 4])
def test_exponents_on_any_address(bs):
    c = Case8([700, 33, 0], S=5, H=2, G=4, D=64, bs=bs, seed=21)
    want = c.run()
    c.check(want)
    scale = torch.from_numpy(c.scales).cuda()
    for at in (1, 2, 4):
        held = torch.empty(scale.numel() + 8, dtype=torch.uint8, device="cuda")[at:at + scale.numel()].view(scale.shape)
        held.copy_(scale)
        pos, a = c.args()
        a.pop("temp_kv")
        r = api.verify_attention_q8(pos[0], api.QuantKV(on_gpu(c.codes, c.scales).codes, held), *pos[2:], **a)
        c.check(r)
        assert at < 4 or torch.equal(r.out, want.out)


@pytest.mark.parametrize("kw", [dict(G=2), dict(G=8), dict(G=20), dict(G=4, bs=5), dict(G=2, shared=128, lens=[128, 300, 700])])
def test_repeats_graphs_and_streams_agree(kw):
    kw = dict(kw)
    c = Case8(kw.pop("lens", [2100, 5, 700]), S=6, H=2, D=128, seed=2, **kw)
    want = c.run()
    pos, a = c.args()
    a.pop("temp_kv")
    cache = on_gpu(c.codes, c.scales)
    call = lambda **k: api.verify_attention_q8(pos[0], cache, *pos[2:], **a, **k)  # noqa: E731
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        held = call()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        graph.replay()
        other, here = call(stream=side), call()
        torch.cuda.synchronize()
        for r in (held, other, here):
            assert torch.equal(r.out, want.out) and torch.equal(r.lse, want.lse)


def test_many_requests_ragged():
    rng = np.random.default_rng(0)
    c = Case8([int(x) for x in rng.integers(0, 500, 70)], S=3, H=2, G=2, D=64, seed=12)
    c.check(c.run())


@pytest.mark.parametrize("D,G,S,H", [(128, 4, 5, 8), (64, 8, 8, 4), (128, 8, 14, 2), (128, 1, 1, 8)])
def test_many_tiles_per_block(D, G, S, H):
    """Rings, buffers and barriers past many rounds, many items a block."""
    c = Case8([1500, 900, 2048, 640, 1, 1300, 2000, 129], S=S, H=H, G=G, D=D, seed=13)
    c.check(c.run())


def test_offsets_past_32_bits():
    """Entries whose codes lie past 2^32 bytes: written, read by the attention, kept, read back."""
    H, D, bs, nb = 8, 128, 16, 300000                     # 4.9 GB of codes a plane
    codes = torch.zeros((1, 2, nb, bs, H, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    cache = api.QuantKV(codes, torch.zeros((1, 2, nb, H, bs), dtype=torch.uint8, device="cuda"))
    g = torch.Generator(device="cuda").manual_seed(0)
    k, v = (torch.randn((2, 40, H, D), generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    q = torch.randn((2, 4, 16, D), generator=g, device="cuda", dtype=torch.bfloat16)
    results = []
    for ids in ([[nb - 1, nb - 7, nb - 3], [nb - 2, nb - 9, nb - 4]], [[0, 3, 1], [2, 5, 7]]):
        table, lens = i32(ids), i32([36, 36])
        api.write_kv_q8(k, v, cache, table, i32([0, 0]), block_size=bs)
        r = api.verify_attention_q8(q, cache, table, lens, block_size=bs)
        f = api.verify_attention_q8(q.float(), cache, table, lens, block_size=bs)
        api.commit_kv_q8(cache, table, i32([[0, 2, 3, -1], [1, 3, -1, -1]]), i32([3, 2]), lens, block_size=bs)
        back = api.read_kv_q8(cache, table, n_max=40, block_size=bs)
        results.append((r.out, r.lse, f.out, f.lse, lens, back.k[:, :38], back.v[:, :38]))
    for a, b in zip(*results):
        assert torch.equal(a, b)
    assert results[0][4].tolist() == [39, 38] and torch.isfinite(results[0][0]).all()


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
def test_rounds_of_chain_decoding():
    """Prompts written, rounds of write, attention, chain verification with the
    in-place commit in two layers: the cache holds the accepted tokens' rows, and
    the attention of each round is the oracle's over them."""
    rng, g = np.random.default_rng(5), torch.Generator().manual_seed(5)
    B, H, G, D, bs, Ly, gamma, V = 3, 2, 4, 128, 16, 2, 4, 64
    S, prompts = gamma + 1, [37, 5, 64]
    table, nb, _ = tables(rng, [n + 60 for n in prompts], bs)
    cache, lens, dt = api.quant_kv(Ly, nb, bs, H, D), i32([0] * B), i32(table)
    held = [[[] for _ in range(2)] for _ in range(B)]     # [b][K/V]: what each entry's rows stand for, by layer
    bf = lambda *s: torch.randn(s, generator=g).bfloat16()  # noqa: E731

    def values(x):
        return O.kv8_values(*O.kv8_quantise(x.double().numpy()))

    p = bf(2, Ly, B, max(prompts), H, D)
    for layer in range(Ly):
        api.write_kv_q8(p[0, layer].cuda(), p[1, layer].cuda(), cache, dt, lens, block_size=bs, layer=layer, n_new=i32(prompts))
    for b in range(B):
        for i in (0, 1):
            held[b][i] = [values(p[i, :, b, e]) for e in range(prompts[b])]
    lens += i32(prompts)
    for _ in range(3):
        kv, q = bf(2, Ly, B, S, H, D), bf(Ly, B, S, H * G, D)
        start = lens.tolist()
        for layer in range(Ly):
            api.write_kv_q8(kv[0, layer].cuda(), kv[1, layer].cuda(), cache, dt, lens, block_size=bs, layer=layer)
            r = api.verify_attention_q8(q[layer].cuda(), cache, dt, lens, block_size=bs, layer=layer)
            for b in range(B):
                k, v = (np.array([e[layer] for e in held[b][i]] + [values(kv[i, layer, b, j]) for j in range(S)]) for i in (0, 1))
                n = start[b]
                off = np.zeros((S, n + S), bool)
                off[:, n:] = O.candidate_mask(S)
                ref = O.attend(q[layer, b].double().numpy(), k, v, np.arange(n, n + S), np.arange(n + S), off, scale=D ** -0.5)
                e = 2.0 ** -24 * (D + 4) * D ** -0.5 * 40 * D + D ** -0.5 * 2.0 ** -17 * 5 * np.abs(k).sum(-1).max()
                tol = (2 * e + 2.0 ** -8 + (n + S + 16) * 2.0 ** -24) * ref.mass + 2.0 ** -8 * np.abs(ref.out)
                assert (np.abs(r.out[b].double().cpu().numpy() - ref.out) <= tol).all()
        logits = torch.randn((B * (gamma + 1), V), generator=g)
        drafts = logits.view(B, gamma + 1, V).argmax(-1)[:, :gamma].int()
        miss = rng.integers(0, gamma + 1, B)              # the first draft that does not match
        for b in range(B):
            if miss[b] < gamma:
                drafts[b, miss[b]] = (drafts[b, miss[b]] + 1) % V
        out = api.verify_chain(logits.cuda(), drafts.cuda(), gamma=gamma, temperature=0.0, committed_len=lens)
        assert out.n_out.tolist() == [int(m) + 1 for m in miss]
        for b in range(B):
            for i in (0, 1):
                held[b][i] += [values(kv[i, :, b, j]) for j in range(int(miss[b]) + 1)]
    assert lens.tolist() == [len(x[0]) for x in held]
    for layer in range(Ly):
        back = api.read_kv_q8(cache, dt, count=lens, n_max=max(lens.tolist()), block_size=bs, layer=layer, dtype=torch.float32)
        for b in range(B):
            for i, x in enumerate((back.k, back.v)):
                assert np.array_equal(x[b, :len(held[b][i])].double().cpu().numpy(), np.array([e[layer] for e in held[b][i]]))


def test_a_round_of_tree_decoding_in_a_graph():
    """verify_tree's mask and positions to the attention, its path to the commit;
    the same round eagerly and captured."""
    rng, g = np.random.default_rng(6), torch.Generator().manual_seed(6)
    B, H, G, D, bs, V = 4, 2, 2, 64, 8, 32
    parent = np.tile(np.array([0, 0, 0, 1, 1, 2]), (B, 1))
    N, R = 6, 7
    S, lens0 = N + 1, [21, 0, 40, 7]
    table, nb, _ = tables(rng, [n + S + 9 for n in lens0], bs)
    logits = torch.randn((B * R, V), generator=g).cuda()
    best = logits.view(B, R, V).argmax(-1).cpu().numpy()
    tokens = np.array([[(best[b, parent[b, i]] + (0 if i in (1, 4) else 1 + i)) % V for i in range(N)] for b in range(B)])
    rows = np.tile(np.arange(R), (B, 1))
    k, v, q = (torch.randn((B, S, n, D), generator=g).bfloat16().cuda() for n in (H, H, H * G))
    dt, node_t, node_p, row = i32(table), i32(tokens), i32(parent), i32(rows)

    def round_(cache, lens):
        tree = api.verify_tree(logits, node_t, node_p, row, lens, R=R)
        api.write_kv_q8(k, v, cache, dt, lens, block_size=bs)
        r = api.verify_attention_q8(q, cache, dt, lens, block_size=bs, tree_mask=tree.tree_mask, pos=tree.pos)
        api.commit_kv_q8(cache, dt, tree.commit_slots, tree.n_commit, lens, block_size=bs)
        return tree, r

    start = random_cache(rng, 1, nb, bs, H, D)
    start[1][:] = start[1] % 20 + 118
    start[0][start[0] & 127 == 127] = 3
    cache, lens = on_gpu(*start), i32(lens0)
    tree, r = round_(cache, lens)
    torch.cuda.synchronize()
    codes, scale = start[0].copy(), start[1].copy()
    for b in range(B):
        for i, x in enumerate((k, v)):
            c, s = O.kv8_quantise(x[b].double().cpu().numpy())
            for e in range(S):
                codes[0, i, table[b, (lens0[b] + e) // bs], (lens0[b] + e) % bs] = c[e]
                scale[0, i, table[b, (lens0[b] + e) // bs], :, (lens0[b] + e) % bs] = s[e]
        path = tree.commit_slots[b, :int(tree.n_commit[b])].tolist()
        assert len(path) >= 2 and O.kv8_commit(codes, scale, table[b], bs, lens0[b], path, S) == int(lens[b])
    got = off_gpu(cache)
    assert np.array_equal(got[0], codes) and np.array_equal(got[1], scale)
    held, hl = on_gpu(*start), i32(lens0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tree2, r2 = round_(held, hl)
    for _ in range(2):
        for dst, src in zip((held.codes.view(torch.uint8), held.scale), (torch.from_numpy(x).cuda() for x in start)):
            dst.copy_(src)
        hl.copy_(i32(lens0))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(r2.out, r.out) and torch.equal(r2.lse, r.lse) and torch.equal(hl, lens)
        assert torch.equal(held.codes.view(torch.uint8), cache.codes.view(torch.uint8)) and torch.equal(held.scale, cache.scale)
