"""Measured cases of the 8-bit paged K/V cache: writing new tokens' keys and
values into it, the verify forward's attention over it, keeping a tree's
accepted candidates, and reading entries back.

``own = False`` computes each operator in elementary torch operations in 32
bits; ``own = True`` calls the library.

Layout (the library's): codes float8_e4m3fn [layers][2][num_blocks][block][H][D],
K at 0 and V at 1; scale uint8 [layers][2][num_blocks][H][block].  A row (one
entry, one cached head) stands for code * 2^(scale - 127), scale the smallest
with every |value| <= 448 * 2^(scale - 127), at least 1.  A round's candidates
lie in the cache at committed_len[b] .. + S - 1.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _case(op, name, **kw):
    base = {
        "attention": dict(H=8, G=4, D=128, block=16, ragged=False, tree=False, cap=0.0, slopes=False, window=0,
                          docs=False, gaps=False, shared=0, dtype="bf16"),
        "write": dict(H=8, D=128, block=16, layers=1, ragged=False, packed=False, dtype="bf16"),
        "commit": dict(H=8, D=128, block=16, ragged=True),
        "read": dict(H=8, D=128, block=16, ragged=False, dtype="bf16"),
    }[op]
    c = dict(op=op, **base)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # the first rounds after short prompts: latency, not bandwidth
        _case("attention", "attention-short", B=8, S=5, len=40, ragged=True),
        # one layer of the chain benchmark's target forward: 64 requests, 4 drafts, 2,048 cached tokens
        _case("attention", "attention-chain", B=64, S=5, len=2048),
        # one layer of the tree benchmark's target forward, scores capped and biased by distance
        _case("attention", "attention-tree-capped", B=128, S=13, len=2048, tree=True, cap=50.0, slopes=True),
        # plain decoding: single tokens over long ragged caches
        _case("attention", "attention-single", B=64, S=1, len=32768, ragged=True),
        # a system prompt of 4,096 tokens shared by the chain benchmark's batch, short turns behind it
        _case("attention", "attention-shared", B=64, S=5, len=300, ragged=True, shared=4096),
        # a small float32 model with an odd head size and odd blocks
        _case("attention", "attention-f32", B=8, S=5, len=777, ragged=True, H=2, D=80, G=3, block=5, dtype="f32",
              slopes=True),
        # the candidates of one round of the chain benchmark, one layer, before its attention
        _case("write", "write-candidates", B=64, S=5, len=2048),
        # prompts of up to 8,192 tokens entering the cache, one layer, padded to the longest; K and V are
        # parts of the fused projection's output
        _case("write", "write-prompts", B=16, S=8192, len=0, ragged=True, packed=True),
        # a small tree round: nothing but latency
        _case("commit", "commit-small", B=4, S=13, len=40, layers=2, H=2, D=64),
        # the tree benchmark's accepted paths, every layer
        _case("commit", "commit-tree", B=128, S=13, len=128, layers=32),
        # the last few entries of a small cache, for a look at them in float32
        _case("read", "read-small", B=8, n=21, len=64, H=2, D=80, block=5, ragged=True, dtype="f32"),
        # long prefixes read back for the next chunk of their prompts
        _case("read", "read-prefix", B=16, n=8192, len=8192, ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "write", "commit", "read"])
    head = dict(H=rng.choice([1, 2, 4, 8]), D=rng.choice([32, 64, 80, 96, 128, 128, 128, 160, 256]),
                block=rng.choice([1, 5, 8, 16, 16, 32, 48, 64]))
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    ragged = rng.random() < 0.7
    if op == "attention":
        S, B, length = _log(rng, 1, 40), _log(rng, 1, 128), _log(rng, 1, 32768)
        c = _case(op, "", B=B, S=S, len=length, G=rng.choice([1, 2, 3, 4, 7, 8]), ragged=ragged,
                  tree=rng.random() < 0.4, cap=rng.choice([0.0, 0.0, 20.0, 50.0]), slopes=rng.random() < 0.4,
                  docs=rng.random() < 0.3, gaps=rng.random() < 0.3, dtype=dtype, **head)
        if rng.random() < 0.3:
            c["window"] = _log(rng, 1, 2 * length)
        size = "len"
        if rng.random() < 0.25:
            c.update(shared=_log(rng, 64, 8192), gaps=False, len=_log(rng, 1, 512))
            size = "shared"
        # no dearer than the largest listed case; wide heads and odd pages run on the CUDA cores
        slow = dtype == "f32" or head["D"] > 128 or head["block"] % 8
        while c[size] > 1 and (work(c)["bytes"] > 2e9 or work(c)["flops"] > (1e10 if slow else 5e10)):
            c[size] = max(1, c[size] * 2 // 3)
        return c
    if op == "write":
        B = _log(rng, 1, 128)
        S = _log(rng, 1, min(16384, (1 << 17) // B))
        return _case(op, "", B=B, S=S, len=_log(rng, 1, 512) - 1, ragged=ragged, packed=rng.random() < 0.5, dtype=dtype,
                     layers=rng.choice([1, 1, 2]), **head)
    if op == "commit":
        B, layers = _log(rng, 1, 128), _log(rng, 1, 32)
        return _case(op, "", B=B, S=_log(rng, 2, 64), len=_log(rng, 1, 128), layers=layers, ragged=ragged, **head)
    B = _log(rng, 1, 128)
    n = _log(rng, 1, min(16384, (1 << 17) // B))
    return _case(op, "", B=B, n=n, len=n + _log(rng, 1, 256) - 1, ragged=ragged, dtype=dtype, **head)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _spread(n, B, ragged, least=1):
    """B sizes: n, or spread over least..n (both ends among them)."""
    least = min(least, n)
    if not ragged:
        return [n] * B
    return [n if b == 0 else least + (b * 2654435761 % 4294967296) * (n + 1 - least) // 4294967296 for b in range(B)]


def _slots_of(case):
    """Committed candidates of each request: 1 .. half of its S."""
    return [1 + (b * 7 + 3) % max(1, (case["S"] + 1) // 2) for b in range(case["B"])]


def _table(rng, needed, block, max_blocks):
    """A block table over blocks in random order: needed[b] entries each."""
    counts = [-(-n // block) for n in needed]
    order = torch.randperm(sum(counts), generator=rng, device="cuda").to(torch.int32)
    table = torch.zeros((len(needed), max_blocks), dtype=torch.int32, device="cuda")
    rows = torch.repeat_interleave(torch.arange(len(needed)), torch.tensor(counts))
    cols = torch.cat([torch.arange(k) for k in counts])
    table[rows.cuda(), cols.cuda()] = order
    return table, sum(counts)


def _normal(rng, shape, dtype, sigma=1.0):
    return torch.randn(shape, generator=rng, device="cuda", dtype=dtype).mul_(sigma)


def _heads(rng, H):
    """Heads differ in size, as trained ones do."""
    return torch.exp(0.7 * torch.randn((H, 1), generator=rng, device="cuda"))


def _filled(rng, shape):
    """Codes and scales of a cache [layers, 2, blocks, block, H, D] of normal values."""
    codes = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty(shape[:3] + (shape[4], shape[3]), dtype=torch.uint8, device="cuda")
    for layer in range(shape[0]):
        for i in (0, 1):
            x = torch.randn(shape[2:], generator=rng, device="cuda") * _heads(rng, shape[4])
            c, sc = _quantised(x)
            codes[layer, i] = c
            scale[layer, i] = sc.transpose(1, 2)
    return codes, scale


def _prepare_attention(case, rng):
    B, S, H, G, D, bs, P = (case[k] for k in ("B", "S", "H", "G", "D", "block", "shared"))
    total = [P + n for n in _spread(case["len"], B, case["ragged"])]
    whole = P // bs                                  # blocks that hold shared entries only
    table, blocks = _table(rng, [n + S - whole * bs for n in total], bs, -(-(max(total) + S) // bs) - whole)
    s = dict(case)
    if P:
        # one more run of blocks holds the shared prefix; each request's own
        # table names them too, as a prefix cache leaves them
        count = -(-P // bs)
        s["shared_table"] = torch.arange(blocks, blocks + count, dtype=torch.int32, device="cuda")
        blocks += count
        table = torch.cat([s["shared_table"][:whole].expand(B, whole), table], 1).contiguous()
    width = table.shape[1] * bs
    s["codes"], s["scale"] = _filled(rng, (1, 2, blocks, bs, H, D))
    s.update(table=table, q=_normal(rng, (B, S, H * G, D), DTYPES[case["dtype"]], 2.0),
             lens=torch.tensor(total, dtype=torch.int32, device="cuda"), softmax_scale=1.0 / math.sqrt(D),
             mask=None, pos=None, key_pos=None, first=None, slope=None)
    if case["slopes"]:
        heads = H * G
        s["slope"] = 2.0 ** (-8.0 * (torch.arange(heads, device="cuda", dtype=torch.float32) + 1) / heads)
    text = s["lens"].to(torch.int64)                 # position of the first candidate
    if case["gaps"]:                                 # thinned caches: ascending positions with gaps
        step = torch.randint(1, 4, (B, width), generator=rng, device="cuda")
        s["key_pos"] = (step.cumsum(1) - 1).to(torch.int32)
        text = s["key_pos"].gather(1, text[:, None] - 1)[:, 0].to(torch.int64) + 1
    if case["docs"]:                                 # the current document began in the first half
        s["first"] = (text * torch.rand(B, generator=rng, device="cuda") * 0.5).to(torch.int32)
    if case["tree"]:
        # a random tree over the candidates: node i's parent is an earlier one
        parent = [[-1] + [int(x) for x in row] for row in
                  (torch.rand((B, S - 1), generator=rng, device="cuda") * torch.arange(1, S, device="cuda")).int().tolist()]
        depth = torch.zeros((B, S), dtype=torch.int64)
        bits = torch.zeros((B, S, (S + 31) // 32), dtype=torch.int64)
        for b in range(B):
            for i in range(S):
                if i:
                    depth[b, i] = depth[b, parent[b][i]] + 1
                    bits[b, i] = bits[b, parent[b][i]]
                bits[b, i, i // 32] |= 1 << (i % 32)
        s["mask"] = bits.cuda().to(torch.int32)
        s["pos"] = (text[:, None] + depth.cuda()).to(torch.int32)
    elif case["gaps"]:
        s["pos"] = (text[:, None] + torch.arange(S, device="cuda")).to(torch.int32)
    return s


def _prepare_write(case, rng):
    B, S, H, D, bs, L = (case[k] for k in ("B", "S", "H", "D", "block", "layers"))
    lens, new = _spread(case["len"], B, True), _spread(S, B, case["ragged"])
    table, blocks = _table(rng, [n + m for n, m in zip(lens, new)], bs, -(-(max(lens) + S) // bs))
    dtype = DTYPES[case["dtype"]]
    if case["packed"]:                               # [q | k | v] of one projection
        qkv = _normal(rng, (B, S, 6 * H, D), dtype)
        qkv.mul_(_heads(rng, 6 * H).to(dtype))
        k, v = qkv[:, :, 4 * H:5 * H], qkv[:, :, 5 * H:]
    else:
        k, v = (_normal(rng, (B, S, H, D), dtype).mul_(_heads(rng, H).to(dtype)) for _ in range(2))
    return dict(case, k=k, v=v, table=table, layer=L - 1,
                codes=torch.zeros((L, 2, blocks, bs, H, D), device="cuda").to(torch.float8_e4m3fn),
                scale=torch.zeros((L, 2, blocks, H, bs), dtype=torch.uint8, device="cuda"),
                lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                new=torch.tensor(new, dtype=torch.int32, device="cuda") if case["ragged"] else None)


def _prepare_commit(case, rng):
    B, S, H, D, bs, L = (case[k] for k in ("B", "S", "H", "D", "block", "layers"))
    lens, n_slots = _spread(case["len"], B, case["ragged"]), _slots_of(case)
    table, blocks = _table(rng, [n + S for n in lens], bs, -(-(max(lens) + S) // bs))
    codes, scale = _filled(rng, (L, 2, blocks, bs, H, D))
    # the root and an ascending path through nodes past the places that it moves to
    # (a path along the first ranks is where it belongs already)
    n = torch.tensor(n_slots, device="cuda")[:, None]
    at = torch.arange(S, device="cuda")[None]
    rank = torch.where(at >= n, torch.rand((B, S), generator=rng, device="cuda"), 2.0).argsort(1)
    pick = torch.where(at < n - 1, rank, S).sort(1).values
    slots = torch.cat([torch.zeros((B, 1), dtype=torch.int64, device="cuda"), pick[:, :S - 1]], 1)
    slots = torch.where(at < n, slots, -1).to(torch.int32)
    return dict(case, codes=codes, scale=scale, table=table, slots=slots,
                n_slots=n[:, 0].to(torch.int32), lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))


def _prepare_read(case, rng):
    B, H, D, bs = (case[k] for k in ("B", "H", "D", "block"))
    count = _spread(case["n"], B, case["ragged"])
    start = [(b * 40503 % 65536) * (case["len"] - c + 1) // 65536 for b, c in enumerate(count)]
    table, blocks = _table(rng, [case["len"]] * B, bs, -(-case["len"] // bs))
    codes, scale = _filled(rng, (1, 2, blocks, bs, H, D))
    return dict(case, codes=codes, scale=scale, table=table,
                start=torch.tensor(start, dtype=torch.int32, device="cuda"),
                count=torch.tensor(count, dtype=torch.int32, device="cuda"))


def prepare(case, seed):
    rng = torch.Generator(device="cuda").manual_seed(seed)
    return {"attention": _prepare_attention, "write": _prepare_write, "commit": _prepare_commit,
            "read": _prepare_read}[case["op"]](case, rng)


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _power(e):
    """2^(e - 127) of 1 <= e <= 254, from its bits."""
    return (e.to(torch.int32) << 23).view(torch.float32)


def _quantised(x):
    """Codes and biased exponents of the rows of x (float32)."""
    bits = x.abs().amax(-1).view(torch.int32)
    scale = ((bits >> 23) - 8 + ((bits & 0x7fffff) > 0x600000).int()).clamp(min=1)
    return (x * _power(254 - scale)[..., None]).to(torch.float8_e4m3fn), scale.to(torch.uint8)


def _values(codes, scale, table, bs, at):
    """[B, n, H, D] in 32 bits: the entries `at` [B or 1, n] of one plane (codes
    [blocks, block, H, D], scale [blocks, H, block])."""
    at = at.expand(table.shape[0], -1)
    blk, off = table.long().gather(1, at // bs), at % bs
    x = codes.view(torch.uint8)[blk, off].view(torch.float8_e4m3fn).float()
    return x.mul_(_power(scale.transpose(1, 2)[blk, off])[..., None])


def _plain_attention(s):
    B, S, H, G, D, bs, P = s["B"], s["S"], s["H"], s["G"], s["D"], s["block"], s["shared"]
    q = s["q"].float().view(B, S, H, G, D).permute(0, 2, 3, 1, 4)  # [B,H,G,S,D]
    lens = s["lens"].long()[:, None]
    at = torch.arange(P, s["table"].shape[1] * bs, device="cuda")[None]  # own entries
    k, v = (_values(s["codes"][0, i], s["scale"][0, i], s["table"], bs, at) for i in (0, 1))
    qp = s["pos"].long() if s["pos"] is not None else lens + torch.arange(S, device="cuda")
    mine = (at >= lens) & (at < lens + S)                             # candidates
    j = (at - lens).clamp(0, S - 1)
    kp = s["key_pos"][:, P:].long() if s["key_pos"] is not None else at.expand(B, -1)
    kp = torch.where(mine, qp.gather(1, j), kp)
    if s["mask"] is not None:
        i = torch.arange(S, device="cuda")
        seen = (s["mask"][:, :, i // 32] >> (i % 32)) & 1 != 0
    else:
        seen = torch.ones((S, S), dtype=torch.bool, device="cuda").tril()[None].expand(B, S, S)
    seen = seen.gather(2, j[:, None, :].expand(B, S, -1))
    visible = torch.where(mine[:, None, :], seen, (at < lens)[:, None, :])

    def scores(dots, kp, visible):
        x = dots.mul_(s["softmax_scale"])
        if s["cap"]:
            x = s["cap"] * torch.tanh(x / s["cap"])
        dist = qp[:, :, None] - kp[:, None, :]
        if s["slope"] is not None:
            x = x - s["slope"].view(1, H, G, 1, 1) * dist[:, None, None].float()
        if s["window"]:
            visible = visible & (dist < s["window"])
        if s["first"] is not None:
            visible = visible & (kp >= s["first"][:, None])[:, None, :]
        return x.masked_fill_(~visible[:, None, None], -math.inf)

    x = scores(torch.einsum("bhgsd,bnhd->bhgsn", q, k), kp, visible)
    if P:
        at = torch.arange(P, device="cuda")[None]
        ks, vs = (_values(s["codes"][0, i], s["scale"][0, i], s["shared_table"][None], bs, at)[0] for i in (0, 1))
        every = torch.ones((1, 1, P), dtype=torch.bool, device="cuda").expand(B, 1, P)
        x = torch.cat([scores(torch.einsum("bhgsd,nhd->bhgsn", q, ks), at, every), x], -1)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = x.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.einsum("bhgsn,bnhd->bhgsd", p[..., P:], v)
    if P:
        out += torch.einsum("bhgsn,nhd->bhgsd", p[..., :P], vs)
    out = torch.where(total > 0, out / total, 0.0)
    lse = (m + total.log())[..., 0]
    return {"out": out.permute(0, 3, 1, 2, 4).reshape(B, S, H * G, D).to(s["q"].dtype),
            "lse": lse.permute(0, 3, 1, 2).reshape(B, S, H * G)}


def _plain_write(s):
    S, bs, layer = s["S"], s["block"], s["layer"]
    i = torch.arange(S, device="cuda")[None]
    at = s["lens"].long()[:, None] + i
    blk = s["table"].long().gather(1, (at // bs).clamp(max=s["table"].shape[1] - 1))
    off = at % bs
    if s["new"] is not None:
        kept = i < s["new"][:, None]
        blk, off = blk[kept], off[kept]
    codes, scale = s["codes"].view(torch.uint8), s["scale"]
    for j, x in enumerate((s["k"], s["v"])):
        c, e = _quantised(x.float())
        c = c.view(torch.uint8)
        if s["new"] is not None:
            c, e = c[kept], e[kept]
        codes[layer, j, blk, off] = c
        scale[layer, j].transpose(1, 2)[blk, off] = e
    return {"codes": s["codes"], "scale": scale}


def _plain_commit(s, lens):
    S, bs = s["S"], s["block"]
    i = torch.arange(S, device="cuda")[None]
    b, at = ((i < s["n_slots"][:, None]) & (s["slots"] > i)).nonzero().T
    src, dst = lens[b].long() + s["slots"][b, at], lens[b].long() + at
    sb, db = s["table"][b, src // bs].long(), s["table"][b, dst // bs].long()
    codes, scale = s["codes"].view(torch.uint8), s["scale"].transpose(3, 4)
    codes[:, :, db, dst % bs] = codes[:, :, sb, src % bs]
    scale[:, :, db, dst % bs] = scale[:, :, sb, src % bs]
    lens += s["n_slots"]
    return {"codes": s["codes"], "scale": s["scale"], "len": lens, "blocks": ((lens + bs - 1) // bs).to(torch.int32)}


def _plain_read(s):
    i = torch.arange(s["n"], device="cuda")[None]
    at = (s["start"].long()[:, None] + i).clamp(max=s["len"] - 1)
    kept = (i < s["count"][:, None])[..., None, None]
    return {name: torch.where(kept, _values(s["codes"][0, j], s["scale"][0, j], s["table"], s["block"], at), 0.0)
            .to(DTYPES[s["dtype"]]) for j, name in enumerate("kv")}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    if not own:
        if s["op"] == "commit":
            return _plain_commit(s, s["lens"].clone())
        return {"attention": _plain_attention, "write": _plain_write, "read": _plain_read}[s["op"]](s)
    from speculative_decoding_verification_37_gb300 import api
    cache = api.QuantKV(s["codes"], s["scale"])
    if s["op"] == "attention":
        shared = dict(shared_table=s["shared_table"], shared_len=s["shared"]) if s["shared"] else {}
        r = api.verify_attention_q8(s["q"], cache, s["table"], s["lens"], block_size=s["block"], tree_mask=s["mask"],
                                    pos=s["pos"], key_pos=s["key_pos"], first_pos=s["first"], slopes=s["slope"],
                                    scale=s["softmax_scale"], softcap=s["cap"], window=s["window"], **shared)
        return {"out": r.out, "lse": r.lse}
    if s["op"] == "write":
        api.write_kv_q8(s["k"], s["v"], cache, s["table"], s["lens"], block_size=s["block"], layer=s["layer"],
                        n_new=s["new"])
        return {"codes": s["codes"], "scale": s["scale"]}
    if s["op"] == "commit":
        lens = s["lens"].clone()
        blocks = torch.empty_like(lens)
        api.commit_kv_q8(cache, s["table"], s["slots"], s["n_slots"], lens, block_size=s["block"], blocks_in_use=blocks)
        return {"codes": s["codes"], "scale": s["scale"], "len": lens, "blocks": blocks}
    r = api.read_kv_q8(cache, s["table"], s["start"], s["count"], n_max=s["n"], block_size=s["block"],
                       dtype=DTYPES[s["dtype"]])
    return {"k": r.k, "v": r.v}


# ---------------------------------------------------------------------------
# the work of a pass
# ---------------------------------------------------------------------------
def work(case):
    B, H, D = case["B"], case["H"], case["D"]
    row = H * (D + 1)                                # codes and exponents of one entry's K or V
    if case["op"] == "commit":
        moved = sum(n - 1 for n in _slots_of(case))
        return {"bytes": 2 * moved * case["layers"] * 2 * row + sum(_slots_of(case)) * 4, "flops": 0}
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("write", "read"):
        n = sum(_spread(case["S" if case["op"] == "write" else "n"], B, case["ragged"]))
        # (a read's rows behind the last entry are written too, as zeros)
        plain = n if case["op"] == "write" else B * case["n"]
        return {"bytes": 2 * (n * row + plain * H * D * e), "flops": n * 2 * H * D * 2}
    S, G, P = case["S"], case["G"], case["shared"]
    docs = 0.75 if case["docs"] else 1.0             # the document starts a quarter in, on average
    seen = lambda n: min(n, case["window"] + S) if case["window"] and not case["gaps"] else n  # noqa: E731
    n = sum(seen(P + t) for t in _spread(case["len"], B, case["ragged"])) * docs
    unique = n - max(0, B - 1) * seen(P) if P else n
    return {"bytes": (max(unique, 0) + B * S) * 2 * row + B * S * G * H * (2 * D * e + 4),
            "flops": (n + B * S) * H * S * G * D * 4}


# ---------------------------------------------------------------------------
# 64 bits, a request at a time, from the definitions
# ---------------------------------------------------------------------------
def _entry_rows(s, which, table, places):
    """[n, H, D]: K (0) or V (1) of the entries `places` under one block table."""
    blk, off = table.long()[places // s["block"]], places % s["block"]
    code = s["codes"][0, which].view(torch.uint8)[blk, off].long()
    sign, e, m = 1.0 - 2.0 * (code >> 7), (code >> 3) & 15, (code & 7).double()
    mag = torch.where(e == 0, m * 2.0 ** -9, (8.0 + m) * torch.exp2((e - 10).double()))
    power = torch.exp2(s["scale"][0, which][blk, :, off].double() - 127.0)
    return sign * mag * power[..., None]


def _exact_attention(s):
    S, H, G, P = s["S"], s["H"], s["G"], s["shared"]
    outs, lses = [], []
    if P:
        i = torch.arange(P, device="cuda")
        common = [_entry_rows(s, w, s["shared_table"], i) for w in (0, 1)]
    for b, n in enumerate(s["lens"].tolist()):
        places = torch.arange(P, n + S, device="cuda")
        k, v = (_entry_rows(s, w, s["table"][b], places) for w in (0, 1))
        if P:
            k, v = torch.cat([common[0], k]), torch.cat([common[1], v])
        qp = (torch.arange(n, n + S, device="cuda") if s["pos"] is None else s["pos"][b]).double()
        kp = (torch.arange(n, device="cuda") if s["key_pos"] is None else s["key_pos"][b, :n]).double()
        kp = torch.cat([kp, qp])
        ok = torch.ones((S, n + S), dtype=torch.bool, device="cuda")
        if s["mask"] is None:
            ok[:, n:] = torch.tril(ok[:, n:])
        else:
            words = s["mask"][b].tolist()
            ok[:, n:] = torch.tensor([[bool(words[i][j // 32] >> (j % 32) & 1) for j in range(S)] for i in range(S)],
                                     device="cuda")
        gap = qp[:, None] - kp[None, :]
        if s["window"]:
            ok &= gap < s["window"]
        if s["first"] is not None:
            ok &= kp[None, :] >= int(s["first"][b])
        q = s["q"][b].double().permute(1, 0, 2).reshape(H, G * S, -1)
        x = torch.bmm(q, k.permute(1, 2, 0)).reshape(H * G, S, n + S) * s["softmax_scale"]
        if s["cap"]:
            x = torch.tanh(x / s["cap"]) * s["cap"]
        if s["slope"] is not None:
            x = x - s["slope"].double()[:, None, None] * gap
        x = torch.where(ok, x, -math.inf)
        lse = torch.logsumexp(x, -1)
        p = torch.exp(x - torch.where(lse.isinf(), 0.0, lse)[..., None])
        o = torch.bmm(p.reshape(H, G * S, -1), v.permute(1, 0, 2)).reshape(H * G, S, -1)
        outs.append(o.permute(1, 0, 2))
        lses.append(lse.T)
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}


def _exact_write(s):
    codes, scale, bs = s["codes"].double(), s["scale"], s["block"]
    new = [s["S"]] * s["B"] if s["new"] is None else s["new"].tolist()
    for b, n in enumerate(s["lens"].tolist()):
        places = torch.arange(n, n + new[b], device="cuda")
        blk, off = s["table"][b].long()[places // bs], places % bs
        for j, t in enumerate((s["k"], s["v"])):
            x = t[b, :new[b]].double()
            mant, e = torch.frexp(x.abs().amax(-1))  # 448 = 0.875 * 2^9
            e = (e - 9 + (mant > 0.875).int()).clamp(min=-126)
            y = x * torch.exp2(-e.double())[..., None]
            # neighbours of e4m3 are 2^-3 of a value's power of two apart, 2^-9 at least
            step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
            codes[s["layer"], j, blk, off] = torch.round(y / step) * step
            scale[s["layer"], j, blk, :, off] = (e + 127).to(torch.uint8)
    return {"codes": codes, "scale": scale}


def _exact_commit(s):
    bs, lens, table = s["block"], s["lens"].tolist(), s["table"].cpu()
    for b, n in enumerate(s["n_slots"].tolist()):
        for i, j in enumerate(s["slots"][b, :n].tolist()):
            src, dst = lens[b] + j, lens[b] + i
            sb, db = int(table[b, src // bs]), int(table[b, dst // bs])
            s["codes"].view(torch.uint8)[:, :, db, dst % bs] = s["codes"].view(torch.uint8)[:, :, sb, src % bs].clone()
            s["scale"][:, :, db, :, dst % bs] = s["scale"][:, :, sb, :, src % bs].clone()
        lens[b] += n
    whole = torch.tensor(lens, dtype=torch.int32)
    return {"codes": s["codes"], "scale": s["scale"], "len": whole,
            "blocks": torch.tensor([-(-n // bs) for n in lens], dtype=torch.int32)}


def _exact_read(s):
    k, v = (torch.zeros((s["B"], s["n"], s["H"], s["D"]), dtype=torch.float64, device="cuda") for _ in range(2))
    for b, (i, n) in enumerate(zip(s["start"].tolist(), s["count"].tolist())):
        for w, t in enumerate((k, v)):
            t[b, :n] = _entry_rows(s, w, s["table"][b], torch.arange(i, i + n, device="cuda"))
    return {"k": k, "v": v}


def exact(case, seed):
    return {"attention": _exact_attention, "write": _exact_write, "commit": _exact_commit,
            "read": _exact_read}[case["op"]](prepare(case, seed))
