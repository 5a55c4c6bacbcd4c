"""Measured cases of the operators around the paged K/V cache: the verify
forward's attention (scores capped by a tanh, biased by distance, masked by
document, window and draft tree), the same for a batch that shares a long
prefix, the attention weight each cached entry accumulates, and the eviction
that goes by it.

``own = False`` computes each operator in elementary torch operations in 32
bits; ``own = True`` calls the library.

Layout (the library's): cache [layers][2][num_blocks][block][H][D], K at 0 and
V at 1; block_table int32 [B][max_blocks]; q [B][S][H*G][D] with G query heads
per cached head; candidate K/V temp_kv [B][layers][2][S][H][D].
"""
import math

import torch

own = False

PACKAGE = "speculative_decoding_verification_37_gb300"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _attention(name, B, S, length, **kw):
    c = dict(op="attention", B=B, S=S, H=8, G=4, D=128, block=16, len=length, ragged=False, tree=False,
             inplace=False, cap=0.0, slopes=False, window=0, docs=False, gaps=False, shared=0, dtype="bf16")
    c.update(kw)
    if name:
        c["name"] = name
    return c


def _weights(name, B, S, length, **kw):
    c = dict(op="weights", B=B, S=S, H=8, G=4, D=128, block=16, len=length, ragged=False, cap=0.0,
             slopes=False, window=0, docs=False, gaps=False, shared=0, dtype="bf16")
    c.update(kw)
    if name:
        c["name"] = name
    return c


def _evict(name, B, length, budget, **kw):
    c = dict(op="evict", B=B, layers=32, H=8, D=128, block=16, len=length, budget=budget, sink=4,
             ragged=False, again=False, dtype="bf16")
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # the first rounds after short prompts: latency, not bandwidth
        _attention("attention-short", 8, 5, 40, ragged=True),
        # one layer of the chain benchmark's target forward: 64 requests, 4 drafts, 2,048 cached tokens
        _attention("attention-chain", 64, 5, 2048),
        # one layer of the tree benchmark's target forward, scores capped and biased by distance
        _attention("attention-tree-capped", 128, 13, 2048, tree=True, cap=50.0, slopes=True),
        # single tokens over long ragged caches that have been thinned out, biased by the entries' own positions
        _attention("attention-single", 64, 1, 32768, ragged=True, inplace=True, gaps=True, slopes=True),
        # two long documents alone on the GPU: the keys have to be split to fill it; a local layer's window
        _attention("attention-long-docs", 2, 8, 32768, docs=True, cap=30.0, window=24576),
        # a small float32 model with an odd head size and odd blocks
        _attention("attention-f32", 8, 5, 777, ragged=True, H=2, D=72, G=3, block=5, dtype="f32", slopes=True),
        # a system prompt of 4,096 tokens shared by the chain benchmark's batch, short turns behind it
        _attention("shared-chain", 64, 5, 300, ragged=True, shared=4096),
        # the largest batch of the benchmarks on a long shared document
        _attention("shared-large", 512, 8, 256, ragged=True, shared=8192),
        # the accepted tokens' weights over the chain benchmark's cache, one layer
        _weights("weights-chain", 64, 5, 2048),
        # ragged, capped and biased, large batch
        _weights("weights-ragged-capped", 512, 8, 4096, ragged=True, cap=50.0, slopes=True),
        # a small cache trimmed after every few rounds
        _evict("evict-small", 8, 100, 64, layers=2, H=2, D=64, ragged=True),
        # every layer of 16 requests cut back from up to 2,304 to 2,048 tokens
        _evict("evict-layers", 16, 2304, 2048, ragged=True, again=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _bounded(c, size):
    """The case with its length cut until it costs less than the largest listed one."""
    flops = 1.5e11 if c["dtype"] == "bf16" else 1e10
    while c[size] > c["S"] + 1 and (work(c)["bytes"] > 1.5e9 or work(c)["flops"] > flops):
        c[size] = max(c["S"] + 1, c[size] * 2 // 3)
        if c["op"] == "weights":
            c["shared"] = min(c["shared"], c["len"] // 2)
    return c


def draw(rng):
    kind = rng.choice(["attention", "attention", "shared", "weights", "evict"])
    head = dict(H=rng.choice([1, 2, 4, 8]), G=rng.choice([1, 2, 3, 4, 7, 8]),
                D=rng.choice([64, 72, 96, 128, 128, 128, 160, 256]), block=rng.choice([1, 5, 16, 16, 32, 48, 64]))
    score = dict(cap=rng.choice([0.0, 0.0, 20.0, 50.0]), slopes=rng.random() < 0.4, docs=rng.random() < 0.3)
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if kind in ("attention", "shared"):
        S = _log(rng, 1, 40)
        B = _log(rng, 1, 128)
        length = _log(rng, 1, 32768)
        c = _attention("", B, S, length, ragged=rng.random() < 0.7, tree=rng.random() < 0.4,
                       inplace=rng.random() < 0.4, gaps=rng.random() < 0.3, dtype=dtype, **head, **score)
        if rng.random() < 0.3:
            c["window"] = _log(rng, 1, 2 * length)
        if kind == "shared":
            c.update(shared=_log(rng, 64, 8192), gaps=False, len=_log(rng, 1, 512))
        return _bounded(c, "shared" if kind == "shared" else "len")
    if kind == "weights":
        S, B = _log(rng, 1, 16), _log(rng, 1, 128)
        length = _log(rng, S, 32768)
        c = _weights("", B, S, length, ragged=rng.random() < 0.7, gaps=rng.random() < 0.3, dtype=dtype, **head,
                     **score)
        if rng.random() < 0.3:
            c["window"] = _log(rng, 1, 2 * length)
        if rng.random() < 0.2:
            c["shared"] = length // 2
        return _bounded(c, "len")
    B, layers = _log(rng, 1, 32), _log(rng, 1, 32)
    length = _log(rng, 16, max(17, min(8192, (1 << 20) // (B * layers))))
    budget = max(8, length - _log(rng, 1, max(2, length // 4)))
    return _evict("", B, length, budget, layers=layers, H=head["H"], D=head["D"], block=head["block"],
                  ragged=rng.random() < 0.7, again=rng.random() < 0.5, sink=rng.choice([0, 1, 4]), dtype=dtype)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _lengths(case, least):
    """Entries of each request after the shared prefix: `len`, or spread over
    least..len (a request of each end among them)."""
    n, B = case["len"], case["B"]
    if not case["ragged"]:
        return [max(n, least)] * B
    least = min(least, n)
    return [n if b == 0 else least + (b * 2654435761 % 4294967296) * (n + 1 - least) // 4294967296
            for b in range(B)]


def _slots_of(case):
    """Committed slots of each request: 1 .. S of its S candidates, slot 0 first."""
    S = case["S"]
    return [1 + (b * 7 + 3) % S for b in range(case["B"])]


def _table(rng, needed, block, max_blocks):
    """A block table over blocks in random order: needed[b] entries (tokens) each."""
    counts = [-(-n // block) for n in needed]
    total = sum(counts)
    order = torch.randperm(total, generator=rng, device="cuda").to(torch.int32)
    table = torch.zeros((len(needed), max_blocks), dtype=torch.int32, device="cuda")
    rows = torch.repeat_interleave(torch.arange(len(needed)), torch.tensor(counts))
    cols = torch.cat([torch.arange(k) for k in counts])
    table[rows.cuda(), cols.cuda()] = order
    return table, total


def _normal(rng, shape, dtype, sigma=1.0):
    x = torch.randn(shape, generator=rng, device="cuda", dtype=dtype)
    return x.mul_(sigma) if sigma != 1.0 else x


def _slopes(case):
    heads = case["H"] * case["G"]
    return 2.0 ** (-8.0 * (torch.arange(heads, device="cuda", dtype=torch.float32) + 1) / heads)


def _thinned(rng, B, n, per_entry=4):
    """Ascending positions with gaps: n entries left of up to per_entry * n tokens."""
    step = torch.randint(1, per_entry, (B, n), generator=rng, device="cuda")
    return (step.cumsum(1) - 1).to(torch.int32)


def _prepare_attention(case, rng):
    B, S, H, G, D, bs = (case[k] for k in ("B", "S", "H", "G", "D", "block"))
    dtype, shared, weights = DTYPES[case["dtype"]], case["shared"], case["op"] == "weights"
    entries = _lengths(case, case["S"] if weights else 1)
    if weights:  # the shared entries are the first part of `len`
        total = entries
        shared = min(shared, min(total))
    else:
        total = [shared + n for n in entries]
    room = 0 if weights or not case["inplace"] else S
    whole = 0 if weights else shared // bs          # blocks that hold shared entries only
    s = dict(case)
    table, blocks = _table(rng, [n + room - whole * bs for n in total], bs, -(-(max(total) + room) // bs) - whole)
    if shared and not weights:
        # one more run of blocks holds the shared prefix; each request's own
        # table names them too, as a prefix cache leaves them
        count = -(-shared // bs)
        s["shared_table"] = torch.arange(blocks, blocks + count, dtype=torch.int32, device="cuda")
        blocks += count
        table = torch.cat([s["shared_table"][:whole].expand(B, whole), table], 1).contiguous()
    max_blocks = table.shape[1]
    s.update(total=max(total), shared=shared, table=table,
             cache=_normal(rng, (1, 2, blocks, bs, H, D), dtype),
             q=_normal(rng, (B, S, H * G, D), dtype, 2.0),
             lens=torch.tensor(total, dtype=torch.int32, device="cuda"),
             scale=1.0 / math.sqrt(D), temp=None, mask=None, pos=None, key_pos=None, first=None, slopes=None)
    if case["slopes"]:
        s["slopes"] = _slopes(case)
    text = s["lens"].to(torch.int64)  # position of the first candidate
    if case["gaps"]:
        s["key_pos"] = torch.zeros((B, max_blocks * bs), dtype=torch.int32, device="cuda")
        s["key_pos"][:, :max(total)] = _thinned(rng, B, max(total))
        text = s["key_pos"].gather(1, text[:, None] - 1)[:, 0].to(torch.int64) + 1
    if case["docs"]:  # the current document began in the first half
        s["first"] = (text * torch.rand(B, generator=rng, device="cuda") * 0.5).to(torch.int32)
    if weights:
        n_slots = _slots_of(case)
        s["n_slots"] = torch.tensor(n_slots, dtype=torch.int32, device="cuda")
        # the committed candidates are slot 0 and an ascending choice of the others
        rest = torch.rand((B, S), generator=rng, device="cuda")
        rest[:, 0] = -1.0
        kept = torch.arange(S, device="cuda") < s["n_slots"][:, None]
        pick = torch.where(kept, rest.argsort(1), S).sort(1).values
        s["slots"] = torch.where(kept, pick, -1).to(torch.int32)
        # their positions are the last n_slots of the text
        rank = torch.where(kept, torch.arange(S, device="cuda"), 0)
        pos = torch.zeros((B, S), dtype=torch.int64, device="cuda")
        pos.scatter_(1, s["slots"].clamp(min=0).to(torch.int64) * kept, (text[:, None] - s["n_slots"][:, None] + rank) * kept)
        pos[:, 0] = text - s["n_slots"]
        s["pos"] = pos.to(torch.int32)
        s["weight"] = torch.zeros((B, max_blocks * bs), device="cuda")
        old = torch.arange(max_blocks * bs, device="cuda") < (s["lens"] - s["n_slots"])[:, None]
        s["weight"].masked_fill_(old, 1.0)
        s["weight"].mul_(torch.rand(s["weight"].shape, generator=rng, device="cuda"))
        s["lse"] = _lse_of_slots(s)
        return s
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
    if not case["inplace"]:
        s["temp"] = _normal(rng, (B, 1, 2, S, H, D), dtype)
    return s


def _prepare_evict(case, rng):
    B, L, H, D, bs = (case[k] for k in ("B", "layers", "H", "D", "block"))
    lens = _evict_lengths(case)
    max_blocks = -(-max(lens) // bs)
    table, blocks = _table(rng, lens, bs, max_blocks)
    width = max_blocks * bs
    s = dict(case, table=table, cache=_normal(rng, (L, 2, blocks, bs, H, D), DTYPES[case["dtype"]]),
             recent=max(1, case["len"] - case["budget"]), most=max(lens))
    # one buffer holds what the call updates per request, so that a copy of it
    # puts the batch back: lengths, positions, weights
    held = torch.zeros(B * (1 + 2 * width), dtype=torch.int32, device="cuda")
    held_len, held_pos, held_weight = _held(held, B)
    held_len.copy_(torch.tensor(lens))
    if case["again"]:  # thinned before: gaps, and older entries out of order
        pos = _thinned(rng, B, width)
        cut = min(case["budget"], width)
        swap = torch.rand((B, cut), generator=rng, device="cuda") < 0.1
        other = torch.rand((B, cut), generator=rng, device="cuda").argsort(1)
        key = torch.where(swap, other.double(), torch.arange(cut, device="cuda").double())
        pos[:, :cut] = pos[:, :cut].gather(1, key.argsort(dim=1, stable=True))
    else:
        pos = torch.arange(width, dtype=torch.int32, device="cuda").expand(B, width)
    valid = torch.arange(width, device="cuda") < held_len[:, None]
    held_pos.copy_(pos * valid)
    held_weight.copy_(torch.exp(1.5 * torch.randn((B, width), generator=rng, device="cuda")) * valid)
    s["held"] = held
    return s


def _held(held, B):
    """Lengths [B], positions [B][width] and weights [B][width] of a buffer."""
    width = (held.numel() // B - 1) // 2
    return (held[:B], held[B:B + B * width].view(B, width),
            held[B + B * width:].view(torch.float32).view(B, width))


def _evict_lengths(case):
    """Lengths from half an overrun below the budget up to `len`."""
    n, over = case["len"], case["len"] - case["budget"]
    if not case["ragged"]:
        return [n] * case["B"]
    lo = max(1, case["budget"] - over // 2)
    return [n if b == 0 else lo + (b * 2654435761 % 4294967296) * (n + 1 - lo) // 4294967296
            for b in range(case["B"])]


def prepare(case, seed):
    rng = torch.Generator(device="cuda").manual_seed(seed)
    return _prepare_evict(case, rng) if case["op"] == "evict" else _prepare_attention(case, rng)


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _pages(plane, table, first_block, count):
    """[B, count*block, H, D] in 32 bits: entries of the table's blocks from first_block on."""
    rows = plane[table[:, first_block:first_block + count].long()]
    return rows.float().flatten(1, 2)


def _score(s, dots, qp, kp, visible):
    """dots [B,H,G,S,N] -> masked scores; qp [B,S], kp [B,N] (or [1,N]), visible [B,S,N] or [B,1,N]."""
    x = dots.mul_(s["scale"])
    if s["cap"]:
        x = s["cap"] * torch.tanh(x / s["cap"])
    dist = qp[:, :, None] - kp[:, None, :]
    if s["slopes"] is not None:
        x = x - s["slopes"].view(1, s["H"], s["G"], 1, 1) * dist[:, None, None].float()
    if s["window"]:
        visible = visible & (dist < s["window"])
    if s["first"] is not None:
        visible = visible & (kp >= s["first"][:, None])[:, None, :]
    return x.masked_fill_(~visible[:, None, None], -math.inf)


def _plain_attention(s):
    B, S, H, G, D, bs, P = s["B"], s["S"], s["H"], s["G"], s["D"], s["block"], s["shared"]
    q = s["q"].float().view(B, S, H, G, D).permute(0, 2, 3, 1, 4)  # [B,H,G,S,D]
    lens = s["lens"].long()[:, None]
    qp = s["pos"].long() if s["pos"] is not None else lens + torch.arange(S, device="cuda")
    kc, vc = s["cache"][0, 0], s["cache"][0, 1]
    # own entries: from the shared prefix's last block on
    b0 = P // bs
    nblk = s["table"].shape[1] - b0
    k, v = _pages(kc, s["table"], b0, nblk), _pages(vc, s["table"], b0, nblk)
    at = torch.arange(b0 * bs, (b0 + nblk) * bs, device="cuda")[None]
    kp = s["key_pos"][:, b0 * bs:].long() if s["key_pos"] is not None else at.expand(B, -1)
    visible = ((at >= P) & (at < lens))[:, None, :].expand(B, S, -1)
    causal = torch.ones((S, S), dtype=torch.bool, device="cuda").tril()[None]
    if s["mask"] is not None:
        j = torch.arange(S, device="cuda")
        causal = (s["mask"][:, :, j // 32] >> (j % 32)) & 1 != 0
    if s["temp"] is not None:
        k = torch.cat([k, s["temp"][:, 0, 0].float()], 1)
        v = torch.cat([v, s["temp"][:, 0, 1].float()], 1)
        kp = torch.cat([kp, qp], 1)
        visible = torch.cat([visible, causal.expand(B, S, S)], 2)
    else:
        j = (at - lens).clamp(0, S - 1)                             # candidate held by an entry
        mine = (at >= lens) & (at < lens + S)
        seen = causal.expand(B, S, S).gather(2, j[:, None, :].expand(B, S, -1))
        visible = torch.where(mine[:, None, :], seen, visible)
        kp = torch.where(mine, qp.gather(1, j), kp)
    x = _score(s, torch.einsum("bhgsd,bnhd->bhgsn", q, k), qp, kp, visible)
    if P:
        ids = s["shared_table"].long()
        ks, vs = (p[ids].float().flatten(0, 1)[:P] for p in (kc, vc))
        at = torch.arange(P, device="cuda")[None]
        y = torch.einsum("bhgsd,nhd->bhgsn", q, ks)
        y = _score(s, y, qp, at, torch.ones((1, 1, P), dtype=torch.bool, device="cuda").expand(B, 1, P))
        x = torch.cat([y, x], -1)
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


def _slot_scores(s):
    """Masked scores [B,H,G,S,N] of the committed candidates, in commit order, against the entries."""
    B, S, H, G, D, P = s["B"], s["S"], s["H"], s["G"], s["D"], s["shared"]
    slots = s["slots"].long().clamp(min=0)
    q = s["q"].float().gather(1, slots[:, :, None, None].expand(B, S, H * G, D))
    q = q.view(B, S, H, G, D).permute(0, 2, 3, 1, 4)
    qp = s["pos"].long().gather(1, slots)
    lens, n = s["lens"].long()[:, None], s["n_slots"].long()[:, None]
    k = _pages(s["cache"][0, 0], s["table"], 0, s["table"].shape[1])
    at = torch.arange(k.shape[1], device="cuda")[None]
    kp = s["key_pos"].long() if s["key_pos"] is not None else at.expand(B, -1)
    j = (at - (lens - n)).clamp(0, S - 1)
    kp = torch.where((at >= lens - n) & (at < lens), qp.gather(1, j), kp)
    order = torch.arange(S, device="cuda")[None]
    last = torch.where(order < n, lens - n + order, -1)             # the candidate's own entry
    x = torch.einsum("bhgsd,bnhd->bhgsn", q, k)
    return _score(s, x, qp, kp, (at[:, None, :] <= last[:, :, None]) & (at >= P)[:, None, :]), slots, kp


def _lse_of_slots(s):
    """What the attention left for the committed candidates (the shared entries take part)."""
    whole = dict(s, shared=0)
    x, slots, _ = _slot_scores(whole)
    B, S, heads = s["B"], s["S"], s["H"] * s["G"]
    lse = torch.logsumexp(x, -1).permute(0, 3, 1, 2).reshape(B, S, heads)
    full = torch.zeros((B, S, heads), device="cuda")
    order = torch.arange(S, device="cuda")
    for j in range(S):
        rows = order[j] < s["n_slots"]
        full[rows, slots[rows, j]] = lse[rows, j]
    return full


def _plain_weights(s):
    x, slots, kp = _slot_scores(s)
    B, S, H, G = s["B"], s["S"], s["H"], s["G"]
    lse = s["lse"].gather(1, slots[:, :, None].expand(B, S, H * G))
    x = x.sub_(lse.view(B, S, H, G).permute(0, 2, 3, 1)[..., None]).exp_()
    done = {"weight": s["weight"] + x.sum((1, 2, 3))}
    if s["key_pos"] is not None:
        done["key_pos"] = kp.to(torch.int32)
    return done


def _plain_evict(s, lens, pos, weight):
    """New lengths, positions, weights and blocks in use; the cache in place."""
    B, bs, width, most = s["B"], s["block"], pos.shape[1], s["budget"]
    at = torch.arange(width, device="cuda")[None]
    valid = at < lens[:, None]
    newest = torch.where(valid, pos, -1).amax(1, keepdim=True)
    safe = valid & ((pos < s["sink"]) | (pos > newest - s["recent"]))
    order = torch.where(safe, math.inf, torch.where(valid, weight, -math.inf)).argsort(dim=1, descending=True, stable=True)
    rank = order.argsort(dim=1)
    kept = valid & (rank < most)
    hole, fill = (~kept & (at < most) & (lens[:, None] > most)).nonzero(), (kept & (at >= most)).nonzero()
    (hb, hi), (fb, fi) = hole.T, fill.T
    cache = s["cache"]
    cache[:, :, s["table"][hb, hi // bs].long(), hi % bs] = cache[:, :, s["table"][fb, fi // bs].long(), fi % bs]
    pos[hb, hi], weight[hb, hi] = pos[fb, fi], weight[fb, fi]
    now = lens.clamp(max=most)
    weight.masked_fill_(at >= now[:, None], 0.0)
    pos.masked_fill_(at >= now[:, None], 0)
    lens.copy_(now)
    return {"cache": cache, "len": lens, "pos": pos, "weight": weight,
            "blocks": ((now + bs - 1) // bs).to(torch.int32)}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _score_args(s):
    return dict(pos=s["pos"], key_pos=s["key_pos"], first_pos=s["first"], slopes=s["slopes"], scale=s["scale"],
                softcap=s["cap"], window=s["window"])


def run(s):
    if own:
        from speculative_decoding_verification_37_gb300 import api
    if s["op"] == "attention":
        if not own:
            return _plain_attention(s)
        shared = dict(shared_table=s["shared_table"], shared_len=s["shared"]) if s["shared"] else {}
        r = api.verify_attention(s["q"], s["cache"], s["table"], s["lens"], block_size=s["block"],
                                 temp_kv=s["temp"], tree_mask=s["mask"], **_score_args(s), **shared)
        return {"out": r.out, "lse": r.lse}
    if s["op"] == "weights":
        if not own:
            return _plain_weights(s)
        weight = s["weight"].clone()
        api.attention_weights(s["q"], s["lse"], s["cache"], s["table"], s["lens"], s["n_slots"], weight,
                              block_size=s["block"], slots=s["slots"], shared_len=s["shared"], **_score_args(s))
        return {"weight": weight} if s["key_pos"] is None else {"weight": weight, "key_pos": s["key_pos"]}
    lens, pos, weight = _held(s["held"].clone(), s["B"])
    if not own:
        return _plain_evict(s, lens, pos, weight)
    blocks = torch.empty_like(lens)
    api.evict_kv(s["cache"], s["table"], lens, weight, pos, block_size=s["block"], budget=s["budget"],
                 sink=s["sink"], recent=s["recent"], blocks_in_use=blocks)
    return {"cache": s["cache"], "len": lens, "pos": pos, "weight": weight, "blocks": blocks}


# ---------------------------------------------------------------------------
# the work of a pass
# ---------------------------------------------------------------------------
def _seen(case, total, S):
    """Cached entries the queries of a request can see, by count."""
    if case["gaps"]:
        return total
    return min(total, case["window"] + S) if case["window"] else total


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    B, H, D = case["B"], case["H"], case["D"]
    if case["op"] == "evict":
        lens = _evict_lengths(case)
        moved = sum(max(0, n - case["budget"]) for n in lens)
        return {"bytes": 2 * moved * case["layers"] * 2 * H * D * e + sum(lens) * 8, "flops": 0}
    S, G, P = case["S"], case["G"], case["shared"]
    docs = 0.75 if case["docs"] else 1.0     # the document starts a quarter in, on average
    if case["op"] == "weights":
        lens = _lengths(case, S)
        n = sum(_seen(case, max(0, t - min(P, min(lens))), S) for t in lens) * docs
        rows = sum(_slots_of(case)) / B * G
        return {"bytes": n * H * D * e + sum(_slots_of(case)) * G * H * (D * e + 4) + 8 * n, "flops": n * H * rows * D * 2}
    n = sum(_seen(case, P + t, S) for t in _lengths(case, 1)) * docs
    once = _seen(case, P, S) if P else 0
    unique = n - max(0, B - 1) * once if P else n
    rows = B * S * G * H
    return {"bytes": (max(unique, 0) + B * S) * H * D * 2 * e + rows * (2 * D * e + 4),
            "flops": (n + B * S) * H * S * G * D * 4}


# ---------------------------------------------------------------------------
# 64 bits, a request at a time, from the definition
# ---------------------------------------------------------------------------
def _entry_rows(s, b, plane, lo, hi):
    i = torch.arange(lo, hi, device="cuda")
    return plane[s["table"][b].long()[i // s["block"]], i % s["block"]].double()


def _exact_scores(s, qb, keys, qp, kp, allowed):
    """qb [R,heads,D], keys [N,H,D], qp [R], kp [N], allowed [R,N] -> [heads,R,N]."""
    heads, G = qb.shape[1], s["G"]
    rows = qb.permute(1, 0, 2).reshape(s["H"], -1, qb.shape[2])        # heads of one group are neighbours
    x = torch.bmm(rows, keys.permute(1, 2, 0)).reshape(heads, len(qp), len(kp)) * s["scale"]
    if s["cap"]:
        x = torch.tanh(x / s["cap"]) * s["cap"]
    gap = (qp[:, None] - kp[None, :]).double()
    if s["slopes"] is not None:
        x = x - s["slopes"].double()[:, None, None] * gap
    ok = allowed.clone()
    if s["window"]:
        ok &= gap < s["window"]
    if s["first_b"] is not None:
        ok &= kp[None, :] >= s["first_b"]
    return torch.where(ok, x, torch.full_like(x, -math.inf))


def _exact_attention(s):
    out, lses = [], []
    S, H, G, P = s["S"], s["H"], s["G"], s["shared"]
    kc, vc = s["cache"][0, 0], s["cache"][0, 1]
    if P:
        i = torch.arange(P, device="cuda")
        common = [p[s["shared_table"].long()[i // s["block"]], i % s["block"]].double() for p in (kc, vc)]
    for b, n in enumerate(s["lens"].tolist()):
        s["first_b"] = None if s["first"] is None else int(s["first"][b])
        qp = (torch.arange(n, n + S, device="cuda") if s["pos"] is None else s["pos"][b]).double()
        kp = (torch.arange(n, device="cuda") if s["key_pos"] is None else s["key_pos"][b, :n]).double()
        mine = [_entry_rows(s, b, p, P, n) for p in (kc, vc)]
        if s["temp"] is not None:
            new = [s["temp"][b, 0, i].double() for i in (0, 1)]
        else:
            new = [_entry_rows(s, b, p, n, n + S) for p in (kc, vc)]
        k, v = (torch.cat(([common[i]] if P else []) + [mine[i], new[i]]) for i in (0, 1))
        allowed = torch.ones((S, n + S), dtype=torch.bool, device="cuda")
        if s["mask"] is None:
            allowed[:, n:] = torch.tril(allowed[:, n:])
        else:
            words = s["mask"][b].tolist()
            allowed[:, n:] = torch.tensor([[bool(words[i][j // 32] >> (j % 32) & 1) for j in range(S)] for i in range(S)], device="cuda")
        x = _exact_scores(s, s["q"][b].double(), k, qp, torch.cat([kp, qp]), allowed)
        lse = torch.logsumexp(x, -1)
        p = torch.exp(x - torch.where(lse.isinf(), 0.0, lse)[..., None])
        o = torch.bmm(p.reshape(H, G * S, -1), v.permute(1, 0, 2)).reshape(H * G, S, -1)
        out.append(o.permute(1, 0, 2))
        lses.append(lse.T)
    return {"out": torch.stack(out), "lse": torch.stack(lses)}


def _exact_weights(s):
    w, kept = s["weight"].double(), s["key_pos"]
    for b, n in enumerate(s["lens"].tolist()):
        s["first_b"] = None if s["first"] is None else int(s["first"][b])
        m = int(s["n_slots"][b])
        slots = s["slots"][b, :m].long()
        qp = s["pos"][b, slots].double()
        kp = (torch.arange(n, device="cuda") if s["key_pos"] is None else s["key_pos"][b, :n]).double()
        kp[n - m:] = qp
        if kept is not None:
            kept[b, n - m:n] = qp.to(torch.int32)
        own_entry = torch.arange(n - m, n, device="cuda")
        allowed = torch.arange(n, device="cuda")[None] <= own_entry[:, None]
        x = _exact_scores(s, s["q"][b, slots].double(), _entry_rows(s, b, s["cache"][0, 0], 0, n), qp, kp, allowed)
        p = torch.exp(x - s["lse"][b, slots].double().T[..., None]).sum((0, 1))
        w[b, s["shared"]:n] += p[s["shared"]:]
    return {"weight": w} if kept is None else {"weight": w, "key_pos": kept}


def _exact_evict(s):
    bs, most = s["block"], s["budget"]
    lens, pos, weight = _held(s["held"].cpu(), s["B"])
    cache, table, blocks = s["cache"], s["table"].cpu(), []
    for b, n in enumerate(lens.tolist()):
        if n > most:
            p, w = pos[b, :n].tolist(), weight[b, :n].tolist()
            newest = max(p)
            safe = [i for i in range(n) if p[i] < s["sink"] or p[i] > newest - s["recent"]]
            others = sorted(set(range(n)) - set(safe), key=lambda i: (-w[i], i))
            kept = set(safe) | set(others[:most - len(safe)])
            holes = [i for i in range(most) if i not in kept]
            fills = [i for i in range(most, n) if i in kept]
            src, dst = (torch.tensor(v, dtype=torch.int64) for v in (fills, holes))
            sb, db = (table[b, v // bs].long().cuda() for v in (src, dst))
            cache[:, :, db, (dst % bs).cuda()] = cache[:, :, sb, (src % bs).cuda()]
            pos[b, dst], weight[b, dst] = pos[b, src], weight[b, src]
            lens[b] = most
        pos[b, int(lens[b]):] = 0
        weight[b, int(lens[b]):] = 0
        blocks.append(-(-int(lens[b]) // bs))
    return {"cache": cache, "len": lens, "pos": pos, "weight": weight.double(), "blocks": torch.tensor(blocks, dtype=torch.int32)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "evict":
        return _exact_evict(s)
    return _exact_weights(s) if case["op"] == "weights" else _exact_attention(s)
