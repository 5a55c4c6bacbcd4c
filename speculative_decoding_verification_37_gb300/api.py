"""Convenience layer over the C ABI: allocates outputs and workspaces with
torch and calls the library.  No arithmetic of the method happens here."""
from __future__ import annotations

from contextlib import nullcontext
from dataclasses import dataclass
from typing import Dict, Optional, Tuple

import torch

from . import _lib as L

_WORKSPACES: Dict[Tuple, torch.Tensor] = {}


# kinds that hold a call's intermediate results: one for each stream
_PER_STREAM = (L.SPEC_WS_ATTENTION, L.SPEC_WS_ATTENTION_SHARED, L.SPEC_WS_EVICT)


def workspace(kind: int, B: int, n: int, V: int, device, stream: Optional[int] = None) -> torch.Tensor:
    """A cached zero-filled workspace for (device, kind, B, n, V) (the size of
    some kinds depends on V).  Every call leaves it zeroed, so it is reused
    without clearing; calls that share it must be ordered on one stream.
    The cache lives as long as the process; clear_workspaces() frees it.
    A call captured into a CUDA graph before any eager one of its sizes gets a
    workspace of the graph's own, zeroed by each replay: a cached one would
    not be zero before the first replay.
    The attention's and the eviction's kinds (zero in the SPEC_WS_ZEROED bytes
    that have to be) are cached for each stream (the raw handle of a stream that
    is current; None: the current one), so that calls in flight on two streams do
    not meet; a stream has one of each kind, as large as its largest call so far
    wanted.  Every captured call gets its own: its graph may be replayed on any
    stream, beside eager calls and other graphs."""
    dev = device if isinstance(device, torch.device) else torch.device(device)
    if dev.type == "cuda" and dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    per_stream = kind in _PER_STREAM
    if per_stream and dev.type == "cuda" and torch.cuda.is_current_stream_capturing():
        return L.new_workspace(kind, B, n, V, device=dev)
    if not per_stream:
        stream = 0
    elif stream is None:  # (before CUDA's first use the default stream is current)
        on_gpu = dev.type == "cuda" and torch.cuda.is_initialized()
        stream = torch.cuda.current_stream(dev).cuda_stream if on_gpu else 0
    key = (dev.type, dev.index, kind, B, n, V, stream)
    ws = _WORKSPACES.get(key)
    if ws is None and per_stream:
        return _grown(key, dev)
    if ws is None:
        ws = L.new_workspace(kind, B, n, V, device=dev)
        if dev.type != "cuda" or not torch.cuda.is_current_stream_capturing():
            _WORKSPACES[key] = ws
    return ws


def _grown(key: Tuple, dev: torch.device) -> torch.Tensor:
    """The stream's workspace of this kind, kept under its sizes too; a larger one
    takes its place, status word included, where these sizes want it (the other
    parts are scratch, or zero between calls)."""
    kind, B, n, V, stream = key[2:]
    one = (dev.type, dev.index, kind, stream)
    old = _WORKSPACES.get(one)
    if old is None or old.numel() < L.spec_workspace_bytes(kind, B, n, V):
        ws = L.new_workspace(kind, B, n, V, device=dev)
        if old is not None:
            ws[:4].copy_(old[:4])
            for k in [k for k, x in _WORKSPACES.items() if x is old]:
                _WORKSPACES[k] = ws
        _WORKSPACES[one] = ws
    _WORKSPACES[key] = _WORKSPACES[one]
    return _WORKSPACES[one]


def clear_workspaces() -> None:
    """Drops every cached workspace (after the work using them has finished),
    e.g. after a timeout (SPEC_FLAG_TIMEOUT asks for a fresh workspace) or
    when batch shapes change for good."""
    _WORKSPACES.clear()


@dataclass
class ChainOut:
    n_acc: torch.Tensor                   # int32 [B]
    out_tokens: torch.Tensor              # int32 [B, gamma+1]
    n_out: torch.Tensor                   # int32 [B]
    accept_prob: Optional[torch.Tensor]   # f32 [B, gamma]
    residual_mass: Optional[torch.Tensor] # f32 [B, gamma]
    flags: torch.Tensor                   # uint32 stored as int32 [B]


def chain_workspace_kind(sampled: bool, top_k: int, V: int, residual_mass: bool = False) -> int:
    """The workspace kind that lets a chain call take its fastest path."""
    if not sampled:
        return L.SPEC_WS_CHAIN
    if 0 < top_k <= L.TOPK_FAST_MAX and top_k < V:
        return L.SPEC_WS_CHAIN_TOPK
    if (top_k == 0 or top_k >= V) and not residual_mass:
        return L.SPEC_WS_CHAIN_FULL
    return L.SPEC_WS_CHAIN


def verify_chain(target: torch.Tensor, draft_tokens: torch.Tensor, *, gamma: int,
                 temperature: float, draft: Optional[torch.Tensor] = None,
                 uniforms: Optional[torch.Tensor] = None, top_k: int = 0,
                 fallback_eps: float = 1e-6, accept_prob: bool = True,
                 residual_mass: bool = False, ws: Optional[torch.Tensor] = None,
                 committed_len: Optional[torch.Tensor] = None,
                 draft_len: Optional[torch.Tensor] = None,
                 blocks_in_use: Optional[torch.Tensor] = None, block_size: int = 0,
                 kv_capacity: int = 0, eos_token: Optional[int] = None,
                 max_new: Optional[torch.Tensor] = None, top_p: float = 0.0,
                 gamma_per_request: Optional[torch.Tensor] = None,
                 temperature_per_request: Optional[torch.Tensor] = None,
                 top_k_per_request: Optional[torch.Tensor] = None,
                 top_p_per_request: Optional[torch.Tensor] = None,
                 stream=None) -> ChainOut:
    """target [B*(gamma+1), V], draft [B*gamma, V] (bf16 or f32, rows may be
    strided), draft_tokens int32 [B, gamma], uniforms f32 [B, gamma+1].

    With committed_len (int32 [B], on the device) the call also commits the
    in-place K/V of the candidates: committed_len advances by n_out,
    draft_len (if given) is cut back to it and blocks_in_use (if given)
    follows, all on the device.  eos_token / max_new (int32 [B] on the
    device) end the round early: its output is cut right after the first
    EOS, then to max_new[b] tokens.  0 < top_p < 1 adds the nucleus after
    top-k.  The *_per_request tensors (on the device, [B]) give each request
    its own gamma (<= gamma; the arrays stay padded to gamma), temperature (0:
    greedy), top-k and top-p."""
    dev = target.device
    V = target.shape[-1]
    B = target.shape[0] // (gamma + 1)
    per_request = any(x is not None for x in (gamma_per_request, temperature_per_request,
                                               top_k_per_request, top_p_per_request))
    sampled = temperature > 0 or temperature_per_request is not None
    out = ChainOut(
        n_acc=torch.empty(B, dtype=torch.int32, device=dev),
        out_tokens=torch.full((B, gamma + 1), -1, dtype=torch.int32, device=dev),
        n_out=torch.empty(B, dtype=torch.int32, device=dev),
        accept_prob=torch.empty((B, gamma), dtype=torch.float32, device=dev)
        if (sampled and accept_prob) else None,
        residual_mass=torch.empty((B, gamma), dtype=torch.float32, device=dev)
        if (sampled and residual_mass) else None,
        flags=torch.zeros(B, dtype=torch.int32, device=dev))
    if ws is None:
        kind = L.SPEC_WS_CHAIN if per_request else chain_workspace_kind(sampled, top_k, V, residual_mass)
        ws = workspace(kind, B, gamma, V, dev)
    L.spec_verify_chain(target_logits=target, draft_tokens=draft_tokens, n_acc=out.n_acc,
                        out_tokens=out.out_tokens, n_out=out.n_out, workspace=ws, gamma=gamma,
                        temperature=temperature, draft_logits=draft, uniforms=uniforms,
                        top_k=top_k, fallback_eps=fallback_eps, accept_prob=out.accept_prob,
                        residual_mass=out.residual_mass, flags=out.flags,
                        committed_len=committed_len, draft_len=draft_len,
                        blocks_in_use=blocks_in_use, block_size=block_size,
                        kv_capacity=kv_capacity, eos_token=eos_token, max_new=max_new,
                        top_p=top_p, gamma_per_request=gamma_per_request,
                        temperature_per_request=temperature_per_request,
                        top_k_per_request=top_k_per_request, top_p_per_request=top_p_per_request,
                        stream=stream)
    return out


@dataclass
class TreeOut:
    path: torch.Tensor          # int32 [B, N]
    n_acc: torch.Tensor         # int32 [B]
    out_tokens: torch.Tensor    # int32 [B, N+1]
    n_out: torch.Tensor         # int32 [B]
    tree_mask: torch.Tensor     # int32 view of uint32 [B, N+1, W]
    pos: torch.Tensor           # int32 [B, N+1]
    commit_slots: torch.Tensor  # int32 [B, N+1]
    n_commit: torch.Tensor      # int32 [B]
    flags: torch.Tensor         # int32 [B]


def verify_tree(logits: torch.Tensor, node_token: torch.Tensor, node_parent: torch.Tensor,
                row_of_node: torch.Tensor, committed_len: torch.Tensor, *, R: int,
                ws: Optional[torch.Tensor] = None, stream=None) -> TreeOut:
    dev = logits.device
    V = logits.shape[-1]
    B = logits.shape[0] // R
    N = node_token.shape[-1]
    W = (N + 1 + 31) // 32
    i32 = dict(dtype=torch.int32, device=dev)
    out = TreeOut(path=torch.full((B, N), -1, **i32), n_acc=torch.empty(B, **i32),
                  out_tokens=torch.full((B, N + 1), -1, **i32), n_out=torch.empty(B, **i32),
                  tree_mask=torch.zeros((B, N + 1, W), **i32), pos=torch.empty((B, N + 1), **i32),
                  commit_slots=torch.full((B, N + 1), -1, **i32), n_commit=torch.empty(B, **i32),
                  flags=torch.zeros(B, **i32))
    if ws is None:
        ws = workspace(L.SPEC_WS_TREE, B, R, V, dev)
    L.spec_verify_tree(logits=logits, R=R, node_token=node_token, node_parent=node_parent,
                       row_of_node=row_of_node, path=out.path, n_acc=out.n_acc,
                       out_tokens=out.out_tokens, n_out=out.n_out, workspace=ws,
                       committed_len=committed_len, tree_mask=out.tree_mask, pos=out.pos,
                       commit_slots=out.commit_slots, n_commit=out.n_commit, flags=out.flags,
                       stream=stream)
    return out


def commit_kv(temp_kv: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor,
              n_slots: torch.Tensor, committed_len: torch.Tensor, *, block_size: int,
              slots: Optional[torch.Tensor] = None, blocks_in_use: Optional[torch.Tensor] = None,
              flags: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
              stream=None) -> None:
    """Commits in place: cache and committed_len are updated on the device."""
    if ws is None:
        ws = workspace(L.SPEC_WS_COMMIT, temp_kv.shape[0], 0, 0, temp_kv.device)
    L.spec_commit_kv(temp_kv=temp_kv, cache=cache, block_table=block_table, n_slots=n_slots,
                     committed_len=committed_len, block_size=block_size, workspace=ws,
                     slots=slots, blocks_in_use=blocks_in_use, flags=flags, stream=stream)


def _allocating_on(stream):
    """Context in which outputs and a first workspace are allocated (and the
    workspace zeroed) on the stream the call runs on."""
    if stream is None:
        return nullcontext()
    return torch.cuda.stream(stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream)))


def _stream_of(stream, t: torch.Tensor):
    """The stream a call runs on (the current one of t's device for None) and its raw handle."""
    if stream is None:
        if not t.is_cuda:  # (the call refuses it)
            return None, 0
        stream = torch.cuda.current_stream(t.device)
    return stream, stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


@dataclass
class AttentionOut:
    out: torch.Tensor            # [B, S, Hq, D], q's type
    lse: torch.Tensor            # f32 [B, S, Hq]


def verify_attention(q: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor,
                     committed_len: torch.Tensor, *, block_size: int, layer: int = 0,
                     temp_kv: Optional[torch.Tensor] = None, tree_mask: Optional[torch.Tensor] = None,
                     pos: Optional[torch.Tensor] = None, key_pos: Optional[torch.Tensor] = None,
                     first_pos: Optional[torch.Tensor] = None, slopes: Optional[torch.Tensor] = None,
                     scale: Optional[float] = None, softcap: float = 0.0, window: int = 0,
                     shared_table: Optional[torch.Tensor] = None, shared_len: int = 0,
                     flags: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                     stream=None) -> AttentionOut:
    """One layer's attention of a round's candidates (the last emitted token
    and the drafts, or a tree's nodes) over the paged cache and the candidates
    themselves.

    q [B, S, Hq, D] (bf16 or f32, Hq a multiple of the cache's H; strides are
    free but for the last dimension's), cache [L, 2, num_blocks, block_size,
    H, D].  The candidates' K/V are temp_kv [B, L, 2, S, H, D], or without it
    the cache's entries committed_len[b] .. + S - 1.  tree_mask and pos as
    verify_tree returns them (without: a chain at committed_len[b] + i);
    key_pos int32 [B, max_blocks*block_size]: the entries' positions once some
    were evicted.  scale defaults to D**-0.5; softcap > 0 caps the scores by a
    tanh; slopes f32 [Hq] subtract slope * distance; window > 0 and first_pos
    (int32 [B]) mask by position.  With shared_len > 0 every request's first
    shared_len entries lie in shared_table's blocks and are read once for the
    whole batch.  A query that sees no key gets 0 and an lse of -inf.
    Calls on different streams, and captured ones, may be in flight together;
    with a ws of the caller's own only those that do not share it (a captured
    call's status word can be read only there)."""
    B, S, Hq, D = q.shape
    with _allocating_on(stream):
        out = AttentionOut(out=torch.empty((B, S, Hq, D), dtype=q.dtype, device=q.device),
                           lse=torch.empty((B, S, Hq), dtype=torch.float32, device=q.device))
        stream, raw = _stream_of(stream, q)
        if ws is None:
            ws = workspace(L.SPEC_WS_ATTENTION_SHARED if shared_len > 0 else L.SPEC_WS_ATTENTION, B, S * Hq, D, q.device, raw)
    L.spec_verify_attention(q=q, cache=cache, block_table=block_table, committed_len=committed_len,
                            block_size=block_size, out=out.out, lse=out.lse, workspace=ws, layer=layer,
                            scale=D ** -0.5 if scale is None else scale, temp_kv=temp_kv, tree_mask=tree_mask,
                            pos=pos, key_pos=key_pos, first_pos=first_pos, slopes=slopes, softcap=softcap,
                            window=window, shared_table=shared_table, shared_len=shared_len, flags=flags,
                            stream=stream)
    return out


def attention_weights(q: torch.Tensor, lse: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor,
                      committed_len: torch.Tensor, n_slots: torch.Tensor, weight: torch.Tensor, *,
                      block_size: int, layer: int = 0, slots: Optional[torch.Tensor] = None,
                      pos: Optional[torch.Tensor] = None, key_pos: Optional[torch.Tensor] = None,
                      first_pos: Optional[torch.Tensor] = None, slopes: Optional[torch.Tensor] = None,
                      scale: Optional[float] = None, softcap: float = 0.0, window: int = 0,
                      shared_len: int = 0, flags: Optional[torch.Tensor] = None,
                      ws: Optional[torch.Tensor] = None, stream=None) -> None:
    """After a commit, adds to weight (f32 [B, max_blocks*block_size], in
    place) what each cached entry got of the committed candidates' attention
    in one layer: n_slots and slots as passed to commit_kv, committed_len as it
    left it, q and lse those of verify_attention, and the same scoring
    arguments.  key_pos, if given, gets the new entries' positions."""
    if ws is None:
        with _allocating_on(stream):
            ws = workspace(L.SPEC_WS_COMMIT, q.shape[0], 0, 0, q.device)
    L.spec_attention_weights(q=q, lse=lse, cache=cache, block_table=block_table, committed_len=committed_len,
                             n_slots=n_slots, weight=weight, block_size=block_size, workspace=ws, layer=layer,
                             scale=q.shape[-1] ** -0.5 if scale is None else scale, slots=slots, pos=pos,
                             key_pos=key_pos, first_pos=first_pos, slopes=slopes, softcap=softcap,
                             window=window, shared_len=shared_len, flags=flags, stream=stream)


def evict_kv(cache: torch.Tensor, block_table: torch.Tensor, committed_len: torch.Tensor, weight: torch.Tensor,
             key_pos: torch.Tensor, *, block_size: int, budget: int, sink: int = 0, recent: int = 0,
             blocks_in_use: Optional[torch.Tensor] = None, flags: Optional[torch.Tensor] = None,
             ws: Optional[torch.Tensor] = None, stream=None) -> None:
    """Cuts every request with more than `budget` entries back to it, in place
    and in every layer: the entries at positions below `sink`, the `recent`
    newest positions and the heaviest others stay; those at or past the
    budget move into the places of the evicted ones.  cache, committed_len,
    weight and key_pos are updated on the device.  Streams, captures and ws as
    for verify_attention."""
    if ws is None:
        with _allocating_on(stream):
            stream, raw = _stream_of(stream, cache)
            ws = workspace(L.SPEC_WS_EVICT, block_table.shape[0], budget, block_table.shape[1] * block_size, cache.device, raw)
    L.spec_evict_kv(cache=cache, block_table=block_table, committed_len=committed_len, weight=weight,
                    key_pos=key_pos, block_size=block_size, budget=budget, workspace=ws, sink=sink, recent=recent,
                    blocks_in_use=blocks_in_use, flags=flags, stream=stream)


@dataclass
class NgramOut:
    draft_tokens: torch.Tensor   # int32 [B, gamma], -1 past n_draft
    n_draft: torch.Tensor        # int32 [B]
    match_n: torch.Tensor        # int32 [B], 0 if no match
    match_start: torch.Tensor    # int32 [B], -1 if no match
    flags: torch.Tensor          # int32 [B]


def ngram_draft(history: torch.Tensor, hist_len: torch.Tensor, *, gamma: int, n_min: int = 1,
                n_max: int = 4, stream=None) -> NgramOut:
    """Prompt-lookup drafts: history int32 [B, max_len] on the device (row b's
    first hist_len[b] tokens are its history)."""
    dev = history.device
    B = history.shape[0]
    i32 = dict(dtype=torch.int32, device=dev)
    out = NgramOut(draft_tokens=torch.empty((B, gamma), **i32), n_draft=torch.empty(B, **i32),
                   match_n=torch.empty(B, **i32), match_start=torch.empty(B, **i32),
                   flags=torch.empty(B, **i32))
    L.spec_ngram_draft(history=history, hist_len=hist_len, gamma=gamma, n_min=n_min, n_max=n_max,
                       draft_tokens=out.draft_tokens, n_draft=out.n_draft, match_n=out.match_n,
                       match_start=out.match_start, flags=out.flags, stream=stream)
    return out


class TreeBuilder:
    """Builds draft trees for B requests one level at a time on the device
    (topKSpec / topHead shape).  Between levels the caller runs the draft
    model at ``next_parents`` and passes its logits rows, in that order, to
    the next ``level`` call.  Node arrays follow the tree verify's layout:
    node_token / node_parent [B, N] (node id i at index i-1), node_logp /
    row_of_node [B, N+1] (indexed by node id, the root is 0)."""

    def __init__(self, B: int, V: int, topKSpec, topHead, device, flags: bool = True):
        if len(topKSpec) != len(topHead) or not len(topHead) or topHead[0] != 1:
            raise ValueError("topHead must start with 1 (the root) and match topKSpec")
        self.B, self.V = B, V
        self.topKSpec = [list(map(int, ks)) for ks in topKSpec]
        self.topHead = list(map(int, topHead))
        self.N = sum(sum(ks) for ks in self.topKSpec)
        dev = torch.device(device)
        i32 = dict(dtype=torch.int32, device=dev)
        self.node_token = torch.full((B, self.N), -1, **i32)
        self.node_parent = torch.full((B, self.N), -1, **i32)
        self.node_logp = torch.zeros((B, self.N + 1), dtype=torch.float32, device=dev)
        self.row_of_node = torch.full((B, self.N + 1), -1, **i32)
        self.flags = torch.zeros(B, **i32) if flags else None
        self.next = [torch.empty((B, h), **i32) for h in self.topHead[1:]] + [None]
        self.ws = [workspace(L.SPEC_WS_TREE_LEVEL, B, h, V, dev) for h in self.topHead]
        self.level_index = 0

    def level(self, logits: torch.Tensor, i: Optional[int] = None, stream=None) -> Optional[torch.Tensor]:
        """Expand level i (default: the next one) from its draft rows
        [B*topHead[i], V]; returns the next level's parents [B, topHead[i+1]]
        (None after the last level)."""
        i = self.level_index if i is None else i
        H = self.topHead[i]
        n_before = sum(sum(ks) for ks in self.topKSpec[:i])
        next_row0 = sum(self.topHead[:i + 1])
        n_next = self.topHead[i + 1] if i + 1 < len(self.topHead) else 0
        L.spec_tree_level(logits=logits, H=H, k=self.topKSpec[i], n_next=n_next, n_before=n_before,
                          next_row0=next_row0, node_token=self.node_token,
                          node_parent=self.node_parent, node_logp=self.node_logp,
                          row_of_node=self.row_of_node, workspace=self.ws[i],
                          parents=None if i == 0 else self.next[i - 1],
                          next_parents=self.next[i], flags=self.flags, stream=stream)
        self.level_index = i + 1
        return self.next[i]
