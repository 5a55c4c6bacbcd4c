"""The attention, entry-weight and eviction entry points on the CPU: struct
layouts, workspace sizes and the refusals, all before anything is enqueued."""
import contextlib
import ctypes
import os
import subprocess
import tempfile

import pytest
import torch

from conftest import ROOT
from speculative_decoding_verification_37_gb300 import _lib as L
from speculative_decoding_verification_37_gb300 import api
from speculative_decoding_verification_37_gb300 import build as B

HEADER = os.path.join(ROOT, "include", "spec_verify.h")


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.lib()


def test_struct_layouts_match_c():
    structs = {"SpecAttentionArgs": L.SpecAttentionArgs, "SpecWeightsArgs": L.SpecWeightsArgs,
               "SpecEvictArgs": L.SpecEvictArgs}
    lines = []
    for name, cls in structs.items():
        lines.append('printf("%s %%zu\\n", sizeof(%s));' % (name, name))
        lines += ['printf("%s.%s %%zu\\n", offsetof(%s, %s));' % (name, f, name, f) for f, _ in cls._fields_]
    src = "#include <stdio.h>\n#include <stddef.h>\n#include \"spec_verify.h\"\nint main(void) {\n%s\nreturn 0; }\n" % "\n".join(lines)
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "l.c"), os.path.join(d, "l")
        open(c, "w").write(src)
        subprocess.run(["gcc", "-I", os.path.dirname(HEADER), c, "-o", exe], check=True)
        out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout
    for line in out.split("\n"):
        if line:
            key, val = line.split()
            s, _, f = key.partition(".")
            assert int(val) == (getattr(structs[s], f).offset if f else ctypes.sizeof(structs[s])), key


def test_workspace_sizes(lib):
    one = L.spec_workspace_bytes(L.SPEC_WS_ATTENTION, 4, 20, 128)
    assert one == L.spec_workspace_bytes(L.SPEC_WS_ATTENTION, 400, 20, 128) > 256
    shared = L.spec_workspace_bytes(L.SPEC_WS_ATTENTION_SHARED, 4, 20, 128)
    assert shared >= one + 4 * 20 * (128 + 1) * 4
    # a request's moves: at most what lies past the budget, or below it
    ev = lambda budget, cap: L.spec_workspace_bytes(L.SPEC_WS_EVICT, 3, budget, cap)  # noqa: E731
    assert ev(100, 100) <= 512 + 256 and ev(100, 130) >= 3 * 30 * 8 and ev(10, 1000) < 3 * 20 * 8 + 1024


def attention(**over):
    a = L.SpecAttentionArgs(B=2, S=3, Hq=4, H=2, D=64, L=2, layer=1, dtype=L.SPEC_DTYPE_BF16, q=4096,
                            q_stride_b=768, q_stride_s=256, q_stride_h=64, cache=4096, num_blocks=9, block_size=16,
                            max_blocks=4, block_table=4096, committed_len=4096, scale=0.125, out=4096, lse=4096)
    for k, v in over.items():
        setattr(a, k, v)
    return a


def weights(**over):
    a = L.SpecWeightsArgs(B=2, S=3, Hq=4, H=2, D=64, L=2, layer=1, dtype=L.SPEC_DTYPE_BF16, q=4096, q_stride_b=768,
                          q_stride_s=256, q_stride_h=64, lse=4096, cache=4096, num_blocks=9, block_size=16,
                          max_blocks=4, block_table=4096, committed_len=4096, n_slots=4096, scale=0.125,
                          weight=4096, weight_stride=64)
    for k, v in over.items():
        setattr(a, k, v)
    return a


def evict(**over):
    a = L.SpecEvictArgs(B=2, L=2, H=2, D=64, block_size=16, elem_bytes=2, cache=4096, num_blocks=9, block_table=4096,
                        max_blocks=4, budget=20, sink=2, recent=4, committed_len=4096, weight=4096, weight_stride=64,
                        key_pos=4096, key_pos_stride=64)
    for k, v in over.items():
        setattr(a, k, v)
    return a


NAN, INF = float("nan"), float("inf")
SCORED = [dict(B=-1), dict(B=32769), dict(S=0), dict(S=1025), dict(H=0), dict(Hq=0), dict(Hq=5), dict(D=0),
          dict(L=0), dict(layer=-1), dict(layer=2), dict(dtype=2), dict(block_size=0), dict(max_blocks=0),
          dict(num_blocks=0), dict(scale=NAN), dict(scale=INF), dict(softcap=-1.0), dict(softcap=NAN),
          dict(softcap=INF), dict(softcap=1e-45), dict(window=-1), dict(shared_len=-1), dict(shared_len=65),
          dict(key_pos=4096, key_pos_stride=63), dict(q=None), dict(cache=None), dict(block_table=None),
          dict(committed_len=None), dict(q=4104), dict(cache=4100), dict(q_stride_b=4), dict(q_stride_s=7),
          dict(q_stride_h=65)]


def refused(lib, fn, a, nbytes=1 << 28):
    # no kernel may start: on a host without a GPU it would return SPEC_ERR_CUDA
    return getattr(lib, fn)(ctypes.byref(a), ctypes.c_void_p(4096), nbytes, None)


@pytest.mark.parametrize("bad", SCORED + [
    dict(out=None), dict(out=4104), dict(temp_kv=4104), dict(shared_len=8), dict(shared_len=8, shared_table=4096,
                                                                                key_pos=4096, key_pos_stride=64)])
def test_attention_refusals(lib, bad):
    assert refused(lib, "spec_verify_attention", attention(**bad)) == L.SPEC_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", SCORED + [
    dict(lse=None), dict(n_slots=None), dict(weight=None), dict(weight_stride=63), dict(slots=4096, slots_stride=2)])
def test_weights_refusals(lib, bad):
    assert refused(lib, "spec_attention_weights", weights(**bad)) == L.SPEC_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [
    dict(B=-1), dict(B=32769), dict(L=0), dict(H=0), dict(D=0), dict(block_size=0), dict(num_blocks=0),
    dict(max_blocks=0), dict(elem_bytes=3), dict(budget=0), dict(sink=-1), dict(recent=-1), dict(sink=10, recent=11),
    dict(weight_stride=63), dict(key_pos_stride=63), dict(cache=None), dict(cache=4104), dict(block_table=None),
    dict(committed_len=None), dict(weight=None), dict(key_pos=None)])
def test_evict_refusals(lib, bad):
    assert refused(lib, "spec_evict_kv", evict(**bad)) == L.SPEC_ERR_INVALID_ARG


def test_unsupported_sizes_and_workspaces(lib):
    for fn, make in (("spec_verify_attention", attention), ("spec_attention_weights", weights)):
        for bad in (dict(D=260), dict(D=12), dict(max_blocks=1 << 30, weight_stride=1 << 40) if make is weights else
                    dict(max_blocks=1 << 30)):
            assert refused(lib, fn, make(**bad)) == L.SPEC_ERR_UNSUPPORTED, bad
        assert getattr(lib, fn)(None, None, 0, None) == L.SPEC_ERR_INVALID_ARG
        assert getattr(lib, fn)(ctypes.byref(make()), None, 1 << 28, None) == L.SPEC_ERR_INVALID_ARG
        assert getattr(lib, fn)(ctypes.byref(make()), ctypes.c_void_p(4096), 64, None) == L.SPEC_ERR_INVALID_ARG
        assert getattr(lib, fn)(ctypes.byref(make()), ctypes.c_void_p(4097), 1 << 28, None) == L.SPEC_ERR_INVALID_ARG
        assert getattr(lib, fn)(ctypes.byref(make(B=0, q=None)), None, 0, None) == L.SPEC_OK
    assert refused(lib, "spec_verify_attention", attention(shared_len=8, shared_table=4096),
                   L.spec_workspace_bytes(L.SPEC_WS_ATTENTION, 2, 12, 64)) == L.SPEC_ERR_INVALID_ARG
    assert refused(lib, "spec_evict_kv", evict(D=65, H=1)) == L.SPEC_ERR_UNSUPPORTED
    assert refused(lib, "spec_evict_kv", evict(), 300) == L.SPEC_ERR_INVALID_ARG
    assert lib.spec_evict_kv(ctypes.byref(evict(B=0)), None, 0, None) == L.SPEC_OK


def test_binding_refuses_cpu_tensors_and_wrong_shapes(lib):
    from speculative_decoding_verification_37_gb300 import api
    cache = torch.zeros((1, 2, 4, 16, 2, 64), dtype=torch.bfloat16)
    table, lens = torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    q = torch.zeros((1, 3, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA device"):
        api.verify_attention(q, cache, table, lens, block_size=16)
    with pytest.raises(ValueError, match="CUDA device"):
        api.attention_weights(q, torch.zeros((1, 3, 4)), cache, table, lens, lens, torch.zeros((1, 32)), block_size=16)
    with pytest.raises(ValueError, match="CUDA device"):
        api.evict_kv(cache, table, lens, torch.zeros((1, 32)), torch.zeros((1, 32), dtype=torch.int32), block_size=16,
                     budget=4)
    # the checks of shape and type themselves
    cpu, i32 = cache.device, torch.int32
    with pytest.raises(ValueError, match="cache must be contiguous"):
        L._cache_shape("f", cache, 8)
    with pytest.raises(ValueError, match="CUDA device"):
        L._cache_shape("f", cache, 16)
    with pytest.raises(TypeError, match="block_table must be"):
        L._checked("f", "block_table", table.long(), i32, (1, 2), cpu)
    with pytest.raises(ValueError, match="committed_len has shape"):
        L._checked("f", "committed_len", torch.zeros(2, dtype=i32), i32, (1,), cpu)
    with pytest.raises(ValueError, match="must be contiguous"):
        L._checked("f", "pos", torch.zeros((3, 2), dtype=i32).T, i32, (2, 3), cpu)
    with pytest.raises(ValueError, match="is on cpu"):
        L._checked("f", "pos", torch.zeros((2, 3), dtype=i32), i32, (2, 3), torch.device("meta"))
    assert L._checked("f", "pos", None, i32, (2, 3), cpu) is None
    assert L._checked("f", "t", table, i32, (-1, 2), cpu) == table.data_ptr()
    with pytest.raises(ValueError, match="contiguous rows"):
        L._rows("f", "weight", torch.zeros((1, 31)), torch.float32, 1, 32, cpu)
    with pytest.raises(ValueError, match="contiguous rows"):
        L._rows("f", "weight", torch.zeros((32, 2)).T, torch.float32, 2, 32, cpu)
    wide = torch.zeros((2, 40))
    assert L._rows("f", "weight", wide[:, 3:36], torch.float32, 2, 32, cpu) == (wide.data_ptr() + 12, 40)
    with pytest.raises(TypeError, match="q is"):
        L._query_strides("f", q.float(), cache, 1)
    with pytest.raises(ValueError, match="contiguous last dimension"):
        L._query_strides("f", q.transpose(2, 3), cache, 1)
    assert L._query_strides("f", q, cache, 1) == [0, 256, 64]


def test_softcaps_that_the_arithmetic_does_not_hold(lib):
    """A bf16 cap past 1024 would round the scores; one far below the scale overflows."""
    for fn, make in (("spec_verify_attention", attention), ("spec_attention_weights", weights)):
        assert refused(lib, fn, make(softcap=1025.0)) == L.SPEC_ERR_UNSUPPORTED
        assert refused(lib, fn, make(softcap=1e-30, scale=1e10)) == L.SPEC_ERR_INVALID_ARG


def test_binding_refuses_integers_past_32_bits(monkeypatch):
    monkeypatch.setattr(L, "_cache_shape", lambda fn, cache, bs: cache.shape)  # a CPU cache, nothing is launched
    cache = torch.zeros(1, 2, 4, 16, 1, 64)
    q, lse, w = torch.zeros(2, 3, 1, 64), torch.zeros(2, 3, 1), torch.zeros(2, 32)
    kw = dict(cache=cache, block_table=torch.zeros(2, 2, dtype=torch.int32),
              committed_len=torch.zeros(2, dtype=torch.int32), block_size=16, workspace=torch.zeros(1))
    for bad in (dict(layer=1 << 32), dict(window=1 << 32), dict(window=-(1 << 31) - 1)):
        with pytest.raises(ValueError, match="32 bits"):
            L.spec_verify_attention(q=q, out=q, scale=1.0, **kw, **bad)
        with pytest.raises(ValueError, match="32 bits"):
            L.spec_attention_weights(q=q, lse=lse, n_slots=kw["committed_len"], weight=w, scale=1.0, **kw, **bad)
    with pytest.raises(ValueError, match="32 bits"):
        L.spec_verify_attention(q=q, out=q, scale=1.0, shared_len=1 << 32, **kw)
    for bad in (dict(budget=(1 << 32) + 20), dict(budget=8, sink=1 << 32), dict(budget=8, recent=1 << 32)):
        with pytest.raises(ValueError, match="32 bits"):
            L.spec_evict_kv(weight=w, key_pos=w.int(), **kw, **bad)


def test_a_captured_first_call_does_not_leave_its_workspace_in_the_cache(monkeypatch):
    """Under capture the zeroing only happens at a replay."""
    api.clear_workspaces()
    monkeypatch.setattr(L, "new_workspace", lambda *a, device: torch.zeros(1))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    a = api.workspace(L.SPEC_WS_ATTENTION, 1, 2, 64, torch.device("cuda", 0))
    b = api.workspace(L.SPEC_WS_ATTENTION, 1, 2, 64, torch.device("cuda", 0))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    c = api.workspace(L.SPEC_WS_ATTENTION, 1, 2, 64, torch.device("cuda", 0))
    d = api.workspace(L.SPEC_WS_ATTENTION, 1, 2, 64, torch.device("cuda", 0))
    api.clear_workspaces()
    assert len({id(x) for x in (a, b, c)}) == 3 and c is d


def test_a_workspace_for_each_stream(lib):
    """The kinds that hold a call's intermediate results are not shared between
    streams, whose calls may be in flight together; the others' only state is theirs."""
    api.clear_workspaces()
    for kind in (L.SPEC_WS_ATTENTION, L.SPEC_WS_ATTENTION_SHARED, L.SPEC_WS_EVICT):
        a, b, c = (api.workspace(kind, 2, 8, 64, "cpu", stream=s) for s in (0, 7, 7))
        assert b is c and a.data_ptr() != b.data_ptr() and a is api.workspace(kind, 2, 8, 64, "cpu")
        assert a.numel() >= L.spec_workspace_bytes(kind, 2, 8, 64) and not a[:L.SPEC_WS_ZEROED].any()
    assert api.workspace(L.SPEC_WS_COMMIT, 2, 0, 0, "cpu", stream=7) is api.workspace(L.SPEC_WS_COMMIT, 2, 0, 0, "cpu")
    api.clear_workspaces()


def test_calls_use_their_streams_workspace(lib, monkeypatch):
    """verify_attention and evict_kv on two streams: workspaces apart, the same
    one again on the same stream, the caller's own where it gives one."""
    used = []
    monkeypatch.setattr(L, "spec_verify_attention", lambda **kw: used.append((kw["workspace"], kw["stream"])))
    monkeypatch.setattr(L, "spec_evict_kv", lambda **kw: used.append((kw["workspace"], kw["stream"])))
    monkeypatch.setattr(api, "_allocating_on", lambda stream: contextlib.nullcontext())
    api.clear_workspaces()
    cache, table, lens = torch.zeros(1, 2, 4, 16, 1, 64), torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    q, w, pos = torch.zeros(2, 3, 1, 64), torch.zeros(2, 32), torch.zeros(2, 32, dtype=torch.int32)
    calls = (lambda **kw: api.verify_attention(q, cache, table, lens, block_size=16, **kw),
             lambda **kw: api.verify_attention(q, cache, table, lens, block_size=16, shared_len=5, shared_table=table[0], **kw),
             lambda **kw: api.evict_kv(cache, table, lens, w, pos, block_size=16, budget=8, **kw))
    for call in calls:
        used.clear()
        mine = torch.zeros(1)
        for kw in (dict(stream=3), dict(stream=4), dict(stream=3), dict(stream=4, ws=mine)):
            call(**kw)
        (a, s), (b, t), (c, _), (d, _) = used
        assert a is c and a.data_ptr() != b.data_ptr() and d is mine and (s, t) == (3, 4)
    api.clear_workspaces()


def test_every_captured_call_gets_a_workspace_of_its_own(monkeypatch):
    """Also after an eager call of its sizes, on the stream that captures: two
    graphs, or a graph and eager calls, can be in flight together."""
    api.clear_workspaces()
    monkeypatch.setattr(L, "new_workspace", lambda *a, device: torch.zeros(1))
    capturing = False
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing)
    dev = torch.device("cuda", 0)
    for kind in (L.SPEC_WS_ATTENTION, L.SPEC_WS_ATTENTION_SHARED, L.SPEC_WS_EVICT):
        eager = api.workspace(kind, 1, 2, 64, dev)
        capturing = True
        graphs = [api.workspace(kind, 1, 2, 64, dev) for _ in range(2)]
        capturing = False
        assert len({id(x) for x in (eager, *graphs)}) == 3 and api.workspace(kind, 1, 2, 64, dev) is eager
    api.clear_workspaces()


def test_a_stream_has_one_workspace_of_a_kind(lib):
    """Batches that grow and shrink, other heads, other budgets: one workspace of
    the largest size so far, with the status word of the one it replaced."""
    for kind, V in ((L.SPEC_WS_ATTENTION, 64), (L.SPEC_WS_ATTENTION_SHARED, 64), (L.SPEC_WS_EVICT, 2048)):
        api.clear_workspaces()
        first = api.workspace(kind, 1, 8, V, "cpu", stream=5)
        first.view(torch.int32)[0] = 1
        other = api.workspace(kind, 1, 8, V, "cpu", stream=6)
        for B in list(range(1, 65)) + list(range(64, 0, -1)):
            for n, v in ((8, V), (40, V), (300, 2 * V)):
                w = api.workspace(kind, B, n, v, "cpu", stream=5)
                assert w.numel() >= L.spec_workspace_bytes(kind, B, n, v) and w.view(torch.int32)[0] == 1
        held = {w.data_ptr(): w.numel() for k, w in api._WORKSPACES.items() if k[-1] == 5}
        assert list(held.values()) == [L.spec_workspace_bytes(kind, 64, 300, 2 * V)]
        assert api.workspace(kind, 1, 8, V, "cpu", stream=5) is w and api.workspace(kind, 1, 8, V, "cpu", stream=6) is other
        assert not w[4:L.SPEC_WS_ZEROED].any() and other.view(torch.int32)[0] == 0
    api.clear_workspaces()
