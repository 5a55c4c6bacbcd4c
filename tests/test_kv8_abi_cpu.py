"""The 8-bit cache's entry points on the CPU: struct layouts, workspace sizes and
the refusals, all before anything is enqueued."""
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

STRUCTS = {"SpecWriteKvQ8Args": L.SpecWriteKvQ8Args, "SpecAttentionQ8Args": L.SpecAttentionQ8Args,
           "SpecCommitKvQ8Args": L.SpecCommitKvQ8Args, "SpecReadKvQ8Args": L.SpecReadKvQ8Args}


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.lib()


def test_struct_layouts_match_c():
    lines = []
    for name, cls in STRUCTS.items():
        lines.append('printf("%s %%zu\\n", sizeof(%s));' % (name, name))
        lines += ['printf("%s.%s %%zu\\n", offsetof(%s, %s));' % (name, f, name, f) for f, _ in cls._fields_]
    src = "#include <stdio.h>\n#include <stddef.h>\n#include \"spec_verify.h\"\nint main(void) {\n%s\nreturn 0; }\n" % "\n".join(lines)
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "l.c"), os.path.join(d, "l")
        open(c, "w").write(src)
        subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), c, "-o", exe], check=True)
        out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout
    seen = 0
    for line in filter(None, out.split("\n")):
        key, val = line.split()
        s, _, f = key.partition(".")
        assert int(val) == (getattr(STRUCTS[s], f).offset if f else ctypes.sizeof(STRUCTS[s])), key
        seen += 1
    assert seen == sum(1 + len(c._fields_) for c in STRUCTS.values())


COMMON = dict(B=2, S=3, H=2, D=64, L=2, num_blocks=9, block_size=16, max_blocks=4, block_table=4096)
GOOD = {
    "spec_write_kv_q8": dict(COMMON, layer=1, dtype=L.SPEC_DTYPE_BF16, k=4096, v=4096, k_stride_b=384, k_stride_s=128,
                             k_stride_h=64, v_stride_b=384, v_stride_s=128, v_stride_h=64, codes=4096, scale=4096,
                             committed_len=4096),
    "spec_verify_attention_q8": dict(COMMON, Hq=4, layer=1, dtype=L.SPEC_DTYPE_BF16, q=4096, q_stride_b=768,
                                     q_stride_s=256, q_stride_h=64, cache=4096, cache_scale=4096, committed_len=4096,
                                     scale=0.125, out=4096, lse=4096),
    "spec_commit_kv_q8": dict(COMMON, codes=4096, scale=4096, slots=4096, slots_stride=3, n_slots=4096,
                              committed_len=4096),
    "spec_read_kv_q8": dict(COMMON, layer=1, dtype=L.SPEC_DTYPE_BF16, codes=4096, scale=4096, k=4096, v=4096),
}
ARGS = {"spec_write_kv_q8": L.SpecWriteKvQ8Args, "spec_verify_attention_q8": L.SpecAttentionQ8Args,
        "spec_commit_kv_q8": L.SpecCommitKvQ8Args, "spec_read_kv_q8": L.SpecReadKvQ8Args}
NAN, INF = float("nan"), float("inf")
SIZES = [dict(B=-1), dict(B=32769), dict(S=0), dict(H=0), dict(D=0), dict(L=0), dict(block_size=0), dict(max_blocks=0),
         dict(num_blocks=0), dict(block_table=None)]
LAYER = [dict(layer=-1), dict(layer=2), dict(dtype=2), dict(dtype=-1)]
CODES = [dict(codes=None), dict(codes=4104), dict(scale=None)]
BAD = {
    "spec_write_kv_q8": SIZES + LAYER + CODES + [
        dict(k=None), dict(v=None), dict(k=4104), dict(v=4098), dict(committed_len=None), dict(k_stride_b=4),
        dict(k_stride_s=7), dict(k_stride_h=65), dict(v_stride_b=1), dict(v_stride_s=12), dict(v_stride_h=66),
        dict(dtype=L.SPEC_DTYPE_F32, k_stride_h=66)],
    "spec_verify_attention_q8": SIZES + LAYER + [
        dict(S=1025), dict(Hq=0), dict(Hq=5), dict(scale=NAN), dict(scale=INF), dict(softcap=-1.0), dict(softcap=NAN),
        dict(softcap=INF), dict(softcap=1e-45), dict(window=-1), dict(shared_len=-1), dict(shared_len=65),
        dict(shared_len=8), dict(shared_len=8, shared_table=4096, key_pos=4096, key_pos_stride=64),
        dict(key_pos=4096, key_pos_stride=63), dict(q=None), dict(cache=None), dict(cache_scale=None),
        dict(committed_len=None), dict(q=4104), dict(cache=4100), dict(out=None), dict(out=4104), dict(q_stride_b=4),
        dict(q_stride_s=7), dict(q_stride_h=65)],
    "spec_commit_kv_q8": SIZES + CODES + [dict(n_slots=None), dict(committed_len=None), dict(slots_stride=2)],
    "spec_read_kv_q8": SIZES + LAYER + CODES + [dict(k=None), dict(v=None), dict(k=4104), dict(v=4098)],
}
UNSUPPORTED = {
    fn: [dict(D=8), dict(D=72), dict(D=272), dict(max_blocks=1 << 28)] for fn in GOOD}
UNSUPPORTED["spec_commit_kv_q8"] += [dict(S=1025, slots_stride=1025), dict(H=65536), dict(B=32768, L=1 << 20)]
UNSUPPORTED["spec_verify_attention_q8"] += [dict(softcap=1025.0), dict(Hq=65536)]
UNSUPPORTED["spec_write_kv_q8"] += [dict(H=65536), dict(S=(1 << 30) + 1), dict(B=32768, S=1 << 26)]
UNSUPPORTED["spec_read_kv_q8"] += [dict(H=65536), dict(S=(1 << 30) + 1), dict(B=32768, S=1 << 26)]


def call(lib, fn, over=(), ws=4096, nbytes=1 << 28):
    # no kernel may start: on a host without a GPU it would return SPEC_ERR_CUDA
    a = ARGS[fn](**dict(GOOD[fn], **dict(over)))
    return getattr(lib, fn)(ctypes.byref(a), ctypes.c_void_p(ws), nbytes, None)


@pytest.mark.parametrize("fn", GOOD)
def test_refusals(lib, fn):
    for bad in BAD[fn]:
        assert call(lib, fn, bad) == L.SPEC_ERR_INVALID_ARG, bad
    for bad in UNSUPPORTED[fn]:
        assert call(lib, fn, bad) == L.SPEC_ERR_UNSUPPORTED, bad
    assert getattr(lib, fn)(None, None, 0, None) == L.SPEC_ERR_INVALID_ARG
    for ws, nbytes in ((None, 1 << 28), (4096, 64), (4097, 1 << 28)):
        assert call(lib, fn, ws=ws, nbytes=nbytes) == L.SPEC_ERR_INVALID_ARG
    assert getattr(lib, fn)(ctypes.byref(ARGS[fn](**dict(GOOD[fn], B=0))), None, 0, None) == L.SPEC_OK


def test_shared_prefix_wants_its_workspace(lib):
    over = dict(shared_len=8, shared_table=4096)
    small = L.spec_workspace_bytes(L.SPEC_WS_ATTENTION, 2, 12, 64)
    assert call(lib, "spec_verify_attention_q8", over, nbytes=small) == L.SPEC_ERR_INVALID_ARG


def test_workspace_of_the_rows_calls(lib):
    api.clear_workspaces()
    assert L.spec_workspace_bytes(L.SPEC_WS_KV8, 5, 0, 0) == L.spec_workspace_bytes(L.SPEC_WS_COMMIT, 5, 0, 0)
    a, b, c = (api.workspace(L.SPEC_WS_KV8, 2, 0, 0, "cpu", stream=s) for s in (0, 7, 7))
    assert b is c and a.data_ptr() != b.data_ptr() and not a.any() and not b.any()
    big = api.workspace(L.SPEC_WS_KV8, 500, 0, 0, "cpu", stream=7)
    assert big is api.workspace(L.SPEC_WS_KV8, 2, 0, 0, "cpu", stream=7) and not big.any()
    api.clear_workspaces()


def test_calls_use_their_streams_workspace(lib, monkeypatch):
    used = []
    for fn in GOOD:
        monkeypatch.setattr(L, fn, lambda **kw: used.append((kw["workspace"], kw["stream"])))
    monkeypatch.setattr(api, "_allocating_on", lambda stream: contextlib.nullcontext())
    api.clear_workspaces()
    cache = api.quant_kv(1, 4, 16, 1, 64, device="cpu")
    table, lens = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    q, k = torch.zeros(2, 3, 1, 64), torch.zeros(2, 3, 1, 64)
    calls = (lambda **kw: api.write_kv_q8(k, k, cache, table, lens, block_size=16, **kw),
             lambda **kw: api.verify_attention_q8(q, cache, table, lens, block_size=16, **kw),
             lambda **kw: api.commit_kv_q8(cache, table, None, lens, lens, block_size=16, S=3, **kw),
             lambda **kw: api.read_kv_q8(cache, table, n_max=3, block_size=16, **kw))
    for f in calls:
        used.clear()
        mine = torch.zeros(1)
        for kw in (dict(stream=3), dict(stream=4), dict(stream=3), dict(stream=4, ws=mine)):
            f(**kw)
        (a, s), (b, t), (c, _), (d, _) = used
        assert a is c and a.data_ptr() != b.data_ptr() and d is mine and (s, t) == (3, 4)
    with pytest.raises(ValueError, match="S is needed"):
        api.commit_kv_q8(cache, table, None, lens, lens, block_size=16)
    api.clear_workspaces()


def test_binding_refuses_wrong_tensors(lib, monkeypatch):
    cache = api.quant_kv(1, 4, 16, 2, 64, device="cpu")
    table, lens = torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    k = torch.zeros((1, 3, 2, 64), dtype=torch.bfloat16)
    q = torch.zeros((1, 3, 4, 64), dtype=torch.bfloat16)
    on_cpu = (lambda: api.write_kv_q8(k, k, cache, table, lens, block_size=16),
              lambda: api.verify_attention_q8(q, cache, table, lens, block_size=16),
              lambda: api.commit_kv_q8(cache, table, None, lens, lens, block_size=16, S=3),
              lambda: api.read_kv_q8(cache, table, n_max=3, block_size=16))
    for f in on_cpu:
        with pytest.raises(ValueError, match="CUDA device"):
            f()
    with pytest.raises(TypeError, match="codes must be"):
        L._cache8_shape("f", cache.codes.view(torch.uint8), cache.scale, 16)
    monkeypatch.setattr(L, "_cache_shape", lambda fn, c, bs: c.shape)  # a CPU cache, nothing is launched
    with pytest.raises(ValueError, match="scale has shape"):
        L._cache8_shape("f", cache.codes, cache.scale.transpose(3, 4), 16)
    with pytest.raises(TypeError, match="scale must be"):
        L._cache8_shape("f", cache.codes, cache.scale.float(), 16)
    ws = torch.zeros(1)
    base = dict(codes=cache.codes, block_table=table, block_size=16, workspace=ws)
    w = dict(base, scale=cache.scale, committed_len=lens)
    for bad, err in ((dict(k=k, v=k[:, :2]), ValueError), (dict(k=k, v=k.float()), TypeError),
                     (dict(k=k[0], v=k), ValueError), (dict(k=k.half(), v=k.half()), TypeError),
                     (dict(k=k.transpose(2, 3), v=k), ValueError), (dict(k=k, v=k, layer=1 << 32), ValueError),
                     (dict(k=k, v=k, n_new=lens.long()), TypeError)):
        with pytest.raises(err):
            L.spec_write_kv_q8(**w, **bad)
    a = dict(base, cache_scale=cache.scale, committed_len=lens, scale=1.0, out=q)
    for bad, err in ((dict(q=q[..., :32]), ValueError), (dict(q=q.float()), TypeError), (dict(q=q[0]), ValueError),
                     (dict(q=q, window=1 << 32), ValueError), (dict(q=q, shared_len=20), ValueError),
                     (dict(q=q, key_pos=torch.zeros((1, 31), dtype=torch.int32)), ValueError)):
        with pytest.raises(err):
            L.spec_verify_attention_q8(**a, **bad)
    c = dict(base, scale=cache.scale, committed_len=lens, n_slots=lens)
    for bad in (dict(S=1 << 32), dict(S=3, slots=torch.zeros((1, 2), dtype=torch.int32)), dict(S=3, blocks_in_use=table)):
        with pytest.raises(ValueError):
            L.spec_commit_kv_q8(**c, **bad)
    r = dict(base, scale=cache.scale)
    for bad, err in ((dict(k=k, v=k[:, :2]), ValueError), (dict(k=k, v=k.float()), TypeError), (dict(k=k[0], v=k), ValueError),
                     (dict(k=k, v=k, start=table), ValueError), (dict(k=k, v=k, layer=-(1 << 32)), ValueError)):
        with pytest.raises(err):
            L.spec_read_kv_q8(**r, **bad)
