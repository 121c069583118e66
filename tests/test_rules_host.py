"""Host-side checks of sv_history_*, sv_logits_process and sv_head_w4 (no GPU):
bad arguments are refused before any CUDA call, by the library and by the
Python binding."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import speculative_decoding_verification_93_b200 as sv
from speculative_decoding_verification_93_b200 import _binding as bd

import _plain_rules as plain

ARG, SHAPE, DTYPE, WORKSPACE = 1, 2, 3, 4
A = [1 << 20, 1 << 30, 1 << 31, 1 << 32, 1 << 33]


def _history(**kw):
    d = dict(prompt_bits=A[0], output_bits=A[0] + 4096, output_counts=A[0] + 8192, R=4, V=1000)
    d.update(kw)
    return bd._History(*(d[n] for n, _ in bd._History._fields_))


@pytest.mark.parametrize("kw,code", [
    (dict(prompt_bits=None), ARG), (dict(output_bits=None), ARG), (dict(output_counts=None), ARG),
    (dict(prompt_bits=A[0] + 2), ARG), (dict(output_counts=A[0] + 1), ARG),
    (dict(R=0), SHAPE), (dict(V=0), SHAPE), (dict(V=(1 << 20) + 1), SHAPE),
])
def test_history_descriptor_refused(kw, code):
    L, h = sv.lib(), _history(**kw)
    assert L.sv_history_add(h, None, 2, A[1], 5, None, 0, 1, None, None) == code
    assert L.sv_history_reset(h, None, 2, None, None) == code


def test_history_arguments():
    L, h = sv.lib(), _history()
    assert L.sv_history_add(None, None, 2, A[1], 5, None, 0, 1, None, None) == ARG
    assert L.sv_history_add(h, None, 2, None, 5, None, 0, 1, None, None) == ARG
    assert L.sv_history_add(h, None, 2, A[1], 5, None, 0, 2, None, None) == ARG
    assert L.sv_history_add(h, None, -1, A[1], 5, None, 0, 1, None, None) == SHAPE
    assert L.sv_history_add(h, None, 2, A[1], -1, None, 0, 1, None, None) == SHAPE
    assert L.sv_history_add(h, None, 5, A[1], 5, None, 0, 1, None, None) == SHAPE   # row b is slot b
    assert L.sv_history_add(h, None, 0, None, 5, None, 0, 1, None, None) == 0       # nothing to do
    assert L.sv_history_add(h, None, 4, None, 0, None, 0, 1, None, None) == 0
    assert L.sv_history_reset(h, None, 5, None, None) == SHAPE
    assert L.sv_history_reset(h, None, -1, None, None) == SHAPE
    assert L.sv_history_reset(h, None, 0, None, None) == 0


def _process(rules=None, **kw):
    d = dict(logits=A[1], out=A[1], dtype=sv.SV_BF16, B=4, P=5, V=1000, v0=0, Vs=1000, drafts=A[0],
             K=4, pos0=0, lengths=None, extra=0)
    d.update(kw)
    return sv.lib().sv_logits_process(
        d["logits"], d["out"], d["dtype"], d["B"], d["P"], d["V"], d["v0"], d["Vs"], d["drafts"],
        d["K"], d["pos0"], d["lengths"], d["extra"],
        None if rules == "none" else (rules or bd._Rules()), None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(logits=None), ARG), (dict(out=None), ARG), (dict(drafts=None), ARG),
    (dict(logits=A[1] + 1, out=A[1] + 1), ARG), (dict(out=A[1] + 2), ARG),   # overlap
    (dict(out=A[1] + 4 * 5 * 1000 * 2 - 2), ARG), (dict(dtype=2), DTYPE),
    (dict(B=-1), SHAPE), (dict(P=0), SHAPE), (dict(P=66), SHAPE), (dict(V=0), SHAPE),
    (dict(Vs=0), SHAPE), (dict(Vs=1001), SHAPE), (dict(v0=1), SHAPE), (dict(v0=-1), SHAPE),
    (dict(K=65), SHAPE), (dict(K=-1), SHAPE), (dict(pos0=-1), SHAPE), (dict(pos0=65), SHAPE),
    (dict(B=0, logits=None, out=None), 0),
])
def test_process_arguments(kw, code):
    assert _process(**kw) == code


def _rules(**kw):
    r = bd._Rules()
    for k, v in kw.items():
        setattr(r, k, ctypes.pointer(v) if k == "history" else v)
    return r


@pytest.mark.parametrize("kw,code", [
    (dict(history=_history(V=999)), SHAPE), (dict(history=_history(R=3)), SHAPE),
    (dict(history=_history(output_counts=None)), ARG),
    (dict(bias_begin=A[0], n_bias=3), ARG), (dict(bias_begin=A[0], n_bias=-1), ARG),
    (dict(mask=A[0], n_masks=0), ARG), (dict(mask=A[0], n_masks=19), SHAPE),
    (dict(bias_begin=A[0], bias_tokens=A[1], bias_values=A[2], n_bias=2**30 + 1), SHAPE),
])
def test_process_rules(kw, code):
    assert _process(_rules(**kw)) == code


def test_process_needs_rules():
    assert _process("none") == ARG


def _head(weight=None, **kw):
    d = dict(x=A[1], B=2, P=3, lengths=None, extra=0, out=A[2], out_dtype=sv.SV_BF16, ws=A[3],
             wsb=1 << 40)
    w = dict(codes=A[0], scale=A[4], zero=None, scale_dtype=sv.SV_BF16, V=100, H=256, group=64)
    for k, v in kw.items():
        (w if k in w else d)[k] = v
    w = bd._W4(*(w[n] for n, _ in bd._W4._fields_))
    return sv.lib().sv_head_w4(w, d["x"], d["B"], d["P"], d["lengths"], d["extra"], d["out"],
                               d["out_dtype"], d["ws"], d["wsb"], None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(codes=None), ARG), (dict(scale=None), ARG), (dict(x=None), ARG), (dict(out=None), ARG),
    (dict(codes=A[0] + 8), ARG), (dict(x=A[1] + 2), ARG), (dict(scale=A[4] + 1), ARG),
    (dict(scale_dtype=sv.SV_F32, scale=A[4] + 2), ARG), (dict(out=A[2] + 1), ARG),
    (dict(out_dtype=sv.SV_F32, out=A[2] + 2), ARG), (dict(ws=A[3] + 8), ARG),
    (dict(ws=None, B=20), ARG), (dict(wsb=1000, B=20), WORKSPACE),
    (dict(out_dtype=2), DTYPE), (dict(scale_dtype=7), DTYPE),
    (dict(V=0), SHAPE), (dict(V=(1 << 20) + 1), SHAPE), (dict(H=0), SHAPE), (dict(H=96), SHAPE),
    (dict(group=16), SHAPE), (dict(group=256), SHAPE), (dict(H=32768 + 64), SHAPE),
    (dict(B=-1), SHAPE), (dict(P=0), SHAPE), (dict(B=1 << 20, P=2), SHAPE),
    (dict(B=0, x=None), 0),
])
def test_head_arguments(kw, code):
    assert _head(**kw) == code


def test_binding_refuses():
    i32 = torch.int32
    h = sv.TokenHistory.empty(2, 100, "cpu")
    assert h.prompt_bits.shape == (2, 4) and h.output_counts.shape == (2, 100)
    with pytest.raises(TypeError, match="on a GPU"):
        sv.sv_history_add(h, torch.zeros(2, 3, dtype=i32))
    with pytest.raises(TypeError, match="shape"):
        sv.TokenHistory(101, h.prompt_bits, h.output_bits, h.output_counts)
    with pytest.raises(TypeError, match="int32"):
        sv.TokenHistory(100, h.prompt_bits.long(), h.output_bits, h.output_counts)
    with pytest.raises(TypeError, match="lens"):
        sv.sv_history_add(h, torch.zeros(2, 3, dtype=i32), torch.zeros(3, dtype=i32))
    with pytest.raises(TypeError, match="go together"):
        sv.LogitRules(bias_begin=torch.zeros(3, dtype=i32))
    with pytest.raises(TypeError, match="same length"):
        sv.LogitRules(repetition=torch.ones(2), presence=torch.ones(3))
    with pytest.raises(TypeError, match="needs a mask"):
        sv.LogitRules(mask_index=torch.zeros(2, 1, dtype=i32))
    z = torch.zeros(2, 3, 100)
    with pytest.raises(TypeError, match="rows"):
        sv.sv_logits_process(z, z, sv.LogitRules(repetition=torch.ones(3)))
    with pytest.raises(TypeError, match="words"):
        sv.sv_logits_process(z, z, sv.LogitRules(mask=torch.zeros(6, 3, dtype=i32)))
    with pytest.raises(TypeError, match="mask_index"):
        sv.sv_logits_process(z, z, sv.LogitRules(mask=torch.zeros(6, 4, dtype=i32),
                                                 mask_index=torch.zeros(2, 2, dtype=i32)))
    with pytest.raises(TypeError):
        sv.sv_logits_process(z.double(), z.double(), sv.LogitRules())
    with pytest.raises(TypeError, match="out"):
        sv.sv_logits_process(z, z.bfloat16(), sv.LogitRules())
    codes = torch.zeros(7, 64, dtype=torch.uint8)
    with pytest.raises(TypeError, match="scale"):
        sv.W4Weight(codes, torch.zeros(7, 3))
    with pytest.raises(TypeError, match="scale"):
        sv.W4Weight(codes, torch.zeros(7, 2, dtype=torch.float16))
    w = sv.W4Weight(codes, torch.zeros(7, 2))
    assert (w.V, w.H, w.group) == (7, 128, 64)
    with pytest.raises(TypeError, match="x must be"):
        sv.sv_head_w4(w, torch.zeros(1, 1, 64, dtype=torch.bfloat16), torch.zeros(1, 1, 7), z)
    with pytest.raises(TypeError, match="out"):
        sv.sv_head_w4(w, torch.zeros(1, 1, 128, dtype=torch.bfloat16), torch.zeros(1, 2, 7), z)


def test_plain_bit_planes_round_trip():
    flags = np.random.default_rng(0).random((3, 77)) < 0.4
    assert np.array_equal(plain.unpack(plain.pack(flags), 77), flags)


@pytest.mark.parametrize("off", [1, 2, 3])
def test_misaligned_arrays_refused(off):
    """Every int32, uint32 and float32 array, before anything could be launched."""
    L, bad = sv.lib(), A[2] + off
    h = _history()
    for kind in (0, 1):
        for slots, tokens, lens, status in ((bad, A[1], None, None), (None, bad, None, None),
                                            (None, A[1], bad, None), (None, A[1], None, bad)):
            assert L.sv_history_add(h, slots, 2, tokens, 5, lens, 0, kind, status, None) == ARG
    assert L.sv_history_reset(h, bad, 2, None, None) == ARG
    assert L.sv_history_reset(h, None, 2, bad, None) == ARG
    for name in ("prompt_bits", "output_bits", "output_counts"):
        assert _process(_rules(history=_history(**{name: bad}))) == ARG, name
    for name in ("slots", "repetition", "frequency", "presence", "bias_begin", "bias_tokens",
                 "bias_values", "mask", "mask_index"):
        kw = dict(bias_begin=A[0], bias_tokens=A[0], bias_values=A[0], n_bias=3, mask=A[0],
                  n_masks=20, mask_index=A[0])
        kw[name] = bad
        assert _process(_rules(**kw)) == ARG, name
    assert _process(drafts=bad) == ARG
    assert _process(lengths=bad) == ARG
    assert L.sv_logits_process(A[1], A[1], sv.SV_BF16, 4, 5, 1000, 0, 1000, None, 0, 0, None, 0,
                               bd._Rules(), bad, None) == ARG
    for B in (2, 20):
        assert _head(B=B, lengths=bad) == ARG
        w = bd._W4(A[0], A[4], None, sv.SV_BF16, 100, 256, 64)
        assert L.sv_head_w4(w, A[1], B, 3, None, 0, A[2], sv.SV_BF16, A[3], 1 << 40, bad, None) == ARG


@pytest.mark.parametrize("V,H,group", [(1000, 12288, 128), (1000, 4096, 32), (33, 4096, 64),
                                       (31, 256, 32), (2752, 4608, 128), (10007, 1120, 32),
                                       (129280, 4096, 128), (64, 32768, 64)])
def test_head_workspace_serves_smaller_batches(V, H, group):
    """A workspace made for the largest batch is large enough for every smaller one."""
    w = bd._W4(A[0], A[4], None, sv.SV_BF16, V, H, group)
    sizes = list(range(1, 1200)) + list(range(1200, 5000, 61)) + [1 << 14, 1 << 17, 1 << 20]
    need = [sv.lib().sv_head_w4_workspace_bytes(w, M, 1) for M in sizes]
    for i in range(1, len(need)):
        assert need[i] >= need[i - 1], (sizes[i - 1:i + 1], need[i - 1:i + 1])
    assert sv.lib().sv_head_w4_workspace_bytes(w, 1 << 10, 1 << 10) == need[-1]


def test_binding_names_every_status_bit():
    header = open(os.path.join(os.path.dirname(__file__), "..", "include", "sv.h")).read()
    bits = re.findall(r"#define (SV_(?:ROW|NOTE)_\w+)\s+(\d+)", header)
    assert len(bits) == 11
    for name, value in bits:
        assert getattr(sv, name) == int(value), name
