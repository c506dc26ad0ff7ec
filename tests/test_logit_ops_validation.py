"""Refusals of the logit adjustment, the row top-k and the top-k distillation calls (CPU only): by the C
entry points before any HIP call, and by the binding before any pointer reaches the library."""

import ctypes
import math
import os

import pytest
import torch

import draft_model_distillation_amd as m
from draft_model_distillation_amd import _binding as binding
from draft_model_distillation_amd import build as B

F32, BF16 = 0, 1
WS = 1 << 20  # fake pointers: validation must reject before dereferencing (a call that passes is never made)
P = 1 << 24
R, V = 6, 64


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.lib_path()):
        B.build()
    return m.load_library()


def _adjust(lib, x=P, dt=BF16, n=4, v=64, ld=64, out=P + (1 << 20), ld_out=64, wsb=None, null=False, **fields):
    a = binding.OpdAdjust(P, 2)
    for k, f in fields.items():
        setattr(a, k, f)
    return lib.opd_adjust_logits(x, dt, n, v, ld, None if null else ctypes.byref(a), out, ld_out, WS,
                                 lib.opd_workspace_size() if wsb is None else wsb, None)


def test_adjust_c_entry(lib):
    assert _adjust(lib, x=None) == 1 and _adjust(lib, out=None) == 1 and _adjust(lib, null=True) == 1
    assert _adjust(lib, offsets=None) == 1 and _adjust(lib, n_blocks=-1) == 2
    assert _adjust(lib, n=-1) == 2 and _adjust(lib, v=0) == 2 and _adjust(lib, v=(1 << 19) + 1, ld=(1 << 19) + 8) == 2
    assert _adjust(lib, ld=56) == 2 and _adjust(lib, ld_out=56) == 2
    assert _adjust(lib, dt=5) == 3
    assert _adjust(lib, x=P + 2) == 4 and _adjust(lib, out=P + 8) == 4 and _adjust(lib, v=60, ld=60) == 4
    assert _adjust(lib, history=P, max_history=4, ld_history=4) == 1  # no history_len
    assert _adjust(lib, history=P, history_len=P, max_history=8, ld_history=4) == 2
    assert _adjust(lib, history=P, history_len=P, max_history=-1) == 2
    assert _adjust(lib, bias_tokens=P, max_bias=1, ld_bias=1) == 1
    assert _adjust(lib, bias_values=P, bias_len=P, max_bias=1, ld_bias=1) == 1
    full = dict(bias_tokens=P, bias_values=P, bias_len=P)
    assert _adjust(lib, **full, max_bias=16385, ld_bias=16385) == 2 and _adjust(lib, **full, max_bias=4, ld_bias=3) == 2
    assert _adjust(lib, mask=P, ld_mask=1, n_masks=4) == 2
    assert _adjust(lib, mask=P, ld_mask=2, n_masks=3) == 2  # four rows, three masks, no mask_row
    assert _adjust(lib, mask=P, ld_mask=2, n_masks=-1, mask_row=P) == 2
    assert _adjust(lib, mask=P, ld_mask=2, n_masks=4, masked_value=math.nan) == 5
    assert _adjust(lib, out=P, ld_out=72) == 2  # in place with another pitch
    assert _adjust(lib, wsb=64) == 6
    assert _adjust(lib, n=0, x=None, out=None) == 0 and _adjust(lib, n_blocks=0, offsets=None) == 0


def _topk(lib, y=P, dt=BF16, n=4, v=4096, ld=4096, k=8, values=P, index=P, rest=P, scratch=P, scb=1 << 30, wsb=None):
    return lib.opd_topk_rows(y, dt, n, v, ld, k, values, index, rest, scratch, scb, WS,
                             lib.opd_workspace_size() if wsb is None else wsb, None)


def test_topk_c_entry(lib):
    assert _topk(lib, y=None) == 1 and _topk(lib, values=None) == 1 and _topk(lib, index=None) == 1
    assert _topk(lib, rest=None) == 1
    assert _topk(lib, k=0) == 2 and _topk(lib, k=257) == 2 and _topk(lib, v=4, ld=8, k=5) == 2
    assert _topk(lib, n=-1) == 2 and _topk(lib, ld=4000) == 2 and _topk(lib, dt=9) == 3 and _topk(lib, y=P + 4) == 4
    assert _topk(lib, wsb=64) == 6
    wide = dict(n=1, v=151936, ld=151936)
    need = lib.opd_topk_scratch_size(1, 151936, BF16, 8)
    assert need > 0
    assert _topk(lib, **wide, scb=need - 1) == 6 and _topk(lib, **wide, scratch=None) == 6
    assert "opd_topk_scratch_size" in lib.opd_last_error().decode()
    assert _topk(lib, **wide, scratch=P + 4) == 4
    assert _topk(lib, n=0, y=None, values=None, index=None, rest=None, scratch=None, scb=0) == 0
    for bad in ((0, 64, BF16, 8), (1, 0, BF16, 8), (1, 64, 7, 8), (1, 64, BF16, 0), (1, 64, BF16, 257),
                (1, (1 << 19) + 1, BF16, 8)):
        assert lib.opd_topk_scratch_size(*bad) == 0


def _loss(lib, which, z=P, dt=BF16, n=4, v=64, ld=64, idx=P, logit=P, k=8, rest=P, kl=0, a=0.5, t=0.05, loss=P,
          stats=P, dz=P, dz_dt=BF16, ld_dz=64, scratch=P, scb=1 << 30, wsb=None):
    wsb = lib.opd_workspace_size() if wsb is None else wsb
    top = (z, dt, n, v, ld, idx, logit, k, rest, kl, a, t)
    if which == "fwd":
        return lib.opd_topk_loss_fwd(*top, loss, stats, scratch, scb, WS, wsb, None)
    if which == "bwd":
        return lib.opd_topk_loss_bwd(*top, stats, None, dz, dz_dt, ld_dz, WS, wsb, None)
    return lib.opd_topk_fused_fwd_bwd(*top, None, loss, stats, dz, dz_dt, ld_dz, scratch, scb, WS, wsb, None)


@pytest.mark.parametrize("which", ["fwd", "bwd", "fused"])
def test_topk_loss_c_entries(lib, which):
    def call(**kw):
        return _loss(lib, which, **kw)

    assert call(z=None) == 1 and call(idx=None) == 1 and call(logit=None) == 1 and call(stats=None) == 1
    assert call(n=-1) == 2 and call(v=0) == 2 and call(ld=56) == 2 and call(k=0) == 2 and call(k=257) == 2
    assert call(dt=4) == 3 and call(z=P + 4) == 4
    assert call(a=1.5) == 5 and call(a=math.nan) == 5 and call(t=math.nan) == 5 and call(kl=2) == 5
    assert call(rest=None, t=math.inf) == 5
    assert call(wsb=64) == 6
    assert call(n=0, z=None, idx=None, logit=None, rest=None, loss=None, stats=None, dz=None, scratch=None, scb=0) == 0
    if which != "bwd":
        assert call(loss=None) == 1
        wide = dict(n=2, v=151936, ld=151936, ld_dz=151936)
        need = lib.opd_topk_loss_scratch_size(2, 151936, BF16)
        assert need > 0 and call(**wide, scb=need - 1) == 6 and call(**wide, scratch=None) == 6
        assert call(**wide, scratch=P + 8) == 4
    if which != "fwd":
        assert call(dz=None) == 1 and call(dz_dt=3) == 3 and call(ld_dz=32) == 2 and call(dz=P + 4) == 4


def _raises(fn, match):
    with pytest.raises(ValueError, match=match):
        fn()


def _i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def test_adjust_binding():
    x, off = torch.zeros(R, V, dtype=torch.bfloat16), torch.tensor([0, 2, R], dtype=torch.int32)

    def bad(match, **kw):
        _raises(lambda: m.adjust_logits(kw.pop("x", x), kw.pop("offsets", off), **kw), match)

    bad("unsupported dtype", x=x.half())
    bad("2-D", x=x[0])
    bad("offsets must be torch.int32", offsets=off.long())
    bad("draft_tokens must have 6", draft_tokens=_i32(5))
    bad("repetition must have 2", repetition=torch.ones(3))
    bad("frequency must be torch.float32", frequency=torch.ones(2, dtype=torch.float64))
    bad("need history", history_len=_i32(2))
    bad("history_len is required", history=_i32(2, 4))
    bad(r"history must be \[2, n\]", history=_i32(3, 4), history_len=_i32(2))
    bad("unit stride", history=_i32(4, 2).t(), history_len=_i32(2))
    bad("rows must not overlap", history=_i32(8).as_strided((2, 4), (1, 1)), history_len=_i32(2))
    bad("need bias_tokens", bias_len=_i32(2))
    bad("bias_values is required", bias_tokens=_i32(2, 3))
    bad("same layout", bias_tokens=_i32(2, 3), bias_values=torch.zeros(2, 4), bias_len=_i32(2))
    bad("bias_len is required", bias_tokens=_i32(2, 3), bias_values=torch.zeros(2, 3))
    bad("mask_row needs mask", mask_row=_i32(R))
    bad("mask must be torch.int32", mask=torch.zeros(R, 2))
    bad("2 words per row", mask=_i32(R, 1))
    bad("one mask per row", mask=_i32(R - 1, 2))
    bad("mask_row must have 6", mask=_i32(R, 2), mask_row=_i32(R - 1))
    bad("out must be torch.bfloat16", out=x.float())
    bad(r"out must be \[6, 64\]", out=x[:5].clone())
    wide = torch.zeros(R + 1, V, dtype=torch.bfloat16)
    bad("out must not overlap x", x=wide[:R], out=wide[1:])
    bad("CUDA", out=x)  # in place is fine: the device check is the last one


def test_topk_binding():
    y = torch.zeros(R, V)
    for k in (0, 65, 257):
        _raises(lambda: m.topk_rows(y, k), "k must be in")
    _raises(lambda: m.topk_rows(y.half(), 4), "unsupported dtype")
    _raises(lambda: m.topk_rows(y, 4, out={"values": torch.zeros(R, 4)}), "index")
    good = {"values": torch.zeros(R, 4), "index": _i32(R, 4), "rest_lse": torch.zeros(R)}
    _raises(lambda: m.topk_rows(y, 3, out=good), "values must be a contiguous")
    _raises(lambda: m.topk_rows(y, 4, scratch=torch.zeros(8, 2).t()), "scratch must be contiguous")
    _raises(lambda: m.topk_rows(y, 4, out=good), "CUDA")


def test_topk_loss_binding():
    z, idx, logit, rest = torch.zeros(R, V), _i32(R, 4), torch.zeros(R, 4), torch.zeros(R)

    def each(match, z=z, idx=idx, logit=logit, rest=rest, **kw):
        _raises(lambda: m.topk_loss_fwd(z, idx, logit, rest, 0.5, 0.1, **kw), match)
        _raises(lambda: m.topk_loss_bwd(z, idx, logit, rest, 0.5, 0.1, torch.zeros(R, 4), **kw), match)
        _raises(lambda: m.topk_fused_fwd_bwd(z, idx, logit, rest, 0.5, 0.1, **kw), match)

    each("top_index must be torch.int32", idx=idx.long())
    each("k must be in", idx=_i32(R, 0), logit=torch.zeros(R, 0))
    each("k must be in", idx=_i32(R, 257), logit=torch.zeros(R, 257))
    each("top_index must be a contiguous", idx=_i32(R - 1, 4))
    each("top_logit must be a contiguous", logit=torch.zeros(R, 5))
    each("top_logit must be torch.float32", logit=logit.double())
    each("rest_lse must have 6", rest=torch.zeros(R - 1))
    each("kl must be one of", kl="jensen")
    each("unsupported dtype", z=z.half())
    each("CUDA")
    args = (z, idx, logit, rest, 0.5, 0.1)
    _raises(lambda: m.topk_loss_bwd(*args, torch.zeros(R, 8)), "row_stats must be a contiguous")
    _raises(lambda: m.topk_loss_bwd(*args, torch.zeros(R, 4), dz=torch.zeros(R, V - 1)), "dz must be")
    _raises(lambda: m.topk_loss_bwd(*args, torch.zeros(R, 4), dz=z), "dz must not overlap z")
    good = {"loss": torch.zeros(R), "row_stats": torch.zeros(R, 4), "dz": torch.zeros(R, V)}
    for call in (m.topk_fused_fwd_bwd, lambda *a, **kw: m.topk_loss_bwd(*a, torch.zeros(R, 4), **kw)):
        _raises(lambda: call(*args, grad_loss=torch.zeros(R - 1)), "grad_loss must have 6")
    for call in (m.topk_fused_fwd_bwd, m.topk_loss_fwd):
        _raises(lambda: call(*args, scratch=torch.zeros(8, 2).t()), "scratch must be contiguous")
    for name in good:
        _raises(lambda: m.topk_fused_fwd_bwd(*args, out={k: v for k, v in good.items() if k != name}), name)
    _raises(lambda: m.topk_fused_fwd_bwd(*args, out=dict(good, dz=z)), "dz must not overlap z")
    _raises(lambda: m.topk_fused_fwd_bwd(*args, out=dict(good, dz=torch.zeros(R, V).half())), "unsupported dtype")
    _raises(lambda: m.topk_fused_fwd_bwd(*args, out=good), "CUDA")
