"""GPU parity of the logit adjustment against its float64 oracle.

Tolerance: the kernel forms x * m (m the factor, at worst a rounded reciprocal) and subtracts in one
fused step a number that took at most (2 + earlier rows of the block) fp32 additions. With u = 2^-24 and
A the sum of the magnitudes added up, the fp32 result is within (4 + rows) u A of the exact one; the
rounding to the logits' type adds half a step of the result.
"""

import numpy as np
import pytest

import synth
from oracle import adjust as A

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}  # half a rounding step of the type, relative


@pytest.fixture(scope="module")
def lib(gpu_available):
    import draft_model_distillation_amd as m

    m.load_library()
    return m


def _logits(x, dtype, pad=0):
    """(device view [n, v] of a wider buffer, the exact float64 values)."""
    import torch

    n, v = x.shape
    per = 8 if dtype == "bf16" else 4
    ld = (v + per - 1) // per * per + pad * per
    buf = torch.full((n, ld), float("inf"), dtype=torch.bfloat16 if dtype == "bf16" else torch.float32)
    t = torch.from_numpy(x.astype(np.float32)).to(buf.dtype)
    buf[:, :v] = t
    return buf.cuda()[:, :v], t.double().numpy()


def _bits(mask):
    """bool [M, V] -> int32 words [M, ceil(V / 32)], with set bits past the vocabulary."""
    import torch

    n, v = mask.shape
    w = (v + 31) // 32
    full = np.ones((n, w * 32), dtype=np.uint8)
    full[:, :v] = mask
    words = np.packbits(full, axis=1, bitorder="little").view(np.uint32)
    return torch.from_numpy(words.view(np.int32).copy()).cuda()


def _dev(a, dtype):
    import torch

    return None if a is None else torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype=dtype))).cuda()


def _check(lib, x, dtype, offsets, pad=0, out_pad=0, inplace=False, masked_value=-1e4, expect_flags=0, **kw):
    import torch

    xt, exact = _logits(x, dtype, pad)
    f64 = {k: v for k, v in kw.items()}
    for name in ("repetition", "frequency", "presence", "bias_values"):  # what the kernel is given, exactly
        if kw.get(name) is not None:
            f64[name] = np.asarray(kw[name], dtype=np.float32).astype(np.float64)
    ref, size, flags = A.adjust_rows(exact, offsets, masked_value=masked_value, **f64)
    assert flags == expect_flags
    args = {k: _dev(v, np.float32 if k in ("repetition", "frequency", "presence", "bias_values") else np.int32)
            for k, v in kw.items() if k != "mask"}
    if kw.get("mask") is not None:
        args["mask"] = _bits(kw["mask"])
    if inplace:
        out = xt
        before = xt.clone()
    else:
        out, _ = _logits(np.full_like(x, 77.0), dtype, out_pad)
        before = out.clone()
    lib.read_flags(clear=True)
    got = lib.adjust_logits(xt, _dev(offsets, np.int32), masked_value=masked_value, out=out, **args)
    torch.cuda.synchronize()
    assert got is out and lib.read_flags(clear=True) == expect_flags
    g = got.double().cpu().numpy()
    keep = np.isnan(ref).all(axis=1) & ~np.isnan(exact).any(axis=1)
    assert np.array_equal(g[keep], before.double().cpu().numpy()[keep])  # rows outside every block
    r, s, gg = ref[~keep], size[~keep], g[~keep]
    fine = np.isfinite(r)
    assert np.array_equal(np.isnan(r), np.isnan(gg))
    assert np.array_equal(gg[~fine & ~np.isnan(r)], r[~fine & ~np.isnan(r)])
    n_max = max([int(b) - int(a) for a, b in zip(offsets, offsets[1:])] + [1])
    tol = (4 + min(n_max, len(x))) * U32 * s[fine] + HALF[dtype] * np.abs(r[fine])
    worst = np.abs(gg[fine] - r[fine]) - tol
    assert worst.size == 0 or worst.max() <= 0, worst.max()
    storage = got.untyped_storage()
    if out_pad and not inplace:  # the pad of the rows is not written
        whole = torch.empty(0, dtype=got.dtype, device="cuda").set_(storage)
        ld = got.stride(0)
        assert torch.isinf(whole.view(-1, ld)[:, got.shape[1]:]).all()
    return got


def _case(seed, offsets, vocab, hist=0, draft=False, bias=0, mask=False):
    rng = np.random.default_rng(seed)
    R, Bn = int(max(offsets[-1], 1)), len(offsets) - 1
    kw = {"repetition": 1 + rng.random(Bn), "frequency": rng.random(Bn), "presence": rng.random(Bn)}
    if hist:
        kw["history"] = rng.integers(0, vocab, (Bn, hist))
        kw["history"][:, ::3] = rng.integers(0, min(vocab, 5), kw["history"][:, ::3].shape)  # repeated tokens
        kw["history_len"] = rng.integers(0, hist + 1, Bn)
        kw["prompt_len"] = (kw["history_len"] * rng.random(Bn)).astype(np.int64)
    if draft:
        kw["draft_tokens"] = rng.integers(0, min(vocab, 40), R)
    if bias:
        kw["bias_tokens"] = rng.integers(0, vocab, (Bn, bias))
        kw["bias_values"] = rng.normal(0, 5, (Bn, bias))
        kw["bias_len"] = rng.integers(0, bias + 1, Bn)
    if mask:
        kw["mask"] = rng.random((R, vocab)) < 0.3
        kw["mask_row"] = np.where(rng.random(R) < 0.7, rng.integers(0, R, R), -1)  # shared by some rows
        kw["mask"][:, 0] = True
    return rng.normal(0, 4, (R, vocab)), kw


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [1, 7, 33, 1000, 8197, 40001])
def test_everything_at_ragged_sizes(lib, dtype, vocab):
    offsets = [0, 1, 1, 4, 21, 23]  # one row, none, and a block longer than a row group
    x, kw = _case(vocab, offsets, vocab, hist=50, draft=True, bias=9, mask=True)
    _check(lib, x, dtype, offsets, pad=1, out_pad=2, **kw)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("parts", [dict(), dict(hist=7), dict(draft=True), dict(bias=3), dict(mask=True),
                                   dict(hist=3000, draft=True)])
def test_each_part_alone(lib, dtype, parts):
    offsets = [0, 2, 18]
    x, kw = _case(3, offsets, 2000, **parts)
    _check(lib, x, dtype, offsets, **kw)


def test_no_penalties_is_a_copy_with_masks(lib):
    x, kw = _case(4, [0, 3], 515, mask=True)
    got = _check(lib, x, "bf16", [0, 3], mask=kw["mask"], masked_value=-np.inf)
    import torch

    assert torch.isinf(got).any()


def test_default_mask_rows(lib):
    x, kw = _case(5, [0, 4], 100, mask=True)
    _check(lib, x, "f32", [0, 4], mask=kw["mask"])


def test_long_blocks_and_many(lib):
    # a block of several row groups beside empty ones, so that workgroups take more than one group each
    offsets = [0, 0, 0, 0, 150, 150, 151]
    x, kw = _case(6, offsets, 300, hist=11, draft=True, bias=2)
    _check(lib, x, "bf16", offsets, **kw)
    offsets = list(range(0, 601, 2))
    x, kw = _case(7, offsets, 64, hist=5, draft=True)
    _check(lib, x, "f32", offsets, **kw)


def test_bias_of_a_token_listed_twice(lib):
    n = 700  # more entries than threads: the two may be one thread's or two threads'
    rng = np.random.default_rng(8)
    tok = rng.integers(0, 40, (1, n))
    val = rng.normal(0, 3, (1, n))
    x = rng.normal(0, 2, (1, 64))
    for length in (n, 1, 0, 300):
        _check(lib, x, "f32", [0, 1], bias_tokens=tok, bias_values=val, bias_len=[length])


def test_special_values(lib):
    x = np.array([[np.inf, -np.inf, np.nan, 0.0, -0.0, 1e30, -1e30, 1.0]] * 2)
    mask = np.array([[1, 1, 1, 1, 1, 1, 1, 1], [0, 0, 0, 0, 1, 1, 1, 1]], dtype=bool)
    for dtype in ("f32", "bf16"):
        got = _check(lib, x, dtype, [0, 1, 2], history=np.array([[0, 1, 2, 3], [4, 4, 5, 7]]), history_len=[4, 4],
                     prompt_len=[4, 0], repetition=[1.5, 2.0], frequency=[0.1, 0.2], presence=[0.0, 0.0], mask=mask)
        assert (got[1, :4].float().cpu().numpy() == float(got[1, 0])).all()


def test_flags_and_clamps(lib):
    x, _ = _case(9, [0, 6], 50)
    hist = np.array([[1, 60, 2], [-3, 1, 1], [2, 2, 2]])
    _check(lib, x, "f32", [0, 2, 4, 6], history=hist, history_len=[3, 2, 2], expect_flags=A.FLAG_BAD_TOKEN)
    _check(lib, x, "f32", [0, 2, 4, 6], history=hist % 50, history_len=[9, -1, 2], prompt_len=[1, 5, 9],
           expect_flags=A.FLAG_BAD_LIST)
    _check(lib, x, "f32", [0, 2, 7, 6], repetition=[2.0, 2.0, 2.0], expect_flags=A.FLAG_BAD_OFFSETS)
    _check(lib, x, "f32", [0, 6], draft_tokens=[1, 2, 99, 3, -4, 5], frequency=[0.5], expect_flags=A.FLAG_BAD_TOKEN)
    _check(lib, x, "f32", [0, 6], bias_tokens=np.array([[77, 3]]), bias_values=np.array([[1.0, 2.0]]), bias_len=[2],
           expect_flags=A.FLAG_BAD_TOKEN)
    mask = np.zeros((2, 50), dtype=bool)
    mask[0, 49] = True
    _check(lib, x, "f32", [0, 6], mask=mask, mask_row=[0, 0, -5, 0, 0, 0])
    _check(lib, x, "f32", [0, 6], mask=mask, mask_row=[0, 1, -1, 0, 0, 0], expect_flags=A.FLAG_EMPTY_MASK)
    _check(lib, x, "f32", [0, 6], mask=mask, mask_row=[0, 0, 0, 0, 0, 2], expect_flags=A.FLAG_BAD_LIST)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_in_place_and_no_rows(lib, dtype):
    import torch

    offsets = [0, 2, 5]
    x, kw = _case(10, offsets, 1003, hist=20, draft=True, bias=4, mask=True)
    _check(lib, x, dtype, offsets, inplace=True, **kw)
    e = torch.empty(0, 8, device="cuda")
    assert lib.adjust_logits(e, torch.zeros(2, dtype=torch.int32, device="cuda")).shape == (0, 8)
    assert lib.adjust_logits(torch.zeros(2, 8, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")).shape == (2, 8)


def test_serving_size(lib):
    import torch

    V = synth.VOCAB
    offsets = [0, 16, 17, 33]
    x, kw = _case(11, offsets, V, hist=5000, draft=True, bias=300, mask=True)
    _check(lib, x, "bf16", offsets, **kw)
    # the same bits every time
    xt, _ = _logits(x, "bf16")
    a = lib.adjust_logits(xt, _dev(offsets, np.int32), history=_dev(kw["history"], np.int32),
                          history_len=_dev(kw["history_len"], np.int32), frequency=_dev(kw["frequency"], np.float32))
    b = lib.adjust_logits(xt, _dev(offsets, np.int32), history=_dev(kw["history"], np.int32),
                          history_len=_dev(kw["history_len"], np.int32), frequency=_dev(kw["frequency"], np.float32))
    torch.cuda.synchronize()
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
