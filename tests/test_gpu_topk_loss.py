"""GPU parity of distillation from a teacher's top logits (forward, backward and fused calls) against its
float64 oracle, within the bounds of tests/topk_check.py, and against differences of the loss."""

import numpy as np
import pytest

import synth
from oracle import topk as T
from tests import topk_check as C

pytestmark = pytest.mark.gpu

HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module")
def lib(gpu_available):
    import draft_model_distillation_amd as m

    m.load_library()
    return m


def _to(x, dtype, pad=1):
    import torch

    n, v = x.shape
    per = 8 if dtype == "bf16" else 4
    buf = torch.full((n, (v + per - 1) // per * per + pad * per), float("inf"),  # the pad must never count
                     dtype=torch.bfloat16 if dtype == "bf16" else torch.float32)
    t = torch.from_numpy(x.astype(np.float32)).to(buf.dtype)
    buf[:, :v] = t
    return buf.cuda()[:, :v], t.double().numpy()


def _lists(y, k):
    got = [T.topk_row(r.astype(np.float32).astype(np.float64), k) for r in y]
    return (np.stack([g[1] for g in got]).astype(np.int32), np.stack([g[0] for g in got]).astype(np.float32),
            np.array([g[2] for g in got], dtype=np.float32))


def _run(lib, zt, idx, logit, rest, alpha, tau, kl, w, dz_dtype, split):
    import torch

    t = [None if a is None else torch.from_numpy(a).cuda() for a in (idx, logit, rest, w)]
    dt = torch.bfloat16 if dz_dtype == "bf16" else torch.float32
    if split:
        loss, stats = lib.topk_loss_fwd(zt, t[0], t[1], t[2], alpha, tau, kl=kl)
        dz = lib.topk_loss_bwd(zt, t[0], t[1], t[2], alpha, tau, stats, kl=kl, grad_loss=t[3], dz_dtype=dt)
    else:
        out = lib.topk_fused_fwd_bwd(zt, t[0], t[1], t[2], alpha, tau, kl=kl, grad_loss=t[3], dz_dtype=dt)
        loss, stats, dz = out["loss"], out["row_stats"], out["dz"]
    torch.cuda.synchronize()
    return loss.cpu().numpy().astype(np.float64), stats.cpu().numpy().astype(np.float64), dz.double().cpu().numpy()


def _check(lib, z, idx, logit, rest, alpha=0.7, tau=0.02, kl="reverse", dtype="f32", dz="f32", w=None, rows=None, flags=0):
    zt, exact = _to(z, dtype)
    for split in (False, True):
        lib.read_flags(clear=True)
        loss, stats, grad = _run(lib, zt, idx, logit, rest, alpha, tau, kl, w, dz, split)
        assert lib.read_flags(clear=True) == flags
        for r in range(len(z)) if rows is None else rows:
            weight = 1.0 if w is None else float(w[r])
            rl = -np.inf if rest is None else float(rest[r])
            ref, info = T.row_grad(exact[r], idx[r], logit[r], rl, alpha, np.float32(tau).astype(float), kl)
            info["loss"] = T.row_loss(exact[r], idx[r], logit[r], rl, alpha, np.float32(tau).astype(float), kl)[0]
            C.check_row(exact[r], info, weight * ref, loss[r], grad[r], alpha, float(np.float32(tau)), kl, weight, HALF[dz])
            if np.isfinite(info["lse"]):
                V = z.shape[1]
                assert abs(stats[r, 2] - info["lse"]) <= C.U * ((V + 255) // 256 + 100 + 4 * abs(info["lse"]))


def _rows(seed, n, V, noise=1.5):
    rng = np.random.default_rng(seed)
    y = rng.normal(0, 3, (n, V))
    y[np.arange(n), rng.integers(0, V, n)] += 8
    return y, y + rng.normal(0, noise, (n, V)), rng


@pytest.mark.parametrize("kl", ["reverse", "forward"])
@pytest.mark.parametrize("dtype,dz", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("V,k", [(2, 1), (9, 9), (33, 4), (1000, 20), (2048, 256), (8197, 64), (40001, 1), (66000, 100)])
def test_random_rows(lib, kl, dtype, dz, V, k):
    y, z, rng = _rows(V + k, 4, V)
    idx, logit, rest = _lists(y, k)
    _check(lib, z, idx, logit, rest, kl=kl, dtype=dtype, dz=dz, w=rng.normal(0, 1, 4).astype(np.float32))


@pytest.mark.parametrize("kl", ["reverse", "forward"])
@pytest.mark.parametrize("alpha", [0.0, 0.5, 1.0])
@pytest.mark.parametrize("tau", [-0.1, 0.0, 0.3, np.inf])
def test_mixtures_and_clips(lib, kl, alpha, tau):
    y, z, _ = _rows(7, 5, 700)
    idx, logit, rest = _lists(y, 12)
    _check(lib, z, idx, logit, rest, alpha=alpha, tau=tau, kl=kl)


@pytest.mark.parametrize("kl", ["reverse", "forward"])
def test_lists_in_any_order_padded_and_repeated(lib, kl):
    y, z, rng = _rows(8, 6, 5000)
    idx, logit, rest = _lists(y, 10)
    for r in range(6):
        o = rng.permutation(10)
        idx[r], logit[r] = idx[r, o], logit[r, o]
    idx[1, 3:] = -1
    idx[2] = -7  # no entry: the row takes no part
    logit[3] = -np.inf
    _check(lib, z, idx, logit, rest, kl=kl)
    again = idx.copy()
    again[4, 7] = again[4, 2]
    _check(lib, z, again, logit, rest, kl=kl, flags=16)
    out = idx.copy()
    out[5, 0], out[0, 9] = 5000, 2 ** 31 - 1
    _check(lib, z, out, logit, rest, kl=kl, flags=8)


@pytest.mark.parametrize("kl", ["reverse", "forward"])
def test_ties_of_the_largest_teacher_logit(lib, kl):
    y, z, _ = _rows(9, 2, 300)
    idx = np.array([[50, 7, 200], [3, 2, 1]], dtype=np.int32)
    logit = np.array([[2.0, 2.0, 1.0], [0.5, 0.5, 0.5]], dtype=np.float32)
    _check(lib, z, idx, logit, np.zeros(2, dtype=np.float32), alpha=0.2, kl=kl)


@pytest.mark.parametrize("kl", ["reverse", "forward"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_zero_probabilities(lib, kl, dtype):
    y, z, rng = _rows(10, 5, 3000)
    idx, logit, rest = _lists(y, 16)
    rest[0] = -np.inf                    # the teacher gives nothing to the others
    logit[1, 5:] = -np.inf               # nor to some listed tokens
    z[2, idx[2, 3:]] = -np.inf           # the drafter gives nothing to some listed tokens
    others = np.setdiff1d(np.arange(3000), idx[3])
    z[3, others] = -np.inf               # nor to any of the others
    z[4, rng.permutation(others)[:2000]] = -np.inf
    _check(lib, z, idx, logit, rest, tau=0.1, kl=kl, dtype=dtype)
    if kl == "forward":
        _check(lib, z, idx, logit, None, tau=np.inf, alpha=1.0, kl=kl, dtype=dtype, rows=[0, 1, 4])
    _check(lib, z, idx, logit, None, tau=0.1, kl=kl, dtype=dtype)


@pytest.mark.parametrize("kl", ["reverse", "forward"])
def test_the_others_are_no_difference(lib, kl):
    # the drafter holds nearly all of its mass on the list, or nearly none of it
    y, z, _ = _rows(11, 4, 20000)
    idx, logit, rest = _lists(y, 8)
    z[0, idx[0]] += 60
    z[1, idx[1]] += 5000
    z[2, idx[2]] -= 60
    z[3, idx[3]] -= 5000
    _check(lib, z, idx, logit, rest, tau=1e3, alpha=1.0, kl=kl)


@pytest.mark.parametrize("rows,V", [(1, 151936), (3, 151936), (40, 151936), (300, 20000), (1200, 4000)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_row_counts_split_differently(lib, rows, V, dtype):
    y, z, rng = _rows(rows, min(rows, 40), V)
    pick = np.arange(rows) % len(y)
    idx, logit, rest = _lists(y, 64)
    w = rng.random(rows).astype(np.float32)
    _check(lib, z[pick], idx[pick], logit[pick], rest[pick], dtype=dtype, dz=dtype, w=w,
           rows=sorted({0, rows // 3, rows // 2, rows - 1}))


@pytest.mark.parametrize("rows", [3, 130])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_the_widest_rows(lib, dtype, rows):
    y, z, _ = _rows(14, 2, 524288)
    pick = np.arange(rows) % 2
    idx, logit, rest = _lists(y, 256)
    _check(lib, z[pick], idx[pick], logit[pick], rest[pick], dtype=dtype, dz=dtype, rows=[0, rows - 1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_rows_same_bits_every_time(lib, dtype):
    import torch

    g = torch.Generator(device="cuda").manual_seed(3)
    z = torch.randn(600, synth.VOCAB, device="cuda", generator=g).mul_(4).to(
        torch.float32 if dtype == "f32" else torch.bfloat16)
    kept = lib.topk_rows(z, 64)
    first = None
    for _ in range(4):
        out = lib.topk_fused_fwd_bwd(z, kept["index"], kept["values"] * 0.5, kept["rest_lse"], 0.7, 0.02, dz_dtype=torch.float32)
        torch.cuda.synchronize()
        if first is None:
            first = out
        assert torch.equal(out["dz"], first["dz"]) and torch.equal(out["loss"], first["loss"])
    # the gradient of a softmax adds up to 0 along each row
    total = first["dz"].double().sum(1).abs().max()
    assert float(total) <= 1e-5
    split = lib.topk_loss_fwd(z, kept["index"], kept["values"] * 0.5, kept["rest_lse"], 0.7, 0.02)
    dz = lib.topk_loss_bwd(z, kept["index"], kept["values"] * 0.5, kept["rest_lse"], 0.7, 0.02, split[1],
                           dz_dtype=torch.float32)
    torch.cuda.synchronize()
    assert float((dz - first["dz"]).abs().max()) <= 1e-5


@pytest.mark.parametrize("kl", ["reverse", "forward"])
def test_gradient_against_differences(lib, kl):
    # A central difference is off by h^2 / 6 times the third derivative. A class's term p l has the third
    # derivative p''' l + 3 p'' l' + 3 p' l'' + p l''', at most 0.9 for |l| < 2.5 (derivatives of p: 1/4, 0.1,
    # 1/8, of l: 1, 1/4, 0.1); all classes together at most twice that, the hard label 0.1: under 4. The
    # losses' own errors (below 1e-5 at this size, tests/topk_check.py) add 1e-5 / h.
    y, z, _ = _rows(12, 1, 40, noise=0.5)
    idx, logit, rest = _lists(y, 6)
    h = 1.0 / 16
    zs = np.repeat(z, 81, 0)
    for j in range(40):
        zs[2 * j, j] += h
        zs[2 * j + 1, j] -= h
    zt, _ = _to(zs, "f32")
    rep = [np.repeat(a, 81, 0) for a in (idx, logit, rest)]
    loss, _, dz = _run(lib, zt, *rep, 0.6, 1e3, kl, None, "f32", False)
    diff = (loss[0:80:2] - loss[1:80:2]) / (2 * h)
    assert np.abs(diff - dz[80]).max() <= 4 * h * h / 6 + 2e-5 / h


def test_separate_and_fused_outputs_of_the_caller(lib):
    import torch

    y, z, _ = _rows(13, 3, synth.VOCAB)
    idx, logit, rest = (torch.from_numpy(a).cuda() for a in _lists(y, 30))
    zt, _ = _to(z, "bf16")
    want = lib.topk_fused_fwd_bwd(zt, idx, logit, rest, 0.5, 0.05)
    wide = torch.full((3, synth.VOCAB + 16), 5.0, dtype=torch.bfloat16, device="cuda")
    out = {"loss": torch.zeros(3, device="cuda"), "row_stats": torch.zeros(3, 4, device="cuda"),
           "dz": wide[:, : synth.VOCAB]}
    scratch = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    got = lib.topk_fused_fwd_bwd(zt, idx, logit, rest, 0.5, 0.05, out=out, scratch=scratch)
    torch.cuda.synchronize()
    assert all(got[n] is out[n] and torch.equal(got[n], want[n]) for n in out)
    assert (wide[:, synth.VOCAB:] == 5.0).all()  # the pad of the rows is not written
    again = lib.topk_fused_fwd_bwd(zt, idx, logit, rest, 0.5, 0.05)
    assert torch.equal(again["dz"].view(torch.int16), want["dz"].view(torch.int16))  # the same bits every time
    empty = lib.topk_fused_fwd_bwd(zt[:0], idx[:0], logit[:0], rest[:0], 0.5, 0.05)
    assert empty["dz"].shape == (0, synth.VOCAB) and empty["loss"].shape == (0,)
