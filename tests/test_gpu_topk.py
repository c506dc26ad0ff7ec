"""GPU parity of the row top-k against its float64 oracle: values and indices are exact; the log-sum-exp
of the others is within a bound derived from its additions.

Bound: with u = 2^-24, a term 2^(x log2 e - ref) has the relative error of its exponent (at most 24 in
magnitude where the term counts: 24 u ln 2) and of exp2 (2 u); a thread adds at most n = ceil(V / 256) +
16 of them (n u) and the joins add at most 32 more rounding steps; the result is rounded once (u |lse|),
and log2 e is rounded (its multiples are divided out: u (|lse| + ln V + the span of what counts, 24)).
"""

import numpy as np
import pytest

import synth
from oracle import topk as T

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24


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


def _check(lib, x, dtype, k, rows=None):
    import torch

    yt, exact = _to(x, dtype)
    out = lib.topk_rows(yt, k)
    torch.cuda.synchronize()
    v, i, r = (out[n].cpu().numpy() for n in ("values", "index", "rest_lse"))
    n, V = x.shape
    for row in range(n) if rows is None else rows:
        rv, ri, rr = T.topk_row(exact[row], k)
        assert np.array_equal(i[row], ri), row
        assert np.array_equal(v[row].astype(np.float64), rv), row
        if np.isinf(rr):
            assert r[row] == rr
        else:
            tol = U32 * (24 * 0.7 + 2 + (V + 255) // 256 + 16 + 32 + 2 * abs(rr) + np.log(V) + 24)
            assert abs(float(r[row]) - rr) <= tol, (row, float(r[row]) - rr, tol)
    return out


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V,k", [(1, 1), (5, 5), (33, 2), (300, 256), (1000, 20), (2049, 256), (8200, 1), (40001, 64),
                                 (151936, 100)])
def test_random_rows(lib, dtype, V, k):
    rng = np.random.default_rng(V + k)
    _check(lib, rng.normal(0, 3, (5, V)), dtype, k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("order", ["rising", "falling", "equal", "two values", "late peaks", "early peaks"])
@pytest.mark.parametrize("V,k", [(20011, 256), (70001, 33)])
def test_orders_that_fill_the_buffer(lib, dtype, order, V, k):
    rng = np.random.default_rng(1)
    x = {"rising": np.linspace(-5, 5, V), "falling": np.linspace(5, -5, V), "equal": np.full(V, 1.25),
         "two values": rng.integers(0, 2, V).astype(float), "late peaks": np.r_[np.zeros(V - 500), np.full(500, 9.0)],
         "early peaks": np.r_[np.full(500, 9.0), np.zeros(V - 500)]}[order]
    _check(lib, np.stack([x, -x]), dtype, k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_masked_and_far_apart_rows(lib, dtype):
    rng = np.random.default_rng(2)
    V = 9001
    x = rng.normal(0, 2, (6, V))
    x[0] = -np.inf                       # nothing left
    x[1, 10:] = -np.inf                  # fewer tokens than the list
    x[2, rng.permutation(V)[:8000]] = -np.inf
    x[3, :64] = 9000.0                   # the list far above the others: their sum is not a difference
    x[4] = np.where(np.arange(V) % 1000 == 0, 1e4, -1e4)
    x[5] *= 0.0
    x[5, ::2] = -0.0                     # equal values of both signs
    for k in (1, 9, 10, 64, 256):
        _check(lib, x, dtype, k)


@pytest.mark.parametrize("rows", [1, 2, 7, 300, 700])
def test_row_counts_split_differently(lib, rows):
    rng = np.random.default_rng(rows)
    x = rng.normal(0, 3, (rows, 30000 if rows > 100 else 151936)).astype(np.float32)
    _check(lib, x, "bf16", 64, rows=range(0, rows, max(1, rows // 7)))


def test_ties_across_segments(lib):
    x = np.zeros((1, 151936))
    x[0, [3, 70000, 70001, 151935]] = 4.0
    out = _check(lib, x, "bf16", 6)
    assert out["index"][0].tolist() == [3, 70000, 70001, 151935, 0, 1]


def test_nan_rows_keep_to_the_memory(lib):
    import torch

    y = torch.full((3, 5000), float("nan"), device="cuda")
    y[1, 7] = 2.0
    y[2] = float("inf")
    out = lib.topk_rows(y, 16)
    torch.cuda.synchronize()
    assert int(out["index"].min()) >= -1 and int(out["index"].max()) < 5000


def test_outputs_and_scratch_of_the_caller(lib):
    import torch

    rng = np.random.default_rng(5)
    yt, exact = _to(rng.normal(0, 3, (2, 151936)), "bf16")
    want = lib.topk_rows(yt, 20)
    out = {"values": torch.zeros(2, 20, device="cuda"), "index": torch.zeros(2, 20, dtype=torch.int32, device="cuda"),
           "rest_lse": torch.zeros(2, device="cuda")}
    scratch = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    got = lib.topk_rows(yt, 20, scratch=scratch, out=out)
    torch.cuda.synchronize()
    for n in out:
        assert got[n] is out[n] and torch.equal(out[n], want[n])
    assert lib.topk_rows(yt[:0], 4)["index"].shape == (0, 4)
    assert synth.VOCAB == 151936
