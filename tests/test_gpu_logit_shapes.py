"""The three logit operators over the row counts, row lengths and list lengths that their kernels divide
work by, against the float64 oracles, within the bounds of the operators' own tests."""

import numpy as np
import pytest

from oracle import topk as T
from tests import test_gpu_adjust as GA
from tests import test_gpu_topk as GT
from tests import test_gpu_topk_loss as GL

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib(gpu_available):
    import draft_model_distillation_amd as m

    m.load_library()
    return m


def _topk_rows(kind, V, rng):
    if kind == "random":
        return rng.normal(0, 3, (4, V))
    x = rng.normal(0, 3, (4, V))
    if kind == "grammar":  # a few allowed tokens, all others the same low number
        for r, allowed in enumerate((3, 40, 200, 4000)):
            keep = rng.permutation(V)[:allowed]
            y = np.full(V, -1e4)
            y[keep] = x[r, keep]
            x[r] = y
    if kind == "masked":
        for r, allowed in enumerate((0, 1, 60, 2000)):
            keep = rng.permutation(V)[:allowed]
            y = np.full(V, -np.inf)
            y[keep] = x[r, keep]
            x[r] = y
    if kind == "steps":  # rising, falling, equal, and a list far above what the rest's sum starts from
        x[0], x[1], x[2] = np.linspace(-5, 5, V), np.linspace(5, -5, V), -2.5
        x[3] = np.where(np.arange(V) % 97 == 0, 12.0 + np.arange(V) * 1e-5, -2.0)
    if kind == "crowded":  # every vector has an element of the same high value, the rest just matters
        x[:] = -1.0
        for r, step in enumerate((4, 8, 16, 64)):
            x[r, ::step] = 9.5
            x[r, :40] = 14.0
    return x


@pytest.mark.parametrize("kind", ["random", "grammar", "masked", "steps", "crowded"])
@pytest.mark.parametrize("rows,V,dtype,k", [
    (3, 262144, "f32", 128), (30, 140000, "bf16", 20), (47, 66000, "f32", 1), (2, 70001, "f32", 129),
    (200, 262144, "bf16", 64), (60, 100003, "f32", 200), (400, 60000, "bf16", 64), (300, 33333, "f32", 256),
    (300, 40000, "bf16", 128), (500, 16000, "bf16", 100), (65, 8192, "f32", 7), (70, 2500, "f32", 256)])
def test_top_lists(lib, kind, rows, V, dtype, k):
    base = _topk_rows(kind, V, np.random.default_rng(rows + V + k)).astype(np.float32)
    x = base[np.arange(rows) % 4]
    out = GT._check(lib, x, dtype, k, rows=range(min(rows, 4)))
    for name in ("values", "index", "rest_lse"):  # equal rows have equal answers, whoever computes them
        got = out[name].view(rows, -1)
        for r in range(4):
            same = got[r::4]
            assert bool((same == same[:1]).all()), (name, r)


@pytest.mark.parametrize("kl", ["reverse", "forward"])
@pytest.mark.parametrize("rows,V,dtype,dz,k", [
    (259, 17003, "bf16", "bf16", 64), (259, 17003, "bf16", "f32", 64), (259, 140003, "bf16", "f32", 33),
    (257, 140003, "bf16", "bf16", 256), (258, 232000, "bf16", "bf16", 100), (256, 140003, "bf16", "bf16", 64),
    (300, 60001, "f32", "f32", 64), (300, 9001, "f32", "bf16", 20), (300, 12000, "bf16", "bf16", 20),
    (130, 120001, "f32", "bf16", 64), (159, 70001, "f32", "f32", 9), (5, 36000, "f32", "f32", 64)])
def test_distillation(lib, kl, rows, V, dtype, dz, k):
    y, z, rng = GL._rows(rows + V, 4, V)
    pick = np.arange(rows) % 4
    idx, logit, rest = GL._lists(y, k)
    w = rng.normal(0, 1, rows).astype(np.float32)
    GL._check(lib, z.astype(np.float32)[pick], idx[pick], logit[pick], rest[pick], kl=kl, dtype=dtype, dz=dz, w=w,
              rows=[0, 1, rows // 2, rows - 1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("blocks,per,hist", [(3, 70, 40), (20, 24, 300), (40, 8, 2000), (300, 1, 100), (2, 3, 20000)])
def test_blocks_and_histories(lib, dtype, blocks, per, hist):
    rng = np.random.default_rng(blocks)
    offsets = np.r_[0, np.cumsum(rng.integers(max(per - 3, 1), per + 4, blocks) if per > 1 else np.ones(blocks, int))]
    vocab = 30011 if dtype == "f32" else 20003
    x, kw = GA._case(blocks, offsets.tolist(), vocab, hist=hist, draft=True, bias=5, mask=blocks < 100)
    GA._check(lib, x, dtype, offsets.tolist(), inplace=blocks == 20, **kw)


def test_masked_rows_keep_their_tokens(lib):
    # adjusted rows under a grammar, then their lists: only allowed tokens come first, in both fills
    import torch

    rng = np.random.default_rng(4)
    R, V, k = 300, 60000, 64
    x = torch.from_numpy(rng.normal(0, 3, (R, V)).astype(np.float32)).bfloat16().cuda()
    allowed = rng.random((R, V)) < 0.002
    mask = GA._bits(allowed)
    off = torch.arange(0, R + 1, 3, dtype=torch.int32, device="cuda")
    for fill in (-1e4, -float("inf")):
        a = lib.adjust_logits(x, off, mask=mask, masked_value=fill)
        out = lib.topk_rows(a, k)
        torch.cuda.synchronize()
        exact = a.double().cpu().numpy()
        for r in (0, 17, R - 1):
            rv, ri, rr = T.topk_row(exact[r], k)
            assert np.array_equal(out["index"][r].cpu().numpy(), ri)
            n = min(k, int(allowed[r].sum()))
            assert allowed[r][ri[:n]].all()
