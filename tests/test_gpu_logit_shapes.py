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
    (300, 40000, "bf16", 128), (1600, 30000, "bf16", 33), (1540, 33333, "f32", 64), (500, 16000, "bf16", 100), (65, 8192, "f32", 7), (70, 2500, "f32", 256)])
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
    (1100, 1003, "f32", "f32", 33), (1100, 8001, "bf16", "bf16", 256), (1100, 8001, "bf16", "f32", 20),
    (1100, 3001, "f32", "bf16", 9), (200, 7001, "bf16", "f32", 33), (130, 120001, "f32", "bf16", 64), (159, 70001, "f32", "f32", 9), (5, 36000, "f32", "f32", 64)])
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


def test_more_rows_than_a_grid_counts(lib):
    # 2^24 rows of a workgroup each have more threads than 32 bits count
    import torch

    R, V = (1 << 24) + 5, 8
    g = torch.Generator(device="cuda").manual_seed(5)
    y = torch.randn(R, V, device="cuda", generator=g).bfloat16()
    out = lib.topk_rows(y, 2)
    torch.cuda.synchronize()
    v, i = y.float().topk(2)
    assert torch.equal(out["values"], v)
    assert torch.equal(torch.gather(y.float(), 1, out["index"].long()), v)
    rest = torch.scatter(y.double(), 1, out["index"].long(), -float("inf")).logsumexp(1)
    assert float((out["rest_lse"].double() - rest).abs().max()) <= GT.U32 * 110  # GT's bound for V = 8 and |rest| < 8
    w = torch.rand(R, device="cuda", generator=g)
    args = (y, out["index"], out["values"] * 0.5, out["rest_lse"], 0.7, 0.05)
    loss, stats = lib.topk_loss_fwd(*args)
    dz = lib.topk_loss_bwd(*args, stats, grad_loss=w)
    both = lib.topk_fused_fwd_bwd(*args, grad_loss=w)
    last = tuple(t[-3:].contiguous() for t in args[:4]) + args[4:]
    few = lib.topk_fused_fwd_bwd(*last, grad_loss=w[-3:].contiguous())
    torch.cuda.synchronize()
    assert float((loss - both["loss"]).abs().max()) <= 1e-5 and float((loss[-3:] - few["loss"]).abs().max()) <= 1e-5
    # (gradients below 2 that differ by fp32's roundings: to bf16 they round to neighbours, 2^-7 apart, at most)
    assert float((dz.float() - both["dz"].float()).abs().max()) <= 2.0 ** -7 + 1e-5
    assert float((dz[-3:].float() - few["dz"].float()).abs().max()) <= 2.0 ** -7 + 1e-5


@pytest.mark.parametrize("rows", [3, 130])
def test_the_widest_rows_replayed(lib, rows):
    # their bitmap takes more LDS than a kernel has without asking for it
    import torch

    V = 524288
    y, z, _ = GL._rows(21, 2, V)
    pick = np.arange(rows) % 2
    idx, logit, rest = (torch.from_numpy(a[pick].copy()).cuda() for a in GL._lists(y, 20))
    zt = torch.from_numpy(z[pick].astype(np.float32)).cuda()
    eager = lib.topk_fused_fwd_bwd(zt, idx, logit, rest, 0.6, 0.05)
    torch.cuda.synchronize()
    want = [eager[n].clone() for n in ("loss", "dz")]
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        lib.topk_fused_fwd_bwd(zt, idx, logit, rest, 0.6, 0.05)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = lib.topk_fused_fwd_bwd(zt, idx, logit, rest, 0.6, 0.05)
    for _ in range(3):
        out["dz"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out["loss"], want[0]) and torch.equal(out["dz"], want[1])
        lib.topk_fused_fwd_bwd(zt, idx, logit, rest, 0.6, 0.05)
        torch.cuda.synchronize()
