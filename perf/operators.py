"""Cases, plain forms and 64-bit values of three operators on vocabulary-wide rows of logits:

* ``adjust``: penalties for repeated tokens, biases and grammar masks on the rows of packed draft
  blocks, before they are verified;
* ``topk``: the k largest logits of every row, their indices, and the log-sum-exp of all the others
  (what is stored of a target row for training later on);
* ``loss``: the clipped distillation loss of the drafter's rows against such a stored row, and its
  gradient, in one call or as a forward and a backward call.

Where ``own`` is false, ``run`` computes them in elementary torch operations in 32 bits; where it is
true it calls the library.
"""

import math
import random

import torch

own = False

VOCAB = 151936
# what a masked token's logit becomes: for a softmax of the caller's own, or, where the library verifies
# the rows next, the lowest logit that its row kernels' contract allows
FILL = {"none": -math.inf, "low": -1.0e4}

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases


def listed():
    return [
        # one request's next token: the smallest call of a decoding loop, latency counts
        {"name": "adjust_decode_1", "op": "adjust", "blocks": 1, "rows": 1, "vocab": VOCAB, "dtype": "bf16",
         "history": 517, "bias": 0, "masked": 0.0, "fill": "none"},
        # 128 requests decoding one token each, with a bias list, one in eight under a grammar
        {"name": "adjust_decode_128", "op": "adjust", "blocks": 128, "rows": 1, "vocab": VOCAB, "dtype": "bf16",
         "history": 4096, "bias": 300, "masked": 0.125, "fill": "none"},
        # 128 drafted blocks of at most 16 positions, packed, one in four under a grammar
        {"name": "adjust_verify_128", "op": "adjust", "blocks": 128, "rows": 16, "vocab": VOCAB, "dtype": "bf16",
         "history": 4096, "bias": 0, "masked": 0.25, "fill": "low"},
        # fp32 rows of a small ragged vocabulary behind long contexts
        {"name": "adjust_long_f32", "op": "adjust", "blocks": 61, "rows": 16, "vocab": 32003, "dtype": "f32",
         "history": 65536, "bias": 17, "masked": 1.0, "fill": "none"},
        # the target row of one position, for a log-probability list of 20
        {"name": "topk_1", "op": "topk", "rows": 1, "vocab": VOCAB, "dtype": "bf16", "k": 20},
        # one round of 16 requests with 16 drafted positions each
        {"name": "topk_256_f32", "op": "topk", "rows": 256, "vocab": VOCAB, "dtype": "f32", "k": 64},
        # a trainer's whole batch, half of the training workload's positions
        {"name": "topk_8192", "op": "topk", "rows": 8192, "vocab": VOCAB, "dtype": "bf16", "k": 64},
        # a long list over a ragged vocabulary
        {"name": "topk_wide_k", "op": "topk", "rows": 1531, "vocab": 50257, "dtype": "f32", "k": 256},
        # one drafted block of 16 positions, trained on at once
        {"name": "loss_16", "op": "loss", "rows": 16, "vocab": VOCAB, "dtype": "bf16", "dz": "bf16", "k": 64,
         "kl": "reverse", "call": "fused"},
        # a trainer's whole batch
        {"name": "loss_8192", "op": "loss", "rows": 8192, "vocab": VOCAB, "dtype": "bf16", "dz": "bf16", "k": 64,
         "kl": "reverse", "call": "fused"},
        # fp32 logits and gradient, the forward divergence
        {"name": "loss_2048_f32", "op": "loss", "rows": 2048, "vocab": VOCAB, "dtype": "f32", "dz": "f32", "k": 100,
         "kl": "forward", "call": "fused"},
        # forward and backward as calls of their own (the loss is weighted between them)
        {"name": "loss_split", "op": "loss", "rows": 1111, "vocab": 50257, "dtype": "bf16", "dz": "f32", "k": 33,
         "kl": "forward", "call": "split"},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["adjust", "topk", "loss"])
    vocab = _log_int(rng, 1000, 262144)
    dtype = rng.choice(["f32", "bf16"])
    # at most a quarter of the largest listed case's elements
    rows = _log_int(rng, 1, max(1, min(8192, 2048 * VOCAB // vocab)))
    if op == "adjust":
        per = rng.choice([1, rng.randint(2, 16), rng.randint(17, 64)])
        return {"op": op, "blocks": max(1, rows // per), "rows": per, "vocab": vocab, "dtype": dtype,
                "history": _log_int(rng, 1, 65536), "bias": rng.choice([0, rng.randint(1, 300)]),
                "masked": rng.choice([0.0, round(rng.random(), 3), 1.0]), "fill": rng.choice(["none", "low"])}
    k = _log_int(rng, 1, 256)
    if op == "topk":
        return {"op": op, "rows": rows, "vocab": vocab, "dtype": dtype, "k": k}
    return {"op": op, "rows": rows, "vocab": vocab, "dtype": dtype, "dz": rng.choice(["f32", "bf16"]), "k": k,
            "kl": rng.choice(["reverse", "forward"]), "call": rng.choice(["fused", "fused", "split"])}


# ------------------------------------------------------------------ inputs


def _matrix(rows, vocab, dtype):
    """An uninitialised [rows, vocab] matrix whose row pitch is whole 16-byte vectors."""
    per = 16 // torch.empty((), dtype=dtype).element_size()
    return torch.empty(rows, (vocab + per - 1) // per * per, dtype=dtype, device="cuda")[:, :vocab]


def _logits(rows, vocab, dtype, g, sigma=3.0, peak=8.0, base=None):
    """Rows of N(0, sigma^2) with one token raised to `peak` above the row's largest, or base + noise."""
    x = torch.randn(rows, vocab, device="cuda", generator=g).mul_(sigma)
    if base is None:
        tok = torch.randint(vocab, (rows, 1), device="cuda", generator=g)
        x.scatter_(1, tok, x.amax(1, keepdim=True) + peak)
    else:
        x += base
    out = _matrix(rows, vocab, dtype)
    out.copy_(x)
    return out


def _layout(case):
    """Rows of each block, lengths of its history and prompt: of the case alone."""
    rng = random.Random("%(blocks)d/%(rows)d/%(history)d" % case)
    n = case["blocks"]
    rows = [case["rows"] if case["rows"] < 2 or n == 1 else rng.randint(1, case["rows"]) for _ in range(n)]
    hist = [case["history"] if n == 1 else rng.randint(case["history"] // 8, case["history"]) for _ in range(n)]
    prompt = [int(h * rng.random()) for h in hist]
    return rows, hist, prompt


def _prepare_adjust(case, g):
    rows, hist, prompt = _layout(case)
    n, vocab, dtype = case["blocks"], case["vocab"], DTYPES[case["dtype"]]
    total = sum(rows)
    i32 = dict(dtype=torch.int32, device="cuda")

    def tokens(*shape):  # frequent tokens have low indices, as in a vocabulary sorted by merges
        u = torch.rand(*shape, device="cuda", generator=g)
        return (vocab * u ** 4).to(torch.int32).clamp_(0, vocab - 1)

    offsets = torch.zeros(n + 1, **i32)
    offsets[1:] = torch.tensor(rows, **i32).cumsum(0)
    state = {
        "case": case, "rows": total, "x": _logits(total, vocab, dtype, g), "offsets": offsets,
        "history": tokens(n, (case["history"] + 3) // 4 * 4), "history_len": torch.tensor(hist, **i32),
        "prompt_len": torch.tensor(prompt, **i32), "draft_tokens": tokens(total),
        "repetition": 1.0 + 0.3 * torch.rand(n, device="cuda", generator=g),
        "frequency": 0.5 * torch.rand(n, device="cuda", generator=g),
        "presence": torch.rand(n, device="cuda", generator=g),
        "bias_tokens": None, "bias_values": None, "bias_len": None, "mask": None, "mask_row": None,
    }
    if case["bias"]:
        m = min(case["bias"], vocab)
        order = torch.rand(n, vocab, device="cuda", generator=g).topk(m, 1).indices  # no token twice
        state["bias_tokens"] = order.to(torch.int32)
        state["bias_values"] = 4.0 * torch.randn(n, m, device="cuda", generator=g)
        state["bias_len"] = torch.randint(0, m + 1, (n,), device="cuda", generator=g, dtype=torch.int32)
    if case["masked"] > 0:
        # rows of the blocks under a grammar have a bit mask each, the others none
        every = max(1, round(1.0 / case["masked"]))
        block = torch.repeat_interleave(torch.arange(n, device="cuda"), torch.tensor(rows, device="cuda"))
        held = block % every == 0
        words = (vocab + 31) // 32
        count = int(held.sum())
        bits = torch.randint(-2 ** 31, 2 ** 31, (2, count, words), device="cuda", generator=g)
        state["mask"] = (bits[0] & bits[1]).to(torch.int32)  # a quarter of the tokens allowed
        state["mask_row"] = torch.where(held, held.cumsum(0) - 1, -1).to(torch.int32)
    return state


def _prepare_topk(case, g):
    return {"case": case, "y": _logits(case["rows"], case["vocab"], DTYPES[case["dtype"]], g)}


def _prepare_loss(case, g):
    rows, vocab, k = case["rows"], case["vocab"], case["k"]
    y = _logits(rows, vocab, torch.float32, g)
    top, index = y.topk(k, 1)
    rest = y.scatter(1, index, -math.inf)
    rest_lse = torch.logsumexp(rest, 1)
    del rest
    z = _logits(rows, vocab, DTYPES[case["dtype"]], g, sigma=1.5, base=y)
    return {"case": case, "z": z, "top_logit": top.contiguous(), "top_index": index.to(torch.int32),
            "rest_lse": rest_lse, "grad_loss": torch.rand(rows, device="cuda", generator=g) / rows,
            "alpha": 0.7, "tau": 0.02}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"adjust": _prepare_adjust, "topk": _prepare_topk, "loss": _prepare_loss}[case["op"]](case, g)


# ------------------------------------------------------------------ the plain forms


def _row_blocks(state):
    """Block of every row, and the row's place in it."""
    rows = torch.arange(state["rows"], device="cuda")
    block = (rows[:, None] >= state["offsets"][None, 1:]).sum(1)
    return rows, block, rows - state["offsets"][block]


def _plain_adjust(s):
    x = s["x"].float()
    vocab = x.shape[1]
    rows, block, _ = _row_blocks(s)
    n = s["offsets"].numel() - 1
    at = torch.arange(s["history"].shape[1], device="cuda")
    hist = s["history"].long()
    live = at[None, :] < s["history_len"][:, None]
    out = live & (at[None, :] >= s["prompt_len"][:, None])
    count = torch.zeros(n, vocab, device="cuda").scatter_add_(1, hist, out.float())[block]
    seen = torch.zeros(n, vocab, device="cuda").scatter_add_(1, hist, live.float())[block]
    # the proposals of a block's earlier rows count as its output
    earlier = (block[:, None] == block[None, :]) & (rows[None, :] < rows[:, None])
    later, before = earlier.nonzero(as_tuple=True)
    one = torch.ones((), device="cuda")
    count.index_put_((later, s["draft_tokens"].long()[before]), one, accumulate=True)
    seen += count
    rho = s["repetition"][block][:, None]
    x = torch.where(seen > 0, torch.where(x > 0, x / rho, x * rho), x)
    x = x - s["frequency"][block][:, None] * count - s["presence"][block][:, None] * (count > 0)
    if s["bias_tokens"] is not None:
        live = torch.arange(s["bias_tokens"].shape[1], device="cuda")[None, :] < s["bias_len"][:, None]
        add = torch.zeros(n, vocab, device="cuda")
        add.scatter_add_(1, s["bias_tokens"].long(), torch.where(live, s["bias_values"], 0.0))
        x = x + add[block]
    if s["mask"] is not None:
        tok = torch.arange(vocab, device="cuda")
        row = s["mask_row"].long()
        words = s["mask"][row.clamp(min=0)][:, tok >> 5]
        allowed = ((words >> (tok & 31)) & 1).bool() | (row < 0)[:, None]
        x = torch.where(allowed, x, FILL[s["case"]["fill"]])
    return x.to(s["x"].dtype)


def _plain_topk(s):
    y = s["y"].float()
    k, vocab = s["case"]["k"], y.shape[1]
    # whole numbers in the order of the values, then of falling indices: no two are the same
    bits = (y + 0.0).contiguous().view(torch.int32).long()
    key = torch.where(bits < 0, (-2 ** 31) - bits - 1, bits)
    key = key * 2 ** 20 + (vocab - 1 - torch.arange(vocab, device="cuda"))
    index = vocab - 1 - (key.topk(k, 1).values & (2 ** 20 - 1))
    del bits, key
    rest = y.scatter(1, index, -math.inf)
    m = rest.amax(1, keepdim=True)
    rest_lse = m[:, 0] + (rest - m).exp().sum(1).log()
    return {"values": y.gather(1, index), "index": index.to(torch.int32), "rest_lse": rest_lse}


def _log_softmax(x):
    x = x - x.amax(1, keepdim=True)
    return x - x.exp().sum(1, keepdim=True).log()


def _plain_loss(s):
    alpha, tau, case = s["alpha"], s["tau"], s["case"]
    z = s["z"].float()
    index = s["top_index"].long()
    rest = z.scatter(1, index, -math.inf)
    m = rest.amax(1, keepdim=True)
    rest = (rest - m).exp()
    total = rest.sum(1, keepdim=True)
    # every row's distribution over its listed tokens and, as one class, all the others
    log_p = _log_softmax(torch.cat([z.gather(1, index), m + total.log()], 1))
    log_q = _log_softmax(torch.cat([s["top_logit"], s["rest_lse"][:, None]], 1))
    p, q = log_p.exp(), log_q.exp()
    if case["kl"] == "reverse":
        term = p * (log_p - log_q)
        g = torch.where(term <= tau, log_p - log_q + 1.0, 0.0)
        d = alpha * p * (g - (p * g).sum(1, keepdim=True))
    else:
        term = q * (log_q - log_p)
        u = torch.where(term <= tau, q, 0.0)
        d = alpha * (u.sum(1, keepdim=True) * p - u)
    hard = torch.zeros_like(p).scatter_(1, s["top_logit"].argmax(1, keepdim=True), 1.0)
    loss = alpha * term.clamp(max=tau).sum(1) - (1.0 - alpha) * (hard * log_p).sum(1)
    d = (d + (1.0 - alpha) * (p - hard)) * s["grad_loss"][:, None]
    # the class of the others: its derivative goes to them by their shares of it
    dz = rest * (d[:, -1:] / total)
    dz.scatter_(1, index, d[:, :-1])
    return {"loss": loss, "dz": dz.to(DTYPES[case["dz"]])}


# ------------------------------------------------------------------ the library's calls


def _own_adjust(s):
    import draft_model_distillation_amd as lib

    return lib.adjust_logits(s["x"], s["offsets"], history=s["history"], history_len=s["history_len"],
                             prompt_len=s["prompt_len"], draft_tokens=s["draft_tokens"], repetition=s["repetition"],
                             frequency=s["frequency"], presence=s["presence"], bias_tokens=s["bias_tokens"],
                             bias_values=s["bias_values"], bias_len=s["bias_len"], mask=s["mask"],
                             mask_row=s["mask_row"], masked_value=FILL[s["case"]["fill"]])


def _own_topk(s):
    import draft_model_distillation_amd as lib

    got = lib.topk_rows(s["y"], s["case"]["k"])
    return {"values": got["values"], "index": got["index"], "rest_lse": got["rest_lse"]}


def _own_loss(s):
    import draft_model_distillation_amd as lib

    case = s["case"]
    args = (s["z"], s["top_index"], s["top_logit"], s["rest_lse"], s["alpha"], s["tau"])
    if case["call"] == "fused":
        got = lib.topk_fused_fwd_bwd(*args, kl=case["kl"], grad_loss=s["grad_loss"], dz_dtype=DTYPES[case["dz"]])
        return {"loss": got["loss"], "dz": got["dz"]}
    loss, row_stats = lib.topk_loss_fwd(*args, kl=case["kl"])
    dz = lib.topk_loss_bwd(*args, row_stats, kl=case["kl"], grad_loss=s["grad_loss"], dz_dtype=DTYPES[case["dz"]])
    return {"loss": loss, "dz": dz}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"adjust": _own_adjust, "topk": _own_topk, "loss": _own_loss}[op](state)
    return {"adjust": _plain_adjust, "topk": _plain_topk, "loss": _plain_loss}[op](state)


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    size = {"f32": 4, "bf16": 2}
    vocab, s = case["vocab"], size[case["dtype"]]
    if case["op"] == "adjust":
        rows, hist, _ = _layout(case)
        every = max(1, round(1.0 / case["masked"])) if case["masked"] > 0 else 0
        held = sum(r for b, r in enumerate(rows) if every and b % every == 0)
        n = sum(rows) * vocab
        return {"bytes": 2 * n * s + held * (vocab + 31) // 32 * 4 + 4 * sum(hist) + 4 * case["bias"] * len(rows),
                "flops": 4 * n}
    n = case["rows"] * vocab
    if case["op"] == "topk":
        return {"bytes": n * s + case["rows"] * (8 * case["k"] + 4), "flops": 3 * n}
    dz = size[case["dz"]]
    reads = 2 if case["call"] == "split" else 1  # a backward call of its own reads the logits again
    return {"bytes": n * (reads * s + dz) + case["rows"] * (reads * 8 * case["k"] + 12), "flops": 6 * n}


# ------------------------------------------------------------------ the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"adjust": _exact_adjust, "topk": _exact_topk, "loss": _exact_loss}[case["op"]](case, s)


def _chunks(rows, vocab):
    step = max(1, (1 << 28) // vocab)
    return [(a, min(rows, a + step)) for a in range(0, rows, step)]


def _exact_adjust(case, s):
    """Row by row, from the list of what the row's request has read and written so far."""
    vocab = case["vocab"]
    off, hist_len, prompt = s["offsets"].tolist(), s["history_len"].tolist(), s["prompt_len"].tolist()
    bias_len = s["bias_len"].tolist() if case["bias"] else None
    picks = s["mask_row"].tolist() if case["masked"] > 0 else None
    shift = torch.arange(32, device="cuda", dtype=torch.int32)
    out = torch.empty(s["rows"], vocab, dtype=torch.float64, device="cuda")
    for b in range(case["blocks"]):
        said = s["history"][b, : hist_len[b]].long()
        written = torch.bincount(said[prompt[b]:], minlength=vocab).double()
        known = torch.bincount(said, minlength=vocab) > 0
        rho, freq, pres = (float(s[name][b]) for name in ("repetition", "frequency", "presence"))
        for r in range(off[b], off[b + 1]):
            x = s["x"][r].double()
            x = torch.where(known & (x > 0), x / rho, torch.where(known, x * rho, x))
            x = x - freq * written - pres * written.clamp(max=1.0)
            if bias_len is not None:
                x[s["bias_tokens"][b, : bias_len[b]].long()] += s["bias_values"][b, : bias_len[b]].double()
            if picks is not None and picks[r] >= 0:
                bits = (s["mask"][picks[r]][:, None] >> shift) & 1
                x = x.masked_fill(bits.reshape(-1)[:vocab] == 0, FILL[case["fill"]])
            out[r] = x
            tok = s["draft_tokens"][r].long()
            written[tok] += 1.0
            known[tok] = True
    return out


def _exact_topk(case, s):
    values, lse = [], []
    for a, b in _chunks(case["rows"], case["vocab"]):
        y = s["y"][a:b].double()
        y = torch.sort(y, 1, descending=True).values
        values.append(y[:, : case["k"]].clone())
        lse.append(torch.logsumexp(y[:, case["k"]:], 1))
    return {"values": torch.cat(values), "index": None, "rest_lse": torch.cat(lse)}


def _exact_loss(case, s):
    """The gradient by the chain rule over the classes' logits (a class of one token has its logit, the class of
    all the others the log-sum-exp of theirs)."""
    alpha, tau, k = s["alpha"], s["tau"], case["k"]
    losses, grads = [], []
    for a, b in _chunks(case["rows"], case["vocab"]):
        z, index = s["z"][a:b].double(), s["top_index"][a:b].long()
        others = torch.ones_like(z, dtype=torch.bool).scatter_(1, index, False)
        lse = torch.logsumexp(z.masked_fill(~others, -math.inf), 1, keepdim=True)
        c = torch.cat([z.gather(1, index), lse], 1)
        t = torch.cat([s["top_logit"][a:b].double(), s["rest_lse"][a:b, None].double()], 1)
        with torch.enable_grad():
            c.requires_grad_(True)
            log_p, log_q = torch.log_softmax(c, 1), torch.log_softmax(t, 1)
            if case["kl"] == "reverse":
                term = log_p.exp() * (log_p - log_q)
            else:
                term = log_q.exp() * (log_q - log_p)
            first = s["top_logit"][a:b].argmax(1, keepdim=True)
            loss = alpha * torch.where(term <= tau, term, torch.full_like(term, tau)).sum(1)
            loss = loss - (1.0 - alpha) * log_p.gather(1, first)[:, 0]
            (d,) = torch.autograd.grad((loss * s["grad_loss"][a:b].double()).sum(), c)
        dz = torch.where(others, (z - lse).exp() * d[:, k:], 0.0)
        dz.scatter_(1, index, d[:, :k])
        losses.append(loss.detach())
        grads.append(dz)
    return {"loss": torch.cat(losses), "dz": torch.cat(grads)}
