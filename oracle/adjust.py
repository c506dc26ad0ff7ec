"""Float64 oracle of penalties, biases and grammar masks on the rows of packed draft blocks (test
infrastructure only; see opd_oracle for the rules of its use).

The published pages name no such step; the rule is the one stated in the library's header: with c_v the
count of token v in the request's output (history behind the prompt, and the proposals of the block's
earlier rows) and known_v whether prompt or output holds it,

    x1 = known_v ? (x > 0 ? x / rho : x rho) : x
    x2 = x1 - f c_v - g [c_v > 0] + bias_v        (the last entry of a token listed twice counts)
    out = (masked) ? masked_value : x2
"""

from __future__ import annotations

import numpy as np

__all__ = ["adjust_rows", "FLAG_BAD_OFFSETS", "FLAG_BAD_TOKEN", "FLAG_BAD_LIST", "FLAG_EMPTY_MASK"]

FLAG_BAD_OFFSETS = 2
FLAG_BAD_TOKEN = 8
FLAG_BAD_LIST = 16
FLAG_EMPTY_MASK = 32


def _clamped(n, most, flags):
    if n < 0 or n > most:
        flags[0] |= FLAG_BAD_LIST
    return min(max(int(n), 0), most)


def adjust_rows(x, offsets, history=None, history_len=None, prompt_len=None, draft_tokens=None, repetition=None,
                frequency=None, presence=None, bias_tokens=None, bias_values=None, bias_len=None, mask=None,
                mask_row=None, masked_value=-1.0e4):
    """Returns (out [R, V] float64, NaN in rows outside every block, size [R, V] of the numbers added up,
    flag word). mask: bool [M, V], true = allowed."""
    x = np.asarray(x, dtype=np.float64)
    n_rows, vocab = x.shape
    out = np.full_like(x, np.nan)
    size = np.zeros_like(x)
    flags = [0]
    for b in range(len(offsets) - 1):
        s, e = int(offsets[b]), int(offsets[b + 1])
        if s < 0 or e < s or e > n_rows:
            flags[0] |= FLAG_BAD_OFFSETS
            continue
        if e == s:
            continue
        prompt, output = [], []
        if history is not None:
            n = _clamped(history_len[b], history.shape[1], flags)
            p = 0 if prompt_len is None else _clamped(prompt_len[b], n, flags)
            tokens = [int(t) for t in history[b, :n]]
            prompt, output = tokens[:p], tokens[p:]
        bias = {}
        if bias_tokens is not None:
            for i in range(_clamped(bias_len[b], bias_tokens.shape[1], flags)):
                bias[int(bias_tokens[b, i])] = float(bias_values[b, i])
        rho = 1.0 if repetition is None else float(repetition[b])
        f = 0.0 if frequency is None else float(frequency[b])
        g = 0.0 if presence is None else float(presence[b])
        if any(not 0 <= t < vocab for t in prompt + output + list(bias)):
            flags[0] |= FLAG_BAD_TOKEN
        if draft_tokens is not None and any(not 0 <= int(t) < vocab for t in draft_tokens[s:e]):
            flags[0] |= FLAG_BAD_TOKEN
        for r in range(s, e):
            said = output + ([int(t) for t in draft_tokens[s:r]] if draft_tokens is not None else [])
            row = x[r].copy()
            for t in set(prompt) | set(said):
                if 0 <= t < vocab:
                    row[t] = row[t] / rho if row[t] > 0 else row[t] * rho
            size[r] = np.abs(row)
            for t in set(said):
                if 0 <= t < vocab:
                    c = said.count(t)
                    row[t] -= f * c + g
                    size[r, t] += abs(f) * c + abs(g)
            for t, v in bias.items():
                if 0 <= t < vocab:
                    row[t] += v
                    size[r, t] += abs(v)
            if mask is not None:
                i = r if mask_row is None else int(mask_row[r])
                if i >= len(mask):
                    flags[0] |= FLAG_BAD_LIST
                elif i >= 0:
                    if not mask[i].any():
                        flags[0] |= FLAG_EMPTY_MASK
                    row[~mask[i]] = masked_value
                    size[r][~mask[i]] = 0.0  # nothing is added up there
            out[r] = row
    return out, size, flags[0]
