"""Pins of the logit-adjustment oracle against things other than itself (CPU only): worked examples by
hand, and step-by-step decoding (a block's row j is the first row of a block whose history ends with the
proposals before it)."""

import numpy as np

from oracle import adjust as A


def test_worked_example():
    x = np.array([[2.0, -2.0, 1.0, 0.5, -1.0, 3.0]])
    out, _, flags = A.adjust_rows(
        x, [0, 1], history=np.array([[0, 1, 2, 2]]), history_len=[4], prompt_len=[2], repetition=[2.0],
        frequency=[0.25], presence=[0.5], bias_tokens=np.array([[3, 3, 5]]), bias_values=np.array([[9.0, 1.0, -1.0]]),
        bias_len=[3], mask=np.array([[1, 1, 1, 1, 0, 1]], dtype=bool), masked_value=-7.0)
    # 0, 1: prompt only; 2: twice in the output; 3: bias, its last entry; 4: masked; 5: bias
    assert out[0].tolist() == [1.0, -4.0, 1.0 / 2 - 2 * 0.25 - 0.5, 1.5, -7.0, 2.0]
    assert flags == 0


def test_rows_of_a_block_are_steps_of_decoding():
    rng = np.random.default_rng(3)
    V, n = 40, 5
    x = rng.normal(0, 3, (n, V))
    hist = rng.integers(0, V, (1, 12))
    draft = rng.integers(0, V, n)
    args = dict(repetition=[1.3], frequency=[0.2], presence=[0.4])
    block, _, _ = A.adjust_rows(x, [0, n], history=hist, history_len=[12], prompt_len=[5], draft_tokens=draft, **args)
    for j in range(n):
        grown = np.concatenate([hist, draft[None, :j]], 1)
        step, _, _ = A.adjust_rows(x[j:j + 1], [0, 1], history=grown, history_len=[12 + j], prompt_len=[5], **args)
        assert np.array_equal(step[0], block[j])


def test_flags_and_untouched_rows():
    x = np.zeros((4, 8))
    out, _, flags = A.adjust_rows(x, [0, 2, 1], history=np.array([[1, 9], [0, 0]]), history_len=[5, 0])
    assert flags == A.FLAG_BAD_OFFSETS | A.FLAG_BAD_TOKEN | A.FLAG_BAD_LIST
    assert np.isnan(out[2:]).all() and not np.isnan(out[:2]).any()
    mask = np.zeros((1, 8), dtype=bool)
    out, _, flags = A.adjust_rows(x, [0, 2], mask=mask, mask_row=[0, -1])
    assert flags == A.FLAG_EMPTY_MASK and (out[0] == -1e4).all() and (out[1] == 0).all()
