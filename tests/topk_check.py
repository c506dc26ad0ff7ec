"""What an fp32 evaluation of the top-k distillation loss may be off by, for the GPU tests.

With u = 2^-24: every log-probability of a class (lp, lq) is a difference of numbers each rounded once,
with the error e = u (n + 64) of the sums behind it, n = additions one thread makes (at most ceil(V / 256)
+ 16; the joins, exp2 and the exponents' rounding, at most 24 u ln 2 where terms count, are in the 64),
and 4 u of its own magnitude. A class's probability has that as its relative error. So term and
derivative of class c are off by at most w_c ((|l_c| + 2) d_c + d_c), d_c = e + 4 u (|lp_c| + |lq_c|), where
w_c is the probability in front of the logarithms. A term within its own error of tau may be clipped or not:
its whole derivative is allowed for. Results below the smallest normal number may be flushed to 0.
"""

import numpy as np

U = 2.0 ** -24
TINY = 2.0 ** -125


def _finite(x):
    return np.where(np.isfinite(x), x, 0.0)


def bounds(info, alpha, tau, kl, V):
    """(loss, each class's derivative, jump allowed to the sum of the derivatives) error bounds."""
    lp, lq = _finite(info["lp"]), _finite(info["lq"])
    p, q = np.exp(info["lp"]), np.exp(info["lq"])
    e = U * ((V + 255) // 256 + 16 + 64)
    d = e + 4 * U * (np.abs(lp) + np.abs(lq))
    l = np.abs(lp - lq)
    w = p if kl == "reverse" else q
    err = w * ((l + 2) * d + d) + p * d
    near = np.abs(info["term"] - tau) <= err
    jump = float(np.sum(np.where(near, w * (l + 1), 0.0)))
    beta = 1 - alpha
    loss = alpha * float(err.sum()) + beta * float(d[info["place"]] * (1 + abs(lp[info["place"]])))
    total = float(err.sum()) + jump
    # d_c = alpha (p_c g_c - p_c sum) + beta (p_c - hard)
    der = alpha * (err + p * (total + float(np.sum(w * (l + 1))) * d) + np.where(near, w * (l + 1), 0.0)) + 2 * beta * p * d
    der = der + 4 * U * (alpha * w * (l + 1) + alpha * p * float(np.sum(w * (l + 1))) + beta)
    return loss + 4 * U, der


def check_row(z, info, dz_ref, got_loss, got_dz, alpha, tau, kl, weight, half):
    V = z.size
    if not info["active"]:
        assert got_loss == 0.0 and not np.any(got_dz)
        return
    loss_tol, der = bounds(info, alpha, tau, kl, V)
    ref = info["loss"]
    if np.isinf(ref):
        assert got_loss == ref
    else:
        assert abs(got_loss - ref) <= loss_tol + 2 * U * abs(ref), (got_loss, ref, loss_tol)
    # a listed token has its class's error, any other its share of the rest's and that of its own exponent
    tol = np.zeros(V)
    tol[info["tok"]] = der[:-1]
    if np.isfinite(info["rest"]):
        o = info["others"]
        share = np.exp(z[o] - info["rest"])
        e = U * ((V + 255) // 256 + 16 + 64)
        expo = e + 4 * U * np.abs(_finite(z[o] - info["rest"]))
        tol[o] = share * der[-1] + np.abs(dz_ref[o]) / max(abs(weight), 1e-300) * expo
    tol = abs(weight) * tol * (1 + half) + half * np.abs(dz_ref) + 2 * U * np.abs(dz_ref) + TINY * max(1.0, abs(weight))
    worst = np.abs(got_dz - dz_ref) - tol
    j = int(np.argmax(worst))
    assert worst[j] <= 0, (j, got_dz[j], dz_ref[j], tol[j])
