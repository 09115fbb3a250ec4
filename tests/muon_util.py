"""Plain 64-bit and binary32 forms of the matrix-orthogonalising step that the
tests compare the library with (numpy / torch on the host; no library code)."""
import math

import numpy as np
import torch

COEFFS = (3.4445, -4.7750, 2.0315)

# Error of dpg_orthogonalize, relative Frobenius norm: the bf16 result rounds
# each value by at most 2^-9; the steps are held to four unit roundoffs of
# fp16 (4 * 2^-11), the precision of the stored products, over all steps.
ORTHO_REL = 2.0 ** -9 + 4 * 2.0 ** -11
# One element: its own bf16 rounding, and twelve times the steps' error spread
# evenly over the matrix.
ORTHO_ELEM = 12 * 4 * 2.0 ** -11


def newton_schulz_64(u, coeffs, eps):
    """u: [rows, cols] float64 -> float64, the steps as they are defined."""
    x = np.asarray(u, np.float64)
    x = x / max(np.linalg.norm(x), eps)
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    for a, b, c in coeffs:
        g = x @ x.T
        x = a * x + (b * g + c * (g @ g)) @ x
    return x.T if tall else x


def check_ortho(got, want, what=""):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    norm = np.linalg.norm(want)
    err = np.abs(got - want)
    assert np.all(np.isfinite(got)), what
    if norm == 0.0:
        assert np.all(got == 0.0), what
        return
    rel = np.linalg.norm(got - want) / norm
    assert rel <= ORTHO_REL, f"{what}: relative error {rel:.3e}"
    bound = 2.0 ** -8 * np.abs(want) + ORTHO_ELEM * norm / math.sqrt(want.size)
    assert np.all(err <= bound), f"{what}: element error {np.max(err / bound):.2f} of its bound"


def momentum_f32(grads, last, tokens, mu, nesterov, m):
    """The binary32 operations of dpg_muon_momentum, in their order."""
    f = np.float32
    s = None
    for r, g in enumerate(grads):
        x = np.asarray(g, f)
        if last is not None:
            x = x + np.asarray(last[r], f)
        s = x if s is None else s + x
    g = s * f(1.0 / float(sum(tokens)))
    omu, muf = f(1.0 - mu), f(mu)
    g = g * omu
    m = muf * m + g
    return m, (g + muf * m if nesterov else m)


def scale_of(rule_rms, rows, cols):
    return 0.2 * math.sqrt(max(rows, cols)) if rule_rms else math.sqrt(max(1.0, rows / cols))


def apply_f32(w, o, lr, wd, scale):
    f = np.float32
    if wd != 0.0:
        w = w - f(lr * wd) * w
    return w - f(lr * scale) * np.asarray(o, f)


def bf16_round(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16)


def make_matrix(kind, rows, cols, rng, scale=1e-3):
    n = rng.standard_normal
    if kind == "gauss":
        u = n((rows, cols))
    elif kind == "spiked":
        u = n((rows, cols)) + 0.5 * n((rows, 4)) @ n((4, cols))
    elif kind == "lowrank":
        k = max(1, min(rows, cols) // 16)
        u = n((rows, k)) @ n((k, cols)) + 0.01 * n((rows, cols))
    elif kind == "rank1":
        u = n((rows, 1)) @ n((1, cols))
    elif kind == "outlier":
        u = n((rows, cols))
        u[rows // 2, cols // 3] = 1000.0 * math.sqrt(max(rows, cols))
    elif kind == "equal":
        u = np.ones((rows, cols))
    elif kind == "diag":
        u = np.eye(rows, cols)
    else:
        raise ValueError(kind)
    return (scale * u).astype(np.float32)
