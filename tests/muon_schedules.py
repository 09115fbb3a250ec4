"""Schedules, matrices and bounds for tests of the Newton-Schulz steps beyond
the five default ones (numpy on the host; no library code)."""
import math

import numpy as np

from muon_util import COEFFS, bf16_round, make_matrix, newton_schulz_64

# A minimax schedule for singular values from 1e-3 on (Amsel et al. 2025, "The
# Polar Express"), its published coefficients with the published 1 % of safety.
_MINIMAX = [(8.28721201814563, -23.595886519098837, 17.300387312530933),
            (4.107059111542203, -2.9478499167379106, 0.5448431082926601),
            (3.9486908534822946, -2.908902115962949, 0.5518191394370137),
            (3.3184196573706015, -2.488488024314874, 0.51004894012372),
            (2.300652019954817, -1.6689039845747493, 0.4188073119525673),
            (1.891301407787398, -1.2679958271945868, 0.37680408948524835),
            (1.8750014808534479, -1.2500016453999487, 0.3750001645474248)]
MINIMAX8 = [(a / 1.01, b / 1.01 ** 3, c / 1.01 ** 5) for a, b, c in _MINIMAX] + [(1.875, -1.25, 0.375)]

SCHEDULES = {
    "5": [COEFFS] * 5, "6": [COEFFS] * 6, "8": [COEFFS] * 8, "12": [COEFFS] * 12, "16": [COEFFS] * 16,
    "minimax5": MINIMAX8[:5], "minimax8": MINIMAX8,
    "8then2": [COEFFS] * 8 + [(2.0, -1.5, 0.5)] * 2,
    "cubic16": [(1.5, -0.5, 0.0)] * 16,
}

# Relative Frobenius error of the steps alone: any matrix at up to five default
# steps; longer schedules.
STEPS_REL = 3e-3
# five default steps where all but a few rows are zero and those depend on one
# another: bf16 updates, fp32 ones
FEW_ROWS_REL = {True: 1.2e-2, False: 6e-2}
LONG_REL = 1.5e-3
# The steps are those of a matrix this close to the given one (relative): what
# the fp32 sums and the 22 bits of X can move.
BACKWARD = 2.0 ** -21


def make_low_rank(kind, rows, cols, rng):
    n = rng.standard_normal
    m = min(rows, cols)
    if kind == "rank4":
        u = n((rows, 4)) @ n((4, cols))
    elif kind == "rank2":
        u = n((rows, 2)) @ n((2, cols))
    elif kind.startswith("rows"):   # rank two in the first rows of the shorter side, zero elsewhere
        h = int(kind[4:])
        u = np.zeros((m, max(rows, cols)))
        u[:h] = n((h, 2)) @ n((2, max(rows, cols)))
        u = u if rows <= cols else u.T
    elif kind == "near1":     # rank one and a hundredth of noise
        u = n((rows, 1)) @ n((1, cols)) + 0.01 * n((rows, cols))
    elif kind == "half":
        u = n((rows, max(1, m // 2))) @ n((max(1, m // 2), cols))
    elif kind == "tail":      # one singular value 1, the others 1e-4
        q, _ = np.linalg.qr(n((rows, m)))
        p, _ = np.linalg.qr(n((cols, m)))
        s = np.full(m, 1e-4)
        s[0] = 1.0
        u = (q * s) @ p.T
    elif kind == "repeated":  # every row (of the shorter side) twice
        u = np.repeat(n(((m + 1) // 2, max(rows, cols))), 2, axis=0)[:m]
        u = u if rows <= cols else u.T
    else:
        return make_matrix(kind, rows, cols, rng)
    return (1e-3 * u).astype(np.float32)


def condition(u, coeffs, eps, rng):
    """How far the exact result moves (relative) when u moves by BACKWARD."""
    want = newton_schulz_64(u, coeffs, eps)
    moved = 0.0
    for _ in range(2):
        e = rng.standard_normal(u.shape)
        e *= BACKWARD * np.linalg.norm(u) / np.linalg.norm(e)
        moved = max(moved, np.linalg.norm(newton_schulz_64(u + e, coeffs, eps) - want))
    return want, moved / np.linalg.norm(want)


def allowed(steps_rel, moved, elements=1 << 20):
    """The steps' own error and the rounding of the result to bf16 (at most
    2^-8 of a value, under 2^-9 in the root mean square over values of all
    mantissas), which are independent, and the conditioning: the sampled
    movements stand for others of their size up to a factor of two.  A handful
    of elements has no mean to speak of: the largest rounding counts."""
    if elements < 16:
        return 2.0 ** -8 + steps_rel + 2.0 * moved
    return 1.05 * math.hypot(2.0 ** -9, steps_rel) + 2.0 * moved


def to_dtype(u, bf16):
    return bf16_round(u).double().numpy() if bf16 else np.asarray(u, np.float64)
