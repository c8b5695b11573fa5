"""Inputs on which the sum for drate cancels, and what it comes to.

Every token resets and x, r and g are the same at each, so drate's term of a
token is C dy_t with one C a channel.  dy is 1 over the first tokens and -1 over
the rest, 8 tokens (a run of the kernel) more of the first kind: the true sum is
8 C, while partial sums reach K = T / 16 / (threads of a channel) runs.

Bound.  C = s_r a (a / m) s_g: both sigmoids, a twice, m, and 6 roundings.  A
run's sum: 8 roundings, the same for 1 and -1 but for the sign, so whole runs
cancel without a rest.  The runs' sum keeps what its roundings lose: a loss is at
most E K runs, 2 K of them at most 2 K^2 E, and their own additions lose 2 K E of
that, 4 K^3 E^2: below E for K <= 128.  Then the addition of the loss, 3 warps and
15 CTAs over sums of at most two runs each: with 64 of those, 2 E a run and
addition."""
import numpy as np

import glr_reference as ref

E = ref.E
TOKENS, CHANNELS = (1 << 17) + 8, 64
PLUS = (TOKENS // 8 // 2 + 1) * 8       # tokens with dy = 1


def constants():
    """x, r, g and rate of the channels; values that bf16 holds."""
    rng = np.random.default_rng(71)
    x = np.full(CHANNELS, 1.0)
    r, g = (np.round(rng.normal(size=CHANNELS) * 32) / 32 for _ in range(2))
    return x, r, g, rng.uniform(0.2, 0.8, CHANNELS).astype(np.float32).astype(np.float64)


def want():
    """drate and its bound."""
    x, r, g, rate = constants()
    sr, sg, a, m, e_a, d_m = ref.gates(x, r, g, rate)
    C = sr * a * (a / m) * sg * x
    rel = 2 * e_a / a + d_m + ref.rel_sig(r) + ref.rel_sig(g) + 6 * E
    return 8 * C, 8 * C * (rel + 8 * E + E + (1 + 3 + 15) * 2 * E)
