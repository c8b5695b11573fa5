"""What the cancelling sum's bound tells apart: the kernel's order of additions in
fp32, with and without what its roundings lose."""
import numpy as np

import glr_sums as sums


def drate(kept, ctas=16, warps=4):
    """The sum in the kernel's order: runs of 8 tokens, dealt to 4 warps of each
    CTA of a cluster, last to first; then the warps, then the CTAs."""
    f = np.float32
    x, r, g, rate = sums.constants()
    C = (sums.want()[0] / 8).astype(f)
    run = np.zeros_like(C)
    for _ in range(8):
        run = (run.astype(np.float64) + C.astype(np.float64)).astype(f)     # an FMA with dy = 1
    n = sums.TOKENS // 8
    total = np.zeros((warps, ctas, C.size), f)
    lost = np.zeros_like(total)
    for i in range(n - 1, -1, -1):
        at = i % warps, i // warps % ctas
        part = run if 8 * i < sums.PLUS else -run
        s = total[at] + part
        back = s - total[at]
        lost[at] = lost[at] + ((total[at] - (s - back)) + (part - back))
        total[at] = s
    if kept:
        total = total + lost
    out = np.zeros_like(C)
    for c in range(ctas):
        w = total[0, c]
        for k in range(1, warps):
            w = w + total[k, c]
        out = out + w
    return out.astype(np.float64)


def test_the_bound_holds_with_the_losses_and_not_without():
    value, bound = sums.want()
    for ctas in (15, 16):
        assert np.all(np.abs(drate(True, ctas) - value) <= bound)
        assert np.mean(np.abs(drate(False, ctas) - value) > bound) > 0.5
