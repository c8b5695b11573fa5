"""route_sort at the numbers of partitions around which its kernels' shared memory
passes 48 KB, each in a process of its own: the limit that a launch needs raised
stays raised for the calls behind it."""
import os
import subprocess
import sys

import pytest

from helpers import need_gpu

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
RUN = """
import sys, torch
import delta_rule_memory_gb300 as sdm
M, N = int(sys.argv[1]), int(sys.argv[2])
sel = torch.randint(0, N, (M, 2), generator=torch.Generator().manual_seed(N), dtype=torch.int32)
order, place, offsets = (x.cpu().long() for x in sdm.route_sort(sel.cuda(), N))
flat = sel.flatten().long()
want = torch.argsort(flat, stable=True)
inverse = torch.empty_like(want)
inverse[want] = torch.arange(2 * M)
assert torch.equal(order, want) and torch.equal(place.flatten(), inverse)
assert torch.equal(offsets[1:], torch.bincount(flat, minlength=N).cumsum(0)) and int(offsets[0]) == 0
"""


@pytest.mark.parametrize("M,N", [(500, 680), (500, 681), (500, 682), (5000, 682), (500, 683), (5000, 768), (500, 769)])
def test_first_call_of_a_process(M, N):
    need_gpu()
    r = subprocess.run([sys.executable, "-c", RUN, str(M), str(N)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
