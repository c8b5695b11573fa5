"""gdn_train and gdn_backward: a row that starts with a reset does not depend on the
state that was given, whatever that holds."""
import pytest

from helpers import need_gpu
from test_gpu_gdn_train import Case, check

pytestmark = pytest.mark.gpu

# one, two and four tiles of columns a CTA; rows by tensor copies and by the helping warps
DIMS = [(1, 150, 1, 2, 64, 48), (2, 130, 2, 2, 100, 33), (1, 100, 20, 20, 32, 128), (1, 100, 40, 40, 36, 116)]


@pytest.mark.parametrize("dims", DIMS, ids=str)
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_a_state_that_was_never_set(dims, what):
    """NaN or infinities in S_0, a reset at token 0: the call of a state of zeros."""
    sdm = need_gpu()
    c = Case(*dims, seed=1, reset=0.02)
    c.reset[:, 0] = 1
    f, b = c.reference()
    c.S0[:] = what
    check(c, c.run(sdm), f, b)
