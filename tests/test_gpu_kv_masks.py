"""The 16-bit cache's attentions beside what a row does not attend to: requests
whose length is below the step's own tokens.  Against the plain 64-bit forms
(tests/kv_ref.py, which derives the tolerances)."""
import math

import pytest

torch = pytest.importorskip("torch")

from tests import kv_ref as ref  # noqa: E402
from tests.test_gpu_kv import BF16, F16, _attend, _lists  # noqa: E402

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


def _shorten(step, r, n):
    """Request r's length, of which its pages in hand are more."""
    step.lens[r], step.lens_list[r] = n, n


@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("H,new", [(8, [3, 5, 40]), (8, [40, 70, 3]), (1, [200, 1, 150]), (128, [2, 3, 2])])
def test_rows_without_a_position(H, new, dtype, sparse):
    """A NaN or an infinity in the pages of a request whose tokens attend to nothing."""
    step = ref.Step([300, 300, 400], new, H=H, Hk=1, page=16, dtype=dtype, seed=H + new[0], pad=1)
    q, k, v = step.rows()
    idx = _lists(step, 5) if sparse else None
    if sparse:  # they list pages all the same, the first ones among them
        idx[:step.first_list[2], :, :3] = torch.arange(3, dtype=torch.int32, device=idx.device)
        idx[:step.first_list[2], :, 3:] = -1
    _shorten(step, 0, new[0] - 1)
    _shorten(step, 1, -7)
    for kk, vv in ((math.nan, 1.0), (math.inf, 1.0), (-math.inf, 1.0), (1.0, math.nan), (1.0, -math.inf)):
        for r in (0, 1):
            ids = step.tables[r, :3].long()
            k[ids, 1::2], v[ids, 1::2] = kk, vv
        o, lse = _attend(step, q, k, v, 0.1, idx)
        few = step.first_list[2]
        assert (o[:few] == 0).all() and (lse[:few] == -math.inf).all()
