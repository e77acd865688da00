"""The choice of pages by a warp a row (608 rows and more, 48 free pages at most)
on inputs that it does not settle at once: equal and neighbouring scores, NaN,
infinities, pages without an id, lists that do not fit, parts of a step.  Against
the plain 64-bit form (tests/kv_ref.py)."""
import math

import pytest

torch = pytest.importorskip("torch")

from tests import kv_ref as ref  # noqa: E402
from tests.test_gpu_kv import BF16, F16, _select  # noqa: E402

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


def _step(dtype=BF16, lens=(9000, 4000, 40, 12000), new=(300, 200, 1, 204), Hk=2, n=4, seed=1, **kw):
    step = ref.Step(list(lens), list(new), H=Hk * n, Hk=Hk, page=16, dtype=dtype, seed=seed, pad=2, **kw)
    assert sum(new) * Hk >= 4 * 160  # a warp a row on any device of up to 160 SMs
    return step, step.normal(step.T, step.H, 128), step.normal(step.pages, Hk, 128)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("kinds", [1, 5, 150])
def test_equal_scores(kinds, dtype):
    """Hundreds of equal scores: more than a row's list holds."""
    step, q, means = _step(dtype, seed=kinds)
    means = means[:kinds][torch.arange(step.pages, device=q.device) % kinds].contiguous()
    _select(step, means, q, 16, 1, 1)
    _select(step, means, q, 50, 1, 1)  # 48 free ones, the most
    _select(step, torch.zeros_like(means), q, 16, 1, 1)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_neighbours_in_rank(dtype):
    """Scores apart by one element's last bit."""
    step, q, means = _step(dtype, seed=7)
    means = means[:1].repeat(step.pages, 1, 1).contiguous()
    bits = means.view(torch.int16)
    for g, d in ((0, 1), (1, -1)):
        bits[torch.arange(step.pages), g, torch.randint(128, (step.pages,), generator=step.gen)] += d
    for n, lead, trail in ((16, 1, 1), (50, 1, 1), (3, 0, 2)):
        _select(step, means, q, n, lead, trail)


@pytest.mark.parametrize("alike", [0.9, 0.98, 0.999])
def test_pages_like_their_neighbours(alike):
    """Means that vary slowly along the context: those that score highest stand side by side."""
    step, q, means = _step(BF16, lens=(12000, 30000), new=(320, 320), seed=int(1000 * alike))
    noise, x = torch.randn(2, step.P, 2, 128, generator=step.gen, dtype=torch.float64), torch.zeros(2, 2, 128, dtype=torch.float64)
    for j in range(step.P):
        x = alike * x + math.sqrt(1 - alike * alike) * noise[:, j]
        for r in range(2):
            if int(step.tables[r, j]) >= 0:
                means[int(step.tables[r, j])] = x[r].to(BF16).to(means.device)
    _select(step, means, q, 16, 1, 2)
    _select(step, means, q, 40, 0, 1)


@pytest.mark.parametrize("q_size,m_size,dtype", [(1e30, 1e-30, BF16), (1e-36, 1e-20, BF16), (6e4, 6e4, F16), (1e-6, 1e-6, F16),
                                                 (1e38, 1e38, BF16)])
def test_magnitudes(q_size, m_size, dtype):
    step, _, _ = _step(dtype, lens=(5000, 6000), new=(320, 320), seed=11)
    top = 6e4 if dtype == F16 else 3e38
    q = (step.normal(step.T, step.H, 128, dtype=torch.float64) * q_size).clamp(-top, top).to(dtype)
    means = (step.normal(step.pages, 2, 128, dtype=torch.float64) * m_size).clamp(-top, top).to(dtype)
    _select(step, means, q, 12, 1, 2)


def test_nan_and_infinities():
    step, q, means = _step(BF16, seed=13)
    for r in (0, 1, 3):
        ids = step.tables[r].long()
        means[ids[5], 0, 7] = math.nan
        means[ids[9], 0, 1] = math.inf
        means[ids[11], 1, 1] = -math.inf
        means[ids[12], 1, 1], means[ids[12], 1, 2] = math.inf, -math.inf
    q[3::50] = math.nan
    q[4::50, 0, 0] = math.inf
    q[5::50, :, 1] = -math.inf
    _select(step, means, q, 12, 1, 2)
    _select(step, means, q, 51, 1, 2)
    means[:] = math.nan
    _select(step, means, q, 12, 1, 2)


def test_pages_without_an_id():
    step, q, means = _step(F16, seed=17)
    step.tables[0, 2:300] = -1
    step.tables[0, 333] = step.pages
    step.tables[1, :] = 2 ** 31 - 1
    step.tables[3, ::2] = -1
    _select(step, means, q, 24, 1, 1)
    _select(step, means, q, 50, 1, 1)


def test_parts_of_a_step():
    """Rows of scores so wide that tokens are taken 128 at a time, one request running through all parts."""
    step = ref.Step([60, 3000, 500], [20, 390, 33], H=16, Hk=16, page=16, dtype=BF16, seed=19, pad=3, width=8192)
    means = step.normal(step.pages, 16, 128)
    _select(step, means, step.normal(step.T, 16, 128), 9, 1, 1)
    means[::2] = means[:1]  # lists that do not fit in each of them
    _select(step, means, step.normal(step.T, 16, 128), 9, 1, 1)
