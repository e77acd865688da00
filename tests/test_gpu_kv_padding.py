"""PagedKV's steps with room for more tokens than they have, and steps that are
refused."""
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_kv import BF16, _dsa  # noqa: E402

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


def test_padding_of_a_step():
    """Rows past the step's last token, and all of a step that is refused, come back as zeros."""
    dsa, dev = _dsa(), "cuda:0"
    i32 = dict(dtype=torch.int32, device=dev)
    c = dsa.PagedKV(requests=2, pages=8, pages_per_request=4, page_size=16, kv_heads=2, inv_freq=[0.5, 0.25] * 4)
    for lens, fresh, taken in (([20, 3], [20, 3], 23), ([20, 70], [0, 67], 0), ([21, 4], [1, 1], 2)):
        x = torch.randn(40 if taken else 70, 12, 128, device=dev).to(BF16)
        c.step(torch.tensor(lens, **i32), torch.tensor(fresh, **i32), x.shape[0])
        # memory that has been used: what is left as it was is not zeros
        junk = [torch.full((x.shape[0], 8, 128), 7.0, dtype=BF16, device=dev) for _ in range(4)]
        del junk
        q = c.append(x[:, :8], x[:, 8:10], x[:, 10:])
        assert (q[taken:] == 0).all() and (q[:taken] != 0).any(-1).all()
