"""Pins of the plain 64-bit forms that the cache's GPU tests compare with, and
the page plan's invariants on them (no GPU)."""
import numpy as np
import pytest

from tests import cache_ref as ref


def test_number_tables():
    assert ref.E4M3[0x7E] == 448.0 and ref.E4M3[0x01] == 2.0 ** -9 and ref.E4M3[0x38] == 1.0
    torch = pytest.importorskip("torch")
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, ref.E4M3, equal_nan=True)


def test_rounding_by_hand():
    # scale = e4m3(6 / 6) = 1: the elements are rounded to e2m1 as they are
    x = np.zeros(128)
    x[:16] = [6, 0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.3, -1.2, -2.4, -2.6, -5.1, 0]
    k, v = ref.expand(ref.pack(x, -x))
    assert k[:16].tolist() == [6, 0, 0.5, 1, 1, 2, 2, 4, 4, 0, -0.5, -1, -2, -3, -6, 0]
    assert np.array_equal(v, -k) and not k[16:].any()


def test_rounding_limits():
    x = np.zeros((4, 128))
    x[0, 0] = 1e6            # clipped at 6 * 448
    x[1, 3], x[1, 5] = np.inf, -7.0
    x[2, 7], x[2, 20] = np.nan, 3.0
    x[3, :16] = 2.0 ** -12   # its scale rounds to 0
    k, _ = ref.expand(ref.pack(x, x))
    assert k[0, 0] == 2688.0
    assert k[1, 3] == 2688.0 and k[1, 5] == 0.0
    assert np.isnan(k[2, :16]).all() and k[2, 20] == 3.0
    assert not k[3].any()


def test_error_of_a_rounded_row():
    # half a step of e2m1 at the top of the range (1 of 6) and a scale off by 1/16
    x = np.random.default_rng(1).standard_normal((50, 128))
    k, _ = ref.expand(ref.pack(x, x))
    top = np.abs(x.reshape(50, 8, 16)).max(-1).repeat(16, -1)
    assert (np.abs(k - x) <= top * (1 / 6 + 1 / 16)).all()


def test_attention_by_hand():
    rng = np.random.default_rng(2)
    k, v = rng.standard_normal((2, 4, 8, 1, 128))
    cache = ref.pack(k, v)
    q = rng.standard_normal((3, 2, 128))
    tables = np.array([[2, 0], [1, -1]])
    idx = np.array([[9, -1, -1], [8, 3, -1], [-1, -1, -1]])
    o, lse, _, _ = ref.attention(cache, 8, q, idx, [0, 1, 0], tables, 0.5)
    kr, vr = ref.expand(cache)
    assert np.allclose(o[0], vr[0, 1, 0]) and np.allclose(lse[0], 0.5 * q[0] @ kr[0, 1, 0])
    assert np.allclose(o[1], vr[1, 3, 0])  # position 8 of request 1 has no page
    assert not o[2].any() and np.isneginf(lse[2]).all()


def test_plan_takes_and_gives_back():
    rng = np.random.default_rng(3)
    R, P, page, pages = 7, 6, 8, 40
    tables, held = np.full((R, P), -1), np.zeros(R, int)
    free, count = rng.permutation(pages), pages
    lens = np.zeros(R, int)
    for _ in range(60):
        fresh = rng.integers(0, 9, R)
        new_lens = np.minimum(np.maximum(lens + rng.integers(-12, 14, R), fresh), P * page)
        before = (tables.copy(), held.copy(), free[:count].copy())
        s = ref.plan(page, pages, new_lens, fresh, tables, held, free, count, 64)
        if s["status"][0]:
            assert np.array_equal(s["tables"], tables) and s["count"][0] == count
            continue
        out = np.concatenate([s["tables"][s["tables"] >= 0], s["free"][:s["count"][0]]])
        assert np.array_equal(np.sort(out), np.arange(pages))  # every page once
        # a step taken back leaves everything as it was
        grown = np.maximum(new_lens, held * page)
        up = ref.plan(page, pages, grown, fresh * 0, tables, held, free, count, 0)
        if up["status"][0] == 0:
            down = ref.plan(page, pages, held * page, fresh * 0, up["tables"], up["held"], up["free"],
                            int(up["count"][0]), 0)
            assert np.array_equal(down["tables"], before[0]) and np.array_equal(down["held"], before[1])
            assert np.array_equal(down["free"][:count], before[2])
        tables, held, free, count = s["tables"], s["held"], s["free"], int(s["count"][0])
        lens = new_lens
