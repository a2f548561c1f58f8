"""Pins of the 8-bit decoder's float64 oracle (oracle/fp8.py): the e4m3 values by enumeration, blocks by hand, the norm's
gradient by differences, the product by dequantised values (CPU)."""
import numpy as np
import pytest
import torch

from oracle import fp8


def _all_e4m3():
    """Every finite value of the format, from its bits."""
    v = []
    for bits in range(128):
        e, m = bits >> 3, bits & 7
        if bits != 127:  # NaN
            v.append(m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return np.array(v)


def test_rounding_takes_the_nearest_value_and_even_ones_of_two():
    table = _all_e4m3()
    assert table[-1] == fp8.TOP and len(table) == 127 and (np.diff(table) > 0).all()
    v = np.concatenate([np.random.default_rng(0).uniform(-500, 500, 4000), np.random.default_rng(1).uniform(-0.05, 0.05, 4000), table,
                        (table[1:] + table[:-1]) / 2])
    for x, got in zip(v, fp8.round_e4m3(v)):
        off = np.abs(table - abs(x))
        near = np.flatnonzero(off == off.min())
        want = table[near[0] if len(near) == 1 or near[0] % 2 == 0 else near[1]]
        assert got == np.sign(x) * want, x
    assert (torch.tensor(v).float().clamp(-448, 448).to(torch.float8_e4m3fn).double().numpy() == fp8.round_e4m3(v.astype(np.float32))).all()


@pytest.mark.parametrize("rows,cols,block", [(3, 300, 1), (130, 129, 128), (1, 1, 128), (256, 128, 128)])
def test_blocks(rows, cols, block):
    x = np.random.default_rng(rows).standard_normal((rows, cols)) * 10
    x[0, :] = 0
    q, s = fp8.quantize(x, block)
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            part = x[i * block:(i + 1) * block, j * 128:(j + 1) * 128]
            assert s[i, j] == (np.abs(part).max() / 448 if np.abs(part).max() else 1)
            got = q[i * block:(i + 1) * block, j * 128:(j + 1) * 128] * s[i, j]
            assert np.abs(got).max() == pytest.approx(np.abs(part).max(), rel=1e-15)
            assert (np.abs(got - part) <= np.maximum(2.0 ** -4 * np.abs(part), 2.0 ** -10 * s[i, j]) * (1 + 1e-12)).all()
    b = np.random.default_rng(7).standard_normal((5, cols))
    qb, sb = fp8.quantize(b, 1)
    out, size = fp8.matmul(qb, sb, q, s)
    for m in range(5):
        for n in range(min(rows, 4)):
            terms = [qb[m, k] * sb[m, k // 128] * q[n, k] * s[n // block, k // 128] for k in range(cols)]
            assert out[m, n] == pytest.approx(sum(terms), rel=1e-12, abs=1e-12 * sum(map(abs, terms)))
            assert size[m, n] == pytest.approx(sum(map(abs, terms)), rel=1e-12, abs=0)


def test_norm_gradient_by_differences():
    g = np.random.default_rng(3)
    h, w, dy, dh = g.standard_normal((4, 30)), g.standard_normal(30), g.standard_normal((4, 30)), g.standard_normal((4, 30))
    dx, dw = fp8.rms_norm_bwd(dy, h, w, dh, 1e-3)

    def loss(h, w):
        return (fp8.rms_norm_fwd(h, None, w, 1e-3)[0] * dy).sum() + (h * dh).sum()

    for got, at in ((dx, 0), (dw, 1)):
        u = g.standard_normal(got.shape)
        args = [[h, w], [h, w]]
        args[0][at], args[1][at] = args[0][at] + 1e-5 * u, args[1][at] - 1e-5 * u
        assert (got * u).sum() == pytest.approx((loss(*args[0]) - loss(*args[1])) / 2e-5, rel=1e-7, abs=1e-8)


def test_clip_by_hand():
    norm, got = fp8.clip([np.array([3.0]), np.array([[0.0, 4.0]])], 1.0, 0.0)
    assert norm == 5 and got[0][0] == pytest.approx(0.6) and got[1][0, 1] == pytest.approx(0.8)
    assert fp8.clip([np.array([3.0])], 4.0, 0.0)[1][0][0] == 3
