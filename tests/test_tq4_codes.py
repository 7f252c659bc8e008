"""The TQ4 code of a value without its division: |y| > s * midpoint decides as the
rounded quotient does, for every fp16 scale (the arithmetic of csrc/tq4_code.cuh, in
numpy's IEEE fp32)."""
import numpy as np
import pytest

MAG = np.array([0.12841796875, 0.387939453125, 0.65673828125, 0.9423828125, 1.255859375, 1.6181640625, 2.068359375,
                2.732421875], np.float32)
MID = (MAG[:-1] + MAG[1:]) * np.float32(0.5)
SCALES = np.arange(1, 0x7C00, dtype=np.uint16).view(np.float16).astype(np.float32)  # every positive finite one


@pytest.mark.parametrize("j", range(7))
def test_thresholds_are_exact_products(j):
    t = SCALES * MID[j]
    assert (t.astype(np.float64) == SCALES.astype(np.float64) * float(MID[j])).all()
    up, down = np.nextafter(t, np.float32(np.inf)), np.nextafter(t, np.float32(0))
    for y in (t, up, down, np.nextafter(up, np.float32(np.inf)), np.nextafter(down, np.float32(0))):
        assert ((y / SCALES > MID[j]) == (y > t)).all()


def test_sign_of_a_quotient_that_underflows():
    y = -np.concatenate([np.arange(1 << 17, dtype=np.uint32).view(np.float32),
                         np.array([1e-38, 1e-30, 1.0, 1e38, 3e38, np.inf], np.float32)])
    with np.errstate(all="ignore"):
        for s in SCALES[::37]:
            assert ((y / s < 0) == (y * np.float32(2.0 ** 126) < np.float32(-2.0 ** -24) * s)).all()
