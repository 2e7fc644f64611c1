"""The sines and cosines of sage_rope by themselves: x = (1, 0) turns into (cos, sin), in float32 without a
further rounding.

Tolerance: freq / 2 pi in float64, |p freq| 2^-52; what is left of the angle beside the nearest quarter turn,
r half turns, is cut at 2^-33 and rounded once, pi (2^-33 + 2^-24 |r|); the sine and cosine of that are within
2 units in the last place, 2^-22 of the value.  Near the quarter turns the smaller of the two is small, and exact to its own size."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("near", [True, False])
def test_sines_and_cosines(near, inverse):
    import bit_trainable_attention_sage_gb300 as sg
    rng = np.random.default_rng(int(near))
    n = 4096
    pos = np.concatenate([rng.integers(-20000, 20000, n - 5), [0, 1, -1, 2, 3]]).astype(np.int64)
    # frequencies that put positions all around, or next to quarter turns
    eps = 10.0 ** np.linspace(-9, -4, 8)
    freqs = [float(q * np.pi / 2 + (e if near else 0.1 + 1e3 * e)) for q, e in zip((1, 2, 3, 4, -1, -2, 5, 0), eps)]
    rope = sg.make_rope(64, (8,), freqs=freqs)
    Q = torch.zeros(1, 1, n, 64)
    Q[..., :8] = 1.0
    out, _ = sg.sage_rope(Q.cuda(), None, torch.from_numpy(pos).int().view(1, 1, n).cuda(), rope, inverse=inverse)
    got = out[0, 0].double().cpu().numpy()
    for j, f in enumerate(freqs):
        # the angle in extended precision; the quarter turn taken off with pi to 36 digits in two parts
        a = pos.astype(np.longdouble) * np.longdouble(f)
        want = {0: np.cos(a), 8: np.sin(-a if inverse else a)}
        half_pi = np.longdouble("1.57079632679489661923132169163975144")
        r = np.abs(a - np.rint(a / half_pi) * half_pi) / (2 * half_pi)
        for at, w in want.items():
            tol = np.abs(a) * 2.0 ** -52 + np.pi * (2.0 ** -33 + 2.0 ** -24 * r) + 2.0 ** -22 * np.abs(w)
            err = np.abs(got[:, at + j] - w)
            assert np.all(err <= tol), (j, at, float((err / tol).max()))
