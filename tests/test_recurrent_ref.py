"""The plain 64-bit forms that the gated recurrence and the state cache are
tested against, themselves pinned on the CPU: gradients by differences, code
grids by their definitions, the random bytes by what a generator of its kind
must satisfy."""
import numpy as np
import pytest

import recurrent_ref as ref


def _inputs(rng, lead, D):
    x, ga, gx, dout = (rng.standard_normal(lead + (D,)) for _ in range(4))
    return x, ga, gx, dout, rng.standard_normal(D)


@pytest.mark.parametrize("cu", [None, [0, 0, 1, 5, 5, 7, 9]])
def test_gradients_are_the_differences(cu):
    rng = np.random.default_rng(7)
    lead = (2, 9) if cu is None else (9,)
    n = 2 if cu is None else len(cu) - 1
    x, ga, gx, dout, lam = _inputs(rng, lead, 3)
    h0, dlast = rng.standard_normal((n, 3)), rng.standard_normal((n, 3))

    def loss(x, ga, gx, lam, h0):
        v, _ = ref.gated_scan(x, ga, gx, lam, h0=h0, cu=cu)
        return (v["out"] * dout).sum() + (v["last"] * dlast).sum()

    g, _ = ref.gated_scan(x, ga, gx, lam, h0=h0, cu=cu, dout=dout, dlast=dlast)
    args = dict(x=x, ga=ga, gx=gx, lam=lam, h0=h0)
    for name, key in (("x", "dx"), ("ga", "dgate_a"), ("gx", "dgate_x"), ("lam", "dlam"), ("h0", "dh0")):
        for idx in np.ndindex(args[name].shape):
            step = 1e-5
            up, dn = ({k: t.copy() for k, t in args.items()} for _ in range(2))
            up[name][idx] += step
            dn[name][idx] -= step
            d = (loss(**up) - loss(**dn)) / (2 * step)
            # central differences: step^2 of the third derivative, and 2^-53 |loss| / step
            assert abs(d - g[key][idx]) <= 1e-6 * (1 + abs(d)), (key, idx)


def test_empty_and_outside_tokens():
    rng = np.random.default_rng(8)
    x, ga, gx, dout, lam = _inputs(rng, (8,), 2)
    h0 = rng.standard_normal((3, 2))
    v, _ = ref.gated_scan(x, ga, gx, lam, h0=h0, cu=[2, 2, 5, 6], dout=dout)
    assert np.array_equal(v["last"][0], h0[0]) and np.array_equal(v["dh0"][0], np.zeros(2))
    assert not v["out"][:2].any() and not v["out"][6:].any() and not v["dx"][6:].any()


def test_grids():
    g8, g4 = ref.grid("fp8"), ref.grid("fp4")
    assert g8[1] == 2.0 ** -9 and g8[8] == 2.0 ** -6 and g8[-1] == 448 and len(g8) == 127
    assert np.all(np.diff(g8) > 0) and np.all(np.diff(g4) > 0)


@pytest.mark.parametrize("fmt", ["int8", "fp8", "fp4"])
def test_encode_is_nearest_and_in_range(fmt):
    rng = np.random.default_rng(9)
    v = rng.standard_normal((40, 50)) * np.exp(3 * rng.standard_normal((40, 1)))
    codes, scales = ref.encode(v, fmt)
    back = ref.decode(codes, scales, fmt)
    unit = np.repeat(2.0 ** (scales.astype(float) - 127), 32, -1)[:, :50]
    assert np.all(np.abs(v) <= ref.MOST[fmt] * unit)
    assert np.all(np.maximum.reduceat(np.abs(v), [0, 32], 1) > ref.MOST[fmt] * unit[:, [0, 32]] / 2)
    if fmt == "int8":
        assert np.all(np.abs(back - v) <= unit / 2)
    else:
        every = np.concatenate((-ref.grid(fmt)[::-1], ref.grid(fmt)))
        best = np.abs(v[..., None] - every * unit[..., None]).min(-1)
        assert np.array_equal(np.abs(back - v), best)


def test_philox_is_a_bijection_of_the_counter_and_flat():
    """Different counters never meet (each round is invertible), and the bytes
    of many are even: 4096 x 16 bytes over 256 values, chi-square within 6
    sigma of its mean 255 (sigma = sqrt(2 * 255))."""
    seen, counts = set(), np.zeros(256)
    for ch in range(4096):
        b = ref.philox_bytes(0x123456789ABCDEF, ch, 3, 16)
        seen.add(bytes(b.astype(np.uint8)))
        counts += np.bincount(b, minlength=256)
    assert len(seen) == 4096
    mean = 4096 * 16 / 256
    assert abs(((counts - mean) ** 2 / mean).sum() - 255) < 6 * np.sqrt(510)
