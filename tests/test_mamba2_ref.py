"""The plain 64-bit forms of the Mamba-2 layer's parts, pinned on the CPU:
gradients by differences, the convolution by numpy's, steps by whole sequences."""
import numpy as np
import pytest

import mamba2_ref as ref


def test_conv_is_numpys():
    rng = np.random.default_rng(1)
    x, w, b = rng.standard_normal((1, 30, 4)), rng.standard_normal((4, 3)), rng.standard_normal(4)
    v, _ = ref.token_conv(x, w, b, silu=False)
    for d in range(4):
        full = np.convolve(x[0, :, d], w[d, ::-1])[:30] + b[d]
        assert np.allclose(v["out"][0, :, d], full, rtol=0, atol=1e-13)
    assert np.array_equal(v["state"][0], x[0, -3:].T)


@pytest.mark.parametrize("cu", [None, [1, 1, 2, 6, 6, 8]])
@pytest.mark.parametrize("K", [1, 3, 4])
def test_conv_gradients_are_the_differences(cu, K):
    rng = np.random.default_rng(2)
    lead, n = ((2, 5), 2) if cu is None else ((9,), len(cu) - 1)
    args = dict(x=rng.standard_normal(lead + (2,)), w=rng.standard_normal((2, K)), b=rng.standard_normal(2),
                state=rng.standard_normal((n, 2, K)))
    dout, dstate = rng.standard_normal(lead + (2,)), rng.standard_normal((n, 2, K))

    def loss(x, w, b, state):
        v, _ = ref.token_conv(x, w, b, state=state, cu=cu)
        return (v["out"] * dout).sum() + (v["state"] * dstate).sum()

    g, _ = ref.token_conv(args["x"], args["w"], args["b"], state=args["state"], cu=cu, dout=dout, dstate=dstate)
    for name, key in (("x", "dx"), ("w", "dweight"), ("b", "dbias"), ("state", "dstate_in")):
        for idx in np.ndindex(args[name].shape):
            step = 1e-5
            up, dn = ({k: t.copy() for k, t in args.items()} for _ in range(2))
            up[name][idx] += step
            dn[name][idx] -= step
            d = (loss(**up) - loss(**dn)) / (2 * step)
            # central differences: step^2 of the third derivative, and 2^-53 |loss| / step
            assert abs(d - g[key][idx]) <= 1e-6 * (1 + abs(d)), (key, idx)


def test_conv_steps_are_the_sequence():
    rng = np.random.default_rng(3)
    x, w, b, state = rng.standard_normal((2, 7, 3)), rng.standard_normal((3, 4)), rng.standard_normal(3), rng.standard_normal((2, 3, 4))
    v, _ = ref.token_conv(x, w, b, state=state)
    pool = state
    for t in range(7):
        out, _, pool = ref.conv_step(pool, x[:, t], w, b)
        assert np.allclose(out, v["out"][:, t], rtol=0, atol=1e-13)
    assert np.array_equal(pool, v["state"])


def test_ssd_step_is_the_recurrence():
    """One channel and one state, written out."""
    rng = np.random.default_rng(4)
    state = rng.standard_normal((1, 1, 1, 1))
    h = state[0, 0, 0, 0]
    for _ in range(5):
        x, dt, B, C, z = rng.standard_normal(5)
        A, D, bias = -abs(rng.standard_normal()), rng.standard_normal(), rng.standard_normal()
        out, _, state, _ = ref.ssd_step(state, [[[x]]], [[dt]], [A], [[[B]]], [[[C]]], D=np.array([D]), z=np.array([[[z]]]),
                                        bias=np.array([bias]))
        step = np.log(1 + np.exp(dt + bias))
        h = np.exp(step * A) * h + step * B * x
        assert np.isclose(state[0, 0, 0, 0], h, rtol=1e-12)
        assert np.isclose(out[0, 0, 0], (C * h + D * x) * z / (1 + np.exp(-z)), rtol=1e-12)


def _scan_inputs(rng, lead, n, H=2, P=2, G=1, N=2):
    return dict(x=rng.standard_normal(lead + (H, P)), dt=rng.standard_normal(lead + (H,)), A=-np.exp(rng.standard_normal(H)),
                B=rng.standard_normal(lead + (G, N)), C=rng.standard_normal(lead + (G, N)), D=rng.standard_normal(H),
                z=rng.standard_normal(lead + (H, P)), bias=rng.standard_normal(H), h0=rng.standard_normal((n, H, P, N)))


def test_ssd_steps_are_the_scan():
    rng = np.random.default_rng(5)
    t = _scan_inputs(rng, (2, 6), 2, H=4, P=3, G=2, N=5)
    v, _ = ref.ssd_scan(**t)
    state = t["h0"]
    for k in range(6):
        out, _, state, _ = ref.ssd_step(state, t["x"][:, k], t["dt"][:, k], t["A"], t["B"][:, k], t["C"][:, k], D=t["D"],
                                        z=t["z"][:, k], bias=t["bias"])
        assert np.allclose(out, v["out"][:, k], rtol=1e-12, atol=1e-12)
    assert np.allclose(state, v["last"], rtol=1e-12)


@pytest.mark.parametrize("cu", [None, [1, 1, 2, 5, 5, 8]])
def test_ssd_gradients_are_the_differences(cu):
    rng = np.random.default_rng(6)
    lead, n = ((2, 4), 2) if cu is None else ((9,), len(cu) - 1)
    args = _scan_inputs(rng, lead, n)
    dout, dlast = rng.standard_normal(lead + (2, 2)), rng.standard_normal((n, 2, 2, 2))

    def loss(**kw):
        v, _ = ref.ssd_scan(cu=cu, **kw)
        return (v["out"] * dout).sum() + (v["last"] * dlast).sum()

    g, _ = ref.ssd_scan(cu=cu, dout=dout, dlast=dlast, **args)
    for name, key in (("x", "dx"), ("dt", "ddt"), ("A", "dA"), ("B", "dB"), ("C", "dC"), ("D", "dD"), ("z", "dz"),
                      ("bias", "ddt_bias"), ("h0", "dh0")):
        for idx in np.ndindex(args[name].shape):
            step = 1e-5
            up, dn = ({k: t.copy() for k, t in args.items()} for _ in range(2))
            up[name][idx] += step
            dn[name][idx] -= step
            d = (loss(**up) - loss(**dn)) / (2 * step)
            # central differences: step^2 of the third derivative, and 2^-53 |loss| / step
            assert abs(d - g[key][idx]) <= 1e-6 * (1 + abs(d)), (key, idx)
