"""Tensors whose offsets pass 32 bits: what lies at their end is the same bits as
the same inputs in small tensors of their own."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU machines only to be skipped
    pytest.skip("no GPU", allow_module_level=True)

import selective_state_space_74_amd as ssm  # noqa: E402

DEV = "cuda"
FAR = 2 ** 31   # elements


@pytest.fixture(autouse=True)
def room():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("less than 60 GiB of GPU memory free")
    yield
    torch.cuda.empty_cache()


def randn(*shape, seed=0, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


def far(t, rows):
    """t at the end of a tensor of that many rows, zeros before it."""
    out = torch.zeros((rows,) + t.shape[1:], dtype=t.dtype, device=DEV)
    out[rows - t.shape[0]:] = t
    return out


def bounds(*b):
    return torch.tensor(b, dtype=torch.int32, device=DEV)


def test_convolution():
    D, n = 2176, 300
    rows = FAR // D + 5000
    x, dout, w, b = randn(n, D, seed=1), randn(n, D, seed=2), randn(D, 4, seed=3, dtype=torch.float32), randn(D, seed=4, dtype=torch.float32)
    fx, fd = far(x, rows), far(dout, rows)
    near, far_ = bounds(0, 0, n), bounds(0, rows - n, rows)
    out, state = ssm.token_conv_fwd(x, w, b, cu_seqlens=near, return_state=True)
    fout, fstate = ssm.token_conv_fwd(fx, w, b, cu_seqlens=far_, return_state=True)
    assert torch.equal(fout[rows - n:], out) and torch.equal(fstate[1], state[1])
    del fout
    g = ssm.token_conv_bwd(dout, x, w, b, cu_seqlens=near)
    fg = ssm.token_conv_bwd(fd, fx, w, b, cu_seqlens=far_)
    assert torch.equal(fg["dx"][rows - n:], g["dx"])


def test_ssm():
    H, P, N, n = 32, 64, 16, 300
    rows = FAR // (H * P) + 5000
    t = dict(x=randn(n, H, P, seed=1), dt=randn(n, H, seed=2), B=randn(n, 1, N, seed=3), C=randn(n, 1, N, seed=4), z=randn(n, H, P, seed=5))
    dout = randn(n, H, P, seed=6)
    rest = dict(A=-torch.rand(H, device=DEV) - 0.5, D=randn(H, seed=7, dtype=torch.float32))
    f = {k: far(v, rows) for k, v in t.items()}
    near, far_ = bounds(0, 0, n), bounds(0, rows - n, rows)
    out, last = ssm.ssd_scan_fwd(**t, **rest, cu_seqlens=near, return_last_state=True)
    fout, flast = ssm.ssd_scan_fwd(**f, **rest, cu_seqlens=far_, return_last_state=True)
    assert torch.equal(fout[rows - n:], out) and torch.equal(flast[1], last[1])
    del fout
    g = ssm.ssd_scan_bwd(dout, **t, **rest, cu_seqlens=near)
    fg = ssm.ssd_scan_bwd(far(dout, rows), **f, **rest, cu_seqlens=far_)
    for k in ("dx", "ddt", "dz"):
        assert torch.equal(fg[k][rows - n:], g[k]), k
    # dB and dC: sums over the heads, whose split over workgroups goes by the sizes
    for k in ("dB", "dC"):
        off = (fg[k][rows - n:].double() - g[k].double()).norm() / g[k].double().norm()
        assert off <= 2 ** -8, k   # one rounding to bf16 of the same sums


def test_steps_on_pools():
    H, P, N, batch = 80, 64, 128, 2
    slots = FAR // (H * P * N) + 2
    pool = torch.zeros(slots, H, P, N, device=DEV)
    start = randn(batch, H, P, N, seed=1, dtype=torch.float32)
    at = torch.tensor([slots - 1, 3], dtype=torch.int32, device=DEV)
    pool[at.long()] = start
    args = dict(x=randn(batch, H, P, seed=2), dt=randn(batch, H, seed=3), A=-torch.rand(H, device=DEV), B=randn(batch, 1, N, seed=4),
                C=randn(batch, 1, N, seed=5))
    y = ssm.ssd_state_update(pool, slots=at, **args)
    assert torch.equal(y, ssm.ssd_state_update(start, **args)) and torch.equal(pool[at.long()], start)
    assert not pool[:3].any() and not pool[slots - 2].any()
    del pool
    D, K = 5376, 4
    slots = FAR // (D * K) + 2
    pool, start = torch.zeros(slots, D, K, device=DEV), randn(batch, D, K, seed=6, dtype=torch.float32)
    at = torch.tensor([slots - 1, 3], dtype=torch.int32, device=DEV)
    pool[at.long()] = start
    x, w = randn(batch, D, seed=7), randn(D, K, seed=8, dtype=torch.float32)
    y = ssm.token_conv_update(pool, x, w, slots=at)
    assert torch.equal(y, ssm.token_conv_update(start, x, w)) and torch.equal(pool[at.long()], start)
    assert not pool[:3].any() and not pool[slots - 2].any()


def test_steps_far_apart():
    """dt a view whose tokens lie 2^25 values apart, where many rows are made in a
    walk: next to the same values side by side, to the bar of a scan in fp32."""
    b, L, H, P, N, apart = 16, 64, 16, 16, 16, 2 ** 25
    dt = randn(1, L, H, seed=1, dtype=torch.float32)
    wide = torch.empty((L - 1) * apart + H, device=DEV).as_strided((1, L, H), (0, apart, 1))
    wide.copy_(dt)
    f32 = dict(dtype=torch.float32)
    args = dict(x=randn(b, L, H, P, seed=2, **f32), A=-torch.rand(H, device=DEV) - 0.5, B=randn(b, L, 1, N, seed=3, **f32),
                C=randn(b, L, 1, N, seed=4, **f32))
    dout = randn(b, L, H, P, seed=5, **f32)
    a, w = (ssm.ssd_scan_bwd(dout, dt=v.expand(b, -1, -1), **args) for v in (dt, wide))
    for k in a:
        assert (a[k].double() - w[k].double()).norm() <= 1e-4 * a[k].double().norm(), k
