"""Gradients of batched rows on both sides of where a row's states are made in one
walk instead of chunk by chunk (192 workgroups: rows x heads x 64 channels x both
directions, heads of more than 16 channels)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU machines only to be skipped
    pytest.skip("no GPU", allow_module_level=True)

import selective_state_space_74_amd as ssm  # noqa: E402
from test_gpu_ssd_grad import call, check, expected, make, run_and_check  # noqa: E402

SHAPES = [(3, 130, 32, 64, 1, 64), (2, 130, 32, 64, 1, 64), (2, 100, 16, 136, 2, 16), (6, 66, 16, 24, 2, 64), (1, 65, 96, 32, 1, 32),
          (7, 70, 16, 16, 1, 32), (3, 64, 32, 64, 1, 24)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_sides_of_the_rule(shape, io):
    b, L, H, P, G, N = shape
    t = make((b, L), H, P, G, N, io, seed=sum(shape), gate=P != 64, h0=L % 2 == 0)
    g = run_and_check(t, io, f"{shape} {io}", dlast=b != 2)
    again = call(t, ssm.ssd_scan_bwd, t["dout"], dlast=t["dlast"] if b != 2 else None)
    assert all(torch.equal(g[k], again[k]) for k in g)


@pytest.mark.parametrize("rows", [2, 3])
def test_128_states(rows):
    t = make((rows, 129), 32, 64, 1, 128, "bf16", seed=rows, gate=rows == 3)
    val, bnd = expected(t, "bf16")
    check(call(t, ssm.ssd_scan_bwd, t["dout"], dlast=t["dlast"]), val, bnd, "bf16", f"{rows} rows, 128 states")
