"""With bf16 IO, what the Mamba-2 SSM returns in fp32 is as good as fp32 products
make it: the gradients of A, of the step bias, of D and of the first state, and the
last state.  Their terms are products of bf16 inputs, which are exact, and of states
and a gated dout, which enter with 24 bits; a term is off by a few half steps of
2^-24, and the sums' errors mostly average out: 16 half steps of the norm are
asked.  Operands of 16 bits (2^-17) would leave two to five times that."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU machines only to be skipped
    pytest.skip("no GPU", allow_module_level=True)

import mamba2_ref as ref  # noqa: E402
import selective_state_space_74_amd as ssm  # noqa: E402
from test_gpu_ssd_grad import DEV, call, expected, f64, make  # noqa: E402


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("shape", [(2, 512, 8, 64, 1, 64), (1, 500, 4, 64, 1, 128), (4, 256, 32, 64, 1, 64), (1, 300, 6, 130, 2, 33)],
                         ids=lambda s: "x".join(map(str, s)))
def test_fp32_results_of_bf16_inputs(shape, gate):
    b, L, H, P, G, N = shape
    t = make((b, L), H, P, G, N, "bf16", seed=sum(shape), gate=gate)
    val, _ = expected(t, "bf16")
    g = call(t, ssm.ssd_scan_bwd, t["dout"], dlast=t["dlast"])
    if b == 1:
        cu = torch.tensor([0, L], dtype=torch.int32, device=DEV)
        one = {k: v[0] if k in ("x", "dt", "B", "C", "z") and v is not None else v for k, v in t.items()}
        _, g["last"] = call(one, ssm.ssd_scan_fwd, cu=cu, return_last_state=True)
    off = {k: np.linalg.norm(f64(g[k]) - val[k]) / np.linalg.norm(val[k]) for k in ("dA", "ddt_bias", "dD", "dh0", "last") if k in g}
    print(f"[{shape} gate {gate}]", {k: f"{v:.1e}" for k, v in off.items()}, flush=True)
    assert max(off.values()) <= 16 * ref.U
