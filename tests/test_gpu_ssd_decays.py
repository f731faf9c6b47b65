"""The Mamba-2 SSM where steps of one chunk differ by orders of magnitude, as a
selective model's do where it drops its state: what comes after such a step, and
the gradients of every step, are as exact as without it.  The bounds are those of
mamba2_ref with every term's own exponent in them."""
import numpy as np
import pytest

import mamba2_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU machines only to be skipped
    pytest.skip("no GPU", allow_module_level=True)

import selective_state_space_74_amd as ssm  # noqa: E402
from test_gpu_ssd_grad import DEV, TYPES, call, check, f64, make  # noqa: E402


def steps(lead, H, where, big, io, seed):
    """Steps of 0.001 to 0.02, but `big` at the tokens that `where` names."""
    g = torch.Generator().manual_seed(seed)
    dt = 1e-3 * 20 ** torch.rand(*lead, H, generator=g)
    at = {"one": [3], "ends": [0, 63, 64, 127], "every 8th": list(range(5, lead[-1], 8)), "block ends": [15, 16, 47, 48, 80]}[where]
    dt[..., [t for t in at if t < lead[-1]], :] = big
    return dt.to(TYPES[io]).to(DEV)


def scan(lead, H, P, G, N, where, big, io, gate=False, n=None, seed=0):
    t = make(lead, H, P, G, N, io, n=n, seed=seed, gate=gate, h0=False)
    t.update(dt=steps(lead, H, where, big, io, seed), dt_bias=None,
             A=-torch.tensor([16.0, 4.0, 1.0, 0.25], device=DEV).repeat(H)[:H])
    return t


def expected(t, io, cu=None):
    return ref.ssd_scan(*(f64(t[k]) for k in ("x", "dt", "A", "B", "C", "D", "z")), softplus_on=False,
                        cu=None if cu is None else cu.tolist(), dout=f64(t["dout"]), dlast=f64(t["dlast"]), io=io, sharp=True)


PATTERNS = [("one", 1.0), ("one", 100.0), ("one", 1000.0), ("ends", 20.0), ("every 8th", 1.0), ("every 8th", 20.0), ("every 8th", 100.0),
            ("block ends", 100.0)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("where,big", PATTERNS, ids=lambda v: str(v))
def test_packed(where, big, io):
    cu = torch.tensor([0, 70, 71, 240], dtype=torch.int32, device=DEV)
    t = scan((240,), 4, 64, 2, 64, where, big, io, gate=io == "f32", n=3, seed=int(big))
    val, bnd = expected(t, io, cu)
    out, last = call(t, ssm.ssd_scan_fwd, softplus=False, cu=cu, return_last_state=True)
    check(dict(out=out, last=last), val, bnd, io, f"{where} {big} {io}")
    check(call(t, ssm.ssd_scan_bwd, t["dout"], softplus=False, cu=cu, dlast=t["dlast"]), val, bnd, io, f"{where} {big} {io}")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("where,big", PATTERNS, ids=lambda v: str(v))
@pytest.mark.parametrize("shape", [(1, 150, 4, 33, 1, 20), (1, 70, 4, 130, 1, 16), (16, 70, 16, 64, 1, 64)], ids=lambda s: "x".join(map(str, s)))
def test_gradients(shape, where, big, io):
    """Chunk by chunk, heads of more channels than a pass has, and a row's states in one walk."""
    b, L, H, P, G, N = shape
    t = scan((b, L), H, P, G, N, where, big, io, gate=P == 33, seed=int(big))
    val, bnd = expected(t, io)
    check(call(t, ssm.ssd_scan_bwd, t["dout"], softplus=False, dlast=t["dlast"]), val, bnd, io, f"{shape} {where} {big} {io}")


def test_many_states():
    t = scan((150,), 4, 64, 1, 128, "every 8th", 20.0, "bf16", gate=True, n=1, seed=5)
    cu = torch.tensor([0, 150], dtype=torch.int32, device=DEV)
    val, bnd = expected(t, "bf16", cu)
    check(call(t, ssm.ssd_scan_bwd, t["dout"], softplus=False, cu=cu, dlast=t["dlast"]), val, bnd, "bf16", "128 states")


@pytest.mark.parametrize("big", [20.0, 1000.0])
def test_after_a_large_step_as_before_it(big):
    """In fp32, tokens after a step that drops the state are off by no more than
    1e-5 of their size, and the sums over steps likewise: ten times less than the
    bar, with room for the sums' own roundings (some 300 of 2^-24, mostly
    averaging out)."""
    cu = torch.tensor([0, 128], dtype=torch.int32, device=DEV)
    t = scan((128,), 4, 64, 1, 64, "one", big, "f32", n=1, seed=9)
    val, _ = expected(t, "f32", cu)
    got = call(t, ssm.ssd_scan_bwd, t["dout"], softplus=False, cu=cu, dlast=t["dlast"])
    got["out"] = call(t, ssm.ssd_scan_fwd, softplus=False, cu=cu)
    off = {}
    for k in ("out", "dx", "dB", "dC", "ddt"):
        off[k] = np.linalg.norm(f64(got[k])[4:] - val[k][4:]) / np.linalg.norm(val[k][4:])
    off["dA"] = np.linalg.norm(f64(got["dA"]) - val["dA"]) / np.linalg.norm(val["dA"])
    print(f"[{big}] {off}", flush=True)
    assert max(off.values()) <= 1e-5, off


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("where,big", PATTERNS, ids=lambda v: str(v))
def test_batched(where, big, io):
    """The batched prefill, along a row."""
    t = scan((2, 150), 4, 64, 2, 64, where, big, io, gate=io == "f32", seed=int(big) + 1)
    val, bnd = expected(t, io)
    out, last = call(t, ssm.ssd_scan_fwd, softplus=False, return_last_state=True)
    got = dict(out=out)
    if io == "f32":   # in bf16 what enters the state is rounded to bf16, which the bounds do not know
        got["last"] = last
    check(got, val, bnd, io, f"batched {where} {big} {io}")
