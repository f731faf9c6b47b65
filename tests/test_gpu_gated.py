"""The gated linear recurrence on the GPU against its 64-bit form, within the
error bound that form computes (recurrent_ref) plus the rounding of the IO
type."""
import numpy as np
import pytest

import recurrent_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU machines only to be skipped
    pytest.skip("no GPU", allow_module_level=True)

import selective_state_space_74_amd as ssm  # noqa: E402

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def make(lead, D, io="f32", n=None, seed=0, h0=True, gates=1.0, strided=False):
    """Inputs on the device; with `strided` the gates are slices of one wider
    tensor and x of another, with rows longer than they need to be."""
    g = torch.Generator().manual_seed(seed)
    dt = TYPES[io]
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    if strided:
        wide = r(*lead, 2 * D + 3).to(dt).to(DEV)
        ga, gx = wide[..., :D], wide[..., D + 3:]
        x = r(*lead, D + 1).to(dt).to(DEV)[..., 1:]
    else:
        x, ga, gx = (t.to(dt).to(DEV) for t in (r(*lead, D), gates * r(*lead, D), gates * r(*lead, D)))
    n = lead[0] if n is None else n
    u = 0.9 + 0.099 * torch.rand(D, generator=g)
    lam = torch.log(1 / u - 1).to(DEV)
    return dict(x=x, gate_a=ga, gate_x=gx, lam=lam, h0=r(n, D).to(DEV) if h0 else None,
                dout=r(*lead, D).to(dt).to(DEV), dlast=r(n, D).to(DEV))


def forward(t, cu=None, **kw):
    ck = torch.empty(ssm.gated_checkpoint_shape(t["x"].shape), device=DEV)
    out, last = ssm.gated_scan_fwd(t["x"], t["gate_a"], t["gate_x"], t["lam"], h0=t["h0"], cu_seqlens=cu,
                                   return_last_state=True, checkpoints=ck, **kw)
    return out, last, ck


def backward(t, ck, cu=None, dlast=True, **kw):
    return ssm.gated_scan_bwd(t["dout"], t["x"], t["gate_a"], t["gate_x"], t["lam"], ck, h0=t["h0"],
                              cu_seqlens=cu, dlast=t["dlast"] if dlast else None, **kw)


def expected(t, cu=None, dlast=True, c=8.0):
    with np.errstate(all="ignore"):
        return ref.gated_scan(f64(t["x"]), f64(t["gate_a"]), f64(t["gate_x"]), f64(t["lam"]), c=c,
                              h0=None if t["h0"] is None else f64(t["h0"]),
                              cu=None if cu is None else cu.tolist(), dout=f64(t["dout"]),
                              dlast=f64(t["dlast"]) if dlast else None)


def check(got, val, bnd, io, what):
    for k, g in got.items():
        half = ref.HALF_STEP[io] if k in ("out", "dx", "dgate_a", "dgate_x") else ref.HALF_STEP["f32"]
        y = f64(g)
        # 2^-126: where fp32 stops being relative
        room = (bnd[k] + half * (np.abs(val[k]) + bnd[k])) + 2.0 ** -126
        assert np.all(np.isfinite(y)), (what, k)
        worst = np.max(np.abs(y - val[k]) / room, initial=0)
        print(f"[{what}] {k}: {worst:.3f} of the bound", flush=True)
        assert worst <= 1, (what, k)


def run_and_check(t, io, what, cu=None, dlast=True):
    val, bnd = expected(t, cu, dlast)
    out, last, ck = forward(t, cu)
    check(dict(out=out, last=last), val, bnd, io, what)
    g = backward(t, ck, cu, dlast)
    assert ("dh0" in g) == (t["h0"] is not None)
    check(g, val, bnd, io, what)
    return out, last, ck, g


SHAPES = [(1, 1, 1), (2, 3, 5), (1, 15, 64), (1, 16, 66), (3, 17, 65), (2, 64, 128), (1, 127, 130), (2, 128, 256),
          (1, 129, 8), (2, 300, 33), (5, 500, 100), (1, 2049, 130), (1, 5000, 34), (40, 2, 258), (300, 1, 7),
          # up to 32 channels: several blocks of tokens a wavefront
          (1, 5000, 13), (2, 3000, 8), (1, 2100, 32), (3, 700, 20), (1, 20000, 3), (2, 1024, 16), (1, 1025, 1),
          # four groups of 128 channels and more: two bf16 channels a lane backward
          (4, 200, 100), (1, 1030, 514), (5, 129, 2)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_batched(shape, io):
    t = make(shape[:2], shape[2], io, seed=sum(shape), h0=shape[1] % 2 == 1)
    run_and_check(t, io, f"{shape} {io}", dlast=shape[0] % 2 == 1)


PACKED = {
    "one": [0, 40],
    "ends_on_blocks": [0, 16, 32, 64, 128, 130],
    "empty_and_single": [0, 0, 1, 2, 2, 2, 19, 20, 150, 150],
    "outside": [5, 9, 140, 260],
    "all_empty": [7, 7, 7],
    "none": [0],
    "many": list(range(0, 400, 3)),
    "long": [0, 3, 1500, 1501, 3333],
    "longer": [1, 1, 2, 2050, 2051, 4100, 9000, 9000],
}


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("name", PACKED)
@pytest.mark.parametrize("D,h0", [(64, True), (131, False), (256, True), (7, True), (13, False), (32, True), (400, True)])
def test_packed(name, D, h0, io):
    cu = torch.tensor(PACKED[name], dtype=torch.int32, device=DEV)
    T = PACKED[name][-1] + (13 if name in ("outside", "all_empty", "none") else 0)
    t = make((T,), D, io, n=cu.numel() - 1, seed=T + D, h0=h0)
    out, last, ck, g = run_and_check(t, io, f"packed {name} {D} {io}", cu)
    # rows in no sequence: zeros in what is made here, untouched in what is given
    given = torch.full_like(t["x"], 7.0)
    ssm.gated_scan_fwd(t["x"], t["gate_a"], t["gate_x"], t["lam"], h0=t["h0"], cu_seqlens=cu, out=given)
    lo, hi = PACKED[name][0], PACKED[name][-1]
    assert torch.equal(given[lo:hi], out[lo:hi])
    for part in (slice(0, lo), slice(hi, T)):
        assert not out[part].any() and torch.all(given[part] == 7.0) and not g["dx"][part].any()


def test_packed_is_the_batched_form_of_each_sequence():
    """A sequence's result does not depend on where it lies: the batched call
    and the packed one agree within both their bounds."""
    t = make((4, 77), 96, "f32", seed=5)
    out, last, ck = forward(t)
    cu = torch.arange(0, 4 * 77 + 1, 77, dtype=torch.int32, device=DEV)
    flat = {k: (v.reshape(-1, v.shape[-1]) if k in ("x", "gate_a", "gate_x", "dout") else v) for k, v in t.items()}
    run_and_check(flat, "f32", "packed rows", cu)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("lead,D", [((2, 150), 64), ((2, 33), 31), ((1, 400), 256)])
def test_slices_of_wider_tensors(lead, D, io):
    t = make(lead, D, io, seed=11, strided=True)
    assert not t["x"].is_contiguous() and not t["gate_a"].is_contiguous()
    run_and_check(t, io, f"slices {lead} {D} {io}")
    # sequence-major storage, and an input broadcast over the batch
    s = {k: (v.transpose(0, 1).contiguous().transpose(0, 1) if k in ("x", "gate_a", "gate_x", "dout") else v)
         for k, v in t.items()}
    s["gate_x"] = s["gate_x"][:1].expand(lead[0], -1, -1)
    run_and_check(s, io, f"sequence-major {lead} {D} {io}")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("L,D", [(1, 12), (300, 12), (150, 66), (133, 512)])
def test_inputs_that_are_one_row_for_all_tokens(L, D, io):
    t = make((2, L), D, io, seed=27)
    for k in ("gate_a", "x", "dout"):
        t[k] = t[k][:, :1].expand(-1, L, -1)
    run_and_check(t, io, f"one row {L} {D} {io}")
    p = {k: (v[1] if v.dim() == 3 else v) for k, v in t.items()}
    cu = torch.tensor([0, L // 2, L], dtype=torch.int32, device=DEV)
    run_and_check(p, io, f"one row, packed {L} {D} {io}", cu)


def test_out_as_a_slice_next_to_the_input():
    t = make((2, 70), 48, "f32", seed=12)
    both = torch.zeros(2, 70, 96, device=DEV)
    both[..., :48] = t["x"]
    ref_out, _, _ = forward(t)
    ssm.gated_scan_fwd(both[..., :48], t["gate_a"], t["gate_x"], t["lam"], h0=t["h0"], out=both[..., 48:])
    assert torch.equal(both[..., 48:], ref_out) and torch.equal(both[..., :48], t["x"])


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("L", [1, 70])
def test_out_next_to_the_input_in_a_sequence_major_tensor(L, io):
    t = make((3, L), 48, io, seed=41)
    both = torch.zeros(L, 3, 96, device=DEV, dtype=TYPES[io]).transpose(0, 1)
    both[..., :48] = t["x"]
    ref_out, _, _ = forward(t)
    ssm.gated_scan_fwd(both[..., :48], t["gate_a"], t["gate_x"], t["lam"], h0=t["h0"], out=both[..., 48:])
    assert torch.equal(both[..., 48:], ref_out) and torch.equal(both[..., :48], t["x"])


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_extreme_gates(io):
    """Gates at both ends: a of 0 and 1, an input scale of 0 with its root's
    derivative taken as 0, huge and tiny decay rates."""
    t = make((2, 200), 64, io, seed=13)
    big = torch.tensor([float("-inf"), -1e4, -60.0, -20.0, 0.0, 20.0, 60.0, 1e4, float("inf")])
    idx = torch.arange(200) % 9
    t["gate_a"] = big[idx][None, :, None].expand(2, 200, 64).to(TYPES[io]).to(DEV).contiguous()
    t["gate_x"] = big[(idx + 4) % 9][None, :, None].expand(2, 200, 64).to(TYPES[io]).to(DEV).contiguous()
    t["lam"] = torch.linspace(-30, 30, 64, device=DEV)
    val, bnd = expected(t)
    out, last, ck = forward(t)
    g = backward(t, ck)
    check(dict(out=out, last=last, dx=g["dx"], dgate_x=g["dgate_x"], dh0=g["dh0"]), val, bnd, io, f"extreme {io}")
    for k in ("dgate_a", "dlam"):
        assert torch.isfinite(g[k]).all(), k


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("D", [20, 64])
def test_extreme_gates_all_gradients(D, io):
    """dgate_a and dlam too, against the 64-bit form.  Added to its bounds, with
    |e| <= E, the sum of the upstreams' magnitudes: where 1 - a^2 is below 2^-126
    (here: 2^-125) fp32 has 2^63 for 1 / beta, so dv sigma(gate_a) is off by
    E |x| (1 / beta + 2^63) sigma(gate_a); and a decay below 2^-126 is 0, which is
    E 2^-126 |h| there."""
    t = make((2, 200), D, io, seed=43)
    big = torch.tensor([float("-inf"), -1e4, -60.0, -20.0, 0.0, 20.0, 60.0, 1e4, float("inf")])
    idx = torch.arange(200) % 9
    t["gate_a"] = big[idx][None, :, None].expand(2, 200, D).to(TYPES[io]).to(DEV).contiguous()
    t["gate_x"] = big[(idx + 4) % 9][None, :, None].expand(2, 200, D).to(TYPES[io]).to(DEV).contiguous()
    t["lam"] = torch.linspace(-30, 30, D, device=DEV)
    val, bnd = expected(t)
    with np.errstate(all="ignore"):
        sa = 1 / (1 + np.exp(-f64(t["gate_a"])))
        s = 8 * (np.maximum(f64(t["lam"]), 0) + np.log1p(np.exp(-np.abs(f64(t["lam"])))))
        q = -np.expm1(-2 * s * sa)
        inv = np.where(q > 0, 1 / np.sqrt(q), 0) + 2.0 ** 63
    E = np.abs(f64(t["dout"])).sum(1, keepdims=True) + np.abs(f64(t["dlast"]))[:, None]
    size = max(np.abs(val["out"]).max(), np.abs(f64(t["h0"])).max())
    off = E * (np.abs(f64(t["x"])) * np.where(q < 2.0 ** -125, inv, 0) + 2.0 ** -126 * size) * sa
    bnd["dgate_a"] = bnd["dgate_a"] + off * s
    bnd["dlam"] = bnd["dlam"] + 8 / (1 + np.exp(-f64(t["lam"]))) * off.sum((0, 1))
    out, last, ck = forward(t)
    check(backward(t, ck), val, bnd, io, f"extreme {D} {io}")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("D,L", [(3, 70000), (13, 36000), (31, 20000)])
def test_few_channels_over_several_groups_of_tiles(D, L, io):
    """The carry from group to group where a group is 32,768 tokens (up to 8
    channels), 16,384 (16) or 8192 (32); batched, and packed with sequences that
    end in other groups than they begin in.  The same bits every time."""
    t = make((1, L), D, io, seed=D)
    t["lam"] = t["lam"] - 6      # decays close to 1: a state reaches over groups
    first = run_and_check(t, io, f"groups {D} {io}")
    p = {k: (v[0] if v.dim() == 3 else v) for k, v in t.items()}
    cu = torch.tensor([0, 11, L // 2 + 5, L // 2 + 5, L - 3], dtype=torch.int32, device=DEV)
    p["h0"], p["dlast"] = torch.randn(4, D, device=DEV), torch.randn(4, D, device=DEV)
    packed = run_and_check(p, io, f"packed groups {D} {io}", cu)
    for i in range(3):
        again = forward(t)
        assert all(torch.equal(a, b) for a, b in zip(again, first))
        assert all(torch.equal(g, first[3][k]) for k, g in backward(t, again[2]).items())
        again = forward(p, cu)
        assert all(torch.equal(a, b) for a, b in zip(again[:2], packed))
        assert all(torch.equal(g, packed[3][k]) for k, g in backward(p, again[2], cu).items())


def test_nan_stays_in_its_channel_and_sequence():
    t = make((2, 300), 66, "f32", seed=14)
    clean, _, _ = forward(t)
    t["x"][0, 100, 10] = float("nan")
    out, last, ck = forward(t)
    assert torch.isnan(out[0, 100:, 10]).all() and torch.isnan(last[0, 10])
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[0, 100:, 10] = True
    assert torch.equal(out[~bad], clean[~bad])
    # packed: a sequence's first token takes nothing from the sequence before
    cu = torch.tensor([0, 150, 300], dtype=torch.int32, device=DEV)
    p, last = ssm.gated_scan_fwd(t["x"][0], t["gate_a"][0], t["gate_x"][0], t["lam"], cu_seqlens=cu,
                                 return_last_state=True)
    assert torch.isnan(p[100:150, 10]).all() and torch.isfinite(p[150:]).all() and torch.isfinite(last[1]).all()


@pytest.mark.parametrize("D", [12, 66])
def test_nan_of_one_sequence_spares_the_others_gradients(D):
    """In x (the states after it are NaN) and in dout (the adjoints before it),
    next to a border inside a block of tokens and far from one."""
    t = make((700,), D, "f32", n=3, seed=24)
    cu = torch.tensor([0, 300, 317, 700], dtype=torch.int32, device=DEV)
    t["x"][305, 5] = float("nan")
    t["dout"][310, 7] = float("inf")
    out, last, ck = forward(t, cu)
    g = backward(t, ck, cu)
    for k in ("dx", "dgate_a", "dgate_x"):
        assert torch.isfinite(g[k][:300]).all() and torch.isfinite(g[k][317:]).all(), k
        keep = torch.ones(D, dtype=torch.bool, device=DEV)
        keep[5] = keep[7] = False
        assert torch.isfinite(g[k][:, keep]).all(), k
    assert torch.isfinite(g["dh0"][[0, 2]]).all()
    assert torch.isfinite(out[:300]).all() and torch.isfinite(out[317:]).all() and torch.isfinite(last[[0, 2]]).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("D", [12, 66, 512])
def test_nan_outside_every_sequence_reaches_nothing(D, io):
    """Rows before, between and behind the sequences' bounds, an odd tail too."""
    cu = torch.tensor([37, 60, 60, 301], dtype=torch.int32, device=DEV)
    t = make((333,), D, io, n=3, seed=25)
    outside = torch.ones(333, dtype=torch.bool, device=DEV)
    outside[37:301] = False
    out, last, ck = forward(t, cu)
    g = backward(t, ck, cu)
    for k in ("x", "gate_a", "gate_x", "dout"):
        t[k][outside] = float("nan")
    out2, last2, ck2 = forward(t, cu)
    g2 = backward(t, ck2, cu)
    assert torch.equal(out, out2) and torch.equal(last, last2)
    for k in g:
        assert torch.equal(g[k], g2[k]), k
    for v in (out2, g2["dx"], g2["dgate_a"], g2["dgate_x"]):
        assert not v[outside].any()


@pytest.mark.parametrize("D", [12, 66])
def test_an_infinite_upstream_of_the_last_state_passes_the_rows_end(D):
    """One token: every gradient of the channel is e = inf times a factor that is
    not 0, and the places behind the row's end in its block add nothing."""
    t = make((2, 1), D, "f32", seed=26)
    t["dlast"][0, 5] = float("inf")
    _, _, ck = forward(t)
    g = backward(t, ck)
    for k in ("dx", "dgate_a", "dgate_x"):
        assert torch.isinf(g[k][0, 0, 5]), k
    assert torch.isinf(g["dh0"][0, 5]) and torch.isinf(g["dlam"][5])
    for k in ("dx", "dgate_a", "dgate_x", "dh0"):
        bad = torch.zeros_like(g[k], dtype=torch.bool)
        bad[0, ..., 5] = True
        assert torch.isfinite(g[k][~bad]).all(), k


def test_zero_sizes():
    for lead in ((0, 5), (3, 0)):
        t = make(lead, 8, "f32", n=lead[0], seed=15)
        out, last, ck = forward(t)
        assert out.shape == lead + (8,) and torch.equal(last, t["h0"])
        g = backward(t, ck)
        assert not g["dlam"].any()
        if lead[1] == 0:
            assert torch.equal(g["dh0"], t["dlast"])
    t = make((2, 3), 0, "f32", seed=16)
    assert forward(t)[0].shape == (2, 3, 0)


def test_packed_without_tokens():
    """Sequences that are all empty, and no token outside either."""
    cu = torch.zeros(4, dtype=torch.int32, device=DEV)
    t = make((0,), 8, "f32", n=3, seed=16)
    out, last, ck = forward(t, cu)
    g = backward(t, ck, cu)
    assert out.shape == (0, 8) and torch.equal(last, t["h0"])
    assert torch.equal(g["dh0"], t["dlast"]) and not g["dlam"].any() and g["dx"].shape == (0, 8)


def test_state_carried_in_place():
    t = make((3, 333), 70, "f32", seed=17)
    _, last, _ = forward(t)
    h = t["h0"].clone()
    ssm.gated_scan_fwd(t["x"], t["gate_a"], t["gate_x"], t["lam"], h0=h, last_state=h)
    assert torch.equal(h, last)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("D", [12, 66, 256])
@pytest.mark.parametrize("L", [1, 40, 100, 128, 333, 1100])
def test_state_in_place_gives_the_bits_of_two_tensors(L, D, io):
    """last_state that is h0: one tile of several wavefronts, chains that end inside
    their first group, narrow calls and packed rows; the outputs and checkpoints,
    which a state read too late would change, too."""
    t = make((24, L), D, io, seed=L + D)
    want = forward(t)
    h, ck = t["h0"].clone(), torch.empty_like(want[2])
    out, last = ssm.gated_scan_fwd(t["x"], t["gate_a"], t["gate_x"], t["lam"], h0=h, last_state=h,
                                   return_last_state=True, checkpoints=ck)
    assert last is h and all(torch.equal(a, b) for a, b in zip((out, h, ck), want))
    # the same rows packed, with an empty sequence between them
    p = {k: (v.reshape(-1, D) if v.dim() == 3 else v) for k, v in t.items()}
    bounds = [k * L for k in range(12)] + [k * L for k in range(11, 24)]
    cu = torch.tensor(bounds, dtype=torch.int32, device=DEV)
    want = forward(p, cu)
    h = t["h0"].clone()
    out, last = ssm.gated_scan_fwd(p["x"], p["gate_a"], p["gate_x"], p["lam"], h0=h, last_state=h, cu_seqlens=cu,
                                   return_last_state=True)
    assert torch.equal(out, want[0]) and torch.equal(h, want[1]) and torch.equal(h[11], t["h0"][11])


def test_split_sequence_carries_the_state():
    t = make((2, 1000), 130, "f32", seed=18)
    val, bnd = expected(t)
    outs, h = [], t["h0"]
    for a, b in ((0, 1), (1, 400), (400, 417), (417, 1000)):
        o, h = ssm.gated_scan_fwd(*(t[k][:, a:b] for k in ("x", "gate_a", "gate_x")), t["lam"], h0=h,
                                  return_last_state=True)
        outs.append(o)
    check(dict(out=torch.cat(outs, 1), last=h), val, bnd, "f32", "split")


def test_same_bits_every_time():
    t = make((2, 3000), 200, "bf16", seed=19)
    first = [*forward(t)]
    first += list(backward(t, first[2]).values())
    for _ in range(5):
        again = [*forward(t)]
        again += list(backward(t, again[2]).values())
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_offsets_past_32_bits():
    """Token rows 2^25 elements apart: the last one's byte offset is past 2^32."""
    D, L = 40, 70
    big = torch.empty(L * (1 << 25), dtype=torch.bfloat16, device=DEV)
    view = lambda at: big.as_strided((1, L, D), (L << 25, 1 << 25, 1), at)  # noqa: E731
    t = make((1, L), D, "bf16", seed=20)
    far = dict(t)
    for i, k in enumerate(("x", "gate_a", "gate_x", "dout")):
        far[k] = view(i * 64)
        far[k].copy_(t[k])
    near_out, near_last, ck = forward(t)
    out, last, ck2 = forward(far)
    assert torch.equal(out, near_out) and torch.equal(last, near_last)
    given = view(1024)
    ssm.gated_scan_fwd(far["x"], far["gate_a"], far["gate_x"], t["lam"], h0=t["h0"], out=given)
    assert torch.equal(given, near_out)
    a, b = backward(t, ck), backward(far, ck2)
    assert all(torch.equal(a[k], b[k]) for k in a)


@pytest.mark.parametrize("D", [3, 12, 30])
def test_few_channels_with_rows_far_apart(D):
    """Up to 32 channels, rows 2^25 elements apart: too far for several blocks of
    tokens behind one descriptor."""
    L = 200
    big = torch.empty(L << 25, dtype=torch.bfloat16, device=DEV)
    view = lambda at: big.as_strided((1, L, D), (L << 25, 1 << 25, 1), at)  # noqa: E731
    t = make((1, L), D, "bf16", seed=D)
    for i, k in enumerate(("x", "gate_a", "gate_x", "dout")):
        far = view(i * 64)
        far.copy_(t[k])
        t[k] = far
    out, _, _, _ = run_and_check(t, "bf16", f"far rows {D}")
    given = view(1024)
    ssm.gated_scan_fwd(t["x"], t["gate_a"], t["gate_x"], t["lam"], h0=t["h0"], out=given)
    assert torch.equal(given, out)


def test_another_stream_and_two_at_once():
    """The same call on two streams at once, each with its own workspace."""
    ts = [make((1, 6000), 300, "f32", seed=21 + i) for i in range(2)]
    want = []
    for t in ts:
        o, l, ck = forward(t)
        want.append((o, l, backward(t, ck)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ts]
    got = []
    for _ in range(4):
        for t, s in zip(ts, streams):
            o, l, ck = forward(t, stream=s)
            with torch.cuda.stream(s):
                got.append((o, l, backward(t, ck)))
    torch.cuda.synchronize()
    for i, (o, l, g) in enumerate(got):
        wo, wl, wg = want[i % 2]
        assert torch.equal(o, wo) and torch.equal(l, wl) and all(torch.equal(g[k], wg[k]) for k in g)


def test_a_stream_by_its_handle():
    t = make((2, 500), 70, "f32", seed=44)
    want = forward(t)
    g = backward(t, want[2])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = forward(t, stream=s.cuda_stream)
    s.synchronize()   # the checkpoints were allocated on the current stream
    got += (backward(t, got[2], stream=s.cuda_stream),)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and all(torch.equal(got[3][k], g[k]) for k in g)


def test_captured_and_replayed():
    t = make((1, 4000), 192, "bf16", seed=23)
    cu = torch.tensor([0, 5, 5, 2222, 4000], dtype=torch.int32, device=DEV)
    p = {k: (v[0] if v.dim() == 3 else v) for k, v in t.items()}
    p["h0"], p["dlast"] = torch.randn(4, 192, device=DEV), torch.randn(4, 192, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o, l, ck = forward(p, cu)
        backward(p, ck, cu)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, l, ck = forward(p, cu)
        g = backward(p, ck, cu)
    for i in range(4):
        p["x"].normal_()
        p["dout"].normal_()
        if i == 2:  # the bounds too are read at each replay
            cu.copy_(torch.tensor([0, 100, 1000, 1001, 3990], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        eo, el, eck = forward(p, cu)
        eg = backward(p, eck, cu)
        torch.cuda.synchronize()
        assert torch.equal(o, eo) and torch.equal(l, el) and all(torch.equal(g[k], eg[k]) for k in g)


@pytest.mark.parametrize("D,L", [(12, 90), (130, 100), (130, 900)])
def test_state_carried_in_place_through_two_captured_graphs(D, L):
    """A layer's chunk and token, the state carried in place by both, captured
    twice and replayed on two streams at once."""
    def layer(t, h):
        out = ssm.gated_scan_fwd(t["x"], t["gate_a"], t["gate_x"], t["lam"], h0=h, last_state=h)
        return out, ssm.gated_state_update(h, *(t[k][:, 0] for k in ("x", "gate_a", "gate_x")), t["lam"])

    ts = [make((3, L), D, "f32", seed=50 + i) for i in range(2)]
    hs, streams = [t["h0"].clone() for t in ts], [torch.cuda.Stream() for _ in ts]
    graphs, got = [], []
    for t, h, s in zip(ts, hs, streams):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            layer(t, h.clone())
        torch.cuda.current_stream().wait_stream(s)
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(layer(t, h))
    for h, t in zip(hs, ts):
        h.copy_(t["h0"])
    eager = [t["h0"].clone() for t in ts]
    for _ in range(4):
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for t, h, e, (out, y) in zip(ts, hs, eager, got):
            eout, ey = layer(t, e)
            assert torch.equal(out, eout) and torch.equal(y, ey) and torch.equal(h, e)


def test_workspace_kept_across_calls_of_different_sizes():
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device=DEV)
    for L in (3000, 40, 5000, 3000):
        t = make((1, L), 140, "f32", seed=L)
        o, l, ck = forward(t)
        o2, l2, ck2 = forward(t, workspace=ws)
        g, g2 = backward(t, ck), backward(t, ck2, workspace=ws)
        assert torch.equal(o, o2) and torch.equal(l, l2) and all(torch.equal(g[k], g2[k]) for k in g)


@pytest.mark.parametrize("D", [12, 140])
def test_workspace_aligned_to_8_bytes_and_no_more(D):
    t = make((2, 3000), D, "f32", seed=D)
    out, last, ck = forward(t)
    g = backward(t, ck)
    ws = torch.full((16 << 20,), 255, dtype=torch.uint8, device=DEV)[8:]
    assert ws.data_ptr() % 16 == 8
    out2, last2, ck2 = forward(t, workspace=ws)
    g2 = backward(t, ck2, workspace=ws)
    assert torch.equal(out, out2) and torch.equal(last, last2) and all(torch.equal(g[k], g2[k]) for k in g)


def test_autograd():
    t = make((2, 90), 40, "f32", seed=25)
    leaves = {k: t[k].clone().requires_grad_() for k in ("x", "gate_a", "gate_x", "lam", "h0")}
    out, last = ssm.gated_scan(**leaves, return_last_state=True)
    ((out * t["dout"]).sum() + (last * t["dlast"]).sum()).backward()
    val, bnd = expected(t)
    check(dict(out=out, last=last, dx=leaves["x"].grad, dgate_a=leaves["gate_a"].grad,
               dgate_x=leaves["gate_x"].grad, dlam=leaves["lam"].grad, dh0=leaves["h0"].grad), val, bnd, "f32", "autograd")
    # through the last state alone, with a gate shared by the batch rows
    one = t["gate_x"][:1].clone().requires_grad_()
    _, last = ssm.gated_scan(t["x"], t["gate_a"], one.expand(2, -1, -1), t["lam"], return_last_state=True)
    last.sum().backward()
    s = dict(t, gate_x=one.detach().expand(2, -1, -1), h0=None, dout=torch.zeros_like(t["x"]),
             dlast=torch.ones(2, 40, device=DEV))
    val, bnd = expected(s)
    k = "dgate_x"
    room = bnd[k].sum(0) + 2.0 ** -23 * np.abs(val[k]).sum(0) + 2.0 ** -126
    assert np.all(np.abs(f64(one.grad[0]) - val[k].sum(0)) <= room)


# -- the single-token step ------------------------------------------------------------------------------------------

@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("batch,D", [(1, 1), (1, 5120), (3, 65), (7, 130), (256, 96)])
def test_step_is_one_token_of_the_scan(batch, D, io):
    t = make((batch, 1), D, io, seed=batch + D)
    val, bnd = expected(t)
    for pool in (None, batch + 5):
        state = torch.full((pool or batch, D), 3.0, device=DEV)
        slots = None if pool is None else torch.randperm(pool)[:batch].to(torch.int32).to(DEV)
        at = slice(0, batch) if slots is None else slots.long()
        state[at] = t["h0"]
        kept = state.clone()
        out = ssm.gated_state_update(state, t["x"][:, 0], t["gate_a"][:, 0], t["gate_x"][:, 0], t["lam"], slots=slots)
        check(dict(out=out[:, None], last=state[at]), val, bnd, io, f"step {batch} {D} {io}")
        mask = torch.ones(state.shape[0], dtype=torch.bool, device=DEV)
        mask[at] = False
        assert torch.equal(state[mask], kept[mask])


def test_step_padding_rows_and_a_slot_named_twice():
    D, slots = 70, [2, -1, 0, 2, 9, 2]
    t = make((6, 1), D, "f32", seed=31)
    x, ga, gx = (t[k][:, 0] for k in ("x", "gate_a", "gate_x"))
    state = torch.randn(4, D, device=DEV)
    want, outs = state.clone(), torch.zeros(6, D, device=DEV)
    for b, s in enumerate(slots):
        if 0 <= s < 4:
            outs[b] = ssm.gated_state_update(want[s:s + 1], x[b:b + 1], ga[b:b + 1], gx[b:b + 1], t["lam"])[0]
    out = ssm.gated_state_update(state, x, ga, gx, t["lam"], slots=torch.tensor(slots, dtype=torch.int32, device=DEV))
    assert torch.equal(out, outs) and torch.equal(state, want)


def test_step_strided_rows_and_pool():
    t = make((5, 1), 40, "bf16", seed=32)
    wide = torch.randn(9, 64, device=DEV)
    state = wide[:, 8:48]
    kept = wide.clone()
    flat = [t[k][:, 0].repeat_interleave(2, 0)[::2] for k in ("x", "gate_a", "gate_x")]
    plain = state.contiguous()
    a = ssm.gated_state_update(state, *flat, t["lam"])
    b = ssm.gated_state_update(plain, *(f.contiguous() for f in flat), t["lam"])
    assert torch.equal(a, b) and torch.equal(state, plain)
    assert torch.equal(wide[:, :8], kept[:, :8]) and torch.equal(wide[:, 48:], kept[:, 48:])


def test_prompt_then_tokens_is_the_whole_scan():
    t = make((3, 60), 90, "f32", seed=33)
    val, bnd = expected(t)
    o, h = ssm.gated_scan_fwd(*(t[k][:, :50] for k in ("x", "gate_a", "gate_x")), t["lam"], h0=t["h0"],
                              return_last_state=True)
    outs = [o]
    for i in range(50, 60):
        outs.append(ssm.gated_state_update(h, *(t[k][:, i] for k in ("x", "gate_a", "gate_x")), t["lam"])[:, None])
    check(dict(out=torch.cat(outs, 1), last=h), val, bnd, "f32", "prompt and tokens")
