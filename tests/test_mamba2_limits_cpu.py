"""Sizes at the edge of what the Mamba-2 layer's launches can run: what passes the
host-side checks fits a grid (less than 2^32 threads) and the kernels' index types,
what does not is refused.  No GPU is touched."""
import selective_state_space_74_amd as ssm
from test_mamba2_abi_cpu import OK, UNSUP, conv, conv_bwd, ssd_step


def test_step_heads_fill_a_grid():
    """Four wavefronts a workgroup of 256: 2^24 - 1 workgroups hold 2^26 - 4 heads of up to 64 channels."""
    most = (1 << 26) - 4
    for P in (1, 8):
        assert ssm.validate_ssd_update(ssd_step(H=most, P=P, G=1, N=1)) == OK
        assert ssm.validate_ssd_update(ssd_step(H=most + 1, P=P, G=1, N=1)) == UNSUP
    assert ssm.validate_ssd_update(ssd_step(H=1 << 24, P=100, G=1, N=1)) == OK
    assert ssm.validate_ssd_update(ssd_step(H=(1 << 31) - 1, P=1, G=1, N=1)) == UNSUP


def test_step_rows_stay_within_ints():
    """Rows are counted in 32 bits up to a wavefront's share, 128 at most, past the last one."""
    for N in (1, 2):
        assert ssm.validate_ssd_update(ssd_step(batch=1, H=1, P=1 << 29, G=1, N=N)) == OK
    assert ssm.validate_ssd_update(ssd_step(batch=1, H=1, P=1 << 30, G=1, N=1)) == OK
    assert ssm.validate_ssd_update(ssd_step(batch=1, H=1, P=(1 << 30) + 1, G=1, N=1)) == UNSUP
    assert ssm.validate_ssd_update(ssd_step(batch=1, H=1, P=(1 << 31) - 1, G=1, N=1)) == UNSUP


def test_convolution_workgroups_fill_a_grid():
    """2^24 - 1 workgroups of 256 threads: 16 runs of tokens by 64 channels each, and up to
    256 for sequences without tokens."""
    def both(status, **kw):
        for make, check, states in ((conv, ssm.validate_token_conv, ("state_in", "state_out")),
                                    (conv_bwd, ssm.validate_token_conv_bwd, ("state_in", "dstate_out", "dstate_in"))):
            a = make(**kw)
            for k in states:   # larger than the addresses made up are apart
                setattr(a, k, None)
            assert check(a) == status, (make.__name__, kw)
    most = (1 << 24) - 257
    both(OK, batch=16 * most, L=1, D=4)
    both(UNSUP, batch=16 * most + 1, L=1, D=4)
    both(UNSUP, batch=(1 << 28) - 1, L=1, D=1)
    both(OK, batch=240, L=1, D=1 << 26)
    both(UNSUP, batch=255, L=1, D=1 << 26)     # 16 x 2^20
    both(OK, batch=1, L=(1 << 31) - 65, D=4)
    both(UNSUP, batch=1, L=(1 << 31) - 65, D=129)
