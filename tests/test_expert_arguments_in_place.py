"""Calls of the expert operators in place, on the CPU: a buffer given twice with rows that lie otherwise is
refused, since a row would be written over others that are yet to be read."""
import pytest

from tests.test_expert_arguments import ACT, COMB, NORM, _code, nat

N = dict(NORM, residual=1 << 20, sum=2 << 20, y=3 << 20, d_y=4 << 20, d_sum=5 << 20, d_x=6 << 20)


@pytest.mark.parametrize("fn,make,base,over,code", [
    (nat.moer_rms_norm, nat.make_norm, N, dict(sum=64, ld_sum=128), 2),
    (nat.moer_rms_norm, nat.make_norm, N, dict(sum=1 << 20, ld_sum=72), 2),
    (nat.moer_rms_norm, nat.make_norm, N, dict(y=64, ld_y=128), 2),
    (nat.moer_rms_norm, nat.make_norm, N, dict(y=64, ld_x=128), 2),
    (nat.moer_rms_norm, nat.make_norm, N, dict(sum=64, y=64), 1),
    (nat.moer_rms_norm_grad, nat.make_norm, N, dict(d_x=4 << 20, ld_d_x=72), 2),
    (nat.moer_rms_norm_grad, nat.make_norm, N, dict(d_x=5 << 20, ld_d_sum=72), 2),
    (nat.moer_expert_act_grad, nat.make_expert_act, dict(ACT, d_y=1 << 20), dict(ld_d_h=136), 2),
    (nat.moer_expert_combine, nat.make_expert_combine, dict(COMB, z=1 << 20), dict(ld_out=72), 2)])
def test_other_rows_of_the_same_buffer(fn, make, base, over, code):
    args = () if make is nat.make_expert_act else (64, 1 << 20)
    assert _code(fn, make(**{**base, **over}), *args, 0) == code
