"""How far apart the rows of the short convolution and the selective scan may be, on
addresses that are not dereferenced: a call that passes the check of its pitches is
refused for an output that overlaps an input.
"""
import pytest

from test_blocks_cpu import CBWD, CFWD, CONV, SBWD, SCAN, SFWD, _call, needs_lib

ROW, ALIAS = -15, -9
FAR = 1 << 24


@needs_lib
@pytest.mark.parametrize("case,status", [
    (dict(ur=FAR), ROW), (dict(dr=FAR), ROW), (dict(gr=FAR), ROW), (dict(br=FAR), ROW),
    (dict(cr=FAR), ROW), (dict(ur=1 << 23), ALIAS), (dict(T=1, ur=FAR), ALIAS),
    (dict(T=1, dr=FAR, gr=FAR, br=FAR + 1, cr=FAR + 3), ALIAS), (dict(T=1, ur=1 << 58), ROW),
    (dict(T=1, br=(1 << 57) + 1), ROW), (dict(T=1, ur=FAR + 4), ROW)])
def test_scan_pitches(case, status):
    assert _call("mlstm_scan_fwd", SFWD, SCAN, dict(y=SCAN["A"], **case)) == status
    if case.get("T") == 1 and status == ALIAS:  # the gradients of one token are a sequence's
        status = ROW
    assert _call("mlstm_scan_bwd", SBWD, SCAN, dict(du=SCAN["A"], **case)) == status


@needs_lib
@pytest.mark.parametrize("case,status", [
    (dict(x_row=FAR), ALIAS), (dict(T=1, x_row=1 << 26), ALIAS), (dict(x_row=1 << 54), ROW),
    (dict(x_row=FAR + 4), ROW)])
def test_conv_pitches(case, status):
    assert _call("mlstm_short_conv_fwd", CFWD, CONV, dict(y=CONV["weight"], **case)) == status
    assert _call("mlstm_short_conv_bwd", CBWD, CONV, dict(dx=CONV["weight"], **case)) == status
