"""The form in which ssm_prefill runs a call: lanes for each channel, whether scanning and the rest go to
waves of their own (roles), segments, tokens of a segment."""
import ctypes as C

import gated_delta_rule_rgdr_amd as rg

CUS = 256  # of an MI355X


def prefill_form(B, T, channels, N, G, one_pass=False, cus=CUS, f32=False):
    form = (C.c_int32 * 4)()
    rc = rg.library().ssm_prefill_form(B, T, channels, N, G, int(f32), int(one_pass), cus, form)
    assert rc == 0, rg.status_string(rc)
    ways, roles, segs, seg_len = form
    return ways, bool(roles), segs, seg_len
