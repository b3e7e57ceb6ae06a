"""Rows behind a sequence's length, and of skipped entries, in the segmented long-sequence form: each is written, into
a buffer that holds other values before the call, as +0.0. A failure names the rows, and whether a second copy of the
buffer to the host, and the device itself, see the same."""
import numpy as np
import pytest
import torch

import workloads
from gpu_util import check_decode, dev_to_bits, oracle_decode, upload

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rg():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import gated_delta_rule_rgdr_amd as m
    m.library()
    return m


def padding_report(out, lens):
    """Which rows past the lengths [B] are not zero bits, at most 8 of them; empty if none."""
    first, second = dev_to_bits(out), dev_to_bits(out.clone())
    on_device = (out.view(torch.int16) != 0).any(-1).cpu().numpy()
    lines = []
    for b, n in enumerate(lens):
        for h in range(out.shape[1]):
            for t in range(n, out.shape[2]):
                if first[b, h, t].any() or second[b, h, t].any() or on_device[b, h, t]:
                    at = np.flatnonzero(first[b, h, t])
                    lines.append(f"entry {b} head {h} row {t} of {n} valid: {len(at)} columns from {at[:1].tolist()}, "
                                 f"bits {[hex(x) for x in first[b, h, t][at][:8]]}; second copy "
                                 f"{np.count_nonzero(second[b, h, t])}; on the device {on_device[b, h, t]}")
    return "\n".join([f"{len(lines)} rows", *lines[:8]]) if lines else ""


def test_padding_report():
    """The report itself finds a row."""
    out = torch.zeros(2, 1, 4, 8, dtype=torch.bfloat16, device="cuda")
    assert not padding_report(out, [4, 1])
    out[1, 0, 2, 5], out[1, 0, 0, 1] = -0.0, 1.0
    text = padding_report(out, [4, 1])
    assert text.startswith("1 rows\nentry 1 head 0 row 2 of 1 valid: 1 columns from [5], bits ['0x8000']")


@pytest.mark.parametrize("Dk,Dv", [(128, 128), (64, 256)])
def test_rows_behind_the_lengths(rg, Dk, Dv):
    inp = workloads.make_case(6, 2, 4, 640, Dk, Dv, 8, seed=8200, indices="choice", lengths="uniform")
    inp.actual_seq_lengths[:] = [640, 500, 0, 640, 311, 640]
    inp.num_accepted_tokens[:] = [0, 500, 0, 640, 64, 200]
    inp.ssm_state_indices[5] = 8  # skipped
    lens = [640, 500, 0, 640, 311, 0]
    assert rg.rgdr_prefill_workspace_size(6, 4, 640, Dk, Dv) > 0
    ref = oracle_decode(inp)
    for value in (float("nan"), 3.0, 0.0):
        d = upload(inp)
        out = torch.full((6, 4, 640, Dv), value, dtype=torch.bfloat16, device="cuda")
        got, st = rg.rgdr_prefill_ws(d["query"], d["key"], d["value"], d["beta"], d["state"], d["actual_seq_lengths"],
                                     d["ssm_state_indices"], d["g"], d["gk"], d["num_accepted_tokens"], inp.scale, out=out)
        torch.cuda.synchronize()
        report = padding_report(got, lens)
        assert not report, f"buffer of {value} before the call: {report}"
        check_decode(inp, got, st, ref, f"buffer of {value}")


@pytest.mark.parametrize("fn", ["rgdr_prefill_ws", "rgdr_prefill_noalloc"])
def test_skipped_entries_with_counts(rg, fn):
    """Entries without a slot, whose lengths and accepted counts span many segments: no segment of theirs has a
    token, so that none writes into the rows that the first one clears."""
    inp = workloads.make_case(6, 2, 4, 640, 128, 128, 8, seed=8201, indices="choice", lengths="uniform")
    inp.actual_seq_lengths[:] = [640, 640, 512, 640, 1000, 640]
    inp.num_accepted_tokens[:] = [640, 640, 500, 64, 1000, 640]
    inp.ssm_state_indices[1:] = [8, -1, 100, 8, -5]
    d = upload(inp)
    out = torch.full((6, 4, 640, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    got, st = getattr(rg, fn)(d["query"], d["key"], d["value"], d["beta"], d["state"], d["actual_seq_lengths"],
                              d["ssm_state_indices"], d["g"], d["gk"], d["num_accepted_tokens"], inp.scale, out=out)
    torch.cuda.synchronize()
    report = padding_report(got, [640, 0, 0, 0, 0, 0])
    assert not report, report
    check_decode(inp, got, st, oracle_decode(inp), fn)
