"""The bounds-checked build checks something in every kernel file that reports to
it: a source scan, on the CPU (the checks themselves pass or fail on the GPU)."""

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "mixture_experts_layer_deepseekmoe_amd", "csrc")
FILES = {os.path.basename(p): open(p).read() for p in sorted(glob.glob(os.path.join(CSRC, "*.hip")))}
REPORTING = [n for n, s in FILES.items() if re.search(r"^MOE_DEBUG_FILE\(", s, re.M)]


def _checks(source):
    """The ids of the file's checks: the last argument of each MOE_CHECK call."""
    ids = []
    for m in re.finditer(r"MOE_CHECK\(", source):
        depth, i = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(source[i], 0)
            i += 1
        ids.append(int(source[m.end():i - 1].rsplit(",", 1)[1]))
    return ids


@pytest.mark.parametrize("name", REPORTING)
def test_reporting_files_check(name):
    ids = _checks(FILES[name])
    assert ids and len({i // 100 for i in ids}) == 1, (name, ids)   # one series to a file


@pytest.mark.parametrize("name,kernels", [
    ("block.hip", ["block_in_kernel", "block_out_kernel", "block_bwd_kernel", "block_colsum_kernel"]),
    ("loss.hip", ["loss_gather_kernel", "loss_logits_kernel", "loss_stream_kernel", "loss_finish_kernel",
                  "loss_dh_kernel", "loss_dh_out_kernel", "loss_dw_kernel"])])
def test_kernels_check(name, kernels):
    s = FILES[name]
    starts = [(m.start(), m.group(1)) for m in re.finditer(r"__global__[^;{]*?(\w+_kernel)\(\w+ a\)", s, re.S)]
    for k, (at, kernel) in enumerate(starts):
        end = starts[k + 1][0] if k + 1 < len(starts) else s.index("MOE_DEBUG_FILE")
        if kernel in kernels:
            assert _checks(s[at:end]), kernel
    assert set(kernels) <= {n for _, n in starts}
