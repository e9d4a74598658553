"""The plan that attention's kernels make for themselves, on the CPU: what two
kernels of a call have to agree on is computed in one of them."""
import os
import re

import numpy as np

SOURCE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "lossless_bit_weight_w12_gb300", "csrc",
                      "attend_device.cuh")

F = np.float32


def _fma(a, b, c):
    return F(np.float64(a) * np.float64(b) + np.float64(c))


def _prefix_sms(fused, heads, pu, w, tiles, requests, sms=152):
    """att_prefix_sms() for units of 256 rows under the prefix and requests in
    the register kernel, both with more work than the GPU has SMs; fused: with
    products contracted into the sums that follow them."""
    tp = F(heads) * F(pu) * F(w) * F(33.0)
    each = F(requests) * F(40.0)
    tq = F(heads) * (_fma(F(tiles), F(7.0), each) if fused else F(tiles) * F(7.0) + each)
    x = F(sms) * tp / (tp + tq)
    for _ in range(4):
        top = _fma(F(250.0), x, tp) if fused else tp + F(250.0) * x
        x = F(sms) * top / (top + tq)
    return max(1, min(sms - 1, int(x + F(0.5))))


def test_the_shares_of_the_sms_depend_on_the_compilation():
    """What the next test is for: contracted and not, the same arithmetic cuts
    the SMs in different places (86 requests under two key heads and a prefix
    of 429 tiles, 4988 tiles of their own)."""
    assert _prefix_sms(False, 2, 1, 429, 4988, 86) != _prefix_sms(True, 2, 1, 429, 4988, 86)


def test_the_prefixs_kernel_tells_its_own_number_of_workers():
    """The join takes the slots of the prefix's results from the number of
    workers that wrote them.  That number comes from float arithmetic, so the
    kernel that used it says it; the requests' kernel, another compilation,
    does not."""
    s = re.sub(r"//[^\n]*", "", open(SOURCE).read())
    plan = s[s.index("AttPlan att_plan("):s.index("AttPlan p;")]
    writes = re.findall(r"if \(([^)]*)\) a\.plan\[1\] = gp;", plan)
    assert len(writes) == 1 and plan.count("a.plan[1]") == 1
    names = dict(re.findall(r"const bool (\w+) = ([^;]*);", plan))
    cond = writes[0]
    for _ in range(3):
        cond = re.sub(r"\w+", lambda m: "(" + names[m[0]] + ")" if m[0] in names else m[0], cond)
    assert "a.join" in cond and "blockIdx.x == 0" in cond and "a.self == kLinePrefix" in cond
