"""What include/batch.h says of the accuracy of probabilities from scores, against the polynomial in
csrc/batch_verify.hip (host arithmetic with 64 bits of mantissa)."""
import math
import os
import re

import numpy as np

from selective_state_update_ssu_amd import build

INCLUDE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")


def test_probabilities_are_as_accurate_as_the_header_says():
    text = open(os.path.join(build.CSRC, "batch_verify.hip")).read()
    body = re.search(r"double exp2_of\(double t\).*?double c\[8\] = \{(.*?)\}", text, re.S).group(1)
    c = [np.longdouble(float(x)) for x in body.split(",")]
    assert len(c) == 8 and np.finfo(np.longdouble).nmant >= 63
    x = np.linspace(np.longdouble(-0.5), np.longdouble(0.5), 400001)
    e = c[7]
    for k in reversed(c[:7]):
        e = e * x + k
    worst = float(np.max(np.abs((1 + e * x) / np.exp2(x) - 1)))
    assert worst < 2.2e-12  # as written beside the polynomial
    # A probability is a weight over a sum of weights. The exponent's argument, at most 1,100 in size,
    # comes from three roundings; the polynomial's own are below 10 of them.
    each = worst + (3 * 1100 * math.log(2) + 10) * 2.0 ** -53
    stated = int(re.search(r"Probabilities from scores\s*\*?\s*\(accurate to 2\^-(\d+)\)",
                           open(os.path.join(INCLUDE, "batch.h")).read()).group(1))
    assert (1 + each) / (1 - each) - 1 < 2.0 ** -stated
