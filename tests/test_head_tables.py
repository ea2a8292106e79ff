"""The table of the exact weights' exponential, against 60 digits."""
import os
import re
from decimal import Decimal, localcontext

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_powers_of_two_as_float_pairs():
    src = open(os.path.join(ROOT, "canvas_sampler_gb300", "csrc", "ds_head_sample.cuh")).read()
    body = re.search(r"kExp2Table\[33\] = \{(.*?)\};", src, re.S).group(1)
    pairs = re.findall(r"\{(-?0x[0-9a-fp.+-]+?)f, (-?0x[0-9a-fp.+-]+?)f\}", body)
    assert len(pairs) == 33
    with localcontext() as c:
        c.prec = 60
        for j, (hi, lo) in zip(range(-16, 17), pairs):
            want = Decimal(2) ** (Decimal(j) / 32)
            hi, lo = float.fromhex(hi), float.fromhex(lo)
            assert hi == float(np.float32(float(want))), j
            rest = want - Decimal(hi)
            assert lo == float(np.float32(float(rest))), j
            # the pair is good to 2^-49 (half a step of a rest below 2^-24)
            assert abs(rest - Decimal(lo)) <= Decimal(2) ** -49 * want
