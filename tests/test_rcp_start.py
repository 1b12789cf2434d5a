"""CPU: the start of the capped prefill's reciprocal (csrc/sp_prefill.cuh), its
constant read from the source: 5.06 % off at most, and past three Newton steps
in fp32 what is left is the roundings of the last one.  Proof of its bound: the
exact steps leave 0.0506^8 = 4.3e-11; 2 - d r and its product with r are rounded
to 2^-24 of themselves each, which moves r by (1 + 2^-24)^2 at most."""
import os
import re

import numpy as np

SRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "head_aware_paged_gb300", "csrc", "sp_prefill.cuh")


def test_start_and_steps():
    with open(SRC) as f:
        m = re.search(r"kRcpStart = 0x7F000000u - \(uint32_t\)\(([0-9.]+) \* 8388608.0 \+ 0.5\);", f.read())
    s = float(m.group(1))
    assert abs(s - (5 - np.sqrt(24.0))) < 1e-12
    start = np.uint32(0x7F000000 - int(s * 8388608.0 + 0.5))
    d = (1 + np.arange(0, 1 << 23, 7) / float(1 << 23)).astype(np.float32)
    for e in (0, 1, 13, 30):                    # d = 1 + 2^x, x <= 30
        de = d * np.float32(2.0 ** e)
        r = (start - de.view(np.uint32)).view(np.float32)
        assert np.abs(1 - de.astype(np.float64) * r).max() <= 0.0506
        for _ in range(3):
            # one rounding of 2 - d r, as the fused operation has
            r = r * (2 - de.astype(np.float64) * r).astype(np.float32)
        assert np.abs(1 - de.astype(np.float64) * r).max() <= (1 + 2.0 ** -24) ** 2 - 1 + 0.0506 ** 8
