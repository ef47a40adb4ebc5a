"""Cases of the experts' int8 products with more experts than one wave's lanes hold: empty ones among them, single rows
and ragged ends, all of lanes 64 to 127 empty, the last expert not.  test_i8_rules_host.py asserts their kernels."""
from collections import namedtuple

import numpy as np

Many = namedtuple("Many", "kernel gate_up experts t topk n k")
MANY = [Many("I8_STREAM_16", True, 512, 300, 4, 70, 192), Many("I8_STREAM_16", False, 512, 300, 4, 140, 192),
        Many("I8_STREAM_16", True, 65, 40, 2, 65, 576), Many("I8_STREAM_16", False, 130, 60, 2, 33, 576),
        Many("I8_TILES_128", True, 130, 8400, 2, 150, 192), Many("I8_TILES_128", False, 65, 4200, 2, 300, 192),
        Many("I8_TILES_128x256", True, 512, 2100, 4, 150, 192), Many("I8_TILES_128x256", False, 512, 2100, 4, 300, 192),
        Many("I8_TILES_256", True, 65, 4200, 2, 550, 192), Many("I8_TILES_256", False, 130, 8400, 2, 700, 192)]


def counts_of(case):
    """Rows of every expert, a twentieth of the pairs dropped."""
    rng = np.random.default_rng(case.experts + case.n)
    share = rng.random(case.experts) ** 2 * (rng.random(case.experts) < 0.7)
    share[64: min(128, case.experts - 1)] = 0
    share[-1] = 1
    pairs = case.t * case.topk
    counts = np.floor(share / share.sum() * pairs * 0.95).astype(int)
    counts[0] += 1
    return counts.tolist()
