"""Clipping refuses outputs that overlap (no GPU: the calls return before any CUDA call)."""
import random

import pytest

from test_layer_ops_host import A, clip

WIDE = 1 << 22


def refused(grads, numels, outs, dtypes=None, out_dtypes=None):
    n = len(grads)
    return clip(grads=grads, numels=numels, dtypes=dtypes or (0,) * n, outs=outs, out_dtypes=out_dtypes or (0,) * n)


@pytest.mark.parametrize("grads,numels,outs", [
    ((A, A), (4, 4), (A, A)),                                       # a gradient listed twice, in place
    ((A, A + 1024), (257, 4), (A, A + 1024)),                       # the first ends inside the second
    ((A + 1024, A), (4, 257), (A + 1024, A)),
    ((A, A + 4096), (4, 4), (WIDE, WIDE + 8)),                      # outputs over one another
    ((A, A + 4096), (4, 4), (A + 4096, WIDE)),                      # an output over another's gradient
    ((A, A + 4096), (4, 4), (A + 8, WIDE)),                         # or over its own, shifted
    ((A, A + 4096, A + 8192), (2048, 4, 4), (A, WIDE, WIDE + 16)),  # or a gradient inside one
])
def test_clip_refuses_outputs_that_overlap(grads, numels, outs):
    assert refused(grads, numels, outs) == 1


def test_clip_refuses_one_overlap_among_many():
    at = [A + 4096 * i for i in range(400)]
    random.Random(1).shuffle(at)
    at[17] = at[301] + 2
    assert refused(at, (2048,) * 400, at, (1,) * 400, (1,) * 400) == 1
