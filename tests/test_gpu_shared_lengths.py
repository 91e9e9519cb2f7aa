"""Groups of which one sequence's queries are inconsistent: the others' rows are
written, as dsa_span_attn writes them."""
import numpy as np
import pytest

from tests.span_util import SpanCase
from tests.test_gpu_spans import FMTS, ctx  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("nds", [[1, 2, 1], [40, 3, 90]])
@pytest.mark.parametrize("groups", [None, [(3, 128)], [(1, 0), (2, 128)]])
def test_a_group_that_ends_past_the_queries(ctx, fmt, nds, groups):  # noqa: F811
    import torch
    c = SpanCase(36, [200, 300, 129], nds, 1, 4, 64, fmt, groups=groups, cap=20.0)
    ref = c.reference()
    d = c.device()
    d["cu"][3] = c.Tq + 5                       # the last sequence's: past the rows of q
    out, lse = c.run(ctx, d=d)
    assert ctx.device_status() == 4 and ctx.device_status() == 0
    good = np.arange(nds[0] + nds[1])
    c.check(out, lse, ref=ref, rows=good)
    rest = slice(len(good), None)
    assert (out[rest] == 77.0).all() and (lse[rest] == 77.0).all()
    torch.cuda.synchronize()
