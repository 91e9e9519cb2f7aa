"""The example of a speculative decoding step: rotary positions, both caches,
the indexer's selection and the attention over it, together."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "draft_step.py")


def _example():
    spec = importlib.util.spec_from_file_location("draft_step", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
def test_selection_of_everything_is_the_whole_attention(fmt):
    # 500 committed tokens, 512 selected: every committed key, in the order of
    # its score; both attentions see the same keys, so the results differ by
    # the roundings of two orders of summation
    import torch
    r = _example().run(batch=3, ctx_len=500, draft=7, k=512, fmt=fmt)
    assert r["status"] == 0
    assert torch.all((r["chosen"] >= 0).sum(1) == 500)
    # fp32 sums of about 500 weights in two orders (2^-24 an addition), scores
    # of up to some tens rounded in two forms
    assert float((r["lse"] - r["full_lse"]).abs().max()) < 1e-4
    # two roundings of weights to bf16 and of results to bf16
    tol = 4 * 2.0 ** -8 * float(r["full"].abs().max())
    assert float((r["out"].float() - r["full"].float()).abs().max()) <= tol


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
def test_selection_keeps_part_of_the_weight(fmt):
    import torch
    r = _example().run(batch=2, ctx_len=3000, draft=9, k=512, fmt=fmt)
    assert r["status"] == 0
    assert torch.all(r["chosen"] >= 0)
    kept = r["kept"]
    assert torch.all(kept > 0) and torch.all(kept < 1 + 1e-4) and float(kept.mean()) < 0.9


def test_tree_rows():
    depth, rows = _example().draft_tree(6)
    assert depth[0] == 0 and rows[0] == 1
    for i in range(1, 6):
        assert rows[i] >> i == 1 and depth[i] == bin(rows[i]).count("1") - 1
