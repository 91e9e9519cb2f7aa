"""The example of samples behind a prompt: page plans, the cache, span and
shared attention together, over several steps."""
import importlib.util
import os

import numpy as np
import pytest

from oracle import attention as A
from oracle import spans as S

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "shared_prompt.py")


def _example():
    spec = importlib.util.spec_from_file_location("shared_prompt", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("prompt", [130, 640])       # a page shared in part, and none
def test_samples_behind_a_prompt(fmt, prompt):
    samples, steps, heads, kv, D, cap = 3, 3, 8, 2, 64, 20.0
    r = _example().run(prompt, samples, steps, fmt, heads, kv, D, cap)
    assert r["status"] == 0
    keys, vals = A.values(r["cache"].cpu().numpy(), r["pages"], kv, D, {"bf16": 0, "fp8": 1, "fp4": 2}[fmt])
    table = r["table"].cpu().numpy()
    near = lambda got, lse, ref, n: _close(got, lse, ref, D, n, cap)  # noqa: E731
    first = np.arange(prompt) - np.arange(prompt) % 700
    ref = S.attend(r["prompt_q"].double().cpu().numpy(), kv, keys, vals, table, [prompt], [0, prompt], D ** -0.5, first=first, cap=cap)
    near(r["prompt_out"], r["prompt_lse"], ref, prompt)
    for i, s in enumerate(r["steps"]):
        lens = s["lens"].cpu().numpy()
        assert lens.tolist() == [prompt] + [prompt + i + 1] * samples
        ref = S.attend(s["q"].double().cpu().numpy(), kv, keys, vals, table[1:], lens[1:], np.arange(samples + 1), D ** -0.5, cap=cap)
        near(s["out"], s["lse"], ref, lens[-1])
        near(s["alone"], s["alone_lse"], ref, lens[-1])
    # what came back is the samples' own pages, and every page is in one place
    whole = prompt // 64
    each = -(-(prompt + steps) // 64) - whole
    assert r["after_end"] - r["before_end"] == samples * each
    used = table[0, :-(-prompt // 64)].tolist()
    assert sorted(used + r["pool"][:r["after_end"]].tolist()) == list(range(r["pages"]))


def _close(got, lse, ref, D, n, cap):
    to, tl = S.tolerance(*ref, D ** -0.5, D, float(n), cap)
    assert np.all(np.abs(got.double().cpu().numpy() - ref[0]) <= to)
    assert np.all(np.abs(lse.double().cpu().numpy() - ref[1]) <= tl)
