"""The example of samples behind a prompt with documents shorter than the prompt,
and with steps that take each sample over several pages."""
import numpy as np
import pytest

from oracle import attention as A
from oracle import spans as S
from tests.test_gpu_shared_prompt import _close, _example

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("document", [1, 100, 130])
def test_documents_of_a_prompt(fmt, document):
    prompt, heads, kv, D, cap = 130, 8, 2, 64, 20.0
    r = _example().run(prompt, 2, 1, fmt, heads, kv, D, cap, document=document)
    assert r["status"] == 0
    keys, vals = A.values(r["cache"].cpu().numpy(), r["pages"], kv, D, {"bf16": 0, "fp8": 1, "fp4": 2}[fmt])
    first = np.arange(prompt) - np.arange(prompt) % document
    args = (r["prompt_q"].double().cpu().numpy(), kv, keys, vals, r["table"].cpu().numpy(), [prompt], [0, prompt], D ** -0.5)
    ref = S.attend(*args, first=first, cap=cap)
    _close(r["prompt_out"], r["prompt_lse"], ref, D, prompt, cap)
    if document < prompt:                       # the tolerance tells documents from one prompt
        to = S.tolerance(*ref, D ** -0.5, D, float(prompt), cap)[0]
        assert np.mean(np.abs(S.attend(*args, cap=cap)[0] - ref[0]) > to) > 0.1


@pytest.mark.parametrize("prompt", [128, 130])
def test_many_steps(prompt):
    samples, steps = 2, 200                     # three or four pages each
    r = _example().run(prompt, samples, steps, "bf16", 8, 2, 64, 20.0)
    assert r["status"] == 0
    whole = prompt // 64
    assert r["after_end"] - r["before_end"] == samples * (-(-(prompt + steps) // 64) - whole)
    used = r["table"].cpu().numpy()[0, :-(-prompt // 64)].tolist()
    assert sorted(used + r["pool"][:r["after_end"]].tolist()) == list(range(r["pages"]))
