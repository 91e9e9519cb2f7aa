"""Every kernel waits for the launches before it, whoever calls it: only after
griddepcontrol.wait are their writes visible to a kernel that was allowed to
start early. Read from the sources, for a missing wait shows rarely."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dsa_sparse_attention_store_gb300", "csrc")


def _body(text, at):
    """The braces that open at or after `at`, and what is between them."""
    i = text.index("{", at)
    depth, j = 1, i + 1
    while depth:
        depth += {"{": 1, "}": -1}.get(text[j], 0)
        j += 1
    return text[i:j]


def test_every_early_kernel_waits_first():
    files = {p: re.sub(r"//[^\n]*", "", open(p).read()) for p in glob.glob(os.path.join(CSRC, "*.cu*"))}
    bodies = {}
    for path, text in files.items():
        for m in re.finditer(r"__global__", text):
            head = text[m.end():text.index("{", m.end())]
            name = re.findall(r"(\w+)\s*\(", re.sub(r"__launch_bounds__\s*\((?:[^()]|\([^()]*\))*\)", "", head))[0]
            bodies[name] = _body(text, m.end())
    early = {n for t in files.values() for n in re.findall(r"(\w+_kernel)\b", t)} & set(bodies)
    assert {"attn_kernel", "span_plan_kernel", "rows_join_kernel", "join_kernel", "batch_plan_kernel"} <= early
    waiting = [n for n in sorted(bodies) if "pdl_wait" in bodies[n] or "pdl_trigger" in bodies[n]]
    assert set(waiting) >= {"attn_kernel", "span_plan_kernel", "rows_join_kernel", "join_kernel", "batch_plan_kernel"}
    for name in waiting:
        calls = [line for line in bodies[name].split("\n") if "pdl_wait" in line or "pdl_trigger" in line]
        # at the top of the kernel's body, on no condition, and before its own successor may start
        assert calls[0] == "  pdl_wait();", (name, calls)
        assert all(x.strip() in ("pdl_wait();", "pdl_trigger();") for x in calls), (name, calls)
