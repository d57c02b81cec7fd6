"""Grouped choice of every number of experts in a process of its own, the
larger ones last: what a launch may have of shared memory is not to depend
on the calls before."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))

CHILD = """
import torch
import route_reference as ref
from test_gpu_route import check_route, gen, make_logits
for dtype in ("fp32", "bf16", "fp16"):
    for E, G in ((1488, 16), (1500, 20), (1504, 16), (1520, 16), (1536, 16), (1552, 16), (2048, 16)):
        l = make_logits(gen(E), 40, E, dtype)
        bias = torch.round(torch.randn(E, generator=gen(E + 1), device="cuda") * 30) * 0.001
        check_route(l, 8, "sigmoid", bias=bias, groups=G, topk_groups=8)
        check_route(l, 8, "softmax", groups=G, topk_groups=8)
print("all held")
"""


def test_grouped_choice_without_a_larger_call_before():
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([HERE, os.path.dirname(HERE)]))
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=HERE, env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "all held" in r.stdout, r.stdout[-2000:] + r.stderr[-3000:]
