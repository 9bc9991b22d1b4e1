"""Runs one case of perf/operators.py for a profiler: three states of it (seeds 0, 1, 2) in
turn, six passes.  From the repository root: python profiles/cases.py "<case's name>"."""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from perf import operators  # noqa: E402

operators.own = True
case = next(c for c in operators.listed() if c["name"] == sys.argv[1])
states = [operators.prepare(case, seed) for seed in range(3)]
for i in range(6):
    operators.run(states[i % 3])
torch.cuda.synchronize()
print("ok")
