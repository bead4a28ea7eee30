"""Drawn cases of the measured work: what their inputs index is there."""
import importlib.util
import os
import random

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_rotations_stay_inside_their_tables():
    spec = importlib.util.spec_from_file_location("measured_work",
                                                  os.path.join(ROOT, "perf", "operators.py"))
    ops = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ops)
    seen = 0
    for seed in range(1500):
        case = ops.draw(random.Random(seed))
        if case["op"] == "rotate":
            seen += 1
            # positions start .. start + T - 1 with start below max(1, pos_max - T)
            assert case["T"] <= case["pos_max"]
    assert seen > 100
