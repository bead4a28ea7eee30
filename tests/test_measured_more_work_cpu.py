"""Drawn cases of the second measured work: they lie in the operators' limits, and what their inputs index is
there."""
import importlib.util
import os
import random

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OPS = ("append", "window", "tree", "plan", "accept")


@pytest.fixture(scope="module")
def ops():
    spec = importlib.util.spec_from_file_location("measured_more_work",
                                                  os.path.join(ROOT, "perf", "more_operators.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.fixture(scope="module")
def cases(ops):
    return ops.listed() + [ops.draw(random.Random(seed)) for seed in range(400)]


def test_every_operator_is_listed_and_drawn(ops, cases):
    assert {c["op"] for c in ops.listed()} == {c["op"] for c in cases if "name" not in c} == set(OPS)


def test_drawn_cases_cost_no_more_than_listed_ones(ops, cases):
    most = {k: max(ops.work(c)[k] for c in ops.listed()) for k in ("bytes", "flops")}
    for case in cases:
        work = ops.work(case)
        assert all(0 <= work[k] <= most[k] for k in most) and any(work.values()), case


def test_cases_lie_in_the_operators_limits(cases):
    for c in cases:
        if c["op"] != "plan":
            assert c["D"] in (64, 128, 256) and c["page"] in (16, 32, 64, 128, 256), c
            assert c["Hq"] % c["Hkv"] == 0 and c["Hq"] // c["Hkv"] <= 16 and c["Hkv"] <= 128, c
        if c["op"] == "append":
            assert c["rot"] % 16 == 0 and c["rot"] <= c["D"] and c["T"] <= 1 << 20, c
            continue
        assert 1 <= c["B"] <= 1024 and 0 <= c["q_min"] <= c["q_max"] and c["q_max"] >= 1, c
        if c["op"] in ("plan", "tree"):
            assert c["q_max"] <= 256, c
        if c["op"] == "tree" and c["window"]:
            assert c["q_max"] <= c["window"], c


def test_lengths_parents_and_paths_fit_together(ops, cases):
    for c in cases:
        if c["op"] == "append":
            continue
        new, ctx = ops._lengths(c)
        assert len(new) == len(ctx) == c["B"] and max(new) == c["q_max"], c
        assert all(n >= 0 for n in new) and all(x >= 0 for x in ctx), c
        if c["op"] in ("plan", "tree"):
            for n, tree in zip(new, ops._parents(c, 3)):
                assert len(tree) == n and all(-1 <= p < i for i, p in enumerate(tree)), c
        if c["op"] == "accept":
            for n, path in zip(new, ops._accepted(c)):
                assert path == sorted(set(path)) and all(0 <= x < n for x in path), c
