"""The products' schedule on the CPU: the GPU tests' sizes take every plan that
calls in the operators' range take, and the scratch that is asked for holds the
parts of every plan, of fewer rows too."""
from __future__ import annotations

import random

import pytest

import _plan as P
import test_gpu_ffn
import test_gpu_ffn_plans


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    return P.compile_plan(str(tmp_path_factory.mktemp("plan")))


def gpu_sizes():
    """The product calls (rows, in, out, dtype) of the GPU tests that run all four of linear, glu and their gradients."""
    calls = [(*s, d) for s in test_gpu_ffn.LINEAR_SHAPES for d in ("bf16", "f32")]
    calls += [(*s, "bf16") for s in test_gpu_ffn.TILE_SHAPES_16 + test_gpu_ffn_plans.PLANS_16]
    return calls + [(*s, "f32") for s in test_gpu_ffn.TILE_SHAPES_32 + test_gpu_ffn_plans.PLANS_32]


def test_every_plan_of_the_range_is_tested(lib):
    reached, have = P.keys(lib, P.sample(60000)), P.keys(lib, gpu_sizes())
    missing = sorted((k for k in reached if k not in have), key=lambda k: -reached[k])
    assert not missing, f"{len(missing)} of {len(reached)} plans are in no GPU test: {missing[:8]}"
    # among them whole and split tiles in one launch, of every product
    assert {k[1] for k in have if k[4] == "mixed"} == set(P.products(1, 8, 8, "bf16"))


def test_split_tiles_of_the_second_weight(lib):
    """One launch of both weights' gradients whose split tiles lie in the second one's."""
    q = P.products(1229, 8264, 904, "bf16")["dw of glu"]
    bm, bn, whole, rest, splits = P.ask(lib, [q])[0][:5]
    tiles = -(-q[1] // bm) * -(-q[2] // bn)
    assert (bm, bn) == (256, 256) and splits > 1 and rest > 0 and whole >= tiles


def test_scratch_holds_every_plan_of_as_many_rows_or_fewer(lib):
    rng = random.Random(3)
    # beside the operators' range, widths whose tiles leave any remainder, at every row count up to two tiles
    calls = P.sample(8000, seed=5) + [(m, 2560, n, d) for m in range(1, 513) for n in (136, 2056, 10240) for d in ("bf16", "f32")]
    large, small = [], []
    for m, k, n, dtype in calls:
        r = rng.randint(1, m)
        for name, q in P.products(m, k, n, dtype).items():
            large.append(q)
            small.append(P.products(r, k, n, dtype)[name])
    for q, a, b in zip(large, P.ask(lib, large), P.ask(lib, small)):
        assert a[7] <= a[6] and b[7] <= b[6] <= a[6], (q, a, b)
