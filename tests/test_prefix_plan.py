"""wh_prefix_attention_plan: which kernels sizes lead to, on the host alone (no GPU needed).  The GPU tests' cases are
pinned here to the path that each is there for, so that a changed rule cannot leave a path untested unnoticed."""
import ctypes

import pytest

from prefix_paths import PATHS, plan_of
from whisper_audio_encoder_gb300 import build, wh


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    wh.lib()


@pytest.mark.parametrize("name", PATHS)
def test_cases_take_their_path(name):
    plan = plan_of(PATHS[name])
    assert {f: plan[f] for f in PATHS[name]["plan"]} == PATHS[name]["plan"], plan


def test_every_path_has_a_case():
    seen = {(p["prefix_rows"], min(p["prefix_cluster"], 2), p["merge"]) for p in map(plan_of, PATHS.values()) if not p["own_warps"]}
    for rows in (16, 32, 64, 128):
        assert {(rows, 1, 0), (rows, 2, 0), (rows, 0, 1)} <= seen


def test_launches():
    plan = lambda *a, **kw: wh.wh_prefix_attention_plan(*a, **kw)["launches"]  # noqa: E731
    both = wh.WH_PREFIX_WEIGHT + wh.WH_OWN_WEIGHT
    assert plan(5, 1, 6, n_prefix=1, max_prefix=1500) == 1
    assert plan(5, 1, 6, n_prefix=1, max_prefix=1500, needs=both) == 2          # own keys' weights of no own keys: nothing
    assert plan(64, 1, 20, n_prefix=1, max_prefix=223, max_own=224) == 2
    assert plan(80, 1, 20, max_own=448, needs=both) == 1                         # from the scores kept on chip
    assert plan(32, 1, 20, n_prefix=1, max_prefix=30000) == 2                    # joined by a kernel


def test_refusals():
    out = wh.wh_prefix_plan()
    call = lambda *a, to=out: wh.lib().wh_prefix_attention_plan(*a, None if to is None else ctypes.byref(to))  # noqa: E731
    assert call(4, 1, 6, 6, 2, 100, 0, 0) == wh.WH_OK
    assert call(4, 1, 6, 6, 2, 100, 0, 0, to=None) == wh.WH_EINVAL
    for args in ((0, 1, 6, 6, 2, 100, 0, 0), (4, 1, 6, 5, 2, 100, 0, 0), (4, 1, 6, 6, -1, 100, 0, 0), (4, 1, 6, 6, 3, 100, 0, 2),
                 (4, 1, 6, 6, 2, 100, 0, 8), (4, 1, 6, 6, 0, 0, 0, 0), (4, 0, 6, 6, 2, 100, 0, 0), (4, 1, 6, 6, 2, -1, 0, 0)):
        assert call(*args) == wh.WH_EINVAL, args


@pytest.mark.parametrize("max_own", range(1, 97))
def test_short_own_caches_take_one_launch(max_own):
    """Fewer warps than four take an item only where it is short, or where items fill the device: one range either way."""
    for batch, heads in ((1, 1), (2, 6), (5, 20), (80, 20)):
        plan = wh.wh_prefix_attention_plan(batch, 1, heads, max_own=max_own, needs=wh.WH_OWN_WEIGHT)
        assert (plan["own_ranges"], plan["own_cluster"], plan["merge"], plan["launches"]) == (1, 1, 0, 1), (batch, heads, plan)


def test_short_own_caches_fill_the_device_or_take_four_warps():
    for batch in range(1, 400, 7):
        for max_own in (1, 32, 33, 64, 96, 97, 200, 448, 3000):
            for prefix in (0, 100):
                plan = wh.wh_prefix_attention_plan(batch, 1, 6, n_prefix=1 if prefix else 0, max_prefix=prefix, max_own=max_own)
                assert plan["own_warps"] == 4 or plan["own_ranges"] == 1, plan
