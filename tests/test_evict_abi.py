"""wh_cache_evict rejects bad arguments on the host before it touches a device (no GPU needed)."""
import ctypes

import pytest
import torch

from whisper_audio_encoder_gb300 import build, wh

FAKE, P = ctypes.c_void_p(1 << 30), 1 << 30          # never dereferenced
ROWS = 3 * 100 * 128                                  # elements of the caches below


@pytest.fixture(scope="module")
def L():
    build.build()
    return wh.lib()


def _keys(at=P, **kw):
    base = dict(k=at, v=at + 2 * ROWS, row_stride=128, set_stride=12800, n_keys=None, weight=at + 4 * ROWS, n_set=3,
                max_keys=100)
    base.update(kw)
    return wh.wh_keys(*[base[f] for f, _ in wh.wh_keys._fields_])


def _call(L, cache=None, n_kv=2, budget=40, recent=8, out=None, n_out=FAKE, kept=None, ws=FAKE, ws_bytes=1 << 40):
    return L.wh_cache_evict(None if cache is None else ctypes.byref(cache), n_kv, budget, recent,
                            None if out is None else ctypes.byref(out), n_out, kept, ws, ws_bytes, None)


def test_rejects_bad_arguments(L):
    bad = [dict(budget=0), dict(budget=-1), dict(recent=-1), dict(recent=41), dict(n_kv=0), dict(n_kv=3), dict(n_out=None),
           dict(n_out=ctypes.c_void_p(P + 1)), dict(kept=ctypes.c_void_p(P + 2)), dict(ws=ctypes.c_void_p(P + 16))]
    for kw in bad:
        assert _call(L, _keys(), **kw) == wh.WH_EINVAL, kw
    assert _call(L) == wh.WH_EINVAL
    for kw in (dict(k=None), dict(v=None), dict(weight=None), dict(k=P + 8), dict(n_keys=P + 1), dict(n_set=0),
               dict(n_set=65536), dict(max_keys=0), dict(row_stride=120), dict(row_stride=132), dict(set_stride=-8),
               dict(set_stride=12801)):
        assert _call(L, _keys(**kw)) == wh.WH_EINVAL, kw


def test_rejects_what_shares_memory(L):
    assert _call(L, _keys(set_stride=0)) == wh.WH_EINVAL              # sets on top of each other
    assert _call(L, _keys(set_stride=12800 - 128)) == wh.WH_EINVAL
    assert _call(L, _keys(v=P)) == wh.WH_EINVAL                       # keys and values the same memory
    assert _call(L, _keys(v=P + 2 * 64)) == wh.WH_EINVAL              # or a head apart
    assert _call(L, _keys(n_keys=FAKE.value + 4)) == wh.WH_EINVAL     # new counts one off the old ones
    far = P + (1 << 24)
    assert _call(L, _keys(), out=_keys(at=far, n_set=2)) == wh.WH_EINVAL
    assert _call(L, _keys(), out=_keys(at=far, max_keys=39)) == wh.WH_EINVAL
    assert _call(L, _keys(), out=_keys(at=far, weight=None)) == wh.WH_EINVAL
    assert _call(L, _keys(), out=_keys()) == wh.WH_EINVAL             # the cache itself: out = NULL says that
    assert _call(L, _keys(), out=_keys(at=far, k=P + 256)) == wh.WH_EINVAL
    assert _call(L, _keys(), out=_keys(at=far, weight=P + 4 * ROWS)) == wh.WH_EINVAL


def test_workspace(L):
    size = L.wh_cache_evict_workspace
    assert size(3, 2, 100, 40) == 0                       # one kernel
    need = size(3, 300, 100, 40)
    assert need >= 3 * 4 + 3 * 300 * 40 * 4
    wide = dict(row_stride=19200, set_stride=1920000, v=P + (1 << 26), weight=P + (1 << 27))
    assert _call(L, _keys(**wide), n_kv=300, ws_bytes=need - 1) == wh.WH_ENOSPC
    assert _call(L, _keys(**wide), n_kv=300, ws=None) == wh.WH_ENOSPC
    for args in ((0, 300, 100, 40), (3, 0, 100, 40), (3, 300, 0, 40), (3, 300, 100, 0)):
        assert size(*args) == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")
def test_layouts_that_are_fine(L):
    far = P + (1 << 24)
    fine = [_keys(), _keys(v=P + 2 * 128, row_stride=256, set_stride=25600),          # [K | V] rows
            _keys(row_stride=384, set_stride=128, v=P + 2 * 3 * 384 * 100),           # sets side by side in a row
            _keys(n_set=1, set_stride=0)]
    for keys in fine:
        assert _call(L, keys) == wh.WH_ENODEV
    assert _call(L, _keys(), out=_keys(at=far, max_keys=40)) == wh.WH_ENODEV
    assert _call(L, _keys(max_keys=30), budget=40, out=_keys(at=far, max_keys=30)) == wh.WH_ENODEV


def test_interleaved_layouts_by_their_rows(L):
    """Sets beside each other in rows, keys and values in the same rows: only what overlaps is refused."""
    W = 2 * 128                                                # bytes of a row of a set (two heads)
    beside = dict(n_set=2, row_stride=640, max_keys=100)
    assert _call(L, _keys(v=P + W, set_stride=128, **beside)) == wh.WH_EINVAL          # set 1's keys are set 0's values
    assert _call(L, _keys(v=P + 2 * W + 16, set_stride=256, **beside)) == wh.WH_EINVAL  # a part of them
    assert _call(L, _keys(v=P + 4 * W, set_stride=128, n_set=2, row_stride=512)) == wh.WH_EINVAL   # the next row's keys
    # sets half a row out of step: the last value row of set 0, 99 rows and a half on, is set 1's first key row
    assert _call(L, _keys(v=P + W, n_set=2, row_stride=256, set_stride=99 * 256 + 128)) == wh.WH_EINVAL
    if not torch.cuda.is_available():
        assert _call(L, _keys(v=P + W, set_stride=256, **beside)) == wh.WH_ENODEV       # K0 V0 K1 V1
        assert _call(L, _keys(v=P + 2 * W, set_stride=128, **beside)) == wh.WH_ENODEV   # K0 K1 V0 V1
        assert _call(L, _keys(v=P - W, k=P, n_set=2, row_stride=512, set_stride=256)) == wh.WH_ENODEV   # V0 K0 V1 K1
        assert _call(L, _keys(v=P + W, n_set=2, row_stride=256, set_stride=100 * 256 + 128)) == wh.WH_ENODEV


def test_workspace_holds_what_can_stay_and_no_more(L):
    size = L.wh_cache_evict_workspace
    assert size(3, 300, 100, 1 << 30) == size(3, 300, 100, 100) > 3 * 300 * 100 * 4      # a budget past the cache
    wide = dict(row_stride=19200, set_stride=1920000, v=P + (1 << 26), weight=P + (1 << 27))
    # the indices go to kept: the counts are all that is left
    assert _call(L, _keys(**wide), n_kv=300, kept=FAKE, ws_bytes=255) == wh.WH_ENOSPC
    if not torch.cuda.is_available():
        assert _call(L, _keys(**wide), n_kv=300, kept=FAKE, ws_bytes=256) == wh.WH_ENODEV
