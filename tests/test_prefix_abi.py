"""wh_prefix_attention rejects bad arguments on the host before it touches a device (no GPU needed)."""
import ctypes

import pytest
import torch

from whisper_audio_encoder_gb300 import build, wh

FAKE, ODD = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 4)   # never dereferenced
P = 1 << 20


@pytest.fixture(scope="module")
def L():
    build.build()
    return wh.lib()


def _keys(**kw):
    base = dict(k=P, v=P, row_stride=384, set_stride=384 * 100, n_keys=None, weight=None, n_set=2, max_keys=100)
    base.update(kw)
    return wh.wh_keys(*[base[f] for f, _ in wh.wh_keys._fields_])


def _call(L, q=FAKE, q_stride=384, batch=4, n_query=1, n_head=6, n_kv=6, prefix=None, start=None, own=None, out=FAKE,
          ws=FAKE, ws_bytes=1 << 40):
    ref = lambda s: None if s is None else ctypes.byref(s)  # noqa: E731
    return L.wh_prefix_attention(q, q_stride, batch, n_query, n_head, n_kv, ref(prefix), start, ref(own), out, ws,
                                 ws_bytes, None)


def test_rejects_bad_shapes_and_pointers(L):
    ok = _keys()
    bad = [dict(n_query=0), dict(n_query=2000), dict(n_head=0), dict(n_kv=4), dict(n_kv=0), dict(batch=-1),
           dict(batch=65536), dict(q_stride=376), dict(q_stride=388), dict(batch=3), dict(q=None), dict(q=ODD),
           dict(out=None), dict(out=ODD), dict(ws=ctypes.c_void_p(P + 16)),
           dict(start=ctypes.c_void_p(P + 2)), dict(batch=65535, n_query=1024, n_head=1020, n_kv=6, q_stride=65536)]
    for kw in bad:
        assert _call(L, prefix=ok, **kw) == wh.WH_EINVAL, kw
    assert _call(L) == wh.WH_EINVAL                                        # neither prefix nor own keys
    assert _call(L, own=_keys(n_set=3)) == wh.WH_EINVAL                    # own sets must be the sequences
    assert _call(L, own=_keys(n_set=4), start=FAKE) == wh.WH_EINVAL        # groups of no prefix
    for kw in (dict(k=None), dict(v=None), dict(k=P + 8), dict(row_stride=376), dict(row_stride=388), dict(set_stride=-8),
               dict(set_stride=12), dict(n_set=0), dict(n_set=65536), dict(max_keys=0), dict(max_keys=(1 << 30) + 1),
               dict(n_keys=P + 2), dict(weight=P + 1)):
        assert _call(L, prefix=_keys(**kw)) == wh.WH_EINVAL, kw


def test_workspace(L):
    size = L.wh_prefix_attention_workspace
    assert size(4, 1, 6, 6, 2, 100, 0, 0) == 0                             # nothing to keep between kernels
    need = size(4, 1, 6, 6, 2, 100, 0, wh.WH_PREFIX_WEIGHT)
    assert need >= 4 * 6 * 8                                               # every row's maximum and sum
    weighed = _keys(weight=P)
    assert _call(L, prefix=weighed, ws_bytes=need - 1) == wh.WH_ENOSPC
    assert _call(L, prefix=weighed, ws=None) == wh.WH_ENOSPC
    for args in ((0, 1, 6, 6, 2, 100, 0, 0), (4, 1, 6, 5, 2, 100, 0, 0), (4, 1, 6, 6, -1, 100, 0, 0), (4, 1, 6, 6, 3, 100, 0, 2),
                 (4, 1, 6, 6, 2, 100, 0, 8)):
        assert size(*args) == 0
    # partial results: of long keys for few rows, and of a prefix before own keys
    assert size(1, 1, 6, 6, 1, 300000, 0, 0) > 6 * 17 * 64 * 4
    assert size(4, 1, 6, 6, 2, 100, 50, wh.WH_GROUP_TABLE) >= 4 * 6 * (64 * 4 + 8)


def test_empty_batch_is_a_no_op(L):
    assert _call(L, batch=0, prefix=_keys(), q=None, out=None, ws=None, ws_bytes=0) == wh.WH_OK
    assert _call(L, batch=0, own=_keys(n_set=0, k=None, v=None), q=None, out=None, ws=None, ws_bytes=0) == wh.WH_OK


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")
def test_no_device_is_reported(L):
    assert _call(L, prefix=_keys()) == wh.WH_ENODEV


def test_binding_checks_its_tensors():
    k = torch.zeros(2, 10, 128, dtype=torch.bfloat16)
    for args in ((k, k), (k.float(), k.float()), (k, k[:, :5]), (k[0], k[0]), (k.transpose(1, 2), k.transpose(1, 2))):
        with pytest.raises(wh.WhError):                                    # not on a CUDA device, or not such a tensor
            wh.Keys(*args)
    with pytest.raises(wh.WhError):
        wh.wh_prefix_attention(k[0], 2)


def test_keys_are_packed_field_by_field():
    c = wh.wh_keys.from_buffer_copy(wh._pack_keys(1 << 40, 2, 3, 4, 5, 0, 7, 8))
    assert [getattr(c, f) for f, _ in wh.wh_keys._fields_] == [1 << 40, 2, 3, 4, 5, None, 7, 8]
