"""Memory that the binding takes by itself: it belongs to the stream that the call is launched on, and a call can be
recorded without handing it any."""
import pytest
import torch

from whisper_audio_encoder_gb300 import build, wh

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    build.build()
    wh.lib()


def stream_of(t):
    """The stream (its handle) in whose order the allocator hands t's memory out."""
    at = t.data_ptr()
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= at < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("memory of no segment")


def _bf(*shape, seed=0):
    gen = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(*shape, generator=gen, device="cuda").bfloat16()


def _prefix():
    q, k, v = _bf(40, 128), _bf(1, 300, 128, seed=1), _bf(1, 300, 128, seed=2)
    return lambda stream=None: wh.wh_prefix_attention(q, 2, prefix=wh.Keys(k, v), stream=stream)


def _evict():
    k, v, w = _bf(3, 300, 128), _bf(3, 300, 128, seed=1), torch.rand(3, 2, 300, device="cuda")
    to = wh.Keys(torch.zeros_like(k), torch.zeros_like(v), None, torch.zeros_like(w))
    return lambda stream=None: wh.wh_cache_evict(wh.Keys(k, v, None, w), 2, 100, 10, out=to, stream=stream)


CALLS = {"wh_prefix_attention": _prefix, "wh_cache_evict": _evict}


@pytest.mark.parametrize("name", CALLS)
def test_results_belong_to_the_launching_stream(name):
    call = CALLS[name]()
    ref = call()
    assert stream_of(ref) == torch.cuda.current_stream().cuda_stream
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = call(s)
    assert stream_of(got) == s.cuda_stream
    s.synchronize()
    assert torch.equal(got, ref)
    with torch.cuda.stream(s):
        assert stream_of(call()) == s.cuda_stream and stream_of(call(s)) == s.cuda_stream
    s.synchronize()


@pytest.mark.parametrize("name", CALLS)
def test_memory_is_not_handed_out_again_while_the_caller_s_stream_reads_it(name):
    """A result of another stream that the current one still reads when it is dropped."""
    call, s = CALLS[name](), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(s)
    s.synchronize()
    a = torch.randn(8192, 8192, device="cuda").bfloat16()
    for _ in range(20):                                # several ms of work that the read below comes behind
        a @ a
    copy, at = got.clone(), got.data_ptr()
    busy = torch.cuda.Event()
    busy.record()
    del got
    again = call(s)
    assert not busy.query(), "the current stream was to be busy still"
    assert again.data_ptr() != at
    torch.cuda.synchronize()
    assert torch.equal(copy, again)


def test_recorded_without_a_workspace():
    """Calls that need workspace, recorded with none given: the graph keeps what they took, and later calls of the same
    sizes do not disturb it."""
    B, H, n, cap = 40, 4, 700, 3000
    q, k, v = _bf(B, 64 * H), _bf(1, n, 64 * H, seed=1), _bf(1, n, 64 * H, seed=2)
    ko, vo = _bf(B, 60, 64 * H, seed=3), _bf(B, 60, 64 * H, seed=4)
    ck, cv, cw = _bf(2, cap, 64 * H, seed=5), _bf(2, cap, 64 * H, seed=6), torch.rand(2, H, cap, device="cuda")
    assert wh.lib().wh_prefix_attention_workspace(B, 1, H, H, 1, n, 60, 0) > 0
    assert wh.lib().wh_cache_evict_workspace(2, H, cap, 1200) > 0
    def fresh():
        return wh.Keys(torch.zeros(2, 1200, 64 * H, dtype=torch.bfloat16, device="cuda"),
                       torch.zeros(2, 1200, 64 * H, dtype=torch.bfloat16, device="cuda"),
                       torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(2, H, 1200, device="cuda"))

    def calls(out, to, queries):
        wh.wh_prefix_attention(queries, H, prefix=wh.Keys(k, v), own=wh.Keys(ko, vo), out=out)
        wh.wh_cache_evict(wh.Keys(ck, cv, None, cw), H, 1200, 30, out=to)

    ref, ref_to = torch.empty_like(q), fresh()
    calls(ref, ref_to, q)
    out, to = torch.zeros_like(q), fresh()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        calls(out, to, q)
        calls(out, to, q)
    other, other_to = torch.empty_like(q), fresh()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(10):
        graph.replay()
        with torch.cuda.stream(s):                     # eager calls of the same sizes beside the replay
            calls(other, other_to, q if i % 2 else q * 2)
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and wh.wh_status() == wh.WH_OK
    for a, b in ((to.k, ref_to.k), (to.v, ref_to.v), (to.weight, ref_to.weight), (to.n_keys, ref_to.n_keys)):
        assert torch.equal(a, b)


def _older():
    """The calls that take their results' and their workspace's memory themselves."""
    pcm = torch.randn(2, 16000, device="cuda")
    x, g, w = torch.randn(64, 384, device="cuda"), torch.ones(384, device="cuda"), _bf(384, 384)
    kv, rows = _bf(2, 1500, 768), _bf(200, 576)
    cross = wh.CrossKV(384, [{"wk": _bf(384, 384).float().cpu().numpy(), "wv": _bf(384, 384).float().cpu().numpy(), "bv": None}])
    mem = torch.randn(1, 100, 384, device="cuda")
    return {
        "wh_frontend": lambda s=None: wh.wh_frontend(pcm, 80, stream=s),
        "wh_frontend_long": lambda s=None: wh.wh_frontend_long(pcm[0], 80, stream=s),
        "wh_resample": lambda s=None: wh.wh_resample(pcm, 44100, stream=s),
        "wh_layer_norm": lambda s=None: wh.wh_layer_norm(x, g, g, stream=s),
        "wh_linear": lambda s=None: wh.wh_linear(w, w, stream=s),
        "wh_attention": lambda s=None: wh.wh_attention(rows, 1, 200, 3, stream=s),
        "wh_decode_attention": lambda s=None: wh.wh_decode_attention(w[:2], kv, kv[..., 384:], 768, 768 * 1500, 1500, 6, stream=s),
        "wh_prepare_cross": lambda s=None: cross.wh_prepare_cross(mem, stream=s),
    }


@pytest.mark.parametrize("name", ["wh_frontend", "wh_frontend_long", "wh_resample", "wh_layer_norm", "wh_linear", "wh_attention",
                                  "wh_decode_attention", "wh_prepare_cross"])
def test_older_calls_take_the_launching_stream_s_memory_too(name, monkeypatch):
    call = _older()[name]
    ref = call()                                       # (with whatever a class keeps)
    torch.cuda.synchronize()
    s, taken, empty = torch.cuda.Stream(), [], torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: (taken.append(torch.cuda.current_stream().cuda_stream), empty(*a, **kw))[1])
    s.wait_stream(torch.cuda.current_stream())
    got = call(s)
    monkeypatch.undo()
    assert taken and set(taken) == {s.cuda_stream} and stream_of(got) == s.cuda_stream
    s.synchronize()
    assert torch.equal(got, ref) and wh.wh_status() == wh.WH_OK
