"""GPU results of wh_cache_evict against the oracle's choice: every kept row, weight, index and count must
be the very bits of the cache, every other byte must stay as it was."""
import numpy as np
import pytest
import torch

from oracle import whisper_ref as R
from whisper_audio_encoder_gb300 import build, wh

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    build.build()
    wh.lib()


def _bits(shape, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    return torch.randint(-2 ** 15, 2 ** 15, shape, generator=gen, device="cuda", dtype=torch.int16).view(torch.bfloat16)


def _weights(shape, kind, seed):
    rng = np.random.default_rng(seed)
    w = rng.random(shape).astype(np.float32) ** 6
    if kind == "ties":
        w = np.round(w * 4) / 4
    elif kind == "equal":
        w[:] = 0.5
    elif kind == "odd":
        for x in (np.nan, np.inf, -np.inf, -0.0, 0.0, -1.0, np.float32(1e-42)):
            w[rng.random(shape) < 0.1] = x
    return w


def same(a, b):
    """Bit for bit (NaN payloads too)."""
    view = {torch.bfloat16: torch.int16, torch.float32: torch.int32, torch.int32: torch.int32}[a.dtype]
    return torch.equal(a.contiguous().view(view), b.contiguous().view(view))


class Case:
    def __init__(self, heads, cap, counts, budget, recent, kind="plain", layout="apart", seed=0):
        self.h, self.cap, self.counts, self.m, self.r = heads, cap, counts, budget, recent
        s, d = len(counts), 64 * heads
        if layout == "kv":                                       # [K | V] rows, some columns of neither
            x = _bits((s, cap, 2 * d + 64), seed)
            self.k, self.v = x[..., :d], x[..., d:2 * d]
        elif layout == "beside":                                 # [key][set]
            x = _bits((2, cap, s, d), seed)
            self.k, self.v = x[0].transpose(0, 1), x[1].transpose(0, 1)
        else:
            x = _bits((2, s, cap, d), seed)
            self.k, self.v = x[0], x[1]
        self.store = x
        self.w = torch.from_numpy(_weights((s, heads, cap), kind, seed)).cuda()
        self.n = torch.tensor(counts, dtype=torch.int32, device="cuda")

    def expected(self, k_to, v_to, w_to, kept):
        """The buffers after the call, from what they and the cache held before."""
        k_to, v_to, w_to, kept = k_to.clone(), v_to.clone(), w_to.clone(), kept.clone()
        w = self.w.cpu().numpy()
        for i, n in enumerate(self.counts):
            for h in range(self.h):
                at = torch.from_numpy(R.cache_evict(w[i, h, :n], self.m, self.r)).cuda()
                c, cols = len(at), slice(64 * h, 64 * h + 64)
                k_to[i, :c, cols], v_to[i, :c, cols] = self.k[i, at, cols], self.v[i, at, cols]
                w_to[i, h, :c] = self.w[i, h, at]
                kept[i, h, :c] = at.int()
        return k_to, v_to, w_to, kept

    def check(self, in_place, cap_out=None, stream=None, with_kept=True):
        s, d = len(self.counts), 64 * self.h
        kept = torch.full((s, self.h, self.m), -7, dtype=torch.int32, device="cuda")
        if in_place:
            k, v, w, n = self.k, self.v, self.w, self.n
        else:
            cap_out = cap_out or min(self.m, self.cap)
            k, v = _bits((2, s, cap_out, d), 99)
            w, n = torch.full((s, self.h, cap_out), 3.0, device="cuda"), torch.full((s,), -1, dtype=torch.int32, device="cuda")
        ek, ev, ew, ekept = self.expected(k, v, w, kept)
        others = self.store.clone() if in_place else None
        cache = wh.Keys(self.k, self.v, self.n, self.w)
        got = wh.wh_cache_evict(cache, self.h, self.m, self.r, out=None if in_place else wh.Keys(k, v, n, w),
                                kept=kept if with_kept else None, stream=stream)
        torch.cuda.synchronize()
        assert wh.wh_status() == wh.WH_OK
        assert got is n and n.tolist() == [min(x, self.m) for x in self.counts]
        assert same(k, ek) and same(v, ev) and same(w, ew)
        assert not with_kept or torch.equal(kept, ekept)
        if in_place and self.store.shape[-1] > 2 * d:
            assert same(self.store[..., 2 * d:], others[..., 2 * d:])


CASES = {
    "one key of two": dict(heads=1, cap=2, counts=[2], budget=1, recent=0),
    "ragged": dict(heads=3, cap=448, counts=[448, 0, 1, 223, 224, 225, 300], budget=224, recent=32),
    "ties": dict(heads=4, cap=300, counts=[300, 299, 257, 256, 255], budget=100, recent=7, kind="ties"),
    "all equal": dict(heads=2, cap=700, counts=[700, 513], budget=512, recent=0, kind="equal"),
    "odd weights": dict(heads=4, cap=333, counts=[333, 200, 90], budget=77, recent=5, kind="odd"),
    "mostly NaN": dict(heads=2, cap=40, counts=[40, 39], budget=38, recent=1, kind="odd"),
    "only recent": dict(heads=2, cap=100, counts=[100, 33], budget=32, recent=32),
    "long": dict(heads=2, cap=40001, counts=[40001, 17, 33000], budget=5003, recent=100, kind="ties"),
    "budget past the cache": dict(heads=2, cap=20, counts=[20, 3], budget=50, recent=10),
    "kv rows": dict(heads=5, cap=150, counts=[150, 149, 60], budget=50, recent=9, layout="kv"),
    "sets beside each other": dict(heads=2, cap=90, counts=[90, 10, 64], budget=33, recent=1, layout="beside"),
    "a few long heads": dict(heads=2, cap=1900, counts=[1900, 1025, 1024], budget=900, recent=50, kind="ties"),
    "many long heads": dict(heads=8, cap=1030, counts=[1030 - 7 * i for i in range(40)], budget=700, recent=50, kind="odd"),
    "long, many heads": dict(heads=20, cap=9001, counts=[9001, 9000, 8193, 700], budget=333, recent=3, kind="ties"),
    "longer, many heads": dict(heads=20, cap=17001, counts=[17001, 16385, 15000, 333], budget=500, recent=3, kind="odd"),
    "thousands of keys, many heads": dict(heads=20, cap=4001, counts=[4001 - 37 * i for i in range(31)], budget=133, recent=3, kind="ties"),
    "most of it stays": dict(heads=20, cap=1500, counts=[1500 - 11 * i for i in range(16)], budget=1200, recent=3, kind="ties"),
    "few heads, most of it stays": dict(heads=1, cap=30000, counts=[30000, 20000, 16001], budget=16000, recent=500, layout="kv"),
    "long, equal": dict(heads=1, cap=33333, counts=[33333], budget=32768, recent=0, kind="equal"),
    "long, odd weights": dict(heads=2, cap=50001, counts=[50001, 40000], budget=49999, recent=7, kind="odd"),
    "many sets": dict(heads=2, cap=64, counts=[(7 * i) % 65 for i in range(300)], budget=31, recent=4, kind="ties"),
}


@pytest.mark.parametrize("in_place", [False, True], ids=["out", "in_place"])
@pytest.mark.parametrize("name", CASES)
def test_choice(name, in_place):
    Case(seed=len(name), **CASES[name]).check(in_place)


@pytest.mark.parametrize("n", [1, 31, 32, 33, 255, 256, 257, 511, 512, 513, 1023, 1024, 1025, 2047, 2048, 2049, 4096, 4097, 8191, 8192, 8193, 16384, 16385, 32768, 32769, 65535, 65536])
def test_lengths(n):
    Case(heads=2, cap=n, counts=[n, n // 2], budget=max(1, n // 3), recent=min(5, max(1, n // 3)), seed=n).check(n % 2 == 0)


@pytest.mark.parametrize("in_place", [False, True], ids=["out", "in_place"])
def test_weights_of_any_size(in_place):
    """Long caches, whose threshold is looked for by ranges of sizes: a set each of small, large, negative and mixed
    weights, of weights next to the powers of two and of two values only."""
    cap = 9000
    c = Case(heads=2, cap=cap, counts=[cap] * 8 + [8999], budget=4000, recent=10)
    rng = np.random.default_rng(3)
    for i, f in enumerate((1e-30, 2.0 ** -19, 512.0, 1e30, -1.0)):
        c.w[i] *= f
    powers = np.float32(2.0) ** rng.integers(-24, 13, (2, cap)).astype(np.float32)
    c.w[5] = torch.from_numpy(np.nextafter(powers, powers * rng.choice([0.0, 1.0, 2.0], (2, cap)).astype(np.float32)))
    c.w[6] = torch.from_numpy(rng.choice(np.float32([2.0 ** -19, 512.0]), (2, cap)))
    c.w[7] = torch.from_numpy(np.where(rng.random((2, cap)) < 0.44, np.float32(512.0), np.float32(2.0 ** -20)))
    c.check(in_place)


@pytest.mark.parametrize("kept", [1, 2, 65534])
@pytest.mark.parametrize("value", [0.0, float("nan"), -1.0, 1.0])
def test_as_many_equal_weights_as_a_cluster_counts(value, kept):
    """65535 keys of one weight: their number is the largest that the choice's counters hold."""
    c = Case(heads=1, cap=65535, counts=[65535], budget=kept, recent=0)
    c.w.fill_(value)
    c.check(False)


def test_into_a_larger_cache_on_another_stream_without_indices():
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    Case(heads=3, cap=200, counts=[200, 150], budget=60, recent=10, seed=1).check(False, cap_out=111, stream=s, with_kept=False)
    Case(heads=3, cap=200, counts=[200, 150], budget=60, recent=10, seed=1).check(True, stream=s, with_kept=False)


def test_counts_out_of_range_and_without_counts():
    c = Case(heads=2, cap=50, counts=[50, 50], budget=20, recent=3, seed=2)
    k, v = torch.zeros(2, 2, 20, 128, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(2, 2, 20, device="cuda")
    got = wh.wh_cache_evict(wh.Keys(c.k, c.v, None, c.w), 2, 20, 3, out=wh.Keys(k, v, None, w))
    assert got.tolist() == [20, 20] and wh.wh_status() == wh.WH_OK
    first = (k.clone(), v.clone(), w.clone())
    c.n.copy_(torch.tensor([51, -1]))
    got = wh.wh_cache_evict(wh.Keys(c.k, c.v, c.n, c.w), 2, 20, 3, out=wh.Keys(k, v, None, w))
    assert got.tolist() == [20, 0] and wh.wh_status() == wh.WH_EBOUNDS
    assert same(k, first[0]) and same(v, first[1]) and same(w, first[2])      # set 1 keeps nothing: nothing is written


def test_recorded_and_replayed():
    c = Case(heads=4, cap=300, counts=[300, 250, 100], budget=120, recent=20, seed=3)
    k, v = torch.zeros(2, 3, 120, 256, dtype=torch.bfloat16, device="cuda")
    w, n = torch.zeros(3, 4, 120, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    cache, out = wh.Keys(c.k, c.v, c.n, c.w), wh.Keys(k, v, n, w)
    kept = torch.zeros(3, 4, 120, dtype=torch.int32, device="cuda")
    ws = torch.empty(max(256, wh.lib().wh_cache_evict_workspace(3, 4, 300, 120)), dtype=torch.uint8, device="cuda")
    wh.wh_cache_evict(cache, 4, 120, 20, out=out, kept=kept, workspace=ws)
    ref = [x.clone() for x in (k, v, w, n, kept)]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        wh.wh_cache_evict(cache, 4, 120, 20, out=out, kept=kept, workspace=ws)
    for x in (k, v, w, n):
        x.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(same(a, b) for a, b in zip((k, v, w, n, kept), ref)) and wh.wh_status() == wh.WH_OK


def test_offsets_past_32_bits():
    rows, stride = 130, 1 << 25
    if torch.cuda.mem_get_info()[0] < 3 * rows * stride * 2:
        pytest.skip("needs 18 GB of device memory")
    big = torch.empty(rows * stride, dtype=torch.bfloat16, device="cuda").as_strided((1, rows, 256), (0, stride, 1))
    small = _bits((1, rows, 256), 5)
    big.copy_(small)
    c = Case(heads=2, cap=rows, counts=[rows], budget=50, recent=4, seed=6)
    c.k, c.v, c.store = big[..., :128], big[..., 128:], small
    c.check(True)


def test_attend_evict_attend():
    """A decoder's use: attend with accumulators, cut the cache in place, attend over what stayed.  The
    attention after eviction is the attention over the kept keys."""
    rng = np.random.default_rng(7)
    H, cap, counts, m, r = 4, 60, [60, 41, 10], 30, 6
    from whisper_audio_encoder_gb300 import synth
    bf = lambda *s: synth.bf16_round(rng.standard_normal(s).astype(np.float32))  # noqa: E731
    k, v = bf(3, cap, 64 * H), bf(3, cap, 64 * H)
    dev = lambda a: torch.from_numpy(a).to(torch.bfloat16).cuda()  # noqa: E731
    own = wh.Keys(dev(k), dev(v), torch.tensor(counts, dtype=torch.int32, device="cuda"), torch.zeros(3, H, cap, device="cuda"))
    for _ in range(5):
        wh.wh_prefix_attention(dev(bf(3, 64 * H)), H, own=own)
    w = own.weight.cpu().numpy()
    assert np.allclose(w.sum(2), 5.0, atol=1e-4)
    wh.wh_cache_evict(own, H, m, r)
    q = bf(3, 64 * H)
    out = wh.wh_prefix_attention(dev(q), H, own=own).float().cpu().numpy()
    assert own.n_keys.tolist() == [30, 30, 10]
    for b, n in enumerate(counts):
        for h in range(H):
            at, cols = R.cache_evict(w[b, h, :n], m, r), slice(64 * h, 64 * h + 64)
            ref, spread, _, _ = R.prefix_attention(q[b:b + 1, cols], 1, 1, 1, [], [None], [(k[b, at, cols], v[b, at, cols])])
            assert np.all(np.abs(out[b, cols] - ref[0]) <= 2.0 ** -8 * np.abs(ref[0]) + (2.0 ** -11 + 2.0 ** -12) * spread[0])
    assert wh.wh_status() == wh.WH_OK


def test_beam_search_loop_with_a_bounded_cache():
    """Three decoder layers as beam search uses them: the hypotheses of two windows share their window's
    cross-attention keys (wh_prepare_cross rows) and their utterance's prompt, keep their own tokens' keys with
    accumulated weight, and all layers' caches are cut in one call whenever they are full.  Every step's attention
    is compared with the oracle on the very keys that the caches hold."""
    from whisper_audio_encoder_gb300 import synth
    rng = np.random.default_rng(8)
    bf = lambda *s: synth.bf16_round(rng.standard_normal(s).astype(np.float32))  # noqa: E731
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(torch.bfloat16).cuda()  # noqa: E731
    layers, windows, beams, H, cap, m, r, n_ctx, prompt = 3, 2, 5, 2, 12, 7, 2, 90, 20
    B, d = windows * beams, 64 * H
    cross, pre = bf(layers, windows, n_ctx, 2 * d), bf(layers, windows, prompt, 2 * d)
    crossd, pred = dev(cross), dev(pre)
    kc, vc = torch.zeros(2, layers * B, cap, d, dtype=torch.bfloat16, device="cuda")
    weight = torch.zeros(layers * B, H, cap, device="cuda")
    n = torch.zeros(layers * B, dtype=torch.int32, device="cuda")
    whole = wh.Keys(kc, vc, n, weight)
    own = [wh.Keys(*(x[l * B:(l + 1) * B] for x in (kc, vc, n, weight))) for l in range(layers)]
    host = lambda x: x.float().cpu().numpy()  # noqa: E731
    group = [b // beams for b in range(B)]
    for step in range(19):
        if step and int(n[0]) == cap:
            before = host(weight).astype(np.float32), host(kc)
            wh.wh_cache_evict(whole, H, m, r)
            assert n.tolist() == [m] * (layers * B)
            for i in (0, layers * B - 1):
                for h in range(H):
                    at = R.cache_evict(before[0][i, h], m, r)
                    assert np.array_equal(host(kc)[i, :m, 64 * h:64 * h + 64], before[1][i, at, 64 * h:64 * h + 64])
        at = int(n[0])
        kc[:, at], vc[:, at] = dev(bf(layers * B, d)), dev(bf(layers * B, d))
        n += 1
        for l in range(layers):
            q = bf(B, d)
            w0 = host(own[l].weight)
            o_self = wh.wh_prefix_attention(dev(q), H, prefix=wh.Keys(pred[l][..., :d], pred[l][..., d:]), own=own[l])
            o_cross = wh.wh_prefix_attention(dev(q), H, prefix=wh.Keys(crossd[l][..., :d], crossd[l][..., d:]))
            k, v = host(own[l].k), host(own[l].v)
            ref, spread, _, wo = R.prefix_attention(q, 1, H, H, [(x[:, :d], x[:, d:]) for x in pre[l]], group,
                                                    [(k[b, :at + 1], v[b, :at + 1]) for b in range(B)])
            assert np.all(np.abs(host(o_self) - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -12) * spread)
            add = host(own[l].weight)[:, :, :at + 1] - w0[:, :, :at + 1]
            assert np.allclose(add, np.stack(wo), rtol=2.0 ** -11, atol=2.0 ** -20)
            ref, spread, _, _ = R.prefix_attention(q, 1, H, H, [(x[:, :d], x[:, d:]) for x in cross[l]], group, [None] * B)
            assert np.all(np.abs(host(o_cross) - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -12) * spread)
    assert wh.wh_status() == wh.WH_OK


def test_refusals_of_the_binding():
    c = Case(heads=2, cap=10, counts=[10], budget=4, recent=1)
    cache = wh.Keys(c.k, c.v, c.n, c.w)
    small = torch.zeros(2, 1, 4, 128, dtype=torch.bfloat16, device="cuda")
    bad = [dict(cache=wh.Keys(c.k, c.v, c.n)), dict(n_kv_head=3), dict(n_kv_head=1), dict(budget=0), dict(recent=5),
           dict(out=wh.Keys(small[0], small[1])), dict(out=wh.Keys(c.k[:, :4], c.v[:, :4], None, torch.zeros(1, 2, 4, device="cuda"))),
           dict(kept=torch.zeros(1, 2, 5, dtype=torch.int32, device="cuda")), dict(workspace=torch.zeros(64, device="cuda")[1:])]
    before = c.store.clone()
    for kw in bad:
        args = dict(cache=cache, n_kv_head=2, budget=4, recent=1)
        args.update(kw)
        with pytest.raises(wh.WhError):
            wh.wh_cache_evict(**args)
    assert same(c.store, before) and wh.wh_status() == wh.WH_OK


def test_numbers_past_the_library_s_types_are_refused():
    """A count that a 32-bit argument would silently cut."""
    c = Case(heads=2, cap=10, counts=[10], budget=4, recent=1)
    cache = wh.Keys(c.k, c.v, c.n, c.w)
    before = c.store.clone()
    for kw in (dict(budget=(1 << 32) + 4), dict(recent=1 << 32), dict(n_kv_head=2 - (1 << 32)), dict(recent=-1)):
        with pytest.raises(wh.WhError):
            wh.wh_cache_evict(**{**dict(cache=cache, n_kv_head=2, budget=4, recent=1), **kw})
    q = torch.zeros(1, 128, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(wh.WhError):
        wh.wh_prefix_attention(q, 2, prefix=wh.Keys(c.k, c.v), n_kv_head=2 - (1 << 32))
    for shape in ((1, (1 << 32) + 1, 128), ((1 << 32) + 1, 1, 128), (65536, 1, 128)):
        with pytest.raises(wh.WhError):
            wh.Keys(q[None].expand(*shape), q[None].expand(*shape))
    assert same(c.store, before) and wh.wh_status() == wh.WH_OK


def test_no_sets_and_single_rows_of_odd_width():
    e = torch.zeros(0, 9, 128, dtype=torch.bfloat16, device="cuda")
    none = wh.Keys(e, e.clone(), None, torch.zeros(0, 2, 9, device="cuda"))
    assert wh.wh_cache_evict(none, 2, 4, 1).shape == (0,)
    # one key of a row of 131 values: the stride of a dimension of size one is not used
    k, v = (torch.randn(1, 1, 131, device="cuda").bfloat16() for _ in range(2))
    w = torch.ones(1, 2, 1, device="cuda")
    assert wh.wh_cache_evict(wh.Keys(k, v, None, w), 2, 1, 0).tolist() == [1]
    out = wh.wh_prefix_attention(torch.zeros(1, 128, dtype=torch.bfloat16, device="cuda"), 2, own=wh.Keys(k, v, None, w))
    assert torch.equal(out, v[:, 0, :128]) and w.tolist() == [[[2.0], [2.0]]] and wh.wh_status() == wh.WH_OK


@pytest.mark.parametrize("in_place", [False, True], ids=["out", "in_place"])
@pytest.mark.parametrize("budget", [33, 64, 65, 1000])
def test_budgets_up_to_and_past_the_cache_without_indices(budget, in_place):
    """The indices then stand in the workspace, as many a head as can stay."""
    Case(heads=20, cap=64, counts=[(7 * i) % 65 for i in range(40)], budget=budget, recent=4, kind="ties",
         seed=9).check(in_place, cap_out=64, with_kept=False)


def test_a_budget_of_any_size_needs_no_more_memory_than_the_cache():
    c = Case(heads=20, cap=64, counts=[(7 * i) % 65 for i in range(40)], budget=1 << 30, recent=1 << 30, seed=9)
    k, v, w = torch.zeros_like(c.k), torch.zeros_like(c.v), torch.zeros_like(c.w)
    n = torch.zeros_like(c.n)
    wh.wh_cache_evict(wh.Keys(c.k, c.v, c.n, c.w), 20, 1 << 30, 1 << 30, out=wh.Keys(k, v, n, w))
    assert torch.equal(n, c.n) and wh.wh_status() == wh.WH_OK
    for i, x in enumerate(c.counts):
        assert same(k[i, :x], c.k[i, :x]) and same(v[i, :x], c.v[i, :x]) and same(w[i, :, :x], c.w[i, :, :x])
        assert not k[i, x:].any() and not v[i, x:].any() and not w[i, :, x:].any()
