"""GPU parity of wh_prefix_attention against the oracle in 64 bits.

Tolerances, counted from the roundings:
- out: its bf16 rounding, 2^-8 |ref|; the softmax weights enter the value product with 11 bits of
  mantissa (half a step: 2^-11) where a prefix has at most 16 rows (queries x query heads of a key head)
  on average, with 8 bits (half a step: 2^-8) where it has more, an error of at most that times
  sum p |v|; and fp32 scores, 2^-12 sum p |v|: a score of 64 products in fp32 is off by at most
  64 2^-24 sum |q k| / 8 < 2^-13.5 for the inputs here (sum |q k| < 180), and so is the maximum's part.
- weights: each weight is off by twice the score's error (its own and the sum's), 2^-12.5, plus the
  exponential's 2^-22, relative; sums of up to 400 rows add 400 2^-24 < 2^-15.
"""
import numpy as np
import pytest
import torch

from oracle import whisper_ref as R
from whisper_audio_encoder_gb300 import build, synth, wh

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    build.build()
    wh.lib()


def out_tol(ref, spread, rows_a_prefix=0):
    return 2.0 ** -8 * np.abs(ref) + ((2.0 ** -8 if rows_a_prefix > 16 else 2.0 ** -11) + 2.0 ** -12) * spread


def _bf(rng, *shape):
    return synth.bf16_round(rng.standard_normal(shape).astype(np.float32))


def _dev(a, dtype=torch.bfloat16):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()


class Case:
    """A batch with its prefixes and own caches; rows past a set's count hold NaN."""

    def __init__(self, seed, n_head, n_kv, nq, groups=(), n_pre=(), cap_pre=0, n_own=None, cap_own=0, batch=None,
                 weigh=False, start=None):
        rng = np.random.default_rng(seed)
        self.H, self.KV, self.nq = n_head, n_kv, nq
        self.start = start if start is not None else np.concatenate([[0], np.cumsum(groups)]).astype(np.int32)
        self.B = batch if batch is not None else (len(n_own) if n_own is not None else int(self.start[-1]))
        self.q = _bf(rng, self.B * nq, 64 * n_head)
        self.pre, self.own = None, None
        if len(n_pre):
            self.pre = [(_bf(rng, n, 64 * n_kv), _bf(rng, n, 64 * n_kv)) for n in n_pre]
        if n_own is not None:
            self.own = [(_bf(rng, n, 64 * n_kv), _bf(rng, n, 64 * n_kv)) for n in n_own]
        self.cap_pre, self.cap_own = cap_pre or max(n_pre, default=0), cap_own or max(n_own or [0])
        self.w0 = {}
        if weigh:
            for what, sets, cap in (("pre", self.pre, self.cap_pre), ("own", self.own, self.cap_own)):
                if sets is not None:
                    self.w0[what] = rng.random((len(sets), n_kv, cap)).astype(np.float32)

    def group_of(self):
        g = [None] * self.B
        for i in range(len(self.start) - 1 if self.pre is not None else 0):
            for b in range(self.start[i], self.start[i + 1]):
                g[b] = i
        return g

    def keys(self, what):
        sets = getattr(self, what)
        if sets is None:
            return None
        cap = self.cap_pre if what == "pre" else self.cap_own
        kv = torch.full((2, len(sets), cap, 64 * self.KV), float("nan"), dtype=torch.bfloat16, device="cuda")
        for i, (k, v) in enumerate(sets):
            kv[0, i, :len(k)], kv[1, i, :len(k)] = _dev(k), _dev(v)
        n = torch.tensor([len(k) for k, _ in sets], dtype=torch.int32, device="cuda")
        w = _dev(self.w0[what], torch.float32) if what in self.w0 else None
        return wh.Keys(kv[0], kv[1], n, w)

    def run(self, uniform=False, **kw):
        self.pk, self.ok = self.keys("pre"), self.keys("own")
        start = None if uniform or self.pre is None else torch.from_numpy(np.asarray(self.start, np.int32)).cuda()
        out = wh.wh_prefix_attention(_dev(self.q), self.H, prefix=self.pk, own=self.ok, n_kv_head=self.KV,
                                     group_start=start, n_query=self.nq, **kw)
        assert wh.wh_status() == wh.WH_OK
        return out

    def check(self, out):
        ref, spread, wp, wo = R.prefix_attention(self.q, self.nq, self.H, self.KV, self.pre or [], self.group_of(),
                                                 self.own or [None] * self.B)
        got = out.float().cpu().numpy()
        rows = -(-self.B * self.nq * (self.H // self.KV) // len(self.pre)) if self.pre else 0
        bad = ~(np.abs(got - ref) <= out_tol(ref, spread, rows))
        assert not bad.any(), f"{bad.sum()} of {bad.size} outside; worst {np.nanmax(np.abs(got - ref)):.3e}"
        for what, ws, keys in (("pre", wp, self.pk), ("own", wo, self.ok)):
            if what not in self.w0:
                continue
            got = keys.weight.cpu().numpy()
            for i, w in enumerate(ws):
                n = w.shape[1]
                add = got[i, :, :n].astype(np.float64) - self.w0[what][i, :, :n]
                # the accumulator itself rounds: half a step of what it holds
                tol = (2.0 ** -12.5 + 2.0 ** -15) * w + 2.0 ** -23 * (self.w0[what][i, :, :n] + w) + 1e-30
                assert np.all(np.abs(add - w) <= tol), f"{what} {i}: {np.max(np.abs(add - w) - tol):.3e}"
                assert np.array_equal(got[i, :, n:], self.w0[what][i, :, n:])      # keys past the count


CASES = {
    "one key, one sequence": dict(n_head=2, n_kv=2, nq=1, groups=[1], n_pre=[1]),
    "five hypotheses": dict(n_head=6, n_kv=6, nq=1, groups=[5], n_pre=[1500]),
    "16 and 17 rows": dict(n_head=3, n_kv=3, nq=1, groups=[16, 17, 15], n_pre=[65, 64, 63]),
    "33 rows": dict(n_head=2, n_kv=2, nq=1, groups=[33, 33], n_pre=[129, 1], cap_pre=150),
    "ragged, empty groups, empty prefix": dict(n_head=2, n_kv=2, nq=1, groups=[0, 3, 0, 1, 7], n_pre=[9, 0, 3, 100, 31],
                                               weigh=True),
    "prefix and own": dict(n_head=4, n_kv=4, nq=1, groups=[3, 4], n_pre=[223, 100], n_own=[1, 0, 224, 17, 16, 15, 3],
                           cap_own=230, weigh=True),
    "own only, some empty": dict(n_head=5, n_kv=5, nq=1, n_own=[0, 1, 448, 447, 63, 64, 65], cap_own=448, weigh=True),
    "long prefix, few rows": dict(n_head=2, n_kv=2, nq=1, groups=[2], n_pre=[20011], weigh=True),
    "long own keys": dict(n_head=2, n_kv=2, nq=1, n_own=[10007]),
    "draft of four, grouped heads": dict(n_head=8, n_kv=2, nq=4, groups=[2, 3], n_pre=[300, 41], n_own=[4, 5, 30, 4, 64],
                                         weigh=True),
    "queries that see nothing": dict(n_head=4, n_kv=2, nq=5, n_own=[0, 1, 3, 5, 9], cap_own=20, weigh=True),
    "queries that see only the prefix": dict(n_head=2, n_kv=2, nq=3, groups=[2], n_pre=[7], n_own=[0, 1]),
    "32 rows, ranges": dict(n_head=2, n_kv=2, nq=1, groups=[32], n_pre=[9001], weigh=True),
    "64 rows": dict(n_head=2, n_kv=2, nq=1, groups=[64, 64, 61], n_pre=[128, 127, 129], cap_pre=131),
    "65 rows, short prefixes": dict(n_head=3, n_kv=3, nq=1, groups=[65, 65, 65, 65], n_pre=[0, 1, 2, 300], n_own=[i % 3 for i in range(260)]),
    "128 rows, ranges": dict(n_head=4, n_kv=2, nq=2, groups=[32], n_pre=[5003], n_own=[2] * 32, weigh=True),
    "300 and 3 rows": dict(n_head=2, n_kv=2, nq=1, groups=[300, 3], n_pre=[1000, 515], weigh=True),
    "own keys in ranges": dict(n_head=3, n_kv=3, nq=1, n_own=[0, 700, 1, 64, 65, 3000, 129], cap_own=3001, weigh=True),
    "own keys in many ranges": dict(n_head=1, n_kv=1, nq=2, n_own=[40000, 2], weigh=True),
    "prefix and long own keys": dict(n_head=1, n_kv=1, nq=1, groups=[1, 1], n_pre=[700, 0], n_own=[900, 4000], weigh=True),
    "long prefix and own keys": dict(n_head=1, n_kv=1, nq=1, groups=[3], n_pre=[30000], n_own=[900, 0, 4000], weigh=True),
    "long prefix of many rows and own keys": dict(n_head=1, n_kv=1, nq=1, groups=[20], n_pre=[40000], n_own=[9 * i for i in range(20)], weigh=True),
    "many queries": dict(n_head=2, n_kv=1, nq=41, groups=[1, 2], n_pre=[50, 77], n_own=[41, 43, 100], weigh=True),
    "two ranges a cluster, the second often empty": dict(
        n_head=6, n_kv=6, nq=1, groups=[24, 20, 0, 31, 24, 24, 24, 24, 24, 24, 24, 45],
        n_pre=[1700, 0, 1699, 5, 895, 896, 897, 1024, 1, 128, 900, 640], weigh=True),
    "wide group": dict(n_head=2, n_kv=1, nq=1, groups=[201], n_pre=[333], n_own=[i % 7 for i in range(201)], weigh=True),
}


@pytest.mark.parametrize("name", CASES)
def test_parity(name):
    c = Case(seed=len(name), **CASES[name])
    c.check(c.run())


def test_equal_groups_need_no_table():
    kw = dict(n_head=4, n_kv=4, nq=2, groups=[3, 3, 3], n_pre=[70, 9, 200], weigh=True)
    a, b = Case(3, **kw), Case(3, **kw)
    x = a.run(uniform=True)
    a.check(x)
    b.check(b.run())


@pytest.mark.parametrize("keys", [50, 700, 20000])
@pytest.mark.parametrize("wide", [1, 20])
@pytest.mark.parametrize("own", [True, False])
def test_sequences_outside_every_group_have_no_prefix(keys, wide, own):
    kw = dict(n_own=[4, 0, 3, 0, 1, 6, 0] + [2] * (3 * wide)) if own else dict(batch=7 + 3 * wide)
    c = Case(4, n_head=2, n_kv=2, nq=1, start=np.array([2, 2, 5 + 3 * wide], np.int32), n_pre=[3, keys], weigh=True, **kw)
    out = c.run()
    c.check(out)
    assert torch.all(out[1] == 0) and (own or torch.all(out[[0, -1]] == 0))    # no prefix, no keys


@pytest.mark.parametrize("beams", [4, 20, 40])
def test_prepare_cross_rows_and_strided_queries(beams):
    """[K | V] rows of wh_prepare_cross, one set per window, and queries inside wider rows."""
    rng = np.random.default_rng(5)
    H, d, n_ctx = 6, 384, 77
    kv = _bf(rng, 3, n_ctx, 2 * d)
    wide = _dev(_bf(rng, 3 * beams, 3 * d))
    q = wide[:, d:2 * d]
    kvd = _dev(kv)
    out = wh.wh_prefix_attention(q, H, prefix=wh.Keys(kvd[..., :d], kvd[..., d:]))
    ref, spread, _, _ = R.prefix_attention(q.float().cpu().numpy(), 1, H, H, [(x[:, :d], x[:, d:]) for x in kv],
                                           [b // beams for b in range(3 * beams)], [None] * 3 * beams)
    assert np.all(np.abs(out.float().cpu().numpy() - ref) <= out_tol(ref, spread, beams))


@pytest.mark.parametrize("beams", [3, 20])
@pytest.mark.parametrize("layout", ["one set for all groups", "sets beside each other", "odd set stride"])
def test_set_strides(layout, beams):
    rng = np.random.default_rng(15)
    H, d, n, sets = 2, 128, 200, 3
    if layout == "one set for all groups":
        k, v = (_dev(_bf(rng, 1, n, d)).expand(sets, n, d) for _ in range(2))
    elif layout == "sets beside each other":
        k, v = (_dev(_bf(rng, n, sets, d)).transpose(0, 1) for _ in range(2))
    else:
        k, v = (_dev(_bf(rng, sets * (n * d + 8))).as_strided((sets, n, d), (n * d + 8, d, 1)) for _ in range(2))
    q = _bf(rng, sets * beams, d)
    out = wh.wh_prefix_attention(_dev(q), H, prefix=wh.Keys(k, v))
    host = lambda x: x.float().cpu().numpy()  # noqa: E731
    ref, spread, _, _ = R.prefix_attention(q, 1, H, H, list(zip(host(k), host(v))), [b // beams for b in range(sets * beams)],
                                           [None] * sets * beams)
    assert np.all(np.abs(host(out) - ref) <= out_tol(ref, spread, beams))


@pytest.mark.parametrize("beams", [3, 20])
def test_offsets_past_32_bits(beams):
    rng = np.random.default_rng(6)
    n, stride = 130, 1 << 25                             # the last key starts 4.3e9 elements in
    if torch.cuda.mem_get_info()[0] < 3 * n * stride * 2:
        pytest.skip("needs 18 GB of device memory")
    k, v, q = _bf(rng, n, 128), _bf(rng, n, 128), _bf(rng, beams, 128)
    big = torch.empty(n * stride, dtype=torch.bfloat16, device="cuda").as_strided((1, n, 256), (0, stride, 1))
    big[0, :, :128], big[0, :, 128:] = _dev(k), _dev(v)
    out = wh.wh_prefix_attention(_dev(q), 2, prefix=wh.Keys(big[..., :128], big[..., 128:]))
    ref, spread, _, _ = R.prefix_attention(q, 1, 2, 2, [(k, v)], [0] * beams, [None] * beams)
    assert np.all(np.abs(out.float().cpu().numpy() - ref) <= out_tol(ref, spread, beams))


@pytest.mark.parametrize("nq", [1, 3, 17])
def test_same_bits_again_with_a_dirty_workspace_on_another_stream(nq):
    kw = dict(n_head=4, n_kv=2, nq=nq, groups=[5, 9, 2], n_pre=[700, 64, 3], n_own=[i + 3 for i in range(16)], weigh=True)
    a = Case(7, **kw)
    x = a.run()
    wp, wo = a.pk.weight.clone(), a.ok.weight.clone()
    b = Case(7, **kw)
    need = wh.lib().wh_prefix_attention_workspace(16, nq, 4, 2, 3, 700, 18, 7)
    ws = torch.full((need // 4,), float("nan"), device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y = b.run(workspace=ws, stream=s)
    s.synchronize()
    assert torch.equal(x, y) and torch.equal(wp, b.pk.weight) and torch.equal(wo, b.ok.weight)


def test_recorded_and_replayed():
    c = Case(8, n_head=4, n_kv=4, nq=1, groups=[3, 2], n_pre=[300, 90], n_own=[5, 6, 7, 8, 9], weigh=True)
    ref = c.run()
    once = c.pk.weight.cpu().numpy() - c.w0["pre"]
    pk, ok, q = c.keys("pre"), c.keys("own"), _dev(c.q)
    start = torch.from_numpy(c.start).cuda()
    out = torch.zeros_like(ref)
    ws = torch.empty(wh.lib().wh_prefix_attention_workspace(5, 1, 4, 4, 2, 300, 9, 7), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        wh.wh_prefix_attention(q, 4, prefix=pk, own=ok, group_start=start, out=out, workspace=ws)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and wh.wh_status() == wh.WH_OK
    three = pk.weight.cpu().numpy() - c.w0["pre"]
    assert np.allclose(three, 3 * once, rtol=1e-5, atol=1e-6)       # each replay adds its weights
    # the counts are read at every replay
    ok.n_keys.zero_()
    pk.n_keys.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.all(out == 0)


def test_counts_and_groups_out_of_range_are_cut_and_reported():
    c = Case(9, n_head=2, n_kv=2, nq=1, groups=[2, 3], n_pre=[40, 40], n_own=[8] * 5)
    ref = c.run()
    pk, ok, q = c.keys("pre"), c.keys("own"), _dev(c.q)
    start = torch.from_numpy(c.start).cuda()
    call = lambda: wh.wh_prefix_attention(q, 2, prefix=pk, own=ok, group_start=start)  # noqa: E731
    pk.n_keys.copy_(torch.tensor([40, 41]))
    assert torch.equal(call(), ref) and wh.wh_status() == wh.WH_EBOUNDS
    pk.n_keys.fill_(40)
    ok.n_keys[4] = 9
    assert torch.equal(call(), ref) and wh.wh_status() == wh.WH_EBOUNDS
    ok.n_keys[4] = 8
    ok.n_keys[0] = -3
    none = call()
    assert wh.wh_status() == wh.WH_EBOUNDS and torch.equal(none[1:], ref[1:])
    ok.n_keys[0] = 8
    start.copy_(torch.tensor([0, 2, 6]))                     # one past the batch
    assert torch.equal(call(), ref) and wh.wh_status() == wh.WH_EBOUNDS
    start.copy_(torch.tensor([-1, 2, 5]))
    assert torch.equal(call(), ref) and wh.wh_status() == wh.WH_EBOUNDS
    start.copy_(torch.tensor([0, 5, 2]))                     # descending: reported, nothing out of range touched
    call()
    assert wh.wh_status() == wh.WH_EBOUNDS
    start.copy_(torch.from_numpy(c.start))
    assert torch.equal(call(), ref) and wh.wh_status() == wh.WH_OK


def test_agrees_with_the_one_query_attention():
    rng = np.random.default_rng(10)
    H, d, n = 20, 1280, 1500
    kv, q = _dev(_bf(rng, 2, n, 2 * d)), _dev(_bf(rng, 2, d))
    a = wh.wh_decode_attention(q, kv, kv[..., d:], 2 * d, 2 * d * n, n, H).float()
    b = wh.wh_prefix_attention(q, H, prefix=wh.Keys(kv[..., :d], kv[..., d:])).float()
    assert torch.all((a - b).abs() <= 2.0 ** -7 * a.abs() + 2.0 ** -10 * kv.abs().max())


@pytest.mark.parametrize("beams", [3, 20])
def test_huge_scores(beams):
    """Scores of 1e12: the softmax picks the largest.  Every query is a multiple of one key, whose score is the
    largest by far more than fp32 rounding (64 2^-24 of the sum's magnitude)."""
    rng = np.random.default_rng(16)
    n = 300
    k = _bf(rng, n, 128) * np.float32(2.0 ** 20)
    v = _bf(rng, n, 128)
    pick = rng.integers(0, n, size=(beams, 2))
    q = np.concatenate([k[pick[:, h], 64 * h:64 * h + 64] for h in range(2)], axis=1)
    own = [(k[:5], v[:5])] * beams
    weight = torch.zeros(1, 2, n, device="cuda")
    keys = wh.Keys(_dev(k[None]), _dev(v[None]), None, weight)
    mine = wh.Keys(_dev(np.stack([a for a, _ in own])), _dev(np.stack([b for _, b in own])))
    for extra in (None, mine):
        out = wh.wh_prefix_attention(_dev(q), 2, prefix=keys, own=extra).float().cpu().numpy()
        for b in range(beams):
            for h in range(2):
                cols = slice(64 * h, 64 * h + 64)
                assert np.array_equal(out[b, cols], v[pick[b, h], cols])
    assert abs(float(weight.sum()) - 2 * 2 * beams) < 2.01 * beams      # the picked key may also be an own one
    for h in range(2):
        seen = set(pick[:, h])
        assert all(weight[0, h, t] == 0 for t in range(n) if t not in seen)


def test_empty_batch():
    k = torch.zeros(0, 9, 128, dtype=torch.bfloat16, device="cuda")
    out = wh.wh_prefix_attention(torch.zeros(0, 128, dtype=torch.bfloat16, device="cuda"), 2, own=wh.Keys(k, k))
    assert out.shape == (0, 128)


def test_two_calls_at_once():
    """Two streams, each its own calls over shared inputs: nothing in the library is shared between them."""
    kw = dict(n_head=4, n_kv=2, nq=2, n_own=[40 + i for i in range(24)])
    cases = [Case(17, groups=[8, 8, 8], n_pre=[900, 1000, 1100], **kw), Case(18, groups=[20, 4], n_pre=[3000, 50], **kw)]
    refs = [c.run() for c in cases]
    args = [dict(q=_dev(c.q), n_head=4, prefix=c.pk, own=c.ok, n_kv_head=2, n_query=2,
                 group_start=torch.from_numpy(c.start).cuda()) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(wh.wh_prefix_attention(**args[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(x, refs[i]) for i in range(2) for x in outs[i]) and wh.wh_status() == wh.WH_OK


def test_refusals_of_the_binding():
    c = Case(11, n_head=2, n_kv=2, nq=1, groups=[2, 2], n_pre=[8, 8], weigh=True)
    c.run()
    q, start = _dev(c.q), torch.from_numpy(c.start).cuda()
    bad = [dict(q=q.float()), dict(q=q[:3]), dict(n_kv_head=4), dict(n_query=3), dict(group_start=start.long()),
           dict(group_start=start[:2]), dict(out=torch.empty(4, 64, dtype=torch.bfloat16, device="cuda")),
           dict(workspace=torch.empty(16, device="cuda")), dict(prefix=None), dict(n_head=3), dict(q=q.cpu())]
    for kw in bad:
        args = dict(q=q, n_head=2, prefix=c.pk)
        args.update(kw)
        with pytest.raises(wh.WhError):
            wh.wh_prefix_attention(**args)
    assert wh.wh_status() == wh.WH_OK
