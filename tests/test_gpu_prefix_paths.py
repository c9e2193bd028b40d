"""wh_prefix_attention on every path of its kernels (the cases of prefix_paths, pinned to their paths on the CPU by
test_prefix_plan), against the oracle in 64 bits.

Queries and keys are small whole numbers, so the scores are exact in fp32.  Tolerance, counted from the roundings:
- out: test_gpu_prefix_precision's (bf16 output, weights of 16 bits, sums), with the weights of up to 24 partial results
  or rescalings more, each off by 2^-22 of what is added: 2^-17 sum p |v|;
- weights: the exponential, the sum of n weights and its inverse, 2^-20 + n 2^-24, and the sum over the queries, 2^-24
  for each of them, relative; half a step of the accumulator before and after.
"""
import numpy as np
import pytest
import torch

from oracle import whisper_ref as R
from prefix_paths import PATHS
from whisper_audio_encoder_gb300 import build, synth, wh

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    build.build()
    wh.lib()


def _dev(a, dtype=torch.bfloat16):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()


def out_tol(ref, spread, n):
    return (2.0 ** -8 + n * 2.0 ** -24) * np.abs(ref) + (2.0 ** -16 + 2.0 ** -17 + 2.0 ** -20 + (n // 16 + 1) * 2.0 ** -18) * spread


def _whole(rng, low, high, *shape):
    return rng.integers(low, high + 1, shape).astype(np.float32)


def _buffers(sets, cap, d, layout):
    """Two [sets][cap][d] views full of NaN, laid out as the case says."""
    full = lambda *shape: torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")  # noqa: E731
    if layout == "kv":
        x = full(sets, cap, 2 * d)
        return x[..., :d], x[..., d:]
    if layout == "one":
        return tuple(full(1, cap, d).expand(sets, cap, d) for _ in range(2))
    if layout == "beside":
        return tuple(full(cap, sets, d).transpose(0, 1) for _ in range(2))
    if layout == "odd":
        return tuple(full(sets * (cap * d + 8)).as_strided((sets, cap, d), (cap * d + 8, d, 1)) for _ in range(2))
    return tuple(full(sets, cap, d) for _ in range(2))


class Run:
    def __init__(self, c, seed):
        rng = np.random.default_rng(seed)
        self.c, d = c, 64 * c["KV"]
        self.q = _whole(rng, -2, 2, c["batch"] * c["nq"], 64 * c["H"])
        one = c["layout"] == "one"
        make = lambda n: (_whole(rng, -2, 2, n, d), synth.bf16_round(rng.standard_normal((n, d)).astype(np.float32)))  # noqa: E731
        self.pre = [make(n) for n in c["n_pre"][:1]] * len(c["n_pre"]) if one else [make(n) for n in c["n_pre"]]
        self.own = None if c["n_own"] is None else [make(n) for n in c["n_own"]]
        self.w0 = {}

        def keys(what, sets, cap, layout):
            k, v = _buffers(len(sets), cap, d, layout)
            for i, (x, y) in enumerate(sets[:1] if layout == "one" else sets):
                k[i, :len(x)], v[i, :len(x)] = _dev(x), _dev(y)
            n = torch.tensor([len(x) for x, _ in sets], dtype=torch.int32, device="cuda")
            w = None
            if c["weigh"]:
                self.w0[what] = rng.random((len(sets), c["KV"], cap)).astype(np.float32) * 50
                w = _dev(self.w0[what], torch.float32)
            return wh.Keys(k, v, n, w)

        self.pk = keys("pre", self.pre, c["cap"], c["layout"])
        self.ok = None if self.own is None else keys("own", self.own, c["cap_own"], "apart")

    def call(self, table=None, **kw):
        c = self.c
        start = _dev(np.array(c["starts"], np.int32), torch.int32) if (c["table"] if table is None else table) else None
        out = wh.wh_prefix_attention(_dev(self.q), c["H"], prefix=self.pk, own=self.ok, n_kv_head=c["KV"], group_start=start,
                                     n_query=c["nq"], **kw)
        assert wh.wh_status() == wh.WH_OK
        return out

    def check(self, out):
        c = self.c
        group = [None] * c["batch"]
        for g in range(len(c["starts"]) - 1):
            group[c["starts"][g]:c["starts"][g + 1]] = [g] * (c["starts"][g + 1] - c["starts"][g])
        ref, spread, wp, wo = R.prefix_attention(self.q, c["nq"], c["H"], c["KV"], self.pre, group, self.own or [None] * c["batch"])
        n = np.array([(c["n_pre"][g] if g is not None else 0) + (c["n_own"][b] if c["n_own"] else 0) for b, g in enumerate(group)])
        over = np.abs(out.float().cpu().numpy() - ref) - out_tol(ref, spread, np.repeat(n, c["nq"])[:, None])
        assert np.all(over <= 0), f"{(~(over <= 0)).sum()} of {over.size} outside, by {np.nanmax(over):.3e}"
        for what, sets, keys in (("pre", wp, self.pk), ("own", wo, self.ok)):
            if what not in self.w0:
                continue
            got, w0 = keys.weight.cpu().numpy().astype(np.float64), self.w0[what]
            for i, w in enumerate(sets):
                m = w.shape[1]
                rows = max((b - a for a, b in zip(c["starts"], c["starts"][1:])), default=1) * c["nq"] * (c["H"] // c["KV"])
                tol = (2.0 ** -20 + (n.max() + rows) * 2.0 ** -24) * w + 2.0 ** -23 * (w0[i, :, :m] + w) + 1e-30
                assert np.all(np.abs(got[i, :, :m] - w0[i, :, :m] - w) <= tol), f"{what} {i}"
                assert np.array_equal(got[i, :, m:], w0[i, :, m:])


@pytest.mark.parametrize("name", PATHS)
def test_paths(name):
    run = Run(PATHS[name], seed=len(name))
    run.check(run.call())


@pytest.mark.parametrize("name", [n for n in PATHS if not PATHS[n]["table"] and PATHS[n]["layout"] == "apart"])
def test_equal_groups_given_as_a_table(name):
    run = Run(PATHS[name], seed=2)
    run.check(run.call(table=True))


@pytest.mark.parametrize("name", ["64 rows, one range, weights", "32 rows, clusters", "32 rows, merge", "128 rows, own keys, ranges"])
def test_same_bits_again(name):
    a, b = Run(PATHS[name], seed=3), Run(PATHS[name], seed=3)
    x, y = a.call(), b.call()
    assert torch.equal(x, y) and all(torch.equal(p.weight, q.weight) for p, q in ((a.pk, b.pk), (a.ok, b.ok)) if p is not None and p.weight is not None)


@pytest.mark.parametrize("groups", [[20] * 20, [40] * 12, [100] * 8], ids=["32 rows", "64 rows", "128 rows"])
@pytest.mark.parametrize("step", [7, -7, 3])
def test_maxima_that_grow_from_step_to_step(groups, step):
    """Scores that rise (or fall, or rise slowly) by 7 from one step of 128 keys to the next, for some queries, and the other
    way round for the others: rising ones are rescaled at every step."""
    rng = np.random.default_rng(4)
    H, cap = (8 if groups[0] == 100 else 12), 700
    sets, B = len(groups), sum(groups)
    plan = wh.wh_prefix_attention_plan(B, 1, H, n_prefix=sets, max_prefix=cap)
    assert (plan["prefix_rows"], plan["prefix_ranges"]) == ({20: 32, 40: 64, 100: 128}[groups[0]], 1)
    q = _whole(rng, -1, 1, B, H, 64)
    q[:, :, :8] = rng.choice(np.float32([-1, 1]), (B, H, 1))                # the way that the query looks
    k, v = _whole(rng, -1, 1, sets, cap, H, 64), synth.bf16_round(rng.standard_normal((sets, cap, H * 64)).astype(np.float32))
    k[..., :8] = (step * (np.arange(cap) // 128)).astype(np.float32)[None, :, None, None]
    q, k = q.reshape(B, -1), k.reshape(sets, cap, -1)
    weight = torch.zeros(sets, H, cap, device="cuda")
    out = wh.wh_prefix_attention(_dev(q), H, prefix=wh.Keys(_dev(k), _dev(v), None, weight)).float().cpu().numpy()
    ref, spread, wp, _ = R.prefix_attention(q, 1, H, H, list(zip(k, v)), [b // groups[0] for b in range(B)], [None] * B)
    assert np.all(np.abs(out - ref) <= out_tol(ref, spread, cap))
    for i, w in enumerate(wp):
        assert np.all(np.abs(weight[i].cpu().numpy() - w) <= (2.0 ** -18 + (cap + groups[0]) * 2.0 ** -24) * w + 1e-30)
    assert wh.wh_status() == wh.WH_OK


def test_offsets_past_32_bits():
    rng = np.random.default_rng(6)
    n, stride, beams = 130, 1 << 25, 40                  # the last key starts 4.3e9 elements in
    if torch.cuda.mem_get_info()[0] < 3 * n * stride * 2:
        pytest.skip("needs 18 GB of device memory")
    k, v, q = _whole(rng, -2, 2, n, 128), synth.bf16_round(rng.standard_normal((n, 128)).astype(np.float32)), _whole(rng, -2, 2, beams, 128)
    big = torch.empty(n * stride, dtype=torch.bfloat16, device="cuda").as_strided((1, n, 256), (0, stride, 1))
    big[0, :, :128], big[0, :, 128:] = _dev(k), _dev(v)
    mine = [(_whole(rng, -2, 2, 3, 128), synth.bf16_round(rng.standard_normal((3, 128)).astype(np.float32))) for _ in range(beams)]
    own = wh.Keys(_dev(np.stack([a for a, _ in mine])), _dev(np.stack([b for _, b in mine])))
    assert wh.wh_prefix_attention_plan(beams, 1, 2, n_prefix=1, max_prefix=n, max_own=3)["prefix_rows"] == 64
    out = wh.wh_prefix_attention(_dev(q), 2, prefix=wh.Keys(big[..., :128], big[..., 128:]), own=own).float().cpu().numpy()
    ref, spread, _, _ = R.prefix_attention(q, 1, 2, 2, [(k, v)], [0] * beams, mine)
    assert np.all(np.abs(out - ref) <= out_tol(ref, spread, n + 3)) and wh.wh_status() == wh.WH_OK


@pytest.mark.parametrize("beams", [20, 40, 100])
def test_huge_scores(beams):
    """Scores of 1e12: the softmax picks the largest.  Every query is a multiple of one key, whose score is the
    largest by far more than fp32 rounding (64 2^-24 of the sum's magnitude)."""
    rng = np.random.default_rng(16)
    n, cap, H = 300, 40000, 4
    assert wh.wh_prefix_attention_plan(beams, 1, H, n_prefix=1, max_prefix=cap)["prefix_rows"] == {20: 32, 40: 64, 100: 128}[beams]
    k = synth.bf16_round(rng.standard_normal((n, 64 * H)).astype(np.float32)) * np.float32(2.0 ** 20)
    v = synth.bf16_round(rng.standard_normal((n, 64 * H)).astype(np.float32))
    pick = rng.integers(0, n, size=(beams, H))
    q = np.concatenate([k[pick[:, h], 64 * h:64 * h + 64] for h in range(H)], axis=1)
    kd, vd = torch.full((2, 1, cap, 64 * H), float("nan"), dtype=torch.bfloat16, device="cuda")
    kd[0, :n], vd[0, :n] = _dev(k), _dev(v)
    weight = torch.zeros(1, H, cap, device="cuda")
    keys = wh.Keys(kd, vd, torch.tensor([n], dtype=torch.int32, device="cuda"), weight)
    out = wh.wh_prefix_attention(_dev(q), H, prefix=keys).float().cpu().numpy()
    for h in range(H):
        cols = slice(64 * h, 64 * h + 64)
        assert np.array_equal(out[:, cols], v[pick[:, h], cols])
        count = np.bincount(pick[:, h], minlength=cap)
        got = weight[0, h].cpu().numpy()
        # (the second pass rounds the same score in another order: off by 64 2^-24 of 1e13 or so, and cut to 1)
        assert np.all(got[count == 0] == 0) and np.all(got <= count)
    assert wh.wh_status() == wh.WH_OK


@pytest.mark.parametrize("sets", [3, 40])
@pytest.mark.parametrize("rows", [16, 64])
@pytest.mark.parametrize("bad", [-1, 701])
def test_counts_of_groups_without_sequences_are_reported(sets, rows, bad):
    H, cap = 2, 700
    sizes = [0] + [1 if rows == 16 else 80 if sets > 3 else 150] * (sets - 2) + [0]
    B = sum(sizes)
    k = torch.zeros(sets, cap, 64 * H, dtype=torch.bfloat16, device="cuda")
    own = wh.Keys(k[:1, :4].expand(B, 4, 64 * H).contiguous(), k[:1, :4].expand(B, 4, 64 * H).contiguous())
    plan = wh.wh_prefix_attention_plan(B, 1, H, n_prefix=sets, max_prefix=cap, max_own=4, needs=wh.WH_GROUP_TABLE)
    assert (plan["prefix_rows"] == 16) == (rows == 16)
    starts = torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32, device="cuda")
    n = torch.full((sets,), cap, dtype=torch.int32, device="cuda")
    q = torch.zeros(B, 64 * H, dtype=torch.bfloat16, device="cuda")
    call = lambda: wh.wh_prefix_attention(q, H, prefix=wh.Keys(k, k, n), own=own, group_start=starts)  # noqa: E731
    call()
    assert wh.wh_status() == wh.WH_OK
    for g in (0, sets - 1):
        n.fill_(cap)
        n[g] = bad
        call()
        assert wh.wh_status() == wh.WH_EBOUNDS, g
        assert wh.wh_status() == wh.WH_OK


@pytest.mark.parametrize("cap", [33, 64, 65, 80, 96, 97])
@pytest.mark.parametrize("nq", [1, 2])
def test_short_own_caches_of_few_sequences(cap, nq):
    rng = np.random.default_rng(cap)
    B, H = 3, 6
    counts = [cap, cap // 2, 0]
    own = [(_whole(rng, -2, 2, n, 64 * H), synth.bf16_round(rng.standard_normal((n, 64 * H)).astype(np.float32))) for n in counts]
    q = _whole(rng, -2, 2, B * nq, 64 * H)
    k, v = _buffers(B, cap, 64 * H, "apart")
    for i, (x, y) in enumerate(own):
        k[i, :len(x)], v[i, :len(x)] = _dev(x), _dev(y)
    weight = torch.zeros(B, H, cap, device="cuda")
    wh.lib().wh_launch_count()                         # (counts from here on)
    out = wh.wh_prefix_attention(_dev(q), H, n_query=nq, own=wh.Keys(k, v, torch.tensor(counts, dtype=torch.int32, device="cuda"), weight))
    launches = wh.lib().wh_launch_count()
    assert launches == wh.wh_prefix_attention_plan(B, nq, H, max_own=cap, needs=wh.WH_OWN_WEIGHT)["launches"]
    ref, spread, _, w = R.prefix_attention(q, nq, H, H, [], [None] * B, own)
    assert np.all(np.abs(out.float().cpu().numpy() - ref) <= out_tol(ref, spread, cap))
    for i, x in enumerate(w):
        assert np.all(np.abs(weight[i, :, :counts[i]].cpu().numpy() - x) <= (2.0 ** -20 + (cap + nq) * 2.0 ** -24) * x + 1e-30)
    assert wh.wh_status() == wh.WH_OK
