"""wh_prefix_attention where only the softmax weights' precision decides: queries and keys are small whole numbers, so
the scores (sums of 64 products below 2^8) are exact in fp32, and the values are taken off their weighted mean, so
that the output is far smaller than the terms that cancel in it.

Tolerance, counted from the roundings:
- out's bf16 rounding: 2^-8 |ref|; the fp32 sum of n weights: n 2^-24 |ref| (it divides the whole output);
- the weights as the sum of two bf16 values, each off by at most half a step: 2^-8 2^-8 = 2^-16 of sum p |v|;
- the exponentials and their arguments: below 2^-20;
- the sum over the keys: products of 16 keys and the running sum are added after alignment to the largest of them,
  17 terms off by at most 2^-23 each: below 2^-18 sum p |v| for every 16 keys, of the high and of the low parts
  (which are 2^-8 as large).
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


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(torch.bfloat16).cuda()


def _tol(ref, spread, n):
    return (2.0 ** -8 + n * 2.0 ** -24) * np.abs(ref) + (2.0 ** -16 + 2.0 ** -20 + (n // 16 + 1) * 2.0 ** -18) * spread


def _set(rng, n, H):
    """One query and n keys of whole numbers, and values whose weighted mean is (nearly) zero."""
    q = rng.integers(-2, 3, (1, 64 * H)).astype(np.float32)
    k = rng.integers(-2, 3, (n, 64 * H)).astype(np.float32)
    v = rng.standard_normal((n, 64 * H))
    mean = R.prefix_attention(q, 1, H, H, [(k, v)], [0], [None])[0][0]
    return q, k, synth.bf16_round((v - mean).astype(np.float32))


# capacities far above the counts send even these few keys through the kernel for many rows
@pytest.mark.parametrize("beams", [5, 16, 20, 32, 40, 64, 100, 300])
def test_prefix(beams):
    rng = np.random.default_rng(beams)
    H, cap, counts = 6, 8000, [3, 17, 64, 65, 100, 128, 129, 400]
    sets = [_set(rng, n, H) for n in counts]
    k, v = torch.full((2, len(counts), cap, 64 * H), float("nan"), dtype=torch.bfloat16, device="cuda")
    for i, (_, x, y) in enumerate(sets):
        k[i, :len(x)], v[i, :len(x)] = _dev(x), _dev(y)
    q = np.repeat(np.concatenate([s[0] for s in sets]), beams, axis=0)
    keys = wh.Keys(k, v, torch.tensor(counts, dtype=torch.int32, device="cuda"))
    out = wh.wh_prefix_attention(_dev(q), H, prefix=keys).float().cpu().numpy()
    assert wh.wh_status() == wh.WH_OK
    for i, (one, x, y) in enumerate(sets):
        ref, spread, _, _ = R.prefix_attention(one, 1, H, H, [(x, y)], [0], [None])
        over = np.abs(out[i * beams:(i + 1) * beams] - ref) / _tol(ref, spread, counts[i])
        assert over.max() <= 1.0, f"{counts[i]} keys: {over.max():.1f} times the tolerance"


@pytest.mark.parametrize("beams", [5, 40, 100])
def test_prefix_and_own_keys(beams):
    """The keys of one softmax, some of them in the prefix, the others in every sequence's own cache."""
    rng = np.random.default_rng(beams)
    H, n, n_own = 4, 90, 37
    q, k, v = _set(rng, n, H)
    dev = lambda x, b: _dev(x)[None].expand(b, -1, -1).contiguous()  # noqa: E731
    out = wh.wh_prefix_attention(_dev(np.repeat(q, beams, axis=0)), H, prefix=wh.Keys(dev(k[n_own:], 1), dev(v[n_own:], 1)),
                                 own=wh.Keys(dev(k[:n_own], beams), dev(v[:n_own], beams))).float().cpu().numpy()
    ref, spread, _, _ = R.prefix_attention(q, 1, H, H, [(k, v)], [0], [None])
    over = np.abs(out - ref) / _tol(ref, spread, n)
    assert over.max() <= 1.0, f"{over.max():.1f} times the tolerance"
    assert wh.wh_status() == wh.WH_OK


def test_own_keys():
    rng = np.random.default_rng(1)
    H, counts = 4, [2, 16, 33, 64, 100, 448]
    sets = [_set(rng, n, H) for n in counts]
    k, v = torch.full((2, len(counts), max(counts), 64 * H), float("nan"), dtype=torch.bfloat16, device="cuda")
    for i, (_, x, y) in enumerate(sets):
        k[i, :len(x)], v[i, :len(x)] = _dev(x), _dev(y)
    own = wh.Keys(k, v, torch.tensor(counts, dtype=torch.int32, device="cuda"))
    out = wh.wh_prefix_attention(_dev(np.concatenate([s[0] for s in sets])), H, own=own).float().cpu().numpy()
    for i, (one, x, y) in enumerate(sets):
        ref, spread, _, _ = R.prefix_attention(one, 1, H, H, [(x, y)], [0], [None])
        over = np.abs(out[i] - ref[0]) / _tol(ref[0], spread[0], counts[i])
        assert over.max() <= 1.0, f"{counts[i]} keys: {over.max():.1f} times the tolerance"
    assert wh.wh_status() == wh.WH_OK


@pytest.mark.parametrize("n_query, rep, n", [(4, 4, 100), (8, 2, 120), (1, 1, 120), (3, 5, 60)])
def test_weights_are_added_to_large_accumulators_once(n_query, rep, n):
    """The sum over the queries is made first: an accumulator of several hundred is rounded once, by half a step, however
    many rows there are.  Sums off by 2^-20 + (keys + rows) 2^-24 of themselves as they come in (exponential, sum, order)."""
    rng = np.random.default_rng(n)
    B, KV = 9, 2
    assert wh.wh_prefix_attention_plan(B, n_query, KV * rep, KV, max_own=n, needs=wh.WH_OWN_WEIGHT)["own_scores_kept"]
    q = rng.integers(-1, 2, (B * n_query, 64 * KV * rep)).astype(np.float32)
    own = [(rng.integers(-1, 2, (n, 64 * KV)).astype(np.float32), rng.standard_normal((n, 64 * KV))) for _ in range(B)]
    w0 = (512 + 500 * rng.random((B, KV, n))).astype(np.float32)
    weight = torch.from_numpy(w0).cuda()
    keys = wh.Keys(_dev(np.stack([k for k, _ in own])), _dev(np.stack([v for _, v in own])), None, weight)
    wh.wh_prefix_attention(_dev(q), KV * rep, own=keys, n_kv_head=KV, n_query=n_query)
    _, _, _, w = R.prefix_attention(q, n_query, KV * rep, KV, [], [None] * B, own)
    exact = w0 + np.stack(w)
    tol = 2.0 ** -24 * exact + (2.0 ** -20 + (n + n_query * rep) * 2.0 ** -24) * np.stack(w)
    over = np.abs(weight.cpu().numpy() - exact) / tol
    assert over.max() <= 1.0, f"{over.max():.1f} times the tolerance, {(over > 1).sum()} of {over.size}"
