"""Cases of wh_prefix_attention by the path that their sizes take, shared by the CPU test that pins the paths and the GPU
test of their results.  `plan` holds what wh_prefix_attention_plan has to say."""
from whisper_audio_encoder_gb300 import wh


def _counts(sets, cap):
    """Unequal prefixes; the first one whole, and borders of the steps of 128 keys among the rest."""
    odd = [cap, 0, 1, 127, 128, 129, 255, 256, 257, cap - 1]
    return [min(cap, odd[i]) if i < len(odd) else 1 + (cap * (7 * i + 3)) // (7 * sets + 5) for i in range(sets)]


def _case(plan, heads, groups, cap, kv=None, nq=1, n_pre=None, own=None, outside=0, table=True, weigh=False, layout="apart"):
    """groups: sequences of every set; own: own keys' capacity (the counts go through 0 .. own) or None; outside: sequences
    before the first group, and as many behind the last."""
    batch = sum(groups) + 2 * outside
    starts = [outside]
    for g in groups:
        starts.append(starts[-1] + g)
    return dict(plan=plan, H=heads, KV=kv or heads, nq=nq, starts=starts, batch=batch, cap=cap,
                n_pre=n_pre or _counts(len(groups), cap), cap_own=own or 0,
                n_own=None if own is None else [(5 * b) % (own + 1) for b in range(batch)], table=table, weigh=weigh, layout=layout)


def _tc(rows, ranges, cluster, merge=0, **kw):
    return dict(prefix_rows=rows, prefix_ranges=ranges, prefix_cluster=cluster, merge=merge, **kw)


PATHS = {
    # one range a block, which finishes its rows
    "32 rows, one range": _case(_tc(32, 1, 1), 12, [20] * 20, 700, table=False),
    "64 rows, one range, weights": _case(_tc(64, 1, 1), 12, [40] * 12, 700, table=False, weigh=True),
    "128 rows, one range": _case(_tc(128, 1, 1), 8, [100] * 8, 700, table=False),
    "128 rows, one range, grouped heads, several queries": _case(_tc(128, 1, 1), 8, [9] * 24, 700, kv=4, nq=5, table=False, weigh=True),
    "64 rows, one range, groups of all sizes": _case(_tc(64, 1, 1), 12, [i * 7 % 81 for i in range(14)], 700),
    "32 rows, one range, sequences outside": _case(_tc(32, 1, 1), 12, [20, 0, 31, 33] * 5, 700, outside=3, weigh=True),
    "128 rows, one range, sequences outside": _case(_tc(128, 1, 1), 8, [100, 129, 0, 101] * 2 + [128], 700, outside=70),
    # two ranges, joined in clusters
    "32 rows, clusters": _case(_tc(32, 2, 2), 9, [24] * 12, 1500, table=False, weigh=True),
    "64 rows, clusters, sequences outside": _case(_tc(64, 2, 2), 8, [40, 65, 3, 0, 64, 41, 60, 50], 1500, outside=2),
    "128 rows, clusters": _case(_tc(128, 2, 2), 8, [90, 128, 129, 10, 97], 1500, weigh=True),
    # more ranges, joined by a kernel
    "32 rows, merge": _case(_tc(32, 32, 0, 1), 8, [32], 20000, table=False),
    "32 rows, merge, few ranges": _case(_tc(32, 6, 0, 1), 8, [30, 20, 27, 9], 6000, weigh=True),
    "64 rows, merge, sequences outside": _case(_tc(64, 6, 0, 1), 8, [60, 33, 50, 45], 6000, outside=1),
    "128 rows, merge, many ranges": _case(_tc(128, 64, 0, 1), 2, [100], 40400, table=False),
    # beside own keys
    "64 rows, own keys": _case(_tc(64, 1, 0), 2, [40] * 3, 200, own=5, table=False),
    "64 rows, own keys, [K | V] rows": _case(_tc(64, 1, 0), 2, [40] * 3, 200, own=5, table=False, layout="kv"),
    "64 rows, own keys, one set for all groups": _case(_tc(64, 1, 0), 2, [40] * 3, 200, n_pre=[200] * 3, own=5, table=False, layout="one"),
    "64 rows, own keys, sets beside each other": _case(_tc(64, 1, 0), 2, [40] * 3, 200, own=5, table=False, layout="beside"),
    "64 rows, own keys, odd set stride": _case(_tc(64, 1, 0), 2, [40] * 3, 200, own=5, table=False, layout="odd"),
    "128 rows, own keys, ranges": _case(_tc(128, 16, 0), 2, [130, 70], 6000, own=9, weigh=True),
    "128 rows, own keys in ranges": _case(_tc(128, 8, 0, 1), 1, [33, 34], 3000, nq=3, own=1300, weigh=True),
    # 32 rows without own keys in the layouts of tensor maps
    "32 rows, [K | V] rows": _case(_tc(32, 8, 0, 1), 8, [20] * 4, 6000, table=False, layout="kv"),
    "32 rows, one set for all groups": _case(_tc(32, 8, 0, 1), 8, [20] * 4, 6000, n_pre=[6000] * 4, table=False, layout="one"),
    "32 rows, sets beside each other": _case(_tc(32, 8, 0, 1), 8, [20] * 4, 6000, table=False, layout="beside"),
    # few rows, for comparison
    "16 rows, one range": _case(dict(prefix_rows=16, prefix_ranges=1, prefix_cluster=1), 20, [5] * 20, 300, table=False),
    "16 rows, clusters": _case(dict(prefix_rows=16, prefix_ranges=16, prefix_cluster=16), 2, [5], 30000, table=False),
    "16 rows, merge": _case(dict(prefix_rows=16, prefix_cluster=0, merge=1), 1, [5], 60000, table=False),
}


def plan_of(c):
    needs = (wh.WH_GROUP_TABLE if c["table"] else 0) + ((wh.WH_PREFIX_WEIGHT + (wh.WH_OWN_WEIGHT if c["cap_own"] else 0)) if c["weigh"] else 0)
    return wh.wh_prefix_attention_plan(c["batch"], c["nq"], c["H"], c["KV"], len(c["starts"]) - 1, c["cap"], c["cap_own"], needs)
