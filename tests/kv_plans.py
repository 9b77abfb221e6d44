"""Calls of tq_kv_attn that between them take every launch plan, with the
workspace each one needs: it shows the plan (which kernel, how many workgroups
or pieces), so a threshold that moves a call to another plan shows in its test."""
import numpy as np


def _ragged(n, most, rows=1, empty=0, seed=1):
    """n sequences of `rows` rows, lengths up to `most` with the ones around a
    page, a whole unit and nothing; every `empty`-th has no rows."""
    rng = np.random.default_rng(seed)
    kv = [most, 0, 1, 64, 65, 1024, 1025, most - 1] + rng.integers(1, most, n).tolist()
    return [(0 if empty and s % empty == 3 else rows, min(t, most)) for s, t in enumerate(kv[:n])]


# (query heads, KV heads, head_dim, [(rows, kv_len)...], window, sinks, max_kv_len, workspace bytes)
PLANS = {
    # tiles of 16 rows, shares of all pages that run over the units' borders
    "shares": (16, 8, 128, _ragged(40, 3000), 0, 0, 3000, 4260864),
    "shares_64": (16, 8, 64, _ragged(40, 3000, seed=2), 0, 0, 3000, 2163712),
    "shares_window": (16, 8, 64, _ragged(40, 3000, seed=3), 700, 70, 3000, 2163712),
    # ... of more sequences than a wave has lanes, some without rows
    "shares_many": (8, 4, 64, _ragged(100, 3000, empty=10, seed=4), 0, 0, 3000, 2163712),
    "shares_many_window": (8, 4, 128, _ragged(100, 2500, empty=7, seed=5), 1000, 3, 2500, 4260864),
    # ... tiles of 32 rows
    "shares_rows": (16, 4, 128, _ragged(70, 2500, rows=5, seed=6), 0, 0, 2500, 8520704),
    "shares_rows_64": (16, 4, 64, _ragged(70, 2500, rows=5, empty=9, seed=7), 900, 65, 2500, 4326400),
    # one piece a workgroup
    "pieces": (16, 2, 128, [(1, 5000), (1, 70), (0, 9), (1, 3000)], 0, 0, 5000, 2663040),
    # whole units, four waves a workgroup
    "whole_4": (16, 8, 128, _ragged(40, 1000, seed=8), 0, 0, 1000, 0),
    "whole_4_64": (16, 8, 64, _ragged(40, 1000, seed=9), 300, 5, 1000, 0),
    # 128 rows: full rounds of whole tiles, the rest of a last round in three pieces
    "rest_cut": (40, 8, 128, [(1025, 1400), (1025, 1100)], 0, 0, 1400, 28754496),
    "rest_cut_window": (40, 8, 64, [(1025, 1400), (1025, 1026)], 400, 70, 1400, 14598720),
    # ... one round of them on few pages, as many pieces as should take least: one, two, three
    "prompt_1": (64, 8, 128, [(256, 2000)], 0, 0, 2000, 0),
    "prompt_2": (64, 8, 128, [(180, 2000)], 0, 0, 2000, 12779904),
    "prompt_3": (32, 8, 128, [(300, 2000)], 0, 0, 2000, 15974720),
    "prompt_1_64": (24, 4, 64, [(300, 1000), (300, 700), (300, 300)], 0, 0, 1000, 0),
    "prompt_2_64": (64, 8, 64, [(256, 2000)], 500, 4, 2000, 9191968),
    "prompt_3_64": (32, 8, 64, [(300, 2000)], 0, 0, 2000, 8110400),
    # ... tiles half empty
    "half_empty": (40, 8, 128, [(13, 2000 - 31 * s) for s in range(30)], 0, 0, 2000, 47924640),
}
