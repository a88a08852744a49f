"""NaN queries and keys: a row whose every score is NaN is NaN, not empty."""

import math

import pytest
import torch

import hierarchical_sparse_attention_build_b200 as R
from test_gpu_dense import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("L,n,lens", [(5, 1, None), (400, 3, [400, 2]), (9000, 1, [9000, 0]), (700, 150, None)])
@pytest.mark.parametrize("what", ["query", "keys"])
def test_rows_of_nan_scores(what, L, n, lens):
    c = Case(2, 2, 4, L, n, seed=n, lens=lens, garbage=0.0)
    view = R.View(causal=True, own_token=True)
    hit = torch.zeros(2, n, 8, dtype=torch.bool)
    if what == "query":
        c.qd[0, n // 2, 5, 7] = math.nan
        hit[0, n // 2, 5] = True
    else:  # every key of one KV head
        c.cache.k_tok[1, 1, :, 64] = math.nan
        for i in range(n):
            hit[1, i, 4:] = c.lens[1] - n + i + 1 > 0
    for fp32, kernel in ((True, R.DENSE_ROWS), (False, R.DENSE_ROWS), (False, R.DENSE_CHUNK)):
        view.kernel = kernel
        got = c.attend(fp32, view).cpu()
        assert torch.isnan(got[hit]).all() and torch.isfinite(got[~hit]).all()
    for view in (R.View(causal=True, own_token=True), R.View()):
        w = torch.zeros(2, 2, c.cap, device="cuda")
        R.accumulate_weights(c.p, c.cache, c.qd, w, c.ws, view)
        R.check_device_errors(c.ws)
        for b in range(2):
            for h in range(2):
                rows = hit[b, :, 4 * h:4 * h + 4]
                seen = c.lens[b] if not view.causal or not rows.any() else c.lens[b] - n + int(rows.any(1).nonzero().max()) + 1
                if view.causal or what == "query":
                    bad = bool(rows.any())
                else:
                    bad = (b, h) == (1, 1) and c.lens[b] > 0
                got = w[b, h, :max(seen, 0)]
                assert torch.isnan(got).all() if bad else torch.isfinite(got).all(), (b, h, view.causal)
