"""The serving operators at operands and sizes where 16-bit parts, split sums
or 32-bit counts could fail, against plain 64-bit forms."""
import math

import numpy as np
import pytest
import torch

import activation_sparse_decode_rank_gb300 as pi
from test_gpu_serve import DEV, TD, U, Cache, i32, new_status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    pi.build()


# ------------------------------------------------------------------ page numbers
@pytest.mark.parametrize("P", [16, 8, 5])
@pytest.mark.parametrize("bad", [-2, -3, -2 ** 31, 2 ** 31 - 1])
@pytest.mark.parametrize("append", [False, True])
def test_attention_reports_every_bad_page_number(P, bad, append):
    # a page in the middle, the first one, the new token's
    for s, j in ((0, 40 // P), (1, 0), (2, 44 // P)):
        c = Cache("f16", 8, 2, 64, P, [100, 60, 45], append=append)
        tab = c.np_table.copy()
        tab[s, j] = bad
        y, lse = c.run(table=i32(tab))
        c.check(y, lse, {s: set(range(j * P, j * P + P))})
        assert int(c.status[0]) == pi.PI_ERR_INDEX
        if append and s == 2:  # not stored anywhere
            pg = int(c.np_table[s, j])
            assert torch.isnan(c.pool[0, pg, :, :, 44 % P]).all()


# ------------------------------------------------------------------ large scores
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("qscale", [1e7, 1e8, 1e12, 1e20])
@pytest.mark.parametrize("shape,lens", [((8, 2, 128, 16), [1, 40, 300, 2]), ((4, 1, 64, 5), [70, 900]),
                                        ((16, 2, 256, 8), [7001, 33])])
def test_attention_of_large_finite_scores(dtype, sign, qscale, shape, lens):
    # Scores are off by da = scale |q|.|k| (2^-21 + D u); where the largest lies
    # more than 2 da + 40 above the second, the others weigh under e^-40 2^13
    # together, and y is the largest one's value (kept to 22 bits), lse its score.
    c = Cache(dtype, *shape, lens, qscale=qscale)
    c.scale *= sign
    y, lse = c.run()
    torch.cuda.synchronize()
    assert torch.isfinite(y).all() and torch.isfinite(lse[:-1]).all()
    y, lse = y.double().cpu().numpy(), lse.double().cpu().numpy()
    seen, G = 0, c.heads // c.kv
    for s, n in enumerate(lens):
        for h in range(c.heads):
            q, k = c.q[s, h].astype(np.float64), c.rows[0, s, :n, h // G]
            a = c.scale * (k @ q)
            da = abs(c.scale) * (np.abs(k) @ np.abs(q)).max() * (2.0 ** -21 + c.D * U)
            top = int(a.argmax())
            if n > 1 and a[top] - np.partition(a, -2)[-2] <= 2 * da + 40:
                continue
            seen += 1
            want = c.rows[1, s, top, h // G]
            assert np.abs(y[s, h] - want).max() <= 2.0 ** -20 * np.abs(want).max(), (s, h)
            assert abs(lse[s, h] - a[top]) <= da + 8 * U * abs(a[top]), (s, h)
    assert seen >= len(lens) * c.heads // 2
