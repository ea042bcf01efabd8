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
