"""The calls around the 4-bit cache at the ends of what they accept, against the float64 oracle, with the tolerances of the
other tests unless one is derived here.
"""

import pytest
import torch

import helpers

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    helpers.ensure_built()

import context_blockwise_attention_gb300 as cpa  # noqa: E402
import test_gpu_kv4 as kv4  # noqa: E402
from context_blockwise_attention_gb300 import PosMap  # noqa: E402
from test_gpu_kv4 import BF16, DEV, F32, Pool, _i32  # noqa: E402


@pytest.mark.parametrize("d,page,hq,dtype", [(64, 16, 8, BF16), (64, 64, 24, F32), (128, 32, 8, F32), (128, 128, 40, BF16)])
def test_rows_whose_query_is_not_finite_give_no_weight(d, page, hq, dtype):
    """Their LSE, the attention's own answer, is not finite, so they give nothing; the rows beside them give what they give
    without them."""
    rows, held = [3, 1, 2], [200, 70, 33]
    pool = Pool(3, held, page, 2, d, 201)
    pool.fill(held, 202)
    q = torch.randn((6, hq, d), generator=torch.Generator().manual_seed(203)).to(dtype)
    first = [m - n for n, m in zip(rows, held)]
    clean = cpa.kv4_cache_attn(q.to(DEV), pool.device(), _i32([0, 3, 4, 6]), _i32(held), _i32(pool.table), q_first=_i32(first))[1]
    spoilt = torch.zeros((6, hq), dtype=torch.bool)
    for i, h, e, x in ((0, 0, 3, "nan"), (1, hq - 1, 0, "inf"), (1, 1, d - 1, "-inf"), (2, hq // 2, 17, "nan"), (4, 2, 40, "inf"),
                       (4, hq // 2, 40, "nan")):
        q[i, h, e] = float(x)
        spoilt[i, h] = True
    q[5, 3] = float("inf")  # all of a row
    spoilt[5, 3] = True
    lse = cpa.kv4_cache_attn(q.to(DEV), pool.device(), _i32([0, 3, 4, 6]), _i32(held), _i32(pool.table), q_first=_i32(first))[1]
    assert torch.equal(lse.isfinite().cpu(), ~spoilt) and torch.equal(lse.cpu()[~spoilt], clean.cpu()[~spoilt])
    kv4._check_weigh(pool, q, rows, held, first, PosMap(0, 1), None, 1.0, 204)
    kv4._check_weigh(pool, q, rows, held, first, PosMap(0, 1), [190, 0, 33], 0.5, 205)
