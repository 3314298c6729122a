"""Rotated queries that leave between the rows of the projection they come from:
the same bits as into a buffer of their own, and nothing else of the rows written."""

import pytest
import torch

from test_gpu_fp4 import Fp4Case
from test_gpu_paged import B, BF16, F32, SETS, _geom  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("x_type", [BF16, F32])
@pytest.mark.parametrize("r", [64, 62])
def test_queries_between_the_rows_of_the_projection(B, r, x_type):
    g = _geom(B)
    g.full_rotary_dim = r
    case = Fp4Case(SETS["mixed"], seed=3, pad=3)
    rope = torch.zeros(max(case.ctx), r // 2, 2, device="cuda")
    B.spark_rope_table(g, B.SPARK_FULL, rope)
    x = torch.randn(case.n_tokens, 10240, generator=case.g, device="cuda").to(x_type)
    old, ws, pool = x.clone(), B.make_paged_workspace(g), B.PagePool(case.k, case.v)
    args = (g, x[:, :4096], x[:, 4096:5120], x[:, 5120:6144], B.SPARK_FULL, rope, pool, case.batch(B))
    own = old[:, 6144:].clone()
    B.spark_paged_rope_append(*args, own, ws)
    pages = case.k.clone(), case.v.clone()
    B.spark_paged_rope_append(*args, x[:, 6144:], ws)
    assert B.spark_attn_error_word(ws) == 0
    assert torch.equal(x[:, 6144:], own) and torch.equal(x[:, :6144], old[:, :6144])
    assert torch.equal(case.k, pages[0]) and torch.equal(case.v, pages[1])
