"""Limits of the serving operators' C entry points, without a GPU: what does not
fit a grid, a workspace or a count is refused before any CUDA call."""

from ctypes import byref

import pytest

from moe_persistent_cta_b200 import mk
from tests.test_ops import append_args, attention_args

MOST = 2 ** 31 - 1


@pytest.mark.parametrize("src", [mk.MK_FP32, mk.MK_BF16, mk.MK_FP16])
@pytest.mark.parametrize("hd", [64, 128])
def test_append_grid_fits(src, hd):
    # rows of stride 0 are allowed, so that memory does not limit their number
    kw = dict(n_rows=MOST, head_dim=hd, rotary_dim=hd, src_type=src, q_token_stride=0, k_token_stride=0,
              v_token_stride=0)
    for tokens, hq, hkv in ((MOST, 1024, 1024), (MOST // 8, 1000, 500), (MOST // 16, 1024, 1024)):
        a = append_args(n_tokens=tokens, n_q_heads=hq, n_kv_heads=hkv, **kw)
        assert mk.lib.mk_rope_append(byref(a), None) == mk.MK_ERR_CAPACITY, (tokens, hq, hkv)
