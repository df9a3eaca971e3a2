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


def test_attention_workspace_goes_by_the_batch():
    size = lambda **kw: mk.lib.mk_prefix_attention_workspace(byref(attention_args(**kw)))  # noqa: E731
    # one entry of 4 query heads on 1 KV head: 320 shares of 2 x 4 rows, 4 x 4 whole ones; a row
    # is head_dim sums of 32 bits and two more numbers
    rows = 320 * 2 * 4 + 4 * 4
    assert rows * (128 * 4 + 8) <= size(batch=1, n_q_heads=4, n_kv_heads=1, head_dim=128) <= rows * (128 * 4 + 8) + 2048
    last = 0
    for b in (1, 2, 3, 8, 15, 16, 17, 32, 33, 100, 1000, 4096):
        now = size(batch=b, n_q_heads=16, n_kv_heads=4, head_dim=128)
        assert now > last, b
        last = now


def test_attention_selftest_refusals():
    call = mk.lib.mk_prefix_attention_selftest
    assert call(None, None) == mk.MK_ERR_INVALID
    assert call(byref(attention_args()), None) == mk.MK_ERR_INVALID                # no status word
    assert call(byref(attention_args(status=4096, batch=-1)), None) == mk.MK_ERR_INVALID
