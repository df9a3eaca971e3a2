"""The serving operators without a GPU: refusals of the C entry points (all of
them before any CUDA call) and of the Python functions, the frequency tables,
and the 64-bit definitions against independent restatements."""

import ctypes
import math
from ctypes import byref

import numpy as np
import pytest
import torch

from moe_persistent_cta_b200 import mk, ops
from tests import ops_oracle

P = 4096   # a stand-in device address; the calls below are refused before using it


def append_args(**kw):
    d = dict(device=0, n_tokens=4, n_rows=4, max_pages=2, n_pages=8, n_q_heads=4, n_kv_heads=2, head_dim=64,
             rotary_dim=64, interleaved=0, src_type=mk.MK_BF16, dst_type=mk.MK_BF16, magnitude=1.0,
             q=P, k=P, v=P, q_token_stride=256, q_head_stride=64, k_token_stride=128, k_head_stride=64,
             v_token_stride=128, v_head_stride=64, q_out=P, k_pool=P, v_pool=P, inv_freq=P, positions=P,
             seq=None, page_table=P, status=None)
    d.update(kw)
    a = mk.mk_rope_append_args()
    for n, v in d.items():
        setattr(a, n, v)
    return a


def attention_args(**kw):
    d = dict(device=0, batch=4, n_groups=1, max_pages=2, n_pages=8, n_q_heads=4, n_kv_heads=2, head_dim=64,
             type=mk.MK_BF16, scale=0.125, q=P, q_token_stride=256, k_pool=P, v_pool=P, page_table=P,
             positions=P, group_start=P, prefix_lens=P, out=P, lse=None, workspace=P,
             workspace_bytes=1 << 40, status=None)
    d.update(kw)
    a = mk.mk_prefix_attention_args()
    for n, v in d.items():
        setattr(a, n, v)
    return a


def sample_args(**kw):
    d = dict(device=0, batch=2, vocab=100, type=mk.MK_FP32, logits=P, row_stride=100, u=P, temperature=None,
             top_k=None, top_p=None, min_p=None, tokens=P, logprobs=None, status=None)
    d.update(kw)
    a = mk.mk_sample_args()
    for n, v in d.items():
        setattr(a, n, v)
    return a


@pytest.mark.parametrize("kw", [
    dict(n_tokens=-1), dict(max_pages=0), dict(n_pages=0), dict(n_kv_heads=0), dict(n_q_heads=-1),
    dict(head_dim=96), dict(rotary_dim=63), dict(rotary_dim=66), dict(rotary_dim=-2), dict(src_type=3),
    dict(dst_type=mk.MK_FP32), dict(k=None), dict(v=None), dict(q=None), dict(q_out=None), dict(k_pool=None),
    dict(v_pool=None), dict(inv_freq=None), dict(positions=None), dict(page_table=None), dict(n_tokens=5),
    dict(k_pool=P + 8), dict(q_out=P + 2), dict(k=P + 1)])
def test_append_refusals(kw):
    assert mk.lib.mk_rope_append(byref(append_args(**kw)), None) == mk.MK_ERR_INVALID


@pytest.mark.parametrize("kw", [
    dict(batch=-1), dict(n_groups=-1), dict(max_pages=0), dict(n_pages=0), dict(n_kv_heads=0), dict(n_q_heads=3),
    dict(head_dim=32), dict(type=mk.MK_FP32), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan),
    dict(scale=math.inf), dict(q=None), dict(k_pool=None), dict(page_table=None), dict(positions=None),
    dict(group_start=None), dict(prefix_lens=None), dict(out=None), dict(workspace=None),
    dict(q_token_stride=255), dict(q_token_stride=248), dict(q=P + 2), dict(out=P + 4), dict(workspace=P + 16)])
def test_attention_refusals(kw):
    assert mk.lib.mk_prefix_attention(byref(attention_args(**kw)), None) == mk.MK_ERR_INVALID


def test_attention_capacity():
    for kw in (dict(batch=4097), dict(n_q_heads=130), dict(n_pages=1 << 26), dict(max_pages=1 << 26),
               dict(workspace_bytes=1000)):
        assert mk.lib.mk_prefix_attention(byref(attention_args(**kw)), None) == mk.MK_ERR_CAPACITY, kw
    assert mk.lib.mk_prefix_attention_workspace(byref(attention_args(batch=4097))) == 0
    assert mk.lib.mk_prefix_attention_workspace(None) == 0
    small, large = (mk.lib.mk_prefix_attention_workspace(byref(attention_args(batch=b))) for b in (1, 4096))
    assert 0 < small < large


@pytest.mark.parametrize("kw", [dict(batch=-1), dict(vocab=0), dict(type=3), dict(logits=None), dict(u=None),
                                dict(tokens=None), dict(logits=P + 2)])
def test_sample_refusals(kw):
    assert mk.lib.mk_sample(byref(sample_args(**kw)), None) == mk.MK_ERR_INVALID


def test_null_and_empty_calls():
    assert mk.lib.mk_rope_append(None, None) == mk.MK_ERR_INVALID
    assert mk.lib.mk_prefix_attention(None, None) == mk.MK_ERR_INVALID
    assert mk.lib.mk_sample(None, None) == mk.MK_ERR_INVALID
    assert mk.lib.mk_sample(byref(sample_args(vocab=mk.MK_SAMPLE_MAX_VOCAB + 1)), None) == mk.MK_ERR_CAPACITY
    # nothing to do: no CUDA call either
    assert mk.lib.mk_prefix_attention(byref(attention_args(batch=0)), None) == mk.MK_OK
    assert mk.lib.mk_prefix_attention(byref(attention_args(n_groups=0)), None) == mk.MK_OK
    assert mk.lib.mk_sample(byref(sample_args(batch=0)), None) == mk.MK_OK


def test_python_functions_refuse_cpu_tensors():
    x, i = torch.zeros((2, 2, 64)), torch.zeros(2, dtype=torch.int32)
    pool = torch.zeros((2, 2, 64, 64), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        ops.rope_append(None, x, x, i, i[None], pool, pool, torch.zeros(32, dtype=torch.float64))
    with pytest.raises(TypeError):
        ops.prefix_attention(x, pool, pool, i[None], i, i, i[:1])
    with pytest.raises(TypeError):
        ops.sample(torch.zeros((2, 8)), torch.zeros(2))


def test_binding_matches_the_header_layout():
    # sizes of the argument structs as the C compiler lays them out (64-bit)
    assert ctypes.sizeof(mk.mk_rope_append_args) == 12 * 4 + 4 + 4 + 3 * 8 + 6 * 8 + 3 * 8 + 5 * 8
    assert ctypes.sizeof(mk.mk_prefix_attention_args) == 10 * 4 + 8 + 8 + 9 * 8 + 8 + 8
    assert ctypes.sizeof(mk.mk_sample_args) == 4 * 4 + 8 + 8 + 8 * 8


def test_frequencies():
    f, m = ops.rope_frequencies(8, 1e4, device="cpu")
    assert m == 1.0 and np.allclose(f, [1.0, 0.1, 0.01, 0.001], rtol=1e-15)
    f, m = ops.rope_frequencies(8, 1e4, scaling="even", factor=4.0, device="cpu")
    assert m == 1.0 and np.allclose(f, [0.25, 0.025, 0.0025, 0.00025], rtol=1e-15)
    # the base form keeps the fastest pair and slows the slowest by the factor
    f, m = ops.rope_frequencies(8, 1e4, scaling="base", factor=4.0, device="cpu")
    assert m == 1.0 and f[0] == 1.0 and math.isclose(f[3], 0.00025, rel_tol=1e-12)
    # by parts: over 4096 positions the pairs turn 651.9, 65.2, 6.52 and 0.652 times
    f, m = ops.rope_frequencies(8, 1e4, scaling="parts", factor=4.0, device="cpu")
    keep = (4096 * 0.01 / (2 * math.pi) - 1) / 31
    assert np.allclose(f, [1.0, 0.1, 0.01 * keep + 0.0025 * (1 - keep), 0.00025], rtol=1e-14)
    assert math.isclose(m, 0.1 * math.log(4.0) + 1.0)
    assert ops.rope_frequencies(0, device="cpu")[0].numel() == 0
    for bad in (dict(rotary_dim=3), dict(rotary_dim=8, factor=0.5), dict(rotary_dim=8, theta=0.0),
                dict(rotary_dim=8, scaling="other"), dict(rotary_dim=8, scaling="parts", fast_turns=1.0)):
        with pytest.raises(ValueError):
            ops.rope_frequencies(device="cpu", **bad)


def test_oracle_rotation_keeps_lengths_and_relative_angles():
    g = torch.Generator().manual_seed(0)
    x = torch.randn((3, 2, 16), generator=g, dtype=torch.float64)
    f, _ = ops.rope_frequencies(8, device="cpu")
    for il in (False, True):
        y, _ = ops_oracle.rotate(x, torch.tensor([0, 5, 1000]), f, il, 1.0)
        assert torch.allclose(y.norm(dim=-1), x.norm(dim=-1))
        assert torch.equal(y[0], x[0]) and torch.equal(y[..., 8:], x[..., 8:])
        a, _ = ops_oracle.rotate(x[:1], torch.tensor([17]), f, il, 1.0)
        b, _ = ops_oracle.rotate(x[1:2], torch.tensor([12]), f, il, 1.0)
        c, _ = ops_oracle.rotate(x[:1], torch.tensor([5]), f, il, 1.0)
        assert torch.allclose((a * b).sum(-1), (c * x[1:2]).sum(-1))


def test_oracle_sampling_follows_the_kept_distribution():
    x = np.array([1.0, 3.0, 2.0, 3.0, -1.0])
    ids, w = ops_oracle.kept(x, 1.0, 0, 1.0, 0.0)
    assert ids.tolist() == [1, 3, 2, 0, 4] and w[0] == w[1] == 1.0
    assert ops_oracle.kept(x, 1.0, 1, 1.0, 0.0)[0].tolist() == [1]
    assert ops_oracle.kept(x, 1.0, 3, 0.5, 0.0)[0].tolist() == [1, 3]
    assert ops_oracle.kept(x, 1.0, 0, 1.0, 0.3)[0].tolist() == [1, 3, 2]
    draws = [ops_oracle.sample(x, (i + 0.5) / 1000, 1.0)[0] for i in range(1000)]
    p = np.exp(x) / np.exp(x).sum()
    assert np.allclose(np.bincount(draws, minlength=5) / 1000, p, atol=2e-3)


def test_oracle_attention_is_softmax_over_the_pages():
    g = torch.Generator().manual_seed(1)
    kp, vp = (torch.randn((4, 1, 64, 64), generator=g, dtype=torch.float64) for _ in range(2))
    q = torch.randn((2, 2, 64), generator=g, dtype=torch.float64)
    table = torch.tensor([[2, 0], [3, 1]])
    out, lse, _, _ = ops_oracle.attention(q, kp, vp, table, [69, 80], [0, 2], [64], 0.125)
    k = torch.cat((kp[2, 0], kp[1, 0]))[:81]
    v = torch.cat((vp[2, 0], vp[1, 0]))[:81]
    want = torch.softmax(q[1] @ k.T * 0.125, -1) @ v
    assert torch.allclose(out[1], want)
    assert torch.allclose(lse[1], torch.logsumexp(q[1] @ k.T * 0.125, -1))


def test_decode_loop_refusals_without_a_context():
    how = mk.mk_sampling()
    assert mk.lib.mk_decode_step_shared(None, P, P, P, P, 1, P, P, P, None) == mk.MK_ERR_INVALID
    assert mk.lib.mk_decode_sample(None, 1, P, P, P, P, P, P, byref(how), None) == mk.MK_ERR_INVALID
    # the struct as the C compiler lays it out: eight pointers and a count
    assert ctypes.sizeof(mk.mk_sampling) == 8 * 8 + 8


def test_sampling_rules():
    from moe_persistent_cta_b200 import serving
    r = serving.sampling_rules(dict(temperature=0.5, top_k=7), 3, "cpu")
    assert r["temperature"].tolist() == [0.5] * 3 and r["top_k"].tolist() == [7] * 3
    assert r["top_k"].dtype == torch.int32 and set(r) == {"temperature", "top_k"}
    with pytest.raises(ValueError):
        serving.sampling_rules(dict(top_q=0.5), 3, "cpu")


def test_attention_line_of_tiles_fits_32_bits():
    big = dict(batch=4096, n_kv_heads=8, n_q_heads=8, q_token_stride=512, n_pages=8)
    assert mk.lib.mk_prefix_attention_workspace(byref(attention_args(max_pages=65531, **big))) > 0
    assert mk.lib.mk_prefix_attention_workspace(byref(attention_args(max_pages=65532, **big))) == 0
    assert mk.lib.mk_prefix_attention(byref(attention_args(max_pages=65532, **big)), None) == mk.MK_ERR_CAPACITY
