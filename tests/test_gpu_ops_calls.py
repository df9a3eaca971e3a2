"""How the serving operators' Python functions are called on the GPU: other
streams than the current one, outputs that the functions allocate, status words,
workspaces and waits that run out."""

import ctypes
import math

import pytest
import torch

from moe_persistent_cta_b200 import mk, ops
from tests import ops_oracle

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BUSY = 200_000_000          # cycles: about a tenth of a second


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32).to(DEV)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def attention_case(seed=1, lens=(90, 200, 131), hq=4, hkv=2, hd=64, dtype=torch.bfloat16, prefix=64):
    """Entries of one group, `prefix` tokens shared; the arguments and the 64-bit result."""
    g = gen(seed)
    b, width = len(lens), max(lens) // 64 + 1
    kp, vp = (torch.randn((b * width, hkv, 64, hd), generator=g).to(dtype) for _ in range(2))
    q = torch.randn((b, hq, hd), generator=g).to(dtype)
    table = torch.randperm(b * width, generator=g).view(b, width).to(torch.int32)
    pos = [n - 1 for n in lens]
    want = ops_oracle.attention(q, kp, vp, table, pos, [0, b], [prefix], 1 / math.sqrt(hd))
    args = [x.to(DEV) for x in (q, kp, vp, table)] + [i32(pos), i32([0, b]), i32([prefix])]
    return args, want


def check_attention(out, want, dtype=torch.bfloat16):
    # P's rounding moves a row by half a step of the weighted |v|, the output's by half a
    # step of itself; 32-bit scores and sums by 2e-5 (1 + the largest score)
    exact, _, mass, high = want
    h = torch.finfo(dtype).eps / 2
    bound = h * mass + h * exact.abs() + 2e-5 * (1 + high[..., None]) * mass + 1e-30
    assert ((out.cpu().double() - exact).abs() <= bound).all()


def check_tokens(tokens, logits, u):
    x, u = logits.cpu().numpy(), u.cpu().numpy()
    assert tokens.cpu().tolist() == [ops_oracle.sample(x[b], float(u[b]))[0] for b in range(len(u))]


# ---------------------------------------------------------------- streams --

def test_outputs_of_a_call_on_another_stream_than_the_current_one():
    """The functions' own outputs, with the current stream behind its work: what
    that stream does later reaches neither their values nor their memory."""
    args, want = attention_case()
    logits = torch.randn((5, 700), generator=gen(2)).to(DEV)
    u = torch.rand(5, generator=gen(3)).to(DEV)
    x = torch.randn((6, 4, 64), generator=gen(4)).to(torch.bfloat16).to(DEV)
    pool = torch.zeros((2, 1, 64, 64), dtype=torch.bfloat16, device=DEV)
    rope = (x[:, :2], x[:, 2:3], x[:, 3:], i32(range(6)), i32([[0, 1]]), pool, pool.clone(),
            ops.rope_frequencies(64, device=DEV)[0])
    kw = dict(seq=i32([0] * 6))
    side = torch.cuda.Stream()
    plain_q = ops.rope_append(*rope, **kw)
    ops.prefix_attention(*args, stream=side)             # loads the modules and fills the allocator's pools
    ops.sample(logits, u, stream=side)
    ops.rope_append(*rope, stream=side, **kw)
    torch.cuda.synchronize()
    # blocks that go back to the current stream's pool with a write of that stream still to come
    late = [torch.empty_like(plain_q), torch.empty(5, dtype=torch.int32, device=DEV), torch.empty_like(args[0])]
    for t in late:
        t.fill_(7)                                       # loads the kernel, which may wait for the device
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    for t in late:
        t.fill_(77)
    del late, t
    out = ops.prefix_attention(*args, stream=side)
    tokens = ops.sample(logits, u, stream=side)
    q_out = ops.rope_append(*rope, stream=side, **kw)
    torch.cuda.synchronize()
    check_attention(out, want)
    check_tokens(tokens, logits, u)
    assert torch.equal(q_out, plain_q)


def test_outputs_of_another_stream_outlive_their_release():
    """An output released while the current stream still reads it is not handed
    out again on the call's stream before that read."""
    logits = torch.randn((64, 300), generator=gen(5)).to(DEV)
    u = torch.rand(64, generator=gen(6)).to(DEV)
    other = torch.rand(64, generator=gen(7)).to(DEV)
    side = torch.cuda.Stream()
    ops.sample(logits, u, stream=side)
    torch.cuda.synchronize()
    tokens = ops.sample(logits, u, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(BUSY)
    kept = torch.empty_like(tokens).copy_(tokens)
    del tokens
    again = ops.sample(logits, other, stream=side)
    torch.cuda.synchronize()
    check_tokens(kept, logits, u)
    check_tokens(again, logits, other)


# ----------------------------------------------------------------- status --

def test_status_waits_for_calls_on_other_streams():
    logits = torch.randn((3, 50), generator=gen(8)).to(DEV)
    bad = torch.tensor([0.5, 1.5, 0.5], device=DEV)      # a number outside [0, 1)
    side = torch.cuda.Stream()
    status = ops.Status(DEV)
    ops.sample(logits, bad, stream=side, status=status)  # loads the module
    assert status.check()[0] == mk.MK_ERR_DEVICE
    for wait_for in (None, side):
        with torch.cuda.stream(side):
            torch.cuda._sleep(BUSY)
        ops.sample(logits, bad, stream=side, status=status)
        rc, detail = status.check() if wait_for is None else status.check(wait_for)
        assert rc == mk.MK_ERR_DEVICE and detail[:2] == [mk.MK_OP_SAMPLE, 1]
        status.check_ok(wait_for)                        # cleared
    # the clearing is past before a call on another stream can latch the next one
    ops.sample(logits, bad, stream=side, status=status)
    assert status.check()[0] == mk.MK_ERR_DEVICE


def test_status_word_is_clear_before_its_first_use():
    logits = torch.randn((1, 50), generator=gen(8)).to(DEV)
    bad = torch.tensor([-1.0], device=DEV)
    side = torch.cuda.Stream()
    ops.sample(logits, bad, stream=side)
    torch.zeros(8, dtype=torch.int32, device=DEV)        # loads the kernels
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    status = ops.Status(DEV)
    ops.sample(logits, bad, stream=side, status=status)
    side.synchronize()
    assert status.check()[0] == mk.MK_ERR_DEVICE


def test_status_of_a_captured_call():
    logits = torch.randn((2, 50), generator=gen(9)).to(DEV)
    u = torch.tensor([0.5, 0.25], device=DEV)
    status, tokens = ops.Status(DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    ops.sample(logits, u, tokens=tokens, status=status)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.sample(logits, u, tokens=tokens, status=status)
    side = torch.cuda.Stream()
    for good in (True, False, True):
        u.copy_(torch.tensor([0.5, 0.25 if good else math.nan]))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(BUSY // 10)
            graph.replay()
        rc, detail = status.check()
        assert (rc == mk.MK_OK) if good else (rc == mk.MK_ERR_DEVICE and detail[1] == 1)


# ------------------------------------------------- values that are no numbers --

@pytest.mark.parametrize("lens", [(200, 94, 131), (94, 70)])
@pytest.mark.parametrize("hd", [64, 128])
def test_attention_nan_beside_far_larger_scores(hd, lens):
    """A key that is NaN in a short remainder shows in the row's result, also where
    the prefix's scores are so much larger that the remainder's weight is 0; other
    rows are as if it were not there."""
    g = gen(11)
    n, width = len(lens), 4
    bad = lens.index(94)
    kp, vp = (torch.randn((n * width, 2, 64, hd), generator=g).to(torch.bfloat16) for _ in range(2))
    q = torch.randn((n, 4, hd), generator=g).to(torch.bfloat16)
    table = torch.randperm(n * width, generator=g).view(n, width).to(torch.int32)
    for h in range(4):                                   # scores of some hundreds in the prefix
        kp[int(table[0, 0]), h // 2, 5 + h] = 320.0 / hd ** 0.5 * q[bad, h] / (q[bad, h].float() ** 2).mean() ** 0.5
    pos = [x - 1 for x in lens]
    want = ops_oracle.attention(q, kp, vp, table, pos, [0, n], [64], hd ** -0.5)
    assert want[3][bad].min() > 200
    kp[int(table[bad, 1]), 1, 7] = math.nan              # token 71 of the entry, in KV head 1
    lse = torch.zeros((n, 4), device=DEV)
    out = ops.prefix_attention(q.to(DEV), kp.to(DEV), vp.to(DEV), table.to(DEV), i32(pos), i32([0, n]), i32([64]),
                               lse=lse).cpu()
    assert torch.isnan(out[bad, 2:]).all() and torch.isnan(lse[bad, 2:]).all()
    out[bad, 2:] = want[0][bad, 2:].to(torch.bfloat16)
    check_attention(out, want)


def test_attention_infinite_value_beside_far_larger_scores():
    # the weight's exponential is 0, the value infinite: no finite result
    g = gen(12)
    kp, vp = (torch.randn((4, 1, 64, 64), generator=g).to(torch.float16) for _ in range(2))
    q = torch.randn((1, 1, 64), generator=g).to(torch.float16)
    kp[0, 0, 3] = 40.0 * q[0, 0]
    args = lambda: (q.to(DEV), kp.to(DEV), vp.to(DEV), i32([[0, 1, 2, 3]]), i32([250]), i32([0, 1]), i32([64]))  # noqa: E731
    assert torch.isfinite(ops.prefix_attention(*args())).all()
    vp[2, 0, 9, :7] = math.inf
    out = ops.prefix_attention(*args()).cpu()[0, 0]
    assert not torch.isfinite(out[:7]).any() and torch.isfinite(out[7:]).all()


# ---------------------------------------------------- rows that are left out --

def test_queries_of_padding_are_zero_in_an_allocated_output():
    x = torch.randn((6, 4, 64), generator=gen(13)).to(torch.bfloat16).to(DEV)
    pool = torch.zeros((2, 1, 64, 64), dtype=torch.bfloat16, device=DEV)
    freq = ops.rope_frequencies(64, device=DEV)[0]
    status = ops.Status(DEV)
    want = torch.zeros((6, 2, 64), dtype=torch.bfloat16, device=DEV)
    for kept, seq, pos in ((range(6), [0] * 6, range(6)), ([0, 2, 3], [0, -1, 0, 0, -1, -1], range(6)),
                           ([1], [0, 0, 9, 0, -1, 0], [-1, 1, 2, 128, 4, 200])):
        stale = torch.full((6, 2, 64), math.nan, dtype=torch.bfloat16, device=DEV)
        del stale                                        # the allocator hands its memory out next
        got = ops.rope_append(x[:, :2], x[:, 2:3], x[:, 3:], i32(pos), i32([[0, 1]]), pool, pool.clone(), freq,
                              seq=i32(seq), status=status)
        kept = list(kept)
        if len(kept) == 6:
            want, all_rows = torch.zeros_like(want), got
            continue
        expect = torch.zeros_like(want)
        expect[kept] = all_rows[kept]
        assert torch.equal(got, expect)
        # a q_out that is passed keeps what it held there
        mine = torch.full_like(want, 5.0)
        ops.rope_append(x[:, :2], x[:, 2:3], x[:, 3:], i32(pos), i32([[0, 1]]), pool, pool.clone(), freq,
                        seq=i32(seq), q_out=mine, status=status)
        rest = [t for t in range(6) if t not in kept]
        assert torch.equal(mine[kept], expect[kept]) and (mine[rest] == 5.0).all()


# -------------------------------------------------------------- workspaces --

def c_arguments(args, out, **more):
    """mk_prefix_attention_args of prefix_attention's tensors (no workspace)."""
    q, kp, vp, table, pos, start, prefix = args
    a = mk.mk_prefix_attention_args()
    d = dict(device=0, batch=q.shape[0], n_groups=prefix.numel(), max_pages=table.shape[1], n_pages=kp.shape[0],
             n_q_heads=q.shape[1], n_kv_heads=kp.shape[1], head_dim=q.shape[2],
             type=mk.MK_BF16 if q.dtype is torch.bfloat16 else mk.MK_FP16, scale=q.shape[2] ** -0.5,
             q_token_stride=q.stride(0), q=q.data_ptr(), k_pool=kp.data_ptr(), v_pool=vp.data_ptr(),
             page_table=table.data_ptr(), positions=pos.data_ptr(), group_start=start.data_ptr(),
             prefix_lens=prefix.data_ptr(), out=out.data_ptr(), **more)
    for name, value in d.items():
        setattr(a, name, value)
    return a


@pytest.mark.parametrize("lens,hq,hkv,prefix", [
    ((20000,), 4, 1, 20000), ((20000,), 2, 2, 0), ((9000, 9100), 3, 1, 8000), ((700, 650, 9), 8, 2, 600),
    (tuple(range(300, 300 + 40)), 4, 1, 256)])
def test_attention_stays_inside_its_workspace(lens, hq, hkv, prefix):
    """A workspace of just the size asked for, in the midst of other memory, at
    batches of few rows (whose shares are small) and of more rows than a tile's."""
    b, hd = len(lens), 64
    g = gen(14)
    width = max(lens) // 64 + 1
    kp, vp = (torch.randn((b * width, hkv, 64, hd), generator=g).to(torch.bfloat16) for _ in range(2))
    q = torch.randn((b, hq, hd), generator=g).to(torch.bfloat16)
    table = torch.randperm(b * width, generator=g).view(b, width).to(torch.int32)
    pos = [n - 1 for n in lens]
    dev = [x.to(DEV) for x in (q, kp, vp, table)] + [i32(pos), i32([0, b]), i32([prefix])]
    want = ops.prefix_attention(*dev)
    out = torch.zeros_like(dev[0])
    a = c_arguments(dev, out)
    size, edge = mk.lib.mk_prefix_attention_workspace(ctypes.byref(a)), 1 << 20
    for fill in (0, 255):
        memory = torch.full((size + 2 * edge,), fill, dtype=torch.uint8, device=DEV)
        assert memory.data_ptr() % 256 == 0
        a.workspace, a.workspace_bytes = memory.data_ptr() + edge, size
        assert mk.lib.mk_prefix_attention(ctypes.byref(a), torch.cuda.current_stream().cuda_stream) == mk.MK_OK
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert (memory[:edge] == fill).all() and (memory[edge + size:] == fill).all()
        a.workspace_bytes = size - 1
        assert mk.lib.mk_prefix_attention(ctypes.byref(a), None) == mk.MK_ERR_CAPACITY


# --------------------------------------------------- waits that run out --

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("hd,lens,hq,hkv,prefix", [
    (64, (90, 200, 131), 4, 2, 64),                      # a block's share is a tile: it ends at once
    (128, (900, 1000, 1100, 40), 4, 1, 830),             # more than one tile, two streams of one unit
    (64, (1500,), 2, 1, 0),
    (128, tuple(range(130, 130 + 40)), 16, 4, 128)])     # two tiles of rows, one warp a row in the join
def test_attention_rows_of_a_wait_that_ran_out(hd, lens, hq, hkv, prefix, dtype):
    """One block's tiles never come: its waits give up, the status says so, and the
    rows that it held shares of are right all the same."""
    args, want = attention_case(15, lens, hq, hkv, hd, dtype, prefix)
    b = len(lens)
    out, lse = torch.full_like(args[0], 9.0), torch.full((b, hq), 9.0, device=DEV)
    status = ops.Status(DEV)
    a = c_arguments(args, out, lse=lse.data_ptr(), status=status.word.data_ptr())
    size = mk.lib.mk_prefix_attention_workspace(ctypes.byref(a))
    work = torch.full((size,), 255, dtype=torch.uint8, device=DEV)
    a.workspace, a.workspace_bytes = work.data_ptr(), size
    stream = torch.cuda.current_stream().cuda_stream
    assert mk.lib.mk_prefix_attention_selftest(ctypes.byref(a), stream) == mk.MK_OK
    rc, detail = status.check()
    assert rc == mk.MK_ERR_TIMEOUT and detail[:2] == [mk.MK_OP_PREFIX_ATTENTION, 0]
    check_attention(out, want, dtype)
    # 32-bit scores and sums move the logarithm by 2e-5 (1 + the largest score)
    assert ((lse.cpu().double() - want[1]).abs() <= 2e-5 * (1 + want[3])).all()
    # the next call in the same workspace is as ever
    out.fill_(9.0)
    assert mk.lib.mk_prefix_attention(ctypes.byref(a), stream) == mk.MK_OK
    status.check_ok()
    assert torch.equal(out, ops.prefix_attention(*args))
    check_attention(out, want, dtype)


# ---------------------------------------------------------------- strides --

def test_attention_strides_of_single_entries_and_heads():
    """Strides along a size of one say nothing: any value is accepted."""
    args, want = attention_case(16, (90, 200), 1, 1, 64)
    wide = torch.zeros((2, 3, 64), dtype=torch.bfloat16, device=DEV)
    wide[:, 1:2] = args[0]
    odd = torch.zeros(2 * 72 + 64, dtype=torch.bfloat16, device=DEV)
    for q in (wide[:, 1:2], torch.as_strided(args[0], (2, 1, 64), (64, 5, 1))):
        check_attention(ops.prefix_attention(q, *args[1:]), want)
    one, want1 = attention_case(17, (150,), 4, 2, 64)
    for q in (torch.as_strided(one[0], (1, 4, 64), (7, 64, 1)), torch.as_strided(one[0], (1, 4, 64), (0, 64, 1))):
        check_attention(ops.prefix_attention(q, *one[1:]), want1)
    for strides in ((72, 65, 1), (100, 64, 1), (8, 64, 1)):   # heads apart, rows that overlap or start off the boundary
        with pytest.raises((ValueError, mk.MKError)):
            ops.prefix_attention(torch.as_strided(odd, (2, 1 + (strides[1] == 65), 64), strides), args[1], args[2],
                                 *args[3:])


@pytest.mark.parametrize("hd", [64, 128])
def test_attention_values_near_the_largest(hd):
    """Finite values whose weighted sum leaves the 32-bit range: their mean does not."""
    g = gen(18)
    lens, width = (300, 500), 8
    kp, vp = (torch.randn((2 * width, 2, 64, hd), generator=g) for _ in range(2))
    vp = (vp.sign() * (2.0 + vp.abs().clamp(max=1.3)) * 1e38).to(torch.bfloat16)
    vp[:, :, :, 0] = torch.finfo(torch.bfloat16).min     # a column of the type's lowest value
    kp, q = kp.to(torch.bfloat16), torch.randn((2, 4, hd), generator=g).to(torch.bfloat16)
    assert torch.isfinite(vp).all()
    table = torch.randperm(2 * width, generator=g).view(2, width).to(torch.int32)
    pos = [n - 1 for n in lens]
    out, lse, mass, high = ops_oracle.attention(q, kp, vp, table, pos, [0, 2], [128], hd ** -0.5)
    assert torch.isfinite(out).all()
    got_lse = torch.zeros((2, 4), device=DEV)
    got = ops.prefix_attention(q.to(DEV), kp.to(DEV), vp.to(DEV), table.to(DEV), i32(pos), i32([0, 2]), i32([128]),
                               lse=got_lse)
    assert torch.isfinite(got).all()
    check_attention(got, (out, lse, mass, high))
    assert ((got_lse.cpu().double() - lse).abs() <= 2e-5 * (1 + high)).all()
