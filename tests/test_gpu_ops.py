"""The serving operators on the GPU against their 64-bit definitions.

Tolerances, from the arithmetic (h is half a step of the output's type):
* rope_append: values are converted once, so they are equal; keys and queries
  carry the angle's last 32-bit rounding (pi 2^-24), two ulp of sine and
  cosine and three roundings of the products, together below 8e-7 of the
  pair's |a| + |b|, then the output's rounding: h |y|.
* prefix_attention: P is rounded to the type before P V, which moves the
  result by at most h of the weighted |v|; the output is rounded: h |o|; the
  32-bit scores, exponents and sums move weights by less than 2e-5 (1 + the
  largest score).  lse: the same 2e-5 (1 + largest score), absolute.
* sample: tokens are equal; log-probabilities are 64-bit values rounded once.
"""

import math

import numpy as np
import pytest
import torch

from moe_persistent_cta_b200 import mk, ops
from tests import ops_oracle

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
PAGE = 64


def gen(seed):
    return torch.Generator().manual_seed(seed)


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32).to(DEV)


# ------------------------------------------------------------ rope_append --

def append_case(seed, counts, starts, hq, hkv, hd, rot, src, dst, interleaved=False, magnitude=1.0,
                offset=0, in_place=False, pad=()):
    g = gen(seed)
    t = sum(counts)
    seq = [i for i, n in enumerate(counts) for _ in range(n)]
    pos = [s + j for s, n in zip(starts, counts) for j in range(n)]
    for i in pad:
        seq[i] = -1
    width = max(p // PAGE + 1 for p in pos)
    n_pages = len(counts) * width + 3
    table = torch.randperm(n_pages, generator=g)[:len(counts) * width].view(len(counts), width)
    wide = torch.randn((t, hq + 2 * hkv, hd + offset), generator=g).to(TYPES[src])
    qkv = wide.to(DEV)[:, :, offset:] if offset else wide.to(DEV)
    rows = wide[:, :, offset:]
    kp = torch.full((n_pages, hkv, PAGE, hd), 7.0, dtype=TYPES[dst])
    vp = torch.full_like(kp, -7.0)
    freq, _ = ops.rope_frequencies(rot, device="cpu")
    kd, vd = kp.to(DEV), vp.to(DEV)
    q_in = qkv[:, :hq]
    if in_place:
        q_in = q_in.contiguous()
    q_out = q_in if in_place else torch.full((t, hq, hd), 3.0, dtype=TYPES[dst], device=DEV)
    status = ops.Status(DEV)
    got_q = ops.rope_append(q_in if hq else None, qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], i32(pos),
                            i32(table), kd, vd, freq.to(DEV), seq=i32(seq), interleaved=interleaved,
                            magnitude=magnitude, q_out=q_out if hq else None, status=status)
    status.check_ok()
    p = torch.tensor(pos)
    want_q, reach_q = ops_oracle.rotate(rows[:, :hq], p, freq, interleaved, magnitude)
    want_k, reach_k = ops_oracle.rotate(rows[:, hq:hq + hkv], p, freq, interleaved, magnitude)
    h = torch.finfo(TYPES[dst]).eps / 2
    tiny = float(torch.finfo(TYPES[dst]).smallest_normal) * h
    if hq:
        err = (got_q.cpu().double() - want_q).abs()
        for i in pad:
            assert in_place or (got_q[i].cpu() == 3.0).all()
            err[i] = 0.0
        assert (err <= h * want_q.abs() + 8e-7 * reach_q + tiny).all(), float(err.max())
    k_got, v_got = kd.cpu(), vd.cpu()
    for i in range(t):
        if seq[i] < 0:
            continue
        page, slot = int(table[seq[i], pos[i] // PAGE]), pos[i] % PAGE
        err = (k_got[page, :, slot].double() - want_k[i]).abs()
        assert (err <= h * want_k[i].abs() + 8e-7 * reach_k[i] + tiny).all(), (i, float(err.max()))
        assert torch.equal(v_got[page, :, slot], rows[i, hq + hkv:].float().to(TYPES[dst]))
        k_got[page, :, slot], v_got[page, :, slot] = 7.0, -7.0
    assert (k_got == 7.0).all() and (v_got == -7.0).all()       # nothing else was written


@pytest.mark.parametrize("src,dst", [("bf16", "bf16"), ("fp32", "bf16"), ("fp16", "fp16"),
                                     ("fp32", "fp16"), ("bf16", "fp16"), ("fp16", "bf16")])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_types(src, dst, interleaved):
    append_case(1, [1, 70, 5], [63, 0, 300], 4, 2, 64, 64, src, dst, interleaved)


@pytest.mark.parametrize("hd,rot", [(64, 2), (64, 36), (64, 48), (128, 0), (128, 16), (128, 50),
                                    (128, 64), (128, 126), (128, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_part_of_the_head(hd, rot, interleaved):
    append_case(2, [3, 1, 66], [10, 4095, 120], 6, 2, hd, rot, "fp32", "bf16", interleaved, 1.25)


@pytest.mark.parametrize("offset", [0, 1, 2, 8])
def test_append_strides(offset):
    append_case(3, [5, 9], [0, 700], 3, 3, 64, 64, "bf16", "bf16", offset=offset)
    append_case(3, [5, 9], [0, 700], 3, 3, 64, 20, "fp32", "bf16", offset=offset)


def test_append_far_position():
    append_case(4, [2], [(1 << 20) - 2], 1, 1, 64, 64, "fp32", "bf16")


def test_append_without_queries_and_one_token():
    append_case(5, [1], [0], 0, 1, 128, 128, "bf16", "bf16")
    append_case(6, [1], [64], 16, 4, 128, 128, "bf16", "bf16")


@pytest.mark.parametrize("rot,interleaved", [(128, False), (128, True), (36, False)])
def test_append_rotates_queries_in_place_and_skips_padding(rot, interleaved):
    append_case(7, [4, 8], [5, 60], 8, 2, 128, rot, "bf16", "bf16", interleaved, in_place=True)
    append_case(8, [4, 8], [5, 60], 8, 2, 128, rot, "bf16", "bf16", interleaved, pad=(0, 6, 11))


def test_append_faults_are_latched_and_left_out():
    k = torch.ones((5, 1, 64), dtype=torch.bfloat16, device=DEV)
    freq, _ = ops.rope_frequencies(64, device=DEV)
    for positions, seq, table, value in (
            ([0, 1, 2, 128, 4], [0] * 5, [[1, 2]], 128),       # beyond the row
            ([0, 1, -1, 3, 4], [0] * 5, [[1, 2]], -1),
            ([0, 1, 2, 3, 4], [0, 0, 1, 0, 0], [[1, 2]], 1),   # no such row
            ([0, 1, 2, 70, 4], [0] * 5, [[1, 4]], 4),          # no such page
            ([0, 1, 2, 70, 4], [0] * 5, [[1, -1]], -1)):
        kp = torch.zeros((4, 1, PAGE, 64), dtype=torch.bfloat16, device=DEV)
        vp, status = torch.zeros_like(kp), ops.Status(DEV)
        ops.rope_append(None, k, k, i32(positions), i32(table), kp, vp, freq, seq=i32(seq), status=status)
        rc, detail = status.check()
        assert rc == mk.MK_ERR_DEVICE and detail[0] == mk.MK_OP_ROPE_APPEND and detail[2] == value
        assert float(vp.float().sum()) == 4 * 64               # the other four tokens
        assert status.check() == (mk.MK_OK, [0, 0, 0, 0])
        with pytest.raises(mk.MKError):
            ops.rope_append(None, k, k, i32(positions), i32(table), kp, vp, freq, seq=i32(seq),
                            status=status)
            status.check_ok()


# ------------------------------------------------------- prefix_attention --

def attention_case(seed, members, prefix, positions, hq, hkv, hd, dt, first=0, behind=0, scale=None,
                   causal=False, spread=1.0, q_pad=0, run=None):
    """members per group, prefix tokens per group, positions per entry; `first`
    and `behind` entries of no group around them.  All cache memory that no
    entry sees is NaN."""
    g = gen(seed)
    b, n = first + sum(members) + behind, len(members)
    start = [first]
    for m in members:
        start.append(start[-1] + m)
    positions = [5] * first + list(positions) + [5] * behind
    assert len(positions) == b
    width = max(1, max(max(positions) + 1, max(prefix, default=0)) + PAGE - 1) // PAGE + 1
    table = torch.full((b, width), -3, dtype=torch.int32)
    nxt = 0
    for k in range(n):
        lead = start[k]
        shared = (prefix[k] + PAGE - 1) // PAGE
        for i in range(start[k], start[k + 1]):
            for page in range((max(positions[i] + 1, prefix[k] if i == lead else 0) + PAGE - 1) // PAGE):
                if i != lead and (page < prefix[k] // PAGE or (causal and page < shared)):
                    table[i, page] = table[lead, page] if table[lead, page] >= 0 else 0
                else:
                    table[i, page] = nxt
                    nxt += 1
    n_pages = nxt + 2
    order = torch.randperm(n_pages, generator=g).to(torch.int32)
    table = torch.where(table >= 0, order[table.clamp(min=0).long()], table)
    kp = torch.full((n_pages, hkv, PAGE, hd), math.nan, dtype=TYPES[dt])
    vp = kp.clone()
    for k in range(n):
        top = max((positions[i] + 1 for i in range(start[k], start[k + 1])), default=0)
        for i in range(start[k], start[k + 1]):
            lo = 0 if i == start[k] else prefix[k]
            hi = positions[i] + 1
            if i == start[k]:
                hi = max(hi, min(prefix[k], top))
            for t in range(lo, hi):
                page = int(table[i, t // PAGE])
                kp[page, :, t % PAGE] = torch.randn((hkv, hd), generator=g).to(TYPES[dt])
                vp[page, :, t % PAGE] = torch.randn((hkv, hd), generator=g).to(TYPES[dt])
    q = (spread * torch.randn((b, hq, hd + q_pad), generator=g)).to(TYPES[dt])[..., :hq, :hd]
    qd = torch.zeros((b, hq * hd + 8 * q_pad), dtype=TYPES[dt], device=DEV)[:, :hq * hd].view(b, hq, hd) \
        if q_pad else torch.empty((b, hq, hd), dtype=TYPES[dt], device=DEV)
    qd.copy_(q)
    scale = scale if scale is not None else 1.0 / math.sqrt(hd)
    out = torch.full((b, hq, hd), 9.0, dtype=TYPES[dt], device=DEV)
    lse = torch.full((b, hq), 9.0, device=DEV)
    status = ops.Status(DEV)
    args = (qd, kp.to(DEV), vp.to(DEV), i32(table), i32(positions), i32(start), i32(prefix))
    if run is None:
        ops.prefix_attention(*args, scale=scale, out=out, lse=lse, status=status)
    else:
        run(args, dict(scale=scale, out=out, lse=lse, status=status))
    status.check_ok()
    check_attention(out, lse, ops_oracle.attention(q, kp, vp, table, positions, start, prefix, scale), dt)


def check_attention(out, lse, want, dt):
    o, s, mass, high = want
    none = torch.isnan(s)
    got, got_lse = out.cpu().double(), lse.cpu().double()
    assert (got[none] == 9.0).all() and (got_lse[none] == 9.0).all()     # of no group: as they were
    h = torch.finfo(TYPES[dt]).eps / 2
    slack = 2e-5 * (1.0 + high)
    ok = ~none
    err = (got - o).abs()
    tol = h * (mass + o.abs()) + slack[..., None] * mass + 1e-7
    assert (err[ok] <= tol[ok]).all(), (float(err[ok].max()), float((err[ok] / tol[ok]).max()))
    empty = torch.isneginf(s)
    assert torch.equal(torch.isneginf(got_lse), empty)
    some = ok & ~empty
    assert ((got_lse - s).abs()[some] <= slack[some]).all()


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("prefix", [0, 1, 63, 64, 65, 127, 128, 129, 200, 256, 300])
def test_attention_prefix_lengths(prefix, hd, dt):
    attention_case(prefix, [4], [prefix], [prefix + x for x in (0, 1, 62, 130)], 4, 2, hd, dt)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (6, 2), (8, 2), (5, 1), (14, 2), (8, 1), (32, 2),
                                    (64, 1), (8, 8)])
def test_attention_head_layouts(hq, hkv):
    attention_case(3, [3, 2], [90, 10], [91, 95, 300, 12, 10], hq, hkv, 64, "bf16")


@pytest.mark.parametrize("length", [1, 2, 63, 64, 65, 128, 129, 1000])
def test_attention_of_single_sequences(length):
    attention_case(length, [1, 1], [0, length], [length - 1, length - 1], 4, 2, 128, "bf16")


def test_attention_idle_short_and_outside_entries():
    # idle entries, entries that end inside the prefix, an empty group, entries of no group
    attention_case(11, [4, 0, 3], [150, 7, 70], [-1, 0, 149, 200, 30, -1, 69], 4, 2, 64, "bf16", first=2,
                   behind=3)
    attention_case(12, [2], [100], [-1, -1], 4, 2, 64, "bf16")
    attention_case(13, [1], [100], [20], 4, 2, 128, "fp16", behind=1)


@pytest.mark.parametrize("hq,hkv,members", [(16, 4, 33), (16, 4, 64), (16, 4, 70), (4, 4, 129),
                                            (3, 1, 43), (3, 1, 90), (7, 1, 37)])
def test_attention_more_rows_than_one_tile(hq, hkv, members):
    pos = [200 + (7 * i) % 90 for i in range(members)]
    attention_case(members, [members], [200], pos, hq, hkv, 64, "bf16")


@pytest.mark.parametrize("hd,past,piece", [(64, 0, 1), (64, 0, 150), (128, 100, 77), (128, 3, 40)])
def test_attention_causal_piece(hd, past, piece):
    attention_case(past + piece, [piece], [past + piece], range(past, past + piece), 8, 2, hd, "bf16",
                   causal=True)


def test_attention_long_split_over_all_blocks():
    attention_case(21, [2], [6000], [6100, 6300], 2, 1, 64, "bf16")


def test_attention_many_short_sequences():
    # far more shares per block than one pass lists
    n = 700
    attention_case(22, [1] * n, [0] * n, [(i * 5) % 23 for i in range(n)], 8, 8, 64, "bf16")


def test_attention_large_scores_and_scale():
    # scores up to some hundreds: the running reference is moved many times
    attention_case(23, [3], [500], [520, 499, 700], 4, 2, 64, "bf16", spread=20.0)
    attention_case(24, [3], [500], [520, 499, 700], 4, 2, 64, "fp16", spread=20.0)
    attention_case(25, [3], [500], [520, 499, 700], 4, 2, 64, "bf16", scale=0.01)


def test_attention_flat_fp16_tail():
    # one token far above very many equal ones, whose weights fp16 alone would lose
    n, hd = 4096, 64
    kp = torch.zeros((n // PAGE, 1, PAGE, hd), dtype=torch.float16)
    vp = torch.ones_like(kp)
    kp[0, 0, 0, 0] = 8.0
    vp[0, 0, 0] = 0.0
    q = torch.zeros((1, 1, hd), dtype=torch.float16)
    q[0, 0, 0] = 2.0 * math.log(2.0) + 0.01
    out, lse = torch.full((1, 1, hd), 9.0, dtype=torch.float16, device=DEV), torch.zeros((1, 1), device=DEV)
    table = torch.arange(n // PAGE, dtype=torch.int32)[None]
    ops.prefix_attention(q.to(DEV), kp.to(DEV), vp.to(DEV), table.to(DEV), i32([n - 1]), i32([0, 1]),
                         i32([n]), scale=1.5, out=out, lse=lse)
    check_attention(out, lse, ops_oracle.attention(q, kp, vp, table, [n - 1], [0, 1], [n], 1.5), "fp16")


def test_attention_token_stride_of_queries():
    attention_case(26, [3], [70], [75, 100, 70], 4, 2, 64, "bf16", q_pad=1)


def test_attention_on_another_stream_twice_at_once():
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []

    def run(args, kw):
        torch.cuda.synchronize()
        for s in (s1, s2):
            o = {**kw, "out": torch.full_like(kw["out"], 9.0), "lse": torch.full_like(kw["lse"], 9.0)}
            torch.cuda.synchronize()
            outs.append(o)
        for _ in range(5):
            for s, o in zip((s1, s2), outs):
                ops.prefix_attention(*args, **o, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(outs[0]["out"], outs[1]["out"])
        kw["out"].copy_(outs[0]["out"])
        kw["lse"].copy_(outs[0]["lse"])

    attention_case(27, [5, 2], [1000, 300], [1001, 1200, 999, 1500, 1000, 305, 300], 8, 2, 128, "bf16",
                   run=run)


def test_attention_captured_and_replayed_with_other_lengths():
    def run(args, kw):
        q, kp, vp, table, positions, start, prefix = args
        want_pos = positions.clone()
        ops.prefix_attention(*args, **kw)                 # loads the module outside the capture
        torch.cuda.synchronize()
        positions.copy_(torch.where(positions >= 0, 0, positions))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ops.prefix_attention(*args, **kw)
        positions.copy_(want_pos)
        kw["out"].fill_(9.0)
        kw["lse"].fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()

    attention_case(28, [4, 1], [300, 0], [301, 400, 299, -1, 50], 4, 2, 64, "bf16", run=run)


def test_attention_faults():
    q = torch.zeros((2, 1, 64), dtype=torch.bfloat16, device=DEV)
    pool = torch.ones((4, 1, PAGE, 64), dtype=torch.bfloat16, device=DEV)
    status = ops.Status(DEV)

    def call(positions, table, start=(0, 2), prefix=(0,)):
        out = ops.prefix_attention(q, pool, pool, i32(table), i32(positions), i32(start), i32(prefix),
                                   status=status)
        return status.check(), out

    (rc, d), out = call([128, 3], [[0, 1], [2, 3]])             # beyond the row: sees nothing
    assert rc == mk.MK_ERR_DEVICE and d == [mk.MK_OP_PREFIX_ATTENTION, 0, 128, 128]
    assert (out[0] == 0).all() and (out[1] == 1).all()
    (rc, d), out = call([3, 3], [[0, 1], [4, 3]])               # no such page
    assert rc == mk.MK_ERR_DEVICE and d[2] == 4 and (out[0] == 1).all()
    (rc, _), _ = call([3, 3], [[0, 1], [2, 3]], start=(2, 0))   # out of order
    assert rc == mk.MK_ERR_DEVICE
    (rc, _), _ = call([3, 3], [[0, 1], [2, 3]], start=(0, 3))
    assert rc == mk.MK_ERR_DEVICE
    (rc, d), _ = call([3, 3], [[0, 1], [2, 3]], prefix=(-1,))
    assert rc == mk.MK_ERR_DEVICE and d[2] == -1
    (rc, _), out = call([3, 3], [[0, 1], [2, 3]])
    assert rc == mk.MK_OK and (out == 1).all()


# ------------------------------------------------------------------ sample --

def sample_case(x, u, temperature=None, k=None, p=None, m=None, dt="fp32", stride=0):
    x = torch.as_tensor(np.asarray(x), dtype=torch.float32).to(TYPES[dt])
    b, v = x.shape
    xd = x.to(DEV)
    if stride:
        wide = torch.full((b, v + stride), 50.0, dtype=TYPES[dt], device=DEV)
        wide[:, stride // 2:stride // 2 + v] = xd
        xd = wide[:, stride // 2:stride // 2 + v]
    f = lambda t: None if t is None else torch.tensor(t, dtype=torch.float32, device=DEV)  # noqa: E731
    logprobs, status = torch.full((b,), 5.0, device=DEV), ops.Status(DEV)
    got = ops.sample(xd, f(u), temperature=f(temperature), top_k=None if k is None else i32(k), top_p=f(p),
                     min_p=f(m), logprobs=logprobs, status=status)
    status.check_ok()
    rows = x.double().numpy()
    r32 = lambda t, i, d: d if t is None else float(np.float32(t[i]))  # noqa: E731
    for i in range(b):
        tok, lp = ops_oracle.sample(rows[i], r32(u, i, 0), r32(temperature, i, 1.0), 0 if k is None else k[i],
                                    r32(p, i, 1.0), r32(m, i, 0.0))
        assert int(got[i]) == tok, (i, int(got[i]), tok)
        g = float(logprobs[i])
        assert g == lp or abs(g - lp) <= 2.0 ** -23 * abs(lp) + 1e-14, (i, g, lp)


def rules(b, seed, names):
    r = np.random.default_rng(seed)
    full = dict(temperature=(0.3 + 1.5 * r.random(b)).tolist(), k=r.integers(0, 60, b).tolist(),
                p=(0.05 + r.random(b)).tolist(), m=(0.2 * r.random(b)).tolist())
    return {n: full[n] for n in names}


@pytest.mark.parametrize("names", [(), ("temperature",), ("k",), ("p",), ("m",), ("k", "p"), ("p", "m"),
                                   ("temperature", "k", "p", "m")])
@pytest.mark.parametrize("v", [1, 2, 31, 1000, 2049, 40001])
def test_sample_rules(v, names):
    r = np.random.default_rng(v)
    b = 7
    sample_case(3 * r.standard_normal((b, v)), r.random(b), **rules(b, v, names))


@pytest.mark.parametrize("dt", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("v,stride", [(151552, 0), (151541, 3), (4100, 1)])
def test_sample_types_strides_and_ties(dt, v, stride):
    # 16-bit logits repeat: cuts fall among equal ones
    r = np.random.default_rng(5)
    b = 9
    sample_case(2 * r.standard_normal((b, v)), r.random(b), dt=dt, stride=stride,
                **rules(b, 6, ("temperature", "k", "p", "m")))
    sample_case(2 * r.standard_normal((b, v)), r.random(b), dt=dt, stride=stride, **rules(b, 7, ("p",)))


def test_sample_many_kept():
    # cuts far down the row: thousands by count, nearly all by probability
    r = np.random.default_rng(8)
    x = r.standard_normal((6, 60000))
    sample_case(x, r.random(6), k=[2000, 2048, 2049, 5000, 30000, 59999])
    sample_case(x, r.random(6), p=[0.9, 0.99, 0.999, 0.9999, 0.5, 0.7])
    sample_case(x, r.random(6), k=[40000] * 6, p=[0.9, 0.99, 0.3, 0.8, 0.95, 0.6], temperature=[2.0] * 6)


def test_sample_equal_logits():
    x = np.zeros((8, 10000))
    u = [0.0, 0.25, 0.5, 0.999, 0.1, 0.2, 0.3, 0.9999999]
    sample_case(x, u)
    sample_case(x, u, k=[1, 2, 3, 100, 9999, 10000, 5000, 4096])
    sample_case(x, u, p=[0.5, 0.25, 0.125, 0.75, 0.001, 0.0, 0.9375, 0.5])
    sample_case(x, u, m=[1.0] * 8)
    # signed zeros are equal; so the ties run over both
    x[:, ::2] = -0.0
    sample_case(x, u, k=[1, 2, 3, 100, 9999, 10000, 5000, 4096])


def test_sample_masked_and_unusual_logits():
    inf, nan = math.inf, math.nan
    x = np.full((10, 3000), -inf)
    x[0, 2999] = 1.0                                     # one token left
    x[2] = nan                                           # nothing to draw, like row 1
    x[3, 10:20] = nan
    x[3, 20:40] = 0.5
    x[4, [5, 70, 900]] = inf                             # only these
    x[5, [5, 70]] = [3e38, -3e38]
    x[6, :100] = np.linspace(-80, 20, 100)
    x[7, 100:200] = -3.4028234663852886e38               # a mask of the type's lowest value
    x[8, 5] = 1e-40
    x[8, 6] = -1e-40
    x[9, ::3] = np.linspace(-5, 5, 1000)
    u = [0.0, 0.5, 0.5, 0.99, 0.4, 0.9, 0.99, 0.35, 0.7, 0.6]
    sample_case(x, u)
    sample_case(x, u, k=[5] * 10, p=[0.9] * 10, m=[0.01] * 10, temperature=[0.7] * 10)
    sample_case(x, u, p=[0.3] * 10)
    sample_case(x, u, temperature=[0.0] * 10)
    sample_case(x, u, temperature=[1e-38] * 10)
    sample_case(x, u, temperature=[1e30] * 10, k=[7] * 10)


def test_sample_one_far_above():
    x = np.random.default_rng(3).standard_normal((4, 20000))
    x[:, 17] = 1e4
    sample_case(x, [0.1, 0.5, 0.9, 0.99], k=[3, 300, 3000, 0], p=[0.9, 1.0, 1.0, 0.99])


def test_sample_bad_parameters():
    x = torch.zeros((6, 100), device=DEV)
    nan = math.nan
    u = torch.tensor([0.5, 1.0, -0.1, nan, 0.5, 0.5], device=DEV)
    t = torch.tensor([1.0, 1.0, 1.0, 1.0, -1.0, math.inf], device=DEV)
    status, lp = ops.Status(DEV), torch.zeros(6, device=DEV)
    got = ops.sample(x, u, temperature=t, logprobs=lp, status=status)
    rc, d = status.check()
    assert rc == mk.MK_ERR_DEVICE and d[0] == mk.MK_OP_SAMPLE
    assert got.tolist() == [50, -1, -1, -1, -1, -1] and torch.isneginf(lp[1:]).all()
    half = torch.full((6,), 0.5, device=DEV)
    got = ops.sample(x, half, top_p=torch.full((6,), nan, device=DEV), status=status)
    assert got.tolist() == [-1] * 6 and status.check()[0] == mk.MK_ERR_DEVICE


def test_sample_same_result_every_time():
    x = torch.randn((16, 151552), device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)).to(torch.bfloat16)
    u = torch.rand(16, device=DEV)
    p, k = torch.full((16,), 0.97, device=DEV), i32([0, 3000] * 8)
    lp0, lp = torch.zeros(16, device=DEV), torch.zeros(16, device=DEV)
    first = ops.sample(x, u, top_p=p, top_k=k, logprobs=lp0)
    for _ in range(20):
        again = ops.sample(x, u, top_p=p, top_k=k, logprobs=lp)
        assert torch.equal(first, again) and torch.equal(lp0, lp)


# --------------------------------------------- calls at the edge of the rules --

@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_attention_values_of_other_entries_do_not_leak(hd, dt):
    """Infinities and NaN that one entry sees stay with it: in its own tokens,
    whose tiles share rows with other entries, and in prefix tokens that a
    shorter member of the group does not reach."""
    g = gen(31)
    n, prefix, hkv, hq = 5, 192, 2, 4
    positions = [250, 300, 100, 199, 260]                # entry 2 ends inside the prefix
    width = 5
    table = torch.full((n, width), 0, dtype=torch.int32)
    nxt = 3
    for i in range(n):
        table[i, :3] = torch.arange(3)
        for page in range(3, width):
            table[i, page] = nxt
            nxt += 1
    kp, vp = (torch.randn((nxt, hkv, PAGE, hd), generator=g).to(TYPES[dt]) for _ in range(2))
    q = torch.randn((n, hq, hd), generator=g).to(TYPES[dt])
    clean = ops_oracle.attention(q, kp, vp, table, positions, [0, n], [prefix], hd ** -0.5)
    vp[int(table[0, 3]), 0, 5] = math.inf                # entry 0 sees it, in KV head 0
    kp[int(table[1, 4]), 1, 3] = math.nan                # entry 1 sees it, in KV head 1
    vp[2, 1, 10] = -math.inf                             # prefix token 138: all but entry 2 see it
    out = torch.full((n, hq, hd), 9.0, dtype=TYPES[dt], device=DEV)
    lse = torch.full((n, hq), 9.0, device=DEV)
    ops.prefix_attention(q.to(DEV), kp.to(DEV), vp.to(DEV), table.to(DEV), i32(positions), i32([0, n]),
                         i32([prefix]), out=out, lse=lse)
    got = out.cpu().float()
    assert not torch.isfinite(got[0, :2]).any()          # its own infinity
    assert torch.isnan(got[1, 2:]).all() and torch.isnan(lse.cpu()[1, 2:]).all()
    for b in (0, 1, 3, 4):
        assert not torch.isfinite(got[b, 2:]).any()      # the prefix's, in KV head 1
    # the others are as if nothing were there
    for b, heads in ((1, slice(0, 2)), (2, slice(0, 4)), (3, slice(0, 2)), (4, slice(0, 2))):
        o, s, mass, high = (x[b, heads] for x in clean)
        h = torch.finfo(TYPES[dt]).eps / 2
        tol = h * (mass + o.abs()) + (2e-5 * (1.0 + high))[..., None] * mass + 1e-7
        assert ((got[b, heads].double() - o).abs() <= tol).all()
        assert ((lse.cpu()[b, heads].double() - s).abs() <= 2e-5 * (1.0 + high)).all()


def test_attention_full_rows_and_largest_batch():
    # the last token of a row that has no page to spare
    attention_case(32, [2], [128], [191, 150], 4, 2, 64, "bf16")
    g = gen(33)
    kp, vp = (torch.randn((6, 2, PAGE, 64), generator=g).to(torch.bfloat16) for _ in range(2))
    q = torch.randn((2, 4, 64), generator=g).to(torch.bfloat16)
    table = torch.tensor([[4, 0, 2], [1, 5, 3]], dtype=torch.int32)
    out, lse = torch.full((2, 4, 64), 9.0, dtype=torch.bfloat16, device=DEV), torch.full((2, 4), 9.0, device=DEV)
    status = ops.Status(DEV)
    ops.prefix_attention(q.to(DEV), kp.to(DEV), vp.to(DEV), table.to(DEV), i32([191, 191]), i32([0, 2]), i32([100]),
                         out=out, lse=lse, status=status)
    status.check_ok()
    # tokens behind the prefix come from the entry's own row
    check_attention(out, lse, ops_oracle.attention(q, kp, vp, table, [191, 191], [0, 2], [100], 0.125), "bf16")
    n = 4096
    attention_case(34, [1] * n, [0] * n, [(i * 7) % 5 for i in range(n)], 1, 1, 64, "bf16")
    attention_case(35, [40] + [0] * 4000 + [3], [70] + [0] * 4000 + [5], [70 + i for i in range(40)] + [5, 4, 9],
                   8, 2, 64, "bf16")


@pytest.mark.parametrize("members,prefix", [(3, 0), (40, 130), (70, 200)])
def test_attention_many_heads_over_many_blocks(members, prefix):
    # one KV head per query head and eight of them: chunks of entries at every place of the line
    attention_case(members + prefix, [members, 2], [prefix, 64],
                   [prefix + (i * 37) % 300 for i in range(members)] + [64, 400], 16, 8, 64, "fp16")


def test_a_step_of_all_three_captured_and_replayed():
    """Append, attend and sample as a decode loop would, captured twice on a side
    stream (two graphs alive at once) and replayed in turn with other inputs."""
    hq, hkv, hd, b, vocab = 4, 2, 64, 3, 500
    freq, _ = ops.rope_frequencies(hd, device=DEV)
    table = i32([[0, 1], [2, 3], [4, 5]])
    proj = torch.randn((vocab, hq * hd), generator=gen(50)).to(DEV)

    def state(seed):
        g = gen(seed)
        s = dict(qkv=torch.randn((b, hq + 2 * hkv, hd), generator=g).to(DEV),
                 kp=torch.randn((6, hkv, PAGE, hd), generator=g).to(torch.bfloat16).to(DEV),
                 vp=torch.randn((6, hkv, PAGE, hd), generator=g).to(torch.bfloat16).to(DEV),
                 pos=i32([70, 5, 127]), u=torch.rand(b, generator=g).to(DEV), tokens=i32([-9] * b),
                 out=torch.zeros((b, hq, hd), dtype=torch.bfloat16, device=DEV))
        s["q"] = torch.zeros_like(s["out"])
        return s

    def step(s):
        ops.rope_append(s["qkv"][:, :hq], s["qkv"][:, hq:hq + hkv], s["qkv"][:, hq + hkv:], s["pos"], table, s["kp"],
                        s["vp"], freq, q_out=s["q"])
        ops.prefix_attention(s["q"], s["kp"], s["vp"], table, s["pos"], i32_start, i32_prefix, out=s["out"])
        logits = s["out"].view(b, -1).float() @ proj.t()
        ops.sample(logits, s["u"], tokens=s["tokens"], top_k=topk)
        return logits

    i32_start, i32_prefix, topk = i32([0, 1, 2, 3]), i32([0, 0, 0]), i32([50] * b)
    graphs = []
    for seed in (41, 42):
        s = state(seed)
        step(s)
        torch.cuda.synchronize()
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=side):
            logits = step(s)
        graphs.append((graph, s, logits))
    for turn in range(3):
        for n, (graph, s, logits) in enumerate(graphs):
            fresh = state(100 + 10 * turn + n)
            for k in ("qkv", "kp", "vp", "u"):
                s[k].copy_(fresh[k])
            s["pos"].copy_(i32([turn, 64 + turn, 100 - turn]))
            fresh["pos"].copy_(s["pos"])
            graph.replay()
            want = step(fresh)
            torch.cuda.synchronize()
            for k in ("kp", "vp", "q", "out", "tokens"):
                assert torch.equal(s[k], fresh[k]), (turn, n, k)
            assert torch.equal(logits, want)


def test_streams_are_waited_for():
    """Each operator on a side stream, behind work of that stream that makes its
    inputs: launches overlap the kernel ahead but not its results."""
    side = torch.cuda.Stream()
    freq, _ = ops.rope_frequencies(64, device=DEV)
    big = torch.randn((4096, 4096), device=DEV)
    k_src = torch.randn((40, 1, 64), device=DEV)
    table = i32([[0]])
    positions, seq = torch.arange(40, dtype=torch.int32, device=DEV), torch.zeros(40, dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    results = []
    for stream in (None, side):
        with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream()):
            k = torch.zeros_like(k_src)
            kp, vp = (torch.zeros((1, 1, PAGE, 64), dtype=torch.bfloat16, device=DEV) for _ in range(2))
            for _ in range(3):
                big @ big
            k.copy_(k_src)
            q = ops.rope_append(k, k, k, positions, table, kp, vp, freq, seq=seq, stream=stream)
            o = ops.prefix_attention(q[39:], kp, vp, table, positions[39:], seq[:2].clone() + i32([0, 1]),
                                     seq[:1], stream=stream)
            t = ops.sample(o.view(1, -1), torch.full((1,), 0.5, device=DEV), stream=stream)
        torch.cuda.synchronize()
        results.append((q, kp, vp, o, t))
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_sample_small_batches_and_wide_rows():
    # rows spread over the most blocks, and those that just are not
    r = np.random.default_rng(14)
    for b, v in ((1, 151552), (2, 16384), (2, 16385), (7, 40000), (8, 40000), (1, mk.MK_SAMPLE_MAX_VOCAB)):
        x = 2.5 * r.standard_normal((b, v))
        sample_case(x, r.random(b))
        sample_case(x, r.random(b), p=[0.9] * b)
        sample_case(x, r.random(b), k=[300] * b, p=[0.95] * b)
        sample_case(x, r.random(b), k=[700] * b)
        sample_case(x, r.random(b), p=[0.95] * b, m=[0.01] * b, temperature=[1.5] * b)


def test_sample_top_p_where_the_weights_lie_flat():
    # the cut among thousands of nearly equal logits, at every level of narrowing
    r = np.random.default_rng(15)
    x = np.concatenate((1e-3 * r.standard_normal((4, 30000)), 1e-6 * r.standard_normal((4, 30000)) + 0.5), axis=1)
    for p in (0.05, 0.3, 0.62, 0.9, 0.999):
        sample_case(x, r.random(4), p=[p] * 4)
    sample_case(x.astype(np.float16), r.random(4), p=[0.6] * 4, dt="fp16")


@pytest.mark.parametrize("b,v", [(2, 40000), (9, 40000), (3, 5000)])
def test_sample_over_clusters_captured(b, v):
    # clusters of 16, 8 and 4 blocks; two graphs alive, replayed with other inputs
    g = gen(60 + b)
    graphs = []
    for _ in range(2):
        s = dict(x=torch.randn((b, v), generator=g).to(DEV), u=torch.rand(b, generator=g).to(DEV),
                 p=torch.full((b,), 0.9, device=DEV), k=i32([0, 40, 600] * 3)[:b], t=i32([-9] * b))
        kw = dict(top_p=s["p"], top_k=s["k"])
        ops.sample(s["x"], s["u"], **kw)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ops.sample(s["x"], s["u"], tokens=s["t"], **kw)
        graphs.append((graph, s, kw))
    for _ in range(3):
        for graph, s, kw in graphs:
            s["x"].copy_(torch.randn((b, v), generator=g))
            s["u"].copy_(torch.rand(b, generator=g))
            graph.replay()
            assert torch.equal(s["t"], ops.sample(s["x"], s["u"], **kw))
