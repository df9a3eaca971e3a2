"""The serving operators inside the decode loop on the GPU (tiny model): steps
that read shared prefixes once, sampled steps, several samples of one prompt and
prompts handed over in one piece, against the 64-bit oracle and one another."""

import numpy as np
import pytest
import torch

import oracle
from moe_persistent_cta_b200 import configs, engine, mk, ops, serving, synth
from tests import ops_oracle
from tests.gpu_common import MAX_ABS, REL_L2, TinyRig, compare_logits, to_dev
from tests.oracle_io import array_kv, array_weights, oracle_shape

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device=DEV)


def shared_rig(lens, groups, prefix, seed=3):
    """A rig whose entries of a group name the same pages for the whole pages of
    their prefix; groups: entries per group, prefix: tokens per group."""
    r = TinyRig(configs.TINY, lens, seed=seed)
    at = 0
    for n, p in zip(groups, prefix):
        for b in range(at + 1, at + n):
            r.table[b, :p // 64] = r.table[at, :p // 64]
        at += n
    start = np.concatenate(([0], np.cumsum(groups)))
    return r, i32(start), i32(prefix)


def shared_step(r, start, prefix, tokens=None, lens=None):
    tokens = r.tokens if tokens is None else tokens
    lens = r.lens if lens is None else lens
    r.dec.step_shared(r.i32(tokens), r.i32(lens), r.table.to(DEV), r.i32(lens), start, prefix, r.logits)
    r.dec.check_ok()
    return r.logits.cpu().double().numpy()


@pytest.mark.parametrize("lens,groups,prefix", [
    ([200, 130, 300, 64], [3, 1], [128, 64]),
    ([5], [1], [0]),
    ([0, 1, 700], [1, 1, 1], [0, 0, 512]),
    ([640, 650, 641, 777, 640, 900, 703, 648], [8], [640]),
])
def test_shared_step_matches_the_oracle(lens, groups, prefix):
    r, start, ends = shared_rig(lens, groups, prefix)
    try:
        ref = r.oracle_step()
        got = shared_step(r, start, ends)
        err, rel = compare_logits(got, ref)
        assert err <= MAX_ABS and rel <= REL_L2, (err, rel)
    finally:
        r.close()


def test_shared_and_fused_steps_alternate():
    # both count on the same counters and append to the same cache
    lens = [190, 200, 129]
    r, start, ends = shared_rig(lens, [3], [128])
    try:
        kv = array_kv(r.k, r.v)
        S, W = oracle_shape(r.shape), array_weights(r.W)
        tokens = list(r.tokens)
        for step in range(6):
            ref = oracle.decode_step(S, W, kv, tokens, lens, r.table.numpy())
            got = shared_step(r, start, ends, tokens, lens) if step % 2 else r.step(tokens, lens)
            err, rel = compare_logits(got, ref)
            assert err <= MAX_ABS and rel <= REL_L2, (step, err, rel)
            kv = array_kv(r.kd.cpu(), r.vd.cpu())
            tokens = [int(t) for t in got.argmax(-1)]
            lens = [n + 1 for n in lens]
    finally:
        r.close()


def test_shared_step_with_a_prefill_group():
    # three prompt tokens of one sequence as consecutive entries, and a fourth sequence
    lens = [100, 100, 100, 70]
    r = TinyRig(configs.TINY, lens, seed=5)
    try:
        r.table[1], r.table[2] = r.table[0], r.table[0]
        pos = [100, 101, 102, 70]
        args = (r.i32(r.tokens), r.i32(pos), r.table.to(DEV), r.i32(lens))
        r.dec.step(*args, r.logits)
        r.dec.check_ok()
        want = r.logits.cpu().double().numpy()
        r.kd.copy_(r.k)
        r.vd.copy_(r.v)
        r.dec.step_shared(*args, i32([0, 3, 4]), i32([100, 0]), r.logits)
        r.dec.check_ok()
        err, rel = compare_logits(r.logits.cpu().double().numpy(), want)
        assert err <= MAX_ABS and rel <= REL_L2, (err, rel)
    finally:
        r.close()


def test_shared_step_faults():
    r, start, ends = shared_rig([100, 90], [2], [64])
    try:
        ref = r.oracle_step()
        # an entry of no group is a fault; so is a page out of range; both leave the context usable
        r.dec.step_shared(r.i32(r.tokens), r.i32(r.lens), r.table.to(DEV), r.i32(r.lens), i32([0, 1]), i32([64]),
                          r.logits)
        rc, d = r.dec.check()
        assert rc == mk.MK_ERR_DEVICE and d[1] == mk.MK_OP_PREFIX_ATTENTION and d[2] == 1
        bad = r.table.clone()
        bad[1, 1] = r.n_pages
        r.dec.step_shared(r.i32(r.tokens), r.i32(r.lens), bad.to(DEV), r.i32(r.lens), start, ends, r.logits)
        rc, d = r.dec.check()
        assert rc == mk.MK_ERR_DEVICE and d[3] == r.n_pages
        for args in ((i32([0, 2]), i32([])), (i32([0]), i32([64])), (i32([0, 1, 2, 2]), i32([0, 0, 0]))):
            with pytest.raises(ValueError):
                shared_step(r, *args)
        r.kd.copy_(r.k)
        r.vd.copy_(r.v)
        err, rel = compare_logits(shared_step(r, start, ends), ref)
        assert err <= MAX_ABS and rel <= REL_L2
    finally:
        r.close()


RULES = dict(temperature=0.8, top_k=50, top_p=0.9, min_p=0.02)


@pytest.mark.parametrize("groups", [None, ([4], [128])])
def test_sampled_steps_follow_the_logits(groups):
    """Every step's tokens are those the 64-bit definition draws from the step's
    own logits, replayed one step at a time; the state moves on by one."""
    lens, steps = [130, 200, 140, 131], 5
    r, start, ends = shared_rig(lens, *(groups or ([4], [128])))
    kw = {} if groups is None else dict(group_start=start, prefix_lens=ends)
    rules = serving.sampling_rules(RULES, 4, DEV)
    u = torch.rand((steps, 4), generator=torch.Generator().manual_seed(1)).to(DEV)
    try:
        tok, pos = r.i32(r.tokens), r.i32(lens)
        out = torch.full((steps, 4), -7, dtype=torch.int32, device=DEV)
        lp = torch.zeros((steps, 4), device=DEV)
        r.dec.sample(steps, tok, pos, r.table.to(DEV), pos, r.logits, out, u, logprobs=lp, **kw, **rules)
        r.dec.check_ok()
        assert pos.tolist() == [n + steps for n in lens] and torch.equal(tok, out[-1])
        last = r.logits.clone()
        r.kd.copy_(r.k)
        r.vd.copy_(r.v)
        tokens, at = list(r.tokens), list(lens)
        for i in range(steps):
            x = shared_step(r, start, ends, tokens, at) if groups else r.step(tokens, at)
            x32 = x.astype(np.float32)
            assert (x32 == x).all()
            tokens = []
            for b in range(4):
                t, p = ops_oracle.sample(x32[b], float(u[i, b]), float(np.float32(0.8)), 50, float(np.float32(0.9)),
                                         float(np.float32(0.02)))
                assert int(out[i, b]) == t, (i, b)
                assert abs(float(lp[i, b]) - p) <= 2.0 ** -23 * abs(p) + 1e-14
                tokens.append(t)
            at = [n + 1 for n in at]
        assert torch.equal(last, r.logits)
        # separate position and length buffers both move on
        pos, ln = r.i32(lens), r.i32(lens)
        r.dec.sample(2, r.i32(r.tokens), pos, r.table.to(DEV), ln, r.logits, out, u, **kw)
        r.dec.check_ok()
        assert pos.tolist() == ln.tolist() == [n + 2 for n in lens]
    finally:
        r.close()


def test_one_token_kept_is_greedy_decoding():
    lens, steps = [70, 10], 6
    r = TinyRig(configs.TINY, lens, seed=9)
    try:
        outs = []
        for greedy in (True, False):
            r.kd.copy_(r.k)
            r.vd.copy_(r.v)
            tok, pos = r.i32(r.tokens), r.i32(lens)
            out = torch.full((steps, 2), -7, dtype=torch.int32, device=DEV)
            if greedy:
                r.dec.greedy(steps, tok, pos, r.table.to(DEV), pos, r.logits, out)
            else:
                r.dec.sample(steps, tok, pos, r.table.to(DEV), pos, r.logits, out,
                             torch.full((steps, 2), 0.7, device=DEV), top_k=i32([1, 1]))
            r.dec.check_ok()
            outs.append(out)
        assert torch.equal(*outs)
        bad = torch.full((1, 2), 1.5, device=DEV)          # a number outside [0, 1)
        r.dec.sample(1, r.i32(r.tokens), r.i32(lens), r.table.to(DEV), r.i32(lens), r.logits, out, bad)
        rc, d = r.dec.check()
        assert rc == mk.MK_ERR_DEVICE and d[1] == mk.MK_OP_SAMPLE and (out[0] == -1).all()
        for kw in (dict(top_k=i32([1])), dict(temperature=torch.ones(1, device=DEV)),
                   dict(group_start=i32([0, 2]))):
            with pytest.raises(ValueError):
                r.dec.sample(1, r.i32(r.tokens), r.i32(lens), r.table.to(DEV), r.i32(lens), r.logits, out,
                             torch.rand((1, 2), device=DEV), **kw)
    finally:
        r.close()


@pytest.mark.parametrize("prompt_len", [128, 150])
def test_samples_of_one_prompt(prompt_len):
    """append_kv hands the prompt over, sample_prompt draws from it: the tokens
    fed and drawn, put through the oracle on a cache of its own, give the same
    logits, and no page is lost."""
    shape = configs.TINY
    n, steps, max_pages, n_pages = 3, 4, 6, 40
    L, hkv, hd = shape["n_layers"], shape["n_kv_heads"], shape["head_dim"]
    W = synth.make_weights(shape, 0, "cpu")
    k = torch.zeros((L, n_pages, hkv, 64, hd), dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    dec = engine.Decoder(shape, to_dev(W, DEV), k, v, max_batch=n)
    pool = serving.PagePool(n_pages)
    pages = pool.alloc(serving.pages_for(prompt_len))
    g = torch.Generator().manual_seed(4)
    try:
        table = torch.full((1, max_pages), -1, dtype=torch.int32)
        table[0, :len(pages)] = torch.tensor(pages, dtype=torch.int32)
        freq, _ = ops.rope_frequencies(hd, shape.get("rope_theta", 1.0e4), device="cpu")
        pos = torch.arange(prompt_len, dtype=torch.int32)
        for l in range(L):
            kk, vv = (torch.randn((prompt_len, hkv, hd), generator=g) for _ in range(2))
            dec.append_kv(l, kk.to(DEV), vv.to(DEV), pos.to(DEV), table.to(DEV), seq=i32([0] * prompt_len))
            want, reach = ops_oracle.rotate(kk, pos, freq, False, 1.0)
            got = k[l].cpu()[pages].transpose(1, 2).reshape(-1, hkv, hd)[:prompt_len].double()
            assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + 8e-7 * reach + 1e-40).all()
        dec.build_schedule([prompt_len] * n, max_pages)
        kv0 = array_kv(k.cpu(), v.cpu())
        free = pool.free_count()
        first = [3, 700, 41]
        r = serving.sample_prompt(dec, k, v, pool, pages, prompt_len, first, steps, max_pages_per_seq=max_pages,
                                  seed=2, sampling=dict(temperature=1.3))
        assert pool.free_count() == free and ((r["tokens"] >= 0) & (r["tokens"] < shape["vocab"])).all()
        assert (r["logprobs"] < 0).all()
        own = pool.alloc(3 * (max_pages - prompt_len // 64))
        rows = np.full((n, max_pages), -1, dtype=np.int32)
        per = len(own) // 3
        kv = kv0
        for i in range(n):
            rows[i, :prompt_len // 64] = pages[:prompt_len // 64]
            rows[i, prompt_len // 64:] = own[i * per:(i + 1) * per]
        kc, vc = k.cpu(), v.cpu()
        if prompt_len % 64:
            for i in range(n):
                kc[:, rows[i, prompt_len // 64]] = kc[:, pages[-1]]
                vc[:, rows[i, prompt_len // 64]] = vc[:, pages[-1]]
        kd, vd = kc.to(DEV), vc.to(DEV)
        dec2 = engine.Decoder(shape, to_dev(W, DEV), kd, vd, max_batch=n)
        try:
            dec2.build_schedule([prompt_len] * n, max_pages)
            logits = torch.empty((n, shape["vocab"]), device=DEV)
            toks = first
            for i in range(steps):
                lens = [prompt_len + i] * n
                kv = array_kv(kd.cpu(), vd.cpu())
                dec2.step(i32(toks), i32(lens), torch.from_numpy(rows).to(DEV), i32(lens), logits)
                dec2.check_ok()
                last = toks
                toks = r["tokens"][i].tolist()
            ref = oracle.decode_step(oracle_shape(shape), array_weights(W), kv, last, lens, rows)
            err, rel = compare_logits(r["logits"].cpu().double().numpy(), ref)
            assert err <= MAX_ABS and rel <= REL_L2, (err, rel)
        finally:
            dec2.close()
        pool.release(own)
    finally:
        dec.close()


def test_continuous_batching_with_sampling():
    shape = configs.TINY
    slots, steps, max_pages = 3, 30, 8
    W = synth.make_weights(shape, 0, "cpu")
    n_pages = 3 * slots * max_pages
    kshape = (shape["n_layers"], n_pages, shape["n_kv_heads"], 64, shape["head_dim"])
    common = dict(slots=slots, steps=steps, seed=21, start_lo=5, start_hi=250, mean_new=6, max_new=steps,
                  max_pages_per_seq=max_pages)
    runs = []
    for sampling in (dict(top_k=1), None, dict(temperature=2.0), dict(temperature=2.0)):
        k = torch.zeros(kshape, dtype=torch.bfloat16, device=DEV)
        v = torch.zeros_like(k)
        dec = engine.Decoder(shape, to_dev(W, DEV), k, v, max_batch=slots)
        try:
            runs.append(serving.run_continuous(dec, shape, k, v, sampling=sampling, **common)["tokens"])
        finally:
            dec.close()
    assert np.array_equal(runs[0], runs[1])          # one token kept: the greedy run
    assert np.array_equal(runs[2], runs[3]) and not np.array_equal(runs[1], runs[2])
    assert ((runs[2] >= 0) & (runs[2] < shape["vocab"])).all()
