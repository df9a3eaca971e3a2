"""How the decode loop's shared and sampled steps are called on the GPU: captures,
arguments that do not fit the schedule, faults outside a step, other streams."""

import numpy as np
import pytest
import torch

import oracle
from moe_persistent_cta_b200 import configs, engine, mk, ops, serving, synth
from tests.gpu_common import MAX_ABS, REL_L2, TinyRig, compare_logits, to_dev
from tests.oracle_io import array_kv, array_weights, oracle_shape
from tests.test_gpu_shared import DEV, i32, shared_rig, shared_step

pytestmark = pytest.mark.gpu


def test_steps_refuse_a_capture():
    r, start, ends = shared_rig([100, 90], [2], [64])
    try:
        ref = r.oracle_step()
        args = (r.i32(r.tokens), r.i32(r.lens), r.table.to(DEV), r.i32(r.lens))
        out, u = torch.zeros((1, 2), dtype=torch.int32, device=DEV), torch.rand((1, 2), device=DEV)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for call in (lambda: r.dec.step_shared(*args, start, ends, r.logits),
                         lambda: r.dec.sample(1, *args, r.logits, out, u),
                         lambda: r.dec.sample(1, *args, r.logits, out, u, group_start=start, prefix_lens=ends)):
                with pytest.raises(mk.MKError) as e:
                    call()
                assert e.value.status == mk.MK_ERR_STATE
            out.fill_(5)
        graph.replay()
        err, rel = compare_logits(shared_step(r, start, ends), ref)
        assert err <= MAX_ABS and rel <= REL_L2 and (out == 5).all()
    finally:
        r.close()


@pytest.mark.parametrize("grouped", [False, True])
def test_sampled_steps_refuse_prefill_groups(grouped):
    # two prompt tokens of one sequence: their rows would go on as two sequences
    r = TinyRig(configs.TINY, [100, 100], seed=5)
    try:
        apart = r.table.clone()
        r.table[1] = r.table[0]
        kw = dict(group_start=i32([0, 2]), prefix_lens=i32([64])) if grouped else {}
        out, u = torch.zeros((1, 2), dtype=torch.int32, device=DEV), torch.rand((1, 2), device=DEV)
        r.dec.sample(1, r.i32(r.tokens), r.i32([100, 101]), r.table.to(DEV), r.i32([100, 100]), r.logits, out, u, **kw)
        rc, d = r.dec.check()
        assert rc == mk.MK_ERR_DEVICE and d[1:5] == [mk.MK_OP_SAMPLE, 1, 101, 100]
        r.dec.sample(1, r.i32(r.tokens), r.i32([100, 100]), apart.to(DEV), r.i32([100, 100]), r.logits, out, u, **kw)
        r.dec.check_ok()
    finally:
        r.close()


def test_faults_of_append_kv_reach_the_decoder():
    shape = configs.TINY
    L, hkv, hd = shape["n_layers"], shape["n_kv_heads"], shape["head_dim"]
    r = TinyRig(shape, [100], seed=6)
    try:
        k = torch.randn((3, hkv, hd), device=DEV)
        table, seq = r.table.to(DEV), i32([0, 0, 0])
        r.dec.append_kv(0, k, k, i32([100, 101, 102]), table, seq=seq)
        r.dec.check_ok()
        limit = r.table.shape[1] * 64
        # a position behind the table, a page of the pool that is not there
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(50_000_000)
        r.dec.append_kv(1, k, k, i32([100, limit, 102]), table, seq=seq, stream=side)
        rc, d = r.dec.check()
        assert rc == mk.MK_ERR_DEVICE and d == [rc, mk.MK_OP_ROPE_APPEND, 1, limit, limit, 0, 0, 0]
        r.dec.check_ok()
        bad = table.clone()
        bad[0, 1] = r.n_pages
        r.dec.append_kv(1, k, k, i32([1, 2, 100]), bad, seq=seq)
        with pytest.raises(mk.MKError) as e:
            r.dec.check_ok()
        assert e.value.detail[1:5] == [mk.MK_OP_ROPE_APPEND, 2, r.n_pages, r.n_pages]
        # a status of the caller's keeps it from the decoder
        own = ops.Status(DEV)
        r.dec.append_kv(1, k, k, i32([1, 2, 100]), bad, seq=seq, status=own)
        r.dec.check_ok()
        assert own.check()[0] == mk.MK_ERR_DEVICE
        # a fault of a step comes first, then that of the append
        r.dec.append_kv(1, k, k, i32([1, 2, 100]), bad, seq=seq)
        r.dec.step(r.i32(r.tokens), r.i32([100]), bad, r.i32([100]), r.logits)
        rc, d = r.dec.check()
        assert rc == mk.MK_ERR_DEVICE
        rc, d = r.dec.check()
        assert rc == mk.MK_ERR_DEVICE and d[1] == mk.MK_OP_ROPE_APPEND
        ref = r.oracle_step()
        r.kd.copy_(r.k)
        r.vd.copy_(r.v)
        err, rel = compare_logits(r.step(), ref)
        assert err <= MAX_ABS and rel <= REL_L2
    finally:
        r.close()


def test_continuous_batching_on_another_stream_than_the_current_one():
    """What the run makes for itself is made on its stream: a current stream that
    is behind its work neither delays the rules nor clears the tokens late."""
    shape = configs.TINY
    slots, steps, max_pages = 3, 12, 8
    W = to_dev(synth.make_weights(shape, 0, "cpu"), DEV)
    kshape = (shape["n_layers"], 3 * slots * max_pages, shape["n_kv_heads"], 64, shape["head_dim"])
    common = dict(slots=slots, steps=steps, seed=21, start_lo=5, start_hi=250, mean_new=6, max_new=steps,
                  max_pages_per_seq=max_pages, sampling=dict(temperature=2.0, top_k=40, top_p=0.95, min_p=0.001))
    runs = []
    side = torch.cuda.Stream()
    for stream in (None, side, side):
        k, v = (torch.zeros(kshape, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        dec = engine.Decoder(shape, W, k, v, max_batch=slots)
        try:
            torch.cuda.synchronize()
            if stream is not None:
                torch.cuda._sleep(400_000_000)
            runs.append(serving.run_continuous(dec, shape, k, v, stream=stream, **common)["tokens"])
            torch.cuda.synchronize()
        finally:
            dec.close()
    assert np.array_equal(runs[0], runs[1]) and np.array_equal(runs[0], runs[2])


@pytest.mark.parametrize("prompt_len", [128, 150, 20])
def test_samples_of_one_prompt_by_fused_and_by_shared_steps(prompt_len):
    """Either kind of step draws from the oracle's logits; the kind is the one asked
    for, or the faster one, or the one that the schedule's plan allows."""
    shape = configs.TINY
    n, max_pages, n_pages = 3, 6, 40
    L, hkv, hd = shape["n_layers"], shape["n_kv_heads"], shape["head_dim"]
    W = synth.make_weights(shape, 0, "cpu")
    g = torch.Generator().manual_seed(4)
    kc, vc = (torch.randn((L, n_pages, hkv, 64, hd), generator=g).to(torch.bfloat16) for _ in range(2))
    k, v = kc.to(DEV), vc.to(DEV)
    dec = engine.Decoder(shape, to_dev(W, DEV), k, v, max_batch=n)
    first = [3, 700, 41]
    took, sample = [], dec.sample
    dec.sample = lambda *a, **kw: (took.append("group_start" in kw), sample(*a, **kw))
    try:
        pool = serving.PagePool(n_pages)
        pages = pool.alloc(serving.pages_for(prompt_len))
        rows = np.full((n, max_pages), -1, dtype=np.int32)
        for i in range(n):                               # the oracle's own copies of the prompt
            rows[i, :len(pages)] = pages
        rows[:, len(pages)] = [30, 31, 32]
        if prompt_len % 64:
            for i in range(n):
                rows[i, len(pages) - 1] = 33 + i
                kc[:, 33 + i], vc[:, 33 + i] = kc[:, pages[-1]], vc[:, pages[-1]]
        ref = oracle.decode_step(oracle_shape(shape), array_weights(W), array_kv(kc, vc), first, [prompt_len] * n, rows)
        dec.build_schedule([prompt_len] * n, max_pages)
        common = dict(max_pages_per_seq=max_pages, seed=2, sampling=dict(temperature=1.3))
        for shared in (None, False, True):
            r = serving.sample_prompt(dec, k, v, pool, pages, prompt_len, first, 1, shared=shared, **common)
            err, rel = compare_logits(r["logits"].cpu().double().numpy(), ref)
            assert err <= MAX_ABS and rel <= REL_L2, (shared, err, rel)
        assert took == [False, False, True]
        # steps past the plan: shared ones alone can
        free, steps = pool.free_count(), 66
        with pytest.raises(ValueError):
            serving.sample_prompt(dec, k, v, pool, pages, prompt_len, first, steps, shared=False, **common)
        r = serving.sample_prompt(dec, k, v, pool, pages, prompt_len, first, steps, **common)
        assert took[-1] and ((r["tokens"] >= 0) & (r["tokens"] < shape["vocab"])).all()
        assert pool.free_count() == free
        dec.build_schedule([prompt_len] * n, max_pages, plan_len=[64 * max_pages - 1] * n)
        r = serving.sample_prompt(dec, k, v, pool, pages, prompt_len, first, steps, **common)
        assert not took[-1] and ((r["tokens"] >= 0) & (r["tokens"] < shape["vocab"])).all()
    finally:
        dec.close()


def test_append_kv_first_called_in_a_capture():
    shape = configs.TINY
    hkv, hd = shape["n_kv_heads"], shape["head_dim"]
    r = TinyRig(shape, [100], seed=6)
    try:
        k = torch.randn((3, hkv, hd), device=DEV, generator=torch.Generator(device=DEV).manual_seed(1))
        table, seq, pos = r.table.to(DEV), i32([0, 0, 0]), i32([100, 101, 102])
        ops.rope_append(None, k, k, pos, table, r.kd[0].clone(), r.vd[0].clone(), ops.rope_frequencies(hd)[0], seq=seq)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            r.dec.append_kv(1, k, k, pos, table, seq=seq)
        want_k, want_v = r.kd[1].clone(), r.vd[1].clone()
        graph.replay()
        r.dec.check_ok()
        ops.rope_append(None, k, k, pos, table, want_k, want_v, ops.rope_frequencies(hd)[0], seq=seq)
        assert torch.equal(r.kd[1], want_k) and torch.equal(r.vd[1], want_v)
        pos.copy_(i32([100, -5, 102]))                   # a replayed call's fault reaches the decoder too
        graph.replay()
        rc, d = r.dec.check()
        assert rc == mk.MK_ERR_DEVICE and d[1:4] == [mk.MK_OP_ROPE_APPEND, 1, -5]
        r.dec.check_ok()
    finally:
        r.close()


def test_logits_of_sample_prompt_outlive_their_release():
    """Logits that the current stream still reads are not written by the next call
    on the samples' stream."""
    shape = configs.TINY
    n, max_pages, n_pages = 3, 6, 40
    kshape = (shape["n_layers"], n_pages, shape["n_kv_heads"], 64, shape["head_dim"])
    g = torch.Generator().manual_seed(9)
    k, v = (torch.randn(kshape, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    dec = engine.Decoder(shape, to_dev(synth.make_weights(shape, 0, "cpu"), DEV), k, v, max_batch=n)
    try:
        dec.build_schedule([100] * n, max_pages)
        pool, side = serving.PagePool(n_pages), torch.cuda.Stream()
        pages = pool.alloc(2)
        run = lambda first: serving.sample_prompt(dec, k, v, pool, pages, 100, first, 1, max_pages_per_seq=max_pages,  # noqa: E731
                                                  stream=side)
        torch.cuda.synchronize()
        want, other = run([3, 700, 41])["logits"].clone(), run([5, 6, 7])["logits"].clone()
        kept = torch.empty_like(want)
        torch.cuda.synchronize()
        with torch.cuda.stream(torch.cuda.Stream()):     # the library's status copy waits for the default one
            logits = run([3, 700, 41])["logits"]
            at = logits.data_ptr()
            torch.cuda._sleep(400_000_000)
            kept.copy_(logits)
            del logits
            again = run([5, 6, 7])["logits"]
            assert again.data_ptr() != at
        torch.cuda.synchronize()
        assert torch.equal(kept, want) and torch.equal(again, other) and not torch.equal(want, other)
    finally:
        dec.close()
