"""Refusals of the decode loop's Python functions, without a GPU: tensors that do
not fit the schedule are refused before the library is called."""

import pytest
import torch

from moe_persistent_cta_b200 import engine, mk, serving

B, PAGES, V = 3, 4, 50


class OnDevice:
    """What the checks look at of a tensor on a device."""

    def __init__(self, *shape, dtype=torch.int32, device=0):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, device

    def get_device(self):
        return self.device

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096


class Stream:
    cuda_stream, device_index = 0, 0


def decoder():
    d = engine.Decoder.__new__(engine.Decoder)
    d.shape, d.batch, d.max_pages, d.device, d._ctx = dict(vocab=V), B, PAGES, 0, None
    d.planned = [64 * PAGES] * B
    return d


F32 = torch.float32


def inputs(**kw):
    d = dict(tokens=OnDevice(B), positions=OnDevice(B), page_table=OnDevice(B, PAGES), seq_lens=OnDevice(B),
             logits=OnDevice(B, V, dtype=F32), group_start=OnDevice(3), prefix_lens=OnDevice(2), stream=Stream())
    d.update(kw)
    return d


def sample_inputs(**kw):
    return inputs(n_steps=2, out_tokens=OnDevice(2, B), u=OnDevice(2, B, dtype=F32), **kw)


BAD_STEP = [
    (ValueError, dict(tokens=OnDevice(B - 1))), (ValueError, dict(positions=OnDevice(B - 1))),
    (ValueError, dict(seq_lens=OnDevice(1))), (ValueError, dict(page_table=OnDevice(B - 1, PAGES))),
    (ValueError, dict(page_table=OnDevice(B, PAGES + 1))), (ValueError, dict(logits=OnDevice(B, V - 1, dtype=F32))),
    (ValueError, dict(group_start=OnDevice(2))), (ValueError, dict(prefix_lens=OnDevice(0), group_start=OnDevice(1))),
    (ValueError, dict(prefix_lens=OnDevice(B + 1), group_start=OnDevice(B + 2))),
    (TypeError, dict(tokens=OnDevice(B, dtype=torch.int64))), (TypeError, dict(seq_lens=OnDevice(B, device=-1))),
    (TypeError, dict(positions=OnDevice(B, device=1))), (TypeError, dict(logits=OnDevice(B, V, dtype=torch.float16))),
    (TypeError, dict(page_table=OnDevice(B, PAGES, device=1))), (TypeError, dict(prefix_lens=OnDevice(2, device=1))),
]
BAD_SAMPLE = [
    (ValueError, dict(out_tokens=OnDevice(2 * B - 1))), (ValueError, dict(u=OnDevice(B, dtype=F32))),
    (ValueError, dict(temperature=OnDevice(B - 1, dtype=F32))), (ValueError, dict(logprobs=OnDevice(B, dtype=F32))),
    (ValueError, dict(group_start=None)), (TypeError, dict(top_k=OnDevice(B, dtype=F32))),
    (TypeError, dict(top_p=OnDevice(B, dtype=F32, device=1))), (TypeError, dict(out_tokens=OnDevice(2, B, device=1))),
]


@pytest.mark.parametrize("error,kw", BAD_STEP)
def test_step_shared_refusals(error, kw):
    with pytest.raises(error):
        decoder().step_shared(**inputs(**kw))


@pytest.mark.parametrize("error,kw", BAD_STEP + BAD_SAMPLE)
def test_sample_refusals(error, kw):
    with pytest.raises(error):
        decoder().sample(**{**sample_inputs(), **kw})


def test_streams_of_another_device_are_refused():
    other = Stream()
    other.device_index = 1
    with pytest.raises(ValueError):
        decoder().step_shared(**inputs(stream=other))
    with pytest.raises(ValueError):
        decoder().sample(**sample_inputs(stream=other))


def test_fitting_tensors_reach_the_library():
    # which has no context here
    for call in (lambda: decoder().step_shared(**inputs()), lambda: decoder().sample(**sample_inputs())):
        with pytest.raises(mk.MKError) as e:
            call()
        assert e.value.status == mk.MK_ERR_INVALID


@pytest.mark.parametrize("kw", [dict(tokens=[1, 2]), dict(tokens=[1, 2, 3, 4]), dict(tokens=[]), dict(steps=-1),
                                dict(prompt_len=-1), dict(prompt_len=129), dict(steps=64 * PAGES - 63)])
def test_sample_prompt_refusals(kw):
    # samples that are not the schedule's, a prompt longer than its pages, more tokens than the table
    # holds; the pool keeps its pages
    pool = serving.PagePool(20)
    pages = pool.alloc(2)
    k = torch.zeros((1, 20, 1, 64, 64), dtype=torch.bfloat16)
    args = dict(prompt_len=64, tokens=[1, 2, 3], steps=2)
    args.update(kw)
    with pytest.raises(ValueError):
        serving.sample_prompt(decoder(), k, k, pool, pages, max_pages_per_seq=PAGES, **args)
    assert pool.free_count() == 18


def test_shared_steps_where_they_save_more_than_they_cost():
    d = decoder()
    d.shape.update(n_kv_heads=4, head_dim=128)           # 2048 bytes a token and layer
    takes = lambda n, prefix, last=100, **kw: (setattr(d, "batch", n), setattr(d, "planned", [10 ** 6] * n),  # noqa: E731
                                               serving.takes_shared_steps(d, prefix, last, **kw))[2]
    # as measured: 8 samples from 16384 .. 32768 on, 4 from 32768 .. 65536 on, 2 not at 131072, 1 never
    assert [takes(8, p) for p in (0, 8192, 16384, 32768, 131072)] == [False, False, False, True, True]
    assert [takes(4, p) for p in (16384, 32768, 65536)] == [False, False, True]
    assert not takes(2, 131072) and not takes(1, 10 ** 7)
    assert takes(2, 64, shared=True) and not takes(8, 131072, shared=False)
    # fused steps cannot pass the schedule's plan
    d.batch, d.planned = 2, [200, 190]
    assert not serving.takes_shared_steps(d, 128, 190)
    assert serving.takes_shared_steps(d, 128, 191) and serving.takes_shared_steps(d, 128, 191, True)
    with pytest.raises(ValueError):
        serving.takes_shared_steps(d, 128, 191, False)
