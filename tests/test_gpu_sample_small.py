"""Sampling from vocabularies of a few thousand tokens, where a few likely tokens
carry most of the weight: every rule, type and size of batch against the 64-bit
definition (tokens equal; a log-probability is a 64-bit value rounded once)."""

import numpy as np
import pytest
import torch

from moe_persistent_cta_b200 import ops
from tests import ops_oracle

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.mark.parametrize("dt", sorted(TYPES))
@pytest.mark.parametrize("rule", ["none", "k", "p", "min", "mixed"])
@pytest.mark.parametrize("b,v", [(42, 1473), (17, 1007), (8, 2191), (5, 4099), (3, 12463)])
def test_sample_small_vocabularies(b, v, rule, dt):
    g = torch.Generator().manual_seed(v + b)
    x = torch.randn((b, v), generator=g) * 2.5
    likely = torch.stack([torch.randperm(v, generator=g)[:40] for _ in range(b)])   # no token twice
    x.scatter_(1, likely, 8.0 + 3.0 * torch.randn((b, 40), generator=g))
    x = x.to(TYPES[dt])
    t = 0.6 + 0.6 * torch.rand(b, generator=g)
    k = torch.randint(1, 200, (b,), generator=g).to(torch.int32)
    p, m = 0.8 + 0.19 * torch.rand(b, generator=g), 0.02 + 0.1 * torch.rand(b, generator=g)
    u = torch.rand(b, generator=g)
    pick = torch.arange(b) % 4
    if rule == "mixed":
        k[(pick == 1) | (pick == 2)], p[pick == 2], m[pick < 2] = 0, 1.0, 0.0
    kw = dict(temperature=t)
    kw.update({"none": {}, "k": dict(top_k=k), "p": dict(top_p=p), "min": dict(min_p=m),
               "mixed": dict(top_k=k, top_p=p, min_p=m)}[rule])
    lp = torch.zeros(b, device=DEV)
    got = ops.sample(x.to(DEV), u.to(DEV), logprobs=lp, **{n: a.to(DEV) for n, a in kw.items()}).cpu()
    for i in range(b):
        of = lambda n, other: kw[n][i].item() if n in kw else other  # noqa: E731
        token, want = ops_oracle.sample(x[i].double().numpy(), float(u[i]), of("temperature", 1.0), of("top_k", 0),
                                        of("top_p", 1.0), of("min_p", 0.0))
        assert int(got[i]) == token, i
        # half a step of 32 bits, and the 64-bit sums' own rounding
        assert abs(float(lp[i]) - want) <= 2.0 ** -24 * abs(want) * (1 + 2.0 ** -20) + 1e-13 and np.isfinite(want)
