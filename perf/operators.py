"""What the serving operators beside the decode step are measured on.

Three operators that a serving loop around the decode step needs when several
sequences continue one prompt:

* ``rope_append``: keys rotated and written, with their values, into the paged
  cache that the decode step reads; queries rotated on the way.
* ``prefix_attention``: attention of one query token per batch entry over the
  paged cache, groups of entries sharing a prefix whose pages are read once
  for the whole group.
* ``sample``: one token per row of logits by temperature, top-k, top-p and
  min-p from a given uniform number.

Sizes follow the 30B-MoE shape (16 query heads, 4 KV heads of 128, vocabulary
151552) and the tiny shape (4 and 2 heads of 64, vocabulary 1024).
"""

import math

import torch

own = False

PAGE = 64
VOCAB = 151552
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # -- appending to the cache ------------------------------------------
        # one decode step of 8 sequences: the projection's 32-bit rows
        dict(name="append step of 8", op="append", seqs=8, tokens=8, hq=16, hkv=4, hd=128, rot=128,
             interleaved=False, scaling="none", src="fp32", dst="bf16", past=8192),
        # a prompt computed outside the step, handed over in one piece
        dict(name="append prompt 8192", op="append", seqs=1, tokens=8192, hq=16, hkv=4, hd=128, rot=128,
             interleaved=False, scaling="none", src="bf16", dst="bf16", past=0),
        # a ragged batch of prompt pieces far into a stretched context, half of each head rotated
        dict(name="append ragged 16381", op="append", seqs=7, tokens=16381, hq=16, hkv=4, hd=128, rot=64,
             interleaved=True, scaling="parts", src="fp16", dst="fp16", past=200000),
        # small heads, a rotated part that no wide load fits, stretched evenly
        dict(name="append odd 333", op="append", seqs=3, tokens=333, hq=4, hkv=2, hd=64, rot=36,
             interleaved=False, scaling="even", src="bf16", dst="bf16", past=131),
        # -- attention over a shared prefix ----------------------------------
        # one decode step: 8 samples of an 8192-token prompt
        dict(name="attend 8 on 8192", op="attend", groups=1, batch=8, prefix=8192, suffix=128, hq=16, hkv=4,
             hd=128, type="bf16", causal=False),
        # a served system prompt: 61 sequences in 4 groups, lengths ragged, an idle row in the batch
        dict(name="attend 61 in 4 groups", op="attend", groups=4, batch=61, prefix=4999, suffix=777, hq=16,
             hkv=4, hd=64, type="fp16", causal=False),
        # many samples of a long document
        dict(name="attend 256 on 32768", op="attend", groups=1, batch=256, prefix=32768, suffix=300, hq=16,
             hkv=4, hd=128, type="bf16", causal=False),
        # a piece of a prompt against its cached past: one group, each query one token further
        dict(name="attend piece of 500", op="attend", groups=1, batch=500, prefix=12345, suffix=0, hq=16,
             hkv=4, hd=128, type="bf16", causal=True),
        # -- sampling ----------------------------------------------------------
        # one row of the tiny vocabulary: latency
        dict(name="sample 1 of 1024", op="sample", batch=1, vocab=1024, type="fp32", rule="k"),
        # one step of 8 sequences, the step's own logits, the usual mix of rules
        dict(name="sample 8 of 151552", op="sample", batch=8, vocab=VOCAB, type="fp32", rule="mixed"),
        # temperature alone: every token may be drawn
        dict(name="sample 33 untruncated", op="sample", batch=33, vocab=VOCAB - 11, type="bf16", rule="none"),
        # the largest batch
        dict(name="sample 256 of 151552", op="sample", batch=256, vocab=VOCAB, type="fp32", rule="mixed"),
    ]


def _span(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("append", "attend", "sample"))
    if op == "append":
        hkv, hd = rng.choice((1, 2, 4, 8)), rng.choice((64, 128))
        tokens = _span(rng, 1, 16000)
        return dict(op=op, seqs=min(tokens, _span(rng, 1, 64)), tokens=tokens, hq=hkv * rng.choice((1, 2, 3, 4)),
                    hkv=hkv, hd=hd, rot=rng.choice((hd, hd, hd // 2, 2 * rng.randint(1, hd // 2))),
                    interleaved=rng.random() < 0.5, scaling=rng.choice(("none", "even", "parts")),
                    src=rng.choice(("bf16", "fp16", "fp32")), dst=rng.choice(("bf16", "fp16")),
                    past=_span(rng, 1, 250000))
    if op == "attend":
        hkv, hd = rng.choice((1, 2, 4)), rng.choice((64, 128))
        causal = rng.random() < 0.25
        batch = _span(rng, 1, 400 if causal else 200)
        return dict(op=op, groups=1 if causal else min(batch, _span(rng, 1, 8)), batch=batch,
                    prefix=_span(rng, 1, 30000), suffix=0 if causal else _span(rng, 1, 1500),
                    hq=hkv * rng.choice((1, 2, 3, 4)), hkv=hkv, hd=hd, type=rng.choice(("bf16", "fp16")),
                    causal=causal)
    return dict(op=op, batch=_span(rng, 1, 200), vocab=_span(rng, 1000, 160000),
                type=rng.choice(("fp32", "bf16", "fp16")), rule=rng.choice(("none", "k", "p", "min", "mixed")))


# ------------------------------------------------------------------ inputs --

def _cut(total, parts, gen):
    """`total` split into `parts` whole numbers >= 1, as a list."""
    w = torch.rand(parts, generator=gen) + 0.2
    n = 1 + ((total - parts) * w / w.sum()).long()
    n[-1] += total - int(n.sum())
    return n.tolist()


def _inv_freq(rot, scaling, theta=1.0e4):
    """The angle of each rotated pair for one position, in 64 bits: as trained,
    slowed evenly by 8, or slowed by 8 only where a pair turns fewer than once
    (kept where it turns more than 32 times) over 4096 positions."""
    f = theta ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if scaling == "even":
        return f / 8.0
    if scaling == "parts":
        keep = ((4096.0 * f / (2.0 * math.pi) - 1.0) / 31.0).clamp(0.0, 1.0)
        return f * keep + f / 8.0 * (1.0 - keep)
    return f


def _prepare_append(c, gen, dev, cuda_gen):
    t, hq, hkv, hd = c["tokens"], c["hq"], c["hkv"], c["hd"]
    counts = _cut(t, c["seqs"], gen)
    starts = [int(x) for x in torch.randint(max(0, c["past"] - 50), c["past"] + 1, (c["seqs"],), generator=gen)]
    seq = torch.cat([torch.full((n,), i, dtype=torch.int32) for i, n in enumerate(counts)])
    pos = torch.cat([torch.arange(s, s + n, dtype=torch.int32) for s, n in zip(starts, counts)])
    first = [s // PAGE for s in starts]
    pages = [(s + n - 1) // PAGE + 1 for s, n in zip(starts, counts)]
    used = t // PAGE + 2 * c["seqs"]             # enough wherever the pieces start
    order = torch.randperm(used, generator=gen).to(torch.int32)
    table, at = torch.full((c["seqs"], max(pages)), -1, dtype=torch.int32), 0
    for i, (f, p) in enumerate(zip(first, pages)):
        table[i, f:p] = order[at:at + p - f]     # the pages before the piece are not looked at
        at += p - f
    src, dst = TYPES[c["src"]], TYPES[c["dst"]]
    # one row per token: query, key and value heads as the projection leaves them
    qkv = torch.randn((t, hq + 2 * hkv, hd), generator=cuda_gen, device=dev).to(src)
    pool = torch.randn((2, used, hkv, PAGE, hd), generator=cuda_gen, device=dev).to(dst)
    return dict(q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], seq=seq.to(dev), positions=pos.to(dev),
                table=table.to(dev), k_pool=pool[0], v_pool=pool[1],
                inv_freq=_inv_freq(c["rot"], c["scaling"]).to(dev),
                magnitude=1.0 if c["scaling"] != "parts" else 0.1 * math.log(8.0) + 1.0,
                q_out=torch.zeros((t, hq, hd), dtype=dst, device=dev))


def _prepare_attend(c, gen, dev, cuda_gen):
    b, n, hkv, hd = c["batch"], c["groups"], c["hkv"], c["hd"]
    members = _cut(b, n, gen)
    start = [0]
    for m in members:
        start.append(start[-1] + m)
    if c["causal"]:
        # queries of one sequence: entry i sees the past and the piece up to itself
        prefix = [c["prefix"] + b]
        pos = torch.arange(c["prefix"], c["prefix"] + b)
    else:
        prefix = [max(1, int(c["prefix"] * f)) for f in (1.0 - 0.5 * torch.rand(n, generator=gen)).tolist()]
        prefix[0] = c["prefix"]
        pos = torch.cat([p + torch.randint(0, c["suffix"], (m,), generator=gen) for p, m in zip(prefix, members)])
        if n > 1:
            pos[start[n] - 1] = -1               # an idle row: it sees nothing
    longest = int(pos.max()) + 1
    own_pages, rows = 0, []
    for g in range(n):
        shared = prefix[g] // PAGE if not c["causal"] else (longest + PAGE - 1) // PAGE
        rows.append((own_pages, shared))
        own_pages += shared
    table = torch.zeros((b, (longest + PAGE - 1) // PAGE), dtype=torch.int32)
    for g in range(n):
        at, shared = rows[g]
        for i in range(start[g], start[g + 1]):
            table[i, :shared] = torch.arange(at, at + shared)
            mine = max(0, (int(pos[i]) + PAGE) // PAGE - shared)
            if i == start[g] and not c["causal"]:
                mine = max(mine, (prefix[g] + PAGE - 1) // PAGE - shared)   # the prefix may end inside a page
            table[i, shared:shared + mine] = torch.arange(own_pages, own_pages + mine)
            own_pages += mine
    order = torch.randperm(own_pages, generator=gen).to(torch.int32)
    table = order[table.long().clamp(max=own_pages - 1)]
    dt = TYPES[c["type"]]
    pool = torch.randn((2, own_pages, hkv, PAGE, hd), generator=cuda_gen, device=dev, dtype=dt)
    q = torch.randn((b, c["hq"], hd), generator=cuda_gen, device=dev).mul_(1.5).to(dt)
    table = table.to(dev)
    # a prefix that ends inside a page: each member's own page holds the same first tokens
    for g in range(n):
        rest = prefix[g] % PAGE
        if rest and not c["causal"] and members[g] > 1:
            page = prefix[g] // PAGE
            mine = [i for i in range(start[g] + 1, start[g + 1]) if int(pos[i]) >= prefix[g]]
            if mine:
                to = table[torch.tensor(mine, device=dev), page].long()
                pool[:, to, :, :rest] = pool[:, table[start[g], page].long()][:, None, :, :rest]
    i32 = dict(dtype=torch.int32, device=dev)
    return dict(q=q, k_pool=pool[0], v_pool=pool[1], table=table, positions=pos.to(**i32),
                group_start=torch.tensor(start, **i32), prefix_lens=torch.tensor(prefix, **i32),
                members=max(members), longest_prefix=max(prefix), longest=longest, shortest_prefix=min(prefix),
                out=torch.zeros_like(q), lse=torch.zeros((b, c["hq"]), dtype=torch.float32, device=dev))


def _prepare_sample(c, gen, dev, cuda_gen):
    b, v = c["batch"], c["vocab"]
    # a language model's logits: a broad bulk and a few likely tokens, how few differing by row
    x = torch.randn((b, v), generator=cuda_gen, device=dev) * 2.5
    likely = torch.randint(0, v, (b, 40), generator=cuda_gen, device=dev)
    x.scatter_(1, likely, 8.0 + 3.0 * torch.randn((b, 40), generator=cuda_gen, device=dev))
    rule, rows = c["rule"], torch.arange(b)
    pick = rows % 4
    temperature = 0.6 + 0.6 * torch.rand(b, generator=gen)
    k = torch.randint(1, 200, (b,), generator=gen)
    p = 0.8 + 0.19 * torch.rand(b, generator=gen)
    m = 0.02 + 0.1 * torch.rand(b, generator=gen)
    use = {"none": (0, 0, 0), "k": (1, 0, 0), "p": (0, 1, 0), "min": (0, 0, 1), "mixed": (1, 1, 1)}[rule]
    if rule == "mixed":                          # k and p, p alone, min-p alone, all three
        k = torch.where((pick == 0) | (pick == 3), k, torch.zeros_like(k))
        p = torch.where(pick != 2, p, torch.ones_like(p))
        m = torch.where(pick >= 2, m, torch.zeros_like(m))
    f32 = dict(dtype=torch.float32, device=dev)
    return dict(logits=x.to(TYPES[c["type"]]), u=torch.rand(b, generator=gen).to(dev), temperature=temperature.to(**f32),
                top_k=k.to(dtype=torch.int32, device=dev) if use[0] else None, top_p=p.to(**f32) if use[1] else None,
                min_p=m.to(**f32) if use[2] else None, tokens=torch.zeros(b, dtype=torch.int32, device=dev),
                logprobs=torch.zeros(b, **f32))


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator().manual_seed(seed)
    cuda_gen = torch.Generator(device=dev).manual_seed(seed)
    make = {"append": _prepare_append, "attend": _prepare_attend, "sample": _prepare_sample}[case["op"]]
    return dict(make(case, gen, dev, cuda_gen), op=case["op"], case=dict(case))


# ------------------------------------------------------------- plain forms --

def _rotated(x, angle, interleaved, magnitude):
    rot = 2 * angle.shape[-1]
    cos, sin = (angle.cos() * magnitude).float()[:, None], (angle.sin() * magnitude).float()[:, None]
    y = x.float()
    part, rest = y[..., :rot], y[..., rot:]
    if interleaved:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, rest), -1)


def _plain_append(s):
    pos = s["positions"].long()
    angle = pos.double()[:, None] * s["inv_freq"]
    page = s["table"][s["seq"].long(), pos // PAGE].long()
    dt, il = s["k_pool"].dtype, s["case"]["interleaved"]
    s["q_out"].copy_(_rotated(s["q"], angle, il, s["magnitude"]).to(dt))
    s["k_pool"][page, :, pos % PAGE] = _rotated(s["k"], angle, il, s["magnitude"]).to(dt)
    s["v_pool"][page, :, pos % PAGE] = s["v"].float().to(dt)
    return {"q": s["q_out"], "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def _gather(pool, pages):
    """[..., pages] of a pool as [..., heads, tokens, head size] in 32 bits."""
    x = pool[pages.long()].transpose(-4, -3)
    return x.flatten(-3, -2).float()


def _plain_attend(s):
    c = s["case"]
    b, hq, hd = s["q"].shape
    hkv, start, prefix = c["hkv"], s["group_start"].long(), s["prefix_lens"].long()
    g, n, mm = hq // hkv, len(s["prefix_lens"]), s["members"]
    seen = s["positions"].long() + 1
    q = s["q"].float().view(b, hkv, g, hd) / math.sqrt(hd)
    # the shared part: every group's members against the group's keys
    member = start[:-1, None] + torch.arange(mm, device=q.device)
    real = member < start[1:, None]
    member = member.clamp(max=b - 1)
    np_ = (s["longest_prefix"] + PAGE - 1) // PAGE
    row = s["table"][start[:-1], :np_]
    kp, vp = _gather(s["k_pool"], row), _gather(s["v_pool"], row)
    qg = q[member].transpose(1, 2).flatten(2, 3)                      # [n, hkv, mm * g, hd]
    sp = qg @ kp.transpose(-1, -2)
    limit = torch.minimum(seen[member], prefix[:, None]).repeat_interleave(g, 1)[:, None, :, None]
    sp.masked_fill_(torch.arange(np_ * PAGE, device=q.device) >= limit, -math.inf)
    mp = sp.amax(-1, keepdim=True).clamp(min=-3e38)
    sp.sub_(mp).exp_()
    lp, op = sp.sum(-1, keepdim=True), sp @ vp
    back = lambda x: x.view(n, hkv, mm, g, -1).transpose(1, 2)[real]  # noqa: E731  rows in batch order
    mp, lp, op = back(mp.expand_as(lp)), back(lp), back(op)
    # what each member has of its own
    p0 = s["shortest_prefix"] // PAGE
    rest = s["table"][:, p0:]
    if rest.shape[1] and not c["causal"]:
        mine = torch.repeat_interleave(prefix, start.diff())
        ks, vs = _gather(s["k_pool"], rest), _gather(s["v_pool"], rest)
        ss = q @ ks.transpose(-1, -2)
        token = p0 * PAGE + torch.arange(rest.shape[1] * PAGE, device=q.device)
        ss.masked_fill_(((token < mine[:, None]) | (token >= seen[:, None]))[:, None, None], -math.inf)
        m = torch.maximum(mp, ss.amax(-1, keepdim=True))
        ss.sub_(m).exp_()
        f = (mp - m).exp()
        l, o = lp * f + ss.sum(-1, keepdim=True), op * f + ss @ vs
    else:
        m, l, o = mp, lp, op
    out = torch.where(l > 0, o / l, 0.0)
    lse = torch.where(l > 0, m + l.log(), -math.inf)
    return {"out": out.view(b, hq, hd).to(s["q"].dtype), "lse": lse.view(b, hq)}


def _plain_sample(s):
    x = s["logits"].double() + 0.0
    b, v = x.shape
    w = ((x - x.amax(-1, keepdim=True)) / s["temperature"].double()[:, None]).exp()
    keep = torch.ones_like(w, dtype=torch.bool)
    if s["top_k"] is not None or s["top_p"] is not None:
        order = x.sort(dim=-1, descending=True, stable=True).indices    # equal logits: the lowest token first
        ws = w.gather(1, order)
        ks = torch.ones_like(keep)
        if s["top_k"] is not None:
            k = s["top_k"][:, None]
            ks = (torch.arange(v, device=x.device) < k) | (k <= 0)
            ws = ws * ks
        if s["top_p"] is not None:
            p, before = s["top_p"].double()[:, None], ws.cumsum(-1) - ws
            ks &= (before < p * ws.sum(-1, keepdim=True)) | (p >= 1)
        keep = torch.zeros_like(keep).scatter_(1, order, ks)
    if s["min_p"] is not None:
        keep &= w >= s["min_p"].double()[:, None]
    w = w * keep
    cum = w.cumsum(-1)                                              # in the order of the token ids
    token = (cum <= s["u"].double()[:, None] * cum[:, -1:]).sum(-1).clamp(max=v - 1)
    logprob = (w.gather(1, token[:, None]) / cum[:, -1:]).log()[:, 0]
    return {"tokens": token.to(torch.int32), "logprobs": logprob.float()}


def run(state):
    s = state
    if own:
        from moe_persistent_cta_b200 import ops
        if s["op"] == "append":
            ops.rope_append(s["q"], s["k"], s["v"], s["positions"], s["table"], s["k_pool"], s["v_pool"], s["inv_freq"],
                            seq=s["seq"], interleaved=s["case"]["interleaved"], magnitude=s["magnitude"], q_out=s["q_out"])
            return {"q": s["q_out"], "k_pool": s["k_pool"], "v_pool": s["v_pool"]}
        if s["op"] == "attend":
            ops.prefix_attention(s["q"], s["k_pool"], s["v_pool"], s["table"], s["positions"], s["group_start"],
                                 s["prefix_lens"], out=s["out"], lse=s["lse"])
            return {"out": s["out"], "lse": s["lse"]}
        ops.sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                   min_p=s["min_p"], tokens=s["tokens"], logprobs=s["logprobs"])
        return {"tokens": s["tokens"], "logprobs": s["logprobs"]}
    return {"append": _plain_append, "attend": _plain_attend, "sample": _plain_sample}[s["op"]](s)


# --------------------------------------------------------------------- work --

def _lens(case):
    """Tokens of prefix (per group) and of everything (per entry) that a case's
    queries see, at their means over the seeds."""
    b, n, p = case["batch"], case["groups"], case["prefix"]
    if case["causal"]:
        return p + b, 0.0, b * (p + (b + 1) / 2)
    mean = (p + (n - 1) * 0.75 * p) / n
    own_tokens = (case["suffix"] + 1) / 2
    return n * mean, b * own_tokens, b * (mean + own_tokens)


def work(case):
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    if case["op"] == "append":
        row = (case["hq"] + 2 * case["hkv"]) * case["hd"]
        turned = (case["hq"] + case["hkv"]) * case["rot"]
        return {"bytes": case["tokens"] * (row * (size[case["src"]] + size[case["dst"]]) + 12),
                "flops": case["tokens"] * 3 * turned}
    if case["op"] == "attend":
        shared, mine, seen = _lens(case)
        hd = case["hd"]
        return {"bytes": (shared + mine) * case["hkv"] * hd * 4 + case["batch"] * case["hq"] * (hd * 4 + 4),
                "flops": 4 * seen * case["hq"] * hd}
    return {"bytes": case["batch"] * (case["vocab"] * size[case["type"]] + 28), "flops": 4 * case["batch"] * case["vocab"]}


# ------------------------------------------------------------------ 64 bits --

def _exact_append(s):
    c, out = s["case"], {}
    half = s["inv_freq"].numel()
    turn = torch.polar(torch.full_like(s["inv_freq"], s["magnitude"]).expand(c["tokens"], half).contiguous(),
                       s["positions"].double()[:, None] * s["inv_freq"])[:, None]
    lo = torch.arange(half, device=turn.device) * (2 if c["interleaved"] else 1)
    hi = lo + (1 if c["interleaved"] else half)
    for name in ("q", "k"):
        x = s[name].double()
        z = torch.complex(x[..., lo], x[..., hi]) * turn
        x[..., lo], x[..., hi] = z.real, z.imag
        out[name] = x
    kp, vp = s["k_pool"].double(), s["v_pool"].double()
    flat = s["table"].long()[s["seq"].long(), s["positions"].long() // PAGE] * PAGE + s["positions"].long() % PAGE
    for pool, rows in ((kp, out["k"]), (vp, s["v"].double())):
        view = pool.transpose(1, 2).clone(memory_format=torch.contiguous_format).view(-1, c["hkv"], c["hd"])
        view[flat] = rows
        pool.copy_(view.view(-1, PAGE, c["hkv"], c["hd"]).transpose(1, 2))
    return {"q": out["q"], "k_pool": kp, "v_pool": vp}


def _exact_attend(s):
    c = s["case"]
    b, hq, hd = s["q"].shape
    out = torch.zeros((b, hq, hd), dtype=torch.float64, device=s["q"].device)
    lse = torch.full((b, hq), -math.inf, dtype=torch.float64, device=s["q"].device)
    table, pos, start = s["table"].long(), s["positions"].tolist(), s["group_start"].tolist()
    prefix = s["prefix_lens"].tolist()
    for g in range(len(prefix)):
        for i in range(start[g], start[g + 1]):
            n = pos[i] + 1
            if n <= 0:
                continue
            t = torch.arange(n, device=table.device)
            # the first prefix tokens by the first member's row, the others by its own
            page = torch.where(t < prefix[g], table[start[g], t // PAGE], table[i, t // PAGE])
            k, v = (p[page, :, t % PAGE].double() for p in (s["k_pool"], s["v_pool"]))    # [n, hkv, hd]
            q = s["q"][i].double().view(c["hkv"], -1, hd)
            score = torch.einsum("hgd,nhd->hgn", q, k) * hd ** -0.5
            lse[i] = torch.logsumexp(score, -1).flatten()
            out[i] = torch.einsum("hgn,nhd->hgd", torch.softmax(score, -1), v).reshape(hq, hd)
    return {"out": out, "lse": lse}


def _exact_sample(s):
    tokens, logprobs = [], []
    for i in range(len(s["u"])):
        x = s["logits"][i].double()
        value, index = torch.sort(x, descending=True, stable=True)
        w = torch.exp((value - value[0]) / s["temperature"][i].double())
        n = len(w)
        if s["top_k"] is not None and int(s["top_k"][i]) > 0:
            n = min(n, int(s["top_k"][i]))
        if s["top_p"] is not None and float(s["top_p"][i]) < 1:
            cum = torch.cumsum(w[:n], 0)
            n = min(n, int((cum < s["top_p"][i].double() * cum[-1]).sum()) + 1)
        if s["min_p"] is not None:
            n = min(n, int((w >= s["min_p"][i].double()).sum()))
        kept, at = torch.sort(index[:n])
        cum = torch.cumsum(w[:n][at], 0)
        j = int(torch.searchsorted(cum, s["u"][i].double() * cum[-1], right=True))
        tokens.append(int(kept[j]))
        logprobs.append(float(torch.log(w[:n][at][j] / cum[-1])))
    return {"tokens": torch.tensor(tokens, dtype=torch.int32), "logprobs": torch.tensor(logprobs, dtype=torch.float64)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "sample": _exact_sample}[case["op"]](s)
