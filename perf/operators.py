"""Timed cases of the prefill operators over the paged latent cache.

Four calls, as a serving program makes them for a chunk of new tokens:

* ``read``    - cache rows of ragged sequences back from the paged cache (bf16, or fp8 codes with their scales)
* ``expand``  - per-head keys and values of those rows, ``wkv_b [H, 256, 512]`` times each 512-wide latent
* ``attend``  - ragged attention of the new tokens' 192-wide query heads over them
* ``prefill`` - all three, over the paged cache, in one call

With ``own`` false ``run`` computes them from elementary torch operations in float32, with ``own`` true it calls
the library.
"""

import math
import random

import torch

own = False

PAGE = 64
SCALE = 1.0 / math.sqrt(192.0)


def listed():
    return [
        # a few short chats read back from a bf16 cache: the call's latency counts
        {"name": "read-bf16-short", "op": "read", "cache": "bf16", "batch": 4, "past_lo": 40, "past_hi": 700, "new_lo": 0,
         "new_hi": 0, "offset": 0, "mix": 11},
        # the contexts of a ragged long-context batch (1k-32k tokens) out of the fp8 cache
        {"name": "read-fp8-long", "op": "read", "cache": "fp8", "batch": 16, "past_lo": 1024, "past_hi": 32768,
         "new_lo": 0, "new_hi": 0, "offset": 77, "mix": 12},
        # 16 heads, a short batch of prompts
        {"name": "expand-h16-short", "op": "expand", "heads": 16, "rows": 1001},
        # 128 heads, one chunk's worth of context
        {"name": "expand-h128-8k", "op": "expand", "heads": 128, "rows": 8209},
        # one new token in each of eight chats: the smallest calls
        {"name": "attend-h16-single", "op": "attend", "heads": 16, "batch": 8, "past_lo": 30, "past_hi": 900, "new_lo": 1,
         "new_hi": 1, "causal": True, "mix": 13},
        # whole prompts of odd lengths, 16 heads
        {"name": "attend-h16-prompts", "op": "attend", "heads": 16, "batch": 6, "past_lo": 0, "past_hi": 0, "new_lo": 90,
         "new_hi": 1700, "causal": True, "mix": 14},
        # a few new tokens after a long context, few heads: work along the keys only
        {"name": "attend-h16-long-keys", "op": "attend", "heads": 16, "batch": 1, "past_lo": 32771, "past_hi": 32771,
         "new_lo": 100, "new_hi": 100, "causal": True, "mix": 15},
        # the older part of a context, seen by every new token (merged with the rest by its log-sum-exp)
        {"name": "attend-h128-part", "op": "attend", "heads": 128, "batch": 2, "past_lo": 3500, "past_hi": 6500,
         "new_lo": 300, "new_hi": 700, "causal": False, "mix": 16},
        # one 2048-token chunk of a long prompt, 128 heads
        {"name": "attend-h128-chunk", "op": "attend", "heads": 128, "batch": 1, "past_lo": 14336, "past_hi": 14336,
         "new_lo": 2048, "new_hi": 2048, "causal": True, "mix": 17},
        # short prompts in one call over a bf16 cache, 16 heads
        {"name": "prefill-bf16-h16", "op": "prefill", "cache": "bf16", "heads": 16, "batch": 5, "past_lo": 0,
         "past_hi": 600, "new_lo": 60, "new_hi": 500, "causal": True, "mix": 18},
        # chunks of two conversations over an fp8 cache, 128 heads
        {"name": "prefill-fp8-h128", "op": "prefill", "cache": "fp8", "heads": 128, "batch": 2, "past_lo": 2000,
         "past_hi": 7000, "new_lo": 512, "new_hi": 1024, "causal": True, "mix": 19},
    ]


def _between(rng, lo, hi):
    """A size between lo and hi, its logarithm uniform."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    """One more case of the same four kinds. Sizes that would cost more than the largest listed case are drawn again."""
    op = rng.choice(["read", "expand", "attend", "attend", "prefill"])
    most = max(work(c)["flops"] for c in listed())
    while True:
        c = {"op": op}
        if op == "read":
            lo = _between(rng, 1, 16384)
            c.update(cache=rng.choice(["bf16", "fp8"]), batch=_between(rng, 1, 16), past_lo=lo,
                     past_hi=min(32768, lo + _between(rng, 1, 4 * lo)), new_lo=0, new_hi=0, offset=rng.randint(0, 200))
        elif op == "expand":
            c.update(heads=rng.choice([4, 16, 24, 40, 64, 128]), rows=_between(rng, 1, 16384))
        else:
            n, past = _between(rng, 1, 2048), rng.choice([0, _between(rng, 1, 16384)])
            c.update(heads=rng.choice([4, 16, 24, 40, 64, 128]), batch=_between(rng, 1, 8), past_lo=past // 2, past_hi=past,
                     new_lo=max(1, n // 2), new_hi=n, causal=True)
            if op == "attend":
                c["causal"] = rng.random() < 0.75
            else:
                c["cache"] = rng.choice(["bf16", "fp8"])
        if op != "expand":
            c["mix"] = rng.randint(100, 1 << 20)
        padded = c.get("heads", 0) * c.get("batch", 0) * c.get("new_hi", 0) * (c.get("past_hi", 0) + c.get("new_hi", 0))
        if work(c)["flops"] <= most and padded <= 1 << 32:
            return c


def _lengths(case):
    """(cached before the chunk, new) tokens of every sequence: from the case alone."""
    rng = random.Random(case["mix"])
    return [(rng.randint(case["past_lo"], case["past_hi"]), rng.randint(case["new_lo"], case["new_hi"]))
            for _ in range(case["batch"])]


def _pairs(case):
    """Visible (query, key) pairs of one head."""
    return sum(n * past + (n * (n + 1) // 2 if case["causal"] else n * n) for past, n in _lengths(case))


def work(case):
    op = case["op"]
    if op == "expand":
        m, h = case["rows"], case["heads"]
        return {"bytes": m * 1024 + h * 256 * 1024 + m * h * 512, "flops": 2 * m * 512 * 256 * h}
    lens = _lengths(case)
    keys, new = sum(p + n for p, n in lens), sum(n for _, n in lens)
    row = 1152 if case.get("cache") == "bf16" else 644
    if op == "read":
        return {"bytes": keys * (row + 1152), "flops": 512 * keys if case["cache"] == "fp8" else 0}
    h = case["heads"]
    attend = 2 * 320 * h * _pairs(case)
    queries = new * h * (384 + 256 + 4)
    if op == "attend":
        return {"bytes": keys * (h * 512 + 128) + queries, "flops": attend}
    return {"bytes": keys * row + h * 256 * 1024 + queries, "flops": attend + 2 * keys * 512 * 256 * h}


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def _offsets(counts):
    return torch.tensor([0] + counts, dtype=torch.int64).cumsum(0).to("cuda", torch.int32)


def _paged(case, g):
    """A paged cache whose pages lie in random order, and the block table of the case's sequences."""
    total = [p + n + case.get("offset", 0) for p, n in _lengths(case)]
    pages = [max(1, -(-t // PAGE)) for t in total]
    count, width = sum(pages) + 3, max(pages)
    order = torch.randperm(count, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(pages), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, p in enumerate(pages):
        table[b, :p] = order[at:at + p]
        at += p
    latent = _normal(g, count, PAGE, 512)
    rope = _normal(g, count, PAGE, 64)
    if case["cache"] == "bf16":
        return torch.cat([latent, rope], -1), table
    raw = torch.zeros(count, PAGE, 656, dtype=torch.uint8, device="cuda")
    scale = latent.float().abs().amax(-1, keepdim=True) / 448.0
    raw[..., :512] = (latent.float() / scale).to(torch.float8_e4m3fn).view(torch.uint8)
    raw[..., 512:640] = rope.view(torch.uint8)
    raw[..., 640:644] = scale.view(torch.uint8)
    return raw, table


def _inputs(case, seed):
    """What the program has before the call: tensors made from the seed alone."""
    g, op, d = _generator(seed), case["op"], {}
    if op == "expand":
        d["rows"] = _normal(g, case["rows"], 576)
        d["wkv_b"] = _normal(g, case["heads"], 256, 512, std=0.05)
        return d
    lens = _lengths(case)
    keys, new = [p + n for p, n in lens], [n for _, n in lens]
    d["cu_k"], d["cu_q"] = _offsets(keys), _offsets(new)
    if op in ("read", "prefill"):
        d["cache"], d["table"] = _paged(case, g)
    if op == "read":
        d["starts"] = torch.full((len(lens),), case["offset"], dtype=torch.int32, device="cuda")
        return d
    h = case["heads"]
    d["q"] = _normal(g, sum(new), h, 192)
    if op == "prefill":
        d["wkv_b"] = _normal(g, h, 256, 512, std=0.05)
    else:
        d["kv"] = _normal(g, sum(keys), h, 256)
        d["k_pe"] = _normal(g, sum(keys), 64)
    return d


def prepare(case, seed):
    d = _inputs(case, seed)
    d["op"], d["causal"] = case["op"], case.get("causal", True)
    if case["op"] != "expand":
        lens = _lengths(case)
        d["total_k"] = sum(p + n for p, n in lens)
        d["max_k"], d["max_q"] = max(p + n for p, n in lens), max(n for _, n in lens)
    if own:
        from mla_latent_kv_26_b200 import prefill

        if case["op"] == "read":
            d["out"] = torch.empty(d["total_k"], 576, dtype=torch.bfloat16, device="cuda")
        elif case["op"] == "expand":
            d["out"] = torch.empty(case["rows"], case["heads"], 256, dtype=torch.bfloat16, device="cuda")
        elif case["op"] == "attend":
            d["out"] = torch.empty(d["q"].shape[0], case["heads"], 128, dtype=torch.bfloat16, device="cuda")
            d["lse"] = torch.empty(d["q"].shape[0], case["heads"], dtype=torch.float32, device="cuda")
            d["workspace"] = torch.empty(prefill.attention_workspace_bytes(d["q"].shape[0], case["heads"],
                                                                           d["total_k"]),
                                         dtype=torch.uint8, device="cuda")
        else:
            d["prefill"] = prefill.MlaPrefill(max_queries=d["q"].shape[0], max_keys=d["total_k"],
                                              num_heads=case["heads"])
    return d


def _plain_read(cache, table, cu, starts, total):
    """Rows in float32: a row index per output row, then one gather."""
    at = torch.arange(total, device="cuda")
    seq = torch.searchsorted(cu[1:].long(), at, right=True)
    pos = at - cu.long()[seq] + (starts.long()[seq] if starts is not None else 0)
    page = table[seq, pos // PAGE].long()
    row = cache.view(-1, cache.shape[-1])[page * PAGE + pos % PAGE]
    if cache.dtype == torch.bfloat16:
        return row.float()
    scale = row[:, 640:644].contiguous().view(torch.float32)
    rope = row[:, 512:640].contiguous().view(torch.bfloat16).float()
    # the format's value of a code is bf16(code * scale)
    latent = (row[:, :512].contiguous().view(torch.float8_e4m3fn).float() * scale).to(torch.bfloat16).float()
    return torch.cat([latent, rope], 1)


def _plain_attend(q, k_nope, v, k_pe, cu_q, cu_k, max_q, max_k, causal):
    """Softmax attention of every sequence at once, queries and keys padded to the longest."""
    nq, nk = (cu_q[1:] - cu_q[:-1]).long()[:, None], (cu_k[1:] - cu_k[:-1]).long()[:, None]
    i, t = torch.arange(max_q, device="cuda")[None], torch.arange(max_k, device="cuda")[None]
    qi = (cu_q[:-1].long()[:, None] + i).clamp(max=q.shape[0] - 1)
    kt = (cu_k[:-1].long()[:, None] + t).clamp(max=k_nope.shape[0] - 1)
    qp = q.float()[qi].permute(0, 2, 1, 3)
    keys = torch.cat([k_nope[kt], k_pe[kt][:, :, None].expand(-1, -1, q.shape[1], -1)], -1)
    s = torch.matmul(qp, keys.permute(0, 2, 3, 1)).mul_(SCALE)
    seen = (t < nk)[:, None, :].expand(-1, max_q, -1)
    if causal:
        seen = seen & (t[:, None, :] <= (nk - nq + i)[:, :, None])
    s.masked_fill_(~seen[:, None], -math.inf)
    top = s.amax(-1, keepdim=True).clamp_(min=-1e30)
    p = s.sub_(top).exp_()
    total = p.sum(-1)
    out = torch.matmul(p, v[kt].permute(0, 2, 1, 3)) / total[..., None]
    lse = total.log() + top[..., 0]
    live = (i < nq).reshape(-1)
    out = out.permute(0, 2, 1, 3).reshape(-1, q.shape[1], 128)[live]
    return out.to(torch.bfloat16), lse.permute(0, 2, 1).reshape(-1, q.shape[1])[live]


def _plain(s):
    op = s["op"]
    if op == "read":
        return _plain_read(s["cache"], s["table"], s["cu_k"], s["starts"], s["total_k"]).to(torch.bfloat16)
    if op == "expand":
        h = s["wkv_b"].shape[0]
        kv = torch.matmul(s["rows"][:, :512].float(), s["wkv_b"].float().view(h * 256, 512).t())
        return kv.to(torch.bfloat16).view(-1, h, 256)
    if op == "attend":
        kv = s["kv"].float()
        return _plain_attend(s["q"], kv[..., :128], kv[..., 128:], s["k_pe"].float(), s["cu_q"], s["cu_k"], s["max_q"],
                             s["max_k"], s["causal"])
    rows = _plain_read(s["cache"], s["table"], s["cu_k"], None, s["total_k"])
    h = s["wkv_b"].shape[0]
    kv = torch.matmul(rows[:, :512], s["wkv_b"].float().view(h * 256, 512).t()).view(-1, h, 256)
    return _plain_attend(s["q"], kv[..., :128], kv[..., 128:], rows[:, 512:], s["cu_q"], s["cu_k"], s["max_q"],
                         s["max_k"], True)[0]


def run(state):
    if not own:
        return _plain(state)
    from mla_latent_kv_26_b200 import prefill

    s, op = state, state["op"]
    if op == "read":
        return prefill.cache_read(s["cache"], s["table"], s["cu_k"], starts=s["starts"], out=s["out"])
    if op == "expand":
        return prefill.expand_kv(s["rows"], s["wkv_b"], out=s["out"])
    if op == "attend":
        return prefill.prefill_attention(s["q"], s["kv"], s["k_pe"], s["cu_q"], s["cu_k"], causal=s["causal"],
                                         out=s["out"], lse=s["lse"], workspace=s["workspace"])
    return s["prefill"](s["q"], s["wkv_b"], s["cache"], s["table"], s["cu_q"], s["cu_k"])


def _exact_rows(d, b, first, count):
    """Cache rows [first, first + count) of sequence b in float64, page by page."""
    parts = []
    for p in range(first // PAGE, (first + count - 1) // PAGE + 1):
        parts.append(d["cache"][int(d["table"][b, p])])
    page = torch.cat(parts)[first % PAGE:first % PAGE + count]
    if page.dtype == torch.bfloat16:
        return page.double()
    code = page[:, :512].contiguous().view(torch.float8_e4m3fn).double()
    scale = page[:, 640:644].contiguous().view(torch.float32).double()
    # code * scale has at most 28 significant bits: float32 rounds it once, then the format's bf16
    latent = (code * scale).float().to(torch.bfloat16).double()
    return torch.cat([latent, page[:, 512:640].contiguous().view(torch.bfloat16).double()], 1)


def _exact_heads(q, key, value, past, causal):
    """One sequence in float64: q [n, H, 192], key(h) [L, 192], value(h) [L, 128]."""
    n, heads = q.shape[:2]
    out = torch.empty(n, heads, 128, dtype=torch.float64, device="cuda")
    lse = torch.empty(n, heads, dtype=torch.float64, device="cuda")
    for h in range(heads):
        s = q[:, h].double() @ key(h).t() / math.sqrt(192.0)
        if causal:
            s += torch.full_like(s, -math.inf).triu(past + 1)
        lse[:, h] = torch.logsumexp(s, 1)
        out[:, h] = torch.exp(s - lse[:, h, None]) @ value(h)
    return out, lse


def exact(case, seed):
    d, op = _inputs(case, seed), case["op"]
    if op == "expand":
        lat = d["rows"][:, :512].double()
        return torch.stack([lat @ w.double().t() for w in d["wkv_b"]], 1)
    lens = _lengths(case)
    if op == "read":
        return torch.cat([_exact_rows(d, b, case["offset"], p + n) for b, (p, n) in enumerate(lens)])
    outs, lses, q0, k0 = [], [], 0, 0
    for b, (past, n) in enumerate(lens):
        q = d["q"][q0:q0 + n]
        if op == "attend":
            kv, pe = d["kv"][k0:k0 + past + n], d["k_pe"][k0:k0 + past + n].double()
            key = lambda h: torch.cat([kv[:, h, :128].double(), pe], 1)
            value = lambda h: kv[:, h, 128:].double()
        else:
            rows = _exact_rows(d, b, 0, past + n)
            key = lambda h: torch.cat([rows[:, :512] @ d["wkv_b"][h, :128].double().t(), rows[:, 512:]], 1)
            value = lambda h: rows[:, :512] @ d["wkv_b"][h, 128:].double().t()
        o, l = _exact_heads(q, key, value, past, case["causal"])
        outs.append(o)
        lses.append(l)
        q0, k0 = q0 + n, k0 + past + n
    if op == "attend":
        return torch.cat(outs), torch.cat(lses)
    return torch.cat(outs)
