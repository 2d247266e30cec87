"""Cases, plain forms and 64-bit values of the operators that decide what a serving step works on.

Four operators around the products of a decoder layer's serving step:

* gate   -- the router's logits: tokens times the gate's rows, summed in 32 bits.
* route  -- logits to experts: softmax or sigmoid scores, a bias for balance, groups, top-k, weights.
* pages  -- the paged key/value cache from request lengths: sequences keep, lose and gain tokens, pages
  come from and go back to a free list, and every new row learns its sequence, position and slot.
* verify -- drafted tokens against the target's probabilities from given random numbers, and the token behind them.

With ``own`` false, ``run`` computes them with elementary torch operations, in 32 bits, or in 64 where a
decision hangs on them; with ``own`` true it calls the library.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    gate = {"op": "gate", "dtype": "bf16"}
    route = {"op": "route", "score": "sigmoid", "bias": True, "groups": 8, "top_groups": 4, "pair": True, "renorm": True, "scale": 2.5,
             "top_k": 8, "experts": 256, "dtype": "f32", "masked": 0.0, "padded": 0}
    pages = {"op": "pages", "keep": "all", "short": False}
    verify = {"op": "verify", "dtype": "f32", "draft_probs": True, "ragged": False}
    return [
        # one user, one token: the gate of the all-experts layer as a decode step waits for it
        dict(gate, name="gate_one_token", tokens=1, hidden=7168, experts=256),
        # a decode batch of a smaller model, an odd number of tokens and experts
        dict(gate, name="gate_decode_odd", tokens=333, hidden=2040, experts=60, dtype="f16"),
        # prompts that go through the layer together
        dict(gate, name="gate_prompts", tokens=16384, hidden=7168, experts=256),
        # one token's experts: latency
        dict(route, name="route_one_token", tokens=1),
        # a padded decode batch, softmax scores in 16 bits, no bias, some experts masked out
        dict(route, name="route_decode_odd", tokens=1021, experts=160, dtype="bf16", score="softmax", bias=False, top_groups=3, pair=False,
             renorm=False, top_k=6, scale=16.0, masked=0.05, padded=24),
        # prompts' routing, as many rows as the prefill of a node brings together
        dict(route, name="route_prompts", tokens=65536),
        # a full decode batch, one token more for each sequence, small pages
        dict(pages, name="pages_decode", batch=256, new=1, ctx=2048, page=16),
        # drafts: rejected ones leave the cache, new ones come; some requests end, some begin, pages run out at the last ones
        dict(pages, name="pages_drafts", batch=61, new=5, ctx=9001, page=64, keep="some", short=True),
        # prompts of many requests, the whole cache in small pages
        dict(pages, name="pages_prompts", batch=1024, new=2048, ctx=0, page=16),
        # one user, three drafts
        dict(verify, name="verify_one", batch=1, drafts=3, vocab=128000),
        # drafts of a lookup, which have no probabilities, in 16 bits, an odd vocabulary, ragged
        dict(verify, name="verify_ragged", batch=37, drafts=7, vocab=50021, dtype="bf16", draft_probs=False, ragged=True),
        # a full batch with three drafts each
        dict(verify, name="verify_batch", batch=256, drafts=3, vocab=128000),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi, max(lo, v))


def draw(rng):
    ops = ("gate", "route", "pages", "verify")
    most = {op: [max(work(c)[k] for c in listed() if c["op"] == op) for k in ("bytes", "flops")] for op in ops}
    while True:
        case = {"op": rng.choice(ops)}
        if case["op"] == "gate":
            case.update(dtype=rng.choice(["bf16", "f16"]), tokens=_spread(rng, 1, 16384), hidden=8 * _spread(rng, 16, 1024),
                        experts=_spread(rng, 4, 512))
        elif case["op"] == "route":
            groups = rng.choice([1, 1, 2, 4, 8, 16])
            experts = groups * _spread(rng, 4, 512 // groups)
            top_groups = rng.randint(1, groups)
            case.update(dtype=rng.choice(["f32", "bf16", "f16"]), tokens=_spread(rng, 1, 65536), experts=experts, groups=groups,
                        top_groups=top_groups, score=rng.choice(["sigmoid", "softmax"]), bias=rng.random() < 0.6,
                        pair=rng.random() < 0.5, renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5, 16.0]),
                        top_k=rng.randint(1, min(16, top_groups * (experts // groups))),
                        masked=rng.choice([0.0, 0.0, 0.3]), padded=rng.choice([0, 0, 17]))
        elif case["op"] == "pages":
            form = rng.choice(["one", "draft", "chunk"])
            case.update(batch=_spread(rng, 1, 1024), new={"one": 1, "draft": rng.randint(2, 9), "chunk": _spread(rng, 10, 4096)}[form],
                        ctx=0 if rng.random() < 0.2 else _spread(rng, 1, 32768), page=rng.choice([16, 32, 64, 128]),
                        keep=rng.choice(["all", "some"]), short=rng.random() < 0.3)
        else:
            case.update(dtype=rng.choice(["f32", "f32", "bf16", "f16"]), batch=_spread(rng, 1, 256), drafts=rng.randint(0, 8),
                        vocab=_spread(rng, 1000, 160000), draft_probs=rng.random() < 0.7, ragged=rng.random() < 0.5)
            if case["batch"] * (case["drafts"] + 1) * case["vocab"] > 1 << 28:        # the probabilities that are in hand
                continue
        if all(work(case)[k] <= m for k, m in zip(("bytes", "flops"), most[case["op"]])):
            return case


# ---------------------------------------------------------------- properties of a case
def _page_lengths(case):
    """Tokens that each sequence has, keeps and gains."""
    r = random.Random("pages %d %d %d" % (case["batch"], case["new"], case["ctx"]))
    old, keep, new = [], [], []
    for _ in range(case["batch"]):
        o = r.randint(case["ctx"] // 8, case["ctx"])
        n = case["new"] if case["new"] < 10 else r.randint(1, case["new"])
        k, fate = o, r.random()
        if case["keep"] == "some":
            if fate < 0.08:                      # a request that has ended
                k, n = 0, 0
            elif fate < 0.16:                    # one that begins with a prompt
                o = k = 0
                n = max(1, case["ctx"] // 16)
            else:                                # rejected drafts
                k = max(0, o - r.randint(0, min(8, case["new"])))
        old.append(o)
        keep.append(k)
        new.append(n)
    return old, keep, new


def _draft_counts(case):
    r = random.Random("drafts %d %d" % (case["batch"], case["drafts"]))
    return [r.randint(0, case["drafts"]) if case["ragged"] else case["drafts"] for _ in range(case["batch"])]


def work(case):
    if case["op"] == "gate":
        t, h, e = case["tokens"], case["hidden"], case["experts"]
        return {"bytes": 2 * (t + e) * h + 4 * t * e, "flops": 2 * t * h * e}
    if case["op"] == "route":
        t, e, k = case["tokens"] - case["padded"], case["experts"], case["top_k"]
        return {"bytes": t * e * (4 if case["dtype"] == "f32" else 2) + 8 * case["tokens"] * k + 4 * e * case["bias"], "flops": 6 * t * e}
    if case["op"] == "pages":
        old, keep, new = _page_lengths(case)
        p = case["page"]
        moved = sum(abs(-(-(k + n) // p) - -(-o // p)) for o, k, n in zip(old, keep, new))
        return {"bytes": 20 * case["batch"] + 8 * moved + 16 * sum(new), "flops": 4 * sum(new)}
    # one row of the target's probabilities for each sequence, and one of the draft's where a draft is rejected: with drafts
    # that are taken three times in four
    size = 4 if case["dtype"] == "f32" else 2
    rows = sum(1 + (1 - 0.75 ** n if case["draft_probs"] else 0) for n in _draft_counts(case))
    return {"bytes": int(rows * case["vocab"] * size) + 16 * sum(n + 1 for n in _draft_counts(case)), "flops": int(2 * rows * case["vocab"])}


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev).manual_seed(seed)
    return {"gate": _prepare_gate, "route": _prepare_route, "pages": _prepare_pages, "verify": _prepare_verify}[case["op"]](case, g, dev)


def _prepare_gate(c, g, dev):
    # normed tokens with a few large dimensions, as residual streams have them
    t, h, e, dtype = c["tokens"], c["hidden"], c["experts"], TYPES[c["dtype"]]
    x = torch.randn((t, h), generator=g, device=dev)
    x[:, torch.randperm(h, generator=g, device=dev)[: max(1, h // 100)]] *= 8.0
    w = torch.randn((e, h), generator=g, device=dev) / math.sqrt(h)
    return {"case": c, "x": x.to(dtype), "w": w.to(dtype), "logits": torch.empty((t, e), device=dev)}


def _prepare_route(c, g, dev):
    t, e = c["tokens"], c["experts"]
    z = torch.randn((t, e), generator=g, device=dev) * 1.5 + 0.5 * torch.randn((1, e), generator=g, device=dev)
    z = torch.where(torch.rand((t, e), generator=g, device=dev) < c["masked"], -torch.inf, z).to(TYPES[c["dtype"]])
    return {"case": c, "logits": z, "bias": 0.1 * torch.randn(e, generator=g, device=dev) if c["bias"] else None,
            "n_tokens": torch.tensor([t - c["padded"]], dtype=torch.int32, device=dev) if c["padded"] else None,
            "ids": torch.empty((t, c["top_k"]), dtype=torch.int32, device=dev), "weights": torch.empty((t, c["top_k"]), device=dev)}


def _prepare_pages(c, g, dev):
    P, B = c["page"], c["batch"]
    old, keep, new = _page_lengths(c)
    held = [-(-o // P) for o in old]
    need = [-(-(k + n) // P) for k, n in zip(keep, new)]
    demand = sum(max(0, n - h) for n, h in zip(need, held)) - sum(max(0, h - n) for n, h in zip(need, held))
    free = max(0, demand) * 4 // 5 if c["short"] else max(0, demand) + 5
    pool = sum(held) + free + 7
    order = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
    table = torch.full((B, max(held + need) + 1), -1, dtype=torch.int32, device=dev)
    table[torch.arange(table.shape[1], device=dev)[None] < torch.tensor(held, device=dev)[:, None]] = order[: sum(held)]
    stack = torch.full((pool,), -1, dtype=torch.int32, device=dev)
    stack[:free] = order[sum(held): sum(held) + free]
    i32 = {"dtype": torch.int32, "device": dev}
    rows = sum(new) + 3                          # a few rows behind the last, as a captured step has them
    return {"case": c, "kv_old": torch.tensor(old, **i32), "kv_keep": torch.tensor(keep, **i32) if c["keep"] == "some" else None,
            "n_new": torch.tensor(new, **i32), "table": table, "stack": stack, "count": torch.tensor([free], **i32),
            "kv_len": torch.empty(B, **i32), "cu_new": torch.empty(B + 1, **i32), "count_out": torch.empty(1, **i32),
            "seqs": torch.empty(rows, **i32), "positions": torch.empty(rows, **i32), "slots": torch.empty(rows, dtype=torch.int64, device=dev)}


def _prepare_verify(c, g, dev):
    counts, V, dtype = _draft_counts(c), c["vocab"], TYPES[c["dtype"]]
    B, T = len(counts), sum(counts) + len(counts)
    z = 4.0 * torch.randn((T, V), generator=g, device=dev)
    p = torch.softmax(z, 1).to(dtype)
    q = torch.softmax(z + 0.5 * torch.randn((T, V), generator=g, device=dev), 1)
    picked = torch.multinomial(q, 1, generator=g).flatten().to(torch.int32)      # each row's draft for the next token
    tokens = torch.zeros(T, dtype=torch.int32, device=dev)
    tokens[1:] = picked[:-1]
    cu = torch.tensor([sum(counts[:b]) + b for b in range(B + 1)], dtype=torch.int32, device=dev)
    return {"case": c, "probs": p, "draft_probs": q.to(dtype) if c["draft_probs"] else None, "tokens": tokens, "cu_new": cu,
            "u_accept": torch.rand(T, generator=g, device=dev), "u_sample": torch.rand(B, generator=g, device=dev),
            "kv_len": cu[1:] - cu[:-1] + 1000, "kv_keep": torch.empty(B, dtype=torch.int32, device=dev),
            "accepted": torch.empty(B, dtype=torch.int32, device=dev),
            "out": torch.empty((B, c["drafts"] + 1), dtype=torch.int32, device=dev)}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"gate": _own_gate, "route": _own_route, "pages": _own_pages, "verify": _own_verify}[op](state)
    return {"gate": _plain_gate, "route": _plain_route, "pages": _plain_pages, "verify": _plain_verify}[op](state)


def _own_gate(s):
    import fp8_grouped_expert_x128_gb300 as moe
    return moe.moe_gate(s["x"], s["w"], s["logits"])


def _own_route(s):
    import fp8_grouped_expert_x128_gb300 as moe
    c = s["case"]
    flags = ((moe.MOE_ROUTE_SOFTMAX if c["score"] == "softmax" else 0) | (moe.MOE_ROUTE_RENORM if c["renorm"] else 0)
             | (moe.MOE_ROUTE_GROUP_PAIR if c["pair"] else 0))
    moe.moe_route(s["logits"], s["ids"], s["weights"], bias=s["bias"], n_group=c["groups"], topk_group=c["top_groups"], scale=c["scale"],
                  flags=flags, n_tokens=s["n_tokens"])
    return {"ids": s["ids"], "weights": s["weights"]}


def _own_pages(s):
    import fp8_grouped_expert_x128_gb300 as moe
    moe.moe_kv_pages(s["kv_old"], s["n_new"], s["table"], s["stack"], s["count"], s["case"]["page"], s["kv_len"], s["cu_new"], s["count_out"],
                     kv_keep=s["kv_keep"], seqs=s["seqs"], positions=s["positions"], slots=s["slots"])
    return _paged(s)


def _own_verify(s):
    import fp8_grouped_expert_x128_gb300 as moe
    moe.moe_verify_drafts(s["probs"], s["tokens"], s["cu_new"], s["u_accept"], s["u_sample"], s["accepted"], s["out"],
                          draft_probs=s["draft_probs"], kv_len=s["kv_len"], kv_keep=s["kv_keep"])
    return _verified(s)


def _paged(s):
    return {"table": s["table"], "stack": s["stack"], "count": s["count_out"], "kv_len": s["kv_len"], "cu_new": s["cu_new"], "seqs": s["seqs"],
            "positions": s["positions"], "slots": s["slots"]}


def _verified(s):
    return {"accepted": s["accepted"], "tokens": s["out"], "kv_keep": s["kv_keep"]}


# ---------------------------------------------------------------- plain forms
def _plain_gate(s):
    return s["logits"].copy_(s["x"].float() @ s["w"].float().T)


def _plain_route(s):
    c, z = s["case"], s["logits"].double()               # ranks hang on differences: 64 bits
    t, e = z.shape
    z = torch.where(torch.isnan(z), -torch.inf, z.clamp(max=torch.finfo(torch.float32).max))
    alive = z > -torch.inf
    if c["score"] == "softmax":
        top = z.amax(1, keepdim=True)
        score = torch.where(alive, torch.exp(z - torch.where(top > -torch.inf, top, 0.0)), 0.0)
        score = score / score.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        score = 1.0 / (1.0 + torch.exp(-z))
    value = score + s["bias"].double() if c["bias"] else z
    if c["groups"] > 1:
        by = (value if c["bias"] or not c["pair"] else score).masked_fill(~alive, -torch.inf).view(t, c["groups"], -1)
        best = by.sort(2, descending=True).values
        second = best[..., 1:2].masked_fill(best[..., 1:2] == -torch.inf, 0.0).sum(2) if c["pair"] else 0.0
        order = (best[..., 0] + second).sort(dim=1, descending=True, stable=True).indices
        kept = torch.zeros_like(order, dtype=torch.bool).scatter_(1, order[:, : c["top_groups"]], True)
        alive = alive & kept.repeat_interleave(e // c["groups"], 1)
    order = value.masked_fill(~alive, -torch.inf).sort(dim=1, descending=True, stable=True).indices[:, : c["top_k"]]
    ok = alive.gather(1, order)
    if s["n_tokens"] is not None:
        ok = ok & (torch.arange(t, device=z.device) < s["n_tokens"])[:, None]
    weight = torch.where(ok, score.gather(1, order), 0.0)
    if c["renorm"]:
        weight = weight / weight.sum(1, keepdim=True).clamp(min=1e-300)
    s["ids"].copy_(torch.where(ok, order, -1))
    s["weights"].copy_(weight * c["scale"])
    return {"ids": s["ids"], "weights": s["weights"]}


def _plain_pages(s):
    P, table, stack, f = s["case"]["page"], s["table"], s["stack"], s["count"].long()
    dev, B = table.device, table.shape[0]
    old, new = s["kv_old"].long(), s["n_new"].long()
    keep = old if s["kv_keep"] is None else s["kv_keep"].long()
    held, need = (old + P - 1) // P, (keep + new + P - 1) // P
    wants = (need - held).clamp(min=0)
    granted = (wants == 0) | (wants.cumsum(0) <= f + (held - need).clamp(min=0).sum())
    new = torch.where(granted, new, 0)
    need = (keep + new + P - 1) // P
    gain, loss = (need - held).clamp(min=0), (held - need).clamp(min=0)
    gains, losses = gain.cumsum(0), loss.cumsum(0)
    s["kv_len"].copy_(keep + new)
    s["cu_new"].zero_()[1:] = new.cumsum(0)
    # pages that go back, in the sequences' order, and then pages that are taken, from the end of the list
    j, pool = torch.arange(table.shape[1], device=dev), stack.numel()
    number = (losses - loss)[:, None] + j - need[:, None]
    at = torch.where((j >= need[:, None]) & (j < held[:, None]), f + number, pool)
    back = torch.cat([stack, stack[:1]]).scatter_(0, at.flatten(), table.flatten())
    total = f + losses[-1] - gains[-1]
    number = (gains - gain)[:, None] + j - held[:, None]
    taken = back[(f + losses[-1] - 1 - number).clamp(0, pool)]
    table.copy_(torch.where((j >= held[:, None]) & (j < need[:, None]), taken, table))
    r = torch.arange(pool, device=dev)
    stack.copy_(torch.where((r >= f) & (r < total), back[:-1], stack))
    s["count_out"].copy_(total)
    row = torch.arange(s["seqs"].numel(), device=dev)
    cu = s["cu_new"].long()
    b = torch.searchsorted(cu[1:], row, right=True)
    used = b < B
    b = b.clamp(max=B - 1)
    pos = keep[b] + row - cu[b]
    page = table[b, (pos // P).clamp(max=table.shape[1] - 1)].long()
    s["seqs"].copy_(torch.where(used, b, -1))
    s["positions"].copy_(torch.where(used, pos, -1))
    s["slots"].copy_(torch.where(used, page * P + pos % P, -1))
    return _paged(s)


def _plain_verify(s):
    c, cu, V = s["case"], s["cu_new"].long(), s["case"]["vocab"]
    n = cu[1:] - cu[:-1] - 1                              # drafts of each sequence
    i = torch.arange(c["drafts"] + 1, device=cu.device)
    at = (cu[:-1, None] + i).clamp(max=s["tokens"].numel() - 1)
    draft = s["tokens"][(at + 1).clamp(max=s["tokens"].numel() - 1)].long()
    p = s["probs"][at, draft].double()
    q = 1.0 if s["draft_probs"] is None else s["draft_probs"][at, draft].double()
    taken = (s["u_accept"][at].double() * q < p) & (i < n[:, None])
    accepted = taken.long().cumprod(1).sum(1)
    row = cu[:-1] + accepted
    whole = s["probs"][row].double()
    turned_down = (accepted < n)[:, None]
    wrong = draft.gather(1, accepted[:, None])
    if s["draft_probs"] is None:
        left = whole.scatter(1, wrong, 0.0)
    else:
        left = (whole - s["draft_probs"][row].double()).clamp(min=0.0)
    left = torch.where(turned_down, left, whole)
    left = torch.where(left.sum(1, keepdim=True) > 0, left, whole)
    sums = left.cumsum(1)                                 # 64 bits: a token's borders lie 1e-6 apart and less
    token = torch.searchsorted(sums, s["u_sample"].double()[:, None] * sums[:, -1:], right=True).flatten()
    last = torch.where(left > 0, torch.arange(V, device=cu.device), -1).amax(1)
    token = torch.minimum(token, last)
    out = torch.where(i < accepted[:, None], draft, -1)
    s["out"].copy_(out.scatter(1, accepted[:, None], token[:, None]))
    s["accepted"].copy_(accepted)
    s["kv_keep"].copy_(s["kv_len"].long() - (n - accepted))
    return _verified(s)


# ---------------------------------------------------------------- 64-bit values
def exact(case, seed):
    s = prepare(case, seed)
    return {"gate": _exact_gate, "route": _exact_route, "pages": _exact_pages, "verify": _exact_verify}[case["op"]](s)


def _exact_gate(s):
    w = s["w"].double().t().contiguous()
    return torch.cat([part.double() @ w for part in s["x"].split(2048)])


def _exact_route(s):
    c, z = s["case"], s["logits"].double()
    t, e = z.shape
    number = torch.arange(e, device=z.device)
    open_ = torch.isfinite(z)
    # the cases' logits are finite or -inf
    if c["score"] == "softmax":
        score = torch.exp(z - torch.logsumexp(z, 1, keepdim=True)).nan_to_num(0.0)
    else:
        score = 0.5 + 0.5 * torch.tanh(0.5 * z)
    value = torch.where(open_, score + s["bias"].double() if c["bias"] else z, -torch.inf)

    def first(v, count, n):
        """The `count` largest of the last axis, one after another, the lowest number among equals."""
        v, found = v.clone(), []
        for _ in range(count):
            m = v.amax(-1, keepdim=True)
            at = torch.where(v == m, n, n.numel()).amin(-1, keepdim=True)
            found.append((at, m))
            v.scatter_(-1, at, torch.nan)
            v.nan_to_num_(nan=-torch.inf, posinf=torch.inf, neginf=-torch.inf)
        return torch.cat([a for a, _ in found], -1), torch.cat([m for _, m in found], -1)

    if c["groups"] > 1:
        size = e // c["groups"]
        rank = value if c["bias"] or not c["pair"] else torch.where(open_, score, -torch.inf)
        _, two = first(rank.view(t, c["groups"], size), min(2, size) if c["pair"] else 1, number[:size])
        value_of = torch.where(torch.isfinite(two), two, 0.0).sum(-1) + torch.where(torch.isfinite(two[..., 0]), 0.0, -torch.inf)
        kept = torch.zeros((t, c["groups"]), device=z.device)
        used = torch.zeros_like(kept, dtype=torch.bool)
        for _ in range(c["top_groups"]):
            free = torch.where(used, -torch.inf, value_of)
            m = free.amax(1, keepdim=True)
            at = torch.where((free == m) & ~used, number[: c["groups"]], e).amin(1, keepdim=True)
            used.scatter_(1, at, True)
        value = torch.where(used.repeat_interleave(size, 1), value, -torch.inf)
    at, m = first(value, c["top_k"], number)
    ok = m > -torch.inf
    if s["n_tokens"] is not None:
        ok[int(s["n_tokens"]):] = False
    w = torch.where(ok, score.gather(1, at), 0.0)
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return {"ids": torch.where(ok, at, -1).int(), "weights": c["scale"] * w}


def _exact_pages(s):
    P = s["case"]["page"]
    old, new = s["kv_old"].tolist(), s["n_new"].tolist()
    keep = old if s["kv_keep"] is None else s["kv_keep"].tolist()
    table, stack, f = s["table"].tolist(), s["stack"].tolist(), int(s["count"])
    room = f + sum(max(0, -(-o // P) - -(-(k + n) // P)) for o, k, n in zip(old, keep, new))
    asked, total = 0, []
    for o, k, n in zip(old, keep, new):
        want = -(-(k + n) // P) - -(-o // P)
        asked += max(0, want)
        total.append(k + (n if want <= 0 or asked <= room else 0))
    free = stack[:f]
    for b, (o, t) in enumerate(zip(old, total)):
        free += table[b][-(-t // P): -(-o // P)]
    for b, (o, t) in enumerate(zip(old, total)):
        for j in range(-(-o // P), -(-t // P)):
            table[b][j] = free.pop()
    cu, seqs, positions, slots = [0], [], [], []
    for b, (k, t) in enumerate(zip(keep, total)):
        cu.append(cu[-1] + t - k)
        for pos in range(k, t):
            seqs.append(b)
            positions.append(pos)
            slots.append(table[b][pos // P] * P + pos % P)
    stack[f:max(f, len(free))] = free[f:]
    behind = [-1] * (s["seqs"].numel() - len(seqs))

    def whole(x, like):
        return torch.tensor(x, dtype=like.dtype, device=like.device)

    return {"table": whole(table, s["table"]), "stack": whole(stack, s["stack"]), "count": whole([len(free)], s["count"]),
            "kv_len": whole(total, s["kv_len"]), "cu_new": whole(cu, s["cu_new"]), "seqs": whole(seqs + behind, s["seqs"]),
            "positions": whole(positions + behind, s["positions"]), "slots": whole(slots + behind, s["slots"])}


def _exact_verify(s):
    c, cu, tokens = s["case"], s["cu_new"].tolist(), s["tokens"].tolist()
    u, v = s["u_accept"].tolist(), s["u_sample"].tolist()
    out, accepted, keep = [], [], []
    for b in range(c["batch"]):
        n, a = cu[b + 1] - cu[b] - 1, 0
        for a in range(n + 1):
            r = cu[b] + a
            if a == n:
                rest = s["probs"][r].double()
                break
            d = tokens[r + 1]
            if not u[r] * (1.0 if s["draft_probs"] is None else float(s["draft_probs"][r, d])) < float(s["probs"][r, d]):
                rest = s["probs"][r].double()
                if s["draft_probs"] is None:
                    rest[d] = 0.0
                else:
                    rest = torch.relu(rest - s["draft_probs"][r].double())
                break
        sums = torch.cumsum(rest, 0)
        if not float(sums[-1]) > 0:
            rest = s["probs"][r].double()
            sums = torch.cumsum(rest, 0)
        beyond = torch.nonzero(sums > v[b] * sums[-1])
        t = int(beyond[0]) if len(beyond) else int(torch.nonzero(rest > 0)[-1])
        taken = tokens[cu[b] + 1: cu[b] + 1 + a]
        out.append(taken + [t] + [-1] * (c["drafts"] - a))
        accepted.append(a)
        keep.append(int(s["kv_len"][b]) - (n - a))

    def whole(x, like):
        return torch.tensor(x, dtype=like.dtype, device=like.device)

    return {"accepted": whole(accepted, s["accepted"]), "tokens": whole(out, s["out"]), "kv_keep": whole(keep, s["kv_keep"])}
