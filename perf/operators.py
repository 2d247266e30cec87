"""Cases, plain forms and 64-bit values of the paged 8-bit key/value cache operators.

Two operators of one serving step, the attention half of a decoder layer beside
the routed-expert FFN:

* append  -- the step's keys and values (keys rotated by position) go into a
  paged E4M3 cache with one power-of-two scale for each page and head; the
  step's queries are rotated in the same call.
* attend  -- the step's queries attend over that cache: causal, ragged, grouped
  heads, with an optional window and an optional tanh cap on the scores.

With ``own`` false, ``run`` computes them with elementary torch operations in 32
bits; with ``own`` true it calls the library.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
SCALE_FLOOR = 1e-4            # the smallest block maximum a scale is taken from
WORKSPACE_BYTES = 64 << 20    # what a serving program sets aside once for split rows
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    base = {"dtype": "bf16", "dim": 128, "page": 64, "layout": "hnd", "ragged": False}
    append = dict(base, op="append", rot=128, interleaved=False)
    attend = dict(base, op="attend", window=0, softcap=0.0)
    return [
        # one user, one token: the latency of a decode step's append
        dict(append, name="append_one_token", batch=1, new=1, ctx=1000, q_heads=32, kv_heads=8),
        # a full decode batch, one token for each sequence, small pages
        dict(append, name="append_decode_batch", batch=256, new=1, ctx=2048, q_heads=32, kv_heads=8, page=16, ragged=True),
        # ragged chunks of prompts, half of each head rotated in adjacent pairs, token-major pages
        dict(append, name="append_ragged_chunks", batch=7, new=4099, ctx=777, q_heads=16, kv_heads=16, dim=64, page=32,
             dtype="f16", rot=32, interleaved=True, layout="nhd", ragged=True),
        # whole prompts: as many rows as the prefill workload of the FFN benchmark
        dict(append, name="append_prompts", batch=4, new=8192, ctx=0, q_heads=64, kv_heads=8),
        # one user, one token, a short context: the latency of a decode step's attention
        dict(attend, name="attend_one_sequence", batch=1, new=1, ctx=1009, q_heads=32, kv_heads=8),
        # a decode batch of very different lengths, small pages
        dict(attend, name="attend_decode_ragged", batch=64, new=1, ctx=16384, q_heads=32, kv_heads=8, page=16, ragged=True),
        # few users with long contexts
        dict(attend, name="attend_decode_long", batch=4, new=1, ctx=131072, q_heads=64, kv_heads=8, page=128),
        # draft tokens checked together, an odd group of heads
        dict(attend, name="attend_draft", batch=32, new=4, ctx=8192, q_heads=28, kv_heads=4, dtype="f16", ragged=True),
        # a head of its own for each query head, short heads, a window and capped scores
        dict(attend, name="attend_window_capped", batch=16, new=1, ctx=8000, q_heads=16, kv_heads=16, dim=64, page=32,
             layout="nhd", window=1024, softcap=30.0, ragged=True),
        # a whole prompt
        dict(attend, name="attend_prompt", batch=1, new=8192, ctx=0, q_heads=64, kv_heads=8),
        # ragged chunks of prompts on contexts that are already cached
        dict(attend, name="attend_ragged_chunks", batch=5, new=1111, ctx=12000, q_heads=40, kv_heads=8, dim=64,
             dtype="f16", ragged=True),
        # prompts under a window with capped scores
        dict(attend, name="attend_prompts_window", batch=3, new=2500, ctx=900, q_heads=32, kv_heads=4, window=600,
             softcap=50.0, ragged=True),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi, max(lo, v))


def draw(rng):
    most = {op: [max(work(c)[k] for c in listed() if c["op"] == op) for k in ("bytes", "flops")] for op in ("append", "attend")}
    while True:
        kv_heads = rng.choice([1, 2, 4, 8, 16])
        dim = rng.choice([64, 128])
        case = {"op": rng.choice(["append", "attend"]), "dtype": rng.choice(["bf16", "f16"]), "dim": dim,
                "page": rng.choice([16, 32, 64, 128]), "layout": rng.choice(["hnd", "nhd"]), "ragged": rng.random() < 0.7,
                "kv_heads": kv_heads, "q_heads": kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8, 16])}
        form = rng.choice(["one", "draft", "chunk"])      # decode, draft tokens, prompts
        case["batch"] = _spread(rng, 1, {"one": 256, "draft": 64, "chunk": 8}[form])
        case["new"] = {"one": 1, "draft": rng.randint(2, 9), "chunk": _spread(rng, 10, 8192)}[form]
        case["ctx"] = 0 if rng.random() < 0.1 else _spread(rng, 1, 2048 if case["op"] == "append" else 131072)
        if case["op"] == "append":
            case["rot"] = rng.choice([0, dim // 4, dim // 2, dim])
            case["interleaved"] = rng.random() < 0.5
        else:
            case["window"] = _spread(rng, 1, 4096) if rng.random() < 0.25 else 0
            case["softcap"] = rng.choice([20.0, 30.0, 50.0]) if rng.random() < 0.25 else 0.0
        if 3072 in (case["new"], case["ctx"], case["q_heads"] * dim, (case["q_heads"] + 2 * kv_heads) * dim):
            continue
        new, total = _lengths(case)
        # the plain form's padded keys, and its scores, have to fit the card
        room = 4 * case["batch"] * max(total) * (2 * kv_heads * dim + case["q_heads"] * case["new"])
        if sum(new) and room <= (24 << 30) and all(work(case)[k] <= m for k, m in zip(("bytes", "flops"), most[case["op"]])):
            return case


def _lengths(case):
    """New tokens and total length (new ones included) of each sequence: a property of the case."""
    r = random.Random("lengths %d %d %d" % (case["batch"], case["new"], case["ctx"]))
    new, total = [], []
    for _ in range(case["batch"]):
        n, c = case["new"], case["ctx"]
        if case["ragged"]:
            n = n if n == 1 else r.randint(1, n)
            c = r.randint(c // 8, c)
        new.append(n)
        total.append(n + c)
    return new, total


def _visible(case):
    """(key/value tokens that have to be read, pairs of a token and a visible token) over all sequences."""
    read = pairs = 0
    for n, total in zip(*_lengths(case)):
        w = case["window"] or total
        read += total - max(0, total - n - w + 1)
        pairs += sum(min(w, total - n + i + 1) for i in range(n))
    return read, pairs


def work(case):
    new, total = _lengths(case)
    tokens, heads, dim = sum(new), case["kv_heads"], case["dim"]
    queries = 2 * tokens * case["q_heads"] * dim
    if case["op"] == "append":
        pages = sum((t - 1) // case["page"] - (t - n) // case["page"] + 1 for n, t in zip(new, total) if n)
        moved = 2 * tokens * heads * dim * (2 + 1) + 2 * queries + 4 * tokens * case["rot"] + 2 * pages * heads * 8 + 4 * pages
        return {"bytes": moved, "flops": tokens * (3 * case["rot"] * (case["q_heads"] + heads) + 4 * heads * dim)}
    read, pairs = _visible(case)
    pages = -(-read // case["page"])
    return {"bytes": 2 * read * heads * dim + 8 * pages * heads + 4 * pages + 2 * queries, "flops": 4 * pairs * case["q_heads"] * dim}


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev).manual_seed(seed)
    new, total = _lengths(case)
    B, P, H, D = case["batch"], case["page"], case["kv_heads"], case["dim"]
    dtype, tokens = TYPES[case["dtype"]], sum(new)
    counts = [-(-t // P) for t in total]
    pool = sum(counts) + 3
    order = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
    table = torch.full((B, max(counts)), -1, dtype=torch.int32, device=dev)   # -1 past a sequence's pages
    where = torch.arange(max(counts), device=dev)[None] < torch.tensor(counts, device=dev)[:, None]
    table[where] = order[: sum(counts)]
    cu = torch.tensor([sum(new[:i]) for i in range(B + 1)], dtype=torch.int32, device=dev)
    kv_len = torch.tensor(total, dtype=torch.int32, device=dev)

    def cache(gain):
        # values of different size from head to head and page to page, as a model's are, in 8 bits with their scales
        shape = (pool, H, P, D) if case["layout"] == "hnd" else (pool, P, H, D)
        codes = torch.empty(shape, dtype=torch.uint8, device=dev)
        ordered = codes if case["layout"] == "hnd" else codes.transpose(1, 2)
        scale = torch.empty((pool, H), dtype=torch.float32, device=dev)
        size = gain * torch.exp(0.3 * torch.randn((pool, H, 1, 1), generator=g, device=dev))
        step = max(1, (1 << 27) // (H * P * D))
        for i in range(0, pool, step):
            x = size[i:i + step] * torch.randn((min(step, pool - i), H, P, D), generator=g, device=dev)
            s = _plain_scale(x.abs().amax((2, 3)))
            scale[i:i + step] = s
            ordered[i:i + step] = (x / s[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        return ordered, scale

    k_cache, k_scale = cache(1.0)
    v_cache, v_scale = cache(0.5)
    # the sequences whose new tokens join a page that holds earlier ones
    joins = torch.tensor([b for b in range(B) if (total[b] - new[b]) % P], dtype=torch.int64, device=dev)
    state = {"case": case, "joins": joins, "k_cache": k_cache, "v_cache": v_cache, "k_scale": k_scale, "v_scale": v_scale,
             "table": table, "cu": cu, "kv_len": kv_len}
    # queries, keys and values as slices of one projection's output, as a layer has them
    heads = case["q_heads"] + (2 * H if case["op"] == "append" else 0)
    rows = torch.randn((tokens, heads, D), generator=g, device=dev)
    rows[:, : case["q_heads"]] *= 2.0
    rows = rows.to(dtype)
    state["q"] = rows[:, : case["q_heads"]]
    state["out"] = torch.empty((tokens, case["q_heads"], D), dtype=dtype, device=dev)
    if case["op"] == "append":
        state["k"], state["v"] = rows[:, case["q_heads"]: case["q_heads"] + H], rows[:, case["q_heads"] + H:]
        if case["rot"]:
            half = case["rot"] // 2
            angle = torch.arange(max(total), device=dev)[:, None] * 10000.0 ** (-torch.arange(half, device=dev) / half)
            state["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
        else:
            state["cos_sin"] = None
    else:
        state["sm_scale"] = 1.0 / math.sqrt(D)
        state["workspace"] = torch.zeros(WORKSPACE_BYTES, dtype=torch.uint8, device=dev)
    return state


def run(state):
    if own:
        return _own_append(state) if state["case"]["op"] == "append" else _own_attend(state)
    return _plain_append(state) if state["case"]["op"] == "append" else _plain_attend(state)


def _own_append(s):
    import fp8_grouped_expert_x128_gb300 as moe
    moe.moe_kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"], s["cu"], s["kv_len"],
                      cos_sin=s["cos_sin"], flags=moe.MOE_KV_INTERLEAVED if s["case"]["interleaved"] else 0, q=s["q"],
                      q_out=s["out"])
    return _appended(s, s["out"])


def _own_attend(s):
    import fp8_grouped_expert_x128_gb300 as moe
    c = s["case"]
    return moe.moe_kv_attention(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"], s["cu"],
                                s["kv_len"], s["out"], s["workspace"], sm_scale=s["sm_scale"], max_q=c["new"],
                                window=c["window"], softcap=c["softcap"])


def _appended(s, q):
    return {"k_cache": s["k_cache"].view(torch.float8_e4m3fn), "v_cache": s["v_cache"].view(torch.float8_e4m3fn),
            "k_scale": s["k_scale"], "v_scale": s["v_scale"], "q": q}


# ---------------------------------------------------------------- plain forms
def _plain_scale(amax):
    """The smallest power of two that takes a block's maximum to at most 448."""
    m, e = torch.frexp(amax.float().clamp(min=SCALE_FLOOR))
    return torch.ldexp(torch.ones_like(m), e - 9 + (m > 0.875).to(e.dtype))


def _plain_tokens(s):
    """For each new token: its sequence, its number among the sequence's new tokens, its position."""
    cu, new = s["cu"].long(), (s["cu"][1:] - s["cu"][:-1]).long()
    t = torch.arange(s["q"].shape[0], device=cu.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    i = t - cu[b]
    return b, i, s["kv_len"].long()[b] - new[b] + i


def _plain_rotate(x, s, pos):
    """x [tokens, heads, dim] in 32 bits, its first `rot` dimensions turned by the position's angles."""
    x, rot = x.float(), s["case"]["rot"]
    if not rot:
        return x
    cos, sin = (c[:, None] for c in s["cos_sin"][pos].split(rot // 2, 1))
    if s["case"]["interleaved"]:
        a, b = x[..., :rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_append(s):
    P, table = s["case"]["page"], s["table"].long()
    b, i, pos = _plain_tokens(s)
    page, slot = table[b, pos // P], pos % P
    first = (s["kv_len"].long() - (s["cu"][1:] - s["cu"][:-1]).long())[s["joins"]]
    joined = table[s["joins"], first // P]
    kept = (torch.arange(P, device=table.device)[None] < (first % P)[:, None])[:, None, :, None]
    for x, cache, scale in ((_plain_rotate(s["k"], s, pos), s["k_cache"], s["k_scale"]),
                            (s["v"].float(), s["v_cache"], s["v_scale"])):
        H = x.shape[1]
        need = torch.zeros_like(scale).scatter_reduce_(0, page[:, None].expand(-1, H), x.abs().amax(2), "amax")
        touched = torch.zeros_like(scale).index_fill_(0, page, 1.0) > 0
        fresh = torch.zeros_like(scale).index_fill_(0, page, 0.0).scatter_reduce_(
            0, page[:, None].expand(-1, H), (slot == 0).float()[:, None].expand(-1, H), "amax") > 0
        wanted = torch.where(touched, _plain_scale(need), 0.0)
        scale_new = torch.where(touched, torch.maximum(torch.where(fresh, 0.0, scale), wanted), scale)
        # tokens that were there keep their values under the page's new scale
        old = cache[joined]
        factor = (scale / scale_new)[joined][:, :, None, None]
        again = (old.view(torch.float8_e4m3fn).float() * factor).to(torch.float8_e4m3fn).view(torch.uint8)
        cache[joined] = torch.where(kept, again, old)
        codes = (x / scale_new[page][:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        cache[page, :, slot] = codes.view(torch.uint8)
        scale.copy_(scale_new)
    s["out"].copy_(_plain_rotate(s["q"], s, pos))
    return _appended(s, s["out"])


def _plain_attend(s):
    c, cu, kv_len = s["case"], s["cu"].long(), s["kv_len"].long()
    B, N, H, D = c["batch"], c["new"], c["kv_heads"], c["dim"]
    G, dev = c["q_heads"] // H, cu.device
    table = s["table"].long().clamp(min=0)
    new = cu[1:] - cu[:-1]
    L = table.shape[1] * c["page"]
    j = torch.arange(L, device=dev)
    valid = (j[None] < kv_len[:, None])[:, None, :, None]

    def gathered(cache, scale):                              # [B, H, L, D] in 32 bits
        x = cache[table].view(torch.float8_e4m3fn).float() * scale[table][..., None, None]
        return torch.where(valid, x.transpose(1, 2).reshape(B, H, L, D), 0.0)

    i = torch.arange(N, device=dev)
    at = (cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)  # the sequences padded to the longest
    q = s["q"][at].float().view(B, N, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * N, D)
    score = q @ gathered(s["k_cache"], s["k_scale"]).transpose(2, 3) * s["sm_scale"]
    if c["softcap"]:
        score = c["softcap"] * torch.tanh(score / c["softcap"])
    pos = (kv_len - new)[:, None] + i                        # [B, N]
    seen = j <= pos[..., None]
    if c["window"]:
        seen &= j > pos[..., None] - c["window"]
    seen = seen[:, None, None].expand(B, H, G, N, L).reshape(B, H, G * N, L)
    score = torch.where(seen, score, -torch.inf)
    p = torch.exp(score - score.amax(3, keepdim=True))
    p /= p.sum(3, keepdim=True)
    y = (p @ gathered(s["v_cache"], s["v_scale"])).view(B, H, G, N, D)
    b, i, _ = _plain_tokens(s)
    s["out"].copy_(y.permute(0, 3, 1, 2, 4)[b, i].reshape(-1, H * G, D))
    return s["out"]


# ---------------------------------------------------------------- 64-bit values
def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attend(s)


def _decoded(codes):
    """E4M3 codes as 64-bit values: sign, 4 bits of exponent with bias 7, 3 of mantissa."""
    bits = torch.arange(256, dtype=torch.int64, device=codes.device)
    expo, man = (bits >> 3) & 15, (bits & 7).double()
    mag = torch.where(expo == 0, man * 2.0 ** -9, (8 + man) * torch.exp2(expo.double() - 10))
    mag = torch.where((bits & 127) == 127, torch.nan, mag)
    return torch.where(bits >= 128, -mag, mag)[codes.long()]


def _to_e4m3(x):
    """64-bit values to the nearest E4M3 value, ties to the even one."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_append(s):
    c = s["case"]
    P, half = c["page"], c["rot"] // 2
    new, total = _lengths(c)
    tables = s["table"].tolist()

    def turned(x, n, t):
        x = x.double()
        if half:
            cs = s["cos_sin"][t - n:t].double()[:, None]
            z = torch.complex(cs[..., :half], cs[..., half:])
            pairs = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if c["interleaved"] else (x[..., :half], x[..., half:2 * half])
            w = torch.complex(*pairs) * z
            x = x.clone()
            if c["interleaved"]:
                x[..., 0:2 * half:2], x[..., 1:2 * half:2] = w.real, w.imag
            else:
                x[..., :half], x[..., half:2 * half] = w.real, w.imag
        return x

    out = {"q": torch.empty(s["out"].shape, dtype=torch.float64, device=s["out"].device)}
    for name in ("k", "v"):
        out[name + "_cache"] = _decoded(s[name + "_cache"])
        out[name + "_scale"] = s[name + "_scale"].double()
    t0 = 0
    for b, (n, t) in enumerate(zip(new, total)):
        out["q"][t0:t0 + n] = turned(s["q"][t0:t0 + n], n, t)
        for name in ("k", "v"):
            x = s[name][t0:t0 + n]
            x = turned(x, n, t) if name == "k" else x.double()
            a = t - n                                          # whole pages at a time: [pages, heads, P, D]
            lo, hi = a // P, -(-t // P)
            ids = torch.tensor(tables[b][lo:hi], device=x.device)
            values = torch.zeros(((hi - lo) * P,) + x.shape[1:], dtype=torch.float64, device=x.device)
            values[a - lo * P: t - lo * P] = x
            values = values.view(hi - lo, P, *x.shape[1:]).transpose(1, 2)
            number = torch.arange(lo * P, hi * P, device=x.device).view(hi - lo, 1, P, 1)
            amax = values.abs().amax((2, 3)).clamp(min=SCALE_FLOOR)
            scale = torch.exp2(torch.ceil(torch.log2(amax / E4M3_MAX)))
            before = out[name + "_scale"][ids]
            if a % P:
                scale[0] = torch.maximum(scale[0], before[0])
            codes = out[name + "_cache"][ids]
            kept = _to_e4m3(codes * (before / scale)[:, :, None, None])
            fresh = _to_e4m3(values / scale[:, :, None, None])
            codes = torch.where((number >= a) & (number < t), fresh, torch.where(number < a, kept, codes))
            out[name + "_cache"][ids] = codes
            out[name + "_scale"][ids] = scale
        t0 += n
    return out


def _exact_attend(s):
    c = s["case"]
    G = c["q_heads"] // c["kv_heads"]
    out = torch.empty(s["out"].shape, dtype=torch.float64, device=s["out"].device)
    t0 = 0
    for b, (n, t) in enumerate(zip(*_lengths(c))):
        ids = s["table"][b, : -(-t // c["page"])].long()
        j = torch.arange(t, device=ids.device)
        pos = torch.arange(t - n, t, device=ids.device)[:, None]
        hidden = (j > pos) | ((j <= pos - c["window"]) if c["window"] else (j < 0))
        for h in range(c["kv_heads"]):
            k, v = ((_decoded(s[x + "_cache"][ids, h]) * s[x + "_scale"][ids, h].double()[:, None, None]).flatten(0, 1)[:t]
                    for x in ("k", "v"))
            q = s["q"][t0:t0 + n, h * G:(h + 1) * G].double()
            score = torch.einsum("igd,jd->gij", q, k) * s["sm_scale"]
            if c["softcap"]:
                score = torch.tanh(score / c["softcap"]) * c["softcap"]
            p = torch.softmax(score.masked_fill_(hidden, -torch.inf), -1)
            out[t0:t0 + n, h * G:(h + 1) * G] = torch.einsum("gij,jd->igd", p, v)
        t0 += n
    return out
