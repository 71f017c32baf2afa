"""Cases of the attention layers between the recurrences, their plain forms and their definitions in 64 bits.

Four operators, in the order in which a server's step calls them:

* the plan of a paged key-value cache: new blocks for the requests that need them, and each new token's slot;
* the writing of the new tokens' keys and values into the cache (bf16, or e4m3 with a scale a head);
* attention of one new token of every request over the paged cache;
* attention of prompts, dense or packed, causal, with an optional window and first tokens that stay visible.

Prompts are those of this repository's prefill workloads: 64 to 16,381 tokens, a packed batch of 32
candidate prompts of 200 to 4,096 tokens, generation for 1 and 128 sequences; 32 query heads of 128.
"""

import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0


# ---- cases ------------------------------------------------------------------------------------

def listed():
    packed = dict(B=32, T=0, packed=True, lo=200, hi=4096, lens=0)
    heads = dict(Hq=32, Hkv=8, d=128)
    return [
        # one new token for each of 128 requests in generation: a few of them begin a block; only latency counts
        dict(name="plan_step_b128", op="plan", B=128, new=False, lo=200, hi=4096, lens=1, page=64, spare=64),
        # the blocks and slots of 32 candidate prompts that are taken in at once
        dict(name="plan_varlen32", op="plan", B=32, new=True, lo=200, hi=4096, lens=0, page=64, spare=64),
        # the new tokens' keys and values of 128 requests in generation, into an 8-bit cache
        dict(name="append_step_b128_e4m3", op="append", T=128, **heads, page=64, e4m3=True),
        # those of 32 candidate prompts (72,102 tokens)
        dict(name="append_varlen32", op="append", T=72102, **heads, page=64, e4m3=False),
        # one request at the default prompt limit: the split over its length decides
        dict(name="step_b1_t4096", op="step", B=1, lo=4096, hi=4096, lens=0, **heads, page=64, e4m3=False, window=0,
             sinks=0),
        # 128 requests of ragged lengths
        dict(name="step_b128", op="step", B=128, lo=200, hi=4096, lens=2, **heads, page=64, e4m3=False, window=0,
             sinks=0),
        # 32 long requests of ragged lengths over an 8-bit cache in small blocks
        dict(name="step_b32_e4m3", op="step", B=32, lo=1024, hi=16381, lens=3, **heads, page=16, e4m3=True, window=0,
             sinks=0),
        # 128 long requests that look back 1,024 tokens, and at their first four
        dict(name="step_b128_w1024", op="step", B=128, lo=1024, hi=8192, lens=4, **heads, page=64, e4m3=False,
             window=1024, sinks=4),
        # the smallest prompt: one tile, one narrow head; only latency counts
        dict(name="attn_t64_d32", op="attn", B=1, T=64, packed=False, Hq=1, Hkv=1, d=32, window=0, sinks=0),
        # one candidate prompt at the default limit
        dict(name="attn_t4096", op="attn", B=1, T=4096, packed=False, **heads, window=0, sinks=0),
        # 32 candidate prompts of ragged lengths in one packed batch, windowed
        dict(name="attn_varlen32_w1024", op="attn", **packed, **heads, window=1024, sinks=4),
        # the longest prompt (a ragged last tile), few shared key heads
        dict(name="attn_t16381", op="attn", B=1, T=16381, packed=False, Hq=16, Hkv=2, d=128, window=0, sinks=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("plan", "append", "step", "step", "attn", "attn"))
    page = rng.choice((16, 32, 48, 64, 128, 256))
    seed = rng.randrange(1 << 20)
    if op == "plan":
        new = rng.random() < 0.5
        hi = _log(rng, 1, 4096)
        return dict(op=op, B=_log(rng, 1, 32 if new else 1024), new=new, lo=rng.choice((0, hi // 2)), hi=hi, lens=seed,
                    page=page, spare=rng.choice((-3, 0, 5, 300)))
    Hkv = rng.choice((1, 2, 3, 4, 8))
    heads = dict(Hq=Hkv * rng.choice((1, 2, 3, 4, 5, 8, 16)), Hkv=Hkv, d=rng.choice((32, 64, 80, 96, 128)))
    if op == "append":
        return dict(op=op, T=_log(rng, 1, 72102), **heads, page=page, e4m3=rng.random() < 0.5)
    view = dict(window=0, sinks=0)
    if rng.random() < 0.5:
        view = dict(window=_log(rng, 16, 4096), sinks=rng.choice((0, 1, 4, 150)))
    if op == "step":
        hi = _log(rng, 1, 16381)
        most = max(1, (128 * 4096 * 8 * 128) // (hi * Hkv * heads["d"]))
        return dict(op=op, B=_log(rng, 1, min(128, most)), lo=rng.choice((1, hi // 2, hi)) or 1, hi=hi, lens=seed, **heads,
                    page=page, e4m3=rng.random() < 0.5, **view)
    if rng.random() < 0.5:
        hi = _log(rng, 1, 4096)
        most = max(1, int(16 * 128 * 16381 ** 2 / (heads["Hq"] * heads["d"] * hi * hi)))
        batch = dict(B=_log(rng, 1, min(32, most)), T=0, packed=True, lo=rng.choice((0, hi // 2)), hi=hi, lens=seed)
    else:
        B = rng.choice((1, 1, 2, 3))
        top = math.sqrt(16 * 128 * 16381 ** 2 / (heads["Hq"] * heads["d"] * B))
        batch = dict(B=B, T=_log(rng, 1, min(16381 // B, top)), packed=False)
    return dict(op=op, **batch, **heads, **view)


def _lengths(case):
    """Tokens of each sequence (attn), cached tokens (step, plan in generation), or new ones (plan of prompts)."""
    if case["op"] == "attn" and not case["packed"]:
        return [case["T"]] * case["B"]
    lens = [int(n) for n in np.random.default_rng(case["lens"]).integers(case["lo"], case["hi"] + 1, case["B"])]
    return [max(lens[0], 1)] + lens[1:]


def _seen(n, m, window, sinks):
    """Visible (query, key) pairs of n queries that end a sequence of m keys."""
    p = np.arange(m - n, m, dtype=np.int64)
    if window == 0:
        return int((p + 1).sum())
    far = np.maximum(p + 1 - window, 0)  # keys before the window
    return int((p + 1 - far + np.minimum(far, sinks)).sum())


def work(case):
    op = case["op"]
    if op == "plan":
        lens, page = np.array(_lengths(case), dtype=np.int64), case["page"]
        old, new = (np.zeros_like(lens), lens) if case["new"] else (lens, np.ones_like(lens))
        taken = max(0, int((-(-(old + new) // page) - -(-old // page)).sum()) + min(0, case["spare"]))
        T, B = int(new.sum()), case["B"]
        return {"bytes": 4 * (T + 2 * B + (B + 1 if case["new"] else 0) + 2 * taken + B + 3), "flops": 4 * T}
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    if op == "append":
        return {"bytes": 2 * case["T"] * Hkv * d * (2 + (1 if case["e4m3"] else 2)) + 4 * case["T"],
                "flops": 2 * case["T"] * Hkv * d if case["e4m3"] else 0}
    lens = _lengths(case)
    if op == "step":
        seen = sum(_seen(1, n, case["window"], case["sinks"]) for n in lens if n > 0)
        return {"bytes": 2 * seen * Hkv * d * (1 if case["e4m3"] else 2) + 2 * len(lens) * Hq * d * 2 +
                4 * (len(lens) + seen // case["page"]), "flops": 4 * seen * Hq * d}
    seen = sum(_seen(n, n, case["window"], case["sinks"]) for n in lens)
    return {"bytes": 2 * sum(lens) * (Hq + Hkv) * d * 2, "flops": 4 * seen * Hq * d}


# ---- inputs -----------------------------------------------------------------------------------

def prepare(case, seed):
    """A program's tensors before the call: slices of the projection's output, the cache with its blocks in the
    order in which they came free, output buffers."""
    dev = torch.device("cuda" if torch.cuda.is_available() else "cpu")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    bf16, i32 = torch.bfloat16, torch.int32

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    def shuffled(n):
        return torch.randperm(n, generator=gen, device=dev).to(i32)

    op, s = case["op"], dict(case)
    if op == "plan":
        lens, page, B = _lengths(case), case["page"], case["B"]
        s["old"] = torch.tensor([0] * B if case["new"] else lens, dtype=i32, device=dev)
        s["cu"] = None
        s["T"] = sum(lens) if case["new"] else B
        if case["new"]:
            s["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=i32, device=dev)
        held = [0 if case["new"] else -(-n // page) for n in lens]
        most = max(lens) if case["new"] else max(lens) + 1
        # all that are needed and some to spare, or a few too few: the last requests then have to wait
        total = max(sum(held), sum(-(-(n if case["new"] else n + 1) // page) for n in lens) + case["spare"])
        blocks = shuffled(total)
        s["table"] = torch.full((B, -(-most // page)), -1, dtype=i32, device=dev)
        at = 0
        for b, n in enumerate(held):
            s["table"][b, :n] = blocks[at : at + n]
            at += n
        s["free"] = torch.zeros(max(total, 1), dtype=i32, device=dev)
        s["free"][: total - at] = blocks[at:]
        s["count"] = torch.tensor([total - at], dtype=i32, device=dev)
        s["slots"] = torch.empty(s["T"], dtype=i32, device=dev)
        s["new_lens"], s["new_count"], s["refused"] = (torch.empty(n, dtype=i32, device=dev) for n in (B, 1, 1))
        return s
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    if op in ("append", "step"):
        page = case["page"]
        cache_type = torch.float8_e4m3fn if case["e4m3"] else bf16
        # scales from a calibration's largest values, a head each
        s["ks"], s["vs"] = ((4.0 + torch.rand(Hkv, generator=gen, device=dev)) / E4M3_MAX if case["e4m3"] else None
                            for _ in range(2))
    if op == "append":
        T = case["T"]
        n = -(-T // page) + 3
        qkv = normal(T, (Hq + 2 * Hkv) * d).to(bf16)
        s["k"] = qkv[:, Hq * d : (Hq + Hkv) * d].unflatten(1, (Hkv, d))
        s["v"] = qkv[:, (Hq + Hkv) * d :].unflatten(1, (Hkv, d))
        # whole blocks, in any order, filled one after the other
        s["slots"] = (shuffled(n)[:-3, None] * page + torch.arange(page, dtype=i32, device=dev)).flatten()[:T].contiguous()
        s["kc"], s["vc"] = (torch.zeros(n, Hkv, page, d, dtype=cache_type, device=dev) for _ in range(2))
        return s
    if op == "step":
        lens = _lengths(case)
        B, held = case["B"], [-(-n // page) for n in lens]
        n = sum(held) + 3
        s["q"] = (1.5 * normal(B, (Hq + 2 * Hkv) * d)).to(bf16)[:, : Hq * d].unflatten(1, (Hq, d))
        for name, scale in (("kc", s["ks"]), ("vc", s["vs"])):
            s[name] = torch.empty(n, Hkv, page, d, dtype=cache_type, device=dev)
            for part in s[name].split(max(1, (1 << 28) // (Hkv * page * d))):
                values = normal(*part.shape)
                if scale is not None:
                    values = torch.clamp(values / scale[:, None, None], -E4M3_MAX, E4M3_MAX)
                part.copy_(values.to(cache_type))
        blocks = shuffled(n)
        s["table"] = torch.full((B, max(held)), -1, dtype=i32, device=dev)
        at = 0
        for b, m in enumerate(held):
            s["table"][b, :m] = blocks[at : at + m]
            at += m
        s["n"] = torch.tensor(lens, dtype=i32, device=dev)
        s["out"] = torch.empty(B, Hq, d, dtype=bf16, device=dev)
        return s
    lens = _lengths(case)
    T = sum(lens)
    qkv = normal(T, (Hq + 2 * Hkv) * d).to(bf16)
    s["q"] = qkv[:, : Hq * d].unflatten(1, (Hq, d))
    s["k"] = qkv[:, Hq * d : (Hq + Hkv) * d].unflatten(1, (Hkv, d))
    s["v"] = qkv[:, (Hq + Hkv) * d :].unflatten(1, (Hkv, d))
    s["cu"] = None
    if case["packed"]:
        s["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=i32, device=dev)
    s["each"] = lens  # the server knows its requests' lengths
    s["out"] = torch.empty(T, Hq, d, dtype=bf16, device=dev)
    return s


# ---- one pass ---------------------------------------------------------------------------------

def run(s):
    if own:
        return _run_own(s)
    return {"plan": _plan, "append": _append, "step": _step, "attn": _attn}[s["op"]](s)


def _run_own(s):
    from hybrid_linear_attention_prefill_gb300 import gdn

    op = s["op"]
    if op == "plan":
        slots, lens, count, refused = gdn.cache_plan(s["old"], s["table"], s["free"], s["count"], s["cu"], page=s["page"],
                                                     slots=s["slots"], new_lens=s["new_lens"],
                                                     new_count=s["new_count"], refused=s["refused"])
        return {"slots": slots, "lens": lens, "count": count, "refused": refused, "table": s["table"]}
    if op == "append":
        gdn.cache_append(s["k"], s["v"], s["kc"], s["vc"], s["slots"], s["ks"], s["vs"])
        return {"k": s["kc"], "v": s["vc"]}
    if op == "step":
        out, _ = gdn.attention_step(s["q"], s["kc"], s["vc"], s["table"], s["n"], s["ks"], s["vs"], window=s["window"],
                                    sinks=s["sinks"], out=s["out"])
        return {"y": out}
    out, _ = gdn.attention(s["q"], s["k"], s["v"], s["cu"], B=s["B"], window=s["window"], sinks=s["sinks"],
                           out=s["out"])
    return {"y": out}


# ---- plain forms: elementary torch operations in 32 bits ----------------------------------------

def _plan(s):
    """Blocks in the requests' order from the top of the stack of free ones, then a slot for every token."""
    dev, page, T = s["old"].device, s["page"], s["T"]
    old, W = s["old"].long(), s["table"].shape[1]
    B = old.numel()
    cu = s["cu"].long() if s["cu"] is not None else torch.arange(B + 1, device=dev)
    total = old + cu[1:] - cu[:-1]
    have, want = (old + page - 1) // page, (total + page - 1) // page
    able = (old >= 0) & (want <= W)
    need = torch.where(able, want - have, 0)
    base = torch.cumsum(need, 0) - need
    granted = able & ((need == 0) | (base + need <= s["count"]))
    taken = torch.where(granted & (need > 0), base + need, 0).amax().reshape(1)
    col = torch.arange(W, device=dev)
    fresh = granted[:, None] & (col >= have[:, None]) & (col < want[:, None])
    at = s["count"] - 1 - base[:, None] - (col - have[:, None])
    s["table"].copy_(torch.where(fresh, s["free"][at.clamp(0, s["free"].numel() - 1)], s["table"]))
    t = torch.arange(T, device=dev)
    b = (torch.searchsorted(cu, t, right=True) - 1).clamp(0, B - 1)
    p = old[b] + t - cu[b]
    ok = granted[b] & (t < cu[-1])
    block = s["table"][b, (p // page).clamp(0, W - 1)].long()
    slots = torch.where(ok & (block >= 0), block * page + p % page, -1)
    i32 = torch.int32
    return {"slots": slots.to(i32), "lens": torch.where(granted, total, old).to(i32), "count": (s["count"] - taken).to(i32),
            "refused": (~granted & (old >= 0)).sum().reshape(1).to(i32), "table": s["table"]}


def _append(s):
    page, slots = s["page"], s["slots"].long()
    for x, cache, scale in ((s["k"], s["kc"], s["ks"]), (s["v"], s["vc"], s["vs"])):
        x = x.float()
        if scale is not None:
            x = torch.clamp(x / scale[:, None], -E4M3_MAX, E4M3_MAX)
        cache[slots // page, :, slots % page] = x.to(cache.dtype)
    return {"k": s["kc"], "v": s["vc"]}


def _soft(scores, seen, v):
    """Rows of scores and which of them count, to weighted sums of v: rows that see nothing give 0."""
    scores = torch.where(seen, scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    w = torch.exp(scores - torch.where(top == -math.inf, 0.0, top))
    total = w.sum(-1, keepdim=True)
    return torch.matmul(w, v) / torch.where(total == 0, 1.0, total)


def _step(s):
    B, Hq, d = s["q"].shape
    Hkv, page = s["Hkv"], s["page"]
    dev, window, sinks = s["q"].device, s["window"], s["sinks"]
    most, n = s["table"].shape[1] * page, s["n"].long()[:, None]
    if 0 < window and window + sinks < most:  # only the positions that may be seen
        first = torch.arange(sinks, device=dev).expand(B, sinks)
        last = n - window + torch.arange(window, device=dev)
        at = torch.cat([first, last], 1)
        seen = torch.cat([first < n, last >= sinks], 1)
    else:
        at = torch.arange(most, device=dev).expand(B, most)
        seen = (at < n) & ((at >= n - window) | (at < sinks) if window else True)
    at = torch.where(seen, at, 0)
    block = torch.gather(s["table"].long(), 1, at // page).clamp_min(0)
    k, v = (c[block, :, at % page].float().transpose(1, 2) for c in (s["kc"], s["vc"]))  # B, Hkv, keys, d
    if s["ks"] is not None:
        k, v = k * s["ks"][:, None, None], v * s["vs"][:, None, None]
    q = s["q"].float().reshape(B, Hkv, Hq // Hkv, d)
    scores = torch.matmul(q, k.transpose(2, 3)) / math.sqrt(d)
    return {"y": _soft(scores, seen[:, None, None], v).reshape(B, Hq, d).to(torch.bfloat16)}


def _attn(s):
    T, Hq, d = s["q"].shape
    Hkv, window, sinks, dev = s["Hkv"], s["window"], s["sinks"], s["q"].device
    G, out, at = Hq // Hkv, torch.empty(T, Hq, d, dtype=torch.bfloat16, device=dev), 0
    for n in s["each"]:
        q = s["q"][at : at + n].float().unflatten(1, (Hkv, G)).permute(1, 2, 0, 3)  # Hkv, G, n, d
        k, v = (s[x][at : at + n].float().transpose(0, 1)[:, None] for x in ("k", "v"))
        for i in range(0, n, 1024):
            e = min(i + 1024, n)
            lo = max(0, i + 1 - window) if window else 0
            j = torch.arange(lo, e, device=dev)
            if lo > 0 and sinks:
                j = torch.cat([torch.arange(min(sinks, lo), device=dev), j])
            p = torch.arange(i, e, device=dev)[:, None]
            seen = (j <= p) & ((j > p - window) | (j < sinks) if window else True)
            kj, vj = (k[:, :, j], v[:, :, j]) if window else (k[:, :, :e], v[:, :, :e])
            scores = torch.matmul(q[:, :, i:e], kj.transpose(2, 3)) / math.sqrt(d)
            out[at + i : at + e] = _soft(scores, seen, vj).permute(2, 0, 1, 3).flatten(1, 2).to(torch.bfloat16)
        at += n
    return {"y": out}


# ---- the definitions in 64 bits -----------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": _plan64, "append": _append64, "step": _step64, "attn": _attn64}[case["op"]](case, s)


def _plan64(case, s):
    """Request by request, token by token."""
    page, dev = case["page"], s["old"].device
    old, table = s["old"].tolist(), s["table"].tolist()
    cu = s["cu"].tolist() if s["cu"] is not None else list(range(case["B"] + 1))
    stack = s["free"].tolist()[: int(s["count"])]
    slots, lens, refused, short = [], [], 0, False
    for b, n in enumerate(old):
        new = cu[b + 1] - cu[b]
        need = -(-(n + new) // page) + (-n // page)
        short = short or need > len(stack)  # once a request goes without, so do those after it that need any
        if need > 0 and short:
            refused += 1
            lens.append(n)
            slots += [-1] * new
            continue
        for i in range(need):
            table[b][-(-n // page) + i] = stack.pop()
        slots += [table[b][p // page] * page + p % page for p in range(n, n + new)]
        lens.append(n + new)
    made = {"slots": slots, "lens": lens, "count": [len(stack)], "refused": [refused], "table": table}
    return {k: torch.tensor(v, dtype=torch.int32, device=dev) for k, v in made.items()}


def _append64(case, s):
    out = {}
    for name, scale in (("k", s["ks"]), ("v", s["vs"])):
        rows = s[name].double()
        if scale is not None:
            rows = (rows / scale.double()[None, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
        blocks = torch.zeros(s[name + "c"].shape, dtype=torch.float64, device=rows.device)
        tokens = blocks.transpose(1, 2).reshape(-1, *rows.shape[1:])
        tokens[s["slots"].long()] = rows
        out[name] = tokens.unflatten(0, (-1, case["page"])).transpose(1, 2).contiguous()
    return out


def _weigh64(q, k, v, hidden):
    logits = torch.einsum("...qd,...kd->...qk", q, k) / math.sqrt(q.shape[-1])
    return torch.einsum("...qk,...kd->...qd", torch.softmax(logits.masked_fill(hidden, -math.inf), -1), v)


def _step64(case, s):
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    y = torch.zeros(case["B"], Hq, d, dtype=torch.float64, device=s["q"].device)
    for b, n in enumerate(_lengths(case)):
        if n == 0:
            continue
        held = s["table"][b, : -(-n // case["page"])].long()
        k, v = (s[c][held].double().transpose(0, 1).flatten(1, 2)[:, :n] for c in ("kc", "vc"))
        if case["e4m3"]:
            k, v = k * s["ks"].double()[:, None, None], v * s["vs"].double()[:, None, None]
        j = torch.arange(n, device=y.device)
        hidden = (j < n - case["window"]) & (j >= case["sinks"]) if case["window"] else j < 0
        y[b] = _weigh64(s["q"][b].double().reshape(Hkv, Hq // Hkv, d), k, v, hidden).reshape(Hq, d)
    return {"y": y}


def _attn64(case, s):
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    window, sinks = case["window"], case["sinks"]
    y = torch.empty(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    at = 0
    for n in _lengths(case):
        for h in range(Hq):
            k, v = (s[x][at : at + n, h // (Hq // Hkv)].double() for x in ("k", "v"))
            for i in range(0, n, 4096):
                e = min(i + 4096, n)
                p = torch.arange(i, e, device=y.device)[:, None]
                j = torch.arange(e, device=y.device)
                hidden = j > p
                if window:
                    hidden = hidden | ((p - j >= window) & (j >= sinks))
                y[at + i : at + e, h] = _weigh64(s["q"][at + i : at + e, h].double(), k[:e], v[:e], hidden)
        at += n
    return {"y": y}
