"""Cases of the operators around the hybrid layers' recurrences, their plain forms and their definitions in 64 bits.

Three operators, for prompts (dense or packed batches) and for single tokens:

* the short causal convolution over the channels that feed a recurrence, with its carried inputs;
* the selective state space scan, one decay per (token, value head), with its carried state;
* the root-mean-square norm that opens a layer, with the residual's addition, and an output in
  bf16 or in 8 bits (e4m3) with scales.

Shapes are those of the prefill workloads of this repository: 16 key heads, 32 value heads of 128,
a state of 128, prompts of 64 to 16,381 tokens, a packed batch of 32 candidate prompts of 200 to
4,096 tokens, and decode batches of 1 and 128.
"""

import math

import numpy as np
import torch
import torch.nn.functional as F

own = False

BF16_STEP = 2  # bytes
CHUNK = 128    # tokens per chunk of the plain scan
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -96  # smallest |value| a scale is made for


# ---- cases ------------------------------------------------------------------------------------

def listed():
    heads = dict(Hk=16, Hv=32, dk=128, dv=128)
    packed = dict(B=32, T=0, packed=True, lo=200, hi=4096, lens=0)
    return [
        # the q, k, v (or x, B, C) channels of one candidate prompt at the default limit
        dict(name="conv_t4096", op="conv", B=1, T=4096, packed=False, C=8192, K=4, bias=True, init=False),
        # the same channels of 32 candidate prompts at once, each continuing from carried inputs
        dict(name="conv_varlen32", op="conv", **packed, C=8192, K=4, bias=True, init=True),
        # one token of each of 128 sequences in generation
        dict(name="conv_step_b128", op="conv_step", B=128, C=8192, K=4, bias=True),
        # the smallest prompt: one chunk, one narrow head; only latency counts
        dict(name="scan_t64_d32", op="scan", B=1, T=64, packed=False, Hk=1, Hv=1, dk=32, dv=32, gate=False,
             init=False, dt32=True),
        # a short prompt with as many key heads as value heads
        dict(name="scan_t1024_h16", op="scan", B=1, T=1024, packed=False, Hk=16, Hv=16, dk=128, dv=128, gate=True,
             init=False, dt32=False),
        # one candidate prompt at the default limit
        dict(name="scan_t4096", op="scan", B=1, T=4096, packed=False, **heads, gate=True, init=False, dt32=False),
        # 32 candidate prompts of ragged lengths in one packed batch
        dict(name="scan_varlen32", op="scan", **packed, **heads, gate=True, init=False, dt32=False),
        # the longest prompt (a ragged last chunk) with few heads, from a carried state
        dict(name="scan_t16381_h4_carry", op="scan", B=1, T=16381, packed=False, Hk=4, Hv=4, dk=128, dv=128,
             gate=True, init=True, dt32=False),
        # one token of one sequence: the launch is most of it
        dict(name="scan_step_b1", op="scan_step", B=1, **heads, gate=True, dt32=False),
        # one token of each of 128 sequences
        dict(name="scan_step_b128", op="scan_step", B=128, **heads, gate=True, dt32=False),
        # the norm before a layer, for one token in generation, to 8 bits with one scale a row
        dict(name="norm_r1_e4m3_row", op="norm", rows=1, D=4096, group=0, e4m3=True, residual=True),
        # the norm before a layer, for a prompt, to 8 bits with a scale per 128 columns
        dict(name="norm_r4096_e4m3_g128", op="norm", rows=4096, D=4096, group=128, e4m3=True, residual=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("conv", "conv_step", "scan", "scan", "scan_step", "norm"))
    if op == "norm":
        D = 8 * _log(rng, 8, 1024)
        rows = _log(rng, 1, min(72102, (72102 * 8192) // D))
        e4m3 = rng.random() < 0.6
        return dict(op=op, rows=rows, D=D, group=rng.choice((0, 32, 64, 128)) if e4m3 else 0, e4m3=e4m3,
                    residual=rng.random() < 0.7)
    if op == "conv_step":
        return dict(op=op, B=_log(rng, 1, 256), C=8 * _log(rng, 8, 1024), K=rng.choice((2, 3, 4)),
                    bias=rng.random() < 0.5)
    if op == "scan_step":
        Hk = _log(rng, 1, 16)
        return dict(op=op, B=_log(rng, 1, 128), Hk=Hk, Hv=Hk * rng.randint(1, max(1, 32 // Hk)),
                    dk=rng.choice((32, 64, 128)), dv=rng.choice((32, 64, 128)), gate=rng.random() < 0.5,
                    dt32=rng.random() < 0.5)
    if rng.random() < 0.5:
        n = _log(rng, 1, 32)
        hi = _log(rng, 1, 4096)
        batch = dict(B=n, T=0, packed=True, lo=rng.choice((0, hi // 8, hi // 2)), hi=hi, lens=rng.randrange(1 << 20))
    else:
        B = rng.choice((1, 1, 2, 3, 5))
        batch = dict(B=B, T=_log(rng, 1, 16381 // B), packed=False)
    if op == "conv":
        return dict(op=op, **batch, C=8 * _log(rng, 8, 1024), K=rng.choice((2, 3, 4)), bias=rng.random() < 0.5,
                    init=rng.random() < 0.5)
    Hk = _log(rng, 1, 16)
    return dict(op=op, **batch, Hk=Hk, Hv=Hk * rng.randint(1, max(1, 32 // Hk)), dk=rng.choice((32, 64, 128)),
                dv=rng.choice((32, 64, 128)), gate=rng.random() < 0.5, init=rng.random() < 0.5,
                dt32=rng.random() < 0.5)


def _lengths(case):
    if not case["packed"]:
        return [case["T"]] * case["B"]
    lens = [int(n) for n in np.random.default_rng(case["lens"]).integers(case["lo"], case["hi"] + 1, case["B"])]
    return [max(lens[0], 1)] + lens[1:]


def work(case):
    op = case["op"]
    if op == "norm":
        n = case["rows"] * case["D"]
        groups = -(-case["D"] // case["group"]) if case["group"] else 1
        reads = n * 2 * (2 if case["residual"] else 1) + case["D"] * 2
        writes = (n * 2 if case["residual"] else 0) + (n + case["rows"] * groups * 4 if case["e4m3"] else n * 2)
        return {"bytes": reads + writes, "flops": 5 * n}
    if op in ("conv", "conv_step"):
        B, C, K = case["B"], case["C"], case["K"]
        T = sum(_lengths(case)) if op == "conv" else B
        states = (1 + (op == "conv_step" or case["init"])) * B * C * (K - 1) * 2
        return {"bytes": 2 * T * C * 2 + C * K * 2 + (C * 2 if case["bias"] else 0) + states,
                "flops": T * C * (2 * K + 4)}
    B, Hk, Hv, dk, dv = (case[k] for k in ("B", "Hk", "Hv", "dk", "dv"))
    T = sum(_lengths(case)) if op == "scan" else B
    tokens = T * (Hv * dv * (3 if case["gate"] else 2) * 2 + 2 * Hk * dk * 2 + Hv * (4 if case["dt32"] else 2))
    states = (1 + (op == "scan_step" or case["init"])) * B * Hv * dv * dk * 4
    return {"bytes": tokens + states + 3 * Hv * 4, "flops": T * Hv * dv * dk * 5}


# ---- inputs -----------------------------------------------------------------------------------

def prepare(case, seed):
    """A program's tensors before the call: activations in bf16 (x, B and C as slices of the
    convolution's output, as they come), decay parameters in fp32, carried states, output buffers."""
    dev = torch.device("cuda" if torch.cuda.is_available() else "cpu")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    bf16 = torch.bfloat16

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device=dev)

    op, s = case["op"], {"op": case["op"]}
    if op == "norm":
        rows, D = case["rows"], case["D"]
        s["x"] = normal(rows, D).to(bf16)
        s["residual"] = (4.0 * normal(rows, D)).to(bf16) if case["residual"] else None
        s["weight"] = (1.0 + 0.1 * normal(D)).to(bf16)
        s["group"], s["e4m3"], s["eps"] = case["group"], case["e4m3"], 1e-6
        s["out"] = torch.empty(rows, D, dtype=torch.float8_e4m3fn if case["e4m3"] else bf16, device=dev)
        s["residual_out"] = torch.empty_like(s["x"]) if case["residual"] else None
        groups = -(-D // case["group"]) if case["group"] else 1
        s["scales"] = torch.empty(rows, groups, device=dev) if case["e4m3"] else None
        return s
    B = s["B"] = case["B"]
    s["cu"] = None
    if op in ("conv", "scan"):
        lens = _lengths(case)
        T = sum(lens)
        if case["packed"]:
            s["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=dev)
    else:
        T = B
    if op in ("conv", "conv_step"):
        C, K = case["C"], case["K"]
        s["x"] = normal(T, C).to(bf16)
        s["weight"] = (normal(C, K) / math.sqrt(K)).to(bf16)
        s["bias"] = (0.1 * normal(C)).to(bf16) if case["bias"] else None
        s["out"] = torch.empty_like(s["x"])
        if op == "conv":
            s["init"] = normal(B, K - 1, C).to(bf16) if case["init"] else None
            s["final"] = torch.empty(B, K - 1, C, dtype=bf16, device=dev)
        else:
            s["state"] = normal(B, K - 1, C).to(bf16)
        return s
    Hk, Hv, dk, dv = (case[k] for k in ("Hk", "Hv", "dk", "dv"))
    xbc = F.silu(normal(T, Hv * dv + 2 * Hk * dk)).to(bf16)
    s["x"] = xbc[:, : Hv * dv].unflatten(1, (Hv, dv))
    s["Bm"] = xbc[:, Hv * dv : Hv * dv + Hk * dk].unflatten(1, (Hk, dk))
    s["Cm"] = xbc[:, Hv * dv + Hk * dk :].unflatten(1, (Hk, dk))
    # steps of 0.001 to 0.1 around a learnt bias, decays of exp(-0.001) to exp(-1.6) a token
    step = torch.exp(math.log(1e-3) + uniform(Hv) * math.log(100.0))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    s["dt"] = (0.5 * normal(T, Hv)).to(torch.float32 if case["dt32"] else bf16)
    s["A"] = -(1.0 + 15.0 * uniform(Hv))
    s["D"] = 1.0 + 0.1 * normal(Hv)
    s["z"] = normal(T, Hv, dv).to(bf16) if case["gate"] else None
    s["out"] = torch.empty(T, Hv, dv, dtype=bf16, device=dev)
    if op == "scan":
        s["init"] = 0.1 * normal(B, Hv, dv, dk) if case["init"] else None
        s["final"] = torch.empty(B, Hv, dv, dk, device=dev)
    else:
        s["state"] = 0.1 * normal(B, Hv, dv, dk)
    return s


# ---- one pass ---------------------------------------------------------------------------------

def run(s):
    if own:
        return _run_own(s)
    return {"conv": _conv, "conv_step": _conv_step, "scan": _scan, "scan_step": _scan_step, "norm": _norm}[s["op"]](s)


def _run_own(s):
    from hybrid_linear_attention_prefill_gb300 import gdn

    op = s["op"]
    if op == "conv":
        out, fin = gdn.causal_conv(s["x"], s["weight"], s["bias"], s["cu"], s["init"], B=s["B"], out=s["out"],
                                   final_state=s["final"])
        return {"y": out, "state": fin}
    if op == "conv_step":
        out = gdn.causal_conv_step(s["x"], s["weight"], s["state"], s["bias"], out=s["out"])
        return {"y": out, "state": s["state"]}
    if op == "scan":
        out, fin = gdn.ssm_scan(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["D"], s["z"], s["dt_bias"], s["cu"],
                                s["init"], B=s["B"], out=s["out"], final_state=s["final"])
        return {"y": out, "state": fin}
    if op == "scan_step":
        out = gdn.ssm_step(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["state"], s["D"], s["z"], s["dt_bias"],
                           out=s["out"])
        return {"y": out, "state": s["state"]}
    out, scales, res = gdn.add_norm(s["x"], s["weight"], s["residual"], eps=s["eps"], group=s["group"], out=s["out"],
                                    scales=s["scales"], residual_out=s["residual_out"])
    return {k: v for k, v in (("y", out), ("scales", scales), ("residual", res)) if v is not None}


# ---- plain forms: elementary torch operations in 32 bits ----------------------------------------

def _silu(x):
    return x / (1.0 + torch.exp(-x))


def _softplus(x):
    return torch.where(x > 20.0, x, torch.log1p(torch.exp(torch.clamp(x, max=20.0))))


def _bounds(s, T):
    """Sequence boundaries and each token's sequence."""
    dev = s["x"].device
    cu = s["cu"].long() if s["cu"] is not None else torch.arange(s["B"] + 1, device=dev) * (T // s["B"])
    return cu, torch.searchsorted(cu, torch.arange(T, device=dev), right=True) - 1


def _conv(s):
    """y_t = silu(bias + sum_k w_k x_{t - K + 1 + k}); inputs before a sequence come from its state."""
    x, w = s["x"].float(), s["weight"].float()
    T, C = x.shape
    K = w.shape[1]
    cu, sid = _bounds(s, T)
    B = cu.numel() - 1
    init = s["init"].float() if s["init"] is not None else torch.zeros(B, K - 1, C, device=x.device)
    # every sequence behind its K - 1 carried inputs, one after the other
    at = torch.arange(T, device=x.device) + (sid + 1) * (K - 1)
    ext = torch.empty(T + B * (K - 1), C, device=x.device)
    ext[at] = x
    head = (cu[:-1] + torch.arange(B, device=x.device) * (K - 1))[:, None] + torch.arange(K - 1, device=x.device)
    ext[head.reshape(-1)] = init.reshape(-1, C)
    y = sum(ext[at - (K - 1 - k)] * w[:, k] for k in range(K))
    if s["bias"] is not None:
        y = y + s["bias"].float()
    tail = (cu[1:] + torch.arange(1, B + 1, device=x.device) * (K - 1))[:, None] - (K - 1) + \
        torch.arange(K - 1, device=x.device)
    return {"y": _silu(y).to(torch.bfloat16), "state": ext[tail].to(torch.bfloat16)}


def _conv_step(s):
    seen = torch.cat([s["state"].float(), s["x"].float()[:, None]], 1)  # [B, K, C]
    y = (seen * s["weight"].float().t()).sum(1)
    if s["bias"] is not None:
        y = y + s["bias"].float()
    s["state"].copy_(seen[:, 1:])
    return {"y": _silu(y).to(torch.bfloat16), "state": s["state"]}


def _scan(s):
    """S_t = exp(dt_t A) S_{t-1} + dt_t x_t B_t^T, y_t = (S_t C_t + D x_t) silu(z_t), in chunks of tokens:
    products of a chunk's tokens with one another, the chunks' sums, and those carried on."""
    T, Hv, dv = s["x"].shape
    Hk, dk = s["Bm"].shape[1:]
    R, dev, Q = Hv // Hk, s["x"].device, CHUNK
    cu, sid = _bounds(s, T)
    B = cu.numel() - 1
    state = s["init"].clone() if s["init"] is not None else torch.zeros(B, Hv, dv, dk, device=dev)
    if T == 0:
        return {"y": s["out"], "state": state}
    nc = -(-T // Q)

    def chunks(t):
        return F.pad(t.float(), (0, 0) * (t.dim() - 1) + (0, nc * Q - T)).unflatten(0, (nc, Q))

    x = chunks(s["x"]).unflatten(2, (Hk, R))                       # c i g r p
    Bm, Cm = chunks(s["Bm"]), chunks(s["Cm"])                      # c i g n
    dt = chunks(_softplus(s["dt"].float() + s["dt_bias"]))         # c i h
    sid = F.pad(sid, (0, nc * Q - T), value=B).unflatten(0, (nc, Q))
    first, last = sid[:, 0], sid[:, -1]                            # the sequences at a chunk's ends
    a = dt * s["A"]
    L = torch.cumsum(a, 1)
    xd = x * dt.unflatten(2, (Hk, R))[..., None]
    # a chunk's tokens with one another
    seen = (sid[:, :, None] == sid[:, None, :]) & torch.ones(Q, Q, dtype=torch.bool, device=dev).tril()
    decay = torch.exp(torch.where(seen[:, None], L.transpose(1, 2)[..., None] - L.transpose(1, 2)[:, :, None],
                                  -math.inf))                      # c h i j
    scores = torch.einsum("cign,cjgn->cgij", Cm, Bm)
    y = torch.einsum("cgrij,cjgrp->cigrp", decay.unflatten(1, (Hk, R)) * scores[:, :, None], xd)
    del decay, scores
    # what each chunk adds to the state of the sequence at its end
    to_end = torch.exp(L[:, -1:] - L) * (sid == last[:, None])[..., None]
    E = torch.einsum("cjgrp,cjgn->cgrpn", xd * to_end.unflatten(2, (Hk, R))[..., None], Bm).flatten(1, 2)
    live = cu[1:] > cu[:-1]
    c0 = torch.clamp(cu[:-1] // Q, max=nc - 1)                     # where a sequence starts
    i0 = cu[:-1] % Q
    before = L[c0, i0] - a[c0, i0]                                 # b h
    reach = live & (last[c0] == torch.arange(B, device=dev))
    w0 = torch.where(reach[:, None], torch.exp(torch.clamp(L[c0, -1] - before, max=0.0)), 0.0)
    E.index_add_(0, c0, w0[..., None, None] * state)
    if s["init"] is not None:                                      # the first chunk's tokens read the carried state
        mine = (sid[c0] == torch.arange(B, device=dev)[:, None]) & live[:, None]
        wi = torch.where(mine[..., None], torch.exp(torch.clamp(L[c0] - before[:, None], max=0.0)), 0.0)
        yi = torch.einsum("bign,bgrpn->bigrp", Cm[c0], state.unflatten(1, (Hk, R)))
        y.index_add_(0, c0, yi * wi.unflatten(2, (Hk, R))[..., None])
    # the chunks' sums carried on: decays over whole chunks between them
    ids = torch.arange(nc, device=dev)
    span = torch.cumsum(torch.where((ids[:, None] > ids)[..., None], L[:, -1][:, None], 0.0), 0)  # k, c', h
    span = torch.cat([torch.zeros_like(span[:1]), span[:-1]], 0)
    carried = (ids[:, None] > ids) & (first[:, None] == last)
    span = torch.exp(torch.where(carried[..., None], span, -math.inf)).permute(2, 0, 1)
    S = torch.matmul(span, E.flatten(2).transpose(0, 1)).transpose(0, 1).unflatten(2, (dv, dk))   # c h p n
    wi = torch.exp(L) * (sid == first[:, None])[..., None]
    yi = torch.einsum("cign,cgrpn->cigrp", Cm, S.unflatten(1, (Hk, R)))
    y = y + yi * wi.unflatten(2, (Hk, R))[..., None]
    # the state after each sequence's last token
    end = torch.clamp(cu[1:] - 1, min=0)
    ce, ie = end // Q, end % Q
    Le = L[ce, ie]
    upto = (sid[ce] == torch.arange(B, device=dev)[:, None]) & (torch.arange(Q, device=dev) <= ie[:, None])
    wj = torch.where(upto[..., None], torch.exp(torch.clamp(Le[:, None] - L[ce], max=0.0)), 0.0)
    fin = torch.einsum("bjgrp,bjgn->bgrpn", xd[ce] * wj.unflatten(2, (Hk, R))[..., None], Bm[ce]).flatten(1, 2)
    fin = fin + torch.where((first[ce] == torch.arange(B, device=dev))[:, None], torch.exp(Le), 0.0)[..., None, None] * S[ce]
    fin = fin + torch.where((c0 == ce)[:, None], torch.exp(torch.clamp(Le - before, max=0.0)), 0.0)[..., None, None] * state
    state = torch.where(live[:, None, None, None], fin, state)
    y = y + s["D"].unflatten(0, (Hk, R))[..., None] * x
    y = y.flatten(0, 1)[:T].flatten(1, 2)
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    return {"y": y.to(torch.bfloat16), "state": state}


def _scan_step(s):
    Hv, dv = s["x"].shape[1:]
    R = Hv // s["Bm"].shape[1]
    x = s["x"].float()
    dt = _softplus(s["dt"].float() + s["dt_bias"])
    Bm, Cm = (s[k].float().repeat_interleave(R, 1) for k in ("Bm", "Cm"))
    S = torch.exp(dt * s["A"])[..., None, None] * s["state"] + (dt[..., None] * x)[..., None] * Bm[:, :, None]
    y = (S * Cm[:, :, None]).sum(-1) + s["D"][:, None] * x
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    s["state"].copy_(S)
    return {"y": y.to(torch.bfloat16), "state": s["state"]}


def _norm(s):
    r = s["x"].float()
    if s["residual"] is not None:
        r = r + s["residual"].float()
    y = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + s["eps"]) * s["weight"].float()
    if s["e4m3"]:
        rows, D = y.shape
        g = s["group"] or D
        parts = F.pad(y, (0, -D % g)).unflatten(1, (-1, g))
        scales = parts.abs().amax(-1).clamp_min(AMAX_FLOOR) / E4M3_MAX
        q = torch.clamp(parts / scales[..., None], -E4M3_MAX, E4M3_MAX).flatten(1)[:, :D]
        out = {"y": q.contiguous().to(torch.float8_e4m3fn), "scales": scales}
    else:
        out = {"y": y.to(torch.bfloat16)}
    if s["residual"] is not None:
        out["residual"] = r.to(torch.bfloat16)
    return out


# ---- the definitions in 64 bits -----------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    f64 = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and k not in ("out", "final", "cu")}
    op = case["op"]
    if op == "norm":
        return _norm64(case, s, f64)
    gate = (lambda v: v * torch.sigmoid(v))
    if op == "conv_step":
        window = torch.cat((f64["state"], f64["x"].unsqueeze(1)), dim=1)
        y = torch.einsum("bkc,ck->bc", window, f64["weight"])
        y = y + f64["bias"] if "bias" in f64 else y
        return {"y": gate(y), "state": window[:, 1:]}
    if op == "conv":
        K, lens = case["K"], _lengths(case)
        ys, states, t = [], [], 0
        for b, n in enumerate(lens):
            head = f64["init"][b] if "init" in f64 else torch.zeros(K - 1, case["C"], dtype=torch.float64,
                                                                   device=s["x"].device)
            seq = torch.cat((head, f64["x"][t : t + n]))
            y = torch.einsum("tck,ck->tc", seq.unfold(0, K, 1), f64["weight"]) if n else seq[:0]
            y = y + f64["bias"] if "bias" in f64 else y
            ys.append(gate(y).float())  # only compared in 32 bits: halves what is held
            states.append(seq[n:])
            t += n
        return {"y": torch.cat(ys), "state": torch.stack(states)}
    lens = _lengths(case) if op == "scan" else [1] * case["B"]
    most = max(lens)
    Hv, dv, Hk = case["Hv"], case["dv"], case["Hk"]
    h_of = torch.arange(Hv, device=s["x"].device) // (Hv // Hk)
    start = np.concatenate([[0], np.cumsum(lens)])
    dt = F.softplus(f64["dt"] + f64["dt_bias"], threshold=40.0)
    S = f64["state"] if op == "scan_step" else f64.get("init")
    if S is None:
        S = torch.zeros(case["B"], Hv, dv, case["dk"], dtype=torch.float64, device=s["x"].device)
    y = torch.zeros(f64["x"].shape, dtype=torch.float64, device=s["x"].device)
    # the longest sequences first, so that those still running are always the leading ones
    order = sorted(range(len(lens)), key=lambda b: -lens[b])
    S = S[order].clone()
    starts = torch.tensor([int(start[b]) for b in order], device=s["x"].device)
    running = [lens[b] for b in order]
    for t in range(most):
        n = sum(1 for m in running if m > t)
        at = starts[:n] + t
        step = dt[at]
        S[:n] *= torch.exp(step * f64["A"])[:, :, None, None]
        S[:n] += (step[:, :, None] * f64["x"][at])[..., None] * f64["Bm"][at][:, h_of][:, :, None, :]
        y[at] = torch.matmul(S[:n], f64["Cm"][at][:, h_of].unsqueeze(-1)).squeeze(-1)
    y = y + f64["D"][None, :, None] * f64["x"]
    if "z" in f64:
        y = y * f64["z"] * torch.sigmoid(f64["z"])
    back = torch.empty_like(S)
    back[order] = S
    return {"y": y, "state": back}


def _norm64(case, s, f64):
    r = f64["x"] + f64["residual"] if case["residual"] else f64["x"]
    y = f64["weight"] * r / torch.sqrt(r.square().mean(dim=1, keepdim=True) + s["eps"])
    out = {"y": y}
    if case["e4m3"]:
        g = case["group"] or case["D"]
        scales = torch.stack([part.abs().amax(dim=1) for part in y.split(g, dim=1)], dim=1) / E4M3_MAX
        out = {"y": y / scales.repeat_interleave(g, dim=1)[:, : case["D"]], "scales": scales}
    if case["residual"]:
        out["residual"] = r
    return out
