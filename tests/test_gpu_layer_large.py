"""The operators around the recurrence at sizes where the launch rules take their long forms (GPU): segments of many
chunks, whole sequences of many chunks, runs of 16 to 128 tokens, 8 and 16 state rows a warp, two vectors a thread.

References are float64 torch operations on the GPU, token by token where there is a recurrence; tolerances as in
test_gpu_layer.py, from the roundings alone.
"""

import pytest

from test_gpu_layer import cu_of, gdn, gen, rnd, scan_inputs  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def within(got, want, mag, rel, mag_rel):
    got = got.double()
    err = (got - want).abs_().sub_(rel * want.abs()).sub_(mag_rel * mag)
    assert bool(torch.isfinite(got).all())
    assert float(err.max()) <= 1e-30, f"{float(err.max()):.3g} beyond its tolerance"


def scan64(s, lens):
    """(y, magnitude, final state, its magnitude) of ssm_scan's operands, every sequence's token t at once."""
    f = {k: None if v is None else v.double() for k, v in s.items()}
    T, Hv, dv = f["x"].shape
    hk = torch.arange(Hv, device="cuda") // (Hv // f["Bm"].shape[1])
    step = torch.nn.functional.softplus(f["dt"] + (f["dt_bias"] if f["dt_bias"] is not None else 0.0), threshold=40.0)
    order = sorted(range(len(lens)), key=lambda b: -lens[b])  # the longest first: those still running lead
    start = torch.tensor([sum(lens[:b]) for b in order], device="cuda")
    S = f["init_state"][order] if f["init_state"] is not None else torch.zeros(
        len(lens), Hv, dv, f["Bm"].shape[2], dtype=torch.float64, device="cuda")
    M = S.abs()
    y, mag = torch.zeros_like(f["x"]), torch.zeros_like(f["x"])
    for t in range(max(lens)):
        n = sum(1 for b in order if lens[b] > t)
        at = start[:n] + t
        decay = torch.exp(step[at] * f["A"])[..., None, None]
        put = (step[at][..., None] * f["x"][at])[..., None] * f["Bm"][at][:, hk][:, :, None]
        S[:n] = S[:n] * decay + put
        M[:n] = M[:n] * decay + put.abs_()
        c = f["Cm"][at][:, hk][..., None]
        y[at] = (S[:n] @ c)[..., 0]
        mag[at] = (M[:n] @ c.abs())[..., 0]
    if f["D"] is not None:
        skip = f["D"][:, None] * f["x"]
        y, mag = y + skip, mag + skip.abs_()
    if f["z"] is not None:
        g = torch.nn.functional.silu(f["z"])
        y, mag = y * g, mag * g.abs_()
    back = torch.empty_like(S), torch.empty_like(M)
    back[0][order], back[1][order] = S, M
    return y, mag, *back


def scan_within(gdn, s, lens, packed):
    out, fin = gdn.ssm_scan(**s, cu_seqlens=cu_of(lens) if packed else None, B=len(lens))
    y, mag, f, fmag = scan64(s, lens)
    within(out, y, mag, 2.0 ** -8, 2.0 ** -8)
    within(fin, f, fmag, 0.0, 2.0 ** -18)


def segments(gdn, B, T, Hk, Hv, dk, dv, packed):
    """Segments of the whole batch, from the workspace they take (0: none is cut)."""
    heads = Hv // (2 if dv < 128 and (Hv // Hk) % 2 == 0 else 1)
    extra = gdn.gdn_ssm_workspace_bytes(B, T, Hk, Hv, dk, dv, packed) - gdn.gdn_ssm_workspace_bytes(
        B, 1, Hk, Hv, dk, dv, packed) - B * Hv * dv * dk * 4
    return max(0, extra) // (heads * dk * 512)


@pytest.mark.parametrize("T,dk,dv,Hk,Hv,init", [(20000, 128, 128, 2, 4, True), (20000, 64, 64, 4, 8, False),
                                                (20000, 32, 128, 4, 4, True), (30000, 128, 32, 2, 2, False),
                                                (4100, 128, 128, 16, 32, True)])
def test_scan_segments_of_many_chunks(gdn, T, dk, dv, Hk, Hv, init):
    n = segments(gdn, 1, T, Hk, Hv, dk, dv, False)
    assert n > 1 and (T + 127) // 128 > 3 * n  # four chunks a segment and more
    scan_within(gdn, scan_inputs(gen(60), T, 1, Hk, Hv, dk, dv, init=init, slow=True), [T], False)


def test_scan_packed_segments_of_many_chunks(gdn):
    lens = [9000, 0, 100, 20001, 128, 3000]
    assert sum(lens) // 128 >= 4 * segments(gdn, 6, sum(lens), 2, 4, 64, 128, True) > 0
    scan_within(gdn, scan_inputs(gen(61), sum(lens), 6, 2, 4, 64, 128, init=True, slow=True), lens, True)


@pytest.mark.parametrize("dk,dv,Hk,Hv,B", [(128, 128, 4, 8, 24), (64, 64, 4, 16, 24), (128, 64, 8, 8, 24),
                                           (32, 32, 8, 16, 24)])
def test_scan_whole_sequences_of_many_chunks(gdn, dk, dv, Hk, Hv, B):
    T = 1300
    assert segments(gdn, B, T, Hk, Hv, dk, dv, False) == 0
    scan_within(gdn, scan_inputs(gen(62), B * T, B, Hk, Hv, dk, dv, init=True, slow=True), [T] * B, False)


def test_scan_packed_whole_sequences_of_many_chunks(gdn):
    lens = [1300 + 37 * b for b in range(23)] + [0, 1]
    assert segments(gdn, 25, sum(lens), 2, 8, 128, 128, True) == 0
    scan_within(gdn, scan_inputs(gen(63), sum(lens), 25, 2, 8, 128, 128, init=True, slow=True), lens, True)


@pytest.mark.parametrize("dv", [64, 128])
@pytest.mark.parametrize("dk", [32, 64, 128])
def test_scan_step_with_several_rows_in_flight(gdn, dk, dv):
    B, Hk, Hv = 128, 16, 32  # dv / 8 state rows a warp: the device is full without fewer
    s = scan_inputs(gen(64), B, B, Hk, Hv, dk, dv, init=True)
    y, mag, f, fmag = scan64(s, [1] * B)
    st = s.pop("init_state")
    out = gdn.ssm_step(**s, state=st)
    within(out, y, mag, 2.0 ** -8, 2.0 ** -16)
    within(st, f, fmag, 0.0, 2.0 ** -18)


# Runs of r tokens where 2 Ttot / r blocks of 512 channels are 21 times the SMs: 16, 32, 64 and 128 of them.
@pytest.mark.parametrize("Ttot,C,K", [(9001, 1032, 4), (9001, 1032, 2), (4097, 8192, 4), (7001, 8192, 3),
                                      (14001, 8192, 4)])
@pytest.mark.parametrize("init", [False, True])
def test_conv_runs_of_many_tokens(gdn, Ttot, C, K, init):
    g = gen(65)
    lens, left = [], Ttot
    while left:  # ends inside runs, at their ends, and several in one run
        lens.append(min(left, [1, 700, 128, 0, 64, 3, 2500, 16, 5][len(lens) % 9]))
        left -= lens[-1]
    x, w, b = rnd(g, Ttot, C + 8)[:, 8:], rnd(g, C, K), rnd(g, C)
    st = rnd(g, len(lens), K - 1, C) if init else None
    out, fin = gdn.causal_conv(x, w, b, cu_of(lens), st)
    at = 0
    for i, n in enumerate(lens):
        head = st[i] if init else torch.zeros(K - 1, C, dtype=x.dtype, device="cuda")
        seen = torch.cat([head, x[at:at + n]])
        assert torch.equal(fin[i], seen[n:])
        if n:
            terms = [seen[k:k + n].double() * w[:, k].double() for k in range(K)] + [b.double()]
            within(out[at:at + n], torch.nn.functional.silu(sum(terms)), sum(t.abs() for t in terms), 2.0 ** -8,
                   2.0 ** -16)
        at += n


@pytest.mark.parametrize("D", [512, 4096, 4104, 16392])
@pytest.mark.parametrize("group", [None, 0, 32, 128])
def test_norm_with_two_vectors_a_thread(gdn, D, group):
    g, rows = gen(66), 700
    x, r0, w = rnd(g, rows, D), rnd(g, rows, D), rnd(g, D)
    out, sc, ro = gdn.add_norm(x, w, r0, group=group or 0, e4m3=group is not None)
    r = x.double() + r0.double()
    y = w.double() * r / torch.sqrt(r.square().mean(1, keepdim=True) + 1e-6)
    within(ro, r, x.double().abs() + r0.double().abs(), 2.0 ** -8, 2.0 ** -16)
    if group is None:
        within(out, y, y.abs(), 2.0 ** -8, 2.0 ** -16)
        return
    want = torch.stack([p.abs().amax(1) for p in y.split(group or D, 1)], 1) / 448.0
    within(sc, want, want, 0.0, 2.0 ** -18)
    v = y / want.repeat_interleave(group or D, 1)[:, :D]
    within(out.float(), v, torch.full_like(v, 448.0), 2.0 ** -4, 2.0 ** -10 / 448 + 2.0 ** -16)
