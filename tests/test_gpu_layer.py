"""The operators around the recurrence against their formulas in float64 (GPU).

Tolerances, from the roundings alone:
* bf16 results: half a unit of the last of 8 bits is 2^-9 of the value; sums in fp32 add far less, so
  |err| <= 2^-8 |y| + 2^-16 magnitude, where magnitude is the sum over the terms' absolute values.
* The scan's outputs may round the state and the token-to-token weights to bf16 as matrix operands
  (2^-9 of each term at most, both in one term never): |err| <= 2^-8 |y| + 2^-8 magnitude.
* fp32 states: a term passes through a softplus, an exponential of a sum and two products, each good
  to a few 2^-23: |err| <= 2^-18 magnitude.
* e4m3: scales to 2^-18; values to half a unit of 4 bits, 2^-4 of the value, or 2^-10 below the
  smallest normal number (2^-6), plus the scale's and the sum's share (2^-16 of the largest, 448).
"""

import numpy as np
import pytest

import layer_refs as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from hybrid_linear_attention_prefill_gb300 import build
    from hybrid_linear_attention_prefill_gb300 import gdn as g

    build.build()
    g.load()
    return g


def n64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def close(got, want, mag, rel, mag_rel):
    got = n64(got)
    err = np.abs(got - want)
    tol = rel * np.abs(want) + mag_rel * mag + 1e-30
    assert np.all(np.isfinite(got))
    assert np.all(err <= tol), f"worst error {np.max(err / tol):.3g} of its tolerance"


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rnd(g, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g).to(dtype).cuda()


def cu_of(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


# ---- causal convolution -----------------------------------------------------------------------

CONV = [  # B, T (dense) or lengths, C, K, bias, init, silu
    (1, 1, 8, 4, True, False, True), (1, 2, 64, 4, False, True, True), (3, 5, 72, 3, True, True, True),
    (1, 65, 1032, 4, True, False, True), (2, 33, 64, 2, False, True, False), (5, 1, 16, 4, True, True, True),
    (1, 130, 2056, 2, True, True, True),
    ([1], 0, 64, 4, True, True, True), ([0, 3, 0, 0, 40, 1, 2, 17, 0], 0, 264, 4, True, True, True),
    ([16, 16, 1, 31], 0, 64, 3, False, False, True), ([0, 0, 7], 0, 8, 2, True, True, False),
]


@pytest.mark.parametrize("B,T,C,K,bias,init,act", CONV)
def test_conv(gdn, B, T, C, K, bias, init, act):
    g = gen(1)
    cu = None
    if isinstance(B, list):
        cu, B, T = cu_of(B), len(B), sum(B)
    n = T if cu is not None else B * T
    wide = rnd(g, n, C + 24)
    x = wide[:, 16:16 + C]  # a slice of wider rows
    w, bv = rnd(g, C, K), rnd(g, C) if bias else None
    st = rnd(g, B, K - 1, C) if init else None
    out, fin = gdn.causal_conv(x, w, bv, cu, st, B=B, silu=act)
    y, mag, f = R.conv(n64(x), n64(w), n64(bv), R.bounds(B, T, None if cu is None else cu.cpu()), n64(st), act)
    close(out, y, mag, 2.0 ** -8, 2.0 ** -16)
    assert np.array_equal(n64(fin), f)  # copies


def test_conv_no_tokens(gdn):
    st = rnd(gen(2), 2, 3, 64)
    out, fin = gdn.causal_conv(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), rnd(gen(3), 64, 4), None,
                               cu_of([0, 0]), st)
    assert out.shape == (0, 64) and torch.equal(fin, st)


@pytest.mark.parametrize("K", [2, 3, 4])
def test_conv_steps_continue_a_prompt(gdn, K):
    g = gen(4)
    x, w, b = rnd(g, 2 * 9, 72), rnd(g, 72, K), rnd(g, 72)
    whole, fin = gdn.causal_conv(x, w, b, B=2)
    x3 = x.view(2, 9, 72)
    out, st = gdn.causal_conv(x3[:, :4].reshape(8, 72), w, b, B=2)
    assert torch.equal(out.view(2, 4, 72), whole.view(2, 9, 72)[:, :4])
    for t in range(4, 9):
        y = gdn.causal_conv_step(x3[:, t], w, st, b)  # rows 9 * 72 apart
        assert torch.equal(y, whole.view(2, 9, 72)[:, t])
    assert torch.equal(st, fin)


def test_conv_sequences_do_not_meet(gdn):
    g = gen(5)
    lens = [5, 20, 3]
    x, w = rnd(g, 28, 64), rnd(g, 64, 4)
    ref, rfin = gdn.causal_conv(x, w, None, cu_of(lens))
    x[5:25] = float("nan")
    out, fin = gdn.causal_conv(x, w, None, cu_of(lens))
    for sl in (slice(0, 5), slice(25, 28)):
        assert torch.equal(out[sl], ref[sl])
    assert torch.equal(fin[0], rfin[0]) and torch.equal(fin[2], rfin[2]) and bool(fin[1].isnan().all())


@pytest.mark.parametrize("bad", [[0, 9, 4, 16], [3, 5, 8, 12], [0, 5, 400, 16], [-7, 5, 8, 16]])
def test_conv_malformed_boundaries_stay_in_bounds(gdn, bad):
    # 16 tokens in the middle of a larger buffer of sentinels: nothing outside may change
    g = gen(6)
    x, w, st = rnd(g, 16, 64), rnd(g, 64, 4), rnd(g, 3, 3, 64)
    buf = torch.full((64, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    fbuf = torch.full((9, 3, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    gdn.causal_conv(x, w, None, torch.tensor(bad, dtype=torch.int32, device="cuda"), st, out=buf[24:40],
                    final_state=fbuf[3:6])
    assert bool((buf[:24] == 7).all()) and bool((buf[40:] == 7).all())
    assert bool((fbuf[:3] == 7).all()) and bool((fbuf[6:] == 7).all())


def test_conv_offsets_past_32_bits(gdn):
    # rows 2^30 elements apart: the last one starts past 2^31 elements
    g = gen(7)
    big = torch.empty(3 * 2 ** 30 + 64, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((4, 64), (2 ** 30, 1))
    x.copy_(rnd(g, 4, 64))
    w = rnd(g, 64, 4)
    a, fa = gdn.causal_conv(x, w)
    b, fb = gdn.causal_conv(x.contiguous(), w)
    assert torch.equal(a, b) and torch.equal(fa, fb)


# ---- selective scan -----------------------------------------------------------------------------

def scan_inputs(g, n, B, Hk, Hv, dk, dv, *, init=False, gate=True, skip=True, dt32=False, bias=True, slow=False,
                strong=False):
    """x, B and C as slices of one wider tensor, steps of 0.001 to 0.3, as a layer has them."""
    pad = 8
    xbc = rnd(g, n, Hv * dv + 2 * Hk * dk + pad)
    xs = xbc[:, :Hv * dv].unflatten(1, (Hv, dv))
    bm = xbc[:, Hv * dv:Hv * dv + Hk * dk].unflatten(1, (Hk, dk))
    cm = xbc[:, Hv * dv + Hk * dk:Hv * dv + 2 * Hk * dk].unflatten(1, (Hk, dk))
    f32 = torch.float32
    step = torch.exp(torch.rand(Hv, generator=g) * np.log(300.0) + np.log(1e-3)).cuda()
    A = -(0.05 if slow else 200.0 if strong else 4.0) * (0.2 + torch.rand(Hv, generator=g)).cuda()
    return dict(x=xs, dt=(0.5 * rnd(g, n, Hv, dtype=f32)).to(f32 if dt32 else torch.bfloat16), A=A, Bm=bm, Cm=cm,
                D=rnd(g, Hv, dtype=f32) if skip else None, z=rnd(g, n, Hv, dv) if gate else None,
                dt_bias=(step + torch.log(-torch.expm1(-step))) if bias else None,
                init_state=rnd(g, B, Hv, dv, dk, dtype=f32) if init else None)


def scan_check(gdn, s, B, T, cu=None, **kw):
    out, fin = gdn.ssm_scan(**s, cu_seqlens=cu, B=B, **kw)
    seqs = R.bounds(B, T, None if cu is None else cu.cpu())
    y, mag, f, fmag = R.scan(*(n64(s[k]) for k in ("x", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias")), seqs,
                             n64(s["init_state"]), kw.get("softplus", True))
    close(out, y, mag, 2.0 ** -8, 2.0 ** -8)
    close(fin, f, fmag, 0.0, 2.0 ** -18)
    return out, fin


@pytest.mark.parametrize("T", [1, 2, 15, 63, 64, 65, 127, 128, 129, 200, 255, 256, 257, 513])
def test_scan_lengths(gdn, T):
    scan_check(gdn, scan_inputs(gen(10 + T), T, 1, 1, 2, 128, 64, init=T % 2 == 1), 1, T)


@pytest.mark.parametrize("dk", [32, 64, 128])
@pytest.mark.parametrize("dv", [32, 64, 128])
@pytest.mark.parametrize("Hk,Hv", [(1, 1), (2, 2), (1, 3), (2, 8)])
def test_scan_heads(gdn, dk, dv, Hk, Hv):
    scan_check(gdn, scan_inputs(gen(dk + dv + Hv), 2 * 150, 2, Hk, Hv, dk, dv, init=True), 2, 150)


@pytest.mark.parametrize("opts", [dict(gate=False), dict(skip=False), dict(dt32=True), dict(bias=False),
                                  dict(slow=True, init=True), dict(strong=True, init=True),
                                  dict(gate=False, skip=False, bias=False, dt32=True)])
def test_scan_options(gdn, opts):
    scan_check(gdn, scan_inputs(gen(20), 200, 1, 1, 2, 64, 128, **opts), 1, 200)


def test_scan_without_softplus(gdn):
    s = scan_inputs(gen(21), 140, 1, 1, 2, 64, 64, bias=False, dt32=True)
    s["dt"] = s["dt"].abs() * 0.1
    s["dt"][::7] = 0.0  # tokens of step 0 leave the state as it is
    scan_check(gdn, s, 1, 140, softplus=False)


@pytest.mark.parametrize("lens", [[1], [0, 5, 0], [128, 128], [130, 0, 1, 127, 300, 64], [1] * 40, [700, 3]])
@pytest.mark.parametrize("init", [False, True])
def test_scan_packed(gdn, lens, init):
    n = sum(lens)
    s = scan_inputs(gen(22), n, len(lens), 2, 4, 64, 64, init=init)
    scan_check(gdn, s, len(lens), n, cu_of(lens))


@pytest.mark.parametrize("B,T,Hk,Hv,dk,dv", [(1, 4000, 1, 2, 128, 128), (1, 2500, 1, 1, 32, 32),
                                             (2, 1700, 1, 3, 64, 64)])
@pytest.mark.parametrize("init", [False, True])
def test_scan_long_prompts_with_few_heads(gdn, B, T, Hk, Hv, dk, dv, init):
    s = scan_inputs(gen(23), B * T, B, Hk, Hv, dk, dv, init=init, slow=True)
    scan_check(gdn, s, B, T)


def test_scan_long_packed_with_few_heads(gdn):
    lens = [1500, 0, 900, 1, 2600]
    s = scan_inputs(gen(24), sum(lens), 5, 1, 1, 128, 64, init=True, slow=True)
    scan_check(gdn, s, 5, sum(lens), cu_of(lens))


def test_scan_no_tokens_returns_the_initial_state(gdn):
    s = scan_inputs(gen(25), 0, 2, 1, 2, 64, 64, init=True)
    out, fin = gdn.ssm_scan(**s, cu_seqlens=cu_of([0, 0]))
    assert out.shape[0] == 0 and torch.equal(fin, s["init_state"])
    s["init_state"] = None
    assert not bool(gdn.ssm_scan(**s, cu_seqlens=cu_of([0, 0]))[1].any())


def test_scan_state_in_place_and_split(gdn):
    T, cut = 333, 150
    s = scan_inputs(gen(26), T, 1, 1, 2, 128, 128, init=True)
    whole, fin = gdn.ssm_scan(**s)
    st = s["init_state"].clone()
    part = lambda lo, hi: {k: (v[lo:hi] if k in ("x", "dt", "Bm", "Cm", "z") else v) for k, v in s.items()}  # noqa: E731
    a, _ = gdn.ssm_scan(**{**part(0, cut), "init_state": st}, final_state=st)
    b, _ = gdn.ssm_scan(**{**part(cut, T), "init_state": st}, final_state=st)
    # the pieces cut the chunks elsewhere: equal up to the outputs' operand roundings
    y, mag, f, fmag = R.scan(*(n64(s[k]) for k in ("x", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias")), [(0, T)],
                             n64(s["init_state"]))
    close(torch.cat([a, b]), y, mag, 2.0 ** -8, 2.0 ** -8)
    close(st, f, fmag, 0.0, 2.0 ** -18)


def test_scan_in_place_state_of_a_long_prompt(gdn):
    T = 3000
    s = scan_inputs(gen(27), T, 1, 1, 1, 64, 64, init=True, slow=True)
    ref, fin = gdn.ssm_scan(**s)
    st = s["init_state"].clone()
    out, _ = gdn.ssm_scan(**{**s, "init_state": st}, final_state=st)
    assert torch.equal(out, ref) and torch.equal(st, fin)


@pytest.mark.parametrize("dk,dv,Hk,Hv", [(32, 32, 1, 1), (64, 128, 1, 3), (128, 64, 2, 4), (128, 128, 2, 2)])
def test_scan_steps_continue_a_prompt(gdn, dk, dv, Hk, Hv):
    B, T = 3, 9
    s = scan_inputs(gen(28), B * T, B, Hk, Hv, dk, dv, init=True)
    y, mag, f, fmag = R.scan(*(n64(s[k]) for k in ("x", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias")),
                             R.bounds(B, T, None), n64(s["init_state"]))
    st = s["init_state"].clone()
    for t in range(T):  # token t of every sequence: rows T apart
        row = {k: (v[t::T] if k in ("x", "dt", "Bm", "Cm", "z") else v) for k, v in s.items() if k != "init_state"}
        out = gdn.ssm_step(**row, state=st)
        close(out, y[t::T], mag[t::T], 2.0 ** -8, 2.0 ** -16)  # no rounding but the last
    close(st, f, fmag, 0.0, 2.0 ** -18)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_scan_sequences_do_not_meet(gdn, bad):
    lens = [70, 130, 200, 5]
    s = scan_inputs(gen(29), sum(lens), 4, 1, 2, 64, 64, init=True)
    ref, rfin = gdn.ssm_scan(**s, cu_seqlens=cu_of(lens))
    for k in ("x", "Bm", "Cm", "z", "dt"):
        s[k][70:200] = bad
    out, fin = gdn.ssm_scan(**s, cu_seqlens=cu_of(lens))
    for sl in (slice(0, 70), slice(200, 405)):
        assert torch.equal(out[sl], ref[sl])
    for b in (0, 2, 3):
        assert torch.equal(fin[b], rfin[b])


def test_scan_reads_nothing_beside_its_slices(gdn):
    # NaN in the columns beside the slices of the wider rows and in other heads' groups of columns
    s = scan_inputs(gen(30), 150, 1, 1, 1, 32, 32)
    ref = gdn.ssm_scan(**s)
    t = dict(s)
    for k, w in (("x", 32), ("Bm", 32), ("Cm", 32), ("z", 32)):
        wide = torch.full((150, 96), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[:, 32:64] = s[k].reshape(150, w)
        t[k] = wide[:, 32:64].unflatten(1, (1, w))
    got = gdn.ssm_scan(**t)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_silu_far_below_zero(gdn):
    # silu goes to zero there; a neighbour's value and a NaN keep their own results
    far = torch.tensor([-50.0, -100.0, -1e10, -3e38, float("-inf")], device="cuda").bfloat16()
    s = scan_inputs(gen(38), 10, 1, 1, 1, 32, 32)
    ref = gdn.ssm_scan(**s)[0]
    row = {k: (v[:2] if k in ("x", "dt", "Bm", "Cm", "z") else v) for k, v in s.items() if k != "init_state"}
    st = torch.zeros(2, 1, 32, 32, device="cuda")
    ref1 = gdn.ssm_step(**row, state=st.clone())
    for i, v in enumerate(far):
        z = s["z"].clone()
        z[0::2, 0, 2 * i + 1] = v
        z[0, 0, 20] = float("nan")
        for out, want in ((gdn.ssm_scan(**{**s, "z": z})[0], ref), (gdn.ssm_step(**{**row, "z": z[:2]},
                                                                                 state=st.clone()), ref1)):
            assert bool((out[0::2, 0, 2 * i + 1].abs() < 1e-15).all()) and bool(out[0, 0, 20].isnan())
            same = torch.ones_like(out, dtype=torch.bool)
            same[0::2, 0, 2 * i + 1] = False
            same[0, 0, 20] = False
            assert torch.equal(out[same], want[same])
    x, w = torch.zeros(4, 16, dtype=torch.bfloat16, device="cuda"), torch.zeros(16, 2, device="cuda").bfloat16()
    x[1, :4], w[:, 1] = far[:4], 1.0
    x[2, 5] = float("nan")
    out, _ = gdn.causal_conv(x, w)
    assert bool((out[1].abs() < 1e-15).all()) and bool(out[2, 5].isnan())


def test_scan_infinite_step_and_zero_rows(gdn):
    # a head whose inputs are all zero returns zeros whatever its decay
    s = scan_inputs(gen(31), 100, 1, 1, 2, 64, 64, gate=False)
    s["x"][:, 1] = 0
    out, fin = gdn.ssm_scan(**s)
    assert not bool(out[:, 1].any()) and not bool(fin[0, 1].any())


def test_scan_is_deterministic_and_runs_on_a_side_stream(gdn):
    s = scan_inputs(gen(32), 2000, 1, 1, 2, 128, 128, init=True)
    a = gdn.ssm_scan(**s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = gdn.ssm_scan(**s)
    side.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("T,Hv", [(200, 2), (3000, 1)])
def test_scan_with_a_caller_workspace_in_a_graph(gdn, T, Hv):
    s = scan_inputs(gen(33), T, 1, 1, Hv, 64, 64, init=True)
    ref = gdn.ssm_scan(**s)
    ws = torch.zeros(gdn.gdn_ssm_workspace_bytes(1, T, 1, Hv, 64, 64, False), dtype=torch.uint8, device="cuda")
    out, fin = torch.empty_like(ref[0]), torch.empty_like(ref[1])
    gdn.ssm_scan(**s, out=out, final_state=fin, workspace=ws)  # the kernels' one-time settings
    torch.cuda.synchronize()
    out.zero_(), fin.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.ssm_scan(**s, out=out, final_state=fin, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref[0]) and torch.equal(fin, ref[1])
    assert int(ws[:4].view(torch.int32)) == 0


@pytest.mark.parametrize("bad", [[0, 190, 100, 200], [3, 50, 90, 120], [0, 50, 4000, 200], [-70, 50, 80, 200]])
@pytest.mark.parametrize("Hv", [1, 4])
def test_scan_malformed_boundaries_stay_in_bounds(gdn, bad, Hv):
    s = scan_inputs(gen(34), 200, 3, 1, Hv, 64, 64, init=True)
    buf = torch.full((600, Hv, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    fbuf = torch.full((9, Hv, 64, 64), 7.0, device="cuda")
    gdn.gdn_device_status()
    gdn.ssm_scan(**s, cu_seqlens=torch.tensor(bad, dtype=torch.int32, device="cuda"), out=buf[200:400],
                 final_state=fbuf[3:6])
    rc, bits = gdn.gdn_device_status()
    assert rc == 0 and bits & gdn.GDN_STATUS_BAD_CU_SEQLENS
    assert bool((buf[:200] == 7).all()) and bool((buf[400:] == 7).all())
    assert bool((fbuf[:3] == 7).all()) and bool((fbuf[6:] == 7).all())


def test_scan_offsets_past_32_bits(gdn):
    s = scan_inputs(gen(35), 3, 1, 1, 1, 64, 64)
    ref = gdn.ssm_scan(**s)
    big = torch.empty(2 * (2 ** 30 + 8) + 64, dtype=torch.bfloat16, device="cuda")
    for k in ("x", "Bm", "Cm", "z"):
        v = big.as_strided((3, 1, 64), (2 ** 30 + 8, 64, 1))
        v.copy_(s[k])
        got = gdn.ssm_scan(**{**s, k: v})
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_scan_in_place_over_many_segments(gdn):
    # enough segments for several waves: the first ones' start must not be the final state of the last
    s = scan_inputs(gen(36), 40000, 1, 1, 4, 64, 128, init=True)
    out, fin = gdn.ssm_scan(**s)
    packed = cu_of([30000, 0, 100, 9900])
    s4 = {**s, "init_state": s["init_state"].repeat(4, 1, 1, 1)}
    out4, fin4 = gdn.ssm_scan(**s4, cu_seqlens=packed)
    for _ in range(5):
        st, st4 = s["init_state"].clone(), s4["init_state"].clone()
        o, _ = gdn.ssm_scan(**{**s, "init_state": st}, final_state=st)
        assert torch.equal(o, out) and torch.equal(st, fin)
        o, _ = gdn.ssm_scan(**{**s4, "init_state": st4}, cu_seqlens=packed, final_state=st4)
        assert torch.equal(o, out4) and torch.equal(st4, fin4)


def test_scan_without_memory_for_its_workspace(gdn):
    s = scan_inputs(gen(37), 2000, 1, 1, 2, 32, 64)
    ref = gdn.ssm_scan(**s)
    gdn.gdn_release_workspace()
    assert gdn.gdn_debug_fail_allocations(1) == 0
    try:
        with pytest.raises(gdn.GdnError) as e:
            gdn.ssm_scan(**s)
        assert e.value.status == gdn.GDN_ERR_ALLOC
    finally:
        gdn.gdn_debug_fail_allocations(0)
    again = gdn.ssm_scan(**s)
    assert torch.equal(again[0], ref[0]) and torch.equal(again[1], ref[1])


# ---- norm -----------------------------------------------------------------------------------------

@pytest.mark.parametrize("rows,D", [(1, 8), (1, 4096), (3, 64), (5, 264), (33, 520), (2, 1000), (7, 2056), (3, 8192),
                                    (2, 16392), (2, 32768), (129, 32)])
@pytest.mark.parametrize("res", [False, True])
def test_norm(gdn, rows, D, res):
    g = gen(D + rows)
    x, w = rnd(g, rows, D + 8)[:, 8:] if rows > 1 else rnd(g, rows, D), rnd(g, D)
    r0 = rnd(g, rows, D) if res else None
    r, y = R.norm(n64(x), n64(r0), n64(w), 1e-6)
    out, sc, ro = gdn.add_norm(x, w, r0)
    assert sc is None and (ro is None) == (not res)
    close(out, y, np.abs(y), 2.0 ** -8, 2.0 ** -16)
    if res:
        close(ro, r, np.abs(n64(x)) + np.abs(n64(r0)), 2.0 ** -8, 2.0 ** -16)
    for group in (0, 32, 64, 128):
        q, sc, _ = gdn.add_norm(x, w, r0, group=group, e4m3=True)
        want = R.scales(y, group)
        assert sc.shape == want.shape
        close(sc, want, want, 0.0, 2.0 ** -18)
        v = y / np.repeat(want, group or D, 1)[:, :D]
        close(q, v, 448.0, 2.0 ** -4, 2.0 ** -10 / 448 + 2.0 ** -16)


def test_norm_in_place_residual(gdn):
    g = gen(40)
    x, w, r0 = rnd(g, 9, 512), rnd(g, 512), rnd(g, 9, 512)
    out, _, ro = gdn.add_norm(x, w, r0)
    keep = r0.clone()
    out2, _, ro2 = gdn.add_norm(x, w, keep, residual_out=keep)
    assert ro2 is keep and torch.equal(out, out2) and torch.equal(ro, keep)


def test_norm_zero_rows_and_tiny_values(gdn):
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    x = torch.zeros(3, 256, dtype=torch.bfloat16, device="cuda")
    x[1, 7] = 2.0 ** -60
    q, sc, _ = gdn.add_norm(x, w, eps=1e-6, group=128, e4m3=True)
    assert not bool(q[0].float().any()) and bool((sc[0] == 2.0 ** -96 / 448).all())
    assert float(q[1, 7].float()) == 448.0 and not bool(q[2].float().any())
    assert bool(torch.isfinite(sc).all())


def test_norm_keeps_nan_and_infinity_in_their_rows(gdn):
    g = gen(41)
    x, w = rnd(g, 5, 512), rnd(g, 512)
    ref = gdn.add_norm(x, w, group=128, e4m3=True)
    refb = gdn.add_norm(x, w)[0]
    x[1, 200], x[3, 0] = float("nan"), float("inf")
    q, sc, _ = gdn.add_norm(x, w, group=128, e4m3=True)
    out = gdn.add_norm(x, w)[0]
    for row in (0, 2, 4):
        assert torch.equal(q[row].view(torch.uint8), ref[0][row].view(torch.uint8)) and torch.equal(sc[row], ref[1][row])
        assert torch.equal(out[row], refb[row])
    assert bool(out[1].isnan().all()) and bool(sc[1].isnan().all())
    # an infinite sum leaves 0 for the finite values and NaN in the infinite one's place
    assert bool(out[3, 0].isnan()) and not bool(out[3, 1:].any())
    assert bool(sc[3, 0].isnan()) and bool(torch.isfinite(sc[3, 1:]).all())


def test_norm_offsets_past_32_bits(gdn):
    g = gen(42)
    x, w = rnd(g, 3, 512), rnd(g, 512)
    big = torch.empty(2 * (2 ** 30 + 8) + 512, dtype=torch.bfloat16, device="cuda")
    v = big.as_strided((3, 512), (2 ** 30 + 8, 1))
    v.copy_(x)
    assert torch.equal(gdn.add_norm(v, w)[0], gdn.add_norm(x, w)[0])


# ---- both ways to a call --------------------------------------------------------------------------

def test_calls_with_outputs_given_are_the_same_calls(gdn, monkeypatch):
    """With every output given a call may take a shorter way through the binding: the same results and refusals."""
    g = gen(50)
    x, w, b, st = rnd(g, 40, 72), rnd(g, 72, 4), rnd(g, 72), rnd(g, 2, 3, 72)
    s = scan_inputs(gen(51), 40, 2, 1, 2, 32, 64, init=True)
    one = {k: (v[:2] if k in ("x", "dt", "Bm", "Cm", "z") else v) for k, v in s.items() if k != "init_state"}
    r, nw = rnd(g, 40, 72), rnd(g, 72)

    def calls():
        o, f = torch.empty_like(x), torch.empty_like(st)
        yield gdn.causal_conv(x, w, b, cu_of([15, 25]), st, out=o, final_state=f)
        o, st1 = torch.empty_like(x[:2]), st.clone()
        yield gdn.causal_conv_step(x[:2], w, st1, b, out=o), st1
        o, f = torch.empty_like(s["x"]), torch.empty_like(s["init_state"])
        yield gdn.ssm_scan(**s, B=2, out=o, final_state=f)
        o, f = torch.empty_like(one["x"]), s["init_state"].clone()
        yield gdn.ssm_step(**one, state=f, out=o), f
        o, rr = torch.empty_like(x), r.clone()
        yield gdn.add_norm(x, nw, rr, out=o, residual_out=rr)[0], rr
        q, sc = torch.empty(40, 72, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(40, 3, device="cuda")
        q, sc, _ = gdn.add_norm(x, nw, group=32, e4m3=True, out=q, scales=sc)
        yield q.view(torch.uint8), sc

    def refusals():
        o = torch.empty_like(x)
        yield lambda: gdn.causal_conv(x, w.float(), b, want_final=False, out=o)
        yield lambda: gdn.causal_conv(x, w[:, :1], b, want_final=False, out=o)
        yield lambda: gdn.causal_conv_step(x[:2], w, st, b, out=o)
        yield lambda: gdn.ssm_scan(**s, B=2, want_final=False, out=torch.empty_like(s["x"])[:39])
        yield lambda: gdn.ssm_step(**one, state=s["init_state"].double(), out=torch.empty_like(one["x"]))
        yield lambda: gdn.add_norm(x, nw[:64], out=o)

    short = [(a.clone(), c.clone()) for a, c in calls()]
    for f in refusals():
        with pytest.raises((ValueError, gdn.GdnError)):
            f()
    monkeypatch.setattr(gdn, "_fast", None)
    for (a, c), (a2, c2) in zip(short, calls()):
        assert torch.equal(a, a2) and torch.equal(c, c2)
    for f in refusals():
        with pytest.raises((ValueError, gdn.GdnError)):
            f()
