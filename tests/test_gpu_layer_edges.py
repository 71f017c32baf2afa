"""Edges of the operators around the recurrence that their other tests leave out (GPU)."""

import pytest

from test_gpu_layer import cu_of, gdn, gen, rnd, scan_check, scan_inputs  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def rows_of(s, sl):
    return {k: (v[sl] if k in ("x", "dt", "Bm", "Cm", "z") else v) for k, v in s.items() if k != "init_state"}


# ---- outputs and streams ------------------------------------------------------------------------

def test_outputs_come_from_the_memory_of_the_stream_of_the_call(gdn):
    """Memory that a call on another stream returned must not go to the current stream's next tensor, whose work
    may run beside the call's (nor come from one that such work still uses)."""
    s = scan_inputs(gen(70), 128, 1, 1, 2, 64, 64)
    one = rows_of(s, slice(0, 64))
    x, w, st = rnd(gen(71), 128, 64), rnd(gen(72), 64, 4), rnd(gen(73), 64, 3, 64)
    state = torch.zeros(64, 2, 64, 64, device="cuda")
    q = rnd(gen(74), 128, 2, 64)
    g = torch.zeros(128, 2, device="cuda")
    for side in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        for call in (lambda: gdn.causal_conv(x, w, stream=side),
                     lambda: [gdn.causal_conv_step(x[:64], w, st, stream=side)],
                     lambda: gdn.ssm_scan(**s, stream=side), lambda: [gdn.ssm_step(**one, state=state, stream=side)],
                     lambda: gdn.add_norm(x, w[:, 0].contiguous(), x, e4m3=True, stream=side),
                     lambda: gdn.prefill(q, q, q, g, g, stream=side)):
            call()  # the library's own memory is there
            torch.cuda.synchronize()
            torch.cuda.empty_cache()
            got = [t for t in call() if t is not None]
            torch.cuda.synchronize()
            was = {t.data_ptr(): t.numel() * t.element_size() for t in got}
            del got
            fresh = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in was.values() for _ in range(4)]
            assert not was.keys() & {t.data_ptr() for t in fresh}


def test_a_first_calls_status_survives_what_another_stream_has_to_do(gdn):
    s = scan_inputs(gen(75), 200, 3, 1, 1, 64, 64, init=True)
    bad = torch.tensor([0, 190, 100, 200], dtype=torch.int32, device="cuda")
    out, fin = torch.empty_like(s["x"]), torch.empty_like(s["init_state"])
    side = torch.cuda.Stream()
    gdn.ssm_scan(**s, cu_seqlens=bad, out=out, final_state=fin, stream=side)
    gdn.gdn_device_status()
    gdn.gdn_release_workspace()
    torch.cuda._sleep(500_000_000)  # about a quarter of a second of the default stream
    gdn.ssm_scan(**s, cu_seqlens=bad, out=out, final_state=fin, stream=side)
    side.synchronize()
    rc, bits = gdn.gdn_device_status()
    assert rc == 0 and bits == gdn.GDN_STATUS_BAD_CU_SEQLENS


def prefill_inputs(n):
    q = torch.nn.functional.normalize(rnd(gen(92), n, 1, 32).float(), dim=-1).bfloat16()  # keys that leave the state finite
    return q, q, q, torch.zeros(n, 1, device="cuda"), torch.full((n, 1), 0.5, device="cuda")


@pytest.mark.parametrize("which", ["prefill", "scan"])
def test_status_outlives_a_larger_workspace(gdn, which):
    bad = torch.tensor([0, 190, 100, 200], dtype=torch.int32, device="cuda")

    def call(n, cu):
        if which == "prefill":
            return gdn.prefill(*prefill_inputs(n), cu)
        B = 1 if cu is None else 3
        return gdn.ssm_scan(**scan_inputs(gen(93), n, B, 1, 1, 128, 128), cu_seqlens=cu, B=B)

    gdn.gdn_release_workspace()
    call(200, bad)
    call(60000, None)  # takes more
    rc, bits = gdn.gdn_device_status()
    assert rc == 0 and bits == gdn.GDN_STATUS_BAD_CU_SEQLENS
    assert gdn.gdn_device_status() == (0, 0)


@pytest.mark.parametrize("which", ["prefill", "scan"])
def test_status_of_a_new_workspace_is_clear(gdn, which):
    gdn.gdn_release_workspace()
    torch.cuda.empty_cache()
    used = torch.full((2 ** 30,), 255, dtype=torch.uint8, device="cuda")  # what a new allocation may find
    small = [torch.full((2 ** 21,), 255, dtype=torch.uint8, device="cuda") for _ in range(16)]
    torch.cuda.synchronize()
    del used, small
    torch.cuda.empty_cache()
    if which == "prefill":
        gdn.prefill(*prefill_inputs(3000))
    else:
        gdn.ssm_scan(**scan_inputs(gen(94), 3000, 1, 1, 1, 128, 128))
    assert gdn.gdn_device_status() == (0, 0)


# ---- arguments ----------------------------------------------------------------------------------

def test_arguments_beyond_their_range_are_refused(gdn):
    """The same errors by both ways through the binding, and the object's own where it has no truth value."""
    class Neither:
        def __bool__(self):
            raise KeyError("neither")

    x, w, st = rnd(gen(76), 8, 64), rnd(gen(77), 64, 4), rnd(gen(78), 8, 3, 64)
    s = scan_inputs(gen(79), 8, 1, 1, 1, 64, 64)
    o, so = torch.empty_like(x), torch.empty_like(s["x"])
    q = torch.empty(8, 64, dtype=torch.float8_e4m3fn, device="cuda")
    state = torch.zeros(8, 1, 64, 64, device="cuda")
    for out in (None, 1):
        kw = dict(want_final=False)
        for n in (2 ** 70, 2 ** 32 + 1, -1, -2 ** 70):
            with pytest.raises(ValueError):
                gdn.causal_conv(x, w, B=n, out=out and o, **kw)
            with pytest.raises(ValueError):
                gdn.ssm_scan(**{**s, "init_state": None}, B=n, out=out and so, **kw)
            with pytest.raises((ValueError, gdn.GdnError)):
                gdn.add_norm(x, w[:, 0].contiguous(), group=n, e4m3=True, out=out and q)
        with pytest.raises(KeyError):
            gdn.causal_conv(x, w, silu=Neither(), out=out and o, **kw)
        with pytest.raises(KeyError):
            gdn.causal_conv_step(x, w, st, silu=Neither(), out=out and o)
        with pytest.raises(KeyError):
            gdn.ssm_scan(**s, softplus=Neither(), out=out and so, **kw)
        with pytest.raises(KeyError):
            gdn.ssm_step(**rows_of(s, slice(0, 8)), state=state, softplus=Neither(), out=out and so)


def test_norm_returns_no_scales_with_a_bf16_output(gdn, monkeypatch):
    x, w = rnd(gen(80), 4, 64), rnd(gen(81), 64)
    sc = torch.full((4, 1), 7.0, device="cuda")
    for _ in range(2):
        out, none, _ = gdn.add_norm(x, w, scales=sc, out=torch.empty_like(x))
        assert none is None and bool((sc == 7).all())
        monkeypatch.setattr(gdn, "_fast", None)


def test_norm_of_nearly_2_to_the_31_rows(gdn):
    rows = 2 ** 31 - 1
    x = torch.zeros(rows, 8, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(8, dtype=torch.bfloat16, device="cuda")
    x[-3:] = rnd(gen(82), 3, 8)
    out, _, _ = gdn.add_norm(x, w, out=torch.full_like(x, 7.0))
    assert torch.equal(out[-3:], gdn.add_norm(x[-3:], w)[0]) and not bool(out[:1000].any())
    assert not bool(out[2 ** 30:2 ** 30 + 1000].any())
    del x, out
    torch.cuda.empty_cache()


# ---- waits that run out ---------------------------------------------------------------------------

@pytest.mark.parametrize("T,Hv,dk,dv", [(100, 1, 64, 64), (300, 2, 128, 32), (1000, 1, 128, 128),
                                        (6000, 2, 32, 128)])
def test_scan_whose_waits_run_out_ends_and_says_so(gdn, T, Hv, dk, dv):
    """The issuing threads give up at once, copies in flight, and what waits for them after its own limit: in one
    pass, two and three."""
    s = scan_inputs(gen(89), T, 1, 1, Hv, dk, dv, init=True)
    ref = gdn.ssm_scan(**s)
    timeouts = gdn.GDN_STATUS_MMA_TIMEOUT | gdn.GDN_STATUS_LOAD_TIMEOUT
    assert gdn.gdn_device_status() == (0, 0)
    usual = gdn.gdn_debug_ssm_wait_polls(0)
    try:
        gdn.ssm_scan(**s)
        rc, bits = gdn.gdn_device_status()
        assert rc == 0 and bits & timeouts and not bits & ~timeouts
    finally:
        assert gdn.gdn_debug_ssm_wait_polls(-1) == 0
    assert gdn.gdn_debug_ssm_wait_polls(usual) == usual
    again = gdn.ssm_scan(**s)
    assert torch.equal(again[0], ref[0]) and torch.equal(again[1], ref[1])
    assert gdn.gdn_device_status() == (0, 0)


# ---- strong decays, steps below zero --------------------------------------------------------------

@pytest.mark.parametrize("dk,dv,Hk,Hv", [(64, 64, 1, 2), (128, 128, 1, 1), (32, 64, 1, 1)])
@pytest.mark.parametrize("dt", [20.0, 50.0, 200.0, 2000.0, 1e6])
def test_scan_long_steps(gdn, dt, dk, dv, Hk, Hv):
    # s A of -320 to -1.6e7 a token: what is left is s_i (C_i . B_i) x_i, to the roundings of any other call
    s = scan_inputs(gen(83), 300, 1, Hk, Hv, dk, dv, dt32=True, bias=False, init=True)
    s["A"] = torch.full((Hv,), -16.0, device="cuda")
    s["dt"] = dt * (0.5 + torch.rand(300, Hv, generator=gen(84))).cuda()
    scan_check(gdn, s, 1, 300)


@pytest.mark.parametrize("every", [0, 3, 29, 37, 64])
@pytest.mark.parametrize("reset", [20.0, 1e4, 1e6, 1e30])
def test_scan_resets_between_slow_decays(gdn, reset, every):
    # single tokens of a very long step forget the state; the tokens after them decay slowly. A reset token's own
    # input is left out, since its step would put it above all others.
    s = scan_inputs(gen(85), 400, 1, 1, 2, 64, 64, dt32=True, bias=False, init=True)
    s["A"] = torch.tensor([-16.0, -1.0], device="cuda")
    at = slice(3, 4) if every == 0 else slice(1, None, every)
    s["dt"] = torch.full((400, 2), -4.0, device="cuda") + 0.3 * rnd(gen(86), 400, 2, dtype=torch.float32)
    s["dt"][at] = reset
    s["x"][at] = 0
    scan_check(gdn, s, 1, 400)


def test_scan_nan_step_reaches_later_tokens_only(gdn):
    # in its chunk and after it, the chunk's tokens before it left as they are
    s = scan_inputs(gen(87), 200, 1, 1, 1, 64, 64, dt32=True, bias=False)
    ref, _ = gdn.ssm_scan(**s)
    s["dt"][140] = float("nan")
    out, fin = gdn.ssm_scan(**s)
    assert torch.equal(out[:140], ref[:140])
    assert bool(out[140:].isnan().all()) and bool(fin.isnan().all())


@pytest.mark.parametrize("T", [300, 3000])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_scan_value_that_is_not_finite_stays_in_its_column(gdn, T, bad):
    # from the start of its chunk on, as documented; other columns, heads and earlier chunks are left as they are
    s = scan_inputs(gen(90), T, 1, 1, 2, 64, 64, init=True)
    ref, rfin = gdn.ssm_scan(**s)
    s["x"][200, 1, 5] = bad
    out, fin = gdn.ssm_scan(**s)
    assert not bool(out[200:, 1, 5].isfinite().any()) and not bool(fin[0, 1, 5].isfinite().any())
    mine = torch.zeros_like(out, dtype=torch.bool)
    mine[128:, 1, 5] = True
    assert torch.equal(out[~mine], ref[~mine])
    keep = torch.ones_like(fin, dtype=torch.bool)
    keep[0, 1, 5] = False
    assert torch.equal(fin[keep], rfin[keep])


@pytest.mark.parametrize("T", [300, 3000])
@pytest.mark.parametrize("which", ["Bm", "Cm", "z"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_scan_b_c_and_gate_that_are_not_finite_reach_no_token_before(gdn, T, which, bad):
    s = scan_inputs(gen(91), T, 1, 1, 2, 64, 64, init=True)
    ref, _ = gdn.ssm_scan(**s)
    s[which][200, 0, 5] = bad
    out, _ = gdn.ssm_scan(**s)
    assert torch.equal(out[:200], ref[:200]) and not bool(out[200, 0].isfinite().all())
    if which != "Bm":  # C and the gate are of one token
        assert torch.equal(out[201:], ref[201:])


@pytest.mark.parametrize("dk,dv,Hk,Hv", [(64, 64, 1, 2), (128, 128, 2, 2), (32, 32, 1, 1), (128, 64, 1, 2)])
@pytest.mark.parametrize("T", [1, 140, 1500])
def test_scan_steps_below_zero(gdn, dk, dv, Hk, Hv, T):
    # without softplus a step may be below zero: prompts and single tokens agree with the formula
    s = scan_inputs(gen(88), T, 1, Hk, Hv, dk, dv, bias=False, dt32=True, init=True)
    s["dt"] *= 0.1
    out, fin = scan_check(gdn, s, 1, T, softplus=False)
    if T == 140:
        st = s["init_state"].clone()
        for t in range(5):
            y = gdn.ssm_step(**rows_of(s, slice(t, t + 1)), state=st, softplus=False)
            assert float((y - out[t:t + 1]).abs().max()) <= 2.0 ** -5 * float(out.abs().max())
