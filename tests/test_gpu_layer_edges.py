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
