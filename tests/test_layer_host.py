"""Refusals of the operators around the recurrence: before any GPU work, with the status codes the header
states (C entries), and as ValueError from the tensor wrappers (CPU only)."""

import pytest
import torch

from hybrid_linear_attention_prefill_gb300 import build as B
from hybrid_linear_attention_prefill_gb300 import gdn

FAKE = 1 << 20  # a 256-byte aligned address that is never dereferenced
FAR = 1 << 40


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()
    return gdn.load()


CONV = dict(x=FAKE, x_stride=64, weight=FAKE, bias=None, cu_seqlens=None, init_state=None, out=FAR, final_state=None,
            B=1, T=16, C=64, K=4, flags=1, stream=0)
STEP = dict(x=FAKE, x_stride=64, weight=FAKE, bias=None, state=FAKE, out=FAR, B=2, C=64, K=4, flags=1, stream=0)
SSM = dict(x=FAKE, x_stride=256, dt=FAKE, dt_stride=4, A=FAKE, Bm=FAKE, b_stride=128, Cm=FAKE, c_stride=128, D=None,
           z=None, z_stride=0, dt_bias=None)
SCAN = dict(**SSM, cu_seqlens=None, init_state=None, out=FAR, final_state=None, B=1, T=16, Hk=2, Hv=4, dk=64, dv=64,
            flags=1, workspace=FAKE, workspace_bytes=1 << 40, stream=0)
SSTEP = dict(**SSM, state=FAKE, out=FAR, B=2, Hk=2, Hv=4, dk=64, dv=64, flags=1, stream=0)
NORM = dict(x=FAKE, x_stride=64, residual=None, weight=FAKE, residual_out=None, out=FAR, scales=None, rows=2, D=64,
            group=0, eps=1e-6, flags=0, stream=0)
ARG, ALIGN = gdn.GDN_ERR_ARG, gdn.GDN_ERR_ALIGN


@pytest.mark.parametrize("kw, code", [
    (dict(B=-1), ARG), (dict(T=-1), ARG), (dict(C=60), ARG), (dict(C=0), ARG), (dict(K=1), ARG), (dict(K=5), ARG),
    (dict(flags=2), ARG), (dict(x=None), ARG), (dict(weight=None), ARG), (dict(out=None), ARG),
    (dict(x_stride=56), ARG), (dict(x_stride=68), ALIGN), (dict(x=FAKE + 8), ALIGN), (dict(out=FAR + 2), ALIGN),
    (dict(bias=FAKE + 4), ALIGN), (dict(cu_seqlens=FAKE + 2), ALIGN), (dict(out=FAKE), ARG),
    (dict(init_state=FAR, final_state=FAR), ARG), (dict(B=1 << 20, T=1 << 20), ARG)])
def test_conv_refusals(kw, code):
    assert gdn.gdn_conv(**{**CONV, **kw}) == code


@pytest.mark.parametrize("kw, code", [
    (dict(B=-1), ARG), (dict(C=12), ARG), (dict(K=9), ARG), (dict(state=None), ARG), (dict(out=None), ARG),
    (dict(state=FAKE + 8), ALIGN), (dict(x_stride=65), ALIGN), (dict(flags=4), ARG)])
def test_conv_step_refusals(kw, code):
    assert gdn.gdn_conv_step(**{**STEP, **kw}) == code


@pytest.mark.parametrize("kw, code", [
    (dict(B=-1), ARG), (dict(T=-1), ARG), (dict(Hk=0), ARG), (dict(Hk=3), ARG), (dict(dk=48), ARG), (dict(dv=16), ARG),
    (dict(flags=4), ARG), (dict(x=None), ARG), (dict(dt=None), ARG), (dict(A=None), ARG), (dict(Bm=None), ARG),
    (dict(Cm=None), ARG), (dict(out=None), ARG), (dict(x_stride=255), ARG), (dict(x_stride=260), ALIGN),
    (dict(b_stride=64), ARG), (dict(c_stride=130), ALIGN), (dict(dt_stride=3), ARG), (dict(z=FAKE, z_stride=8), ARG),
    (dict(z=FAKE + 2, z_stride=256), ALIGN), (dict(dt=FAKE + 1), ALIGN), (dict(dt=FAKE + 2, flags=2), ALIGN),
    (dict(init_state=FAKE + 4), ALIGN), (dict(final_state=FAKE + 8), ALIGN), (dict(workspace=FAKE + 64), ALIGN),
    (dict(workspace_bytes=16), gdn.GDN_ERR_SCRATCH), (dict(B=1 << 20, T=1 << 20), ARG)])
def test_scan_refusals(kw, code):
    assert gdn.gdn_ssm_scan(**{**SCAN, **kw}) == code


@pytest.mark.parametrize("kw, code", [
    (dict(B=-1), ARG), (dict(dk=256), ARG), (dict(state=None), ARG), (dict(state=FAKE + 4), ALIGN), (dict(x=None), ARG),
    (dict(out=FAR + 8), ALIGN), (dict(flags=8), ARG)])
def test_scan_step_refusals(kw, code):
    assert gdn.gdn_ssm_step(**{**SSTEP, **kw}) == code


@pytest.mark.parametrize("kw, code", [
    (dict(rows=-1), ARG), (dict(D=12), ARG), (dict(D=32776, x_stride=32776), ARG), (dict(flags=2), ARG),
    (dict(group=128), ARG), (dict(flags=1), ARG), (dict(flags=1, scales=FAKE, group=48), ARG), (dict(x=None), ARG),
    (dict(weight=None), ARG), (dict(x_stride=63), ARG), (dict(x_stride=66), ALIGN), (dict(residual=FAKE + 8), ALIGN),
    (dict(residual_out=FAKE + 2), ALIGN), (dict(out=FAR + 8), ALIGN), (dict(flags=1, scales=FAKE + 2), ALIGN)])
def test_norm_refusals(kw, code):
    assert gdn.gdn_add_norm(**{**NORM, **kw}) == code


def test_nothing_to_do():
    assert gdn.gdn_conv(**{**CONV, "B": 0}) == gdn.GDN_OK
    assert gdn.gdn_conv(**{**CONV, "T": 0}) == gdn.GDN_OK
    assert gdn.gdn_conv_step(**{**STEP, "B": 0}) == gdn.GDN_OK
    assert gdn.gdn_ssm_scan(**{**SCAN, "B": 0}) == gdn.GDN_OK
    assert gdn.gdn_ssm_scan(**{**SCAN, "T": 0}) == gdn.GDN_OK
    assert gdn.gdn_ssm_step(**{**SSTEP, "B": 0}) == gdn.GDN_OK
    assert gdn.gdn_add_norm(**{**NORM, "rows": 0}) == gdn.GDN_OK


def test_workspace_bytes_refuses_bad_sizes():
    assert gdn.gdn_ssm_workspace_bytes(1, 64, 2, 3, 64, 64, 0) == 0
    assert gdn.gdn_ssm_workspace_bytes(1, 64, 2, 4, 48, 64, 0) == 0
    assert gdn.gdn_ssm_workspace_bytes(1, 64, 2, 4, 64, 64, 0) >= 256


def test_wrappers_refuse_wrong_tensors():
    bf, z = torch.bfloat16, torch.zeros
    x, w = z(8, 64, dtype=bf), z(64, 4, dtype=bf)
    for bad in (lambda: gdn.causal_conv(x.float(), w), lambda: gdn.causal_conv(x, w.float()),
                lambda: gdn.causal_conv(x, z(32, 4, dtype=bf)), lambda: gdn.causal_conv(x.t(), z(8, 4, dtype=bf)),
                lambda: gdn.causal_conv(x, w, B=3), lambda: gdn.causal_conv(x, w, z(32, dtype=bf)),
                lambda: gdn.causal_conv(x, w, cu_seqlens=z(3, dtype=torch.int64)),
                lambda: gdn.causal_conv(x, w, init_state=z(1, 4, 64, dtype=bf)),
                lambda: gdn.causal_conv(x, w, out=z(8, 64)),
                lambda: gdn.causal_conv_step(x, w, z(8, 3, 32, dtype=bf)),
                lambda: gdn.add_norm(x, z(32, dtype=bf)), lambda: gdn.add_norm(x, z(64, dtype=bf), z(8, 64)),
                lambda: gdn.add_norm(x, z(64, dtype=bf), e4m3=True, scales=z(8, 2)),
                lambda: gdn.add_norm(x[:, ::2], z(32, dtype=bf))):
        with pytest.raises(ValueError):
            bad()
    s = dict(x=z(8, 4, 64, dtype=bf), dt=z(8, 4), A=z(4), Bm=z(8, 2, 32, dtype=bf), Cm=z(8, 2, 32, dtype=bf))
    for kw in (dict(x=z(8, 4, 64)), dict(dt=z(8, 3)), dict(dt=z(8, 4, dtype=torch.float16)), dict(A=z(4, dtype=bf)),
               dict(Cm=z(8, 2, 64, dtype=bf)), dict(Bm=z(7, 2, 32, dtype=bf)), dict(D=z(3)), dict(z=z(8, 4, 32, dtype=bf)),
               dict(dt_bias=z(4, 1)), dict(x=z(8, 64, 4, dtype=bf).transpose(1, 2))):
        with pytest.raises(ValueError):
            gdn.ssm_scan(**{**s, **kw})
        with pytest.raises(ValueError):
            gdn.ssm_step(**{**s, **kw}, state=z(8, 4, 64, 32))
    with pytest.raises(ValueError):
        gdn.ssm_scan(**s, init_state=z(1, 4, 32, 64))
    with pytest.raises(ValueError):
        gdn.ssm_step(**s, state=z(8, 4, 64, 64))


def test_wrappers_refuse_host_tensors():
    bf, z = torch.bfloat16, torch.zeros
    x, w = z(8, 64, dtype=bf), z(64, 4, dtype=bf)
    s = dict(x=z(8, 4, 64, dtype=bf), dt=z(8, 4), A=z(4), Bm=z(8, 2, 32, dtype=bf), Cm=z(8, 2, 32, dtype=bf))
    for call in (lambda: gdn.causal_conv(x, w), lambda: gdn.causal_conv_step(x, w, z(8, 3, 64, dtype=bf)),
                 lambda: gdn.add_norm(x, z(64, dtype=bf)), lambda: gdn.ssm_scan(**s),
                 lambda: gdn.ssm_step(**s, state=z(8, 4, 64, 32))):
        with pytest.raises(ValueError, match="CUDA tensors"):
            call()
