"""Refusals of attention and its paged cache: before any GPU work, with the status codes the header states
(C entries), and as ValueError from the tensor functions (CPU only)."""

import pytest
import torch

from hybrid_linear_attention_prefill_gb300 import build as B
from hybrid_linear_attention_prefill_gb300 import gdn

FAKE = 1 << 20  # a 256-byte aligned address that is never dereferenced
FAR = 1 << 40
ARG, ALIGN, OK = gdn.GDN_ERR_ARG, gdn.GDN_ERR_ALIGN, gdn.GDN_OK


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()
    return gdn.load()


PLAN = dict(lens=FAKE, block_table=FAKE, table_stride=8, free_blocks=FAKE, free_count=FAKE, cu_seqlens=None, slots=FAR,
            new_lens=FAR, new_count=FAR, refused=None, B=4, T=4, W=8, capacity=64, page=16, stream=0)
APPEND = dict(k=FAKE, k_stride=128, v=FAKE, v_stride=128, k_cache=FAR, k_block_stride=2048, v_cache=FAR,
              v_block_stride=2048, k_scale=None, v_scale=None, slots=FAKE, T=4, Hkv=2, d=64, page=16, blocks=8, flags=0,
              stream=0)
ATTN = dict(q=FAKE, q_stride=256, k=FAKE, k_stride=128, v=FAKE, v_stride=128, cu_seqlens=None, cu_seqlens_k=None, out=FAR,
            lse=None, B=1, T=16, Tk=16, Hq=4, Hkv=2, d=64, window=0, sinks=0, scale=0.125, flags=0, workspace=FAKE,
            workspace_bytes=1 << 40, stream=0)
STEP = dict(q=FAKE, q_stride=256, k_cache=FAKE, k_block_stride=2048, v_cache=FAKE, v_block_stride=2048, k_scale=None,
            v_scale=None, block_table=FAKE, table_stride=8, lens=FAKE, out=FAR, lse=None, B=3, Hq=4, Hkv=2, d=64, page=16,
            blocks=8, W=8, window=0, sinks=0, scale=0.125, flags=0, workspace=FAKE, workspace_bytes=1 << 40, stream=0)
NAN = float("nan")


@pytest.mark.parametrize("kw, code", [
    (dict(B=-1), ARG), (dict(T=-1), ARG), (dict(W=-1), ARG), (dict(capacity=-1), ARG), (dict(page=0), ARG),
    (dict(page=24), ARG), (dict(page=-16), ARG), (dict(B=16385, T=16385), ARG), (dict(T=5), ARG), (dict(lens=None), ARG),
    (dict(block_table=None), ARG), (dict(free_blocks=None), ARG), (dict(free_count=None), ARG), (dict(slots=None), ARG),
    (dict(new_lens=None), ARG), (dict(new_count=None), ARG), (dict(table_stride=7), ARG), (dict(lens=FAKE + 2), ALIGN),
    (dict(block_table=FAKE + 1), ALIGN), (dict(slots=FAR + 2), ALIGN), (dict(refused=FAR + 3), ALIGN),
    (dict(cu_seqlens=FAKE + 2), ALIGN), (dict(new_count=FAR + 2), ALIGN)])
def test_plan_refusals(kw, code):
    assert gdn.gdn_cache_plan(**{**PLAN, **kw}) == code


@pytest.mark.parametrize("kw, code", [
    (dict(T=-1), ARG), (dict(Hkv=0), ARG), (dict(d=60), ARG), (dict(d=136), ARG), (dict(d=0), ARG), (dict(page=8), ARG),
    (dict(page=20), ARG), (dict(blocks=-1), ARG), (dict(blocks=1 << 28), ARG), (dict(flags=2), ARG), (dict(k=None), ARG),
    (dict(v=None), ARG), (dict(k_cache=None), ARG), (dict(v_cache=None), ARG), (dict(slots=None), ARG),
    (dict(flags=1), ARG), (dict(k_scale=FAKE), ARG), (dict(flags=1, k_scale=FAKE), ARG), (dict(k_stride=120), ARG),
    (dict(v_stride=132), ALIGN), (dict(k=FAKE + 8), ALIGN), (dict(k_cache=FAR + 8), ALIGN), (dict(k_block_stride=2032), ARG),
    (dict(v_block_stride=2056), ALIGN), (dict(slots=FAKE + 1), ALIGN),
    (dict(flags=1, k_scale=FAKE, v_scale=FAKE + 2), ALIGN), (dict(T=0), OK), (dict(blocks=0), OK)])
def test_append_refusals(kw, code):
    assert gdn.gdn_cache_append(**{**APPEND, **kw}) == code


@pytest.mark.parametrize("kw, code", [
    (dict(B=-1), ARG), (dict(T=-1), ARG), (dict(Tk=-1), ARG), (dict(Hq=3), ARG), (dict(Hkv=0), ARG), (dict(d=12), ARG),
    (dict(d=256), ARG), (dict(Hq=258, Hkv=1, d=8, q_stride=2064), ARG), (dict(window=-1), ARG), (dict(sinks=-1), ARG),
    (dict(scale=NAN), ARG), (dict(scale=float("inf")), ARG), (dict(flags=1), ARG), (dict(q=None), ARG), (dict(k=None), ARG),
    (dict(v=None), ARG), (dict(out=None), ARG), (dict(q_stride=248), ARG), (dict(k_stride=130), ALIGN),
    (dict(v=FAKE + 8), ALIGN), (dict(out=FAR + 8), ALIGN), (dict(lse=FAR + 2), ALIGN), (dict(cu_seqlens_k=FAKE), ARG),
    (dict(cu_seqlens=FAKE, Tk=17), ARG), (dict(cu_seqlens=FAKE + 2), ALIGN), (dict(out=FAKE + 512), ARG),
    (dict(workspace=FAKE + 16), ALIGN), (dict(workspace_bytes=255), gdn.GDN_ERR_SCRATCH), (dict(B=1 << 20, T=1 << 20), ARG),
    (dict(B=0), OK), (dict(T=0), OK),
    (dict(B=1, T=2 ** 31 - 1, Tk=2 ** 31 - 1), ARG), (dict(B=2 ** 20, T=2048, Tk=1), ARG)])
def test_attn_refusals(kw, code):
    assert gdn.gdn_attn(**{**ATTN, **kw}) == code


@pytest.mark.parametrize("kw, code", [
    (dict(B=-1), ARG), (dict(W=-1), ARG), (dict(Hq=5), ARG), (dict(d=20), ARG), (dict(page=24), ARG), (dict(blocks=-2), ARG),
    (dict(flags=4), ARG), (dict(window=-2), ARG), (dict(sinks=-1), ARG), (dict(scale=NAN), ARG), (dict(W=1 << 28), ARG),
    (dict(q=None), ARG), (dict(k_cache=None), ARG), (dict(v_cache=None), ARG), (dict(lens=None), ARG), (dict(out=None), ARG),
    (dict(block_table=None), ARG), (dict(table_stride=4), ARG), (dict(flags=1), ARG), (dict(v_scale=FAKE), ARG),
    (dict(q=FAKE + 2), ALIGN), (dict(q_stride=260), ALIGN), (dict(k_block_stride=2047), ARG), (dict(k_cache=FAKE + 4), ALIGN),
    (dict(v_block_stride=2049), ALIGN), (dict(lens=FAKE + 2), ALIGN), (dict(block_table=FAKE + 3), ALIGN),
    (dict(out=FAR + 4), ALIGN), (dict(lse=FAR + 1), ALIGN), (dict(out=FAKE), ARG), (dict(workspace=FAKE + 128), ALIGN),
    (dict(workspace_bytes=16), gdn.GDN_ERR_SCRATCH), (dict(B=0), OK)])
def test_step_refusals(kw, code):
    assert gdn.gdn_attn_step(**{**STEP, **kw}) == code


def test_no_arguments():
    lib = gdn.load()
    for name in ("gdn_cache_plan", "gdn_cache_append", "gdn_attn", "gdn_attn_step"):
        assert getattr(lib, name)(None) == ARG


def test_workspace_bytes():
    assert gdn.gdn_attn_workspace_bytes(4, 8, 3, 64) == 0
    assert gdn.gdn_attn_workspace_bytes(-1, 8, 2, 64) == 0
    assert gdn.gdn_attn_workspace_bytes(4, 8, 2, 64) >= 256


# ---- the tensor functions ------------------------------------------------------------------------

BF, I32, F8 = torch.bfloat16, torch.int32, torch.float8_e4m3fn


class Entries:
    """Stands in for the library: notes the calls of its entries and returns 0."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def entry(*args):
            self.calls.append(name)
            return 0
        return entry


@pytest.fixture
def entries(monkeypatch):
    e = Entries()
    monkeypatch.setattr(gdn, "load", lambda *a: e)
    monkeypatch.setattr(gdn, "_fast", None)
    monkeypatch.setattr(gdn, "_raw_stream", lambda *a: 0)
    monkeypatch.setattr(gdn, "_call", lambda entry, args, dev: entry(args))
    return e


def z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


def plan_args(**kw):
    return {**dict(lens=z(4, dtype=I32), block_table=z(4, 8, dtype=I32), free_blocks=z(64, dtype=I32),
                   free_count=z(1, dtype=I32), page=16), **kw}


def append_args(**kw):
    return {**dict(k=z(4, 2, 64), v=z(4, 2, 64), k_cache=z(8, 2, 16, 64), v_cache=z(8, 2, 16, 64),
                   slots=z(4, dtype=I32)), **kw}


def attn_args(**kw):
    return {**dict(q=z(16, 4, 64), k=z(16, 2, 64), v=z(16, 2, 64)), **kw}


def step_args(**kw):
    return {**dict(q=z(3, 4, 64), k_cache=z(8, 2, 16, 64), v_cache=z(8, 2, 16, 64), block_table=z(3, 8, dtype=I32),
                   lens=z(3, dtype=I32)), **kw}


@pytest.mark.parametrize("name, args", [("cache_plan", plan_args), ("cache_append", append_args), ("attention", attn_args),
                                        ("attention_step", step_args)])
def test_calls_reach_their_entry(entries, name, args):
    getattr(gdn, name)(**args())
    assert entries.calls == [{"attention": "gdn_attn", "attention_step": "gdn_attn_step"}.get(name, "gdn_" + name)]


@pytest.mark.parametrize("f, args", [
    (gdn.cache_plan, plan_args(lens=z(4))), (gdn.cache_plan, plan_args(block_table=z(3, 8, dtype=I32))),
    (gdn.cache_plan, plan_args(block_table=z(4, 16, dtype=I32)[:, ::2])), (gdn.cache_plan, plan_args(T=5)),
    (gdn.cache_plan, plan_args(cu_seqlens=z(5, dtype=I32))), (gdn.cache_plan, plan_args(cu_seqlens=z(4, dtype=I32), T=4)),
    (gdn.cache_plan, plan_args(free_count=z(2, dtype=I32))), (gdn.cache_plan, plan_args(slots=z(5, dtype=I32), T=4)),
    (gdn.cache_plan, plan_args(page=16.0)), (gdn.cache_plan, plan_args(page=0)),
    (gdn.cache_append, append_args(v=z(4, 1, 64))), (gdn.cache_append, append_args(slots=z(5, dtype=I32))),
    (gdn.cache_append, append_args(slots=torch.zeros(4, dtype=torch.int64))),
    (gdn.cache_append, append_args(k_cache=z(8, 2, 16, 64, dtype=F8))), (gdn.cache_append, append_args(k_scale=z(2, dtype=torch.float32))),
    (gdn.cache_append, append_args(v_cache=z(8, 2, 32, 64))),
    (gdn.cache_append, append_args(k_cache=z(8, 16, 2, 64).transpose(1, 2))),
    (gdn.cache_append, append_args(k=z(4, 2, 128)[:, :, ::2])), (gdn.cache_append, append_args(k_cache=z(2, 16, 64))),
    (gdn.attention, attn_args(q=z(16, 4, 64, dtype=torch.float16))), (gdn.attention, attn_args(v=z(16, 2, 32))),
    (gdn.attention, attn_args(k=z(17, 2, 64), v=z(17, 2, 64), cu_seqlens=z(2, dtype=I32))),
    (gdn.attention, attn_args(cu_seqlens_k=z(2, dtype=I32))), (gdn.attention, attn_args(B=3)),
    (gdn.attention, attn_args(cu_seqlens=z(3, dtype=I32), cu_seqlens_k=z(2, dtype=I32))),
    (gdn.attention, attn_args(window=-1)), (gdn.attention, attn_args(window=1.5)), (gdn.attention, attn_args(sinks=1 << 40)),
    (gdn.attention, attn_args(out=z(16, 4, 32))), (gdn.attention, attn_args(lse=z(16, 4))),
    (gdn.attention, attn_args(workspace=torch.zeros(0, dtype=torch.uint8))),
    (gdn.attention, attn_args(workspace=torch.zeros(1024, dtype=torch.uint8)[::2])),
    (gdn.attention_step, step_args(lens=z(4, dtype=I32))), (gdn.attention_step, step_args(q=z(3, 4, 32))),
    (gdn.attention_step, step_args(block_table=z(3, 8, dtype=torch.int64))),
    (gdn.attention_step, step_args(v_cache=z(8, 2, 16, 64, dtype=F8))), (gdn.attention_step, step_args(sinks=-1)),
    (gdn.attention_step, step_args(v_scale=z(2, dtype=torch.float32))),
    (gdn.attention_step, step_args(out=z(4, 4, 64))), (gdn.attention_step, step_args(lse=z(3, 4)))])
def test_tensor_functions_refuse(entries, f, args):
    with pytest.raises(ValueError):
        f(**args)
    assert entries.calls == []


def test_tensor_functions_make_outputs(entries):
    slots, lens, count, refused = gdn.cache_plan(**plan_args(cu_seqlens=z(5, dtype=I32), T=9))
    assert (slots.shape, lens.shape, count.shape, refused.shape) == ((9,), (4,), (1,), (1,))
    given = [z(4, dtype=I32) for _ in range(2)]
    made = gdn.cache_plan(**plan_args(slots=given[0], new_lens=given[1]))
    assert made[0] is given[0] and made[1] is given[1]
    out, lse = gdn.attention(**attn_args(want_lse=True))
    assert out.shape == (16, 4, 64) and lse.shape == (16, 4) and lse.dtype is torch.float32
    out, lse = gdn.attention_step(**step_args())
    assert out.shape == (3, 4, 64) and lse is None


def test_tensor_functions_take_slices(entries):
    qkv = z(16, (4 + 2 + 2) * 64)
    gdn.attention(qkv[:, :256].unflatten(1, (4, 64)), qkv[:, 256:384].unflatten(1, (2, 64)),
                  qkv[:, 384:].unflatten(1, (2, 64)))
    both = z(8, 2, 2, 16, 64)
    gdn.attention_step(**step_args(k_cache=both[:, 0], v_cache=both[:, 1], block_table=z(3, 12, dtype=I32)[:, :8]))
    assert entries.calls == ["gdn_attn", "gdn_attn_step"]


def test_no_cuda_tensors():
    for f, args in ((gdn.cache_plan, plan_args()), (gdn.attention, attn_args()), (gdn.attention_step, step_args())):
        with pytest.raises(ValueError, match="CUDA"):
            f(**args)
