"""Attention and its cache at their long forms, where a launch, a join or a thread takes another way than with few
tokens (GPU).  Tolerances are those of test_gpu_attn.py; of long prompts, some rows are compared.
"""

import numpy as np
import pytest

import attn_refs as R
from test_gpu_attn import BF, I32, close, close_lse, cu_of, gen, ints, n64, rnd, run_plan, slices, torch
from test_gpu_attn import gdn  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn


# ---- one token: parts joined in several rounds, maxima that move ---------------------------------

def sloped_cache(g, n, Hkv, d, page, slope, e4m3):
    """A cache of one request whose first column grows by `slope` / 8 a token, its table and scales."""
    W = -(-n // page)
    order = torch.randperm(W, generator=g)
    kv = torch.randn(2, W * page, Hkv, d, generator=g)
    kv[0, :, :, 0] = slope / 8 * torch.arange(W * page, dtype=torch.float32)[:, None]
    cache = torch.empty(2, W, Hkv, page, d)
    cache[:, order] = kv.unflatten(1, (W, page)).transpose(2, 3)
    scales = []
    if e4m3:
        scale = max(abs(slope) * n / 8 / 400, 0.01)
        scales = [torch.full((Hkv,), scale, device="cuda"), torch.full((Hkv,), 0.01, device="cuda")]
        cache = (cache / torch.tensor([scale, 0.01])[:, None, None, None, None]).clamp(-448, 448)
    cache = cache.to(F8 if e4m3 else BF).cuda()
    return cache[0], cache[1], order.tolist(), scales


def check_sloped(gdn, g, n, Hq, Hkv, d, page, slope, e4m3):
    kc, vc, table, scales = sloped_cache(g, n, Hkv, d, page, slope, e4m3)
    q = rnd(g, 1, Hq, d)
    q[:, :, 0] = 8.0
    args = (q, kc, vc, ints([table]), ints([n]), *scales)
    out, lse = gdn.attention_step(*args, scale=1.0, want_lse=True)
    for _ in range(3):  # the same sums in the same order, whatever finishes first
        again = gdn.attention_step(*args, scale=1.0, want_lse=True)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    k, v = (R.paged(n64(c.float()), table, n) for c in (kc, vc))
    if e4m3:
        k, v = (x * n64(s)[:, None] for x, s in ((k, scales[0]), (v, scales[1])))
    y, mag, l, bound = R.attend(n64(q), k, v, 1.0)
    close(out, y, mag, bound)
    close_lse(lse, l, bound)


@pytest.mark.parametrize("n,Hq,Hkv,d", [(2400, 16, 1, 32), (6000, 16, 1, 32), (9500, 16, 1, 128), (16381, 16, 1, 128),
                                        (16381, 13, 1, 96), (12000, 32, 1, 64)])
@pytest.mark.parametrize("rise", [60.0, -60.0, 0.0])
@pytest.mark.parametrize("e4m3", [False, True])
def test_step_parts_joined_in_rounds(gdn, n, Hq, Hkv, d, rise, e4m3):
    # more parts than the statistics that fit into shared memory at once: 36 of 16 heads of 32 columns, 132 of 128; scores
    # rise or fall by 60 along the cache, so that a later round brings a higher maximum, or none
    check_sloped(gdn, gen(n + d), n, Hq, Hkv, d, 16, rise / n, e4m3)


@pytest.mark.parametrize("slope", [0.005, -0.005, 0.05, -0.05, 0.3, 0.34, 0.5, 3.0, -3.0])
@pytest.mark.parametrize("n", [600, 5000])
@pytest.mark.parametrize("e4m3", [False, True])
def test_step_sizes_of_scores_of_either_cache(gdn, slope, n, e4m3):
    # (a maximum stays in use until a score is 2^8 above it: 16 tokens of 0.34 rise by 2^7.8)
    check_sloped(gdn, gen(n), n, 3, 1, 64, 16, slope, e4m3)


@pytest.mark.parametrize("lens,Hq,Hkv,d,page,window,sinks,e4m3", [
    ([16381, 1024, 9000, 1], 32, 8, 128, 16, 0, 0, True), ([16381, 12345], 32, 8, 128, 64, 0, 0, False),
    ([8192, 1024, 5000, 1023, 1025], 32, 8, 128, 64, 1024, 4, False)])
def test_step_long_requests(gdn, lens, Hq, Hkv, d, page, window, sinks, e4m3):
    g = gen(len(lens))
    W = -(-max(lens) // page)
    table = torch.randperm(len(lens) * W, generator=g).reshape(len(lens), W)
    cache = torch.randn(2, len(lens) * W, Hkv, page, d, generator=g)
    scales = [torch.rand(Hkv, generator=g).cuda() / 100 + 0.01 for _ in range(2)] if e4m3 else []
    if e4m3:
        cache = (cache / torch.stack(scales).cpu()[:, None, :, None, None]).clamp(-448, 448)
    cache = cache.to(F8 if e4m3 else BF).cuda()
    q = rnd(g, len(lens), Hq, d)
    out, lse = gdn.attention_step(q, cache[0], cache[1], ints(table.tolist()), ints(lens), *scales, window=window,
                                  sinks=sinks, want_lse=True)
    for b, n in enumerate(lens):
        blocks = table[b, :-(-n // page)].cuda()
        k, v = (n64(c[blocks].float()).transpose(0, 2, 1, 3).reshape(-1, Hkv, d)[:n] for c in cache)
        if e4m3:
            k, v = (x * n64(s)[:, None] for x, s in zip((k, v), scales))
        y, mag, l, bound = R.attend(n64(q[b:b + 1]), k, v, d ** -0.5, window, sinks)
        close(out[b:b + 1], y, mag, bound)
        close_lse(lse[b:b + 1], l, bound)


# ---- writing: several tokens a thread ------------------------------------------------------------

@pytest.mark.parametrize("T,Hkv,d,page", [(20003, 8, 128, 64), (1003, 40, 128, 16), (90001, 1, 32, 48), (31111, 3, 104, 256)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_append_many_tokens(gdn, T, Hkv, d, page, e4m3):
    g = gen(T)
    blocks = -(-T // page) + 2
    kv = (torch.randn(T, 2 * Hkv * d + 16, generator=g) * 3).to(BF).cuda()
    k, v = kv[:, 8:8 + Hkv * d].unflatten(1, (Hkv, d)), kv[:, 16 + Hkv * d:].unflatten(1, (Hkv, d))
    caches = torch.randn(blocks, 2, Hkv, page, d, generator=g).to(F8 if e4m3 else BF).cuda()
    before = caches.clone()
    slots = torch.randperm(blocks * page, generator=g)[:T].to(I32)
    slots[5::7] = -1 - slots[5::7]  # passed over, as what lies past the cache
    slots[11::501] = blocks * page + slots[11::501].abs()
    slots[T - 1], slots[T - 3], slots[0] = 2 ** 31 - 1, -2 ** 31, blocks * page
    scales = [torch.rand(Hkv, generator=g).cuda() / 50 + 0.01 for _ in range(2)] if e4m3 else [None, None]
    gdn.cache_append(k, v, caches[:, 0], caches[:, 1], slots.cuda(), *scales)
    at = slots.long().cuda()
    there = (at >= 0) & (at < blocks * page)
    at = at[there]
    wrote = torch.zeros(blocks * page, dtype=torch.bool, device="cuda")
    wrote[at] = True
    for i, (x, scale) in enumerate(((k, scales[0]), (v, scales[1]))):
        got, old = (c[:, i].transpose(1, 2).flatten(0, 1) for c in (caches, before))  # [tokens, Hkv, d]
        assert torch.equal(got[~wrote].float(), old[~wrote].float())
        if not e4m3:
            assert torch.equal(got[at], x[there])
            continue
        want = (x[there].double() / scale.double()[:, None]).clamp(-448, 448)
        tol = torch.clamp(2.0 ** -4 * want.abs(), min=2.0 ** -10) + 2.0 ** -20 * want.abs()
        assert bool(((got[at].double() - want).abs() <= tol).all())


# ---- prompts ----------------------------------------------------------------------------------

def check_rows_of(out, lse, q, k, v, rows, keys, window, sinks):
    """Rows (of these queries, the last of these keys) against float64."""
    n, m = q.shape[0], k.shape[0]
    rows = sorted({r for r in rows if 0 <= r < n})
    y, mag, l, bound = R.attend(n64(q[rows]), keys[0], keys[1], q.shape[2] ** -0.5, window, sinks,
                                positions=[m - n + r for r in rows])
    close(out[rows], y, mag, bound)
    close_lse(lse[rows], l, bound)


@pytest.mark.parametrize("n,m,Hq,Hkv,d,window,sinks", [
    (16381, 16381, 16, 2, 128, 0, 0), (16381, 16381, 4, 1, 64, 1000, 4), (500, 16381, 8, 2, 128, 0, 0),
    (4096, 9000, 8, 4, 96, 4000, 130), (16384, 16384, 2, 2, 32, 0, 0)])
def test_attention_long_prompts(gdn, n, m, Hq, Hkv, d, window, sinks):
    g = gen(n)
    q, k, v = slices(g, n, m, Hq, Hkv, d)
    out, lse = gdn.attention(q, k, v, cu_of([n]), cu_of([m]) if m != n else None, window=window, sinks=sinks, want_lse=True)
    rows = [0, 1, 127, 128, n - 1, n - 2, n - 129] + torch.randint(0, n, (40,), generator=g).tolist()
    check_rows_of(out, lse, q, k, v, rows, (n64(k), n64(v)), window, sinks)
    assert bool(out.isfinite().all()) and gdn.gdn_device_status() == (0, 0)


@pytest.mark.parametrize("window,sinks", [(0, 0), (1024, 4)])
def test_a_long_packed_batch(gdn, window, sinks):
    """32 prompts, 70,000 tokens or so: planned, written in both types, attended to."""
    g = gen(31)
    Hq, Hkv, d, page = 16, 4, 128, 64
    lens = torch.randint(200, 4097, (32,), generator=g).tolist()
    T, cu = sum(lens), [0] + np.cumsum(lens).tolist()
    q, k, v = slices(g, T, T, Hq, Hkv, d)
    blocks = sum(-(-n // page) for n in lens) + 3
    stack = torch.randperm(blocks, generator=g).tolist()
    slots = run_plan(gdn, [0] * 32, [[-1] * 64] * 32, stack, blocks, cu, page, T)[0]
    out, lse = gdn.attention(q, k, v, ints(cu), window=window, sinks=sinks, want_lse=True)
    for b, n in enumerate(lens):
        sl = slice(cu[b], cu[b + 1])
        rows = [0, 127, n - 1, n // 2] + torch.randint(0, n, (3,), generator=g).tolist()
        check_rows_of(out[sl], lse[sl], q[sl], k[sl], v[sl], rows, (n64(k[sl]), n64(v[sl])), window, sinks)
    assert bool(out.isfinite().all())
    kc, vc = (torch.zeros(blocks, Hkv, page, d, dtype=BF, device="cuda") for _ in range(2))
    gdn.cache_append(k, v, kc, vc, slots)
    at = slots.long()
    assert torch.equal(kc.transpose(1, 2).flatten(0, 1)[at], k) and torch.equal(vc.transpose(1, 2).flatten(0, 1)[at], v)
    # the last token of every prompt again, over the cache: the same sums in another order
    table = torch.full((32, 64), -1, dtype=I32, device="cuda")
    for b, n in enumerate(lens):
        table[b, :-(-n // page)] = slots[cu[b]:cu[b + 1]:page] // page
    ends = torch.tensor(cu[1:], device="cuda") - 1
    one, one_lse = gdn.attention_step(q[ends], kc, vc, table, ints(lens), window=window, sinks=sinks, want_lse=True)
    for b, n in enumerate(lens):
        sl = slice(cu[b], cu[b + 1])
        check_rows_of(one[b:b + 1], one_lse[b:b + 1], q[ends][b:b + 1], k[sl], v[sl], [0], (n64(k[sl]), n64(v[sl])), window,
                      sinks)
