"""Attention and its cache where they can go wrong: values that are not finite, calls at once, refusals (GPU).

Tolerances are those of test_gpu_attn.py.
"""

import threading

import numpy as np
import pytest

import attn_refs as R
from test_gpu_attn import BF, I32, NAN, close, close_lse, cu_of, gen, ints, n64, rnd, slices, torch
from test_gpu_attn import gdn  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

INF = float("inf")


def fastest(call, n=4):
    """Milliseconds of the fastest of n calls, after one."""
    call()
    times = []
    for _ in range(n):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        call()
        b.record()
        b.synchronize()
        times.append(a.elapsed_time(b))
    return min(times)


# ---- prompts: values that are not finite ---------------------------------------------------------

def sees(n, m, window, sinks):
    p, j = np.arange(m - n, m)[:, None], np.arange(m)[None]
    return (j <= p) & ((j > p - window) | (j < sinks) if window else True)


def check_odd(gdn, q, k, v, lens, window=0, sinks=0, packed=True):
    """Against float64 with the values that are not finite taken out, and put where they are seen: a column in which a
    row sees a NaN, or infinities of both signs, is NaN, one in which it sees an infinity is that."""
    out, lse = gdn.attention(q, k, v, cu_of(lens) if packed else None, B=None if packed else len(lens), window=window,
                             sinks=sinks, want_lse=True)
    G = q.shape[1] // k.shape[1]
    at = 0
    for n in lens:
        sl = slice(at, at + n)
        q64, k64, v64 = n64(q[sl]), n64(k[sl]), n64(v[sl])
        y, mag, l, bound = R.attend(q64, k64, v64, q.shape[2] ** -0.5, window, sinks)
        seen = sees(n, n, window, sinks).astype(np.float64)
        got, kind = n64(out[sl]), {}
        for what, there in (("nan", np.isnan(v64)), ("up", np.isposinf(v64)), ("down", np.isneginf(v64))):
            kind[what] = np.stack([seen @ there[:, h // G] > 0 for h in range(q.shape[1])], 1)
        nan = kind["nan"] | (kind["up"] & kind["down"])
        assert np.array_equal(np.isnan(got), nan)
        assert np.array_equal(np.isposinf(got), kind["up"] & ~nan) and np.array_equal(np.isneginf(got), kind["down"] & ~nan)
        odd = ~np.isfinite(got)
        close(torch.from_numpy(np.where(odd, 0.0, got)), np.where(odd, 0.0, y), np.where(odd, 0.0, mag), bound)
        close_lse(lse[sl], l, bound)
        at += n
    return out


ODD = [  # lens, Hq, Hkv, d, window, sinks
    ([700], 4, 1, 64, 0, 0), ([300, 1, 520], 8, 2, 128, 0, 0), ([900], 2, 2, 80, 0, 0), ([260, 400], 5, 1, 32, 0, 0),
    ([1100], 4, 1, 128, 200, 0), ([1100], 4, 2, 64, 130, 5), ([640, 300], 16, 1, 104, 150, 140), ([500], 128, 1, 16, 60, 1),
]


@pytest.mark.parametrize("lens,Hq,Hkv,d,window,sinks", ODD)
@pytest.mark.parametrize("what", ["first", "middle", "last", "both", "every 128", "every 300", "columns", "all", "huge"])
def test_attention_values_that_are_not_finite(gdn, lens, Hq, Hkv, d, window, sinks, what):
    g = gen(sum(lens) + d)
    T = sum(lens)
    q, k, v = slices(g, T, T, Hq, Hkv, d)
    h = Hkv - 1
    if what == "first":  # seen by every row of the first sequence
        v[0, h, 3] = NAN
        v[0, 0, d - 1] = -INF
    elif what == "middle":
        v[lens[0] // 2, h, 5] = INF
        v[lens[0] // 2 + 1, 0, 6] = NAN
    elif what == "last":  # beside the next sequence's rows, or at the end
        v[lens[0] - 1, h, 0] = NAN
        v[T - 1, 0] = INF
    elif what == "both":  # of both signs, in one column and in two
        v[10, h, 1], v[200, h, 1], v[lens[0] - 3, h, 2], v[lens[0] - 60, h, 4] = INF, -INF, -INF, INF
    elif what == "every 128":
        v[::128, h, 2] = NAN
        v[64::128, 0, 7] = INF
    elif what == "every 300":  # (a window forgets them)
        v[7::300, h, :2] = INF
        v[180::300, 0, 1] = NAN
    elif what == "columns":
        for c in range(d):
            v[(c * 37) % T, h, c] = (NAN, INF, -INF)[c % 3]
    elif what == "all":
        v[:, h] = NAN
        v[:, 0, ::2] = INF
    else:  # finite, but their weighted sums are not before the division
        v[:, h, :3] = 2e38
        v[T // 2, 0, 1] = NAN
    check_odd(gdn, q, k, v, lens, window, sinks)
    assert gdn.gdn_device_status() == (0, 0)


def test_attention_a_value_that_is_not_finite_is_quick(gdn):
    # rows that see it are looked into, not worked out one by one
    g = gen(3)
    q, k, v = rnd(g, 4096, 32, 128), rnd(g, 4096, 8, 128), rnd(g, 4096, 8, 128)
    out = torch.empty_like(q)
    clean = fastest(lambda: gdn.attention(q, k, v, out=out))
    for at in (0, 1000, 4095, slice(None)):
        odd = v.clone()
        odd[at, :, 3] = NAN
        assert fastest(lambda: gdn.attention(q, k, odd, out=out)) < 40 * clean  # 700 and more where every row was


def test_attention_keys_that_are_not_finite(gdn):
    # a score that is not a number reaches its row whole, the others not at all
    g = gen(4)
    q, k, v = rnd(g, 700, 4, 64), rnd(g, 700, 2, 64), rnd(g, 700, 2, 64)
    want, _ = gdn.attention(q, k, v, window=200, sinks=3)
    k[300, 1, 5] = NAN
    v[300, 0, 0] = NAN
    out, lse = gdn.attention(q, k, v, window=200, sinks=3, want_lse=True)
    assert bool(out[300:500, 2:].isnan().all()) and bool(lse[300:500, 2:].isnan().all())
    assert bool(out[300:500, :2, 0].isnan().all())
    for rest in (out[:300], out[500:], out[300:500, :2, 1:]):
        assert bool(rest.isfinite().all())
    assert bool(torch.isfinite(lse[:, :2]).all())
    assert torch.equal(out[640:], want[640:])  # (tiles far from the edge of what sees it)


# ---- the library's own workspaces ----------------------------------------------------------------

def step_of(gdn, g, lens, Hq, Hkv, d, page=16):
    """A step's call without a workspace, its output and what that has to be."""
    W = -(-max(lens) // page)
    kc, vc = rnd(g, W * len(lens), Hkv, page, d), rnd(g, W * len(lens), Hkv, page, d)
    table = torch.randperm(W * len(lens), generator=g).to(I32).cuda().reshape(len(lens), W)
    q, n = rnd(g, len(lens), Hq, d), ints(lens)
    out, lse = torch.empty_like(q), torch.empty(len(lens), Hq, device="cuda")
    ws = torch.zeros(gdn.gdn_attn_workspace_bytes(len(lens), Hq, Hkv, d), dtype=torch.uint8, device="cuda")
    want = [x.clone() for x in gdn.attention_step(q, kc, vc, table, n, want_lse=True, workspace=ws)]
    return (lambda **kw: gdn.attention_step(q, kc, vc, table, n, **{"out": out, "lse": lse, **kw})), out, lse, want


def test_steps_on_streams_at_once_without_a_workspace(gdn):
    # few CTAs each, so that they run beside one another, with parts of their own that share no counter
    g = gen(5)
    cases = [step_of(gdn, g, [n], 8, 1, 128) for n in (4000, 2500, 900, 3300)]
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(20):
        torch.cuda.synchronize()
        wrong = []
        for s in streams:
            with torch.cuda.stream(s):
                torch.cuda._sleep(400_000)
        for _ in range(8):
            for s, (call, out, lse, want) in zip(streams, cases):
                with torch.cuda.stream(s):
                    out.fill_(7)
                    call()
                    wrong.append((out != want[0]).any() | (lse != want[1]).any())
        torch.cuda.synchronize()
        assert not any(bool(w) for w in wrong)
    for call, out, lse, want in cases:  # and afterwards, one by one
        call()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_steps_on_more_streams_than_have_a_workspace(gdn):
    g = gen(6)
    cases = [step_of(gdn, g, lens, 4, 2, 64) for lens in ([1500], [40] * 700, [300, 2000])]  # (the second wants more room)
    streams = [torch.cuda.Stream() for _ in range(20)]
    raw = {s.cuda_stream for s in streams}
    assert len(raw) == 20
    torch.cuda.synchronize()
    for turn in range(4):
        for i, s in enumerate(streams):
            call, out, lse, want = cases[(i + turn) % 3]
            with torch.cuda.stream(s):
                out.fill_(7)
                call()
            s.synchronize()
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    gdn.gdn_release_workspace()
    for call, out, lse, want in cases:
        call()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert gdn.gdn_device_status() == (0, 0)


def test_bad_blocks_on_any_stream_are_reported(gdn):
    g = gen(7)
    kc, vc = rnd(g, 4, 1, 16, 64), rnd(g, 4, 1, 16, 64)
    q, n, table = rnd(g, 1, 2, 64), ints([40]), ints([[0, 4, 1]])
    gdn.gdn_device_status()
    for s in (torch.cuda.current_stream(), torch.cuda.Stream(), torch.cuda.Stream()):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            gdn.attention_step(q, kc, vc, table, n)
        assert gdn.gdn_device_status() == (0, gdn.GDN_STATUS_BAD_PAGE) and gdn.gdn_device_status() == (0, 0)


def test_a_step_without_a_workspace_is_not_captured(gdn):
    g = gen(8)
    call, out, lse, want = step_of(gdn, g, [700], 4, 2, 64)
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out.fill_(3)
        with pytest.raises(gdn.GdnError, match=str(gdn.GDN_ERR_SCRATCH)):
            call()
    graph.replay()
    assert bool((out == 3).all())
    call()
    assert torch.equal(out, want[0])


def test_a_prompt_without_a_workspace_is_captured_after_the_first_call(gdn):
    g = gen(9)
    q, k, v = rnd(g, 300, 4, 64), rnd(g, 300, 2, 64), rnd(g, 300, 2, 64)
    out = torch.empty_like(q)
    gdn.gdn_release_workspace()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out.fill_(3)
        with pytest.raises(gdn.GdnError, match=str(gdn.GDN_ERR_SCRATCH)):
            gdn.attention(q, k, v, out=out)
    want = gdn.attention(q, k, v)[0]
    step_of(gdn, g, [40] * 3000, 4, 2, 64)[0]()  # (a large step moves nothing that the graph holds)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.attention(q, k, v, out=out)
    step_of(gdn, g, [40] * 6000, 4, 2, 64)[0]()
    out.fill_(7)
    graph.replay()
    assert torch.equal(out, want)


@pytest.mark.parametrize("own_streams", [False, True])
def test_steps_from_threads_at_once_without_a_workspace(gdn, own_streams):
    """Threads whose calls want ever more room: what one enlarges, another may be about to use."""
    g = gen(12)
    sizes = ([9], [30] * 900, [2000], [20] * 2500, [700] * 3, [5] * 5000)
    cases = [step_of(gdn, g, lens, 4, 2, 64) for lens in sizes]
    gdn.gdn_release_workspace()
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        try:
            s = torch.cuda.Stream() if own_streams else torch.cuda.default_stream()
            with torch.cuda.stream(s):
                for n in range(12):
                    q_call, _, _, want = cases[(i + n) % len(cases)]
                    out = torch.empty_like(want[0])
                    got, _ = q_call(out=out if n % 2 else None, lse=None)
                    s.synchronize()
                    if not (torch.equal(got, want[0])):
                        wrong.append((i, n))
        except Exception as e:  # noqa: BLE001  (said by the assertion below)
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(6)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == []
    assert gdn.gdn_device_status() == (0, 0)


# ---- the smallest calls --------------------------------------------------------------------------

def test_calls_with_nothing_in_them(gdn):
    g = gen(13)
    none = ints([]).reshape(2, 0)
    cache = torch.empty(0, 2, 16, 64, dtype=BF, device="cuda")
    for lens in ([0, 0], [-5, 0], [40, 3]):  # no columns, no blocks: nothing is seen
        for given in (False, True):
            out = torch.full((2, 4, 64), 3, dtype=BF, device="cuda") if given else None
            out, lse = gdn.attention_step(rnd(g, 2, 4, 64), cache, cache, none, ints(lens), out=out, want_lse=True)
            assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())
    q = rnd(g, 0, 4, 64)
    assert gdn.attention(q, q[:, :2], q[:, :2])[0].shape == (0, 4, 64)
    assert gdn.attention(q, q[:, :2], q[:, :2], ints([0, 0, 0]), want_lse=True)[1].shape == (0, 4)
    assert gdn.attention_step(q, cache, cache, ints([]).reshape(0, 3), ints([]))[0].shape == (0, 4, 64)
    gdn.cache_append(q[:, :2], q[:, :2], cache, cache, ints([]))
    gdn.cache_append(rnd(g, 3, 2, 64), rnd(g, 3, 2, 64), cache, cache, ints([0, 1, 2]))  # nowhere to go
    out = torch.full((5, 4, 64), 3, dtype=BF, device="cuda")
    gdn.attention(rnd(g, 5, 4, 64), rnd(g, 5, 2, 64), rnd(g, 5, 2, 64), ints([0, 0, 0]), out=out)  # no sequence has any
    assert bool((out == 3).all()) and gdn.gdn_device_status() == (0, 0)


def test_a_step_with_more_tokens_than_columns(gdn):
    g = gen(14)
    kc, vc = rnd(g, 9, 2, 16, 64), rnd(g, 9, 2, 16, 64)
    q, table = rnd(g, 1, 4, 64), [[4, 0, 7]]
    out, lse = gdn.attention_step(q, kc, vc, ints(table), ints([2 ** 31 - 1]), want_lse=True)
    want, want_lse = gdn.attention_step(q, kc, vc, ints(table), ints([48]), want_lse=True)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("window,sinks", [(2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31 - 1, 0), (1, 2 ** 31 - 1), (0, 2 ** 31 - 1)])
def test_the_largest_windows_and_sinks(gdn, window, sinks):
    g = gen(15)
    q, k, v = rnd(g, 300, 4, 64), rnd(g, 300, 2, 64), rnd(g, 300, 2, 64)
    want, want_lse = gdn.attention(q, k, v, want_lse=True)  # all of them see everything before them
    out, lse = gdn.attention(q, k, v, window=window, sinks=sinks, want_lse=True)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    kc, vc = (t[:288].unflatten(0, (18, 16)).transpose(1, 2).contiguous() for t in (k, v))
    table, n = ints([list(range(18))]), ints([288])
    want, want_lse = gdn.attention_step(q[:1], kc, vc, table, n, want_lse=True)
    out, lse = gdn.attention_step(q[:1], kc, vc, table, n, window=window, sinks=sinks, want_lse=True)
    y, mag, l, bound = R.attend(n64(q[:1]), n64(k[:288]), n64(v[:288]), 64 ** -0.5)
    for o, s in ((out, lse), (want, want_lse)):
        close(o, y, mag, bound)
        close_lse(s, l, bound)


# ---- devices that prompts' kernels are not made for ------------------------------------------------

def test_another_start_of_shared_memory_is_refused(gdn):
    g = gen(10)
    q, k, v = rnd(g, 100, 4, 64), rnd(g, 100, 2, 64), rnd(g, 100, 2, 64)
    out, lse = torch.full_like(q, 3), torch.full((100, 4), 3.0, device="cuda")
    assert gdn.gdn_debug_attn_smem_base(2048) == 0
    try:
        with pytest.raises(gdn.GdnError, match=str(gdn.GDN_ERR_LAUNCH)):
            gdn.attention(q, k, v, out=out, lse=lse)
    finally:
        assert gdn.gdn_debug_attn_smem_base(0) == 2048
    assert bool((out == 3).all()) and bool((lse == 3).all()) and gdn.gdn_device_status() == (0, 0)
    assert gdn.gdn_debug_attn_smem_base(1024) == 0  # what it is
    want = gdn.attention(q, k, v, out=out)[0].clone()
    assert gdn.gdn_debug_attn_smem_base(0) == 1024
    assert torch.equal(gdn.attention(q, k, v)[0], want) and bool(want.isfinite().all())


# ---- one token: what the weights keep -----------------------------------------------------------

@pytest.mark.parametrize("lens,Hq,Hkv,d,window,sinks", [([3000] * 3, 8, 2, 128, 0, 0), ([700, 41, 2048], 20, 1, 64, 0, 0),
                                                        ([900, 1500], 4, 4, 80, 300, 5)])
def test_step_weights_over_a_bf16_cache(gdn, lens, Hq, Hkv, d, window, sinks):
    """A weight is 2^-16 of it off at most as two operands (the upper 16 bits and the rest, cut and rounded to 8), besides
    the fp32 rounding that `bound` is for: an output is its own rounding to bf16, 2^-8, and that."""
    g = gen(d)
    W = -(-max(lens) // 32)
    kc, vc = rnd(g, W * len(lens), Hkv, 32, d), rnd(g, W * len(lens), Hkv, 32, d)
    table = torch.randperm(W * len(lens), generator=g).reshape(len(lens), W)
    q = rnd(g, len(lens), Hq, d)
    out, lse = gdn.attention_step(q, kc, vc, ints(table.tolist()), ints(lens), window=window, sinks=sinks, want_lse=True)
    for b, n in enumerate(lens):
        k, v = (R.paged(n64(c), table[b].tolist(), n) for c in (kc, vc))
        y, mag, l, bound = R.attend(n64(q[b:b + 1]), k, v, d ** -0.5, window, sinks)
        err, tol = np.abs(n64(out[b:b + 1]) - y), 2.0 ** -8 * np.abs(y) + (2.0 ** -16 + 2 * bound) * mag
        assert np.all(err <= tol), np.max(err / tol)
        close_lse(lse[b:b + 1], l, bound)


@pytest.mark.parametrize("e4m3", [False, True])
def test_step_infinities_that_are_seen(gdn, e4m3):
    """An infinity among the values is one in the output, whatever of its weight the operands hold; two signs are NaN."""
    g = gen(11)
    kc, vc = rnd(g, 8, 1, 16, 64), rnd(g, 8, 1, 16, 64)
    q = rnd(g, 2, 8, 64)
    one = [torch.ones(1, device="cuda")] * 2 if e4m3 else []
    vc[1, 0, 3, 5], vc[2, 0, 1, 5], vc[5, 0, 0, 7] = INF, -INF, -INF
    kc[6] = 0  # weights of a power of two, that one operand holds
    q[1] = 0
    vc[6, 0, 2, 9], vc[7, 0, 15, 9] = INF, INF
    if e4m3:  # (which has no infinities, only NaN)
        kc, vc = (c.to(torch.float8_e4m3fn) for c in (kc, vc))
    out, lse = gdn.attention_step(q, kc, vc, ints([list(range(8))] * 2), ints([128, 128]), *one, want_lse=True)
    if e4m3:
        want = vc.float().isnan().any(0).any(1).expand(2, 8, 64)
        assert torch.equal(out.isnan(), want) and bool(out.isfinite()[~want].all())
    else:
        assert bool(out[:, :, 5].isnan().all()) and bool(torch.isneginf(out[:, :, 7]).all())
        assert bool(torch.isposinf(out[:, :, 9]).all())
        keep = [c for c in range(64) if c not in (5, 7, 9)]
        assert bool(out[:, :, keep].isfinite().all())
    assert bool(lse.isfinite().all())
