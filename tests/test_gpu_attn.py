"""Attention and its paged cache against their definitions in float64 (GPU).

Tolerances, from the roundings alone: the plan is of whole numbers; a bf16 copy is exact; an e4m3 value is within half
a step of 4 bits (2^-4 of it, 2^-10 below 2^-6) of x / scale.  An output is rounded to bf16 (2^-8 of it), its weights to
16 bits as operands (2^-8 of each term, so 2^-8 of the weighted mean of |v|), and a weight carries the fp32 rounding of
its score, `bound` in attn_refs, which is also the log's.
"""

import numpy as np
import pytest

import attn_refs as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF, I32 = torch.bfloat16, torch.int32
NAN = float("nan")


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


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rnd(g, *shape, dtype=BF):
    return torch.randn(shape, generator=g).to(dtype).cuda()


def ints(x):
    return torch.tensor(x, dtype=I32, device="cuda")


def cu_of(lens):
    return ints(np.concatenate([[0], np.cumsum(lens)]))


def close(got, y, mag, bound):
    got = n64(got)
    assert np.all(np.isfinite(got))
    tol = 2.0 ** -8 * np.abs(y) + (2.0 ** -8 + 2 * bound) * mag + 1e-30
    err = np.abs(got - y)
    assert np.all(err <= tol), f"worst error {np.max(err / tol):.3g} of its tolerance at {np.unravel_index(np.argmax(err / tol), y.shape)}"


def close_lse(got, lse, bound):
    got = n64(got)
    assert np.array_equal(np.isneginf(got), np.isneginf(lse))
    some = ~np.isneginf(lse)
    got, lse, bound = got[some], lse[some], bound[..., 0][some]
    assert np.all(np.abs(got - lse) <= 2 * bound + 2.0 ** -20 * (1 + np.abs(lse)))


# ---- the plan -----------------------------------------------------------------------------------

def run_plan(gdn, lens, table, free, count, cu, page, T, **kw):
    """The call on copies, checked against the plan by hand."""
    t, wide = ints(table).reshape(len(table), -1), None
    W = t.shape[1]
    if kw.pop("strided", False):
        wide = torch.full((len(table), W + 5), 77, dtype=I32, device="cuda")
        wide[:, 2:2 + W] = t
        t = wide[:, 2:2 + W]
    got = gdn.cache_plan(ints(lens), t, ints(free), ints([count]), None if cu is None else ints(cu), page=page,
                         T=None if cu is None else T, **kw)
    slots, new_lens, after, left, refused = R.plan(lens, table, free, count, cu, page, T, W)
    assert got[0].tolist() == slots
    assert got[1].tolist() == new_lens
    assert got[2].item() == left and got[3].item() == refused
    assert t.tolist() == after
    if wide is not None:
        assert bool((wide[:, :2] == 77).all()) and bool((wide[:, 2 + W:] == 77).all())
    return got


PLAN = [  # lens, new tokens each (None: one), page, W, free blocks, tokens behind the last
    ([0], None, 16, 1, 1, 0), ([16], None, 16, 2, 1, 0), ([15], None, 16, 1, 0, 0), ([5, -1, 32, 31, 0], None, 16, 4, 9, 0),
    ([16, 16, 3, 16], None, 16, 2, 2, 0),                # the third and fourth: one needs nothing, one goes without
    ([32, 1, 16], None, 16, 2, 9, 0),                    # the first's table is full
    ([0, 0, 0], [5, 0, 40], 16, 3, 7, 0), ([7, 100, 0, 63], [1, 29, 64, 2], 64, 4, 8, 3), ([0], [0], 16, 1, 2, 0),
    ([3, 3], [50, 60], 48, 2, 3, 2),                     # the second's does not fit
    ([0, 0, 0, 0], [33, 16, 1, 16], 16, 3, 5, 0),        # blocks end inside
    ([-5, 0], [9, 17], 16, 2, 2, 7),
]


@pytest.mark.parametrize("lens,new,page,W,free,pad", PLAN)
@pytest.mark.parametrize("strided", [False, True])
def test_plan(gdn, lens, new, page, W, free, pad, strided):
    rng = np.random.default_rng(1)
    table = rng.integers(100, 200, (len(lens), W)).tolist()
    stack = rng.permutation(90)[:max(free, 1) + 3].tolist()
    cu = None if new is None else [0] + np.cumsum(new).tolist()
    run_plan(gdn, lens, table, stack, free, cu, page, len(lens) if new is None else sum(new) + pad, strided=strided)


@pytest.mark.parametrize("seed", range(6))
def test_plan_many_requests(gdn, seed):
    rng = np.random.default_rng(seed)
    B, page = [1, 33, 1024, 1025, 5000, 16384][seed], int(rng.choice([16, 48, 256]))
    lens = rng.integers(-2, 900, B).tolist()
    W = 900 // page + 2
    table = rng.integers(0, 10 ** 6, (B, W)).tolist()
    free = int(rng.integers(B // 64, B // 8 + 2))
    stack = rng.permutation(10 ** 6)[:free + 1].tolist()
    run_plan(gdn, lens, table, stack, free, None, page, B)
    new = rng.integers(0, 9, B)
    run_plan(gdn, lens, table, stack, free * 2, [0] + np.cumsum(new).tolist(), page, int(new.sum()) + 11)


def test_plan_long_prompts(gdn):
    rng = np.random.default_rng(7)
    new = rng.integers(200, 4097, 32)
    new[5] = 0
    lens = rng.integers(0, 200, 32).tolist()
    stack = rng.permutation(5000)[:3000].tolist()
    run_plan(gdn, lens, rng.integers(0, 99, (32, 70)).tolist(), stack, 3000, [0] + np.cumsum(new).tolist(), 64,
             int(new.sum()) + 5)


@pytest.mark.parametrize("cu", [[0, 9, 4, 16], [3, 5, 8, 12], [0, 5, 400, 16], [-7, 5, 8, 16], [16, 0, 0, 0]])
def test_plan_malformed_boundaries_stay_in_bounds(gdn, cu):
    # results are unspecified; nothing outside the outputs may change
    bufs = [torch.full((48,), 7, dtype=I32, device="cuda") for _ in range(4)]
    table = torch.full((9, 12), 7, dtype=I32, device="cuda")
    for i, n in enumerate((16, 3, 1, 1)):
        bufs[i] = (bufs[i], bufs[i][16:16 + n])
    gdn.cache_plan(ints([0, 20, 40]), table[3:6, 4:8], ints(list(range(10))), ints([10]), ints(cu), page=16,
                   slots=bufs[0][1], new_lens=bufs[1][1], new_count=bufs[2][1], refused=bufs[3][1])
    for whole, part in bufs:
        assert bool((whole[:16] == 7).all()) and bool((whole[16 + part.numel():] == 7).all())
    table[3:6, 4:8] = 7
    assert bool((table == 7).all())


def test_plan_bad_entries_and_heights(gdn):
    assert run_plan(gdn, [5, 5], [[-3, 9], [2 ** 31 - 1, 9]], [1, 2], 2, None, 16, 2)[0].tolist() == [-1, -1]
    # a height past the stack, or below zero, counts as its end
    lens, table = ints([0, 16]), ints([[0, 0], [3, 0]])
    slots, new, count, refused = gdn.cache_plan(lens, table, ints([8, 9]), ints([100]), page=16)
    assert slots.tolist() == [144, 128] and count.item() == 0 and refused.item() == 0
    slots, new, count, refused = gdn.cache_plan(lens, table, ints([8, 9]), ints([-100]), page=16)
    assert slots.tolist() == [-1, -1] and count.item() == 0 and refused.item() == 2 and new.tolist() == [0, 16]
    # lengths next to 2^31
    slots, new, _, refused = gdn.cache_plan(ints([2 ** 31 - 1, 2 ** 31 - 17]), table, ints([8, 9]), ints([2]), page=16)
    assert slots.tolist() == [-1, -1] and refused.item() == 2 and new.tolist() == [2 ** 31 - 1, 2 ** 31 - 17]


def test_plan_no_requests(gdn):
    slots, lens, count, refused = gdn.cache_plan(ints([]), ints([]).reshape(0, 4), ints([1, 2]), ints([2]), ints([0]),
                                                 page=16, T=3)
    assert slots.tolist() == [-1] * 3 and count.item() == 2 and refused.item() == 0


def test_plan_in_place_and_captured(gdn):
    lens, table, stack, count = ints([15, 40, -1]), torch.zeros(3, 8, dtype=I32, device="cuda"), ints(list(range(20))), ints([20])
    slots, refused = ints([0, 0, 0]), ints([0])

    def step():
        gdn.cache_plan(lens, table, stack, count, page=16, slots=slots, new_lens=lens, new_count=count, refused=refused)

    by_hand = [15, 40, -1], [[0] * 8 for _ in range(3)], 20
    step()
    for i in range(1, 4):
        want, l, t, c, _ = R.plan(by_hand[0], by_hand[1], list(range(20)), by_hand[2], None, 16, 3, 8)
        by_hand = l, t, c
        assert slots.tolist() == want and lens.tolist() == l and table.tolist() == t and count.item() == c
        if i == 1:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        graph.replay()


# ---- the cache's writing ------------------------------------------------------------------------

APPEND = [  # T, Hkv, d, page, e4m3
    (1, 1, 8, 16, False), (5, 2, 64, 16, False), (37, 3, 80, 48, True), (130, 8, 128, 64, True), (130, 8, 128, 64, False),
    (9, 40, 128, 16, False), (7, 33, 24, 32, True), (1000, 1, 32, 256, True),
]


@pytest.mark.parametrize("T,Hkv,d,page,e4m3", APPEND)
def test_append(gdn, T, Hkv, d, page, e4m3):
    g = gen(T)
    blocks = -(-T // page) + 2
    kv = rnd(g, T, 2 * Hkv * d + 16) * 3
    k, v = kv[:, 8:8 + Hkv * d].unflatten(1, (Hkv, d)), kv[:, 16 + Hkv * d:].unflatten(1, (Hkv, d))
    dtype = torch.float8_e4m3fn if e4m3 else BF
    caches = rnd(g, blocks, 2, Hkv, page, d).to(dtype)  # k and v of a block side by side
    before = caches.clone()
    slots = torch.randperm(blocks * page, generator=g)[:T].to(I32)
    slots[::7] = -1 - slots[::7]  # some are passed over
    if T > 20:
        slots[3], slots[4] = blocks * page, 2 ** 31 - 1
    scales = [torch.rand(Hkv, generator=g).cuda() / 50 + 0.01 for _ in range(2)] if e4m3 else [None, None]
    gdn.cache_append(k, v, caches[:, 0], caches[:, 1], slots.cuda(), *scales)
    want = n64(before.float())
    wrote = np.zeros((blocks, 2, Hkv, page, d), bool)
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < blocks * page:
            for i, (x, scale) in enumerate(((k, scales[0]), (v, scales[1]))):
                row = n64(x[t])
                if e4m3:
                    row = np.clip(row / n64(scale)[:, None], -448, 448)
                want[s // page, i, :, s % page] = row
                wrote[s // page, i, :, s % page] = True
    got = n64(caches.float())
    if e4m3:
        tol = np.where(wrote, np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10) + 2.0 ** -20 * np.abs(want), 0)
        assert np.all(np.abs(got - want) <= tol)
    else:
        assert np.array_equal(got, want)


def test_append_values_that_are_not_finite(gdn):
    k = torch.tensor([NAN, float("inf"), -float("inf"), 1e30, -500.0, 2.0 ** -9, 0.0, -0.0], dtype=BF, device="cuda")
    k = k.expand(1, 1, 8).contiguous()
    one = torch.ones(1, device="cuda")
    kc, vc = (torch.zeros(1, 1, 16, 8, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
    gdn.cache_append(k, k, kc, vc, ints([3]), one, one)
    assert str(kc[0, 0, 3].float().tolist()) == str([NAN, 448.0, -448.0, 448.0, -448.0, 2.0 ** -9, 0.0, -0.0])
    kc, vc = (torch.zeros(1, 1, 16, 8, dtype=BF, device="cuda") for _ in range(2))
    gdn.cache_append(k, k, kc, vc, ints([15]))
    assert torch.equal(kc[0, 0, 15].view(torch.int16), k[0, 0].view(torch.int16))


def test_append_offsets_past_32_bits(gdn):
    # blocks 2^30 elements apart: the last token's place starts past 2^31 elements
    g = gen(3)
    big = torch.zeros(3 * 2 ** 30 + 2 * 16 * 64, dtype=BF, device="cuda")
    kc = big.as_strided((4, 2, 16, 64), (2 ** 30, 16 * 64, 64, 1))
    vc = torch.zeros(4, 2, 16, 64, dtype=BF, device="cuda")
    k, v = rnd(g, 2, 2, 64), rnd(g, 2, 2, 64)
    gdn.cache_append(k, v, kc, vc, ints([63, 5]))
    for c, x in ((kc, k), (vc, v)):
        assert torch.equal(c[3, :, 15], x[0]) and torch.equal(c[0, :, 5], x[1])
    assert int((kc != 0).sum()) <= 256


# ---- one token over the cache -------------------------------------------------------------------

def cache_of(g, lens, Hkv, d, page, e4m3, fill=NAN, spare=2):
    """A cache that holds random tokens for these requests, `fill` elsewhere, in shuffled blocks; its tables, with
    entries that no call may follow behind the requests' blocks."""
    held = [max(0, -(-n // page)) for n in lens]
    blocks = sum(held) + spare
    order = torch.randperm(blocks, generator=g).tolist()
    W = max(held + [1]) + 1
    table = np.full((len(lens), W), 2 ** 30)
    caches = torch.full((blocks, 2, Hkv, page, d), fill)
    at = 0
    for b, m in enumerate(held):
        table[b, :m] = order[at:at + m]
        for i in range(m):
            n = min(page, lens[b] - i * page)
            caches[order[at + i], :, :, :n] = torch.randn((2, Hkv, n, d), generator=g)
        at += m
    scales = [None, None]
    if e4m3:
        scales = [torch.rand(Hkv, generator=g).cuda() / 100 + 0.01 for _ in range(2)]
        caches = (caches / torch.stack(scales).cpu()[None, :, :, None, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    else:
        caches = caches.to(BF)
    caches = caches.cuda()
    return caches[:, 0], caches[:, 1], scales, table


def check_step(gdn, q, kc, vc, scales, table, lens, window=0, sinks=0, scale=None, **kw):
    B, Hq, d = q.shape
    out, lse = gdn.attention_step(q, kc, vc, ints(table), ints(lens), *scales, window=window, sinks=sinks, scale=scale,
                                  want_lse=True, **kw)
    k64, v64 = n64(kc.float()), n64(vc.float())
    if scales[0] is not None:
        k64, v64 = (c * n64(s)[None, :, None, None] for c, s in ((k64, scales[0]), (v64, scales[1])))
    page = kc.shape[2]
    for b, n in enumerate(lens):
        n = max(0, n)
        blocks = table[b, :-(-n // page)]
        y, mag, l, bound = R.attend(n64(q[b:b + 1]), R.paged(k64, blocks, n), R.paged(v64, blocks, n),
                                    d ** -0.5 if scale is None else scale, window, sinks)
        close(out[b:b + 1], y, mag, bound)
        close_lse(lse[b:b + 1], l, bound)
    return out, lse


STEP = [  # lens, Hq, Hkv, d, page, window, sinks
    ([1], 1, 1, 8, 16, 0, 0), ([0], 4, 2, 64, 16, 0, 0), ([2, 15, 16, 17], 4, 2, 64, 16, 0, 0),
    ([31, 32, 33, 0, 63, 64, 65], 8, 1, 128, 32, 0, 0), ([127, 128, 129, -1, 255, 257], 8, 2, 128, 64, 0, 0),
    ([1000, 3], 12, 4, 80, 48, 0, 0), ([700], 20, 1, 96, 256, 0, 0), ([300, 1, 77], 33, 3, 32, 64, 0, 0),
    ([520, 40], 40, 1, 24, 16, 0, 0), ([513], 64, 2, 128, 16, 0, 0), ([2500, 900, 1], 6, 2, 112, 128, 0, 0),
    ([400, 100, 17, 1], 8, 2, 128, 16, 17, 0), ([400, 100, 17, 1], 8, 2, 128, 16, 16, 3), ([400, 130, 30], 4, 4, 64, 64, 1, 0),
    ([400, 130, 30], 4, 1, 64, 64, 1, 1), ([900, 200], 5, 1, 72, 32, 100, 150), ([900, 140], 8, 4, 128, 64, 128, 64),
    ([50], 2, 2, 40, 16, 4000, 9), ([300], 2, 1, 64, 16, 30, 4000),
]


@pytest.mark.parametrize("lens,Hq,Hkv,d,page,window,sinks", STEP)
@pytest.mark.parametrize("e4m3", [False, True])
def test_step(gdn, lens, Hq, Hkv, d, page, window, sinks, e4m3):
    g = gen(len(lens) + Hq + d)
    kc, vc, scales, table = cache_of(g, lens, Hkv, d, page, e4m3)
    wide = rnd(g, len(lens), Hq * d + 24)
    check_step(gdn, wide[:, 8:8 + Hq * d].unflatten(1, (Hq, d)), kc, vc, scales, table, lens, window, sinks)


@pytest.mark.parametrize("B,top,Hq,Hkv,d,page,window,e4m3", [
    (1, 9000, 8, 1, 128, 64, 0, False), (1, 9001, 32, 8, 128, 16, 0, True), (40, 1500, 32, 8, 128, 64, 0, False),
    (300, 200, 8, 2, 64, 16, 0, True), (17, 3000, 16, 2, 96, 128, 500, False), (3, 5000, 48, 1, 128, 32, 0, False)])
def test_step_split_over_the_device(gdn, B, top, Hq, Hkv, d, page, window, e4m3):
    g = gen(B + top)
    lens = torch.randint(top // 3, top, (B,), generator=g).tolist()
    kc, vc, scales, table = cache_of(g, lens, Hkv, d, page, e4m3)
    q = rnd(g, B, Hq, d) * 2
    out, lse = check_step(gdn, q, kc, vc, scales, table, lens, window, 4)
    for _ in range(3):  # the same sums in the same order, whatever finishes first
        again, lse2 = gdn.attention_step(q, kc, vc, ints(table), ints(lens), *scales, window=window, sinks=4, want_lse=True)
        assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("B,top,Hq,Hkv,d,e4m3", [(33, 300, 2, 1, 64, False), (1025, 60, 4, 2, 32, True), (3000, 40, 2, 1, 64, False),
                                                (5000, 2, 1, 1, 8, False)])
def test_step_many_requests(gdn, B, top, Hq, Hkv, d, e4m3):
    g = gen(B)
    lens = torch.randint(0, top, (B,), generator=g)
    lens[torch.randint(0, B, (B // 3,), generator=g)] = 0
    lens[B // 2:B // 2 + B // 20] = 0
    lens[B // 3] = 40 * top  # one long among them
    kc, vc, scales, table = cache_of(g, lens.tolist(), Hkv, d, 16, e4m3)
    check_step(gdn, rnd(g, B, Hq, d), kc, vc, scales, table, lens.tolist())


@pytest.mark.parametrize("given", [False, True])
def test_calls_of_many_sizes_one_after_another(gdn, given):
    # what one call leaves in a workspace is no other's concern
    g = gen(12)
    ws = torch.zeros(gdn.gdn_attn_workspace_bytes(400, 48, 6, 128), dtype=torch.uint8, device="cuda") if given else None
    for B, top, Hq, Hkv, d, e4m3 in ((1, 3000, 48, 6, 128, False), (400, 30, 2, 1, 64, True), (3, 900, 40, 1, 32, False),
                                     (1, 1, 1, 1, 8, True), (37, 700, 16, 4, 96, True), (1, 5000, 8, 8, 128, False)):
        lens = torch.randint(top // 2, top + 1, (B,), generator=g).tolist()
        kc, vc, scales, table = cache_of(g, lens, Hkv, d, 32, e4m3)
        check_step(gdn, rnd(g, B, Hq, d), kc, vc, scales, table, lens, workspace=ws)
        q, k, v = slices(g, top, top, Hq, Hkv, d) if top < 1000 else slices(g, 9, 9, Hq, Hkv, d)
        check_attn(gdn, q, k, v, [q.shape[0]], workspace=ws)
    assert gdn.gdn_device_status() == (0, 0)
    if given:
        assert int(ws[:4].view(I32)) == 0


@pytest.mark.parametrize("d", range(8, 129, 8))
def test_every_width(gdn, d):
    # each column alone: a query that is one at a column, keys that are there what no other column is
    for lens in ([3], [70]):
        n = lens[0]
        q = torch.eye(d).to(BF).cuda()[:, None]  # d queries of one head
        k = torch.zeros(n, 1, d)
        k[0, 0] = torch.arange(1, d + 1) / 8
        v = (torch.arange(n)[:, None, None] % 5 + torch.arange(d) % 3).float()
        k, v = k.to(BF).cuda(), v.to(BF).cuda()
        check_attn(gdn, q, k, v, [d], [n], scale=1.0)
        for e4m3 in (False, True):
            kc, vc = (torch.full((8, 1, 16, d), NAN) for _ in range(2))
            for i in range(0, n, 16):
                m = min(16, n - i)
                kc[i // 16, :, :m] = k[i:i + m].float().cpu().transpose(0, 1)
                vc[i // 16, :, :m] = v[i:i + m].float().cpu().transpose(0, 1)
            t = torch.float8_e4m3fn if e4m3 else BF
            scales = [torch.ones(1, device="cuda")] * 2 if e4m3 else [None, None]
            table = np.tile(np.arange(8), (d, 1))
            check_step(gdn, q, kc.to(t).cuda(), vc.to(t).cuda(), scales, table, [n] * d, scale=1.0)


@pytest.mark.parametrize("e4m3", [False, True])
def test_step_scales(gdn, e4m3):
    g = gen(4)
    kc, vc, scales, table = cache_of(g, [333], 2, 64, 32, e4m3)
    q = rnd(g, 1, 4, 64)
    for scale in (1.0, 0.0, -0.3, 20.0):
        check_step(gdn, q, kc, vc, scales, table, [333], scale=scale)
    check_step(gdn, (q.float() * 1e-18).to(BF), kc, vc, scales, table, [333], scale=1e18)
    check_step(gdn, (q.float() * 1e18).to(BF), kc, vc, scales, table, [333], scale=1e-18)


def test_step_sizes_of_scores(gdn):
    # scores that grow along the cache, that fall, and that are far from one another
    g = gen(8)
    for slope in (0.05, -0.05, 3.0, -3.0):
        kc, vc, scales, table = cache_of(g, [600], 1, 64, 16, False)
        for i, block in enumerate(table[0, :38]):
            for t in range(16):
                kc[int(block), 0, t, 0] = slope * (16 * i + t) / 8
        q = rnd(g, 1, 3, 64)
        q[:, :, 0] = 8.0
        check_step(gdn, q, kc, vc, scales, table, [600], scale=1.0)


def test_step_blocks_that_are_not_there(gdn):
    g = gen(5)
    kc, vc, scales, table = cache_of(g, [100, 200], 2, 64, 16, False, fill=0.0)
    q = rnd(g, 2, 4, 64)
    gdn.gdn_device_status()
    out, lse = gdn.attention_step(q, kc, vc, ints(table), ints([100, 200]), want_lse=True)
    assert gdn.gdn_device_status() == (0, 0)
    bad = table.copy()
    bad[0, 2], bad[1, 0], bad[1, 12] = -1, kc.shape[0], -2 ** 31  # (in the last, eight tokens)
    got, got_lse = gdn.attention_step(q, kc, vc, ints(bad), ints([100, 200]), want_lse=True)
    assert gdn.gdn_device_status() == (0, gdn.GDN_STATUS_BAD_PAGE)
    for b, gone in ((0, [2]), (1, [0, 12])):
        keep = np.concatenate([np.arange(16 * i, min(16 * i + 16, [100, 200][b])) for i in range(13) if i not in gone])
        keep = keep[keep < [100, 200][b]].astype(int)
        k, v = (R.paged(n64(c), table[b, :-(-[100, 200][b] // 16)], [100, 200][b])[keep] for c in (kc, vc))
        y, mag, l, bound = R.attend(n64(q[b:b + 1]), k, v, 0.125)
        close(got[b:b + 1], y, mag, bound)
        close_lse(got_lse[b:b + 1], l, bound)
    none = np.full_like(table, -1)
    got, got_lse = gdn.attention_step(q, kc, vc, ints(none), ints([100, 200]), want_lse=True)
    assert not bool(got.any()) and bool(torch.isneginf(got_lse).all())
    assert gdn.gdn_device_status() == (0, gdn.GDN_STATUS_BAD_PAGE)
    # a length past the table counts as its end
    got, _ = gdn.attention_step(q, kc, vc, ints(table[:, :3]), ints([2 ** 31 - 1, 48]))
    want, _ = gdn.attention_step(q, kc, vc, ints(table[:, :3]), ints([48, 48]))
    assert torch.equal(got, want)


@pytest.mark.parametrize("value", [NAN, float("inf")])
def test_step_values_that_are_not_finite_where_they_are_seen(gdn, value):
    g = gen(6)
    kc, vc, scales, table = cache_of(g, [40, 40], 2, 64, 16, False)
    vc[int(table[0, 1]), 1, 4, 7] = value
    q = rnd(g, 2, 4, 64)
    out, lse = gdn.attention_step(q, kc, vc, ints(table), ints([40, 40]), want_lse=True)
    bad = ~torch.isfinite(out)
    assert bool(bad[0, 2:, 7].all()) and int(bad.sum()) == 2 and bool(torch.isfinite(lse).all())
    if value != value:
        kc[int(table[1, 0]), 0, 0, 0] = value
        out, _ = gdn.attention_step(q, kc, vc, ints(table), ints([40, 40]))
        assert bool(out[1, :2].isnan().all()) and not bool(out[1, 2:].isnan().any())


def test_step_offsets_past_32_bits(gdn):
    g = gen(7)
    big = torch.empty(3 * 2 ** 30 + 2 * 16 * 64, dtype=BF, device="cuda")
    kc = big.as_strided((4, 2, 16, 64), (2 ** 30, 16 * 64, 64, 1))
    for i in range(4):
        kc[i] = rnd(g, 2, 16, 64)
    vc = rnd(g, 4, 2, 16, 64)
    check_step(gdn, rnd(g, 2, 4, 64), kc, vc, [None, None], np.array([[3, 2], [1, 3]]), [32, 30])


def test_step_captured_with_a_workspace(gdn):
    g = gen(9)
    kc, vc, scales, table = cache_of(g, [2000, 700], 2, 128, 16, False)
    q, lens, t = rnd(g, 2, 16, 128), ints([2000, 700]), ints(table)
    ws = torch.zeros(gdn.gdn_attn_workspace_bytes(2, 16, 2, 128), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(2, 16, device="cuda")

    def call(**kw):
        gdn.attention_step(q, kc, vc, t, lens, out=out, lse=lse, workspace=ws, **kw)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for a, b in ((1999, 700), (1, 0), (650, 333)):
        lens.copy_(ints([a, b]))
        q.copy_(rnd(g, 2, 16, 128))
        out.fill_(7)
        graph.replay()
        got, got_lse = out.clone(), lse.clone()
        want, want_lse = check_step(gdn, q, kc, vc, scales, table, [a, b])
        assert torch.equal(got, want) and torch.equal(got_lse, want_lse)
    assert int(ws[:4].view(I32)) == 0
    with pytest.raises(gdn.GdnError, match=str(gdn.GDN_ERR_SCRATCH)):
        gdn.attention_step(q, kc, vc, t, lens, workspace=ws[:128])


# ---- prompts -------------------------------------------------------------------------------------

def check_attn(gdn, q, k, v, lens, klens=None, window=0, sinks=0, scale=None, packed=True, **kw):
    T, Hq, d = q.shape
    klens = lens if klens is None else klens
    cu = cu_of(lens) if packed else None
    cuk = cu_of(klens) if packed and klens is not lens else None
    out, lse = gdn.attention(q, k, v, cu, cuk, B=None if packed else len(lens), window=window, sinks=sinks, scale=scale,
                             want_lse=True, **kw)
    a = b = 0
    q64, k64, v64 = n64(q), n64(k), n64(v)
    for n, m in zip(lens, klens):
        y, mag, l, bound = R.attend(q64[a:a + n], k64[b:b + m], v64[b:b + m], d ** -0.5 if scale is None else scale, window,
                                    sinks)
        if n:
            close(out[a:a + n], y, mag, bound)
            close_lse(lse[a:a + n], l, bound)
        a, b = a + n, b + m
    return out, lse


def slices(g, T, Tk, Hq, Hkv, d):
    wq, wkv = rnd(g, T, Hq * d + 16), rnd(g, Tk, 2 * Hkv * d + 8)
    return (wq[:, 8:8 + Hq * d].unflatten(1, (Hq, d)), wkv[:, :Hkv * d].unflatten(1, (Hkv, d)),
            wkv[:, 8 + Hkv * d:].unflatten(1, (Hkv, d)))


ATTN = [  # lens, Hq, Hkv, d, window, sinks
    ([1], 1, 1, 8, 0, 0), ([2], 2, 1, 64, 0, 0), ([64], 1, 1, 32, 0, 0), ([127], 4, 4, 128, 0, 0), ([128], 4, 2, 128, 0, 0),
    ([129], 4, 1, 128, 0, 0), ([5, 0, 130, 1, 0, 257], 8, 2, 128, 0, 0), ([300, 299], 5, 1, 80, 0, 0),
    ([513], 6, 2, 96, 0, 0), ([100, 28], 7, 1, 24, 0, 0), ([260], 16, 1, 64, 0, 0), ([70, 33], 64, 1, 128, 0, 0),
    ([40], 100, 1, 16, 0, 0), ([9, 200], 128, 1, 128, 0, 0), ([1000], 3, 3, 112, 0, 0), ([640, 1, 385], 2, 1, 128, 0, 0),
    ([300, 17, 1], 4, 2, 64, 1, 0), ([300, 17, 1], 4, 2, 64, 1, 1), ([500], 4, 2, 128, 16, 4), ([700, 90], 8, 1, 128, 128, 0),
    ([700, 90], 8, 2, 64, 127, 150), ([1100], 2, 1, 128, 129, 1), ([1100], 2, 2, 64, 500, 300), ([900], 3, 1, 40, 64, 128),
    ([200], 4, 1, 128, 4000, 3), ([260], 2, 1, 64, 20, 4000), ([1500], 1, 1, 128, 300, 130),
]


@pytest.mark.parametrize("lens,Hq,Hkv,d,window,sinks", ATTN)
def test_attention_packed(gdn, lens, Hq, Hkv, d, window, sinks):
    g = gen(sum(lens) + Hq + d)
    q, k, v = slices(g, sum(lens), sum(lens), Hq, Hkv, d)
    check_attn(gdn, q, k, v, lens, window=window, sinks=sinks)


@pytest.mark.parametrize("top,Hq,Hkv,d,window,sinks", [(80, 4, 1, 64, 0, 0), (40, 8, 2, 128, 0, 0), (150, 4, 2, 32, 20, 2),
                                                       (300, 2, 1, 96, 60, 3)])
def test_attention_many_sequences(gdn, top, Hq, Hkv, d, window, sinks):
    # many more items than CTAs, with tiles that see nothing in any order among them
    g = gen(top)
    lens = torch.randint(0, top, (1500,), generator=g)
    lens[torch.randint(0, 1500, (400,), generator=g)] = 1
    klens = torch.where(torch.rand(1500, generator=g) < 0.2, torch.randint(0, top, (1500,), generator=g), lens)
    q, k, v = slices(g, int(lens.sum()), int(klens.sum()), Hq, Hkv, d)
    check_attn(gdn, q, k, v, lens.tolist(), klens.tolist(), window=window, sinks=sinks)
    assert gdn.gdn_device_status() == (0, 0)


@pytest.mark.parametrize("B,T,Hq,Hkv,d,window,sinks", [
    (1, 1, 2, 1, 64, 0, 0), (3, 65, 4, 2, 128, 0, 0), (2, 400, 8, 2, 80, 0, 0), (4, 130, 3, 3, 32, 40, 2),
    (2, 1027, 8, 4, 128, 256, 4), (1, 3001, 8, 1, 128, 0, 0), (5, 2500, 8, 4, 64, 130, 4), (30, 100, 16, 8, 64, 0, 0)])
def test_attention_dense(gdn, B, T, Hq, Hkv, d, window, sinks):
    g = gen(B + T)
    q, k, v = slices(g, B * T, B * T, Hq, Hkv, d)
    check_attn(gdn, q, k, v, [T] * B, window=window, sinks=sinks, packed=False)


@pytest.mark.parametrize("lens,klens,Hq,Hkv,d,window,sinks", [
    ([1], [500], 8, 2, 128, 0, 0), ([100, 3], [300, 900], 4, 2, 64, 0, 0), ([130, 60, 0], [700, 60, 50], 8, 1, 128, 200, 5),
    ([50, 300], [20, 129], 4, 2, 128, 0, 0),   # fewer keys than queries: the first see none
    ([300, 7], [0, 10], 2, 1, 64, 0, 0), ([260, 300], [100, 40], 6, 2, 96, 16, 3), ([5, 5], [0, 0], 2, 2, 64, 0, 0)])
def test_attention_keys_of_their_own_length(gdn, lens, klens, Hq, Hkv, d, window, sinks):
    g = gen(sum(lens) + sum(klens))
    q, k, v = slices(g, sum(lens), sum(klens), Hq, Hkv, d)
    check_attn(gdn, q, k, v, lens, klens, window=window, sinks=sinks)


def test_attention_dense_keys_of_their_own_length(gdn):
    g = gen(11)
    for T, Tk in ((40, 170), (170, 40), (3, 0)):
        q, k, v = slices(g, 2 * T, 2 * Tk, 4, 2, 64)
        check_attn(gdn, q, k, v, [T] * 2, [Tk] * 2, packed=False)


def test_attention_scales(gdn):
    g = gen(12)
    q, k, v = slices(g, 300, 300, 4, 2, 64)
    for scale in (1.0, 0.0, -0.3, 10.0):
        check_attn(gdn, q, k, v, [300], scale=scale)
    q, k, v = slices(g, 200, 200, 2, 1, 128)
    for a in (1e-18, 1e18):
        check_attn(gdn, (q.float() * a).to(BF), k, v, [200], scale=1 / a)


@pytest.mark.parametrize("slope", [0.05, -0.05, 3.0, -3.0, 40.0])
def test_attention_sizes_of_scores(gdn, slope):
    g = gen(13)
    q, k, v = (rnd(g, 600, h, 64) for h in (2, 1, 1))
    k[:, :, 0] = (slope * torch.arange(600, device="cuda")[:, None] / 8).to(BF)
    q[:, :, 0] = 8.0
    check_attn(gdn, q, k, v, [600], scale=1.0)
    check_attn(gdn, q, k, v, [600], scale=1.0, window=150, sinks=7)


def test_attention_rows_behind_the_last_sequence(gdn):
    g = gen(14)
    q, k, v = slices(g, 400, 400, 4, 2, 128)
    out, lse = torch.full((400, 4, 128), 7.0, dtype=BF, device="cuda"), torch.full((400, 4), 7.0, device="cuda")
    q[301:], k[301:], v[301:] = NAN, NAN, NAN
    gdn.attention(q, k, v, cu_of([100, 201]), out=out, lse=lse)
    assert bool((out[301:] == 7).all()) and bool((lse[301:] == 7).all())
    # (rows beside values that are not finite are worked out apart, with other roundings: both within the tolerance)
    for a, b in ((0, 100), (100, 301)):
        y, mag, l, bound = R.attend(n64(q[a:b]), n64(k[a:b]), n64(v[a:b]), 128 ** -0.5)
        close(out[a:b], y, mag, bound)
        close_lse(lse[a:b], l, bound)


@pytest.mark.parametrize("value", [NAN, float("inf"), -float("inf")])
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 5)])
def test_attention_unseen_values_change_nothing(gdn, value, window, sinks):
    g = gen(15)
    lens = [200, 90, 300]
    q, k, v = (rnd(g, 590, h, 64) for h in (4, 2, 2))
    want, want_lse = check_attn(gdn, q, k, v, lens, window=window, sinks=sinks)
    k[200:290], v[200:290] = value, value  # a whole sequence
    k[290 + 150, 1], v[290 + 150, 0] = value, value  # a token of a head
    out, lse = gdn.attention(q, k, v, cu_of(lens), window=window, sinks=sinks, want_lse=True)
    tol = 2.0 ** -7 * want.abs().float() + 2.0 ** -8
    for sl in (slice(0, 200), slice(290, 290 + 150)):
        assert bool(((out[sl].float() - want[sl].float()).abs() <= tol[sl]).all())
        assert bool(((lse[sl] - want_lse[sl]).abs() < 1e-4).all())
    if value != value:
        seen = slice(290 + 150, 290 + (220 if window else 300))
        assert bool(out[seen].isnan().all())  # heads 0, 1 by their values, 2, 3 by their scores
        assert bool(lse[seen, 2:].isnan().all()) and bool(((lse[seen, :2] - want_lse[seen, :2]).abs() < 1e-4).all())
        if window:
            assert bool(((out[510:].float() - want[510:].float()).abs() <= tol[510:]).all())


def test_attention_one_value_that_is_not_finite(gdn):
    # an infinity in one column reaches that column of the queries that see it, and nothing else
    g = gen(16)
    q, k, v = (rnd(g, 500, h, 128) for h in (2, 1, 1))
    want, _ = gdn.attention(q, k, v)
    v[260, 0, 77] = float("inf")
    out, _ = gdn.attention(q, k, v)
    assert bool(torch.isposinf(out[260:, :, 77]).all())
    keep = torch.ones_like(out, dtype=torch.bool)
    keep[260:, :, 77] = False
    tol = 2.0 ** -7 * want.abs().float() + 2.0 ** -8
    assert bool(((out.float() - want.float()).abs() <= tol)[keep].all())


@pytest.mark.parametrize("bad", [[0, 9, 4, 16], [3, 5, 8, 12], [0, 5, 400, 16], [-7, 5, 8, 16], [0, 2000, 5, 16]])
def test_attention_malformed_boundaries_stay_in_bounds(gdn, bad):
    g = gen(17)
    q, k, v = slices(g, 16, 16, 4, 2, 64)
    buf, lbuf = torch.full((64, 4, 64), 7.0, dtype=BF, device="cuda"), torch.full((64, 4), 7.0, device="cuda")
    gdn.attention(q, k, v, ints(bad), out=buf[24:40], lse=lbuf[24:40])
    gdn.attention(q, k, v, cu_of([4, 6, 6]), ints(bad), out=buf[24:40], lse=lbuf[24:40])
    assert bool((buf[:24] == 7).all()) and bool((buf[40:] == 7).all())
    assert bool((lbuf[:24] == 7).all()) and bool((lbuf[40:] == 7).all())


def test_attention_offsets_past_32_bits(gdn):
    # tokens 2^28 elements apart: the last one starts past 2^31 elements
    g = gen(18)
    big = torch.empty(9 * 2 ** 28 + 256, dtype=BF, device="cuda")
    k = big.as_strided((10, 2, 64), (2 ** 28, 64, 1))
    k.copy_(rnd(g, 10, 2, 64))
    check_attn(gdn, rnd(g, 10, 4, 64), k, rnd(g, 10, 2, 64), [4, 6])
    q = big.as_strided((10, 4, 64), (2 ** 28, 64, 1))
    q.copy_(rnd(g, 10, 4, 64))
    check_attn(gdn, q, rnd(g, 10, 2, 64), rnd(g, 10, 2, 64), [4, 6])


def test_attention_is_the_same_every_time_and_captured(gdn):
    g = gen(19)
    q, k, v = (rnd(g, 900, h, 128) for h in (8, 2, 2))
    cu = cu_of([500, 400])
    out, lse = gdn.attention(q, k, v, cu, window=200, sinks=3, want_lse=True)
    ws = torch.zeros(gdn.gdn_attn_workspace_bytes(2, 8, 2, 128), dtype=torch.uint8, device="cuda")
    got, got_lse = torch.empty_like(out), torch.empty_like(lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gdn.attention(q, k, v, cu, window=200, sinks=3, out=got, lse=got_lse, workspace=ws)
    side.synchronize()
    assert torch.equal(out, got) and torch.equal(lse, got_lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.attention(q, k, v, cu, window=200, sinks=3, out=got, lse=got_lse, workspace=ws)
    q.copy_(rnd(g, 900, 8, 128))
    cu.copy_(cu_of([333, 567]))
    graph.replay()
    want, want_lse = check_attn(gdn, q, k, v, [333, 567], window=200, sinks=3)
    assert torch.equal(got, want) and torch.equal(got_lse, want_lse)
    assert int(ws[:4].view(I32)) == 0


# ---- a run of them together ------------------------------------------------------------------------

@pytest.mark.parametrize("e4m3,window,sinks", [(False, 0, 0), (False, 50, 2), (True, 0, 0), (True, 64, 4)])
def test_prompts_and_then_tokens(gdn, e4m3, window, sinks):
    """Prompts planned, written and attended to, then continued token by token over the cache."""
    g = gen(20)
    Hq, Hkv, d, page, steps = 8, 2, 64, 16, 20
    lens = [70, 1, 129, 40]
    B, total = len(lens), [n + steps for n in lens]
    qkv = [rnd(g, n, (Hq + 2 * Hkv) * d) for n in total]

    def split(x):
        return (x[:, :Hq * d].unflatten(1, (Hq, d)), x[:, Hq * d:(Hq + Hkv) * d].unflatten(1, (Hkv, d)),
                x[:, (Hq + Hkv) * d:].unflatten(1, (Hkv, d)))

    blocks = sum(-(-n // page) for n in total) + 1
    kc, vc = (torch.full((blocks, Hkv, page, d), NAN).to(torch.float8_e4m3fn if e4m3 else BF).cuda() for _ in range(2))
    scales = [torch.full((Hkv,), 0.02, device="cuda") for _ in range(2)] if e4m3 else [None, None]
    held, table = ints([0] * B), torch.full((B, -(-max(total) // page)), -1, dtype=I32, device="cuda")
    stack, count = torch.randperm(blocks, generator=g).to(I32).cuda(), ints([blocks])
    cu = cu_of(lens)
    q, k, v = split(torch.cat([x[:n] for x, n in zip(qkv, lens)]))
    slots, held, count, refused = gdn.cache_plan(held, table, stack, count, cu, page=page, T=sum(lens))
    gdn.cache_append(k, v, kc, vc, slots, *scales)
    out, _ = gdn.attention(q, k, v, cu, window=window, sinks=sinks)
    assert refused.item() == 0 and held.tolist() == lens
    got = [[out[a:a + n]] for a, n in zip(np.cumsum([0] + lens).tolist(), lens)]
    for i in range(steps):
        q, k, v = split(torch.stack([x[n + i] for x, n in zip(qkv, lens)]))
        slots, _, _, _ = gdn.cache_plan(held, table, stack, count, page=page, new_lens=held, new_count=count)
        gdn.cache_append(k, v, kc, vc, slots, *scales)
        out, _ = gdn.attention_step(q, kc, vc, table, held, *scales, window=window, sinks=sinks)
        for b in range(B):
            got[b].append(out[b:b + 1])
    assert held.tolist() == total and count.item() == 1
    for b, x in enumerate(qkv):
        q, k, v = (n64(t) for t in split(x))
        y, mag, _, bound = R.attend(q, k, v, d ** -0.5, window, sinks)
        o = torch.cat(got[b])
        close(o[:lens[b]], y[:lens[b]], mag[:lens[b]], bound[:lens[b]])
        if e4m3:  # the tokens read what the cache holds
            k, v = (n64((torch.tensor(t) / 0.02).clamp(-448, 448).to(torch.float8_e4m3fn).float()) * n64(scales[0][0])
                    for t in (k, v))
            y, mag, _, bound = R.attend(q, k, v, d ** -0.5, window, sinks)
        close(o[lens[b]:], y[lens[b]:], mag[lens[b]:], bound[lens[b]:])


def test_streams_and_devices_memory(gdn):
    """Calls on a stream of their own, in order there, without the current stream's help."""
    g = gen(21)
    q, k, v = (rnd(g, 600, h, 64) for h in (4, 2, 2))
    want, _ = gdn.attention(q, k, v)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out, _ = gdn.attention(q, k, v, stream=s)
    raw, _ = gdn.attention(q, k, v, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(out, want) and torch.equal(raw, want)
    kc, vc, scales, table = cache_of(g, [600], 2, 64, 16, False)
    q1 = rnd(g, 1, 4, 64)
    torch.cuda.synchronize()
    a, _ = gdn.attention_step(q1, kc, vc, ints(table), ints([600]))
    torch.cuda.synchronize()
    t, n = ints(table), ints([600])
    torch.cuda.synchronize()
    b, _ = gdn.attention_step(q1, kc, vc, t, n, stream=s)
    s.synchronize()
    assert torch.equal(a, b)


def captured(call):
    """A graph of the call, which has run before on the stream that it is captured from."""
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    return graph


def step_case(gdn, g, lens, Hq, Hkv, d, e4m3, ws):
    kc, vc, scales, table = cache_of(g, lens, Hkv, d, 32, e4m3)
    wide = torch.full((len(lens), table.shape[1] + 3), -5, dtype=I32, device="cuda")
    wide[:, 1:-2] = ints(table)
    q, out = rnd(g, len(lens), Hq, d), torch.empty(len(lens), Hq, d, dtype=BF, device="cuda")
    lse = torch.empty(len(lens), Hq, device="cuda")
    want = check_step(gdn, q, kc, vc, scales, table, lens)
    args = (q, kc, vc, wide[:, 1:-2], ints(lens), *scales)
    return (lambda: gdn.attention_step(*args, out=out, lse=lse, workspace=ws)), out, lse, want


def test_step_two_graphs_with_one_workspace(gdn):
    g = gen(31)
    ws = torch.zeros(gdn.gdn_attn_workspace_bytes(50, 16, 2, 128), dtype=torch.uint8, device="cuda")
    cases = [step_case(gdn, g, lens, Hq, Hkv, d, e4m3, ws) for lens, Hq, Hkv, d, e4m3 in (
        ([3000, 17], 16, 2, 128, False), ([900] * 50, 4, 2, 64, True))]
    graphs = [captured(c[0]) for c in cases]
    for i in (0, 1, 1, 0, 0, 1, 0):
        call, out, lse, want = cases[i]
        out.fill_(7)
        graphs[i].replay()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_step_two_streams_at_once(gdn):
    g = gen(32)
    size = gdn.gdn_attn_workspace_bytes(40, 8, 2, 128)
    cases = [step_case(gdn, g, lens, 8, 2, 128, e4m3, torch.zeros(size, dtype=torch.uint8, device="cuda"))
             for lens, e4m3 in (([4000, 5], False), ([700] * 40, True))]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(30):
        for s, (call, out, _, _) in zip(streams, cases):
            with torch.cuda.stream(s):
                out.fill_(7)
                call()
    torch.cuda.synchronize()
    for _, out, lse, want in cases:
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_captured_server_step(gdn):
    """Plan, writing and attention of a token as one graph, replayed with new tokens; the same as call by call."""
    g = gen(33)
    B, Hq, Hkv, d, page, steps = 5, 8, 2, 64, 16, 40
    lens = [0, 15, 33, 100, -1]
    blocks = 30
    results = []
    tokens = [rnd(g, B, Hq + 2 * Hkv, d) for _ in range(steps)]
    past = rnd(g, blocks, 2, Hkv, page, d)
    for graphed in (False, True):
        cache = past.clone()
        held, count = ints(lens), ints([blocks - 20])
        table = torch.full((B, 12), -1, dtype=I32, device="cuda")
        for b, n in enumerate(lens):
            m = max(0, -(-n // page))
            table[b, :m] = torch.arange(blocks - 20 + 3 * b, blocks - 20 + 3 * b + m, dtype=I32, device="cuda")
        stack = torch.arange(blocks - 20, dtype=I32, device="cuda")
        x = torch.empty_like(tokens[0])
        slots, refused = ints([0] * B), ints([0])
        out = torch.empty(B, Hq, d, dtype=BF, device="cuda")
        ws = torch.zeros(gdn.gdn_attn_workspace_bytes(B, Hq, Hkv, d), dtype=torch.uint8, device="cuda")

        def step():
            gdn.cache_plan(held, table, stack, count, page=page, slots=slots, new_lens=held, new_count=count,
                           refused=refused)
            gdn.cache_append(x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], cache[:, 0], cache[:, 1], slots)
            gdn.attention_step(x[:, :Hq], cache[:, 0], cache[:, 1], table, held, window=30, sinks=2, out=out, workspace=ws)

        x.copy_(tokens[0])
        step()
        got = [out.clone()]
        graph = torch.cuda.CUDAGraph()
        if graphed:
            with torch.cuda.graph(graph):
                step()
        for t in tokens[1:]:
            x.copy_(t)
            graph.replay() if graphed else step()
            got.append(out.clone())
        results.append((torch.stack(got), held.clone(), count.clone(), refused.clone(), cache))
    for a, b in zip(*results):
        assert torch.equal(a, b)
    assert results[0][1].tolist()[4] == -1
