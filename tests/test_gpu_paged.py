"""The paged cache: page plans and cache writes (whole numbers and copies: exact) and the attention of
one new token, against its formula in 64 bits; and a run of the three together.

Attention's tolerance. u = 2^-24. A score s_t = scale q.k_t is off by at most E_t = (d + 4) u scale
|q|.|k_t|, so a weight exp(s_t - m) is off by a factor within (1 +- (E_t + E_m + 4 u)) up to second
order, E_m <= max E; a weight's maximum shift is rescaled once per tile. The weighted sums add at most
n = L + 64 roundings on top. With p the softmax, |o - o*| <= (4 max_t E_t + (2 n + 16) u) sum_t p_t |v_t|.
Independent roundings add in quadrature: the 2-norm is within (4 max E + 8 sqrt(2 n + 16) u) of the
magnitudes' norm.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
KINDS = [torch.float32, torch.bfloat16]


@pytest.fixture(scope="module")
def stq():
    import quantized_linear_attention_stq_b200 as m

    m.lib()
    return m


# ---------------------------------------------------------------------------------------------
# plan
# ---------------------------------------------------------------------------------------------
def plan_ref(table, lens, fresh, free, head, N, page):
    """The plan's definition, request by request."""
    table, lens_out, smap, starts, bad = [list(r) for r in table], list(lens), [-1] * N, [], False
    B, W, tok, pages, most = len(lens), len(table[0]) if table else 0, 0, 0, 0
    for b in range(B):
        starts.append(min(tok, N))
        add = max(fresh[b], 0)
        ok = lens[b] >= 0 and fresh[b] >= 0 and lens[b] + fresh[b] <= W * page
        now, then = -(-lens[b] // page), -(-(lens[b] + fresh[b]) // page)
        need = then - now if ok else 0
        fits = ok and (need == 0 or pages + need <= len(free) - head) and tok + add <= N
        if fits:
            for i in range(need):
                table[b][now + i] = free[head + pages + i]
            if need:
                most = pages + need
            lens_out[b] = lens[b] + add
            for t in range(add):
                pos = lens[b] + t
                slot = table[b][pos // page] * page + pos % page
                smap[tok + t] = slot if table[b][pos // page] >= 0 else -1
                bad |= smap[tok + t] < 0
        else:
            bad = True
        pages += need
        tok += add
    starts.append(min(tok, N))
    return table, lens_out, smap, starts, head + most, bad


def run_plan(stq, table, lens, fresh, free, head, N, page, inplace=False):
    t = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    B = len(lens)
    tt = t(table) if B else torch.zeros(0, 3, dtype=torch.int32, device=DEV)
    ll, hh = t(lens), t([head])
    lo, ho = (ll, hh) if inplace else (t([-9] * B), t([-9]))
    smap, starts, status = t([-7] * N), t([-7] * (B + 1)), t([0])
    stq.page_plan(tt, ll, t(fresh), t(free), hh, smap, starts, lo, ho, page, status=status)
    return tt.tolist(), lo.tolist(), smap.tolist(), starts.tolist(), ho.item(), status.item()


def check_plan(stq, table, lens, fresh, free, head, N, page):
    want = plan_ref(table, lens, fresh, free, head, N, page)
    for inplace in (False, True):
        got = run_plan(stq, table, lens, fresh, free, head, N, page, inplace)
        for name, g, w in zip(("table", "lens", "slot map", "starts", "head"), got, want):
            assert g == w, name
        assert got[5] == ((1 << 6) if want[5] else 0)


def plan_case(B, page, longest, new, seed, spare=4):
    g = torch.Generator().manual_seed(seed)
    r = lambda n: torch.randint(0, n + 1, (B,), generator=g).tolist()  # noqa: E731
    lens, fresh = r(longest), r(new)
    W = -(-(longest + new) // page) + 1
    held = [-(-n // page) for n in lens]
    need = [-(-(a + b) // page) - h for a, b, h in zip(lens, fresh, held)]
    ids = torch.randperm(sum(held) + sum(need) + spare, generator=g).tolist()
    table, at = [], 0
    for h in held:
        table.append(ids[at:at + h] + [-1] * (W - h))
        at += h
    return table, lens, fresh, ids[at:]


@pytest.mark.parametrize("B,page,longest,new", [(1, 16, 0, 1), (1, 1, 5, 3), (70, 16, 500, 1), (7, 20, 100, 90),
                                                (1023, 16, 40, 1), (1025, 64, 30, 3), (2500, 8, 20, 2), (40, 64, 100, 900),
                                                (33, 1, 9, 700)])
def test_plan(stq, B, page, longest, new):
    table, lens, fresh, free = plan_case(B, page, longest, new, B + page)
    check_plan(stq, table, lens, fresh, free, 0, sum(fresh), page)
    check_plan(stq, table, lens, fresh, [99999] * 3 + free, 3, sum(fresh) + 5, page)  # taken pages, a padded map


def test_plan_large_map(stq):
    """More new tokens than one block writes."""
    table, lens, fresh, free = plan_case(300, 16, 50, 400, 2)
    assert sum(fresh) > 40000
    check_plan(stq, table, lens, fresh, free, 0, sum(fresh) + 100, 16)
    check_plan(stq, table, lens, fresh, free, 0, sum(fresh) - 12345, 16)
    check_plan(stq, table, lens, fresh, free[: len(free) // 2], 0, sum(fresh), 16)


def test_plan_edges(stq):
    # no requests: only the ends are written
    assert run_plan(stq, [], [], [], [5, 6], 1, 3, 16) == ([], [], [-1] * 3, [0], 1, 0)
    # nothing new, an empty free list, an empty slot map
    assert run_plan(stq, [[3]], [16], [0], [], 0, 0, 16) == ([[3]], [16], [], [0, 0], 0, 0)
    # a request of nothing but new tokens between two that get none
    check_plan(stq, [[-1] * 3] * 3, [0, 0, 0], [0, 33, 0], [4, 2, 9], 0, 40, 16)


def test_plan_refuses_requests(stq):
    T = [[1, 2, -1], [3, -1, -1], [-1, -1, -1], [4, 5, 6]]
    for lens, fresh, free, head, N in (
            ([20, 10, 0, 40], [5, 20, 40, 1], [7, 8], 0, 100),        # the list runs out at the third
            ([20, 10, 0, 48], [5, 20, 40, 1], list(range(10, 30)), 0, 100),  # the last has no room in its row
            ([20, 10, 0, 40], [5, -2, 40, 1], list(range(10, 30)), 0, 100),  # a negative count
            ([20, -1, 0, 40], [5, 2, 40, 1], list(range(10, 30)), 0, 100),   # a negative length
            ([20, 10, 0, 40], [5, 20, 40, 1], list(range(10, 30)), 0, 30),   # the map ends inside the third
            ([20, 10, 0, 40], [5, 20, 40, 1], [7, 8, 9], 3, 100),     # nothing left: those who need none are served
            ([2000000000, 10, 0, 40], [2000000000, 20, 40, 1], list(range(10, 30)), 0, 100)):
        check_plan(stq, T, lens, fresh, free, head, N, 16)
    # a list head outside the list: no page is handed out, and the head stays
    for head in (-1, 4):
        got = run_plan(stq, T, [20, 10, 0, 40], [5, 2, 3, 1], [7, 8, 9], head, 20, 16)
        assert got[0] == T and got[1] == [25, 12, 0, 41] and got[4] == head and got[5] == 1 << 6
    # a page that cannot be: its tokens get no slot
    got = run_plan(stq, [[-5]], [3], [2], [7], 0, 2, 16)
    assert got[2] == [-1, -1] and got[5] == 1 << 6
    got = run_plan(stq, [[1 << 30]], [3], [2], [7], 0, 2, 16)
    assert got[2] == [-1, -1] and got[5] == 1 << 6


# ---------------------------------------------------------------------------------------------
# write
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("N,H,d,page", [(1, 1, 16, 1), (5, 3, 32, 20), (70, 8, 128, 16), (301, 2, 64, 64), (1000, 1, 16, 3),
                                        (5000, 8, 128, 64)])
def test_write(stq, N, H, d, page, kind):
    g = torch.Generator(device=DEV).manual_seed(N)
    n = -(-N // page) + 2
    rows = torch.randn(N, 2 * H * d + 32, generator=g, device=DEV).to(kind)
    k, v = rows[:, :H * d].unflatten(1, (H, d)), rows[:, H * d:2 * H * d].unflatten(1, (H, d))
    kp, vp = (torch.randn(n, H, page, d, generator=g, device=DEV).to(kind) for _ in range(2))
    slots = torch.randperm(n * page, generator=g, device=DEV)[:N].to(torch.int32)
    slots[::7] = -1
    want = [kp.clone(), vp.clone()]
    live = slots >= 0
    at = slots[live].long()
    for w, x in zip(want, (k, v)):
        w[at // page, :, at % page] = x[live]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    stq.page_write(kp, vp, slots, k, v, status=status)
    assert status.item() == 0
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])
    # dense rows, and slots outside the pages
    slots[0], slots[-1] = n * page, -2
    stq.page_write(kp, vp, slots, k.contiguous(), v.contiguous(), status=status)
    assert status.item() == 1 << 6
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])


# ---------------------------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------------------------
def cache(lens, Hkv, d, page, kind, seed, spare=3, gap=-1):
    """Pages in random order, a table whose entries behind a request's pages are `gap`, NaN in every row
    that no token holds."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    held = [-(-n // page) for n in lens]
    total = sum(held) + spare
    ids = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    W = max(held) + 2
    table = torch.full((len(lens), W), gap, dtype=torch.int32, device=DEV)
    kp, vp = (torch.full((total, Hkv, page, d), float("nan"), dtype=kind, device=DEV) for _ in range(2))
    at = 0
    for b, (n, h) in enumerate(zip(lens, held)):
        table[b, :h] = ids[at:at + h]
        for i in range(h):
            rows = min(page, n - i * page)
            for pages in (kp, vp):
                pages[ids[at + i], :, :rows] = torch.randn(Hkv, rows, d, generator=g, device=DEV).to(kind)
        at += h
    return kp, vp, table


def attend_ref(q, kp, vp, table, lens, scale):
    """(o, tolerance's magnitudes sum p|v|, max_t E_t) in 64 bits."""
    B, Hq, d = q.shape
    _, Hkv, page, _ = kp.shape
    G = Hq // Hkv
    o, mag = (torch.zeros(B, Hq, d, dtype=torch.float64, device=DEV) for _ in range(2))
    E = torch.zeros(B, Hq, 1, dtype=torch.float64, device=DEV)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        at = table[b, : -(-n // page)].long()
        k, v = (x[at].transpose(0, 1).reshape(Hkv, -1, d)[:, :n].double() for x in (kp, vp))
        qq = q[b].double().view(Hkv, G, d)
        s = abs(scale) * (qq.abs() @ k.abs().transpose(1, 2))
        p = torch.softmax(scale * (qq @ k.transpose(1, 2)), dim=-1)
        o[b] = (p @ v).reshape(Hq, d)
        mag[b] = (p @ v.abs()).reshape(Hq, d)
        E[b] = ((d + 4) * U * s.amax(dim=-1)).reshape(Hq, 1)
    return o, mag, E


def check_attend(stq, lens, Hq, Hkv, d, page, kind, seed=0, scale=None, ws=(True, False), size=1.0):
    kp, vp, table = cache(lens, Hkv, d, page, kind, seed)
    g = torch.Generator(device=DEV).manual_seed(seed + 1)
    q = (size * torch.randn(len(lens), Hq, d, generator=g, device=DEV)).to(kind)
    scale = d ** -0.5 if scale is None else scale
    want, mag, E = attend_ref(q, kp, vp, table, lens, scale)
    tl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    n = max(lens) + 64
    for use in ws:
        o = torch.full((len(lens), Hq, d), 7.0, device=DEV)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        work = torch.full((stq.paged_attention_workspace_bytes(len(lens), Hq, d, Hkv),), 0xFF, dtype=torch.uint8,
                          device=DEV) if use else None
        stq.paged_attention(q, kp, vp, table, tl, o, scale, workspace=work, status=status)
        assert status.item() == 0, stq.status_flags(status)
        err = (o.double() - want).abs()
        allowed = (4 * E + (2 * n + 16) * U) * mag
        assert torch.all(err <= allowed + 1e-37), (err / (allowed + 1e-37)).max().item()
        most = (4 * E.max() + 8 * math.sqrt(2 * n + 16) * U) * mag.norm()
        assert err.norm() <= most + 1e-30, (err.norm() / most).item()
    return q, kp, vp, table, tl


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (8, 2), (10, 2), (16, 2), (16, 1), (20, 1), (34, 2)])
def test_attend_heads(stq, Hq, Hkv, d, kind):
    check_attend(stq, [200, 1, 67], Hq, Hkv, d, 16, kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page", [1, 3, 8, 16, 20, 64, 100, 256])
def test_attend_pages(stq, page, kind):
    check_attend(stq, [300, 64, 63, 65, 16, 17], 4, 2, 64, page, kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lens", [[1], [2], [15], [16], [17], [127], [128], [129], [4097], [0, 5], [0, 0, 3, 0], [0],
                                  [1] * 50, [5000] + [1] * 20, [700, 0, 3, 9000, 128, 64, 0]])
def test_attend_lengths(stq, lens, kind):
    check_attend(stq, lens, 8, 2, 128, 16, kind)


@pytest.mark.parametrize("kind", KINDS)
def test_attend_many_requests(stq, kind):
    g = torch.Generator().manual_seed(6)
    check_attend(stq, torch.randint(0, 400, (300,), generator=g).tolist(), 4, 1, 32, 16, kind)


@pytest.mark.parametrize("kind", KINDS)
def test_attend_long(stq, kind):
    check_attend(stq, [100003, 20001], 8, 2, 64, 64, kind, ws=(True,))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("scale,size", [(0.0, 1.0), (-0.3, 1.0), (1.0, 8.0), (1e-3, 1.0)])
def test_attend_scales(stq, scale, size, kind):
    """Scores that are all equal, negated, and so spread that one token takes all the weight."""
    check_attend(stq, [300, 40], 4, 2, 64, 16, kind, scale=scale, size=size)


@pytest.mark.parametrize("kind", KINDS)
def test_attend_infinities(stq, kind):
    """-inf scores drop their tokens; a row with nothing else is zero; NaN and +inf are flagged."""
    q, kp, vp, table, lens = check_attend(stq, [100, 100], 2, 2, 64, 16, kind)
    q[:, :, 0] = 1.0
    ws = torch.empty(stq.paged_attention_workspace_bytes(2, 2, 64, 2), dtype=torch.uint8, device=DEV)
    k2 = kp.clone()
    for t in range(20, 100):  # request 0: only the first 20 tokens count
        k2[table[0, t // 16].item(), :, t % 16, 0] = float("-inf")
    for t in range(100):      # request 1, head 1: none does
        k2[table[1, t // 16].item(), 1, t % 16, 0] = float("-inf")
    want = attend_ref(q, k2, vp, table, [20, 100], 0.125)[0]
    want[1, 1] = 0
    for work in (ws, None):
        o, status = torch.empty(2, 2, 64, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
        stq.paged_attention(q, k2, vp, table, lens, o, 0.125, workspace=work, status=status)
        assert status.item() == 0
        assert (o.double() - want).abs().max() < 1e-4  # a dropped or kept token moves o by about 1/100
        assert torch.all(o[1, 1] == 0)
    for value in (float("nan"), float("inf")):
        k3 = kp.clone()
        k3[table[0, 2].item(), 0, 3, 0] = value
        status.zero_()
        stq.paged_attention(q, k3, vp, table, lens, o, 0.125, workspace=ws, status=status)
        assert status.item() == 1 << 4
        assert torch.isnan(o[0, 0]).all() and torch.isfinite(o[0, 1]).all() and torch.isfinite(o[1]).all()


@pytest.mark.parametrize("kind", KINDS)
def test_attend_bad_pages_and_lengths(stq, kind):
    q, kp, vp, table, lens = check_attend(stq, [100, 90, 50], 4, 2, 64, 16, kind)
    kp, vp = torch.nan_to_num(kp), torch.nan_to_num(vp)
    bad = table.clone()
    bad[0, 2], bad[1, 0] = -3, kp.shape[0]
    ws = torch.empty(stq.paged_attention_workspace_bytes(3, 4, 64, 2), dtype=torch.uint8, device=DEV)
    want, mag, E = attend_ref(q, kp, vp, table, [100, 90, 50], 0.125)
    for work in (ws, None):
        o, status = torch.empty(3, 4, 64, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
        stq.paged_attention(q, kp, vp, bad, lens, o, 0.125, workspace=work, status=status)
        assert status.item() == 1 << 6
        # the same requests without the tokens of those pages
        k2, v2 = kp[table[0].clamp(min=0).long()], vp[table[0].clamp(min=0).long()]
        keep = [0, 1, 3, 4, 5, 6]
        t2 = torch.tensor([keep], dtype=torch.int32, device=DEV)
        w2, m2, E2 = attend_ref(q[:1], k2, v2, t2, [84], 0.125)
        assert torch.all((o[:1].double() - w2).abs() <= (4 * E2 + 400 * U) * m2)
        assert torch.all((o[2].double() - want[2]).abs() <= (4 * E[2] + 400 * U) * mag[2])
        l2 = torch.tensor([100, -1, table.shape[1] * 16 + 1], dtype=torch.int32, device=DEV)
        status.zero_()
        stq.paged_attention(q, kp, vp, table, l2, o, 0.125, workspace=work, status=status)
        assert status.item() == 1 << 6
        assert torch.all(o[1:] == 0)
        assert torch.all((o[0].double() - want[0]).abs() <= (4 * E[0] + 400 * U) * mag[0])


@pytest.mark.parametrize("kind", KINDS)
def test_attend_without_a_table(stq, kind):
    """A table of no columns: every request is empty."""
    q = torch.randn(2, 4, 64, device=DEV).to(kind)
    pages = torch.zeros(0, 2, 16, 64, device=DEV, dtype=kind)
    ws = torch.empty(stq.paged_attention_workspace_bytes(2, 4, 64, 2), dtype=torch.uint8, device=DEV)
    for work in (ws, None):
        o = torch.full((2, 4, 64), 7.0, device=DEV)
        stq.paged_attention(q, pages, pages, torch.zeros(2, 0, dtype=torch.int32, device=DEV),
                            torch.zeros(2, dtype=torch.int32, device=DEV), o, 0.125, workspace=work)
        assert torch.all(o == 0)


def test_attend_far_pages(stq):
    """Pages whose offsets pass 2^31 elements and 2^32 bytes."""
    page, Hkv, d = 64, 8, 128
    n = (1 << 31) // (page * Hkv * d) + 40
    kp, vp = (torch.empty(n, Hkv, page, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    lens = [130, 64]
    ids = [[n - 1, 0, n - 30], [n - 2, -1, -1]]
    g = torch.Generator(device=DEV).manual_seed(3)
    for row in ids:
        for i in row:
            if i >= 0:
                for pages in (kp, vp):
                    pages[i] = torch.randn(Hkv, page, d, generator=g, device=DEV).to(torch.bfloat16)
    q = torch.randn(2, 16, d, generator=g, device=DEV).to(torch.bfloat16)
    table = torch.tensor(ids, dtype=torch.int32, device=DEV)
    o = torch.empty(2, 16, d, device=DEV)
    ws = torch.empty(stq.paged_attention_workspace_bytes(2, 16, d, Hkv), dtype=torch.uint8, device=DEV)
    stq.paged_attention(q, kp, vp, table, torch.tensor(lens, dtype=torch.int32, device=DEV), o, d ** -0.5, workspace=ws)
    want, mag, E = attend_ref(q, kp, vp, table, lens, d ** -0.5)
    assert torch.all((o.double() - want).abs() <= (4 * E + 500 * U) * mag)
    # and their write
    k = torch.randn(3, Hkv, d, generator=g, device=DEV).to(torch.bfloat16)
    slots = torch.tensor([(n - 1) * page + 5, -1, (n - 2) * page], dtype=torch.int32, device=DEV)
    stq.page_write(kp, vp, slots, k, k)
    assert torch.equal(kp[n - 1, :, 5], k[0]) and torch.equal(vp[n - 2, :, 0], k[2])


# ---------------------------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("graph", [False, True])
def test_plan_write_attend(stq, graph, kind):
    """A few prompts and then decode steps: plan, write, attend, with the lengths kept on the device; also
    with the decode step captured once and replayed. Each step's output is that of the tokens so far."""
    B, Hq, Hkv, d, page, W = 3, 8, 2, 64, 16, 6
    prompts, steps = [30, 0, 17], 20
    i32 = dict(dtype=torch.int32, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    table, lens = torch.full((B, W), -1, **i32), torch.zeros(B, **i32)
    free = torch.randperm(B * W, generator=g, device=DEV).to(torch.int32)
    head, starts, status = torch.zeros(1, **i32), torch.zeros(B + 1, **i32), torch.zeros(1, **i32)
    kp, vp = (torch.full((B * W, Hkv, page, d), float("nan"), dtype=kind, device=DEV) for _ in range(2))
    rand = lambda *s: torch.randn(*s, generator=g, device=DEV).to(kind)  # noqa: E731
    said = [[[], []] for _ in range(B)]  # keys and values of every request, in order

    smap = torch.zeros(64, **i32)  # longer than the prompts: the rest is padding
    k, v = rand(64, Hkv, d), rand(64, Hkv, d)
    stq.page_plan(table, lens, torch.tensor(prompts, **i32), free, head, smap, starts, lens, head, page, status=status)
    stq.page_write(kp, vp, smap, k, v, status=status)
    at = 0
    for b, n in enumerate(prompts):
        said[b][0] += list(k[at:at + n])
        said[b][1] += list(v[at:at + n])
        at += n

    q, k, v = rand(B, Hq, d), rand(B, Hkv, d), rand(B, Hkv, d)
    fresh, smap = torch.ones(B, **i32), torch.zeros(B, **i32)
    o = torch.empty(B, Hq, d, device=DEV)
    ws = torch.empty(stq.paged_attention_workspace_bytes(B, Hq, d, Hkv), dtype=torch.uint8, device=DEV)

    def one():
        stq.page_plan(table, lens, fresh, free, head, smap, starts, lens, head, page, status=status)
        stq.page_write(kp, vp, smap, k, v, status=status)
        stq.paged_attention(q, kp, vp, table, lens, o, 0.125, workspace=ws, status=status)

    if graph:
        keep = [x.clone() for x in (table, lens, head)]
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            cg = torch.cuda.CUDAGraph()
            with torch.cuda.graph(cg, stream=s):
                one()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip((table, lens, head), keep))  # a capture runs nothing
        one_step = cg.replay
    else:
        one_step = one
    for step in range(steps):
        q.copy_(rand(B, Hq, d))
        k.copy_(rand(B, Hkv, d))
        v.copy_(rand(B, Hkv, d))
        for b in range(B):
            said[b][0].append(k[b].clone())
            said[b][1].append(v[b].clone())
        one_step()
        torch.cuda.synchronize()
        assert status.item() == 0
        assert lens.tolist() == [n + step + 1 for n in prompts]
        dense = [torch.zeros(B, Hkv, 64, d, dtype=kind, device=DEV) for _ in range(2)]
        for b in range(B):
            for x, rows in zip(dense, said[b]):
                x[b, :, :len(rows)] = torch.stack(rows).transpose(0, 1)
        want, mag, E = attend_ref(q, *dense, torch.arange(B, device=DEV)[:, None], lens.tolist(), 0.125)
        assert torch.all((o.double() - want).abs() <= (4 * E + 400 * U) * mag)


def test_repeats_are_bit_identical(stq):
    for kind in KINDS:
        q, kp, vp, table, lens = check_attend(stq, [5000, 3, 777], 8, 2, 128, 16, kind)
        outs = []
        for _ in range(3):
            o = torch.empty(3, 8, 128, device=DEV)
            ws = torch.empty(stq.paged_attention_workspace_bytes(3, 8, 128, 2), dtype=torch.uint8, device=DEV)
            stq.paged_attention(q, kp, vp, table, lens, o, 0.1, workspace=ws)
            outs.append(o)
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_two_streams_at_once(stq):
    """Two calls in flight with workspaces of their own."""
    sets = [check_attend(stq, [20000, 9000], 8, 2, 128, 16, torch.bfloat16, seed=s, ws=(True,)) for s in (1, 2)]
    need = stq.paged_attention_workspace_bytes(2, 8, 128, 2)
    alone, both = [], []
    for q, kp, vp, table, lens in sets:
        o = torch.empty(2, 8, 128, device=DEV)
        stq.paged_attention(q, kp, vp, table, lens, o, 0.1, workspace=torch.empty(need, dtype=torch.uint8, device=DEV))
        alone.append(o)
    streams = [torch.cuda.Stream() for _ in sets]
    work = [torch.empty(need, dtype=torch.uint8, device=DEV) for _ in sets]
    both = [torch.empty(2, 8, 128, device=DEV) for _ in sets]
    torch.cuda.synchronize()
    for _ in range(5):
        for (q, kp, vp, table, lens), s, w, o in zip(sets, streams, work, both):
            stq.paged_attention(q, kp, vp, table, lens, o, 0.1, workspace=w, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(alone, both))


def test_compiled_binding_and_python_make_the_same_calls(stq):
    """A tensor subclass and a stream argument go the Python way: the same outputs, bit for bit, and the same
    refusals."""
    from quantized_linear_attention_stq_b200 import _binding as b

    class Sub(torch.Tensor):
        pass

    g = torch.Generator(device=DEV).manual_seed(3)
    rnd = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    side = torch.cuda.Stream()
    N, H, d, page, n = 9, 1, 32, 4, 5
    both = rnd(N, 2 * H * d)
    k, v = (x.view(N, H, d) for x in both.split(H * d, dim=1))
    slots = torch.randperm(n * page, generator=g, device=DEV)[:N].to(torch.int32)
    pages = [torch.zeros(n, H, page, d, device=DEV) for _ in range(6)]
    assert b.page_write(pages[0], pages[1], slots, k, v, None, None) == 0
    assert b.page_write(pages[2], pages[3], slots, k.as_subclass(Sub), v, None, None) == -1
    stq.page_write(pages[2], pages[3], slots, k.as_subclass(Sub), v)
    torch.cuda.synchronize()
    stq.page_write(pages[4], pages[5], slots, k, v, stream=side)
    side.synchronize()
    for x in pages[2:]:
        assert torch.equal(x, pages[0] if torch.equal(x, pages[0]) else pages[1])
    assert torch.equal(pages[0], pages[2]) and torch.equal(pages[1], pages[5])
    q = rnd(2, 4, d)
    table = torch.tensor([[1, 0, 2], [3, 4, 0]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([11, 7], dtype=torch.int32, device=DEV)
    out = [torch.empty(2, 4, d, device=DEV) for _ in range(2)]
    ws = torch.empty(stq.paged_attention_workspace_bytes(2, 4, d, H), dtype=torch.uint8, device=DEV)
    assert b.paged_attention(q, pages[0], pages[1], table, lens, out[0], 0.3, ws, None, None) == 0
    torch.cuda.synchronize()
    stq.paged_attention(q.as_subclass(Sub), pages[0], pages[1], table, lens, out[1], 0.3, workspace=ws)
    assert torch.equal(out[0], out[1])
    # a workspace that is too small is not taken by the compiled call, and named by the Python one
    assert b.paged_attention(q, pages[0], pages[1], table, lens, out[0], 0.3, ws[:64], None, None) == -1
    with pytest.raises(ValueError):
        stq.paged_attention(q, pages[0], pages[1], table, lens, out[0], 0.3, workspace=ws[:64])
    # what the library refuses is raised from either way
    for x in (q, q.as_subclass(Sub)):
        with pytest.raises(stq.StqError):
            stq.paged_attention(x, pages[0], pages[1], table, lens, out[0], float("inf"), workspace=ws)


@pytest.mark.parametrize("captured", [False, True])
def test_calls_keep_the_streams_order(stq, captured):
    """Kernels are set up while the one before them runs: still each reads what was written just before it, by
    a call of the library or by torch, and is done before what follows. Run without a wait between, and with
    one behind every operation."""
    B, Hq, H, d, page, steps = 5, 8, 2, 64, 4, 60
    g = torch.Generator(device=DEV).manual_seed(7)
    rnd = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    noise = [rnd(B, (Hq + 2 * H) * d) for _ in range(steps)]
    gates = [torch.rand(B, H, generator=g, device=DEV) for _ in range(steps)]
    n, W = 200, 40
    i32 = dict(dtype=torch.int32, device=DEV)
    ws = torch.empty(stq.paged_attention_workspace_bytes(B, Hq, d, H), dtype=torch.uint8, device=DEV)

    def run(wait):
        table, lens, head = torch.zeros(B, W, **i32), torch.zeros(B, **i32), torch.zeros(1, **i32)
        fresh, free, starts = torch.ones(B, **i32), torch.arange(n, **i32).flip(0).contiguous(), torch.zeros(B + 1, **i32)
        slots, smap = torch.arange(B, **i32), torch.zeros(B, **i32)
        pages = [torch.zeros(n, H, page, d, device=DEV) for _ in range(2)]
        states, o, o2, x = torch.zeros(B, H, d, d, device=DEV), torch.zeros(B, Hq, d, device=DEV), torch.zeros(B, H, d, device=DEV), torch.zeros(B, d, device=DEV)
        outs = torch.zeros(steps, B, d, device=DEV)

        def body():
            for s in range(steps):
                ops = [
                    lambda: stq.page_plan(table, lens, fresh, free, head, smap, starts, lens, head, page),
                    lambda: torch.add(noise[s], x.repeat(1, Hq + 2 * H), out=qkv),
                    lambda: torch.tanh(qkv, out=qkv),
                    lambda: stq.page_write(*pages, smap, qkv[:, Hq * d:(Hq + H) * d].view(B, H, d), qkv[:, (Hq + H) * d:].view(B, H, d)),
                    lambda: q.copy_(qkv[:, :Hq * d].view(B, Hq, d)),
                    lambda: stq.paged_attention(q, *pages, table, lens, o, 0.125, workspace=ws),
                    lambda: stq.decay_step(states, slots, o[:, :H].contiguous(), o[:, H:2 * H].contiguous(), o[:, 2 * H:3 * H].contiguous(), gates[s], o2),
                    lambda: torch.sum(o2, dim=1, out=x),
                    lambda: outs[s].copy_(x),
                ]
                for op in ops:
                    op()
                    if wait:
                        torch.cuda.synchronize()

        qkv, q = torch.zeros(B, (Hq + 2 * H) * d, device=DEV), torch.zeros(B, Hq, d, device=DEV)
        if captured and not wait:
            first = [t.clone() for t in (table, lens, head, states, x, *pages)]
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                body()
            for t, was in zip((table, lens, head, states, x, *pages), first):
                t.copy_(was)
            graph.replay()
        else:
            body()
        torch.cuda.synchronize()
        return outs, states, pages[0], pages[1], lens

    for a, b in zip(run(False), run(True)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("lens_in_place", [False, True])
@pytest.mark.parametrize("head_in_place", [False, True])
def test_plan_large_map_partly_in_place(stq, lens_in_place, head_in_place):
    """Many blocks' plan with either, both or none of the lengths and the head updated in place."""
    table, lens, fresh, free = plan_case(200, 8, 60, 300, 5)
    N = sum(fresh) + 7
    assert N > 20000
    want = run_plan(stq, table, lens, fresh, free, 0, N, 8, False)
    t = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    for _ in range(5):
        tt, ll, ff, fr, hh = t(table), t(lens), t(fresh), t(free), t([0])
        lo, ho = ll if lens_in_place else t([-9] * len(lens)), hh if head_in_place else t([-9])
        smap, starts, status = t([-7] * N), t([-7] * (len(lens) + 1)), t([0])
        stq.page_plan(tt, ll, ff, fr, hh, smap, starts, lo, ho, 8, status=status)
        assert (tt.tolist(), lo.tolist(), smap.tolist(), starts.tolist(), ho.item(), status.item()) == want


@pytest.mark.parametrize("N", [60, 5000])  # one block's plan, and that of many
def test_plan_refuses_lengths_past_int32(stq, N):
    """A table row may span more than int32 counts: a request whose tokens pass it gets no slots, keeps its
    length and is flagged; one that ends at the last count is served, and so are those behind."""
    page, most = 1 << 30, 2147483647
    table = [[0, 1, -1], [0, 1, -1], [0, -1, -1], [0, 1, -1]]
    lens, fresh = [most - 7, most - 20, 5, most], [20, 20, 3, 1]
    for inplace in (False, True):
        got = run_plan(stq, table, lens, fresh, [2, 3], 0, N, page, inplace)
        assert got[0] == table and got[1] == [most - 7, most, 8, most]
        assert got[2] == [-1] * 20 + list(range(most - 20, most)) + [5, 6, 7] + [-1] * (N - 43)
        assert got[3] == [0, 20, 40, 43, 44] and got[4] == 0 and got[5] == 1 << 6
    # a row of many pages, and the request that is refused in front of its last page
    table, free = [list(range(2048)) + [-1] * 2048], [7, 8]
    got = run_plan(stq, table, [most - 99], [200], free, 0, N, 1 << 20)
    assert got[0] == table and got[1] == [most - 99] and got[4] == 0 and got[5] == 1 << 6
    assert got[2] == [-1] * N and got[3] == [0, min(200, N)]


@pytest.mark.parametrize("kind", KINDS)
def test_attend_up_to_the_last_position(stq, kind):
    """A cache whose last tokens stand within a hundred of the last that a call takes (2^31 - 65). Every
    entry of the table names the same page, so the softmax is that over the page's rows.

    A block's sums are those of 2^31 / (64 * 592) tiles at least, added one after the other: with at most four
    additions a tile and 592 pieces, n = 4 * 56680 + 592 in the bound that stands at the head of this file."""
    page, W, d = 38820, 55319, 16
    L = page * W
    assert 2 ** 31 - 94 <= L <= 2 ** 31 - 65
    g = torch.Generator(device=DEV).manual_seed(12)
    kp, vp = (torch.randn(3, 1, page, d, generator=g, device=DEV).to(kind) for _ in range(2))
    q = torch.randn(1, 1, d, generator=g, device=DEV).to(kind)
    table, lens = torch.ones(1, W, dtype=torch.int32, device=DEV), torch.tensor([L], dtype=torch.int32, device=DEV)
    o, status = torch.empty(1, 1, d, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = torch.empty(stq.paged_attention_workspace_bytes(1, 1, d, 1), dtype=torch.uint8, device=DEV)
    stq.paged_attention(q, kp, vp, table, lens, o, 0.25, workspace=ws, status=status)
    assert status.item() == 0
    want, mag, E = attend_ref(q, kp, vp, table, [page], 0.25)
    n = 4 * 56680 + 592
    assert torch.all((o.double() - want).abs() <= (4 * E + (2 * n + 16) * U) * mag)


@pytest.mark.parametrize("page", [(1 << 32) + 16, 16 - (1 << 32), 1 << 70, -(1 << 70)])
def test_page_sizes_past_int32_are_refused(stq, page):
    """By the compiled module, without a call, and then by name."""
    from quantized_linear_attention_stq_b200 import _binding as b

    i = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    args = [torch.full((1, 3), -1, dtype=torch.int32, device=DEV), i(0), i(2), i(1, 0, 2), i(0), i(5, 5, 5), i(7, 7), i(9), i(9)]
    assert b.page_plan(*args, page, None, None) == -1
    with pytest.raises(ValueError, match="past int32"):
        stq.page_plan(*args, page)
    assert args[5].tolist() == [5, 5, 5] and args[7].item() == 9


def in_order(body, tensors, captured):
    """What body(op) leaves in `tensors` where its operations run without a wait between, directly or captured,
    and where each is waited for."""
    first = [t.clone() for t in tensors]

    def start():
        for t, was in zip(tensors, first):
            t.copy_(was)
        torch.cuda.synchronize()

    def waited(op):
        op()
        torch.cuda.synchronize()

    start()
    body(waited)
    want = [t.clone() for t in tensors]
    start()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            body(lambda op: op())
        start()
        graph.replay()
    else:
        body(lambda op: op())
    torch.cuda.synchronize()
    return zip(tensors, want)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("B", [200, 1100])  # one round of requests, and two
def test_large_plans_in_place_keep_the_streams_order(stq, B, captured):
    """Plans of many blocks that update the lengths and the list's head in place, each right behind kernels
    that write both, and the counts, and in front of ones that read what it wrote."""
    page, W, steps, most = 8, 30, 12, 44
    g = torch.Generator(device=DEV).manual_seed(8)
    i32 = dict(dtype=torch.int32, device=DEV)
    N = B * most // 2
    assert N > 4096
    a = torch.randn(2048, 2048, generator=g, device=DEV)
    counts = torch.randint(0, most, (steps, B), generator=g, device=DEV).to(torch.int32)
    held = torch.randint(0, 100, (steps, B), generator=g, device=DEV).to(torch.int32)
    table, free = torch.arange(B * W, **i32).view(B, W).contiguous(), torch.arange(B * W, **i32).flip(0).contiguous()
    lens, fresh, head, starts, smap = (torch.zeros(n, **i32) for n in (B, B, 1, B + 1, N))
    slow, status = torch.zeros(2048, 2048, device=DEV), torch.zeros(1, **i32)
    kept = [torch.zeros(steps, n, **i32) for n in (B, 1, B + 1, N)]

    def body(do):
        for s in range(steps):
            do(lambda: torch.mm(a, a, out=slow))  # the writes below stand behind a slow kernel
            do(lambda: fresh.copy_(counts[s]))
            do(lambda: torch.add(held[s], lens % 7, out=lens))
            do(lambda: head.copy_(slow[:1, 0].abs().clamp(max=0).int() + s))
            do(lambda: stq.page_plan(table, lens, fresh, free, head, smap, starts, lens, head, page, status=status))
            for to, x in zip(kept, (lens, head, starts, smap)):
                do(lambda: to[s].copy_(x))

    for got, want in in_order(body, [table, lens, head, starts, smap, status, *kept], captured):
        assert torch.equal(got, want)
    assert status.item() == 1 << 6  # the map ends inside some plans


@pytest.mark.parametrize("B,new", [(2500, 20), (1025, 100)])
def test_plan_large_map_of_more_requests_than_threads(stq, B, new):
    """Many blocks' plans that take more than one round of requests, in place and not: all served, and with a
    free list, a slot map or both that end inside the second round."""
    page = 8
    table, lens, fresh, free = plan_case(B, page, 40, new, B)
    need = [-(-(a + b) // page) + -a // page for a, b in zip(lens, fresh)]
    N, pages, tokens = sum(fresh), sum(need), sum(fresh[:1024])
    assert N > 4096 and B > 1024 and tokens < N
    check_plan(stq, table, lens, fresh, free, 0, N + 9, page)
    check_plan(stq, table, lens, fresh, [99999] * 2 + free, 2, N, page)
    inside = sum(need[:1024]) + max(1, (pages - sum(need[:1024])) // 2)
    check_plan(stq, table, lens, fresh, free[:inside], 0, N, page)
    check_plan(stq, table, lens, fresh, free, 0, tokens + (N - tokens) // 2, page)
    check_plan(stq, table, lens, fresh, free[:inside], 0, tokens + (N - tokens) // 2 + 1, page)
    check_plan(stq, table, lens, fresh, free[: sum(need[:1000])], 0, sum(fresh[:1010]), page)  # and inside the first
    # requests that are refused in the first round, and others that need nothing
    bad = list(lens)
    bad[5], bad[1000] = -1, page * len(table[0]) + 1
    none = [0 if i % 3 else n for i, n in enumerate(fresh)]
    if sum(none) > 4096:
        check_plan(stq, table, bad, none, free, 0, sum(none), page)
    check_plan(stq, table, bad, fresh, free, 0, N, page)


def binding_calls(kind):
    """For each call of the binding: its name, valid arguments in order, and which of them may have another
    length than the others ask for."""
    g = torch.Generator(device=DEV).manual_seed(4)
    rnd = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    B, H, T, d = 2, 3, 5, 32
    pages = lambda: rnd(6, H, 4, d).to(kind)  # noqa: E731
    word = lambda: torch.zeros(1, dtype=torch.int32, device=DEV)  # noqa: E731
    return {
        "decay_step": (dict(states=rnd(4, H, d, d), slots=i(1, 3), q=rnd(B, H, d).to(kind), k=rnd(B, H, d).to(kind),
                            v=rnd(B, H, d).to(kind), alpha=torch.rand(B, H, device=DEV), o=rnd(B, H, d), status=word()), {"states"}),
        "decay_prefill": (dict(states=rnd(4, H, d, d), slots=i(1, 3), q=rnd(B, H, T, d).to(kind), k=rnd(B, H, T, d).to(kind),
                               v=rnd(B, H, T, d).to(kind), alpha=torch.rand(B, H, T, device=DEV), o=rnd(B, H, T, d), lens=i(5, 2),
                               workspace=None, status=word()), {"states"}),
        "page_plan": (dict(table=i(0, -1, -1, 1, -1, -1).view(2, 3), lens=i(3, 1), fresh=i(2, 1), free_pages=i(4, 2, 5),
                           free_head=i(0), slot_map=i(0, 0, 0), starts=i(0, 0, 0), lens_out=i(0, 0), head_out=i(0),
                           page_size=4, status=word()), {"free_pages", "slot_map"}),
        "page_write": (dict(k_pages=pages(), v_pages=pages(), slot_map=i(5, -1, 9), k=rnd(3, H, d).to(kind),
                            v=rnd(3, H, d).to(kind), status=word()), set()),
        "paged_attention": (dict(q=rnd(B, 2 * H, d).to(kind), k_pages=pages(), v_pages=pages(), table=i(0, 1, 5, 2).view(2, 2),
                                 lens=i(7, 5), o=rnd(B, 2 * H, d), scale=0.2,
                                 workspace=torch.empty(1 << 22, dtype=torch.uint8, device=DEV), status=word()), set()),
    }


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("name", ["decay_step", "decay_prefill", "page_plan", "page_write", "paged_attention"])
def test_compiled_binding_checks_every_argument(stq, name, kind):
    """From valid CUDA arguments, one is replaced at a time: the compiled module makes no call, and the Python
    one names what is wrong. What is tried is never smaller than what it stands for."""
    from quantized_linear_attention_stq_b200 import _binding as b

    args, free = binding_calls(kind)[name]
    compiled = lambda a: getattr(b, name)(*a.values(), None)  # noqa: E731
    assert compiled(args) == 0 and args["status"].item() == 0
    getattr(stq, name)(**args)
    torch.cuda.synchronize()
    tried = 0
    for what, t in args.items():
        if not isinstance(t, torch.Tensor):
            wrong = [("kind", "x")] if t is not None else []
        else:
            wrong = [("kind", "x"), ("cpu", t.cpu())]
            if what != "workspace":  # that one is bytes of any shape and type
                wrong += [("dtype", t.to(torch.float64 if t.is_floating_point() else torch.int64)), ("dims", t[None]),
                          ("type of another kind", t.int() if t.dtype == torch.float32 else t.float())]
                if what not in free and not (name == "paged_attention" and what == "q"):
                    wrong += [("length", torch.cat([t, t]))]
                wrong += [("width", torch.cat([t, t], -1))] if t.dim() > 1 and what != "table" else []
            else:
                wrong += [("length", t[:1024])]
            if what in ("k", "v") and name == "page_write":  # tokens may be strided, heads may not
                wrong += [("strides", torch.cat([t, t], 1)[:, ::2])]
            elif t.numel() > 1:
                wrong += [("strides", torch.stack([t, t], -1)[..., 0])]
            if what not in ("status", "workspace", "lens"):
                wrong += [("none", None)]
        for how, x in wrong:
            tried += 1
            assert compiled({**args, what: x}) == -1, f"{what}: {how}"
            with pytest.raises((TypeError, ValueError)):
                getattr(stq, name)(**{**args, what: x})
    assert tried > 25
    torch.cuda.synchronize()
    assert args["status"].item() == 0
