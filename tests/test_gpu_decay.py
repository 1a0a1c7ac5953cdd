"""Decayed linear attention (decay_step, decay_prefill) against the recurrence in 64 bits.

Tolerances. u = 2^-24 is fp32's rounding. Let A and m be the recurrence and readout on absolute
values, A <- |a| A + |k||v|^T, m = A^T |q|: every term of a state entry or output is bounded by them.
One step rounds a state entry three times, a readout adds d + 1 roundings. A chunked form multiplies up to
127 decays, sums up to 128 + d terms, and rounds a few times per chunk. So after T tokens a state entry
is off by at most (3 T + 4 d + 300) u A and an output by as much of m; independent roundings add in
quadrature, which bounds the 2-norm of the error by 4 sqrt(3 T + 4 d + 300) u of the magnitudes' norm.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24


@pytest.fixture(scope="module")
def stq():
    import quantized_linear_attention_stq_b200 as m

    m.lib()
    return m


def make(B, H, T, d, kind, seed=0, half=64.0, spare=2):
    g = torch.Generator().manual_seed(seed)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    q, k = (unit(torch.randn(B, H, T, d, generator=g)).to(kind) for _ in range(2))
    v = torch.randn(B, H, T, d, generator=g).to(kind)
    alpha = torch.exp(-2 * torch.rand(B, H, T, generator=g) / half)
    slots = torch.randperm(B + spare, generator=g)[:B].to(torch.int32)
    states = torch.randn(B + spare, H, d, d, generator=g)
    return q, k, v, alpha, slots, states


def recurrence(q, k, v, alpha, S, lens=None):
    """o, S and their magnitudes in 64 bits; tokens behind a prompt's end change nothing (o: NaN there)."""
    q, k, v, alpha, S = (x.double() for x in (q, k, v, alpha, S))
    A = S.abs()
    B, H, T, d = q.shape
    o = torch.full((B, H, T, d), float("nan"), dtype=torch.float64, device=q.device)
    m = torch.zeros_like(o)
    for t in range(T):
        for b in range(B):
            if lens is not None and t >= lens[b]:
                continue
            a = alpha[b, :, t, None, None]
            S[b] = a * S[b] + k[b, :, t, :, None] * v[b, :, t, None, :]
            A[b] = a.abs() * A[b] + k[b, :, t, :, None].abs() * v[b, :, t, None, :].abs()
            o[b, :, t] = torch.einsum("hij,hi->hj", S[b], q[b, :, t])
            m[b, :, t] = torch.einsum("hij,hi->hj", A[b], q[b, :, t].abs())
    return o, S, m, A


def close(got, want, size, T, d, what):
    n = 3 * T + 4 * d + 300
    err = (got.double() - want).abs()
    assert torch.all(err <= n * U * size + 1e-37), f"{what}: {(err / (U * size + 1e-37)).max().item():.1f} u, allowed {n}"
    assert err.norm() <= 4 * n ** 0.5 * U * size.norm() + 1e-30, f"{what}: 2-norm {(err.norm() / (U * size.norm())).item():.1f} u"


def check(stq, B, H, T, d, kind, lens=None, half=64.0, seed=0, ws=True, mutate=None, step=False):
    q, k, v, alpha, slots, states = make(B, H, T, d, kind, seed, half)
    if mutate:
        mutate(q, k, v, alpha, states)
    o_ref, S_ref, m, A = recurrence(*(x.to(DEV) for x in (q, k, v, alpha)), states[slots.long()].to(DEV), lens)
    dev = [x.to(DEV) for x in (states, slots, q, k, v, alpha)]
    if lens is not None:  # what stands behind a prompt's end is not used
        for b, n in enumerate(lens):
            for x in dev[2:6]:
                x[b, :, n:] = float("nan")
    o = torch.full((B, H, T, d), 7.0, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    if step:
        args = [dev[0], dev[1]] + [x[:, :, 0].contiguous() for x in dev[2:6]]
        o = o[:, :, 0].contiguous()
        stq.decay_step(*args, o, status=status)
        o = o[:, :, None]
    else:
        need = stq.decay_prefill_workspace_bytes(B, H, T, d, kind)
        work = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV) if need and ws else None  # NaN bytes
        stq.decay_prefill(*dev, o, lens=None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV),
                          workspace=work, status=status)
    assert status.item() == 0, stq.status_flags(status)
    for b in range(B):
        n = T if lens is None else lens[b]
        if n:
            close(o[b, :, :n], o_ref[b, :, :n], m[b, :, :n], n, d, f"o of request {b}")
        assert torch.all(o[b, :, n:] == 7.0), "rows behind the prompt's end were written"
        close(dev[0][slots[b]], S_ref[b], A[b], n, d, f"state of request {b}")
    rest = [i for i in range(states.shape[0]) if i not in slots.tolist()]
    assert torch.equal(dev[0][rest].cpu(), states[rest]), "a slot that no request names was written"
    return dev[0], o


KINDS = [torch.float32, torch.bfloat16]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("B,H", [(1, 1), (3, 5)])
def test_step(stq, B, H, d, kind):
    check(stq, B, H, 1, d, kind, step=True)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("T", [1, 2, 31, 127, 128, 129, 300])
def test_prefill_lengths(stq, T, d, kind):
    check(stq, 2, 3, T, d, kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [16, 64, 128])
def test_prefill_ragged(stq, d, kind):
    check(stq, 5, 2, 260, d, kind, lens=[260, 0, 1, 129, 128])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [32, 128])
@pytest.mark.parametrize("half", [0.05, 1.0, 1e6])
def test_prefill_decays(stq, half, d, kind):
    """From decays that forget at once (their products underflow) to ones that hardly forget."""
    check(stq, 1, 2, 200, d, kind, half=half)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [16, 128])
def test_prefill_odd_gates(stq, d, kind):
    """Decays of zero (the state is cleared), one, negative and above one."""
    def mutate(q, k, v, alpha, states):
        alpha[:, :, 3] = 0.0
        alpha[:, :, 130] = 0.0
        alpha[:, :, 131] = 0.0
        alpha[:, 0, ::2] = -alpha[:, 0, ::2]
        alpha[:, 1, 140:150] = 1.25
        alpha[:, 1, 0] = 1.0

    check(stq, 2, 2, 190, d, kind, mutate=mutate)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [None, [5000, 1700, 0]])
def test_prefill_long_few_heads(stq, d, lens):
    """Few heads and a long prompt, with and without a workspace."""
    B = 1 if lens is None else 3
    a, oa = check(stq, B, 1, 5000, d, torch.bfloat16, lens=lens, half=500.0)
    b, ob = check(stq, B, 1, 5000, d, torch.bfloat16, lens=lens, half=500.0, ws=False)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [32, 128])
def test_scales_of_inputs(stq, d, kind):
    """Keys and values of very different magnitude from token to token."""
    def mutate(q, k, v, alpha, states):
        s = torch.logspace(-12, 12, k.shape[2])[None, None, :, None]
        k.mul_(s.to(k.dtype))
        v.mul_(s.flip(2).sqrt().to(v.dtype))

    check(stq, 1, 2, 150, d, kind, mutate=mutate)


@pytest.mark.parametrize("kind", KINDS)
def test_prompt_then_tokens_equals_prompt(stq, kind):
    """A prompt and then single tokens end where the whole prompt does, and stop anywhere."""
    B, H, T, d = 2, 2, 140, 64
    q, k, v, alpha, slots, states = (x.to(DEV) for x in make(B, H, T, d, kind, seed=5))
    o_ref, S_ref, m, A = recurrence(q, k, v, alpha, states[slots.long()])
    for cut in (1, 100, 128, 137):
        st = states.clone()
        o = torch.empty(B, H, cut, d, device=DEV)
        stq.decay_prefill(st, slots, *(x[:, :, :cut].contiguous() for x in (q, k, v, alpha)), o)
        close(o, o_ref[:, :, :cut], m[:, :, :cut], T, d, "prompt")
        for t in range(cut, T):
            o1 = torch.empty(B, H, d, device=DEV)
            stq.decay_step(st, slots, *(x[:, :, t].contiguous() for x in (q, k, v, alpha)), o1)
            close(o1, o_ref[:, :, t], m[:, :, t], T, d, f"token {t}")
        close(st[slots.long()], S_ref, A, T, d, "state")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("form", ["step", "prefill"])
def test_bad_slots_and_lengths_are_skipped(stq, form, kind):
    """A slot outside the pool or a length outside the prompt: the request is left alone and flagged."""
    B, H, T, d = 4, 2, 1 if form == "step" else 133, 128
    q, k, v, alpha, slots, states = make(B, H, T, d, kind, seed=3)
    o_ref, S_ref, m, A = recurrence(*(x.to(DEV) for x in (q, k, v, alpha)), states[slots.long()].to(DEV))
    live = slots.clone()
    live[1], live[2] = -1, states.shape[0]
    dev = [x.to(DEV) for x in (states, live, q, k, v, alpha)]
    o = torch.full((B, H, T, d), 7.0, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    if form == "step":
        o = o[:, :, 0].contiguous()
        stq.decay_step(dev[0], dev[1], *(x[:, :, 0].contiguous() for x in dev[2:]), o, status=status)
        o = o[:, :, None]
        good = (0, 3)
    else:
        lens = torch.tensor([T, T, T, T + 1], dtype=torch.int32, device=DEV)
        stq.decay_prefill(*dev, o, lens=lens, status=status)
        good = (0,)
    assert status.item() == 1 << 6
    for b in range(B):
        if b in good:
            close(o[b], o_ref[b], m[b], T, d, "o")
            close(dev[0][slots[b]], S_ref[b], A[b], T, d, "state")
        else:
            assert torch.all(o[b] == 7.0)
            assert torch.equal(dev[0][slots[b]].cpu(), states[slots[b]])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("where", ["v", "state", "alpha"])
def test_nonfinite_is_flagged(stq, where, kind):
    """An infinity or NaN spreads as the formula says and is flagged; other requests are untouched."""
    B, H, T, d = 2, 2, 40, 128
    q, k, v, alpha, slots, states = make(B, H, T, d, kind, seed=4)
    if where == "v":
        v[0, 1, 20, 3] = float("inf")
    elif where == "state":
        states[slots[0], 1, 5, 3] = float("nan")
    else:
        alpha[0, 1, 20] = float("inf")
    o_ref, S_ref, m, A = recurrence(*(x.to(DEV) for x in (q, k, v, alpha)), states[slots.long()].to(DEV))
    dev = [x.to(DEV) for x in (states, slots, q, k, v, alpha)]
    o = torch.empty(B, H, T, d, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    stq.decay_prefill(*dev, o, status=status)
    assert status.item() == 1 << 4
    assert not torch.isfinite(o[0, 1, 20:, 3]).any()
    close(o[1], o_ref[1], m[1], T, d, "the other request")
    close(o[0, 0], o_ref[0, 0], m[0, 0], T, d, "the other head")
    close(dev[0][slots[1]], S_ref[1], A[1], T, d, "the other state")


def test_repeats_are_bit_identical(stq):
    for kind, (B, H, T, d) in ((torch.bfloat16, (1, 2, 3000, 128)), (torch.float32, (2, 3, 200, 64))):
        q, k, v, alpha, slots, states = (x.to(DEV) for x in make(B, H, T, d, kind, seed=8))
        need = stq.decay_prefill_workspace_bytes(B, H, T, d, kind)
        outs = []
        for _ in range(2):
            st, o = states.clone(), torch.empty(B, H, T, d, device=DEV)
            stq.decay_prefill(st, slots, q, k, v, alpha, o, workspace=torch.empty(max(need, 1), dtype=torch.uint8, device=DEV))
            outs.append((st, o))
        assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


@pytest.mark.parametrize("kind", KINDS)
def test_other_stream_and_graph(stq, kind):
    """On a side stream, and captured and replayed on new inputs, a call does what it does directly."""
    B, H, T, d = 2, 2, 200, 128
    q, k, v, alpha, slots, states = (x.to(DEV) for x in make(B, H, T, d, kind, seed=9))
    st0, o0 = states.clone(), torch.empty(B, H, T, d, device=DEV)
    need = stq.decay_prefill_workspace_bytes(B, H, T, d, kind)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device=DEV)
    stq.decay_prefill(st0, slots, q, k, v, alpha, o0, workspace=ws)
    one = [x[:, :, 0].contiguous() for x in (q, k, v, alpha)]
    o1 = torch.empty(B, H, d, device=DEV)
    stq.decay_step(st0, slots, *one, o1)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    st, o, o2 = states.clone(), torch.empty_like(o0), torch.empty_like(o1)
    torch.cuda.synchronize()
    stq.decay_prefill(st, slots, q, k, v, alpha, o, workspace=ws, stream=s)
    stq.decay_step(st, slots, *one, o2, stream=s)
    s.synchronize()
    assert torch.equal(st, st0) and torch.equal(o, o0) and torch.equal(o2, o1)
    st.copy_(states)
    qg = torch.zeros_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        stq.decay_prefill(st, slots, qg, k, v, alpha, o, workspace=ws)
        stq.decay_step(st, slots, *one, o2)
    qg.copy_(q)
    o.zero_()
    st.copy_(states)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(st, st0) and torch.equal(o, o0) and torch.equal(o2, o1)


def test_states_park_as_codes(stq):
    """A finished prompt's states go to the quantized pool and come back within the codes' step."""
    B, H, T, d = 2, 4, 64, 128
    q, k, v, alpha, slots, states = (x.to(DEV) for x in make(B, H, T, d, torch.bfloat16, seed=11))
    o = torch.empty(B, H, T, d, device=DEV)
    stq.decay_prefill(states, slots, q, k, v, alpha, o)
    lay = stq.Layout([8] * H, d)
    pool = lay.alloc_pool(B, DEV)
    at = torch.arange(B, dtype=torch.int32, device=DEV)
    S = states[slots.long()].contiguous()
    stq.init_state(lay, pool, at, S, torch.ones(H, d, device=DEV))
    back = torch.empty_like(S)
    stq.dequantize(lay, pool, at, back)
    # r_i c_j Q_ij with |Q| <= 127 and r_i = max_j |S_ij / c_j| / 127: half a step is r_i c_j / 2
    c = (S * S).mean(dim=2, keepdim=True).sqrt()
    r = (S / c).abs().amax(dim=3, keepdim=True) / 127
    assert torch.all((S - back).abs() <= r * c * (0.5 + 1e-3))


@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("lens", [None, [3000, 1, 0, 129, 2999]])
def test_prefill_segments_of_full_precision_prompts(stq, d, lens):
    """Long float32 prompts of few heads are cut into segments; ends in, at and between their borders."""
    B = 1 if lens is None else len(lens)
    need = stq.decay_prefill_workspace_bytes(B, 2, 3000, d, torch.float32)
    assert need > 0
    check(stq, B, 2, 3000, d, torch.float32, lens=lens, half=300.0, seed=21)
    check(stq, B, 2, 3000, d, torch.float32, lens=lens, half=300.0, seed=21, ws=False)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [32, 64, 128])
def test_prefill_many_heads(stq, d, kind):
    """As many heads as take four columns to a thread token by token, short and ragged."""
    check(stq, 20, 32, 40, d, kind, lens=[40 - 2 * b for b in range(20)], seed=22)


@pytest.mark.parametrize("d", [16, 32, 64, 128])
def test_prefill_ends_inside_a_warps_rows(stq, d):
    """Chunks whose last tokens fill some of the 32-row groups of o, whole or in part."""
    check(stq, 7, 2, 256, d, torch.bfloat16, lens=[32, 33, 63, 64, 160, 191, 255], seed=23)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [16, 128])
def test_prefill_cleared_at_borders(stq, d, kind):
    """Decays of zero at the first and last tokens of chunks and groups, over several segments."""
    def mutate(q, k, v, alpha, states):
        for t in (0, 15, 16, 127, 128, 255, 256, 1023, 1024, 1999):
            alpha[:, 0, t] = 0.0

    check(stq, 1, 2, 2000, d, kind, mutate=mutate, half=2000.0, seed=24)


def test_two_prompts_at_once(stq):
    """Two prompts on two streams, each with its workspace, do what they do alone."""
    B, H, T, d = 1, 3, 4000, 128
    runs = []
    for seed in (31, 32):
        q, k, v, alpha, slots, states = (x.to(DEV) for x in make(B, H, T, d, torch.bfloat16, seed=seed))
        need = stq.decay_prefill_workspace_bytes(B, H, T, d, torch.bfloat16)
        st, o = states.clone(), torch.empty(B, H, T, d, device=DEV)
        stq.decay_prefill(st, slots, q, k, v, alpha, o, workspace=torch.empty(need, dtype=torch.uint8, device=DEV))
        runs.append((q, k, v, alpha, slots, states, st, o, torch.empty(need, dtype=torch.uint8, device=DEV), torch.cuda.Stream()))
    torch.cuda.synchronize()
    out = []
    for _ in range(3):
        for q, k, v, alpha, slots, states, st, o, ws, s in runs:
            with torch.cuda.stream(s):
                st2, o2 = states.clone(), torch.empty_like(o)
                stq.decay_prefill(st2, slots, q, k, v, alpha, o2, workspace=ws)
                out.append((st, st2, o, o2))
    torch.cuda.synchronize()
    for st, st2, o, o2 in out:
        assert torch.equal(st, st2) and torch.equal(o, o2)


def test_status_flags_name_no_wait_that_ran_out(stq):
    """A second of prompts of every shape back to back: no bounded wait gives up."""
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    for i, (B, H, T, d) in enumerate([(1, 1, 1, 128), (3, 7, 4097, 128), (2, 40, 513, 64), (1, 5, 2049, 16), (9, 9, 129, 32)]):
        q, k, v, alpha, slots, states = (x.to(DEV) for x in make(B, H, T, d, torch.bfloat16, seed=40 + i))
        need = stq.decay_prefill_workspace_bytes(B, H, T, d, torch.bfloat16)
        ws = torch.empty(need, dtype=torch.uint8, device=DEV) if need else None
        o = torch.empty(B, H, T, d, device=DEV)
        for _ in range(40):
            stq.decay_prefill(states, slots, q, k, v, alpha, o, workspace=ws, status=status)
    assert status.item() == 0, stq.status_flags(status)


@pytest.mark.parametrize("kind,B,H,T,d,grow,rate", [
    (torch.bfloat16, 1, 2, 7936, 64, 256, 1.8),     # segments of 2 chunks: 1.8^256 = 2e65
    (torch.bfloat16, 1, 60, 13440, 16, 1920, 1.8),  # of 464 tokens: 1.8^464 = 3e118
    (torch.bfloat16, 1, 60, 13440, 32, 1920, 1.8),  # of 15 chunks: 1.8^1920 = 1e490, past fp64 as well
    (torch.float32, 1, 600, 600, 16, 320, 1.4),     # of 320 tokens: 1.4^320 = 6e46
])
def test_prefill_segments_whose_decays_product_passes_fp32(stq, kind, B, H, T, d, grow, rate):
    """Products of 128 decays are finite, a segment's is not: empty states stay empty, a state that is
    cleared again is empty, one so small that it may grow that much does."""
    assert stq.decay_prefill_workspace_bytes(B, H, T, d, kind) > 0

    def mutate(q, k, v, alpha, states):
        k[:, :, :grow] = 0
        alpha[:, :, :grow] = rate
        alpha[:, 1::2, :grow] *= -1
        states.zero_()
        n = math.floor(math.log10(rate) * grow)
        if n < 70:  # S0 2^e rate^grow, some 1e10 (bf16's terms of S0 stay normal)
            states[:, 0] = torch.randn(states.shape[0], d, d, generator=torch.Generator().manual_seed(1)) * 10.0 ** max(10 - n, -30)
        if H > 4:
            states[:, 4] = 1.0
            alpha[:, 4, 0] = 0.0
            alpha[:, 5, grow - 1] = 0.0

    for ws in (True, False):
        check(stq, B, H, T, d, kind, half=50.0, seed=51, mutate=mutate, ws=ws)


@pytest.mark.parametrize("kind", KINDS)
def test_prefill_segments_whose_decays_product_is_below_fp32(stq, kind):
    """States that large decays bring down to where the segment's product is no normal fp32 number."""
    def mutate(q, k, v, alpha, states):
        k.zero_()
        alpha.fill_(0.67)  # 0.67^256 = 3e-45
        alpha[:, :, 256:] = 1.0
        states.mul_(1e30)

    H, T = (2, 7936) if kind == torch.bfloat16 else (600, 512)
    check(stq, 1, H, T, 16, kind, seed=52, mutate=mutate)


@pytest.mark.parametrize("kind,H,d,longest,lengths", [
    (torch.bfloat16, 2, 64, 8000, (7936, 7808, 5300, 2432, 768, 640, 127)),
    (torch.bfloat16, 60, 16, 14000, (13440, 2049, 100)),
    (torch.float32, 3, 32, 3000, (2999, 2500, 1300, 700, 128, 5)),
])
def test_prefill_workspace_of_the_longest_prompt(stq, kind, H, d, longest, lengths):
    """A server's one workspace, made for the longest prompt, serves the shorter ones."""
    need = stq.decay_prefill_workspace_bytes(1, H, longest, d, kind)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)
    for i, T in enumerate(lengths):
        q, k, v, alpha, slots, states = (x.to(DEV) for x in make(1, H, T, d, kind, seed=60 + i, half=200.0))
        o_ref, S_ref, m, A = recurrence(q, k, v, alpha, states[slots.long()])
        o = torch.empty(1, H, T, d, device=DEV)
        stq.decay_prefill(states, slots, q, k, v, alpha, o, workspace=ws)
        close(o, o_ref, m, T, d, f"o of {T} tokens")
        close(states[slots.long()], S_ref, A, T, d, f"states behind {T} tokens")


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("kind,T", [(torch.bfloat16, 2000), (torch.float32, 700), (torch.bfloat16, 20)])
def test_prompts_keep_the_streams_order(stq, kind, T, captured):
    """Prompts (in segments, where they are long), each right behind kernels that write its inputs and lengths,
    one of them a call of the library, and in front of ones that read its outputs: without a wait between, and
    with one behind every operation."""
    B, H, d, steps = 2, 2, 64, 6
    g = torch.Generator(device=DEV).manual_seed(9)
    noise = [0.2 * torch.randn(B, H, T, d, generator=g, device=DEV) for _ in range(steps)]
    need = stq.decay_prefill_workspace_bytes(B, H, T, d, kind)
    assert (need > 0) == (T > 100)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV) if need else None
    states, slots = torch.zeros(B, H, d, d, device=DEV), torch.arange(B, dtype=torch.int32, device=DEV)
    x, o, one = (torch.zeros(B, H, n, d, device=DEV) for n in (T, T, 1))
    gates, lens = torch.zeros(B, H, T, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV)
    kept, status = torch.zeros(steps, B, H, T, d, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    q, k = (torch.zeros(B, H, T, d, dtype=kind, device=DEV) for _ in range(2))

    def body(do):
        for s in range(steps):
            do(lambda: torch.tanh(noise[s] + one, out=x))
            do(lambda: q.copy_(x))
            do(lambda: k.copy_(x.flip(3) * 0.1))
            do(lambda: gates.copy_(torch.sigmoid(x[..., 0] + 3)))
            do(lambda: lens.copy_((one[:, 0, 0, 0].abs() * 5000).int().clamp(max=9).neg() + T))
            do(lambda: stq.decay_prefill(states, slots, q, k, q, gates, o, lens=lens, workspace=ws, status=status))
            do(lambda: stq.decay_step(states, slots, *(t[:, :, 0].contiguous() for t in (q, k, q)), gates[:, :, 0].contiguous(),
                                      one.view(B, H, d), status=status))
            do(lambda: stq.decay_prefill(states, slots, q, k, q, gates, o, lens=lens, workspace=ws, status=status))
            do(lambda: kept[s].copy_(o))

    tensors = [states, x, o, one, gates, lens, kept, q, k, status]
    first = [t.clone() for t in tensors]

    def start():
        for t, was in zip(tensors, first):
            t.copy_(was)
        torch.cuda.synchronize()

    def waited(op):
        op()
        torch.cuda.synchronize()

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
    assert status.item() == 0 and lens.min() < T  # the lengths hang on the outputs before
    for got, w in zip(tensors, want):
        assert torch.equal(got, w)


@pytest.mark.parametrize("H,d,T", [(1, 128, 87), (1, 128, 88), (30, 128, 55), (30, 128, 56), (60, 128, 31), (60, 128, 32),
                                   (3, 64, 63), (3, 64, 64), (3, 32, 103), (3, 32, 104), (300, 32, 127), (300, 32, 128),
                                   (600, 32, 223), (600, 32, 224), (3, 16, 127), (3, 16, 128), (3, 16, 256), (3, 16, 257),
                                   (3, 16, 1500), (150, 16, 200), (1, 16, 24575), (1, 16, 24576)])
@pytest.mark.parametrize("ws", [True, False])
def test_prefill_forms_meet(stq, H, d, T, ws):
    """On both sides of the lengths at which bf16 prompts go by chunks, for few heads and many."""
    check(stq, 1, H, T, d, torch.bfloat16, half=100.0, seed=71, ws=ws)


@pytest.mark.parametrize("kind,T,d", [(torch.float32, 1, 32), (torch.float32, 3, 16), (torch.bfloat16, 40, 16), (torch.bfloat16, 130, 16)])
def test_more_heads_than_a_grid_dimension(stq, kind, T, d):
    """More (request, head) pairs than 32768, with requests of several lengths among them."""
    B, H = 11, 3001
    check(stq, B, H, T, d, kind, step=T == 1, lens=None if T == 1 else [T, 0, 1] + [T] * 7 + [T - 1], seed=81)
