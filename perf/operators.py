"""What is measured of the operators that serve the layers next to the quantized delta-rule ones.

A hybrid stack mixes linear-attention layers with softmax-attention layers. Five operators serve
the layers that the quantized state does not cover:

  step      linear attention with a decay per head, one token: S <- a S + k v^T, o = S^T q
  prefill   the same recurrence over a prompt
  plan      pages, block table and slot map of a step, from the requests' lengths
  write     the new tokens' keys and values into the paged cache, by the slot map
  attend    attention of one new token per request over the paged cache

``run`` computes an operator in its plain form (elementary torch operations) or, where ``own`` is
true, by the call that a user of the framework makes.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
_DEV = "cuda"


def listed():
    return [
        # one request of a small model: the latency of a single token
        dict(name="step 1x16 d64 fp32", op="step", batch=1, heads=16, d=64, type="fp32"),
        # one 48-head layer of 70 concurrent requests
        dict(name="step 70x48 d128 bf16", op="step", batch=70, heads=48, d=128, type="bf16"),
        # a few short prompts of unequal length, small heads, full-precision inputs
        dict(name="prefill 3x5 T77 d32 fp32", op="prefill", batch=3, heads=5, tokens=77, d=32, type="fp32", ragged=True),
        # the prompt of the prefill workload: 16 requests, 16 heads, 8192 tokens each
        dict(name="prefill 16x16 T8192 d128 bf16", op="prefill", batch=16, heads=16, tokens=8192, d=128, type="bf16", ragged=False),
        # one long document: few heads, work split over the length
        dict(name="prefill 1x16 T65521 d128 bf16", op="prefill", batch=1, heads=16, tokens=65521, d=128, type="bf16", ragged=False),
        # the plan of a decode step
        dict(name="plan 70 decode", op="plan", batch=70, new=1, longest=4096, page=16),
        # the plan of a large batch of prompts
        dict(name="plan 1000 prompts", op="plan", batch=1000, new=1000, longest=2000, page=64),
        # the cache write of a decode step
        dict(name="write 70 decode", op="write", tokens=70, kv_heads=8, d=128, type="bf16", page=16),
        # the cache write of prompts
        dict(name="write 50001 prompt", op="write", tokens=50001, kv_heads=8, d=128, type="bf16", page=64),
        # one request over a short cache, no sharing of key-value heads, full precision
        dict(name="attend 1 L1000 fp32", op="attend", batch=1, heads=8, kv_heads=8, d=64, longest=1000, type="fp32", page=16),
        # 70 requests of very different lengths, four query heads to a key-value head
        dict(name="attend 70 L16384 bf16", op="attend", batch=70, heads=32, kv_heads=8, d=128, longest=16384, type="bf16", page=64),
        # two very long documents, sixteen query heads to a key-value head
        dict(name="attend 2 L500001 bf16", op="attend", batch=2, heads=32, kv_heads=2, d=128, longest=500001, type="bf16", page=16),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["step", "prefill", "plan", "write", "attend"])
    kind = rng.choice(["bf16", "bf16", "fp32"])
    if op == "step":
        return dict(op=op, batch=_log_int(rng, 1, 100), heads=_log_int(rng, 1, 32), d=rng.choice([16, 32, 64, 128]), type=kind)
    if op == "prefill":
        d = rng.choice([16, 32, 64, 128])
        batch, heads = _log_int(rng, 1, 16), _log_int(rng, 1, 32)
        most = (2 ** 26 if kind == "bf16" else 2 ** 23) // (batch * heads * d)  # values of one of q, k, v
        return dict(op=op, batch=batch, heads=heads, tokens=_log_int(rng, 1, max(2, min(32768, most))), d=d, type=kind, ragged=rng.random() < 0.5)
    page = rng.choice([1, 8, 16, 20, 32, 64, 128])
    if op == "plan":
        new = rng.choice([1, _log_int(rng, 2, 700)])
        return dict(op=op, batch=_log_int(rng, 1, 1000), new=new, longest=_log_int(rng, 1, 2000), page=page)
    kv_heads, d = rng.choice([1, 2, 3, 4, 8]), rng.choice([16, 32, 64, 128])
    if op == "write":
        return dict(op=op, tokens=_log_int(rng, 1, 32768), kv_heads=kv_heads, d=d, type=kind, page=page)
    batch = _log_int(rng, 1, 64)
    most = 2 ** 27 // (batch * kv_heads * d)
    return dict(op=op, batch=batch, heads=kv_heads * rng.choice([1, 2, 3, 4, 6, 8, 16]), kv_heads=kv_heads, d=d,
                longest=_log_int(rng, 1, min(200000, most)), type=kind, page=page)


def _lengths(n, longest):
    """n lengths spread over 1..longest, in mixed order; the first is the longest."""
    order = sorted(range(n), key=lambda i: (i * 2654435761) % 4294967296)
    out = [0] * n
    for rank, i in enumerate(order):
        out[i] = max(1, longest - (longest * rank) // n)
    return out


def _attend_lengths(case):
    """Lengths of the cached requests; a batch of more than four ends in a padding request without tokens."""
    lens = _lengths(case["batch"], case["longest"])
    if case["batch"] > 4:
        lens[-1] = 0
    return lens


def _plan_lengths(case):
    """Tokens held and tokens new of every request; one request in seven is new (it holds nothing)."""
    held = [0 if i % 7 == 3 else n for i, n in enumerate(_lengths(case["batch"], case["longest"]))]
    return held, list(reversed(_lengths(case["batch"], case["new"])))


def _prompt_lengths(case):
    return _lengths(case["batch"], case["tokens"]) if case["ragged"] else [case["tokens"]] * case["batch"]


def _pages_of(n, page):
    return -(-n // page)


def _unit(x):
    return x / torch.linalg.vector_norm(x, dim=-1, keepdim=True)


def _int(values):
    return torch.tensor(values, dtype=torch.int32, device=_DEV)


def prepare(case, seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(shape, generator=g, device=_DEV)

    def perm(n):
        return torch.randperm(n, generator=g, device=_DEV).to(torch.int32)

    state = dict(case)
    op = case["op"]
    if op in ("step", "prefill"):
        B, H, d = case["batch"], case["heads"], case["d"]
        kind = _TYPES[case["type"]]
        lead = (B, H) if op == "step" else (B, H, case["tokens"])
        state["q"] = _unit(randn(*lead, d)).to(kind)
        state["k"] = _unit(randn(*lead, d)).to(kind)
        state["v"] = randn(*lead, d).to(kind)
        # half-lives of 1 to 4096 tokens per head, the gate of a token near its head's
        half = torch.exp(torch.rand(H, generator=g, device=_DEV) * math.log(4096.0))
        near = 0.5 + torch.rand(lead, generator=g, device=_DEV)
        state["alpha"] = torch.exp(-near / half.view((1, H) + (1,) * (len(lead) - 2)))
        state["slots"] = perm(B + 3)[:B].contiguous()
        state["states"] = 0.5 * randn(B + 3, H, d, d)
        if op == "prefill":  # every other request starts with an empty state
            state["states"][state["slots"][::2].long()] = 0.0
            state["lens"] = _int(_prompt_lengths(case)) if case["ragged"] else None
        state["o"] = torch.full((*lead, d), -1.0, device=_DEV)
        return state
    page = case["page"]
    if op == "plan":
        held, new = _plan_lengths(case)
        now = [_pages_of(h, page) for h in held]
        then = [_pages_of(h + n, page) for h, n in zip(held, new)]
        width = max(then) + 2
        pages = perm(sum(then) + 5)
        table = torch.full((case["batch"], width), -1, dtype=torch.int32, device=_DEV)
        have = torch.arange(width, device=_DEV)[None, :] < _int(now)[:, None]
        table[have] = pages[: sum(now)]
        state.update(table=table, lens=_int(held), new=_int(new), free=pages[sum(now):].contiguous(), head=_int([0]),
                     lens_out=_int([0] * case["batch"]), head_out=_int([0]),
                     slot_map=_int([0] * (sum(new) + 3)), starts=_int([0] * (case["batch"] + 1)))
        return state
    Hkv, d, kind = case["kv_heads"], case["d"], _TYPES[case["type"]]
    if op == "write":
        n = case["tokens"]
        pages = _pages_of(n, page) + 3
        # keys and values are parts of one projection's rows; one token in sixteen is padding
        both = randn(n, 2 * Hkv * d).to(kind)
        state["k"], state["v"] = (x.view(n, Hkv, d) for x in both.split(Hkv * d, dim=1))
        state["k_pages"], state["v_pages"] = (randn(pages, Hkv, page, d).to(kind) for _ in range(2))
        first = torch.randint(0, 2 * page + 1, (1,), generator=g, device=_DEV)
        slot = torch.arange(n, device=_DEV) + first
        slot = perm(pages).long()[slot // page] * page + slot % page
        pad = torch.rand(n, generator=g, device=_DEV) < 1 / 16
        state["slot_map"] = torch.where(pad, -1, slot).to(torch.int32)
        return state
    lens = _attend_lengths(case)
    held = [_pages_of(n, page) for n in lens]
    width = max(held) + 1
    total = sum(held) + 2
    table = torch.full((case["batch"], width), -1, dtype=torch.int32, device=_DEV)
    have = torch.arange(width, device=_DEV)[None, :] < _int(held)[:, None]
    table[have] = perm(total)[: sum(held)]
    state.update(q=randn(case["batch"], case["heads"], d).to(kind), table=table, lens=_int(lens), scale=1.0 / math.sqrt(d),
                 o=torch.full((case["batch"], case["heads"], d), -1.0, device=_DEV))
    state["k_pages"], state["v_pages"] = (torch.empty(total, Hkv, page, d, dtype=kind, device=_DEV).normal_(generator=g) for _ in range(2))
    return state


def _plain_step(s):
    at = s["slots"].long()
    q, k, v = (s[n].float() for n in "qkv")
    S = s["alpha"][..., None, None] * s["states"][at] + k[..., :, None] * v[..., None, :]
    s["states"][at] = S
    return (S * q[..., :, None]).sum(dim=2), s["states"]


def _plain_prefill(s, chunk=128):
    B, H, T, d = s["q"].shape
    lens = torch.full((B,), T, device=_DEV) if s["lens"] is None else s["lens"].long()
    live = (torch.arange(T, device=_DEV)[None] < lens[:, None])[:, None, :]  # [B][1][T]
    N = -(-T // chunk)

    def cut(x):  # [B][H][T][...] -> [B][H][N][chunk][...], padded with zeros
        pad = x.new_zeros((B, H, N * chunk - T) + x.shape[3:])
        return torch.cat([x, pad], dim=2).view((B, H, N, chunk) + x.shape[3:])

    q, k, v = (cut(torch.where(live[..., None], s[n].float(), 0.0)) for n in "qkv")
    g = cut(torch.where(live, torch.log(s["alpha"].double()), 0.0)).cumsum(dim=3)  # log of the decay since the chunk's start
    keep = torch.ones(chunk, chunk, dtype=torch.bool, device=_DEV).tril()
    decay = torch.exp((g[..., :, None] - g[..., None, :]).masked_fill(~keep, -math.inf)).float()
    o = ((q @ k.transpose(-1, -2)) * decay) @ v
    last = g[..., -1:]
    local = (k * torch.exp(last - g).float()[..., None]).transpose(-1, -2) @ v  # [B][H][N][d][d]
    end = last[..., 0].cumsum(dim=2)  # log of the decay at every chunk's end
    start = end - last[..., 0]
    before = torch.ones(N, N, dtype=torch.bool, device=_DEV).tril(-1)
    carry = torch.exp((start[..., :, None] - end[..., None, :]).masked_fill(~before, -math.inf)).float()
    at = s["slots"].long()
    S0 = s["states"][at]
    flat = local.view(B, H, N, d * d)
    S_in = (carry @ flat).view(B, H, N, d, d) + torch.exp(start).float()[..., None, None] * S0[:, :, None]
    o = o + torch.exp(g).float()[..., None] * (q @ S_in)
    S = torch.exp(end[..., -1]).float()[..., None, None] * S0
    S = S + (torch.exp(end[..., -1:] - end).float()[..., None, :] @ flat).view(B, H, d, d)
    s["states"][at] = S
    return torch.where(live[..., None], o.view(B, H, N * chunk, d)[:, :, :T], s["o"]), s["states"]


def _plain_plan(s):
    page, table, lens, new = s["page"], s["table"], s["lens"].long(), s["new"].long()
    now, then = (lens + page - 1) // page, (lens + new + page - 1) // page
    need = then - now
    upto = need.cumsum(0)
    col = torch.arange(table.shape[1], device=_DEV)[None, :]
    fresh = (col >= now[:, None]) & (col < then[:, None])
    pick = s["head"].long() + (upto - need - now)[:, None] + col
    table = torch.where(fresh, s["free"][pick.clamp(0, s["free"].numel() - 1)], table)
    starts = torch.cat([new.new_zeros(1), new.cumsum(0)])
    n = s["slot_map"].numel()
    i = torch.arange(n, device=_DEV)
    b = torch.searchsorted(starts[1:].contiguous(), i, right=True).clamp(max=new.numel() - 1)
    pos = (lens[b] + i - starts[b]).clamp(min=0, max=table.shape[1] * page - 1)
    slot = table[b, pos // page].long() * page + pos % page
    slot = torch.where(i < starts[-1], slot, -1)
    return dict(table=table, lens_out=(lens + new).int(), head_out=s["head"] + upto[-1].int(), slot_map=slot.int(), starts=starts.int())


def _plain_write(s):
    page = s["page"]
    live = s["slot_map"] >= 0
    slot = s["slot_map"][live].long()
    for pages, rows in ((s["k_pages"], s["k"]), (s["v_pages"], s["v"])):
        pages[slot // page, :, slot % page] = rows[live]
    return s["k_pages"], s["v_pages"]


def _plain_attend(s):
    B, Hq, d = s["q"].shape
    _, Hkv, page, _ = s["k_pages"].shape
    pick = s["table"].clamp(min=0).long()
    W = pick.shape[1]

    def cached(pages):  # [B][Hkv][W * page][d]
        return pages[pick].transpose(1, 2).reshape(B, Hkv, W * page, d).float()

    q = s["q"].float().view(B, Hkv, Hq // Hkv, d)
    score = s["scale"] * (q @ cached(s["k_pages"]).transpose(-1, -2))
    live = torch.arange(W * page, device=_DEV)[None] < s["lens"][:, None]
    score = score.masked_fill(~live[:, None, None], -math.inf)
    top = score.amax(dim=-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)  # a request without tokens: no weights
    p = torch.exp(score - top)
    total = p.sum(dim=-1, keepdim=True)
    return ((p @ cached(s["v_pages"])) / torch.where(total > 0, total, 1.0)).view(B, Hq, d)


_PLAIN = dict(step=_plain_step, prefill=_plain_prefill, plan=_plain_plan, write=_plain_write, attend=_plain_attend)


def _scratch(state, need):
    """The workspace that the program keeps beside its inputs, made at the first pass."""
    if "workspace" not in state:
        state["workspace"] = torch.empty(need, dtype=torch.uint8, device=_DEV) if need else None
    return state["workspace"]


def _own(s):
    import quantized_linear_attention_stq_b200 as stq

    op = s["op"]
    if op == "step":
        stq.decay_step(s["states"], s["slots"], s["q"], s["k"], s["v"], s["alpha"], s["o"])
        return s["o"], s["states"]
    if op == "prefill":
        B, H, T, d = s["q"].shape
        ws = s["workspace"] if "workspace" in s else _scratch(s, stq.decay_prefill_workspace_bytes(B, H, T, d, s["q"].dtype))
        stq.decay_prefill(s["states"], s["slots"], s["q"], s["k"], s["v"], s["alpha"], s["o"], lens=s["lens"], workspace=ws)
        return s["o"], s["states"]
    if op == "plan":
        stq.page_plan(s["table"], s["lens"], s["new"], s["free"], s["head"], s["slot_map"], s["starts"], s["lens_out"],
                      s["head_out"], s["page"])
        return {n: s[n] for n in ("table", "lens_out", "head_out", "slot_map", "starts")}
    if op == "write":
        stq.page_write(s["k_pages"], s["v_pages"], s["slot_map"], s["k"], s["v"])
        return s["k_pages"], s["v_pages"]
    ws = s["workspace"] if "workspace" in s else _scratch(s, stq.paged_attention_workspace_bytes(*s["q"].shape, s["k_pages"].shape[1]))
    stq.paged_attention(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["o"], s["scale"], workspace=ws)
    return s["o"]


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["op"]](state)


def work(case):
    op = case["op"]
    size = 2 if case.get("type") == "bf16" else 4
    if op in ("step", "prefill"):
        B, H, d = case["batch"], case["heads"], case["d"]
        tokens = B if op == "step" else sum(_prompt_lengths(case))
        return dict(bytes=H * (B * 8 * d * d + tokens * (3 * d * size + 4 + 4 * d)), flops=H * tokens * 5 * d * d)
    if op == "plan":
        held, new = _plan_lengths(case)
        fresh = sum(_pages_of(h + n, case["page"]) - _pages_of(h, case["page"]) for h, n in zip(held, new))
        return dict(bytes=4 * (5 * case["batch"] + 2 * fresh + sum(new)), flops=2 * sum(new))
    if op == "write":
        return dict(bytes=case["tokens"] * (4 * case["kv_heads"] * case["d"] * size + 4), flops=0)
    kept = sum(_attend_lengths(case))
    return dict(bytes=kept * 2 * case["kv_heads"] * case["d"] * size + case["batch"] * case["heads"] * case["d"] * (size + 4),
                flops=4 * kept * case["heads"] * case["d"])


def exact(case, seed):
    """The definitions in 64 bits: the recurrence token by token, the attention request by request."""
    op = case["op"]
    s = prepare(case, seed)
    if op == "step":
        slots = s["slots"].long()
        states = s["states"].double()
        S = torch.einsum("bh,bhij->bhij", s["alpha"].double(), states[slots])
        S += torch.einsum("bhi,bhj->bhij", s["k"].double(), s["v"].double())
        states[slots] = S
        return torch.einsum("bhij,bhi->bhj", S, s["q"].double()), states
    if op == "prefill":
        slots = s["slots"].long()
        states, o = s["states"].double(), s["o"].double()
        S = states[slots]
        lens = _prompt_lengths(case)
        count = torch.tensor(lens, device=_DEV)[:, None, None]
        T = case["tokens"]
        if T * max(1, S.numel() / 2 ** 23) > 100000:
            return None
        ragged = min(lens) < T
        for t in range(T):
            q, k, v = (s[n][:, :, t].double() for n in "qkv")
            grown = S * s["alpha"][:, :, t, None, None].double()
            grown += k[..., :, None] * v[..., None, :]
            ot = torch.matmul(q[..., None, :], grown)[..., 0, :]
            if ragged:
                grown = torch.where((t < count)[..., None], grown, S)
                ot = torch.where(t < count, ot, o[:, :, t])
            S = grown
            o[:, :, t] = ot
        states[slots] = S
        return o, states
    if op == "attend":
        out = torch.zeros(case["batch"], case["heads"], case["d"], dtype=torch.float64, device=_DEV)
        share = case["heads"] // case["kv_heads"]
        for b, n in enumerate(_attend_lengths(case)):
            if n:
                at = s["table"][b, : _pages_of(n, case["page"])].long()
                for h in range(case["kv_heads"]):
                    k, v = (s[x][at, h].reshape(-1, case["d"])[:n].double() for x in ("k_pages", "v_pages"))
                    w = torch.softmax(s["scale"] * (s["q"][b, h * share:(h + 1) * share].double() @ k.T), dim=-1)
                    out[b, h * share:(h + 1) * share] = w @ v
        return out
    return None  # whole numbers and copies
