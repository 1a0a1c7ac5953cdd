"""Host-side checks (no GPU) of the calls for the layers next to the quantized ones: decayed linear
attention, page plans, cache writes and paged attention. Bad arguments are refused before anything is
enqueued, so the pointers here are never dereferenced."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p
FAKE, ODD4, ODD2 = P(0x10000), P(0x10004), P(0x10002)
OK, INVALID, UNSUPPORTED = 0, 1, 2


@pytest.fixture(scope="module")
def stq():
    from quantized_linear_attention_stq_b200 import build

    build.build()
    import quantized_linear_attention_stq_b200 as m

    return m


def step(L, B=2, H=3, d=64, dt=1, states=FAKE, n=4, slots=FAKE, q=FAKE, k=FAKE, v=FAKE, alpha=FAKE, o=FAKE):
    return L.stq_decay_step(B, H, d, dt, states, n, slots, q, k, v, alpha, o, None, None)


def prefill(L, B=2, H=3, T=5, d=64, dt=1, states=FAKE, n=4, slots=FAKE, q=FAKE, k=FAKE, v=FAKE, alpha=FAKE, lens=None,
            o=FAKE, ws=None, wsn=0):
    return L.stq_decay_prefill(B, H, T, d, dt, states, n, slots, q, k, v, alpha, lens, o, ws, wsn, None, None)


@pytest.mark.parametrize("call", [step, prefill])
def test_decay_refusals(stq, call):
    L = stq.lib()
    for bad in (dict(B=-1), dict(H=0), dict(dt=2), dict(n=-1), dict(states=None), dict(slots=None), dict(q=None),
                dict(k=None), dict(v=None), dict(alpha=None), dict(o=None), dict(states=ODD4), dict(q=ODD4),
                dict(k=ODD4), dict(v=ODD4), dict(o=ODD4), dict(alpha=ODD2), dict(slots=ODD2)):
        assert call(L, **bad) == INVALID, bad
    for d in (0, 8, 96, 256):
        assert call(L, d=d) == UNSUPPORTED
    assert call(L, B=1 << 20, H=1 << 12) == UNSUPPORTED  # more (request, head) pairs than int32 counts
    # no work: nothing is looked at
    assert call(L, B=0, states=None, slots=None, q=None, k=None, v=None, alpha=None, o=None) == OK


def test_decay_prefill_refusals(stq):
    L = stq.lib()
    assert prefill(L, T=-1) == INVALID
    assert prefill(L, lens=ODD2) == INVALID
    assert prefill(L, T=0, states=None, q=None, o=None) == OK
    need = stq.decay_prefill_workspace_bytes(1, 2, 100000, 128, torch.bfloat16)
    if need:
        assert prefill(L, B=1, H=2, T=100000, d=128, ws=FAKE, wsn=need - 1) == INVALID
        assert prefill(L, B=1, H=2, T=100000, d=128, ws=P(0x10010), wsn=need) == INVALID
    for B, H, T, d in ((0, 2, 5, 64), (2, 0, 5, 64), (2, 2, 0, 64), (2, 2, 5, 63), (-1, -1, -1, -1)):
        assert stq.decay_prefill_workspace_bytes(B, H, T, d, torch.bfloat16) == 0
    with pytest.raises(TypeError):
        stq.decay_prefill_workspace_bytes(1, 1, 1, 64, torch.float16)


def plan(L, B=2, W=3, page=16, table=FAKE, lens=FAKE, fresh=FAKE, free=FAKE, F=9, head=FAKE, smap=FAKE, N=8,
         starts=FAKE, lens_out=FAKE, head_out=FAKE):
    return L.stq_page_plan(B, W, page, table, lens, fresh, free, F, head, smap, N, starts, lens_out, head_out, None, None)


def test_plan_refusals(stq):
    L = stq.lib()
    for bad in (dict(B=-1), dict(W=-1), dict(page=0), dict(F=-1), dict(N=-1), dict(table=None), dict(lens=None),
                dict(fresh=None), dict(free=None), dict(head=None), dict(smap=None), dict(starts=None),
                dict(lens_out=None), dict(head_out=None), dict(table=ODD2), dict(lens=ODD2), dict(fresh=ODD2),
                dict(free=ODD2), dict(head=ODD2), dict(smap=ODD2), dict(starts=ODD2), dict(lens_out=ODD2),
                dict(head_out=ODD2)):
        assert plan(L, **bad) == INVALID, bad


def write(L, N=3, H=2, d=64, dt=1, page=16, n=5, kp=FAKE, vp=FAKE, smap=FAKE, k=FAKE, v=FAKE, ks=128, vs=128):
    return L.stq_page_write(N, H, d, dt, page, n, kp, vp, smap, k, v, ks, vs, None, None)


def test_write_refusals(stq):
    L = stq.lib()
    for bad in (dict(N=-1), dict(H=0), dict(dt=2), dict(page=0), dict(n=-1), dict(kp=None), dict(vp=None),
                dict(smap=None), dict(k=None), dict(v=None), dict(kp=ODD4), dict(vp=ODD4), dict(k=ODD4), dict(v=ODD4),
                dict(smap=ODD2), dict(ks=127), dict(vs=64), dict(ks=132), dict(vs=129)):
        assert write(L, **bad) == INVALID, bad
    assert write(L, d=48) == UNSUPPORTED
    assert write(L, page=1 << 20, n=1 << 12) == UNSUPPORTED  # slots past int32
    assert write(L, N=0, kp=None, vp=None, smap=None, k=None, v=None) == OK


def attend(L, B=2, Hq=4, Hkv=2, d=64, dt=1, page=16, n=5, W=3, q=FAKE, kp=FAKE, vp=FAKE, table=FAKE, lens=FAKE,
           scale=1.0, o=FAKE, ws=None, wsn=0):
    return L.stq_paged_attention(B, Hq, Hkv, d, dt, page, n, W, q, kp, vp, table, lens, scale, o, ws, wsn, None, None)


def test_attention_refusals(stq):
    L = stq.lib()
    for bad in (dict(B=-1), dict(Hq=0), dict(Hkv=0), dict(Hq=3), dict(dt=2), dict(page=0), dict(n=-1), dict(W=-1),
                dict(q=None), dict(kp=None), dict(vp=None), dict(table=None), dict(lens=None), dict(o=None),
                dict(q=ODD4), dict(kp=ODD4), dict(vp=ODD4), dict(o=ODD4), dict(table=ODD2), dict(lens=ODD2),
                dict(scale=float("inf")), dict(scale=float("nan"))):
        assert attend(L, **bad) == INVALID, bad
    need = stq.paged_attention_workspace_bytes(2, 4, 64, 2)
    assert need > 0 and need % 4 == 0
    assert attend(L, ws=FAKE, wsn=need - 1) == INVALID
    assert attend(L, ws=P(0x10010), wsn=need) == INVALID
    assert attend(L, d=256) == UNSUPPORTED
    assert attend(L, page=1 << 16, W=1 << 16) == UNSUPPORTED  # positions past int32
    assert attend(L, B=0, q=None, kp=None, vp=None, table=None, lens=None, o=None) == OK
    for args in ((0, 4, 64, 2), (2, 3, 64, 2), (2, 4, 64, 0), (2, 1, 64, 2)):
        assert stq.paged_attention_workspace_bytes(*args) == 0


def test_binding_checks(stq):
    """Types, shapes, contiguity and device are checked before the library is called."""
    f, i = torch.float32, torch.int32
    z = lambda *s, t=f: torch.zeros(*s, dtype=t)  # noqa: E731
    good = dict(states=z(3, 2, 16, 16), slots=z(1, t=i), q=z(1, 2, 16), k=z(1, 2, 16), v=z(1, 2, 16), alpha=z(1, 2),
                o=z(1, 2, 16))
    for name, t, err in (("q", z(2, 16), ValueError), ("k", z(1, 2, 32), ValueError), ("v", z(1, 2, 16, t=torch.bfloat16), TypeError),
                         ("q", z(1, 2, 16, t=torch.float16), TypeError), ("states", z(2, 16, 16), ValueError),
                         ("states", z(3, 1, 16, 16), ValueError), ("slots", z(2, t=i), ValueError),
                         ("slots", z(1, t=torch.int64), TypeError), ("alpha", z(1, 1), ValueError),
                         ("o", z(1, 2, 16, t=torch.bfloat16), TypeError), ("q", None, TypeError)):
        with pytest.raises(err):
            stq.decay_step(**{**good, name: t})
    with pytest.raises(ValueError):  # everything in order, but not on a CUDA device
        stq.decay_step(**good)
    with pytest.raises(ValueError):
        stq.decay_prefill(**good)
    k = z(4, 2, 16)
    pages = z(3, 2, 8, 16)
    for bad in (dict(k=z(4, 2, 32)[..., ::2]), dict(v=z(4, 1, 16)), dict(k_pages=z(3, 1, 8, 16)),
                dict(v_pages=z(3, 2, 8, 32)), dict(slot_map=z(3, t=i)), dict(k=z(1, 2, 16).expand(4, 2, 16))):
        with pytest.raises(ValueError):
            stq.page_write(**{**dict(k_pages=pages, v_pages=pages, slot_map=z(4, t=i), k=k, v=k), **bad})
    att = dict(q=z(2, 4, 16), k_pages=pages, v_pages=pages, table=z(2, 5, t=i), lens=z(2, t=i), o=z(2, 4, 16), scale=1.0)
    for bad in (dict(q=z(8, 16)), dict(table=z(3, 5, t=i)), dict(lens=z(3, t=i)), dict(o=z(2, 4, 8)),
                dict(v_pages=z(2, 2, 8, 16)), dict(workspace=z(1)), dict(q=z(2, 16, 4).transpose(1, 2))):
        with pytest.raises(ValueError):
            stq.paged_attention(**{**att, **bad})
    pl = dict(table=z(2, 5, t=i), lens=z(2, t=i), fresh=z(2, t=i), free_pages=z(9, t=i), free_head=z(1, t=i),
              slot_map=z(8, t=i), starts=z(3, t=i), lens_out=z(2, t=i), head_out=z(1, t=i), page_size=4)
    for bad in (dict(table=z(10, t=i)), dict(lens=z(3, t=i)), dict(starts=z(2, t=i)), dict(free_pages=z(3, 3, t=i)),
                dict(head_out=z(2, t=i))):
        with pytest.raises(ValueError):
            stq.page_plan(**{**pl, **bad})


def test_compiled_binding_leaves_the_unusual_to_python(stq):
    """The compiled module answers -1, without a call, to all that is not a contiguous CUDA tensor of the
    expected kind, and Python then says what is wrong."""
    from quantized_linear_attention_stq_b200 import _binding as b

    z = lambda *s, t=torch.float32: torch.zeros(*s, dtype=t)  # noqa: E731
    i = torch.int32
    step = [z(3, 2, 16, 16), z(1, t=i), z(1, 2, 16), z(1, 2, 16), z(1, 2, 16), z(1, 2), z(1, 2, 16), None, None]
    calls = {
        "decay_step": step,
        "decay_prefill": [step[0], step[1]] + [z(1, 2, 4, 16)] * 3 + [z(1, 2, 4), z(1, 2, 4, 16), None, None, None, None],
        "page_plan": [z(1, 2, t=i), z(1, t=i), z(1, t=i), z(4, t=i), z(1, t=i), z(3, t=i), z(2, t=i), z(1, t=i), z(1, t=i),
                      16, None, None],
        "page_write": [z(2, 1, 4, 16), z(2, 1, 4, 16), z(3, t=i), z(3, 1, 16), z(3, 1, 16), None, None],
        "paged_attention": [z(1, 2, 16), z(2, 1, 4, 16), z(2, 1, 4, 16), z(1, 2, t=i), z(1, t=i), z(1, 2, 16), 1.0, None,
                            None, None],
    }
    for name, args in calls.items():
        f = getattr(b, name)
        assert f(*args) == -1, name
        for n in range(len(args)):
            assert f(*args[:n], "x", *args[n + 1:]) == -1
            assert f(*args[:n], None, *args[n + 1:]) == -1
        with pytest.raises(TypeError):
            f(*args, None)
        with pytest.raises(TypeError):
            f()


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("H", [1, 2, 5, 16, 31, 60, 71, 90, 149, 170, 197, 300, 900])
def test_decay_prefill_workspace_never_falls_with_the_length(stq, H, kind):
    """One workspace, made for the longest prompt, serves every shorter one."""
    for d in (16, 128):
        last = 0
        for T in [*range(1, 9000, 61), *range(9000, 90000, 1277), 1 << 20, 1 << 24, (1 << 31) - 1]:
            need = stq.decay_prefill_workspace_bytes(1, H, T, d, kind)
            assert need >= last, (T, d)
            last = need
    assert stq.decay_prefill_workspace_bytes(1, H, 127, 128, kind) == 0


def test_sizes_past_int32_are_refused(stq):
    """The library's sizes are int32: what passes them is named, not cut."""
    meta = lambda *s, t=torch.int32: torch.empty(*s, dtype=t, device="meta")  # noqa: E731
    big, f = 1 << 32, torch.float32
    pl = dict(table=meta(2, 5), lens=meta(2), fresh=meta(2), free_pages=meta(9), free_head=meta(1), slot_map=meta(8),
              starts=meta(3), lens_out=meta(2), head_out=meta(1), page_size=4)
    for name, bad in (("page_size", dict(page_size=big + 16)), ("page_size", dict(page_size=16 - big)),
                      ("free_pages", dict(free_pages=meta(big + 9))), ("slot_map", dict(slot_map=meta(1 << 31))),
                      ("table", dict(table=meta(2, big)))):
        with pytest.raises(ValueError, match=f"{name}.* past int32"):
            stq.page_plan(**{**pl, **bad})
    with pytest.raises(ValueError, match="page_size.* past int32"):
        stq.page_write(*[meta(1, 2, big + 4, 16, t=f)] * 2, meta(3), *[meta(3, 2, 16, t=f)] * 2)
    with pytest.raises(ValueError, match="N.* past int32"):
        stq.page_write(*[meta(1, 2, 4, 16, t=f)] * 2, meta(big + 3), *[meta(big + 3, 2, 16, t=f)] * 2)
    with pytest.raises(ValueError, match="table.* past int32"):
        stq.paged_attention(meta(2, 4, 16, t=f), *[meta(3, 2, 4, 16, t=f)] * 2, meta(2, big + 1), meta(2), meta(2, 4, 16, t=f), 1.0)
    with pytest.raises(ValueError, match="states.* past int32"):
        stq.decay_step(meta(big + 1, 2, 16, 16, t=f), meta(1), *[meta(1, 2, 16, t=f)] * 3, meta(1, 2, t=f), meta(1, 2, 16, t=f))
    with pytest.raises(ValueError, match="T.* past int32"):
        stq.decay_prefill(meta(3, 1, 16, 16, t=f), meta(1), *[meta(1, 1, big + 5, 16, t=f)] * 3, meta(1, 1, big + 5, t=f),
                          meta(1, 1, big + 5, 16, t=f))
    for args in ((big + 1, 2, 300, 64), (1, big + 2, 300, 64), (1, 2, big + 300, 64), (1, 2, 300, big + 64)):
        with pytest.raises(ValueError, match="past int32"):
            stq.decay_prefill_workspace_bytes(*args, torch.float32)
    for args in ((big + 2, 4, 64, 2), (2, big + 4, 64, 2), (2, 4, big + 64, 2), (2, 4, 64, big + 2)):
        with pytest.raises(ValueError, match="past int32"):
            stq.paged_attention_workspace_bytes(*args)


def test_binding_of_another_torch_is_rebuilt_and_not_used(stq, monkeypatch):
    """The compiled module reads torch's tensors inline: one built against another torch or Python is stale for the
    build, and the calls go through ctypes instead of it; so they do where there is none."""
    import sys

    from quantized_linear_attention_stq_b200 import _binding, api, build

    assert _binding.built_for == build.binding_key() and torch.__version__ in _binding.built_for
    assert not build.binding_stale()
    f, i = torch.float32, torch.int32
    good = [torch.zeros(3, 2, 16, 16), torch.zeros(1, dtype=i), *[torch.zeros(1, 2, 16)] * 3, torch.zeros(1, 2), torch.zeros(1, 2, 16)]
    calls = []
    for name in ("decay_step", "decay_prefill", "page_plan", "page_write", "paged_attention"):
        assert getattr(api._Ctypes, name)(*good) == -1

    def load():
        monkeypatch.setattr(api, "_native", None)
        with pytest.warns(RuntimeWarning, match="ctypes"):
            with pytest.raises(ValueError, match="expected a CUDA device"):  # the Python path's answer to CPU tensors
                stq.decay_step(*good)
        calls.append(api._native)

    with monkeypatch.context() as m:
        m.setattr(build, "binding_key", lambda: "torch 1.0, cpython-27")
        assert build.binding_stale()
        load()
    with monkeypatch.context() as m:
        m.setitem(sys.modules, "quantized_linear_attention_stq_b200._binding", None)
        m.delattr(sys.modules["quantized_linear_attention_stq_b200"], "_binding")
        load()
    assert calls == [api._Ctypes] * 2
    monkeypatch.setattr(api, "_native", None)
    assert api._load() is _binding


@pytest.mark.parametrize("what", ["g++", "Python.h"])
def test_library_is_built_without_the_bindings_tools(stq, monkeypatch, what):
    """Where the compiled module cannot be built the C library still is."""
    from quantized_linear_attention_stq_b200 import build

    if what == "g++":
        which = build.shutil.which
        monkeypatch.setattr(build.shutil, "which", lambda name: None if name == "g++" else which(name))
    else:
        monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": "/nowhere"})
    assert build.build_binding() == build.BINDING  # nothing is missing for one that is up to date
    monkeypatch.setattr(build, "binding_stale", lambda: True)
    with pytest.warns(UserWarning, match="not built"):
        assert build.build() == build.LIB
    with pytest.warns(UserWarning, match="not built"):
        assert build.build_binding(force=True) == ""


def test_workspace_of_another_kind_is_named(stq):
    z = lambda *s, t=torch.float32: torch.zeros(*s, dtype=t)  # noqa: E731
    i = torch.int32
    with pytest.raises(TypeError, match="workspace"):
        stq.paged_attention(z(2, 4, 16), z(3, 2, 8, 16), z(3, 2, 8, 16), z(2, 5, t=i), z(2, t=i), z(2, 4, 16), 1.0, workspace="x")
    with pytest.raises(TypeError, match="workspace"):
        stq.decay_prefill(z(1, 1, 16, 16), z(1, t=i), *[z(1, 1, 2000, 16)] * 3, z(1, 1, 2000), z(1, 1, 2000, 16), workspace=b"x")


def test_attention_refuses_a_scale_that_overflows(stq):
    """Scores are taken in base 2: log2(e) times the scale has to be finite too."""
    L = stq.lib()
    for scale in (2.4e38, -3.4e38):
        assert attend(L, scale=scale) == INVALID
    assert attend(L, scale=2.3e38, d=256) == UNSUPPORTED  # the next check
