"""The 8-bit cache calls where they are most easily wrong, without a GPU: plans
and refusals of the C entry points, and what the Python calls do around them."""
import ast
import ctypes
import inspect
import subprocess

import pytest
import torch

import cross_layer_shared_b200 as sa
from cross_layer_shared_b200 import build
from tests.test_cache_q8_host import append, attn, lib  # noqa: F401


@pytest.mark.parametrize("L,B,Hq,Hkv,n_tokens", [(1, 1, 8, 1, 65536), (6, 1, 320, 80, 4096), (24, 4, 32, 8, 8192),
                                                 (1, 300, 8, 1, 19200)])
def test_a_bound_that_bounds_nothing_plans_like_the_cache(lib, L, B, Hq, Hkv, n_tokens):
    size = sa.decode_attn_q8_workspace_size
    assert size(L, B, n_tokens, 2 ** 31 - 1, Hq, Hkv, 128, 0) == size(L, B, n_tokens, n_tokens, Hq, Hkv, 128, 0)


@pytest.mark.parametrize("kw", [dict(n_tokens=(1 << 30) + 64, k=0, idx=None), dict(k=(1 << 30) + 1)], ids=["tokens", "entries"])
def test_attention_refuses_more_keys_than_it_counts(lib, kw):
    assert attn(lib, **kw) == sa.SA_ERR_UNSUPPORTED
    assert b"2^30" in lib.sa_last_error()


BASE = 0x7F0000100000
CODES = 256 * 8 * 128  # of the default arguments
SCALES = 256 * 8 // 64 * 4


@pytest.mark.parametrize("kw", [dict(V8=0), dict(V8=16), dict(V8=CODES - 16), dict(V8=16 - CODES), dict(Vs=0), dict(Vs=SCALES - 4),
                                dict(Vs=4 - SCALES)], ids=lambda kw: "-".join(f"{k}{v:+d}" for k, v in kw.items()))
def test_append_refuses_one_cache_as_k_and_v(lib, kw):
    """Both are written at the same time.  (Never launched: an overlap is refused.)"""
    at = lambda x: ctypes.c_void_p(x)
    args = dict(K8=at(BASE), V8=at(BASE + 4 * CODES), Ks=at(BASE - 0x10000), Vs=at(BASE - 0x8000))
    for name, base in (("V8", BASE), ("Vs", BASE - 0x10000)):
        if name in kw:
            args[name] = at(base + kw[name])
    assert append(lib, **args) == sa.SA_ERR_INVALID_ARG
    assert b"overlap" in lib.sa_last_error()


class Side:
    """A stream of another library's: its address is all there is."""
    cuda_stream = 1234


def test_what_a_call_allocates_belongs_to_its_stream(monkeypatch):
    """Outputs, temporaries and workspaces that are not given are allocated (and zeroed) on the stream of the call."""
    on, made = [], []
    bf, f8 = torch.bfloat16, torch.float8_e4m3fn
    c, s = torch.zeros((128, 128), dtype=f8), torch.ones(2)
    off, ln = torch.tensor([0, 128]), torch.tensor([5], dtype=torch.int32)
    Q, q, w, x = torch.zeros((1, 1, 4, 128), dtype=bf), torch.zeros((1, 4, 128), dtype=bf), torch.ones((1, 4)), torch.zeros((1, 1, 128))

    class Stream:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            on.append(self.stream)

        def __exit__(self, *a):
            on.pop()

    def recording(make):
        def f(*a, **kw):
            made.append(on[-1] if on else None)
            return make(*a, **{**kw, "device": "cpu"})
        return f

    class Native:  # the compiled marshalling: every call succeeds
        def __getattr__(self, name):
            return lambda *a: 0

    monkeypatch.setattr(sa, "_native", Native())
    monkeypatch.setattr(sa, "topk", lambda *a, **kw: None)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda p: ("stream at", p))
    monkeypatch.setattr(torch.cuda, "stream", Stream)
    monkeypatch.setattr(torch, "empty", recording(torch.empty))
    monkeypatch.setattr(torch, "zeros", recording(torch.zeros))
    calls = {
        1: lambda **kw: sa.cache_append_q8(x, None, c, s, None, None, off, ln, **kw),
        3: lambda **kw: sa.cache_read_q8(c, s, c, s, off, ln, 128, 1, out_off=off, n_out=128, **kw),
        2: lambda **kw: sa.index_score_q8(q, w, c, s, off, ln, 128, **kw),
        -2: lambda **kw: sa.decode_attn_q8(Q, c, s, c, s, off, ln, 128, 1, 0.1, **kw),
        4: lambda **kw: sa.decode_step_q8("F", [q], [w], [(c, s)], [(c, s)], [(c, s)], off, ln, 128, 16, Q, 1, 0.1, **kw),
    }
    for n, call in calls.items():
        for kw, want in ((dict(stream=Side()), ("stream at", 1234)), (dict(), None)):
            made.clear()
            call(**kw)
            assert made == [want] * abs(n)


def test_every_call_with_a_stream_allocates_there():
    for name, f in vars(sa).items():
        if callable(f) and not isinstance(f, type) and name not in ("_empty", "workspace") and f.__module__ == sa.__name__ \
                and "stream" in inspect.signature(f).parameters:
            text = inspect.getsource(f)
            assert "torch.empty(" not in text and "torch.zeros(" not in text, name
            made = ast.walk(ast.parse(text))
            for call in (c for c in made if isinstance(c, ast.Call) and isinstance(c.func, ast.Name)):
                if call.func.id == "_empty":
                    assert getattr(call.args[0], "id", None) == "stream", name
                if call.func.id == "workspace":
                    assert getattr(call.args[-1], "id", None) == "stream", name


@pytest.mark.parametrize("B,Hq,Hkv,S_max", [(1, 64, 8, 8192), (4, 32, 8, 4096), (2, 8, 1, 1000)])
def test_room_to_grow_does_not_change_the_plan(lib, B, Hq, Hkv, S_max):
    """The split goes by the keys there can be (S_max of each sequence), not by the cache's token places."""
    size = sa.decode_attn_q8_workspace_size
    tight = B * (S_max + 63) // 64 * 64
    assert size(1, B, 1 << 20, S_max, Hq, Hkv, 128, 0) == size(1, B, tight, S_max, Hq, Hkv, 128, 0)


# ------------------------------------------------------------------ the build of the marshalling
def test_binding_is_built_again_for_another_torch(monkeypatch, tmp_path):
    built = []

    def gxx(cmd, **kw):
        built.append(cmd[0])
        (tmp_path / "_binding.so.tmp").write_text("")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build.subprocess, "run", gxx)
    build.build_binding()
    build.build_binding()
    assert built == ["g++"]
    monkeypatch.setattr(torch, "__version__", "0.0.0")
    build.build_binding()
    build.build_binding()
    assert built == ["g++"] * 2


def test_libraries_are_built_without_what_the_binding_needs(monkeypatch, tmp_path):
    """A host without g++ or headers still gets libsa and the generator, then the error."""
    done = []
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "SYNTH_LIB", str(tmp_path / "libsasynth.so"))
    monkeypatch.setattr(build, "_build_lib", lambda out, *a: done.append(out))

    def check_call(cmd):
        done.append(cmd[-1])
        (tmp_path / "libsasynth.so.tmp").write_text("")

    def missing(*a, **kw):
        raise FileNotFoundError("g++")

    monkeypatch.setattr(build.subprocess, "check_call", check_call)
    monkeypatch.setattr(build.subprocess, "run", missing)
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_binding.so"))
    with pytest.raises(RuntimeError, match="g\\+\\+"):
        build.build()
    assert done == [build.LIB, build.SYNTH_SRC]
