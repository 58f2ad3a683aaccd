"""The 8-bit cache calls where they are most easily wrong, without a GPU: plans
and refusals of the C entry points, and what the Python calls do around them."""
import ctypes

import pytest
import torch

import cross_layer_shared_b200 as sa
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
