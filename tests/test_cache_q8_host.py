"""The 8-bit cache without a GPU: the oracle's code format against its
definition, and what the entry points refuse before any launch."""
import ctypes

import numpy as np
import pytest
import torch

import cross_layer_shared_b200 as sa
from cross_layer_shared_b200 import build
from oracle import q8

FAKE = ctypes.c_void_p(0x7F0000001000)  # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x7F0000001008)
FAKE_WS = ctypes.c_void_p(0x7F0000002000)
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    build.build()
    return sa.lib()


def test_oracle_codes_are_e4m3():
    table = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(q8.VALUES, table, equal_nan=True)
    finite = np.flatnonzero(~np.isnan(q8.VALUES))
    assert np.array_equal(q8.encode(q8.VALUES[finite]), finite)
    # ties to the even code, and the ends of the range
    for c in range(126):
        tie = (q8.VALUES[c] + q8.VALUES[c + 1]) / 2
        even = c if c % 2 == 0 else c + 1
        assert q8.encode(tie) == even and q8.encode(-tie) == even | 0x80
        assert q8.encode(np.nextafter(tie, 0)) == c and q8.encode(np.nextafter(tie, 1e9)) == c + 1
    assert q8.encode(1e30) == 126 and q8.encode(-np.inf) == 254 and q8.encode(np.nan) & 127 == 127


def test_oracle_scale_is_the_smallest_power_of_two():
    for amax, want in ((0.0, 2.0 ** -126), (448.0, 1.0), (np.nextafter(448.0, 500.0), 2.0), (224.0, 0.5),
                       (1.0, 2.0 ** -8), (3.3e38, 2.0 ** 120), (1e-45, 2.0 ** -126)):
        assert q8.scale_of(amax) == want


def test_oracle_append_by_pieces_keeps_the_scale_and_requantises():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((100, 2, 64)) * np.exp(rng.standard_normal((100, 1, 1)))
    one = [np.zeros((2, 128, 64), np.uint8), np.zeros((2, 2))]
    many = [np.zeros((2, 128, 64), np.uint8), np.zeros((2, 2))]
    q8.append(*one, x, 100)
    at = 0
    for n in (1, 2, 60, 0, 1, 36):
        q8.append(*many, x[at:at + n], at + n)
        at += n
    assert np.array_equal(one[1], many[1])
    v1, v2 = q8.values(*one), q8.values(*many)
    step = np.repeat(one[1], 64, -1)[..., None] * 2.0 ** -9
    assert (np.abs(v1 - v2) <= np.maximum(np.abs(v1) / 8, step)).all()  # rounded twice at most
    assert (np.abs(v1[:, :100] - x.transpose(1, 0, 2)) <= np.maximum(np.abs(v1[:, :100]) / 16, step[:, :100] / 2)).all()


# ------------------------------------------------------------------ refusals
def append(lib, new_K=FAKE, sK=1024, new_V=FAKE, sV=1024, dt=0, n_rows=4, new_off=FAKE, max_new=2, K8=FAKE, Ks=FAKE,
           V8=FAKE, Vs=FAKE, off=FAKE, ln=FAKE, B=2, n_tokens=256, Hkv=8, d=128, ws=FAKE_WS, wsb=4096):
    return lib.sa_cache_append_q8(new_K, sK, new_V, sV, dt, n_rows, new_off, max_new, K8, Ks, V8, Vs, off, ln, B,
                                  n_tokens, Hkv, d, ws, wsb, None)


def read(lib, K8=FAKE, Ks=FAKE, V8=FAKE, Vs=FAKE, off=FAKE, ln=FAKE, B=2, n_tokens=256, S_max=128, Hkv=8, d=128,
         idx=FAKE, k=16, out_off=None, n_out=0, K=FAKE, V=FAKE, dt=0, ws=FAKE_WS, wsb=4096):
    return lib.sa_cache_read_q8(K8, Ks, V8, Vs, off, ln, B, n_tokens, S_max, Hkv, d, idx, k, out_off, n_out, K, V, dt,
                                ws, wsb, None)


def index(lib, q=FAKE, w=FAKE, K8=FAKE, Ks=FAKE, off=FAKE, ln=FAKE, B=2, n_tokens=256, S_max=128, H=16, d=128,
          scores=FAKE, ld=128, ws=FAKE_WS, wsb=4096):
    return lib.sa_index_score_q8(q, w, K8, Ks, off, ln, B, n_tokens, S_max, H, d, scores, ld, ws, wsb, None)


def attn(lib, Q=FAKE, K8=FAKE, Ks=FAKE, V8=FAKE, Vs=FAKE, off=FAKE, ln=FAKE, idx=FAKE, L=1, B=2, n_tokens=256,
         S_max=128, Hq=32, Hkv=8, d=128, k=16, scale=0.1, O=FAKE, dt=0, ws=FAKE_WS, wsb=BIG):
    return lib.sa_decode_attn_q8(Q, K8, Ks, V8, Vs, off, ln, idx, L, B, n_tokens, S_max, Hq, Hkv, d, k, scale, O, dt,
                                 ws, wsb, None)


COMMON = [  # of all four: arguments, status, a word of the message
    (dict(B=-1), sa.SA_ERR_INVALID_ARG, b"B"),
    (dict(B=4097), sa.SA_ERR_INVALID_ARG, b"B"),
    (dict(n_tokens=100), sa.SA_ERR_INVALID_ARG, b"multiple of 64"),
    (dict(n_tokens=1 << 31), sa.SA_ERR_INVALID_ARG, b"multiple of 64"),
    (dict(K8=None), sa.SA_ERR_INVALID_ARG, b"NULL"),
    (dict(Ks=None), sa.SA_ERR_INVALID_ARG, b"NULL"),
    (dict(off=None), sa.SA_ERR_INVALID_ARG, b"NULL"),
    (dict(ln=None), sa.SA_ERR_INVALID_ARG, b"NULL"),
    (dict(K8=ODD), sa.SA_ERR_INVALID_ARG, b"aligned"),
    (dict(Ks=ctypes.c_void_p(0x7F0000001002)), sa.SA_ERR_INVALID_ARG, b"aligned"),
    (dict(wsb=100), sa.SA_ERR_WORKSPACE, b""),
    (dict(ws=None), sa.SA_ERR_WORKSPACE, b""),
]
PAIR = [
    (dict(Hkv=0), sa.SA_ERR_INVALID_ARG, b"Hkv"),
    (dict(V8=None), sa.SA_ERR_INVALID_ARG, b""),
    (dict(Vs=None), sa.SA_ERR_INVALID_ARG, b"together"),
    (dict(V8=ODD), sa.SA_ERR_INVALID_ARG, b"aligned"),
]
APPEND = [
    (dict(d=96), sa.SA_ERR_UNSUPPORTED, b"d=96"),
    (dict(dt=7), sa.SA_ERR_INVALID_ARG, b"in_dtype"),
    (dict(max_new=-1), sa.SA_ERR_INVALID_ARG, b"negative"),
    (dict(n_rows=-1), sa.SA_ERR_INVALID_ARG, b"negative"),
    (dict(new_off=None), sa.SA_ERR_INVALID_ARG, b"one row"),
    (dict(new_V=None), sa.SA_ERR_INVALID_ARG, b"together"),
    (dict(sK=1016), sa.SA_ERR_INVALID_ARG, b"strides"),
    (dict(sV=1028), sa.SA_ERR_INVALID_ARG, b"strides"),
    (dict(new_K=None), sa.SA_ERR_INVALID_ARG, b"NULL"),
    (dict(new_K=ODD), sa.SA_ERR_INVALID_ARG, b"aligned"),
    (dict(new_V=ODD), sa.SA_ERR_INVALID_ARG, b"aligned"),
]
READ = [
    (dict(d=80), sa.SA_ERR_UNSUPPORTED, b"d=80"),
    (dict(dt=3), sa.SA_ERR_INVALID_ARG, b"out_dtype"),
    (dict(k=-1), sa.SA_ERR_INVALID_ARG, b"negative"),
    (dict(S_max=-1), sa.SA_ERR_INVALID_ARG, b"negative"),
    (dict(n_out=-1), sa.SA_ERR_INVALID_ARG, b"negative"),
    (dict(out_off=FAKE), sa.SA_ERR_INVALID_ARG, b"either"),
    (dict(idx=None), sa.SA_ERR_INVALID_ARG, b"either"),
    (dict(V=None), sa.SA_ERR_INVALID_ARG, b"together"),
    (dict(K=None), sa.SA_ERR_INVALID_ARG, b"NULL"),
    (dict(K=ODD), sa.SA_ERR_INVALID_ARG, b"aligned"),
]
INDEX = [
    (dict(S_max=-1), sa.SA_ERR_INVALID_ARG, b"S_max"),
    (dict(ld=100), sa.SA_ERR_INVALID_ARG, b"ld"),
    (dict(H=65), sa.SA_ERR_UNSUPPORTED, b""),
    (dict(d=96), sa.SA_ERR_UNSUPPORTED, b""),
    (dict(q=None), sa.SA_ERR_INVALID_ARG, b"NULL"),
    (dict(scores=None), sa.SA_ERR_INVALID_ARG, b"NULL"),
]
ATTN = [
    (dict(L=0), sa.SA_ERR_INVALID_ARG, b"L_g"),
    (dict(B=0), sa.SA_ERR_INVALID_ARG, b"B"),
    (dict(S_max=-1), sa.SA_ERR_INVALID_ARG, b"S_max"),
    (dict(k=0), sa.SA_ERR_INVALID_ARG, b"k=0"),
    (dict(idx=None), sa.SA_ERR_INVALID_ARG, b"k=16"),
    (dict(d=64), sa.SA_ERR_UNSUPPORTED, b"d=64"),
    (dict(Hq=30), sa.SA_ERR_INVALID_ARG, b"multiple"),
    (dict(Hq=8 * 129), sa.SA_ERR_UNSUPPORTED, b"128"),
    (dict(dt=2), sa.SA_ERR_INVALID_ARG, b"out_dtype"),
    (dict(Q=None), sa.SA_ERR_INVALID_ARG, b"NULL"),
    (dict(O=ODD), sa.SA_ERR_INVALID_ARG, b"aligned"),
    (dict(scale=0.0), sa.SA_ERR_INVALID_ARG, b"scale"),
    (dict(scale=float("inf")), sa.SA_ERR_INVALID_ARG, b"scale"),
    (dict(scale=float("nan")), sa.SA_ERR_INVALID_ARG, b"scale"),
]
REFUSALS = [(f, *c) for f, cases in ((append, COMMON + PAIR + APPEND), (read, COMMON + PAIR + READ),
                                     (index, COMMON + INDEX), (attn, COMMON + PAIR + ATTN)) for c in cases]


@pytest.mark.parametrize("call,kw,status,word", REFUSALS,
                         ids=[f"{f.__name__}-{'-'.join(kw)}-{i}" for i, (f, kw, _, _) in enumerate(REFUSALS)])
def test_refusals(lib, call, kw, status, word):
    assert call(lib, **kw) == status
    assert word in lib.sa_last_error()


def test_nothing_to_do_is_fine(lib):
    assert append(lib, B=0) == append(lib, max_new=0) == append(lib, n_rows=0) == sa.SA_OK
    assert read(lib, B=0) == read(lib, k=0) == read(lib, idx=None, k=0, out_off=FAKE, n_out=0) == sa.SA_OK
    assert index(lib, B=0, n_tokens=0) == index(lib, S_max=0, ld=0) == sa.SA_OK


def test_workspace_size_covers_every_key_split(lib):
    size = sa.decode_attn_q8_workspace_size
    assert size(1, 600, 64 * 600, 64, 8, 8, 128, 0) == sa.WS_HEADER_BYTES  # more units than counters: no split
    # slices of many rows merge as a cluster, in shared memory
    assert size(24, 4, 4 * 131072, 131072, 32, 8, 128, 2048) == sa.WS_HEADER_BYTES
    for L, B, S, Hq, Hkv, k in ((1, 1, 131072, 8, 1, 0), (12, 1, 131072, 8, 1, 0), (1, 2, 20000, 16, 2, 0)):
        n = size(L, B, B * (S + 63) // 64 * 64, S, Hq, Hkv, 128, k)
        assert sa.WS_HEADER_BYTES < n < 1 << 28
        assert attn(lib, L=L, B=B, n_tokens=B * (S + 63) // 64 * 64, S_max=S, Hq=Hq, Hkv=Hkv, k=k,
                    idx=FAKE if k else None, wsb=n - 1) == sa.SA_ERR_WORKSPACE


def test_python_calls_refuse_what_is_not_on_the_gpu():
    c, s = torch.zeros((128, 128), dtype=torch.float8_e4m3fn), torch.ones(2)
    off, ln = torch.tensor([0, 128]), torch.tensor([5], dtype=torch.int32)
    with pytest.raises(ValueError, match="new_K"):
        sa.cache_append_q8(torch.zeros((1, 1, 128)), None, c, s, None, None, off, ln)
    with pytest.raises(ValueError, match="K8"):
        sa.cache_read_q8(c, s, None, None, off, ln, 128, 1, out_off=off, n_out=128)
    with pytest.raises(ValueError, match="qI"):
        sa.index_score_q8(torch.zeros((1, 4, 128), dtype=torch.bfloat16), torch.ones((1, 4)), c, s, off, ln, 128)
    with pytest.raises(ValueError, match="Q"):
        sa.decode_attn_q8(torch.zeros((1, 1, 4, 128), dtype=torch.bfloat16), c, s, c, s, off, ln, 128, 1, 0.1)
    for pat in ("SF", "", "FX"):
        n = len(pat)
        with pytest.raises(ValueError, match="letters"):
            sa.decode_step_q8(pat, [None] * n, [None] * n, [None] * n, [(c, s)] * n, [(c, s)] * n, off, ln, 128, 16,
                              torch.zeros((n, 1, 4, 128), dtype=torch.bfloat16), 1, 0.1)
    with pytest.raises(ValueError, match="one entry per"):
        sa.decode_step_q8("FS", [None], [None], [None], [(c, s)], [(c, s)], off, ln, 128, 16,
                          torch.zeros((2, 1, 4, 128), dtype=torch.bfloat16), 1, 0.1)
