"""The 8-bit cache calls where they are most easily wrong: scales that an
append does not write, bounds of a caller's that bound nothing, layers that
share half of a cache, sizes at the ends.  Oracle and tolerances are those of
test_gpu_cache_q8.py."""
import numpy as np
import pytest
import torch

import cross_layer_shared_b200 as sa
from oracle import q8
from tests.test_gpu_cache_q8 import BF16, F32, Cache, check_attn, dev, filled, i32, i64, ok, picks, rows  # noqa: F401

pytestmark = pytest.mark.gpu


def attend(dev, K, V, lens, Qf, Hkv, idx=None, dt=F32, scale=0.1, S=None):
    """decode_attn_q8 against the oracle; Qf float [L, B, Hq, 128]."""
    L, B, Hq, _ = Qf.shape
    S = max(lens) if S is None else S
    Qt = torch.from_numpy(Qf.astype(np.float32)).to(BF16)
    k = 0 if idx is None else idx.shape[1]
    ws = sa.workspace(sa.decode_attn_q8_workspace_size(L, B, int(K.off[-1]), S, Hq, Hkv, 128, k), dev)
    O = torch.full(Qt.shape, 7.0, dtype=dt, device=dev)
    sa.decode_attn_q8(Qt.to(dev), *K.pair(), *V.pair(), i64(K.off, dev), i32(lens, dev), S, Hkv, scale,
                      idx=None if idx is None else i32(idx, dev), O=O, ws=ws)
    ok(ws)
    assert torch.isfinite(O).all()  # a NaN would pass the comparison below
    check_attn(Qt.float().numpy(), K, V, lens, idx, Hkv, np.float32(scale), O, dt)
    return O


# ------------------------------------------------------------------ scales of a cache from elsewhere
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("e", [-9, -33, -100])  # V scales near 2^-16, 2^-40 and 2^-107
def test_a_zero_v_scale_costs_the_other_tokens_nothing(e, dt, dev):
    """Tokens of a block whose V scale is zero add nothing, and the weights of the others keep their bits, however
    small the others' V scales are: picked so that a pass holds both kinds, and every token, the zero block first."""
    rng = np.random.default_rng(60)
    for Hkv, lens, pick in ((2, [192], 16), (2, [192], 48), (160, [320], 0)):
        K, V = filled(rng, lens, Hkv, 128, dev, strong=[(0, blk, e) for blk in range(5)])
        V.scales[0][:, 0] = 0
        V.upload()
        idx = None if not pick else np.arange(pick)[None] % 3 * 64 + np.arange(pick)[None] // 3
        attend(dev, K, V, lens, rng.standard_normal((2, 1, Hkv, 128)) * 2, Hkv, idx, dt)


def test_scales_below_the_smallest_normal_number(dev):
    """2^-127 and 1.5 * 2^-128 are finite scales too."""
    rng = np.random.default_rng(61)
    K, V = filled(rng, [192], 2, 128, dev)
    V.scales[0][:] = np.array([0.0, 2.0 ** -127, 1.5 * 2.0 ** -128])
    V.upload()
    idx = np.arange(48)[None] % 3 * 64 + np.arange(48)[None] // 3
    O = attend(dev, K, V, [192], rng.standard_normal((1, 1, 4, 128)), 2, idx)
    assert O.abs().max().item() > 1e-37


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("k", [0, 192])
@pytest.mark.parametrize("high", [511.99, 255.999, 448.0, 2.0 ** 9 * (1 - 2.0 ** -24)])
def test_a_scale_just_under_a_power_of_two(high, k, dt, dev):
    """A later block's V scale passes the first one's by as much as the reference allows, times almost two: the
    weights that meet in the second product stay finite."""
    rng = np.random.default_rng(62)
    K, V = filled(rng, [192], 1, 128, dev)
    V.scales[0][:] = np.array([1.0, 1.0, np.float32(high)])
    V.upload()
    idx = np.arange(192)[None] if k else None
    attend(dev, K, V, [192], np.zeros((1, 1, 4, 128)), 1, idx, dt)


# ------------------------------------------------------------------ a step whose layers share half of a cache
@pytest.mark.parametrize("layers", [[("KA", "VA"), ("KA", "VB"), ("KB", "VB")], [("KA", "KA"), ("KA", "VA"), ("VA", "KA")]],
                         ids=["half_shared", "one_cache_as_both"])
def test_step_appends_to_every_listed_cache_once(layers, dev):
    """Layers that share K and not V, V and not K, and layers whose K and V are one cache: each cache gets one row
    per sequence, from the first place that lists it (a layer's K before its V)."""
    rng = np.random.default_rng(63)
    lens, Hkv = [70, 127], 2
    new_lens = [n + 1 for n in lens]
    C = {}
    for name in sorted({name for pair in layers for name in pair}):
        C[name], _ = filled(rng, lens, Hkv, 128, dev)
    KI, _ = filled(rng, lens, 1, 64, dev)
    for c in list(C.values()) + [KI]:  # room for one token more in every sequence
        assert all(n <= cap for n, cap in zip(new_lens, c.caps))
    L = len(layers)
    new_K, new_V = ([rows(rng, 2, Hkv, 128, BF16) for _ in range(L)] for _ in range(2))
    tI, xI = rows(rng, 2, 1, 64, BF16)
    Q = torch.from_numpy(rng.standard_normal((L, 2, 4, 128)).astype(np.float32)).to(BF16)
    qI = torch.from_numpy(rng.standard_normal((2, 4, 64)).astype(np.float32)).to(BF16).to(dev)
    none = [None] * (L - 1)
    O, idx = sa.decode_step_q8("FSS", [qI] + none, [torch.ones((2, 4), device=dev)] + none, [KI.pair()] + none,
                               [C[k].pair() for k, _ in layers], [C[v].pair() for _, v in layers], i64(KI.off, dev),
                               i32(new_lens, dev), 128, 40, Q.to(dev), Hkv, 0.1, out_dtype=F32,
                               new_KI=[tI.to(dev)] + none, new_K=[t.to(dev) for t, _ in new_K],
                               new_V=[t.to(dev) for t, _ in new_V])
    first = {}
    for l, pair in enumerate(layers):
        for name, new in zip(pair, (new_K, new_V)):
            first.setdefault(name, new[l][1])
    for c, x in [(KI, xI)] + [(C[name], x) for name, x in first.items()]:
        for b, n in enumerate(new_lens):
            q8.append(c.codes[b], c.scales[b], x[b:b + 1], n)
        c.check()
    for l, (k, v) in enumerate(layers):
        check_attn(Q[l:l + 1].float().numpy(), C[k], C[v], new_lens, idx.cpu().numpy(), Hkv, np.float32(0.1),
                   O[l:l + 1], F32)


# ------------------------------------------------------------------ sizes at the ends
@pytest.mark.parametrize("L,Hkv,lens", [(6, 80, [130]), (6, 80, [1000]), (1, 80, [300, 70]), (6, 2, [1500, 1])])
def test_a_bound_that_bounds_nothing(L, Hkv, lens, dev):
    """S_max = 2^31 - 1 only says that no length is longer."""
    rng = np.random.default_rng(64)
    K, V = filled(rng, lens, Hkv, 128, dev)
    Qf = rng.standard_normal((L, len(lens), 4 * Hkv, 128))
    attend(dev, K, V, lens, Qf, Hkv, S=2 ** 31 - 1)
    attend(dev, K, V, lens, Qf, Hkv, picks(rng, lens, 100, 0.1), BF16, S=2 ** 31 - 1)


def test_index_keys_up_to_2_31(dev):
    """One sequence of the most token places a cache may have: its last tokens appended, read back and scored."""
    n, d, new = (1 << 31) - 64, 64, 100
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 152 << 30:
        pytest.skip("137 GB of codes, 9 GB of scores and room to compare them")
    rng = np.random.default_rng(65)
    raw = torch.zeros((n, d), dtype=torch.uint8, device=dev)
    K8 = raw.view(torch.float8_e4m3fn)
    Ks = torch.ones(n // 64, device=dev)
    off, ws = i64([0, n], dev), sa.workspace(sa.WS_HEADER_BYTES, dev)
    q = torch.from_numpy(rng.standard_normal((1, 4, d)).astype(np.float32)).to(BF16)
    w = torch.ones((1, 4))
    scores = torch.full((1, n), 7.0, device=dev)
    for length in (n - 5, n - 64):  # the last tile part full, and a length of whole tiles
        t, x = rows(rng, new, 1, d, BF16)
        first = length - new
        codes, scales = np.zeros((1, 256, d), np.uint8), np.ones((1, 4))  # the last 256 places
        raw[n - 256:] = 0
        Ks[-4:] = 1
        sa.cache_append_q8(t.to(dev), None, K8, Ks, None, None, off, i32([length], dev), i64([0, new], dev), ws=ws)
        q8.append(codes, scales, x, length - (n - 256))
        k = q8.values(codes, scales)[0]
        back = sa.cache_read_q8(K8, Ks, None, None, off, i32([length], dev), n, 1,
                                idx=i32([np.arange(first, length)], dev), out_dtype=F32, ws=ws)
        assert np.array_equal(back[0, 0].double().cpu().numpy(), k[first - (n - 256):length - (n - 256)])
        scores.fill_(7.0)
        sa.index_score_q8(q.to(dev), w.to(dev), K8, Ks, off, i32([length], dev), n, scores=scores, ws=ws)
        ok(ws)
        want, mag = q8.index_scores(q[0].float().numpy(), w[0].numpy(), k)
        tol = 140 * 2.0 ** -23 * mag + np.abs(k).sum(1) * np.abs(q[0].float().numpy()).max(1).sum() * 2.0 ** -17
        last = scores[0, n - 256:].double().cpu().numpy()
        end = length - (n - 256)
        assert (np.abs(last[:end] - want[:end]) <= tol[:end]).all() and (last[end:] == 7).all()
        assert sum(int(torch.count_nonzero(scores[0, a:min(a + (1 << 28), n - 256)])) for a in range(0, n - 256, 1 << 28)) == 0
    del raw, K8, Ks, scores
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ another stream, without a workspace
def test_calls_on_another_stream_with_memory_of_their_own(dev):
    """The current stream is busy and has just given back memory full of ones: a call on another stream neither waits
    for it nor reads that memory as its workspace."""
    rng = np.random.default_rng(67)
    lens = [9000, 500]
    K, V = filled(rng, lens, 2, 128, dev)
    KI, _ = filled(rng, lens, 1, 64, dev)
    off, ln = i64(K.off, dev), i32(lens, dev)
    bf = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(dev).to(BF16)
    Q, qI, w = bf(1, 2, 8, 128), bf(2, 4, 64), torch.rand((2, 4), device=dev)
    packed = i64([0, 9000, 9500], dev)
    Kb, Vb = sa.cache_read_q8(*K.pair(), *V.pair(), off, ln, 9000, 2, out_off=packed, n_out=9500)

    def calls(**kw):
        scores = sa.index_score_q8(qI, w, *KI.pair(), off, ln, 9000, **kw)
        with torch.cuda.stream(kw.get("stream")):
            scores[1, 500:] = 0  # not written
        idx = sa.topk(scores, ln, 9000, 256, **kw)
        return (scores, idx, sa.decode_attn_q8(Q, *K.pair(), *V.pair(), off, ln, 9000, 2, 0.1, out_dtype=F32, **kw),
                sa.decode_attn_q8(Q, *K.pair(), *V.pair(), off, ln, 9000, 2, 0.1, idx=idx, **kw),
                *sa.cache_read_q8(*K.pair(), *V.pair(), off, ln, 9000, 2, idx=idx, **kw),
                sa.sparse_decode_attn(Q, Kb, Vb, packed, ln, idx, 2, 0.1, out_dtype=F32, **kw))

    want = calls()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    calls(stream=side)  # memory of the stream's own to use again
    for _ in range(4):
        torch.cuda.synchronize()
        torch.cuda._sleep(50_000_000)
        for n in (4096, 1 << 16, 1 << 20):
            torch.full((n,), 255, dtype=torch.uint8, device=dev)
        got = calls(stream=side)
        side.synchronize()
        assert all(torch.equal(a.cpu(), b.cpu()) for a, b in zip(want, got))


# ------------------------------------------------------------------ appending behind scales from elsewhere
@pytest.mark.parametrize("grow", [1.0, 300.0])
@pytest.mark.parametrize("old", [0.7, 1.9999, 3e-3, 1e-39, 2.5e38])
def test_append_behind_a_scale_that_is_not_a_power_of_two(old, grow, dev):
    """The scale is kept where the new tokens fit, and x / scale is x times its reciprocal in fp32; else the older
    codes move to the new scale."""
    rng = np.random.default_rng(68)
    old = np.float32(old)
    C, Hkv, d, n0, n1 = Cache([64], 2, 128, dev), 2, 128, 20, 50
    codes = rng.integers(0, 127, (Hkv, n0, d)).astype(np.uint8) | (rng.integers(0, 2, (Hkv, n0, d)) * 128).astype(np.uint8)
    C.codes[0][:, :n0] = codes
    C.scales[0][:] = old
    C.upload()
    with np.errstate(over="ignore"):
        x = (rng.standard_normal((n1 - n0, Hkv, d)).astype(np.float32) * np.float32(min(60.0 * float(old) * grow, 3e37)))
    ws = sa.workspace(sa.WS_HEADER_BYTES, dev)
    sa.cache_append_q8(torch.from_numpy(x).to(dev), None, *C.pair(), None, None, i64(C.off, dev), i32([n1], dev),
                       i64([0, n1 - n0], dev), ws=ws)
    ok(ws)
    for h in range(Hkv):
        s = np.float32(max(q8.scale_of(float(np.abs(x[:, h]).max())), float(old)))
        if s != old:
            with np.errstate(under="ignore"):
                ratio = old * (np.float32(1) / s)
                C.codes[0][h, :n0] = q8.encode(q8.VALUES[codes[h]].astype(np.float32) * ratio)
        C.codes[0][h, n0:n1] = q8.encode(x[:, h] * (np.float32(1) / s))
        C.scales[0][h] = s
    C.check()


def test_the_largest_elements(dev):
    """What rounds to 2^128 reads back as infinity, and what is just below does not."""
    x = torch.tensor([3.4028234e38, -3.4028234e38, 3.29e38, -3.29e38] + [1.0] * 60).view(1, 1, 64)
    C = Cache([64], 1, 64, dev, fill=0)
    sa.cache_append_q8(x.to(dev), None, *C.pair(), None, None, i64(C.off, dev), i32([1], dev))
    for dt in (F32, BF16):
        got = sa.cache_read_q8(*C.pair(), None, None, i64(C.off, dev), i32([1], dev), 1, 1, idx=i32([[0]], dev), out_dtype=dt)
        assert got[0, 0, 0, :4].double().tolist() == [np.inf, -np.inf, 240 * 2.0 ** 120, -240 * 2.0 ** 120]


# ------------------------------------------------------------------ the queries' two parts
def test_index_queries_keep_what_is_promised_of_them(dev):
    """One-hot keys give the query elements back: exact down to 2^-9 of their row's largest, and off by at most
    2^-17 of it below, for every mantissa of the largest and elements of 14 binades."""
    rng = np.random.default_rng(66)
    B, d = 128, 128
    C = Cache([128] * B, 1, d, dev, fill=0)
    for b in range(B):
        C.codes[b][0][np.arange(d), np.arange(d)] = 0x38  # 1.0
        C.scales[b][:] = 1.0
    C.upload()
    q = (1 + np.arange(128) / 128)[:, None] * np.ones((1, d))
    q[:, 1:] = (1 + rng.integers(0, 128, (B, d - 1)) / 128) * np.exp2(-1.0 - rng.integers(0, 14, (B, d - 1)))
    qt = torch.from_numpy(q.astype(np.float32)).to(BF16)
    assert np.array_equal(qt.double().numpy(), q)
    s = sa.index_score_q8(qt[:, None].contiguous().to(dev), torch.ones((B, 1), device=dev), *C.pair(), i64(C.off, dev),
                          i32([128] * B, dev), 128).double().cpu().numpy()
    top = q[:, :1]
    assert np.array_equal(s[q >= top * 2.0 ** -9], q[q >= top * 2.0 ** -9])
    assert (np.abs(s - q) <= top * 2.0 ** -17).all()
