"""The operators on a cache held in 8 bits against the oracle (float64):
quantising as it is written, reading back, the indexer's scores, decode
attention over an index and over every token, and a decode step of them.

Tolerances, with u = 2^-24 (half a step of fp32):
* codes, scales and rows read back: equal.
* scores: the products are exact but for query elements below 2^-11 of their
  row's largest, off by 2^-17 of it; n added terms are off by at most n * 2u
  of the sum of their magnitudes, whatever the order and rounding of the adds.
* attention: a logit is a sum of 128 exact products (off by 130 * 2u of the
  sum of their magnitudes, in units where it enters an exponential), the
  exponential and its argument by 2^-20, and by 2u of the V scale's exponent,
  which joins it; the weights go through 22 bits or more (fp32
  outputs) or 11 (bf16 outputs; with more than 16 rows per KV head 8, each
  weight then off by 2^-9 and the sum that divides it by 2^-9: 2^-8); sums
  over n keys by n * 2u; an output element is then off by that share of
  sum_t p_t |v_t|, and bf16 outputs by half a step of the element, 2^-8, more.
"""
import math

import numpy as np
import pytest
import torch

import cross_layer_shared_b200 as sa
from oracle import q8
from synth import bf16_bits_to_f32, f32_to_bf16_bits
from synth import gpu as sgpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def dev():
    from cross_layer_shared_b200 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return torch.device("cuda")


def status(ws):
    return sa.read_status(ws)


def ok(ws):
    code, det = status(ws)
    assert code == 0, (code, det)


class Cache:
    """One 8-bit tensor: sequences of capacities caps, host copies per sequence beside it."""

    def __init__(self, caps, Hkv, d, dev, fill=None):
        self.caps, self.Hkv, self.d = caps, Hkv, d
        self.off = np.concatenate([[0], np.cumsum(caps)]).astype(np.int64)
        rng = np.random.default_rng(99)
        self.codes = [rng.integers(0, 256, (Hkv, c, d)).astype(np.uint8) if fill is None else
                      np.full((Hkv, c, d), fill, np.uint8) for c in caps]
        self.scales = [np.full((Hkv, c // 64), np.nan) for c in caps]
        self.dev = dev
        self.upload()

    def upload(self):
        flat = np.concatenate([c.reshape(-1) for c in self.codes] or [np.zeros(0, np.uint8)])
        self.c8 = torch.from_numpy(flat).to(self.dev).view(torch.float8_e4m3fn).view(-1, self.d)
        s = np.concatenate([c.reshape(-1) for c in self.scales] or [np.zeros(0)])
        self.s = torch.from_numpy(s.astype(np.float32)).to(self.dev)

    def pair(self):
        return self.c8, self.s

    def check(self):
        got = self.c8.view(torch.uint8).cpu().numpy().reshape(-1)
        sc = self.s.cpu().numpy().astype(np.float64)
        at = ats = 0
        for b, (c, s) in enumerate(zip(self.codes, self.scales)):
            g = got[at:at + c.size].reshape(c.shape)
            at += c.size
            nan = np.isnan(q8.VALUES[c]) & np.isnan(q8.VALUES[g])
            assert ((g == c) | nan).all(), (b, np.argwhere((g != c) & ~nan)[:4])
            assert np.array_equal(sc[ats:ats + s.size].reshape(s.shape), s, equal_nan=True), b
            ats += s.size


def rows(rng, n, Hkv, d, dt, kind="normal"):
    x = rng.standard_normal((n, Hkv, d)).astype(np.float32)
    if kind == "growing":
        x *= np.exp2(np.arange(n) // 7).astype(np.float32)[:, None, None] * np.float32(1e-3)
    elif kind == "wild":
        x *= np.exp2(rng.integers(-140, 120, (n, Hkv, 1))).astype(np.float32)
        x[rng.random(x.shape) < 0.02] = np.nan
        x[rng.random(x.shape) < 0.02] = np.inf
        x[rng.random(x.shape) < 0.02] = -np.inf
        x[rng.random(x.shape) < 0.05] = 0
        x[rng.random((n, Hkv)) < 0.2] = 0
    elif kind == "zeros":
        x[:] = 0
    if dt == BF16:
        t = torch.from_numpy(x).to(BF16)
        return t, t.float().numpy()
    return torch.from_numpy(x), x


def i64(x, dev):
    return torch.from_numpy(np.asarray(x, np.int64)).to(dev)


def i32(x, dev):
    return torch.from_numpy(np.asarray(x, np.int32)).to(dev)


# ------------------------------------------------------------------ append
APPENDS = {  # Hkv, d, dtype, kind, rounds of new tokens per sequence
    "one_token_each": (2, 128, BF16, "normal", [(1, 1, 1)] * 3),
    "around_a_block": (1, 128, F32, "normal", [(63, 64, 65), (1, 1, 1), (64, 63, 62), (0, 1, 0)]),
    "scale_grows": (2, 64, BF16, "growing", [(5, 70), (40, 1), (70, 0), (3, 90)]),
    "wild": (3, 128, F32, "wild", [(100, 1), (31, 64), (1, 130)]),
    "wild_bf16": (1, 256, BF16, "wild", [(20, 90), (50, 1)]),
    "zeros_then_values": (1, 192, F32, "zeros", [(10, 0), (64, 3)]),
    "heads8_d128": (8, 128, BF16, "normal", [(200, 0, 1, 333)]),
    "d192": (2, 192, BF16, "normal", [(7, 129)]),
    "d256": (1, 256, F32, "growing", [(65, 1), (1, 65)]),
    "d64_odd_heads": (5, 64, F32, "normal", [(99,), (1,)]),
}


@pytest.mark.parametrize("name", list(APPENDS))
def test_append(name, dev):
    Hkv, d, dt, kind, rounds = APPENDS[name]
    rng = np.random.default_rng(list(APPENDS).index(name))
    B = len(rounds[0])
    total = [sum(r[b] for r in rounds) for b in range(B)]
    caps = [(t + 63) // 64 * 64 + 64 * (b % 2) for b, t in enumerate(total)]
    K, V = Cache(caps, Hkv, d, dev), Cache(caps, Hkv, d, dev)
    ws = sa.workspace(sa.WS_HEADER_BYTES, dev)
    lens = [0] * B
    for r, new in enumerate(rounds):
        lens = [a + n for a, n in zip(lens, new)]
        n = sum(new)
        (tk, xk), (tv, xv) = (rows(rng, n, Hkv, d, dt, "normal" if kind == "zeros" and r else kind) for _ in range(2))
        if r % 2:  # slices of a fused projection
            fused = torch.zeros((n, 3 * Hkv, d), dtype=dt)
            fused[:, Hkv:2 * Hkv], fused[:, 2 * Hkv:] = tk, tv
            fused = fused.to(dev)
            tk, tv = fused[:, Hkv:2 * Hkv], fused[:, 2 * Hkv:]
        off = np.concatenate([[0], np.cumsum(new)])
        new_off = None if all(x == 1 for x in new) else i64(off, dev)
        sa.cache_append_q8(tk.to(dev), tv.to(dev), *K.pair(), *V.pair(), i64(K.off, dev), i32(lens, dev),
                           new_off, None if r else max(new), ws=ws)
        for b in range(B):
            q8.append(K.codes[b], K.scales[b], xk[off[b]:off[b + 1]], lens[b])
            q8.append(V.codes[b], V.scales[b], xv[off[b]:off[b + 1]], lens[b])
        ok(ws)
        K.check(), V.check()


def test_append_of_one_tensor(dev):
    rng = np.random.default_rng(5)
    C = Cache([128, 64], 1, 64, dev)
    t, x = rows(rng, 97, 1, 64, BF16)
    sa.cache_append_q8(t.to(dev), None, *C.pair(), None, None, i64(C.off, dev), i32([90, 7], dev), i64([0, 90, 97], dev))
    q8.append(C.codes[0], C.scales[0], x[:90], 90)
    q8.append(C.codes[1], C.scales[1], x[90:], 7)
    C.check()


BAD = {  # what is wrong: (seq_off, seq_len, new_off); sequence 1 is always right
    "offset_not_a_block": ([0, 100, 256], [3, 3], [0, 2, 4]),
    "offset_past_the_cache": ([-64, 128, 256], [3, 3], [0, 2, 4]),
    "longer_than_its_room": ([0, 128, 256], [129, 3], [0, 2, 4]),
    "negative_length": ([0, 128, 256], [-1, 3], [0, 2, 4]),
    "more_new_than_tokens": ([0, 128, 256], [1, 3], [0, 2, 4]),
    "more_new_than_max_new": ([0, 128, 256], [100, 3], [0, 4, 4]),
    "new_rows_backwards": ([0, 128, 256], [3, 3], [3, 2, 4]),
    "new_rows_past_the_end": ([0, 128, 256], [3, 3], [2, 5, 5]),
}


@pytest.mark.parametrize("name", list(BAD))
def test_append_reports_bad_sequences_and_writes_nothing(name, dev):
    off, ln, new_off = BAD[name]
    C = Cache([128, 128], 1, 128, dev)
    ws = sa.workspace(sa.WS_HEADER_BYTES, dev)
    t, x = rows(np.random.default_rng(0), 4, 1, 128, BF16)
    sa.cache_append_q8(t.to(dev), None, *C.pair(), None, None, i64(off, dev), i32(ln, dev), i64(new_off, dev), 3, ws=ws)
    code, det = status(ws)
    assert code == sa.SA_ERR_DEVICE and det[0] == 10 and det[1] in (0, 1), det
    if name not in ("offset_not_a_block",) and new_off[1:] == [2, 4]:  # the other sequence is written
        q8.append(C.codes[1], C.scales[1], x[2:4], 3)
    C.check()


# ------------------------------------------------------------------ a cache to read
def filled(rng, lens, Hkv, d, dev, spread=0.5, strong=()):
    """Caches K, V of quantised rows; strong: (sequence, block, exponent) factors on V."""
    caps = [(n + 63) // 64 * 64 + 64 * (b % 3) for b, n in enumerate(lens)]
    K, V = Cache(caps, Hkv, d, dev), Cache(caps, Hkv, d, dev)
    for C in (K, V):
        for b, n in enumerate(lens):
            if n == 0:
                continue
            x = rng.standard_normal((n, Hkv, d))
            x *= np.exp(spread * rng.standard_normal((n + 63) // 64))[np.arange(n) // 64][:, None, None]
            if C is V:
                for sb, blk, e in strong:
                    if sb == b:
                        x[blk * 64:(blk + 1) * 64] *= 2.0 ** e
            q8.append(C.codes[b], C.scales[b], x, n)
        C.upload()
    return K, V


@pytest.mark.parametrize("d,Hkv,dt", [(64, 1, BF16), (128, 3, F32), (192, 2, BF16), (256, 1, F32)])
def test_read_picked_and_whole(d, Hkv, dt, dev):
    rng = np.random.default_rng(d)
    lens = [1, 200, 0, 64, 333]
    K, V = filled(rng, lens, Hkv, d, dev)
    off, ln, S = i64(K.off, dev), i32(lens, dev), max(lens)
    ws = sa.workspace(sa.WS_HEADER_BYTES, dev)
    kk = 70
    idx = np.full((len(lens), kk), -1, np.int32)
    for b, n in enumerate(lens):
        if n:
            idx[b] = rng.integers(0, n, kk)
            idx[b, rng.random(kk) < 0.2] = -1
    got = sa.cache_read_q8(*K.pair(), *V.pair(), off, ln, S, Hkv, idx=i32(idx, dev), out_dtype=dt, ws=ws)
    for g, C in zip(got, (K, V)):
        assert g.dtype == dt and tuple(g.shape) == (len(lens), Hkv, kk, d)
        for b in range(len(lens)):
            v = q8.values(C.codes[b], C.scales[b])
            want = np.where((idx[b] >= 0)[None, :, None], v[:, np.maximum(idx[b], 0)], 0.0) if lens[b] else 0.0
            assert np.array_equal(g[b].double().cpu().numpy(), np.broadcast_to(want, g[b].shape))
    # whole sequences, packed, into a buffer with room behind the last one
    out_off = np.concatenate([[0], np.cumsum(lens)])
    n_out = int(out_off[-1]) + 5
    Kp = torch.full((n_out * Hkv, d), 7.0, dtype=dt, device=dev)
    only = sa.cache_read_q8(*K.pair(), None, None, off, ln, S, Hkv, out_off=i64(out_off, dev), K=Kp, ws=ws)
    assert only is Kp
    ok(ws)
    for b, n in enumerate(lens):
        part = Kp[out_off[b] * Hkv:out_off[b + 1] * Hkv].double().cpu().numpy().reshape(Hkv, n, d)
        assert np.array_equal(part, q8.values(K.codes[b], K.scales[b])[:, :n])
    assert (Kp[out_off[-1] * Hkv:] == 7).all()


def test_read_reports_entries_past_the_length_and_bad_output_places(dev):
    rng = np.random.default_rng(3)
    K, V = filled(rng, [100, 40], 1, 128, dev)
    off, ln = i64(K.off, dev), i32([100, 40], dev)
    ws = sa.workspace(sa.WS_HEADER_BYTES, dev)
    k = sa.cache_read_q8(*K.pair(), None, None, off, ln, 100, 1, idx=i32([[0, 99], [40, 1]], dev), out_dtype=F32, ws=ws)
    code, det = status(ws)
    assert code == sa.SA_ERR_DEVICE and det == [10, 2, 40, 40]
    assert (k[1, 0, 0] == 0).all() and (k[1, 0, 1] != 0).any() and (k[0, 0, 1] != 0).any()
    for bad in ([0, 99, 140], [0, 100, 141], [-1, 99, 139], [41, 141, 181]):
        sa.clear_status(ws)
        out = torch.full((180, 128), 7.0, device=dev)
        sa.cache_read_q8(*K.pair(), None, None, off, ln, 100, 1, out_off=i64(bad, dev), K=out, ws=ws)
        assert status(ws)[0] == sa.SA_ERR_DEVICE
        assert (out[:1] == 7).all() or bad[0] == 0 and bad[1] == 100


# ------------------------------------------------------------------ indexer
@pytest.mark.parametrize("H,d,lens", [(1, 64, [1, 64, 65]), (4, 64, [127, 128, 129]), (16, 128, [5000]), (16, 128, [0, 300, 0, 1]),
                                      (33, 192, [200, 513]), (64, 256, [130, 1000]), (48, 128, [64] * 40), (17, 64, [20000, 3])])
def test_index_scores(H, d, lens, dev):
    rng = np.random.default_rng(H * d)
    K, _ = filled(rng, lens, 1, d, dev)
    B, S = len(lens), max(lens) + 3
    q = bf16_bits_to_f32(f32_to_bf16_bits(rng.standard_normal((B, H, d)).astype(np.float32)))
    q[:, 0] *= np.exp2(rng.integers(-16, 1, d)).astype(np.float32)  # elements far below their row's largest
    w = (rng.standard_normal((B, H)) * (rng.random((B, H)) < 0.9)).astype(np.float32)
    scores = torch.full((B, S + 2), 7.0, device=dev)
    ws = sa.workspace(sa.WS_HEADER_BYTES, dev)
    sa.index_score_q8(torch.from_numpy(q).to(dev).to(BF16), torch.from_numpy(w).to(dev), *K.pair(), i64(K.off, dev),
                      i32(lens, dev), S, scores=scores, ws=ws)
    ok(ws)
    got = scores.double().cpu().numpy()
    for b, n in enumerate(lens):
        k = q8.values(K.codes[b], K.scales[b])[0, :n]
        want, mag = q8.index_scores(q[b], w[b], k)
        off_q = np.abs(w[b]) * np.abs(q[b]).max(1) * 2.0 ** -17  # per |k_c|
        tol = (2 * d + H + 4) * 2 * U * mag + np.abs(k).sum(1) * off_q.sum() + 1e-37
        assert (np.abs(got[b, :n] - want) <= tol).all(), (np.abs(got[b, :n] - want) / tol).max()
        assert (got[b, n:] == 7).all()


def test_index_zero_queries_and_extreme_sizes(dev):
    """A zero query row scores zero; large and small queries keep their size."""
    rng = np.random.default_rng(8)
    K, _ = filled(rng, [300], 1, 128, dev)
    q = bf16_bits_to_f32(f32_to_bf16_bits(rng.standard_normal((1, 3, 128)).astype(np.float32)))
    q[0, 0] = 0
    for e in (-100, 100):
        qe = q * np.float32(2.0 ** e)
        w = np.array([[1.0, 0.5, 2.0]], np.float32)
        s = sa.index_score_q8(torch.from_numpy(qe).to(dev).to(BF16), torch.from_numpy(w).to(dev), *K.pair(),
                              i64(K.off, dev), i32([300], dev), 300).double().cpu().numpy()[0]
        k = q8.values(K.codes[0], K.scales[0])[0, :300]
        want, mag = q8.index_scores(qe[0], w[0], k)
        tol = 300 * 2 * U * mag + np.abs(k).sum(1) * (w * np.abs(qe[0]).max(1)).sum() * 2.0 ** -17
        assert (np.abs(s - want) <= tol).all()


def test_index_reports_a_length_above_s_max(dev):
    K, _ = filled(np.random.default_rng(1), [100, 90], 1, 64, dev)
    ws = sa.workspace(sa.WS_HEADER_BYTES, dev)
    scores = torch.full((2, 99), 7.0, device=dev)
    q = torch.ones((2, 4, 64), dtype=BF16, device=dev)
    sa.index_score_q8(q, torch.ones((2, 4), device=dev), *K.pair(), i64(K.off, dev), i32([100, 90], dev), 99,
                      scores=scores, ws=ws)
    code, det = status(ws)
    assert code == sa.SA_ERR_DEVICE and det[0] == 11 and det[1] == 0
    assert (scores[0] == 7).all() and (scores[1, :90] != 7).any() and (scores[1, 90:] == 7).all()


# ------------------------------------------------------------------ attention
def attn_tol(pv, mag, o, n, dt, expo, rows):
    dz = 130 * 2 * U * mag[:, None] + 2.0 ** -20 + expo * 2 * U
    rel = 2 * dz + (2.0 ** -21 if dt == F32 else 2.0 ** -11 if rows <= 16 else 2.0 ** -8) + (n + 64) * 2 * U
    return rel * pv + (np.abs(o) * 2.0 ** -8 if dt == BF16 else 0) + 1e-37


def check_attn(Q, K, V, lens, idx, Hkv, scale, O, dt):
    """Q float [L, B, Hq, d]; idx None or int [B, k]."""
    L, B, Hq, d = Q.shape
    G = Hq // Hkv
    got = O.double().cpu().numpy()
    worst = 0.0
    for b in range(B):
        pick = np.arange(lens[b]) if idx is None else idx[b][(idx[b] >= 0) & (idx[b] < lens[b])]
        for g in range(Hkv):
            k, v = (q8.VALUES[C.codes[b][g][pick]] * C.scales[b][g][pick // 64][:, None] for C in (K, V))
            q = Q[:, b, g * G:(g + 1) * G].reshape(L * G, d)
            want, pv, mag = q8.attention(q, k, v, scale)
            have = got[:, b, g * G:(g + 1) * G].reshape(L * G, d)
            vs = V.scales[b][g][np.unique(pick // 64)]
            expo = np.abs(np.log2(vs[vs > 0])).max(initial=0)
            tol = attn_tol(pv, mag, want, len(pick), dt, expo, L * G)
            worst = max(worst, float((np.abs(have - want) / tol).max()))
    assert worst <= 1, worst


def picks(rng, lens, k, pad=0.0):
    idx = np.full((len(lens), k), -1, np.int32)
    for b, n in enumerate(lens):
        m = min(k, n)
        idx[b, :m] = np.sort(rng.choice(n, m, replace=False)) if m else []
        idx[b, rng.random(k) < pad] = -1
    return idx


ATTN = {  # L, Hq, Hkv, lens, k (0: every token), share of -1 entries, dtype
    "one_token": (1, 4, 4, [1, 1], 0, 0, F32),
    "no_token": (1, 8, 2, [0, 5, 0], 0, 0, F32),
    "every_token_mha": (1, 3, 3, [63, 64, 65, 200], 0, 0, F32),
    "every_token_gqa8": (1, 16, 2, [1000, 17], 0, 0, F32),
    "every_token_bf16": (1, 8, 1, [3000], 0, 0, BF16),
    "every_token_split": (1, 5, 1, [40000], 0, 0, F32),
    "every_token_group": (6, 8, 2, [500, 129], 0, 0, BF16),
    "k1": (1, 8, 2, [100, 50], 1, 0, F32),
    "k16": (2, 8, 2, [100, 5], 16, 0, F32),
    "k17_padded": (1, 32, 4, [300, 90], 17, 0.3, F32),
    "k2048_layer": (1, 32, 8, [5000, 3000], 2048, 0.1, BF16),
    "rows9": (3, 6, 2, [700], 333, 0, F32),
    "rows16": (2, 16, 2, [700], 500, 0, BF16),
    "rows20": (5, 4, 1, [900, 31], 257, 0.2, F32),
    "rows48": (12, 8, 2, [2000], 1000, 0, BF16),
    "rows96": (24, 8, 2, [4000, 100], 2048, 0, F32),
    "rows128": (16, 8, 1, [600], 300, 0, BF16),
    "rows200": (25, 16, 2, [600], 300, 0.5, F32),
    "heads128": (1, 128, 1, [400], 0, 0, BF16),
    "gqa5_odd": (3, 15, 3, [333, 1], 100, 0, F32),
}


@pytest.mark.parametrize("name", list(ATTN))
def test_attention(name, dev):
    L, Hq, Hkv, lens, k, pad, dt = ATTN[name]
    rng = np.random.default_rng(list(ATTN).index(name))
    K, V = filled(rng, lens, Hkv, 128, dev)
    B, S = len(lens), max(lens)
    Qt = torch.from_numpy(rng.standard_normal((L, B, Hq, 128)).astype(np.float32) * 2).to(BF16)
    idx = picks(rng, lens, k, pad) if k else None
    n_tokens = int(K.off[-1])
    ws = sa.workspace(sa.decode_attn_q8_workspace_size(L, B, n_tokens, S, Hq, Hkv, 128, k), dev)
    O = torch.full((L, B, Hq, 128), 7.0, dtype=dt, device=dev)
    args = (Qt.to(dev), *K.pair(), *V.pair(), i64(K.off, dev), i32(lens, dev), S, Hkv, 0.1)
    sa.decode_attn_q8(*args, idx=None if idx is None else i32(idx, dev), O=O, ws=ws)
    ok(ws)
    check_attn(Qt.float().numpy(), K, V, lens, idx, Hkv, np.float32(0.1), O, dt)
    assert (ws[256:sa.WS_HEADER_BYTES] == 0).all()  # the counters are back at zero
    again = sa.decode_attn_q8(*args, idx=None if idx is None else i32(idx, dev), out_dtype=dt, ws=ws)
    assert torch.equal(O, again)  # the order of the slices does not matter


def test_attention_empty_rows_and_repeated_entries(dev):
    rng = np.random.default_rng(4)
    lens = [300, 200, 0]
    K, V = filled(rng, lens, 2, 128, dev)
    Qt = torch.from_numpy(rng.standard_normal((1, 3, 4, 128)).astype(np.float32)).to(BF16)
    idx = np.full((3, 40), -1, np.int32)
    idx[0] = rng.integers(0, 10, 40)  # the same tokens many times
    O = sa.decode_attn_q8(Qt.to(dev), *K.pair(), *V.pair(), i64(K.off, dev), i32(lens, dev), 300, 2, 0.1,
                          idx=i32(idx, dev), out_dtype=F32)
    check_attn(Qt.float().numpy(), K, V, lens, idx, 2, np.float32(0.1), O, F32)
    assert (O[:, 1:] == 0).all()


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("k", [0, 250])
def test_attention_sharp_logits_and_far_apart_scales(k, dt, dev):
    """Logits over hundreds of units, V blocks 2^+-40 apart, a strong block without weight: what counts is the
    sum of the weighted values, not the largest V of the cache."""
    rng = np.random.default_rng(6)
    lens = [700, 130]
    K, V = filled(rng, lens, 1, 128, dev, spread=1.0, strong=[(0, 3, 40), (0, 5, -40), (0, 7, 20), (1, 0, -60)])
    q = rng.standard_normal((2, 2, 4, 128)).astype(np.float32)
    q[0] *= 12
    q[1, :, :2] *= np.float32(1e-3)
    # keys of the strong block point away from the first two heads' queries
    Qt = torch.from_numpy(q).to(BF16)
    k3 = -np.repeat(Qt[0, 0, :1].float().numpy(), 64, 0)[:, None]
    codes, scales = K.codes[0][:, 192:256], K.scales[0][:, 3:4]
    q8.append(codes, scales, k3, 64)
    K.upload()
    idx = picks(rng, lens, k) if k else None
    O = sa.decode_attn_q8(Qt.to(dev), *K.pair(), *V.pair(), i64(K.off, dev), i32(lens, dev), 700, 1, 0.25,
                          idx=None if idx is None else i32(idx, dev), out_dtype=dt)
    check_attn(Qt.float().numpy(), K, V, lens, idx, 1, 0.25, O, dt)


def test_attention_queries_of_any_size(dev):
    rng = np.random.default_rng(7)
    K, V = filled(rng, [200], 1, 128, dev)
    for e in (-120, -60, 0, 30):
        q = torch.from_numpy(rng.standard_normal((1, 1, 3, 128)) * 2.0 ** e).to(BF16)
        q[..., 0] *= 2 ** -20  # an element far below its row's largest
        scale = 0.1 * 2.0 ** min(-e, 100)
        O = sa.decode_attn_q8(q.to(dev), *K.pair(), *V.pair(), i64(K.off, dev), i32([200], dev), 200, 1, scale,
                              out_dtype=F32)
        check_attn(q.float().numpy(), K, V, [200], None, 1, np.float32(scale), O, F32)


def test_attention_zero_and_other_scales(dev):
    """A cache from elsewhere: zero scales are blocks of zeros, scales need not be powers of two."""
    rng = np.random.default_rng(10)
    lens = [320]
    K, V = filled(rng, lens, 2, 128, dev)
    for C in (K, V):
        C.scales[0] *= 0.7 + 0.6 * rng.random(C.scales[0].shape)
        C.scales[0] = C.scales[0].astype(np.float32).astype(np.float64)
    K.scales[0][0, 1] = 0
    V.scales[0][1, 2] = V.scales[0][0, 0] = 0
    K.upload(), V.upload()
    Qt = torch.from_numpy(rng.standard_normal((1, 1, 8, 128)).astype(np.float32)).to(BF16)
    O = sa.decode_attn_q8(Qt.to(dev), *K.pair(), *V.pair(), i64(K.off, dev), i32(lens, dev), 320, 2, 0.1,
                          out_dtype=F32)
    check_attn(Qt.float().numpy(), K, V, lens, None, 2, np.float32(0.1), O, F32)


def test_attention_reports_entries_past_the_length(dev):
    rng = np.random.default_rng(12)
    lens = [100, 0]
    K, V = filled(rng, lens, 1, 128, dev)
    Qt = torch.from_numpy(rng.standard_normal((1, 2, 2, 128)).astype(np.float32)).to(BF16)
    for idx, where in (([[3, 100, 7], [-1, -1, -1]], (1, 100, 100)), ([[3, 4, 7], [-1, 0, -1]], (4, 0, 0))):
        ws = sa.workspace(1 << 20, dev)
        O = sa.decode_attn_q8(Qt.to(dev), *K.pair(), *V.pair(), i64(K.off, dev), i32(lens, dev), 100, 1, 0.1,
                              idx=i32(idx, dev), out_dtype=F32, ws=ws)
        code, det = status(ws)
        assert code == sa.SA_ERR_DEVICE and tuple(det) == (12, *where)
        check_attn(Qt.float().numpy(), K, V, lens, np.array(idx), 1, np.float32(0.1), O, F32)


def test_attention_of_a_bad_sequence_is_zero_and_reported(dev):
    rng = np.random.default_rng(13)
    lens = [100, 70]
    K, V = filled(rng, lens, 1, 128, dev)
    Qt = torch.from_numpy(rng.standard_normal((1, 2, 2, 128)).astype(np.float32)).to(BF16)
    ws = sa.workspace(1 << 20, dev)
    O = sa.decode_attn_q8(Qt.to(dev), *K.pair(), *V.pair(), i64(K.off, dev), i32([129, 70], dev), 128, 1, 0.1,
                          out_dtype=F32, ws=ws)
    code, det = status(ws)
    assert code == sa.SA_ERR_DEVICE and det[0] == 12 and det[1] == 0
    assert (O[:, 0] == 0).all()
    check_attn(Qt.float().numpy()[:, 1:], _only(K, 1), _only(V, 1), [70], None, 1, np.float32(0.1), O[:, 1:], F32)


class _only:
    def __init__(self, C, b):
        self.codes, self.scales = [C.codes[b]], [C.scales[b]]


def test_what_lies_past_the_length_does_not_matter(dev):
    """NaN codes and NaN scales behind the last token, and in tokens an index does not name."""
    rng = np.random.default_rng(14)
    lens = [70, 129]
    K, V = filled(rng, lens, 1, 128, dev)
    for C in (K, V):
        for b, n in enumerate(lens):
            C.codes[b][:, n:] = 127
        C.upload()
    Qt = torch.from_numpy(rng.standard_normal((1, 2, 2, 128)).astype(np.float32)).to(BF16)
    O = sa.decode_attn_q8(Qt.to(dev), *K.pair(), *V.pair(), i64(K.off, dev), i32(lens, dev), 129, 1, 0.1, out_dtype=F32)
    check_attn(Qt.float().numpy(), K, V, lens, None, 1, np.float32(0.1), O, F32)


# ------------------------------------------------------------------ more than 16 query rows per KV head
def group_case(dev, rng, lens, L, Hq, Hkv, k=0, pad=0.0, dt=BF16, scale=0.1, K=None, V=None, Qf=None, S=None):
    if K is None:
        K, V = filled(rng, lens, Hkv, 128, dev)
    B, S = len(lens), max(lens) if S is None else S
    Qt = torch.from_numpy((rng.standard_normal((L, B, Hq, 128)) if Qf is None else Qf).astype(np.float32)).to(BF16)
    idx = picks(rng, lens, k, pad) if k else None
    ws = sa.workspace(sa.decode_attn_q8_workspace_size(L, B, int(K.off[-1]), S, Hq, Hkv, 128, k), dev)
    O = torch.full((L, B, Hq, 128), 7.0, dtype=dt, device=dev)
    sa.decode_attn_q8(Qt.to(dev), *K.pair(), *V.pair(), i64(K.off, dev), i32(lens, dev), S, Hkv, scale,
                      idx=None if idx is None else i32(idx, dev), O=O, ws=ws)
    ok(ws)
    check_attn(Qt.float().numpy(), K, V, lens, idx, Hkv, np.float32(scale), O, dt)
    return O


GROUP = {  # L, Hq, Hkv, lens, k, share of -1, dtype
    "r17_one_token": (17, 1, 1, [1], 0, 0, BF16),
    "r18_empty_sequences": (9, 4, 2, [0, 70, 0], 0, 0, F32),
    "r24_k1": (6, 8, 2, [300, 5], 1, 0, F32),
    "r24_one_tile_short": (6, 8, 2, [127, 3], 0, 0, BF16),
    "r24_one_tile_long": (6, 8, 2, [129, 128], 0, 0, F32),
    "r32_cluster2": (8, 4, 1, [250], 0, 0, BF16),
    "r32_cluster4": (8, 4, 1, [400, 90], 0, 0, F32),
    "r32_cluster8_ragged": (8, 4, 1, [1024, 1, 513], 0, 0, BF16),
    "r20_k2048_padded": (5, 8, 2, [9000, 100], 2048, 0.4, F32),
    "r96_k2048": (24, 4, 1, [5000, 2048, 2049], 2048, 0.05, BF16),
    "r40_through_the_workspace": (10, 4, 1, [9000], 0, 0, F32),
    "r40_through_the_workspace_bf16": (10, 4, 1, [8193, 4500], 0, 0, BF16),
    "r129_two_row_tiles": (43, 3, 1, [300], 0, 0, F32),
    "r256_many_units": (2, 256, 2, [130] * 40, 0, 0, BF16),
    # units enough that tiles of 128 rows are taken, in clusters of 8, 4, 2 and 1
    "r128_cluster8": (16, 16, 2, [3000, 2000], 0, 0, F32),
    "r96_cluster4": (24, 32, 8, [700, 1, 300], 0, 0, BF16),
    "r96_cluster4_f32_k": (24, 32, 8, [2500, 800, 2100, 500], 600, 0.1, F32),
    "r24_cluster2": (3, 64, 8, [1100, 5, 600, 0, 129, 128, 900, 64], 0, 0, BF16),
    "r130_two_row_tiles_cluster1": (13, 80, 8, [300] * 9, 0, 0, F32),
    # 16 rows a CTA: several row tiles
    "r35_rows16_k": (7, 10, 2, [900, 2000], 500, 0.2, F32),
    "r100_rows16": (25, 4, 1, [1000], 0, 0, BF16),
    # 8 rows: one cluster, several of them, and slices through the workspace
    "r4_clusters": (1, 4, 1, [30000, 9000], 0, 0, F32),
    "r8_workspace_slices": (1, 64, 8, [6000, 100, 5000], 0, 0, BF16),
}


@pytest.mark.parametrize("name", list(GROUP))
def test_attention_of_many_rows(name, dev):
    L, Hq, Hkv, lens, k, pad, dt = GROUP[name]
    rng = np.random.default_rng(100 + list(GROUP).index(name))
    group_case(dev, rng, lens, L, Hq, Hkv, k, pad, dt)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("rising,L,Hkv", [(1, 8, 1), (-1, 8, 1), (1, 32, 6), (-1, 32, 6)])  # rows of 16, and of 128
def test_attention_of_many_rows_moves_its_reference(rising, L, Hkv, dt, dev):
    """Logits that climb (or fall) by hundreds of units over a slice's tiles: sums and outputs move to new references,
    rows on their own; one row's logits stay."""
    rng = np.random.default_rng(7)
    n, Hq = 1500, 4 * Hkv
    K, V = Cache([1536], Hkv, 128, dev), Cache([1536], Hkv, 128, dev)
    k = rng.standard_normal((n, Hkv, 128))
    k[:, :, 0] = rising * np.linspace(-200, 200, n)[:, None]
    q8.append(K.codes[0], K.scales[0], k, n)
    q8.append(V.codes[0], V.scales[0], rng.standard_normal((n, Hkv, 128)), n)
    K.upload(), V.upload()
    q = rng.standard_normal((L, 1, Hq, 128))
    q[:, 0, :, 0] = 12 * rng.random((L, Hq))
    q[0, 0, 0, 0] = 0
    group_case(dev, rng, [n], L, Hq, Hkv, dt=dt, K=K, V=V, Qf=q)
    group_case(dev, rng, [n], L, Hq, Hkv, k=900, dt=dt, K=K, V=V, Qf=q)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("L,Hkv", [(9, 1), (62, 16)])  # rows of 16, and of 128
def test_attention_of_many_rows_far_apart_scales(L, Hkv, dt, dev):
    rng = np.random.default_rng(6)
    lens = [700, 130]
    K, V = filled(rng, lens, Hkv, 128, dev, spread=1.0, strong=[(0, 3, 40), (0, 5, -40), (0, 7, 20), (1, 0, -60)])
    group_case(dev, rng, lens, L, 2 * Hkv, Hkv, dt=dt, K=K, V=V, scale=0.25)
    group_case(dev, rng, lens, L, 2 * Hkv, Hkv, k=250, dt=dt, K=K, V=V, scale=0.25)


@pytest.mark.parametrize("Hkv", [1, 80])  # rows of 16, and of 128
def test_attention_of_many_rows_ignores_what_it_does_not_read(Hkv, dev):
    """NaN codes and scales past the length and in tokens the index does not name; a bad sequence; an entry past the
    length."""
    rng = np.random.default_rng(14)
    lens = [70, 300]
    K, V = filled(rng, lens, Hkv, 128, dev)
    for C in (K, V):
        for b, n in enumerate(lens):
            C.codes[b][:, n:] = 127
        C.codes[1][:, 5] = 127
        C.upload()
    Qt = torch.from_numpy(rng.standard_normal((6, 2, 4 * Hkv, 128)).astype(np.float32)).to(BF16)
    idx = picks(rng, lens, 60)
    idx[1][idx[1] == 5] = -1
    args = (Qt.to(dev), *K.pair(), *V.pair(), i64(K.off, dev))
    O = sa.decode_attn_q8(*args, i32(lens, dev), 300, Hkv, 0.1, idx=i32(idx, dev), out_dtype=F32)
    check_attn(Qt.float().numpy(), K, V, lens, idx, Hkv, np.float32(0.1), O, F32)
    idx[0, 7] = 70
    ws = sa.workspace(1 << 16, dev)
    O = sa.decode_attn_q8(*args, i32(lens, dev), 300, Hkv, 0.1, idx=i32(idx, dev), out_dtype=F32, ws=ws)
    code, det = status(ws)
    assert code == sa.SA_ERR_DEVICE and det == [12, 7, 70, 70]
    check_attn(Qt.float().numpy(), K, V, lens, idx, Hkv, np.float32(0.1), O, F32)
    sa.clear_status(ws)
    O = sa.decode_attn_q8(*args, i32([129, 300], dev), 300, Hkv, 0.1, idx=i32(idx, dev), out_dtype=F32, ws=ws)
    code, det = status(ws)
    assert code == sa.SA_ERR_DEVICE and det[0] == 12 and det[1] == 0
    assert (O[:, 0] == 0).all() and not (O[:, 1] == 0).any()


def test_attention_of_many_rows_repeats_itself(dev):
    """The same call twice, and on two streams at once, gives the same bits (no order of arrival enters)."""
    rng = np.random.default_rng(15)
    lens = [3000, 500]
    K, V = filled(rng, lens, 2, 128, dev)
    off, ln = i64(K.off, dev), i32(lens, dev)
    Q = torch.from_numpy(rng.standard_normal((12, 2, 8, 128)).astype(np.float32)).to(dev).to(BF16)
    idx = i32(picks(rng, lens, 700), dev)
    one = sa.decode_attn_q8(Q, *K.pair(), *V.pair(), off, ln, 3000, 2, 0.1, idx=idx)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    wss = [sa.workspace(sa.WS_HEADER_BYTES, dev) for _ in streams]
    outs = [[torch.zeros_like(one) for _ in range(6)] for _ in streams]
    torch.cuda.synchronize()
    for r in range(6):
        for st, ws, o in zip(streams, wss, outs):
            sa.decode_attn_q8(Q, *K.pair(), *V.pair(), off, ln, 3000, 2, 0.1, idx=idx, O=o[r], ws=ws, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(one, x) for o in outs for x in o)


# ------------------------------------------------------------------ sizes at the ends
def test_many_sequences(dev):
    """4096 sequences of up to 64 tokens: one decode step's append, scores and attention."""
    rng = np.random.default_rng(40)
    B = 4096
    lens = rng.integers(1, 64, B)
    off = np.arange(B + 1) * 64
    C = Cache([64 * B], 1, 64, dev)
    C.off = off
    x = torch.from_numpy(rng.standard_normal((int(lens.sum()), 1, 64)).astype(np.float32))
    ws = sa.workspace(sa.WS_HEADER_BYTES, dev)
    sa.cache_append_q8(x.to(dev), None, *C.pair(), None, None, i64(off, dev), i32(lens, dev),
                       i64(np.concatenate([[0], np.cumsum(lens)]), dev), 64, ws=ws)
    one = torch.from_numpy(rng.standard_normal((B, 1, 64)).astype(np.float32))
    sa.cache_append_q8(one.to(dev), None, *C.pair(), None, None, i64(off, dev), i32(lens + 1, dev), ws=ws)
    ok(ws)
    q = torch.from_numpy(rng.standard_normal((B, 4, 64)).astype(np.float32)).to(BF16)
    w = torch.ones((B, 4))
    scores = sa.index_score_q8(q.to(dev), w.to(dev), *C.pair(), i64(off, dev), i32(lens + 1, dev), 64, ws=ws)
    ok(ws)
    got = scores.double().cpu().numpy()
    at = np.concatenate([[0], np.cumsum(lens)])
    for b in (0, 1, 777, 2048, B - 1):
        codes, scales = np.zeros((1, 64, 64), np.uint8), np.zeros((1, 1))
        q8.append(codes, scales, x.numpy()[at[b]:at[b + 1]], int(lens[b]))
        q8.append(codes, scales, one.numpy()[b:b + 1], int(lens[b]) + 1)
        k = q8.values(codes, scales)[0, :lens[b] + 1]
        want, mag = q8.index_scores(q[b].float().numpy(), w[b].numpy(), k)
        tol = 140 * 2 * U * mag + np.abs(k).sum(1) * np.abs(q[b].float().numpy()).max(1).sum() * 2.0 ** -17
        assert (np.abs(got[b, :lens[b] + 1] - want) <= tol).all()


def test_empty_cache_and_empty_batch(dev):
    """No token place at all: rows of zeros, scores untouched, new tokens reported."""
    e8 = lambda d: torch.empty((0, d), dtype=torch.float8_e4m3fn, device=dev)
    s0 = torch.empty(0, device=dev)
    off, ln = i64([0, 0, 0], dev), i32([0, 0], dev)
    ws = sa.workspace(1 << 16, dev)
    for L in (1, 9):
        Q = torch.ones((L, 2, 2, 128), dtype=BF16, device=dev)
        O = torch.full((L, 2, 2, 128), 7.0, device=dev)
        sa.decode_attn_q8(Q, e8(128), s0, e8(128), s0, off, ln, 0, 1, 0.1, O=O, ws=ws)
        assert (O == 0).all()
        O.fill_(7)
        sa.decode_attn_q8(Q, e8(128), s0, e8(128), s0, off, ln, 0, 1, 0.1, idx=i32([[-1] * 3] * 2, dev), O=O, ws=ws)
        assert (O == 0).all()
    ok(ws)
    scores = torch.full((2, 4), 7.0, device=dev)
    sa.index_score_q8(torch.ones((2, 4, 64), dtype=BF16, device=dev), torch.ones((2, 4), device=dev), e8(64), s0, off,
                      ln, 4, scores=scores, ws=ws)
    assert (scores == 7).all()
    K, V = sa.cache_read_q8(e8(64), s0, e8(64), s0, off, ln, 0, 1, idx=i32([[-1], [-1]], dev), ws=ws)
    assert (K == 0).all() and (V == 0).all()
    ok(ws)
    x = torch.ones((2, 1, 64), device=dev)
    sa.cache_append_q8(x, x, e8(64), s0, e8(64), s0, off, i32([1, 1], dev), ws=ws)
    assert status(ws)[0] == sa.SA_ERR_DEVICE
    none = torch.empty((0, 1, 64), device=dev)
    sa.cache_append_q8(none, None, e8(64), s0, None, None, i64([0], dev), i32([], dev))


def test_offsets_past_32_bits(dev):
    """The last sequence of a cache of more than 2^31 bytes of codes per tensor, and more than 2^32 with it."""
    rng = np.random.default_rng(41)
    Hkv, d, n, first = 8, 128, 300, (1 << 22) + 64 * 3
    n_tokens = first + 320
    K8, V8 = (torch.zeros((n_tokens * Hkv, d), dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn) for _ in range(2))
    Ks, Vs = (torch.zeros(n_tokens * Hkv // 64, device=dev) for _ in range(2))
    off, ln = i64([0, first, n_tokens], dev), i32([0, n], dev)
    (tk, xk), (tv, xv) = (rows(rng, n, Hkv, d, BF16) for _ in range(2))
    ws = sa.workspace(1 << 20, dev)
    sa.cache_append_q8(tk.to(dev), tv.to(dev), K8, Ks, V8, Vs, off, ln, i64([0, 0, n], dev), ws=ws)
    C = []
    for x in (xk, xv):
        c = Cache([320], Hkv, d, dev, fill=0)
        q8.append(c.codes[0], c.scales[0], x, n)
        C.append(c)
    K, V = sa.cache_read_q8(K8, Ks, V8, Vs, off, ln, n, Hkv, out_off=i64([0, 0, n], dev), n_out=n, out_dtype=F32, ws=ws)
    for got, c in ((K, C[0]), (V, C[1])):
        assert np.array_equal(got.double().cpu().numpy().reshape(Hkv, n, d), q8.values(c.codes[0], c.scales[0])[:, :n])
    for L, G in ((1, 4), (6, 4)):
        Q = torch.from_numpy(rng.standard_normal((L, 2, Hkv * G, d)).astype(np.float32)).to(BF16)
        O = sa.decode_attn_q8(Q.to(dev), K8, Ks, V8, Vs, off, ln, n, Hkv, 0.1, out_dtype=F32, ws=ws)
        assert (O[:, 0] == 0).all()
        check_attn(Q[:, 1:].float().numpy(), *C, [n], None, Hkv, np.float32(0.1), O[:, 1:], F32)
    ok(ws)
    # the same memory as one indexer-key cache of 2^25 tokens and more
    kI = K8.view(-1, d)
    scores = torch.zeros((1, 64), device=dev)
    at = (n_tokens * Hkv // 64 - 5 * Hkv) * 64  # head 0 of the last sequence
    q = torch.from_numpy(rng.standard_normal((1, 16, d)).astype(np.float32)).to(BF16)
    w = torch.ones((1, 16))
    sa.index_score_q8(q.to(dev), w.to(dev), kI, Ks, i64([at, at + 64], dev), i32([64], dev), 64, scores=scores, ws=ws)
    ok(ws)
    k = q8.values(C[0].codes[0], C[0].scales[0])[0, :64]
    want, mag = q8.index_scores(q[0].float().numpy(), w[0].numpy(), k)
    tol = 300 * 2 * U * mag + np.abs(k).sum(1) * np.abs(q[0].float().numpy()).max(1).sum() * 2.0 ** -17
    assert (np.abs(scores[0].double().cpu().numpy() - want) <= tol).all()


def test_read_into_outputs_between_two_sectors(dev):
    """Outputs that are 16- but not 32-byte aligned."""
    rng = np.random.default_rng(42)
    K, V = filled(rng, [100], 2, 128, dev)
    for dt, skip in ((BF16, 8), (F32, 4)):
        base = [torch.full((100 * 2 * 128 + 2 * skip,), 7.0, dtype=dt, device=dev) for _ in range(2)]
        out = [t[skip:-skip].view(200, 128) for t in base]
        assert out[0].data_ptr() % 32 == 16
        sa.cache_read_q8(*K.pair(), *V.pair(), i64(K.off, dev), i32([100], dev), 100, 2, out_off=i64([0, 100], dev),
                         K=out[0], V=out[1])
        for o, t, C in zip(out, base, (K, V)):
            assert np.array_equal(o.double().cpu().numpy().reshape(2, 100, 128), q8.values(C.codes[0], C.scales[0])[:, :100])
            assert (t[:skip] == 7).all() and (t[-skip:] == 7).all()


def test_calls_refuse_wrong_tensors(dev):
    rng = np.random.default_rng(43)
    K, V = filled(rng, [100], 2, 128, dev)
    off, ln = i64(K.off, dev), i32([100], dev)
    Q = torch.zeros((1, 1, 4, 128), dtype=BF16, device=dev)
    good = dict(Q=Q, K8=K.c8, K_scale=K.s, V8=V.c8, V_scale=V.s, seq_off=off, seq_len=ln, S_max=100, Hkv=2, scale=0.1)
    sa.decode_attn_q8(**good)
    for name, wrong in (("Q", Q.float()), ("Q", Q.cpu()), ("Q", Q[0]), ("Q", Q.expand(2, 1, 4, 128)), ("K8", K.c8.view(torch.uint8)),
                        ("K8", K.c8[:-64]), ("K8", K.c8.cpu()), ("V8", V.c8[:128]), ("V8", None), ("V_scale", None),
                        ("K_scale", K.s.double()), ("K_scale", K.s[:-1]), ("seq_off", off.int()), ("seq_off", off[:1]),
                        ("seq_len", ln.long()), ("Hkv", 0), ("Hkv", 3), ("S_max", 1 << 40), ("scale", "x"),
                        ("idx", torch.zeros((1, 4), device=dev)), ("idx", torch.zeros((2, 4), dtype=torch.int32, device=dev)),
                        ("idx", torch.zeros(4, dtype=torch.int32, device=dev)), ("O", Q.half()), ("O", Q[..., :64]),
                        ("O", torch.zeros((1, 1, 4, 256), dtype=BF16, device=dev)[..., ::2]),
                        ("ws", torch.zeros(4096, device=dev)), ("ws", torch.zeros(4096, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            sa.decode_attn_q8(**dict(good, **{name: wrong}))
    with pytest.raises(sa.SAError, match="WORKSPACE"):
        sa.decode_attn_q8(**dict(good, ws=torch.zeros(256, dtype=torch.uint8, device=dev)))
    x = torch.zeros((1, 2, 128), device=dev)
    good = dict(new_K=x, new_V=x, K8=K.c8, K_scale=K.s, V8=V.c8, V_scale=V.s, seq_off=off, seq_len=ln)
    for name, wrong in (("new_K", x.half()), ("new_K", x.transpose(1, 2)), ("new_K", x[:, :1]), ("new_V", None), ("V8", None),
                        ("new_V", x.to(BF16)), ("new_K", x.cpu()), ("new_K", torch.zeros((2, 2, 128), device=dev)),
                        ("new_off", i32([0, 1], dev)), ("new_off", i64([0, 1, 1], dev)), ("K8", None)):
        with pytest.raises((ValueError, AttributeError)):
            sa.cache_append_q8(**dict(good, **{name: wrong}))
    idx = i32([[1, 2]], dev)
    good = dict(K8=K.c8, K_scale=K.s, V8=V.c8, V_scale=V.s, seq_off=off, seq_len=ln, S_max=100, Hkv=2, idx=idx)
    out = torch.zeros((1, 2, 2, 128), device=dev)
    for name, wrong in (("idx", None), ("out_off", i64([0, 100], dev)), ("K", out[:, :1]), ("K", out.half()), ("K", out.cpu()),
                        ("V", out), ("Hkv", 5)):
        with pytest.raises(ValueError):
            sa.cache_read_q8(**dict(good, **{name: wrong}))
    k1, _ = filled(rng, [100], 1, 64, dev)
    q = torch.zeros((1, 4, 64), dtype=BF16, device=dev)
    good = dict(qI=q, w=torch.zeros((1, 4), device=dev), KI8=k1.c8, KI_scale=k1.s, seq_off=i64(k1.off, dev), seq_len=ln, S_max=100)
    for name, wrong in (("qI", q.float()), ("qI", q[0]), ("w", torch.zeros((1, 3), device=dev)), ("KI8", k1.c8.view(-1, 128)),
                        ("scores", torch.zeros((1, 99), device=dev)), ("scores", torch.zeros(100, device=dev)),
                        ("scores", torch.zeros((1, 100), dtype=BF16, device=dev)), ("ld", 50),
                        ("seq_len", i32([100, 1], dev))):
        with pytest.raises((ValueError, sa.SAError)):
            sa.index_score_q8(**dict(good, **{name: wrong}))


# ------------------------------------------------------------------ together
def step_case(dev, B=3, L=5, Hq=8, Hkv=2, H=4, d_I=64, k=128, lens=(300, 700, 1500)):
    rng = np.random.default_rng(20)
    caps = [(n + 20 + 63) // 64 * 64 for n in lens]
    caches = {}
    for name, h, w in (("KI0", 1, d_I), ("KI3", 1, d_I), ("K0", Hkv, 128), ("V0", Hkv, 128), ("K3", Hkv, 128), ("V3", Hkv, 128)):
        C = caches[name] = Cache(caps, h, w, dev)
        t, _ = rows(rng, sum(lens), h, w, BF16)
        sa.cache_append_q8(t.to(dev), None, *C.pair(), None, None, i64(C.off, dev), i32(lens, dev),
                           i64(np.concatenate([[0], np.cumsum(lens)]), dev))
    bf = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(dev).to(BF16)
    qI = [bf(B, H, d_I), None, None, bf(B, H, d_I), None]
    w = [torch.from_numpy(rng.random((B, H)).astype(np.float32)).to(dev) if t is not None else None for t in qI]
    at = lambda n: [caches[n + "0"].pair()] * 3 + [caches[n + "3"].pair()] * 2
    KI = [caches["KI0"].pair(), None, None, caches["KI3"].pair(), None]
    new_KI = [bf(B, 1, d_I) if t is not None else None for t in qI]
    new = lambda: [bf(B, Hkv, 128) for _ in range(L)]
    return dict(caches=caches, qI=qI, w=w, KI=KI, K=at("K"), V=at("V"), Q=bf(L, B, Hq, 128), new_KI=new_KI, new_K=new(),
                new_V=new(), off=i64(caches["K0"].off, dev), lens=list(lens), B=B, L=L, Hq=Hq, Hkv=Hkv, k=k, S=max(caps))


def plain_step(c, lens, dev):
    """The step by its parts on the caches' values: read back, score and attend in float64."""
    O = np.zeros((c["L"], c["B"], c["Hq"], 128))
    G = c["Hq"] // c["Hkv"]
    off = c["off"].tolist()
    for l in range(c["L"]):
        f = 0 if l < 3 else 3
        for b, n in enumerate(lens):
            def vals(pair, Hkv):
                codes, s = pair
                d = codes.shape[1]
                r = slice(off[b] * Hkv, off[b + 1] * Hkv)
                cap = off[b + 1] - off[b]
                v = codes[r].double().view(Hkv, cap, d) * s[off[b] * Hkv // 64:off[b + 1] * Hkv // 64].double() \
                    .repeat_interleave(64).view(Hkv, cap, 1)
                return v[:, :n].cpu().numpy()
            k, v = vals(c["K"][l], c["Hkv"]), vals(c["V"][l], c["Hkv"])
            pick = c["idx"][f][b]
            pick = pick[pick >= 0]
            for g in range(c["Hkv"]):
                q = c["Q"][l, b, g * G:(g + 1) * G].double().cpu().numpy()
                O[l, b, g * G:(g + 1) * G] = q8.attention(q, k[g][pick], v[g][pick], 0.1)[0]
    return O


@pytest.mark.parametrize("Hq", [8, 16])  # 12 and 8 query rows per KV head and group of layers, or 24 and 16
def test_decode_steps_with_append_eager_and_captured(Hq, dev):
    """Two steps: one eager, one replayed from a graph captured on another stream; new tokens, lengths and queries
    change in place between them."""
    c = step_case(dev, Hq=Hq)
    ln = i32([n + 1 for n in c["lens"]], dev)
    n_tokens = int(c["off"][-1])
    ws = sa.workspace(sa.decode_step_q8_workspace_size(c["L"], c["B"], n_tokens, c["S"], c["Hq"], c["Hkv"], 128, c["k"]), dev)
    O = torch.zeros((c["L"], c["B"], c["Hq"], 128), dtype=F32, device=dev)
    idx = torch.zeros((c["B"], c["k"]), dtype=torch.int32, device=dev)
    scores = torch.zeros((c["B"], c["S"]), dtype=F32, device=dev)

    def step():
        sa.decode_step_q8("FSSFS", c["qI"], c["w"], c["KI"], c["K"], c["V"], c["off"], ln, c["S"], c["k"], c["Q"],
                          c["Hkv"], 0.1, O=O, idx=idx, scores=scores, ws=ws, new_KI=c["new_KI"], new_K=c["new_K"],
                          new_V=c["new_V"])

    def check():
        lens = ln.tolist()
        ok(ws)
        c["idx"] = {}
        for f in (0, 3):
            s = sa.index_score_q8(c["qI"][f], c["w"][f], *c["KI"][f], c["off"], ln, c["S"])
            c["idx"][f] = sa.topk(s, ln, c["S"], c["k"]).cpu().numpy()
        assert np.array_equal(c["idx"][3], idx.cpu().numpy())
        want = plain_step(c, lens, dev)
        # |logits| stay below 2^5 and sums of p |v| below 2^3 here
        assert np.abs(O.double().cpu().numpy() - want).max() <= 8 * (2 * (130 * 2 * U * 32 + 2.0 ** -20) + 2.0 ** -15)
        # the new rows are in the caches
        got = sa.cache_read_q8(*c["K"][3], *c["V"][3], c["off"], ln, c["S"], c["Hkv"],
                               idx=(ln - 1)[:, None].contiguous(), out_dtype=F32)
        for g, new in zip(got, (c["new_K"][3], c["new_V"][3])):
            x = new.float()
            assert ((g[:, :, 0] - x).abs() <= x.abs() / 8 + x.abs().amax() * 2.0 ** -12).all()

    step()
    check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for i in range(3):
        ln += 1
        for t in c["new_K"] + c["new_V"] + [c["Q"]] + [x for x in c["new_KI"] + c["qI"] if x is not None]:
            t.copy_(torch.roll(t, 1, 0) * 0.9)
        graph.replay()
        torch.cuda.synchronize()
        check()


def test_calls_on_two_streams_at_once(dev):
    """Each with its own workspace, over one cache."""
    rng = np.random.default_rng(30)
    lens = [9000, 500]
    K, V = filled(rng, lens, 2, 128, dev)
    off, ln = i64(K.off, dev), i32(lens, dev)
    n = sa.decode_attn_q8_workspace_size(1, 2, int(K.off[-1]), 9000, 8, 2, 128, 0)
    streams = [torch.cuda.Stream() for _ in range(2)]
    Qs = [torch.from_numpy(rng.standard_normal((1, 2, 8, 128)).astype(np.float32)).to(dev).to(BF16) for _ in streams]
    wss = [sa.workspace(n, dev) for _ in streams]
    alone = [sa.decode_attn_q8(q, *K.pair(), *V.pair(), off, ln, 9000, 2, 0.1, out_dtype=F32) for q in Qs]
    outs = [[torch.zeros_like(alone[0]) for _ in range(8)] for _ in streams]
    torch.cuda.synchronize()
    for r in range(8):
        for s, q, ws, o in zip(streams, Qs, wss, outs):
            sa.decode_attn_q8(q, *K.pair(), *V.pair(), off, ln, 9000, 2, 0.1, O=o[r], ws=ws, stream=s)
    torch.cuda.synchronize()
    for a, o, ws in zip(alone, outs, wss):
        ok(ws)
        assert all(torch.equal(a, x) for x in o)


def test_a_cache_read_back_feeds_the_bf16_path(dev):
    """Prefill over an 8-bit cache: whole sequences read back packed are what sparse_decode_attn takes."""
    rng = np.random.default_rng(31)
    lens = [400, 130]
    K, V = filled(rng, lens, 2, 128, dev)
    off, ln = i64(K.off, dev), i32(lens, dev)
    out_off = i64(np.concatenate([[0], np.cumsum(lens)]), dev)
    idx = i32(picks(rng, lens, 64), dev)
    Q = torch.from_numpy(rng.standard_normal((2, 2, 8, 128)).astype(np.float32)).to(dev).to(BF16)
    Kb, Vb = sa.cache_read_q8(*K.pair(), *V.pair(), off, ln, 400, 2, out_off=out_off, n_out=sum(lens))
    a = sa.sparse_decode_attn(Q, Kb, Vb, out_off, ln, idx, 2, 0.1, out_dtype=F32)
    b = sa.decode_attn_q8(Q, *K.pair(), *V.pair(), off, ln, 400, 2, 0.1, idx=idx, out_dtype=F32)
    # the bf16 path rounds its weights to bf16 pairs or keeps them in fp32: its own stated tolerance
    assert (a - b).abs().max().item() <= 1e-4
