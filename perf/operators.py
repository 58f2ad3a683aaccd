"""Measured cases of the operators on a cache held in 8 bits.

The cache: e4m3 codes with one fp32 scale, a power of two, for each block of
64 tokens and KV head.  Sequence b owns cap_b = seq_off[b+1] - seq_off[b]
token places (a multiple of 64) laid out [Hkv, cap_b, d] from row
seq_off[b]*Hkv; the scale of row r is scales[r // 64].  A block's scale is
the smallest 2^e >= 2^-126 with max|x| <= 448 * 2^e; when later tokens of the
block need a larger one, the codes already there are requantised to it.

Operators (`op` of a case):
  append  new tokens' rows quantised into the cache behind the tokens there
  read    cache rows back as bf16 / fp32: picked rows, or whole sequences packed
  index   the indexer's scores over an 8-bit key cache
  attn    decode attention over the cache: the tokens of an index, or all

`own` false: plain torch in fp32; true: the framework's entry points.
"""
import math

import torch

own = False

BLOCK = 64
D = 128
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one decode step's K and V rows of 4 sequences, most blocks part full
        dict(name="append-token", op="append", B=4, Hkv=8, d=128, len_lo=4099, len_hi=131072, n_lo=1, n_hi=1,
             pair=True, fused=True, dtype="bf16"),
        # one chunk of a chunked prefill behind 100,037 cached tokens, K and V sliced from a fused projection
        dict(name="append-chunk", op="append", B=1, Hkv=8, d=128, len_lo=102085, len_hi=102085, n_lo=2048, n_hi=2048,
             pair=True, fused=True, dtype="bf16"),
        # 16 whole prompts of ragged lengths, fp32 rows (a projection that keeps its accumulator)
        dict(name="append-prompts", op="append", B=16, Hkv=4, d=128, len_lo=517, len_hi=16384, n_lo=517, n_hi=16384,
             pair=True, fused=False, dtype="f32"),
        # the selected rows of 8 sequences for a caller's own attention
        dict(name="read-picked", op="read", B=8, Hkv=4, d=128, len_lo=32768, len_hi=32768, k=2048, pair=True,
             dtype="bf16"),
        # one long sequence back as a packed bf16 cache, before a prefill chunk attends to it
        dict(name="read-whole", op="read", B=1, Hkv=8, d=128, len_lo=131009, len_hi=131009, k=0, pair=True,
             dtype="bf16"),
        # indexer of one short sequence: latency
        dict(name="index-short", op="index", B=1, H=4, d=64, len_lo=4096, len_hi=4096),
        # indexer of four long sequences, the bulk of a decode step's bytes
        dict(name="index-long", op="index", B=4, H=16, d=128, len_lo=131072, len_hi=131072),
        # a ragged batch of 32
        dict(name="index-ragged", op="index", B=32, H=16, d=128, len_lo=8192, len_hi=131072),
        # one layer's attention over the shared index (8 query rows per KV head)
        dict(name="attn-picked-layer", op="attn", B=8, L=1, Hq=32, Hkv=4, len_lo=32768, len_hi=32768, k=2048,
             dtype="bf16"),
        # the 24 layers of a group over one index and one cache (96 query rows per KV head)
        dict(name="attn-picked-group", op="attn", B=4, L=24, Hq=32, Hkv=8, len_lo=131072, len_hi=131072, k=2048,
             dtype="bf16"),
        # a short conversation, every token, fp32 out: latency
        dict(name="attn-all-short", op="attn", B=2, L=1, Hq=8, Hkv=1, len_lo=333, len_hi=1021, k=0, dtype="f32"),
        # a dense layer over four long sequences
        dict(name="attn-all-long", op="attn", B=4, L=1, Hq=32, Hkv=8, len_lo=131072, len_hi=131072, k=0,
             dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "read", "index", "attn"])
    if op == "append":
        Hkv, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 192, 256])
        n = 1 if rng.random() < 0.3 else _log(rng, 2, 16384)
        B = _log(rng, 1, max(1, min(32, 131072 * 4 // (n * Hkv * d // 128 + 1))))
        hi = n + _log(rng, 1, max(1, 500000 // B))
        return dict(op=op, B=B, Hkv=Hkv, d=d, len_lo=max(n, hi // 3), len_hi=hi, n_lo=max(1, n // 2), n_hi=n,
                    pair=rng.random() < 0.7, fused=rng.random() < 0.5, dtype=rng.choice(["bf16", "f32"]))
    if op == "read":
        Hkv, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 192, 256])
        B = _log(rng, 1, 16)
        hi = _log(rng, 1, max(1, 131072 * 8 * 128 // (B * Hkv * d)) if B * Hkv * d > 8 * 128 else 131072)
        return dict(op=op, B=B, Hkv=Hkv, d=d, len_lo=max(1, hi // 4), len_hi=hi,
                    k=0 if rng.random() < 0.5 else _log(rng, 1, 2048), pair=rng.random() < 0.7,
                    dtype=rng.choice(["bf16", "f32"]))
    if op == "index":
        B = _log(rng, 1, 32)
        hi = _log(rng, 1, 131072)
        return dict(op=op, B=B, H=rng.choice([1, 4, 8, 16]), d=rng.choice([64, 128]), len_lo=max(1, hi // 8),
                    len_hi=hi)
    Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 8])
    if rng.random() < 0.5:  # the tokens of an index, one layer or a group
        B, L, k = _log(rng, 1, 8), rng.choice([1, 1, 2, 4, 12]), _log(rng, 16, 2048)
        hi = _log(rng, 64, 131072)
    else:
        B, L, k = _log(rng, 1, 16), 1, 0
        hi = _log(rng, 1, min(131072, 131072 * 32 // (B * Hkv)))
    return dict(op=op, B=B, L=L, Hq=Hkv * G, Hkv=Hkv, len_lo=max(1, hi // 3), len_hi=hi, k=k,
                dtype=rng.choice(["bf16", "f32"]))


def _spread(lo, hi, n):
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _lens(case):
    return _spread(case["len_lo"], case["len_hi"], case["B"])


def _caps(case):
    return [(n + BLOCK - 1) // BLOCK * BLOCK + BLOCK * (i % 3) for i, n in enumerate(_lens(case))]


def _news(case):
    return [min(n, m) for n, m in zip(_spread(case["n_lo"], case["n_hi"], case["B"]), _lens(case))]


def _pow2_scale(amax):
    """The smallest 2^e >= 2^-126 with amax <= 448 * 2^e = 1.75 * 2^(e+8), from the bits of amax."""
    bits = amax.contiguous().view(torch.int32)
    e = (bits >> 23) - 135 + ((bits & 0x7FFFFF) > 0x600000).int()
    return ((e.clamp(min=-126) + 127) << 23).view(torch.float32)


def _cache(rows, d, g):
    """A cache as quantising gives it: ~N(0, 1) rows, a few strong channels, blocks of differing strength."""
    codes = torch.empty((rows, d), dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty(rows // BLOCK, dtype=torch.float32, device="cuda")
    chan = torch.where(torch.arange(d, device="cuda") % 37 == 5, 6.0, 1.0)
    step = 1 << 20
    for a in range(0, rows, step):
        n = min(step, rows - a)
        x = torch.randn((n // BLOCK, BLOCK, d), device="cuda", generator=g) * chan
        x *= torch.exp(0.5 * torch.randn((n // BLOCK, 1, 1), device="cuda", generator=g))
        s = _pow2_scale(x.abs().amax((1, 2)))
        scales[a // BLOCK:(a + n) // BLOCK] = s
        codes[a:a + n] = (x / s[:, None, None]).to(torch.float8_e4m3fn).view(n, d)
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    lens, caps = _lens(case), _caps(case)
    off = [0]
    for c in caps:
        off.append(off[-1] + c)
    B, op, d = case["B"], case["op"], case.get("d", D)
    Hkv = case.get("Hkv", 1)
    s = {"case": dict(case), "off": torch.tensor(off, dtype=torch.int64, device="cuda"),
         "len": torch.tensor(lens, dtype=torch.int32, device="cuda"), "S": max(lens), "n_tokens": off[-1]}
    rows = off[-1] * Hkv
    s["K8"], s["Ks"] = _cache(rows, d, g)
    if case.get("pair") or op == "attn":
        s["V8"], s["Vs"] = _cache(rows, d, g)
    dt = DTYPES.get(case.get("dtype"))
    if op == "append":
        new = _news(case)
        new_off = [0]
        for n in new:
            new_off.append(new_off[-1] + n)
        s["new_off"] = torch.tensor(new_off, dtype=torch.int64, device="cuda")
        s["max_new"] = max(new)
        s["touched"] = sum((n - 1) // BLOCK - (n - m) // BLOCK + 1 for n, m in zip(lens, new))
        N = new_off[-1]
        if case["fused"]:  # K and V as slices of one projection's output rows [queries | K | V]
            x = torch.randn((N, 3 * Hkv, d), device="cuda", generator=g).to(dt)
            s["newK"], s["newV"] = x[:, Hkv:2 * Hkv], x[:, 2 * Hkv:]
        else:
            s["newK"], s["newV"] = (torch.randn((N, Hkv, d), device="cuda", generator=g).to(dt) for _ in range(2))
        if not case["pair"]:
            s["newV"] = None
    elif op == "read" or op == "attn":
        if case["k"]:
            k = case["k"]
            idx = torch.full((B, k), -1, dtype=torch.int32, device="cuda")
            for b in range(B):
                m = min(k, lens[b])
                idx[b, :m] = torch.randperm(lens[b], device="cuda", generator=g)[:m].sort().values.int()
            s["idx"] = idx
        elif op == "read":
            out = [0]
            for n in lens:
                out.append(out[-1] + n)
            s["out_off"], s["n_out"] = torch.tensor(out, dtype=torch.int64, device="cuda"), out[-1]
        if op == "read":
            shape = (B, Hkv, case["k"], d) if case["k"] else (s["n_out"] * Hkv, d)
            s["K"] = torch.zeros(shape, dtype=dt, device="cuda")
            s["V"] = torch.zeros(shape, dtype=dt, device="cuda") if case["pair"] else None
        else:
            s["Q"] = torch.randn((case["L"], B, case["Hq"], d), device="cuda", generator=g).to(torch.bfloat16)
            s["O"] = torch.zeros((case["L"], B, case["Hq"], d), dtype=dt, device="cuda")
            s["scale"] = d ** -0.5
    else:
        H = case["H"]
        s["qI"] = torch.randn((B, H, d), device="cuda", generator=g).to(torch.bfloat16)
        s["w"] = torch.rand((B, H), device="cuda", generator=g) + 0.1
        s["scores"] = torch.zeros((B, s["S"]), dtype=torch.float32, device="cuda")
    return s


# ------------------------------------------------------------------ plain form
def _rows(s, Hkv, t):
    """Cache row of token t [B, n] of every head: [B, Hkv, n]."""
    off, cap = s["off"][:-1], s["off"][1:] - s["off"][:-1]
    head = off[:, None] * Hkv + cap[:, None] * torch.arange(Hkv, device="cuda")
    return head[:, :, None] + t[:, None, :]


def _values(codes, scales, rows):
    return codes.view(torch.uint8)[rows].view(torch.float8_e4m3fn).float() * scales[rows // BLOCK][..., None]


def _plain_append_one(s, x, codes, scales):
    Hkv = x.shape[1]
    n = s["new_off"][1:] - s["new_off"][:-1]
    length = s["len"].long()
    pos0 = length - n
    blocks = (length - 1) // BLOCK - pos0 // BLOCK + 1
    seq = torch.repeat_interleave(torch.arange(len(n), device="cuda"), blocks, output_size=s["touched"])
    first = torch.cumsum(blocks, 0) - blocks
    blk = pos0[seq] // BLOCK + torch.arange(s["touched"], device="cuda") - first[seq]
    t = blk[:, None] * BLOCK + torch.arange(BLOCK, device="cuda")  # [T, 64]
    is_old = t < pos0[seq][:, None]
    is_new = ~is_old & (t < length[seq][:, None])
    src = (s["new_off"][seq][:, None] + t - pos0[seq][:, None]).clamp(0, x.shape[0] - 1)
    xn = torch.where(is_new[:, :, None, None], x[src].float(), 0.0).transpose(1, 2)  # [T, Hkv, 64, d]
    off, cap = s["off"][seq], s["off"][seq + 1] - s["off"][seq]
    rows = (off * Hkv)[:, None, None] + cap[:, None, None] * torch.arange(Hkv, device="cuda")[:, None] + t[:, None, :]
    old_scale = torch.where(is_old[:, :1], scales[rows[:, :, 0] // BLOCK], 2.0 ** -126)
    scale = torch.maximum(_pow2_scale(xn.abs().amax((2, 3))), old_scale)
    raw = codes.view(torch.uint8)
    had = raw[rows]
    ratio = torch.where(is_old[:, :1], old_scale / scale, 0.0)
    was = torch.where(is_old[:, None, :, None], had.view(torch.float8_e4m3fn).float() * ratio[:, :, None, None], 0.0)
    now = (was + xn / scale[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    raw[rows] = torch.where((is_old | is_new)[:, None, :, None], now, had)
    scales[rows[:, :, 0] // BLOCK] = scale


def _plain_read_one(s, case, codes, scales, dt):
    Hkv, d = case["Hkv"], case["d"]
    if case["k"]:
        t = s["idx"].long()
        v = _values(codes, scales, _rows(s, Hkv, t.clamp(min=0)))
        return torch.where((t >= 0)[:, None, :, None], v, 0.0).to(dt)
    r = torch.arange(s["n_out"] * Hkv, device="cuda")
    b = torch.searchsorted(s["out_off"] * Hkv, r, right=True) - 1
    length, off = s["len"].long()[b], s["off"]
    at = r - s["out_off"][b] * Hkv
    rows = off[b] * Hkv + at // length * (off[b + 1] - off[b]) + at % length
    return _values(codes, scales, rows).to(dt)


def _plain_index(s):
    t = torch.arange(s["S"], device="cuda").expand(len(s["len"]), -1)
    seen = t < s["len"][:, None]
    k = _values(s["K8"], s["Ks"], s["off"][:-1, None] + torch.where(seen, t, 0))  # [B, S, d]
    dots = torch.relu(s["qI"].float() @ k.transpose(1, 2))  # [B, H, S]
    return torch.where(seen, (s["w"][:, :, None] * dots).sum(1), 0.0)


def _plain_attn(s, case):
    Hkv, L, B = case["Hkv"], case["L"], case["B"]
    G = case["Hq"] // Hkv
    if case["k"]:
        t = s["idx"].long()
        seen = t >= 0
    else:
        t = torch.arange(s["S"], device="cuda").expand(B, -1)
        seen = t < s["len"][:, None]
    rows = _rows(s, Hkv, torch.where(seen, t, 0))
    q = s["Q"].float().view(L, B, Hkv, G, D).permute(1, 2, 0, 3, 4).reshape(B, Hkv, L * G, D)
    z = (q @ _values(s["K8"], s["Ks"], rows).transpose(2, 3)) * s["scale"]
    z = torch.where(seen[:, None, None, :], z, -math.inf)
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(m > -math.inf, m, 0.0))
    total = p.sum(-1, keepdim=True)
    o = (p @ _values(s["V8"], s["Vs"], rows)) / torch.where(total > 0, total, 1.0)
    return o.view(B, Hkv, L, G, D).permute(2, 0, 1, 3, 4).reshape(L, B, case["Hq"], D).to(DTYPES[case["dtype"]])


def _own(s, case):
    import cross_layer_shared_b200 as sa

    op = case["op"]
    if "ws" not in s:  # a user's program keeps its workspace
        if op == "attn":
            n = sa.decode_attn_q8_workspace_size(case["L"], case["B"], s["n_tokens"], s["S"], case["Hq"], case["Hkv"], D,
                                                 case["k"])
        else:
            n = sa.WS_HEADER_BYTES
        s["ws"] = sa.workspace(n)
    if op == "append":
        sa.cache_append_q8(s["newK"], s["newV"], s["K8"], s["Ks"], s.get("V8"), s.get("Vs"), s["off"], s["len"],
                           s["new_off"], s["max_new"], ws=s["ws"])
    elif op == "read":
        sa.cache_read_q8(s["K8"], s["Ks"], s.get("V8"), s.get("Vs"), s["off"], s["len"], s["S"], case["Hkv"],
                         idx=s.get("idx"), out_off=s.get("out_off"), K=s["K"], V=s["V"], ws=s["ws"])
    elif op == "index":
        return sa.index_score_q8(s["qI"], s["w"], s["K8"], s["Ks"], s["off"], s["len"], s["S"], scores=s["scores"],
                                 ws=s["ws"])
    else:
        return sa.decode_attn_q8(s["Q"], s["K8"], s["Ks"], s["V8"], s["Vs"], s["off"], s["len"], s["S"], case["Hkv"],
                                 s["scale"], idx=s.get("idx"), O=s["O"], ws=s["ws"])
    return [x for x in ((s["K8"], s["Ks"], s.get("V8"), s.get("Vs")) if op == "append" else (s["K"], s["V"]))
            if x is not None]


def run(state):
    s, case = state, state["case"]
    if own:
        return _own(s, case)
    if case["op"] == "append":
        _plain_append_one(s, s["newK"], s["K8"], s["Ks"])
        if s["newV"] is None:
            return [s["K8"], s["Ks"]]
        _plain_append_one(s, s["newV"], s["V8"], s["Vs"])
        return [s["K8"], s["Ks"], s["V8"], s["Vs"]]
    if case["op"] == "read":
        dt = DTYPES[case["dtype"]]
        k = _plain_read_one(s, case, s["K8"], s["Ks"], dt)
        return [k, _plain_read_one(s, case, s["V8"], s["Vs"], dt)] if case["pair"] else [k]
    return _plain_index(s) if case["op"] == "index" else _plain_attn(s, case)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    lens, B, op = _lens(case), case["B"], case["op"]
    d, Hkv = case.get("d", D), case.get("Hkv", 1)
    row = d + 4.0 / BLOCK  # a cached row and its share of the block's scale
    size = 2 if case.get("dtype") == "bf16" else 4
    pair = 2 if case.get("pair") or op == "attn" else 1
    if op == "append":
        n = sum(_news(case)) * Hkv * pair
        return {"bytes": n * (d * size + row) + 16 * B, "flops": 3.0 * n * d}
    if op == "read":
        n = (sum(min(case["k"], m) for m in lens) if case["k"] else sum(lens)) * Hkv * pair
        out = (B * case["k"] * Hkv * pair if case["k"] else n) * d * size
        return {"bytes": n * row + out + 4 * B * case["k"] + 24 * B, "flops": 1.0 * n * d}
    if op == "index":
        n = sum(lens)
        return {"bytes": n * (row + 4) + B * case["H"] * (2 * d + 4) + 12 * B, "flops": n * case["H"] * (2.0 * d + 3)}
    n = sum(min(case["k"], m) for m in lens) if case["k"] else sum(lens)
    q = case["L"] * B * case["Hq"] * d
    return {"bytes": 2.0 * n * Hkv * row + q * (2 + size) + 4 * B * case["k"] + 12 * B,
            "flops": 4.0 * n * case["L"] * case["Hq"] * d}


# ------------------------------------------------------------------ the definition in 64 bits, sequence by sequence
def _e4m3(y):
    """y rounded to the nearest e4m3 value, ties to the even code, |y| <= 448."""
    _, e = torch.frexp(y)
    ulp = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return torch.round(y / ulp) * ulp


def exact(case, seed):
    s = prepare(case, seed)
    op, d, Hkv = case["op"], case.get("d", D), case.get("Hkv", 1)
    lens, off = s["len"].tolist(), s["off"].tolist()

    def head(name, b, h, t0=0, t1=None):
        r = off[b] * Hkv + h * (off[b + 1] - off[b])
        t1 = off[b + 1] - off[b] if t1 is None else t1
        sc = s[name + "s"][r // BLOCK:(r + t1 + BLOCK - 1) // BLOCK].double().repeat_interleave(BLOCK)[t0:t1]
        return s[name + "8"][r + t0:r + t1].double() * sc[:, None]

    if op == "append":
        got, new_off = [], s["new_off"].tolist()
        for name in ("K", "V") if case["pair"] else ("K",):
            codes, scales, x = s[name + "8"].double(), s[name + "s"].double(), s["new" + name]
            for b, n in enumerate(lens):
                p0 = n - (new_off[b + 1] - new_off[b])
                start, end = p0 // BLOCK * BLOCK, (n + BLOCK - 1) // BLOCK * BLOCK
                for h in range(Hkv):
                    r = off[b] * Hkv + h * (off[b + 1] - off[b])
                    y = x[new_off[b]:new_off[b + 1], h].double()
                    pad = torch.zeros((end - start, d), dtype=torch.float64, device="cuda")
                    pad[p0 - start:n - start] = y
                    amax = pad.view(-1, BLOCK * d).abs().amax(1)
                    m, e = torch.frexp(amax / 448.0)  # amax / 448 = m 2^e, m in [0.5, 1)
                    e = torch.where(m == 0.5, e - 1, e)
                    sc = torch.exp2(torch.where(amax > 0, e, -126).clamp(min=-126).double())
                    if p0 > start:
                        was = scales[(r + start) // BLOCK].clone()
                        sc[0] = torch.maximum(sc[0], was)
                        part = codes[r + start:r + p0]
                        codes[r + start:r + p0] = _e4m3(part * (was / sc[0]))
                    scales[(r + start) // BLOCK:(r + end) // BLOCK] = sc
                    codes[r + p0:r + n] = _e4m3(y / sc.repeat_interleave(BLOCK)[p0 - start:n - start, None])
            got += [codes, scales]
        return got
    if op == "read":
        got = []
        for name in ("K", "V") if case["pair"] else ("K",):
            if case["k"]:
                out = torch.zeros((case["B"], Hkv, case["k"], d), dtype=torch.float64, device="cuda")
                for b in range(case["B"]):
                    pick = s["idx"][b][s["idx"][b] >= 0].long()
                    for h in range(Hkv):
                        out[b, h, :len(pick)] = head(name, b, h)[pick]
                got.append(out)
            else:
                got.append(torch.cat([head(name, b, h, 0, n) for b, n in enumerate(lens) for h in range(Hkv)]))
        return got
    if op == "index":
        out = torch.zeros((case["B"], s["S"]), dtype=torch.float64, device="cuda")
        for b, n in enumerate(lens):
            dots = head("K", b, 0, 0, n) @ s["qI"][b].double().T
            out[b, :n] = torch.clamp(dots, min=0) @ s["w"][b].double()
        return out
    G = case["Hq"] // Hkv
    out = torch.zeros((case["L"], case["B"], case["Hq"], D), dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        for h in range(Hkv):
            k, v = (head(name, b, h, 0, n) for name in ("K", "V"))
            if case["k"]:
                pick = s["idx"][b][s["idx"][b] >= 0].long()
                k, v = k[pick], v[pick]
            q = s["Q"][:, b, h * G:(h + 1) * G].double()
            out[:, b, h * G:(h + 1) * G] = torch.softmax(q @ k.T * s["scale"], -1) @ v
    return out
