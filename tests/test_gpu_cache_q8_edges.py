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
