"""Pins of the oracle of the windowed attention and the 8-bit cache (CPU)."""
import numpy as np
import pytest
import torch

from oracle import frames_oracle as F


def test_e4m3_table_and_rounding_match_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    ours = F.TABLE
    theirs = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ours, theirs, equal_nan=True)
    g = torch.Generator().manual_seed(0)
    x = torch.cat([torch.randn(4000, generator=g) * s for s in (1e-3, 0.02, 1.0, 60.0)])
    x = x.clamp(-448, 448)
    # every midpoint between neighbours: the ties
    pos = torch.from_numpy(F._POS)
    mid = ((pos[1:] + pos[:-1]) / 2).float()
    x = torch.cat([x, mid, -mid])
    assert np.array_equal(F.e4m3_encode(x.double().numpy()),
                          x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())


@pytest.mark.parametrize("amax,scale", [
    (448.0, 1.0), (np.nextafter(448.0, 500.0), 2.0), (224.0, 0.5), (1.0, 2.0 ** -8),
    (0.0, 2.0 ** -110), (3.3e38, 2.0 ** 120)])
def test_scale(amax, scale):
    assert F.scale_for(amax) == scale


def test_visibility_by_hand():
    # frames of 2 tokens; position 7 lies in frame 3
    assert F.visible(7, 10, 2, 2, 1, 1).nonzero()[0].tolist() == [0, 1, 4, 5, 6, 7]
    assert F.visible(7, 10, 2, 2, 1, 0).nonzero()[0].tolist() == [0, 1, 4, 5, 6, 7, 8, 9]
    assert F.visible(6, 7, 2, 1, 0, 1).nonzero()[0].tolist() == [6]
    assert F.visible(0, 3, 1, 0, 0, 1).nonzero()[0].tolist() == [0]
    assert F.visible(0, 3, 1, 0, 0, 0).all()
    assert not F.visible(-1, 3, 1, 0, 2, 0).any()


def test_attention_of_one_visible_key_is_that_value():
    rng = np.random.default_rng(0)
    q, k, v = rng.normal(size=(2, 3, 4)), rng.normal(size=(1, 3, 4)), rng.normal(size=(1, 3, 4))
    r = F.attention(q, k, v, 3, dict(frame=1, window=1, sinks=0, causal=1))
    assert np.allclose(r["out"], np.broadcast_to(v, (2, 3, 4)))
    assert np.allclose(r["lse"], 0.5 * np.einsum("hid,xid->hi", q, k))


def test_model_fork_copies_on_write_and_packs():
    p = dict(B=3, Hkv=1, d=64, page=16, n_pages=8, max_pages=4)
    m = F.CacheModel(p)
    rng = np.random.default_rng(1)
    start = m.reserve([20, 0, 0])
    x = rng.normal(size=(3, 1, 20, 64))
    m.append(x, x, start, [20, 0, 0])
    assert m.fork([0], [1]) and m.ref.tolist()[:2] == [2, 2]
    start = m.reserve([0, 1, 0])
    assert start.tolist() == [20, 20, 0]
    assert m.table[1].tolist() == [0, 2, -1, -1] and m.ref.tolist()[:3] == [2, 1, 1]
    before = m.tokens(0)
    m.append(10 * x[:, :, :1], x[:, :, :1], start, [0, 1, 0])
    assert np.array_equal(m.tokens(0), before)
    m.free([0, 0])
    assert m.ref.tolist()[:3] == [1, 0, 1] and m.len.tolist() == [0, 21, 0]
    kept = m.tokens(1)
    assert m.compact() == 2 and m.table[1].tolist() == [0, 1, -1, -1]
    assert np.array_equal(m.tokens(1), kept)
    assert m.reserve([0, 40, 0]) is not None and m.reserve([64, 64, 64]) is None
