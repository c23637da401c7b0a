"""Helpers of the GPU tests of the windowed attention and the 8-bit cache."""
import numpy as np
import torch

from oracle import frames_oracle as F

# half a step of each type, relative to the value
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def bounds(ref, dtype, d, weights, qk_round, v_round):
    """Largest allowed errors of out and lse.

    A logit is a sum of d fp32 products (each add rounds to 2^-24 of at most
    the sum of magnitudes, `spread`), scaled and shifted with a handful more
    roundings: |ds| <= (2 d + 16) 2^-24 spread, plus the rounding of q and k
    where they are rounded (qk_round, relative, both together). A weight then
    is off by at most 2 |ds| (itself and the sum that divides it) + 2^-16 (the
    exponential and the fp32 sums) + the rounding of the weights before the
    second product; v_round: the rounding of the values. The output adds its own
    rounding."""
    ds = ((2 * d + 16) * 2.0 ** -24 + qk_round) * ref["spread"]
    rel = 2 * ds + 2.0 ** -16 + weights + v_round
    out = rel[..., None] * ref["mass"] + HALF[dtype] * np.abs(ref["out"]) * (1 + 2.0 ** -8)
    lse = ds + 2.0 ** -16 + 2.0 ** -22 * np.abs(np.where(np.isfinite(ref["lse"]), ref["lse"], 0))
    return out + 1e-30, lse


def check(out, lse, ref, dtype, d, weights, qk_round=0.0, v_round=0.0, what=""):
    """out [Hq, n, d] and lse [Hq, n] of one sequence against the oracle."""
    tol_o, tol_l = bounds(ref, dtype, d, weights, qk_round, v_round)
    o, x = out.double().cpu().numpy(), lse.double().cpu().numpy()
    nan = np.isnan(ref["out"])
    assert np.array_equal(np.isnan(o), nan), (what, "NaN in other places")
    with np.errstate(invalid="ignore"):
        far = np.where(nan, 0, np.abs(o - ref["out"]) / tol_o)
    assert far.size == 0 or far.max() <= 1, (what, "out", float(far.max()),
                                             np.unravel_index(far.argmax(), far.shape))
    empty = np.isneginf(ref["lse"])
    assert np.array_equal(np.isneginf(x), empty), (what, "empty rows")
    bad = np.isnan(ref["lse"]) | empty
    with np.errstate(invalid="ignore"):
        far = np.where(bad, 0, np.abs(x - ref["lse"]) / tol_l)
    assert far.size == 0 or far.max() <= 1, (what, "lse", float(far.max()),
                                             np.unravel_index(far.argmax(), far.shape))


def f64(t):
    return t.detach().double().cpu().numpy()


def status(ws):
    """The device status word at the start of a workspace."""
    return int(ws[:4].view(torch.int32).item())


def normal(shape, seed, dtype=torch.bfloat16, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def to_model(p, c):
    """The host model of a device cache."""
    m = F.CacheModel(p)
    m.k8, m.v8 = (x.view(torch.uint8).cpu().numpy().copy() for x in (c.k8, c.v8))
    m.k_scale, m.v_scale = f64(c.k_scale), f64(c.v_scale)
    m.table = c.table.cpu().numpy().astype(np.int64)
    m.len, m.ref = (x.cpu().numpy().astype(np.int64) for x in (c.len, c.ref))
    return m


def same_cache(m, c, what=""):
    """The device cache holds what the model does, pages in use bit for bit (NaN
    codes count as equal)."""
    assert np.array_equal(c.table.cpu().numpy(), m.table), (what, "table")
    assert np.array_equal(c.len.cpu().numpy(), m.len), (what, "len")
    assert np.array_equal(c.ref.cpu().numpy(), m.ref), (what, "ref")
    assert np.array_equal(f64(c.k_scale), m.k_scale), (what, "k_scale")
    assert np.array_equal(f64(c.v_scale), m.v_scale), (what, "v_scale")
    for name in ("k8", "v8"):
        got, want = getattr(c, name).view(torch.uint8).cpu().numpy(), getattr(m, name)
        same = (got == want) | (np.isnan(F.TABLE[got]) & np.isnan(F.TABLE[want]))
        assert same.all(), (what, name, int((~same).sum()))
