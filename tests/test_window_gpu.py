"""Windowed attention against the fp64 oracle on the GPU: sizes around the
tiles, shared heads, ragged batches, windows and sinks that leave tiles or
rows empty, hidden NaN, large logits, streams and graphs."""
import numpy as np
import pytest
import torch

from free_block_sparse_eigenbasis_b200 import sparsepr as S
from oracle import frames_oracle as F
import frames_util as U

pytestmark = pytest.mark.gpu

# bf16 weights in the second product: half a step of bf16
WEIGHTS = U.HALF[torch.bfloat16]
ROUND = dict(qk_round=2 * 2.0 ** -8 + 2.0 ** -16, v_round=2.0 ** -8)  # fp32 inputs go to bf16


def params(B, Hq, Hkv, Nq, Nk, d, frame=1, window=0, sinks=0, causal=1, **kw):
    return dict(B=B, Hq=Hq, Hkv=Hkv, Nq=Nq, Nk=Nk, d=d, frame=frame, window=window, sinks=sinks,
                causal=causal, **kw)


def inputs(p, dtype, seed, scale=1.0):
    q = U.normal((p["B"], p["Hq"], p["Nq"], p["d"]), seed, dtype, scale)
    k = U.normal((p["B"], p["Hkv"], p["Nk"], p["d"]), seed + 1, dtype, scale)
    v = U.normal((p["B"], p["Hkv"], p["Nk"], p["d"]), seed + 2, dtype)
    return q, k, v


def call(p, q, k, v, n_q=None, n_k=None, stream=None):
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:3], 7.0, device="cuda")
    ws = S.allocate_window_workspace(p, q.dtype)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    S.sparsepr_window_attention(q, k, v, p, out, ws, lse=lse,
                                n_q=None if n_q is None else U.i32(n_q),
                                n_k=None if n_k is None else U.i32(n_k), stream=stream)
    torch.cuda.synchronize()
    return out, lse, U.status(ws)


def see(p):
    return dict(frame=p["frame"], window=p["window"], sinks=p["sinks"], causal=p["causal"])


def verify(p, q, k, v, out, lse, n_q=None, n_k=None, what=""):
    extra = ROUND if q.dtype == torch.float32 else {}
    for b in range(p["B"]):
        n = p["Nq"] if n_q is None else n_q[b]
        L = p["Nk"] if n_k is None else n_k[b]
        ref = F.attention(U.f64(q[b]), U.f64(k[b, :, :L]), U.f64(v[b, :, :L]), n, see(p),
                          p.get("scale", 0.0))
        U.check(out[b, :, :n], lse[b, :, :n], ref, q.dtype, p["d"], WEIGHTS, what=(what, b), **extra)
        # rows behind the sequence are left as they were
        assert (out[b, :, n:] == 7).all() and (lse[b, :, n:] == 7).all()


CASES = [
    # one token, one key; one token over lengths around a tile
    params(1, 1, 1, 1, 1, 64), params(2, 4, 2, 1, 127, 128), params(1, 8, 1, 1, 129, 64),
    params(3, 3, 3, 1, 700, 128, window=200, sinks=3),
    params(1, 2, 2, 1, 2500, 128), params(1, 2, 1, 2, 2500, 64, window=2100, sinks=5),
    # lengths around one and two query tiles
    params(1, 2, 1, 128, 128, 128), params(1, 1, 1, 129, 129, 64), params(1, 2, 2, 255, 255, 128),
    params(1, 1, 1, 257, 257, 128), params(1, 1, 1, 300, 500, 64),
    # windows narrower and wider than a tile, sinks
    params(1, 2, 1, 300, 300, 128, window=1), params(1, 1, 1, 300, 300, 64, window=2, sinks=1),
    params(1, 1, 1, 400, 400, 128, window=128), params(1, 2, 1, 333, 600, 64, window=130, sinks=4),
    params(1, 1, 1, 513, 513, 128, window=200, sinks=140),
    params(1, 1, 1, 300, 300, 128, window=1000, sinks=2000),
    # both directions
    params(1, 2, 2, 200, 300, 128, causal=0), params(1, 1, 1, 300, 300, 64, window=40, causal=0),
    params(1, 2, 1, 260, 700, 128, window=70, sinks=3, causal=0),
    # frames
    params(1, 1, 1, 300, 300, 128, frame=52, window=2, sinks=1),
    params(1, 2, 1, 210, 420, 64, frame=70, window=3, sinks=1, causal=0),
    params(1, 1, 1, 390, 390, 128, frame=130), params(1, 1, 1, 100, 333, 64, frame=1000, window=1),
    # more queries than keys: the first queries stand before the sequence
    params(1, 2, 1, 200, 130, 64), params(1, 1, 1, 70, 3, 128, causal=0),
    # no keys
    params(1, 2, 1, 40, 0, 64),
    # a scale of its own
    params(1, 1, 1, 140, 140, 64, scale=0.5),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_cases(i, dtype):
    p = CASES[i]
    q, k, v = inputs(p, dtype, 10 * i)
    out, lse, st = call(p, q, k, v)
    assert st == 0
    verify(p, q, k, v, out, lse)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kw", [dict(), dict(window=100, sinks=2), dict(causal=0),
                                dict(frame=33, window=2, causal=0)])
def test_ragged_batch(d, kw):
    p = params(5, 4, 2, 150, 290, d, **kw)
    n_q, n_k = [150, 0, 1, 131, 90], [290, 20, 1, 129, 0]
    q, k, v = inputs(p, torch.bfloat16, 3)
    for b in range(5):  # what lies behind a sequence may be anything
        q[b, :, n_q[b]:] = float("nan")
        k[b, :, n_k[b]:] = float("nan")
        v[b, :, n_k[b]:] = float("inf")
    out, lse, st = call(p, q, k, v, n_q, n_k)
    assert st == 0
    verify(p, q, k, v, out, lse, n_q, n_k)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_hidden_keys_do_not_matter(d, value):
    """Keys and values that only some rows see: the others must not meet them."""
    p = params(1, 2, 1, 200, 200, d, window=64, sinks=2)
    q, k, v = inputs(p, torch.bfloat16, 4)
    for j in (5, 77, 130, 199):
        k[0, 0, j, 3] = value
        v[0, 0, j] = value
    k[0, 0, 140] = 1.0
    v[0, 0, 140, 5] = value  # a plain key with such a value
    out, lse, st = call(p, q, k, v)
    assert st == 0
    on = np.stack([F.visible(i, 200, **see(p)) for i in range(200)])
    clean = ~on[:, [5, 77, 130, 140, 199]].any(1)
    assert clean.sum() > 10
    k2, v2 = k.clone(), v.clone()
    for t in (k2, v2):
        t[0, 0, [5, 77, 130, 140, 199]] = 0
    ref = F.attention(U.f64(q[0]), U.f64(k2[0]), U.f64(v2[0]), 200, see(p))
    some = {n: x[:, clean] for n, x in ref.items()}
    U.check(out[0][:, clean], lse[0][:, clean], some, q.dtype, d, WEIGHTS)
    # rows that see key 140 alone of these: NaN or infinite in column 5 only
    only = on[:, 140] & ~on[:, [5, 77, 130, 199]].any(1)
    assert only.sum() >= 5
    o = out[0][:, only].float()
    assert not torch.isfinite(o[..., 5]).any()
    assert torch.isfinite(torch.cat([o[..., :5], o[..., 6:]], -1)).all()


def test_query_rows_with_nan_keep_to_themselves():
    p = params(1, 1, 1, 140, 140, 64)
    q, k, v = inputs(p, torch.bfloat16, 6)
    q[0, 0, 7] = float("nan")
    out, lse, _ = call(p, q, k, v)
    assert torch.isnan(out[0, 0, 7]).all()
    ref = F.attention(U.f64(q[0]), U.f64(k[0]), U.f64(v[0]), 140, see(p))
    rest = [i for i in range(140) if i != 7]
    U.check(out[0][:, rest], lse[0][:, rest], {n: x[:, rest] for n, x in ref.items()}, q.dtype, 64,
            WEIGHTS)


@pytest.mark.parametrize("d", [64, 128])
def test_rising_and_falling_logits(d):
    """Logits that climb by far more than 2^32 in weight along the keys, in
    both halves of a tile, and that fall again."""
    p = params(1, 2, 1, 130, 600, d, causal=0)
    q, k, v = inputs(p, torch.bfloat16, 8, 0.3)
    q[..., 0] = 4.0
    ramp = torch.cat([torch.linspace(-60, 60, 450), torch.linspace(60, -60, 150)])
    k[0, 0, :, 0] = (ramp * (d ** 0.5) / 4).to(torch.bfloat16).cuda()
    q[0, 1, :, 0] = -4.0  # the other head sees them fall first
    out, lse, st = call(p, q, k, v)
    assert st == 0
    verify(p, q, k, v, out, lse)


def test_counts_outside_the_buffers_are_reported_and_clamped():
    p = params(2, 1, 1, 20, 30, 64)
    q, k, v = inputs(p, torch.bfloat16, 9)
    out, lse, st = call(p, q, k, v, [21, -3], [30, 99])
    assert st == 1 << S.ERR_INVALID_ARG
    verify(p, q, k, v, out, lse, [20, 0], [30, 30])


def test_other_stream_graph_and_workspace_of_one_run():
    p = params(2, 4, 2, 150, 260, 128, window=90, sinks=2)
    q, k, v = inputs(p, torch.bfloat16, 11)
    side = torch.cuda.Stream()
    want, want_lse, _ = call(p, q, k, v)
    got, got_lse, _ = call(p, q, k, v, stream=side)
    assert torch.equal(got, want) and torch.equal(got_lse, want_lse)
    # captured, replayed on new inputs
    ws = S.allocate_window_workspace(p, q.dtype)
    sq, sk, sv = (torch.zeros_like(t) for t in (q, k, v))
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:3], device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        S.sparsepr_window_attention(sq, sk, sv, p, out, ws, lse=lse)
    for t, s in zip((q, k, v), (sq, sk, sv)):
        s.copy_(t)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    # without lse
    out2 = torch.zeros_like(q)
    S.sparsepr_window_attention(q, k, v, p, out2, ws)
    assert torch.equal(out2, want)


def test_rows_beyond_32_bit_offsets():
    """The last keys of a buffer of more than 2^32 bytes."""
    N, W = 17_000_000, 300
    k = torch.zeros((1, 1, N, 128), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    k[:, :, -W:], v[:, :, -W:] = U.normal((1, 1, W, 128), 1), U.normal((1, 1, W, 128), 2)
    q = U.normal((1, 2, 5, 128), 3)
    p = params(1, 2, 1, 5, N, 128, window=200)
    out, lse, st = call(p, q, k, v)
    assert st == 0
    ref = F.attention(U.f64(q[0]), U.f64(k[0, :, -W:]), U.f64(v[0, :, -W:]), 5, see(p))
    U.check(out[0], lse[0], ref, q.dtype, 128, WEIGHTS)


def test_calls_on_two_streams_with_workspaces_of_their_own():
    p = params(2, 4, 2, 300, 400, 128, window=130, sinks=2)
    q, k, v = inputs(p, torch.bfloat16, 31)
    want, want_lse, _ = call(p, q, k, v)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [(torch.zeros_like(q), torch.zeros(q.shape[:3], device="cuda"),
             S.allocate_window_workspace(p, q.dtype)) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(10):
        for st, (out, lse, ws) in zip(streams, outs):
            S.sparsepr_window_attention(q, k, v, p, out, ws, lse=lse, stream=st)
    torch.cuda.synchronize()
    for out, lse, ws in outs:
        assert torch.equal(out, want) and torch.equal(lse, want_lse) and U.status(ws) == 0


def test_no_query_rows():
    p = params(1, 2, 1, 0, 10, 64)
    q, k, v = inputs(p, torch.bfloat16, 12)
    out, lse, st = call(p, q, k, v)
    assert st == 0 and out.numel() == 0


def test_same_as_the_dense_kernel_without_a_window():
    """causal = 0 and no window is the dense attention that the library has."""
    H, N, d = 2, 640, 128
    q, k, v = (U.normal((H, N, d), 20 + i) for i in range(3))
    dense = torch.empty((H, N, d), device="cuda")
    S.dense_attention(q, k, v, dense)
    p = params(1, H, H, N, N, d, causal=0)
    out, _, _ = call(p, q[None], k[None], v[None])
    # both round their weights to bf16 and the output here once more
    assert (out[0].double() - dense.double()).abs().max() <= 4 * 2.0 ** -8


@pytest.mark.parametrize("see_", [
    dict(frame=2 ** 31 - 1, window=2 ** 31 - 1, sinks=2 ** 31 - 1, causal=0),
    dict(frame=2 ** 31 - 1, window=1, causal=1), dict(frame=2 ** 30, window=2 ** 31 - 1, causal=1),
    dict(frame=1, window=2 ** 31 - 1, sinks=2 ** 31 - 1, causal=1),
    dict(frame=3, window=2 ** 31 - 1, causal=0)])
def test_largest_frames_windows_and_sinks(see_):
    p = params(1, 6, 2, 150, 420, 64, **see_)
    q, k, v = inputs(p, torch.bfloat16, 31)
    out, lse, status = call(p, q, k, v)
    assert status == 0
    verify(p, q, k, v, out, lse)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("sizes", [(3, 21, 7, 37, 301), (2, 10, 2, 131, 517), (1, 13, 13, 257, 259),
                                   (5, 6, 3, 43, 1025)])
def test_sizes_that_divide_nothing(sizes, dtype):
    """Rows, heads, groups, frames and splits that no power of two divides."""
    for d, frame, window, sinks, causal in ((128, 7, 5, 3, 1), (64, 11, 3, 0, 0), (64, 1, 0, 0, 1)):
        p = params(*sizes, d, frame, window, sinks, causal)
        q, k, v = inputs(p, dtype, 77)
        B, Nq, Nk = p["B"], p["Nq"], p["Nk"]
        n_q, n_k = [Nq - 3 * b for b in range(B)], [Nk - 101 * b for b in range(B)]
        out, lse, status = call(p, q, k, v, n_q, n_k)
        assert status == 0
        verify(p, q, k, v, out, lse, n_q, n_k, what=(d, frame))


@pytest.mark.parametrize("splits", [False, True])
def test_behind_copies_and_other_streams(splits):
    """The inputs are the results of copies, fills and of another stream's work
    right before the call, eagerly and in a captured graph; calls that depend on
    one another follow without a pause."""
    # one unit of many keys is cut, many units are not
    p = params(1, 2, 2, 3, 5000, 128) if splits else params(2, 40, 40, 300, 400, 128, window=64)
    q, k, v = inputs(p, torch.bfloat16, 41)
    k2, v2 = k.flip(2).contiguous(), v.flip(2).contiguous()
    first, _, _ = call(p, q, k, v)
    want, want_lse, _ = call(p, first, k2, v2)
    side = torch.cuda.Stream()
    sq, sk, sv, mid, out = (torch.zeros_like(t) for t in (q, k, v, q, q))
    lse = torch.zeros(q.shape[:3], device="cuda")
    ws = S.allocate_window_workspace(p, q.dtype)

    def step():
        out.zero_()
        sk.copy_(k)
        sv.copy_(v)
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            sq.copy_(q)
        here.wait_stream(side)
        S.sparsepr_window_attention(sq, sk, sv, p, mid, ws)
        sk.copy_(k2)
        sv.fill_(0)
        sv.copy_(v2)
        S.sparsepr_window_attention(mid, sk, sv, p, out, ws, lse=lse)  # the same workspace
        S.sparsepr_window_attention(mid, sk, sv, p, out, ws, lse=lse)

    for _ in range(5):
        step()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(5):
        for t in (sq, sk, sv, mid, out, lse):
            t.fill_(5)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert U.status(ws) == 0


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("H,Nk,weak", [(2, 5000, 4000), (2, 256, 128), (296, 256, 128)])
def test_values_that_are_not_finite_under_vanishing_weights(H, Nk, weak, value):
    """The first keys lie 512 log2 units below the others, so that whole parts of the sum
    weigh 0 in fp32 where they are joined; 0 times a NaN or an infinity is NaN there as
    everywhere, whether the keys are cut into ranges or not."""
    p = params(1, H, H, 3, Nk, 128, causal=0, scale=1.0)
    q, k, v = inputs(p, torch.bfloat16, 5, 0.1)
    q[..., 0], k[..., 0] = 16.0, 0.0
    k[:, :, :weak, 0] = -22.25
    ref = F.attention(U.f64(q[0]), U.f64(k[0]), U.f64(v[0]), 3, see(p), 1.0)
    v[0, :, 10, 5] = value
    out, lse, st = call(p, q, k, v)
    assert st == 0
    assert not torch.isfinite(out[..., 5]).any()
    keep = [c for c in range(128) if c != 5]
    U.check(out[0][..., keep], lse[0], dict(ref, out=ref["out"][..., keep], mass=ref["mass"][..., keep]),
            q.dtype, 128, WEIGHTS)


@pytest.mark.parametrize("scale", [1e-300, 1e-42, 1e-39])
def test_scales_below_the_normal_numbers(scale):
    """All visible keys weigh the same, and masked ones nothing."""
    p = params(1, 2, 1, 200, 300, 64, window=70, sinks=2, scale=scale)
    q, k, v = inputs(p, torch.bfloat16, 51)
    out, lse, st = call(p, q, k, v)
    assert st == 0
    verify(p, q, k, v, out, lse)


@pytest.mark.parametrize("bad", ["values", "keys", "both"])
@pytest.mark.parametrize("p", [
    params(1, 2, 1, 700, 700, 128, window=150, sinks=3), params(1, 3, 1, 40, 900, 64, window=300, sinks=5),
    params(1, 1, 1, 600, 600, 64, frame=50, window=3, sinks=1, causal=0),
    params(1, 2, 2, 300, 300, 128, frame=130, window=1, sinks=2),
    params(2, 4, 2, 257, 511, 128, causal=0), params(1, 1, 1, 500, 500, 128),
    params(1, 2, 2, 3, 4000, 64, window=3900), params(1, 1, 1, 300, 200, 64, window=60, sinks=1)])
def test_nan_shows_where_it_is_seen_and_nowhere_else(p, bad):
    """NaN values in single columns, and NaN keys, seen by some rows and hidden from others
    of the same tile."""
    q, k, v = inputs(p, torch.bfloat16, 61)
    rng = np.random.default_rng(p["Nk"])
    for b in range(p["B"]):
        for h in range(p["Hkv"]):
            for j in rng.integers(0, p["Nk"], 4):
                if bad != "keys":
                    v[b, h, int(j), int(rng.integers(p["d"]))] = float("nan")
            if bad != "values":
                k[b, h, int(rng.integers(p["Nk"])), 3] = float("nan")
    out, lse, st = call(p, q, k, v)
    assert st == 0
    verify(p, q, k, v, out, lse)


@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("d", [64, 128])
def test_what_every_row_sees_costs_no_second_pass(d, causal):
    """A NaN and an infinity in the sink frame, and a NaN key there: columns that they do not
    touch are those of the call without them, bit for bit, and the calls take no more than
    a few times as long (rows taken again one by one took 100 to 250 times as long here). So
    are rows from whose tiles a NaN is hidden altogether, though it lies right behind the sinks."""
    p = params(1, 2, 1, 4000, 4000, d, frame=200, window=3, sinks=1, causal=causal)
    q, k, v = inputs(p, torch.bfloat16, 5)
    ws = S.allocate_window_workspace(p, q.dtype)
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:3], device="cuda")

    def go(k, v):
        best = 1e9
        for _ in range(6):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            torch.cuda.synchronize()
            a.record()
            S.sparsepr_window_attention(q, k, v, p, out, ws, lse=lse)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        return out.clone(), lse.clone(), best
    clean, clean_lse, t0 = go(k, v)
    v2, k2 = v.clone(), k.clone()
    v2[0, 0, 7, 5], v2[0, 0, 9, 6], k2[0, 0, 7, 5] = float("nan"), float("inf"), float("nan")
    got, got_lse, t1 = go(k, v2)
    keep = [c for c in range(d) if c not in (5, 6)]
    assert torch.isnan(got[..., 5]).all() and (got[..., 6] == float("inf")).all()
    assert torch.equal(got_lse, clean_lse) and torch.equal(got[..., keep], clean[..., keep])
    got, got_lse, t2 = go(k2, v)
    assert torch.isnan(got).all() and torch.isnan(got_lse).all()
    v3 = v.clone()
    v3[0, 0, 210] = float("nan")  # frame 1: seen up to frame 3
    got, got_lse, _ = go(k, v3)
    assert torch.isnan(got[:, :, 200:800]).all() and torch.isfinite(got[:, :, 800:]).all()
    # (rows 800 to 1023 share their unit with rows that see it, and are taken again)
    assert torch.equal(got[:, :, 1024:], clean[:, :, 1024:])
    assert torch.equal(got_lse[:, :, 1024:], clean_lse[:, :, 1024:])
    got, _, t3 = go(k, torch.full_like(v, float("nan")))
    assert torch.isnan(got).all()
    assert max(t1, t2, t3) < 20 * t0, (t0, t1, t2, t3)


@pytest.mark.parametrize("d", [64, 128])
def test_leaps_of_logits(d):
    """Logits that leap by 20,000 and more log2 units between groups of keys: whole numbers up
    to 2^14 and a little, which fp32 sums exactly. (Not further: at 2^24 fp32 rounds the logits
    themselves by whole units, and the bounds, linear in that rounding, say nothing.)"""
    p = params(1, 2, 1, 600, 600, d, scale=1.0)
    q, k, v = inputs(p, torch.bfloat16, 71)
    q, k = torch.round(q), torch.round(k)
    q[..., 0] = 16.0
    for n, x in ((0, -1024.0), (200, 0.0), (300, 1024.0)):
        k[:, :, n:, 0] = x
    q[:, 1, :, 0] = -16.0  # the other head leaps down
    out, lse, st = call(p, q, k, v)
    assert st == 0
    verify(p, q, k, v, out, lse)
