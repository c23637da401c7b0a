"""The paged 8-bit cache on the GPU: pages, scales and codes against the host
model bit for bit, attention against the fp64 oracle, and a whole rollout."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from free_block_sparse_eigenbasis_b200 import sparsepr as S
from oracle import frames_oracle as F
import frames_util as U

pytestmark = pytest.mark.gpu

F16 = U.HALF[torch.float16]  # weights are rounded to 11 bits at least
Q32 = 2.0 ** -11             # fp32 queries too


def weights(rows):
    """Half a step of the weights' type: fp16 while the cache is read in place
    (up to 32 query rows per key head), bf16 beyond."""
    return F16 if rows <= 32 else U.HALF[torch.bfloat16]


def rounding(rows, dtype):
    """Rounding of the queries: none for bf16 values; fp32 goes to 11 bits, beyond
    32 rows to bf16."""
    return 0.0 if dtype == torch.bfloat16 else Q32 if rows <= 32 else U.HALF[torch.bfloat16]


def cache_params(B, Hkv, d, page, n_pages, max_pages):
    return dict(B=B, Hkv=Hkv, d=d, page=page, n_pages=n_pages, max_pages=max_pages)


class Run:
    """A device cache beside its host model."""

    def __init__(self, p, seed=0):
        self.p, self.rng = p, np.random.default_rng(seed)
        self.c, self.m = S.allocate_cache(p), F.CacheModel(p)
        self.ws = S.allocate_cache_workspace(p)
        self.start = U.i32([0] * p["B"])

    def status(self):
        st = U.status(self.ws)
        S.sparsepr_reset_stats(self.ws)
        return st

    def reserve(self, n):
        S.sparsepr_cache_reserve(U.i32(n), self.p, self.c, self.start, self.ws)
        want = self.m.reserve(n)
        got = self.start.cpu().numpy()
        assert (got == (-1 if want is None else want)).all()
        return want is not None

    def append(self, n, dtype=torch.bfloat16, scale=1.0, T=None):
        p = self.p
        T = max(n) if T is None else T
        seed = int(self.rng.integers(1 << 30))
        k = U.normal((p["B"], p["Hkv"], T, p["d"]), seed, dtype, scale)
        v = U.normal((p["B"], p["Hkv"], T, p["d"]), seed + 1, dtype, 0.1 * scale)
        S.sparsepr_cache_append(k, v, p, self.c, self.start, U.i32(n), self.ws)
        self.m.append(U.f64(k), U.f64(v), self.start.cpu().numpy(), n)

    def grow(self, n, **kw):
        assert self.reserve(n)
        if max(n):
            self.append(n, **kw)

    def same(self, what=""):
        U.same_cache(self.m, self.c, what)

    def attend(self, attn, dtype=torch.bfloat16, n_q=None, seed=5, what="", scale=1.0, ws=None):
        p = self.p
        q = U.normal((p["B"], attn["Hq"], attn["Nq"], p["d"]), seed, dtype, scale)
        out = torch.full_like(q, 7.0)
        lse = torch.full(q.shape[:3], 7.0, device="cuda")
        ws = S.allocate_cache_workspace(p, attn) if ws is None else ws
        S.sparsepr_cache_attention(q, p, self.c, attn, out, ws, lse=lse,
                                   n_q=None if n_q is None else U.i32(n_q))
        torch.cuda.synchronize()
        see = {n: attn.get(n, d) for n, d in (("frame", 1), ("window", 0), ("sinks", 0),
                                              ("causal", 1))}
        for b in range(p["B"]):
            n = attn["Nq"] if n_q is None else n_q[b]
            ref = F.attention(U.f64(q[b]), self.m.tokens(b, "k"), self.m.tokens(b, "v"), n, see,
                              attn.get("scale", 0.0))
            rows = attn["Hq"] // p["Hkv"] * attn["Nq"]
            U.check(out[b, :, :n], lse[b, :, :n], ref, dtype, p["d"], weights(rows),
                    qk_round=rounding(rows, dtype), what=(what, b))
            assert (out[b, :, n:] == 7).all() and (lse[b, :, n:] == 7).all()
        return U.status(ws)


# ---- append -------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_append_codes_and_scales(page, d, dtype):
    r = Run(cache_params(3, 2, d, page, 60, 20), page + d)
    r.grow([1, 0, page], dtype=dtype)
    r.grow([page // 2, 3, 1], dtype=dtype, scale=0.3)
    r.grow([2 * page + 5, 1, page - 1], dtype=dtype, scale=20.0)  # scales grow inside pages
    r.grow([0, 0, 1], dtype=dtype, scale=1e-3)
    r.grow([1, 1, 1], dtype=dtype, scale=500.0)
    r.grow([3, 2, 0], dtype=dtype, T=7)  # a padded batch
    assert r.status() == 0
    r.same()


def test_append_one_token_at_a_time_equals_its_definition():
    r = Run(cache_params(2, 1, 64, 16, 10, 4), 1)
    for i in range(37):
        r.grow([1, i % 2], scale=float(1.0 + (i % 5) ** 3))
    assert r.status() == 0
    r.same()


def test_append_extremes():
    """Zeros, values at the limits of the types, ties between codes, NaN and
    infinities; tiny values under a large one in the same page."""
    p = cache_params(1, 1, 64, 16, 8, 4)
    rows = torch.zeros(1, 1, 40, 64)
    rows[0, 0, 1] = 3.3e38
    rows[0, 0, 2] = torch.linspace(0, 1e-38, 64)
    rows[0, 0, 16] = 448.0
    rows[0, 0, 17] = torch.arange(64) * 2.0 ** -10  # ties and subnormal codes at scale 1
    rows[0, 0, 18] = 448.0 * 2.0 ** -9 * torch.linspace(-1, 1, 64)
    rows[0, 0, 20, 3], rows[0, 0, 20, 4], rows[0, 0, 20, 5] = float("nan"), float("inf"), -float("inf")
    rows[0, 0, 33] = 1e-36  # under the smallest scale
    for dtype in (torch.float32, torch.bfloat16):
        r = Run(p)
        x = rows.to(dtype).cuda()
        assert r.reserve([40])
        S.sparsepr_cache_append(x, -x, p, r.c, r.start, None, r.ws)
        r.m.append(U.f64(x), -U.f64(x), [0], [40])
        assert r.status() == 0
        r.same(dtype)


def test_append_refuses_pages_it_may_not_write():
    p = cache_params(3, 1, 64, 16, 10, 3)
    r = Run(p)
    r.grow([20, 5, 0])
    S.sparsepr_cache_fork(U.i32([0]), U.i32([2]), p, r.c, r.ws)
    r.m.fork([0], [2])
    x = torch.ones(3, 1, 4, 64, dtype=torch.bfloat16, device="cuda")
    for start, n in (([20, -1, -1], [4, 0, 0]),      # a page that two sequences share
                     ([-1, 32, -1], [0, 2, 0]),      # an entry without a page
                     ([-1, 46, -1], [0, 4, 0])):     # past the table (and no page before that)
        S.sparsepr_cache_append(x, x, p, r.c, U.i32(start), U.i32(n), r.ws)
        assert r.status() == 1 << S.ERR_INVALID_ARG, (start, n)
        r.same()
    S.sparsepr_cache_append(x, x, p, r.c, U.i32([-1, 5, -1]), U.i32([0, 9, 0]), r.ws)
    assert r.status() == 1 << S.ERR_INVALID_ARG  # nine tokens of four: four are written
    r.m.append(U.f64(x), U.f64(x), [-1, 5, -1], [0, 4, 0])
    r.same()


# ---- pages ----------------------------------------------------------------------
def test_reserve_all_or_nothing():
    p = cache_params(3, 1, 64, 16, 5, 4)
    r = Run(p)
    r.grow([17, 16, 0])
    assert not r.reserve([20, 16, 1]) and r.status() == 1 << S.ERR_CAPACITY
    r.same()
    assert not r.reserve([48, 0, 0]) and r.status() == 1 << S.ERR_CAPACITY  # row too short
    r.same()
    assert not r.reserve([1, -1, 0]) and r.status() == 1 << S.ERR_INVALID_ARG
    r.same()
    # the last two pages, exactly
    assert r.reserve([15, 1, 16]) and r.status() == 0
    r.same()
    assert r.reserve([0, 0, 0]) and r.status() == 0
    r.same()
    assert not r.reserve([1, 0, 0])


def test_fork_refusals():
    p = cache_params(6, 1, 64, 16, 12, 3)
    r = Run(p)
    r.grow([20, 5, 0, 0, 0, 0])
    # to itself, to a sequence in use, twice to one, from a target, outside; one good pair
    src = [0, 0, 0, 1, 2, 9, 1]
    dst = [0, 1, 3, 3, 5, 4, 2]
    S.sparsepr_cache_fork(U.i32(src), U.i32(dst), p, r.c, r.ws)
    assert r.status() == 1 << S.ERR_INVALID_ARG
    assert not r.m.fork(src, dst)
    r.same()
    S.sparsepr_cache_fork(U.i32([0, 0]), U.i32([3, 4]), p, r.c, r.ws)
    assert r.m.fork([0, 0], [3, 4]) and r.status() == 0
    r.same()
    S.sparsepr_cache_free(U.i32([4, 4, 5, 17, -2]), p, r.c, r.ws)
    r.m.free([4, 4, 5, 17, -2])
    assert r.status() == 1 << S.ERR_INVALID_ARG
    r.same()


@pytest.mark.parametrize("seed", range(6))
def test_random_life_of_a_cache(seed):
    """Rollouts branch, grow, end, lose old frames and are packed, in any order."""
    rng = np.random.default_rng(seed)
    page = [16, 32, 64, 128, 16, 64][seed]
    B = [6, 40, 5, 4, 9, 7][seed]
    p = cache_params(B, [1, 2, 3, 1, 12, 1][seed], [64, 128][seed % 2], page, 7 * B, 9)
    r = Run(p, seed)
    for step in range(40):
        op = rng.integers(6)
        if op <= 1:
            n = [int(x) for x in rng.integers(0, 2 * page, B) * (rng.random(B) < 0.4)]
            if r.reserve(n):
                r.append(n, scale=float(rng.choice([0.1, 1.0, 30.0])), T=max(1, max(n)))
        elif op == 2:
            some = rng.permutation(B)[:rng.integers(1, B + 1)]
            half = len(some) // 2
            s = [int(x) for x in rng.choice(some[:half], half)] if half else []
            t = [int(x) for x in some[half:2 * half]]
            if s:
                S.sparsepr_cache_fork(U.i32(s), U.i32(t), p, r.c, r.ws)
                r.m.fork(s, t)
        elif op == 3:
            s = [int(x) for x in rng.integers(0, B, rng.integers(1, max(2, B // 3)))]
            S.sparsepr_cache_free(U.i32(s), p, r.c, r.ws)
            r.m.free(s)
        elif op == 4:
            see = dict(frame=int(rng.integers(1, 20)), window=int(rng.integers(1, 9)),
                       sinks=int(rng.integers(0, 3)), causal=1)
            S.sparsepr_cache_evict(see, p, r.c, r.ws)
            r.m.evict(see["frame"], see["window"], see["sinks"])
        else:
            used = U.i32([0])
            S.sparsepr_cache_compact(p, r.c, used, r.ws)
            assert int(used) == r.m.compact()
        r.same((seed, step, int(op)))


def test_wide_pool_and_many_sequences():
    """More pages and sequences than one round of the planning block."""
    p = cache_params(1024, 1, 64, 16, 5000, 6)
    r = Run(p)
    rng = np.random.default_rng(0)
    n = [int(x) for x in rng.integers(0, 40, 1024)]
    assert r.reserve(n)
    r.same()
    s = [int(x) for x in rng.permutation(1024)[:600]]
    S.sparsepr_cache_free(U.i32(s), p, r.c, r.ws)
    r.m.free(s)
    n = [int(x) for x in rng.integers(0, 50, 1024)]
    assert r.reserve(n)
    r.same()
    used = U.i32([0])
    S.sparsepr_cache_free(U.i32(list(range(0, 1024, 3))), p, r.c, r.ws)
    r.m.free(list(range(0, 1024, 3)))
    S.sparsepr_cache_compact(p, r.c, used, r.ws)
    assert int(used) == r.m.compact()
    r.same()


# ---- attention ------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("page,d,Hkv,group,Nq,kw", [
    (64, 128, 2, 1, 1, {}), (16, 64, 1, 8, 1, {}), (128, 128, 3, 2, 1, dict(window=50, sinks=3)),
    (32, 64, 2, 4, 2, {}), (64, 128, 1, 16, 1, {}), (16, 128, 1, 3, 5, dict(window=20)),
    (128, 64, 1, 1, 17, dict(causal=0)), (64, 64, 2, 5, 7, dict(frame=10, window=3, sinks=1)),
    (32, 128, 1, 2, 33, dict(window=7, sinks=40)), (16, 64, 1, 1, 130, dict(frame=13, window=4)),
    (64, 128, 2, 1, 140, {}), (128, 128, 1, 4, 70, dict(window=64, causal=0)),
])
def test_attention(page, d, Hkv, group, Nq, kw, dtype):
    p = cache_params(4, Hkv, d, page, 70, 24)
    r = Run(p, page + Nq)
    r.grow([min(23 * page, 300), 1, 0, 129])
    r.grow([70, 6, 0, page], scale=3.0)
    attn = dict(Hq=Hkv * group, Nq=Nq, **kw)
    assert r.attend(attn, dtype) == 0
    assert r.attend(attn, dtype, n_q=[Nq, 0, min(Nq, 1), max(1, Nq - 1)], seed=8) == 0


def test_attention_over_long_and_short_sequences():
    p = cache_params(6, 2, 64, 16, 700, 200)
    r = Run(p, 3)
    r.grow([3000, 1, 17, 0, 640, 2000])
    for Nq, kw in ((1, {}), (1, dict(window=900, sinks=5)), (3, dict(frame=100, window=4, sinks=1))):
        assert r.attend(dict(Hq=8, Nq=Nq, **kw)) == 0


def test_bytes_behind_a_sequence_do_not_matter():
    """Codes of NaN in the rest of the last page and in every page not in use."""
    p = cache_params(3, 2, 128, 64, 20, 4)
    r = Run(p, 4)
    for c in (r.c.k8, r.c.v8):
        c.view(torch.uint8).fill_(0x7F)
    r.c.k_scale.fill_(float("nan"))
    r.c.v_scale.fill_(float("nan"))
    r.m = U.to_model(p, r.c)
    r.grow([70, 1, 128])
    for Nq in (1, 4, 130):
        assert r.attend(dict(Hq=4, Nq=Nq)) == 0


@pytest.mark.parametrize("Nq", [3, 20, 100])
def test_hidden_tokens_do_not_matter(Nq):
    """A NaN token that later queries see and earlier ones do not."""
    p = cache_params(1, 1, 64, 16, 20, 16)
    r = Run(p, 5)
    r.grow([150])
    x = U.normal((1, 1, 2, 64), 3)
    x[0, 0, 1] = float("nan")
    assert r.reserve([2])
    S.sparsepr_cache_append(x, x, p, r.c, r.start, None, r.ws)
    r.m.append(U.f64(x), U.f64(x), r.start.cpu().numpy(), [2])
    r.same()
    assert r.attend(dict(Hq=2, Nq=Nq)) == 0


def test_evicted_pages_are_not_read():
    p = cache_params(2, 1, 64, 16, 40, 16)
    r = Run(p, 6)
    r.grow([200, 90])
    see = dict(frame=5, window=8, sinks=2, causal=1)
    S.sparsepr_cache_evict(see, p, r.c, r.ws)
    r.m.evict(5, 8, 2)
    assert (r.m.table[0] < 0).sum() > 12 - 8
    r.same()
    r.grow([1, 1])
    assert r.attend(dict(Hq=3, Nq=1, **see)) == 0
    # queries that would look at them: reported, and NaN; those that do not are as they were
    for Nq in (1, 70):
        a = dict(Hq=1, Nq=Nq, frame=5, window=25, sinks=2)
        ws = S.allocate_cache_workspace(p, a)
        q = U.normal((2, 1, Nq, 64), 1)
        out = torch.zeros_like(q)
        S.sparsepr_cache_attention(q, p, r.c, a, out, ws)
        assert U.status(ws) == 1 << S.ERR_INVALID_ARG
        for b in range(2):
            k, v = r.m.tokens(b, "k"), r.m.tokens(b, "v")
            ref = F.attention(U.f64(q[b]), k, v, Nq, dict(frame=5, window=25, sinks=2, causal=1))
            lost = np.isnan(ref["out"]).any(-1)
            assert lost.any() and np.isnan(U.f64(out[b])[lost]).all()
            tol, _ = U.bounds(ref, q.dtype, 64, weights(Nq), 0.0, 0.0)
            assert (np.abs(U.f64(out[b]) - ref["out"])[~lost] <= tol[~lost]).all()


def test_what_lies_behind_the_sinks_does_not_matter():
    """Widened pages: the rows between the sinks and the window are whatever the
    workspace held."""
    p = cache_params(2, 1, 64, 16, 80, 40)
    r = Run(p, 17)
    r.grow([600, 400])
    see = dict(frame=1, window=100, sinks=20, causal=1)
    attn = dict(Hq=1, Nq=50, **see)
    S.sparsepr_cache_evict(dict(see, window=150), p, r.c, r.ws)
    r.m.evict(1, 150, 20)
    ws = S.allocate_cache_workspace(p, attn)
    ws.fill_(0xFF)  # NaN in every type
    S.sparsepr_reset_stats(ws)
    assert r.attend(attn, ws=ws) == 0


def test_first_call_inside_a_capture():
    p = cache_params(1, 1, 64, 32, 8, 4)
    r = Run(p, 19)
    r.grow([100])
    for Nq in (1, 40):
        attn = dict(Hq=3, Nq=Nq)
        q = U.normal((1, 3, Nq, 64), 2, torch.float32)
        out, ws = torch.zeros_like(q), S.allocate_cache_workspace(p, attn)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            S.sparsepr_cache_attention(q, p, r.c, attn, out, ws)
        g.replay()
        torch.cuda.synchronize()
        again = torch.zeros_like(q)
        S.sparsepr_cache_attention(q, p, r.c, attn, again, ws)
        assert U.status(ws) == 0 and torch.equal(out, again) and out.abs().sum() > 0


def test_scales_far_apart():
    """Pages whose values differ by thirty powers of two, the weight on the
    small ones; keys likewise."""
    p = cache_params(1, 1, 128, 16, 20, 16)
    r = Run(p, 7)
    for i, s in enumerate([1.0, 2.0 ** -30, 2.0 ** 12, 2.0 ** -15, 1.0]):
        assert r.reserve([16])
        k = U.normal((1, 1, 16, 128), 50 + i, torch.float32, 0.2)
        k[..., 0] = 30.0 if i in (1, 3) else -30.0
        v = U.normal((1, 1, 16, 128), 60 + i, torch.float32, s)
        S.sparsepr_cache_append(k, v, p, r.c, r.start, None, r.ws)
        r.m.append(U.f64(k), U.f64(v), r.start.cpu().numpy(), [16])
    r.same()
    q = torch.zeros(1, 1, 1, 128, device="cuda")
    q[..., 0] = 10.0
    attn = dict(Hq=1, Nq=1, scale=0.1)
    out, ws = torch.zeros_like(q), S.allocate_cache_workspace(p, attn)
    S.sparsepr_cache_attention(q, p, r.c, attn, out, ws)
    ref = F.attention(U.f64(q[0]), r.m.tokens(0, "k"), r.m.tokens(0, "v"), 1,
                      dict(frame=1, window=0, sinks=0, causal=1), 0.1)
    tol, _ = U.bounds(ref, q.dtype, 128, F16, Q32, 0.0)
    assert (np.abs(U.f64(out[0]) - ref["out"]) <= tol).all()


def test_large_logits():
    p = cache_params(1, 1, 64, 32, 20, 16)
    r = Run(p, 9)
    r.grow([300], scale=40.0)
    assert r.attend(dict(Hq=4, Nq=1), scale=40.0) == 0
    assert r.attend(dict(Hq=4, Nq=40), scale=40.0) == 0


def test_pools_beyond_32_bit_offsets():
    """Pages whose bytes lie past 2^32 in the pool: append, copy of a shared last page,
    attention in place and widened, packing back to the front."""
    p = cache_params(3, 8, 128, 128, 34000, 3)  # 4.46 GB of keys, as much of values
    c = S.allocate_cache(p)
    c.ref[:33950] = 1  # all but the last pages are taken
    ws, start = S.allocate_cache_workspace(p), U.i32([0] * 3)
    n = U.i32([200, 0, 5])
    S.sparsepr_cache_reserve(n, p, c, start, ws)
    assert c.table[0].tolist() == [33950, 33951, -1] and c.table[2].tolist() == [33952, -1, -1]
    k, v = U.normal((3, 8, 200, 128), 1), U.normal((3, 8, 200, 128), 2)
    S.sparsepr_cache_append(k, v, p, c, start, n, ws)
    S.sparsepr_cache_fork(U.i32([0]), U.i32([1]), p, c, ws)
    one = U.i32([0, 1, 0])
    S.sparsepr_cache_reserve(one, p, c, start, ws)  # sequence 1 gets a copy of page 33951
    S.sparsepr_cache_append(k, v, p, c, start, one, ws)
    assert c.table[1].tolist() == [33950, 33953, -1] and U.status(ws) == 0

    def same_as_small():
        """The same tokens in a small cache."""
        small = Run(cache_params(3, 8, 128, 128, 8, 3))
        small.start.copy_(U.i32([0, 0, 0]))
        assert small.reserve([200, 201, 5])
        kk, vv = (torch.cat([t[:1], torch.cat([t[:1], t[1:2, :, :1]], 2)[:, :, :201][:, :, :200],
                             t[2:]]) for t in (k, v))
        small.c.len.copy_(U.i32([0, 0, 0]))
        S.sparsepr_cache_append(kk, vv, small.p, small.c, U.i32([0, 0, 0]), U.i32([200, 200, 5]),
                                small.ws)
        tail = [torch.zeros_like(t[:, :, :1]) for t in (k, v)]
        for x, t in zip(tail, (k, v)):
            x[1] = t[1, :, :1]
        S.sparsepr_cache_append(tail[0].contiguous(), tail[1].contiguous(), small.p, small.c,
                                U.i32([-1, 200, -1]), U.i32([0, 1, 0]), small.ws)
        small.c.len.copy_(c.len)
        for Nq in (1, 40):
            a = dict(Hq=8, Nq=Nq)
            q = U.normal((3, 8, Nq, 128), 5)
            outs = []
            for pp, cc in ((p, c), (small.p, small.c)):
                out = torch.zeros_like(q)
                w = S.allocate_cache_workspace(pp, a)
                S.sparsepr_cache_attention(q, pp, cc, a, out, w)
                assert U.status(w) == 0
                outs.append(out)
            assert torch.equal(outs[0], outs[1])

    same_as_small()
    c.ref[:33950] = 0  # and they are given up
    used = U.i32([0])
    S.sparsepr_cache_compact(p, c, used, ws)
    assert int(used) == 4 and int(c.table.max()) == 3 and U.status(ws) == 0
    same_as_small()


def test_widened_pages_of_one_sequence_at_a_time():
    """Table rows so long that the workspace holds the widened rows of one sequence."""
    p = cache_params(3, 1, 64, 128, 12, 24000)
    r = Run(p, 21)
    r.grow([300, 129, 0])
    attn = dict(Hq=1, Nq=40, window=150, sinks=2)
    assert S.allocate_cache_workspace(p, attn).numel() < 900 * 2 ** 20
    assert r.attend(attn) == 0
    assert r.attend(attn, torch.float32, n_q=[40, 7, 3]) == 0


def test_many_branches_of_one_history():
    """1,024 sequences that share their pages: more tiles than 2^22, the same answer for
    all of them."""
    p = cache_params(1024, 32, 64, 16, 520, 520)
    one = Run(dict(p, B=1), 3)
    one.grow([8256])
    c = S.allocate_cache(p)
    for name in ("k8", "v8", "k_scale", "v_scale"):
        getattr(c, name).view(torch.uint8).copy_(getattr(one.c, name).view(torch.uint8))
    c.table[0], c.len[0] = one.c.table[0], one.c.len[0]
    c.ref.copy_(one.c.ref)
    ws = S.allocate_cache_workspace(p)
    S.sparsepr_cache_fork(U.i32([0] * 1023), U.i32(list(range(1, 1024))), p, c, ws)
    assert U.status(ws) == 0 and int(c.ref.max()) == 1024
    q1 = U.normal((1, 32, 1, 64), 4)
    outs = []
    for pp, cc, q in ((one.p, one.c, q1), (p, c, q1.expand(1024, -1, -1, -1).contiguous())):
        a = dict(Hq=32, Nq=1)
        out, w = torch.zeros_like(q), S.allocate_cache_workspace(pp, a)
        S.sparsepr_cache_attention(q, pp, cc, a, out, w)
        assert U.status(w) == 0
        outs.append(out.double())
    # both round fp16 weights (2^-11 of values up to 0.5, over many tokens) and the output once
    assert (outs[1] - outs[0]).abs().max() <= 2 * 2.0 ** -11 * 0.5 + 2.0 ** -8 * outs[0].abs().max()


# ---- a run of them together -------------------------------------------------------
def test_rollout_step_captured_and_replayed():
    """Prompt, then steps of reserve + append + attention captured once in a graph
    and replayed; then a branch, its own last page, and the end of the parent."""
    p = cache_params(4, 2, 128, 16, 64, 12)
    attn = dict(Hq=4, Nq=1, window=60, sinks=3)
    r = Run(p, 11)
    r.grow([30, 47, 1, 0])
    ws = S.allocate_cache_workspace(p, attn)
    one = U.i32([1, 1, 1, 0])
    n_q = U.i32([1, 1, 1, 0])
    k = torch.zeros(4, 2, 1, 128, dtype=torch.bfloat16, device="cuda")
    v, q = torch.zeros_like(k), torch.zeros(4, 4, 1, 128, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.zeros_like(q), torch.zeros(4, 4, 1, device="cuda")

    def step():
        S.sparsepr_cache_reserve(one, p, r.c, r.start, ws)
        S.sparsepr_cache_append(k, v, p, r.c, r.start, one, ws)
        S.sparsepr_cache_attention(q, p, r.c, attn, out, ws, lse=lse, n_q=n_q)
        S.sparsepr_cache_evict(attn, p, r.c, ws)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    see = dict(frame=1, window=60, sinks=3, causal=1)
    for i in range(40):
        for t, s in ((k, 1), (v, 2), (q, 3)):
            t.copy_(U.normal(t.shape, 1000 + 10 * i + s))
        g.replay()
        torch.cuda.synchronize()
        start = r.m.reserve([1, 1, 1, 0])
        r.m.append(U.f64(k), U.f64(v), start, [1, 1, 1, 0])
        if i % 8 == 0:
            for b in range(3):
                ref = F.attention(U.f64(q[b]), r.m.tokens(b, "k"), r.m.tokens(b, "v"), 1, see)
                U.check(out[b], lse[b], ref, q.dtype, 128, F16, what=(i, b))
        r.m.evict(1, 60, 3)
        r.same(i)
    assert U.status(ws) == 0
    # sequence 3 branches off sequence 1 in the middle of a page, both go on
    S.sparsepr_cache_fork(U.i32([1]), U.i32([3]), p, r.c, ws)
    assert r.m.fork([1], [3])
    r.grow([0, 2, 0, 5])
    r.same("branch")
    S.sparsepr_cache_free(U.i32([1]), p, r.c, ws)
    r.m.free([1])
    used = U.i32([0])
    S.sparsepr_cache_compact(p, r.c, used, ws)
    assert int(used) == r.m.compact()
    r.same("packed")
    assert r.attend(attn, n_q=[1, 0, 1, 1]) == 0


def test_cache_agrees_with_the_windowed_attention():
    """A prompt through the windowed attention and through the cache: the same
    visibility, apart from the rounding of keys and values to 8 bits."""
    p = cache_params(1, 1, 64, 32, 16, 8)
    r = Run(p, 13)
    r.grow([200])
    k, v = (torch.tensor(r.m.tokens(0, n), dtype=torch.bfloat16, device="cuda")[None] for n in "kv")
    see = dict(frame=9, window=5, sinks=1, causal=1)
    q = U.normal((1, 2, 60, 64), 3)
    outs = [torch.zeros_like(q) for _ in range(2)]
    wp = dict(B=1, Hq=2, Hkv=1, Nq=60, Nk=200, d=64, **see)
    S.sparsepr_window_attention(q, k, v, wp, outs[0], S.allocate_window_workspace(wp, q.dtype))
    attn = dict(Hq=2, Nq=60, **see)
    S.sparsepr_cache_attention(q, p, r.c, attn, outs[1], S.allocate_cache_workspace(p, attn))
    ref = F.attention(U.f64(q[0]), U.f64(k[0]), U.f64(v[0]), 60, see)
    tol, _ = U.bounds(ref, q.dtype, 64, U.HALF[torch.bfloat16], 0.0, 0.0)
    for o in outs:  # the cached tokens are exactly bf16 values
        assert (np.abs(U.f64(o[0]) - ref["out"]) <= tol).all()


@pytest.mark.parametrize("see", [
    dict(frame=2 ** 31 - 1, window=2 ** 31 - 1, sinks=2 ** 31 - 1, causal=0),
    dict(frame=2 ** 31 - 1, window=1, sinks=0, causal=1),
    dict(frame=2, window=2 ** 31 - 1, sinks=1, causal=1)])
@pytest.mark.parametrize("Nq", [1, 5, 40])
def test_largest_frames_windows_and_sinks(see, Nq):
    r = Run(cache_params(2, 1, 64, 16, 90, 40), 19)
    r.grow([600, 130])
    assert r.attend(dict(Hq=2, Nq=Nq, **see)) == 0


@pytest.mark.parametrize("at", [0, 690])
@pytest.mark.parametrize("ratio,page", [(1, 64), (2.0 ** 6, 64), (2.0 ** 10, 16)])
@pytest.mark.parametrize("gap", [16, 20, 25, 30, 60])
@pytest.mark.parametrize("rows", [1, 8, 32])
@pytest.mark.parametrize("d", [64, 128])
def test_a_strong_key_without_a_value(d, rows, gap, ratio, page, at):
    """A key whose logit lies `gap` log2 units above all others and whose value is 0, in a
    page whose value scale is `ratio` times the others': the output is the other keys',
    whose weights are that much smaller than the largest. The queries are bf16 values, which
    the call takes as they are; the output is fp32, so that the weights' 11 bits show."""
    L, scale = 700, 0.125
    Hq, Nq = {1: (1, 1), 8: (8, 1), 32: (4, 8)}[rows]
    p = cache_params(1, 1, d, page, 50, 48)
    r = Run(p)
    assert r.reserve([L])
    k = U.normal((1, 1, L, d), 1, scale=0.25)
    v = U.normal((1, 1, L, d), 2, scale=0.25) + 1
    k[..., 0], k[0, 0, at, 0] = 0.0, 16.0
    v[0, 0, at] = 0
    v[0, 0, at ^ 1, 0] = 2.0 * ratio
    S.sparsepr_cache_append(k, v, p, r.c, r.start, None, r.ws)
    r.m.append(U.f64(k), U.f64(v), [0], [L])
    r.same()
    q = U.normal((1, Hq, Nq, d), 3, scale=0.25).float()
    q[..., 0] = gap / (scale * 16 * 1.4426950408889634)
    q = q.bfloat16().float()
    attn = dict(Hq=Hq, Nq=Nq, scale=scale)
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:3], device="cuda")
    ws = S.allocate_cache_workspace(p, attn)
    S.sparsepr_cache_attention(q, p, r.c, attn, out, ws, lse=lse)
    ref = F.attention(U.f64(q[0]), r.m.tokens(0, "k"), r.m.tokens(0, "v"), Nq,
                      dict(frame=1, window=0, sinks=0, causal=1), scale)
    U.check(out[0], lse[0], ref, torch.float32, d, F16)
    assert U.status(ws) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("Nq", [1, 3])
@pytest.mark.parametrize("big", [2.0 ** 14, 2.0 ** 20, 2.0 ** 28, 2.0 ** 110])
@pytest.mark.parametrize("d", [64, 128])
def test_a_query_channel_far_above_the_others(d, big, Nq, dtype):
    """One large channel of the queries meets zeros of the keys: the logits are the other
    channels'. The queries are bf16 values that the call can take as they are: multiples of
    2^-39 of the large one (at 2^28 they are rounded to that here)."""
    p = cache_params(1, 1, d, 16, 20, 16)
    r = Run(p, 7)
    assert r.reserve([200])
    k, v = U.normal((1, 1, 200, d), 1), U.normal((1, 1, 200, d), 2)
    k[..., 0] = 0
    S.sparsepr_cache_append(k, v, p, r.c, r.start, None, r.ws)
    r.m.append(U.f64(k), U.f64(v), [0], [200])
    q = U.normal((1, 2, Nq, d), 3)
    if big == 2.0 ** 28:  # multiples of 2^-9
        q = torch.round(q.float() * 16).div(16).bfloat16()
    scale = 1.0
    if big == 2.0 ** 110:
        q, scale = q * 2.0 ** 100, 2.0 ** -100
    q = q.to(dtype)
    q[..., 0] = big
    attn = dict(Hq=2, Nq=Nq, scale=scale)
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:3], device="cuda")
    S.sparsepr_cache_attention(q, p, r.c, attn, out, S.allocate_cache_workspace(p, attn), lse=lse)
    ref = F.attention(U.f64(q[0]), r.m.tokens(0, "k"), r.m.tokens(0, "v"), Nq,
                      dict(frame=1, window=0, sinks=0, causal=1), scale)
    U.check(out[0], lse[0], ref, dtype, d, F16)


def test_append_of_nothing_beside_a_shared_page():
    """Sequences that get no token in this step may share their last, partly filled page, or
    hold none: nothing is written for them and nothing is wrong."""
    p = cache_params(4, 1, 64, 16, 12, 4)
    r = Run(p)
    r.grow([20, 5, 0, 0])
    S.sparsepr_cache_fork(U.i32([0]), U.i32([2]), p, r.c, r.ws)
    r.m.fork([0], [2])
    r.grow([0, 2, 0, 0], T=3)
    assert r.status() == 0
    r.same()
    # a place inside the table without a page, and the end of the row
    x = torch.ones(4, 1, 3, 64, dtype=torch.bfloat16, device="cuda")
    S.sparsepr_cache_append(x, x, p, r.c, U.i32([20, 7, 64, 40]), U.i32([0, 0, 0, 0]), r.ws)
    assert r.status() == 0
    r.same()


@pytest.mark.parametrize("Nq,kw", [(1, {}), (5, {}), (3, dict(window=120, sinks=20)),
                                   (16, dict(frame=7, window=9, sinks=1)), (40, dict(window=70, sinks=3))])
@pytest.mark.parametrize("d", [64, 128])
def test_nan_shows_where_it_is_seen_and_nowhere_else(d, Nq, kw):
    """NaN values in single columns and NaN keys, early, in the window and among the last
    tokens, of which some queries see some."""
    p = cache_params(3, 2, d, 16, 80, 24)
    r = Run(p, 31)
    r.grow([300, 200, 90])
    rng = np.random.default_rng(d + Nq)
    for b, L in enumerate((300, 200, 90)):
        for j in [3, int(rng.integers(L)), L - 1 - int(rng.integers(4)), L - 1]:
            r.c.v8.view(torch.uint8)[int(r.m.table[b, j // 16]), b % 2, j % 16, int(rng.integers(d))] = 0x7F
        j = int(rng.integers(L))
        if b:
            r.c.k8.view(torch.uint8)[int(r.m.table[b, j // 16]), 0, j % 16, 3] = 0xFF
    r.m = U.to_model(p, r.c)
    assert r.attend(dict(Hq=4, Nq=Nq, **kw)) == 0


@pytest.mark.parametrize("Nq", [1, 8])
@pytest.mark.parametrize("d", [64, 128])
def test_what_every_query_sees_costs_no_second_pass(d, Nq):
    """A NaN in the first token: columns that it does not touch are those of the call without
    it, bit for bit; so are the other heads' where a key is NaN. Neither takes more than a few
    times as long (taken again one by one, rows took 100 times as long and more)."""
    p = cache_params(8, 4, d, 64, 8 * 64, 64)
    r = Run(p)
    c = r.c
    g = torch.Generator(device="cuda").manual_seed(1)
    for t in (c.k8, c.v8):
        t.copy_((torch.randn(t.shape, generator=g, device="cuda") * 90).clamp_(-448, 448).to(S.F8))
    c.k_scale.fill_(2.0 ** -6), c.v_scale.fill_(2.0 ** -6)
    c.table.copy_(torch.arange(512, dtype=torch.int32, device="cuda").view(8, 64))
    c.len.fill_(4000), c.ref.fill_(1)
    attn = dict(Hq=4, Nq=Nq)
    q = U.normal((8, 4, Nq, d), 3)
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:3], device="cuda")
    ws = S.allocate_cache_workspace(p, attn)

    def go():
        best = 1e9
        for _ in range(6):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            torch.cuda.synchronize()
            a.record()
            S.sparsepr_cache_attention(q, p, c, attn, out, ws, lse=lse)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        return out.clone(), lse.clone(), best
    clean, clean_lse, t0 = go()
    assert torch.isfinite(clean).all()
    c.v8.view(torch.uint8)[::64, :, 7, 5] = 0x7F
    got, got_lse, t1 = go()
    keep = [i for i in range(d) if i != 5]
    assert torch.isnan(got[..., 5]).all() and torch.equal(got_lse, clean_lse)
    assert torch.equal(got[..., keep], clean[..., keep])
    c.k8.view(torch.uint8)[::64, 2, 9, 3] = 0x7F
    got, got_lse, t2 = go()
    assert torch.isnan(got[:, 2]).all() and torch.isnan(got_lse[:, 2]).all()
    assert torch.equal(got[:, :2][..., keep], clean[:, :2][..., keep])
    c.table[:, 3] = -1  # pages that are missing
    got, _, t3 = go()
    assert torch.isnan(got).all() and U.status(ws) == 1 << S.ERR_INVALID_ARG
    assert max(t1, t2, t3) < 20 * t0, (t0, t1, t2, t3)


@pytest.mark.parametrize("stale", [0x00, 0x01, 0x55, 0xFF])
def test_packing_leaves_entries_without_a_count(stale):
    """An entry that names a page with ref 0, whatever the workspace held."""
    p = cache_params(3, 1, 64, 16, 300, 4)
    r = Run(p)
    r.grow([40, 30, 20])
    S.sparsepr_cache_free(U.i32([0]), p, r.c, r.ws)
    r.m.free([0])
    for t in (r.c.table, r.m.table):
        t[0, 3], t[0, 1], t[2, 3] = 7, 299, 6  # page 6 moves, and so does this entry of it
    r.ws[256:].fill_(stale)
    used = U.i32([0])
    S.sparsepr_cache_compact(p, r.c, used, r.ws)
    assert int(used) == r.m.compact()
    assert r.c.table[0].tolist() == [-1, 299, -1, 7]
    r.same()


def test_first_calls_of_a_process_inside_captures():
    """A process whose first call of every attention kernel is captured: whatever a kernel
    needs once per device is set up in the capture."""
    code = """
import torch
from free_block_sparse_eigenbasis_b200 import sparsepr as S
for d in (64, 128):
    p = dict(B=2, Hkv=1, d=d, page=32, n_pages=8, max_pages=4)
    c = S.allocate_cache(p)
    for t in (c.k8, c.v8):
        t.copy_(torch.randn(t.shape, device="cuda").to(S.F8))
    c.table.copy_(torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4))
    c.len.fill_(100), c.ref.fill_(1)
    for dtype in (torch.bfloat16, torch.float32):
        for rows in (3, 12, 90):  # in place, 8 and 16 rows a unit, and widened
            q = torch.randn(2, 3, rows // 3, d, device="cuda").to(dtype)
            a = dict(Hq=3, Nq=rows // 3)
            calls = [(S.allocate_cache_workspace(p, a), lambda out, ws, q=q, a=a:
                      S.sparsepr_cache_attention(q, p, c, a, out, ws))]
            if rows == 90:  # the windowed kernel's own first call, before the cache's
                k = torch.randn(2, 1, 700, d, device="cuda").to(dtype)
                w = dict(B=2, Hq=3, Hkv=1, Nq=30, Nk=700, d=d)
                calls.insert(0, (S.allocate_window_workspace(w, dtype), lambda out, ws, q=q, k=k, w=w:
                                 S.sparsepr_window_attention(q, k, k, w, out, ws)))
            for ws, call in calls:
                out, again = torch.zeros_like(q), torch.zeros_like(q)
                torch.cuda.synchronize()
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g):
                    call(out, ws)
                g.replay()
                torch.cuda.synchronize()
                call(again, ws)
                assert torch.equal(out, again) and out.abs().sum() > 0
                assert int(ws[:4].view(torch.int32)) == 0
print("captured")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]
