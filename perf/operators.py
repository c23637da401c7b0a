"""Cases for the attention operators of frame-by-frame generation.

A world model that generates video frame by frame keeps the keys and values of
the frames it has made, attends to the last few of them (a sliding window) and
to the first one (a sink), and branches, drops and packs rollouts. Four
operators carry that:

  window    attention with a sliding window of frames and sink frames over
            keys and values in bf16
  append    new tokens' keys and values written to a paged cache in 8 bits
            (e4m3), one power-of-two scale for each page and head
  cached    attention over that cache, for one token or for a whole frame
  pages     the cache's pages: branch rollouts (free, fork, reserve with a
            copy of the shared last page) and pack a fragmented pool

``run`` computes each in plain torch operations in 32 bits, or, where ``own``
is true, by the library's calls.

Which keys a query sees. With frames of F tokens, a query at position p and a
key at position j lie in frames fq = p // F and fj = j // F. The key is
visible if (causal) fj <= fq, and if the window W is 0 or |fq - fj| < W or
fj < S, the number of sink frames. The n queries of a sequence of L keys stand
at its end: p = L - n + i.
"""
import math

import numpy as np
import torch

own = False

E4M3_MAX_MANT, E4M3_MAX_EXP = 0.875, 9  # 448 = 0.875 * 2^9
MIN_SCALE_EXP = -110


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _window(name, B, Hq, Hkv, d, Nq, Nk, frame, window, sinks, causal, ragged=False):
    return dict(name=name, op="window", B=B, Hq=Hq, Hkv=Hkv, d=d, Nq=Nq, Nk=Nk, frame=frame,
                window=window, sinks=sinks, causal=causal, ragged=ragged)


def _cached(name, B, Hq, Hkv, d, page, Nq, length, frame, window, sinks, ragged=False):
    return dict(name=name, op="cached", B=B, Hq=Hq, Hkv=Hkv, d=d, page=page, Nq=Nq, length=length,
                frame=frame, window=window, sinks=sinks, causal=True, ragged=ragged)


def listed():
    return [
        # one new token of a 12-head layer against 4,000 earlier ones kept in bf16
        _window("window-token", 1, 12, 12, 128, 1, 4001, 1, 0, 0, True),
        # three prompts of different lengths in one padded batch, shared key heads,
        # 64 channels, a token-level window with a few first tokens
        _window("window-ragged", 3, 16, 4, 64, 777, 1291, 1, 512, 4, True, ragged=True),
        # the 480p video layer (21 latent frames of 1,560 tokens), every frame
        # attends to its neighbours on both sides and to the first frame
        _window("window-clip", 1, 12, 12, 128, 32760, 32760, 1560, 3, 1, False),
        # the 720p video layer generated frame by frame: causal by frames, the
        # last four frames and the first one
        _window("window-rollout", 1, 12, 12, 128, 75600, 75600, 3600, 4, 1, True),
        # one new token for each of 8 rollouts, in the middle of a page
        dict(name="append-token", op="append", B=8, Hkv=8, d=128, page=64, T=1, start=1000,
             ragged=False),
        # one new 480p frame of a 12-head layer behind six earlier frames
        dict(name="append-frame", op="append", B=1, Hkv=12, d=128, page=64, T=1560, start=9360,
             ragged=False),
        # one token against a short cache: the smallest call
        _cached("cached-token", 1, 12, 12, 128, 64, 1, 1000, 1, 0, 0),
        # a serving batch of rollouts of different lengths, four query heads per key head
        _cached("cached-batch", 32, 32, 8, 128, 64, 1, 8192, 1, 0, 0, ragged=True),
        # long histories seen through a window of 64 frames of 400 tokens, small pages,
        # 64 channels, four tokens at once
        _cached("cached-window", 4, 16, 2, 64, 16, 4, 100003, 400, 64, 1),
        # a whole new 480p frame against the cache of 13 frames and itself
        _cached("cached-frame", 1, 12, 12, 128, 64, 1560, 21840, 1560, 0, 0),
        # 16 rollouts dropped and branched anew from 4 survivors, room for a token each
        dict(name="pages-branch", op="branch", B=20, parents=4, Hkv=12, d=128, page=64,
             length=9383, n_new=1),
        # a pool that many ended rollouts have left full of holes
        dict(name="pages-pack", op="pack", B=24, Hkv=12, d=128, page=64, length=6240, spread=2),
    ]


def _log(rng, lo, hi):
    """A whole number, spread evenly over the logarithm of lo..hi."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["window", "window", "append", "cached", "cached", "cached", "branch", "pack"])
    d = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128])
    Hkv = rng.choice([1, 2, 4, 8, 12])
    group = rng.choice([1, 1, 2, 4, 8])
    if op == "window":
        B = rng.choice([1, 1, 2, 3])
        Hkv = rng.choice([1, 2, 4, 6])
        group = rng.choice([1, 2, 4])
        Nk = _log(rng, 40, 16000)
        Nq = rng.choice([1, Nk, max(1, _log(rng, 1, Nk)), max(1, Nk // 3)])
        frame = rng.choice([1, 1, rng.randint(2, 400)])
        c = _window("", B, Hkv * group, Hkv, d, Nq, Nk, frame,
                    rng.choice([0, max(1, _log(rng, 16, 4000) // frame)]),
                    rng.choice([0, 1, 4]), rng.random() < 0.7, ragged=rng.random() < 0.5)
    elif op == "append":
        T = rng.choice([1, _log(rng, 2, 6000)])
        c = dict(op="append", B=rng.choice([1, 2, 5, 16]) if T < 1500 else 1, Hkv=Hkv, d=d,
                 page=page, T=T, start=_log(rng, 1, 20000) - 1, ragged=rng.random() < 0.5)
    elif op == "cached":
        Nq = rng.choice([1, 1, 1, 2, 5, _log(rng, 8, 1500)])
        length = _log(rng, Nq + 1, 60000)
        B = 1 if Nq * group > 64 else rng.choice([1, 3, 8, 24])
        if Nq * group > 64:
            Hkv = min(Hkv, 4)
            length = min(length, max(Nq + 1, 20000))
        B = max(1, min(B, 400000 * 8 * 128 // (length * Hkv * d)))
        frame = rng.choice([1, 1, rng.randint(2, 400)])
        c = _cached("", B, Hkv * group, Hkv, d, page, Nq, length, frame,
                    rng.choice([0, 0, max(1, _log(rng, 16, 8000) // frame)]),
                    rng.choice([0, 1, 4]), ragged=rng.random() < 0.5)
    elif op == "branch":
        parents = rng.randint(1, 6)
        c = dict(op="branch", B=parents * rng.randint(2, 6), parents=parents, Hkv=Hkv, d=d,
                 page=page, length=_log(rng, 2, 12000), n_new=_log(rng, 1, 300))
    else:
        B = rng.randint(2, 24)
        c = dict(op="pack", B=B, Hkv=Hkv, d=d, page=page, length=_log(rng, 30, 6240),
                 spread=rng.randint(2, 4))
    c.pop("name", None)
    return c


# --------------------------------------------------------------------------
# lengths, tables and counts that follow from a case
# --------------------------------------------------------------------------
def _spread(n, B, ragged):
    """Lengths of B sequences: n, or about 0.35 n to n in an uneven order (the first is n)."""
    if not ragged:
        return [n] * B
    return [n if b == 0 else max(1, int(n * (0.35 + 0.65 * ((b * 0.6180339887) % 1.0))))
            for b in range(B)]


def _attn_lengths(c):
    """(keys, queries) of every sequence of an attention case."""
    n = c["Nk"] if c["op"] == "window" else c["length"]
    keys = _spread(n, c["B"], c["ragged"])
    return keys, [min(k, q) for k, q in zip(keys, _spread(c["Nq"], c["B"], c["ragged"]))]


def _bounds(c, pos, length):
    """Visible keys of queries at positions `pos` (numpy int64): [0, s) and [lo, hi)."""
    F, W, S = c["frame"], c["window"], c["sinks"]
    f = pos // F
    hi = np.full_like(pos, length)
    if c["causal"]:
        hi = np.minimum(hi, (f + 1) * F)
    s = np.minimum(hi, S * F)
    lo = np.zeros_like(pos)
    if W > 0:
        lo = np.maximum(0, (f - W + 1) * F)
        if not c["causal"]:
            hi = np.minimum(length, (f + W) * F)
    return s, lo, hi


def work(case):
    c = case
    if c["op"] in ("window", "cached"):
        pairs = seen = rows = 0
        for L, n in zip(*_attn_lengths(c)):
            s, lo, hi = _bounds(c, np.arange(L - n, L, dtype=np.int64), L)
            pairs += int((np.maximum(hi - np.maximum(lo, s), 0) + s).sum())
            a, b = int(s.max()), int(lo.min())
            seen += a + max(0, int(hi.max()) - max(a, b))
            rows += n
        kv = 2 * seen * c["Hkv"] * c["d"] * (2 if c["op"] == "window" else 1)
        if c["op"] == "cached":
            kv += 2 * 4 * c["Hkv"] * (seen // c["page"] + 1) + 4 * (seen // c["page"] + 1)
        return {"bytes": kv + rows * c["Hq"] * (4 * c["d"] + 4),
                "flops": 4 * c["d"] * c["Hq"] * pairs}
    page_bytes = 2 * c["Hkv"] * (c["page"] * c["d"] + 4)  # keys, values and their scales
    if c["op"] == "append":
        n = sum(_spread(c["T"], c["B"], c["ragged"]))
        return {"bytes": 2 * n * c["Hkv"] * c["d"] * 3 + c["B"] * 2 * c["Hkv"] * 8,
                "flops": 4 * n * c["Hkv"] * c["d"]}
    if c["op"] == "branch":
        lp, mp = _table_shape(c)
        kids = c["B"] - c["parents"]
        copies = kids if c["length"] % c["page"] else 0
        return {"bytes": copies * 2 * page_bytes + kids * lp * 20, "flops": 0}
    lp, mp = _table_shape(c)
    used = c["B"] * lp
    moves = int((_pack_pages(c) >= used).sum())
    return {"bytes": moves * 2 * page_bytes + 2 * 4 * c["B"] * lp + 4 * used * c["spread"],
            "flops": 0}


def _table_shape(c):
    """(pages a sequence holds, width of a table row)."""
    n = c["length"] + c.get("n_new", 0)
    return -(-c["length"] // c["page"]), -(-n // c["page"]) + 1


def _pack_pages(c):
    """Pages of the fragmented pool, in table order: a draw of B * lp of spread times as many."""
    lp, _ = _table_shape(c)
    used = c["B"] * lp
    return np.random.RandomState(used).permutation(used * c["spread"])[:used]


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _rng(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _pool(n_pages, c, g):
    """Pages as earlier calls leave them: e4m3 values with a power-of-two scale for each page
    and head, keys and values of about unit size."""
    shape = (n_pages, c["Hkv"], c["page"], c["d"])
    x8, scale = [], []
    for _ in range(2):
        e = torch.randint(-8, -5, shape[:2], generator=g, device="cuda")
        x8.append((_normal(shape, g) * 90).clamp_(-448, 448).to(torch.float8_e4m3fn))
        scale.append(torch.exp2(e.float()))
    return dict(k8=x8[0], v8=x8[1], k_scale=scale[0], v_scale=scale[1])


def _cache_dict(c, n_pages, max_pages, B):
    return dict(B=B, Hkv=c["Hkv"], d=c["d"], page=c["page"], n_pages=n_pages, max_pages=max_pages)


def prepare(case, seed):
    c, g = dict(case), _rng(seed)
    st = dict(c=c)
    if c["op"] in ("window", "cached"):
        keys, queries = _attn_lengths(c)
        st["q"] = _normal((c["B"], c["Hq"], c["Nq"], c["d"]), g)
        st["out"] = torch.zeros_like(st["q"])
        st["lse"] = torch.zeros((c["B"], c["Hq"], c["Nq"]), device="cuda")
        st["n_q"] = _i32(queries) if c["ragged"] else None
        st["mask"] = dict(frame=c["frame"], window=c["window"], sinks=c["sinks"],
                          causal=int(c["causal"]))
    if c["op"] == "window":
        st["k"] = _normal((c["B"], c["Hkv"], c["Nk"], c["d"]), g)
        st["v"] = _normal((c["B"], c["Hkv"], c["Nk"], c["d"]), g)
        st["n_k"] = _i32(keys) if c["ragged"] else None
        return st
    if c["op"] == "cached":
        mp = -(-c["length"] // c["page"])
        n_pages = c["B"] * mp + 3
        perm = torch.randperm(n_pages, generator=g, device="cuda")[:c["B"] * mp]
        st |= _pool(n_pages, c, g)
        st["table"] = perm.to(torch.int32).view(c["B"], mp)
        st["len"] = _i32(keys)
        st["ref"] = torch.ones(n_pages, dtype=torch.int32, device="cuda")
        st["p"] = _cache_dict(c, n_pages, mp, c["B"])
    elif c["op"] == "append":
        end = c["start"] + c["T"]
        mp = -(-end // c["page"])
        n_pages = c["B"] * mp + 1
        perm = torch.randperm(n_pages, generator=g, device="cuda")[:c["B"] * mp]
        st |= _pool(n_pages, c, g)
        st["table"] = perm.to(torch.int32).view(c["B"], mp)
        st["start"] = _i32([c["start"]] * c["B"])
        st["n_new"] = _i32(_spread(c["T"], c["B"], c["ragged"]))
        st["len"] = st["start"] + st["n_new"]
        st["ref"] = torch.ones(n_pages, dtype=torch.int32, device="cuda")
        st["k"] = _normal((c["B"], c["Hkv"], c["T"], c["d"]), g)
        st["v"] = _normal((c["B"], c["Hkv"], c["T"], c["d"]), g) * 1.5
        st["p"] = _cache_dict(c, n_pages, mp, c["B"])
    elif c["op"] == "branch":
        # parents hold pages of their own; the children are branches of an earlier step, whose
        # last page is their own and whose other pages are a parent's
        lp, mp = _table_shape(c)
        kids = c["B"] - c["parents"]
        n_pages = c["parents"] * lp + 3 * kids * (1 + -(-c["n_new"] // c["page"])) + 5
        perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        table = torch.full((c["B"], mp), -1, dtype=torch.int32, device="cuda")
        table[:c["parents"], :lp] = perm[:c["parents"] * lp].view(c["parents"], lp)
        old = torch.randint(0, c["parents"], (kids,), generator=g, device="cuda")
        table[c["parents"]:] = table[old]
        table[c["parents"]:, lp - 1] = perm[c["parents"] * lp:c["parents"] * lp + kids]
        st |= _pool(n_pages, c, g)
        st["table"] = table
        st["len"] = _i32([c["length"]] * c["B"])
        st["ref"] = torch.bincount(table[table >= 0].long(), minlength=n_pages).to(torch.int32)
        st["kids"] = torch.arange(c["parents"], c["B"], dtype=torch.int32, device="cuda")
        st["src"] = torch.randint(0, c["parents"], (kids,), generator=g, device="cuda",
                                  dtype=torch.int32)
        st["n_new"] = _i32([0] * c["parents"] + [c["n_new"]] * kids)
        st["start"] = torch.zeros(c["B"], dtype=torch.int32, device="cuda")
        st["p"] = _cache_dict(c, n_pages, mp, c["B"])
    else:
        lp, mp = _table_shape(c)
        used = c["B"] * lp
        n_pages = used * c["spread"]
        st |= _pool(n_pages, c, g)
        table = torch.full((c["B"], mp), -1, dtype=torch.int32, device="cuda")
        pages = _i32(_pack_pages(c))
        table[:, :lp] = pages.view(c["B"], lp)
        ref = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
        ref[pages.long()] = 1
        st["holes"] = (table, ref)
        st["table"], st["ref"] = table.clone(), ref.clone()
        st["len"] = _i32([c["length"]] * c["B"])
        st["n_used"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        st["p"] = _cache_dict(c, n_pages, mp, c["B"])
    return st


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(state):
    return _run_own(state) if own else _PLAIN[state["c"]["op"]](state)


def _pool_out(st, **more):
    return dict(k8=st["k8"], v8=st["v8"], k_scale=st["k_scale"], v_scale=st["v_scale"], **more)


def _run_own(st):
    from free_block_sparse_eigenbasis_b200 import sparsepr as S

    c = st["c"]
    if c["op"] == "window":
        if "p" not in st:
            st["p"] = dict(B=c["B"], Hq=c["Hq"], Hkv=c["Hkv"], Nq=c["Nq"], Nk=c["Nk"], d=c["d"],
                           **st["mask"])
            st["ws"] = S.allocate_window_workspace(st["p"], st["q"].dtype)
        S.sparsepr_window_attention(st["q"], st["k"], st["v"], st["p"], st["out"], st["ws"],
                                    lse=st["lse"], n_q=st["n_q"], n_k=st["n_k"])
        return dict(out=st["out"], lse=st["lse"])
    if "cache" not in st:
        st["cache"] = S.Cache(k8=st["k8"], v8=st["v8"], k_scale=st["k_scale"],
                              v_scale=st["v_scale"], table=st["table"], len=st["len"],
                              ref=st["ref"])
        attn = None
        if c["op"] == "cached":
            attn = st["attn"] = dict(Hq=c["Hq"], Nq=c["Nq"], **st["mask"])
        st["ws"] = S.allocate_cache_workspace(st["p"], attn)
    p, cache, ws = st["p"], st["cache"], st["ws"]
    if c["op"] == "cached":
        S.sparsepr_cache_attention(st["q"], p, cache, st["attn"], st["out"], ws, lse=st["lse"],
                                   n_q=st["n_q"])
        return dict(out=st["out"], lse=st["lse"])
    if c["op"] == "append":
        S.sparsepr_cache_append(st["k"], st["v"], p, cache, st["start"], st["n_new"], ws)
        return _pool_out(st)
    if c["op"] == "branch":
        S.sparsepr_cache_free(st["kids"], p, cache, ws)
        S.sparsepr_cache_fork(st["src"], st["kids"], p, cache, ws)
        S.sparsepr_cache_reserve(st["n_new"], p, cache, st["start"], ws)
        return _pool_out(st, table=st["table"], len=st["len"], ref=st["ref"], start=st["start"])
    cache.table.copy_(st["holes"][0])
    cache.ref.copy_(st["holes"][1])
    S.sparsepr_cache_compact(p, cache, st["n_used"], ws)
    return _pool_out(st, table=st["table"], ref=st["ref"], n_used=st["n_used"])


# ---- plain forms ----------------------------------------------------------
def _visible(c, pos, keys, lengths):
    """[B, n, keys] truth: key `keys` (int64) is visible from position `pos` [B, n]."""
    F, W, S = c["frame"], c["window"], c["sinks"]
    fq = torch.div(pos, F, rounding_mode="floor")[:, :, None]
    fk = torch.div(keys, F, rounding_mode="floor")[None, None, :]
    see = (keys[None, None, :] < lengths[:, None, None]) & (pos >= 0)[:, :, None]
    if c["causal"]:
        see = see & (fk <= fq)
    if W > 0:
        see = see & (((fq - fk).abs() < W) | (fk < S))
    return see


def _attend(c, q, k, v, see):
    """softmax over the visible keys: q [B, Hq, n, d], k and v [B, Hkv, m, d] in fp32."""
    B, Hq, n, d = q.shape
    Hkv = k.shape[1]
    s = torch.matmul(q.view(B, Hkv, -1, d), k.transpose(2, 3)).view(B, Hkv, Hq // Hkv, n, -1)
    s = (s / math.sqrt(d)).masked_fill(~see[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = torch.exp(s - top)
    tot = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(B, Hkv, -1, e.shape[-1]), v).view(B, Hkv, Hq // Hkv, n, d)
    o = torch.where(tot > 0, o / tot, torch.zeros_like(o))
    return o.reshape(B, Hq, n, d), (top + torch.log(tot)).reshape(B, Hq, n)


def _attend_rows(st, k, v, lengths, counts):
    """All query rows against k and v (bf16 or fp32), in pieces of the rows that keep the scores
    under a gigabyte; a piece reads the keys that its rows can see. Rows behind a sequence's
    queries keep what they hold."""
    c, q = st["c"], st["q"]
    B, Hq, Nq, d = q.shape
    m = k.shape[2]
    piece = max(1, min(Nq, (1 << 28) // (B * Hq * (m if c["window"] == 0 else min(
        m, (2 * c["window"] + c["sinks"]) * c["frame"] + 4096)))))
    for r0 in range(0, Nq, piece):
        r1 = min(Nq, r0 + piece)
        keys = torch.arange(m, device="cuda")
        if not c["ragged"] and c["window"] > 0:
            s, lo, hi = _bounds(c, np.arange(m - Nq + r0, m - Nq + r1, dtype=np.int64), m)
            a, b, e = int(s.max()), int(lo.min()), int(hi.max())
            keys = torch.cat([keys[:min(a, b)], keys[b:e]])
        i = torch.arange(r0, r1, device="cuda")
        see = _visible(c, (lengths - counts)[:, None] + i[None, :], keys, lengths)
        o, lse = _attend(c, q[:, :, r0:r1].float(), k[:, :, keys].float(), v[:, :, keys].float(),
                         see)
        real = (i[None, :] < counts[:, None])[:, None, :]
        st["out"][:, :, r0:r1] = torch.where(real[..., None], o.to(q.dtype), st["out"][:, :, r0:r1])
        st["lse"][:, :, r0:r1] = torch.where(real, lse, st["lse"][:, :, r0:r1])
    return dict(out=st["out"], lse=st["lse"])


def _counts(st, B, n):
    return torch.full((B,), n, device="cuda") if st["n_q"] is None else st["n_q"].long()


def _plain_window(st):
    c = st["c"]
    lengths = torch.full((c["B"],), c["Nk"], device="cuda") if st["n_k"] is None else st["n_k"].long()
    return _attend_rows(st, st["k"], st["v"], lengths, _counts(st, c["B"], c["Nq"]))


def _gathered(x8, scale, table):
    """The tokens of every sequence in order: [B, Hkv, max_pages * page, d] in fp32."""
    at = table.long().clamp(min=0)
    x = x8.view(torch.uint8)[at].view(torch.float8_e4m3fn).float() * scale[at][..., None, None]
    return x.permute(0, 2, 1, 3, 4).reshape(x.shape[0], x.shape[2], -1, x.shape[4])


def _plain_cached(st):
    c = st["c"]
    k = _gathered(st["k8"], st["k_scale"], st["table"])[:, :, :c["length"]]
    v = _gathered(st["v8"], st["v_scale"], st["table"])[:, :, :c["length"]]
    return _attend_rows(st, k, v, st["len"].long(), _counts(st, c["B"], c["Nq"]))


def _scale_exp(amax):
    """Exponent of the smallest power of two s with amax <= 448 s (amax = 0: the least one)."""
    m, e = torch.frexp(amax)
    e = e - E4M3_MAX_EXP + (m > E4M3_MAX_MANT)
    return torch.where(amax > 0, e.clamp(min=MIN_SCALE_EXP), torch.full_like(e, MIN_SCALE_EXP))


def _plain_append(st):
    c = st["c"]
    B, Hkv, T, d = st["k"].shape
    page, start, n = c["page"], st["start"].long(), st["n_new"].long()
    touched = -(-(T + page - 1) // page)  # pages that T tokens can reach from any offset
    first = start // page
    idx = first[:, None] + torch.arange(touched, device="cuda")  # [B, touched] table columns
    hit = idx * page < (start + n)[:, None]
    pages = st["table"].gather(1, idx.clamp(max=st["table"].shape[1] - 1)).long()
    pos = idx[:, :, None] * page + torch.arange(page, device="cuda")  # [B, touched, page]
    new = ((pos >= start[:, None, None]) & (pos < (start + n)[:, None, None]))[:, :, None, :, None]
    old = (pos < start[:, None, None])[:, :, None, :, None]
    tok = (pos - start[:, None, None]).clamp(0, T - 1)
    at = tok[:, None].expand(B, Hkv, touched, page).reshape(B, Hkv, -1, 1).expand(-1, -1, -1, d)
    for x, x8, scale in ((st["k"], st["k8"], st["k_scale"]), (st["v"], st["v8"], st["v_scale"])):
        xs = x.float().gather(2, at).view(B, Hkv, touched, page, d).transpose(1, 2)
        xs = torch.where(xs.isinf(), torch.full_like(xs, math.nan), xs)
        amax = torch.where(new & ~xs.isnan(), xs.abs(), torch.zeros_like(xs)).amax((3, 4))
        need = torch.exp2(_scale_exp(amax).double()).float()
        was = scale[pages]  # [B, touched, Hkv]
        now = torch.where(old.any(3).squeeze(-1), torch.maximum(was, need), need)
        q8 = x8.view(torch.uint8)[pages]
        kept = q8.view(torch.float8_e4m3fn).float()
        again = (kept * (was / now)[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        fresh = (xs / now[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        q8 = torch.where(new, fresh, torch.where(old, again, q8))
        x8.view(torch.uint8)[pages[hit]] = q8[hit]
        scale[pages[hit]] = now[hit]
    return _pool_out(st)


def _plain_branch(st):
    table, ref, length, kids = st["table"], st["ref"], st["len"], st["kids"].long()
    page, n, B = st["c"]["page"], st["n_new"].long(), table.shape[0]

    def count(rows, by):
        entries = table[rows].long()
        ref.index_add_(0, entries.clamp(min=0).view(-1), (entries >= 0).view(-1).to(ref.dtype) * by)

    count(kids, -1)  # free
    table[kids], length[kids] = -1, 0
    table[kids], length[kids] = table[st["src"].long()], length[st["src"].long()]  # fork
    count(kids, 1)
    # reserve: a page of its own for a shared last page, then new pages, lowest free pages first
    start = length.long()
    have, want = -(-start // page), -(-(start + n) // page)
    last = table.gather(1, (start // page).clamp(max=table.shape[1] - 1)[:, None])[:, 0].long()
    own_copy = (n > 0) & (start % page > 0) & (ref[last.clamp(min=0)] > 1)
    need = want - have + own_copy
    free = torch.argsort(ref != 0, stable=True)  # free pages first, ascending
    before = torch.cumsum(need, 0) - need
    most = -(-st["c"]["n_new"] // page) + 1
    j = torch.arange(most, device="cuda")[None, :]
    give = j < need[:, None]
    pages = free[(before[:, None] + j).clamp(max=free.numel() - 1)]
    col = (have - own_copy.long())[:, None] + j
    wide = torch.cat([table, table.new_full((B, most + 1), -1)], 1)
    wide.scatter_(1, torch.where(give, col, table.shape[1] + j), pages.to(torch.int32))
    table.copy_(wide[:, :table.shape[1]])
    ref.index_add_(0, pages.view(-1), give.view(-1).to(ref.dtype))
    ref.index_add_(0, last.clamp(min=0), -own_copy.to(ref.dtype))
    src, dst = last[own_copy], pages[:, 0][own_copy]
    for name in ("k8", "v8"):
        st[name].view(torch.uint8)[dst] = st[name].view(torch.uint8)[src]
    for name in ("k_scale", "v_scale"):
        st[name][dst] = st[name][src]
    st["start"].copy_(start)
    length.add_(st["n_new"])
    return _pool_out(st, table=table, len=length, ref=ref, start=st["start"])


def _plain_pack(st):
    table, ref = st["table"], st["ref"]
    table.copy_(st["holes"][0])
    ref.copy_(st["holes"][1])
    used = ref > 0
    n = used.sum()
    st["n_used"].copy_(n.view(1))
    at = torch.arange(ref.numel(), device="cuda")
    src, dst = at[used & (at >= n)], at[~used & (at < n)]
    to = at.clone()
    to[src] = dst
    table.copy_(torch.where(table >= 0, to[table.long().clamp(min=0)].to(torch.int32), table))
    for name in ("k8", "v8"):
        st[name].view(torch.uint8)[dst] = st[name].view(torch.uint8)[src]
    for name in ("k_scale", "v_scale"):
        st[name][dst] = st[name][src]
    ref[dst] = ref[src]
    ref[src] = 0
    return _pool_out(st, table=table, ref=ref, n_used=st["n_used"])


_PLAIN = dict(window=_plain_window, cached=_plain_cached, append=_plain_append,
              branch=_plain_branch, pack=_plain_pack)


# --------------------------------------------------------------------------
# the definition in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    c = dict(case)
    st = prepare(c, seed)
    if c["op"] in ("branch", "pack"):
        return None  # whole pages and whole numbers move; nothing is rounded
    if c["op"] == "append":
        return _exact_append(c, st)
    keys, queries = _attn_lengths(c)
    out = torch.zeros((c["B"], c["Hq"], c["Nq"], c["d"]), dtype=torch.float64, device="cuda")
    lse = torch.zeros((c["B"], c["Hq"], c["Nq"]), dtype=torch.float64, device="cuda")
    group = c["Hq"] // c["Hkv"]
    for b in range(c["B"]):
        L, n = keys[b], queries[b]
        for h in range(c["Hkv"]):
            if c["op"] == "window":
                k, v = st["k"][b, h, :L].double(), st["v"][b, h, :L].double()
            else:
                pg = st["table"][b].long()
                k = st["k8"].view(torch.uint8)[pg, h].view(torch.float8_e4m3fn).double()
                v = st["v8"].view(torch.uint8)[pg, h].view(torch.float8_e4m3fn).double()
                k = (k * st["k_scale"][pg, h].double()[:, None, None]).view(-1, c["d"])[:L]
                v = (v * st["v_scale"][pg, h].double()[:, None, None]).view(-1, c["d"])[:L]
            heads = slice(h * group, (h + 1) * group)
            step = max(1, (1 << 27) // (group * L))
            if c["window"] and c["frame"] > 1:
                step = min(n, max(step, c["frame"] // 2))
            for r in range(0, n, step):
                e = min(n, r + step)
                s, lo, hi = _bounds(c, np.arange(L - n + r, L - n + e, dtype=np.int64), L)
                a, z = min(int(s.max()), int(lo.min())), int(hi.max())
                pick = torch.cat([torch.arange(0, a, device="cuda"),
                                  torch.arange(int(lo.min()), z, device="cuda")])
                s, lo, hi = (torch.from_numpy(x).cuda()[:, None] for x in (s, lo, hi))
                unseen = ~((pick < s) | ((pick >= lo) & (pick < hi)))
                logit = torch.einsum("gnd,md->gnm", st["q"][b, heads, r:e].double(), k[pick])
                logit = (logit * c["d"] ** -0.5).masked_fill_(unseen[None], -math.inf)
                norm = torch.logsumexp(logit, -1)
                w = logit.sub_(norm[..., None]).exp_()
                out[b, heads, r:e] = torch.einsum("gnm,md->gnd", w, v[pick])
                lse[b, heads, r:e] = norm
    return dict(out=out, lse=lse)


def _exact_append(c, st):
    """Page by page: the scale from the largest magnitude, then every value's nearest e4m3."""
    B, Hkv, T, d = st["k"].shape
    if B * (T // c["page"] + 2) > 4000:
        return None
    page, res = c["page"], {}
    n = _spread(c["T"], B, c["ragged"])
    for name, x in (("k", st["k"].double()), ("v", st["v"].double())):
        vals = st[name + "8"].to(torch.float64)
        scale = st[name + "_scale"].to(torch.float64)
        for b in range(B):
            for col in range(c["start"] // page, -(-(c["start"] + n[b]) // page)):
                pg = int(st["table"][b, col])
                lo, hi = max(c["start"], col * page), min(c["start"] + n[b], (col + 1) * page)
                fresh = x[b, :, lo - c["start"]:hi - c["start"]]
                top = fresh.abs().amax((1, 2))
                s = torch.exp2(torch.ceil(torch.log2(top / 448.0)))
                s = torch.where(top > 448.0 * s, 2 * s, torch.where(top <= 224.0 * s, s / 2, s))
                held = lo - col * page
                if held:
                    s = torch.maximum(s, scale[pg])
                    old = vals[pg, :, :held] * (scale[pg] / s)[:, None, None]
                    vals[pg, :, :held] = _nearest_e4m3(old)
                vals[pg, :, held:hi - col * page] = _nearest_e4m3(fresh / s[:, None, None])
                scale[pg] = s
        res[name + "8"], res[name + "_scale"] = vals, scale
    return res


def _nearest_e4m3(x):
    """The nearest e4m3 value, ties to the even mantissa (|x| <= 448)."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -30))).clamp(min=-6.0)
    step = torch.exp2(e - 3.0)
    return torch.round(x / step) * step
