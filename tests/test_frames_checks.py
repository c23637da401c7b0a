"""Refusals of the windowed attention and the 8-bit cache calls, all made on
the host before anything is enqueued (CPU)."""
import ctypes

import pytest
import torch

from free_block_sparse_eigenbasis_b200 import sparsepr as S

FAKE = ctypes.c_void_p(1 << 40)  # never dereferenced: every call fails first
ODD = ctypes.c_void_p((1 << 40) + 4)
WIN = dict(B=2, Hq=4, Hkv=2, Nq=8, Nk=16, d=64, frame=1, window=0, sinks=0, causal=1)
CACHE = dict(B=2, Hkv=2, d=64, page=16, n_pages=8, max_pages=4)
ATTN = dict(Hq=4, Nq=1, frame=1, window=0, sinks=0, causal=1)


def window(p=WIN, q=FAKE, k=FAKE, v=FAKE, out=ctypes.c_void_p(1 << 41), lse=None, ws=FAKE,
           nbytes=1 << 40, dt=S.BF16):
    return S.lib.sparsepr_window_attention(q, k, v, dt, ctypes.byref(S.make_window_params(p)),
                                           None, None, out, lse, ws, nbytes, None)


@pytest.mark.parametrize("bad", [
    dict(B=0), dict(Hq=0), dict(Hkv=0), dict(Hq=3), dict(Nq=-1), dict(Nk=-1), dict(frame=0),
    dict(window=-1), dict(sinks=-1), dict(causal=2), dict(scale=-1.0), dict(scale=float("nan"))])
def test_window_parameters(bad):
    p = dict(WIN, **bad)
    assert S.lib.sparsepr_window_workspace_bytes(ctypes.byref(S.make_window_params(p)), S.BF16) == 0
    assert window(p) == S.ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(d=96), dict(B=40000), dict(Nq=1 << 30),
                                 dict(Nk=(1 << 31) - 1)])
def test_window_sizes_that_are_not_built(bad):
    assert window(dict(WIN, **bad)) == S.ERR_UNSUPPORTED


def test_window_pointers():
    assert window(dt=7) == S.ERR_UNSUPPORTED
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(q=ODD),
                dict(out=ODD), dict(lse=ctypes.c_void_p(2)), dict(out=FAKE)):
        assert window(**bad) == S.ERR_INVALID_ARG, bad
    assert window(ws=None) == S.ERR_WORKSPACE
    assert window(ws=ODD) == S.ERR_WORKSPACE
    assert window(nbytes=16) == S.ERR_WORKSPACE
    # nothing to do: no query rows
    assert window(dict(WIN, Nq=0), q=None, out=None) == S.OK


def cache_pointers(**bad):
    return ctypes.byref(S.CachePointers(**{n: bad.get(n, (1 << 40) + (i << 32)) for i, n in enumerate(
        ("k8", "v8", "k_scale", "v_scale", "table", "len", "ref"))}))


def every_cache_call(p, c, nbytes=1 << 40, ws=FAKE):
    pp = ctypes.byref(S.make_cache_params(p))
    a = ctypes.byref(S.make_cache_attention_params(ATTN))
    see = ctypes.byref(S.Visibility(1, 4, 0, 1))
    L = S.lib
    yield L.sparsepr_cache_reserve(pp, c, FAKE, ctypes.c_void_p(1 << 41), ws, nbytes, None)
    yield L.sparsepr_cache_append(FAKE, FAKE, S.BF16, 4, pp, c, FAKE, None, ws, nbytes, None)
    yield L.sparsepr_cache_attention(FAKE, S.BF16, pp, c, a, None, ctypes.c_void_p(1 << 41), None,
                                     ws, nbytes, None)
    yield L.sparsepr_cache_fork(pp, c, FAKE, FAKE, 1, ws, nbytes, None)
    yield L.sparsepr_cache_free(pp, c, FAKE, 1, ws, nbytes, None)
    yield L.sparsepr_cache_evict(pp, c, see, ws, nbytes, None)
    yield L.sparsepr_cache_compact(pp, c, FAKE, ws, nbytes, None)


@pytest.mark.parametrize("bad,code", [
    (dict(B=0), S.ERR_INVALID_ARG), (dict(B=1025), S.ERR_INVALID_ARG),
    (dict(Hkv=0), S.ERR_INVALID_ARG), (dict(n_pages=0), S.ERR_INVALID_ARG),
    (dict(max_pages=0), S.ERR_INVALID_ARG), (dict(d=32), S.ERR_UNSUPPORTED),
    (dict(page=48), S.ERR_UNSUPPORTED), (dict(max_pages=1 << 28), S.ERR_UNSUPPORTED)])
def test_cache_parameters(bad, code):
    p = dict(CACHE, **bad)
    assert S.lib.sparsepr_cache_workspace_bytes(ctypes.byref(S.make_cache_params(p)), None) == 0
    got = list(every_cache_call(p, cache_pointers()))
    if "Hkv" in bad:  # the attention checks the head counts too
        assert all(g in (code, S.ERR_INVALID_ARG) for g in got)
    else:
        assert got == [code] * 7


def test_cache_pointers():
    for name in ("k8", "v8", "k_scale", "v_scale", "table", "len", "ref"):
        assert list(every_cache_call(CACHE, cache_pointers(**{name: None}))) == [1] * 7
        assert list(every_cache_call(CACHE, cache_pointers(**{name: (1 << 40) + 2}))) == [1] * 7
    assert list(every_cache_call(CACHE, None)) == [1] * 7
    assert list(every_cache_call(CACHE, cache_pointers(v8=1 << 40))) == [1] * 7  # one pool twice
    assert list(every_cache_call(CACHE, cache_pointers(), nbytes=64)) == [S.ERR_WORKSPACE] * 7
    assert list(every_cache_call(CACHE, cache_pointers(), ws=ODD)) == [S.ERR_WORKSPACE] * 7


def test_cache_call_arguments():
    pp, c, L = ctypes.byref(S.make_cache_params(CACHE)), cache_pointers(), S.lib
    big, out = 1 << 40, ctypes.c_void_p(1 << 41)

    def attend(bad=None, q=FAKE, out=out, dt=S.BF16):
        a = S.make_cache_attention_params(dict(ATTN, **(bad or {})))
        return L.sparsepr_cache_attention(q, dt, pp, c, ctypes.byref(a), None, out, None, FAKE, big,
                                          None)
    for bad in (dict(Hq=3), dict(Hq=0), dict(Nq=-1), dict(frame=0), dict(window=-2), dict(sinks=-1),
                dict(causal=-1), dict(scale=float("inf"))):
        assert attend(bad) == S.ERR_INVALID_ARG, bad
    assert attend(dict(Nq=1 << 30)) == S.ERR_UNSUPPORTED
    wide = ctypes.byref(S.make_cache_params(dict(CACHE, B=1024, max_pages=1 << 26)))
    a = ctypes.byref(S.make_cache_attention_params(ATTN))
    assert L.sparsepr_cache_workspace_bytes(wide, None) > 0
    assert L.sparsepr_cache_workspace_bytes(wide, a) == 0  # more tiles than 2^31
    assert attend(q=None) == attend(out=None) == attend(out=FAKE) == S.ERR_INVALID_ARG
    assert attend(dt=5) == S.ERR_UNSUPPORTED
    assert attend(dict(Nq=0), q=None, out=None) == S.OK
    # reserve: start may not be the lengths or the counts
    assert L.sparsepr_cache_reserve(pp, c, FAKE, FAKE, FAKE, big, None) == S.ERR_INVALID_ARG
    assert L.sparsepr_cache_reserve(pp, c, None, out, FAKE, big, None) == S.ERR_INVALID_ARG
    # append
    assert L.sparsepr_cache_append(FAKE, FAKE, S.BF16, -1, pp, c, FAKE, None, FAKE, big,
                                   None) == S.ERR_INVALID_ARG
    assert L.sparsepr_cache_append(FAKE, None, S.BF16, 1, pp, c, FAKE, None, FAKE, big,
                                   None) == S.ERR_INVALID_ARG
    assert L.sparsepr_cache_append(ODD, FAKE, S.BF16, 1, pp, c, FAKE, None, FAKE, big,
                                   None) == S.ERR_INVALID_ARG
    assert L.sparsepr_cache_append(FAKE, FAKE, S.BF16, 1, pp, c, None, None, FAKE, big,
                                   None) == S.ERR_INVALID_ARG
    assert L.sparsepr_cache_append(FAKE, FAKE, 9, 1, pp, c, FAKE, None, FAKE, big,
                                   None) == S.ERR_UNSUPPORTED
    assert L.sparsepr_cache_append(None, None, S.BF16, 0, pp, c, FAKE, None, FAKE, big,
                                   None) == S.OK
    # lists
    assert L.sparsepr_cache_fork(pp, c, FAKE, None, 1, FAKE, big, None) == S.ERR_INVALID_ARG
    assert L.sparsepr_cache_fork(pp, c, FAKE, FAKE, -1, FAKE, big, None) == S.ERR_INVALID_ARG
    assert L.sparsepr_cache_fork(pp, c, None, None, 0, FAKE, big, None) == S.OK
    assert L.sparsepr_cache_free(pp, c, None, 1, FAKE, big, None) == S.ERR_INVALID_ARG
    assert L.sparsepr_cache_free(pp, c, None, 0, FAKE, big, None) == S.OK
    # eviction needs a causal window
    for see in ((1, 0, 0, 1), (1, 4, 0, 0), (0, 4, 0, 1), (1, 4, -1, 1)):
        assert L.sparsepr_cache_evict(pp, c, ctypes.byref(S.Visibility(*see)), FAKE, big,
                                      None) == S.ERR_INVALID_ARG, see
    assert L.sparsepr_cache_compact(pp, c, None, FAKE, big, None) == S.ERR_INVALID_ARG


def test_binding_refuses_what_the_library_cannot_see(monkeypatch):
    calls = []

    class Recorder:
        def __getattr__(self, name):
            if name.endswith("_bytes") or name.endswith("string"):
                return getattr(real, name)
            return lambda *a: calls.append(name) or S.OK
    real = S.lib
    monkeypatch.setattr(S, "lib", Recorder())
    monkeypatch.setattr(S, "_DEVICE_TYPE", "cpu")

    class Stream:
        cuda_stream = 0
    st = Stream()
    bf, i32 = torch.bfloat16, torch.int32
    q, k = torch.zeros(2, 4, 8, 64, dtype=bf), torch.zeros(2, 2, 16, 64, dtype=bf)
    ws = S.allocate_window_workspace(WIN, bf, "cpu")
    ok = dict(out=q.clone(), ws=ws, stream=st)
    S.sparsepr_window_attention(q, k, k.clone(), WIN, **ok)
    wide = torch.zeros(2, 2, 16, 128, dtype=bf)[..., :64]
    for args, kw in (((q, wide, k), {}), ((q, k, k.float()), {}), ((q[:, :3], k, k), {}),
                     ((q.half(), k.half(), k.half()), {}),
                     ((q, k, k), dict(lse=torch.zeros(2, 4, 8, dtype=bf))),
                     ((q, k, k), dict(n_q=torch.zeros(2, dtype=torch.int64))),
                     ((q, k, k), dict(n_k=torch.zeros(3, dtype=i32)))):
        with pytest.raises((TypeError, ValueError)):
            S.sparsepr_window_attention(*args, WIN, **ok, **kw)
    c = S.allocate_cache(CACHE, "cpu")
    assert c.table.min() == -1 and c.ref.sum() == 0
    cws = S.allocate_cache_workspace(CACHE, ATTN, "cpu")
    assert cws.numel() >= S.allocate_cache_workspace(CACHE, None, "cpu").numel()
    n = torch.zeros(2, dtype=i32)
    S.sparsepr_cache_reserve(n, CACHE, c, n.clone(), cws, st)
    S.sparsepr_cache_append(k, k, CACHE, c, n, None, cws, st)
    S.sparsepr_cache_attention(q[:, :, :1].contiguous(), CACHE, c, ATTN,
                               torch.zeros(2, 4, 1, 64, dtype=bf), cws, stream=st)
    S.sparsepr_cache_fork(n[:1], n[1:], CACHE, c, cws, st)
    S.sparsepr_cache_free(n, CACHE, c, cws, st)
    S.sparsepr_cache_evict(dict(window=4), CACHE, c, cws, st)
    S.sparsepr_cache_compact(CACHE, c, n[:1], cws, st)
    done = list(calls)
    with pytest.raises(ValueError):
        S.sparsepr_cache_append(k[:, :, :, :32], k, CACHE, c, n, None, cws, st)
    with pytest.raises(ValueError):
        S.sparsepr_cache_fork(n[:1], n, CACHE, c, cws, st)
    with pytest.raises(TypeError):
        S.sparsepr_cache_free(n.long(), CACHE, c, cws, st)
    c.k8 = c.k8.view(torch.uint8)
    with pytest.raises(TypeError):
        S.sparsepr_cache_evict(dict(window=4), CACHE, c, cws, st)
    assert calls == done
    with pytest.raises(S.SparsePRError):
        S.allocate_cache(dict(CACHE, page=20), "cpu")
    with pytest.raises(S.SparsePRError):
        S.allocate_window_workspace(dict(WIN, d=80), bf, "cpu")
    with pytest.raises(S.SparsePRError):
        S.allocate_window_workspace(WIN, torch.float16, "cpu")


def test_host_tensors_are_refused():
    q = torch.zeros(2, 4, 8, 64, dtype=torch.bfloat16)
    k = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA tensor"):
        S.sparsepr_window_attention(q, k, k, WIN, q.clone(), ws)
    with pytest.raises(ValueError, match="CUDA tensor"):
        S.sparsepr_cache_compact(CACHE, S.allocate_cache(CACHE, "cpu"),
                                 torch.zeros(1, dtype=torch.int32), ws)


def test_status_string_of_capacity():
    assert "page" in S.status_string(S.ERR_CAPACITY)


@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("big", [dict(frame=2 ** 31 - 1, window=2 ** 31 - 1, sinks=2 ** 31 - 1),
                                 dict(frame=1 << 20, window=2 ** 31 - 1),
                                 dict(frame=2 ** 31 - 1, window=1)])
def test_workspace_of_the_largest_windows(big, causal):
    """A window that reaches every key needs the scratch of none: products of
    frames and windows do not overflow where the key ranges are planned."""
    p = dict(B=1, Hq=12, Hkv=12, Nq=1, Nk=4001, d=128, frame=1, window=0, sinks=0, causal=causal)
    need = [S.lib.sparsepr_window_workspace_bytes(
        ctypes.byref(S.make_window_params(dict(p, **kw))), S.BF16) for kw in ({}, big)]
    assert need[0] == need[1] > 0


def test_workspace_of_the_longest_run_of_queries():
    """Units are counted without overflow up to the last row count allowed: the
    scratch is at most that of 16 rounds of cut units of 256 rows."""
    p = dict(B=1, Hq=1, Hkv=1, Nq=2 ** 31 - 1, Nk=64, d=64, frame=1, window=0, sinks=0, causal=1)
    need = S.lib.sparsepr_window_workspace_bytes(ctypes.byref(S.make_window_params(p)), S.BF16)
    assert 0 < need <= 16 * 148 * 256 * (64 + 1) * 4 + 4096


@pytest.mark.parametrize("scale,code", [(1e39, S.ERR_INVALID_ARG), (1e300, S.ERR_INVALID_ARG),
                                        (2.0 ** 126, S.OK), (1e-300, S.OK)])
def test_scales_that_fp32_does_not_hold(scale, code):
    """A scale that is infinite in fp32 would make NaN of every logit of 0."""
    assert window(dict(WIN, Nq=0, scale=scale), q=None, out=None) == code
    a = S.make_cache_attention_params(dict(ATTN, Nq=0, scale=scale))
    assert S.lib.sparsepr_cache_attention(None, S.BF16, ctypes.byref(S.make_cache_params(CACHE)),
                                          cache_pointers(), ctypes.byref(a), None, None, None, FAKE,
                                          1 << 40, None) == code
