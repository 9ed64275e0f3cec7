"""Host-side checks of the softmax operators: bad arguments are refused before
anything is launched (these calls never reach the GPU, so they run anywhere)."""
import ctypes

import pytest
import torch

import kernelized_causal_sequence_b200 as la

INVALID, UNSUPPORTED = la.LA_ERR_INVALID_ARG, la.LA_ERR_UNSUPPORTED
BASE = 1 << 40      # dummy addresses, never dereferenced, 4 GiB apart


def P(i, off=0):
    return ctypes.c_void_p(BASE + (i << 32) + off)


@pytest.fixture(scope="module")
def L():
    from kernelized_causal_sequence_b200 import build
    build.build()
    return la.lib()


@pytest.fixture(autouse=True)
def no_kernel_launched(L):
    before = L.la_launch_count()
    yield
    assert L.la_launch_count() == before, "a host-side check let a kernel launch"


def prefill(L, **kw):
    a = dict(q=P(1), k=P(2), v=P(3), dt=la.LA_BF16, H=8, Hkv=2, N=1000, d=128, cu=P(4), n_seq=3, strides=None,
             scale=0.1, out=P(5), odt=la.LA_BF16, ws=P(6), nws=256)
    a.update(kw)
    if a["strides"] is not None:
        a["strides"] = (ctypes.c_int64 * 8)(*a["strides"])
    return L.la_softmax_prefill(a["q"], a["k"], a["v"], a["dt"], a["H"], a["Hkv"], a["N"], a["d"], a["cu"], a["n_seq"],
                                a["strides"], a["scale"], a["out"], a["odt"], a["ws"], a["nws"], None)


C = [1000 * 128, 128]


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(out=None), INVALID),
    (dict(cu=None), INVALID), (dict(cu=P(4, 2)), INVALID), (dict(q=P(1, 8)), INVALID), (dict(out=P(5, 8)), INVALID),
    (dict(dt=7), INVALID), (dict(odt=-1), INVALID), (dict(odt=la.LA_F16), UNSUPPORTED), (dict(dt=la.LA_F32), UNSUPPORTED),
    (dict(d=96), UNSUPPORTED), (dict(d=256), UNSUPPORTED), (dict(d=0), INVALID), (dict(H=-1), INVALID),
    (dict(H=7), INVALID), (dict(Hkv=0), INVALID), (dict(H=0), INVALID), (dict(H=70000, Hkv=70000), UNSUPPORTED),
    (dict(N=-1), INVALID), (dict(N=(1 << 30) + 1), UNSUPPORTED), (dict(n_seq=-1), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(ws=None), INVALID), (dict(nws=255), INVALID), (dict(ws=P(6, 64)), INVALID),
    (dict(out=P(1)), INVALID), (dict(out=P(1, 1000 * 128 * 16 - 16)), INVALID), (dict(out=P(2)), INVALID),
    (dict(out=P(3)), INVALID), (dict(strides=C + [0, 128] + C + C), INVALID), (dict(strides=C + C + C + [1000 * 128, 64]), INVALID),
    (dict(strides=[1000 * 132, 132] + C + C + C), INVALID), (dict(strides=C + C + [1 << 40, 128] + C), INVALID),
    (dict(strides=[-1000 * 128, 128] + C + C + C), INVALID),
])
def test_prefill_refusals(L, kw, want):
    assert prefill(L, **kw) == want


def test_prefill_nothing_to_do(L):
    for kw in (dict(N=0), dict(n_seq=0), dict(H=0, Hkv=0)):
        assert prefill(L, **kw) == la.LA_OK
    assert la.la_softmax_prefill_workspace_size(8, 2, 100, 128, 1) >= 8
    assert la.la_softmax_prefill_workspace_size(8, 3, 100, 128, 1) == 0
    assert la.la_softmax_prefill_workspace_size(8, 2, 100, 80, 1) == 0


def test_prefill_refuses_a_workspace_over_its_arrays(L):
    """The call sets the workspace's first words before it reads the others."""
    for kw in (dict(ws=P(1)), dict(ws=P(2)), dict(ws=P(3)), dict(ws=P(4)), dict(ws=P(5)), dict(ws=P(1, 8 * 1000 * 256 - 256)),
               dict(ws=P(5, 8 * 1000 * 256 - 256)), dict(out=P(4))):
        assert prefill(L, **kw) == INVALID


@pytest.mark.parametrize("scale,ok", [(1e-45, False), (1e-39, False), (2e-38, True), (2.3e38, True), (2.4e38, False), (3.4e38, False)])
def test_scale_range(L, scale, ok):
    """scale log2(e), which the kernels multiply by, has to be a normal number: neither cut short nor infinite."""
    want = la.LA_OK if ok else INVALID
    assert prefill(L, scale=scale, N=0) == want
    assert L.la_kv4_decode(P(1), la.LA_BF16, 0, ctypes.byref(cache(H_kv=0)), P(2), scale, None, None, P(3), la.LA_BF16, P(4), 256, None) == want


def cache(i=10, **kw):
    a = dict(k_codes=P(i), k_par=P(i + 1), v_codes=P(i + 2), v_par=P(i + 3), B=3, H_kv=2, cap=100, d=64)
    a.update(kw)
    return la._Kv4CacheC(*(x.value if isinstance(x, ctypes.c_void_p) else x for x in a.values()))


BAD_CACHES = [(dict(k_codes=None), INVALID), (dict(k_par=P(11, 4)), INVALID), (dict(v_codes=P(12, 8)), INVALID),
              (dict(v_par=None), INVALID), (dict(d=48), UNSUPPORTED), (dict(d=0), INVALID), (dict(B=-1), INVALID),
              (dict(cap=-1), INVALID), (dict(H_kv=-1), INVALID), (dict(cap=(1 << 30) + 1), UNSUPPORTED)]


@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_bad_caches(L, kw, want):
    c = ctypes.byref(cache(**kw))
    good = ctypes.byref(cache(20))
    assert L.la_kv4_append(P(1), P(2), 1, 3, None, None, P(3), c, None) == want
    assert L.la_kv4_read(c, 3, None, P(3), P(1), P(2), 1, None) == want
    assert L.la_kv4_decode(P(1), 1, 4, c, P(2), 0.1, None, None, P(3), 1, P(4), 1 << 30, None) == want
    assert L.la_kv4_evict(c, P(1), P(2), 10, 0, good, None, None, None, P(3), 1 << 30, None) == want
    assert L.la_kv4_evict(good, P(1), P(2), 10, 0, c, None, None, None, P(3), 1 << 30, None) == want


def test_append_read_refusals(L):
    c = ctypes.byref(cache())
    app = lambda k=P(1), v=P(2), dt=1, N=50, st=None, cu=P(3), start=P(4): L.la_kv4_append(
        k, v, dt, N, None if st is None else (ctypes.c_int64 * 4)(*st), cu, start, c, None)
    assert app(k=None) == app(v=None) == app(start=None) == app(k=P(1, 8)) == app(start=P(4, 1)) == INVALID
    assert app(cu=P(3, 2)) == app(dt=5) == app(N=-1) == app(cu=None) == INVALID
    assert app(st=[50 * 64, 63, 50 * 64, 64]) == app(st=[50 * 64, 64, 50 * 64 + 4, 64]) == INVALID
    assert app(N=(1 << 30) + 1) == UNSUPPORTED
    assert app(N=0) == la.LA_OK
    rd = lambda N=50, cu=P(3), start=P(4), k=P(1), v=P(2), dt=1: L.la_kv4_read(c, N, cu, start, k, v, dt, None)
    assert rd(N=-1) == rd(cu=None) == rd(start=None) == rd(k=None) == rd(v=P(2, 4)) == rd(dt=9) == INVALID
    assert rd(N=(1 << 30) + 1) == UNSUPPORTED
    assert rd(N=0) == la.LA_OK


def test_decode_refusals(L):
    c = ctypes.byref(cache())
    need = la.la_kv4_decode_workspace_size(3, 4, 2, 100, 64, True)
    assert need > 0

    def dec(q=P(1), dt=1, H=4, lens=P(2), scale=0.1, wi=P(5), wo=P(6), out=P(3), odt=1, ws=P(4), nws=need):
        return L.la_kv4_decode(q, dt, H, c, lens, scale, wi, wo, out, odt, ws, nws, None)
    assert dec(q=None) == dec(lens=None) == dec(out=None) == dec(q=P(1, 4)) == dec(lens=P(2, 2)) == INVALID
    assert dec(dt=9) == dec(H=3) == dec(H=-2) == dec(scale=0.0) == dec(scale=float("nan")) == INVALID
    assert dec(wo=None) == dec(wi=P(5, 4)) == dec(wo=P(6, 8)) == dec(wi=P(6, 16)) == INVALID
    assert dec(out=P(1)) == dec(out=P(1, 16)) == INVALID
    assert dec(ws=None) == dec(nws=need - 1) == dec(ws=P(4, 16)) == INVALID
    assert dec(odt=2) == dec(H=70000) == UNSUPPORTED
    assert la.la_kv4_decode_workspace_size(3, 5, 2, 100, 64) == 0


def test_evict_refusals(L):
    need = la.la_kv4_evict_workspace_size(3, 2, 100, 10)
    assert need > 0

    def ev(c=None, o=None, w=P(1), lens=P(2), keep=10, recent=0, ow=P(5), kept=P(6), ol=P(7), ws=P(3), nws=need):
        return L.la_kv4_evict(ctypes.byref(c or cache()), w, lens, keep, recent, ctypes.byref(o or cache(20, cap=12)),
                              ow, kept, ol, ws, nws, None)
    assert ev(w=None) == ev(lens=None) == ev(w=P(1, 4)) == ev(lens=P(2, 1)) == ev(kept=P(6, 2)) == INVALID
    assert ev(ol=P(7, 2)) == ev(ow=P(5, 4)) == ev(ow=P(1)) == INVALID
    assert ev(keep=0) == ev(recent=-1) == ev(recent=11) == ev(keep=13) == INVALID
    assert ev(o=cache(20, B=2)) == ev(o=cache(20, H_kv=1)) == ev(o=cache(20, d=32)) == INVALID
    assert ev(o=cache(10)) == ev(o=cache(20, v_codes=P(10))) == ev(o=cache(20, k_par=P(13))) == INVALID
    assert ev(kept=None, ws=None) == ev(kept=None, nws=need - 1) == ev(kept=None, ws=P(3, 32)) == INVALID


def test_evict_refuses_outputs_over_inputs(L):
    """One head's results are written while another's lengths and weights are read."""
    def ev(lens=P(2), kept=P(6), ol=P(7)):
        return L.la_kv4_evict(ctypes.byref(cache()), P(1), lens, 10, 0, ctypes.byref(cache(20, cap=12)), P(5), kept, ol,
                              None, 0, None)
    assert ev(ol=P(2)) == ev(lens=P(2, 8), ol=P(2)) == ev(kept=P(2)) == ev(kept=P(1, 16)) == INVALID


def pairs(names, regions, given):
    """Each (output, other) pair by name, with the output laid over the first and the last bytes of the other."""
    for name in given:
        for other in names:
            if other != name:
                at, n = regions[other]
                yield name, other, at
                yield name, other, at + n - 16


# (bytes of the arrays of cache(): B 3, H_kv 2, cap 100, d 64)
CACHE_BYTES = [600 * 32, 600 * 8, 600 * 32, 600 * 8]


def test_evict_refuses_any_overlap(L):
    """No output over an input or another output, first bytes or last, the workspace among them."""
    size = dict(zip(("kc", "kp", "vc", "vp"), CACHE_BYTES), w=600 * 4, lens=16, okc=72 * 32, okp=72 * 8, ovc=72 * 32, ovp=72 * 8,
                ow=72 * 4, kept=60 * 4, ol=16, ws=256)
    place = {x: (P(i + 1).value, n) for i, (x, n) in enumerate(size.items())}
    outputs = ["okc", "okp", "ovc", "ovp", "ow", "kept", "ol", "ws"]

    def ev(**at):
        a = {x: p for x, (p, _) in place.items()}
        a.update(at)
        kept = a["kept"] if "ws" not in at else None      # the workspace holds the list where `kept` is not given
        return L.la_kv4_evict(ctypes.byref(la._Kv4CacheC(a["kc"], a["kp"], a["vc"], a["vp"], 3, 2, 100, 64)), a["w"], a["lens"],
                              10, 0, ctypes.byref(la._Kv4CacheC(a["okc"], a["okp"], a["ovc"], a["ovp"], 3, 2, 12, 64)),
                              a["ow"], kept, a["ol"], a["ws"], 256, None)
    names = [x for x in size if x != "ws"]
    wrong = [(o, x) for o, x, at in pairs(names, place, outputs)
             if not (o == "ws" and (x == "kept" or at % 256)) and ev(**{o: at}) != INVALID]
    assert not wrong


def test_decode_refuses_any_overlap(L):
    """No output over an input or another output, the workspace among them; weights_in may be weights_out."""
    need = la.la_kv4_decode_workspace_size(3, 4, 2, 100, 64, True)
    size = dict(zip(("kc", "kp", "vc", "vp"), CACHE_BYTES), q=12 * 128, lens=16, wi=600 * 4, wo=600 * 4, out=12 * 128, ws=need)
    place = {x: (P(i + 1).value, n) for i, (x, n) in enumerate(size.items())}

    def dec(**at):
        a = {x: p for x, (p, _) in place.items()}
        a.update(at)
        c = la._Kv4CacheC(a["kc"], a["kp"], a["vc"], a["vp"], 3, 2, 100, 64)
        return L.la_kv4_decode(a["q"], la.LA_BF16, 4, ctypes.byref(c), a["lens"], 0.1, a["wi"], a["wo"], a["out"], la.LA_BF16,
                               a["ws"], need, None)
    wrong = [(o, x) for o, x, at in pairs(size, place, ["out", "wo", "ws"])
             if not (o == "ws" and at % 256) and not (o == "wo" and x == "wi" and at == place["wi"][0]) and dec(**{o: at}) != INVALID]
    assert not wrong


def test_append_read_refuse_any_overlap(L):
    """No cache array over an input or another array in an append, no output over the cache, the indexes or the other
    output in a read."""
    size = dict(zip(("kc", "kp", "vc", "vp"), CACHE_BYTES), k=2 * 50 * 128, v=2 * 50 * 128, cu=16, start=16)
    place = {x: (P(i + 1).value, n) for i, (x, n) in enumerate(size.items())}

    def call(which, **at):
        a = {x: p for x, (p, _) in place.items()}
        a.update(at)
        c = ctypes.byref(la._Kv4CacheC(a["kc"], a["kp"], a["vc"], a["vp"], 3, 2, 100, 64))
        if which == "append":
            return L.la_kv4_append(a["k"], a["v"], la.LA_BF16, 50, None, a["cu"], a["start"], c, None)
        return L.la_kv4_read(c, 50, a["cu"], a["start"], a["k"], a["v"], la.LA_BF16, None)
    wrong = [("append", o, x) for o, x, at in pairs(size, place, ["kc", "kp", "vc", "vp"]) if call("append", **{o: at}) != INVALID]
    wrong += [("read", o, x) for o, x, at in pairs(size, place, ["k", "v"]) if call("read", **{o: at}) != INVALID]
    assert not wrong


def test_evict_lengths_need_a_head(L):
    """The new lengths are written with the heads' results: without a head nobody writes them."""
    def ev(ol, **kw):
        return L.la_kv4_evict(ctypes.byref(cache(H_kv=0, **kw)), P(1), P(2), 10, 0, ctypes.byref(cache(20, H_kv=0, cap=12, **kw)),
                              P(5), P(6), ol, None, 0, None)
    assert ev(P(7)) == INVALID
    assert ev(None) == ev(P(7), B=0) == la.LA_OK


def test_python_checks():
    f = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)
    i = lambda n: torch.zeros(n, dtype=torch.int32)
    with pytest.raises(ValueError):
        la.la_softmax_prefill(f(4, 10, 64), f(2, 10, 64), f(2, 10, 64), i(3))     # not on CUDA
    with pytest.raises(ValueError):
        la.la_softmax_prefill(f(10, 64), f(2, 10, 64), f(2, 10, 64), i(3))
    c = la.KV4Cache.alloc(2, 1, 8, 64, "cpu")
    assert [tuple(x.shape) for x in c] == [(2, 1, 8, 32), (2, 1, 8, 2)] * 2
    for call in (lambda: la.la_kv4_append(f(1, 2, 64), f(1, 2, 64), c, i(2)), lambda: la.la_kv4_read(c, i(2), 2),
                 lambda: la.la_kv4_decode(f(2, 4, 64), c, i(2)), lambda: la.la_kv4_evict(c, f(2, 1, 8), i(2), 4)):
        with pytest.raises(ValueError):
            call()
