"""The softmax operators (packed prompt attention, 4-bit cache: append, read,
decode, evict) against plain float64 implementations, at the sizes and masks
where they can go wrong, and a run of them together.

Tolerances are bounds, with u = half a step of a type (bf16 2^-8, fp16 2^-11,
fp32 2^-24), A = sum_j p_j |v_j| for the output at hand:

- a score q.k is off by at most (d + 3) u32 sum_c |q_c k_c| (products and sums
  in fp32); its exponential by that, by the rounding of the scaled score (twice
  u32 |s|, for the maximum too) and by the exponential function itself (2^-20
  allowed), and numerator and denominator both carry it;
- the sums over n keys add (n + 64) u32 each;
- where the weights are rounded to 16 bits for the product with v, u of that
  type times A more;
- the output's own rounding, u |o|.
"""
import math

import numpy as np
import pytest
import torch

DEV = "cuda"
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
U32 = 2.0 ** -24


# ------------------------------------------------------------------ references
def ref_prefill(q, k, v, lens, scale):
    """(out, bound without roundings to 16 bits, A) in float64, [H, N, d]."""
    H, N, d = q.shape
    G = H // k.shape[0]
    q, k, v = q.double(), k.double(), v.double()
    out, rel, A = torch.zeros_like(q), torch.zeros_like(q[..., :1]), torch.zeros_like(q)
    t = 0
    for n in [x for x in lens if x]:
        r = slice(t, t + n)
        for h in range(H):
            kk, vv = k[h // G, r], v[h // G, r]
            s = scale * q[h, r] @ kk.T
            s = torch.where(torch.ones(n, n, dtype=torch.bool).tril(), s, -math.inf)
            p = torch.softmax(s, -1)
            out[h, r], A[h, r] = p @ vv, p @ vv.abs()
            ds = scale * (d + 3) * U32 * (q[h, r].abs() @ kk.abs().T) + 4 * U32 * s.abs().nan_to_num(posinf=0)
            ds = torch.where(torch.ones(n, n, dtype=torch.bool).tril(), ds, 0).amax(-1)
            rel[h, r, 0] = 2 * ds + 2 * 2.0 ** -20 + 2 * (n + 64) * U32
        t += n
    return out, rel * A, A


def check_prefill(out, q, k, v, lens, scale, in16):
    ref, tol, A = ref_prefill(q, k, v, lens, scale)
    if in16:
        tol = tol + U[q.dtype] * A
    tol = tol + U[out.dtype] * (ref.abs() + tol) + 1e-30
    n = sum(lens)
    err = (out.double().cpu() - ref).abs()[:, :n]
    assert torch.isfinite(out[:, :n]).all()
    worst = float((err / tol[:, :n]).max()) if n else 0.0
    assert worst <= 1.0, f"{worst} of the bound"


def pack_ref(x):
    """(codes uint8, scale float64, offset float64) of rows x [..., d]: the definition."""
    g = x.double().numpy().reshape(*x.shape[:-1], -1, 32)
    lo, hi = g.min(-1), g.max(-1)
    sc = np.maximum((hi - lo) / 15.0, np.abs(g).max(-1) / 1024.0).astype(np.float32)
    sc = torch.from_numpy(sc).to(torch.bfloat16).double().numpy()
    safe = np.where(sc > 0, sc, 1.0)
    off = np.where(sc > 0, lo / safe, 0.0).astype(np.float32).astype(np.float16).astype(np.float64)
    c = np.where(sc[..., None] > 0, np.clip(np.rint(g / safe[..., None] - off[..., None]), 0, 15), 0)
    return c.astype(np.uint8), sc, off


def values_ref(x):
    c, sc, off = pack_ref(x)
    return torch.from_numpy((sc[..., None] * (c + off[..., None])).reshape(x.shape))


def rows_ref(x):
    """The bytes and words of rows x, as linattn.h lays them out."""
    c, sc, off = pack_ref(x)
    d = x.shape[-1]
    G = d // 32
    b = np.zeros((*x.shape[:-1], d // 2), dtype=np.uint8)
    for g in range(G):
        for r in range(8):
            f = c[..., g, 4 * r:4 * r + 4].astype(np.uint32)
            field = f[..., 0] | f[..., 1] << 4 | f[..., 2] << 8 | f[..., 3] << 12
            b[..., r * 2 * G + 2 * g] = field & 255
            b[..., r * 2 * G + 2 * g + 1] = field >> 8
    s = torch.from_numpy(sc).to(torch.bfloat16).view(torch.int16).numpy().astype(np.uint16).astype(np.uint32)
    o = off.astype(np.float16).view(np.uint16).astype(np.uint32)
    return torch.from_numpy(b), torch.from_numpy((s | o << 16).view(np.int32))


def new_cache(la, B, Hkv, cap, d, fill=0xA5):
    c = la.KV4Cache.alloc(B, Hkv, cap, d, DEV)
    for x in c:
        x.view(torch.uint8).fill_(fill)
    return c


def fill_cache(la, k, v):
    """A cache that holds k, v [B, Hkv, T, d] at positions 0 .. T - 1 (garbage behind), and its values."""
    B, Hkv, T, d = k.shape
    c = new_cache(la, B, Hkv, T + 5, d, fill=0xFF)      # scale and offset of the garbage: NaN
    for x, codes, par in ((k, c.k_codes, c.k_par), (v, c.v_codes, c.v_par)):
        b, w = rows_ref(x)
        codes[:, :, :T] = b.to(DEV)
        par[:, :, :T] = w.to(DEV)
    return c, values_ref(k), values_ref(v)


def ref_decode(q, k, v, lens, scale, vscale):
    """(out, bound, A, weights [B, Hkv, T]); vscale: the values' scales [B, Hkv, T, d / 32]."""
    B, H, d = q.shape
    Hkv, T = k.shape[1], k.shape[2]
    G = H // Hkv
    out = torch.zeros(B, H, d, dtype=torch.float64)
    A, tol = out.clone(), out.clone()
    w = torch.zeros(B, Hkv, T, dtype=torch.float64)
    wtol = w.clone()
    for b in range(B):
        n = lens[b]
        if n == 0:
            continue
        for h in range(H):
            kk, vv = k[b, h // G, :n], v[b, h // G, :n]
            s = scale * kk @ q[b, h].double()
            p = torch.softmax(s, -1)
            out[b, h], A[b, h] = p @ vv, p @ vv.abs()
            # a code's contribution is taken around 16: terms up to 31 scales plus the offset's
            ksc = kk.abs().amax(-1)
            big = (q[b, h].double().abs().sum() * ksc * 40)
            ds = float((scale * (d + 8) * U32 * big + 4 * U32 * s.abs()).max())
            rel = 2 * ds + 2 * 2.0 ** -20 + 2 * (n + 64) * U32
            wide = (p[:, None] * vscale[b, h // G, :n] * 64).sum(0).repeat_interleave(32)
            tol[b, h] = rel * A[b, h] + (n + 64) * U32 * wide
            w[b, h // G, :n] += p
            wtol[b, h // G, :n] += rel * p
    return out, tol, A, w, wtol


# ------------------------------------------------------------------ prompt attention
PREFILL = [
    # (dtype, out dtype or None, d, H, Hkv, lens, tail)
    (torch.float32, None, 64, 4, 2, [1, 5, 64, 65, 0, 130], 3),
    (torch.float32, None, 32, 3, 1, [33, 1, 1, 200], 0),
    (torch.float32, None, 128, 2, 2, [129, 300], 1),
    (torch.bfloat16, None, 32, 4, 4, [70, 2, 129], 0),
    (torch.float16, torch.float32, 32, 2, 1, [257], 9),
    (torch.float16, None, 32, 6, 2, [1, 128, 129, 0, 1000], 2),
    (torch.bfloat16, None, 128, 4, 1, [1], 0),
    (torch.bfloat16, None, 128, 4, 2, [1, 2, 3, 127, 128, 129, 0, 255, 256, 257], 5),
    (torch.bfloat16, torch.float32, 128, 6, 2, [385, 513], 0),
    (torch.bfloat16, None, 64, 5, 5, [640, 1, 77], 130),
    (torch.float16, None, 64, 8, 1, [1, 300, 0, 0, 511], 0),
    (torch.float16, torch.float32, 128, 2, 2, [1000, 24], 0),
    (torch.float16, None, 128, 3, 1, [2049], 1),
    # each way the tensor-core kernel fills a CTA: one tile, two heads, two tiles
    (torch.bfloat16, None, 64, 4, 2, [2500, 2100], 1),
    (torch.float16, torch.float32, 64, 2, 1, [2305], 0),
    (torch.bfloat16, None, 128, 32, 16, [2500, 130], 7),
    (torch.float16, torch.float32, 128, 30, 2, [1, 3000], 0),
    (torch.bfloat16, None, 128, 3, 3, [1, 130, 77, 0, 256, 383, 300], 65),
    (torch.float16, torch.float32, 128, 1, 1, [255, 129, 128, 1], 0),
    (torch.bfloat16, torch.float32, 128, 3, 1, [700, 384, 900], 3),
    # two tiles and two heads over sequences of every length, empty ones among them
    (torch.bfloat16, None, 128, 9, 3, [0, 1, 255, 256, 257, 0, 384, 513, 900, 1300, 64, 1100], 11),
    (torch.float16, torch.float32, 128, 12, 2, [65, 0, 0, 1200, 128, 129, 640, 1, 511, 383, 0, 1700], 0),
]


def prefill_inputs(dtype, d, H, Hkv, N, seed):
    g = torch.Generator().manual_seed(seed)
    mk = lambda h: torch.randn(h, N, d, generator=g).to(dtype)
    return mk(H), mk(Hkv), mk(Hkv)


def cu_of(lens):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device=DEV)


def tensor_cores(dtype, d):
    # 16-bit inputs: the weights are rounded to that type
    return dtype != torch.float32


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,od,d,H,Hkv,lens,tail", PREFILL)
def test_prefill(la, dtype, od, d, H, Hkv, lens, tail):
    N = sum(lens) + tail
    q, k, v = prefill_inputs(dtype, d, H, Hkv, N, seed=N + d)
    # rows behind the last sequence hold NaN: they reach nothing
    for x in (q, k, v):
        x[:, sum(lens):] = math.nan
    out = torch.full((H, N, d), 7.0, dtype=od or dtype, device=DEV)
    ret = la.la_softmax_prefill(q.to(DEV), k.to(DEV), v.to(DEV), cu_of(lens), out=out)
    torch.cuda.synchronize()
    assert ret is out
    assert (out[:, sum(lens):] == 7.0).all()
    check_prefill(out, q, k, v, lens, d ** -0.5, tensor_cores(dtype, d))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", [(torch.float32, 64), (torch.bfloat16, 128), (torch.float16, 64)])
def test_prefill_many_single_tokens(la, dtype, d):
    """A token alone attends to itself: its output is its head's value row."""
    S, H, Hkv = 300, 4, 2
    q, k, v = prefill_inputs(dtype, d, H, Hkv, S, seed=1)
    out = la.la_softmax_prefill(q.to(DEV), k.to(DEV), v.to(DEV), cu_of([1] * S))
    assert torch.equal(out.cpu(), v.repeat_interleave(H // Hkv, 0))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", [(torch.float32, 64), (torch.bfloat16, 128), (torch.float16, 64), (torch.bfloat16, 32)])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_prefill_hidden_keys_do_not_reach(la, dtype, d, bad):
    """A NaN or infinity in a key or value leaves the queries before it, the
    other channels and the other sequences exactly as they are without it."""
    hidden_keys(la, dtype, d, 4, 2, bad)


@pytest.mark.gpu
@pytest.mark.parametrize("H,Hkv,first,d", [(3, 3, 300, 64), (3, 3, 300, 128), (32, 16, 2900, 128), (30, 2, 2900, 128)])
def test_prefill_hidden_keys_all_slots(la, H, Hkv, first, d):
    """The same where a CTA holds one tile, two tiles and two heads."""
    hidden_keys(la, torch.bfloat16, d, H, Hkv, math.nan, first=first)


def hidden_keys(la, dtype, d, H, Hkv, bad, first=300):
    lens = [first, 150]
    G = H // Hkv
    q, k, v = prefill_inputs(dtype, d, H, Hkv, first + 150, seed=3)
    run = lambda kk, vv: la.la_softmax_prefill(q.to(DEV), kk.to(DEV), vv.to(DEV), cu_of(lens)).cpu()
    clean = run(k, v)
    for at in (5, 131, first - 1):
        kb, vb = k.clone(), v.clone()
        vb[0, at, 3] = bad
        got = run(k, vb)
        same = torch.ones_like(clean, dtype=torch.bool)
        same[:G, at:first, 3] = False
        assert torch.equal(got[same], clean[same])
        assert not torch.isfinite(got[:G, at:first, 3]).any()
        kb[0, at, 3] = bad
        got = run(kb, v)
        same[:G, at:first] = False
        assert torch.equal(got[same], clean[same])


@pytest.mark.gpu
def test_prefill_strided_views(la):
    """q, k, v as views of one token-major projection, out token-major."""
    N, H, Hkv, d = 333, 6, 2, 128
    lens = [100, 233]
    g = torch.Generator().manual_seed(4)
    qkv = torch.randn(N, (H + 2 * Hkv) * d, generator=g).to(torch.bfloat16).to(DEV)
    heads = qkv.view(N, H + 2 * Hkv, d).transpose(0, 1)
    q, k, v = heads[:H], heads[H:H + Hkv], heads[H + Hkv:]
    out = torch.zeros(N, H, d, dtype=torch.bfloat16, device=DEV)
    la.la_softmax_prefill(q, k, v, cu_of(lens), out=out.transpose(0, 1))
    want = la.la_softmax_prefill(q.contiguous(), k.contiguous(), v.contiguous(), cu_of(lens))
    assert torch.equal(out.transpose(0, 1), want)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_prefill_large_scores(la, dtype):
    """Scores up to several hundred, some rows dominated by one key, one row by equal keys."""
    d, lens = 64, [200]
    q, k, v = prefill_inputs(dtype, d, 2, 1, 200, seed=6)
    q = q * 8
    k = k * 4
    k[0, 50:60] = k[0, 50]
    out = la.la_softmax_prefill(q.to(DEV), k.to(DEV), v.to(DEV), cu_of(lens), scale=0.5)
    check_prefill(out, q, k, v, lens, 0.5, tensor_cores(dtype, d))


@pytest.mark.gpu
def test_prefill_descending_and_rising_maximum(la):
    """The running maximum moves at every key, and never after the first."""
    d, n = 128, 700
    for sign in (1.0, -1.0):
        q = torch.zeros(1, n, d, dtype=torch.bfloat16)
        k = torch.zeros(1, n, d, dtype=torch.bfloat16)
        q[..., 0] = 1
        k[0, :, 0] = sign * torch.arange(n) / 8
        v = torch.randn(1, n, d, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16)
        out = la.la_softmax_prefill(q.to(DEV), k.to(DEV), v.to(DEV), cu_of([n]), scale=1.0)
        check_prefill(out, q, k, v, [n], 1.0, True)


@pytest.mark.gpu
def test_prefill_deterministic_and_long(la):
    lens = [5000, 1, 3333]
    q, k, v = (x.to(DEV) for x in prefill_inputs(torch.bfloat16, 128, 4, 2, sum(lens), seed=8))
    a = la.la_softmax_prefill(q, k, v, cu_of(lens))
    for _ in range(3):
        assert torch.equal(a, la.la_softmax_prefill(q, k, v, cu_of(lens)))
    check_prefill(a, q.cpu(), k.cpu(), v.cpu(), lens, 128 ** -0.5, True)


@pytest.mark.gpu
def test_prefill_graph_streams(la):
    """A captured call follows its device inputs; calls on other streams agree."""
    lens = [40, 300, 7]
    q, k, v = (x.to(DEV) for x in prefill_inputs(torch.bfloat16, 64, 4, 2, 400, seed=9))
    cu = cu_of(lens)
    eager = la.la_softmax_prefill(q, k, v, cu, out=torch.zeros_like(q))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    on_s = la.la_softmax_prefill(q, k, v, cu, out=torch.zeros_like(q), stream=s)
    s.synchronize()
    assert torch.equal(eager, on_s)
    out = torch.zeros_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        la.la_softmax_prefill(q, k, v, cu, out=out)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, eager)
    lens2 = [200, 0, 100]
    cu.copy_(cu_of(lens2))
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    check_prefill(out, q.cpu(), k.cpu(), v.cpu(), lens2, 64 ** -0.5, True)


# ------------------------------------------------------------------ the cache
def awkward_rows(d, dtype, seed):
    """Rows whose groups are ordinary, constant, zero, tiny, far from zero, at halves."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(24, d, generator=g)
    x[1] = 0
    x[2] = 3.25
    x[3] = -1e-3
    x[4] *= 1e-6
    x[5] *= 1e4
    x[6] = 100 + x[6] * 0.5
    x[7] = -2000 + x[7]
    x[8] = torch.arange(d) % 16 - 7.5          # codes exactly 0 .. 15
    x[9] = (torch.arange(d) % 32) / 2 - 7.75   # halves between codes
    x[10, 1:] = 0
    x[11] = x[11].abs()
    x[12] = -x[12].abs()
    x[13] *= 2.0 ** -20
    return x.to(dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_append_read(la, dtype, d):
    """Bytes and words as the format says, exactly; values read back exactly
    (one product of an exact sum in fp32: u32 of the value and of the sum)."""
    Hkv, cap = 2, 50
    lens, start = [24, 0, 1, 23], [3, 7, 49, 27]
    N = sum(lens)
    k = torch.stack([awkward_rows(d, dtype, 1), awkward_rows(d, dtype, 2)]).repeat(1, 2, 1)[:, :N]
    v = torch.stack([awkward_rows(d, dtype, 3), awkward_rows(d, dtype, 4)]).repeat(1, 2, 1)[:, :N]
    c = new_cache(la, len(lens), Hkv, cap, d)
    before = [x.cpu().clone() for x in c]
    st = torch.tensor(start, dtype=torch.int32, device=DEV)
    la.la_kv4_append(k.to(DEV), v.to(DEV), c, st, cu_seqlens=cu_of(lens))
    for x, codes, par, b0, w0 in ((k, c.k_codes, c.k_par, before[0], before[1]), (v, c.v_codes, c.v_par, before[2], before[3])):
        b, w = rows_ref(x)
        t = 0
        for s, n in enumerate(lens):
            at = slice(start[s], start[s] + n)
            b0[s, :, at], w0[s, :, at] = b[:, t:t + n], w[:, t:t + n]
            t += n
        assert torch.equal(codes.cpu(), b0) and torch.equal(par.cpu(), w0)
    for od in (torch.float32, torch.bfloat16, torch.float16):
        rk, rv = la.la_kv4_read(c, st, N, cu_seqlens=cu_of(lens), out_dtype=od)
        for got, x in ((rk, k), (rv, v)):
            want = values_ref(x)
            if od == torch.float16:
                keep = want.abs() < 6e4
            else:
                keep = torch.ones_like(want, dtype=torch.bool)
            sc = torch.from_numpy(pack_ref(x)[1]).repeat_interleave(32, -1)
            tol = 2 * U32 * (want.abs() + 16 * sc) + (U[od] * want.abs() * 1.001 if od != torch.float32 else 0) + \
                (2.0 ** -24 if od == torch.float16 else 1e-38)
            assert ((got.double().cpu() - want).abs() <= tol)[keep].all()


@pytest.mark.gpu
def test_append_borders(la):
    """fp32 values next to the border between two codes, where only the definition's 64 bits decide."""
    d, n = 128, 4000
    rng = np.random.default_rng(0)
    x = np.empty((n, d), dtype=np.float32)
    sc = torch.from_numpy(np.exp(rng.normal(size=(n, 4))).astype(np.float32)).to(torch.bfloat16).float().numpy()
    c = rng.integers(0, 15, size=(n, 4, 32)) + 0.5
    x = ((c - 7.3) * sc[..., None]).astype(np.float32)
    x = np.nextafter(x, np.where(rng.random(x.shape) < 0.5, -np.inf, np.inf).astype(np.float32))
    x[..., 0], x[..., 31] = -7.3 * sc, 7.7 * sc
    x = torch.from_numpy(x.reshape(1, n, d))
    cache = new_cache(la, 1, 1, n, d)
    la.la_kv4_append(x.to(DEV), x.to(DEV), cache, torch.zeros(1, dtype=torch.int32, device=DEV), cu_seqlens=cu_of([n]))
    b, w = rows_ref(x)
    assert torch.equal(cache.k_codes.cpu()[0], b) and torch.equal(cache.k_par.cpu()[0], w)


@pytest.mark.gpu
def test_append_nonfinite_strided_and_dropped(la):
    """NaN and infinities turn their own group to NaN only; token-major views;
    one token per sequence; positions outside the cache are dropped."""
    B, Hkv, cap, d = 5, 3, 8, 64
    kv = torch.randn(B, 2 * Hkv, d, generator=torch.Generator().manual_seed(2)).to(torch.float16)
    kv[1, 0, 5], kv[2, 1, 40], kv[3, 4, 0] = math.nan, math.inf, -math.inf
    x = kv.to(DEV).transpose(0, 1)
    cache = new_cache(la, B, Hkv, cap, d)
    start = torch.tensor([0, 7, 3, 8, -1], dtype=torch.int32, device=DEV)
    before = [t.clone() for t in cache]
    la.la_kv4_append(x[:Hkv], x[Hkv:], cache, start)
    for t, t0 in zip(cache, before):
        assert torch.equal(t[3:], t0[3:])
    k, v = la.la_kv4_read(cache, start, B)
    assert (k[:, 3:] == 0).all() and (v[:, 3:] == 0).all()
    clean = kv.clone()
    clean[~torch.isfinite(clean)] = 0
    bad = ~torch.isfinite(kv).view(B, 2 * Hkv, 2, 32).all(-1).repeat_interleave(32, -1)
    got = torch.cat([k, v]).cpu().double().transpose(0, 1)[:3]
    want = values_ref(clean)[:3]
    assert torch.isnan(got[bad[:3]]).all()
    ok = ~bad[:3]
    assert ((got - want).abs()[ok] <= 1e-6 * (1 + want.abs()[ok])).all()


@pytest.mark.gpu
@pytest.mark.parametrize("n_seq", [1, 2, 31, 32, 33, 70])
def test_append_finds_rows(la, n_seq):
    """Each token reaches its own sequence and position, with empty sequences
    among them and behind; what starts outside the cache, and tokens behind the
    last sequence, are dropped; other rows stay."""
    Hkv, cap, d = 2, 9, 32
    lens = [(3 * s + 5) % 7 * (s % 5 != 1) for s in range(n_seq)]
    first = [(5 * s) % 11 - 2 for s in range(n_seq)]
    n = sum(lens)
    x = torch.randn(2 * Hkv, n + 6, d, generator=torch.Generator().manual_seed(n_seq))
    cache = new_cache(la, n_seq, Hkv, cap, d)
    want = [t.cpu().clone() for t in cache]
    la.la_kv4_append(x[:Hkv].to(DEV), x[Hkv:].to(DEV), cache, torch.tensor(first, dtype=torch.int32, device=DEV),
                     cu_seqlens=cu_of(lens))
    rows = [rows_ref(x[:Hkv]), rows_ref(x[Hkv:])]
    t = 0
    for s in range(n_seq):
        for i in range(lens[s]):
            if 0 <= first[s] + i < cap:
                for j, (b, w) in enumerate(rows):
                    want[2 * j][s, :, first[s] + i] = b[:, t]
                    want[2 * j + 1][s, :, first[s] + i] = w[:, t]
            t += 1
    for got, ref in zip(cache, want):
        assert torch.equal(got.cpu(), ref)


@pytest.mark.gpu
def test_read_tokens_of_no_sequence(la):
    c = new_cache(la, 2, 1, 4, 32)
    k, v = la.la_kv4_read(c, torch.zeros(2, dtype=torch.int32, device=DEV), 6, cu_seqlens=cu_of([1, 2]))
    assert (k[:, 3:] == 0).all() and (v[:, 3:] == 0).all()


DECODE = [
    # (dtype, out dtype, d, H, Hkv, cap tokens, lens)
    (torch.float32, None, 32, 2, 1, 40, [0, 1, 40]),
    (torch.float32, None, 64, 8, 2, 300, [300, 17, 128]),
    (torch.float32, None, 128, 3, 3, 1000, [999]),
    (torch.bfloat16, None, 128, 8, 1, 700, [700, 1, 0, 65]),
    (torch.bfloat16, torch.float32, 128, 16, 1, 130, [129, 130]),
    (torch.bfloat16, None, 64, 6, 2, 2500, [2500, 2047, 2049]),
    (torch.bfloat16, None, 32, 40, 1, 77, [77, 15]),
    (torch.float16, None, 64, 16, 16, 257, [256, 257, 33]),
    (torch.float16, torch.float32, 128, 12, 4, 513, [513]),
    (torch.float16, None, 32, 1, 1, 17, [16, 17, 1, 7]),
    (torch.bfloat16, None, 128, 32, 2, 5000, [4999, 31]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,od,d,H,Hkv,T,lens", DECODE)
def test_decode(la, dtype, od, d, H, Hkv, T, lens):
    g = torch.Generator().manual_seed(T + d)
    B = len(lens)
    k = torch.randn(B, Hkv, T, d, generator=g) + 2 * torch.randn(1, Hkv, 1, d, generator=g)
    v = torch.randn(B, Hkv, T, d, generator=g)
    q = torch.randn(B, H, d, generator=g).to(dtype)
    cache, kv, vv = fill_cache(la, k, v)
    vs = torch.from_numpy(pack_ref(v)[1])
    scale = d ** -0.5
    ref, tol, A, w, wtol = ref_decode(q, kv, vv, lens, scale, vs)
    tl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out = la.la_kv4_decode(q.to(DEV), cache, tl, out_dtype=od)
    # fp32 queries carry the weights as two bf16 terms (2^-16 of them may be missing)
    tol = tol + (U[dtype] if dtype != torch.float32 else 2.0 ** -16) * A
    tol = tol + U[out.dtype] * (ref.abs() + tol) + 1e-30
    assert float(((out.double().cpu() - ref).abs() / tol).max()) <= 1.0
    assert (out[[i for i, n in enumerate(lens) if n == 0]] == 0).all()
    # the weights: added to what is there, none behind the lengths, the output the same
    cap = cache.k_codes.shape[2]
    win = torch.rand(B, Hkv, cap, generator=g).to(DEV)
    for acc in (None, win, "in place"):
        wo = win.clone() if acc == "in place" else torch.full_like(win, 5.0)
        out2 = la.la_kv4_decode(q.to(DEV), cache, tl, out_dtype=od, weights_in=wo if acc == "in place" else acc, weights_out=wo)
        assert torch.equal(out, out2)
        was = win.cpu().double() if acc is not None else torch.zeros(B, Hkv, cap, dtype=torch.float64)
        for b, n in enumerate(lens):
            want = was[b, :, :n] + w[b, :, :n]
            assert ((wo[b, :, :n].cpu().double() - want).abs() <= wtol[b, :, :n] + 4 * U32 * want + 1e-30).all()
            assert (wo[b, :, n:] == (win[b, :, n:] if acc == "in place" else 5.0)).all()


@pytest.mark.gpu
def test_decode_peaked_and_flat(la):
    """One key far above the others, far into the cache; then all keys equal."""
    T, d = 3000, 128
    g = torch.Generator().manual_seed(1)
    q = torch.randn(1, 4, d, generator=g).to(torch.bfloat16)
    k, v = 0.1 * torch.randn(1, 1, T, d, generator=g), torch.randn(1, 1, T, d, generator=g)
    k[0, 0, 2777] = q[0].float().mean(0) * 60
    for kk in (k, torch.ones_like(k)):
        cache, kv, vv = fill_cache(la, kk, v)
        ref, tol, A, _, _ = ref_decode(q, kv, vv, [T], d ** -0.5, torch.from_numpy(pack_ref(v)[1]))
        out = la.la_kv4_decode(q.to(DEV), cache, torch.tensor([T], dtype=torch.int32, device=DEV))
        tol = tol + 2.0 ** -8 * A
        tol = tol + 2.0 ** -8 * (ref.abs() + tol)
        assert float(((out.double().cpu() - ref).abs() / tol).max()) <= 1.0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,H", [(torch.bfloat16, 4), (torch.float32, 4), (torch.float16, 12)])
@pytest.mark.parametrize("T", [50, 900])
def test_decode_nan_values_stay_in_their_group(la, dtype, H, T):
    """A value group of NaN reaches its 32 channels of the output and no others."""
    d = 128
    g = torch.Generator().manual_seed(12)
    k, v = torch.randn(2, 1, T, d, generator=g), torch.randn(2, 1, T, d, generator=g)
    q = torch.randn(2, H, d, generator=g).to(dtype).to(DEV)
    cache, _, _ = fill_cache(la, k, v)
    tl = torch.tensor([T, T], dtype=torch.int32, device=DEV)
    clean = la.la_kv4_decode(q, cache, tl)
    cache.v_par[1, 0, T // 2, 2] = 0x7fc0
    got = la.la_kv4_decode(q, cache, tl)
    assert torch.isnan(got[1, :, 64:96]).all()
    same = torch.ones_like(clean, dtype=torch.bool)
    same[1, :, 64:96] = False
    # (the NaN scale may have been the largest of its tile, by which the others' are held)
    assert torch.allclose(got[same].float(), clean[same].float(), rtol=2 * U[dtype], atol=1e-5)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("mag", [1e-30, 1e-6, 1e30])
def test_decode_value_magnitudes(la, dtype, mag):
    """Values far below and above 16-bit products' range, and growing by 2^12 along the cache."""
    T, d = 600, 64
    g = torch.Generator().manual_seed(13)
    k = torch.randn(1, 2, T, d, generator=g)
    v = torch.randn(1, 2, T, d, generator=g) * mag * torch.logspace(0, 12, T, base=2.0)[:, None]
    q = torch.randn(1, 4, d, generator=g).to(dtype)
    cache, kv, vv = fill_cache(la, k, v)
    ref, tol, A, _, _ = ref_decode(q, kv, vv, [T], d ** -0.5, torch.from_numpy(pack_ref(v)[1]))
    out = la.la_kv4_decode(q.to(DEV), cache, torch.tensor([T], dtype=torch.int32, device=DEV), out_dtype=torch.float32)
    tol = tol + (U[torch.float16] if dtype != torch.float32 else 2.0 ** -16) * A
    tol = tol + U32 * (ref.abs() + tol)
    assert float(((out.double().cpu() - ref).abs() / tol).max()) <= 1.0


@pytest.mark.gpu
def test_decode_lengths_are_clamped(la):
    T, d = 100, 64
    g = torch.Generator().manual_seed(11)
    k, v = torch.randn(2, 1, T, d, generator=g), torch.randn(2, 1, T, d, generator=g)
    cache, _, _ = fill_cache(la, k, v)
    cache = la.KV4Cache(*(x[:, :, :T].contiguous() for x in cache))
    q = torch.randn(2, 4, d, generator=g).to(torch.bfloat16).to(DEV)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    assert torch.equal(la.la_kv4_decode(q, cache, i32(10 ** 9, -5)), la.la_kv4_decode(q, cache, i32(T, 0)))


# ------------------------------------------------------------------ eviction
def ref_evict(w, n, keep, recent):
    if n <= keep:
        return list(range(n))
    old = n - recent
    key = [math.inf if math.isnan(x) else x for x in w[:old]]
    isnan = [math.isnan(x) for x in w[:old]]
    order = sorted(range(old), key=lambda i: (not isnan[i], -key[i], i))
    return sorted(order[:keep - recent]) + list(range(old, n))


EVICT = [
    # (d, Hkv, cap, lens, keep, recent)
    (32, 1, 1, [1], 1, 0),
    (32, 2, 40, [0, 1, 39, 40], 8, 3),
    (64, 2, 600, [599, 256, 257, 600], 256, 0),
    (64, 1, 700, [700, 650], 33, 33),
    (128, 3, 5000, [5000, 4097, 12], 1000, 128),
    (128, 1, 20000, [20000], 19999, 5),
    (32, 1, 20000, [19000], 1, 0),
    # slices that do not fit a block's registers: of one CTA, of a cluster
    (32, 2, 9000, [9000, 8500] + [5] * 73, 100, 7),
    (32, 1, 70000, [70000], 30000, 10),
]


@pytest.mark.gpu
@pytest.mark.parametrize("d,Hkv,cap,lens,keep,recent", EVICT)
@pytest.mark.parametrize("kind", ["random", "ties", "odd"])
def test_evict(la, d, Hkv, cap, lens, keep, recent, kind):
    B = len(lens)
    rng = np.random.default_rng(cap + keep)
    c = la.KV4Cache.alloc(B, Hkv, cap, d, DEV)
    for x in c:
        x.view(torch.uint8).copy_(torch.from_numpy(rng.integers(0, 256, size=tuple(x.view(torch.uint8).shape), dtype=np.uint8)))
    if kind == "random":
        w = rng.random((B, Hkv, cap)).astype(np.float32) ** 8
    elif kind == "ties":
        w = rng.integers(0, 3, size=(B, Hkv, cap)).astype(np.float32)
        w[w == 0] = rng.choice([0.0, -0.0], size=int((w == 0).sum()))
    else:
        w = rng.choice(np.array([math.nan, math.inf, -math.inf, 1e-40, -1.5, 2.0, 2.0000002], dtype=np.float32), size=(B, Hkv, cap))
    wd = torch.from_numpy(w).to(DEV)
    out = new_cache(la, B, Hkv, keep + 3, d)
    before = [x.clone() for x in out]
    ow = torch.full((B, Hkv, keep + 3), 9.0, device=DEV)
    kept, ow2, ol = la.la_kv4_evict(c, wd, torch.tensor(lens, dtype=torch.int32, device=DEV), keep, recent=recent, out=out, out_weights=ow)
    assert ow2 is ow and ol.tolist() == [min(n, keep) for n in lens]
    for b in range(B):
        for h in range(Hkv):
            want = ref_evict(w[b, h].tolist(), lens[b], keep, recent)
            m = len(want)
            assert kept[b, h].tolist() == want + [-1] * (keep - m)
            for x, y, y0 in zip(c, out, before):
                assert torch.equal(y[b, h, :m], x[b, h, want]) and torch.equal(y[b, h, m:], y0[b, h, m:])
            assert torch.equal(ow[b, h, :m].cpu().view(torch.int32), torch.from_numpy(w[b, h, want]).view(torch.int32))
            assert (ow[b, h, m:] == 9.0).all()


# ------------------------------------------------------------------ together
@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d,H,Hkv", [(torch.bfloat16, 128, 8, 2), (torch.float16, 64, 4, 4), (torch.float32, 32, 6, 2)])
def test_serving_run(la, dtype, d, H, Hkv):
    """A packed prompt through the attention and into the cache, decode steps
    that append, attend and collect weights (one captured graph, replayed),
    an eviction, and a step over what it left; each against float64."""
    lens, steps, keep, recent = [70, 1, 33], 6, 24, 5
    B, cap = len(lens), 90
    N = sum(lens)
    q, k, v = prefill_inputs(dtype, d, H, Hkv, N, seed=21)
    out = la.la_softmax_prefill(q.to(DEV), k.to(DEV), v.to(DEV), cu_of(lens))
    check_prefill(out, q, k, v, lens, d ** -0.5, tensor_cores(dtype, d))
    cache = new_cache(la, B, Hkv, cap, d, fill=0xFF)
    pos = torch.zeros(B, dtype=torch.int32, device=DEV)
    la.la_kv4_append(k.to(DEV), v.to(DEV), cache, pos, cu_seqlens=cu_of(lens))
    cur = torch.tensor(lens, dtype=torch.int32, device=DEV)
    wts = torch.zeros(B, Hkv, cap, device=DEV)
    rows = [[torch.cat([x[:, a:b] for a, b in [(sum(lens[:s]), sum(lens[:s + 1]))]], 1) for s in range(B)] for x in (k, v)]
    qs, ks, vs = (torch.zeros(B, h, d, dtype=dtype, device=DEV) for h in (H, Hkv, Hkv))
    o = torch.zeros(B, H, d, dtype=dtype, device=DEV)

    def step():
        la.la_kv4_append(ks.transpose(0, 1), vs.transpose(0, 1), cache, cur)
        cur.add_(1)
        la.la_kv4_decode(qs, cache, cur, weights_in=wts, weights_out=wts, out=o)

    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        step()
    gen = torch.Generator().manual_seed(22)
    wref = torch.zeros(B, Hkv, cap, dtype=torch.float64)
    for _ in range(steps):
        nq, nk, nv = (torch.randn(B, h, d, generator=gen).to(dtype) for h in (H, Hkv, Hkv))
        for dst, x in ((qs, nq), (ks, nk), (vs, nv)):
            dst.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        for s in range(B):
            rows[0][s] = torch.cat([rows[0][s], nk[s][:, None]], 1)
            rows[1][s] = torch.cat([rows[1][s], nv[s][:, None]], 1)
            n = rows[0][s].shape[1]
            ref, tol, A, w, _ = ref_decode(nq[s:s + 1], values_ref(rows[0][s])[None], values_ref(rows[1][s])[None], [n],
                                           d ** -0.5, torch.from_numpy(pack_ref(rows[1][s])[1])[None])
            tol = tol + (U[dtype] if dtype != torch.float32 else 2.0 ** -16) * A
            tol = tol + U[dtype] * (ref.abs() + tol)
            assert float(((o[s].double().cpu() - ref[0]).abs() / tol[0]).max()) <= 1.0
            wref[s, :, :n] += w[0]
    assert float((wts.cpu().double() - wref).abs().max()) < 1e-4
    total = float(wts.sum())
    assert abs(total - steps * B * H) < 1e-3 * total
    small, kept, ow, ol = la.la_kv4_evict(cache, wts, cur, keep, recent=recent)
    o2 = la.la_kv4_decode(qs, small, ol)
    w = wts.cpu()
    for s in range(B):
        n = lens[s] + steps
        sel = [ref_evict(w[s, h].tolist(), n, keep, recent) for h in range(Hkv)]
        assert [x for x in kept[s].tolist()] == [x + [-1] * (keep - len(x)) for x in sel]
        kk = torch.stack([values_ref(rows[0][s])[h, sel[h]] for h in range(Hkv)])[None]
        vv = torch.stack([values_ref(rows[1][s])[h, sel[h]] for h in range(Hkv)])[None]
        sc = torch.stack([torch.from_numpy(pack_ref(rows[1][s])[1])[h, sel[h]] for h in range(Hkv)])[None]
        ref, tol, A, _, _ = ref_decode(qs[s:s + 1].cpu(), kk, vv, [len(sel[0])], d ** -0.5, sc)
        tol = tol + (U[dtype] if dtype != torch.float32 else 2.0 ** -16) * A
        tol = tol + U[dtype] * (ref.abs() + tol)
        assert float(((o2[s].double().cpu() - ref[0]).abs() / tol[0]).max()) <= 1.0


@pytest.mark.gpu
@pytest.mark.parametrize("H,Hkv,d,n", [(4, 2, 64, 700), (4, 2, 128, 700), (32, 16, 128, 2500)])
def test_prefill_wait_limit(la, H, Hkv, d, n):
    """With a wait limit of 0 the kernel gives up and says so in the status
    word; the next call, with the limit back, is right."""
    q, k, v = (x.to(DEV) for x in prefill_inputs(torch.bfloat16, d, H, Hkv, n, seed=31))
    cu = cu_of([n])
    ws = torch.empty(la.la_softmax_prefill_workspace_size(H, Hkv, n, d, 1), dtype=torch.uint8, device=DEV)
    want = la.la_softmax_prefill(q, k, v, cu, workspace=ws)
    assert la.la_workspace_status(ws) == (la.LA_OK, 0)
    old = la.la_set_wait_limit_ns(0)
    try:
        la.la_softmax_prefill(q, k, v, cu, workspace=ws)
        status, waiter = la.la_workspace_status(ws)
    finally:
        la.la_set_wait_limit_ns(old)
    assert status == la.LA_ERR_TIMEOUT and waiter > 0
    assert torch.equal(la.la_softmax_prefill(q, k, v, cu, workspace=ws), want)
    assert la.la_workspace_status(ws) == (la.LA_OK, 0)
