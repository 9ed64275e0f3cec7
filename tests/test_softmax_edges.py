"""The softmax operators where single calls went, or could go, wrong: masks and
weights at the ends of the types' ranges, clusters with nothing to choose,
long lists of tiles, empty extents, arguments that alias.

References and bounds are those of test_softmax_ops, whose notation is used:
u = half a step of a type, A = sum_j p_j |v_j|.
"""
import math

import numpy as np
import pytest
import torch

from test_softmax_ops import (DEV, U, U32, check_prefill, cu_of, fill_cache, pack_ref, prefill_inputs, ref_decode,
                              ref_evict, tensor_cores)


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------ prompt attention
@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d,H,Hkv,lo,hi,S", [(torch.float16, 64, 8, 8, 1, 40, 1500), (torch.bfloat16, 128, 16, 4, 1, 300, 400),
                                                   (torch.bfloat16, 128, 8, 4, 257, 700, 150), (torch.float16, 128, 9, 9, 257, 700, 100)])
def test_prefill_long_lists(la, dtype, d, H, Hkv, lo, hi, S):
    """Tens of tiles a CTA, of every small number of blocks (one tile, two heads, two tiles a CTA): no wait gives up,
    every run gives the same bits, and the first and last sequences' rows are right."""
    lens = np.random.default_rng(S).integers(lo, hi + 1, size=S).tolist()
    N = sum(lens)
    q, k, v = prefill_inputs(dtype, d, H, Hkv, N, seed=S)
    ws = torch.empty(la.la_softmax_prefill_workspace_size(H, Hkv, N, d, S), dtype=torch.uint8, device=DEV)
    dev = [x.to(DEV) for x in (q, k, v)]
    runs = []
    for _ in range(5):
        runs.append(la.la_softmax_prefill(*dev, cu_of(lens), workspace=ws))
        assert la.la_workspace_status(ws) == (la.LA_OK, 0)
        assert torch.equal(runs[-1], runs[0])
    for part, at in ((lens[:20], 0), (lens[-20:], N - sum(lens[-20:]))):
        r = slice(at, at + sum(part))
        check_prefill(runs[0][:, r], q[:, r], k[:, r], v[:, r], part, d ** -0.5, True)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d,H", [(torch.float32, 32, 2), (torch.float32, 64, 80), (torch.float32, 128, 2), (torch.bfloat16, 64, 2),
                                       (torch.bfloat16, 128, 2), (torch.float16, 128, 2)])
@pytest.mark.parametrize("first", [1, 64, 130])
def test_prefill_scores_of_minus_infinity(la, dtype, d, H, first):
    """Keys with an infinite channel score -inf.  Rows that see others too are the softmax of those, however many
    keys of -inf come before, between or behind; rows that see no other are 0 / 0."""
    n = first + 300
    q, k, v = prefill_inputs(dtype, d, H, 2, n, seed=first + d)
    q[..., 0] = 1
    kk = k.clone()
    kk[:, :first, 0] = -math.inf
    out = la.la_softmax_prefill(q.to(DEV), kk.to(DEV), v.to(DEV), cu_of([n]))
    assert torch.isnan(out[:, :first]).all()
    check_prefill(out[:1, first:], q[:1, first:], k[:1, first:], v[:1, first:], [n - first], d ** -0.5, tensor_cores(dtype, d))
    # among the others: as if they were not there
    kk, gap = k.clone(), slice(40, 40 + first)
    kk[:, gap, 0] = -math.inf
    out = la.la_softmax_prefill(q.to(DEV), kk.to(DEV), v.to(DEV), cu_of([n]))
    rest = lambda x: torch.cat([x[:, :40], x[:, 40 + first:]], 1)
    check_prefill(rest(out)[:1], rest(q)[:1], rest(k)[:1], rest(v)[:1], [n - first], d ** -0.5, tensor_cores(dtype, d))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d,H,Hkv", [(torch.float16, 64, 1, 1), (torch.float16, 128, 30, 2), (torch.float16, 128, 37, 37),
                                           (torch.bfloat16, 64, 1, 1), (torch.float32, 64, 1, 1)])
@pytest.mark.parametrize("bits", [4, 12, 20, 24])
@pytest.mark.parametrize("at", [0, 400])
def test_prefill_one_key_takes_the_weight(la, dtype, d, H, Hkv, bits, at):
    """A key of value 0 with 2^bits of every other key's weight: what is left of the output is made of the small
    weights alone, each of which keeps its relative precision (down to 2^-25 of the greatest)."""
    n = 3000 if H > 1 else 1500
    g = torch.Generator().manual_seed(bits + d)
    q, k = torch.zeros(H, n, d, dtype=dtype), torch.zeros(Hkv, n, d, dtype=dtype)
    q[..., 0] = 1
    k[..., 0] = (-(bits + torch.rand(Hkv, n, generator=g)) * math.log(2)).to(dtype)
    v = torch.randn(Hkv, n, d, generator=g).to(dtype)
    k[:, at], v[:, at] = 0, 0
    out = la.la_softmax_prefill(q.to(DEV), k.to(DEV), v.to(DEV), cu_of([n]), scale=1.0, out_dtype=torch.float32)
    check_prefill(out[:1], q[:1], k[:1], v[:1], [n], 1.0, tensor_cores(dtype, d))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("H,Hkv", [(3, 1), (16, 4)])
def test_prefill_fp32_tiles(la, d, H, Hkv):
    """Tiles of 16 queries (few heads) and of 64, over sequences that end on, before and behind a tile's end."""
    lens = [64, 0, 1, 200, 63, 65, 16, 17, 15, 129]
    q, k, v = prefill_inputs(torch.float32, d, H, Hkv, sum(lens) + 2, seed=d + H)
    out = torch.full_like(q, 7.0, device=DEV)
    la.la_softmax_prefill(q.to(DEV), k.to(DEV), v.to(DEV), cu_of(lens), out=out)
    assert (out[:, sum(lens):] == 7.0).all()
    check_prefill(out, q, k, v, lens, d ** -0.5, False)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d,H,Hkv,n", [(torch.float32, 64, 6, 2, 333), (torch.float32, 128, 4, 4, 70), (torch.float32, 32, 64, 8, 333),
                                             (torch.float16, 32, 6, 2, 333)])
def test_prefill_views_of_a_projection(la, dtype, d, H, Hkv, n):
    """q, k, v as views of one token-major projection with a gap behind each token, out token-major."""
    lens = [n // 3, n - n // 3]
    g = torch.Generator().manual_seed(n)
    x = torch.randn(n, (H + 2 * Hkv + 1) * d, generator=g).to(dtype).to(DEV)
    heads = x.view(n, H + 2 * Hkv + 1, d).transpose(0, 1)
    q, k, v = heads[:H], heads[H:H + Hkv], heads[H + Hkv:H + 2 * Hkv]
    out = torch.zeros(n, H, d, dtype=dtype, device=DEV)
    la.la_softmax_prefill(q, k, v, cu_of(lens), out=out.transpose(0, 1))
    want = la.la_softmax_prefill(q.contiguous(), k.contiguous(), v.contiguous(), cu_of(lens))
    assert torch.equal(out.transpose(0, 1), want)
    check_prefill(want, q.cpu(), k.cpu(), v.cpu(), lens, d ** -0.5, tensor_cores(dtype, d))


# ------------------------------------------------------------------ reading back
@pytest.mark.gpu
@pytest.mark.parametrize("od,dtype", [(torch.float32, "LA_F32"), (torch.bfloat16, "LA_BF16")])
@pytest.mark.parametrize("B,cap", [(0, 8), (3, 0)])
def test_read_cache_without_rows(la, od, dtype, B, cap):
    """Tokens of no sequence, where there is no sequence at all, and positions outside a cache of none: zeros."""
    Hkv, N, d = 2, 6, 64
    c = la._Kv4CacheC(None, None, None, None, B, Hkv, cap, d)
    cu, start = i32(*range(B + 1)), torch.zeros(max(B, 1), dtype=torch.int32, device=DEV)
    k, v = (torch.full((Hkv, N, d), 7.0, dtype=od, device=DEV) for _ in range(2))
    assert la.lib().la_kv4_read(c, N, cu.data_ptr(), start.data_ptr(), k.data_ptr(), v.data_ptr(), getattr(la, dtype),
                                torch.cuda.current_stream().cuda_stream) == la.LA_OK
    assert (k == 0).all() and (v == 0).all()


# ------------------------------------------------------------------ decode
@pytest.mark.gpu
@pytest.mark.parametrize("dtype,H", [(torch.float16, 4), (torch.bfloat16, 4), (torch.bfloat16, 12), (torch.float32, 4)])
@pytest.mark.parametrize("T", [2, 20, 150])
@pytest.mark.parametrize("bits", [4, 12, 20, 24])
def test_decode_one_position_takes_the_weight(la, dtype, H, T, bits):
    """A position of value 0 with 2^bits of every other one's weight: what is left of the output is made of the
    small weights alone, each of which keeps its relative precision (times its scale, down to 2^-26 of the largest
    scale).

    Bound.  A score is one product (the queries have one channel): a code's exact number and an offset, both up to 31
    scales, in at most 8 roundings of fp32.  A weight's exponential and the sums as in ref_decode, over n positions
    of which each product is at most 31 scales (16 of code, 15 of offset and the constant 8).  The product p scale is
    rounded to 11 bits, or carried as two terms of 22 bits, at worst to half a step of 2^-36 of the largest scale (fp32
    queries); that number then multiplies a value over its scale, at most 16."""
    d = 64
    g = torch.Generator().manual_seed(bits + T)
    q = torch.zeros(1, H, d, dtype=dtype)
    q[..., 0] = 1
    k = torch.zeros(1, 1, T, d)
    k[..., 0] = -(bits + 0.4 * torch.rand(1, 1, T, generator=g)) * math.log(2)
    v = torch.randn(1, 1, T, d, generator=g)
    k[0, 0, T // 2], v[0, 0, T // 2] = 0, 0
    cache, kv, vv = fill_cache(la, k, v)
    out = la.la_kv4_decode(q.to(DEV), cache, i32(T), scale=1.0, out_dtype=torch.float32)
    s = kv[0, 0, :, 0]
    p = torch.softmax(s, 0)
    vs = torch.from_numpy(pack_ref(v)[1])[0, 0].repeat_interleave(32, -1)
    ref, A = p @ vv[0, 0], p @ vv[0, 0].abs()
    ks = float(torch.from_numpy(pack_ref(k)[1]).max())
    rel = 2 * (8 * U32 * 2 * 31 * ks + 4 * U32 * float(s.abs().max())) + 2 * 2.0 ** -20 + 2 * (T + 64) * U32
    tol = rel * A + (T + 64) * U32 * 31 * (p @ vs) + U32 * ref.abs() + 1e-30
    if dtype == torch.float32:
        tol = tol + 2.0 ** -22 * A + T * 2.0 ** -37 * 16 * float(vs.max())
    else:
        tol = tol + U[torch.float16] * A
    err = (out[0].double().cpu() - ref).abs()
    assert float((err / tol).max()) <= 1.0


@pytest.mark.gpu
@pytest.mark.parametrize("H", [4, 40])
@pytest.mark.parametrize("with_weights", [False, True])
def test_decode_cache_without_positions(la, H, with_weights):
    """cap 0: zeros, for more query heads than one block takes too, and nothing is written to the weights."""
    B, d = 2, 64
    c = la._Kv4CacheC(None, None, None, None, B, 1, 0, d)
    q = torch.ones(B, H, d, dtype=torch.bfloat16, device=DEV)
    out, w, lens = torch.full_like(q, 3.0), torch.full((4,), 5.0, device=DEV), i32(0, 7)
    ws = torch.empty(max(la.la_kv4_decode_workspace_size(B, H, 1, 0, d, with_weights), 256), dtype=torch.uint8, device=DEV)
    status = la.lib().la_kv4_decode(q.data_ptr(), la.LA_BF16, H, c, lens.data_ptr(), 0.1, None,
                                    w.data_ptr() if with_weights else None, out.data_ptr(), la.LA_BF16, ws.data_ptr(),
                                    ws.nbytes, torch.cuda.current_stream().cuda_stream)
    assert status == la.LA_OK
    assert (out == 0).all() and (w == 5.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("H", [1, 4, 12])
@pytest.mark.parametrize("T", [2, 32])
def test_decode_rounding_of_the_weights(la, dtype, d, H, T):
    """The weights times scales are rounded to fp16's 11 bits whatever the 16-bit type of the queries, or carried as
    two such terms (fp32 queries; one value row of the T is not 0 then, so that no sum covers the rounding).

    Bound.  As in test_decode_one_position_takes_the_weight, with no weight below 2^-3 of another's.  A sum of r rows
    in one tile takes at most r products, r offsets and 8 more roundings, each of a number below 31 scales."""
    g = torch.Generator().manual_seed(T + d + H)
    q = torch.zeros(1, H, d, dtype=dtype)
    q[0, :, 0] = 1 + torch.arange(H) / 32
    k = torch.zeros(1, 1, T, d)
    k[..., 0] = 2 * torch.rand(1, 1, T, generator=g) - 1
    v = torch.randn(1, 1, T, d, generator=g)
    rows = T
    if dtype == torch.float32:
        v[:, :, 1:], rows = 0, 1
    cache, kv, vv = fill_cache(la, k, v)
    out = la.la_kv4_decode(q.to(DEV), cache, i32(T), scale=1.0, out_dtype=torch.float32)[0].double().cpu()
    vs = torch.from_numpy(pack_ref(v)[1])[0, 0].repeat_interleave(32, -1)
    ks = float(torch.from_numpy(pack_ref(k)[1]).max())
    for h in range(H):
        s = kv[0, 0, :, 0] * q[0, h, 0].double()
        p = torch.softmax(s, 0)
        ref, A = p @ vv[0, 0], p @ vv[0, 0].abs()
        rel = 2 * (8 * U32 * 2 * 31 * ks + 4 * U32 * float(s.abs().max())) + 2 * 2.0 ** -20 + 2 * (T + 8) * U32
        tol = rel * A + (2 * rows + 8) * U32 * 31 * (p @ vs) + U32 * ref.abs() + 1e-30
        tol = tol + (2.0 ** -22 if dtype == torch.float32 else U[torch.float16]) * A
        assert float(((out[h] - ref).abs() / tol).max()) <= 1.0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("power", [-99, 99])
def test_decode_ranges_of_keys_and_queries(la, dtype, power):
    """Keys of 2^99 under queries of 2^-99, and the other way round: ordinary scores."""
    T, d = 300, 128
    g = torch.Generator().manual_seed(19)
    k, v = torch.randn(1, 1, T, d, generator=g), torch.randn(1, 1, T, d, generator=g)
    q = torch.randn(1, 4, d, generator=g).to(dtype)
    cache, kv, vv = fill_cache(la, k * 2.0 ** power, v)
    ref, tol, A, _, _ = ref_decode(q.double() * 2.0 ** -power, kv, vv, [T], d ** -0.5, torch.from_numpy(pack_ref(v)[1]))
    out = la.la_kv4_decode((q * 2.0 ** -power).to(DEV), cache, i32(T), out_dtype=torch.float32)
    tol = tol + (U[torch.float16] if dtype != torch.float32 else 2.0 ** -22) * A + U32 * ref.abs()
    assert float(((out.double().cpu() - ref).abs() / tol).max()) <= 1.0


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1019, 1020])
def test_decode_on_both_sides_of_whole_rows(la, T):
    """Caches of 1024 and 1025 positions (whole rows and the cut line): right, and within rounding of each other."""
    lens = [T, 700, 1]
    g = torch.Generator().manual_seed(17)
    k, v = (torch.randn(3, 2, 1020, 64, generator=g)[:, :, :T] for _ in range(2))
    q = torch.randn(3, 6, 64, generator=g).to(torch.bfloat16)
    cache, kv, vv = fill_cache(la, k, v)
    assert cache.k_codes.shape[2] == T + 5
    wo = torch.zeros(3, 2, T + 5, device=DEV)
    out = la.la_kv4_decode(q.to(DEV), cache, i32(*lens), weights_out=wo, out_dtype=torch.float32)
    ref, tol, A, w, wtol = ref_decode(q, kv, vv, lens, 0.125, torch.from_numpy(pack_ref(v)[1]))
    tol = tol + U[torch.float16] * A + U32 * ref.abs() + 1e-30
    assert float(((out.double().cpu() - ref).abs() / tol).max()) <= 1.0
    assert ((wo.cpu().double()[:, :, :T] - w).abs() <= wtol + 4 * U32 * w + 1e-30).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d,H,Hkv", [(torch.bfloat16, 64, 4, 1), (torch.float16, 32, 20, 1), (torch.float32, 32, 4, 2),
                                           (torch.bfloat16, 128, 2, 2)])
def test_decode_lengths_of_every_size(la, dtype, d, H, Hkv):
    """Forty sequences from none to thousands of positions in one cut line: each as if it were alone, the weights too,
    and every run with the same bits."""
    T, B = 3000, 40
    rng = np.random.default_rng(d)
    lens = [0, 1, 2, 31, 32, 33, 0, T, T - 1, 2049] + [int(x) for x in np.exp(rng.uniform(0, math.log(T), B - 10))]
    rng.shuffle(lens)
    g = torch.Generator().manual_seed(d)
    k, v = torch.randn(B, Hkv, T, d, generator=g), torch.randn(B, Hkv, T, d, generator=g)
    q = torch.randn(B, H, d, generator=g).to(dtype)
    cache, kv, vv = fill_cache(la, k, v)
    ref, tol, A, w, wtol = ref_decode(q, kv, vv, lens, d ** -0.5, torch.from_numpy(pack_ref(v)[1]))
    tol = tol + (U[torch.float16] if dtype != torch.float32 else 2.0 ** -22) * A
    tol = tol + U[dtype] * (ref.abs() + tol) + 1e-30
    cap = cache.k_codes.shape[2]
    runs = []
    for _ in range(3):
        wo = torch.full((B, Hkv, cap), 5.0, device=DEV)
        runs.append((la.la_kv4_decode(q.to(DEV), cache, i32(*lens), weights_out=wo), wo))
        assert torch.equal(runs[-1][0], runs[0][0]) and torch.equal(wo, runs[0][1])
    assert torch.equal(la.la_kv4_decode(q.to(DEV), cache, i32(*lens)), runs[0][0])
    assert float(((runs[0][0].double().cpu() - ref).abs() / tol).max()) <= 1.0
    for b, n in enumerate(lens):
        assert ((runs[0][1][b, :, :n].cpu().double() - w[b, :, :n]).abs() <= wtol[b, :, :n] + 4 * U32 * w[b, :, :n] + 1e-30).all()
        assert (runs[0][1][b, :, n:] == 5.0).all()


# ------------------------------------------------------------------ eviction
@pytest.mark.gpu
@pytest.mark.parametrize("d,Hkv,cap,lens,keep,recent", [
    # clusters (caches beyond 8192 positions, few rows) whose rows have nothing to choose: within the budget, empty,
    # or with the newest positions alone
    (64, 1, 20000, [20000, 50, 0], 100, 100),
    (32, 2, 20000, [50, 20000, 0], 1000, 0),
    (128, 1, 9000, [9000, 9000], 9000, 0),
    (32, 1, 70000, [70000, 3], 500, 500),
    (32, 1, 70000, [400, 0, 500, 70000], 500, 250),
    # more rows than SMs: one small block each, to its last key
    (32, 2, 2048, [2048, 2047, 0, 900] + [1300] * 76, 1000, 11),
])
def test_evict_clusters_with_nothing_to_choose(la, d, Hkv, cap, lens, keep, recent):
    B = len(lens)
    rng = np.random.default_rng(cap + keep)
    c = la.KV4Cache.alloc(B, Hkv, cap, d, DEV)
    for x in c:
        x.view(torch.uint8).copy_(torch.from_numpy(rng.integers(0, 256, size=tuple(x.view(torch.uint8).shape), dtype=np.uint8)))
    w = rng.random((B, Hkv, cap)).astype(np.float32)
    wd, ld = torch.from_numpy(w).to(DEV), i32(*lens)
    for _ in range(20):
        out, kept, ow, ol = la.la_kv4_evict(c, wd, ld, keep, recent=recent)
        assert ol.tolist() == [min(n, keep) for n in lens]
        for b in range(B):
            for h in range(Hkv):
                want = ref_evict(w[b, h].tolist(), lens[b], keep, recent)
                m = len(want)
                assert kept[b, h].tolist() == want + [-1] * (keep - m)
                assert ow[b, h, :m].tolist() == w[b, h, want].tolist() and (ow[b, h, m:] == 0).all()
                for x, y in zip(c, out):
                    assert torch.equal(y[b, h, :m], x[b, h, want])


@pytest.mark.gpu
@pytest.mark.parametrize("cap,lens,keep,recent", [(300, [300, 7, 0], 64, 10), (20000, [20000, 9000], 4000, 100)])
def test_evict_without_optional_outputs(la, cap, lens, keep, recent):
    """The rows are the same whichever of the other outputs are asked for (without `kept` the workspace holds the list)."""
    B, Hkv, d = len(lens), 2, 64
    rng = np.random.default_rng(cap)
    c = la.KV4Cache.alloc(B, Hkv, cap, d, DEV)
    for x in c:
        x.view(torch.uint8).copy_(torch.from_numpy(rng.integers(0, 256, size=tuple(x.view(torch.uint8).shape), dtype=np.uint8)))
    w = torch.from_numpy(rng.random((B, Hkv, cap)).astype(np.float32)).to(DEV)
    want, kept, ow, ol = la.la_kv4_evict(c, w, i32(*lens), keep, recent=recent)
    ws = torch.empty(la.la_kv4_evict_workspace_size(B, Hkv, cap, keep), dtype=torch.uint8, device=DEV)
    for asked in range(8):
        out = la.KV4Cache.alloc(B, Hkv, keep, d, DEV)
        got = [torch.empty_like(kept), torch.zeros_like(ow), torch.empty_like(ol)]
        at = [x.data_ptr() if asked >> i & 1 else None for i, x in enumerate(got)]
        lens_d = i32(*lens)
        assert la.lib().la_kv4_evict(la._cache_c(c)[0], w.data_ptr(), lens_d.data_ptr(), keep, recent, la._cache_c(out)[0], at[1], at[0],
                                     at[2], ws.data_ptr(), ws.nbytes, torch.cuda.current_stream().cuda_stream) == la.LA_OK
        for b in range(B):
            m = min(lens[b], keep)
            for x, y in zip(out, want):
                assert torch.equal(x[b, :, :m], y[b, :, :m])
        for i, y in enumerate((kept, ow, ol)):
            if asked >> i & 1:
                assert torch.equal(got[i], y)


# ------------------------------------------------------------------ together
@pytest.mark.gpu
def test_calls_at_once(la):
    """Prompts of both kinds of CTA, a decode and an eviction on streams of their own, with workspaces of their own, and
    the same calls replayed from one captured graph after their inputs changed: the bits of the calls one by one."""
    lens = [700, 1300, 64, 257]
    a = [x.to(DEV) for x in prefill_inputs(torch.float16, 64, 8, 8, sum(lens), seed=41)]
    b = [x.to(DEV) for x in prefill_inputs(torch.bfloat16, 128, 32, 16, sum(lens), seed=42)]
    cu = cu_of(lens)
    g = torch.Generator().manual_seed(43)
    k, v = torch.randn(4, 2, 1500, 64, generator=g), torch.randn(4, 2, 1500, 64, generator=g)
    cache, _, _ = fill_cache(la, k, v)
    cap = cache.k_codes.shape[2]
    q = torch.randn(4, 8, 64, generator=g).to(torch.bfloat16).to(DEV)
    tl, w = i32(1500, 3, 0, 900), torch.rand(4, 2, cap, generator=g).to(DEV)
    need = [la.la_softmax_prefill_workspace_size(8, 8, sum(lens), 64, 4), la.la_softmax_prefill_workspace_size(32, 16, sum(lens), 128, 4),
            la.la_kv4_decode_workspace_size(4, 8, 2, cap, 64, True)]
    ws = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in need]
    out = [torch.zeros_like(a[0]), torch.zeros_like(b[0]), torch.zeros_like(q), torch.zeros_like(w)]
    small = la.KV4Cache.alloc(4, 2, 300, 64, DEV)
    ow = torch.zeros(4, 2, 300, device=DEV)
    calls = [lambda: la.la_softmax_prefill(*a, cu, out=out[0], workspace=ws[0]),
             lambda: la.la_softmax_prefill(*b, cu, out=out[1], workspace=ws[1]),
             lambda: la.la_kv4_decode(q, cache, tl, weights_in=w, weights_out=out[3], out=out[2], workspace=ws[2]),
             lambda: la.la_kv4_evict(cache, w, tl, 300, recent=20, out=small, out_weights=ow)]

    def results():
        torch.cuda.synchronize()
        x = [t.clone() for t in (*out, ow)] + [small.k_codes[0].clone(), small.v_par[0].clone()]
        for t in (*out, ow):
            t.zero_()
        return x

    def same(x, y):
        return all(torch.equal(s, t) for s, t in zip(x, y))
    for call in calls:
        call()
    want = results()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(10):
        torch.cuda.synchronize()
        for call, s in zip(calls, streams):
            with torch.cuda.stream(s):
                call()
        assert same(results(), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for call in calls:
            call()
    graph.replay()
    assert same(results(), want)
    cu.copy_(cu_of([1, 0, 1500, 600]))
    tl.copy_(i32(0, 1400, 299, 301))
    q.mul_(-1)
    graph.replay()
    got = results()
    for call in calls:
        call()
    again = results()
    assert same(got, again) and not same(got, want)
    for x in ws[:2]:
        assert la.la_workspace_status(x) == (la.LA_OK, 0)
