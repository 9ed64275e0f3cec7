"""What is measured of the softmax-attention operators that serve the
full-attention layers of a hybrid stack: attention over a packed prompt, the
4-bit key/value cache (append, read back, decode) and its eviction.

Every case can run two ways on the same inputs: in plain torch operations
(``own`` false) and through the package's entry points (``own`` true).

The cache format is part of the inputs.  For each sequence, kv head, position:
d 4-bit codes and, for each group of 32 channels, a bf16 scale and an fp16
offset in one 32-bit word (scale in the low half); a value is
scale * (code + offset).  Codes are stored as 8 chunks per row; chunk r holds,
for each group g, 16 bits with channels 32 g + 4 r + {0, 1, 2, 3}, the lowest
channel in the lowest bits.
"""
import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_ES = {"f32": 4, "bf16": 2, "f16": 2}
_GROUP = 32


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a few short prompts arrive together, fp32: what a call costs at the least
        {"name": "prefill_short_f32_d64", "op": "prefill", "dtype": "f32", "d": 64, "H": 8, "Hkv": 2,
         "S": 4, "lo": 1, "hi": 64, "tail": 3},
        # ordinary serving batch, prompts of a few hundred tokens, half precision, no shared heads
        {"name": "prefill_packed_f16_d64", "op": "prefill", "dtype": "f16", "d": 64, "H": 16, "Hkv": 16,
         "S": 32, "lo": 1, "hi": 700, "tail": 0},
        # a batch of prompts of thousands of tokens with odd lengths, grouped heads, buffer longer than the batch
        {"name": "prefill_packed_bf16_d128", "op": "prefill", "dtype": "bf16", "d": 128, "H": 16, "Hkv": 4,
         "S": 8, "lo": 257, "hi": 4111, "tail": 129},
        # one long document
        {"name": "prefill_long_bf16_d128", "op": "prefill", "dtype": "bf16", "d": 128, "H": 16, "Hkv": 2,
         "S": 1, "lo": 16384, "hi": 16384, "tail": 0},
        # one decode step's keys and values for 64 sequences
        {"name": "append_step_f16_d64", "op": "append", "dtype": "f16", "d": 64, "Hkv": 4, "S": 64, "lo": 1, "hi": 1,
         "cap": 4096},
        # the keys and values of a packed prompt, appended behind what the sequences hold
        {"name": "append_prompt_bf16_d128", "op": "append", "dtype": "bf16", "d": 128, "Hkv": 8, "S": 12, "lo": 3,
         "hi": 1531, "cap": 4096},
        # one user, a short context
        {"name": "decode_one_f32_d64", "op": "decode", "dtype": "f32", "d": 64, "B": 1, "H": 8, "Hkv": 2, "cap": 256,
         "lo": 37, "hi": 37, "weights": True},
        # a batch of mid-size contexts, half precision, heads not shared
        {"name": "decode_batch_f16_d64", "op": "decode", "dtype": "f16", "d": 64, "B": 16, "H": 16, "Hkv": 16,
         "cap": 2048, "lo": 0, "hi": 2048, "weights": False},
        # the repository's decode batch (64 sequences, 16 heads of 128) with ragged contexts up to 8192
        {"name": "decode_batch_bf16_d128", "op": "decode", "dtype": "bf16", "d": 128, "B": 64, "H": 16, "Hkv": 4,
         "cap": 8192, "lo": 1, "hi": 8192, "weights": False},
        # one long document of the repository's long-context length, collecting the weights that eviction goes by
        {"name": "decode_long_bf16_d128", "op": "decode", "dtype": "bf16", "d": 128, "B": 1, "H": 32, "Hkv": 8,
         "cap": 131072, "lo": 131072, "hi": 131072, "weights": True},
        # one sequence steps over its budget
        {"name": "evict_one_d64", "op": "evict", "d": 64, "B": 1, "Hkv": 2, "cap": 320, "lo": 301, "hi": 301,
         "keep": 256, "recent": 32},
        # a batch's prompts cut down to a quarter
        {"name": "evict_batch_d128", "op": "evict", "d": 128, "B": 16, "Hkv": 8, "cap": 8192, "lo": 1500, "hi": 8192,
         "keep": 2048, "recent": 256},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "append", "decode", "evict"])
    d = rng.choice([32, 64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 8])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "prefill":
        hi = _log_int(rng, 1, 2048 if dtype == "f32" else 8192)
        lo = max(1, int(hi * rng.random()))
        S = max(1, min(_log_int(rng, 1, 64), 12000 // hi))
        while Hkv * G > 16:
            G = max(1, G // 2)
        return {"op": op, "dtype": dtype, "d": d, "H": Hkv * G, "Hkv": Hkv, "S": S, "lo": lo,
                "hi": hi, "tail": rng.choice([0, 0, 1, 77])}
    if op == "append":
        hi = _log_int(rng, 1, 4000)
        lo = max(1, int(hi * rng.random()))
        S = max(1, min(_log_int(rng, 1, 256), 16000 // hi))
        return {"op": op, "dtype": dtype, "d": d, "Hkv": Hkv, "S": S, "lo": lo, "hi": hi,
                "cap": hi + _log_int(rng, 1, 4000)}
    cap = _log_int(rng, 1, 131072)
    most = 64 * 4 * 8192 // (Hkv * cap)
    B = max(1, min(_log_int(rng, 1, 128), most))
    lo = int(cap * rng.random())
    if op == "decode":
        return {"op": op, "dtype": dtype, "d": d, "B": B, "H": Hkv * G, "Hkv": Hkv, "cap": cap, "lo": lo, "hi": cap,
                "weights": rng.random() < 0.3}
    B = max(1, min(B, 16 * 8 * 8192 // (Hkv * cap)))
    keep = max(1, int(cap * rng.uniform(0.05, 0.7)))
    return {"op": op, "d": d, "B": B, "Hkv": Hkv, "cap": cap, "lo": lo, "hi": cap, "keep": keep,
            "recent": int(keep * rng.choice([0.0, 0.1, 0.5, 1.0]))}


# ------------------------------------------------------------------ inputs
def _lengths(rng, n, lo, hi):
    return [int(x) for x in rng.integers(lo, hi + 1, size=n)]


def _prompt_lengths(case):
    # a case's prompts add up to the same tokens for every seed
    return _lengths(np.random.default_rng([case["S"], case["lo"], case["hi"]]), case["S"], case["lo"], case["hi"])


def _keys(shape_h, shape_t, d, dtype, gen):
    # keys with a mean per head and channel, a few channels far out, as projections have
    x = torch.randn((shape_h, shape_t, d), generator=gen, device="cuda")
    mean = torch.randn((shape_h, 1, d), generator=gen, device="cuda")
    far = torch.rand((shape_h, 1, d), generator=gen, device="cuda") < 0.03
    return (x + mean * torch.where(far, 4.0, 0.3)).to(dtype)


def _pack(codes, scale, off):
    """codes [..., d] (0..15), scale, off [..., d/32] -> (bytes [..., d/2] uint8, words [..., d/32] int32)."""
    d = codes.shape[-1]
    g = d // _GROUP
    c = codes.to(torch.int32).reshape(*codes.shape[:-1], g, 8, 4)
    f = c[..., 0] | (c[..., 1] << 4) | (c[..., 2] << 8) | (c[..., 3] << 12)    # [..., g, 8]
    f = f.transpose(-1, -2)                                                    # chunk r, group g
    b = torch.stack([f & 255, f >> 8], -1).to(torch.uint8)
    s = scale.to(torch.bfloat16).view(torch.int16).to(torch.int32) & 0xFFFF
    o = off.to(torch.float16).view(torch.int16).to(torch.int32)
    return b.reshape(*codes.shape[:-1], d // 2).contiguous(), ((o << 16) | s).contiguous()


def _unpack(b, w, dtype):
    """The values of packed rows, in ``dtype``."""
    d = b.shape[-1] * 2
    g = d // _GROUP
    x = b.reshape(*b.shape[:-1], 8, g, 2)
    n = torch.stack([x[..., 0] & 15, x[..., 0] >> 4, x[..., 1] & 15, x[..., 1] >> 4], -1)   # [..., 8, g, 4]
    n = n.transpose(-2, -3).reshape(*b.shape[:-1], g, _GROUP).to(dtype)
    scale = (w << 16).view(torch.float32).to(dtype)
    off = (w >> 16).to(torch.int16).view(torch.float16).to(dtype)
    return (scale[..., None] * (n + off[..., None])).reshape(*b.shape[:-1], d)


def _random_cache(B, Hkv, cap, d, gen):
    def half(bias):
        b = torch.randint(0, 256, (B, Hkv, cap, d // 2), generator=gen, device="cuda", dtype=torch.uint8)
        sc = 0.12 + 0.2 * torch.rand((B, Hkv, cap, d // _GROUP), generator=gen, device="cuda")
        of = -7.5 + bias * torch.randn((B, Hkv, cap, d // _GROUP), generator=gen, device="cuda")
        s = sc.to(torch.bfloat16).view(torch.int16).to(torch.int32) & 0xFFFF
        o = of.to(torch.float16).view(torch.int16).to(torch.int32)
        return b, (o << 16) | s
    kc, kp = half(1.5)
    vc, vp = half(0.5)
    return kc, kp, vc, vp


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = {"case": case}
    d = case["d"]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    if case["op"] in ("prefill", "append"):
        lens = [int(x) for x in rng.permutation(_prompt_lengths(case))]
        cu = np.concatenate([[0], np.cumsum(lens)])
        N = int(cu[-1]) + case.get("tail", 0)
        dt = _DT[case["dtype"]]
        st |= {"cu": i32(cu.tolist()), "lens": lens, "N": N, "max_len": max(lens)}
        st["k"] = _keys(case["Hkv"], N, d, dt, gen)
        st["v"] = torch.randn((case["Hkv"], N, d), generator=gen, device="cuda").to(dt)
        if case["op"] == "prefill":
            st["q"] = torch.randn((case["H"], N, d), generator=gen, device="cuda").to(dt)
            st["out"] = torch.zeros((case["H"], N, d), dtype=dt, device="cuda")
        else:
            st["start"] = i32([int(rng.integers(0, case["cap"] - n + 1)) for n in lens])
            shape = (case["S"], case["Hkv"], case["cap"])
            st["cache"] = [torch.zeros((*shape, d // 2), dtype=torch.uint8, device="cuda"),
                           torch.zeros((*shape, d // _GROUP), dtype=torch.int32, device="cuda"),
                           torch.zeros((*shape, d // 2), dtype=torch.uint8, device="cuda"),
                           torch.zeros((*shape, d // _GROUP), dtype=torch.int32, device="cuda")]
        return st
    B, Hkv, cap = case["B"], case["Hkv"], case["cap"]
    st["lens"] = i32(_lengths(rng, B, case["lo"], case["hi"]))
    st["cache"] = list(_random_cache(B, Hkv, cap, d, gen))
    # accumulated weights: heavy tailed, with positions that tie
    w = torch.rand((B, Hkv, cap), generator=gen, device="cuda") ** 6
    st["weights"] = torch.where(w < 1e-4, torch.zeros_like(w), w)
    if case["op"] == "decode":
        st["q"] = torch.randn((B, case["H"], d), generator=gen, device="cuda").to(_DT[case["dtype"]])
        st["weights_out"] = torch.zeros_like(st["weights"])
    else:
        keep = case["keep"]
        st["out"] = [torch.zeros((B, Hkv, keep, d // 2), dtype=torch.uint8, device="cuda"),
                     torch.zeros((B, Hkv, keep, d // _GROUP), dtype=torch.int32, device="cuda"),
                     torch.zeros((B, Hkv, keep, d // 2), dtype=torch.uint8, device="cuda"),
                     torch.zeros((B, Hkv, keep, d // _GROUP), dtype=torch.int32, device="cuda")]
        st["out_weights"] = torch.zeros((B, Hkv, keep), device="cuda")
        st["all_cu"] = torch.arange(0, (B + 1) * keep, keep, dtype=torch.int32, device="cuda")
        st["zero"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    return _RUN[st["case"]["op"]](st)


def _prefill(st):
    if own:
        import kernelized_causal_sequence_b200 as la
        return la.la_softmax_prefill(st["q"], st["k"], st["v"], st["cu"], out=st["out"])
    q, k, v, cu, L = st["q"], st["k"], st["v"], st["cu"].long(), st["max_len"]
    H, N, d = q.shape
    Hkv, S = k.shape[0], cu.numel() - 1
    dev = q.device
    pos = torch.arange(L, device=dev)
    lens = cu[1:] - cu[:-1]
    idx = (cu[:-1, None] + pos).clamp(max=N - 1)                       # [S, L]
    qp = q.float()[:, idx].reshape(Hkv, H // Hkv, S, L, d)
    kp = k.float()[:, idx][:, None]
    vp = v.float()[:, idx][:, None]
    hide = (pos[None, :] > pos[:, None]) | (pos >= lens[:, None])[:, None, :]      # [S, L, L]
    s = torch.matmul(qp * d ** -0.5, kp.transpose(-1, -2))
    s.masked_fill_(hide, -math.inf)
    s.sub_(s.amax(-1, keepdim=True)).exp_()
    o = (torch.matmul(s, vp) / s.sum(-1, keepdim=True)).reshape(H, S, L, d)
    t = torch.arange(N, device=dev)
    seq = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=S - 1)
    at = (t - cu[seq]).clamp(max=L - 1)
    return torch.where((t < cu[-1])[None, :, None], o[:, seq, at], 0.0).to(q.dtype)


def _quantise(x):
    """Codes, scale and offset of rows x [..., d]: the definition, in 64 bits up to each rounding."""
    g = x.double().reshape(*x.shape[:-1], -1, _GROUP)
    lo, hi = g.amin(-1), g.amax(-1)
    sc = torch.maximum((hi - lo) / 15, g.abs().amax(-1) / 1024).to(torch.bfloat16)
    s64 = sc.double()
    of = torch.where(s64 > 0, lo / s64, 0.0).to(torch.float16)
    c = torch.where(s64[..., None] > 0, torch.round(g / s64[..., None] - of.double()[..., None]).clamp(0, 15), 0.0)
    return c.reshape(x.shape), sc, of


def _append(st):
    c = st["cache"]
    cu = None if st["N"] == len(st["lens"]) else st["cu"]
    if own:
        import kernelized_causal_sequence_b200 as la
        cache = la.KV4Cache(*c)
        la.la_kv4_append(st["k"], st["v"], cache, st["start"], cu_seqlens=cu)
        return la.la_kv4_read(cache, st["start"], st["N"], cu_seqlens=cu, out_dtype=torch.float32)
    cu, N = st["cu"].long(), st["N"]
    t = torch.arange(N, device=c[0].device)
    seq = torch.searchsorted(cu, t, right=True) - 1
    at = st["start"].long()[seq] + t - cu[seq]
    for x, b, w in ((st["k"], c[0], c[1]), (st["v"], c[2], c[3])):
        rows, words = _pack(*_quantise(x))
        b[seq, :, at] = rows.transpose(0, 1)
        w[seq, :, at] = words.transpose(0, 1)
    return tuple(_unpack(b[seq, :, at], w[seq, :, at], torch.float32).transpose(0, 1) for b, w in ((c[0], c[1]), (c[2], c[3])))


def _decode(st):
    c, case = st["cache"], st["case"]
    if own:
        import kernelized_causal_sequence_b200 as la
        if case["weights"]:
            o = la.la_kv4_decode(st["q"], la.KV4Cache(*c), st["lens"], weights_in=st["weights"], weights_out=st["weights_out"])
            return o, st["weights_out"]
        return la.la_kv4_decode(st["q"], la.KV4Cache(*c), st["lens"])
    q, lens = st["q"], st["lens"].long()
    B, H, d = q.shape
    Hkv, cap = c[0].shape[1], c[0].shape[2]
    k, v = _unpack(c[0], c[1], torch.float32), _unpack(c[2], c[3], torch.float32)
    hide = (torch.arange(cap, device=q.device) >= lens[:, None])[:, None, None, :]
    s = torch.matmul(q.float().reshape(B, Hkv, H // Hkv, d) * d ** -0.5, k.transpose(-1, -2)).masked_fill_(hide, -math.inf)
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(m > -math.inf, m, 0.0))
    p = e / e.sum(-1, keepdim=True).clamp(min=1e-30)
    o = torch.matmul(p, v).reshape(B, H, d).to(q.dtype)
    if not case["weights"]:
        return o
    return o, torch.where(hide[:, 0], 0.0, st["weights"] + p.sum(2))


def _evict(st):
    c, case = st["cache"], st["case"]
    keep, recent = case["keep"], case["recent"]
    if own:
        import kernelized_causal_sequence_b200 as la
        dst = la.KV4Cache(*st["out"])
        kept, w, n = la.la_kv4_evict(la.KV4Cache(*c), st["weights"], st["lens"], keep, recent=recent, out=dst,
                                     out_weights=st["out_weights"])
        k, v = la.la_kv4_read(dst, st["zero"], keep * case["B"], cu_seqlens=st["all_cu"], out_dtype=torch.float32)
        return kept, w, n, k, v
    B, Hkv, cap = st["weights"].shape
    n = st["lens"].long()
    pos = torch.arange(cap, device=n.device)
    newest = pos >= (n - recent)[:, None]
    rank = st["weights"].masked_fill(newest[:, None], math.inf).masked_fill((pos >= n[:, None])[:, None], -1.0)
    first = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :keep]
    have = torch.arange(keep, device=n.device) < n.clamp(max=keep)[:, None, None]
    kept = torch.sort(torch.where(have, first, cap), dim=-1).values          # [B, Hkv, keep], ascending
    at = kept.clamp(max=cap - 1)
    w = torch.where(have, st["weights"].gather(2, at), 0.0)
    rows = lambda b: torch.where(have[..., None], b.gather(2, at[..., None].expand(-1, -1, -1, b.shape[-1])), 0)
    kv = [_unpack(rows(b), rows(x), torch.float32).transpose(0, 1).reshape(Hkv, B * keep, case["d"])
          for b, x in ((c[0], c[1]), (c[2], c[3]))]
    return torch.where(have, kept, -1).int(), w, n.clamp(max=keep).int(), kv[0], kv[1]


_RUN = {"prefill": _prefill, "append": _append, "decode": _decode, "evict": _evict}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    d = case["d"]
    mean = (case["lo"] + case["hi"]) / 2
    row = 2 * (d // 2 + d // 8)                 # a position's keys and values in the cache, one head
    if case["op"] == "prefill":
        lens = _prompt_lengths(case)
        return {"bytes": _ES[case["dtype"]] * (2 * case["H"] + 2 * case["Hkv"]) * sum(lens) * d,
                "flops": 2 * d * case["H"] * sum(n * (n + 1) for n in lens)}
    if case["op"] == "append":
        n = sum(_prompt_lengths(case)) * case["Hkv"]
        # the inputs, the rows written and read back, their values
        return {"bytes": n * (2 * _ES[case["dtype"]] * d + 2 * row + 8 * d), "flops": n * 12 * d}
    n = case["B"] * case["Hkv"] * mean
    if case["op"] == "decode":
        q = case["B"] * case["H"] * d * _ES[case["dtype"]]
        return {"bytes": n * (row + (8 if case["weights"] else 0)) + 2 * q, "flops": 4 * n * d * case["H"] / case["Hkv"]}
    kept = case["B"] * case["Hkv"] * min(case["keep"], mean)
    # the weights, the kept rows read, written and read back, weights and indices, the values
    return {"bytes": 4 * n + kept * (3 * row + 8 + 8 * d), "flops": n}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    return _EXACT[case["op"]](st, case)


def _exact_prefill(st, case):
    q, k, v = st["q"], st["k"], st["v"]
    H, N, d = q.shape
    G = H // k.shape[0]
    out = torch.zeros((H, N, d), dtype=torch.float64, device="cuda")
    t0 = 0
    for n in st["lens"]:
        for r0 in range(0, n, 2048):            # blocks of queries, each against all keys up to its last
            r1 = min(n, r0 + 2048)
            later = torch.triu(torch.ones((r1 - r0, r1), dtype=torch.bool, device="cuda"), r0 + 1)
            for h in range(H):
                kk, vv = k[h // G, t0:t0 + r1].double(), v[h // G, t0:t0 + r1].double()
                a = (q[h, t0 + r0:t0 + r1].double() @ kk.T) / math.sqrt(d)
                p = torch.softmax(a.masked_fill(later, -math.inf), -1)
                out[h, t0 + r0:t0 + r1] = p @ vv
        t0 += n
    return out


def _exact_values(x):
    xs = x.double().unflatten(-1, (-1, _GROUP))
    lo = xs.min(-1).values
    step = torch.stack([(xs.max(-1).values - lo) / 15, xs.abs().max(-1).values / 1024]).max(0).values.bfloat16().double()
    safe = torch.where(step == 0, 1.0, step)[..., None]
    off = (lo[..., None] / safe).half().double()
    c = torch.clamp(torch.round(xs / safe - off), 0, 15)
    return torch.where(step[..., None] == 0, 0.0, step[..., None] * (c + off)).flatten(-2)


def _exact_append(st, case):
    return _exact_values(st["k"]), _exact_values(st["v"])


def _exact_rows(b, w):
    """Values of packed rows, channel by channel of a group, in 64 bits."""
    d, g = b.shape[-1] * 2, b.shape[-1] // 16
    out = torch.empty((*b.shape[:-1], d), dtype=torch.float64, device=b.device)
    scale = ((w & 0xFFFF) << 16).view(torch.float32).double()
    off = (w >> 16).to(torch.int16).view(torch.float16).double()
    for ch in range(d):
        grp, r, i = ch // 32, (ch % 32) // 4, ch % 4
        byte = b[..., (r * g + grp) * 2 + i // 2].to(torch.int32)
        out[..., ch] = scale[..., grp] * (((byte >> (4 * (i % 2))) & 15).double() + off[..., grp])
    return out


def _exact_decode(st, case):
    q, lens, c = st["q"].double(), st["lens"].tolist(), st["cache"]
    B, H, d = q.shape
    Hkv = c[0].shape[1]
    out = torch.zeros((B, H, d), dtype=torch.float64, device="cuda")
    wts = torch.zeros(st["weights"].shape, dtype=torch.float64, device="cuda")
    for b in range(B):
        n = lens[b]
        if n == 0:
            continue
        k, v = _exact_rows(c[0][b, :, :n], c[1][b, :, :n]), _exact_rows(c[2][b, :, :n], c[3][b, :, :n])
        qs = q[b].unflatten(0, (Hkv, -1))
        p = torch.softmax(torch.einsum("hgd,htd->hgt", qs, k) / math.sqrt(d), -1)
        out[b] = torch.einsum("hgt,htd->hgd", p, v).flatten(0, 1)
        wts[b, :, :n] = st["weights"][b, :, :n].double() + p.sum(1)
    return (out, wts) if case["weights"] else out


def _exact_evict(st, case):
    keep, recent, c = case["keep"], case["recent"], st["cache"]
    B, Hkv, cap = st["weights"].shape
    w = st["weights"].double().cpu().numpy()
    wt = np.zeros((B, Hkv, keep))
    idx = np.full((B, Hkv, keep), -1, dtype=np.int64)
    lens = st["lens"].tolist()
    for b in range(B):
        n = lens[b]
        for h in range(Hkv):
            if n <= keep:
                sel = np.arange(n)
            else:
                old = n - recent
                order = np.lexsort((np.arange(old), -w[b, h, :old]))[:keep - recent]
                sel = np.concatenate([np.sort(order), np.arange(old, n)])
            idx[b, h, :len(sel)] = sel
            wt[b, h, :len(sel)] = w[b, h, sel]
    it = torch.from_numpy(idx).cuda()
    vals = []
    for cb, cw in ((c[0], c[1]), (c[2], c[3])):
        at = it.clamp(min=0)[..., None]
        x = _exact_rows(cb.gather(2, at.expand(-1, -1, -1, cb.shape[-1])), cw.gather(2, at.expand(-1, -1, -1, cw.shape[-1])))
        x = torch.where(it[..., None] >= 0, x, 0.0)
        vals.append(x.transpose(0, 1).reshape(Hkv, B * keep, case["d"]))
    n_out = st["lens"].clamp(max=keep)
    return it.int(), torch.from_numpy(wt).cuda(), n_out, vals[0], vals[1]


_EXACT = {"prefill": _exact_prefill, "append": _exact_append, "decode": _exact_decode, "evict": _exact_evict}
