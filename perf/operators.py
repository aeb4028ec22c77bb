"""What is measured of the cache and sampling operators, and their plain forms.

Three operators of a decode step: keys and values appended to a paged cache with the position
rotation on the way (``append_kv``), attention of a ragged batch over that cache held in
4 bits (``attend``), and the draw of tokens with a request's temperature, top-k, top-p and
min-p (``sample_filtered``).

A 4-bit cache stores, for each block of 16 values along the head dimension, a scale in e4m3
and 16 codes in e2m1 (two to a byte, the even element low); a value is code * scale * the
kv head's fp32 scale.
"""
import math
import random

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # append: one sequence's draft batch (K = 7: its verified rows, the next-token and the
        # mask rows) -- latency
        dict(name="append one sequence", op="append", B=1, rows=15, Hq=64, Hkv=8, D=64, rot=64,
             bs=16, kind="e2m1", dtype="bf16", pad=0.0, base=10000, far=4096, values=False,
             interleaved=False, lens=1),
        # append: 64 sequences at K = 7 into a 16-bit cache, rejected rows padded out
        dict(name="append 64 to 16 bits", op="append", B=64, rows=15, Hq=32, Hkv=8, D=128,
             rot=128, bs=16, kind="16", dtype="bf16", pad=0.25, base=1000000, far=16384,
             values=False, interleaved=False, lens=2),
        # append: the large batch's draft rows, far positions, the stored values asked for
        dict(name="append 1024 to 4 bits", op="append", B=1024, rows=15, Hq=64, Hkv=8, D=64,
             rot=64, bs=16, kind="e2m1", dtype="bf16", pad=0.25, base=150000, far=100000,
             values=True, interleaved=False, lens=3),
        # append: a prompt, fp32, adjacent pairs rotated, half of the head dimension, odd pages
        dict(name="append fp32 prompt", op="append", B=3, rows=1000, Hq=12, Hkv=3, D=80, rot=40,
             bs=20, kind="e2m1", dtype="f32", pad=0.05, base=10000, far=32768, values=True,
             interleaved=True, lens=4),
        # attend: one sequence's draft batch over 4096 keys -- latency
        dict(name="attend one sequence", op="attend", B=1, q_lo=8, q_hi=8, k_lo=4096, k_hi=4096,
             Hq=64, Hkv=8, D=64, bs=16, dtype="bf16", lens=5),
        # attend: one token a sequence, 64 sequences of 512 to 16384 keys
        dict(name="attend 64 single tokens", op="attend", B=64, q_lo=1, q_hi=1, k_lo=512,
             k_hi=16384, Hq=32, Hkv=8, D=128, bs=16, dtype="bf16", lens=6),
        # attend: a draft batch of 64 sequences (1 to 15 live rows each), 64 query heads
        dict(name="attend 64 draft batches", op="attend", B=64, q_lo=1, q_hi=15, k_lo=512,
             k_hi=16384, Hq=64, Hkv=8, D=64, bs=16, dtype="bf16", lens=7),
        # attend: one token over the longest context
        dict(name="attend one long", op="attend", B=1, q_lo=1, q_hi=1, k_lo=100000, k_hi=100000,
             Hq=32, Hkv=8, D=128, bs=16, dtype="bf16", lens=8),
        # attend: prompts' rows (a drafter's first pass), ragged, a page size that is no power of 2
        dict(name="attend prompts", op="attend", B=4, q_lo=200, q_hi=700, k_lo=700, k_hi=4000,
             Hq=16, Hkv=2, D=128, bs=48, dtype="bf16", lens=9),
        # sample: one sequence's K = 7 rows, every filter -- latency
        dict(name="sample one sequence", op="sample", B=1, K=7, V=201088, dtype="bf16",
             filters="mixed", sigma=3.0, zipf=1.1, lens=10),
        # sample: temperature alone, 64 sequences of K = 7 rows, fp32 logits
        dict(name="sample 64 by temperature", op="sample", B=64, K=7, V=151936, dtype="f32",
             filters="none", sigma=3.0, zipf=0.0, lens=11),
        # sample: a large batch, every request with its own filters
        dict(name="sample 256 mixed", op="sample", B=256, K=3, V=201088, dtype="bf16",
             filters="mixed", sigma=3.0, zipf=1.1, lens=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "attend", "sample"))
    lens = rng.randrange(1 << 30)
    if op == "append":
        Hkv = rng.choice((1, 2, 3, 4, 8))
        D = 16 * rng.randint(2, 16)
        rows = _log(rng, 1, 400)
        B = _log(rng, 1, max(1, 1024 * 15 * 8 * 64 // (rows * Hkv * D * 2)))
        return dict(op=op, B=min(B, 1024), rows=rows, Hq=Hkv * rng.randint(1, 8), Hkv=Hkv, D=D,
                    rot=rng.choice((0, D, D, D // 2, 2 * rng.randint(1, D // 2))),
                    bs=rng.choice((1, 4, 16, 16, 32, 20, 64, 128)),
                    kind=rng.choice(("e2m1", "e2m1", "16")), dtype=rng.choice(("bf16", "bf16", "f32")),
                    pad=rng.choice((0.0, 0.2)), base=rng.choice((10000, 150000, 1000000)),
                    far=_log(rng, 1, 1000000), values=rng.random() < 0.5,
                    interleaved=rng.random() < 0.3, lens=lens)
    if op == "attend":
        Hkv = rng.choice((1, 2, 4, 5, 8))
        D = rng.choice((64, 128))
        k_hi = _log(rng, 1, 30000)
        B = _log(rng, 1, min(96, max(1, 64 * 16384 * 8 * 64 // (k_hi * Hkv * D))))
        q_hi = min(k_hi, _log(rng, 1, max(1, min(600, 12000 // B))))
        G = rng.choice((1, 2, 4, 7, 8, 16))
        while G > 1 and B * q_hi * G * Hkv * k_hi > 1 << 30:  # the plain form's scores
            G -= 1
        while q_hi > 1 and B * q_hi * G * Hkv * k_hi > 1 << 30:
            q_hi = q_hi * 2 // 3
        return dict(op=op, B=B, q_lo=rng.randint(1, q_hi), q_hi=q_hi,
                    k_lo=rng.choice((q_hi, k_hi)), k_hi=k_hi, Hq=Hkv * G, Hkv=Hkv, D=D,
                    bs=rng.choice((1, 8, 16, 16, 16, 32, 48, 20, 64, 128)),
                    dtype=rng.choice(("bf16", "bf16", "bf16", "f32")), lens=lens)
    V = _log(rng, 2, 300000)
    K = rng.randint(1, 8)
    return dict(op=op, B=_log(rng, 1, min(1024, max(1, 120_000_000 // (V * K)))), K=K, V=V,
                dtype=rng.choice(("bf16", "f32")),
                filters=rng.choice(("none", "top_k", "top_p", "min_p", "mixed", "mixed")),
                sigma=rng.uniform(0.5, 5.0), zipf=rng.choice((0.0, 1.1)), lens=lens)


# ------------------------------------------------------------- lengths, from the case alone
def _attend_lengths(case):
    rng = random.Random(case["lens"])
    rows, keys = [], []
    for _ in range(case["B"]):
        n = rng.randint(case["q_lo"], case["q_hi"])
        rows.append(n)
        keys.append(max(n, rng.randint(min(case["k_lo"], case["k_hi"]), case["k_hi"])))
    return rows, keys


def _append_live(case):
    """Which rows of the append carry a slot."""
    rng = random.Random(case["lens"])
    return [rng.random() >= case["pad"] for _ in range(case["B"] * case["rows"])]


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _row_bytes(case, D, kind):
    if kind == "e2m1":
        return D // 2 + D // 16
    return D * (2 if case["dtype"] == "bf16" else 4)


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "append":
        n = sum(_append_live(case))
        Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
        b = n * (2 * Hq * D * e + 2 * Hkv * D * e + 2 * Hkv * _row_bytes(case, D, case["kind"]))
        b += n * 2 * Hkv * D * e if case["values"] else 0
        b += case["B"] * case["rows"] * 12 + 2 * case["rot"]
        return dict(bytes=b, flops=n * (Hq + Hkv) * case["rot"] * 3 + n * 2 * Hkv * D * 4)
    if case["op"] == "attend":
        rows, keys = _attend_lengths(case)
        Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
        b = sum(keys) * Hkv * 2 * (D // 2 + D // 16) + sum(rows) * Hq * (2 * D * e + 4)
        b += sum(-(-k // case["bs"]) for k in keys) * 4 + sum(rows) * 4 + case["B"] * 8
        seen = sum(n * (k - n) + n * (n + 1) // 2 for n, k in zip(rows, keys))
        return dict(bytes=b, flops=seen * Hq * D * 4)
    n = case["B"] * case["K"]
    return dict(bytes=n * (case["V"] * e + 12) + case["B"] * 16, flops=n * case["V"] * 4)


# ----------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _nibbles(g, shape):
    """Random cache bytes whose two codes are distributed as a normal value's are."""
    q = (torch.arange(256, device=DEV, dtype=torch.float64) + 0.5) / 256
    v = torch.special.ndtri(q) * 2.4
    code = (v.abs()[:, None] - torch.tensor(E2M1, device=DEV, dtype=torch.float64)).abs().argmin(1)
    lut = (code + 8 * (v < 0)).to(torch.uint8)
    r = torch.randint(0, 65536, shape, generator=g, device=DEV, dtype=torch.int32)
    return lut[r & 255] | (lut[r >> 8] << 4)


def _block_scales(g, shape):
    return (torch.randn(shape, generator=g, device=DEV) * 0.25 - 1.0).exp().to(torch.float8_e4m3fn)


def _prepare_append(case, seed):
    g, dt = _gen(seed), _dtype(case)
    B, n, Hq, Hkv, D, bs = (case[k] for k in ("B", "rows", "Hq", "Hkv", "D", "bs"))
    T = B * n
    # one fused projection's output: the rows of q, k and v are views of it
    qkv = torch.randn((T, (Hq + 2 * Hkv) * D), generator=g, device=DEV).to(dt)
    q = qkv[:, :Hq * D].view(T, Hq, D)
    k = qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
    v = qkv[:, (Hq + Hkv) * D:].view(T, Hkv, D)
    start = torch.randint(0, case["far"], (B,), generator=g, device=DEV)
    pos = (start[:, None] + torch.arange(n, device=DEV)).reshape(T)
    per = -(-(n + bs - 1) // bs)  # pages that a sequence's rows can touch
    table = torch.randperm(B * per, generator=g, device=DEV).view(B, per)
    at = (start % bs)[:, None] + torch.arange(n, device=DEV)
    slot = (table.gather(1, at // bs) * bs + at % bs).reshape(T)
    live = torch.tensor(_append_live(case), device=DEV)
    s = dict(op="append", case=case, q=q, k=k, v=v, positions=pos.to(torch.int32),
             slots=torch.where(live, slot, -1).to(torch.int64),
             inv_freq=(1.0 / case["base"] ** (torch.arange(0, case["rot"], 2, device=DEV, dtype=torch.float64)
                                              / max(1, case["rot"]))).float(),
             k_scale=torch.rand((Hkv,), generator=g, device=DEV) + 0.5,
             v_scale=torch.rand((Hkv,), generator=g, device=DEV) + 0.5)
    if case["kind"] == "e2m1":
        for w in "kv":
            s[w + "_pages"] = _nibbles(g, (B * per, Hkv, bs, D // 2))
            s[w + "_block_scales"] = _block_scales(g, (B * per, Hkv, bs, D // 16))
    else:
        for w in "kv":
            s[w + "_pages"] = torch.randn((B * per, Hkv, bs, D), generator=g, device=DEV).to(dt)
            s[w + "_block_scales"] = None
    s["out"] = dict(q=torch.zeros((T, Hq, D), dtype=dt, device=DEV))
    if case["values"]:
        s["out"] |= {w: torch.zeros((T, Hkv, D), dtype=dt, device=DEV) for w in ("k", "v")}
    return s


def _prepare_attend(case, seed):
    g, dt = _gen(seed), _dtype(case)
    B, Hq, Hkv, D, bs = (case[k] for k in ("B", "Hq", "Hkv", "D", "bs"))
    rows, keys = _attend_lengths(case)
    rows_t, keys_t = torch.tensor(rows, device=DEV), torch.tensor(keys, device=DEV)
    pages = [-(-k // bs) for k in keys]
    pool, widest = sum(pages), max(pages)
    pages_t = torch.tensor(pages, device=DEV)
    ids = torch.randperm(pool, generator=g, device=DEV)
    col = torch.arange(widest, device=DEV)
    first = pages_t.cumsum(0) - pages_t
    table = torch.where(col < pages_t[:, None], ids[(first[:, None] + col).clamp(max=pool - 1)], -1)
    qsl = torch.cat((torch.zeros(1, device=DEV, dtype=torch.int64), rows_t.cumsum(0)))
    T = sum(rows)
    seq = torch.repeat_interleave(torch.arange(B, device=DEV), rows_t)
    pos = (keys_t - rows_t)[seq] + torch.arange(T, device=DEV) - qsl[seq]
    q = (torch.randn((T, Hq, D), generator=g, device=DEV) * 1.5).to(dt)
    s = dict(op="attend", case=case, q=q, qsl=qsl.int(), positions=pos.int(), seq_lens=keys_t.int(),
             table=table.int(), k_scale=torch.rand((Hkv,), generator=g, device=DEV) + 0.5,
             v_scale=torch.rand((Hkv,), generator=g, device=DEV) + 0.5, scale=D ** -0.5,
             widest_rows=max(rows))
    for w in "kv":
        s[w + "_pages"] = _nibbles(g, (pool, Hkv, bs, D // 2))
        s[w + "_block_scales"] = _block_scales(g, (pool, Hkv, bs, D // 16))
    s["out"] = dict(out=torch.zeros((T, Hq, D), dtype=dt, device=DEV),
                    lse=torch.zeros((T, Hq), dtype=torch.float32, device=DEV))
    return s


def _prepare_sample(case, seed):
    g, dt = _gen(seed), _dtype(case)
    B, K, V = case["B"], case["K"], case["V"]
    x = torch.empty((B, K, V), dtype=dt, device=DEV)
    bias = -case["zipf"] * torch.log(torch.arange(V, device=DEV, dtype=torch.float32) + 1.0)
    for i in range(0, B, 64):
        n = min(64, B - i)
        x[i:i + n] = (torch.randn((n, K, V), generator=g, device=DEV) * case["sigma"] + bias).to(dt)
    s = dict(op="sample", case=case, logits=x,
             uniforms=torch.rand((B, K), generator=g, device=DEV).clamp_(max=1 - 2.0 ** -24),
             temperature=torch.rand((B,), generator=g, device=DEV) * 1.2 + 0.3,
             top_k=None, top_p=None, min_p=None,
             out=dict(tokens=torch.zeros((B, K), dtype=torch.int32, device=DEV),
                      probs=torch.zeros((B, K), dtype=torch.float32, device=DEV)))
    f = case["filters"]
    k = torch.randint(1, min(V, 400) + 1, (B,), generator=g, device=DEV)
    p = 1 - 0.5 * torch.rand((B,), generator=g, device=DEV) ** 2
    m = 0.2 * torch.rand((B,), generator=g, device=DEV) ** 2
    if f == "mixed":  # each request has its own: some filters are off, some are greedy
        on = torch.rand((4, B), generator=g, device=DEV)
        k, p, m = torch.where(on[0] < 0.5, k, 0), torch.where(on[1] < 0.5, p, 1.0), torch.where(on[2] < 0.3, m, 0.0)
        s["temperature"] = torch.where(on[3] < 0.1, 0.0, s["temperature"])
    if f in ("top_k", "mixed"):
        s["top_k"] = k.int()
    if f in ("top_p", "mixed"):
        s["top_p"] = p.float()
    if f in ("min_p", "mixed"):
        s["min_p"] = m.float()
    return s


def prepare(case, seed):
    s = dict(append=_prepare_append, attend=_prepare_attend, sample=_prepare_sample)[case["op"]](case, seed)
    if own:  # the call with its fixed buffers marshalled once, as a decode loop keeps it
        import speculative_decoding_step_pspec_b200 as ps
        if s["op"] != "sample":
            cache = ps.KVCache(k=s["k_pages"], v=s["v_pages"], k_block_scales=s["k_block_scales"],
                               v_block_scales=s["v_block_scales"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        if s["op"] == "append":
            s["call"], _ = ps.prepare_append_kv(s["k"], s["v"], s["positions"], s["slots"], cache, q=s["q"],
                                                inv_freq=s["inv_freq"], interleaved=case["interleaved"], out=s["out"])
        elif s["op"] == "attend":
            s["call"], _ = ps.prepare_attend(s["q"], cache, s["table"], s["qsl"], s["positions"], s["seq_lens"],
                                             scale=s["scale"], out=s["out"])
        else:
            s["call"], _ = ps.prepare_sample_filtered(s["logits"], s["uniforms"], temperature=s["temperature"],
                                                      top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"], out=s["out"])
    return s


# ------------------------------------------------------------------- the operators, plainly
def _rotate(x, cos, sin, interleaved):
    """x [T, H, D] with its first 2 * cos.shape[-1] elements rotated by the row's angles."""
    h = cos.shape[-1]
    a, b = (x[..., 0:2 * h:2], x[..., 1:2 * h:2]) if interleaved else (x[..., :h], x[..., h:2 * h])
    c, s = cos[:, None], sin[:, None]
    a, b = a * c - b * s, b * c + a * s
    r = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((r, x[..., 2 * h:]), -1)


def _quantise(x, g):
    """Codes, block scales (as values) of x [T, H, D] with the heads' scales g [H]; 64 bits, for
    a value next to a border takes the other code when it is off by anything."""
    T, H, D = x.shape
    y = (x.double() / g.double()[None, :, None]).view(T, H, D // 16, 16)
    a = y.abs().amax(-1) / 6
    e = (torch.frexp(a)[1] - 1).clamp(min=-6)
    step = torch.exp2((e - 3).double())
    s = (torch.round(a / step) * step).clamp(max=448.0)
    z = torch.where(s[..., None] > 0, y.abs() / s.clamp(min=2.0 ** -9)[..., None], 0.0)
    code = torch.zeros_like(z, dtype=torch.uint8)
    for i, mid in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        code += (z >= mid) if i % 2 else (z > mid)  # ties to the even code
    code += 8 * torch.signbit(y)
    return code.view(T, H, D), s


def _values(code, s, g):
    """What codes [..., D] with block scales [..., D / 16] stand for, with g to broadcast."""
    lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=code.device, dtype=torch.float32)
    return ((lut[code.int()].view(*s.shape, 16) * s.float()[..., None]).flatten(-2) * g).float()


def _plain_append(s):
    c = s["case"]
    bs, live = c["bs"], s["slots"] >= 0
    rows, slot = live.nonzero()[:, 0], s["slots"][live]
    angle = s["positions"][rows].double()[:, None] * s["inv_freq"].double()
    cos, sin = angle.cos(), angle.sin()
    dt = s["q"].dtype
    out = {"q": s["out"]["q"].clone()}
    out["q"][rows] = _rotate(s["q"][rows].float(), cos.float(), sin.float(), c["interleaved"]).to(dt)
    k = _rotate(s["k"][rows].double(), cos, sin, c["interleaved"])
    for w, x in (("k", k), ("v", s["v"][rows].double())):
        pages, scales = s[w + "_pages"].clone(), s[w + "_block_scales"]
        if scales is None:
            pages[slot // bs, :, slot % bs] = x.float().to(dt)
            stored = x.float()
        else:
            scales = scales.clone()
            code, sc = _quantise(x, s[w + "_scale"])
            pages[slot // bs, :, slot % bs] = code[..., ::2] | (code[..., 1::2] << 4)
            scales.view(torch.uint8)[slot // bs, :, slot % bs] = sc.float().to(torch.float8_e4m3fn).view(torch.uint8)
            out[w + "_block_scales"] = scales
            stored = _values(code, sc, s[w + "_scale"][None, :, None])
        out[w + "_pages"] = pages
        if c["values"]:
            out[w] = s["out"][w].clone()
            out[w][rows] = stored.to(dt)
    return out


def _gathered(s, w):
    """The cache's keys or values of every sequence, padded to the longest: [B, Hkv, len, D]."""
    t = s["table"].clamp(min=0).long()
    code, sc = s[w + "_pages"][t], s[w + "_block_scales"].view(torch.uint8)[t].view(torch.float8_e4m3fn)
    code = torch.stack((code & 15, code >> 4), -1).flatten(-2)
    x = _values(code, sc, s[w + "_scale"][:, None, None])  # [B, pages, Hkv, bs, D]
    return x.transpose(1, 2).flatten(2, 3)


def _plain_attend(s):
    c, qsl = s["case"], s["qsl"].long()
    B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
    n, most = qsl[1:] - qsl[:-1], s["widest_rows"]
    j = torch.arange(most, device=DEV)
    there = j < n[:, None]
    at = torch.where(there, qsl[:-1, None] + j, 0)
    q = s["q"].float()[at].view(B, most, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    k = _gathered(s, "k")
    x = (q @ k.transpose(-1, -2)) * s["scale"]  # [B, Hkv, G * most, len]
    del k
    key = torch.arange(x.shape[-1], device=DEV)
    seen = (key <= s["positions"][at].long()[..., None]) & (key < s["seq_lens"].long()[:, None, None])
    x = x.view(B, Hkv, Hq // Hkv, most, -1).masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ _gathered(s, "v")).view(*p.shape[:-1], D) / total
    o = o.permute(0, 3, 1, 2, 4).reshape(B, most, Hq, D)
    lse = (top + total.log()).squeeze(-1).permute(0, 3, 1, 2).reshape(B, most, Hq)
    return dict(out=o[there].to(s["q"].dtype), lse=lse[there])


def _plain_sample(s):
    B, K, V = s["logits"].shape
    row = lambda v, off: (torch.full((B,), off, device=DEV) if v is None else v).repeat_interleave(K)[:, None]  # noqa: E731
    x = s["logits"].view(B * K, V).double()
    t = row(s["temperature"], 1.0).double()
    top_k, top_p, min_p = row(s["top_k"], 0).long(), row(s["top_p"], 1.0).double(), row(s["min_p"], 0.0).double()
    x, ids = x.sort(dim=1, descending=True, stable=True)  # ties: the lowest id first
    w = ((x - x[:, :1]) / torch.where(t > 0, t, 1.0)).exp()
    del x
    rank = torch.arange(V, device=DEV)
    kept = (rank < torch.where(top_k > 0, top_k, V)) & ((t > 0) | (rank == 0))
    w *= kept
    mass = w.cumsum(1)
    kept &= ((mass - w) < top_p * mass[:, -1:]) | (top_p >= 1)
    kept &= (w >= min_p)
    kept[:, 0] = True
    w *= kept
    w = torch.zeros_like(w).scatter_(1, ids, w)  # back in the order of ids
    del ids, kept, mass
    cdf = w.cumsum(1)
    total = cdf[:, -1:]
    over = cdf > row(None, 0.0) + s["uniforms"].view(-1, 1).double() * total
    last = ((w > 0) * rank).amax(1)
    token = torch.where(over.any(1), over.int().argmax(1), last)
    probs = w.gather(1, token[:, None]) / total
    return dict(tokens=token.int().view(B, K), probs=probs.float().view(B, K))


def run(state):
    if own:
        state["call"]()
        r = dict(state["out"])
        if state["op"] == "append":
            for w in "kv":
                r[w + "_pages"] = state[w + "_pages"]
                if state[w + "_block_scales"] is not None:
                    r[w + "_block_scales"] = state[w + "_block_scales"]
        return r
    return dict(append=_plain_append, attend=_plain_attend, sample=_plain_sample)[state["op"]](state)


# ----------------------------------------------------------- the definitions, in 64 bits
def _exact_append(case, s):
    """Row by row of the definition, as values: the rotation as a product of complex numbers, the
    nearest code found among all eight."""
    T, Hq, D = s["q"].shape
    h, live = case["rot"] // 2, (s["slots"] >= 0).nonzero()[:, 0]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                       torch.outer(s["positions"].double(), s["inv_freq"].double()))[live, None]

    def turned(x):
        x = x[live].double()
        if not h:
            return x
        if case["interleaved"]:
            z = torch.view_as_complex(x[..., :2 * h].reshape(*x.shape[:2], h, 2).contiguous()) * turn
            r = torch.view_as_real(z).reshape(*x.shape[:2], 2 * h)
        else:
            z = torch.complex(x[..., :h].contiguous(), x[..., h:2 * h].contiguous()) * turn
            r = torch.cat((z.real, z.imag), -1)
        return torch.cat((r, x[..., 2 * h:]), -1)

    q = torch.zeros((T, Hq, D), dtype=torch.float64, device=DEV)
    q[live] = turned(s["q"])
    out = dict(q=q)
    for w, x in (("k", turned(s["k"])), ("v", s["v"][live].double())):
        at = s["slots"][live]
        if case["kind"] == "e2m1":
            g = s[w + "_scale"].double()[:, None, None]
            y = x.view(*x.shape[:2], -1, 16) / g
            grid = torch.arange(127, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn).double()  # 0 .. 448
            a = y.abs().amax(-1) / 6
            hi = torch.searchsorted(grid, a.contiguous()).clamp(max=126)
            lo = (hi - 1).clamp(min=0)
            up, down = grid[hi] - a, a - grid[lo]
            pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)) | (a > 448), hi, lo)
            sc = grid[pick]
            levels = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
            z = y.abs() / torch.where(sc > 0, sc, 1.0)[..., None]
            far = (z[..., None] - levels).abs() + 1e-300 * (torch.arange(8, device=DEV) % 2)
            best = far.amin(-1, keepdim=True)
            even = torch.tensor([0, 2, 4, 6, 1, 3, 5, 7], device=DEV)  # of two as near, the even code
            code = even[(far[..., even] == best).int().argmax(-1)]
            code = torch.where(sc[..., None] > 0, code, 0)
            x = (levels[code] * torch.where(torch.signbit(y), -1.0, 1.0) * sc[..., None] * g).flatten(-2)
            scales = s[w + "_block_scales"].double()
            scales[at // case["bs"], :, at % case["bs"]] = sc
            out[w + "_block_scales"] = scales
            out[w + "_pages"] = None  # codes: compared as whole numbers
        else:
            pages = s[w + "_pages"].double()
            pages[at // case["bs"], :, at % case["bs"]] = x
            out[w + "_pages"] = pages
        if case["values"]:
            full = torch.zeros((T, case["Hkv"], D), dtype=torch.float64, device=DEV)
            full[live] = x
            out[w] = full
    return out


def _exact_attend(case, s):
    """Sequence by sequence, head by head."""
    levels = torch.tensor(E2M1 + tuple(-x for x in E2M1), dtype=torch.float64, device=DEV)
    T, Hq, D = s["q"].shape
    G = Hq // case["Hkv"]
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device=DEV)
    lse = torch.zeros((T, Hq), dtype=torch.float64, device=DEV)
    qsl, lens = s["qsl"].tolist(), s["seq_lens"].tolist()
    for i in range(case["B"]):
        lo, hi, n = qsl[i], qsl[i + 1], lens[i]
        pages = s["table"][i, :-(-n // case["bs"])].long()
        hidden = torch.arange(n, device=DEV) > s["positions"][lo:hi, None]
        for h in range(case["Hkv"]):
            kv = []
            for w in "kv":
                b = s[w + "_pages"][pages, h].view(-1, D // 2)[:n].int()
                x = levels[torch.stack((b % 16, b // 16), -1)].view(n, D // 16, 16)
                x = x * s[w + "_block_scales"][pages, h].double().view(-1, D // 16)[:n, :, None]
                kv.append(x.view(n, D) * s[w + "_scale"][h].double())
            z = torch.einsum("tgd,nd->gtn", s["q"][lo:hi, h * G:(h + 1) * G].double(), kv[0]) * s["scale"]
            z[:, hidden] = -math.inf
            l = torch.logsumexp(z, -1)
            out[lo:hi, h * G:(h + 1) * G] = torch.einsum("gtn,nd->tgd", (z - l[..., None]).exp(), kv[1])
            lse[lo:hi, h * G:(h + 1) * G] = l.T
    return dict(out=out, lse=lse)


def _exact_sample(case, s):
    """Request by request: the kept set as a list of ids, then the draw along it."""
    B, K, V = s["logits"].shape
    tokens = torch.zeros((B, K), dtype=torch.int32, device=DEV)
    probs = torch.zeros((B, K), dtype=torch.float64, device=DEV)
    get = lambda v, i, off: off if v is None else v[i].item()  # noqa: E731
    for i in range(B):
        t, k = s["temperature"][i].item(), get(s["top_k"], i, 0)
        p, m = get(s["top_p"], i, 1.0), get(s["min_p"], i, 0.0)
        for r in range(K):
            x = s["logits"][i, r].double()
            if t == 0:
                tokens[i, r], probs[i, r] = int((x == x.max()).nonzero()[0, 0]), 1.0
                continue
            best, ids = torch.sort(x / t, descending=True, stable=True)
            if k > 0:
                best, ids = best[:k], ids[:k]
            soft = torch.softmax(best, 0)
            if p < 1:
                before = torch.cat((soft.new_zeros(1), soft.cumsum(0)[:-1]))
                n = max(1, int((before < p).sum()))
                best, ids = best[:n], ids[:n]
            n = max(1, int(((best - best[0]).exp() >= m).sum()))
            ids, order = ids[:n].sort()
            mass = torch.softmax(best[:n], 0)[order]
            cdf = mass.cumsum(0)
            c = min(int((cdf <= s["uniforms"][i, r].double() * cdf[-1]).sum()), n - 1)
            tokens[i, r], probs[i, r] = ids[c].int(), mass[c] / cdf[-1]
    return dict(tokens=tokens, probs=probs)


def exact(case, seed):
    global own
    kept, own = own, False
    s = prepare(case, seed)
    own = kept
    return dict(append=_exact_append, attend=_exact_attend, sample=_exact_sample)[case["op"]](case, s)
