"""The ends of what the cache and sampling operators admit, on the GPU against their 64-bit references."""
import threading

import numpy as np
import pytest
import torch

import speculative_decoding_step_pspec_b200 as ps
from speculative_decoding_step_pspec_b200 import _binding as b
from speculative_decoding_step_pspec_b200 import inputs as I
from tests import ops_reference as R
from tests.test_cache_ops_gpu import (DEV, LAST, attend_case, gen, i32, logits, random_cache, run_attend,
                                      run_filtered, uniforms, wide_heads)

pytestmark = pytest.mark.gpu


# --------------------------------------------------------------------------- attend
def one_signed(c, size, seed):
    """Positive keys against queries of one sign, of about this size."""
    for w in "kv":
        getattr(c["cache"], w).bitwise_and_(0x77).bitwise_or_(0x11)
    c["q"] = (size * (torch.rand(c["q"].shape, device=DEV, generator=gen(seed)) + 0.5)).to(c["q"].dtype)
    return c


def check_largest_alone(c, out):
    """Where a row's largest score lies above the next by more than both are rounded (D + 8 roundings
    of 2^-23 each), and by tens, it has probability 1: the row is its value, with one rounding to the
    dtype and two of factors in fp32.  The weight itself, 2^7 and up to an octave more, is rounded as
    every probability is -- to fp16 for bf16 rows (half a step is 2^-11 of it), to two fp16 terms for
    fp32 rows (2^-22) -- and the sum that divides it is not.  Returns how many (row, head) pairs it were."""
    dtype, (T, Hq, D) = c["q"].dtype, c["q"].shape
    kv, vv = (R.cache_values(c["cache"], w) for w in "kv")
    q, got, lse, sure = R.f64(c["q"]), R.f64(out["out"]), R.f64(out["lse"]), 0
    step = R.HALF_STEP[dtype] + 2.0 ** -22 + (2.0 ** -11 if dtype == torch.bfloat16 else 2.0 ** -22)
    for i in range(len(c["lens"])):
        for t in range(c["qsl"][i], c["qsl"][i + 1]):
            j = np.arange(c["pos"][t] + 1)
            if not len(j):
                continue
            at = c["table"][i, j // c["bs"]], slice(None), j % c["bs"]
            k, v = kv[at], vv[at]
            for h in range(Hq):
                x = k[:, h // (Hq // kv.shape[1])] @ q[t, h] * float(np.float32(D ** -0.5))
                order = np.argsort(-x)
                top = x[order[0]]
                if len(j) > 1 and top - x[order[1]] <= (D + 8) * 2.0 ** -22 * abs(x[order[1]]) + 40:
                    continue
                sure += 1
                want = v[order[0], h // (Hq // kv.shape[1])]
                assert np.all(np.abs(got[t, h] - want) <= step * 1.01 * np.abs(want)), (t, h)
                assert abs(lse[t, h] - top) <= (D + 8) * 2.0 ** -23 * abs(top)
    return sure


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("size", [1e6, 1e8, 1e9, 1e13, 1e20, 1e28])
@pytest.mark.parametrize("D", [64, 128])
def test_attend_scores_without_a_fraction(D, size, dtype, sign):
    """Scores so large that fp32 holds no fraction of them, later no octave."""
    for rows, keys, Hq, Hkv in (([1, 2], [1, 2], 4, 2), ([8], [300], 8, 1), ([130], [200], 8, 4)):
        c = one_signed(attend_case(int(D + keys[0]), rows, keys, Hq, Hkv, D, 16, dtype), sign * size, D)
        assert check_largest_alone(c, run_attend(c)) >= (sum(rows) * Hq // 2 if size > 1e6 else 0)


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("size", [1e6, 1e8, 1e9, 1e13, 1e20, 1e28])
@pytest.mark.parametrize("D", [64, 128])
def test_attend_many_rows_scores_without_a_fraction(D, size, sign):
    H = wide_heads([40, 30], 2, D)
    c = one_signed(attend_case(D, [40, 30], [40, 150], 2 * H, H, D, 16, torch.bfloat16, extra_rows=0), sign * size, D)
    c["pos"][:3] = [-1, 0, 1]
    assert check_largest_alone(c, run_attend(c)) >= (60 * H if size > 1e6 else 0)


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_attend_moderate_scores_after_very_negative_ones(D, many):
    """The first keys' scores lie past 2^28 below zero, the later ones' within some hundreds of it: the
    running maximum comes back to where fractions count."""
    rows = [40, 30] if many else [3, 1]
    H = wide_heads(rows, 2, D) if many else 2
    c = attend_case(D, rows, [300, 200], 2 * H, H, D, 16, torch.bfloat16, extra_rows=0, qscale=100.0)
    pages = c["cache"].k
    pages[..., 0].bitwise_and_(0xF0)                            # element 0 of every key is zero ...
    for i in range(2):
        for j in range(150):                                    # ... but of each sequence's first keys
            pages[c["table"][i, j // 16], :, j % 16, 0].bitwise_or_(6)
            c["cache"].k_block_scales.view(torch.uint8)[c["table"][i, j // 16], :, j % 16, 0] = 0x7E
    c["q"][:, :, 0] = -3e6
    # scores: element 0 gives the far ones, the rest stays within hundreds
    out = run_attend(c)
    q = c["q"].clone()
    q[:, :, 0] = 0
    kv, vv = (R.cache_values(c["cache"], w) for w in "kv")
    _, _, _, a, vmax = R.attend(R.f64(q), kv, vv, c["table"], c["qsl"], c["pos"], c["lens"], D ** -0.5, 16)
    want = np.zeros(q.shape)
    for i in range(2):
        for t in range(c["qsl"][i], c["qsl"][i + 1]):
            j = np.arange(150, c["pos"][t] + 1)
            at = c["table"][i, j // 16], slice(None), j % 16
            for h in range(2 * H):
                x = kv[at][:, h // 2] @ R.f64(q)[t, h] * D ** -0.5
                p = np.exp(x - x.max())
                want[t, h] = p @ vv[at][:, h // 2] / p.sum()
    bound, _ = R.attend_bounds(torch.bfloat16, D, want, a, vmax)
    assert np.all(np.abs(R.f64(out["out"]) - want) <= bound)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("size", [1e30, 1e33, 1e36])
@pytest.mark.parametrize("D", [64, 128])
def test_attend_rows_with_very_negative_scores_alone(D, size, dtype):
    """A row whose visible scores all lie far below zero, of one key or of many, is no empty one."""
    for rows, keys, Hq, Hkv in (([1, 2], [1, 2], 4, 2), ([8], [300], 8, 1), ([130], [200], 8, 4)):
        c = one_signed(attend_case(int(D + keys[0]), rows, keys, Hq, Hkv, D, 16, dtype), -size, D)
        assert check_largest_alone(c, run_attend(c)) >= sum(rows) * Hq // 2


@pytest.mark.parametrize("D", [64, 128])
def test_attend_very_negative_scores_are_the_same_in_wide_tiles(D):
    """The same row alone (narrow tiles) and in a batch of many rows (wide ones)."""
    H = wide_heads([64], 1, D)
    c = one_signed(attend_case(D, [64], [64], H, H, D, 16, torch.bfloat16, extra_rows=0), -1e33, D)
    wide = run_attend(c)
    narrow = run_attend(dict(c, q=c["q"][:1].contiguous(), qsl=np.array([0, 1]), pos=c["pos"][:1]))
    assert torch.equal(narrow["out"][0], wide["out"][0]) and torch.isfinite(narrow["lse"]).all()


@pytest.mark.parametrize("dtype,many", [(torch.bfloat16, False), (torch.bfloat16, True), (torch.float32, False)])
@pytest.mark.parametrize("D", [64, 128])
def test_attend_at_the_ends_of_the_head_scales(D, dtype, many):
    """A power of two moved between the queries and the keys' head scales changes nothing, one in the
    values' only their power, as long as the outputs stay in fp32's normal range."""
    rows = [40, 30] if many else [3, 1]
    H = wide_heads(rows, 2, D) if many else 2
    c = attend_case(D, rows, [300, 20000], 2 * H, H, D, 16, dtype, extra_rows=0)
    cache, args = c["cache"], (i32(c["table"]), i32(c["qsl"]), i32(c["pos"]), i32(c["lens"]))
    k, v = cache.k_scale.clone(), cache.v_scale.clone()
    want = ps.attend(c["q"], cache, *args, want_lse=True)
    for e in (-110, -60, 60, 100):
        cache.k_scale = k * 2.0 ** e
        got = ps.attend(c["q"] * 2.0 ** -e, cache, *args, want_lse=True)
        assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"]), e
    cache.k_scale = torch.full_like(k, 2.0 ** -20)
    want = ps.attend(c["q"], cache, *args, want_lse=True)
    cache.k_scale = torch.full_like(k, 2.0 ** -140)
    got = ps.attend(c["q"] * 2.0 ** 120, cache, *args, want_lse=True)
    assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])
    for e in (-100, 100):
        cache.v_scale = v * 2.0 ** e
        got = ps.attend(c["q"] * 2.0 ** 120, cache, *args, want_lse=True)
        cache.v_scale = v
        want = ps.attend(c["q"] * 2.0 ** 120, cache, *args, want_lse=True)
        here = want["out"].double().abs() > 2.0 ** -25
        assert torch.equal(got["out"].double()[here], (want["out"].double() * 2.0 ** e)[here])


@pytest.mark.parametrize("D", [64, 128])
def test_attend_fp32_sums_along_many_keys(D):
    """fp32 rows over thousands of keys in one go: off by what fp32 rounds, not by what the tensor cores
    cut off.  Of outputs that are means of values of either sign, the relative error in the 2-norm is
    about that of the weights (products and sums of scores of size 10, the exponential: 2^-20 of root
    mean square) and that of some 300 additions in a row (2^-24 sqrt(300) = 2^-20)."""
    B, H, n, bs = 64, 8, 20000, 16
    g, pages = gen(D), n // bs
    cache = random_cache(g, pages * 4, H, bs, D)                # (sequences share four sets of pages)
    table = (torch.arange(B, device=DEV)[:, None] % 4 * pages + torch.arange(pages, device=DEV)).int()
    q = torch.randn((B, H, D), generator=g, device=DEV) * 1.5
    qsl, pos = torch.arange(B + 1, device=DEV).int(), torch.full((B,), n - 1, dtype=torch.int32, device=DEV)
    o = ps.attend(q, cache, table, qsl, pos, pos + 1)
    torch.cuda.synchronize()
    levels = torch.tensor(R.LEVELS, device=DEV)
    levels = torch.cat((levels, -levels))
    err = ref = 0.0
    for i in (0, 1, 63):
        for h in (0, 7):
            kv = []
            for w in "kv":
                b8 = getattr(cache, w)[table[i].long(), h].reshape(n, D // 2).int()
                x = levels[torch.stack((b8 & 15, b8 >> 4), -1)].view(n, D // 16, 16)
                x = x * getattr(cache, w + "_block_scales")[table[i].long(), h].double().view(n, D // 16, 1)
                kv.append(x.view(n, D) * getattr(cache, w + "_scale")[h].double())
            want = torch.softmax(kv[0] @ q[i, h].double() * D ** -0.5, 0) @ kv[1]
            err += (o["out"][i, h].double() - want).square().sum().item()
            ref += want.square().sum().item()
    assert (err / ref) ** 0.5 <= 2.5e-6


# --------------------------------------------------------------------------- append
@pytest.mark.parametrize("rot", [0, 64])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("g", [3e38, 1.5e38, 6e37, 2e-36, 1e-37, 1e-38, 1e-39, 1e-42])
def test_append_at_the_ends_of_the_head_scales(g, dtype, rot):
    """Any positive and finite head scale: codes and block scales as if computed exactly, for rows
    of its size, far smaller and (where fp32 holds them) far larger ones."""
    T, H, D, bs = 64, 2, 64, 16
    x = torch.randn((T, H, D), generator=gen(1), device=DEV, dtype=torch.float64)
    x *= g * 2.0 ** torch.linspace(-12, 12, T, device=DEV, dtype=torch.float64)[:, None, None]
    x = x.clamp(-1.5e38, 1.5e38).to(dtype)                      # (a rotation stays finite in fp32)
    x[1::2].abs_()                                              # blocks of one sign, and of both
    cache = random_cache(gen(2), 4, H, bs, D)
    cache.k_scale = torch.tensor([g, g * 0.75], device=DEV)
    cache.v_scale = torch.tensor([g * 0.8, g], device=DEV)
    pos = torch.arange(T, device=DEV, dtype=torch.int32)
    inv = (10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / max(rot, 1))).float()
    r = ps.append_kv(x, x, pos, torch.arange(T, device=DEV), cache, inv_freq=inv if rot else None)
    torch.cuda.synchronize()
    assert r["err"].item() == 0
    v = R.f64(x)
    for w, y in (("k", R.rotate(v, pos.cpu().numpy(), R.f64(inv), False)), ("v", v)):
        code, sc = R.quantise(y, R.f64(getattr(cache, w + "_scale")))
        got_s = getattr(cache, w + "_block_scales").view(torch.uint8).transpose(1, 2).reshape(T, H, -1).cpu().numpy()
        got_c = R.unpack(getattr(cache, w).transpose(1, 2).reshape(T, H, -1).cpu().numpy())
        assert np.array_equal(got_s, sc), np.argwhere(got_s != sc)[:5]
        mag = np.repeat(sc > 0, 16, -1)                         # a block of scale 0 holds zeros of either sign
        bad = np.where(mag, got_c != code, got_c & 7 != 0)
        # a rotated value on the sign's border may be a zero of either sign
        bad &= ~((got_c & 7 == 0) & (code & 7 == 0) & (np.abs(y) <= 1e-15 * np.abs(v).max(-1, keepdims=True)))
        assert not bad.any(), np.argwhere(bad)[:5]


# --------------------------------------------------------------------------- sample
@pytest.mark.parametrize("rows", [1, 40])
def test_sample_filtered_min_p_borders_next_to_zero(rows):
    """The border value M + t ln(min_p) lies within 1e-15 of 0, where fp32 values are far closer to one
    another than weights are resolved: it is found in a few steps all the same."""
    cases = [(2.0, 96, "0x1.800048p-17"), (1.0, 96, "0x1.800048p-18"), (0.7, 27, "0x1.2e6676p-20"),
             (0.7, 3, "0x1.0ccccep-23"), (1.0, 160, "0x1.400064p-17"), (0.9, 985, "0x1.bb4354p-15")]
    B, V = len(cases) * rows, 3001
    x = -torch.rand((B, 1, V), generator=gen(1), device=DEV) - 1e-3
    t, m = [], []
    for i in range(B):
        temperature, j, top = cases[i % len(cases)]
        top = float.fromhex(top)
        t.append(temperature)
        m.append(1 - j * 2.0 ** -24)
        x[i, 0, 10:20] = top * 0.9                              # kept with the largest
        x[i, 0, 20:30] = -top                                   # not kept
        x[i, 0, 17] = top
    u = uniforms(2, B, 1)
    run_filtered(x, u, t=t, m=m)
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    call, _ = ps.prepare_sample_filtered(x, u, temperature=torch.tensor(t, device=DEV), min_p=torch.tensor(m, device=DEV))
    call()
    torch.cuda.synchronize()
    a.record()
    call()
    b.record()
    torch.cuda.synchronize()
    assert a.elapsed_time(b) < 5.0                              # ms; tens of microseconds


def test_sample_filtered_from_two_threads_with_other_vocabularies():
    """Calls of several host threads, each on its stream: none lowers the shared memory that
    another's launch may take."""
    sizes = [(4, 7, 201088), (1, 2, 2100), (3, 5, 60000), (2, 4, 9001)]
    work = []
    for B, K, V in sizes:
        x, u = logits(V, B, K, V, torch.bfloat16), uniforms(V + 1, B, K)
        k = torch.full((B,), 20, dtype=torch.int32, device=DEV)
        work.append((x, u, k, ps.sample_filtered(x, u, top_k=k)["tokens"]))
    torch.cuda.synchronize()
    failed, streams = [], [torch.cuda.Stream() for _ in sizes]

    def loop(i):
        x, u, k, want = work[i]
        try:
            call, o = ps.prepare_sample_filtered(x, u, top_k=k)
            for _ in range(3000):
                call(streams[i])
            streams[i].synchronize()
            if not torch.equal(o["tokens"], want):
                failed.append((i, "tokens"))
        except Exception as e:                                  # noqa: BLE001 (reported below)
            failed.append((i, repr(e)))

    threads = [threading.Thread(target=loop, args=(i,)) for i in range(len(sizes))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


# --------------------------------------------------------------------------- prepared calls
def test_prepared_calls_do_not_run_ahead_of_their_zeros():
    """Prepared behind work that the current stream has queued, and called at once on another stream:
    counters and error words are zero before the call and not written after it."""
    c = attend_case(1, [1, 4], [9000, 3000], 8, 2, 64, 16, torch.bfloat16)
    args = (c["q"], c["cache"], i32(c["table"]), i32(c["qsl"]), i32(c["pos"]), i32(c["lens"]))
    x, u = logits(2, 3, 2, 5001, torch.float32), uniforms(3, 3, 2)
    t = torch.tensor([-1.0, 1.0, 1.0], device=DEV)              # sets the error word
    k = torch.randn((4, 2, 64), device=DEV).to(torch.bfloat16)
    pos, slots = torch.zeros(4, dtype=torch.int32, device=DEV), torch.tensor([0, -5, 1, 2], device=DEV)
    want = ps.attend(*args)
    n = int(c["qsl"][-1])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(5):
        junk = torch.full((ps.pspec_attend_workspace_bytes(),), 0x5A, dtype=torch.uint8, device=DEV)
        del junk                                                # what the workspace will be made of
        torch.cuda._sleep(50_000_000)                           # some tens of milliseconds
        attend, o = ps.prepare_attend(*args)
        attend(s)
        torch.cuda._sleep(50_000_000)
        draw, d = ps.prepare_sample_filtered(x, u, temperature=t)
        draw(s)
        torch.cuda._sleep(50_000_000)
        append, a = ps.prepare_append_kv(k, k, pos, slots, c["cache"])
        append(s)
        torch.cuda.synchronize()
        assert o["err"].item() == 0 and torch.equal(o["out"][:n], want["out"][:n])
        assert d["err"].item() == b.PSPEC_DEVERR_PARAM_RANGE and a["err"].item() == b.PSPEC_DEVERR_BLOCK_RANGE
        want = ps.attend(*args)                                 # (the cache has changed)
        torch.cuda.synchronize()


def test_calls_prepared_inside_a_capture_belong_to_its_graph():
    c = attend_case(4, [1, 4], [900, 300], 8, 2, 64, 16, torch.bfloat16)
    args = (c["q"], c["cache"], i32(c["table"]), i32(c["qsl"]), i32(c["pos"]), i32(c["lens"]))
    want = ps.attend(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call, o = ps.prepare_attend(*args)
        call()
    for _ in range(3):
        o["out"].fill_(-3)
        graph.replay()
    torch.cuda.synchronize()
    n = int(c["qsl"][-1])
    assert o["err"].item() == 0 and torch.equal(o["out"][:n], want["out"][:n])


@pytest.mark.parametrize("rejection", [False, True])
def test_steps_on_another_stream_do_not_run_ahead_of_their_zeros(rejection):
    """The step, its parts and its prepared call behind work that the current stream has queued, on
    another stream with nothing given: what they allocate is that stream's, or there already."""
    w = I.scaled(I.C64, B=6, V=4000, H=64, ctx="uniform", ctx_args=(20, 300))
    inp = I.build_inputs(w, DEV)
    d = torch.randint(0, w.V, (w.B, w.K), generator=gen(1), device=DEV, dtype=torch.int32)
    target, draft = logits(2, w.B, w.K + 1, w.V, torch.bfloat16), logits(3, w.B, w.K, w.V, torch.bfloat16)
    u = uniforms(4, w.B, w.K + 1)
    uk = u[:, :w.K].contiguous()
    kw = dict(draft_logits=draft, uniforms=u) if rejection else {}

    def same(got, want):
        torch.cuda.synchronize()
        assert got["err"].item() == 0
        for n in want:
            assert torch.equal(got[n], want[n]), n

    want_v, want_b = ps.step(target, d, inp, **kw)
    want_s = ps.sample_drafts(draft, uk)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        junk = [torch.full((n,), 0x5A, dtype=torch.uint8, device=DEV) for n in (1 << 20, 1 << 16, 512, 512, 512)]
        del junk
        torch.cuda._sleep(50_000_000)
        call, v, bo = ps.api.prepare_step(target, d, inp, **kw)
        call(s)
        torch.cuda._sleep(50_000_000)
        v2, b2 = ps.step(target, d, inp, stream=s, **kw)
        if rejection:
            v3 = ps.verify_rejection(target, draft, d, u, stream=s)
        else:
            v3 = ps.verify_greedy(target, d, stream=s)
        s3 = ps.sample_drafts(draft, uk, stream=s.cuda_stream)
        same(v, want_v)
        same(bo, want_b)
        same(v2, want_v)
        same(b2, want_b)
        same(v3, want_v)
        same(s3, want_s)


def repeated(x, times, dtype, pad, offset):
    """x [B, K, V] `times` over, in rows padded by `pad` elements and `offset` of them off alignment."""
    B, K, V = x.shape
    flat = torch.zeros((times * B * K * (V + pad) + 8,), dtype=dtype, device=DEV)
    r = flat[offset:offset + times * B * K * (V + pad)].view(times * B, K, V + pad)[..., :V]
    r.copy_(x.repeat(times, 1, 1))
    return r


STREAMED = [(torch.float32, 0, 0), (torch.float32, 3, 1), (torch.bfloat16, 0, 0), (torch.bfloat16, 5, 3)]


@pytest.mark.parametrize("dtype,pad,offset", STREAMED)
@pytest.mark.parametrize("V,times", [(3000, 4), (30011, 8)])
def test_sample_filtered_many_rows_infinities_and_nan(V, times, dtype, pad, offset):
    """Batches past the few rows whose slices lie in shared memory."""
    x = logits(14, 6, 2, V, torch.float32)
    x[0] = -float("inf")                                        # no mass: token 0, probability 0
    x[1, :, 10:] = -float("inf")                                # masked vocabulary
    x[2, 0, 77] = x[2, 0, 2900] = float("inf")                  # shares of the infinite
    x[2, 1] = float("nan")
    x[3, :, ::2] = float("nan")
    x[4] = -float("inf")
    x[4, :, 1234] = -1e38
    x[5] *= 1e37
    x, B = repeated(x, times, dtype, pad, offset), 6 * times
    u = uniforms(15, B, 2)
    for kw in ({}, dict(k=5), dict(p=0.5), dict(t=0.0), dict(m=0.3), dict(k=2500), dict(p=0.99, m=1e-4), dict(k=2000, p=0.9)):
        r = run_filtered(x, u, **{n: [v] * B for n, v in kw.items()})
        assert (r["tokens"][::6] == 0).all() and (r["probs"][::6] == 0).all() and (r["tokens"][4::6] == 1234).all()


@pytest.mark.parametrize("dtype,pad,offset", STREAMED)
def test_sample_filtered_many_rows_of_ties(dtype, pad, offset):
    """Few distinct logits, -0 among them: cuts inside a class of ties larger than one CTA sorts."""
    V = 30011
    x = torch.randint(0, 3, (6, 2, V), generator=gen(11), device=DEV).float()
    x[5, :, ::2] *= -0.0
    x, B = repeated(x, 4, dtype, pad, offset), 24
    u = uniforms(12, B, 2)
    run_filtered(x, u, k=[1, 4000, 15000, 25000, 29000, 0] * 4, p=[1, 1, 1, 1, 1, 0.3] * 4)
    run_filtered(x, u, p=[0.01, 0.2, 0.5, 0.7, 0.97, 0.9999] * 4)
    run_filtered(x, u, k=[5000, 6000, 12000, 20000, 25000, 29999] * 4, p=[0.5, 0.9, 0.99, 0.8, 0.3, 0.7] * 4)
    run_filtered(x, u, p=[0.01, 0.2, 0.5, 0.7, 0.97, 0.9999] * 4, m=[0.1, 0.3, 1.0, 0.14, 0.5, 0.0] * 4)
    same = repeated(torch.full((3, 2, V), -2.5, device=DEV), 8, dtype, pad, offset)
    run_filtered(same, u, k=[0, 9000, 0] * 8, p=[1, 1, 0.25] * 8, m=[0, 0, 1.0] * 8)


@pytest.mark.parametrize("dtype,pad,offset", STREAMED)
def test_sample_filtered_many_rows_at_extreme_uniforms(dtype, pad, offset):
    x = repeated(logits(16, 4, 2, 4000, torch.float32), 6, dtype, pad, offset)
    edge = torch.tensor([[0.0, LAST]] * 24, device=DEV)
    run_filtered(x, edge, t=[1, 0.3, 1, 1] * 6, k=[0, 0, 30, 0] * 6, p=[1, 1, 1, 0.9] * 6)


@pytest.mark.parametrize("times", [1, 5])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sample_filtered_so_hot_that_the_lowest_logit_weighs(dtype, times):
    """Temperatures at which every finite logit has a share: tokens at -inf, and what lies past a row's
    end, still have none."""
    t = [1e35, 5e35, 1e36, 1e37, 1e38, 3.4e38, 1e36, 1e36]
    B, V = len(t) * times, 5003
    x = logits(23, B, 2, V, torch.float32, sigma=1.0)
    x[::2] *= 1e38
    x[:, :, 1::3] = -float("inf")
    x[6::8] = (x[6::8].clamp(-10, 10) * 1e34) - 3.2e38          # all near the lowest
    x = x.to(dtype)
    u = uniforms(24, B, 2)
    for kw in ({}, dict(k=7), dict(k=2000), dict(p=0.3), dict(p=0.9), dict(m=0.5), dict(p=0.7, m=0.01), dict(k=400, p=0.6)):
        run_filtered(x, u, t=t * times, **{n: [v] * B for n, v in kw.items()})


@pytest.mark.parametrize("times", [1, 3])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1000, 9001])
def test_sample_filtered_extreme_temperatures(V, dtype, times):
    """From the smallest that fp32 holds to near its largest: one token's share, and equal shares."""
    t = [1e-45, 1e-38, 1e-20, 1e-6, 1e-3, 1e3, 1e6, 1e12, 1e30, 3e38]
    B = len(t) * times
    x = logits(21, B, 2, V, dtype)
    u = uniforms(22, B, 2)
    for kw in ({}, dict(k=7), dict(k=2000), dict(p=0.3), dict(p=0.9), dict(m=0.5), dict(p=0.7, m=0.01), dict(k=400, p=0.6)):
        for shift in (0.0, 1000.0, -1e6):
            run_filtered(x + torch.full((), shift, dtype=dtype, device=DEV), u, t=t * times,
                         **{n: [v] * B for n, v in kw.items()})
