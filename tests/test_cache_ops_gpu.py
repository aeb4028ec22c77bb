"""The cache and sampling operators on the GPU against their 64-bit references."""
import numpy as np
import pytest
import torch

import speculative_decoding_step_pspec_b200 as ps
from speculative_decoding_step_pspec_b200 import _binding as b
from speculative_decoding_step_pspec_b200 import inputs as I
from tests import ops_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
LAST = 1 - 2.0 ** -24


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def random_cache(g, n, H, bs, D, spread=0.5):
    """A 4-bit cache of random content (finite scales)."""
    def r(*s):
        return torch.randint(0, 256, s, generator=g, device=DEV, dtype=torch.int32).to(torch.uint8)

    def scales():
        return (torch.randn((n, H, bs, D // 16), generator=g, device=DEV) * spread - 1).exp().to(torch.float8_e4m3fn)

    def heads():
        return torch.rand((H,), generator=g, device=DEV) + 0.5

    return ps.KVCache(r(n, H, bs, D // 2), r(n, H, bs, D // 2), scales(), scales(), heads(), heads())


# --------------------------------------------------------------------------- append
def append_case(seed, T, Hq, Hkv, D, rot, bs, kind, dtype, interleaved=False, far=5000, offset=0, pad=0.3):
    g = gen(seed)
    W = (Hq + 2 * Hkv) * D + 8
    flat = torch.randn((T * W + 8,), generator=g, device=DEV).to(dtype)
    qkv = flat[offset:offset + T * W].view(T, W)
    q = qkv[:, :Hq * D].view(T, Hq, D)
    k = qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
    v = qkv[:, (Hq + Hkv) * D:(Hq + 2 * Hkv) * D].view(T, Hkv, D)
    blocks = -(-2 * T // bs) + 1
    slots = torch.randperm(blocks * bs, generator=g, device=DEV)[:T]
    slots = torch.where(torch.rand((T,), generator=g, device=DEV) < pad, -1, slots)
    pos = torch.randint(0, far, (T,), generator=g, device=DEV).int()
    inv = (10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / max(rot, 1))).float()
    if kind == "e2m1":
        cache = random_cache(g, blocks, Hkv, bs, D)
    else:
        cache = ps.KVCache(*(torch.randn((blocks, Hkv, bs, D), generator=g, device=DEV).to(dtype) for _ in range(2)))
    return q, k, v, pos, slots, cache, inv


def check_append(q, k, v, pos, slots, cache, inv, interleaved, before, out, live=None):
    """Everything the call may and may not have written."""
    dtype, bs = k.dtype, cache.k.shape[2]
    live = (slots >= 0).cpu().numpy() if live is None else live
    sl, p, f = slots.cpu().numpy()[live], pos.cpu().numpy()[live], R.f64(inv)
    half = R.HALF_STEP[dtype]

    def turned_bound(x):
        # cos and sin rounded to fp32 (2^-24 each), two products and a sum in fp32
        m = np.abs(x)
        h = len(f)
        pair = m.copy()
        ia, ib = (np.arange(0, 2 * h, 2), np.arange(1, 2 * h, 2)) if interleaved else (np.arange(h), np.arange(h, 2 * h))
        pair[..., ia] += m[..., ib]
        pair[..., ib] += m[..., ia]
        return 4 * 2.0 ** -24 * pair

    if q is not None:
        x = R.f64(q)[live]
        want = R.rotate(x, p, f, interleaved)
        got = R.f64(out["q"])
        assert np.all(np.abs(got[live] - want) <= half * 1.01 * np.abs(want) + turned_bound(x))
        assert np.all(got[~live] == -7)
    kr = R.rotate(R.f64(k)[live], p, f, interleaved)
    for w, x in (("k", kr), ("v", R.f64(v)[live])):
        pages = getattr(cache, w).clone()
        if getattr(cache, w + "_block_scales") is None:
            got = R.f64(pages)[sl // bs, :, sl % bs]
            bound = half * 1.01 * np.abs(x) + turned_bound(R.f64(k)[live]) if w == "k" else 0
            assert np.all(np.abs(got - x) <= bound)
            stored = got
        else:
            gs = getattr(cache, w + "_scale")
            gs = np.ones(k.shape[1]) if gs is None else R.f64(gs)
            code, sc = R.quantise(x, gs)
            byte_scales = getattr(cache, w + "_block_scales").view(torch.uint8)
            assert np.array_equal(byte_scales.cpu().numpy()[sl // bs, :, sl % bs], sc), w
            assert np.array_equal(R.unpack(pages.cpu().numpy()[sl // bs, :, sl % bs]), code), w
            stored = R.values(code, sc, gs)
            keep = byte_scales.clone()
            keep[sl // bs, :, sl % bs] = before[w + "_block_scales"].view(torch.uint8)[sl // bs, :, sl % bs]
            assert torch.equal(keep, before[w + "_block_scales"].view(torch.uint8))
        pages[sl // bs, :, sl % bs] = before[w][sl // bs, :, sl % bs]
        assert torch.equal(pages, before[w])                  # every other slot as it was
        if w in out:
            got = R.f64(out[w])
            # level * scale exact, one rounding with the head scale, one to the dtype
            assert np.all(np.abs(got[live] - stored) <= (half + 2.0 ** -24) * 1.01 * np.abs(stored))
            assert np.all(got[~live] == -7)


def run_append(seed, interleaved=False, with_q=True, values=True, **kw):
    q, k, v, pos, slots, cache, inv = append_case(seed, interleaved=interleaved, **kw)
    before = {n: getattr(cache, n).clone() for n in ("k", "v", "k_block_scales", "v_block_scales")
              if getattr(cache, n) is not None}
    out = {}
    if with_q:
        out["q"] = torch.full(q.shape, -7.0, dtype=q.dtype, device=DEV)
    if values:
        out |= {n: torch.full(k.shape, -7.0, dtype=k.dtype, device=DEV) for n in ("k", "v")}
    r = ps.append_kv(k, v, pos, slots, cache, q=q if with_q else None, inv_freq=inv if kw["rot"] else None,
                     interleaved=interleaved, out=out)
    torch.cuda.synchronize()
    assert r["err"].item() == 0 and ps.pspec_last_launches() == 1
    check_append(q if with_q else None, k, v, pos, slots, cache, inv, interleaved, before, out)


@pytest.mark.parametrize("kind", ["e2m1", "rows"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,bs,interleaved", [
    (1, 1, 1, 16, 16, 1, False), (7, 4, 2, 64, 64, 16, False), (33, 3, 3, 80, 40, 20, True),
    (5, 8, 1, 128, 128, 16, False), (64, 16, 8, 64, 32, 4, False), (9, 2, 2, 48, 6, 5, False),
    (6, 5, 5, 112, 112, 32, True), (3, 2, 1, 512, 512, 64, False), (300, 6, 2, 128, 0, 16, False),
    (4, 1, 1, 256, 250, 7, False),
])
def test_append(T, Hq, Hkv, D, rot, bs, interleaved, dtype, kind):
    run_append(T + D, T=T, Hq=Hq, Hkv=Hkv, D=D, rot=rot, bs=bs, kind=kind, dtype=dtype, interleaved=interleaved)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("offset", [1, 2, 3])
def test_append_of_unaligned_rows(offset, dtype):
    run_append(offset, T=20, Hq=4, Hkv=2, D=64, rot=64, bs=16, kind="e2m1", dtype=dtype, offset=offset)
    run_append(offset, T=20, Hq=4, Hkv=2, D=64, rot=32, bs=16, kind="rows", dtype=dtype, offset=offset)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_far_positions_and_a_large_batch(dtype):
    run_append(1, T=4000, Hq=8, Hkv=4, D=128, rot=128, bs=16, kind="e2m1", dtype=dtype, far=2 ** 31 - 1)
    run_append(2, T=1000, Hq=8, Hkv=4, D=64, rot=64, bs=16, kind="rows", dtype=dtype, far=10 ** 6, with_q=False,
               values=False)


def test_append_of_extreme_values():
    """Zero blocks, blocks whose scale rounds to 0 or saturates, infinities, NaN, exact ties."""
    g = gen(3)
    T, H, D, bs = 12, 1, 64, 16
    v = torch.randn((T, H, D), generator=g, device=DEV)
    v[0] = 0
    v[1] *= 1e-5                                                # scale rounds to 0
    v[2] *= 1e-2
    v[3] *= 1e6                                                 # scale saturates at 448
    v[4, 0, 5] = float("inf")
    v[5, 0, 20] = float("nan")
    v[6] = float("nan")
    v[7] = torch.arange(64, device=DEV) % 16 * 0.25 + 0.25       # ties of e2m1 borders (largest 4)
    v[8] = -v[7]
    v[9] = 6 * 2.0 ** -10                                        # largest / 6 on the border to 0
    v[10] = 6 * 3 * 2.0 ** -10                                   # on the border of two subnormal scales
    v[11] = -0.0
    cache = random_cache(g, 2, H, bs, D)
    cache.k_scale = cache.v_scale = None
    slots = torch.arange(T, device=DEV)
    pos = torch.zeros((T,), dtype=torch.int32, device=DEV)
    r = ps.append_kv(v, v, pos, slots, cache, want_values=True)
    torch.cuda.synchronize()
    with np.errstate(invalid="ignore"):
        code, sc = R.quantise(R.f64(v), np.ones(1))
    for w in "kv":
        got_s = getattr(cache, w + "_block_scales").view(torch.uint8)[0, :, :T].transpose(0, 1).cpu().numpy()
        got_c = R.unpack(getattr(cache, w)[0, :, :T].transpose(0, 1).cpu().numpy())
        assert np.array_equal(got_s, sc), np.argwhere(got_s != sc)
        # a block of scale 0 holds zeros of either sign
        mag = np.repeat(sc > 0, 16, -1)
        assert np.array_equal(np.where(mag, got_c, got_c & 7), np.where(mag, code, 0))
        assert torch.isfinite(r[w]).all()


def test_append_flags_bad_slots_and_skips_them():
    q, k, v, pos, slots, cache, inv = append_case(4, T=8, Hq=2, Hkv=2, D=64, rot=64, bs=16, kind="e2m1",
                                                  dtype=torch.bfloat16, pad=0.0)
    total = cache.k.shape[0] * 16
    slots[2], slots[5], slots[6] = -2, total, 2 ** 62
    before = {n: getattr(cache, n).clone() for n in ("k", "v", "k_block_scales", "v_block_scales")}
    out = {"q": torch.full(q.shape, -7.0, dtype=q.dtype, device=DEV)}
    r = ps.append_kv(k, v, pos, slots, cache, q=q, inv_freq=inv, out=out)
    torch.cuda.synchronize()
    assert r["err"].item() == b.PSPEC_DEVERR_BLOCK_RANGE
    live = np.ones(8, bool)
    live[[2, 5, 6]] = False
    check_append(q, k, v, pos, slots, cache, inv, False, before, out, live)


# --------------------------------------------------------------------------- attend
def attend_case(seed, rows, keys, Hq, Hkv, D, bs, dtype, extra_rows=3, spread=0.5, qscale=1.5):
    """Sequences with the given row counts and lengths, positions as a decode step has them."""
    g, rng = gen(seed), np.random.default_rng(seed)
    B = len(rows)
    pages = [-(-n // bs) for n in keys]
    pool = sum(pages) + 2
    ids = rng.permutation(pool)
    table = np.full((B, max(max(pages), 1) + 1), -1)
    at = 0
    for i, n in enumerate(pages):
        table[i, :n] = ids[at:at + n]
        at += n
    qsl = np.concatenate(([0], np.cumsum(rows)))
    T = int(qsl[-1]) + extra_rows
    pos = np.zeros(T, np.int64)
    for i, (r, n) in enumerate(zip(rows, keys)):
        pos[qsl[i]:qsl[i + 1]] = n - r + np.arange(r)
    q = (torch.randn((T, Hq, D), generator=g, device=DEV) * qscale).to(dtype)
    return dict(q=q, cache=random_cache(g, pool, Hkv, bs, D, spread), table=table, qsl=qsl, pos=pos,
                lens=np.array(keys), bs=bs)


def i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32, device=DEV)


def run_attend(c, scale=None, row_kind=None, err=0, q=None, workspace=None, either=()):
    q = c["q"] if q is None else q
    T, Hq, D = q.shape
    scale = D ** -0.5 if scale is None else scale
    out = dict(out=torch.full((T, Hq, D), -7.0, dtype=q.dtype, device=DEV),
               lse=torch.full((T, Hq), -7.0, device=DEV))
    kind = None if row_kind is None else torch.as_tensor(row_kind, dtype=torch.uint8, device=DEV)
    r = ps.attend(q, c["cache"], i32(c["table"]), i32(c["qsl"]), i32(c["pos"]), i32(c["lens"]), scale=scale,
                  row_kind=kind, out=out, workspace=workspace)
    torch.cuda.synchronize()
    assert r["err"].item() == err
    assert ps.pspec_last_launches() == 1
    check_attend(c, q, scale, row_kind, out, either)
    return out


def check_attend(c, q, scale, row_kind, out, either=()):
    """either: rows that two sequences claim (a malformed qsl), which may hold either's result."""
    D = q.shape[2]
    kv, vv = (R.cache_values(c["cache"], w) for w in "kv")
    f32 = float(np.float32(scale))
    want, lse, seen, a, vmax = R.attend(R.f64(q), kv, vv, c["table"], c["qsl"], c["pos"], c["lens"], f32, c["bs"],
                                        row_kind)
    bound, d = R.attend_bounds(q.dtype, D, want, a, vmax)
    got, got_lse = R.f64(out["out"]), R.f64(out["lse"])
    for t in either:
        got[t], got_lse[t] = want[t], lse[t]
    assert np.all(got[~seen] == -7) and np.all(got_lse[~seen] == -7)
    bad = np.abs(got - want) > bound
    assert not bad[seen].any(), (np.argwhere(bad & seen[:, None, None])[:5], np.abs(got - want)[seen].max())
    empty = np.isinf(lse) & seen[:, None]
    assert np.all(got[empty] == 0) and np.all(got_lse[empty] == -np.inf)
    full = seen[:, None] & ~empty
    lse_bound = d + 2.0 ** -22 * (np.abs(np.where(full, lse, 0)) + a + 16)
    assert np.all(np.abs(got_lse[full] - lse[full]) <= lse_bound[full])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows,keys,Hq,Hkv,bs", [
    ([1], [1], 1, 1, 16), ([1], [17], 4, 4, 16), ([1, 1, 1], [5, 64, 65], 8, 2, 16),
    ([8], [300], 8, 1, 16), ([3, 0, 7, 1], [3, 40, 129, 1000], 6, 2, 32), ([2, 5], [63, 200], 7, 7, 4),
    ([1, 2], [90, 33], 5, 1, 1), ([40, 17], [40, 100], 4, 2, 20), ([1, 15, 2], [500, 15, 48], 16, 1, 48),
    ([1, 1], [0, 70], 2, 2, 16), ([130], [130], 8, 4, 64), ([1] * 40, list(range(1, 161, 4)), 2, 1, 16),
])
def test_attend(rows, keys, Hq, Hkv, bs, D, dtype):
    run_attend(attend_case(len(rows) + D + bs, rows, keys, Hq, Hkv, D, bs, dtype))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,rows,keys,Hq,Hkv", [(128, [1], [20000], 4, 1), (64, [4, 1], [9000, 12000], 8, 2)])
def test_attend_long_contexts_split_over_the_gpu(D, rows, keys, Hq, Hkv, dtype):
    run_attend(attend_case(7, rows, keys, Hq, Hkv, D, 16, dtype))


def wide_heads(rows, group, D):
    """As many kv heads as it takes for the rows' tiles to fill half of the GPU, and no fewer."""
    per_seq = (sum(rows) + 3) * group / len(rows)
    return -(-80 // (len(rows) * max(1, int(-(-per_seq // 128)))))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows,keys,group,bs", [
    ([40], [40], 1, 16), ([33], [64], 1, 16), ([64, 64], [65, 700], 1, 16), ([128], [300], 1, 32),
    ([129, 1], [129, 1500], 2, 16), ([20, 30, 1, 90], [20, 300, 1, 91], 7, 48), ([70], [2000], 8, 20),
    ([100, 0, 60], [100, 50, 64], 1, 1), ([300, 200], [301, 500], 3, 64), ([8] * 30, [13 * i + 8 for i in range(30)], 8, 16),
])
def test_attend_many_rows(rows, keys, group, bs, D):
    """Rows enough for the wide tiles: parts of a tile, several of them, tiles split over CTAs."""
    H = wide_heads(rows, group, D)
    run_attend(attend_case(sum(rows) + D, rows, keys, H * group, H, D, bs, torch.bfloat16))


@pytest.mark.parametrize("D", [64, 128])
def test_attend_many_rows_masks_and_scores(D):
    """Wide tiles with rows that see nothing, scattered positions, rejected rows, missing pages,
    scores far apart, a negative scale, queries that are not aligned, and keys behind every
    position that hold anything."""
    rows = [60, 50, 0, 45]
    H = wide_heads(rows, 2, D)
    c = attend_case(30 + D, rows, [700, 50, 9, 333], 2 * H, H, D, 16, torch.bfloat16, qscale=8.0)
    g = np.random.default_rng(3)
    c["pos"][:60] = g.integers(-2, 720, 60)
    c["pos"][60:70] = -1
    run_attend(c)
    run_attend(c, scale=-0.2)
    run_attend(c, row_kind=g.integers(0, 5, len(c["pos"])).astype(np.uint8))
    T, Hq, _ = c["q"].shape
    wide = torch.randn((T, Hq * D + 24), device=DEV, generator=gen(1)).to(torch.bfloat16)
    run_attend(c, q=wide[:, 1:1 + Hq * D].view(T, Hq, D))
    c["table"][0, 3], c["table"][3, 20] = -1, c["cache"].k.shape[0]
    run_attend(c, err=b.PSPEC_DEVERR_BLOCK_RANGE)
    rows = [50, 40]
    H = wide_heads(rows, 2, D)
    c = attend_case(31 + D, rows, [500, 90], 2 * H, H, D, 16, torch.bfloat16)
    c["pos"][:50], c["pos"][50:90] = np.arange(50) + 30, np.arange(40)
    want = run_attend(c)
    for w in ("k_block_scales", "v_block_scales"):
        sc = getattr(c["cache"], w).view(torch.uint8)
        keep = torch.zeros(sc.shape[0], sc.shape[2], dtype=torch.bool, device=DEV)
        for i, n in ((0, 80), (1, 40)):
            for j in range(n):
                keep[c["table"][i, j // 16], j % 16] = True
        sc.copy_(torch.where(keep[:, None, :, None], sc, 0x7F if w[0] == "k" else 0xFF))
    got = run_attend(c)
    assert torch.equal(got["out"][:90], want["out"][:90]) and torch.equal(got["lse"][:90], want["lse"][:90])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_attend_large_scores_and_small(dtype):
    """Scores far apart (a running maximum that moves often) and all but equal, negative scale."""
    run_attend(attend_case(8, [3, 1], [700, 260], 4, 2, 64, 16, dtype, qscale=40.0))
    run_attend(attend_case(9, [3, 1], [700, 260], 4, 2, 128, 16, dtype, qscale=1e-6))
    run_attend(attend_case(10, [2], [300], 2, 2, 128, 16, dtype), scale=-0.3)
    run_attend(attend_case(11, [2], [300], 2, 2, 64, 16, dtype), scale=0.0)
    c = attend_case(12, [4], [200], 2, 1, 64, 16, dtype)
    c["q"][0] = 0
    c["q"][1] *= 1e30
    run_attend(c, scale=1e-30)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_attend_masks(dtype):
    """Rows that see nothing, rows that see one key or all, positions past the length, rows of
    rejected and padding kind, sequences without keys or rows."""
    c = attend_case(13, [6, 4, 0, 3], [50, 0, 9, 400], 4, 2, 64, 16, dtype)
    c["pos"][:6] = [-1, 0, 49, 50, 2 ** 31 - 1, -5]
    run_attend(c)
    kind = np.zeros(len(c["pos"]), np.uint8)
    kind[[1, 5, 11]] = [3, 4, 3]
    kind[[2, 3]] = [1, 2]
    run_attend(c, row_kind=kind)
    run_attend(c, row_kind=np.full(len(c["pos"]), 3, np.uint8))


def test_attend_unseen_keys_may_hold_anything():
    """NaN scales and other garbage in keys past every row's position, past the length and in
    pages of no sequence do not reach the outputs."""
    for D in (64, 128):
        c = attend_case(14, [3, 2], [100, 37], 4, 2, D, 16, torch.bfloat16)
        c["pos"][:3], c["pos"][3:5] = [40, 41, 42], [10, 9]
        want = run_attend(c)
        for w in ("k_block_scales", "v_block_scales"):
            sc = getattr(c["cache"], w).view(torch.uint8)
            keep = torch.zeros(sc.shape[0], sc.shape[2], dtype=torch.bool, device=DEV)
            for i, n in ((0, 43), (1, 11)):
                for j in range(n):
                    keep[c["table"][i, j // 16], j % 16] = True
            sc.copy_(torch.where(keep[:, None, :, None], sc, 0x7F if w[0] == "k" else 0xFF))
        got = run_attend(c)
        assert torch.equal(got["out"][:5], want["out"][:5]) and torch.equal(got["lse"][:5], want["lse"][:5])


def test_attend_flags_bad_tables_lengths_and_offsets():
    c = attend_case(15, [2, 3, 1], [100, 60, 30], 4, 2, 64, 16, torch.bfloat16)
    c["table"][0, 2] = -1                                       # a page that is not there
    c["table"][1, 0] = c["cache"].k.shape[0]
    run_attend(c, err=b.PSPEC_DEVERR_BLOCK_RANGE)
    c = attend_case(16, [2, 3], [100, 60], 4, 2, 64, 16, torch.bfloat16)
    c["table"] = c["table"][:, :7].copy()
    c["lens"] = np.array([2 ** 31 - 1, -3])
    c["pos"][:2] = [2 ** 31 - 1, 50]
    run_attend(c, err=b.PSPEC_DEVERR_BLOCK_RANGE)
    c = attend_case(17, [2, 3, 2], [100, 60, 20], 4, 2, 64, 16, torch.bfloat16)
    c["qsl"] = np.array([0, 2, 1, 3])                           # sequence 1 runs backwards
    run_attend(c, err=b.PSPEC_DEVERR_LAYOUT, either=[1])
    c["qsl"] = np.array([-1, 2, 5, 2 ** 30])
    run_attend(c, err=b.PSPEC_DEVERR_LAYOUT)


def test_attend_strided_queries_and_many_sequences():
    c = attend_case(18, [2] * 300, [int(x) for x in np.random.default_rng(1).integers(2, 90, 300)], 4, 1, 64, 16,
                    torch.bfloat16)
    run_attend(c)
    T = len(c["pos"])
    wide = torch.randn((T, 4 * 64 + 24), device=DEV, generator=gen(1)).to(torch.bfloat16)
    for off in (0, 1, 8):
        run_attend(c, q=wide[:, off:off + 256].view(T, 4, 64))


def test_attend_is_deterministic_and_leaves_its_workspace_clean():
    ws = ps.attend_workspace()
    small = attend_case(19, [1, 3], [2000, 700], 8, 2, 128, 16, torch.bfloat16)
    large = attend_case(20, [8] * 6, [3000, 10, 64, 65, 900, 8], 8, 2, 64, 16, torch.bfloat16)
    first = run_attend(small, workspace=ws)
    run_attend(large, workspace=ws)
    again = run_attend(small, workspace=ws)
    assert torch.equal(first["out"], again["out"]) and torch.equal(first["lse"], again["lse"])


# --------------------------------------------------------------------------- sample
def run_filtered(x, u, t=None, k=None, p=None, m=None, err=0, flat=False):
    """Both outputs of every row against the reference; draws whose uniform lies within 1e-9 of a
    border are left out (they are counted and must be few)."""
    B, K, V = x.shape
    dev = lambda v, dt: None if v is None else torch.as_tensor(np.asarray(v), dtype=dt, device=DEV)  # noqa: E731
    r = ps.sample_filtered(x, u, temperature=dev(t, torch.float32), top_k=dev(k, torch.int32),
                           top_p=dev(p, torch.float32), min_p=dev(m, torch.float32), want_probs=True)
    torch.cuda.synchronize()
    assert r["err"].item() == err and ps.pspec_last_launches() == 1
    near = 0
    xn, un = x.float().cpu().numpy(), u.cpu().numpy().astype(np.float64)
    f = lambda v, i, d: d if v is None else float(np.float32(v[i]))  # noqa: E731
    for i in range(B):
        for j in range(K):
            tok, pr, margin = R.filtered(xn[i, j], un[i, j], f(t, i, 1.0), 0 if k is None else int(k[i]),
                                         f(p, i, 1.0), f(m, i, 0.0))
            got, gp = r["tokens"][i, j].item(), r["probs"][i, j].item()
            if margin < 1e-9 and got != tok:
                near += 1
                continue
            assert got == tok, (i, j, got, tok, margin, f(t, i, 1.0), k and k[i], p and p[i], m and m[i])
            assert abs(gp - pr) <= 2.0 ** -24 * 1.01 * pr + 1e-11, (i, j, gp, pr)
    assert near <= B * K // 50
    return r


def logits(seed, B, K, V, dtype, sigma=3.0, pad=0, offset=0):
    g = gen(seed)
    ld = V + pad
    flat = (torch.randn((B * K * ld + 8,), generator=g, device=DEV) * sigma).to(dtype)
    return flat[offset:offset + B * K * ld].view(B, K, ld)[..., :V]


def uniforms(seed, B, K):
    return torch.rand((B, K), generator=gen(seed), device=DEV).clamp_(max=LAST)


FILTERS = {
    "off": {}, "temperature": dict(t=0.7), "hot": dict(t=5.0), "greedy": dict(t=0.0), "k1": dict(k=1),
    "k": dict(k=40), "k_large": dict(k=5000, t=1.3), "k_all": dict(k=1 << 30), "p": dict(p=0.9),
    "p_small": dict(p=1e-4), "p_zero": dict(p=0.0), "p_near_1": dict(p=LAST, t=2.0), "m": dict(m=0.05),
    "m_one": dict(m=1.0), "m_over": dict(m=1.5), "k_p": dict(k=100, p=0.8), "k_p_large": dict(k=9000, p=0.97, t=2.0),
    "p_m": dict(p=0.95, m=0.01), "all": dict(t=0.8, k=300, p=0.95, m=0.002), "k_m": dict(k=60, m=0.1),
    "negative_k": dict(k=-5, p=2.0, m=-1.0),
}


@pytest.mark.parametrize("name", FILTERS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [1, 2, 31, 100, 256, 513, 2048, 2049, 40001])
def test_sample_filtered(V, dtype, name):
    B, K = 3, 2
    kw = {n: [v] * B for n, v in FILTERS[name].items()}
    run_filtered(logits(V, B, K, V, dtype), uniforms(V + 1, B, K), **kw)


@pytest.mark.parametrize("name", ["off", "k", "p", "k_p_large", "all"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_sample_filtered_large_vocabulary(dtype, name):
    B, K, V = 2, 3, 201088
    kw = {n: [v] * B for n, v in FILTERS[name].items()}
    run_filtered(logits(5, B, K, V, dtype), uniforms(6, B, K), **kw)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,K,V", [(20, 2, 40001), (301, 7, 20), (36, 1, 2050), (400, 4, 5003), (14, 3, 151936)])
def test_sample_filtered_many_rows(B, K, V, dtype):
    """Batches past the few rows whose slices live in shared memory, every request its own."""
    g = np.random.default_rng(B + V)
    x = logits(B + 1, B, K, V, dtype, pad=5)
    x[:, :, 3::7] -= 4.0
    for i in range(2):
        kw = dict(t=g.choice([0.3, 0.8, 1.5, 3.0, 0.0], B), k=g.choice([0, 0, 1, 50, 900, 1500, V], B),
                  p=g.choice([1.0, 0.3, 0.9, 0.99, 0.9999], B), m=g.choice([0.0, 0.0, 1e-6, 1e-3, 0.2, 1.0], B))
        run_filtered(x, uniforms(B + V + i, B, K), **kw)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B", [3, 40])
@pytest.mark.parametrize("V", [9001, 70000])
def test_sample_filtered_large_nuclei(V, B, dtype):
    """Top-p sets of thousands of tokens, alone and beside a min-p that ends sooner, later or
    about there, in rows of a narrow and a wide spread."""
    x = logits(V + B, B, 1, V, dtype, sigma=2.0)
    x[::2] *= 0.02
    x[1::3] += 300.0
    u = uniforms(V + B + 1, B, 1)
    for p in (0.5, 0.9, 0.995):
        run_filtered(x, u, p=[p] * B, t=[1.2] * B)
        for m in (1e-9, 2e-4, 1e-2, 0.9):
            run_filtered(x, u, p=[p] * B, t=[1.2] * B, m=[m] * B)


def test_sample_filtered_past_the_shared_memory():
    """A vocabulary whose slices are read from global memory."""
    V = 1200000
    for kw in ({}, dict(k=[50]), dict(p=[0.9])):
        run_filtered(logits(7, 1, 2, V, torch.float32), uniforms(8, 1, 2), **kw)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad,offset", [(3, 0), (8, 0), (0, 1), (5, 3)])
def test_sample_filtered_padded_and_unaligned_rows(pad, offset, dtype):
    x = logits(9, 4, 3, 5001, dtype, pad=pad, offset=offset)
    run_filtered(x, uniforms(10, 4, 3), t=[0.5, 1, 2, 0], k=[0, 70, 0, 0], p=[0.9, 1, 0.99, 1], m=[0, 0, 0.01, 0])


def test_sample_filtered_ties():
    """Few distinct logits: cuts inside a class of ties larger than one CTA sorts keep its lowest
    ids, whatever the filter."""
    g = gen(11)
    V = 30011
    x = torch.randint(0, 3, (6, 2, V), generator=g, device=DEV).float()
    u = uniforms(12, 6, 2)
    run_filtered(x, u, k=[1, 4000, 15000, 25000, 29000, 0], p=[1, 1, 1, 1, 1, 0.3])
    run_filtered(x, u, p=[0.01, 0.2, 0.5, 0.7, 0.97, 0.9999])
    run_filtered(x, u, k=[5000, 6000, 12000, 20000, 25000, 29999], p=[0.5, 0.9, 0.99, 0.8, 0.3, 0.7])
    same = torch.full((3, 1, V), -2.5, device=DEV, dtype=torch.bfloat16)
    run_filtered(same, uniforms(13, 3, 1), k=[0, 9000, 0], p=[1, 1, 0.25], m=[0, 0, 1.0])
    zeros = torch.zeros((1, 2, 5000), device=DEV)
    zeros[:, :, ::2] = -0.0                                     # -0 ties with 0
    run_filtered(zeros, torch.tensor([[0.1, 0.999]], device=DEV), k=[3001])


def test_sample_filtered_infinities_and_nan():
    V = 3000
    x = logits(14, 6, 2, V, torch.float32)
    x[0] = -float("inf")                                        # no mass: token 0, probability 0
    x[1, :, 10:] = -float("inf")                                # masked vocabulary
    x[2, 0, 77] = x[2, 0, 2900] = float("inf")                  # shares of the infinite
    x[2, 1] = float("nan")
    x[3, :, ::2] = float("nan")
    x[4] = -float("inf")
    x[4, :, 1234] = -1e38
    x[5] *= 1e37
    u = uniforms(15, 6, 2)
    for kw in ({}, dict(k=[5] * 6), dict(p=[0.5] * 6), dict(t=[0.0] * 6), dict(m=[0.3] * 6), dict(k=[2500] * 6)):
        r = run_filtered(x, u, **kw)
        assert r["tokens"][0].tolist() == [0, 0] and r["probs"][0].tolist() == [0, 0]
        assert r["tokens"][4].tolist() == [1234, 1234]


def test_sample_filtered_extreme_uniforms_and_bad_parameters():
    x = logits(16, 4, 2, 4000, torch.bfloat16)
    edge = torch.tensor([[0.0, LAST]] * 4, device=DEV)
    run_filtered(x, edge, t=[1, 0.3, 1, 1], k=[0, 0, 30, 0], p=[1, 1, 1, 0.9])
    nan, inf = float("nan"), float("inf")
    u = uniforms(17, 4, 2)
    r = ps.sample_filtered(x, u, temperature=torch.tensor([nan, -1.0, inf, 1.0], device=DEV),
                           top_p=torch.tensor([0.9, 0.9, 0.9, nan], device=DEV),
                           min_p=torch.tensor([0.0, 0.0, nan, 0.0], device=DEV))
    want = ps.sample_filtered(x, u, top_p=torch.tensor([0.9, 0.9, 0.9, 1.0], device=DEV))
    torch.cuda.synchronize()
    assert r["err"].item() == b.PSPEC_DEVERR_PARAM_RANGE and torch.equal(r["tokens"], want["tokens"])


def test_sample_filtered_follows_the_distribution():
    """Evenly spaced uniforms hit every kept token in proportion to its mass."""
    V, n = 50, 20000
    x = logits(18, 1, 1, V, torch.float32, sigma=1.0)
    u = ((torch.arange(n, device=DEV) + 0.5) / n).view(1, n)
    r = ps.sample_filtered(x.expand(1, 1, V).repeat(1, n, 1), u, top_k=torch.tensor([20], device=DEV, dtype=torch.int32))
    got = np.bincount(r["tokens"].view(-1).cpu().numpy(), minlength=V) / n
    w = np.exp(R.f64(x)[0, 0])
    w[np.argsort(-w)[20:]] = 0
    assert np.all(np.abs(got - w / w.sum()) <= 1.01 / n + 1e-6)


def test_sample_filtered_agrees_with_sample_drafts_and_repeats():
    x = logits(19, 16, 7, 20000, torch.bfloat16)
    u = uniforms(20, 16, 7)
    a = ps.sample_filtered(x, u, want_probs=True)
    again = ps.sample_filtered(x, u, want_probs=True)
    d = ps.sample_drafts(x, u, want_probs=True)
    g = ps.sample_filtered(x, u, temperature=torch.zeros(16, device=DEV))
    greedy = ps.sample_drafts(x)
    torch.cuda.synchronize()
    assert torch.equal(a["tokens"], again["tokens"]) and torch.equal(a["probs"], again["probs"])
    assert (a["tokens"] != d["draft_tokens"]).sum() <= 2        # fp32 borders of sample_drafts
    assert torch.equal(g["tokens"], greedy["draft_tokens"])


# --------------------------------------------------------------------------- together
def decode_step(w, seed=0, Hq=8, Hkv=2, D=64, layers=None):
    """A drafter layer around the framework's draft batch: build -> append -> attend -> logits ->
    draw, with a random projection; returns the callable and what it works on."""
    inp = I.build_inputs(w, DEV)
    g = gen(seed)
    H, V = w.H, w.V
    wqkv = (torch.randn((H, (Hq + 2 * Hkv) * D), generator=g, device=DEV) / H ** 0.5).to(w.dtype)
    wout = (torch.randn((Hq * D, V), generator=g, device=DEV) / (Hq * D) ** 0.5).to(w.dtype)
    nblk = int(inp["block_table"].max().item()) + 1
    cache = random_cache(g, nblk, Hkv, w.block_size, D)
    inv = (10000.0 ** (-torch.arange(0, D, 2, device=DEV, dtype=torch.float64) / D)).float()
    u = torch.rand((w.B, w.K), generator=g, device=DEV).clamp_(max=LAST)
    temperature = torch.full((w.B,), 0.9, device=DEV)
    top_k = torch.full((w.B,), 50, dtype=torch.int32, device=DEV)
    ws = ps.attend_workspace()
    build = {k: inp[k] for k in ("K", "block_size", "mask_id", "pad_id", "T_cap", "qsl_in", "verify_tokens",
                                 "verify_pos", "accepted_len", "bonus", "block_table", "verify_hidden", "h_shared")}

    def step():
        d = ps.build_draft_batch(**build)
        qkv = d["draft_hidden"] @ wqkv
        T = qkv.shape[0]
        q = qkv[:, :Hq * D].view(T, Hq, D)
        k = qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
        v = qkv[:, (Hq + Hkv) * D:].view(T, Hkv, D)
        a = ps.append_kv(k, v, d["draft_pos"], d["slot_mapping"], cache, q=q, inv_freq=inv,
                         out=dict(q=torch.zeros((T, Hq, D), dtype=w.dtype, device=DEV)))
        o = ps.attend(a["q"], cache, inp["block_table"], d["qsl_out"], d["draft_pos"], d["seq_lens_out"],
                      row_kind=d["row_kind"], workspace=ws,
                      out=dict(out=torch.zeros((T, Hq, D), dtype=w.dtype, device=DEV),
                               lse=torch.zeros((T, Hq), device=DEV)))
        x = (o["out"].view(T, -1)[d["sample_idx"].view(-1).long()] @ wout).view(w.B, w.K, V)
        s = ps.sample_filtered(x, u, temperature=temperature, top_k=top_k, want_probs=True)
        return dict(batch=d, q=q, k=k, v=v, append=a, attend=o, logits=x, sample=s)

    return step, inp, cache, inv, u


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_decode_step_runs_together(dtype):
    """The draft batch's slots, positions, offsets, lengths and row kinds go into the three
    operators as they are; each one's output is checked from the inputs that it got."""
    w = I.scaled(I.C64, B=5, V=1000, H=64, ctx="uniform", ctx_args=(20, 300), dtype=dtype)
    step, inp, cache, inv, u = decode_step(w)
    before = {n: getattr(cache, n).clone() for n in ("k", "v", "k_block_scales", "v_block_scales")}
    r = step()
    torch.cuda.synchronize()
    d = r["batch"]
    assert all(x["err"].item() == 0 for x in (d, r["append"], r["attend"], r["sample"]))
    live = (d["slot_mapping"] >= 0).cpu().numpy()
    got = {"q": torch.where(torch.as_tensor(live, device=DEV)[:, None, None], r["append"]["q"], -7.0)}
    check_append(r["q"], r["k"], r["v"], d["draft_pos"], d["slot_mapping"], cache, inv, False, before, got)
    kind = d["row_kind"].cpu().numpy()
    assert np.array_equal(live, kind <= 2)
    c = dict(cache=cache, table=inp["block_table"].cpu().numpy(), qsl=d["qsl_out"].cpu().numpy(),
             pos=d["draft_pos"].cpu().numpy(), lens=d["seq_lens_out"].cpu().numpy(), bs=w.block_size)
    rows = torch.as_tensor(live, device=DEV)
    out = dict(out=torch.where(rows[:, None, None], r["attend"]["out"], -7.0),
               lse=torch.where(rows[:, None], r["attend"]["lse"], -7.0))
    check_attend(c, r["append"]["q"], r["q"].shape[2] ** -0.5, kind, out)
    run_filtered(r["logits"], u, t=[0.9] * w.B, k=[50] * w.B)


def test_a_decode_step_in_a_graph_and_on_another_stream():
    """Captured once and replayed (the cache and the inputs keep their storage), and launched on a
    side stream: the same results as eagerly."""
    w = I.scaled(I.C64, B=4, V=3000, H=64, ctx="uniform", ctx_args=(20, 500))
    step, inp, cache, inv, u = decode_step(w)
    start = {n: getattr(cache, n).clone() for n in ("k", "v", "k_block_scales", "v_block_scales")}

    def reset():
        for n, t in start.items():
            getattr(cache, n).view(torch.uint8).copy_(t.view(torch.uint8))

    eager = step()
    torch.cuda.synchronize()
    want = {n: getattr(cache, n).clone() for n in start}
    s = torch.cuda.Stream()
    reset()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        side = step()
    s.synchronize()
    for a, bb in ((eager, side),):
        assert torch.equal(a["attend"]["out"], bb["attend"]["out"])
        assert torch.equal(a["sample"]["tokens"], bb["sample"]["tokens"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for _ in range(3):
        reset()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(eager["attend"]["out"], captured["attend"]["out"])
    assert torch.equal(eager["sample"]["tokens"], captured["sample"]["tokens"])
    assert torch.equal(eager["append"]["q"], captured["append"]["q"])
    for n in start:
        assert torch.equal(getattr(cache, n).view(torch.uint8), want[n].view(torch.uint8))


def test_what_a_call_allocates_belongs_to_its_stream():
    """Calls on a side stream, by object and by handle, with nothing given: their zeros, outputs and
    temporary workspaces are that stream's, whatever the current stream does meanwhile."""
    c = attend_case(23, [1] * 12, [900] * 12, 8, 2, 64, 16, torch.bfloat16)
    x, u = logits(24, 6, 2, 3001, torch.float32), uniforms(25, 6, 2)
    args = (c["q"], c["cache"], i32(c["table"]), i32(c["qsl"]), i32(c["pos"]), i32(c["lens"]))
    want, drawn = ps.attend(*args), ps.sample_filtered(x, u, want_probs=True)
    torch.cuda.synchronize()
    n = int(c["qsl"][-1])
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        for _ in range(10):
            got = ps.attend(*args, stream=stream)
            tok = ps.sample_filtered(x, u, want_probs=True, stream=stream)
            torch.full((ps.pspec_attend_workspace_bytes(),), 255, dtype=torch.uint8, device=DEV)   # over what was let go
        torch.cuda.synchronize()
        assert got["err"].item() == 0 and tok["err"].item() == 0
        assert torch.equal(got["out"][:n], want["out"][:n]) and torch.equal(tok["tokens"], drawn["tokens"])


def test_two_graphs_and_two_prepared_calls_side_by_side():
    """Two captured graphs with workspaces of their own, replayed on two streams at once."""
    cs = [attend_case(26 + i, [4, 1, 9], [700, 90, 2000], 8, 2, D, 16, torch.bfloat16) for i, D in enumerate((64, 128))]
    want, graphs = [], []
    for c in cs:
        args = (c["q"], c["cache"], i32(c["table"]), i32(c["qsl"]), i32(c["pos"]), i32(c["lens"]))
        call, o = ps.prepare_attend(*args, want_lse=True)
        call()
        torch.cuda.synchronize()
        want.append({k: v.clone() for k, v in o.items()})
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        o["out"].fill_(-3)
        graphs.append((g, o, call))
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(20):
        for (g, _, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    n = 14
    for (_, o, _), w in zip(graphs, want):
        assert torch.equal(o["out"][:n], w["out"][:n]) and torch.equal(o["lse"][:n], w["lse"][:n])


def test_two_streams_with_their_own_workspaces():
    c1 = attend_case(21, [1] * 8, [3000] * 8, 8, 2, 128, 16, torch.bfloat16)
    c2 = attend_case(22, [8] * 4, [2000, 100, 900, 8], 8, 2, 64, 16, torch.bfloat16)
    streams = [torch.cuda.Stream() for _ in range(2)]
    calls = []
    for c in (c1, c2):
        out = dict(out=torch.empty_like(c["q"]))
        call, o = ps.prepare_attend(c["q"], c["cache"], i32(c["table"]), i32(c["qsl"]), i32(c["pos"]), i32(c["lens"]),
                                    out=out)
        calls.append((call, o))
    for call, _ in calls:
        call()
    torch.cuda.synchronize()
    want = [o["out"].clone() for _, o in calls]
    for _ in range(20):
        for (call, _), s in zip(calls, streams):
            call(s)
    torch.cuda.synchronize()
    n = [int(c["qsl"][-1]) for c in (c1, c2)]
    assert all(torch.equal(o["out"][:m], w[:m]) for (_, o), w, m in zip(calls, want, n))


def test_prepared_calls_see_new_contents():
    x, u = logits(23, 2, 3, 5000, torch.bfloat16).contiguous(), uniforms(24, 2, 3)
    call, o = ps.prepare_sample_filtered(x, u, top_k=torch.tensor([3, 0], dtype=torch.int32, device=DEV))
    call()
    torch.cuda.synchronize()
    x.copy_(logits(25, 2, 3, 5000, torch.bfloat16))
    call()
    torch.cuda.synchronize()
    want = ps.sample_filtered(x, u, top_k=torch.tensor([3, 0], dtype=torch.int32, device=DEV))
    assert torch.equal(o["tokens"], want["tokens"])
