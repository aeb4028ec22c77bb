"""The cache and sampling operators without a GPU: host-side refusals of the C entry points
(each fails a check before any launch) and of the Python binding, and the 64-bit references
the GPU tests compare with, against small worked values."""
import ctypes

import numpy as np
import pytest
import torch

import speculative_decoding_step_pspec_b200 as ps
from speculative_decoding_step_pspec_b200 import _binding as b
from tests import ops_reference as R

FAR = 1 << 32           # spacing of the fake, never dereferenced device arrays: none overlap


def fakes(struct, *fields, **kw):
    a = struct()
    for i, f in enumerate(fields):
        setattr(a, f, FAR * (i + 1))
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def append_args(**kw):
    d = dict(T=4, Hq=4, Hkv=2, D=64, rot=64, dtype=b.PSPEC_BF16, cache=b.PSPEC_CACHE_E2M1, block_size=16,
             num_blocks=8, q_stride=256, k_stride=128, v_stride=128)
    d.update(kw)
    return fakes(b.pspec_append_args, "q", "k", "v", "positions", "slot_mapping", "inv_freq", "k_pages", "v_pages",
                 "k_block_scales", "v_block_scales", "k_scale", "v_scale", "q_out", "k_out", "v_out", "err", **d)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(Hkv=0), dict(D=0), dict(D=24), dict(D=528), dict(rot=3), dict(rot=66), dict(rot=-2),
    dict(block_size=0), dict(num_blocks=0), dict(dtype=7), dict(cache=3), dict(err=None), dict(Hq=0),
    dict(q_out=None), dict(k=None), dict(v=None), dict(positions=None), dict(slot_mapping=None),
    dict(inv_freq=None), dict(k_pages=None), dict(v_block_scales=None), dict(k_stride=127), dict(q_stride=255),
    dict(k=FAR + 1), dict(k_pages=FAR + 8), dict(slot_mapping=FAR * 5 + 4), dict(positions=FAR * 4 + 2),
    dict(q_out=FAR), dict(q_out=FAR + 512), dict(k_out=FAR * 2), dict(k_pages=FAR * 8),
    dict(k_block_scales=FAR * 8 + 16), dict(k_stride=1 << 61), dict(err=FAR * 16 + 1),
    dict(Hq=1 << 27, q_stride=1 << 33), dict(Hkv=1 << 26, k_stride=1 << 32, v_stride=1 << 32),
])
def test_append_refuses(kw):
    assert b.LIB.pspec_append_kv(ctypes.byref(append_args(**kw)), None) == b.PSPEC_ERR_INVALID_ARG
    assert b.LIB.pspec_append_kv(None, None) == b.PSPEC_ERR_INVALID_ARG


def test_append_of_no_rows_is_a_no_op():
    assert b.LIB.pspec_append_kv(ctypes.byref(append_args(T=0, k=None, v=None)), None) == b.PSPEC_OK
    assert ps.pspec_last_launches() == 0


def attend_args(**kw):
    d = dict(T=4, B=2, Hq=4, Hkv=2, D=64, dtype=b.PSPEC_BF16, block_size=16, num_blocks=8, max_blocks=4, scale=0.125,
             q_stride=256)
    d.update(kw)
    return fakes(b.pspec_attend_args, "q", "k_pages", "v_pages", "k_block_scales", "v_block_scales", "k_scale",
                 "v_scale", "block_table", "qsl", "positions", "seq_lens", "row_kind", "out", "lse", "err", **d)


WS = FAR * 64


@pytest.mark.parametrize("kw,status", [(k, b.PSPEC_ERR_INVALID_ARG) for k in (
    dict(T=-1), dict(B=-1), dict(Hkv=0), dict(Hq=3), dict(Hq=1), dict(D=0), dict(block_size=0), dict(num_blocks=0),
    dict(max_blocks=0), dict(dtype=2), dict(err=None), dict(scale=float("nan")), dict(scale=float("inf")),
    dict(q_stride=255), dict(q=None), dict(k_pages=None), dict(v_block_scales=None), dict(block_table=None),
    dict(qsl=None), dict(positions=None), dict(seq_lens=None), dict(out=None), dict(q=FAR + 1),
    dict(out=FAR * 13 + 8), dict(k_pages=FAR * 2 + 8), dict(out=FAR), dict(lse=FAR * 13 + 16), dict(lse=FAR))]
    + [(dict(D=96), b.PSPEC_ERR_UNSUPPORTED), (dict(D=256), b.PSPEC_ERR_UNSUPPORTED)])
def test_attend_refuses(kw, status):
    a = attend_args(**kw)
    assert b.LIB.pspec_attend(ctypes.byref(a), WS, 1 << 40, None) == status
    assert b.LIB.pspec_attend(None, WS, 1 << 40, None) == b.PSPEC_ERR_INVALID_ARG


def test_attend_workspace_checks_and_no_ops():
    n = ps.pspec_attend_workspace_bytes()
    assert n > 0 and n % 256 == 0
    a = attend_args()
    for ws, size in ((None, n), (WS + 128, n), (WS, n - 1)):
        assert b.LIB.pspec_attend(ctypes.byref(a), ws, size, None) == b.PSPEC_ERR_WORKSPACE
    for kw in (dict(T=0), dict(B=0)):
        assert b.LIB.pspec_attend(ctypes.byref(attend_args(**kw)), None, 0, None) == b.PSPEC_OK
        assert ps.pspec_last_launches() == 0


def filter_args(**kw):
    d = dict(B=2, K=3, V=100, ld=100, dtype=b.PSPEC_F32)
    d.update(kw)
    return fakes(b.pspec_filter_args, "logits", "uniforms", "temperature", "top_k", "top_p", "min_p", "tokens",
                 "probs", "err", **d)


@pytest.mark.parametrize("kw,status", [(k, b.PSPEC_ERR_INVALID_ARG) for k in (
    dict(B=-1), dict(K=0), dict(V=0), dict(ld=99), dict(dtype=9), dict(err=None), dict(logits=None),
    dict(uniforms=None), dict(tokens=None), dict(logits=FAR + 2), dict(top_k=FAR * 4 + 1), dict(ld=1 << 60),
    dict(tokens=FAR), dict(probs=FAR * 2 + 8), dict(probs=FAR * 7 + 4), dict(tokens=FAR * 3))]
    + [(dict(V=(1 << 24) + 1, ld=1 << 25), b.PSPEC_ERR_UNSUPPORTED),
       (dict(B=1 << 24, K=16), b.PSPEC_ERR_UNSUPPORTED)])
def test_sample_filtered_refuses(kw, status):
    assert b.LIB.pspec_sample_filtered(ctypes.byref(filter_args(**kw)), None) == status
    assert b.LIB.pspec_sample_filtered(None, None) == b.PSPEC_ERR_INVALID_ARG


def test_sample_filtered_of_an_empty_batch():
    assert b.LIB.pspec_sample_filtered(ctypes.byref(filter_args(B=0, logits=None)), None) == b.PSPEC_OK
    assert ps.pspec_last_launches() == 0


# ------------------------------------------------------------------ the binding's own checks
def rows(T=3, H=2, D=32, dtype=torch.float32):
    return torch.zeros((T, H, D), dtype=dtype)


def append_kw(**kw):
    c = ps.KVCache.zeros(4, 2, 4, 32, device="cpu")
    d = dict(k=rows(), v=rows(), positions=torch.zeros(3, dtype=torch.int32),
             slot_mapping=torch.zeros(3, dtype=torch.int64), k_pages=c.k, v_pages=c.v,
             k_block_scales=c.k_block_scales, v_block_scales=c.v_block_scales,
             err=torch.zeros(1, dtype=torch.int32))
    d.update(kw)
    return d


@pytest.mark.parametrize("kw,error", [
    (dict(), ValueError),                                              # not on a CUDA device
    (dict(k=rows()[0]), ValueError), (dict(k=rows(dtype=torch.float16)), TypeError),
    (dict(v=rows(dtype=torch.bfloat16)), TypeError), (dict(v=rows(T=4)), ValueError),
    (dict(k=rows(D=64)[..., ::2]), ValueError), (dict(k=rows(H=4)[:, ::2]), ValueError),
    (dict(k=rows(T=1).expand(3, 2, 32)), ValueError),
    (dict(positions=torch.zeros(3, dtype=torch.int64)), TypeError),
    (dict(positions=torch.zeros(2, dtype=torch.int32)), ValueError),
    (dict(slot_mapping=torch.zeros(3, dtype=torch.int32)), TypeError),
    (dict(k_pages=torch.zeros((4, 2, 4, 16))), ValueError),
    (dict(k_block_scales=None), TypeError), (dict(q=rows(H=4)), ValueError),
    (dict(q=rows(D=16), q_out=rows(D=16)), ValueError), (dict(q_out=rows()), ValueError),
    (dict(k_scale=torch.ones(3)), ValueError), (dict(k_out=rows(T=2)), ValueError),
    (dict(inv_freq=torch.ones((2, 2))), ValueError), (dict(inv_freq=torch.ones(4, dtype=torch.float64)), TypeError),
])
def test_append_binding_refuses(kw, error):
    with pytest.raises(error):
        b.pspec_append_kv(**append_kw(**kw))


@pytest.mark.parametrize("given", [(), ("err",), ("q",), ("k",), ("err", "v", "q")])
def test_append_allocates_the_outputs_that_are_not_given(monkeypatch, given):
    seen = {}
    monkeypatch.setattr(b, "pspec_append_kv", lambda **kw: seen.update(kw))
    all_outs = dict(q=rows(H=4), k=rows(), v=rows(), err=torch.ones(1, dtype=torch.int32))
    out = {n: all_outs[n] for n in given}
    kw = append_kw()
    cache = ps.KVCache(kw["k_pages"], kw["v_pages"], kw["k_block_scales"], kw["v_block_scales"])
    r = ps.append_kv(kw["k"], kw["v"], kw["positions"], kw["slot_mapping"], cache, q=rows(H=4), want_values=True,
                     out=out or None)
    assert set(r) == {"q", "k", "v", "err"} and set(out) == set(given)
    for n in r:
        arg = seen[n if n == "err" else n + "_out"]
        assert arg is r[n] and (arg is out[n] if n in given else arg.shape == all_outs[n].shape)


def test_append_binding_refuses_pages_of_another_dtype():
    c = ps.KVCache.zeros(4, 2, 4, 32, dtype=torch.bfloat16, device="cpu")
    with pytest.raises(TypeError):
        b.pspec_append_kv(**append_kw(k_pages=c.k, v_pages=c.v, k_block_scales=None, v_block_scales=None))


def attend_kw(**kw):
    c = ps.KVCache.zeros(4, 2, 4, 64, device="cpu")
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    d = dict(q=rows(3, 4, 64), k_pages=c.k, v_pages=c.v, k_block_scales=c.k_block_scales,
             v_block_scales=c.v_block_scales, block_table=i(2, 4), qsl=i(3), positions=i(3), seq_lens=i(2),
             out=rows(3, 4, 64), err=i(1), workspace=torch.zeros(256, dtype=torch.uint8), scale=1.0)
    d.update(kw)
    return d


@pytest.mark.parametrize("kw,error", [
    (dict(), ValueError), (dict(qsl=torch.zeros(2, dtype=torch.int32)), ValueError),
    (dict(seq_lens=torch.zeros(2, dtype=torch.int64)), TypeError), (dict(out=rows(3, 4, 32)), ValueError),
    (dict(block_table=torch.zeros(8, dtype=torch.int32)), ValueError), (dict(lse=torch.zeros((3, 2))), ValueError),
    (dict(row_kind=torch.zeros(3, dtype=torch.int32)), TypeError),
    (dict(k_pages=torch.zeros((4, 2, 4, 64)), v_pages=torch.zeros((4, 2, 4, 64)), k_block_scales=None,
          v_block_scales=None), TypeError),
])
def test_attend_binding_refuses(kw, error):
    with pytest.raises(error):
        b.pspec_attend(**attend_kw(**kw))


@pytest.mark.parametrize("kw,error", [
    (dict(), ValueError), (dict(logits=torch.zeros((2, 10))), ValueError),
    (dict(uniforms=torch.zeros((2, 2))), ValueError), (dict(top_k=torch.zeros(2)), TypeError),
    (dict(temperature=torch.zeros(3)), ValueError), (dict(logits=torch.zeros((2, 3, 20))[..., ::2]), ValueError),
    (dict(tokens=torch.zeros((2, 3), dtype=torch.int64)), TypeError),
])
def test_sample_filtered_binding_refuses(kw, error):
    d = dict(logits=torch.zeros((2, 3, 10)), uniforms=torch.zeros((2, 3)),
             tokens=torch.zeros((2, 3), dtype=torch.int32), err=torch.zeros(1, dtype=torch.int32))
    d.update(kw)
    with pytest.raises(error):
        b.pspec_sample_filtered(**d)


def test_argument_structs_match_the_header():
    """The binding's structs have the sizes that the header's have (LP64: ints then padding to
    the first 8-byte field)."""
    assert ctypes.sizeof(b.pspec_append_args) == 10 * 4 + 3 * 8 + 16 * 8
    assert ctypes.sizeof(b.pspec_attend_args) == 10 * 4 + 8 + 15 * 8
    assert b.pspec_attend_args.scale.offset == 36 and b.pspec_attend_args.q_stride.offset == 40
    assert ctypes.sizeof(b.pspec_filter_args) == 16 + 8 + 8 + 9 * 8


# ------------------------------------------------------------------ the references themselves
def test_reference_grids_against_torch():
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(R.GRID, codes)
    x = np.array([0.0, 0.25, 0.26, 0.75, 0.74, 1.25, 1.75, 2.5, 2.51, 3.5, 5.0, 5.01, 9.0, np.inf])
    assert R.nearest_code(x, R.LEVELS).tolist() == [0, 0, 1, 2, 1, 2, 4, 4, 5, 6, 6, 7, 7, 7]
    y = torch.rand(4096, dtype=torch.float64, generator=torch.Generator().manual_seed(0)) * 500
    y = torch.cat((y, y / 1e5))
    want = y.clamp(max=448).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(R.nearest_code(y.numpy(), R.GRID), want)


def test_reference_quantise_round_trip_and_rotation():
    rng = np.random.default_rng(0)
    x = rng.normal(size=(5, 3, 64))
    g = np.array([1.0, 0.5, 2.0])
    code, sc = R.quantise(x, g)
    v = R.values(code, sc, g)
    step = np.repeat(R.GRID[sc] * g[:, None], 16, axis=-1)      # half of the widest gap is one unit
    assert np.all(np.abs(v - x) <= step * 1.0 + np.abs(x) * 2.0 ** -3)
    again, sc2 = R.quantise(v, g)
    assert np.array_equal(R.unpack(R.pack(code)), code)
    inv = 10000.0 ** (-np.arange(16) / 16)
    for il in (False, True):
        r = R.rotate(x, np.array([0, 1, 7, 100, 10 ** 6]), inv, il)
        np.testing.assert_allclose(np.linalg.norm(r, axis=-1), np.linalg.norm(x, axis=-1), rtol=1e-12)
        assert np.array_equal(r[0], x[0]) and np.array_equal(r[..., 32:], x[..., 32:])


def test_reference_filtered_worked_example():
    x = np.log(np.array([0.1, 0.4, 0.2, 0.2, 0.1]))
    assert R.filtered(x, 0.0, 1, 0, 1, 0)[0] == 0
    assert R.filtered(x, 0.3, 1, 0, 1, 0)[0] == 1
    assert R.filtered(x, 0.99, 1, 2, 1, 0)[0] == 2              # the two largest: ids 1 and 2 (tie: lower id)
    assert R.filtered(x, 0.99, 1, 0, 0.39, 0)[0] == 1           # the first alone reaches 0.39
    assert R.filtered(x, 0.99, 1, 0, 0.61, 0)[0] == 3
    assert R.filtered(x, 0.99, 1, 0, 1, 0.4)[0] == 3            # weights 0.25, 1, 0.5, 0.5, 0.25
    assert R.filtered(x, 0.5, 0, 0, 1, 0)[:2] == (1, 1.0)
