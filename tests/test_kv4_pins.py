"""CPU: the 4-bit cache's oracle against hand-worked values and its definitions, the sizing
and the refusals of the C ABI (which come before any launch)."""

import ctypes

import numpy as np
import pytest
import torch

import block_sparse_attention_video_b200 as F
from block_sparse_attention_video_b200 import kv4 as K
from oracle import kv4_oracle as O


def test_e4m3_table_is_torchs():
    t = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, O.E4M3)


def test_quantize_hand_worked():
    # largest magnitude 12 -> scale 2; ties go to the even code: 0.5 (0.25 of the scale) -> 0,
    # 1.5 (0.75) -> 1.0, 2.5 (1.25) -> 1.0, 3.5 (1.75) -> 2.0, 5 (2.5) -> 2, 7 (3.5) -> 4, 10 (5) -> 4
    x = np.array([12, 0.5, 1.5, 2.5, 3.5, 5, 7, 10, -0.5, -1.5, -2.5, -3.5, -5, -7, -10, -12.0])[None]
    c, s = O.quantize(x)
    assert O.E4M3[s[0, 0]] == 2.0
    want = np.array([12, 0, 2, 2, 4, 4, 8, 8, 0, -2, -2, -4, -4, -8, -8, -12.0])
    assert np.array_equal(O.dequantize(c, s)[0], want)


def test_quantize_scale_rounds_to_even_and_saturates():
    x = np.zeros((3, 16))
    x[0, 0] = 6 * 1.0625          # between 1 and 1.125: 1 has the even code
    x[1, 0] = 6 * 448 * 4         # above the largest scale
    x[2, 0] = 6 * 2.0 ** -10      # half the smallest scale: 0, and with it every code
    c, s = O.quantize(x[:, None, :])
    assert O.E4M3[s[0, 0, 0]] == 1.0 and O.E4M3[s[1, 0, 0]] == 448.0 and s[2, 0, 0] == 0
    assert O.dequantize(c, s)[1, 0, 0] == 6 * 448 and not c[2].any()


def test_quantize_error_bound():
    # half a step of E2M1 relative to the group's scale (1 at the top: between 4 and 6), and the
    # scale itself off by at most 2^-4: |x^ - x| <= s (1 + 6/16)
    x = np.random.default_rng(0).standard_normal((64, 2, 64)).astype(np.float32)
    c, s = O.quantize(x)
    err = np.abs(O.dequantize(c, s) - x)
    assert np.all(err <= np.repeat(O.E4M3[s], 16, -1) * (1 + 6 / 16))


def test_select_closed_forms():
    o, d = 5, 4
    q, ks = np.zeros((2, d)), np.arange(o * d).reshape(o, d)
    assert O.select_row(q, ks, 64, 1.0, 0.6, 1) == [0, 1, 2, 5]          # uniform: three of five reach 0.6
    assert O.select_row(q, ks, 64, 1.0, 0.1, 4) == [0, 1, 2, 3, 5]       # the floor
    assert O.select_row(q, ks, 64, 1.0, 1.0, 1) == [0, 1, 2, 3, 4, 5]
    assert O.select_row(q, ks[:0], 64, 1.0, 0.5, 3) == [0]               # nothing before the own page
    q[:] = 1e6
    assert O.select_row(q, ks, 64, 1.0, 0.9, 1) == [4, 5]                # one page takes all


def test_attend_closed_forms():
    q = np.zeros(64)
    k, v = np.random.default_rng(1).standard_normal((2, 7, 64))
    out, lse, _, _ = O.attend_row(q, k, v, 0.125)
    assert np.allclose(out, v.mean(0)) and np.isclose(lse, np.log(7))
    out, lse, _, _ = O.attend_row(q, k[:0], v[:0], 0.125)
    assert not out.any() and lse == -np.inf


# ------------------------------------------------------------------ the C ABI, before any launch
FAKE = 1 << 20


def _cache(pages=FAKE, ksum=FAKE, ks=None, vs=None, num_pages=4, H=2, d=64, block=64):
    return K._CacheStruct(pages, ksum, ks, vs, num_pages, H, d, block)


def _batch(table=FAKE, kv_len=FAKE, cu=FAKE, B=2, max_pages=3, rows=5, max_q=4):
    return K._BatchStruct(table, kv_len, cu, B, max_pages, rows, max_q)


def _r(x):
    return None if x is None else ctypes.byref(x)


BAD_COMMON = [dict(cache=None), dict(batch=None), dict(cache=_cache(pages=None)), dict(cache=_cache(pages=FAKE + 8)),
              dict(cache=_cache(num_pages=0)), dict(cache=_cache(H=0)), dict(cache=_cache(d=96)),
              dict(cache=_cache(block=32)), dict(cache=_cache(ksum=FAKE + 4)), dict(cache=_cache(ks=FAKE + 2)),
              dict(batch=_batch(table=None)), dict(batch=_batch(kv_len=None)), dict(batch=_batch(cu=None)),
              dict(batch=_batch(cu=FAKE + 1)), dict(batch=_batch(B=0)), dict(batch=_batch(max_pages=0)),
              dict(batch=_batch(max_pages=1 << 25)), dict(batch=_batch(rows=-1)), dict(batch=_batch(max_q=0)),
              dict(dtype=7)]
FAR = FAKE * 64     # does not overlap the pool


def _append(cache=_cache(), batch=_batch(), k=FAR, v=FAR, ks=128, vs=128, dtype=F.FVATTN_BF16, ws=FAKE, n=256):
    return F._lib.fvattn_kv4_append(_r(cache), _r(batch), k, v, ks, vs, dtype, ws, n, None)


def _read(cache=_cache(), batch=_batch(), k=FAR, v=2 * FAR, dtype=F.FVATTN_BF16, ws=FAKE, n=256):
    return F._lib.fvattn_kv4_read(_r(cache), _r(batch), k, v, dtype, ws, n, None)


def _select(cache=_cache(), batch=_batch(), q=FAR, qs=256, Hq=4, dtype=F.FVATTN_BF16, scale=0.1, p=0.9, k_min=1,
            idx=FAR, cnt=FAR, ws=FAKE, n=1 << 40):
    return F._lib.fvattn_kv4_select(_r(cache), _r(batch), q, qs, Hq, dtype, scale, p, k_min, idx, cnt, ws, n, None)


def _attn(cache=_cache(), batch=_batch(), q=FAR, qs=256, Hq=4, out=2 * FAR, lse=None, dtype=F.FVATTN_BF16, scale=0.1,
          causal=1, idx=None, cnt=None, ws=FAKE, n=1 << 40):
    return F._lib.fvattn_kv4_attn(_r(cache), _r(batch), q, qs, Hq, out, lse, dtype, scale, causal, idx, cnt, ws, n,
                                  None)


@pytest.mark.parametrize("kw", BAD_COMMON, ids=str)
@pytest.mark.parametrize("call", [_append, _read, _select, _attn])
def test_every_call_rejects_bad_caches_and_batches(call, kw):
    assert call(**kw) == F.FVATTN_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [
    dict(k=None), dict(v=None), dict(k=FAR + 4), dict(ks=64), dict(vs=127), dict(ks=129), dict(ks=-128),
    dict(k=FAKE + 64), dict(v=FAKE + 128)], ids=str)
def test_append_rejects(kw):
    assert _append(**kw) == F.FVATTN_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(k=None), dict(v=None), dict(v=FAR), dict(k=FAKE), dict(v=FAR + 8)], ids=str)
def test_read_rejects(kw):
    assert _read(**kw) == F.FVATTN_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(idx=None), dict(cnt=None), dict(Hq=3), dict(Hq=1), dict(Hq=0), dict(Hq=130, qs=8320),
    dict(qs=255), dict(qs=128), dict(scale=0.0), dict(scale=float("inf")), dict(scale=float("nan")), dict(p=0.0),
    dict(p=1.01), dict(p=float("nan")), dict(k_min=0), dict(idx=FAR + 2), dict(cache=_cache(ksum=None)),
    dict(batch=_batch(max_pages=8193))], ids=str)
def test_select_rejects(kw):
    assert _select(**kw) == F.FVATTN_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(out=None), dict(out=FAR), dict(out=FAR + 2048), dict(q=FAR + 8), dict(lse=FAR + 2), dict(Hq=3),
    dict(Hq=130, qs=8320), dict(qs=248), dict(scale=-1.0), dict(scale=float("nan")), dict(idx=FAR), dict(cnt=FAR),
    dict(idx=FAR + 1, cnt=FAR)], ids=str)
def test_attn_rejects(kw):
    assert _attn(**kw) == F.FVATTN_ERR_INVALID_ARG


@pytest.mark.parametrize("call", [_append, _read, _select, _attn])
@pytest.mark.parametrize("kw", [dict(ws=None), dict(ws=FAKE + 16), dict(n=255)], ids=str)
def test_workspaces_are_checked(call, kw):
    assert call(**kw) == F.FVATTN_ERR_WORKSPACE


def test_workspace_bytes():
    def size(op, cache=_cache(), batch=_batch(), Hq=4):
        return F._lib.fvattn_kv4_workspace_bytes(op, _r(cache), _r(batch), Hq)
    ops = (F.FVATTN_OP_KV4_APPEND, F.FVATTN_OP_KV4_READ, F.FVATTN_OP_KV4_SELECT, F.FVATTN_OP_KV4_ATTN)
    for op in ops:
        assert size(op) >= 256 and size(op) % 256 == 0
        assert size(op, cache=_cache(d=80)) == 0 and size(op, batch=_batch(B=0)) == 0 and size(op, cache=None) == 0
        # a path sized for its largest call can make smaller ones
        assert size(op, batch=_batch(B=9, rows=40)) >= size(op)
    assert size(F.FVATTN_OP_KV4_ATTN, Hq=3) == 0
    assert size(F.FVATTN_OP_ROUTE) == 0
    assert F.fvattn_workspace_bytes(F.FVATTN_OP_KV4_ATTN, 1, 1, 64, 64, 64) == 0
