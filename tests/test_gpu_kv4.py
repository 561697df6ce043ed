"""GPU: the paged 4-bit key/value cache against its fp64 oracle: codes, page sums and lists
exactly, attention within bounds derived from its roundings, at the lengths, head layouts,
strides and masks where it can go wrong; refusals; captured and concurrent calls.

Attention's bound, for a row with weights w, A = sum w |v| per channel, S = max |logit| and
T = max sum |q||k| scale:
  a logit's error          e_s = T d 2^-24 (fp32 sums of exact products; the fp32 path's split of q
                                 leaves 2^-22 of T more) + S 2^-22 (product with the scale, exponent's
                                 argument, both rounded to fp32)
  a weight's               2 e_s + 2^-21 (ex2.approx, the quotient) + P's rounding to fp16, 2^-11
                           (bf16 path; the fp32 path keeps 2^-22)
  P below fp16's range     rounds to a grid of 2^-24 of a value at most 2^-4 of the row's largest P: at
                           most N 2^-29 A_max
  output                   half a step of its type, 2^-8 or 2^-24 relative (and 2^-23 for the products
                           with 1/l and the head's scale)
"""

import math

import numpy as np
import pytest
import torch

from oracle import kv4_oracle as O

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import block_sparse_attention_video_b200 as F

BF16, FP32 = torch.bfloat16, torch.float32


class Case:
    """A pool filled through fvattn_kv4_append with ragged sequences, and the oracle's copy of it."""

    def __init__(self, kv, rows, H, d, block, seed=0, scaled=False, Hq=None, dtype=BF16, spread=1.0, fill=True):
        self.g = torch.Generator().manual_seed(seed)
        self.kv, self.nrow, self.H, self.d, self.block, self.dtype = kv, rows, H, d, block, dtype
        self.Hq = Hq or H
        dev = torch.device("cuda")
        need = [max(1, -(-n // block)) for n in kv]
        self.max_pages = max(need) + 1
        slots = sum(need) + 3
        perm = torch.randperm(slots, generator=self.g)
        table = torch.full((len(kv), self.max_pages), -7, dtype=torch.int32)   # never to be read behind the end
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = perm[at:at + n]
            at += n
        self.table_np = table.numpy()
        sc = lambda: (0.3 + torch.rand(H, generator=self.g)) if scaled else None
        self.ks, self.vs = sc(), sc()
        up = lambda t: None if t is None else t.to(dev)
        self.cache = F.KV4Cache(slots, H, d, block, dev, k_scale=up(self.ks), v_scale=up(self.vs))
        self.cache.pages.fill_(0xFF)                        # what was never written has NaN scales
        self.table = table.to(dev)
        rnd = lambda n: spread * torch.randn((n, H, d), generator=self.g)
        self.k = [rnd(n).to(dtype) for n in kv]
        self.v = [rnd(n).to(dtype) for n in kv]
        self.batch = self.batch_of(rows)
        self.rows = sum(rows)
        if fill:
            self.append(kv)

    def batch_of(self, rows, kv=None):
        dev = self.table.device
        return F.KV4Batch(self.table, torch.tensor(kv or self.kv, dtype=torch.int32, device=dev),
                          torch.tensor(np.cumsum([0] + list(rows)), dtype=torch.int32, device=dev), max(max(rows), 1))

    def ws(self, op, rows, batch=None):
        return F.alloc_workspace(F.fvattn_kv4_workspace_bytes(op, self.cache, batch or self.batch, rows, self.Hq),
                                 self.table.device)

    def append(self, rows, kv=None):
        kv = kv or self.kv
        b = self.batch_of(rows, kv)
        cat = lambda x: torch.cat([t[n - r:n] for t, n, r in zip(x, kv, rows)]).cuda()
        ws = self.ws(F.FVATTN_OP_KV4_APPEND, sum(rows), b)
        F.fvattn_kv4_append(self.cache, b, cat(self.k), cat(self.v), ws)
        assert F.fvattn_workspace_status(ws) == F.FVATTN_OK

    def quantized(self, b):
        """The oracle's codes and scales of sequence b's tokens: K codes, K scales, V codes, V scales."""
        f = lambda x, s: O.quantize(x[b].float().numpy(), None if s is None else s.numpy())
        return (*f(self.k, self.ks), *f(self.v, self.vs))

    def values(self, b):
        kc, ks, vc, vs = self.quantized(b)
        h = lambda s: 1.0 if s is None else s.double().numpy()[:, None]
        return O.dequantize(kc, ks) * h(self.ks), O.dequantize(vc, vs) * h(self.vs)

    def records(self):
        """The pool's records split: K codes [slots, H, block, d], K scales, V codes, V scales."""
        p = self.cache.pages.cpu().numpy()
        a, s = self.block * self.d // 2, self.block * self.d // 16
        parts = [p[..., i:j] for i, j in ((0, a), (a, a + s), (a + s, 2 * a + s), (2 * a + s, 2 * a + 2 * s))]
        out = []
        for i, x in enumerate(parts):
            x = x.reshape(*x.shape[:2], self.block, -1)
            out.append(np.stack((x & 15, x >> 4), -1).reshape(*x.shape[:3], -1) if i % 2 == 0 else x)
        return out

    def assert_records(self, want):
        """The pool's records equal ``want`` (an earlier ``records()``), a zero's sign aside."""
        for i, (g, w) in enumerate(zip(self.records(), want)):
            assert np.all((g == w) | (((g & 7) == 0) & ((w & 7) == 0)) if i % 2 == 0 else g == w)

    def make_q(self, dtype=None, spread=1.0, pad=0):
        q = spread * torch.randn((self.rows + pad, self.Hq, self.d), generator=self.g)
        return q.to(dtype or self.dtype)

    def attend(self, q, causal=True, idx=None, cnt=None, scale=None, ws=None, stream=None):
        qd = q if q.is_cuda else q.cuda()
        out = torch.full(tuple(qd.shape), 77.0, dtype=qd.dtype, device=qd.device)
        lse = torch.full(tuple(qd.shape[:2]), 77.0, device=qd.device)
        ws = self.ws(F.FVATTN_OP_KV4_ATTN, qd.shape[0]) if ws is None else ws
        F.fvattn_kv4_attn(self.cache, self.batch, qd, out, ws, scale=scale, causal=causal, lse=lse, kv_idx=idx,
                          kv_cnt=cnt, stream=stream)
        self.last_ws = ws
        return out, lse

    def check(self, q, out, lse, causal=True, lists=None, scale=None, rows=None):
        """Every (row, head) (or the given rows) against the oracle, within the bound above."""
        sc = float(np.float32(1 / math.sqrt(self.d) if scale is None else scale))
        out, lse, qn = out.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().cpu().numpy()
        bf16 = q.dtype == BF16
        half = 2.0 ** -8 if bf16 else 2.0 ** -24
        G = self.Hq // self.H
        r0 = 0
        for b, (n, m) in enumerate(zip(self.kv, self.nrow)):
            kv = self.values(b) if m else None
            for i in range(m):
                if rows is not None and r0 + i not in rows:
                    continue
                pos = n - m + i
                keys = np.arange(max(0, min(n, pos + 1)) if causal else n)
                for hq in range(self.Hq):
                    h = hq // G
                    kk = keys
                    if lists is not None:
                        kk = keys[np.isin(keys // self.block, lists[r0 + i][h])]
                    k, v = kv[0][kk, h], kv[1][kk, h]
                    ref, ref_lse, A, T = O.attend_row(qn[r0 + i, hq], k, v, sc)
                    if len(kk) == 0:
                        assert not out[r0 + i, hq].any() and lse[r0 + i, hq] == -np.inf
                        continue
                    S = abs(ref_lse) + T
                    e_s = T * (self.d * 2.0 ** -24 + 2.0 ** -22) + S * 2.0 ** -22
                    rel = 2 * e_s + 2.0 ** -21 + (2.0 ** -11 if bf16 else 2.0 ** -22)
                    tol = (half + 2.0 ** -23) * np.abs(ref) + rel * A + len(kk) * 2.0 ** -29 * np.abs(v).max()
                    err = np.abs(out[r0 + i, hq] - ref)
                    assert np.all(err <= tol), (b, i, hq, float((err / tol).max()))
                    assert abs(lse[r0 + i, hq] - ref_lse) <= 2 * e_s + 2.0 ** -20 + abs(ref_lse) * 2.0 ** -22, (b, i, hq)
            r0 += m


# ------------------------------------------------------------------ writing and reading back
WRITE = [
    # kv, H, d, block, scaled, dtype
    ([1], 1, 64, 64, False, BF16),
    ([128], 2, 128, 128, False, BF16),
    ([130, 64, 1], 3, 128, 64, False, FP32),
    ([300, 257, 0, 127], 2, 64, 128, True, BF16),
    ([191], 5, 128, 64, True, FP32),
]


@pytest.mark.parametrize("kv,H,d,block,scaled,dtype", WRITE)
def test_codes_scales_and_sums_are_exact(kv, H, d, block, scaled, dtype):
    c = Case(kv, kv, H, d, block, seed=len(kv) + H, scaled=scaled, dtype=dtype, spread=1.3)
    kc, ks, vc, vs = c.records()
    ksum = c.cache.ksum.cpu().numpy()
    for b, n in enumerate(kv):
        want = c.quantized(b)
        for t in range(n):
            slot, at = c.table_np[b, t // block], t % block
            for got, w in zip((kc, ks, vc, vs), want):
                g, e = got[slot, :, at], w[t]
                same = (g == e) | (((g & 7) == 0) & ((e & 7) == 0)) if got is kc or got is vc else g == e
                assert np.all(same), (b, t)
        plain = O.dequantize(want[0], want[1])
        for pg in range(n // block):
            for h in range(H):
                s = O.page_sum(plain[pg * block:(pg + 1) * block, h])
                assert np.array_equal(ksum[c.table_np[b, pg], h], s)
    # what no row owns is as it was
    owned = np.zeros((c.cache.num_pages, block), bool)
    for b, n in enumerate(kv):
        for t in range(n):
            owned[c.table_np[b, t // block], t % block] = True
    assert np.all(kc.transpose(0, 2, 1, 3)[~owned] == 15) and np.all(vs.transpose(0, 2, 1, 3)[~owned] == 0xFF)


@pytest.mark.parametrize("steps", [[1] * 9, [5, 64, 1, 60, 3], [127, 1, 2], [200]])
def test_growing_by_steps_equals_one_write(steps):
    n = sum(steps) + 70
    a = Case([n, n], [n, n], 2, 64, 64, seed=3)
    b = Case([n, n], [n, n], 2, 64, 64, seed=3, fill=False)
    b.append([70, 70], kv=[70, 70])
    at = 70
    for s in steps:
        at += s
        b.append([s, s], kv=[at, at])
    assert torch.equal(a.cache.pages, b.cache.pages)
    full = [a.table_np[i, p] for i in range(2) for p in range(n // 64)]
    assert torch.equal(a.cache.ksum[full], b.cache.ksum[full])


def test_writing_a_position_again_replaces_it():
    a, b = Case([130], [130], 2, 128, 64, seed=5), Case([130], [130], 2, 128, 64, seed=6)
    b.k, b.v = a.k, a.v
    b.append([100])                       # positions 30..129 with the other case's rows
    b.append([130])
    assert torch.equal(a.cache.pages[a.table_np[0, :3]], b.cache.pages[b.table_np[0, :3]])
    assert torch.equal(a.cache.ksum[a.table_np[0, :2]], b.cache.ksum[b.table_np[0, :2]])


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_extreme_inputs(dtype):
    c = Case([4], [4], 1, 64, 64, dtype=dtype, fill=False)
    k = torch.zeros((4, 1, 64))
    k[0, 0, 0], k[0, 0, 1] = 1e30, -5.0
    k[1, 0, :16] = torch.linspace(-1, 1, 16) * 1e-4            # below half the smallest scale: all zero
    k[1, 0, 16:32] = 0.02
    k[2, 0, 0], k[2, 0, 1], k[2, 0, 2] = math.inf, -math.inf, 1.0
    k[3, 0, 3] = -2688.0
    c.k = c.v = [k.to(dtype)]
    c.append([4])
    out = [torch.empty((4, 1, 64), dtype=FP32, device="cuda") for _ in range(2)]
    ws = c.ws(F.FVATTN_OP_KV4_READ, 4)
    F.fvattn_kv4_read(c.cache, c.batch, *out, ws)
    g = out[0].cpu()[:, 0]
    assert g[0, 0] == 2688 and g[2, 0] == 2688 and g[2, 1] == -2688 and g[3, 3] == -2688
    assert not g[1, :16].any() and torch.equal(out[0], out[1])
    x = c.k[0].float().numpy()
    x[2] = 0
    want = O.dequantize(*O.quantize(x))
    assert np.array_equal(g.numpy()[[0, 1, 3]], want[[0, 1, 3], 0])


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("scales", [[1e-25, 0.7], [3.3e20, 2.0 ** 60], [2.0 ** -60, 1.1e-3]])
def test_head_scales_of_any_size(dtype, scales):
    """The stored value is that of the correctly rounded quotient by the head's scale, saturated."""
    c = Case([300], [300], 2, 64, 64, seed=30, dtype=dtype, scaled=True, fill=False)
    c.ks.copy_(torch.tensor(scales))
    c.cache.k_scale.copy_(c.ks)
    k = c.k[0].float() * c.ks[:, None] * torch.logspace(-4, 4, 300)[:, None, None]
    k[7, :, 0], k[8, :, 1] = math.inf, -math.inf
    c.k = [k.to(dtype)]
    c.append(c.kv)
    kc, ks, _, _ = c.records()
    x = c.k[0].float().numpy()
    want, sc = O.quantize(np.clip(x, -3e38, 3e38), c.ks.numpy())
    for t in range(300):
        slot, at = c.table_np[0, t // 64], t % 64
        g, w = kc[slot, :, at], want[t]
        assert np.array_equal(ks[slot, :, at], sc[t]), t
        assert np.all((g == w) | (((g & 7) == 0) & ((w & 7) == 0))), t


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("d,block", [(64, 64), (128, 128), (128, 64)])
def test_every_code_border(dtype, d, block):
    """x on and one step beside every border t * s of two codes, for every scale significand."""
    rows = []
    for m in range(8, 16):
        for e in (-6, 0, 7):
            s = np.float32(m / 8 * 2.0 ** e)
            for t in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
                x = torch.tensor(t * s, dtype=dtype)
                lo, hi = (torch.nextafter(x, torch.tensor(v, dtype=dtype)) for v in (0.0, 1e9))
                r = torch.zeros(16, dtype=dtype)
                r[0] = float(6 * s)
                r[1], r[2], r[3], r[4], r[5], r[6] = x, lo, hi, -x, -lo, -hi
                rows.append(r)
    x = torch.stack(rows)
    x = torch.cat([x, torch.zeros((-len(x)) % (d // 16), 16, dtype=dtype)]).reshape(-1, 1, d)
    c = Case([len(x)], [len(x)], 1, d, block, dtype=dtype, fill=False)
    c.k = c.v = [x]
    c.append([len(x)])
    kc, ks, _, _ = c.records()
    want, sc = O.quantize(x.float().numpy())
    for t in range(len(x)):
        slot = c.table_np[0, t // block]
        g, w = kc[slot, 0, t % block], want[t, 0]
        assert np.array_equal(ks[slot, 0, t % block], sc[t, 0])
        assert np.all((g == w) | (((g & 7) == 0) & ((w & 7) == 0))), t


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("rows,pad", [([1, 1], 0), ([77, 3], 2), ([130, 200], 5)])
def test_read_back(dtype, rows, pad):
    c = Case([150, 200], rows, 3, 128, 64, seed=9, scaled=True)
    c.nrow, rows = [min(a, b) for a, b in zip(rows, c.kv)], rows
    b = c.batch_of(c.nrow)
    n = sum(c.nrow)
    out = [torch.full((n + pad, 3, 128), 55.0, dtype=dtype, device="cuda") for _ in range(2)]
    ws = c.ws(F.FVATTN_OP_KV4_READ, n + pad, b)
    F.fvattn_kv4_read(c.cache, b, *out, ws)
    assert F.fvattn_workspace_status(ws) == F.FVATTN_OK
    r = 0
    for i, m in enumerate(c.nrow):
        kc, ks, vc, vs = c.quantized(i)
        for got, codes, scales, hs in ((out[0], kc, ks, c.ks), (out[1], vc, vs, c.vs)):
            v = (O.dequantize(codes, scales).astype(np.float32) * hs.numpy()[:, None])[c.kv[i] - m:]
            assert torch.equal(got[r:r + m].cpu(), torch.tensor(v).to(dtype))
        r += m
    assert torch.all(out[0][n:] == 55) and torch.all(out[1][n:] == 55)


def test_append_takes_columns_of_a_fused_projection():
    a = Case([90, 10], [90, 10], 2, 64, 64, seed=4)
    b = Case([90, 10], [90, 10], 2, 64, 64, seed=4, fill=False)
    k, v = torch.cat(b.k).cuda(), torch.cat(b.v).cuda()
    fused = torch.randn((100, 8 * 64), device="cuda").to(BF16)
    fused[:, 256:384], fused[:, 384:512] = k.flatten(1), v.flatten(1)
    kk, vv = fused[:, 256:384].unflatten(1, (2, 64)), fused[:, 384:].unflatten(1, (2, 64))
    F.fvattn_kv4_append(b.cache, b.batch, kk, vv, b.ws(F.FVATTN_OP_KV4_APPEND, 100))
    assert torch.equal(a.cache.pages, b.cache.pages)


def test_offsets_past_32_bits():
    # 2^31 bytes of pool lie before the pages used: 117k records of 18,432 bytes and more
    slots = (1 << 31) // 18432 + 40
    cache = F.KV4Cache(slots, 1, 128, 128, "cuda")
    n = 300
    dev = cache.device
    table = torch.tensor([[slots - 1, 3, slots - 7]], dtype=torch.int32, device=dev)
    one = lambda *v: torch.tensor(v, dtype=torch.int32, device=dev)
    batch = F.KV4Batch(table, one(n), one(0, n), n)
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn((n, 1, 128), generator=g).to(BF16) for _ in range(2))
    ws = F.alloc_workspace(1 << 26, dev)
    F.fvattn_kv4_append(cache, batch, k.cuda(), v.cuda(), ws)
    ko, vo = torch.empty_like(k, device=dev), torch.empty_like(v, device=dev)
    F.fvattn_kv4_read(cache, batch, ko, vo, ws)
    want = O.dequantize(*O.quantize(k.float().numpy()))
    assert np.array_equal(ko.float().cpu().numpy(), want)
    q = torch.randn((n, 1, 128), generator=g).to(BF16)
    out, lse = torch.empty_like(q, device=dev), torch.empty((n, 1), device=dev)
    F.fvattn_kv4_attn(cache, batch, q.cuda(), out, ws, lse=lse)
    ref, rl, _, _ = O.attend_row(q[-1, 0].double().numpy(), want[:, 0], O.dequantize(*O.quantize(v.float().numpy()))[:, 0],
                                 128 ** -0.5)
    assert abs(lse[-1, 0].item() - rl) < 1e-4 and np.abs(out[-1, 0].double().cpu().numpy() - ref).max() < 0.02


# ------------------------------------------------------------------ choosing pages
SELECT = [
    # kv, rows, H, Hq, d, block, p, k_min, dtype, scaled
    ([1], [1], 1, 1, 64, 64, 0.9, 1, BF16, False),
    ([64], [1], 1, 2, 64, 64, 0.9, 1, BF16, False),
    ([65], [1], 2, 2, 128, 64, 0.5, 1, FP32, False),
    ([2000, 129, 700], [1, 1, 1], 2, 10, 128, 64, 0.9, 2, BF16, True),
    ([1500, 900], [70, 3], 1, 3, 64, 128, 0.8, 1, BF16, False),
    ([4500], [2], 1, 8, 64, 64, 0.95, 5, FP32, False),
    ([1000, 0, 300], [5, 0, 2], 2, 2, 64, 64, 1.0, 1, BF16, False),
    ([700], [4], 1, 64, 64, 64, 0.7, 3, BF16, False),
    ([900], [3], 2, 4, 128, 64, 0.3, 100, BF16, True),
    ([2900, 700], [330, 41], 7, 7, 64, 64, 0.85, 1, BF16, False),   # blocks for three an SM
    ([600, 410], [100, 20], 5, 15, 128, 64, 0.9, 2, FP32, True),
]


def _select(c, q, p, k_min, scale=None):
    n = q.shape[0]
    idx = torch.full((n, c.H, c.max_pages), -5, dtype=torch.int32, device="cuda")
    cnt = torch.full((n, c.H), -5, dtype=torch.int32, device="cuda")
    ws = c.ws(F.FVATTN_OP_KV4_SELECT, n)
    F.fvattn_kv4_select(c.cache, c.batch, q.cuda(), p, k_min, idx, cnt, ws, scale=scale)
    c.last_ws = ws
    return idx, cnt


def _want_lists(c, q, p, k_min, scale=None):
    sc = float(np.float32(c.d ** -0.5 if scale is None else scale))
    G = c.Hq // c.H
    lists, qn = [], q.double().numpy()
    r = 0
    for b, (n, m) in enumerate(zip(c.kv, c.nrow)):
        kc, ks, _, _ = c.quantized(b) if n else (None,) * 4
        plain = O.dequantize(kc, ks) if n else None
        for i in range(m):
            o = (n - m + i) // c.block
            per = []
            for h in range(c.H):
                sums = np.array([O.page_sum(plain[j * c.block:(j + 1) * c.block, h]) for j in range(o)]).reshape(o, c.d)
                hs = 1.0 if c.ks is None else float(c.ks[h])
                per.append(O.select_row(qn[r + i, h * G:(h + 1) * G], sums, c.block, sc * hs, float(np.float32(p)),
                                        k_min))
            lists.append(per)
        r += m
    return lists


@pytest.mark.parametrize("kv,rows,H,Hq,d,block,p,k_min,dtype,scaled", SELECT)
def test_lists_equal_the_oracles(kv, rows, H, Hq, d, block, p, k_min, dtype, scaled):
    c = Case(kv, rows, H, d, block, seed=11, scaled=scaled, Hq=Hq)
    q = c.make_q(dtype, spread=6.0, pad=2)          # sharp enough for short lists
    idx, cnt = _select(c, q, p, k_min)
    assert F.fvattn_workspace_status(c.last_ws) == F.FVATTN_OK
    want = _want_lists(c, q, p, k_min)
    idx, cnt = idx.cpu().numpy(), cnt.cpu().numpy()
    for r, per in enumerate(want):
        for h, w in enumerate(per):
            assert cnt[r, h] == len(w) and list(idx[r, h, :len(w)]) == w, (r, h)
            assert np.all(idx[r, h, len(w):] == -5)
    assert np.all(cnt[c.rows:] == -5) and np.all(idx[c.rows:] == -5)


def test_tied_pages_go_to_the_lower_index():
    c = Case([64 * 9 + 1], [1], 1, 64, 64, seed=2, Hq=3, fill=False)
    page = torch.randn((64, 1, 64), generator=c.g).to(BF16)
    c.k = [torch.cat([page] * 9 + [page[:1]])]
    c.append(c.kv)
    idx, cnt = _select(c, c.make_q(), 0.5, 1)
    assert idx[0, 0, :cnt[0, 0]].tolist() == [0, 1, 2, 3, 4, 9]
    idx, cnt = _select(c, c.make_q(), 0.01, 3)
    assert idx[0, 0, :cnt[0, 0]].tolist() == [0, 1, 2, 9]


def test_select_takes_columns_of_a_fused_projection():
    c = Case([700, 300], [3, 2], 2, 64, 64, seed=8, Hq=4)
    q = c.make_q(spread=5.0)
    wide = torch.randn((5, 6 * 64), device="cuda").to(BF16)
    wide[:, 64:320] = q.flatten(1).cuda()
    a = _select(c, q, 0.8, 2)
    b = _select(c, wide[:, 64:320].unflatten(1, (4, 64)), 0.8, 2)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


# ------------------------------------------------------------------ attention
ATTEND = [
    # kv, rows, H, Hq, d, block, dtype, causal, scaled
    ([1], [1], 1, 1, 64, 64, BF16, True, False),
    ([1, 2, 63, 64, 65], [1] * 5, 2, 2, 128, 64, BF16, True, False),
    ([127, 128, 129, 700], [1] * 4, 1, 8, 128, 128, BF16, True, True),
    ([1000], [1], 3, 15, 128, 64, BF16, True, False),
    ([513, 40], [1, 1], 1, 16, 64, 128, BF16, True, False),
    ([400], [1], 1, 40, 64, 64, BF16, True, False),
    ([300], [1], 1, 64, 128, 128, BF16, True, False),
    ([700, 90], [5, 3], 2, 6, 64, 64, FP32, True, True),
    ([260], [1], 2, 4, 128, 128, FP32, True, False),
    ([130, 0, 77], [9, 0, 1], 2, 4, 128, 64, BF16, True, False),
    ([200, 100], [33, 100], 1, 4, 128, 128, BF16, True, False),
    ([333, 257], [333, 130], 2, 2, 64, 128, BF16, True, True),
    ([300], [150], 1, 3, 128, 64, BF16, False, False),
    ([513], [300], 1, 1, 128, 128, BF16, False, False),
    ([150], [40], 1, 3, 128, 128, FP32, False, False),
    ([300], [140], 2, 2, 64, 64, BF16, False, True),
]


@pytest.mark.parametrize("kv,rows,H,Hq,d,block,dtype,causal,scaled", ATTEND)
def test_attention(kv, rows, H, Hq, d, block, dtype, causal, scaled):
    c = Case(kv, rows, H, d, block, seed=sum(kv), scaled=scaled, Hq=Hq)
    q = c.make_q(dtype, spread=2.0, pad=3)
    out, lse = c.attend(q, causal)
    assert F.fvattn_workspace_status(c.last_ws) == F.FVATTN_OK
    assert torch.all(out[c.rows:] == 77) and torch.all(lse[c.rows:] == 77)     # rows of no sequence
    some = None if c.rows <= 60 else set(range(0, c.rows, 7)) | {c.rows - 1}
    c.check(q, out, lse, causal, rows=some)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("causal", [True, False])
def test_rows_that_see_nothing(dtype, causal):
    # more rows than tokens: the first ones stand before the sequence; an empty sequence has nothing to see
    c = Case([3, 0, 70], [5, 2, 1], 1, 64, 64, seed=7, Hq=4, dtype=dtype, fill=False)
    c.append([3, 0, 70])
    q = c.make_q()
    out, lse = c.attend(q, causal)
    assert F.fvattn_workspace_status(c.last_ws) == F.FVATTN_OK
    c.check(q, out, lse, causal)
    dead = [0, 1, 5, 6] if causal else [5, 6]
    assert not out[dead].any() and torch.all(lse[dead] == -math.inf)


@pytest.mark.parametrize("rows", [[1, 1], [40, 150]])
@pytest.mark.parametrize("spread", [1e-6, 30.0, 1e4])
def test_blunt_and_sharp_logits(rows, spread):
    c = Case([900, 333], rows, 1, 128, 128, seed=13, Hq=4)
    q = c.make_q(spread=spread)
    scale = 0.01 if spread > 100 else None
    out, lse = c.attend(q, scale=scale)
    c.check(q, out, lse, scale=scale, rows=set(range(0, c.rows, 11)) | {0, c.rows - 1})


@pytest.mark.parametrize("rows", [[1], [70]])
def test_growing_logits(rows):
    """Keys that point ever more along q: the running maximum rises at every page."""
    c = Case([1100], rows, 1, 64, 64, seed=14, Hq=1, fill=False)
    direction = torch.randn(64, generator=c.g)
    ramp = torch.linspace(-3, 3, 1100)[:, None, None]
    c.k = [(ramp * direction + 0.1 * torch.randn((1100, 1, 64), generator=c.g)).to(BF16)]
    c.append(c.kv)
    q = (5 * direction).to(BF16).expand(c.rows, 1, 64).contiguous()
    out, lse = c.attend(q)
    c.check(q, out, lse, rows=set(range(0, c.rows, 9)))


@pytest.mark.parametrize("big", [1e30, 1e-30])
@pytest.mark.parametrize("rows", [[2], [200]])
def test_range_of_q(big, rows):
    c = Case([260], rows, 1, 64, 64, seed=15, Hq=2)
    q = c.make_q()
    ref, rl = c.attend(q, scale=0.125)
    got, gl = c.attend((q.float() * 2.0 ** round(math.log2(big))).to(BF16), scale=0.125 * 2.0 ** -round(math.log2(big)))
    assert torch.equal(ref, got) and torch.equal(rl, gl)


@pytest.mark.parametrize("rows,G", [([1, 1], 1), ([1, 1], 5), ([3, 2], 8), ([2, 1], 20)])
@pytest.mark.parametrize("block,dtype", [(64, BF16), (128, BF16), (64, FP32)])
def test_attention_over_selected_pages(rows, G, block, dtype):
    c = Case([1400, 650], rows, 2, 64, block, seed=16, Hq=2 * G)
    q = c.make_q(dtype, spread=4.0)
    idx, cnt = _select(c, q, 0.7, 2)
    lists = [[idx[r, h, :cnt[r, h]].tolist() for h in range(2)] for r in range(c.rows)]
    for causal in (True, False):
        out, lse = c.attend(q, causal, idx, cnt)
        assert F.fvattn_workspace_status(c.last_ws) == F.FVATTN_OK
        c.check(q, out, lse, causal, lists=lists)


def test_lists_of_every_page_equal_no_lists():
    c = Case([900, 500], [2, 3], 2, 128, 64, seed=17, Hq=8)
    q = c.make_q()
    idx = torch.arange(c.max_pages, dtype=torch.int32, device="cuda").expand(5, 2, -1).contiguous()
    cnt = torch.tensor([15] * 2 + [8] * 3, dtype=torch.int32, device="cuda")[:, None].expand(5, 2).contiguous()
    a, la = c.attend(q, True, idx, cnt)
    b, lb = c.attend(q, True)
    assert (a.float() - b.float()).abs().max() <= 2.0 ** -7 * b.float().abs().max()
    assert (la - lb).abs().max() < 1e-4


def test_bad_lists_are_left_out_and_recorded():
    c = Case([900], [3], 1, 64, 64, seed=18, Hq=2)          # pages 0..14
    q = c.make_q()
    idx = torch.zeros((3, 1, c.max_pages), dtype=torch.int32, device="cuda")
    cnt = torch.tensor([[6], [2], [1]], dtype=torch.int32, device="cuda")
    idx[0, 0, :6] = torch.tensor([2, 2, 1, 5, 99, 14], dtype=torch.int32)      # repeated, descending, out of range
    idx[1, 0, :2] = torch.tensor([-3, 4], dtype=torch.int32)
    out, lse = c.attend(q, True, idx, cnt)
    assert F.fvattn_workspace_status(c.last_ws) == F.FVATTN_ERR_INVALID_ARG
    # each entry has to be above the one before it, whatever became of that one: 14 is not
    c.check(q, out, lse, True, lists=[[[2, 5]], [[4]], [[0]]])
    cnt[1] = 0
    idx[0, 0, :6] = torch.tensor([0, 1, 2, 5, 9, 14], dtype=torch.int32)
    out, lse = c.attend(q, True, idx, cnt)
    assert F.fvattn_workspace_status(c.last_ws) == F.FVATTN_OK
    assert not out[1].any() and torch.all(lse[1] == -math.inf)


@pytest.mark.parametrize("rows", [[1, 1], [60, 100]])
def test_bad_tables_and_lengths_are_recorded(rows):
    c = Case([300, 500], rows, 1, 64, 64, seed=19, Hq=2)
    q = c.make_q()
    first = rows[0]
    # Sequence 1 keeps its result within the bound (where its sums are split depends on the whole batch).
    keeps = set(range(first, c.rows, 7)) | {c.rows - 1}
    table = c.table.clone()
    c.batch.table[0, 1] = c.cache.num_pages + 5             # sequence 0 loses a page
    out, lse = c.attend(q)
    assert F.fvattn_workspace_status(c.last_ws) == F.FVATTN_ERR_INVALID_ARG
    assert torch.isfinite(out).all()
    c.check(q, out, lse, rows=keeps)
    idx, cnt = _select(c, q, 0.9, 1)
    assert F.fvattn_workspace_status(c.last_ws) == F.FVATTN_ERR_INVALID_ARG
    c.batch.table.copy_(table)
    c.batch.kv_len[0] = (c.max_pages + 1) * 64              # longer than its table row
    c.batch.table.clamp_(min=0)
    out, lse = c.attend(q)
    assert F.fvattn_workspace_status(c.last_ws) == F.FVATTN_ERR_INVALID_ARG
    c.check(q, out, lse, rows=keeps)
    c.batch.kv_len[0] = -4
    out, lse = c.attend(q)
    assert F.fvattn_workspace_status(c.last_ws) == F.FVATTN_ERR_INVALID_ARG
    assert not out[:first].any()
    c.check(q, out, lse, rows=keeps)


def test_writes_outside_the_table_are_refused_on_the_device():
    c = Case([100, 100], [100, 100], 1, 64, 64, seed=20)
    before = c.cache.pages.clone()
    k = torch.randn((8, 1, 64), device="cuda").to(BF16)
    ws = c.ws(F.FVATTN_OP_KV4_APPEND, 8)
    for kv, cu in (([2, 100], [0, 8, 8]), ([5000, 100], [0, 4, 4]), ([-3, 100], [0, 8, 8])):
        b = F.KV4Batch(c.table, torch.tensor(kv, dtype=torch.int32, device="cuda"),
                       torch.tensor(cu, dtype=torch.int32, device="cuda"), 8)
        F.fvattn_kv4_append(c.cache, b, k, k, ws)
        assert F.fvattn_workspace_status(ws) == F.FVATTN_ERR_INVALID_ARG
    slot = int(c.table_np[0, 0])
    keep = [s for s in range(c.cache.num_pages) if s not in c.table_np[0]]
    assert torch.equal(c.cache.pages[keep], before[keep])
    # the two valid positions of the first call were written, nothing behind them
    assert not torch.equal(c.cache.pages[slot], before[slot])
    b = F.KV4Batch(c.table, torch.tensor([2, 100], dtype=torch.int32, device="cuda"),
                   torch.tensor([0, 8, 8], dtype=torch.int32, device="cuda"), 8)
    ko, vo = (torch.full((8, 1, 64), 3.0, device="cuda") for _ in range(2))
    F.fvattn_kv4_read(c.cache, b, ko, vo, ws)
    assert F.fvattn_workspace_status(ws) == F.FVATTN_ERR_INVALID_ARG
    assert not ko[:6].any() and ko[6:].abs().sum() > 0


# ------------------------------------------------------------------ many sequences, long tables, odd batches
def test_more_sequences_than_shared_memory_holds():
    """300 sequences: all four calls search the lengths in global memory then."""
    g = torch.Generator().manual_seed(40)
    kv = torch.randint(0, 150, (300,), generator=g).tolist()
    rows = [min(n, i % 3) for i, n in enumerate(kv)]
    c = Case(kv, rows, 1, 64, 64, seed=41, Hq=3)
    q = c.make_q(spread=4.0)
    idx, cnt = _select(c, q, 0.6, 1)
    want = _want_lists(c, q, 0.6, 1)
    assert [idx[r, 0, :cnt[r, 0]].tolist() for r in range(c.rows)] == [w[0] for w in want]
    out, lse = c.attend(q)
    c.check(q, out, lse, rows=set(range(0, c.rows, 13)))
    out, lse = c.attend(q, True, idx, cnt)
    c.check(q, out, lse, lists=want, rows=set(range(0, c.rows, 17)))
    many = c.batch_of([min(n, 40) for n in kv])
    n = sum(min(x, 40) for x in kv)
    ko, vo = (torch.empty((n, 1, 64), device="cuda") for _ in range(2))
    F.fvattn_kv4_read(c.cache, many, ko, vo, c.ws(F.FVATTN_OP_KV4_READ, n, many))
    r = 0
    for i, x in enumerate(kv):
        m = min(x, 40)
        if m and i % 11 == 0:
            k, v = c.values(i)
            assert np.array_equal(ko[r:r + m].cpu().numpy(), k[x - m:]) and np.array_equal(vo[r:r + m].cpu().numpy(), v[x - m:])
        r += m


@pytest.mark.parametrize("Hq,kv,p", [(8, 190_000, 0.9), (1, 70_000, 0.95), (3, 70_000, 0.5)])
def test_selection_over_many_pages(Hq, kv, p):
    """Up to 2,968 pages; with eight heads shared memory holds four at a time."""
    c = Case([kv], [1], 1, 64, 64, seed=42, Hq=Hq)
    q = c.make_q(spread=3.0)
    idx, cnt = _select(c, q, p, 2)
    want = _want_lists(c, q, p, 2)[0][0]
    assert idx[0, 0, :cnt[0, 0]].tolist() == want


def test_widest_table():
    c = Case([1000], [2], 2, 64, 64, seed=43, Hq=6)
    q = c.make_q(spread=4.0)
    want = _want_lists(c, q, 0.8, 1)
    wide = torch.zeros((1, 8192), dtype=torch.int32, device="cuda")
    wide[0, :c.max_pages] = c.table[0].clamp(min=0)
    c.table, c.max_pages = wide, 8192
    c.batch = c.batch_of([2])
    idx, cnt = _select(c, q, 0.8, 1)
    assert [[idx[r, h, :cnt[r, h]].tolist() for h in range(2)] for r in range(2)] == want
    out, lse = c.attend(q, True, idx, cnt)
    c.check(q, out, lse, lists=want)


@pytest.mark.parametrize("p,k_min", [(0.55, 1), (0.1, 40), (0.999, 1)])
def test_equal_masses(p, k_min):
    """q = 0: more pages tie than the quick search takes; they go in index order."""
    c = Case([64 * 100 + 9], [1], 1, 64, 64, seed=44, Hq=2)
    q = torch.zeros((1, 2, 64), dtype=BF16)
    idx, cnt = _select(c, q, p, k_min)
    assert idx[0, 0, :cnt[0, 0]].tolist() == _want_lists(c, q, p, k_min)[0][0]


def test_one_sharp_page_and_a_long_tail():
    """Masses over hundreds of binades, down to 0."""
    c = Case([64 * 400 + 1], [1], 1, 64, 64, seed=45, Hq=1)
    q = c.make_q(spread=300.0)
    for p, k_min in ((0.5, 1), (0.9999, 1), (0.5, 60)):
        idx, cnt = _select(c, q, p, k_min)
        assert idx[0, 0, :cnt[0, 0]].tolist() == _want_lists(c, q, p, k_min)[0][0]


@pytest.mark.parametrize("claimed", [1, 500])
def test_max_q_only_chooses_the_kernel(claimed):
    c = Case([400, 130], [60, 1], 1, 64, 64, seed=46, Hq=2)
    c.batch = F.KV4Batch(c.table, c.batch.kv_len, c.batch.cu, claimed)
    q = c.make_q()
    out, lse = c.attend(q)
    assert F.fvattn_workspace_status(c.last_ws) == F.FVATTN_OK
    c.check(q, out, lse, rows=set(range(0, 61, 7)) | {60})


@pytest.mark.parametrize("rows", [[3, 1], [100, 40]])
def test_a_bad_row_leaves_the_others(rows):
    c = Case([300, 200], rows, 1, 128, 64, seed=47, Hq=4)
    q = c.make_q()
    good, gl = c.attend(q)
    q[1, 2, 5], q[2, 0, 0] = math.nan, math.inf
    out, lse = c.attend(q)
    keep = torch.ones(q.shape[:2], dtype=torch.bool)
    keep[1, 2] = keep[2, 0] = False
    assert torch.equal(out[keep], good[keep]) and torch.equal(lse[keep], gl[keep])
    assert out[1, 2].isnan().all() and out[2, 0].isnan().all()


@pytest.mark.parametrize("cu", [[2, 4, 5], [-3, 1, 2], [0, 4, 2], [0, 3, 900]])
def test_odd_row_starts(cu):
    """Rows before cu[0] belong to no sequence; a negative, falling or too large start is skipped and recorded."""
    c = Case([300, 200], [2, 1], 1, 64, 64, seed=48, Hq=2)
    cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
    n = 6
    q = torch.randn((n, 2, 64), generator=c.g).to(BF16).cuda()
    for max_q in (1, 300):
        c.batch = F.KV4Batch(c.table, c.batch.kv_len, cut, max_q)
        out, lse = c.attend(q)
        bad = F.fvattn_workspace_status(c.last_ws)
        assert bad == (F.FVATTN_OK if cu in ([2, 4, 5], [0, 4, 2]) else F.FVATTN_ERR_INVALID_ARG)
        if cu[0] == 2:
            assert torch.all(out[:2] == 77) and torch.all(out[5:] == 77) and torch.isfinite(out).all()
            c.nrow, c.kv = [2, 1], [300, 200]
            c.check(q[2:].cpu(), out[2:], lse[2:])
    idx, cnt = _select(c, q.cpu(), 0.9, 1)
    before = c.records()
    ko, vo = (torch.full((n, 1, 64), 5.0, device="cuda") for _ in range(2))
    F.fvattn_kv4_read(c.cache, c.batch, ko, vo, c.ws(F.FVATTN_OP_KV4_READ, n))
    if cu[0] == 2:
        assert torch.all(cnt[:2] == -5) and torch.all(cnt[2:5] > 0) and torch.all(cnt[5:] == -5)
        assert torch.all(ko[:2] == 5) and torch.all(ko[5:] == 5)
        F.fvattn_kv4_append(c.cache, c.batch, ko, vo, c.ws(F.FVATTN_OP_KV4_APPEND, n))
        c.assert_records(before)                            # what was read is what is written again


@pytest.mark.parametrize("cu,good", [([2, 4, 4, 5], True), ([0, 1, 4, 2], True), ([0, 4, 2, 6], False),
                                     ([-3, 1, 2, 4], False), ([0, 3, 3, 900], False), ([0, 2, 4, -1], False)])
def test_the_calls_agree_on_the_rows(cu, good):
    """All four calls, on both attention kernels and over lists: rows in front of cu[0], of a sequence with a
    negative start and from cu[B] on are left alone, others get their own sequence's results, and starts that
    are negative or fall are recorded."""
    n = 7
    c = Case([300, 200, 150], [1, 1, 1], 1, 64, 64, seed=63, Hq=2)
    kv, k, v = c.kv, c.k, c.v
    ok = lambda ws: (F.fvattn_workspace_status(ws) == F.FVATTN_OK) == good
    owners = [[b for b in range(3) if 0 <= cu[b] <= r < min(cu[b + 1], cu[3])] for r in range(n)]
    free = [r for r in range(n) if not owners[r]]
    sole = [(r, o[0], kv[o[0]] - (cu[o[0] + 1] - r)) for r, o in enumerate(owners) if len(o) == 1]
    assert free or cu[3] > n
    q = torch.randn((n, 2, 64), generator=c.g).to(BF16)
    lists = torch.arange(c.max_pages, dtype=torch.int32, device="cuda").expand(n, 1, -1).contiguous()
    for max_q in (1, 300):
        c.batch = F.KV4Batch(c.table, c.batch.kv_len, torch.tensor(cu, dtype=torch.int32, device="cuda"), max_q)
        runs = [c.attend(q)]
        assert ok(c.last_ws)
        cnt = torch.ones((n, 1), dtype=torch.int32, device="cuda")
        for r, b, pos in sole:
            cnt[r] = pos // 64 + 1
        runs.append(c.attend(q, True, lists, cnt))
        assert ok(c.last_ws)
        for out, lse in runs:
            assert torch.all(out[free] == 77) and torch.all(lse[free] == 77)
            for r, b, pos in sole:
                c.kv, c.nrow = [pos + 1 if i == b else 0 for i in range(3)], [int(i == b) for i in range(3)]
                c.check(q[r:r + 1], out[r:r + 1], lse[r:r + 1])
    idx, cnt = _select(c, q, 0.8, 1)
    assert ok(c.last_ws) and torch.all(cnt[free] == -5) and torch.all(idx[free] == -5)
    for r, b, pos in sole:
        c.kv, c.nrow = [pos + 1 if i == b else 0 for i in range(3)], [int(i == b) for i in range(3)]
        c.k = [x[:max(m, 0)] for x, m in zip(k, c.kv)]
        want = _want_lists(c, q[r:r + 1], 0.8, 1)[0] if pos >= 0 else [[]]      # in front of the sequence: none
        assert [idx[r, 0, :cnt[r, 0]].tolist()] == want
    c.k = k
    ws = c.ws(F.FVATTN_OP_KV4_READ, n)
    ko, vo = (torch.full((n, 1, 64), 5.0, device="cuda") for _ in range(2))
    F.fvattn_kv4_read(c.cache, c.batch, ko, vo, ws)
    assert ok(ws) and torch.all(ko[free] == 5) and torch.all(vo[free] == 5)
    for r, b, pos in sole:
        assert all(np.array_equal(x[r].cpu().numpy(), y[pos] if pos >= 0 else 0 * y[0])
                   for x, y in zip((ko, vo), c.values(b)))
    want = c.records()
    new = torch.randn((n, 1, 64), generator=c.g)
    codes, scales = O.quantize(new.numpy())
    for r, o in enumerate(owners):                          # (a row that two claim is written for each)
        for b in o:
            pos = kv[b] - (cu[b + 1] - r)
            if pos < 0:
                continue
            for i, x in enumerate((codes, scales, codes, scales)):
                want[i][c.table_np[b, pos // 64], :, pos % 64] = x[r]
    F.fvattn_kv4_append(c.cache, c.batch, new.cuda(), new.cuda(), ws)
    assert ok(ws)
    c.assert_records(want)


@pytest.mark.parametrize("rows,over", [(1, 1), (5, 2), (70, 1), (70, 70), (3, 40), (2, (1 << 31) - 1 - 256)])
@pytest.mark.parametrize("block", [64, 128])
def test_longer_than_the_table_row(rows, over, block):
    """Rows keep their positions where a sequence is longer than its table row holds: those behind it are not
    written, read as zeros and choose no page; what is held stays as it is."""
    cap = 256
    c = Case([cap, 90], [rows, 1], 2, 64, block, seed=62, Hq=4)
    c.max_pages = cap // block
    c.table = c.table[:, :c.max_pages].clamp(min=0).contiguous()
    c.batch = c.batch_of([rows, 1], [cap + over, 90])
    fits = max(0, rows - over)                              # rows at positions below cap
    bad = lambda ws: F.fvattn_workspace_status(ws) == F.FVATTN_ERR_INVALID_ARG
    want = c.records()
    k, v = (torch.randn((rows + 1, 2, 64), generator=c.g).to(BF16) for _ in range(2))
    for mine, new in ((c.k, k), (c.v, v)):
        mine[0][cap - fits:] = new[:fits]
        mine[1][89] = new[rows]
    places = [(0, t) for t in range(cap - fits, cap)] + [(1, 89)]
    parts = [c.quantized(b) for b in range(2)]
    for b, t in places:
        for w, x in zip(want, parts[b]):
            w[c.table_np[b, t // block], :, t % block] = x[t]
    ws = c.ws(F.FVATTN_OP_KV4_APPEND, rows + 1)
    F.fvattn_kv4_append(c.cache, c.batch, k.cuda(), v.cuda(), ws)
    assert bad(ws)
    c.assert_records(want)
    ksum, plain = c.cache.ksum.cpu().numpy(), O.dequantize(*parts[0][:2])
    for pg in range(cap // block):
        for h in range(2):
            assert np.array_equal(ksum[c.table_np[0, pg], h], O.page_sum(plain[pg * block:(pg + 1) * block, h]))
    ko, vo = (torch.full((rows + 1, 2, 64), 5.0, device="cuda") for _ in range(2))
    F.fvattn_kv4_read(c.cache, c.batch, ko, vo, ws)
    assert bad(ws) and not ko[fits:rows].any() and not vo[fits:rows].any()
    for got, x in ((ko, 0), (vo, 1)):
        assert np.array_equal(got[:fits].cpu().numpy(), c.values(0)[x][cap - fits:])
        assert np.array_equal(got[rows].cpu().numpy(), c.values(1)[x][89])
    q = c.make_q(spread=4.0)
    live = list(range(fits)) + [rows]
    idx, cnt = _select(c, q, 0.8, 1)
    assert bad(c.last_ws) and not cnt[fits:rows].any()
    lists = idx[:, :, :1].new_zeros((rows + 1, 2, c.max_pages)) + torch.arange(c.max_pages, device="cuda").int()
    full = torch.full((rows + 1, 2), c.max_pages, dtype=torch.int32, device="cuda")
    full[rows] = 2
    outs = [c.attend(q), c.attend(q, True, lists, full)]
    assert bad(c.last_ws)
    c.nrow = [fits, 1]
    got = [[idx[r, h, :cnt[r, h]].tolist() for h in range(2)] for r in live]
    assert got == _want_lists(c, q[live], 0.8, 1)
    for out, lse in outs:
        c.nrow = [fits, 1]
        c.check(q[live], out[live], lse[live])
        c.nrow = [rows - fits, 0]                           # behind the end: all that is held
        c.check(q[fits:rows], out[fits:rows], lse[fits:rows], causal=False)


@pytest.mark.parametrize("start", [-1, -77, -(1 << 28), -(1 << 30), -(1 << 31)])
@pytest.mark.parametrize("G", [1, 8])
def test_negative_row_starts_with_lists(start, G):
    """The sequence is skipped and recorded, however far below 0 its start is (times G it has no 32-bit value)."""
    c = Case([300, 200], [3, 2], 1, 64, 64, seed=61, Hq=G)
    q = c.make_q()
    idx = torch.zeros((5, 1, c.max_pages), dtype=torch.int32, device="cuda")
    idx[:, 0, :2] = torch.tensor([1, 2], dtype=torch.int32)
    cnt = torch.full((5, 1), 2, dtype=torch.int32, device="cuda")
    c.batch.cu[0] = start
    out, lse = c.attend(q, True, idx, cnt)
    assert F.fvattn_workspace_status(c.last_ws) == F.FVATTN_ERR_INVALID_ARG
    assert torch.all(out[:3] == 77) and torch.all(lse[:3] == 77)
    c.kv, c.nrow, c.k, c.v = c.kv[1:], [2], c.k[1:], c.v[1:]
    c.check(q[3:], out[3:], lse[3:], lists=[[[1, 2]], [[1, 2]]])


@pytest.mark.parametrize("block", [64, 128])
def test_more_rows_than_tokens_behind_rows_of_no_sequence(block):
    """A first sequence that starts at row 260 and has more rows than tokens: the tiles of the rows before it
    touch no page (the entries in front of its table row are valid slots here, which would be written)."""
    c = Case([block + 9], [4], 2, 64, block, seed=60)
    wide = torch.arange(5 * c.max_pages, dtype=torch.int32, device="cuda").reshape(5, -1) % c.cache.num_pages
    wide[4] = c.table[0].clamp(min=0)
    one = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    rows, kv = 3 * block, 5
    b = F.KV4Batch(wide[4:], one(kv), one(260, 260 + rows), rows)
    k, v = (torch.randn((260 + rows + 9, 2, 64), generator=c.g).to(BF16) for _ in range(2))
    want = c.records()
    for i, x in enumerate((k, v)):                          # the last five rows are the tokens held
        codes, scales = O.quantize(x[260 + rows - kv:260 + rows].float().numpy())
        for w, y in ((want[2 * i], codes), (want[2 * i + 1], scales)):
            w[c.table_np[0, 0], :, :kv] = y.transpose(1, 0, 2)
    sums = c.cache.ksum.clone()
    ws = c.ws(F.FVATTN_OP_KV4_APPEND, len(k), b)
    F.fvattn_kv4_append(c.cache, b, k.cuda(), v.cuda(), ws)
    assert F.fvattn_workspace_status(ws) == F.FVATTN_ERR_INVALID_ARG
    c.assert_records(want)
    assert torch.equal(sums, c.cache.ksum)


def test_rewriting_what_was_read_changes_nothing():
    """Quantizing stored values gives them back: codes, scales and sums."""
    c = Case([200, 130], [200, 130], 2, 128, 64, seed=49)
    before, sums = c.records(), c.cache.ksum.clone()
    ko, vo = (torch.empty((330, 2, 128), device="cuda") for _ in range(2))
    F.fvattn_kv4_read(c.cache, c.batch, ko, vo, c.ws(F.FVATTN_OP_KV4_READ, 330))
    F.fvattn_kv4_append(c.cache, c.batch, ko, vo, c.ws(F.FVATTN_OP_KV4_APPEND, 330))
    # (a group's largest stored magnitude is 6 scales, so its scale comes out the same)
    full = [int(c.table_np[i, p]) for i, n in enumerate(c.kv) for p in range(n // 64)]
    c.assert_records(before)
    assert torch.equal(sums[full], c.cache.ksum[full])


# ------------------------------------------------------------------ together, streams, graphs, refusals
def _path_inputs(c, rows, seed):
    g = torch.Generator().manual_seed(seed)
    mk = lambda H: torch.randn((rows, H, c.d), generator=g).to(BF16)
    return mk(c.Hq), mk(c.H), mk(c.H)


@pytest.mark.parametrize("p", [None, 0.8])
def test_path_grows_sequences(p):
    """A prompt, then single tokens: every step writes, chooses and attends; the last step's outputs and lists
    against the oracle on everything written."""
    kv, H, Hq, d, block = [150, 201], 2, 6, 64, 64
    c = Case(kv, kv, H, d, block, seed=21, Hq=Hq, fill=False)
    path = F.KV4Path(c.cache, Hq, sum(kv), 2, c.max_pages, BF16, p=p, k_min=1)
    q0 = [torch.randn((n, Hq, d), generator=c.g).mul(4).to(BF16) for n in kv]
    at = [n - 6 for n in kv]
    take = lambda x, lo, hi: torch.cat([t[a:b] for t, a, b in zip(x, lo, hi)]).cuda()
    path(c.batch_of(at, at), take(q0, [0, 0], at), take(c.k, [0, 0], at), take(c.v, [0, 0], at))
    for _ in range(6):
        nxt = [a + 1 for a in at]
        out = path(c.batch_of([1, 1], nxt), take(q0, at, nxt), take(c.k, at, nxt), take(c.v, at, nxt))
        at = nxt
    for ws in (path.ws_append, path.ws_attn) + (() if p is None else (path.ws_select,)):
        assert F.fvattn_workspace_status(ws) == F.FVATTN_OK
    c.nrow, c.rows = [1, 1], 2
    q = take(q0, [n - 1 for n in kv], kv)
    lists = None if p is None else _want_lists(c, q.cpu(), p, 1)
    c.check(q, out, path.lse[:2], lists=lists)


def test_captured_step_follows_the_lengths():
    """One captured step replayed while the lengths, the rows and the inputs change on the device."""
    c = Case([140, 90], [1, 1], 2, 128, 64, seed=22, Hq=8)
    path = F.KV4Path(c.cache, 8, 2, 2, c.max_pages, BF16, p=0.9, k_min=1)
    batch = c.batch_of([1, 1], [100, 50])
    q, k, v = (t.cuda() for t in _path_inputs(c, 2, 1))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        path(batch, q, k, v)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = path(batch, q, k, v)
    other = F.KV4Path(c.cache, 8, 2, 2, c.max_pages, BF16, p=0.9, k_min=1)
    for step, kv in enumerate(([101, 51], [129, 64], [140, 90])):
        batch.kv_len.copy_(torch.tensor(kv, dtype=torch.int32))
        for t, s in zip((q, k, v), _path_inputs(c, 2, 10 + step)):
            t.copy_(s)
        graph.replay()
        got = out.clone()
        want = other(c.batch_of([1, 1], kv), q, k, v)
        assert torch.equal(got, want), kv


def test_captured_step_past_the_tables_end():
    """A captured step replayed until its stream no longer fits its table row: the cache keeps what it held."""
    c = Case([126], [1], 2, 64, 64, seed=66, Hq=4)
    c.table = c.table[:, :2].contiguous()
    batch = F.KV4Batch(c.table, c.batch.kv_len, c.batch.cu, 1)
    path = F.KV4Path(c.cache, 4, 1, 1, 2, BF16, p=0.9)
    q, k, v = (t.cuda() for t in _path_inputs(c, 1, 4))
    path(batch, q, k, v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        path(batch, q, k, v)
        batch.kv_len.add_(1)
    for n in range(126, 133):
        for t, s in zip((q, k, v), _path_inputs(c, 1, n)):
            t.copy_(s)
        graph.replay()
        bad = [F.fvattn_workspace_status(ws) != F.FVATTN_OK for ws in (path.ws_append, path.ws_select, path.ws_attn)]
        assert bad == [n > 128] * 3, n
        if n == 128:
            pages, sums = c.cache.pages.clone(), c.cache.ksum.clone()
    assert torch.equal(pages, c.cache.pages) and torch.equal(sums, c.cache.ksum)


def test_two_calls_at_once_and_repeats_are_bit_identical():
    c = Case([3000, 1700], [1, 1], 2, 128, 64, seed=23, Hq=8)
    d = Case([700, 900], [100, 130], 1, 64, 128, seed=24, Hq=4)
    qc, qd = c.make_q().cuda(), d.make_q().cuda()
    want_c, want_d = c.attend(qc), d.attend(qd)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    wc, wd = c.ws(F.FVATTN_OP_KV4_ATTN, 2), d.ws(F.FVATTN_OP_KV4_ATTN, 230)
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(s1):
            got_c = c.attend(qc, ws=wc)
        with torch.cuda.stream(s2):
            got_d = d.attend(qd, ws=wd)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got_c + got_d, want_c + want_d))


def test_an_explicit_stream_is_used():
    """The call stands behind the work of the stream it names, not of the current one."""
    c = Case([500], [1], 1, 64, 64, seed=25, Hq=4)
    q = c.make_q().cuda()
    want, want_lse = c.attend(q)
    late, out, lse, ws = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(want_lse), c.ws(F.FVATTN_OP_KV4_ATTN, 1)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)                       # some 10 ms
        late.copy_(q)
    F.fvattn_kv4_attn(c.cache, c.batch, late, out, ws, lse=lse, stream=s)
    s.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("fill", [0x00, 0xFF, 0x5E])
def test_what_a_workspace_holds_does_not_matter(rows, fill):
    """Eager calls clear nothing: any bytes may lie there, the parts of other calls too."""
    c = Case([9000, 77], [rows, 1], 2, 128, 128, seed=50, Hq=4)
    q = c.make_q().cuda()
    out, lse = c.attend(q)
    c.check(q.cpu(), out, lse, rows=[0, rows])
    c.last_ws.view(torch.uint8).fill_(fill)
    other = c.make_q(spread=3.0).cuda()
    c.attend(other, ws=c.last_ws)                           # leaves parts of the same units
    again = c.attend(q, ws=c.last_ws)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    assert F.fvattn_workspace_status(c.last_ws) == F.FVATTN_OK


@pytest.mark.parametrize("rows", [1, 40])
def test_replays_and_eager_calls_share_a_workspace(rows):
    """Replays of a captured call share its number; units that several blocks hold are joined right in each,
    with eager calls between, and an error is the last call's only."""
    c = Case([9000, 77], [rows, 1], 2, 128, 128, seed=51, Hq=4)
    q = c.make_q().cuda()
    ws = c.ws(F.FVATTN_OP_KV4_ATTN, rows + 1)
    batch = c.batch_of(c.nrow)
    kv = batch.kv_len.clone()
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    run = lambda: F.fvattn_kv4_attn(c.cache, batch, q, out, ws, lse=lse)
    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for step in range(8):
        q.copy_(c.make_q(spread=1.0 + step))
        bad = step in (2, 3, 6)
        batch.kv_len.copy_(kv)
        if bad:
            batch.kv_len[1] = c.max_pages * c.block + 1     # clamped, and its last page is in no table
        out.fill_(77.0)
        run() if step % 3 == 1 else graph.replay()
        assert F.fvattn_workspace_status(ws) == (F.FVATTN_ERR_INVALID_ARG if bad else F.FVATTN_OK), step
        if not bad:
            want = c.attend(q)
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1]), step
            c.check(q.cpu(), out, lse, rows=[0, rows])


def test_status_of_a_workspace_that_other_calls_use_too():
    """The status is the last call's, whichever kind of call it was."""
    c = Case([300], [2], 1, 64, 64, seed=52, Hq=2)
    q = c.make_q().cuda()
    ws = F.alloc_workspace(1 << 22, "cuda")
    bad = F.KV4Batch(c.table, torch.tensor([-1], dtype=torch.int32, device="cuda"), c.batch.cu, 2)
    out = torch.empty_like(q)
    dense = [torch.randn((1, 1, 128, 64), device="cuda").to(BF16) for _ in range(3)]
    for batch, want in ((bad, F.FVATTN_ERR_INVALID_ARG), (c.batch, F.FVATTN_OK)):
        F.fvattn_kv4_attn(c.cache, batch, q, out, ws)
        assert F.fvattn_workspace_status(ws) == want
        F.fvattn_dense_fwd(*dense, torch.empty_like(dense[0]), 128, 64, ws)
        assert F.fvattn_workspace_status(ws) == F.FVATTN_OK
        F.fvattn_kv4_attn(c.cache, batch, q, out, ws)
        assert F.fvattn_workspace_status(ws) == want
    e = torch.empty((0, 2, 64), dtype=BF16, device="cuda")
    F.fvattn_kv4_attn(c.cache, bad, e, e.clone(), ws)       # a call without rows looks at nothing
    assert F.fvattn_workspace_status(ws) == F.FVATTN_OK


def test_the_path_refuses_before_it_writes():
    c = Case([100, 60], [1, 1], 2, 64, 64, seed=53, Hq=4)
    path = F.KV4Path(c.cache, 4, 2, 2, c.max_pages, BF16, p=0.5)
    q, k, v = (t.cuda() for t in _path_inputs(c, 2, 3))
    before = c.cache.pages.clone()
    for bad in ((q[:1], k, v), (q, k[:1], v[:1]), (q, k, v[:1]), (q.float(), k, v), (q[:, :2], k, v),
                (q.repeat(2, 1, 1), k.repeat(2, 1, 1), v.repeat(2, 1, 1))):
        with pytest.raises((ValueError, TypeError)):
            path(c.batch, *bad)
    assert torch.equal(before, c.cache.pages)


def test_the_path_refuses_layouts_and_sizes_before_it_writes():
    c = Case([100, 60], [1, 1], 2, 64, 64, seed=64, Hq=4)
    make = lambda **kw: F.KV4Path(c.cache, 4, 2, 2, c.max_pages, BF16, **{**dict(p=0.5), **kw})
    path = make()
    q, k, v = (t.cuda() for t in _path_inputs(c, 2, 3))
    pages, sums = c.cache.pages.clone(), c.cache.ksum.clone()
    wide = torch.zeros(2, 4 * 64 + 4, dtype=BF16, device="cuda")
    flat = torch.zeros(2 * 4 * 64 + 8, dtype=BF16, device="cuda")
    for bad in (wide[:, :256].unflatten(1, (4, 64)),                                 # row stride of 520 bytes
                q.transpose(0, 1).contiguous().transpose(0, 1),                      # a row's heads lie apart
                flat[1:513].view(2, 4, 64), path.out, q.cpu()):
        with pytest.raises((ValueError, TypeError)):
            path(c.batch, bad, k, v)
    claims = F.KV4Batch(c.table, c.batch.kv_len, c.batch.cu, 500)
    with pytest.raises(ValueError):
        path(claims, q, k, v)
    for kw in (dict(p=0.0), dict(p=1.5), dict(p=math.nan), dict(k_min=0), dict(scale=-1.0), dict(scale=math.inf)):
        with pytest.raises(ValueError):
            make(**kw)
    assert torch.equal(pages, c.cache.pages) and torch.equal(sums, c.cache.ksum)
    # a larger max_q that asks for no other kernel is none of its business
    want = path(c.batch, q, k, v).clone()
    assert torch.equal(want, path(F.KV4Batch(c.table, c.batch.kv_len, c.batch.cu, 4), q, k, v))


def test_no_rows():
    c = Case([100], [1], 1, 64, 64, seed=26)
    e = torch.empty((0, 1, 64), dtype=BF16, device="cuda")
    b = F.KV4Batch(c.table, c.batch.kv_len, torch.zeros(2, dtype=torch.int32, device="cuda"), 1)
    before = c.cache.pages.clone()
    ws = c.ws(F.FVATTN_OP_KV4_ATTN, 0)
    F.fvattn_kv4_append(c.cache, b, e, e, ws)
    F.fvattn_kv4_read(c.cache, b, e, e.clone(), ws)
    F.fvattn_kv4_attn(c.cache, b, e, e.clone(), ws)
    assert torch.equal(before, c.cache.pages)


def test_the_binding_refuses():
    c = Case([100, 60], [2, 1], 2, 64, 64, seed=27, Hq=4)
    ws = F.alloc_workspace(1 << 20, "cuda")
    q = c.make_q().cuda()
    out = torch.empty_like(q)
    k = torch.zeros((3, 2, 64), dtype=BF16, device="cuda")
    att = lambda **kw: F.fvattn_kv4_attn(**{**dict(cache=c.cache, batch=c.batch, q=q, out=out, workspace=ws), **kw})
    for bad in (dict(out=out.float()), dict(out=out[:2]), dict(q=q.cpu()), dict(q=q.transpose(0, 1)),
                dict(lse=torch.empty((3, 2), device="cuda")), dict(kv_idx=torch.zeros(3, dtype=torch.int32).cuda()),
                dict(workspace=ws.cpu())):
        with pytest.raises((ValueError, TypeError)):
            att(**bad)
    with pytest.raises(F.FVAttnError):
        att(q=q[:, :3].contiguous(), out=out[:, :3].contiguous())     # 3 query heads for 2 KV heads
    with pytest.raises(F.FVAttnError):
        att(out=q)
    with pytest.raises(F.FVAttnError):
        att(scale=-1.0)
    app = lambda **kw: F.fvattn_kv4_append(**{**dict(cache=c.cache, batch=c.batch, k=k, v=k, workspace=ws), **kw})
    for bad in (dict(v=k.float()), dict(k=k[:2]), dict(k=k.half(), v=k.half()), dict(k=k[..., :32]),
                dict(k=torch.zeros((3, 2 * 64 + 4), dtype=BF16, device="cuda")[:, :128].unflatten(1, (2, 64)))):
        with pytest.raises((ValueError, TypeError)):
            app(**bad)
    with pytest.raises(ValueError):
        F.KV4Batch(c.table, c.batch.kv_len[:1], c.batch.cu, 1)
    with pytest.raises(ValueError):
        F.KV4Batch(c.table, c.batch.kv_len, c.batch.cu, 0)
    with pytest.raises(TypeError):
        F.KV4Batch(c.table.long(), c.batch.kv_len, c.batch.cu, 1)
    with pytest.raises(ValueError):
        F.KV4Cache(4, 2, 96, 64)
