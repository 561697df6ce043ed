"""The 4-bit paged key/value cache: what its four operators compute, and the calls that are timed.

A cache is a pool of pages. The page of KV head h in pool slot s is one record of
``block * (d + d / 8)`` bytes, ``block`` tokens long:

    K codes  [block, d / 2]    two E2M1 codes a byte, the even channel in the low four bits
    K scales [block, d / 16]   one E4M3 scale for each 16 channels of a token
    V codes  [block, d / 2]
    V scales [block, d / 16]

and beside it ``ksum`` [slots, H_kv, d] int32: the sum of a full page's stored keys in units of
2^-10 (every E2M1 value times an E4M3 scale is a whole number of these). A code stands for
``E2M1(code) * E4M3(scale) * head_scale``.

Sequences are described by ``table`` [B, max_pages] (pool slots), ``kv_len`` [B] (tokens held, those
of this call among them) and ``cu`` [B + 1] (first row of each sequence in the call's [rows, H, d]
tensors; rows behind ``cu[B]`` are left alone). Row i of sequence b stands at position
``kv_len[b] - rows_b + i``.

    write   quantises K and V of the rows into the pages; then what the pages hold is read back
    read    reads K and V of the rows back
    select  for every row and KV head, the pages whose mean key scores best: the row's own page, and
            before it the smallest set that reaches the mass p of the softmax over the mean keys
            (averaged over the query heads of the KV head), but at least k_min pages
    attend  attention of the rows over the cache, or over the selected pages alone
"""

import math

import numpy as np
import torch

own = False

_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _case(name, op, B, Hq, H, d, block, ctx, q, ragged=0.0, dtype="bf16", causal=True, scaled=False, pad=0,
          pages=0, p=0.9, k_min=4):
    c = dict(op=op, B=B, Hq=Hq, H=H, d=d, block=block, ctx=ctx, q=q, ragged=ragged, dtype=dtype,
             causal=causal, scaled=scaled, pad=pad, pages=pages, p=p, k_min=k_min)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one new token of 48 streams, as after every decoding step of a serving batch
        _case("write-step", "write", 48, 8, 8, 128, 128, 4096, 1, ragged=0.8),
        # three latent frames of 30 x 52 tokens, 40 heads, for two clips: a generated chunk enters the cache
        _case("write-chunk", "write", 2, 40, 40, 128, 128, 9360, 4680, scaled=True),
        # the last tokens of each stream in full precision, for a check or for a re-quantised copy
        _case("read-tail", "read", 16, 4, 4, 64, 64, 1500, 77, ragged=0.5, dtype="fp32", pad=3),
        # a whole clip (21 frames of 30 x 52) back in bf16, for a layer that is not run over the cache
        _case("read-clip", "read", 1, 12, 12, 128, 128, 32760, 32760),
        # one token of each stream chooses its pages
        _case("select-step", "select", 32, 32, 8, 128, 64, 32768, 1, ragged=0.7, k_min=8),
        # half a frame of 30 x 52 chooses its pages in a 720p clip (21 frames of 45 x 80), head by head
        _case("select-frame", "select", 1, 12, 12, 128, 128, 75600, 780, p=0.95, k_min=8),
        # the smallest call: one token, one short stream
        _case("token-short", "attend", 1, 12, 12, 128, 128, 390, 1),
        # a serving batch, five query heads a KV head, lengths between a fifth and all of 32k
        _case("token-batch", "attend", 64, 40, 8, 128, 128, 32768, 1, ragged=0.8),
        # long streams over 64 selected pages of 2,048
        _case("token-selected", "attend", 16, 32, 4, 128, 64, 131072, 1, ragged=0.3, pages=64),
        # five drafted tokens of three streams, single precision, odd lengths
        _case("draft-fp32", "attend", 3, 6, 2, 64, 64, 2001, 5, ragged=0.5, dtype="fp32", scaled=True, pad=2),
        # a prompt's chunk behind a cached prefix, causal, odd lengths
        _case("chunk-prompt", "attend", 2, 40, 8, 128, 128, 9001, 4099, ragged=0.4),
        # three new latent frames of 30 x 52 attend a whole clip and themselves, both ways
        _case("chunk-clip", "attend", 1, 12, 12, 128, 128, 37440, 4680, causal=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One case more, spread over the same ranges."""
    op = rng.choice(("write", "read", "select", "attend", "attend", "attend"))
    H = rng.choice((1, 2, 3, 4, 8, 12))
    Hq = H * rng.choice((1, 1, 2, 4, 5, 7, 8))
    d, block = rng.choice((64, 128)), rng.choice((64, 128))
    ragged, dtype = rng.choice((0.0, 0.3, 0.8)), rng.choice(("bf16", "bf16", "fp32"))
    more = dict(ragged=ragged, dtype=dtype, scaled=rng.random() < 0.3, pad=rng.choice((0, 0, 1, 5)))
    if op in ("write", "read"):
        q = _log(rng, 1, 8192)
        B = rng.randint(1, max(1, min(64, 16384 // q)))
        return _case("", op, B, Hq, H, d, block, q + _log(rng, 1, 4096), q, **more)
    if op == "select":
        q = _log(rng, 1, 512)
        B = rng.randint(1, max(1, min(32, 512 // q)))
        return _case("", op, B, Hq, H, d, block, q + _log(rng, 4096, 40000), q, p=rng.choice((0.5, 0.9, 0.95)),
                     k_min=rng.choice((1, 4, 16)), **more)
    pages = 0
    if rng.random() < 0.5:                       # single tokens and drafts
        q = rng.choice((1, 1, 2, 3, 5))
        B = _log(rng, 1, 48)
        ctx = q + _log(rng, 1, 32768)
        pages = rng.choice((0, 0, 3, 16, 48))
    else:                                        # chunks
        q = _log(rng, 16, 2048)
        B = rng.randint(1, max(1, min(4, 2048 // q)))
        ctx = q + _log(rng, 1, 16384)
        more["dtype"] = "bf16" if q > 256 else dtype
    c = _case("", op, B, Hq, H, d, block, ctx, q, causal=rng.random() < 0.7, pages=pages, **more)
    most = [work(x) for x in listed()]
    while any(work(c)[k] > max(w[k] for w in most) for k in ("bytes", "flops")):
        c["ctx"] = q + (c["ctx"] - q) // 2
    return c


def _lengths(case):
    """Tokens held by, and rows of, every sequence: the case's alone, the same for each seed."""
    kv, rows = [], []
    for b in range(case["B"]):
        f = 1.0 - case["ragged"] * ((b * 0.6180339887) % 1.0)
        n = max(1, int(round(case["q"] * (f if case["q"] > 1 else 1.0))))
        rows.append(n)
        kv.append(max(n, int(round(case["ctx"] * f))))
    return kv, rows


# ---------------------------------------------------------------- the stored form
def _e4m3(codes):
    return codes.view(torch.float8_e4m3fn).float()


def _split(pages, block, d):
    """Views of a record's four parts: [..., block, d / 2] codes and [..., block, d / 16] scales."""
    a, b = block * d // 2, block * d // 16
    parts = (pages[..., :a], pages[..., a:a + b], pages[..., a + b:2 * a + b], pages[..., 2 * a + b:])
    return [x.unflatten(-1, (block, -1)) for x in parts]


def _values(codes, scales):
    """What codes [..., d / 2] with scales [..., d / 16] stand for, before the head's scale: fp32 [..., d]."""
    lut = torch.tensor(_E2M1, device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    x = lut[c.int()].unflatten(-1, (-1, 16))
    return (x * _e4m3(scales.contiguous())[..., None]).flatten(-2)


def _quantise(x):
    """fp32 [..., d] -> codes [..., d / 2], scales [..., d / 16]: the scale is the nearest E4M3 to the group's
    largest magnitude / 6, the code the nearest E2M1 to x / scale, ties to the even code, 6 the largest."""
    g = x.unflatten(-1, (-1, 16))
    s = (g.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    v = s.float()[..., None]
    r = torch.where(v > 0, g.abs() / v, torch.zeros_like(g))
    code = ((r > 0.25).to(torch.uint8) + (r >= 0.75) + (r > 1.25) + (r >= 1.75) + (r > 2.5) + (r >= 3.5) + (r > 5.0))
    code = (code + 8 * (g < 0)).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), s.view(torch.uint8)


# ---------------------------------------------------------------- inputs
def _inputs(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    B, Hq, H, d, block = (case[k] for k in ("B", "Hq", "H", "d", "block"))
    dtype = _TYPES[case["dtype"]]
    kv, nrow = _lengths(case)
    need = [-(-n // block) for n in kv]
    width, slots = max(need), sum(need) + 2
    perm = torch.randperm(slots, generator=gen, device=dev).int()
    table = torch.zeros((B, width), dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    rec = block * (d + d // 8)
    pages = torch.empty((slots, H, rec), dtype=torch.uint8, device=dev)
    ksum = torch.empty((slots, H, d), dtype=torch.int32, device=dev)
    # keys: noise with a few strong channels and a slow drift from page to page; values: noise
    strong = 1.0 + 3.0 * (torch.rand((H, 1, d), generator=gen, device=dev) < 0.04)
    drift = 0.5 * torch.randn((slots, H, 1, d), generator=gen, device=dev)
    step = max(1, (1 << 25) // (H * block * d))
    for i in range(0, slots, step):
        n = min(step, slots - i)
        kc, ks, vc, vs = _split(pages[i:i + n], block, d)
        x = torch.randn((n, H, block, d), generator=gen, device=dev) * strong + drift[i:i + n]
        kc[:], ks[:] = _quantise(x)
        ksum[i:i + n] = (_values(kc, ks).double().sum(-2) * 1024.0).int()
        vc[:], vs[:] = _quantise(torch.randn((n, H, block, d), generator=gen, device=dev))
    scales = [None, None]
    if case["scaled"]:
        scales = [0.5 + torch.rand((H,), generator=gen, device=dev) for _ in range(2)]
    rows = sum(nrow) + case["pad"]
    s = dict(case=case, pages=pages, ksum=ksum, table=table, rows=rows, max_q=max(nrow),
             kv_len=torch.tensor(kv, dtype=torch.int32, device=dev),
             cu=torch.tensor(np.cumsum([0] + nrow), dtype=torch.int32, device=dev),
             k_scale=scales[0], v_scale=scales[1])
    if case["op"] == "write":
        s["k"] = (1.1 * torch.randn((rows, H, d), generator=gen, device=dev)).to(dtype)
        s["v"] = torch.randn((rows, H, d), generator=gen, device=dev).to(dtype)
    if case["op"] in ("select", "attend"):
        # heads from blunt to sharp; each row leans towards the keys of some page of the pool
        tau = torch.exp(torch.rand((1, Hq, 1), generator=gen, device=dev) * math.log(6.0)) * 0.4
        pick = torch.randint(slots, (rows, H), generator=gen, device=dev)
        lean = drift[pick, torch.arange(H, device=dev), 0].repeat_interleave(Hq // H, 1)
        s["q"] = (tau * torch.randn((rows, Hq, d), generator=gen, device=dev) + 2.0 * tau * lean).to(dtype)
    if case["pages"]:
        # lists as the selection gives them: ascending, the row's own page last
        n = case["pages"]
        idx = torch.full((rows, H, width), -1, dtype=torch.int32, device=dev)
        cnt = torch.zeros((rows, H), dtype=torch.int32, device=dev)
        for b in range(B):
            r0 = sum(nrow[:b])
            for i in range(nrow[b]):
                last = (kv[b] - nrow[b] + i) // block
                m = min(n - 1, last)
                some = torch.rand((H, last), generator=gen, device=dev).argsort(-1)[:, :m].sort(-1).values
                idx[r0 + i, :, :m] = some.int()
                idx[r0 + i, :, m] = last
                cnt[r0 + i] = m + 1
        s["idx"], s["cnt"] = idx, cnt
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    dtype, dev = _TYPES[case["dtype"]], s["pages"].device
    rows, H, Hq, d = s["rows"], case["H"], case["Hq"], case["d"]
    s["scale"] = float(np.float32(1.0 / math.sqrt(d)))
    if case["op"] in ("write", "read"):
        s["k_out"] = torch.zeros((rows, H, d), dtype=dtype, device=dev)
        s["v_out"] = torch.zeros((rows, H, d), dtype=dtype, device=dev)
    elif case["op"] == "select":
        s["idx"] = torch.full((rows, H, s["table"].shape[1]), -1, dtype=torch.int32, device=dev)
        s["cnt"] = torch.zeros((rows, H), dtype=torch.int32, device=dev)
    else:
        s["out"] = torch.zeros((rows, Hq, d), dtype=dtype, device=dev)
        s["lse"] = torch.zeros((rows, Hq), dtype=torch.float32, device=dev)
    if own:
        import block_sparse_attention_video_b200 as F
        s["F"] = F
        s["cache"] = F.KV4Cache(s["pages"].shape[0], H, d, case["block"], device=dev, k_scale=s["k_scale"],
                                v_scale=s["v_scale"], pages=s["pages"], ksum=s["ksum"])
        s["batch"] = F.KV4Batch(s["table"], s["kv_len"], s["cu"], s["max_q"])
        op = {"write": F.FVATTN_OP_KV4_APPEND, "read": F.FVATTN_OP_KV4_READ, "select": F.FVATTN_OP_KV4_SELECT,
              "attend": F.FVATTN_OP_KV4_ATTN}[case["op"]]
        s["ws"] = F.alloc_workspace(F.fvattn_kv4_workspace_bytes(op, s["cache"], s["batch"], rows, Hq), dev)
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if own:
        F, cache, batch, ws = s["F"], s["cache"], s["batch"], s["ws"]
        if op == "write":
            F.fvattn_kv4_append(cache, batch, s["k"], s["v"], ws)
        if op in ("write", "read"):
            F.fvattn_kv4_read(cache, batch, s["k_out"], s["v_out"], ws)
        elif op == "select":
            F.fvattn_kv4_select(cache, batch, s["q"], s["case"]["p"], s["case"]["k_min"], s["idx"], s["cnt"], ws,
                                scale=s["scale"])
        else:
            F.fvattn_kv4_attn(cache, batch, s["q"], s["out"], ws, scale=s["scale"], causal=s["case"]["causal"],
                              lse=s["lse"], kv_idx=s.get("idx"), kv_cnt=s.get("cnt"))
    elif op == "write":
        _plain_write(s)
        _plain_read(s)
    elif op == "read":
        _plain_read(s)
    elif op == "select":
        _plain_select(s)
    else:
        _plain_attend(s)
    if op == "write":
        return {"k": s["k_out"], "v": s["v_out"], "ksum": s["ksum"]}
    if op == "read":
        return {"k": s["k_out"], "v": s["v_out"]}
    if op == "select":
        return {"idx": s["idx"], "cnt": s["cnt"]}
    return {"out": s["out"], "lse": s["lse"]}


def _places(s):
    """Row and position of every (sequence, i), i up to the longest's rows; a shorter one's last row repeats."""
    n = (s["cu"][1:] - s["cu"][:-1]).long()[:, None]
    i = torch.minimum(torch.arange(s["max_q"], device=n.device)[None], n - 1)
    return s["cu"][:-1].long()[:, None] + i, s["kv_len"].long()[:, None] - n + i


def _slots(s, pos):
    block = s["case"]["block"]
    return s["table"].long().gather(1, pos // block), pos % block


def _head(scale):
    return 1.0 if scale is None else scale[:, None]


def _plain_write(s):
    block, d = s["case"]["block"], s["case"]["d"]
    row, pos = _places(s)
    page, slot = _slots(s, pos)
    kc, ks, vc, vs = _split(s["pages"], block, d)
    c, e = _quantise(s["k"][row].float() / _head(s["k_scale"]))
    kc[page, :, slot], ks[page, :, slot] = c, e
    c, e = _quantise(s["v"][row].float() / _head(s["v_scale"]))
    vc[page, :, slot], vs[page, :, slot] = c, e
    # sums of the pages that are full now, of those that the rows touch
    last = pos[:, -1:] // block
    j = torch.arange((s["max_q"] + block - 2) // block + 1, device=pos.device)[None]
    j = torch.minimum(pos[:, :1] // block + j, last)
    p = s["table"].long().gather(1, j)
    full = ((j + 1) * block <= s["kv_len"][:, None])[:, :, None, None]
    total = (_values(kc[p], ks[p]).double().sum(-2) * 1024.0).int()
    s["ksum"][p] = torch.where(full, total, s["ksum"][p])


def _plain_read(s):
    row, pos = _places(s)
    page, slot = _slots(s, pos)
    kc, ks, vc, vs = _split(s["pages"], s["case"]["block"], s["case"]["d"])
    k = _values(kc[page, :, slot], ks[page, :, slot]) * _head(s["k_scale"])
    v = _values(vc[page, :, slot], vs[page, :, slot]) * _head(s["v_scale"])
    s["k_out"][row], s["v_out"][row] = k.to(s["k_out"].dtype), v.to(s["v_out"].dtype)


def _plain_select(s):
    """In 64 bits: a page next to the cut has to fall on the right side of it."""
    case, H, block = s["case"], s["case"]["H"], s["case"]["block"]
    row, pos = _places(s)
    width = s["table"].shape[1]
    j = torch.arange(width, device=row.device)
    q = s["q"][row].double().unflatten(2, (H, -1))                               # [B, n, H, G, d]
    k = s["ksum"][s["table"].long()].double()                                    # [B, width, H, d]
    w = s["scale"] / (1024.0 * block) * (1.0 if s["k_scale"] is None else s["k_scale"].double())
    x = torch.einsum("bnhgd,bjhd->bnhgj", q, k) * (w if s["k_scale"] is None else w[:, None, None])
    mine = (pos // block)[:, :, None, None]                                      # the row's own page
    x = x.masked_fill(j >= mine[..., None], -math.inf)
    e = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-1e300))
    z = e.sum(-1, keepdim=True)
    mass = (e / torch.where(z > 0, z, torch.ones_like(z))).mean(3)               # [B, n, H, width]
    mass = mass.masked_fill(j >= mine, -1.0)
    order = mass.sort(dim=-1, descending=True, stable=True)
    p = float(np.float32(case["p"]))
    need = (order.values.clamp(min=0.0).cumsum(-1) < p).sum(-1) + 1
    if p >= 1.0:
        need = need + width
    cnt = torch.minimum(need.clamp(min=case["k_min"]), mine[..., 0])
    rank = torch.empty_like(order.indices).scatter_(-1, order.indices, j.expand_as(order.indices).contiguous())
    keep = ((rank < cnt[..., None]) & (j < mine)) | (j == mine)
    idx = torch.where(keep, j, width).sort(-1).values
    s["idx"][row] = torch.where(idx < width, idx, -1).int()
    s["cnt"][row] = (cnt + 1).int()


def _plain_attend(s):
    case, H, block, d = s["case"], s["case"]["H"], s["case"]["block"], s["case"]["d"]
    row, pos = _places(s)
    n = row.shape[1]
    kc, ks, vc, vs = _split(s["pages"][s["table"].long()].transpose(1, 2), block, d)
    k = (_values(kc, ks) * (1.0 if s["k_scale"] is None else s["k_scale"][:, None, None, None])).flatten(2, 3)
    v = (_values(vc, vs) * (1.0 if s["v_scale"] is None else s["v_scale"][:, None, None, None])).flatten(2, 3)
    q = s["q"][row].float().unflatten(2, (H, -1)).permute(0, 2, 1, 3, 4)         # [B, H, n, G, d]
    G = q.shape[3]
    x = (q.flatten(2, 3) @ k.transpose(-1, -2)).unflatten(2, (n, G)) * s["scale"]
    del k, kc, ks
    t = torch.arange(x.shape[-1], device=x.device)
    seen = pos + 1 if case["causal"] else s["kv_len"].long()[:, None].expand_as(pos)
    hide = (t >= seen[:, :, None])[:, None, :, None]                             # [B, 1, n, 1, keys]
    if s.get("idx") is not None:
        at = torch.arange(s["idx"].shape[-1], device=x.device)
        idx = torch.where(at < s["cnt"][..., None], s["idx"], at.numel()).long()
        listed_ = torch.zeros((*idx.shape[:2], at.numel() + 1), dtype=torch.bool, device=x.device).scatter_(-1, idx, True)
        listed_ = listed_[row][..., :-1].permute(0, 2, 1, 3).repeat_interleave(block, -1)
        hide = hide | ~listed_[:, :, :, None]
    x.masked_fill_(hide, -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-3e38)
    x.sub_(m).exp_()
    z = x.sum(-1, keepdim=True)
    o = (x.flatten(2, 3) @ v).unflatten(2, (n, G)) / torch.where(z > 0, z, torch.ones_like(z))
    s["out"][row] = o.permute(0, 2, 1, 3, 4).flatten(2, 3).to(s["out"].dtype)
    lse = torch.where(z > 0, m + torch.log(z), torch.full_like(z, -math.inf))[..., 0]
    s["lse"][row] = lse.permute(0, 2, 1, 3).flatten(2, 3)


# ---------------------------------------------------------------- cost and truth
def work(case):
    kv, nrow = _lengths(case)
    Hq, H, d, block = (case[k] for k in ("Hq", "H", "d", "block"))
    rows, es = sum(nrow), 2 if case["dtype"] == "bf16" else 4
    token = d + d // 8                                    # bytes of one token's K and V in one head
    if case["op"] == "write":
        # k, v in; codes out and in again; k, v out; the filled pages' older codes in, their sums out
        old = full = 0
        for n, m in zip(kv, nrow):
            a = n // block - (n - m) // block
            full += a
            old += (n - m) % block if a else 0
        return {"bytes": rows * H * (4 * d * es + 2 * token) + H * (old * token // 2 + full * d * 4),
                "flops": rows * H * d * 8}
    if case["op"] == "read":
        return {"bytes": rows * H * (token + 2 * d * es), "flops": rows * H * d * 2}
    if case["op"] == "select":
        pages = sum((n - 1) // block for n in kv)
        pairs = sum((n - m + i) // block for n, m in zip(kv, nrow) for i in range(m))
        return {"bytes": pages * H * d * 4 + rows * Hq * d * es, "flops": pairs * Hq * (2 * d + 20)}
    seen = keys = 0
    for n, m in zip(kv, nrow):
        for i in range(m):
            k = n - m + 1 + i if case["causal"] else n
            if case["pages"]:
                own_page = (n - m + i) // block
                k = min(case["pages"] - 1, own_page) * block + min(block, k - own_page * block)
            seen += k
            keys += k if case["pages"] else 0
        keys += 0 if case["pages"] else n
    return {"bytes": keys * H * token + rows * Hq * (2 * d * es + 4), "flops": seen * Hq * 4 * d}


def _decoded(codes, scales):
    """Codes and scales to 64-bit values, from the formats' bit fields."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).double()
    sign = torch.where(c >= 8, -1.0, 1.0)
    c = c % 8
    e, m = torch.div(c, 2, rounding_mode="floor"), c % 2
    x = sign * torch.where(e == 0, m / 2, torch.exp2(e - 1) * (1 + m / 2))
    b = scales.double()
    e, m = torch.div(b, 8, rounding_mode="floor") % 16, b % 8
    y = torch.where(e == 0, m / 8 * 2.0 ** -6, torch.exp2(e - 7) * (1 + m / 8))
    return x * y.repeat_interleave(16, -1)


def _nearest(x, grid):
    """The nearest value of the ascending grid, of two equally near ones the one with the even index."""
    hi = torch.searchsorted(grid, x.contiguous()).clamp(1, len(grid) - 1)
    a, b = x - grid[hi - 1], grid[hi] - x
    lower = (a < b) | ((a == b) & ((hi - 1) % 2 == 0))
    return grid[torch.where(lower, hi - 1, hi)]


def _stored(x):
    """64-bit values as the cache holds them."""
    dev = x.device
    small = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=dev)
    e, m = torch.meshgrid(torch.arange(16), torch.arange(8), indexing="ij")
    steps = torch.where(e == 0, m / 8 * 2.0 ** -6, torch.exp2(e.double() - 7) * (1 + m / 8)).flatten()[:127].to(dev)
    g = x.unflatten(-1, (-1, 16))
    s = _nearest(g.abs().amax(-1) / 6, steps.double())[..., None]
    y = torch.where(s > 0, _nearest(g.abs() / torch.where(s > 0, s, torch.ones_like(s)), small) * s, torch.zeros_like(g))
    return (y * torch.sign(g)).flatten(-2)


def exact(case, seed):
    if case["op"] == "select":
        return None
    s = _inputs(case, seed)
    H, Hq, d, block = (case[k] for k in ("H", "Hq", "d", "block"))
    dev, G = s["pages"].device, Hq // H
    kv, nrow = _lengths(case)
    start = np.cumsum([0] + nrow)
    one = torch.ones(H, dtype=torch.float64, device=dev)
    hk = one if s["k_scale"] is None else s["k_scale"].double()
    hv = one if s["v_scale"] is None else s["v_scale"].double()
    if case["op"] == "write":
        outs = []
        for x, h in ((s["k"], hk), (s["v"], hv)):
            y = torch.zeros((s["rows"], H, d), dtype=torch.float64, device=dev)
            # the division by the head's scale is the stored value's definition: one rounding to 32 bits
            z = (x[:start[-1]].float() / h.float()[:, None]).double()
            y[:start[-1]] = _stored(z) * h[:, None]
            outs.append(y)
        return {"k": outs[0], "v": outs[1], "ksum": None}
    a, b = block * d // 2, block * d // 16
    parts = [0, a, a + b, 2 * a + b, 2 * a + 2 * b]

    def sequence(i, which):
        rec = s["pages"][s["table"][i, :-(-kv[i] // block)].long()]
        c, e = (rec[..., parts[2 * which + t]:parts[2 * which + t + 1]].unflatten(-1, (block, -1)) for t in (0, 1))
        x = _decoded(c, e).transpose(1, 2).flatten(0, 1)[:kv[i]]                  # [tokens, H, d]
        return x * (hk, hv)[which][:, None]

    if case["op"] == "read":
        outs = []
        for which in (0, 1):
            y = torch.zeros((s["rows"], H, d), dtype=torch.float64, device=dev)
            for i in range(case["B"]):
                y[start[i]:start[i + 1]] = sequence(i, which)[kv[i] - nrow[i]:]
            outs.append(y)
        return {"k": outs[0], "v": outs[1]}
    out = torch.zeros((s["rows"], Hq, d), dtype=torch.float64, device=dev)
    lse = torch.zeros((s["rows"], Hq), dtype=torch.float64, device=dev)
    scale = float(np.float32(1.0 / math.sqrt(d)))
    for i in range(case["B"]):
        k, v = sequence(i, 0), sequence(i, 1)
        key = torch.arange(kv[i], device=dev)
        step = max(1, (1 << 26) // (kv[i] * Hq))
        for r in range(0, nrow[i], step):
            n = min(step, nrow[i] - r)
            rows = slice(start[i] + r, start[i] + r + n)
            q = s["q"][rows].double().unflatten(1, (H, G))
            x = torch.einsum("nhgd,thd->nhgt", q, k) * scale
            at = kv[i] - nrow[i] + r + torch.arange(n, device=dev)
            if case["causal"]:
                x.masked_fill_(key[None, None, None] > at[:, None, None, None], -math.inf)
            if case["pages"]:
                member = torch.zeros((n, H, s["table"].shape[1]), dtype=torch.bool, device=dev)
                for c in range(min(case["pages"], member.shape[-1])):
                    live = c < s["cnt"][rows]
                    page = s["idx"][rows, :, c].long().clamp(min=0)
                    member |= torch.nn.functional.one_hot(page, member.shape[-1]).bool() & live[..., None]
                x.masked_fill_(~member[:, :, key // block][:, :, None], -math.inf)
            z = torch.logsumexp(x, -1)
            out[rows] = torch.einsum("nhgt,thd->nhgd", torch.exp(x - z[..., None]), v).flatten(1, 2)
            lse[rows] = z.flatten(1, 2)
    return {"out": out, "lse": lse}
