"""The decode-step operators around the MoE layer, as measured cases: each in its plain form (elementary
torch operations in 32 bits) and as the calls a user makes of this package.

  norm    residual addition and root-mean-square norm: the new residual stream, the normed rows in bf16
          and, on request, their MXFP8 form (E4M3 codes, one E8M0 scale per 32 columns)
  append  the new tokens' keys and values into a paged cache, kept in bf16 or in MXFP8
  attend  attention of 1..16 new tokens of every request over that cache (causal among the new tokens)
  layer   the whole MoE layer for up to 8 tokens

The MXFP8 outputs are returned as the element values (float8 E4M3) and the scales (float8 E8M0) they are
held as: the value of an element is their product.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one token of a lone request, MoE width of the model this package serves: launch latency
        dict(name="norm-1", op="norm", T=1, d=4096, residual=True, mx=True, w32=False),
        # a verify batch: 64 requests of 8 rows
        dict(name="norm-512", op="norm", T=512, d=4096, residual=True, mx=True, w32=False),
        # a prefill batch, bf16 only (the next reader is a bf16 projection); memory-bound
        dict(name="norm-8192", op="norm", T=8192, d=4096, residual=True, mx=False, w32=True),
        # a verify step's keys and values, 64 requests of 8 rows, quantised
        dict(name="append-64x8-mxfp8", op="append", B=64, L=8, lo=8, hi=4096, kv=8, D=128, page=64, mx=True),
        # a prompt of 8191 tokens on top of a short context, bf16, pages of 16 tokens
        dict(name="append-8191-bf16", op="append", B=1, L=8191, lo=8500, hi=8500, kv=8, D=128, page=16, mx=False),
        # one request that has just begun: latency
        dict(name="attend-1x333", op="attend", B=1, L=1, lo=333, hi=333, kv=8, g=4, D=128, page=16, mx=False),
        # a verify step of 64 requests, contexts of 100 to 8000 tokens, quantised cache
        dict(name="attend-64x8-mxfp8", op="attend", B=64, L=8, lo=100, hi=8000, kv=8, g=4, D=128, page=64, mx=True),
        # few requests with long contexts, one new token each: the length is split over the GPU
        dict(name="attend-3-long", op="attend", B=3, L=1, lo=30001, hi=131071, kv=8, g=8, D=128, page=64, mx=False),
        # many short ragged requests, some still empty, one shared key-value head of 64
        dict(name="attend-200-ragged", op="attend", B=200, L=2, lo=1, hi=1500, kv=1, g=16, D=64, page=48, mx=True),
        # a lone token through a full-size layer
        dict(name="layer-1", op="layer", T=1, d=4096, f=2048, E=256, k=6, shared=True, hash=False),
        # one request's verify rows through a full-size layer
        dict(name="layer-8", op="layer", T=8, d=4096, f=2048, E=256, k=6, shared=True, hash=False),
        # a small hash-routed layer: latency
        dict(name="layer-5-small", op="layer", T=5, d=256, f=128, E=8, k=2, shared=True, hash=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    while True:
        c = _draw(rng)
        sizes = [v for v in c.values() if isinstance(v, int)]
        sizes += [a * b for i, a in enumerate(sizes) for b in sizes[:i]] + [2 * c.get("f", 0)]
        if 3072 not in sizes:
            return c


def _draw(rng):
    op = rng.choice(["norm", "append", "attend", "layer"])
    if op == "norm":
        T, mx = _log_int(rng, 1, 8192), rng.random() < 0.6
        d = 32 * _log_int(rng, 2, 256) if mx else 8 * _log_int(rng, 4, 1024)
        return dict(op=op, T=max(1, min(T, 8192 * 4096 // d)), d=d, residual=rng.random() < 0.8, mx=mx,
                    w32=rng.random() < 0.5)
    kv, D = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    page, mx = rng.choice([16, 32, 48, 64, 128]), rng.random() < 0.5
    if op == "append":
        B = _log_int(rng, 1, 128)
        L = _log_int(rng, 1, max(1, 8191 // B))
        lo = rng.choice([0, 1, L, L + 7])
        return dict(op=op, B=B, L=L, lo=lo, hi=lo + _log_int(rng, 1, 2000), kv=kv, D=D, page=page, mx=mx)
    if op == "attend":
        B, L = _log_int(rng, 1, 200), rng.choice([1, 1, 2, 3, 5, 8, 16])
        g = rng.choice([1, 2, 4, 7, 8, 16])
        # at most the largest listed case's cache (about 2.2 G tokens x heads x columns)
        hi = _log_int(rng, 64, max(65, min(100000, 200_000 * 8 // (B * kv))))
        lo = rng.choice([0, 1, hi // 7, hi // 2, hi])
        rows = B * hi * kv * g * L
        while rows > 64 * 8000 * 8 * 32 // 2 and L > 1:  # and of its score matrix
            L -= 1
            rows = B * hi * kv * g * L
        return dict(op=op, B=B, L=L, lo=lo, hi=hi, kv=kv, g=g, D=D, page=page, mx=mx)
    E = _log_int(rng, 1, 256)
    return dict(op=op, T=rng.randint(1, 8), d=256 * rng.randint(1, 16), f=128 * rng.randint(1, 16), E=E,
                k=rng.randint(1, min(8, E)), shared=rng.random() < 0.7, hash=rng.random() < 0.3)


def _lens(c):
    """Context lengths of the requests, spread evenly over the logarithm of their range (the same for every
    seed); where the range begins at 0, every seventh request is still empty."""
    B, lo, hi = c["B"], c["lo"], c["hi"]
    a, b = max(lo, 1), max(hi, 1)
    lens = [round(a * (b / a) ** (i / max(B - 1, 1))) if B > 1 else b for i in range(B)]
    if lo <= 1 < hi and B > 1:
        lens = [0 if i % 7 == 3 else n for i, n in enumerate(lens)]
    order = random.Random(B * 1000003 + hi).sample(range(B), B)
    return [lens[i] for i in order]


# ------------------------------------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device=DEV, dtype=F32) * std


def _inputs(case, seed):
    """The operator's inputs, made from the seed alone."""
    c, g = case, _gen(seed)
    if c["op"] == "norm":
        T, d = c["T"], c["d"]
        # hidden states: a few columns are much larger than the rest
        col = torch.exp(0.7 * _randn(g, d))
        s = dict(x=(_randn(g, T, d) * col).to(BF), weight=1.0 + 0.2 * _randn(g, d), eps=1e-6, residual=None)
        if not c["w32"]:
            s["weight"] = s["weight"].to(BF)
        if c["residual"]:
            s["residual"] = (3.0 * _randn(g, T, d) * col).to(BF)
        return s
    if c["op"] == "layer":
        return _layer_inputs(c, g)
    B, L, kv, D, page = c["B"], c["L"], c["kv"], c["D"], c["page"]
    lens = _lens(c)
    per = [-(-n // page) for n in lens]
    need = sum(per)
    n_pages = need + 3
    # the pages of a request lie anywhere in the pool; unused table entries hold no page
    perm = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32).cpu().numpy()
    table = np.full((B, max(max(per), 1) + 1), -1, np.int32)
    at = np.concatenate([[0], np.cumsum(per)])
    col = np.arange(need) - np.repeat(at[:-1], per)
    table[np.repeat(np.arange(B), per), col] = perm[:need]
    s = dict(table=torch.from_numpy(table).to(DEV), lens=torch.tensor(lens, dtype=torch.int32, device=DEV),
             max_len=max(lens), k_s=None, v_s=None)
    # keys have columns of very different sizes, as after a trained projection
    kcol = torch.exp(0.5 * _randn(g, kv, D))
    shape = (n_pages, page, kv, D)
    if c["op"] == "append":
        qkv = torch.cat([_randn(g, B * L, 4 * kv * D, std=1.0), _randn(g, B * L, kv * D) * kcol.reshape(-1),
                         _randn(g, B * L, kv * D)], 1).to(BF)
        # views of the fused projection's output
        s["k_new"] = qkv[:, 4 * kv * D:5 * kv * D].unflatten(0, (B, L)).unflatten(-1, (kv, D))
        s["v_new"] = qkv[:, 5 * kv * D:].unflatten(0, (B, L)).unflatten(-1, (kv, D))
        if c["mx"]:
            s["k"] = torch.zeros(shape, dtype=torch.uint8, device=DEV)
            s["v"] = torch.zeros(shape, dtype=torch.uint8, device=DEV)
            s["k_s"] = torch.zeros(shape[:3] + (D // 32,), dtype=torch.uint8, device=DEV)
            s["v_s"] = torch.zeros(shape[:3] + (D // 32,), dtype=torch.uint8, device=DEV)
        else:
            s["k"] = torch.zeros(shape, dtype=BF, device=DEV)
            s["v"] = torch.zeros(shape, dtype=BF, device=DEV)
        return s
    s["q"] = _randn(g, B, L, kv * c["g"], D, std=1.5).to(BF)
    s["scale"] = D ** -0.5
    if c["mx"]:
        code = lambda: torch.randn(shape, generator=g, device=DEV, dtype=BF).mul_(100).clamp_(-448, 448).to(  # noqa: E731
            torch.float8_e4m3fn).view(torch.uint8)
        s["k"], s["v"] = code(), code()
        s["k_s"] = (120 + torch.randint(-1, 2, shape[:3] + (D // 32,), generator=g, device=DEV)).to(torch.uint8)
        s["v_s"] = (120 + torch.randint(-1, 2, shape[:3] + (D // 32,), generator=g, device=DEV)).to(torch.uint8)
    else:
        s["k"] = torch.randn(shape, generator=g, device=DEV, dtype=BF).mul_(kcol.to(BF))
        s["v"] = torch.randn(shape, generator=g, device=DEV, dtype=BF)
    # what an earlier user of the pool left behind the requests' ends: no reader may let it through
    stale = torch.ones(n_pages, page, dtype=torch.bool, device=DEV)
    left = torch.from_numpy(np.repeat(lens, per) - col * page).to(DEV)  # rows of each page that are in use
    stale[torch.from_numpy(perm[:need].astype(np.int64)).to(DEV)] = torch.arange(page, device=DEV) >= left[:, None]
    for name in ("k", "v"):
        s[name].masked_fill_(stale[..., None, None], 0x7F if c["mx"] else float("nan"))
    return s


def _experts(g, n, d, f):
    def scales(rows, K):
        e0 = math.floor(math.log2(1.0 / (2.93 * math.sqrt(d))))
        return (127 + e0 + torch.randint(0, 2, (n, rows, K // 32), generator=g, device=DEV)).to(torch.uint8)

    def codes(rows, K):
        return torch.randint(0, 256, (n, rows, K // 2), generator=g, device=DEV, dtype=torch.uint8)

    return dict(w13=codes(2 * f, d), s13=scales(2 * f, d), w2=codes(d, f), s2=scales(d, f))


def _layer_inputs(c, g):
    T, d, f, E, k = c["T"], c["d"], c["f"], c["E"], c["k"]
    s = dict(x=_randn(g, T, d).to(BF), experts=_experts(g, E, d, f), shared=_experts(g, 1, d, f) if c["shared"] else None,
             scale=1.5, limit=10.0, k=k, rw=None, rb=None, table=None, tok=None)
    if c["hash"]:
        V = 4096
        s["table"] = torch.rand(V, E, generator=g, device=DEV).argsort(1)[:, :k].to(torch.int32).contiguous()
        s["tok"] = torch.randint(0, V, (T,), generator=g, device=DEV).to(torch.int32)
    else:
        s["rw"] = _randn(g, E, d, std=d ** -0.5)
        s["rb"] = torch.rand(E, generator=g, device=DEV) * 0.2 - 0.1
    return s


def prepare(case, seed):
    c, s = case, _inputs(case, seed)
    s["case"] = c
    if c["op"] == "norm":
        T, d = c["T"], c["d"]
        s["sum"] = torch.empty(T, d, dtype=BF, device=DEV) if c["residual"] else None
        s["y"] = torch.empty(T, d, dtype=BF, device=DEV)
        s["y_q"] = torch.empty(T, d, dtype=torch.uint8, device=DEV) if c["mx"] else None
        s["y_s"] = torch.empty(T, d // 32, dtype=torch.uint8, device=DEV) if c["mx"] else None
    if c["op"] == "attend":
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(s["q"].shape[:3], dtype=F32, device=DEV)
    if c["op"] == "layer":
        s["out"] = torch.empty_like(s["x"])
        s["ids"] = torch.empty(c["T"], c["k"], dtype=torch.int32, device=DEV)
        s["wts"] = torch.empty(c["T"], c["k"], dtype=F32, device=DEV)
    if own:
        import block_scaled_fp4_sqrt_gb300 as moe
        s["moe"] = moe
        if c["op"] in ("append", "attend"):
            s["cache"] = moe.PagedKVCache(s["k"], s["v"], s["table"], s["lens"], s["k_s"], s["v_s"])
        if c["op"] == "layer":
            ex = moe.DeviceExperts(**s["experts"])
            sh = None if s["shared"] is None else moe.DeviceExperts(**s["shared"])
            s["layer"] = moe.MoELayer(c["d"], c["f"], c["E"], c["k"], ex, sh, s["rw"], s["rb"], s["table"], max_T=8,
                                      route_scale=s["scale"], swiglu_limit=s["limit"], device=DEV,
                                      resident_router=not c["hash"])
    return s


# ------------------------------------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if op == "norm":
        if own:
            s["moe"].moe_add_rms_norm(s["x"], s["residual"], s["weight"], s["eps"], s["sum"], s["y"], s["y_q"], s["y_s"])
            out = dict(y=s["y"])
            if s["sum"] is not None:
                out["sum"] = s["sum"]
            if s["y_q"] is not None:
                out["q"], out["s"] = s["y_q"].view(torch.float8_e4m3fn), s["y_s"].view(torch.float8_e8m0fnu)
            return out
        return _plain_norm(s)
    if op == "append":
        if own:
            s["cache"].append(s["k_new"], s["v_new"])
        else:
            _plain_append(s)
        if s["k_s"] is None:
            return dict(k=s["k"], v=s["v"])
        e4, e8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
        return dict(k=s["k"].view(e4), v=s["v"].view(e4), k_s=s["k_s"].view(e8), v_s=s["v_s"].view(e8))
    if op == "attend":
        if own:
            s["cache"].attend(s["q"], s["out"], s["lse"], s["scale"])
            return dict(out=s["out"], lse=s["lse"])
        return _plain_attend(s)
    if own:
        s["layer"].forward_few(s["x"], s["tok"], s["out"], s["ids"], s["wts"])
        return dict(out=s["out"], ids=s["ids"], wts=s["wts"])
    return _plain_layer(s)


def _pow2(e):
    """2^e in fp32 for integer e in [-126, 127], from its bits."""
    return ((e.to(torch.int32) + 127) << 23).view(F32)


def _mx(v):
    """MXFP8 of fp32 v along its last dimension: (element values in block units, exponents)."""
    b = v.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1, keepdim=True)
    e = (torch.frexp(amax)[1] - 9).clamp(-127, 127)
    e = torch.where(amax > 0, e, torch.full_like(e, -127))
    u = b * _pow2(torch.clamp(-e, max=127))
    return u.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).flatten(-2), e.squeeze(-1)


def _plain_norm(s):
    x = s["x"].float()
    t = x if s["residual"] is None else x + s["residual"].float()
    r = torch.rsqrt((t * t).mean(-1, keepdim=True) + s["eps"])
    out = dict(y=(t * r * s["weight"].float()).to(BF))
    if s["residual"] is not None:
        out["sum"] = t.to(BF)
    if s["y_q"] is not None:  # the codes of the bf16 rows, as the expert layer would make them
        q, e = _mx(out["y"].float())
        out["q"], out["s"] = q, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    return out


def _plain_append(s):
    B, L = s["k_new"].shape[:2]
    page = s["k"].shape[1]
    pos = s["lens"].long()[:, None] - L + torch.arange(L, device=DEV)
    ok = pos >= 0
    pages = s["table"].long().gather(1, (pos.clamp(min=0) // page))
    at = (pages[ok], pos[ok] % page)
    for new, dst, sc in (("k_new", "k", "k_s"), ("v_new", "v", "v_s")):
        v = s[new][ok]
        if s[sc] is None:
            s[dst][at] = v
        else:
            q, e = _mx(v.float())
            s[dst][at] = q.view(torch.uint8)
            s[sc][at] = (e + 127).to(torch.uint8)


def _plain_attend(s):
    B, L, Hq, D = s["q"].shape
    page, kv = s["k"].shape[1:3]
    n, g = max(s["max_len"], 1), Hq // kv
    pos = torch.arange(n, device=DEV)
    lens = s["lens"].long()
    live = pos < lens[:, None]
    pages = s["table"].long()[:, pos // page]
    pages = torch.where(live, pages, torch.zeros_like(pages))

    def rows(codes, scales):
        r = codes[pages, pos % page]
        if scales is not None:
            r = r.view(torch.float8_e4m3fn).float().unflatten(-1, (-1, 32))
            r = (r * _pow2(scales[pages, pos % page].int() - 127)[..., None]).flatten(-2)
        r = torch.where(live[..., None, None], r.float(), torch.zeros((), device=DEV))
        return r.transpose(1, 2)  # [B, kv, n, D]

    q = s["q"].float().unflatten(2, (kv, g)).permute(0, 2, 1, 3, 4).reshape(B, kv, L * g, D)
    sc = torch.matmul(q, rows(s["k"], s["k_s"]).transpose(2, 3)).mul_(s["scale"]).unflatten(2, (L, g))
    limit = lens[:, None] - L + 1 + torch.arange(L, device=DEV)  # row l sees positions below limit
    sc.masked_fill_((pos >= limit[..., None])[:, None, :, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    p = sc.sub_(torch.where(m > -math.inf, m, torch.zeros_like(m))).exp_()
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), rows(s["v"], s["v_s"])).unflatten(2, (L, g))
    o = torch.where(z > 0, o / z, torch.zeros_like(o)).permute(0, 2, 1, 3, 4)
    lse = (m + z.log()).squeeze(-1).permute(0, 2, 1, 3)
    return dict(out=o.reshape(B, L, Hq, D).to(BF), lse=lse.reshape(B, L, Hq))


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _fp4_rows(codes, scales):
    """MXFP4 codes [..., K/2] and scale bytes [..., K/32] as fp32 [..., K]."""
    lut = torch.tensor([[E2M1[b & 15], E2M1[b >> 4]] for b in range(256)], dtype=F32, device=codes.device)
    v = lut[codes.int()].flatten(-2).unflatten(-1, (-1, 32))
    return (v * _pow2(scales.int() - 127)[..., None]).flatten(-2)


def _mx_rows(v):
    q, e = _mx(v)
    return (q.float().unflatten(-1, (-1, 32)) * _pow2(e.clamp(min=-126))[..., None]).flatten(-2)


def _plain_layer(s):
    x, k = s["x"].float(), s["k"]
    T = x.shape[0]
    if s["table"] is not None:
        ids = s["table"][s["tok"].long()].long().sort(1)[0]
        w = torch.full((T, k), s["scale"] / k, dtype=F32, device=DEV)
    else:
        l = torch.matmul(x, s["rw"].t())
        score = torch.sqrt(l.clamp(min=0) + torch.log1p(torch.exp(-l.abs())))
        ids = torch.sort(score + s["rb"], dim=1, descending=True, stable=True)[1][:, :k].sort(1)[0]
        w = score.gather(1, ids)
        w = s["scale"] * w / w.sum(1, keepdim=True)

    def ffn(e, rows, xr):
        h = torch.matmul(_fp4_rows(e["w13"][rows], e["s13"][rows]), xr[..., None]).squeeze(-1)
        gate, up = h.chunk(2, -1)
        gate, up = gate.clamp(max=s["limit"]), up.clamp(-s["limit"], s["limit"])
        h = _mx_rows(gate / (1 + torch.exp(-gate)) * up)
        return torch.matmul(_fp4_rows(e["w2"][rows], e["s2"][rows]), h[..., None]).squeeze(-1)

    xr = _mx_rows(x)
    y = (ffn(s["experts"], ids.reshape(-1), xr.repeat_interleave(k, 0)) * w.reshape(-1, 1)).unflatten(0, (T, k)).sum(1)
    if s["shared"] is not None:
        y = y + ffn(s["shared"], torch.zeros(T, dtype=torch.long, device=DEV), xr)
    return dict(out=y.to(BF), ids=ids.to(torch.int32), wts=w)


# ------------------------------------------------------------------------------------------------ work
def work(case):
    c = case
    if c["op"] == "norm":
        T, d = c["T"], c["d"]
        b = 2 * T * d * 2 + (4 if c["w32"] else 2) * d
        b += 2 * T * d * 2 if c["residual"] else 0
        b += T * d + T * d // 32 if c["mx"] else 0
        return dict(bytes=b, flops=5 * T * d)
    if c["op"] == "layer":
        T, d, f, E, k = c["T"], c["d"], c["f"], c["E"], c["k"]
        touched = E * (1 - (1 - k / E) ** T) + (1 if c["shared"] else 0)  # expected distinct experts
        b = touched * 3 * d * f * (1 / 2 + 1 / 32) + 4 * T * d + 8 * T * k
        b += 4 * T * (1 + k) if c["hash"] else 4 * E * d + 4 * E
        rows = T * (k + (1 if c["shared"] else 0))
        return dict(bytes=b, flops=6 * rows * d * f + (0 if c["hash"] else 2 * T * E * d))
    el = 1 + 1 / 32 if c["mx"] else 2
    B, L, kv, D, lens = c["B"], c["L"], c["kv"], c["D"], _lens(c)
    if c["op"] == "append":
        n = sum(min(L, x) for x in lens)
        return dict(bytes=2 * n * kv * D * (2 + el) + 8 * B, flops=2 * n * kv * D)
    pages = sum(-(-x // c["page"]) for x in lens)
    rows = B * L * kv * c["g"]
    seen = sum(max(x - L + 1 + i, 0) for x in lens for i in range(L))
    return dict(bytes=2 * sum(lens) * kv * D * el + 4 * pages + 4 * B + rows * (4 * D + 4),
                flops=4 * seen * kv * c["g"] * D)


# ------------------------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """What run() returns, from the definitions in 64 bits.  Values that are rounded to 16 or 8 bits at the
    end are given before that rounding."""
    c, s = case, _inputs(case, seed)
    return {"norm": _exact_norm, "append": _exact_append, "attend": _exact_attend, "layer": _exact_layer}[c["op"]](c, s)


def _block_exponent(a):
    """floor(log2 a) - 8 of the block maxima a (fp64), -127 where a block is all zero."""
    m, e = torch.frexp(a)
    return torch.where(a > 0, (e - 9).clamp(-127, 127), torch.full_like(e, -127))


def _in_block_units(v):
    b = v.reshape(*v.shape[:-1], v.shape[-1] // 32, 32)
    e = _block_exponent(b.abs().amax(-1))
    return (b * torch.exp2(-e.double())[..., None]).clamp(-448, 448).reshape(v.shape), e


def _exact_norm(c, s):
    t = s["x"].double()
    out = {}
    if c["residual"]:
        t = t + s["residual"].double()
        out["sum"] = t
    y = t / torch.sqrt(torch.sum(t * t, 1, keepdim=True) / c["d"] + s["eps"]) * s["weight"].double()
    out["y"] = y
    if c["mx"]:
        q, e = _in_block_units(y)
        out["q"], out["s"] = q, torch.exp2(e.double())
    return out


def _exact_append(c, s):
    B, L, page = c["B"], c["L"], c["page"]
    lens, table = s["lens"].cpu().numpy().astype(np.int64), s["table"].cpu().numpy()
    b, l = np.divmod(np.arange(B * L), L)
    pos = lens[b] - L + l
    b, l, pos = b[pos >= 0], l[pos >= 0], pos[pos >= 0]
    page_at = torch.from_numpy(table[b, pos // page].astype(np.int64)).to(DEV)
    row = torch.from_numpy(pos % page).to(DEV)
    b, l = torch.from_numpy(b).to(DEV), torch.from_numpy(l).to(DEV)
    out = {}
    for name in ("k", "v"):
        new = s[name + "_new"][b, l].double()
        full = torch.zeros(s[name].shape, dtype=F64, device=DEV)
        if c["mx"]:
            q, e = _in_block_units(new)
            sc = torch.full(s[name + "_s"].shape, 2.0 ** -127, dtype=F64, device=DEV)
            sc[page_at, row] = torch.exp2(e.double())
            full[page_at, row] = q
            out[name], out[name + "_s"] = full, sc
        else:
            full[page_at, row] = new
            out[name] = full
    return out


def _exact_attend(c, s):
    B, L, kv, g, D, page = c["B"], c["L"], c["kv"], c["g"], c["D"], c["page"]
    out = torch.zeros(B, L, kv * g, D, dtype=F64, device=DEV)
    lse = torch.full((B, L, kv * g), -math.inf, dtype=F64, device=DEV)
    lens, table = s["lens"].tolist(), s["table"].cpu()
    for b, n in enumerate(lens):
        if n == 0:
            continue
        pages = table[b, : -(-n // page)].long().to(DEV)

        def seq(codes, scales):
            r = codes[pages].reshape(-1, kv, D)[:n]
            if scales is None:
                return r.double()
            e = scales[pages].reshape(-1, kv, D // 32)[:n].double() - 127
            return (r.view(torch.float8_e4m3fn).double().reshape(n, kv, D // 32, 32) * torch.exp2(e)[..., None]).reshape(n, kv, D)

        K, V = seq(s["k"], s["k_s"]), seq(s["v"], s["v_s"])
        for l in range(L):
            end = n - L + 1 + l
            if end <= 0:
                continue
            q = s["q"][b, l].double().reshape(kv, g, D)
            t = torch.einsum("hgd,thd->hgt", q, K[:end]) / math.sqrt(D)
            z = torch.logsumexp(t, -1)
            lse[b, l] = z.reshape(-1)
            out[b, l] = torch.einsum("hgt,thd->hgd", torch.exp(t - z[..., None]), V[:end]).reshape(kv * g, D)
    return dict(out=out, lse=lse)


def _round_e4m3(v):
    """Nearest E4M3 value of fp64 v with ties to even, |v| <= 448 after saturation."""
    v = v.clamp(-448, 448)
    e = torch.frexp(v)[1].clamp(min=-5) - 1  # floor(log2 |v|), at least -6
    step = torch.exp2((e - 3).double())
    return torch.round(v / step) * step  # torch.round: half to even


def _mxfp8_64(v):
    u, e = _in_block_units(v)
    u = _round_e4m3(u)
    return (u.reshape(*e.shape, 32) * torch.exp2(e.double())[..., None]).reshape(v.shape)


def _fp4_64(codes, scales):
    mag = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=F64, device=DEV)
    nib = torch.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    val = mag[(nib & 7).long()] * torch.where(nib >= 8, -1.0, 1.0).double()
    return val * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


def _exact_layer(c, s):
    T, k = c["T"], c["k"]
    x = s["x"].double()
    ids, wts = [], []
    for t in range(T):
        if c["hash"]:
            chosen = sorted(s["table"][int(s["tok"][t])].tolist())
            weight = [s["scale"] / k] * k
        else:
            l = (s["rw"].double() * x[t]).sum(1)
            score = torch.sqrt(torch.logaddexp(l, torch.zeros_like(l)))
            key = (score + s["rb"].double()).tolist()
            chosen = sorted(sorted(range(c["E"]), key=lambda e: (-key[e], e))[:k])
            total = sum(float(score[e]) for e in chosen)
            weight = [s["scale"] * float(score[e]) / total for e in chosen]
        ids.append(chosen)
        wts.append(weight)
    xq = _mxfp8_64(x)
    out = torch.zeros_like(x)

    def add(e, i, tokens, weight):
        h = xq[tokens] @ _fp4_64(e["w13"][i], e["s13"][i]).t()
        a, b = h[:, : c["f"]], h[:, c["f"]:]
        a, b = a.clamp(max=s["limit"]), b.clamp(-s["limit"], s["limit"])
        h = _mxfp8_64(a * torch.sigmoid(a) * b)
        out[tokens] += weight[:, None] * (h @ _fp4_64(e["w2"][i], e["s2"][i]).t())

    for i in sorted({e for row in ids for e in row}):
        at = [(t, wts[t][row.index(i)]) for t, row in enumerate(ids) if i in row]
        add(s["experts"], i, torch.tensor([t for t, _ in at], device=DEV), torch.tensor([w for _, w in at], dtype=F64, device=DEV))
    if s["shared"] is not None:
        add(s["shared"], 0, torch.arange(T, device=DEV), torch.ones(T, dtype=F64, device=DEV))
    return dict(out=out, ids=None, wts=torch.tensor(wts, dtype=F64, device=DEV))
