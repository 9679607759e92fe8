"""The operators around the paged cache of a decode step, as measured cases: each in its plain form (elementary
torch operations in 32 bits) and as the calls a user makes of this package.

  attend  attention of the newest tokens of every request over a paged cache held in 4 bits (MXFP4: E2M1 codes,
          two a byte, one E8M0 scale per 32 columns)
  rope    root-mean-square norms of every query and key head with the position rotation in the same pass (one or
          several position axes), the keys and values written into a paged cache in its format on request
  pages   the cache's pages: branches that share pages (fork), growth with copy on write, truncation (resize),
          compaction, and the copies of page contents in all layers that these ask for

Cache contents in 4 bits are returned as the values they stand for in their block's units (float8 E4M3 holds every
E2M1 value) and the scales (float8 E8M0).
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
BF, F32, F64, I32, U8 = torch.bfloat16, torch.float32, torch.float64, torch.int32, torch.uint8
E4, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one request that has just begun: latency
        dict(name="attend-1x333", op="attend", B=1, L=1, lo=333, hi=333, kv=8, g=4, D=128, page=16),
        # a decode step of 64 requests, contexts of 100 to 8000 tokens
        dict(name="attend-64x1", op="attend", B=64, L=1, lo=100, hi=8000, kv=8, g=4, D=128, page=64),
        # a verify step of the same requests, eight rows each
        dict(name="attend-64x8", op="attend", B=64, L=8, lo=100, hi=8000, kv=8, g=4, D=128, page=64),
        # few requests with long contexts: the length is split over the GPU
        dict(name="attend-3-long", op="attend", B=3, L=1, lo=30001, hi=131071, kv=8, g=8, D=128, page=64),
        # a chunk of two prompts over what is cached already, heads of 64: bound by the products
        dict(name="attend-2x500", op="attend", B=2, L=500, lo=1500, hi=3001, kv=4, g=4, D=64, page=48),
        # one token of a lone request, 32 query and 8 key-value heads, into a bf16 cache: launch latency
        dict(name="rope-1", op="rope", B=1, L=1, lo=2000, hi=2000, hq=32, kv=8, D=128, rot=128, norm=True, axes=1,
             pairs="half", fmt="bf16", page=64),
        # a verify step's rows, 64 requests of 8, into a quantised cache
        dict(name="rope-64x8-mxfp8", op="rope", B=64, L=8, lo=8, hi=4096, hq=32, kv=8, D=128, rot=128, norm=True,
             axes=1, pairs="half", fmt="mxfp8", page=64),
        # a prompt far into its context, half of every head rotated, into a 4-bit cache
        dict(name="rope-4099-mxfp4", op="rope", B=1, L=4099, lo=120000, hi=120000, hq=32, kv=8, D=128, rot=64,
             norm=True, axes=1, pairs="adjacent", fmt="mxfp4", page=64),
        # image and video tokens: time, height and width, no cache, keys in place of the cache as rows
        dict(name="rope-8191-3d", op="rope", B=1, L=8191, lo=0, hi=0, hq=32, kv=8, D=128, rot=128, norm=True, axes=3,
             pairs="half", fmt="none", page=16),
        # four requests branch, all grow by a verify step's tokens: latency
        dict(name="pages-branch-4", op="pages", job="branch", B=4, lo=50, hi=900, page=16, pool=512, L=8, layers=2,
             kv=2, D=64, fmt="mxfp8"),
        # a full server: 512 requests, half of them with a branch, a pool of 200,000 pages
        dict(name="pages-branch-512", op="pages", job="branch", B=512, lo=100, hi=8000, page=16, pool=200000, L=8,
             layers=1, kv=1, D=64, fmt="mxfp8"),
        # requests have left: a fragmented pool moves together, contents of two layers
        dict(name="pages-compact", op="pages", job="compact", B=64, lo=100, hi=8000, page=64, pool=4000, L=0, layers=2,
             kv=8, D=128, fmt="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["attend", "rope", "pages"])
    D, page = rng.choice([64, 128]), rng.choice([16, 32, 48, 64, 128])
    kv = rng.choice([1, 2, 4, 8])
    if op == "attend":
        B, L, g = _log_int(rng, 1, 200), rng.choice([1, 1, 2, 3, 5, 8, 16, _log_int(rng, 17, 700)]), rng.choice([1, 2, 4, 7, 8, 16])
        # at most the largest listed case's cache (about 1.5 G columns of keys) and score matrices
        hi = _log_int(rng, 64, max(65, min(131071, 200_000 * 8 // (B * kv))))
        lo = rng.choice([0, 1, hi // 7, hi // 2, hi])
        while B * hi * kv * g * L > 64 * 8000 * 8 * 32 // 2 and L > 1:
            L = L // 2
        return dict(op=op, B=B, L=L, lo=lo, hi=hi, kv=kv, g=g, D=D, page=page)
    if op == "rope":
        B = _log_int(rng, 1, 128)
        L = _log_int(rng, 1, max(1, 8191 // B))
        axes = rng.choice([1, 1, 1, 2, 3])
        lo = rng.choice([0, 1, L, L + 7])
        return dict(op=op, B=B, L=L, lo=lo, hi=lo + _log_int(rng, 1, 2000), hq=kv * rng.choice([1, 2, 4, 7]), kv=kv, D=D,
                    rot=2 * rng.randint(max(1, axes), D // 2), norm=rng.random() < 0.8, axes=axes,
                    pairs=rng.choice(["half", "adjacent"]), fmt=rng.choice(["none", "bf16", "mxfp8", "mxfp4"]), page=page)
    B, job = _log_int(rng, 1, 512), rng.choice(["branch", "compact"])
    hi = _log_int(rng, 64, 8000)
    lo = rng.choice([0, 1, hi // 9, hi // 2])
    need = B * (hi // page + 2)
    # contents of at most the largest listed case's
    layers = max(1, min(rng.randint(1, 5), (4000 * 64 * 8 * 128 * 2) // (2 * need * page * kv * D)))
    if 2 * need * page * kv * D * layers > 4000 * 64 * 8 * 128 * 2:
        kv, D = 1, 64
    return dict(op=op, job=job, B=B, lo=lo, hi=hi, page=page, pool=int(need * rng.uniform(2.0, 4.0)) + 8,
                L=rng.choice([1, 2, 8, 33]) if job == "branch" else 0, layers=layers, kv=kv, D=D,
                fmt=rng.choice(["bf16", "mxfp8"]))


def _lens(c):
    """Context lengths of the requests, spread evenly over the logarithm of their range (the same for every
    seed); where the range begins at 0 or 1, every seventh request is still empty."""
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


def _table(g, lens, page, n_pages, rows=None, spare=1):
    """A block table whose requests' pages lie anywhere in the pool (unused entries -1), and the pages in use."""
    per = [-(-n // page) for n in lens]
    need = sum(per)
    perm = torch.randperm(n_pages, generator=g, device=DEV)[:need].to(I32).cpu().numpy()
    table = np.full((rows or len(lens), max(max(per), 1) + spare), -1, np.int32)
    at = np.concatenate([[0], np.cumsum(per)])
    col = np.arange(need) - np.repeat(at[:-1], per)
    table[np.repeat(np.arange(len(lens)), per), col] = perm
    return table, perm, per, col


def _inputs(case, seed):
    """The operator's inputs, made from the seed alone."""
    return {"attend": _attend_inputs, "rope": _rope_inputs, "pages": _pages_inputs}[case["op"]](case, _gen(seed))


def _attend_inputs(c, g):
    B, L, kv, D, page = c["B"], c["L"], c["kv"], c["D"], c["page"]
    lens = _lens(c)
    n_pages = sum(-(-n // page) for n in lens) + 3
    table, used, per, col = _table(g, lens, page, n_pages)
    s = dict(table=torch.from_numpy(table).to(DEV), lens=torch.tensor(lens, dtype=I32, device=DEV), max_len=max(lens),
             q=_randn(g, B, L, kv * c["g"], D, std=1.5).to(BF), scale=D ** -0.5)
    shape = (n_pages, page, kv, D // 2)
    for name in ("k", "v"):  # codes as a quantiser leaves them: few zeros, one large value a block or more
        s[name] = torch.randint(0, 256, shape, generator=g, device=DEV, dtype=U8)
        s[name + "_s"] = (125 + torch.randint(-1, 2, shape[:3] + (D // 32,), generator=g, device=DEV)).to(U8)
    # what an earlier user of the pool left behind the requests' ends: no reader may let it through (scale 255: NaN)
    stale = torch.ones(n_pages, page, dtype=torch.bool, device=DEV)
    left = torch.from_numpy(np.repeat(lens, per) - col * page).to(DEV)  # rows of each page that are in use
    stale[torch.from_numpy(used.astype(np.int64)).to(DEV)] = torch.arange(page, device=DEV) >= left[:, None]
    for name in ("k_s", "v_s"):
        s[name].masked_fill_(stale[..., None, None], 255)
    return s


def _axis_of(c):
    """Position axis of every rotated pair: contiguous sections, the first axis the smallest."""
    n, a = c["rot"] // 2, c["axes"]
    first = max(1, n // (2 * a)) if a > 1 else n
    rest = [first] + [(n - first) // (a - 1)] * (a - 1) if a > 1 else [n]
    rest[-1] += n - sum(rest)
    return sum(([i] * k for i, k in enumerate(rest)), [])


def _rope_inputs(c, g):
    B, L, hq, kv, D = c["B"], c["L"], c["hq"], c["kv"], c["D"]
    # a fused projection's output: heads and columns of very different sizes
    col = torch.exp(0.5 * _randn(g, (hq + 2 * kv) * D))
    qkv = (_randn(g, B * L, (hq + 2 * kv) * D) * col).to(BF).view(B, L, hq + 2 * kv, D)
    s = dict(eps=1e-6, inv_freq=(10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=F64) / c["rot"])), axis=_axis_of(c))
    s["q"], s["k"], s["v"] = qkv.split((hq, kv, kv), dim=2)
    for w in ("qw", "kw"):
        s[w] = (1.0 + 0.2 * _randn(g, D)).to(BF) if c["norm"] else None
    s["pos"] = s["cache"] = None
    if c["fmt"] != "none":
        lens, page = _lens(c), c["page"]
        n_pages = sum(-(-n // page) for n in lens) + 3
        table = _table(g, lens, page, n_pages)[0]
        s["table"], s["lens"] = torch.from_numpy(table).to(DEV), torch.tensor(lens, dtype=I32, device=DEV)
        shape = (n_pages, page, kv, D // 2 if c["fmt"] == "mxfp4" else D)
        s["cache"] = {n: torch.zeros(shape, dtype=BF if c["fmt"] == "bf16" else U8, device=DEV) for n in ("k", "v")}
        if c["fmt"] != "bf16":
            s["cache"].update({n: torch.zeros(shape[:3] + (D // 32,), dtype=U8, device=DEV) for n in ("k_s", "v_s")})
    if c["axes"] > 1:  # frames of 24 x 40 patches after a text of a few tokens
        t = torch.arange(B * L, device=DEV)
        grid = torch.stack([t // 960, t // 40 % 24, t % 40])[:c["axes"]] + torch.randint(1, 200, (1,), generator=g, device=DEV)
        s["pos"] = grid.to(I32).contiguous()
    elif c["fmt"] == "none":
        s["pos"] = (torch.arange(B * L, device=DEV) + torch.randint(0, 4000, (1,), generator=g, device=DEV)).to(I32)[None].contiguous()
    return s


def _pages_inputs(c, g):
    B, page, n_pages = c["B"], c["page"], c["pool"]
    lens = _lens(c)
    rows = B + (B + 1) // 2 if c["job"] == "branch" else B  # room for the branches
    table, used, per, col = _table(g, lens, page, n_pages, rows, spare=2 + c["L"] // page)
    all_lens = np.array(lens + [0] * (rows - B), np.int32)
    refs = np.zeros(n_pages, np.int32)
    refs[used] = 1
    # table, lengths and reference counts lie in one buffer, so that a pass begins with one copy
    ints = torch.from_numpy(np.concatenate([table.reshape(-1), all_lens, refs])).to(DEV)
    s = dict(ints0=ints, ints=ints.clone(), shape=table.shape)
    if c["job"] == "branch":
        # every second request gets a branch; then all grow by L, but every fifth, whose last drafts were rejected, shrinks
        src = np.arange(0, B, 2, dtype=np.int32)
        dst = (B + np.arange(len(src))).astype(np.int32)
        s["src"], s["dst"] = torch.from_numpy(src).to(DEV), torch.from_numpy(dst).to(DEV)
        new = all_lens.copy()
        new[dst] = all_lens[src]
        shrink = np.arange(rows) % 5 == 4
        new = np.where(shrink, np.maximum(new - 5, 0), np.where(new > 0, new + c["L"], 0)).astype(np.int32)
        s["new"] = torch.from_numpy(new).to(DEV)
    shape = (n_pages, page, c["kv"], c["D"])
    s["layers"] = []
    for _ in range(c["layers"]):
        if c["fmt"] == "bf16":
            s["layers"].append({n: torch.randn(shape, generator=g, device=DEV, dtype=BF) for n in ("k", "v")})
        else:  # any codes but NaN
            lay = {n: torch.randint(0, 127, shape, generator=g, device=DEV, dtype=U8) for n in ("k", "v")}
            lay.update({n: torch.randint(100, 140, shape[:3] + (c["D"] // 32,), generator=g, device=DEV, dtype=U8) for n in ("k_s", "v_s")})
            s["layers"].append(lay)
    return s


def _split_ints(s):
    """Views of the block table, the lengths and the reference counts in the state's buffer."""
    rows, cols = s["shape"]
    i = s["ints"]
    return i[:rows * cols].view(rows, cols), i[rows * cols:rows * cols + rows], i[rows * cols + rows:]


def prepare(case, seed):
    c, s = case, _inputs(case, seed)
    s["case"] = c
    if own:
        import block_scaled_fp4_sqrt_gb300 as moe
        s["moe"] = moe
    if c["op"] == "attend":
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(s["q"].shape[:3], dtype=F32, device=DEV)
        if own:
            s["handle"] = moe.PagedKVCache(s["k"], s["v"], s["table"], s["lens"], s["k_s"], s["v_s"])
    if c["op"] == "rope":
        s["q_out"] = torch.empty(s["q"].shape, dtype=BF, device=DEV)
        s["k_out"] = torch.empty(s["k"].shape, dtype=BF, device=DEV) if c["fmt"] == "none" else None
        if c["fmt"] == "mxfp4":  # the rows that the pass writes, and the values of a byte's two codes
            s["rows"] = torch.from_numpy(_written(c, s)[2]).to(DEV)
            s["lut"] = torch.tensor([[E2M1[b & 15], E2M1[b >> 4]] for b in range(256)], device=DEV).to(E4).view(torch.int16).view(256)
        if own:
            s["plan"] = moe.RotaryPlan(s["inv_freq"], axis_of=s["axis"] if c["axes"] > 1 else None,
                                       pairs=c["pairs"], device=DEV)
            if s["cache"] is not None:
                s["handle"] = moe.PagedKVCache(s["cache"]["k"], s["cache"]["v"], s["table"], s["lens"],
                                               s["cache"].get("k_s"), s["cache"].get("v_s"))
        else:
            s["inv_freq"] = s["inv_freq"].to(DEV)
            s["axis"] = torch.tensor(s["axis"], device=DEV)
    if c["op"] == "pages":
        n = s["shape"][0] if c["job"] == "branch" else c["pool"] // 2
        s["copies"] = torch.empty(n, 2, dtype=I32, device=DEV)
        if own:
            table, lens, refs = _split_ints(s)
            s["pool"] = moe.PagePool(table, lens, refs, c["page"])
            s["caches"] = [moe.PagedKVCache(y["k"], y["v"], table, lens, y.get("k_s"), y.get("v_s")) for y in s["layers"]]
    return s


def _written(c, s):
    """(request, token) of every row that the pass writes into the cache, and its flat row in the pool."""
    lens, table = s["lens"].cpu().numpy().astype(np.int64), s["table"].cpu().numpy()
    b, l = np.divmod(np.arange(c["B"] * c["L"]), c["L"])
    pos = lens[b] - c["L"] + l
    b, l, pos = b[pos >= 0], l[pos >= 0], pos[pos >= 0]
    return b, l, table[b, pos // c["page"]].astype(np.int64) * c["page"] + pos % c["page"]


# ------------------------------------------------------------------------------------------------ one pass
def run(s):
    c = s["case"]
    if c["op"] == "attend":
        if own:
            s["handle"].attend(s["q"], s["out"], s["lse"], s["scale"])
            return dict(out=s["out"], lse=s["lse"])
        return _plain_attend(s)
    if c["op"] == "rope":
        if own:
            args = dict(q_weight=s["qw"], k_weight=s["kw"], eps=s["eps"], q_out=s["q_out"], k_out=s["k_out"])
            if s["cache"] is None:
                s["moe"].moe_head_norm_rope(s["q"], s["k"], s["plan"], s["pos"], **args)
            else:
                s["handle"].append_rotated(s["q"], s["k"], s["v"], s["plan"], s["pos"], **args)
        else:
            _plain_rope(s)
        out = dict(q=s["q_out"])
        if s["cache"] is None:
            out["k"] = s["k_out"]
        elif c["fmt"] == "bf16":
            out.update(s["cache"])
        elif c["fmt"] == "mxfp8":
            out.update({n: t.view(E8 if n.endswith("_s") else E4) for n, t in s["cache"].items()})
        else:
            for n, t in s["cache"].items():
                t = t.flatten(0, 1)[s["rows"]]
                out[n] = t.view(E8) if n.endswith("_s") else s["lut"][t.int()].view(E4)
        return out
    s["ints"].copy_(s["ints0"])
    if own:
        if c["job"] == "branch":
            s["pool"].fork(s["src"], s["dst"])
            s["pool"].resize(s["new"], s["copies"])
        else:
            s["pool"].compact(s["copies"])
        s["moe"].moe_copy_pages(s["caches"], s["copies"])
    else:
        _plain_pages(s)
    table, lens, refs = _split_ints(s)
    out = dict(table=table, lens=lens, refs=refs, copies=s["copies"])
    for i, y in enumerate(s["layers"]):
        out.update({f"{n}{i}": t if t.dtype == BF else t.view(E8 if n.endswith("_s") else E4) for n, t in y.items()})
    return out


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _pow2(e):
    """2^e in fp32 for integer e in [-126, 127], from its bits."""
    return ((e.to(I32) + 127) << 23).view(F32)


def _plain_attend(s):
    B, L, Hq, D = s["q"].shape
    page, kv = s["k"].shape[1:3]
    n, g = max(s["max_len"], 1), Hq // kv
    pos = torch.arange(n, device=DEV)
    lens = s["lens"].long()
    live = pos < lens[:, None]
    pages = s["table"].long()[:, pos // page]
    pages = torch.where(live, pages, torch.zeros_like(pages))
    lut = torch.tensor([[E2M1[b & 15], E2M1[b >> 4]] for b in range(256)], dtype=F32, device=DEV)

    def rows(codes, scales):
        r = lut[codes[pages, pos % page].int()].flatten(-2).unflatten(-1, (-1, 32))
        r = (r * _pow2(scales[pages, pos % page].int() - 127)[..., None]).flatten(-2)
        return r.masked_fill_(~live[..., None, None], 0.0).transpose(1, 2)  # [B, kv, n, D]

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


def _block(v, emax):
    """fp32 v along its last dimension in the units of its blocks of 32, and the blocks' exponents."""
    b = v.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1, keepdim=True)
    e = (torch.frexp(amax)[1] - 1 - emax).clamp(-127, 127)
    e = torch.where(amax > 0, e, torch.full_like(e, -127))
    return (b * _pow2(torch.clamp(-e, max=127))).flatten(-2), e.squeeze(-1)


def _e2m1_codes(u):
    """Codes of fp32 u, nearest with ties to the even code, saturating at 6."""
    a = u.abs()
    code = torch.zeros_like(u, dtype=U8)
    for i, (border, down) in enumerate(((0.25, True), (0.75, False), (1.25, True), (1.75, False), (2.5, True), (3.5, False), (5.0, True))):
        code += ((a > border) if down else (a >= border)).to(U8)  # a tie goes to the even of codes i and i + 1
    return code | (torch.signbit(u).to(U8) << 3)


def _plain_rope(s):
    c = s["case"]
    B, L, D, R = c["B"], c["L"], c["D"], c["rot"]
    if s["pos"] is not None:
        pos = s["pos"].double()
    else:
        pos = (s["lens"][:, None] - L + torch.arange(L, device=DEV)).reshape(1, B * L).double()
    a = pos[s["axis"]].t() * s["inv_freq"] if c["axes"] > 1 else pos[0][:, None] * s["inv_freq"]
    cos, sin = (f(a).float().view(B, L, 1, R // 2) for f in (torch.cos, torch.sin))

    def turned(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w.float()
        y = x.clone()
        if c["pairs"] == "half":
            x0, x1 = x[..., :R // 2], x[..., R // 2:R]
            y[..., :R // 2], y[..., R // 2:R] = x0 * cos - x1 * sin, x0 * sin + x1 * cos
        else:
            x0, x1 = x[..., 0:R:2], x[..., 1:R:2]
            y[..., 0:R:2], y[..., 1:R:2] = x0 * cos - x1 * sin, x0 * sin + x1 * cos
        return y

    s["q_out"].copy_(turned(s["q"], s["qw"]))
    k = turned(s["k"], s["kw"])
    if s["cache"] is None:
        s["k_out"].copy_(k)
        return
    page = c["page"]
    at = s["lens"].long()[:, None] - L + torch.arange(L, device=DEV)
    ok = at >= 0
    pages = s["table"].long().gather(1, at.clamp(min=0) // page)
    at = (pages[ok], at[ok] % page)
    for name, v in (("k", k[ok]), ("v", s["v"][ok])):
        dst = s["cache"]
        if c["fmt"] == "bf16":
            dst[name][at] = v.to(BF)
        elif c["fmt"] == "mxfp8":
            u, e = _block(v.float(), 8)
            dst[name][at] = u.clamp(-448.0, 448.0).to(E4).view(U8)
            dst[name + "_s"][at] = (e + 127).to(U8)
        else:
            u, e = _block(v.float(), 2)
            code = _e2m1_codes(u)
            dst[name][at] = code[..., 0::2] | (code[..., 1::2] << 4)
            dst[name + "_s"][at] = (e + 127).to(U8)


def _plain_pages(s):
    c, page = s["case"], s["case"]["page"]
    table, lens, refs = _split_ints(s)
    j = torch.arange(table.shape[1], device=DEV)
    if c["job"] == "branch":
        src, dst = s["src"].long(), s["dst"].long()
        n = -(-lens[src] // page)
        held = j < n[:, None]
        table[dst] = torch.where(held, table[src], table[dst])
        refs.scatter_add_(0, table[src][held].long(), torch.ones_like(table[src][held]))
        lens[dst] = lens[src]
        new, n0, n1 = s["new"], -(-lens // page), -(-s["new"] // page)
        drop = (j >= n1[:, None]) & (j < n0[:, None])
        refs.scatter_add_(0, table[drop].long(), torch.full_like(table[drop], -1))
        table[drop] = -1
        last = table.gather(1, (n0 - 1).clamp(min=0).long()[:, None])[:, 0]
        shared = refs[last.clamp(min=0).long()] > 1
        cow = (new > lens) & (lens % page != 0) & shared
        want = cow.to(torch.int64) + (n1 - n0).clamp(min=0)
        free = torch.nonzero(refs == 0)[:, 0]
        end = want.cumsum(0)
        served = (new <= lens) | (end <= free.numel())
        cow, want = cow & served, want * served
        fresh = (j >= (n0 - cow.to(I32))[:, None]) & (j < n1[:, None]) & ((new > lens) & served & (want > 0))[:, None]
        rank = (end - want)[:, None] + j - (n0 - cow.to(I32))[:, None]
        got = free[rank[fresh]].to(I32)
        table[fresh] = got
        refs[got.long()] = 1
        refs.scatter_add_(0, last[cow].long(), torch.full_like(last[cow], -1))
        now = table.gather(1, (n0 - 1).clamp(min=0).long()[:, None])[:, 0]
        none = torch.full_like(last, -1)
        s["copies"].copy_(torch.stack([torch.where(cow, last, none), torch.where(cow, now, none)], 1))
        lens.copy_(torch.where(served, new, lens))
    else:
        live = refs > 0
        n_live = live.sum()
        index = torch.arange(refs.numel(), device=DEV)
        movers = torch.nonzero(live & (index >= n_live))[:, 0].flip(0)
        holes = torch.nonzero(~live & (index < n_live))[:, 0]
        s["copies"].fill_(-1)
        s["copies"][:movers.numel(), 0] = movers.to(I32)
        s["copies"][:movers.numel(), 1] = holes.to(I32)
        to = index.clone()
        to[movers] = holes
        held = j < (-(-lens // page))[:, None]
        table[held] = to[table[held].long()].to(I32)
        refs[holes] = refs[movers]
        refs[movers] = 0
    pairs = s["copies"][s["copies"][:, 0] >= 0].long()
    for y in s["layers"]:
        for t in y.values():
            t[pairs[:, 1]] = t[pairs[:, 0]]


# ------------------------------------------------------------------------------------------------ work
def work(case):
    c = case
    if c["op"] == "attend":
        B, L, kv, D, lens = c["B"], c["L"], c["kv"], c["D"], _lens(c)
        pages = sum(-(-x // c["page"]) for x in lens)
        rows = B * L * kv * c["g"]
        seen = sum(max(x - L + 1 + i, 0) for x in lens for i in range(L))
        return dict(bytes=2 * sum(lens) * kv * D * (1 / 2 + 1 / 32) + 4 * pages + 4 * B + rows * (4 * D + 4),
                    flops=4 * seen * kv * c["g"] * D)
    if c["op"] == "rope":
        T, D = c["B"] * c["L"], c["D"]
        if c["fmt"] == "none":
            b = T * D * 4 * (c["hq"] + c["kv"]) + 4 * T * c["axes"]
        else:
            n = sum(min(c["L"], x) for x in _lens(c))
            el = {"bf16": 2, "mxfp8": 1 + 1 / 32, "mxfp4": 1 / 2 + 1 / 32}[c["fmt"]]
            b = T * D * 4 * c["hq"] + 2 * n * c["kv"] * D * (2 + el) + 8 * c["B"]
        return dict(bytes=b, flops=T * D * (c["hq"] + c["kv"]) * (8 if c["norm"] else 4))
    lens, page = _lens(c), c["page"]
    pages = sum(-(-x // page) for x in lens)
    el = {"bf16": 2, "mxfp8": 1 + 1 / 32}[c["fmt"]]
    one = 2 * page * c["kv"] * c["D"] * el * c["layers"]  # one page in all layers
    if c["job"] == "branch":
        shared = lens[::2]
        fork = sum(-(-x // page) for x in shared)
        grown = 2 * sum(1 for x in lens if x)
        moved = 2 * sum(1 for x in shared if x % page) * 0.8  # both holders grow, four fifths of them
        return dict(bytes=4 * (4 * fork + 4 * grown + c["pool"] + len(lens) * 3) + 2 * moved * one, flops=c["pool"])
    moved = pages * (1 - pages / c["pool"])  # of pages that lie anywhere
    return dict(bytes=4 * (2 * pages + 2 * c["pool"] + 2 * moved) + 2 * moved * one, flops=c["pool"])


# ------------------------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """What run() returns, from the definitions in 64 bits.  Values that are rounded to 16 or 8 bits at the end are
    given before that rounding; those in 4 bits, whose steps are a part of the definition, after it."""
    c, s = case, _inputs(case, seed)
    return {"attend": _exact_attend, "rope": _exact_rope, "pages": _exact_pages}[c["op"]](c, s)


def _fp4_64(codes, scales):
    mag = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=F64, device=DEV)
    nib = torch.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    val = mag[(nib & 7).long()] * torch.where(nib >= 8, -1.0, 1.0).double()
    return val * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


def _exact_attend(c, s):
    B, L, kv, g, D, page = c["B"], c["L"], c["kv"], c["g"], c["D"], c["page"]
    out = torch.zeros(B, L, kv * g, D, dtype=F64, device=DEV)
    lse = torch.full((B, L, kv * g), -math.inf, dtype=F64, device=DEV)
    lens, table = s["lens"].tolist(), s["table"].cpu()
    for b, n in enumerate(lens):
        if n == 0:
            continue
        pages = table[b, : -(-n // page)].long().to(DEV)
        K, V = (_fp4_64(s[x][pages].reshape(-1, kv, D // 2)[:n], s[x + "_s"][pages].reshape(-1, kv, D // 32)[:n]).transpose(0, 1)
                for x in "kv")  # [kv, n, D]
        q = s["q"][b].double().reshape(L, kv, g, D).permute(1, 0, 2, 3).reshape(kv, L * g, D)
        t = (q @ K.transpose(1, 2) / math.sqrt(D)).reshape(kv, L, g, n)
        end = n - L + 1 + torch.arange(L, device=DEV)
        t = t.masked_fill((torch.arange(n, device=DEV) >= end[:, None])[None, :, None], -math.inf)
        z = torch.logsumexp(t, -1)
        w = torch.exp(t - torch.where(z > -math.inf, z, torch.zeros_like(z))[..., None])
        lse[b] = z.permute(1, 0, 2).reshape(L, kv * g)
        out[b] = (w.reshape(kv, L * g, n) @ V).reshape(kv, L, g, D).permute(1, 0, 2, 3).reshape(L, kv * g, D)
    return dict(out=out, lse=lse)


def _exact_rope(c, s):
    B, L, D, R = c["B"], c["L"], c["D"], c["rot"]
    half = R // 2
    if s["pos"] is not None:
        pos = s["pos"].double().cpu()
    else:
        pos = (s["lens"].cpu()[:, None] - L + torch.arange(L)).reshape(1, -1).double()
    angle = torch.stack([pos[s["axis"][i]] * s["inv_freq"][i] for i in range(half)], 1).to(DEV).view(B, L, 1, half)
    unit = torch.polar(torch.ones_like(angle), angle)

    def turned(x, w):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / D + s["eps"]) * w.double()
        head, tail = x[..., :R], x[..., R:]
        if c["pairs"] == "half":
            z = torch.complex(head[..., :half].contiguous(), head[..., half:].contiguous()) * unit
            head = torch.cat([z.real, z.imag], -1)
        else:
            z = torch.view_as_complex(head.reshape(B, L, -1, half, 2).contiguous()) * unit
            head = torch.view_as_real(z).reshape(B, L, -1, R)
        return torch.cat([head, tail], -1)

    out = dict(q=turned(s["q"], s["qw"]))
    k = turned(s["k"], s["kw"])
    if s["cache"] is None:
        return dict(out, k=k)
    b, l, row = (torch.from_numpy(x).to(DEV) for x in _written(c, s))
    for name, x in (("k", k), ("v", s["v"].double())):
        x = x[b, l]
        full = torch.zeros(*s["cache"][name].shape[:3], D, dtype=F64, device=DEV).flatten(0, 1)
        if c["fmt"] == "bf16":
            full[row] = x
            out[name] = full.view(s["cache"][name].shape)
            continue
        emax, top = (8, 448.0) if c["fmt"] == "mxfp8" else (2, 6.0)
        blocks = x.reshape(*x.shape[:-1], D // 32, 32)
        m, e = torch.frexp(blocks.abs().amax(-1))
        e = torch.where(m > 0, (e - 1 - emax).clamp(-127, 127), torch.full_like(e, -127))
        u = (blocks * torch.exp2(-e.double())[..., None]).clamp(-top, top).reshape(x.shape)
        sc = torch.exp2(e.double())
        if c["fmt"] == "mxfp4":  # steps of 1/2 below 2, of 1 below 4 and of 2 above, half to even
            step = torch.where(u.abs() < 2, 0.5, torch.where(u.abs() < 4, 1.0, 2.0).double())
            u = torch.round(u / step) * step
            out[name], out[name + "_s"] = u.reshape(u.shape[0], -1, D), sc
        else:
            scales = torch.full(s["cache"][name + "_s"].shape, 2.0 ** -127, dtype=F64, device=DEV).flatten(0, 1)
            full[row], scales[row] = u, sc
            out[name] = full.view(s["cache"][name].shape)
            out[name + "_s"] = scales.view(s["cache"][name + "_s"].shape)
    return out


def _exact_pages(c, s):
    """The contents after the copies, from the rules one request and one page at a time."""
    page = c["page"]
    rows, cols = s["shape"]
    ints = s["ints0"].cpu().numpy()
    table = [list(r) for r in ints[:rows * cols].reshape(rows, cols)]
    lens = [int(x) for x in ints[rows * cols:rows * cols + rows]]
    refs = [int(x) for x in ints[rows * cols + rows:]]
    pages_of = lambda n: -(-n // page)  # noqa: E731
    moves = []
    if c["job"] == "branch":
        before = list(lens)
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            lens[b] = before[a]
            for i in range(pages_of(before[a])):
                table[b][i] = table[a][i]
                refs[table[a][i]] += 1
        new = s["new"].tolist()
        for b in range(rows):
            for i in range(pages_of(new[b]), pages_of(lens[b])):
                refs[table[b][i]] -= 1
        free = iter([p for p, r in enumerate(refs) if r == 0])
        for b in range(rows):
            n0, n1 = pages_of(lens[b]), pages_of(new[b])
            if new[b] > lens[b] and lens[b] % page and refs[table[b][n0 - 1]] > 1:
                moves.append((table[b][n0 - 1], next(free)))
            for _ in range(n0, n1):
                next(free)
    else:
        live, free = [p for p, r in enumerate(refs) if r], [p for p, r in enumerate(refs) if not r]
        moves = [(a, b) for a, b in zip(reversed(live), free) if a > b]
    out = dict(table=None, lens=None, refs=None, copies=None)
    a, b = (torch.tensor([m[i] for m in moves], dtype=torch.int64, device=DEV) for i in (0, 1))
    for i, y in enumerate(s["layers"]):
        for n, t in y.items():
            v = t.clone()
            v[b] = t[a]
            out[f"{n}{i}"] = (v.view(E8) if n.endswith("_s") else v if v.dtype == BF else v.view(E4)).double()
    return out
