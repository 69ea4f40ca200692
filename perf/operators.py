"""The serving operators beside the quantized cache: attention of a tree of
drafted tokens over the cache, the attention mass of its pages, and eviction by
that mass.  Each case is one call on the buffers that a serving loop holds: a
paged pool of packed blocks (the layout of include/kvq.h), a shuffled page
table, sequence lengths, and the layer's queries.

Plain form: the blocks are unpacked with elementary torch operations and the
attention is computed in 32 bits; `own` makes the library's calls instead."""
import math

import torch

own = False

PT = 16                                             # tokens of a page
INT4, E2M1, CB2, TIERED = 0, 1, 2, 3                # kvq_format
NAMES = {"int4": INT4, "e2m1": E2M1, "cb2": CB2, "tiered": TIERED}
E2M1_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    tree = dict(op="tree", tree=True, page_lse=False, ragged=False)
    return [
        # the smallest call: five drafted tokens of one short request, one kv head
        dict(tree, name="tree_int4_256", fmt="int4", B=1, Hkv=1, G=4, D=64, N=256, T=5),
        # a verify step of a small batch of ragged requests, 2-bit pages
        dict(tree, name="tree_cb2_4k", fmt="cb2", B=8, Hkv=8, G=4, D=128, N=4096, T=16, ragged=True),
        # a verify step of a full batch over long FP4 contexts: the largest call
        dict(tree, name="tree_fp4_32k", fmt="e2m1", B=16, Hkv=8, G=8, D=128, N=32768, T=16),
        # single-token decode that also reports each page's weight (what eviction accumulates)
        dict(tree, name="token_tiered_32k", fmt="tiered", B=16, Hkv=8, G=8, D=128, N=32768, T=1, tree=False, page_lse=True),
        # one very long request, a wide tree
        dict(tree, name="tree_cb2_128k", fmt="cb2", B=1, Hkv=8, G=4, D=128, N=131072, T=32),
        # the widest tree (more rows than one tile holds), odd length, with page weights
        dict(tree, name="tree_fp4_64nodes", fmt="e2m1", B=2, Hkv=8, G=8, D=128, N=8011, T=64, page_lse=True, ragged=True),
        # the page weights of one short request's decode step
        dict(name="mass_small", op="mass", B=1, Hq=4, T=1, P=16, decay=1.0),
        # a decode step of long requests; an exponentially forgetting score
        dict(name="mass_128k", op="mass", B=4, Hq=32, T=1, P=8192, decay=0.99),
        # the accepted nodes of a verify step of a full batch
        dict(name="mass_tree_32k", op="mass", B=16, Hq=64, T=8, P=2048, decay=1.0),
        # eviction: one short request, a full batch at half the budget, long requests with the short budget of a fixed-size cache
        dict(name="evict_small", op="evict", B=1, P=16, N=256, keep=8, sink=1, recent=2),
        dict(name="evict_32k", op="evict", B=64, P=2048, N=32768, keep=1024, sink=1, recent=4),
        dict(name="evict_128k", op="evict", B=4, P=8704, N=131067, keep=512, sink=4, recent=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "mass", "evict"])
    if op == "mass":
        return dict(op=op, B=_log(rng, 1, 16), Hq=rng.choice([4, 8, 24, 32, 64]), T=_log(rng, 1, 8), P=_log(rng, 5, 2048),
                    decay=rng.choice([1.0, 0.99, 0.9]))
    if op == "evict":
        P = _log(rng, 16, 8704)
        keep = rng.randint(8, P)
        return dict(op=op, B=_log(rng, 1, 64), P=P, N=rng.randint(1, P * PT), keep=keep, sink=rng.randint(0, 3), recent=rng.randint(0, 5))
    while True:
        G, T = rng.choice([1, 2, 3, 4, 7, 8, 16]), _log(rng, 1, 64)
        c = dict(op=op, fmt=rng.choice(["int4", "e2m1", "cb2", "tiered"]), B=_log(rng, 1, 16), Hkv=rng.choice([1, 2, 4, 8]), G=G,
                 D=rng.choice([64, 128, 128]), N=_log(rng, 1, 131072), T=T, tree=rng.random() < 0.8, page_lse=rng.random() < 0.4,
                 ragged=rng.random() < 0.5)
        if c["B"] * c["Hkv"] * c["N"] * c["D"] <= 1 << 28 and c["B"] * c["Hkv"] * c["N"] * G * T <= 1 << 28:
            return c


# ------------------------------------------------------------------ shapes
def _lens(c):
    """Tokens cached per sequence."""
    n = c["N"]
    return [max(1, n - (b * 7919) % (n // 2 + 1)) if c.get("ragged") else n for b in range(c["B"])]


def _stride(fmt, D):
    cap = 3 * (D // 32)
    size = {INT4: 10 * D + 16 + 48 * cap, E2M1: 9 * D, CB2: 12 * D + 4 + 20 * D, "fp8": 16 * D + 16}[fmt]
    return (size + 127) // 128 * 128


def work(case):
    c = case
    if c["op"] == "mass":
        n = c["B"] * c["T"] * c["Hq"]
        return {"bytes": 4 * (n * c["P"] + n + 2 * c["B"] * c["P"]) + 8 * c["B"], "flops": 2 * n * c["P"]}
    if c["op"] == "evict":
        return {"bytes": 4 * c["B"] * (4 * c["P"] + 3), "flops": c["B"] * c["P"]}
    D, rows = c["D"], c["B"] * c["T"] * c["Hkv"] * c["G"]
    # the codes, scales and codebooks of a block; outliers as the inputs have them (about 4 channels a page, 1% of the values)
    block = {"int4": 10 * D + 16 + 3 * D // 8, "e2m1": 9 * D, "cb2": 12 * D + 84, "tiered": 0.9 * (12 * D + 84) + 0.1 * (16 * D + 4)}[c["fmt"]]
    tokens = sum(_lens(c))
    cached = tokens / PT * c["Hkv"] * 2 * block
    P = -(-c["N"] // PT)
    nodes = c["T"] if c["tree"] else 0
    moved = cached + rows * D * 4 + rows * 4 + (rows * P * 4 if c["page_lse"] else 0) + 4 * c["B"] * nodes * c["Hkv"] * D + 4 * c["B"] * P
    return {"bytes": moved, "flops": 4.0 * c["G"] * c["Hkv"] * c["T"] * D * (tokens + c["B"] * nodes / 2)}


# ------------------------------------------------------------------ inputs
def _frag(x, role):
    """[..., 16, D] -> [..., 32 lanes, D/16 steps, 2, 4]: the slots 4 a + b of a lane's step."""
    *n, _, D = x.shape
    k = len(n)
    lead = list(range(k))
    if role == 0:   # (t_hi, t_lo, s, j_hi, jq, j_lo) -> (t_lo, jq, s, j_hi, t_hi, j_lo)
        x = x.reshape(*n, 2, 8, D // 16, 2, 4, 2).permute(*lead, k + 1, k + 4, k + 2, k + 3, k, k + 5)
    else:           # (t_hi, tq, t_b, s, j_hi, j8) -> (j8, tq, s, t_hi, j_hi, t_b)
        x = x.reshape(*n, 2, 4, 2, D // 16, 2, 8).permute(*lead, k + 5, k + 1, k + 3, k, k + 4, k + 2)
    return x.reshape(*n, 32, D // 16, 2, 4)


def _unfrag(x, role):
    """The inverse of _frag: [..., 32, D/16, 2, 4] -> [..., 16, D]."""
    *n, _, S, _, _ = x.shape
    k = len(n)
    lead = list(range(k))
    if role == 0:
        x = x.reshape(*n, 8, 4, S, 2, 2, 2).permute(*lead, k + 4, k, k + 2, k + 3, k + 1, k + 5)
    else:
        x = x.reshape(*n, 8, 4, S, 2, 2, 2).permute(*lead, k + 3, k + 1, k + 5, k + 2, k + 4, k)
    return x.reshape(*n, PT, 16 * S)


def _nibbles(code, role):
    f = _frag(code, role).reshape(*code.shape[:-2], -1, 2)
    return f[..., 0] | (f[..., 1] << 4)


def _slots(D, role, device):
    """Channel c's place in the codebook."""
    c = torch.arange(D, device=device)
    return c if role == 0 else 16 * (c // 16) + 2 * (c % 8) + (c % 16) // 8


def _bytes(x):
    return x.contiguous().view(torch.uint8)


def _e4m3(x):
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def _pack_e2m1(x, blk, role):
    D = x.shape[-1]
    xs = x.view(*x.shape[:-1], D // 16, 16)
    sc = _e4m3(xs.abs().amax(-1) / 6)
    y = xs / sc.float().unsqueeze(-1).clamp_min(1e-12)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    code = (torch.bucketize(y.abs(), edges).to(torch.uint8) | ((y < 0).to(torch.uint8) << 3)).view(x.shape)
    blk[..., :8 * D] = _nibbles(code, role)
    blk[..., 8 * D:9 * D] = _bytes(sc.transpose(-1, -2)).flatten(-2)


def _pack_int4(x, blk, role):
    D = x.shape[-1]
    xs = x.view(*x.shape[:-1], D // 32, 32)
    out = (xs - xs.mean(-1, keepdim=True)).abs() > 3 * xs.std(-1, keepdim=True)
    lo = xs.masked_fill(out, math.inf).amin(-1)
    hi = xs.masked_fill(out, -math.inf).amax(-1)
    S, m = ((hi - lo) / 15).half(), lo.half()
    q = ((xs - m.float().unsqueeze(-1)) / S.float().unsqueeze(-1).clamp_min(1e-12)).round().clamp(0, 15)
    blk[..., :8 * D] = _nibbles(q.masked_fill(out, 0).to(torch.uint8).view(x.shape), role)
    blk[..., 8 * D:10 * D] = _bytes(torch.stack([S, m], -1)).flatten(-2).flatten(-2)
    out, cap = out.view(x.shape), 3 * (D // 32)
    n = out.sum(-1)
    ch = torch.argsort(out.to(torch.uint8), dim=-1, descending=True, stable=True)[..., :cap]
    live = torch.arange(cap, device=x.device) < n.unsqueeze(-1)
    blk[..., 10 * D:10 * D + 16] = n.to(torch.uint8)
    blk[..., 10 * D + 16:10 * D + 16 + 16 * cap] = (ch * live).to(torch.uint8).flatten(-2)
    val = x.gather(-1, ch).half() * live
    blk[..., 10 * D + 16 + 16 * cap:10 * D + 16 + 48 * cap] = _bytes(val).flatten(-2)


def _pack_cb2(x, blk, role):
    D, R = x.shape[-1], 8
    out = (x - x.mean(-1, keepdim=True)).abs() > 3 * x.std(-1, keepdim=True)
    # centroids: the means of the quarters of a channel's 16 values, outliers drawn in to the largest that is none
    y = torch.where(out, torch.zeros_like(x), x).transpose(-1, -2)
    cent = y.sort(-1).values.view(*y.shape[:-1], 4, 4).mean(-1).half()
    code = (y.unsqueeze(-1) - cent.float().unsqueeze(-2)).abs().argmin(-1).transpose(-1, -2).masked_fill(out, 0)
    f = _frag(code.to(torch.uint8), role)
    nib = f[..., 0, :] | (f[..., 1, :] << 2)
    blk[..., :4 * D] = (nib[..., 0::2] | (nib[..., 1::2] << 4)).flatten(-3)
    raw = _bytes(cent).view(*cent.shape[:-1], 4, 2).transpose(-1, -2).flatten(-2)   # 4 low bytes, 4 high bytes
    place = torch.empty_like(raw)
    place[..., _slots(D, role, x.device), :] = raw
    blk[..., 4 * D:12 * D] = place.flatten(-2)
    has = out.any(-2)
    n = has.sum(-1).clamp_max(R)
    ch = torch.argsort(has.to(torch.uint8), dim=-1, descending=True, stable=True)[..., :R].sort(-1).values
    ch = torch.where(has.gather(-1, ch), ch, D).sort(-1).values          # the channels that have outliers, ascending
    live = ch < D
    chc = ch.clamp_max(D - 1)
    o = out.transpose(-1, -2).gather(-2, chc.unsqueeze(-1).expand(*chc.shape, PT)) & live.unsqueeze(-1)
    v = _bytes(_e4m3(x.transpose(-1, -2).gather(-2, chc.unsqueeze(-1).expand(*chc.shape, PT))))
    bits = (o.to(torch.int32) << torch.arange(PT, device=x.device, dtype=torch.int32)).sum(-1)
    rec = torch.zeros(*chc.shape, 20, dtype=torch.uint8, device=x.device)
    rec[..., 0] = (chc * live).to(torch.uint8)
    rec[..., 2] = (bits & 255).to(torch.uint8)
    rec[..., 3] = (bits >> 8).to(torch.uint8)
    rec[..., 4:] = v * o
    blk[..., 12 * D] = n.to(torch.uint8)
    blk[..., 12 * D + 1] = o.sum((-1, -2)).to(torch.uint8)
    blk[..., 12 * D + 4:12 * D + 4 + 20 * R] = rec.flatten(-2)


def _pack_fp8(x, blk, role):
    D = x.shape[-1]
    s = x.abs().amax((-1, -2)) / 448
    blk[..., :16 * D] = _bytes(_frag(_e4m3(x / s[..., None, None]).view(torch.uint8), role)).flatten(-4)
    blk[..., 16 * D:16 * D + 4] = _bytes(s.unsqueeze(-1))


def _values(gen, shape, fmt, loud, device):
    """K or V of some tokens: heavy tails for the format without outliers, else four loud channels a head."""
    x = torch.randn(shape, generator=gen, device=device)
    if fmt == E2M1:   # Student's t with four degrees of freedom, unit variance
        u = [torch.rand(shape, generator=gen, device=device).clamp_min(1e-7).log() for _ in range(2)]
        return x / (-(u[0] + u[1]) / 2).sqrt().clamp_min(1e-2) / math.sqrt(2.0)
    return x * loud


def _ancestors(T, g):
    """Bit j of word i: node i attends to node j (its ancestors and itself); parents come before children."""
    words = []
    for i in range(T):
        p = int(torch.randint(-1, i, (1,), generator=g)) if i else -1
        words.append((1 << i) | (words[p] if p >= 0 else 0))
    return [w - (1 << 64) if w >> 63 else w for w in words]


def _small_cache(B, P, dev):
    """The buffers of a cache of one small FP4 head, for the calls that read no block."""
    return dict(fmt=E2M1, pool=torch.zeros(B * P * 2 * _stride(E2M1, 64), dtype=torch.uint8, device=dev), tiers=None, staging=None,
                table=torch.arange(B * P, dtype=torch.int32, device=dev).view(B, P), lens=torch.full((B,), P * PT, dtype=torch.int32, device=dev),
                status=torch.zeros(1, dtype=torch.int32, device=dev))


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    B = c["B"]
    if c["op"] == "mass":
        # page weights of softmax rows whose logits have unit variance, early and late pages above the rest
        T, Hq, P = c["T"], c["Hq"], c["P"]
        x = torch.randn((B, T, Hq, P), generator=gen, device=dev) + 2.8
        x[..., 0] += 4.0
        x[..., -1] += 2.0
        lse = torch.logsumexp(x, -1) + 0.1
        accepted = [0] * B
        for b in range(B):
            accepted[b] = 1 | int(torch.randint(0, 1 << min(T, 30), (1,), generator=cpu))
        return dict(case=c, page_lse=x, lse=lse, nodes=torch.tensor(accepted, device=dev),
                    mass=torch.rand((B, P), generator=gen, device=dev) * Hq, **_small_cache(B, P, dev))
    if c["op"] == "evict":
        P = c["P"]
        # accumulated weights: heavy-tailed over the pages, some of them never attended to (ties at zero)
        mass = torch.rand((B, P), generator=gen, device=dev).clamp_min(1e-6).pow(-0.9)
        mass = torch.where(torch.rand((B, P), generator=gen, device=dev) < 0.1, torch.zeros_like(mass), mass)
        lens = [max(0, c["N"] - (b * 7919) % (c["N"] // 3 + 1)) for b in range(B)]
        held = _small_cache(B, P, dev)
        held["table"] = torch.randperm(B * P, generator=gen, device=dev).view(B, P).to(torch.int32)
        held["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        return dict(case=c, mass=mass, **held)
    fmt, Hkv, G, D, T = NAMES[c["fmt"]], c["Hkv"], c["G"], c["D"], c["T"]
    lens = _lens(c)
    P = -(-max(lens) // PT)
    main = CB2 if fmt == TIERED else fmt
    order = torch.randperm(B * P, generator=gen, device=dev)
    tier = torch.rand(B * P, generator=gen, device=dev) < 0.1 if fmt == TIERED else torch.zeros(B * P, dtype=torch.bool, device=dev)
    entry = torch.where(tier, tier.cumsum(0) - 1, (~tier).cumsum(0) - 1)          # page i of the draw: its block in its pool
    n_tier = max(int(tier.sum()), 1) if fmt == TIERED else 0
    n_main = max(int((~tier).sum()), 1)
    pool = torch.zeros((n_main, Hkv, 2, _stride(main, D)), dtype=torch.uint8, device=dev)
    tiers = torch.zeros((n_tier, Hkv, 2, _stride("fp8", D)), dtype=torch.uint8, device=dev) if n_tier else None
    loud = torch.ones((2, Hkv, 1, D), device=dev)
    at = torch.rand((2, Hkv, 1, D), generator=gen, device=dev).argsort(-1)[..., :4]
    loud.scatter_(-1, at, 8.0)
    step = max(1, (1 << 26) // (Hkv * PT * D))
    for p in range(0, B * P, step):
        n = min(step, B * P - p)
        t, e = tier[p:p + n], entry[p:p + n]
        for role in (0, 1):
            x = _values(gen, (n, Hkv, PT, D), fmt, loud[role], dev)
            blk = torch.zeros((n, Hkv, _stride(main, D)), dtype=torch.uint8, device=dev)
            (_pack_e2m1 if main == E2M1 else _pack_int4 if main == INT4 else _pack_cb2)(x, blk, role)
            pool[e[~t], :, role] = blk[~t]
            if n_tier:
                blk = torch.zeros((n, Hkv, _stride("fp8", D)), dtype=torch.uint8, device=dev)
                _pack_fp8(x, blk, role)
                tiers[e[t], :, role] = blk[t]
    word = entry.to(torch.int64) - (tier.to(torch.int64) << 31)                   # bit 31 set: the tier pool
    s = dict(case=c, fmt=fmt, pool=pool.view(-1), tiers=None if tiers is None else tiers.view(-1), n_main=n_main, n_tier=n_tier,
             table=word[order].view(B, P).to(torch.int32), lens=torch.tensor(lens, dtype=torch.int32, device=dev), staging=None,
             status=torch.zeros(1, dtype=torch.int32, device=dev), longest=max(lens), scale=D ** -0.5)
    if main == CB2:
        s["staging"] = _values(gen, (B, Hkv, 2, PT, D), fmt, loud.transpose(0, 1), dev).contiguous()
    s["q"] = torch.randn((B, T, Hkv * G, D), generator=gen, device=dev).to(torch.bfloat16)
    s["k"] = s["v"] = s["mask"] = s["nodes"] = None
    if c["tree"]:
        s["k"], s["v"] = [torch.randn((B, T, Hkv, D), generator=gen, device=dev).to(torch.bfloat16) for _ in range(2)]
        s["mask"] = torch.tensor([_ancestors(T, cpu) for _ in range(B)], device=dev)
        if c["ragged"]:   # sequences draft trees of their own sizes
            s["nodes"] = torch.tensor([max(1, T - b % T) for b in range(B)], dtype=torch.int32, device=dev)
    return s


# ------------------------------------------------------------------ plain form
def _by_page(s, pool, stride, index):
    c = s["case"]
    return pool.view(-1, c["Hkv"], 2, stride)[index]                              # [B, P, Hkv, 2, stride]


def _unpack_nibbles(raw, D, role):
    n = torch.stack([raw & 15, raw >> 4], -1)
    return _unfrag(n.view(*raw.shape[:-1], 32, D // 16, 2, 4), role)


def _unpack_e2m1(blk, D, role):
    code = _unpack_nibbles(blk[..., :8 * D], D, role).to(torch.int32)
    value = torch.tensor(E2M1_VALUES + tuple(-v for v in E2M1_VALUES), device=blk.device)[code]
    sc = blk[..., 8 * D:9 * D].contiguous().view(torch.float8_e4m3fn).float().view(*blk.shape[:-1], D // 16, PT)
    return value * sc.transpose(-1, -2).repeat_interleave(16, -1)


def _unpack_int4(blk, D, role):
    cap = 3 * (D // 32)
    q = _unpack_nibbles(blk[..., :8 * D], D, role).float()
    sz = blk[..., 8 * D:10 * D].contiguous().view(torch.float16).float().view(*blk.shape[:-1], PT, D // 32, 2)
    x = (q.view(*sz.shape[:-1], 32) * sz[..., 0:1] + sz[..., 1:2]).flatten(-2)
    n = blk[..., 10 * D:10 * D + 16]
    ch = blk[..., 10 * D + 16:10 * D + 16 + 16 * cap].reshape(*blk.shape[:-1], PT, cap).long()
    val = blk[..., 10 * D + 16 + 16 * cap:10 * D + 16 + 48 * cap].contiguous().view(torch.float16).float().view(ch.shape)
    live = torch.arange(cap, device=blk.device) < n.unsqueeze(-1)
    wide = torch.cat([x, torch.zeros_like(x[..., :1])], -1)                       # one more channel takes the empty places
    return wide.scatter(-1, torch.where(live, ch, D), val)[..., :D]


def _unpack_cb2(blk, D, role):
    w = blk[..., :4 * D].reshape(*blk.shape[:-1], 32, D // 16, 2)
    nib = torch.stack([w & 15, w >> 4], -1).flatten(-2)                           # slots b of a = 0 (low bits) and a = 1
    code = _unfrag(torch.stack([nib & 3, nib >> 2], -2), role).long()
    cb = blk[..., 4 * D:12 * D].reshape(*blk.shape[:-1], D, 2, 4).transpose(-1, -2).contiguous().view(torch.float16).squeeze(-1)
    cb = cb[..., _slots(D, role, blk.device), :].float()                          # [..., channel, centroid]
    x = cb.gather(-1, code.transpose(-1, -2))                                     # [..., channel, token]
    R = 8                                                                         # records the inputs can have
    rec = blk[..., 12 * D + 4:12 * D + 4 + 20 * R].reshape(*blk.shape[:-1], R, 20)
    live = torch.arange(R, device=blk.device) < blk[..., 12 * D].unsqueeze(-1)
    ch = torch.where(live, rec[..., 0].long(), D)
    bits = rec[..., 2].to(torch.int32) | (rec[..., 3].to(torch.int32) << 8)
    flag = ((bits.unsqueeze(-1) >> torch.arange(PT, device=blk.device, dtype=torch.int32)) & 1).bool()
    val = rec[..., 4:].contiguous().view(torch.float8_e4m3fn).float()
    wide = torch.cat([x, torch.zeros_like(x[..., :1, :])], -2)
    at = ch.unsqueeze(-1).expand(val.shape)
    wide = wide.scatter(-2, at, torch.where(flag, val, wide.gather(-2, at)))
    return wide[..., :D, :].transpose(-1, -2)


def _unpack_fp8(blk, D, role):
    v = blk[..., :16 * D].reshape(*blk.shape[:-1], 32, D // 16, 2, 4).contiguous().view(torch.float8_e4m3fn).float()
    return _unfrag(v, role) * blk[..., 16 * D:16 * D + 4].contiguous().view(torch.float32).unsqueeze(-1)


def _cached(s, role):
    """The values the cache stands for: 32 bits [B, Hkv, P * 16, D]."""
    c, fmt, D = s["case"], s["fmt"], s["case"]["D"]
    word = s["table"].to(torch.int64)
    main = CB2 if fmt == TIERED else fmt
    unpack = {INT4: _unpack_int4, E2M1: _unpack_e2m1, CB2: _unpack_cb2}[main]
    tier = word < 0
    x = unpack(_by_page(s, s["pool"], _stride(main, D), word.masked_fill(tier, 0))[..., role, :], D, role)
    if fmt == TIERED:
        blk = _by_page(s, s["tiers"], _stride("fp8", D), (word & 0x7FFFFFFF).masked_fill(~tier, 0))[..., role, :]
        x = torch.where(tier[:, :, None, None, None], _unpack_fp8(blk, D, role), x)
    x = x.permute(0, 2, 1, 3, 4).reshape(c["B"], c["Hkv"], -1, D)
    if s["staging"] is not None:                                                  # the partial last page waits in 32 bits
        t = torch.arange(x.shape[2], device=x.device)
        tail = t[None, :] >= (s["lens"] // PT * PT)[:, None]
        x = torch.where(tail[:, None, :, None], s["staging"][:, :, role].repeat(1, 1, x.shape[2] // PT, 1), x)
    return x


def _tree_plain(s):
    c = s["case"]
    B, Hkv, G, D, T = c["B"], c["Hkv"], c["G"], c["D"], c["T"]
    k, v = _cached(s, 0), _cached(s, 1)
    n = k.shape[2]
    pos = torch.arange(n, device=k.device)
    seen = (pos[None, :] < s["lens"][:, None])[:, None, :].expand(B, T, n)
    if c["tree"]:
        k = torch.cat([k, s["k"].float().permute(0, 2, 1, 3)], 2)
        v = torch.cat([v, s["v"].float().permute(0, 2, 1, 3)], 2)
        node = torch.arange(T, device=k.device)
        sees = ((s["mask"].unsqueeze(-1) >> node) & 1).bool()
        if s["nodes"] is not None:
            live = node[None, :] < s["nodes"][:, None]
            sees = sees & live[:, None, :]
            seen = seen & live[:, :, None]
            sees = sees & live[:, :, None]
        seen = torch.cat([seen, sees], 2)
    q = s["q"].float().view(B, T, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, D)
    a = torch.matmul(q, k.transpose(-1, -2)) * s["scale"]
    a = a.view(B, Hkv, T, G, -1).masked_fill(~seen[:, None, :, None, :], -math.inf)
    top = a.amax(-1, keepdim=True)
    p = torch.exp(a - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, T * G, -1), v).view(B, Hkv, T, G, D) / torch.where(total == 0, torch.ones_like(total), total)
    out = o.permute(0, 2, 1, 3, 4).reshape(B, T, Hkv * G, D).to(torch.bfloat16)
    lse = (top + total.log()).squeeze(-1).permute(0, 2, 1, 3).reshape(B, T, Hkv * G)
    if not c["page_lse"]:
        return {"out": out, "lse": lse}
    a = a[..., :n].reshape(B, Hkv, T, G, n // PT, PT)
    top = a.amax(-1, keepdim=True)
    page = top.squeeze(-1) + torch.exp(a - torch.where(top == -math.inf, torch.zeros_like(top), top)).sum(-1).log()
    return {"out": out, "lse": lse, "page_lse": page.permute(0, 2, 1, 3, 4).reshape(B, T, Hkv * G, n // PT).contiguous()}


def _mass_plain(s):
    c = s["case"]
    on = ((s["nodes"][:, None] >> torch.arange(c["T"], device=s["nodes"].device)) & 1).bool()
    w = torch.exp(s["page_lse"] - s["lse"].unsqueeze(-1)) * on[:, :, None, None]
    return {"mass": c["decay"] * s["mass"] + w.sum((1, 2))}


def _evict_plain(s):
    c, P = s["case"], s["case"]["P"]
    i = torch.arange(P, device=s["mass"].device)[None, :]
    full, used = (s["lens"] // PT)[:, None], ((s["lens"] + PT - 1) // PT)[:, None]
    fixed = (i < c["sink"]) | (i >= full - c["recent"])
    key = torch.where(fixed, torch.full_like(s["mass"], math.inf), s["mass"])
    key = torch.where(i < full, key, torch.full_like(key, -math.inf))
    rank = torch.empty_like(key, dtype=torch.int64)
    rank.scatter_(1, torch.argsort(key, dim=1, descending=True, stable=True), i.expand(key.shape))
    gone = (i < full) & (rank >= c["keep"])
    order = torch.argsort(gone.to(torch.uint8), dim=1, stable=True)               # kept, partial and unused pages, then the evicted
    n = gone.sum(1)
    mass = s["mass"].gather(1, order)
    return {"page_table": s["table"].gather(1, order), "seq_lens": (s["lens"] - PT * n).to(torch.int32), "evicted": n.to(torch.int32),
            "mass": torch.where(i < used - n[:, None], mass, torch.zeros_like(mass))}


# ------------------------------------------------------------------ the library's calls
def _handle(s, kvq):
    """The serving loop's handle on its buffers."""
    if "cache" not in s:
        c = s["case"]
        s["cache"] = kvq.QuantizedKVCache.from_buffers(s["fmt"], c.get("Hkv", 1), c.get("D", 64), s["pool"], s["table"], s["lens"], s["status"],
                                                       staging=s["staging"], tier_pool=s["tiers"])
    return s["cache"]


def _tree_own(s):
    from sub_byte_quantized_kvq_gb300 import kvq
    c, q, cache = s["case"], s["q"], _handle(s, kvq)
    B, T, Hq, _ = q.shape
    if "workspace" not in s:
        s["workspace"] = kvq.alloc_tree_workspace(cache, Hq, T, s["longest"])
    got = {"out": torch.empty_like(q), "lse": torch.empty((B, T, Hq), dtype=torch.float32, device=q.device)}
    if c["page_lse"]:
        got["page_lse"] = torch.empty((B, T, Hq, s["table"].shape[1]), dtype=torch.float32, device=q.device)
    kvq.kvq_tree_attention(cache, q, s["scale"], s["longest"], k_tree=s["k"], v_tree=s["v"], tree_mask=s["mask"],
                           nodes_per_seq=s["nodes"], out=got["out"], lse=got["lse"], page_lse=got.get("page_lse"),
                           workspace=s["workspace"])
    return got


def _mass_own(s):
    from sub_byte_quantized_kvq_gb300 import kvq
    out = torch.empty_like(s["mass"])
    kvq.kvq_page_mass(_handle(s, kvq), s["lse"], s["page_lse"], s["mass"], node_mask=s["nodes"], decay=s["case"]["decay"], mass_out=out)
    return {"mass": out}


def _evict_own(s):
    from sub_byte_quantized_kvq_gb300 import kvq
    c = s["case"]
    got = {"page_table": torch.empty_like(s["table"]), "seq_lens": torch.empty_like(s["lens"]), "evicted": torch.empty_like(s["lens"]),
           "mass": torch.empty_like(s["mass"])}
    kvq.kvq_evict_pages(_handle(s, kvq), s["mass"], c["keep"], sink_pages=c["sink"], recent_pages=c["recent"],
                        page_table_out=got["page_table"], seq_lens_out=got["seq_lens"], mass_out=got["mass"], evicted=got["evicted"])
    return got


def run(state):
    op = state["case"]["op"]
    if own:
        return _tree_own(state) if op == "tree" else _mass_own(state) if op == "mass" else _evict_own(state)
    return _tree_plain(state) if op == "tree" else _mass_plain(state) if op == "mass" else _evict_plain(state)


# ------------------------------------------------------------------ 64 bits
def _minifloat(byte, exp_bits, man_bits, bias):
    """A sign, exponent, mantissa byte (no infinities) as a 64-bit number."""
    b = byte.to(torch.int64)
    man, ex = b & ((1 << man_bits) - 1), (b >> man_bits) & ((1 << exp_bits) - 1)
    frac = torch.where(ex == 0, man.double(), man.double() + (1 << man_bits))
    return torch.where((b >> (exp_bits + man_bits)) & 1 == 1, -1.0, 1.0) * frac * torch.pow(2.0, (ex.clamp_min(1) - bias - man_bits).double())


def _half(lo, hi):
    """IEEE half precision from its two bytes."""
    return _minifloat(lo.to(torch.int64) | (hi.to(torch.int64) << 8), 5, 10, 15)


def _element(role, t, ch, per, blk):
    """Where element (t, ch) lies: the index of its code among the block's lanes x steps x 8 slots."""
    j = ch % 16
    lane = 4 * (t % 8) + (j % 8) // 2 if role == 0 else 4 * (j % 8) + (t % 8) // 2
    slot = 2 * (t // 8 + 2 * (j // 8)) + j % 2 if role == 0 else 2 * (j // 8 + 2 * (t // 8)) + t % 2
    return lane, ch // 16, slot


def _exact_values(blk, kind, role, D):
    """[n, stride] bytes -> [n, 16, D] in 64 bits, element by element from the layout."""
    dev = blk.device
    t = torch.arange(PT, device=dev)[:, None].expand(PT, D)
    ch = torch.arange(D, device=dev)[None, :].expand(PT, D)
    lane, step, slot = _element(role, t, ch, D // 16, blk)
    cell = lane * (D // 16) + step
    if kind == "fp8":
        bits = blk[:, 16 * D:16 * D + 4].contiguous().view(torch.float32).double()
        return _minifloat(blk[:, cell * 8 + slot], 4, 3, 7) * bits[:, :, None]
    if kind in (E2M1, INT4):
        code = (blk[:, cell * 4 + slot // 2].to(torch.int64) >> (4 * (slot % 2))) & 15
        if kind == E2M1:
            return _minifloat(code, 2, 1, 1) * _minifloat(blk[:, 8 * D + 16 * (ch // 16) + t], 4, 3, 7)
        at = 8 * D + 4 * (t * (D // 32) + ch // 32)
        x = code.double() * _half(blk[:, at], blk[:, at + 1]) + _half(blk[:, at + 2], blk[:, at + 3])
        cap = 3 * (D // 32)
        for i in range(cap):
            row = torch.arange(PT, device=dev)
            c_i = blk[:, 10 * D + 16 + row * cap + i].to(torch.int64)
            a = 10 * D + 16 + 16 * cap + 2 * (row * cap + i)
            hit = (ch[None] == c_i[:, :, None]) & (blk[:, 10 * D:10 * D + 16].to(torch.int64) > i)[:, :, None]
            x = torch.where(hit, _half(blk[:, a], blk[:, a + 1])[:, :, None], x)
        return x
    code = (blk[:, cell * 2 + (slot % 4) // 2].to(torch.int64) >> (4 * (slot % 2) + 2 * (slot // 4))) & 3
    place = ch if role == 0 else 16 * (ch // 16) + 2 * (ch % 8) + (ch % 16) // 8
    at = (4 * D + 8 * place)[None] + code
    x = _half(blk.gather(1, at.flatten(1)).view(at.shape), blk.gather(1, (at + 4).flatten(1)).view(at.shape))
    for i in range(8):
        r = 12 * D + 4 + 20 * i
        row = torch.arange(PT, device=dev)
        flags = (blk[:, r + 2].to(torch.int64) | (blk[:, r + 3].to(torch.int64) << 8))[:, None] >> row & 1
        hit = (blk[:, 12 * D] > i)[:, None, None] & (ch[None] == blk[:, r].to(torch.int64)[:, None, None]) & (flags == 1)[:, :, None]
        x = torch.where(hit, _minifloat(blk[:, r + 4:r + 20], 4, 3, 7)[:, :, None], x)
    return x


def _exact_tree(s):
    c, dev = s["case"], s["q"].device
    B, Hkv, G, D, T = c["B"], c["Hkv"], c["G"], c["D"], c["T"]
    main = CB2 if s["fmt"] == TIERED else s["fmt"]
    pool = s["pool"].view(-1, Hkv, 2, _stride(main, D))
    tiers = s["tiers"].view(-1, Hkv, 2, _stride("fp8", D)) if s["tiers"] is not None else None
    P = s["table"].shape[1]
    out = torch.zeros((B, T, Hkv * G, D), dtype=torch.float64, device=dev)
    lse = torch.full((B, T, Hkv * G), -math.inf, dtype=torch.float64, device=dev)
    page = torch.full((B, T, Hkv * G, P), -math.inf, dtype=torch.float64, device=dev)
    for b in range(B):
        L = int(s["lens"][b])
        n = T if s["nodes"] is None else int(s["nodes"][b])
        pages = -(-L // PT)
        word = s["table"][b, :pages].to(torch.int64)
        for h in range(Hkv):
            kv = []
            for role in (0, 1):
                x = torch.zeros((pages, PT, D), dtype=torch.float64, device=dev)
                main_at = torch.nonzero(word >= 0).flatten()
                x[main_at] = _exact_values(pool[word[main_at], h, role], main, role, D)
                if tiers is not None:
                    at = torch.nonzero(word < 0).flatten()
                    x[at] = _exact_values(tiers[word[at] & 0x7FFFFFFF, h, role], "fp8", role, D)
                if s["staging"] is not None and L % PT:
                    x[-1] = s["staging"][b, h, role].double()
                x = x.view(-1, D)[:L]
                kv.append(torch.cat([x, s["k" if role == 0 else "v"][b, :n, h].double()]) if c["tree"] else x)
            rows = s["q"][b, :n, h * G:(h + 1) * G].double().reshape(n * G, D)
            a = rows @ kv[0].T * s["scale"]
            if c["tree"]:
                for i in range(n):
                    w = int(s["mask"][b, i])
                    hide = torch.tensor([not (w >> j) & 1 for j in range(n)], device=dev)
                    a[i * G:(i + 1) * G, L:] = a[i * G:(i + 1) * G, L:].masked_fill(hide, -math.inf)
            lse[b, :n, h * G:(h + 1) * G] = torch.logsumexp(a, -1).view(n, G)
            out[b, :n, h * G:(h + 1) * G] = (torch.softmax(a, -1) @ kv[1]).view(n, G, D)
            if c["page_lse"]:
                wide = torch.full((n * G, pages * PT), -math.inf, dtype=torch.float64, device=dev)
                wide[:, :L] = a[:, :L]
                page[b, :n, h * G:(h + 1) * G, :pages] = torch.logsumexp(wide.view(n, G, pages, PT), -1)
    return {"out": out, "lse": lse, "page_lse": page} if c["page_lse"] else {"out": out, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "tree":
        return _exact_tree(s)
    if case["op"] == "mass":
        w = (s["page_lse"].double() - s["lse"].double()[..., None]).exp()
        total = case["decay"] * s["mass"].double()
        for t in range(case["T"]):
            total += w[:, t].sum(1) * ((s["nodes"] >> t) & 1)[:, None]
        return {"mass": total}
    table, lens, mass = s["table"].cpu(), s["lens"].cpu().tolist(), s["mass"].double().cpu()
    kept_mass = torch.zeros_like(mass)
    for b, L in enumerate(lens):
        full, used = L // PT, -(-L // PT)
        fixed = set(range(min(case["sink"], full))) | set(range(max(0, full - case["recent"]), full))
        free = sorted((i for i in range(full) if i not in fixed), key=lambda i: (-float(mass[b, i]), i))
        stay = sorted(fixed | set(free[:max(0, case["keep"] - len(fixed))])) + list(range(full, used))
        kept_mass[b, :len(stay)] = mass[b, stay]
        gone = sorted(set(range(used)) - set(stay))
        table[b] = table[b, stay + list(range(used, case["P"])) + gone]
        lens[b] = L - PT * len(gone)
    n = s["lens"].cpu() - torch.tensor(lens, dtype=torch.int32)
    return {"page_table": table, "seq_lens": torch.tensor(lens, dtype=torch.int32), "evicted": (n // PT).to(torch.int32), "mass": kept_mass}
