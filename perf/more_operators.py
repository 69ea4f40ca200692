"""The operators before the quantized cache when a prompt arrives or a token is
decoded: per-head norms of queries and keys with the rotary positions in the
same pass, and attention of whole prompts (causal, grouped heads, padded or
packed sequences of different lengths).  Each case is one call on what a
layer's projection has just written.

Plain form: elementary torch operations in 32 bits (angles in 64); `own` makes
the library's calls instead."""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6


def listed():
    prompt = dict(op="prompt", dtype="bf16", packed=False, ragged=False, fused=False, causal=True)
    rope = dict(op="rope", dtype="bf16", out="bf16", axes=1, interleaved=False, norm=True, fused=False)
    return [
        # the smallest call: the question of one short chat turn, one kv head
        dict(prompt, name="prompt_17", B=1, Hkv=1, G=4, D=64, N=17),
        # one short request of the smallest cache
        dict(prompt, name="prompt_256", B=1, Hkv=1, G=4, D=64, N=256),
        # a padded batch of ordinary prompts
        dict(prompt, name="prompt_4k", B=8, Hkv=8, G=4, D=128, N=4096),
        # one long document: the largest call
        dict(prompt, name="prompt_32k", B=1, Hkv=8, G=8, D=128, N=32768),
        # a packed batch from one token to long prompts, read from the fused projection's rows, unused rows behind the last
        dict(prompt, name="prompt_packed", B=16, Hkv=8, G=8, D=128, N=6007, packed=True, ragged=True, fused=True),
        # fp16, narrow heads in groups of three, odd padded lengths
        dict(prompt, name="prompt_f16", dtype="f16", B=16, Hkv=2, G=3, D=64, N=1021, ragged=True),
        # the decode step of one request
        dict(rope, name="rope_token", B=1, T=1, Hkv=8, G=4, D=128, R=128, far=True),
        # the decode step of a full batch, far positions
        dict(rope, name="rope_batch", B=64, T=1, Hkv=8, G=8, D=128, R=128, far=True, fused=True),
        # a batch of ordinary prompts
        dict(rope, name="rope_4k", B=8, T=4096, Hkv=8, G=4, D=128, R=128, far=False),
        # one very long prompt, read from the fused projection's rows: the largest call
        dict(rope, name="rope_128k", B=1, T=131072, Hkv=8, G=4, D=128, R=128, far=False, fused=True),
        # image and video tokens: time, height and width positions, an odd count
        dict(rope, name="rope_axes", B=1, T=7777, Hkv=8, G=4, D=128, R=128, far=False, axes=3, fused=True),
        # fp32 rows, a quarter of the channels rotated in neighbouring pairs, no norm
        dict(rope, name="rope_part", dtype="f32", out="f32", B=3, T=1021, Hkv=4, G=2, D=64, R=16, far=True, interleaved=True, norm=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    if rng.random() < 0.5:
        while True:
            D = rng.choice([64, 128, 128])
            c = dict(op="rope", dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), B=_log(rng, 1, 64), T=_log(rng, 1, 131072),
                     Hkv=rng.choice([1, 2, 4, 8]), G=rng.choice([1, 2, 3, 4, 7, 8, 16]), D=D, R=16 * rng.randint(1, D // 16),
                     far=rng.random() < 0.5, axes=rng.choice([1, 1, 2, 3]), interleaved=rng.random() < 0.4, norm=rng.random() < 0.7,
                     fused=rng.random() < 0.5)
            c["out"] = rng.choice([c["dtype"], c["dtype"], "bf16"])
            if c["B"] * c["T"] * c["Hkv"] * (c["G"] + 1) * D <= 1 << 28:
                return c
    while True:
        c = dict(op="prompt", dtype=rng.choice(["bf16", "bf16", "f16"]), B=_log(rng, 1, 16), Hkv=rng.choice([1, 2, 4, 8]),
                 G=rng.choice([1, 2, 3, 4, 7, 8, 16]), D=rng.choice([64, 128, 128]), N=_log(rng, 1, 32768), packed=rng.random() < 0.5,
                 ragged=rng.random() < 0.6, fused=rng.random() < 0.5, causal=rng.random() < 0.8)
        heads = c["B"] * c["Hkv"] * c["G"]
        if heads * c["N"] * c["D"] <= 1 << 28 and heads * c["N"] ** 2 * c["D"] <= 1 << 40:
            return c


# ------------------------------------------------------------------ shapes
def _lens(c):
    """Tokens of each prompt: the first has all N, the others of a ragged batch anything down to one token."""
    n = c["N"]
    return [n if b == 0 or not c["ragged"] else max(1, int(n * ((b * 0.618034) % 1.0) ** 2)) for b in range(c["B"])]


def _rows(c):
    """First row of each prompt, and the rows there are."""
    lens = _lens(c)
    if not c["packed"]:
        return [b * c["N"] for b in range(c["B"])], c["B"] * c["N"]
    first = [sum(lens[:b]) for b in range(c["B"])]
    return first, sum(lens) + 37


def work(case):
    c = case
    if c["op"] == "rope":
        rows, heads = c["B"] * c["T"], c["Hkv"] * (c["G"] + 1)
        size = {"bf16": 2, "f16": 2, "f32": 4}
        moved = rows * heads * c["D"] * (size[c["dtype"]] + size[c["out"]]) + 4 * rows * c["axes"] + 2 * c["R"] + 8 * c["D"] * c["norm"]
        return {"bytes": moved, "flops": rows * heads * (3 * c["R"] + 4 * c["D"] * c["norm"])}
    lens, D, Hq, Hkv = _lens(c), c["D"], c["Hkv"] * c["G"], c["Hkv"]
    seen = sum(n * (n + 1) // 2 if c["causal"] else n * n for n in lens)
    return {"bytes": sum(lens) * (2 * D * (2 * Hq + 2 * Hkv) + 4 * Hq) + 8 * c["B"], "flops": 4.0 * D * Hq * seen}


# ------------------------------------------------------------------ inputs
def _cache(c, dev):
    """The buffers of the cache that the rows are meant for (neither operator reads them)."""
    B, Hkv, D = c["B"], c["Hkv"], c["D"]
    block = (9 * D + 127) // 128 * 128                                            # an FP4 block
    return dict(pool=torch.zeros(2 * Hkv * block, dtype=torch.uint8, device=dev), table=torch.zeros((B, 1), dtype=torch.int32, device=dev),
                lens=torch.zeros(B, dtype=torch.int32, device=dev), status=torch.zeros(1, dtype=torch.int32, device=dev))


def _split(c, rows, gen, dev, scale_kv):
    """q, k, v [rows, heads, D] in the case's type: parts of one projection's rows, or tensors of their own.  K and V
    have four loud channels a head."""
    Hq, Hkv, D = c["Hkv"] * c["G"], c["Hkv"], c["D"]
    dt = DTYPES[c["dtype"]]
    loud = torch.ones((2, Hkv, D), device=dev)
    at = torch.rand((2, Hkv, D), generator=gen, device=dev).argsort(-1)[..., :4]
    loud.scatter_(-1, at, scale_kv)
    wide = (Hq + 2 * Hkv) * D
    buf = torch.empty((rows, wide), dtype=dt, device=dev)
    step = max(1, (1 << 27) // wide)
    for r in range(0, rows, step):
        n = min(step, rows - r)
        x = torch.randn((n, Hq + 2 * Hkv, D), generator=gen, device=dev)
        x[:, Hq:Hq + Hkv] *= loud[0]
        x[:, Hq + Hkv:] *= loud[1]
        buf[r:r + n] = x.view(n, wide)
    parts = [p.unflatten(1, (-1, D)) for p in buf.split([Hq * D, Hkv * D, Hkv * D], 1)]
    return parts if c["fused"] else [p.contiguous() for p in parts]


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    Hq, Hkv, D, B = c["Hkv"] * c["G"], c["Hkv"], c["D"], c["B"]
    s = dict(case=c, **_cache(c, dev))
    if c["op"] == "rope":
        T, R, rows = c["T"], c["R"], c["B"] * c["T"]
        s["q"], s["k"], _ = _split(c, rows, gen, dev, 8.0)
        start = torch.randint(0, 131072 if c["far"] else 64, (B, 1), generator=gen, device=dev)
        pos = (start + torch.arange(T, device=dev)).flatten()
        if c["axes"] == 1:
            pos = pos[None]
        else:                                                                     # frames of 16 x 24 patches
            t, i = pos // 384, pos % 384
            pos = torch.stack([t, t + i // 24, t + i % 24][:c["axes"]])
        s["pos"] = pos.to(torch.int32).contiguous()
        s["freq"] = (1e6 ** (-torch.arange(0, R, 2, dtype=torch.float64, device=dev) / R)).float()
        s["pair_axis"] = None
        if c["axes"] > 1:                                                         # a quarter of the pairs turns with time
            s["pair_axis"] = [0 if i < R // 8 else 1 + (i - R // 8) * (c["axes"] - 1) // (R // 2 - R // 8) for i in range(R // 2)]
        s["wq"], s["wk"] = [1 + 0.3 * torch.randn(D, generator=gen, device=dev) for _ in range(2)] if c["norm"] else (None, None)
        dt = DTYPES[c["out"]]
        s["q_out"], s["k_out"] = [torch.zeros((rows, h, D), dtype=dt, device=dev) for h in (Hq, Hkv)]
        return s
    first, rows = _rows(c)
    lens = _lens(c)
    s["q"], s["k"], s["v"] = _split(c, rows, gen, dev, 4.0)
    live = torch.zeros(rows, dtype=torch.bool, device=dev)
    for f, n in zip(first, lens):
        live[f:f + n] = True
    for x in (s["q"], s["k"], s["v"]):                                            # rows of no prompt hold stale memory: anything
        x[~live] = math.nan
    s["first_rows"], s["lens_list"] = first, lens
    s["first"] = torch.tensor(first, dtype=torch.int32, device=dev)
    s["n"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    s["scale"] = D ** -0.5
    s["out"] = torch.zeros((rows, Hq, D), dtype=DTYPES[c["dtype"]], device=dev)
    s["lse"] = torch.zeros((rows, Hq), dtype=torch.float32, device=dev)
    return s


# ------------------------------------------------------------------ plain form
def _rotated(s, x, weight):
    c, R = s["case"], s["case"]["R"]
    x = x.float()
    if c["norm"]:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight
    axis = torch.tensor(s["pair_axis"] or [0] * (R // 2), device=x.device)
    phi = s["pos"][axis].double().T * s["freq"].double()                          # [rows, R / 2]
    cos, sin = phi.cos().float()[:, None], phi.sin().float()[:, None]
    part = x[..., :R].unflatten(-1, (R // 2, 2)) if c["interleaved"] else x[..., :R].unflatten(-1, (2, R // 2)).transpose(-1, -2)
    a, b = part[..., 0], part[..., 1]
    turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1)
    turned = turned.flatten(-2) if c["interleaved"] else turned.transpose(-1, -2).flatten(-2)
    return torch.cat([turned, x[..., R:]], -1).to(DTYPES[c["out"]])


def _rope_plain(s):
    rows = s["q"].shape[0]
    step = max(1, (1 << 27) // (s["q"].shape[1] * s["q"].shape[2]))
    got = {"q": torch.empty_like(s["q_out"]), "k": torch.empty_like(s["k_out"])}
    for r in range(0, rows, step):                                                # (long prompts: a part of the rows at a time)
        part = dict(s, pos=s["pos"][:, r:r + step])
        got["q"][r:r + step] = _rotated(part, s["q"][r:r + step], s["wq"])
        got["k"][r:r + step] = _rotated(part, s["k"][r:r + step], s["wk"])
    return got


def _prompt_plain(s):
    c = s["case"]
    G, Hkv, D = c["G"], c["Hkv"], c["D"]
    out, lse = torch.zeros_like(s["out"]), torch.zeros_like(s["lse"])
    for f, n in zip(s["first_rows"], s["lens_list"]):
        k, v = [s[x][f:f + n].float().transpose(0, 1) for x in "kv"]              # [Hkv, n, D]
        per = max(1, (1 << 29) // (Hkv * G * n))                                  # query tokens at a time
        for i in range(0, n, per):
            m = min(per, n - i)
            top = i + m if c["causal"] else n                                     # keys that any of them sees
            q = s["q"][f + i:f + i + m].float().view(m, Hkv, G, D).permute(1, 0, 2, 3).reshape(Hkv, m * G, D)
            a = torch.matmul(q, k[:, :top].transpose(1, 2)) * s["scale"]
            if c["causal"]:
                hide = torch.arange(top, device=q.device)[None, :] > i + torch.arange(m, device=q.device)[:, None]
                a.view(Hkv, m, G, top).masked_fill_(hide[None, :, None, :], -math.inf)
            peak = a.amax(-1, keepdim=True)
            p = a.sub_(peak).exp_()
            total = p.sum(-1, keepdim=True)
            o = torch.matmul(p, v[:, :top]) / total
            rows = slice(f + i, f + i + m)
            out[rows] = o.view(Hkv, m, G, D).permute(1, 0, 2, 3).reshape(m, Hkv * G, D).to(out.dtype)
            lse[rows] = (peak + total.log()).view(Hkv, m, G).permute(1, 0, 2).reshape(m, Hkv * G)
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------ the library's calls
def _handle(s, kvq):
    """The serving loop's handle on its cache."""
    if "cache" not in s:
        c = s["case"]
        s["cache"] = kvq.QuantizedKVCache.from_buffers(kvq.KVQ_FMT_FP4_E2M1_S16, c["Hkv"], c["D"], s["pool"], s["table"], s["lens"], s["status"])
    return s["cache"]


def _rope_own(s):
    from sub_byte_quantized_kvq_gb300 import kvq
    c = s["case"]
    kvq.kvq_norm_rope(_handle(s, kvq), s["q"], s["k"], s["pos"], s["freq"], q_weight=s["wq"], k_weight=s["wk"],
                      eps=EPS if c["norm"] else None, interleaved=c["interleaved"], pair_axis=s["pair_axis"], q_out=s["q_out"], k_out=s["k_out"])
    return {"q": s["q_out"], "k": s["k_out"]}


def _prompt_own(s):
    from sub_byte_quantized_kvq_gb300 import kvq
    c = s["case"]
    cache = _handle(s, kvq)
    if c["packed"]:
        kvq.kvq_prompt_attention(cache, s["q"], s["k"], s["v"], s["scale"], t_per_seq=s["n"], first_row=s["first"], t_new=c["N"],
                                 causal=c["causal"], out=s["out"], lse=s["lse"])
    else:
        q, k, v, out, lse = [s[x].unflatten(0, (c["B"], c["N"])) for x in ("q", "k", "v", "out", "lse")]
        kvq.kvq_prompt_attention(cache, q, k, v, s["scale"], t_per_seq=s["n"] if c["ragged"] else None, causal=c["causal"], out=out, lse=lse)
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    if state["case"]["op"] == "rope":
        return _rope_own(state) if own else _rope_plain(state)
    return _prompt_own(state) if own else _prompt_plain(state)


# ------------------------------------------------------------------ 64 bits
def _exact_rope(s):
    c, R, D = s["case"], s["case"]["R"], s["case"]["D"]
    got = {}
    for name, w in (("q", s["wq"]), ("k", s["wk"])):
        rows = s[name].shape[0]
        y = torch.empty(s[name].shape, dtype=torch.float64, device=s[name].device)
        step = max(1, (1 << 26) // (s[name].shape[1] * D))
        for r in range(0, rows, step):
            x = s[name][r:r + step].double()
            if c["norm"]:
                x = x / ((x ** 2).sum(-1, keepdim=True) / D + EPS).sqrt() * w.double()
            z = x.clone()
            for i in range(R // 2):
                a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + R // 2)
                axis = s["pair_axis"][i] if s["pair_axis"] else 0
                turn = torch.polar(torch.ones(x.shape[0], dtype=torch.float64, device=x.device),
                                   s["pos"][axis, r:r + step].double() * float(s["freq"][i]))
                t = torch.complex(x[..., a], x[..., b]) * turn[:, None]
                z[..., a], z[..., b] = t.real, t.imag
            y[r:r + step] = z
        got[name] = y
    return got


def _exact_prompt(s):
    c = s["case"]
    G, D = c["G"], c["D"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=s["out"].device)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=s["out"].device)
    for f, n in zip(s["first_rows"], s["lens_list"]):
        for h in range(c["Hkv"] * G):
            q, k, v = s["q"][f:f + n, h].double(), s["k"][f:f + n, h // G].double(), s["v"][f:f + n, h // G].double()
            step = max(64, (1 << 25) // n)
            for i in range(0, n, step):
                j = min(n, i + step)
                top = j if c["causal"] else n
                a = torch.einsum("id,jd->ij", q[i:j], k[:top]) * s["scale"]
                if c["causal"]:
                    a += torch.full_like(a, -math.inf).triu(i + 1)
                lse[f + i:f + j, h] = a.logsumexp(-1)
                out[f + i:f + j, h] = (a - lse[f + i:f + j, h, None]).exp() @ v[:top]
    return {"out": out, "lse": lse}


def exact(case, seed):
    if case["op"] == "prompt" and work(case)["flops"] > 3e12:
        return None                                                               # (too long in 64 bits)
    s = prepare(case, seed)
    return _exact_rope(s) if case["op"] == "rope" else _exact_prompt(s)
