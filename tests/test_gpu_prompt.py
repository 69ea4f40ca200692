"""kvq_prompt_attention against its 64-bit definition."""
import math

import pytest
import torch

import _prompt_reference as ref
from sub_byte_quantized_kvq_gb300 import kvq

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
NAN = float("nan")


def handle(B, Hkv, D):
    return kvq.QuantizedKVCache(kvq.KVQ_FMT_FP4_E2M1_S16, B, Hkv, D, 1, 1)


def inputs(rows, Hq, Hkv, D, dtype, seed, fused=False):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    wide = torch.randn((rows, (Hq + 2 * Hkv) * D), generator=gen, device="cuda")
    wide[:, :Hq * D] *= 1.5
    parts = [p.unflatten(1, (-1, D)) for p in wide.to(dtype).split([Hq * D, Hkv * D, Hkv * D], 1)]
    return parts if fused else [p.contiguous() for p in parts]


def check(out, lse, q, k, v, scale, causal):
    """One sequence's rows."""
    n = q.shape[0]
    if n == 0:
        return
    y, z, size, reach = ref.prompt(q, k, v, scale, causal)
    bound, zbound = ref.prompt_bounds(y, z, size, reach, float(v.double().abs().max()), n, q.shape[-1], q.dtype, out.dtype)
    err = (out.double() - y).abs()
    assert (err <= bound).all(), float((err / bound).max())
    if lse is not None:
        assert ((lse.double() - z).abs() <= zbound).all(), float(((lse.double() - z).abs() / zbound).max())


def run(lens, Hkv, G, D, dtype=BF, causal=True, packed=True, fused=False, out_dtype=None, seed=0, scale=None, change=None, gap=3):
    """Sequences of `lens` tokens in one call; rows of none hold NaN.  change(q, k, v, first): further edits of the inputs."""
    B, Hq = len(lens), Hkv * G
    live = [max(n, 0) for n in lens]
    if packed:   # out of order, with gaps
        order = list(range(1, B)) + [0]
        first, at = [0] * B, 2
        for b in order:
            first[b] = at
            at += live[b] + gap
        rows, t_new = at, max(live + [1])
    else:
        t_new = max(live + [1]) + 1
        first, rows = [b * t_new for b in range(B)], B * t_new
    q, k, v = inputs(rows, Hq, Hkv, D, dtype, seed, fused)
    used = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for f, n in zip(first, live):
        used[f:f + n] = True
    if change:
        change(q, k, v, first)
    for x in (q, k, v):
        x[~used] = NAN
    scale = D ** -0.5 if scale is None else scale
    cache = handle(B, Hkv, D)
    out = torch.full((rows, Hq, D), 7.0, dtype=out_dtype or dtype, device="cuda")
    lse = torch.full((rows, Hq), 7.0, device="cuda")
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if packed:
        got = kvq.kvq_prompt_attention(cache, q, k, v, scale, t_per_seq=n, first_row=torch.tensor(first, dtype=torch.int32, device="cuda"),
                                       t_new=t_new, causal=causal, out=out, lse=lse)
        assert got is out
    else:
        kvq.kvq_prompt_attention(cache, *[x.unflatten(0, (B, t_new)) for x in (q, k, v)], scale, t_per_seq=n, causal=causal,
                                 out=out.unflatten(0, (B, t_new)), lse=lse.unflatten(0, (B, t_new)))
    assert cache.status_word() == 0
    assert (out[~used] == 7).all() and (lse[~used] == 7).all()   # rows of no sequence
    return out, lse, q, k, v, first, scale


def run_and_check(lens, *args, causal=True, **kw):
    out, lse, q, k, v, first, scale = run(lens, *args, causal=causal, **kw)
    for f, n in zip(first, lens):
        s = slice(f, f + max(n, 0))
        check(out[s], lse[s], q[s], k[s], v[s], scale, causal)


LENGTHS = [[1], [2, 1, 3], [15, 16, 17, 0, 5, 31, 32, 33], [63, 64, 65, -3, 127], [128], [129, 1, 128], [255, 256, 257], [300, 511],
           [513, 640], [1000], [1, 1500, 7, 384]]


@pytest.mark.parametrize("lens", LENGTHS, ids=lambda x: "-".join(map(str, x)))
@pytest.mark.parametrize("Hkv,G,D", [(2, 4, 128), (1, 8, 64), (2, 1, 64), (1, 3, 128), (1, 16, 128)])
@pytest.mark.parametrize("causal", [True, False])
def test_lengths(lens, Hkv, G, D, causal):
    run_and_check(lens, Hkv, G, D, causal=causal, seed=len(lens))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("packed,fused,out", [(True, True, None), (False, False, None), (False, True, F32)])
@pytest.mark.parametrize("G", [1, 2, 5, 6, 7, 12])
def test_types_layouts_and_groups(dtype, D, packed, fused, out, G):
    run_and_check([200, 0, 333, 64], 2, G, D, dtype=dtype, packed=packed, fused=fused, out_dtype=out, seed=G)


@pytest.mark.parametrize("n,Hkv,G,D,dtype", [(4133, 1, 2, 128, BF), (2999, 2, 4, 64, HF), (6001, 1, 1, 64, BF)])
def test_many_tiles(n, Hkv, G, D, dtype):
    run_and_check([n, 700], Hkv, G, D, dtype=dtype)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("causal", [True, False])
def test_growing_scores(D, dtype, causal):
    """Scores that rise (and fall) along the keys by far more than the exponential's range: the maximum has to follow."""
    def change(q, k, v, first):
        n = q.shape[0]
        ramp = torch.linspace(-12, 12, n, device="cuda")
        q[..., 0], k[..., 0] = 16.0, ramp[:, None].to(k.dtype)
        q[::2, ..., 0] = -16.0
    run_and_check([700, 400], 1, 4, D, dtype=dtype, causal=causal, scale=1.0, change=change)


@pytest.mark.parametrize("scale", [0.0, -0.25, 3.0])
def test_any_scale(scale):
    run_and_check([300, 40], 2, 2, 64, scale=scale)


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), NAN])
@pytest.mark.parametrize("D,G", [(128, 1), (64, 8)])
def test_later_tokens_do_not_reach_earlier_ones(bad, D, G):
    """Infinities and NaN in K and V of some tokens: what does not attend to them is as without them, what does is not finite
    in V's channel."""
    lens, at = [290, 130], {0: [289, 150, 131], 1: [129]}
    clean = run(lens, 1, G, D, seed=4)
    def change_v(q, k, v, first):
        for b, js in at.items():
            for j in js:
                v[first[b] + j, 0, 5] = bad
    def change_k(q, k, v, first):
        for b, js in at.items():
            for j in js:
                k[first[b] + j, 0, 9] = NAN if bad != bad else bad
    out, lse, *_, first, _ = run(lens, 1, G, D, seed=4, change=change_v)
    assert torch.equal(lse, clean[1])
    for b, js in at.items():
        for i in range(lens[b]):
            r = first[b] + i
            hit = min(js) <= i
            same = out[r] == clean[0][r]
            assert same[:, [c for c in range(D) if c != 5]].all()
            assert (~torch.isfinite(out[r][:, 5])).all() if hit else same[:, 5].all()
            if hit and bad == bad and all(j <= i for j in js if j <= i):
                assert (out[r][:, 5] == bad).all()
    out, lse, *_, first, _ = run(lens, 1, G, D, seed=4, change=change_k)
    for b, js in at.items():
        s = slice(first[b], first[b] + min(js))
        assert torch.equal(out[s], clean[0][s]) and torch.equal(lse[s], clean[1][s])
        if bad != bad:
            late = slice(first[b] + min(js), first[b] + lens[b])
            assert torch.isnan(out[late]).all() and torch.isnan(lse[late]).all()


def test_rows_that_do_not_fit_are_skipped():
    """A sequence that is too long, or lies outside the rows, is left out and flagged; the others are computed."""
    Hkv, G, D, rows = 1, 2, 64, 100
    q, k, v = inputs(rows, 2, 1, D, BF, 1)
    for first, lens, good in (([0, 40], [41, 30], [False, True]), ([0, 90], [30, 11], [True, False]), ([-1, 50], [10, 40], [False, True]),
                              ([2 ** 31 - 1, 0], [5, 40], [False, True]), ([60, 0], [40, 40], [True, True])):
        cache = handle(2, Hkv, D)
        out = torch.full((rows, 2, D), 7.0, dtype=BF, device="cuda")
        kvq.kvq_prompt_attention(cache, q, k, v, 0.125, t_per_seq=torch.tensor(lens, dtype=torch.int32).cuda(),
                                 first_row=torch.tensor(first, dtype=torch.int32).cuda(), t_new=40, out=out)
        assert cache.status_word() == (0 if all(good) else kvq.KVQ_STATUS_BAD_ROWS)
        used = torch.zeros(rows, dtype=torch.bool, device="cuda")
        for f, n, g in zip(first, lens, good):
            if g:
                used[f:f + n] = True
                s = slice(f, f + n)
                check(out[s], None, q[s], k[s], v[s], 0.125, True)
        assert (out[~used] == 7).all()


def test_many_short_sequences():
    """More sequences than a warp has lanes, their lengths from none up."""
    lens = [(7 * b) % 23 for b in range(151)]
    run_and_check(lens, 1, 2, 64)
    run_and_check([5] * 70 + [300] + [0] * 40 + [129] * 3, 2, 1, 128)


def test_scores_that_jump_within_a_tile():
    """Each run of 64 keys scores far above (or below) the one before: the maximum has to follow between the halves of a tile."""
    steps = torch.tensor([0, 40, 3, 90, -50, 91, 150, 0, 151, 260, 20, 261], dtype=torch.float32, device="cuda")
    for dtype, D in ((BF, 128), (HF, 64)):
        def change(q, k, v, first):
            q[..., 0] = 1.0
            n = 12 * 64
            k[first[0]:first[0] + n, ..., 0] = steps.repeat_interleave(64)[:, None].to(k.dtype)
        for causal in (True, False):
            run_and_check([12 * 64, 100], 1, 2, D, dtype=dtype, causal=causal, scale=1.0, change=change, seed=2)


@pytest.mark.parametrize("dtype,D,G", [(BF, 128, 1), (HF, 64, 4), (BF, 64, 2), (HF, 128, 1)])
@pytest.mark.parametrize("causal", [True, False])
def test_scores_that_jump_in_both_halves_of_a_tile(dtype, D, G, causal):
    """Behind the first tile, both halves of a tile raise the maximum of rows of one warp: every third token in the first
    half, every third in the second, every third in both.  O is then scaled twice in a row, by 1 where a row does not jump."""
    first_half = torch.tensor([0, 0, 40, 40, 90, 90, 90, 90, 130, 130, 0, 0], dtype=torch.float32, device="cuda")
    second_half = torch.tensor([0, 0, 0, 30, 30, 75, 75, 75, 75, 110, 110, 0], dtype=torch.float32, device="cuda")
    n = 64 * first_half.numel()
    def change(q, k, v, first):
        s = slice(first[0], first[0] + n)
        q.mul_(0.05)
        q[..., :2] = 0.0
        third = torch.arange(n, device="cuda") % 3
        q[s, :, 0] = (third != 1).to(q.dtype)[:, None]
        q[s, :, 1] = (third != 0).to(q.dtype)[:, None]
        for c, steps in enumerate((first_half, second_half)):
            k[s, :, c] = steps.repeat_interleave(64)[:, None].to(k.dtype)
    run_and_check([n, 100], 1, G, D, dtype=dtype, causal=causal, scale=1.0, change=change, seed=6)


@pytest.mark.parametrize("below", [8.0, 14.0, 17.0, 20.0, 24.0])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_one_key_far_above_the_rest(dtype, below):
    """A first key that takes nearly all the weight and whose V is 0: what is left of the output are the small weights, which
    fp16 holds to 2^-31 of the largest (a relative bound alone does not hold there), bf16 to 2^-8 of each."""
    n, D = 2500, 64
    def change(q, k, v, first):
        q.mul_(0.02)
        q[..., 0] = 1.0
        k[..., 0] = 0.0
        k[first[0], :, 0] = below
        v[first[0]] = 0.0
        v.copy_(v.abs())
    out, lse, q, k, v, first, scale = run([n], 1, 2, D, dtype=dtype, scale=1.0, change=change, out_dtype=F32, seed=12)
    s = slice(first[0], first[0] + n)
    check(out[s], lse[s], q[s], k[s], v[s], scale, True)
    y, _, size, reach = ref.prompt(q[s], k[s], v[s], scale, True)
    e = 2.0 ** -11 if dtype is HF else 2.0 ** -8
    loss = (((out[s].double() - y).abs() / size.clamp_min(1e-300))[n // 2:]).max()
    # 2^-31 of the largest weight, over what the small ones hold: e^-below of it each, the noise of the other channels included
    few = 2.0 ** -31 / math.exp(-below - 1.5) if dtype is HF else 0.0
    # scores: 2 (2^-23 (D + 2) sum |q k| + 2^-21), sums 2^-23 n, as in prompt_bounds
    rest = 2 * (2.0 ** -23 * (D + 2) * float(reach.max()) + 2.0 ** -21) + 2.0 ** -23 * n
    assert loss <= e + few + rest, float(loss)


def test_scores_of_minus_infinity():
    """Keys that score -inf have no weight; a token that sees no other gets 0 and lse -inf."""
    n, m, G, D = 700, 333, 2, 128
    def change(q, k, v, first):
        q[..., 0] = q[..., 0].abs() + 0.5
        k[first[0]:first[0] + m, ..., 0] = -math.inf
    out, lse, q, k, v, first, scale = run([n], 1, G, D, change=change)
    s = slice(first[0], first[0] + m)
    assert (out[s] == 0).all() and (lse[s] == -math.inf).all()
    s = slice(first[0] + m, first[0] + n)   # the rest attends to itself alone
    check(out[s], lse[s], q[s], k[s], v[s], scale, True)


@pytest.mark.parametrize("offset,pad", [(8, 0), (0, 8), (16, 24)])
def test_out_rows_of_any_alignment(offset, pad):
    """Output rows that are 16-byte, not 32-byte aligned, with a gap behind each."""
    n, Hq, Hkv, D = 300, 4, 2, 64
    q, k, v = inputs(n, Hq, Hkv, D, BF, 7)
    cache = handle(1, Hkv, D)
    want = kvq.kvq_prompt_attention(cache, q[None], k[None], v[None], 0.125)
    flat = torch.full((offset + n * (Hq * D + pad),), 3.0, dtype=BF, device="cuda")
    rows = flat[offset:].view(n, Hq * D + pad)
    out = rows[:, :Hq * D].unflatten(1, (Hq, D))[None]
    kvq.kvq_prompt_attention(cache, q[None], k[None], v[None], 0.125, out=out)
    assert torch.equal(out, want) and (rows[:, Hq * D:] == 3).all() and (flat[:offset] == 3).all()


def test_more_sequences_than_registers_hold():
    gen = torch.Generator().manual_seed(5)
    lens = torch.randint(-2, 200, (700,), generator=gen).tolist()
    out, lse, q, k, v, first, scale = run(lens, 1, 2, 64, gap=0)
    for b in [0, 1, 255, 256, 257, 511, 698, 699] + torch.randint(0, 700, (40,), generator=gen).tolist():
        s = slice(first[b], first[b] + max(lens[b], 0))
        check(out[s], lse[s], q[s], k[s], v[s], scale, True)
    # every row was written (run() looked at the others)
    for f, n in zip(first, lens):
        assert n <= 0 or bool((lse[f:f + n] != 7).all())


def test_runs_of_sequences_without_tokens():
    """Hundreds of sequences in a row without tokens, and the longest ones far behind the first."""
    lens = [3] + [0] * 599 + [700, 1] + [0] * 290 + [5, 1500] + [-1] * 300 + [130]
    run_and_check(lens, 1, 2, 64, gap=0)
    run_and_check([0] * 1000 + [17], 2, 4, 128)
    run_and_check([0] * 300, 1, 1, 64)


def padded_and_packed(B, t_new, lens, Hkv, G, D, seed):
    """The same sequences as a padded batch, NaN behind each, and packed."""
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    first = (n.cumsum(0) - n).to(torch.int32)
    packed = inputs(sum(lens), Hkv * G, Hkv, D, BF, seed)
    at = torch.cat([b * t_new + torch.arange(m) for b, m in enumerate(lens)]).cuda()   # of each packed row
    padded = []
    for x in packed:
        y = torch.full((B * t_new, *x.shape[1:]), NAN, dtype=BF, device="cuda")
        y[at] = x
        padded.append(y.unflatten(0, (B, t_new)))
    return n, first, packed, padded, at


@pytest.mark.parametrize("B,t_new", [(300, 2400), (67, 12300), (515, 1000)])
def test_short_prompts_padded_to_a_long_one(B, t_new):
    """Few sequences are taken at a time where their padded length is long: the same bits as the same sequences packed."""
    Hkv, G, D = 4, 2, 128
    lens = torch.randint(0, 65, (B,), generator=torch.Generator().manual_seed(B)).tolist()
    for b in (3, B // 2, B - 2):
        lens[b] = t_new - b % 5
    n, first, packed, padded, at = padded_and_packed(B, t_new, lens, Hkv, G, D, 17)
    cache, rows = handle(B, Hkv, D), B * t_new
    wlse = torch.empty((sum(lens), Hkv * G), device="cuda")
    want = kvq.kvq_prompt_attention(cache, *packed, 0.09, t_per_seq=n, first_row=first, t_new=max(lens), lse=wlse)
    out, lse = torch.full((rows, Hkv * G, D), 7.0, dtype=BF, device="cuda"), torch.full((rows, Hkv * G), 7.0, device="cuda")
    kvq.kvq_prompt_attention(cache, *padded, 0.09, t_per_seq=n, out=out.unflatten(0, (B, t_new)), lse=lse.unflatten(0, (B, t_new)))
    assert torch.equal(out[at], want) and torch.equal(lse[at], wlse) and cache.status_word() == 0
    out[at], lse[at] = 7.0, 7.0
    assert (out == 7).all() and (lse == 7).all()
    for b in (0, 3, B - 1):
        s = slice(int(first[b]), int(first[b]) + lens[b])
        check(want[s], wlse[s], *[x[s] for x in packed], 0.09, True)


def test_padding_costs_little():
    """256 prompts of up to 64 tokens take about as long padded to 6200 as packed (and not a memory latency for each sequence more:
    four times as long)."""
    B, t_new, Hkv, G, D = 256, 6200, 4, 1, 128
    lens = torch.randint(1, 65, (B,), generator=torch.Generator().manual_seed(2)).tolist()
    n, first, packed, padded, _ = padded_and_packed(B, t_new, lens, Hkv, G, D, 18)
    cache, out, wide = handle(B, Hkv, D), torch.empty_like(packed[0]), torch.empty_like(padded[0])
    def us(call):
        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(5):
                call()
        best = math.inf
        for _ in range(10):
            a, b = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
            a.record()
            graph.replay()
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b) * 200)
        return best
    apart = us(lambda: kvq.kvq_prompt_attention(cache, *packed, 0.09, t_per_seq=n, first_row=first, t_new=64, out=out))
    filled = us(lambda: kvq.kvq_prompt_attention(cache, *padded, 0.09, t_per_seq=n, out=wide))
    assert filled < 2 * apart, (filled, apart)


def test_a_sequence_that_does_not_fit_among_many():
    n, at = 5, 801
    B, Hkv, G, D = 1000, 1, 1, 64
    q, k, v = inputs(B * n, Hkv * G, Hkv, D, BF, 3)
    first = torch.arange(0, B * n, n, dtype=torch.int32, device="cuda")
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    lens[at] = n + 1
    cache = handle(B, Hkv, D)
    out = torch.full_like(q, 7.0)
    kvq.kvq_prompt_attention(cache, q, k, v, 0.125, t_per_seq=lens, first_row=first, t_new=n, out=out)
    assert cache.status_word() == kvq.KVQ_STATUS_BAD_ROWS
    skipped = slice(at * n, at * n + n)
    assert (out[skipped] == 7).all()
    for b in (0, at - 1, at + 1, B - 1):
        s = slice(b * n, b * n + n)
        check(out[s], None, q[s], k[s], v[s], 0.125, True)


def test_two_calls_at_once():
    """Calls on two streams share nothing but their inputs, and give the same bits as one after the other."""
    a = inputs(4096, 8, 2, 128, BF, 1)
    b = inputs(3000, 6, 2, 64, HF, 2)
    ca, cb = handle(2, 2, 128), handle(3, 2, 64)
    one = [x.view(2, 2048, *x.shape[1:]) for x in a], [x.view(3, 1000, *x.shape[1:]) for x in b]
    want = kvq.kvq_prompt_attention(ca, *one[0], 0.1), kvq.kvq_prompt_attention(cb, *one[1], 0.1, causal=False)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(5):
        got.append((kvq.kvq_prompt_attention(ca, *one[0], 0.1, stream=s1), kvq.kvq_prompt_attention(cb, *one[1], 0.1, causal=False, stream=s2)))
    s1.synchronize()
    s2.synchronize()
    for x, y in got:
        assert torch.equal(x, want[0]) and torch.equal(y, want[1])
    assert ca.status_word() == 0 and cb.status_word() == 0


def test_long_prompt_sampled():
    """20,011 tokens: some tokens against all the keys that they see."""
    n, Hq, Hkv, D = 20011, 4, 1, 128
    q, k, v = inputs(n, Hq, Hkv, D, BF, 9)
    lse = torch.empty((1, n, Hq), device="cuda")
    out = kvq.kvq_prompt_attention(handle(1, Hkv, D), q[None], k[None], v[None], 0.09, lse=lse, out_dtype=F32)[0]
    for i in [0, 1, 127, 128, 129, 4095, 9999, 12345, n - 2, n - 1]:
        a = q[i].double() @ k[:i + 1, 0].double().T * 0.09
        z = a.logsumexp(-1)
        p = (a - z[:, None]).exp()
        y, size = p @ v[:i + 1, 0].double(), p @ v[:i + 1, 0].double().abs()
        reach = (q[i].double().abs() @ k[:i + 1, 0].double().abs().T * 0.09).amax(-1)
        bound, zbound = ref.prompt_bounds(y, z, size, reach, float(v.double().abs().max()), i + 1, D, BF, F32)
        assert ((out[i].double() - y).abs() <= bound).all() and ((lse[0, i].double() - z).abs() <= zbound).all()


@pytest.mark.parametrize("lens,padded", [([20011, 5, 0, 12000], False), ([9001, 9001], True), ([3001] * 7, True), ([2999, 3100] * 4, False),
                                         ([70, 9100, 130], False)])
@pytest.mark.parametrize("causal", [True, False])
def test_more_keys_than_are_taken_at_once(lens, padded, causal):
    """K and V far beyond what the order of the pairs takes at a time: each head's rows are, bit for bit, those of a call of its
    own, and every row is written."""
    B, Hkv, G, D = len(lens), 8, 2 if padded else 1, 128
    first = torch.tensor([sum(lens[:b]) for b in range(B)], dtype=torch.int32, device="cuda")
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q, k, v = inputs(sum(lens), Hkv * G, Hkv, D, BF, 21)
    def attend(Hkv, q, k, v):
        lse = torch.full(q.shape[:2], 7.0, device="cuda")
        if padded:
            shape = (B, lens[0])
            out = kvq.kvq_prompt_attention(handle(B, Hkv, D), *[x.unflatten(0, shape) for x in (q, k, v)], 0.09, causal=causal, lse=lse.unflatten(0, shape))
            return out.flatten(0, 1), lse
        return kvq.kvq_prompt_attention(handle(B, Hkv, D), q, k, v, 0.09, t_per_seq=n, first_row=first, t_new=max(lens), causal=causal, lse=lse), lse
    out, lse = attend(Hkv, q, k, v)
    assert (lse != 7).all()
    for h in range(Hkv):
        heads = slice(h * G, h * G + G)
        o, z = attend(1, q[:, heads], k[:, h:h + 1], v[:, h:h + 1])
        assert torch.equal(out[:, heads], o) and torch.equal(lse[:, heads], z)
    s = slice(0, min(lens[0], 2000))
    if causal:
        check(out[s], lse[s], q[s], k[s], v[s], 0.09, True)


def test_rows_far_apart():
    """Rows so far apart that their elements lie behind 2^31, of the inputs and of out."""
    rows, step, Hq, Hkv, D, lens, first = 700, 1 << 22, 2, 1, 64, [130, 40], [560, 3]
    q, k, v = inputs(rows, Hq, Hkv, D, BF, 13)
    want = torch.full((rows, Hq, D), 7.0, dtype=BF, device="cuda")
    n, f = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (lens, first)]
    cache = handle(2, Hkv, D)
    kvq.kvq_prompt_attention(cache, q, k, v, 0.125, t_per_seq=n, first_row=f, t_new=130, out=want)
    wide = torch.empty((rows, step), dtype=BF, device="cuda")
    parts, at = [], 0
    for x in (q, k, v, want):
        parts.append(wide[:, at:at + x[0].numel()].unflatten(1, x.shape[1:]))
        at += x[0].numel()
        parts[-1].copy_(x)
    parts[3].fill_(7)
    kvq.kvq_prompt_attention(cache, *parts[:3], 0.125, t_per_seq=n, first_row=f, t_new=130, out=parts[3])
    assert torch.equal(parts[3], want) and cache.status_word() == 0


def test_graph_streams_and_repeats():
    gen_lens = [700, 33]
    out, lse, q, k, v, first, scale = run(gen_lens, 2, 4, 128)
    cache = handle(2, 2, 128)
    n, f = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (gen_lens, first)]
    again, relse = torch.full_like(out, 7), torch.full_like(lse, 7)
    args = dict(t_per_seq=n, first_row=f, t_new=700, out=again, lse=relse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kvq.kvq_prompt_attention(cache, q, k, v, scale, stream=side, **args)
    side.synchronize()
    assert torch.equal(again, out) and torch.equal(relse, lse)   # the same bits
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvq.kvq_prompt_attention(cache, q, k, v, scale, **args)
    n.copy_(torch.tensor([129, 31]))
    q.neg_()
    again.fill_(7)
    graph.replay()
    for b, m in enumerate((129, 31)):
        s = slice(first[b], first[b] + m)
        check(again[s], relse[s], q[s], k[s], v[s], scale, True)
        assert (again[first[b] + m:first[b] + gen_lens[b]] == 7).all()
    assert cache.status_word() == 0


def test_prompt_then_decode():
    """The calls together: norms and rotation, the prompt's attention, the append, and a decoded token."""
    B, T, Hq, Hkv, D, P = 2, 45, 8, 2, 64, 4
    gen = torch.Generator(device="cuda").manual_seed(11)
    lens = torch.tensor([45, 18], dtype=torch.int32, device="cuda")
    cache = kvq.QuantizedKVCache(kvq.KVQ_FMT_FP4_E2M1_S16, B, Hkv, D, P, B * P)
    wide = torch.randn((B, T, (Hq + 2 * Hkv) * D), generator=gen, device="cuda").to(BF)
    q, k, v = [p.unflatten(-1, (-1, D)) for p in wide.split([Hq * D, Hkv * D, Hkv * D], -1)]
    f = (1e4 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().cuda()
    w = 1 + 0.1 * torch.randn(D, generator=gen, device="cuda")
    pos = torch.arange(T, device="cuda", dtype=torch.int32).repeat(B, 1)
    qr, kr = kvq.kvq_norm_rope(cache, q, k, pos, f, w, w)
    lse = torch.zeros((B, T, Hq), device="cuda")
    out = kvq.kvq_prompt_attention(cache, qr, kr, v, D ** -0.5, t_per_seq=lens, lse=lse)
    for b, n in enumerate(lens.tolist()):
        check(out[b, :n], lse[b, :n], qr[b, :n], kr[b, :n], v[b, :n], D ** -0.5, True)
    kvq.kvq_quantize_append(cache, kr, v.contiguous(), t_per_seq=lens)
    assert cache.seq_lens.tolist() == [45, 18]
    one = torch.randn((B, 1, (Hq + 2 * Hkv) * D), generator=gen, device="cuda").to(BF)
    q1, k1, v1 = [p.unflatten(-1, (-1, D)) for p in one.split([Hq * D, Hkv * D, Hkv * D], -1)]
    q1, k1 = kvq.kvq_norm_rope(cache, q1, k1, cache.seq_lens, f, w, w)     # positions 45 and 18
    kvq.kvq_quantize_append(cache, k1, v1.contiguous())
    got = kvq.kvq_decode_attention(cache, q1[:, 0].contiguous(), D ** -0.5, 64, out_dtype=F32)
    for b, n in enumerate((46, 19)):
        kd, vd = [torch.stack([kvq.kvq_dequantize(cache, b, h, r, 0, n) for h in range(Hkv)], 1).double() for r in (0, 1)]
        # the rotation at the cache's own length is that of position n - 1
        pq, _ = ref.norm_rope(one[b, :, :Hq * D].unflatten(-1, (Hq, D)), w, 1e-6, torch.tensor([[n - 1]]), f, None, False)
        assert (q1[b].double().cpu() - pq).abs().max() <= 2.0 ** -8 * pq.abs().max() + 1e-5
        a = torch.einsum("hgd,nhd->hgn", q1[b, 0].double().unflatten(0, (Hkv, Hq // Hkv)), kd) * D ** -0.5
        want = torch.einsum("hgn,nhd->hgd", a.softmax(-1), vd).flatten(0, 1)
        assert (got[b].double() - want).abs().max() <= 2e-3
    assert cache.status_word() == 0 and math.isfinite(float(got.sum()))
