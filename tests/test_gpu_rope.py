"""kvq_norm_rope against its 64-bit definition."""
import math

import pytest
import torch

import _prompt_reference as ref
from sub_byte_quantized_kvq_gb300 import kvq

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def handle(Hkv, D, B=1):
    return kvq.QuantizedKVCache(kvq.KVQ_FMT_FP4_E2M1_S16, B, Hkv, D, 1, 1)


def freqs(R, base=1e6):
    return (base ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)).float().cuda() if R else None


def close(got, x, weight, eps, pos, inv_freq, pair_axis, interleaved):
    y, size = ref.norm_rope(x, weight, eps, pos, inv_freq, pair_axis, interleaved)
    err = (got.double().cpu() - y).abs()
    bound = ref.norm_rope_bound(y, size, got.dtype)
    assert (err <= bound).all(), float((err / bound.clamp_min(1e-300)).max())


@pytest.mark.parametrize("D,R", [(64, 64), (64, 16), (64, 48), (128, 128), (128, 112), (128, 32), (128, 0), (64, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tin,tout", [(BF, BF), (HF, HF), (F32, F32), (F32, BF), (BF, F32), (HF, BF)])
def test_types_and_channels(D, R, interleaved, tin, tout):
    gen = torch.Generator(device="cuda").manual_seed(D + R)
    rows, Hq, Hkv = 37, 10, 5
    q, k = [(2 * torch.randn((rows, h, D), generator=gen, device="cuda")).to(tin) for h in (Hq, Hkv)]
    wq, wk = [1 + 0.5 * torch.randn(D, generator=gen, device="cuda") for _ in range(2)]
    pos = torch.randint(0, 200000, (1, rows), generator=gen, device="cuda", dtype=torch.int32)
    f = freqs(R)
    got = kvq.kvq_norm_rope(handle(Hkv, D), q, k, pos if R else None, f, wq, wk, eps=1e-5, interleaved=interleaved, out_dtype=tout)
    for y, x, w in zip(got, (q, k), (wq, wk)):
        assert y.dtype is tout and y.shape == x.shape
        close(y, x, w, 1e-5, pos, f, None, interleaved)


@pytest.mark.parametrize("rows", [1, 2, 3, 7, 64, 4097, 20011])
@pytest.mark.parametrize("Hq,Hkv,D", [(1, 1, 64), (4, 1, 128), (32, 8, 128), (21, 3, 64), (64, 4, 64)])
def test_rows_and_heads(rows, Hq, Hkv, D):
    gen = torch.Generator(device="cuda").manual_seed(rows)
    q, k = [torch.randn((rows, h, D), generator=gen, device="cuda").to(BF) for h in (Hq, Hkv)]
    w = 1 + 0.5 * torch.randn(D, generator=gen, device="cuda")
    pos, f = torch.arange(rows, device="cuda", dtype=torch.int32)[None] + 31000, freqs(D)
    qo, ko = kvq.kvq_norm_rope(handle(Hkv, D), q, k, pos, f, w, None)
    pick = torch.randperm(rows, generator=torch.Generator().manual_seed(1))[:200].sort().values.cuda()
    close(qo[pick], q[pick], w, 1e-6, pos[:, pick], f, None, False)
    close(ko[pick], k[pick], None, 1e-6, pos[:, pick], f, None, False)
    if rows > 200:   # every row was written: once more, into NaN, gives the same bits
        out = [torch.full_like(x, float("nan")) for x in (q, k)]
        kvq.kvq_norm_rope(handle(Hkv, D), q, k, pos, f, w, None, q_out=out[0], k_out=out[1])
        assert torch.equal(out[0], qo) and torch.equal(out[1], ko)


@pytest.mark.parametrize("axes,interleaved", [(2, False), (3, False), (3, True), (4, False)])
def test_axes(axes, interleaved):
    """Time, height and width: the axis of each pair, in sections or alternating."""
    gen = torch.Generator(device="cuda").manual_seed(axes)
    D, rows, Hq, Hkv = 128, 131, 6, 2
    q, k = [torch.randn((rows, h, D), generator=gen, device="cuda").to(BF) for h in (Hq, Hkv)]
    pos = torch.randint(-50, 3000, (axes, rows), generator=gen, device="cuda", dtype=torch.int32)
    f = freqs(D)
    for pair_axis in ([i * axes // 64 for i in range(64)], [i % axes for i in range(64)]):
        qo, ko = kvq.kvq_norm_rope(handle(Hkv, D), q, k, pos, f, interleaved=interleaved, pair_axis=pair_axis)
        close(qo, q, None, 1e-6, pos, f, pair_axis, interleaved)
        close(ko, k, None, 1e-6, pos, f, pair_axis, interleaved)


def test_positions_of_any_size():
    """Angles far beyond binary32's whole numbers, negative ones, and frequencies of more than a turn a position."""
    D, R = 64, 64
    pos = torch.tensor([[0, 1, -1, 131071, 1 << 20, (1 << 24) + 1, 2 ** 31 - 1, -2 ** 31, 123456789, -987654321]], dtype=torch.int32).cuda()
    q = torch.randn((pos.numel(), 3, D), generator=torch.Generator().manual_seed(0)).cuda()
    f = torch.cat([freqs(56), torch.tensor([0.0, 3.25, -0.75, 6.0]).cuda()])
    assert f.numel() == R // 2
    qo, none = kvq.kvq_norm_rope(handle(1, D), q, None, pos, f, eps=None)
    assert none is None
    y, size = ref.norm_rope(q, None, None, pos, f, None, False)
    # the phase itself: a frequency's fraction of a turn is below 1 and rounded twice in binary64 (2^-53 a position), and 32 bits
    # of the phase are kept (2^-33); and the reference's product, 2^-53 of up to 2^31 x 6.25 radians
    angle = 6.2832 * (2.0 ** -53 * pos.double().abs().cpu()[0] + 2.0 ** -33) + 2.0 ** -53 * 6.25 * pos.double().abs().cpu()[0]
    err = (qo.double().cpu() - y).abs()
    assert (err <= ref.norm_rope_bound(y, size, F32) + angle[:, None, None] * size).all()


def test_phase_of_the_farthest_positions():
    """The phase itself, against exact fractions, at frequencies whose product with a rounded 1 / (2 pi) would be off by more than
    2^-22 of a turn there: within 2^-27 of a turn at any int32 position."""
    inv_tau = 0x28BE60DB9391054A7F09D5F47D4D377036D8A5664F10E410   # 1 / (2 pi) 2^192: 2^64 turns' worth of bits behind any product here
    f = torch.tensor([6.2800726890563965, 6.279623508453369, 6.2367072105407715, 6.252718925476074, -6.282087802886963, -0.9548900127410889,
                      0.9847080707550049, 1.0, 2.0 ** -20, 1e-6, -1e-6, 1e-30, 0.0, 3.0, 5.5, -2.0 ** -12])
    pos = [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 123, 1500000001, -2000000011, 1 << 30, 12345, 131071, 1, 0]
    D, R = 64, 32
    q = torch.zeros((len(pos), 1, D))
    q[..., :R // 2] = 1.0
    qo, _ = kvq.kvq_norm_rope(handle(1, D), q.cuda(), None, torch.tensor(pos, dtype=torch.int32).cuda(), f.cuda(), eps=None)
    qo = qo.double().cpu()
    # 2^-27 of a turn, the sine's or cosine's own error (2 steps of 2^-24) and the rotation's rounding (one)
    bound = 2 * math.pi * 2.0 ** -27 + 3 * 2.0 ** -24
    for j, x in enumerate(f.tolist()):
        num, den = x.as_integer_ratio()
        for r, p in enumerate(pos):
            turn = (p * num * inv_tau // den) % (1 << 192) / (1 << 192)
            assert abs(float(qo[r, 0, j]) - math.cos(2 * math.pi * turn)) <= bound, (x, p)
            assert abs(float(qo[r, 0, R // 2 + j]) - math.sin(2 * math.pi * turn)) <= bound, (x, p)


def test_parts_of_one_projection_and_in_place():
    """Rows that are parts of a wider row, 4-D batches, and the outputs over the inputs."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    B, T, Hq, Hkv, D = 3, 50, 8, 2, 64
    wide = torch.randn((B, T, (Hq + 2 * Hkv) * D + 16), generator=gen, device="cuda").to(BF)
    q, k = wide[..., :Hq * D].unflatten(-1, (Hq, D)), wide[..., Hq * D:(Hq + Hkv) * D].unflatten(-1, (Hkv, D))
    pos, f, cache = torch.arange(B * T, device="cuda", dtype=torch.int32).view(B, T), freqs(D), handle(Hkv, D, B)
    qo, ko = kvq.kvq_norm_rope(cache, q, k, pos, f)
    want = kvq.kvq_norm_rope(cache, q.contiguous(), k.contiguous(), pos, f)
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1]) and qo.is_contiguous()
    before = wide.clone()
    got = kvq.kvq_norm_rope(cache, q, k, pos, f, q_out=q, k_out=k)
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(wide[..., (Hq + Hkv) * D:], before[..., (Hq + Hkv) * D:])   # V and what lies behind
    only, none = kvq.kvq_norm_rope(cache, None, before[..., Hq * D:(Hq + Hkv) * D].unflatten(-1, (Hkv, D)), pos, f)[::-1]
    assert none is None and torch.equal(only, want[1])
    empty = kvq.kvq_norm_rope(cache, q[:0], k[:0], pos[:0], f)
    assert empty[0].shape == (0, T, Hq, D)


def test_outputs_with_gaps():
    """Output rows that are parts of a wider row; what lies between stays."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    rows, Hq, Hkv, D = 300, 5, 1, 128
    q, k = [torch.randn((rows, h, D), generator=gen, device="cuda").to(HF) for h in (Hq, Hkv)]
    pos, f, cache = torch.arange(rows, device="cuda", dtype=torch.int32), freqs(96), handle(Hkv, D)
    want = kvq.kvq_norm_rope(cache, q, k, pos, f, out_dtype=BF)
    wide = torch.full((rows, 8 + (Hq + Hkv) * D + 8), 5.0, dtype=BF, device="cuda")
    qo, ko = wide[:, 8:8 + Hq * D].unflatten(1, (Hq, D)), wide[:, 8 + Hq * D:-8].unflatten(1, (Hkv, D))
    kvq.kvq_norm_rope(cache, q, k, pos, f, q_out=qo, k_out=ko)
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
    assert (wide[:, :8] == 5).all() and (wide[:, -8:] == 5).all()
    one = q[:1].expand(rows, Hq, D)   # one row for every position
    y, _ = kvq.kvq_norm_rope(cache, one, None, pos, f)
    z, _ = kvq.kvq_norm_rope(cache, one.contiguous(), None, pos, f)
    assert torch.equal(y, z)


def test_rows_far_apart():
    """Rows so far apart that their elements lie behind 2^31, of the inputs and of the outputs."""
    rows, step, Hq, Hkv, D = 601, 1 << 22, 3, 1, 64
    gen = torch.Generator(device="cuda").manual_seed(8)
    q, k = [torch.randn((rows, h, D), generator=gen, device="cuda").to(BF) for h in (Hq, Hkv)]
    pos, f, cache = torch.arange(rows, device="cuda", dtype=torch.int32), freqs(D), handle(Hkv, D)
    want = kvq.kvq_norm_rope(cache, q, k, pos, f)
    wide = torch.empty((rows, step), dtype=BF, device="cuda")
    qi, ki = wide[:, :Hq * D].unflatten(1, (Hq, D)), wide[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
    qo, ko = wide[:, 512:512 + Hq * D].unflatten(1, (Hq, D)), wide[:, 512 + Hq * D:512 + (Hq + Hkv) * D].unflatten(1, (Hkv, D))
    qi.copy_(q)
    ki.copy_(k)
    kvq.kvq_norm_rope(cache, qi, ki, pos, f, q_out=qo, k_out=ko)
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])


def test_special_values():
    """A NaN or an infinity stays in its head; rows of zeros stay zero; channels behind rot_dim do not meet the rotation."""
    D, R = 128, 32
    q = torch.randn((4, 4, D), generator=torch.Generator().manual_seed(5)).cuda()
    q[0, 1, 100] = float("inf")
    q[1, 2, 3] = float("nan")
    q[2, 3] = 0
    pos, f, cache = torch.tensor([5, 6, 7, 8], dtype=torch.int32).cuda(), freqs(R), handle(4, D)
    qo, _ = kvq.kvq_norm_rope(cache, q, None, pos, f)
    bad = ~torch.isfinite(qo).all(-1)
    assert bad.nonzero().tolist() == [[0, 1], [1, 2]] and (qo[2, 3] == 0).all()
    plain, _ = kvq.kvq_norm_rope(cache, q, None, pos, f, eps=None)
    assert not torch.isfinite(plain[0, 1, 100]) and torch.isfinite(plain[0, 1]).sum() == D - 1
    assert torch.equal(plain[0, 1, R:], q[0, 1, R:]) and torch.isnan(plain[1, 2, [3, 3 + R // 2]]).all()


def test_graph_and_stream():
    gen = torch.Generator(device="cuda").manual_seed(8)
    q, k = [torch.randn((9, h, 128), generator=gen, device="cuda").to(BF) for h in (16, 4)]
    pos, f, cache = torch.arange(9, device="cuda", dtype=torch.int32), freqs(128), handle(4, 128, 9)
    want = kvq.kvq_norm_rope(cache, q, k, pos, f)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = kvq.kvq_norm_rope(cache, q, k, pos, f, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    out = [torch.empty_like(q), torch.empty_like(k)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvq.kvq_norm_rope(cache, q, k, pos, f, q_out=out[0], k_out=out[1])
    pos += 11
    want = kvq.kvq_norm_rope(cache, q, k, pos, f)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
