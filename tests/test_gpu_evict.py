"""Page mass and page eviction against their definitions, and a run of them with
tree attention and the append, as a serving loop makes it."""
import types

import numpy as np
import pytest
import torch

from _kvq_pairs import Pair, make_kv
from _tree_reference import evict, page_mass, sees_from_parents, tree_rows
from sub_byte_quantized_kvq_gb300 import kvq

pytestmark = pytest.mark.gpu


def handle(B, P, fmt=kvq.KVQ_FMT_FP4_E2M1_S16):
    return kvq.QuantizedKVCache(fmt, B, 1, 64, P, B * P)


@pytest.mark.parametrize("B,T,Hq,P,ppsm", [(1, 1, 4, 16, 16), (3, 5, 7, 33, 40), (2, 64, 8, 130, 130), (1, 1, 1, 1, 3),
                                           (2, 3, 64, 2049, 2050), (2, 2, 4, 0, 5)])
def test_page_mass(B, T, Hq, P, ppsm):
    """Sums of n terms e^x: each off by 2^-20 relative, the fp32 sum by n 2^-24 of the total."""
    g = torch.Generator().manual_seed(B * 1000 + P)
    x = torch.randn((B, T, Hq, P), generator=g) * 2
    lse = torch.logsumexp(x, -1) + 0.2 if P else torch.zeros((B, T, Hq))
    if P > 2:
        x[0, 0, 0, 1:] = -np.inf                        # a page without tokens of a short sequence
        lse[-1, -1] = -np.inf                           # an empty row
        x[-1, -1] = -np.inf
    mass = torch.rand((B, ppsm), generator=g) * 5
    on = torch.rand((B, T), generator=g) < 0.6
    word = torch.from_numpy((on.numpy().astype(np.uint64) << np.arange(T, dtype=np.uint64)).sum(-1, dtype=np.uint64).view(np.int64))
    cache = handle(B, ppsm)
    for node_mask, marks in ((None, np.ones((B, T), bool)), (word, on.numpy())):
        for decay in (1.0, 0.9, 0.0):
            exp = page_mass(lse.numpy(), x.numpy(), mass.numpy(), np.float32(decay), marks)
            m = mass.cuda()
            out = torch.full_like(m, 9.0)
            args = (cache, lse.cuda(), x.cuda())
            nm = None if node_mask is None else node_mask.cuda()
            kvq.kvq_page_mass(*args, m, nm, decay, mass_out=out)
            assert torch.equal(m.cpu(), mass)
            bound = (2.0 ** -20 + (T * Hq + 2) * 2.0 ** -24) * np.abs(exp) + 1e-30
            assert (np.abs(out.cpu().numpy() - exp) <= bound).all()
            kvq.kvq_page_mass(*args, m, nm, decay)      # in place: the same bits
            assert torch.equal(m, out)


def rows(B, P, seed, kind="random"):
    g = np.random.default_rng(seed)
    table = np.stack([g.permutation(P) + b * P for b in range(B)]).astype(np.int32)
    mass = g.random((B, P)).astype(np.float32) ** 3
    if kind == "ties":
        mass = g.integers(0, 3, (B, P)).astype(np.float32)
    elif kind == "odd":
        mass[:, ::5] = np.nan
        mass[:, 1::7] = np.inf
        mass[:, 2::9] = -0.0
        mass[:, 3::11] = 0.0
        mass[:, 4::13] = -np.inf
        mass[:, 5::17] = 1e-42
    return table, mass


@pytest.mark.parametrize("kind", ["random", "ties", "odd"])
@pytest.mark.parametrize("fmt", [kvq.KVQ_FMT_FP4_E2M1_S16, kvq.KVQ_FMT_CB2_GROUP4], ids=["page", "group"])
@pytest.mark.parametrize("P", [16, 260, 2048, 5003])
def test_evict(kind, fmt, P):
    unit = 4 if fmt == kvq.KVQ_FMT_CB2_GROUP4 else 1
    lens = np.array([0, 1, 15, 16, 64, 16 * P, 16 * P - 5, 16 * (P // 2) + 3, 100], np.int32).clip(0, 16 * P)
    B = len(lens)
    table, mass = rows(B, P, P, kind)
    cache = handle(B, P, fmt)
    for keep, sink, recent in ((8, 0, 0), (8, 4, 4), (P // 2 // 4 * 4, 4, 8), (P // 4 * 4, 0, 0), (0, 0, 0), (12, 0, 4)):
        if sink + recent > keep:
            continue
        exp = evict(table, lens, mass, keep, sink, recent, unit)
        outs = [torch.full((B, P), -7, dtype=torch.int32, device="cuda"), torch.full((B,), -7, dtype=torch.int32, device="cuda"),
                torch.full((B, P), -7.0, device="cuda")]
        cache.page_table.copy_(torch.from_numpy(table))
        cache.seq_lens.copy_(torch.from_numpy(lens))
        m = torch.from_numpy(mass).cuda()
        n = kvq.kvq_evict_pages(cache, m, keep, sink, recent, *outs)
        for got, e in zip((*outs, n), exp):
            np.testing.assert_array_equal(got.cpu().numpy(), e)
        np.testing.assert_array_equal(cache.page_table.cpu().numpy(), table)
        n2 = kvq.kvq_evict_pages(cache, m, keep, sink, recent)   # in place
        for got, e in zip((cache.page_table, cache.seq_lens, m, n2), outs + [n]):
            np.testing.assert_array_equal(got.cpu().numpy(), e.cpu().numpy())


def test_evict_longest_row():
    P = 28672
    table, mass = rows(1, P, 1)
    lens = np.array([16 * P - 3], np.int32)
    cache = handle(1, P)
    cache.page_table.copy_(torch.from_numpy(table))
    cache.seq_lens.copy_(torch.from_numpy(lens))
    m = torch.from_numpy(mass).cuda()
    n = kvq.kvq_evict_pages(cache, m, 10000, 4, 64)
    exp = evict(table, lens, mass, 10000, 4, 64)
    for got, e in zip((cache.page_table, cache.seq_lens, m, n), exp):
        np.testing.assert_array_equal(got.cpu().numpy(), e)


@pytest.mark.parametrize("fmt", [kvq.KVQ_FMT_INT4_G32, kvq.KVQ_FMT_FP4_E2M1_S16, kvq.KVQ_FMT_CB2_OUTLIER, kvq.KVQ_FMT_TIERED,
                                 kvq.KVQ_FMT_CB2_GROUP4], ids=["int4", "e2m1", "cb2", "tiered", "cb2g"])
def test_serving_loop_on_a_fixed_page_budget(fmt):
    """Verify a drafted tree, append the accepted path, accumulate its page weights,
    evict: longer than the page table could hold without eviction.  Each step is
    checked against the 64-bit definitions on the values the cache then holds."""
    unit = 4 if fmt == kvq.KVQ_FMT_CB2_GROUP4 else 1
    B, Hkv, G, D, P, T = 2, 2, 4, 128, 14 if unit == 4 else 12, 6   # a group more than is kept fits
    tiers = np.zeros((B, P), bool)
    if fmt == kvq.KVQ_FMT_TIERED:
        tiers[:, 2::3] = True
    cache, total = Pair(fmt, B, Hkv, D, P, seed=5, tiers=tiers).gpu, 0
    k, v = make_kv(11, B, 400, Hkv, D, *(("student_t4", 0, 1.0) if fmt == kvq.KVQ_FMT_FP4_E2M1_S16 else ("normal", 4, 8.0)))
    kvq.kvq_quantize_append(cache, k[:, :70].contiguous().cuda(), v[:, :70].contiguous().cuda())
    at = 70
    mass = torch.zeros((B, P), device="cuda")
    g = torch.Generator().manual_seed(2)
    parents = np.array([[-1, 0, 1, 0, 2, 4]] * B)
    mask = kvq.tree_mask_from_parents(parents).cuda()
    accepted = [0, 1, 2, 4]
    marks = np.zeros((B, T), bool)
    marks[:, accepted] = True
    for step in range(40):
        lens = cache.seq_lens.cpu().numpy()
        n_max = int(lens.max())
        q = torch.randn((B, T, Hkv * G, D), generator=g).to(torch.bfloat16)
        kt, vt = [x[:, at:at + T].to(torch.bfloat16).contiguous() for x in (k, v)]
        lse = torch.empty((B, T, Hkv * G), device="cuda")
        page = torch.empty((B, T, Hkv * G, -(-n_max // 16)), device="cuda")
        kvq.kvq_tree_attention(cache, q.cuda(), D ** -0.5, n_max, kt.cuda(), vt.cuda(), mask, lse=lse, page_lse=page)
        held = types.SimpleNamespace(   # the cache as it is: what kvq_dequantize says
            Hkv=Hkv, seq_lens=lens,
            dequantize=lambda b, h, role, t0, t1: kvq.kvq_dequantize(cache, b, h, role, t0, t1).cpu().numpy())
        _, e_lse, e_page, _ = tree_rows(held, q.float().numpy(), D ** -0.5, kt.float().numpy(), vt.float().numpy(),
                                        sees_from_parents(parents))
        assert np.abs(lse.cpu().numpy() - e_lse).max() < 1e-4
        fin = np.isfinite(e_page)
        assert np.array_equal(fin, np.isfinite(page.cpu().numpy()))
        assert np.abs(page.cpu().numpy()[fin] - e_page[fin]).max() < 1e-4
        path = torch.tensor(accepted)
        kvq.kvq_quantize_append(cache, kt[:, path].contiguous().cuda(), vt[:, path].contiguous().cuda())
        before = mass.cpu().numpy()
        kvq.kvq_page_mass(cache, lse, page, mass, torch.full((B,), sum(1 << i for i in accepted), device="cuda"), 0.95)
        exp = page_mass(e_lse, e_page, before, np.float32(0.95), marks)
        assert np.abs(mass.cpu().numpy() - exp).max() < 1e-3
        old = (cache.page_table.cpu().numpy(), cache.seq_lens.cpu().numpy(), mass.cpu().numpy())
        n = kvq.kvq_evict_pages(cache, mass, 8 if unit == 4 else 6, unit, unit)
        e = evict(*old, 8 if unit == 4 else 6, unit, unit, unit)
        for got, x in zip((cache.page_table, cache.seq_lens, mass, n), e):
            np.testing.assert_array_equal(got.cpu().numpy(), x)
        total += int(n.sum())
        at += 6
    assert cache.status_word() == 0 and total >= 4


@pytest.mark.parametrize("fmt", range(7), ids=["int4", "e2m1", "cb2", "tiered", "cb2s", "a3", "cb2g"])
def test_recycled_pages_hold_what_fresh_ones_would(fmt):
    """Tokens appended into evicted blocks dequantize to what they would in zeroed ones."""
    B, Hkv, D, P = 1, 2, 128, 8
    sc = 2 if fmt == kvq.KVQ_FMT_CB2_STATIC else 0
    mk = lambda: kvq.QuantizedKVCache(fmt, B, Hkv, D, P, P, 1 if fmt == kvq.KVQ_FMT_TIERED else 0, static_channels=sc)
    used, fresh = mk(), mk()
    k, v = [x.cuda() for x in make_kv(3, B, 300, Hkv, D, "normal", 4, 8.0)]
    for c in (used, fresh):
        if sc:
            c.static_mask.copy_(torch.tensor([5, 77], dtype=torch.uint8, device="cuda"))
    kvq.kvq_quantize_append(used, k[:, :128].contiguous(), v[:, :128].contiguous())
    mass = torch.zeros((B, P), device="cuda")
    assert int(kvq.kvq_evict_pages(used, mass, 0)) == 8
    for t0, t1 in ((128, 157), (157, 200)):
        for c in (used, fresh):
            kvq.kvq_quantize_append(c, k[:, t0:t1].contiguous(), v[:, t0:t1].contiguous())
        n = t1 - 128
        q = torch.randn((B, 3, 8, D), device="cuda").to(torch.bfloat16)
        assert torch.equal(*[kvq.kvq_tree_attention(c, q, D ** -0.5, n) for c in (used, fresh)])
        for h in range(Hkv):
            for role in (0, 1):
                assert torch.equal(*[kvq.kvq_dequantize(c, 0, h, role, 0, n) for c in (used, fresh)])
