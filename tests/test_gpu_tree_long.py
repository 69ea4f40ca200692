"""Tree attention over contexts of many tiles against the 64-bit definition: both
head dimensions, every format, splits long enough that each buffer, barrier
phase and tensor-memory column is used many times over.

Error bounds as in test_gpu_tree.py (u = 2^-24, h = 2^-11, fp16's half step):
  E = scale (D + 4) 2u max_j sum_c |q_c k_jc| for a score,
  out: 2 (2E + 2^-20 + 2h) sum_j p_j |v_j|, lse: E + 2^-20 + 2^-22 |lse|."""
import pytest
import torch

from sub_byte_quantized_kvq_gb300 import kvq

pytestmark = pytest.mark.gpu

FORMATS = dict(int4=kvq.KVQ_FMT_INT4_G32, e2m1=kvq.KVQ_FMT_FP4_E2M1_S16, cb2=kvq.KVQ_FMT_CB2_OUTLIER, tiered=kvq.KVQ_FMT_TIERED,
               cb2s=kvq.KVQ_FMT_CB2_STATIC, a3=kvq.KVQ_FMT_ASYM3_OUTLIER, cb2g=kvq.KVQ_FMT_CB2_GROUP4)


def filled(fmt, lens, Hkv, D, seed=1, change=None):
    """A cache of random tokens; every seventh page of a tiered one is an FP8 page.  change(k, v): edits of them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, L = len(lens), max(lens)
    P = -(-L // 16) + 3
    pt = torch.arange(B * P).view(B, P)
    tiers = torch.zeros((B, P), dtype=torch.bool)
    if fmt == kvq.KVQ_FMT_TIERED:
        tiers[:, ::7] = True
        pt = torch.where(tiers, (tiers.view(-1).cumsum(0) - 1).view(B, P) - (1 << 31), pt)
    cache = kvq.QuantizedKVCache(fmt, B, Hkv, D, P, B * P, int(tiers.sum()), page_table=pt,
                                 static_channels=2 if fmt == kvq.KVQ_FMT_CB2_STATIC else 0)
    k, v = [torch.randn((B, L, Hkv, D), generator=g, device="cuda") for _ in range(2)]
    if change:
        change(k, v)
    if fmt == kvq.KVQ_FMT_CB2_STATIC:
        kvq.kvq_select_static_channels(cache, k[0, :64].contiguous(), v[0, :64].contiguous())
    kvq.kvq_quantize_append(cache, k, v, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    return cache, g


def exact(cache, lens, q, scale):
    """(out, lse, sum_j p_j |v_j|, max_j sum_c |q_c k_jc|) in 64 bits, over the values that the cache holds."""
    B, T, Hq, D = q.shape
    Hkv = cache.cfg.num_kv_heads
    G = Hq // Hkv
    out, weight = [torch.zeros((B, T, Hq, D), dtype=torch.float64, device="cuda") for _ in range(2)]
    lse, reach = [torch.zeros((B, T, Hq), dtype=torch.float64, device="cuda") for _ in range(2)]
    for b, L in enumerate(lens):
        for h in range(Hkv):
            k, v = [kvq.kvq_dequantize(cache, b, h, r, 0, L).double() for r in (0, 1)]
            hs = slice(h * G, h * G + G)
            x = q[b, :, hs].double()
            a = scale * (x @ k.T)
            lse[b, :, hs] = torch.logsumexp(a, -1)
            p = torch.exp(a - lse[b, :, hs, None])
            out[b, :, hs], weight[b, :, hs] = p @ v, p @ v.abs()
            reach[b, :, hs] = (x.abs() @ k.abs().T).amax(-1)
    return out, lse, weight, reach


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("name", list(FORMATS))
def test_many_tiles(name, D):
    """Odd lengths, 47 tiles (94 of INT4) a split at the longest; few rows, a tile of them, more than one."""
    lens, Hkv = [6007, 2500], 2
    cache, g = filled(FORMATS[name], lens, Hkv, D)
    scale = D ** -0.5
    for T, Hq in ((1, 2), (3, 16), (16, 16), (40, 16)):
        q = (2 * torch.randn((2, T, Hq, D), generator=g, device="cuda")).to(torch.bfloat16)
        e_out, e_lse, weight, reach = exact(cache, lens, q, scale)
        E = scale * (D + 4) * 2.0 ** -23 * reach
        for splits in (1, 2, 0):
            lse = torch.empty((2, T, Hq), device="cuda")
            out = kvq.kvq_tree_attention(cache, q, scale, max(lens), num_splits=splits, out_dtype=torch.float32, lse=lse)
            assert ((out - e_out).abs() <= 2 * (2 * E[..., None] + 2.0 ** -20 + 2.0 ** -10) * weight).all()
            assert ((lse - e_lse).abs() <= E + 2.0 ** -20 + 2.0 ** -22 * e_lse.abs()).all()
    assert cache.status_word() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("name", list(FORMATS))
def test_scores_that_jump_between_the_chunks_of_a_tile(name, D):
    """Each run of 64 tokens scores far above the one before, for every second node: the maximum rises between the chunks of
    a tile, whose earlier weights are then scaled where they lie, by 1 for the nodes that do not jump."""
    lens, Hkv, scale = [7 * 64 + 50, 300], 2, D ** -0.5
    def change(k, v):
        run = torch.arange(k.shape[1], device="cuda") // 64
        k[..., 0] = (12.0 * 2.0 ** run)[None, :, None]
    cache, g = filled(FORMATS[name], lens, Hkv, D, seed=3, change=change)
    for T, Hq in ((3, 16), (16, 16), (33, 16)):
        q = (2 * torch.randn((2, T, Hq, D), generator=g, device="cuda")).to(torch.bfloat16)
        q[..., 0] = 0
        q[:, ::2, :, 0] = 1 / scale
        e_out, e_lse, weight, reach = exact(cache, lens, q, scale)
        E = scale * (D + 4) * 2.0 ** -23 * reach
        for splits in (1, 0):
            lse = torch.empty((2, T, Hq), device="cuda")
            out = kvq.kvq_tree_attention(cache, q, scale, max(lens), num_splits=splits, out_dtype=torch.float32, lse=lse)
            assert ((out - e_out).abs() <= 2 * (2 * E[..., None] + 2.0 ** -20 + 2.0 ** -10) * weight).all()
            assert ((lse - e_lse).abs() <= E + 2.0 ** -20 + 2.0 ** -22 * e_lse.abs()).all()
    assert cache.status_word() == 0
