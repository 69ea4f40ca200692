"""Tree attention over FP8 tier pages whose V lies far outside fp16's range.

Error bounds (u = 2^-24, h = 2^-11, fp16's half step): a weight is off by
2E + 2^-20 relative and rounded to fp16 (h), a value of V times its page's scale
is rounded to fp16 once, relative to itself (h), so out is off by at most
2 (2E + 2^-20 + 2h) sum_j p_j |v_j|, E = scale (D + 4) 2u max_j sum_c |q_c k_jc|.
A weight is an fp16 number relative to the largest p_j s_j of the row's split (s_j the
page's power of two, or 1), which is stored as 2^6 at least: what it loses to
fp16's subnormals is at most 2^-25 / 2^6 = 2^-31 max_i(p_i s_i) |v_j| / s_j in O."""
import numpy as np
import pytest
import torch

from _kvq_pairs import Pair, make_kv
from _tree_reference import sees_from_parents, tree_rows, words
from sub_byte_quantized_kvq_gb300 import kvq

pytestmark = pytest.mark.gpu
TIERED = kvq.KVQ_FMT_TIERED
B, HKV, D, PAGES = 2, 2, 128, 16
LENS = [16 * 13 + 5, 16 * 9]


def pair_of(factor, tier, seed=3):
    """A cache whose page p is an FP8 page where tier[p], its V scaled by factor[p]."""
    pair = Pair(TIERED, B, HKV, D, PAGES, seed=seed, tiers=np.repeat(np.asarray(tier, bool)[None], B, 0), extra_pages=1)
    k, v = make_kv(seed + 4, B, 16 * PAGES, HKV, D, "normal", 4, 8.0)
    v = v * torch.tensor(factor, dtype=torch.float32).repeat_interleave(16)[None, :, None, None]
    pair.append(k, v, t_per_seq=LENS)
    return pair


def check(pair, q, k=None, v=None, sees=None, splits=(0, 1, 2)):
    f = lambda x: None if x is None else x.float().numpy()
    scale, L = D ** -0.5, max(LENS)
    e_out, e_lse, e_page, (reach, weight) = tree_rows(pair.ref, f(q), scale, f(k), f(v), sees, None, L)
    E = scale * (D + 4) * 2.0 ** -23 * reach
    b_out = 2 * (2 * E[..., None] + 2.0 ** -20 + 2.0 ** -10) * weight
    up = lambda x: None if x is None else torch.as_tensor(x).cuda().contiguous()
    for s in splits:
        lse = torch.empty(q.shape[:3], device="cuda")
        page = torch.empty((*q.shape[:3], -(-L // 16)), device="cuda")
        out = kvq.kvq_tree_attention(pair.gpu, up(q), scale, L, up(k), up(v), None if sees is None else up(words(sees)),
                                     num_splits=s, out_dtype=torch.float32, lse=lse, page_lse=page).cpu().numpy()
        assert np.isfinite(out).all()
        err = np.abs(out - e_out)
        assert (err <= b_out).all(), f"off by up to {(err / b_out).max():.3g} of the bound"
        assert (np.abs(lse.cpu().numpy() - e_lse) <= E + 2.0 ** -20 + 2.0 ** -22 * np.abs(e_lse)).all()
        g, fin = page.cpu().numpy(), np.isfinite(e_page)
        assert np.array_equal(np.isneginf(g), ~fin)
        assert (np.abs(g[fin] - e_page[fin]) <= (E[..., None] + 2.0 ** -20 + 2.0 ** -22 * np.abs(np.where(fin, e_page, 0)))[fin]).all()
    return e_out, weight


def queries(T, Hq, seed=1):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((B, T, Hq, D), generator=g).to(torch.bfloat16)
    k, v = [torch.randn((B, T, HKV, D), generator=g).to(torch.bfloat16) for _ in range(2)]
    parents = np.array([[-1 if t == 0 else int(torch.randint(-1, t, (1,), generator=g)) for t in range(T)] for _ in range(B)])
    return q, k, v, sees_from_parents(parents)


SHAPES = [(1, 2), (3, 16), (16, 16), (33, 16)]   # 1, 24, 128 and 264 rows a kv head


@pytest.mark.parametrize("factor", [1e9, 1e6, 300.0, 1e-2, 1e-4, 1e-6, 1e-8, 1e-12])
@pytest.mark.parametrize("T,Hq", SHAPES)
def test_tier_pages_of_any_magnitude(factor, T, Hq):
    """All pages FP8, every V of the same magnitude; with and without drafted tokens of ordinary size."""
    pair = pair_of([factor] * PAGES, [True] * PAGES)
    # the staged tail's V (fp32) are of that magnitude too
    q, k, v, sees = queries(T, Hq)
    e, _ = check(pair, q)
    assert np.abs(e).max() < 8 * 8 * factor    # (the case is what it says)
    check(pair, q, k, (v.float() * factor).to(torch.bfloat16), sees)


@pytest.mark.parametrize("factor", [1e6, 1e-6, 1e-8])
@pytest.mark.parametrize("T,Hq", SHAPES)
def test_tier_pages_beside_codebook_pages(factor, T, Hq):
    """FP8 pages of an odd magnitude between 2-bit pages of an ordinary one."""
    tier = [p % 3 == 1 for p in range(PAGES)]
    pair = pair_of([factor if t else 1.0 for t in tier], tier)
    q, k, v, sees = queries(T, Hq)
    check(pair, q)
    check(pair, q, k, v, sees)


@pytest.mark.parametrize("T,Hq", SHAPES)
def test_mixed_magnitudes(T, Hq):
    """Pages of very different magnitudes in one tile."""
    tier = [p % 4 != 0 for p in range(PAGES)]
    pair = pair_of([(1.0, 1e6, 1e-9, 1e-3)[p % 4] for p in range(PAGES)], tier)
    q, k, v, sees = queries(T, Hq)
    check(pair, q, splits=(1, 2))
    check(pair, q, k, v, sees, splits=(1, 2))


@pytest.mark.parametrize("T,Hq", SHAPES)
@pytest.mark.parametrize("small", [1e-6, 1e-9])
def test_a_row_that_looks_at_the_small_page(T, Hq, small):
    """The weight lies on an FP8 page of tiny V; a page of huge V, with a weight of about e^-60, does not hide it:
    what reaches the result is the small page's."""
    tier = [False, True, True] + [False] * (PAGES - 3)
    pair = Pair(TIERED, B, HKV, D, PAGES, seed=9, tiers=np.repeat(np.asarray(tier)[None], B, 0))
    g = torch.Generator().manual_seed(4)
    u = torch.randn((HKV, D), generator=g)
    u = u / u.norm(dim=-1, keepdim=True)
    height = torch.full((16 * PAGES,), -60.0)
    height[32:48] = 0.0                             # page 2: where the queries look
    k = height[None, :, None, None] * u + 0.02 * torch.randn((B, 16 * PAGES, HKV, D), generator=g)
    v = torch.randn((B, 16 * PAGES, HKV, D), generator=g)
    v[:, 16:32] *= 1e6
    v[:, 32:48] *= small
    pair.append(k, v, t_per_seq=LENS)
    q = (D ** 0.5 * u.repeat_interleave(Hq // HKV, 0))[None, None].repeat(B, T, 1, 1)
    e, _ = check(pair, q.to(torch.bfloat16))
    assert np.abs(e).max() < 8 * small


def test_one_node_is_decode_attention():
    """num_nodes = 1 over the cache alone, at every magnitude: both calls within their bounds of each other
    (decode keeps P and V as fp16 pairs: 2^-10 of sum_j p_j |v_j| covers it)."""
    for factor in (1e6, 1.0, 1e-6, 1e-8):
        pair = pair_of([factor] * PAGES, [True] * PAGES)
        q = queries(1, 16)[0]
        _, weight = check(pair, q)
        tree = kvq.kvq_tree_attention(pair.gpu, q.cuda(), D ** -0.5, max(LENS), out_dtype=torch.float32)[:, 0]
        dec = kvq.kvq_decode_attention(pair.gpu, q[:, 0].cuda().contiguous(), D ** -0.5, max(LENS), out_dtype=torch.float32)
        assert (np.abs((tree - dec).cpu().numpy()) <= 2.0 ** -8 * weight[:, 0]).all()
