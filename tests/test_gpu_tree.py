"""Tree attention over the quantized cache against the 64-bit definition.

Error bounds (u = 2^-24, fp32's half step; h = 2^-11, fp16's):
  scores: K and V of a block are exact in the tensor cores' fp16 operands (INT4:
    K as an fp16 pair, 2^-22; V as one fp16, h) and the query is exact, so a
    score of D products accumulated in fp32 is off by at most
    E = scale * (D + 4) * 2u * max_j sum_c |q_c k_jc|   (2u: a truncating add);
  lse, page_lse: E, plus 2^-20 for the exponentials (ex2.approx: 2 ulp), their
    fp32 sums and the logarithm, plus the rounding of the result;
  out: each weight is off by 2E + 2^-20 relative and is rounded to fp16 for the
    tensor cores (h), V by at most h: (2E + 2^-20 + 2h) sum_j p_j |v_j|, twice
    where the normaliser counts too, plus the output's own rounding."""
import numpy as np
import pytest
import torch

from _kvq_pairs import Pair, make_kv
from _tree_reference import sees_from_parents, tree_rows, words
from sub_byte_quantized_kvq_gb300 import kvq

pytestmark = pytest.mark.gpu

INT4, E2M1, CB2, TIERED = (kvq.KVQ_FMT_INT4_G32, kvq.KVQ_FMT_FP4_E2M1_S16, kvq.KVQ_FMT_CB2_OUTLIER,
                           kvq.KVQ_FMT_TIERED)
CB2S, A3, CB2G = kvq.KVQ_FMT_CB2_STATIC, kvq.KVQ_FMT_ASYM3_OUTLIER, kvq.KVQ_FMT_CB2_GROUP4
NAMES = ["int4", "e2m1", "cb2", "tiered", "cb2s", "a3", "cb2g"]
ALL = [INT4, E2M1, CB2, TIERED, CB2S, A3, CB2G]


def build(fmt, D, lens, Hkv=2, P=16, seed=3, dist=None):
    B = len(lens)
    tiers = np.zeros((B, P), bool)
    if fmt == TIERED:
        tiers[:, 1::3] = True
    pair = Pair(fmt, B, Hkv, D, P, seed=seed, tiers=tiers)
    k, v = make_kv(seed + 4, B, max(max(lens), 1), Hkv, D, *(dist or (("student_t4", 0, 1.0) if fmt == E2M1 else ("normal", 4, 8.0))))
    pair.append(k, v, t_per_seq=lens)
    return pair


def draft(seed, B, T, Hkv, Hq, D, loud=1.0):
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn((B, T, Hq, D), generator=g) * loud).to(torch.bfloat16)
    k, v = [torch.randn((B, T, Hkv, D), generator=g).to(torch.bfloat16) for _ in range(2)]
    parents = np.array([[int(torch.randint(-1, t, (1,), generator=g)) if t else -1 for t in range(T)] for _ in range(B)])
    return q, k, v, parents


def bounds(exp, slack, scale, D):
    out, lse, page, (reach, weight) = exp[0], exp[1], exp[2], slack
    E = scale * (D + 4) * 2.0 ** -23 * reach
    b_lse = E + 2.0 ** -20 + 2.0 ** -22 * np.abs(np.where(np.isinf(lse), 0, lse))
    b_page = E[..., None] + 2.0 ** -20 + 2.0 ** -22 * np.abs(np.where(np.isinf(page), 0, page))
    b_out = 2 * (2 * E[..., None] + 2.0 ** -20 + 2.0 ** -10) * weight
    return b_out, b_lse, b_page


def run(pair, q, k=None, v=None, mask=None, nodes=None, splits=0, out_dtype=torch.float32, max_len=None, **kw):
    dev = "cuda"
    B, T, Hq, D = q.shape
    max_len = int(pair.ref.seq_lens.max()) if max_len is None else max_len
    lse = torch.full((B, T, Hq), 77.0, device=dev)
    page = torch.full((B, T, Hq, -(-min(max_len, 16 * pair.P) // 16)), 77.0, device=dev)
    up = lambda x: None if x is None else torch.as_tensor(x).to(dev).contiguous()
    out = kvq.kvq_tree_attention(pair.gpu, up(q), D ** -0.5, max_len, k_tree=up(k), v_tree=up(v), tree_mask=up(mask),
                                 nodes_per_seq=None if nodes is None else torch.tensor(nodes, dtype=torch.int32, device=dev),
                                 num_splits=splits, out_dtype=out_dtype, lse=lse, page_lse=page, **kw)
    torch.cuda.synchronize()
    return out.float().cpu().numpy(), lse.cpu().numpy().astype(np.float64), page.cpu().numpy().astype(np.float64)


def check(got, pair, q, k=None, v=None, sees=None, nodes=None, max_len=None, out_dtype=torch.float32):
    D = q.shape[-1]
    f = lambda x: None if x is None else x.float().numpy()
    out, lse, page, slack = tree_rows(pair.ref, f(q), D ** -0.5, f(k), f(v), sees, nodes, max_len)
    b_out, b_lse, b_page = bounds((out, lse, page), slack, D ** -0.5, D)
    if out_dtype == torch.bfloat16:
        b_out = b_out + 2.0 ** -8 * np.abs(out)
    for name, g, e, b in (("out", got[0], out, b_out), ("lse", got[1], lse, b_lse), ("page_lse", got[2], page, b_page)):
        assert np.array_equal(np.isneginf(g), np.isneginf(e)), name
        fin = np.isfinite(e)
        err = np.abs(g[fin] - e[fin])
        assert np.isfinite(g[fin]).all() and (err <= b[fin]).all(), (
            f"{name}: off by up to {err.max():.3e}, {(err / np.maximum(b[fin], 1e-30)).max():.2f} of the bound")


@pytest.mark.parametrize("fmt", ALL, ids=NAMES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,T", [(1, 1), (4, 5), (8, 3), (3, 7), (16, 9), (8, 33)])
def test_tree_parity(fmt, D, G, T):
    """Ragged lengths (whole pages, partial pages, one token, none), random trees,
    one split and the library's choice, both output types."""
    pair = build(fmt, D, [209, 77, 1, 0, 128])
    Hq = 2 * G
    q, k, v, parents = draft(G * 100 + T, 5, T, 2, Hq, D)
    sees = sees_from_parents(parents)
    for splits, od in ((0, torch.bfloat16), (1, torch.float32), (3, torch.float32)):
        got = run(pair, q, k, v, words(sees), splits=splits, out_dtype=od)
        check(got, pair, q, k, v, sees, out_dtype=od)
    assert pair.gpu.status_word() == 0


@pytest.mark.parametrize("fmt", ALL, ids=NAMES)
def test_queries_over_the_cache_alone(fmt):
    """No tree: T independent queries; one of them is decode attention."""
    pair = build(fmt, 128, [209, 77, 1])
    for T in (1, 4):
        q, _, _, _ = draft(5 + T, 3, T, 2, 16, 128)
        got = run(pair, q)
        check(got, pair, q)
    q1 = draft(6, 3, 1, 2, 16, 128)[0]
    dec = kvq.kvq_decode_attention(pair.gpu, q1[:, 0].cuda().contiguous(), 128 ** -0.5, 209, out_dtype=torch.float32)
    _, _, _, (_, weight) = tree_rows(pair.ref, q1.float().numpy(), 128 ** -0.5)
    assert (np.abs(run(pair, q1)[0][:, 0] - dec.cpu().numpy()) <= 2.0 ** -9 * weight[:, 0] + 2e-3).all()


@pytest.mark.parametrize("T", [1, 2, 16, 17, 63, 64])
def test_chain_and_shared_tree(T):
    """No mask is a chain; one tree for every sequence; the last bit of the word."""
    pair = build(E2M1, 128, [130, 40])
    q, k, v, parents = draft(T, 2, T, 2, 4, 128)
    check(run(pair, q, k, v), pair, q, k, v)
    sees = sees_from_parents(np.repeat(parents[:1], 2, 0))
    got = run(pair, q, k, v, words(sees[0]))
    check(got, pair, q, k, v, sees)
    np.testing.assert_array_equal(kvq.tree_mask_from_parents(parents).numpy(), words(sees_from_parents(parents)))


def test_rows_that_attend_to_nothing():
    """Empty cache and an empty word: 0 and -inf; a word without the node itself is taken as it is."""
    pair = build(CB2, 128, [0, 33])
    q, k, v, _ = draft(3, 2, 6, 2, 8, 128)
    sees = np.zeros((2, 6, 6), bool)
    sees[:, 1, 0] = sees[:, 2, 5] = True
    got = run(pair, q, k, v, words(sees))
    check(got, pair, q, k, v, sees)
    assert (got[0][0, 0] == 0).all() and np.isneginf(got[1][0, 0]).all()


@pytest.mark.parametrize("fmt", [INT4, CB2], ids=["int4", "cb2"])
def test_what_is_masked_never_arrives(fmt):
    """NaN and infinities in nodes a row does not see, in nodes past the count and in
    their queries; rows past the count are empty rows."""
    pair = build(fmt, 128, [100, 50, 64])
    T = 20
    q, k, v, parents = draft(9, 3, T, 2, 8, 128)
    parents[:, 5] = -1
    parents[:, 6:][parents[:, 6:] == 5] = 4
    sees = sees_from_parents(parents)
    nodes = [20, 13, 0]
    clean = run(pair, q, k, v, words(sees), nodes)
    check(clean, pair, q, k, v, sees, nodes)
    k2, v2, q2 = k.clone(), v.clone(), q.clone()
    k2[:, 5], v2[:, 5] = float("nan"), float("inf")     # node 5: only itself sees it
    for b in (1, 2):
        k2[b, nodes[b]:], v2[b, nodes[b]:], q2[b, nodes[b]:] = float("inf"), float("nan"), float("nan")
    wide = sees.copy()
    wide[1, :, 13:] = True                              # bits past the count are ignored
    got = run(pair, q2, k2, v2, words(wide), nodes)
    keep = np.arange(T) != 5
    for a, e in zip(got, clean):
        np.testing.assert_array_equal(a[:, keep], e[:, keep])
    for b in (1, 2):
        assert (got[0][b, nodes[b]:] == 0).all()
        assert np.isneginf(got[1][b, nodes[b]:]).all() and np.isneginf(got[2][b, nodes[b]:]).all()


def test_loud_and_quiet_queries():
    """Queries far outside fp16's range (each row is scaled by a power of two), one
    page that holds nearly all the weight: the others' page_lse stay finite."""
    pair = build(CB2, 128, [200, 90], dist=("normal", 4, 8.0))
    for loud in (1e5, 1e-6, 30.0):
        q, k, v, parents = draft(4, 2, 5, 2, 8, 128, loud)
        sees = sees_from_parents(parents)
        got = run(pair, q, k, v, words(sees))
        check(got, pair, q, k, v, sees)
        assert np.isfinite(got[2][0]).all()


@pytest.mark.parametrize("G,T", [(4, 2), (8, 8), (8, 16)])
def test_running_maximum_rises_all_along(G, T):
    """Scores that climb by about 40 (natural units) over the context in uneven steps, some rows down instead:
    the state is rescaled many times, early pages end up far below the maximum, late ones in the other rows."""
    L, Hkv, D = 900, 2, 128
    pair = Pair(E2M1, 1, Hkv, D, 64, seed=2)
    g = torch.Generator().manual_seed(5)
    u = torch.randn((Hkv, D), generator=g)
    u = u / u.norm(dim=-1, keepdim=True)
    height = 40.0 * torch.cumsum(torch.rand(L, generator=g) ** 6, 0) / torch.cumsum(torch.rand(L, generator=g) ** 6, 0)[-1]
    k = (height[:, None, None] * u)[None] + 0.05 * torch.randn((1, L, Hkv, D), generator=g)
    v = torch.randn((1, L, Hkv, D), generator=g)
    pair.append(k, v)
    q = (D ** 0.5 * u.repeat_interleave(G, 0))[None, None].repeat(1, T, 1, 1)
    q[:, ::2] *= -1.0
    q = (q + 0.1 * torch.randn(q.shape, generator=g)).to(torch.bfloat16)
    for splits in (1, 0, 3):
        got = run(pair, q, splits=splits)
        check(got, pair, q)


def test_more_queries_than_a_tile_and_many_splits():
    pair = build(E2M1, 128, [700, 333], Hkv=1, P=48)
    q, k, v, parents = draft(21, 2, 64, 1, 16, 128)
    sees = sees_from_parents(parents)
    nodes = [64, 41]
    for splits in (0, 1, 7, 44, 60):
        got = run(pair, q, k, v, words(sees), nodes, splits=splits)
        check(got, pair, q, k, v, sees, nodes)


@pytest.mark.parametrize("fmt", [E2M1, CB2, CB2G], ids=["e2m1", "cb2", "cb2g"])
def test_shorter_bound_than_the_sequences(fmt):
    """Tokens past max_seq_len are left out and flagged, also inside a block."""
    pair = build(fmt, 128, [209, 64, 30])
    q, k, v, parents = draft(2, 3, 4, 2, 8, 128)
    got = run(pair, q, k, v, max_len=70)
    check(got, pair, q, k, v, max_len=70)
    assert pair.gpu.status_word() == kvq.KVQ_STATUS_SEQ_TOO_LONG
    got = run(pair, q, k, v, max_len=0)
    check(got, pair, q, k, v, max_len=0)


@pytest.mark.parametrize("fmt", [E2M1, CB2, CB2G, TIERED], ids=["e2m1", "cb2", "cb2g", "tiered"])
def test_bad_page_table_entries(fmt):
    """An entry outside its pool is flagged and its page (group) left out; the other sequences are whole."""
    pair = build(fmt, 64, [150, 209, 40])
    q, k, v, parents = draft(8, 3, 3, 2, 8, 64)
    sees = sees_from_parents(parents)
    good = run(pair, q, k, v, words(sees))
    for entry in (1 << 20, -1, -(1 << 31) + (1 << 20)):
        pair.gpu.page_table[1, 5] = entry
        pair.gpu.status.zero_()
        got = run(pair, q, k, v, words(sees))
        assert pair.gpu.status_word() == kvq.KVQ_STATUS_BAD_PAGE
        for a, e in zip(got, good):
            np.testing.assert_array_equal(a[[0, 2]], e[[0, 2]])
        left_out = range(4, 8) if fmt == CB2G else [5]
        others = [p for p in range(14) if p not in left_out]
        assert np.isneginf(got[2][1][..., list(left_out)]).all()
        assert np.abs(got[2][1][..., others] - good[2][1][..., others]).max() < 1e-4
        w = np.concatenate([good[2][1][..., list(left_out)]], -1)
        exp = np.log(np.exp(good[1][1]) - np.exp(w).sum(-1))
        assert np.abs(got[1][1] - exp).max() < 1e-3


def test_blocks_past_four_gigabytes():
    """Physical pages whose byte offset passes 32 bits."""
    D, Hkv, L = 128, 8, 100
    n = (1 << 32) // (2 * Hkv * 1152) + 64
    g = torch.Generator().manual_seed(0)
    pt = (torch.arange(2 * 8, dtype=torch.int64).view(2, 8) + n - 20).to(torch.int32)
    cache = kvq.QuantizedKVCache(E2M1, 2, Hkv, D, 8, n, page_table=pt)
    small = kvq.QuantizedKVCache(E2M1, 2, Hkv, D, 8, 16)
    k, v = [torch.randn((2, L, Hkv, D), generator=g).cuda() for _ in range(2)]
    q, kt, vt, _ = draft(1, 2, 6, Hkv, 32, D)
    outs = []
    for c in (cache, small):
        kvq.kvq_quantize_append(c, k, v)
        outs.append(kvq.kvq_tree_attention(c, q.cuda(), D ** -0.5, L, kt.cuda(), vt.cuda(), out_dtype=torch.float32))
    assert torch.equal(*outs)


def test_streams_graphs_and_workspaces():
    """The same call on another stream, captured and replayed after its inputs
    changed, and two graphs with a workspace each replayed at once."""
    pair = build(CB2, 128, [209, 77])
    Hq, T = 8, 6
    qs = [draft(s, 2, T, 2, Hq, 128) for s in (1, 2)]
    args = [[x.cuda() for x in d[:3]] for d in qs]
    want = [kvq.kvq_tree_attention(pair.gpu, *[a[0]], 128 ** -0.5, 209, a[1], a[2]) for a in args]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = kvq.kvq_tree_attention(pair.gpu, args[0][0], 128 ** -0.5, 209, args[0][1], args[0][2], stream=side)
    side.synchronize()
    assert torch.equal(got, want[0])
    graphs, outs, ins = [], [], []
    for i in range(2):
        x = [t.clone() for t in args[i]]
        o = torch.zeros_like(x[0])
        ws = kvq.alloc_tree_workspace(pair.gpu, Hq, T, 209)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kvq.kvq_tree_attention(pair.gpu, x[0], 128 ** -0.5, 209, x[1], x[2], out=o, workspace=ws)
        graphs.append((g, ws)), outs.append(o), ins.append(x)
    for swap in (0, 1):
        for i in range(2):
            for t, s in zip(ins[i], args[i ^ swap]):
                t.copy_(s)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i][0].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(outs[i], want[i ^ swap])


def test_from_buffers_reads_the_same_cache():
    for fmt in (INT4, TIERED, CB2S, CB2G):
        pair = build(fmt, 128, [209, 77])
        c = pair.gpu
        same = kvq.QuantizedKVCache.from_buffers(fmt, 2, 128, c.pool, c.page_table, c.seq_lens, c.status, c.staging, c.tier_pool,
                                                 c.static_mask)
        assert (same.cfg.num_pages, same.cfg.num_tier_pages) == (c.cfg.num_pages, c.cfg.num_tier_pages)
        q, k, v, _ = [x.cuda() if isinstance(x, torch.Tensor) else x for x in draft(1, 2, 4, 2, 8, 128)]
        assert torch.equal(*[kvq.kvq_tree_attention(x, q, 128 ** -0.5, 209, k, v) for x in (c, same)])


def test_first_call_after_another_format():
    """What an earlier kernel left in shared or tensor memory never shows: each format's
    first call after another's gives the bits of its later ones."""
    q, k, v, _ = [x.cuda() if isinstance(x, torch.Tensor) else x for x in draft(1, 2, 4, 2, 8, 128)]
    pairs = [build(fmt, 128, [209, 77]) for fmt in ALL]
    big = build(E2M1, 128, [250, 250], dist=("student_t4", 0, 1.0))
    for pair in pairs:
        for splits in (0, 1):
            kvq.kvq_tree_attention(big.gpu, q * 3, 0.3, 250, v, k, num_splits=1)
            outs = [kvq.kvq_tree_attention(pair.gpu, q, 128 ** -0.5, 209, k, v, num_splits=splits) for _ in range(3)]
            assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("fmt", ALL, ids=NAMES)
def test_no_wait_gives_up_over_many_tiles(fmt):
    """Long splits of every format, few and many rows, repeated: no wait times out and
    every call gives the same bits."""
    D, Hkv, L = 128, 2, 6000
    g = torch.Generator(device="cuda").manual_seed(1)
    P = L // 16 + 1
    pt = torch.arange(2 * P).view(2, P)
    tiers = torch.zeros((2, P), dtype=torch.bool)
    if fmt == TIERED:
        tiers[:, ::7] = True
        pt = torch.where(tiers, (tiers.view(-1).cumsum(0) - 1).view(2, P) - (1 << 31), pt)
    cache = kvq.QuantizedKVCache(fmt, 2, Hkv, D, P, 2 * P, int(tiers.sum()), page_table=pt, static_channels=2 if fmt == CB2S else 0)
    k, v = [torch.randn((2, L, Hkv, D), generator=g, device="cuda") for _ in range(2)]
    if fmt == CB2S:
        kvq.kvq_select_static_channels(cache, k[0, :64].contiguous(), v[0, :64].contiguous())
    kvq.kvq_quantize_append(cache, k, v)
    for T, Hq in ((1, 2), (3, 16), (16, 16), (40, 16)):
        q = torch.randn((2, T, Hq, D), generator=g, device="cuda").to(torch.bfloat16)
        ws = kvq.alloc_tree_workspace(cache, Hq, T, L, 3)
        first = kvq.kvq_tree_attention(cache, q, D ** -0.5, L, num_splits=1, workspace=ws)
        for splits in (1, 1, 1, 2, 3):
            out = kvq.kvq_tree_attention(cache, q, D ** -0.5, L, num_splits=splits, workspace=ws)
            if splits == 1:
                assert torch.equal(out, first)
    assert cache.status_word() == 0


@pytest.mark.parametrize("fmt", [INT4, CB2, E2M1], ids=["int4", "cb2", "e2m1"])
@pytest.mark.parametrize("G,T", [(4, 8), (4, 9), (8, 8), (8, 9), (8, 16), (8, 17)])
def test_row_counts_at_the_kernels_borders(fmt, G, T):
    """32, 36, 64, 72, 128 and 136 rows, and fewer live ones in some sequences."""
    pair = build(fmt, 128, [180, 209, 77, 50])
    q, k, v, parents = draft(G + T, 4, T, 2, 2 * G, 128)
    sees = sees_from_parents(parents)
    for nodes in (None, [T, T // 2, 1, T - 1]):
        check(run(pair, q, k, v, words(sees), nodes, splits=1), pair, q, k, v, sees, nodes)


@pytest.mark.parametrize("fmt", [E2M1, CB2], ids=["e2m1", "cb2"])
def test_a_nan_query_stays_in_its_row(fmt):
    """A NaN query gives NaN (not an empty row) in its own row, over the cache and over the tree; no other row changes."""
    pair = build(fmt, 128, [209, 0])
    T = 6
    q, k, v, _ = draft(14, 2, T, 2, 8, 128)
    bad = q.clone()
    bad[:, 2, 3, 7] = bad[:, 4, 0] = float("nan")
    keep = np.ones((2, T, 8), bool)
    keep[:, 2, 3] = keep[:, 4, 0] = False
    for tree in ((k, v), (None, None)):
        clean, got = run(pair, q, *tree), run(pair, bad, *tree)
        live = [0, 1] if tree[0] is not None else [0]
        for a, e in zip(got, clean):
            np.testing.assert_array_equal(a[keep], e[keep])
            for b in live:
                assert np.isnan(a[b, 2, 3][~np.isneginf(e[b, 2, 3])]).all() and np.isnan(a[b, 4, 0][~np.isneginf(e[b, 4, 0])]).all()


@pytest.mark.parametrize("G,T", [(4, 2), (8, 16)])
def test_zero_keys_in_a_cut_fp8_page(G, T):
    """A tier page of zeros has scale 0; the bound on the length ends inside it: uniform weights over what is visible."""
    pair = Pair(TIERED, 2, 2, 128, 8, seed=3, tiers=np.array([[False, True, False, False] * 2] * 2))
    k, v = make_kv(5, 2, 64, 2, 128, "normal", 4, 8.0)
    pair.append(torch.zeros_like(k), v)
    q, kt, vt, _ = draft(2, 2, T, 2, 2 * G, 128)
    for max_len in (24, 17, 64):
        got = run(pair, q, max_len=max_len)
        check(got, pair, q, max_len=max_len)


@pytest.mark.parametrize("scale", [0.0, -0.125, 1e-30])
def test_scales_that_are_not_positive(scale):
    for fmt in (INT4, TIERED):
        pair = build(fmt, 128, [209, 40])
        q, k, v, parents = draft(31, 2, 5, 2, 8, 128)
        sees = sees_from_parents(parents)
        lse = torch.empty((2, 5, 8), device="cuda")
        out = kvq.kvq_tree_attention(pair.gpu, q.cuda(), scale, 209, k.cuda(), v.cuda(), torch.from_numpy(words(sees)).cuda(),
                                     out_dtype=torch.float32, lse=lse)
        f = lambda x: x.float().numpy()
        e_out, e_lse, e_page, slack = tree_rows(pair.ref, f(q), scale, f(k), f(v), sees, None, 209)
        b_out, b_lse, _ = bounds((e_out, e_lse, e_page), slack, abs(scale), 128)
        assert (np.abs(out.cpu().numpy() - e_out) <= b_out).all()
        assert (np.abs(lse.cpu().numpy() - e_lse) <= b_lse).all()
