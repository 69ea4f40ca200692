"""What kvq_tree_attention, kvq_page_mass and kvq_evict_pages refuse, before any
buffer is touched (the pointers are never read: no GPU is needed)."""
import ctypes
import os
import shutil

import numpy as np
import pytest
import torch

from _tree_reference import sees_from_parents, words

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="nvcc not available")


@pytest.fixture(scope="module")
def kvq():
    from sub_byte_quantized_kvq_gb300 import build
    build.build()
    from sub_byte_quantized_kvq_gb300 import kvq as mod
    return mod


FAKE = 1 << 20   # 16-byte aligned, never read


def cfg_of(kvq, fmt=1, D=128, **kw):
    c = kvq.kvq_config(4, 8, D, 16, 64, 0, fmt, 16, 3.0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def cache_of(kvq, **kw):
    p = dict(pool=FAKE, tier_pool=None, page_table=FAKE, seq_lens=FAKE, staging=None, status=FAKE, static_mask=None)
    p.update(kw)
    return kvq.kvq_cache(*[p[f] for f, _ in kvq.kvq_cache._fields_])


def tree(kvq, cfg, cache, q=FAKE, Hq=32, T=4, k=FAKE, v=FAKE, mask=None, per_seq=0, nodes=None, scale=0.1, max_len=100, splits=2,
         out=FAKE, od=0, ws=FAKE, nbytes=0):
    return kvq.lib().kvq_tree_attention(ctypes.byref(cfg), ctypes.byref(cache), q, Hq, T, k, v, mask, per_seq, nodes,
                                        ctypes.c_float(scale), max_len, splits, out, od, None, None, ws, nbytes, None)


def test_tree_attention_refusals(kvq):
    INVALID, UNSUPPORTED, WORKSPACE, CAPACITY = (kvq.KVQ_ERR_INVALID_ARG, kvq.KVQ_ERR_UNSUPPORTED, kvq.KVQ_ERR_WORKSPACE,
                                                 kvq.KVQ_ERR_CAPACITY)
    c, k = cfg_of(kvq), cache_of(kvq)
    assert tree(kvq, c, k) == WORKSPACE                 # all else is right
    for bad in (dict(q=None), dict(q=FAKE + 2), dict(out=None), dict(out=FAKE + 4), dict(od=kvq.KVQ_F16), dict(ws=None), dict(ws=FAKE + 8),
                dict(k=None), dict(v=None), dict(k=FAKE + 4), dict(k=None, v=None, mask=FAKE), dict(per_seq=2), dict(Hq=0),
                dict(Hq=30), dict(T=0), dict(max_len=-1), dict(splits=-1), dict(scale=float("inf")),
                dict(scale=float("nan"))):
        assert tree(kvq, c, k, **bad) == INVALID, bad
    assert tree(kvq, c, k, T=65) == UNSUPPORTED
    assert tree(kvq, c, k, Hq=8 * 17) == UNSUPPORTED
    assert tree(kvq, cfg_of(kvq, D=96), k) == UNSUPPORTED
    assert tree(kvq, cfg_of(kvq, num_kv_heads=10000), k, Hq=160000, T=64) == UNSUPPORTED   # 80,000 row tiles in the grid
    assert tree(kvq, c, k, splits=257) == CAPACITY
    assert tree(kvq, cfg_of(kvq, 2), k) == INVALID      # a page format without staging
    assert tree(kvq, c, cache_of(kvq, page_table=None)) == INVALID
    n = ctypes.c_size_t()
    L = kvq.lib()
    assert L.kvq_tree_workspace_bytes(ctypes.byref(c), 32, 4, 100, 3, ctypes.byref(n)) == kvq.KVQ_OK
    assert n.value >= 4 * 32 * 4 * 3 * (128 * 4 + 8)    # rows x splits x (o, m, l)
    assert tree(kvq, c, k, splits=3, nbytes=n.value - 1) == WORKSPACE
    assert L.kvq_tree_workspace_bytes(ctypes.byref(c), 32, 4, 100, 3, None) == INVALID
    assert L.kvq_tree_workspace_bytes(ctypes.byref(c), 32, 65, 100, 3, ctypes.byref(n)) == UNSUPPORTED


def test_page_mass_refusals(kvq):
    c = cfg_of(kvq)

    def mass(Hq=32, T=4, P=16, lse=FAKE, page=FAKE, decay=1.0, src=FAKE, dst=FAKE, cfg=c):
        return kvq.lib().kvq_page_mass(ctypes.byref(cfg), Hq, T, P, lse, page, None, ctypes.c_float(decay), src, dst, None)
    for bad in (dict(lse=None), dict(page=None), dict(src=None), dict(dst=None), dict(P=17), dict(P=-1), dict(decay=float("nan")),
                dict(T=0), dict(Hq=31)):
        assert mass(**bad) == kvq.KVQ_ERR_INVALID_ARG, bad
    assert mass(T=65) == kvq.KVQ_ERR_UNSUPPORTED


def test_evict_refusals(kvq):
    def evict(cfg, keep=8, sink=0, recent=0, mass=FAKE, table=FAKE, lens=FAKE, out=FAKE, cache=None):
        return kvq.lib().kvq_evict_pages(ctypes.byref(cfg), ctypes.byref(cache or cache_of(kvq, staging=FAKE)), mass, keep, sink, recent,
                                         table, lens, out, None, None)
    c = cfg_of(kvq)
    for bad in (dict(mass=None), dict(table=None), dict(lens=None), dict(out=None), dict(sink=-1), dict(recent=-1), dict(keep=-1),
                dict(keep=5, sink=3, recent=3), dict(keep=8, sink=2 ** 31 - 1, recent=2 ** 31 - 1)):
        assert evict(c, **bad) == kvq.KVQ_ERR_INVALID_ARG, bad
    g = cfg_of(kvq, 6)
    for bad in (dict(keep=6), dict(sink=2), dict(recent=1)):
        assert evict(g, **bad) == kvq.KVQ_ERR_INVALID_ARG, bad
    assert evict(cfg_of(kvq, pages_per_seq_max=28673)) == kvq.KVQ_ERR_UNSUPPORTED


def test_mask_from_parents(kvq):
    rng = np.random.default_rng(1)
    for T in (1, 2, 63, 64):
        parents = np.array([[-1 if t == 0 else int(rng.integers(-1, t)) for t in range(T)] for _ in range(3)])
        np.testing.assert_array_equal(kvq.tree_mask_from_parents(parents).numpy(), words(sees_from_parents(parents)))
    for bad in ([0], [-1, 1], [-2], [-1] * 65):
        with pytest.raises(ValueError):
            kvq.tree_mask_from_parents(torch.tensor(bad))


def test_tensors_of_another_device_are_refused(kvq):
    """A host tensor never reaches the library."""
    with pytest.raises(ValueError):
        kvq._check_on(0, None, torch.zeros(1))
    with pytest.raises(ValueError):
        kvq._check_on(-1, torch.zeros(1))   # a cache that lies on the host
