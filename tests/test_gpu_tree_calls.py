"""What surrounds a tree attention call: one workspace for calls of several
shapes, and tensors made for a call on another stream."""
import numpy as np
import pytest
import torch

from sub_byte_quantized_kvq_gb300 import kvq

pytestmark = pytest.mark.gpu
E2M1 = kvq.KVQ_FMT_FP4_E2M1_S16


def empty_cache(B, Hkv, L, D=64):
    """A cache with room for L tokens a sequence (its pages all share one block) that holds none."""
    return kvq.QuantizedKVCache(E2M1, B, Hkv, D, -(-L // 16), 1)


@pytest.mark.parametrize("B,Hkv,G,T,L", [(16, 8, 8, 16, 23424), (1, 8, 4, 16, 39000), (2, 2, 8, 64, 12000), (3, 1, 16, 9, 4000)])
def test_one_workspace_for_shorter_calls(B, Hkv, G, T, L):
    """What kvq_tree_workspace_bytes asks for with the library's choice of splits is enough for every smaller bound on the
    lengths and for fewer nodes, and never shrinks as they grow."""
    cache = empty_cache(B, Hkv, L)
    ws = kvq.alloc_tree_workspace(cache, Hkv * G, T, L)
    rng = np.random.default_rng(0)
    lengths = sorted({0, 1, 127, 128, 129, 2432, 23296, L - 1, L, *rng.integers(1, L, 40).tolist()} & set(range(L + 1)))
    for t in sorted({1, T // 2, T - 1, T}):
        q = torch.zeros((B, t, Hkv * G, 64), dtype=torch.bfloat16, device="cuda")
        out = torch.ones_like(q)
        before = 0
        for n in lengths:
            kvq.kvq_tree_attention(cache, q, 0.1, n, out=out, workspace=ws)
            need = kvq.kvq_tree_workspace_bytes(cache, Hkv * G, t, n)
            assert before <= need <= ws.nbytes
            before = need
        assert (out == 0).all()
    with pytest.raises(kvq.KVQError):   # a workspace for one split does not do for two
        one = kvq.alloc_tree_workspace(cache, Hkv * G, T, L, 1)
        kvq.kvq_tree_attention(cache, q, 0.1, L, num_splits=2, out=out, workspace=one)
    assert cache.status_word() == 0
