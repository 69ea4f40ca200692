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


def pointers(monkeypatch, name, position, call):
    """The pointer that `call` hands to the library as argument `position` of `name` (nothing is launched)."""
    seen = []
    monkeypatch.setattr(kvq, "_call", lambda what, index, stream, *args: seen.append((what, args)))
    result = call()
    monkeypatch.undo()
    assert [w for w, _ in seen] == [name]
    return seen[0][1][position], result


def test_memory_made_for_another_stream_is_that_streams_own(monkeypatch):
    """What a call on another stream allocates does not come from blocks that the current stream has just given
    up (its pending work may still use them), and what it returns is held for the current stream."""
    cache = empty_cache(4, 2, 4096)
    side = torch.cuda.Stream()
    q = torch.zeros((4, 8, 8, 64), dtype=torch.bfloat16, device="cuda")
    mass = torch.zeros((4, 256), device="cuda")
    tree = lambda: kvq.kvq_tree_attention(cache, q, 0.1, 4096, stream=side)
    for name, position, nbytes, call in (("kvq_tree_attention", 13, q.nbytes, tree),
                                         ("kvq_tree_attention", 17, kvq.alloc_tree_workspace(cache, 8, 8, 4096).nbytes, tree),
                                         ("kvq_evict_pages", 9, 16, lambda: kvq.kvq_evict_pages(cache, mass, 8, stream=side))):
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        held = [torch.empty(nbytes, dtype=torch.uint8, device="cuda") for _ in range(2)]
        given_up = {t.data_ptr() for t in held}
        del held
        ptr, result = pointers(monkeypatch, name, position, call)
        assert ptr and ptr not in given_up
        if position != 17:
            assert result.data_ptr() == ptr


def test_call_on_another_stream_beside_pending_work():
    """Work pending on the current stream reads memory that was given up; a call on another stream, its tensors made
    inside, leaves it alone and gives the same bits."""
    cache = kvq.QuantizedKVCache(E2M1, 2, 2, 64, 16, 32)
    k, v = [torch.randn((2, 200, 2, 64), device="cuda") for _ in range(2)]
    kvq.kvq_quantize_append(cache, k, v)
    q = torch.randn((2, 4, 8, 64), device="cuda").to(torch.bfloat16)
    want = kvq.kvq_tree_attention(cache, q, 0.125, 200)
    nbytes = kvq.alloc_tree_workspace(cache, 8, 4, 200).nbytes
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for n in (want.nbytes, nbytes):
        x = torch.full((n // 2,), 3, dtype=torch.int16, device="cuda")
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)           # about 10 ms
        total = x.sum()
        del x
        got = kvq.kvq_tree_attention(cache, q, 0.125, 200, stream=side)
        side.synchronize()
        assert torch.equal(got, want)
        assert int(total) == 3 * (n // 2)
