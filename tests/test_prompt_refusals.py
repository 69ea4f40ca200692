"""What kvq_norm_rope and kvq_prompt_attention refuse, before any buffer is
touched (the pointers are never read: no GPU is needed)."""
import ctypes
import os
import shutil

import pytest
import torch

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="nvcc not available")


@pytest.fixture(scope="module")
def kvq():
    from sub_byte_quantized_kvq_gb300 import build
    build.build()
    from sub_byte_quantized_kvq_gb300 import kvq as mod
    return mod


FAKE = 1 << 20   # 16-byte aligned, never read


def cfg_of(kvq, D=128, **kw):
    c = kvq.kvq_config(4, 8, D, 16, 64, 0, 1, 16, 3.0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def test_norm_rope_refusals(kvq):
    def rope(cfg=None, q=FAKE, qs=4096, Hq=32, k=FAKE, ks=1024, tin=0, rows=0, wq=None, wk=None, eps=1e-6, pos=FAKE, axes=1, f=FAKE, R=128,
             pair=None, inter=0, qo=2 * FAKE, qos=4096, ko=2 * FAKE, kos=1024, tout=0):
        return kvq.lib().kvq_norm_rope(ctypes.byref(cfg or cfg_of(kvq)), q, qs, Hq, k, ks, tin, rows, wq, wk, ctypes.c_float(eps), pos, axes, f,
                                       R, pair, inter, qo, qos, ko, kos, tout, None)
    INVALID = kvq.KVQ_ERR_INVALID_ARG
    assert rope() == kvq.KVQ_OK                       # no rows: nothing to do, and nothing read
    assert rope(q=None, qo=None) == kvq.KVQ_OK and rope(k=None, ko=None) == kvq.KVQ_OK
    assert rope(R=0, pos=None, f=None) == kvq.KVQ_OK and rope(eps=-1.0) == kvq.KVQ_OK
    assert rope(qo=FAKE, ko=FAKE) == kvq.KVQ_OK       # in place
    assert rope(qs=0, ks=0) == kvq.KVQ_OK             # one row for all
    assert rope(axes=3, pair=bytes([2] * 64)) == kvq.KVQ_OK
    for bad in (dict(q=None, k=None), dict(qo=None), dict(ko=None), dict(q=FAKE + 8), dict(k=FAKE + 2), dict(qo=FAKE + 4), dict(ko=FAKE + 8),
                dict(qs=4097), dict(ks=1028), dict(qos=4090), dict(qos=4088), dict(kos=1016), dict(qs=-8), dict(qs=1 << 38), dict(Hq=0),
                dict(Hq=30), dict(tin=3), dict(tout=-1), dict(rows=-1), dict(eps=float("nan")), dict(eps=float("inf")),
                dict(eps=-1.0, wq=FAKE), dict(eps=-1.0, wk=FAKE), dict(pos=None), dict(f=None), dict(R=-16), dict(R=144), dict(R=8),
                dict(axes=0), dict(axes=256), dict(axes=3, pair=bytes([0] * 63 + [3])), dict(inter=2), dict(qo=FAKE, tout=2),
                dict(qo=FAKE, qos=8192)):
        assert rope(**bad) == INVALID, bad
    assert rope(cfg_of(kvq, 96)) == kvq.KVQ_ERR_UNSUPPORTED


def test_prompt_refusals(kvq):
    def prompt(cfg=None, q=FAKE, qs=4096, k=FAKE, ks=1024, v=FAKE, vs=1024, t=0, Hq=32, rows=0, n=None, t_new=9, scale=0.1, causal=1, out=FAKE,
               os=4096, tout=0, status=FAKE):
        return kvq.lib().kvq_prompt_attention(ctypes.byref(cfg or cfg_of(kvq)), q, qs, k, ks, v, vs, t, Hq, rows, n, n, t_new, ctypes.c_float(scale),
                                              causal, out, os, tout, None, status, None)
    assert prompt() == kvq.KVQ_OK and prompt(rows=5, t_new=0) == kvq.KVQ_OK     # no rows, no tokens
    assert prompt(t=1, tout=1) == kvq.KVQ_OK and prompt(t=1, tout=2) == kvq.KVQ_OK and prompt(tout=2) == kvq.KVQ_OK
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(status=None), dict(q=FAKE + 8), dict(k=FAKE + 8),
                dict(v=FAKE + 2), dict(out=FAKE + 4), dict(qs=4100), dict(ks=1020), dict(vs=-1024), dict(qs=4088), dict(ks=0), dict(os=4088), dict(t=2), dict(t=2, tout=2),
                dict(tout=1), dict(tout=3), dict(Hq=0), dict(Hq=31), dict(rows=-1), dict(t_new=-1), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(causal=2)):
        assert prompt(**bad) == kvq.KVQ_ERR_INVALID_ARG, bad
    assert prompt(cfg_of(kvq, 96)) == kvq.KVQ_ERR_UNSUPPORTED
    assert prompt(Hq=8 * 17) == kvq.KVQ_ERR_UNSUPPORTED
    assert prompt(t_new=(1 << 21) + 1) == kvq.KVQ_ERR_UNSUPPORTED and prompt(t_new=1 << 21) == kvq.KVQ_OK


def test_rows_of_a_tensor(kvq):
    """The binding's reading of a tensor as evenly spaced rows."""
    rows = kvq._token_rows
    x = torch.zeros((3, 5, 96))
    assert rows(x.view(3, 5, 6, 16), 6, 16) == (15, 96)
    assert rows(x[..., 32:64].unflatten(-1, (2, 16)), 2, 16) == (15, 96)
    assert rows(x[:, :1, :32].unflatten(-1, (2, 16)), 2, 16) == (3, 480)
    assert rows(x[1:2, 2:3, :32].unflatten(-1, (2, 16)), 2, 16) == (1, 32)
    assert rows(torch.zeros((1, 2, 16)).expand(7, 2, 16), 2, 16) == (7, 0)
    assert rows(torch.zeros((0, 2, 16)), 2, 16)[0] == 0
    assert rows(torch.zeros((4, 16, 1)).transpose(1, 2), 1, 16) == (4, 16)
    for bad in (x[:, :4].unflatten(-1, (6, 16)),        # every fifth row is missing
                x.view(3, 5, 16, 6).transpose(2, 3)):   # channels apart
        with pytest.raises(ValueError):
            rows(bad, 6, 16)
    for shape in ((3, 6, 8), (6, 16)):
        with pytest.raises(ValueError):
            rows(torch.zeros(shape), 6, 16)


def test_binding_refusals(kvq):
    """What the binding refuses before it looks for a device (tensors and cache on the host)."""
    cache = kvq.QuantizedKVCache(1, 2, 2, 64, 1, 1, device="cpu")
    bf = torch.bfloat16
    q, k, pos, f = torch.zeros((6, 4, 64), dtype=bf), torch.zeros((6, 2, 64), dtype=bf), torch.zeros(6, dtype=torch.int32), torch.zeros(32)
    rope = lambda *a, **kw: kvq.kvq_norm_rope(cache, *a, **kw)
    for call in (lambda: rope(None, None, pos, f), lambda: rope(q, k[:5], pos, f), lambda: rope(q, k.float(), pos, f), lambda: rope(q, k, pos[:5], f),
                 lambda: rope(q, k, pos, f, eps=-1.0), lambda: rope(q, k, pos, f, pair_axis=[0] * 31), lambda: rope(q, k, torch.zeros((2, 6), dtype=torch.int32), f),
                 lambda: rope(q, k, pos[None], f, pair_axis=[1] * 32), lambda: rope(q, k, pos[None], f, pair_axis=[-1] * 32),
                 lambda: rope(q, k, pos, f, q_out=q[:5]), lambda: rope(q, k, pos, f, q_out=q, k_out=k.float()),
                 lambda: rope(q[..., :32], k, pos, f), lambda: rope(q, torch.zeros((6, 4, 64), dtype=bf), pos, f),
                 lambda: rope(q, k, pos, f)):                                   # (all is right but the device)
        with pytest.raises(ValueError):
            call()
    for call in (lambda: rope(q, k, pos.long(), f), lambda: rope(q, k, None, f), lambda: rope(q, k, pos, f.double()),
                 lambda: rope(q, k, pos, f, q_weight=torch.zeros(64, dtype=bf)), lambda: rope(q, k, pos, f, k_weight=torch.zeros(65))):
        with pytest.raises(AssertionError):
            call()
    prompt = lambda *a, **kw: kvq.kvq_prompt_attention(cache, *a, **kw)
    n = torch.zeros(2, dtype=torch.int32)
    pq, pk = q.view(2, 3, 4, 64), k.view(2, 3, 2, 64)
    for call in (lambda: prompt(pq.float(), pk.float(), pk.float(), 0.1), lambda: prompt(pq, pk.half(), pk, 0.1), lambda: prompt(q, k, k, 0.1, first_row=n),
                 lambda: prompt(q, k, k, 0.1, first_row=n, t_per_seq=n), lambda: prompt(pq, pk[..., :1, :], pk, 0.1),
                 lambda: prompt(pq, pk[:, :2], pk, 0.1),                        # (rows that are not evenly spaced)
                 lambda: prompt(pq, pk, pk, 0.1)):                              # (all is right but the device)
        with pytest.raises(ValueError):
            call()
    for call in (lambda: prompt(q, k, k, 0.1), lambda: prompt(pq[:1], pk[:1], pk[:1], 0.1), lambda: prompt(pq, pk, pk, 0.1, t_new=2),
                 lambda: prompt(pq, pk, pk, 0.1, t_per_seq=n.long()),
                 lambda: prompt(pq, pk, pk, 0.1, out=torch.zeros((2, 3, 4, 64), dtype=torch.float16)), lambda: prompt(pq, pk, pk, 0.1, lse=torch.zeros((2, 3))),
                 lambda: prompt(q, k, k, 0.1, first_row=n[:1], t_per_seq=n, t_new=3)):
        with pytest.raises(AssertionError):
            call()
