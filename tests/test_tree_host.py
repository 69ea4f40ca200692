"""The host side of the calls beside decode attention: what a cache handle on
the caller's buffers accepts, and what the binding hands to the library (no GPU
is needed: nothing is launched)."""
import ctypes
import os
import shutil

import numpy as np
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


def buffers(kvq, fmt, Hkv=2, D=64, pages=8):
    """Host tensors of a cache of two sequences, the pools 16 bytes into larger ones."""
    c = kvq.kvq_config(2, Hkv, D, 4, pages, 1 if fmt == kvq.KVQ_FMT_TIERED else 0, fmt, 16, 3.0, 2)
    main = 2 * Hkv * kvq.kvq_block_bytes(c, 0) * pages
    tier = 2 * Hkv * kvq.kvq_block_bytes(c, 1) * pages if fmt == kvq.KVQ_FMT_TIERED else 0
    big = torch.zeros(main + 64, dtype=torch.uint8)
    base = -big.data_ptr() % 16 + 16
    big_t = torch.zeros(tier + 64, dtype=torch.uint8)
    base_t = -big_t.data_ptr() % 16 + 16
    b = dict(pool=big[base:base + main], page_table=torch.zeros((2, 4), dtype=torch.int32),
             seq_lens=torch.zeros(2, dtype=torch.int32), status=torch.zeros(1, dtype=torch.int32))
    if tier:
        b["tier_pool"] = big_t[base_t:base_t + tier]
    if fmt >= kvq.KVQ_FMT_CB2_OUTLIER:
        b["staging"] = torch.zeros(2 * Hkv * 2 * 64 * D, dtype=torch.float32)
    if fmt == kvq.KVQ_FMT_CB2_STATIC:
        b["static_mask"] = torch.zeros((Hkv, 2, 2), dtype=torch.uint8)
    return b, (big, base, main), (big_t, base_t, tier)


def test_from_buffers_checks_the_pools(kvq):
    """Pools are bytes and 16-byte aligned: the kernels copy blocks 16 bytes at a time."""
    for fmt in range(7):
        b, main, tier = buffers(kvq, fmt)
        make = lambda **kw: kvq.QuantizedKVCache.from_buffers(fmt, 2, 64, **{**b, **kw})
        assert make().cfg.num_pages == 8
        for off in (1, 4, 8):
            t, base, n = main
            with pytest.raises(AssertionError):
                make(pool=t[base + off:base + off + n])
        with pytest.raises(AssertionError):
            make(pool=b["pool"].view(torch.float32))
        if tier[2]:
            t, base, n = tier
            with pytest.raises(AssertionError):
                make(tier_pool=t[base + 8:base + 8 + n])
            with pytest.raises(AssertionError):
                make(tier_pool=b["tier_pool"].view(torch.int32))
        if "static_mask" in b:
            with pytest.raises(AssertionError):
                make(static_mask=b["static_mask"].float())


@pytest.mark.parametrize("field", ["pool", "tier_pool"])
def test_misaligned_pools_are_refused(kvq, field):
    """By every call that reads or writes blocks, before anything is launched."""
    A = 1 << 20   # an address that is never read
    cfg = kvq.kvq_config(4, 8, 128, 16, 64, 64, kvq.KVQ_FMT_TIERED, 16, 3.0)
    for off in (1, 4, 8):
        p = dict(pool=A, tier_pool=A, page_table=A, seq_lens=A, staging=A, status=A, static_mask=None)
        p[field] = A + off
        cache = kvq.kvq_cache(*[p[f] for f, _ in kvq.kvq_cache._fields_])
        L, c, k, z = kvq.lib(), ctypes.byref(cfg), ctypes.byref(cache), ctypes.c_float(0.1)
        assert L.kvq_tree_attention(c, k, A, 32, 4, A, A, None, 0, None, z, 100, 2, A, 0, None, None, A, 0, None) == kvq.KVQ_ERR_INVALID_ARG
        assert L.kvq_decode_attention(c, k, A, 32, z, 100, 2, A, 0, A, 0, None) == kvq.KVQ_ERR_INVALID_ARG
        assert L.kvq_quantize_append(c, k, A, A, 0, 0, None, None) == kvq.KVQ_ERR_INVALID_ARG
        assert L.kvq_project_append(c, k, A, 128, A, A, 0, None, None, None) == kvq.KVQ_ERR_INVALID_ARG


def test_a_handle_whose_structures_are_replaced(kvq):
    """Calls read the handle's present cfg and c, not those of an earlier call."""
    b, _, _ = buffers(kvq, kvq.KVQ_FMT_FP4_E2M1_S16)
    cache = kvq.QuantizedKVCache.from_buffers(kvq.KVQ_FMT_FP4_E2M1_S16, 2, 64, **b)
    assert kvq._refs(cache)[0]._obj is cache.cfg and kvq._refs(cache)[1]._obj is cache.c
    c = kvq.kvq_cache.from_buffer_copy(cache.c)
    cfg = kvq.kvq_config.from_buffer_copy(cache.cfg)
    cache.c, cache.cfg = c, cfg
    assert kvq._refs(cache)[0]._obj is cfg and kvq._refs(cache)[1]._obj is c


@pytest.mark.parametrize("number", [0.5, 1, np.float32(0.5), np.float64(0.5), torch.tensor(0.5)], ids=str)
def test_scales_of_any_number_type(kvq, monkeypatch, number):
    """The scale and the decay are taken as decode attention takes its scale: anything that is a number."""
    b, _, _ = buffers(kvq, kvq.KVQ_FMT_FP4_E2M1_S16)
    cache = kvq.QuantizedKVCache.from_buffers(kvq.KVQ_FMT_FP4_E2M1_S16, 2, 64, **b)
    seen = []
    monkeypatch.setattr(kvq, "_check_on", lambda *a: None)   # (the tensors lie on the host)
    monkeypatch.setattr(kvq, "_call", lambda what, index, stream, *args: seen.append(args))
    kvq.kvq_tree_attention(cache, torch.zeros((2, 1, 4, 64), dtype=torch.bfloat16), number, 64)
    mass = torch.zeros((2, 4))
    kvq.kvq_page_mass(cache, torch.zeros((2, 1, 4)), torch.zeros((2, 1, 4, 4)), mass, decay=number)
    for args, types in zip(seen, (kvq.lib().kvq_tree_attention.argtypes, kvq.lib().kvq_page_mass.argtypes)):
        floats = [a for a, t in zip(args, types) if t is ctypes.c_float]
        assert len(floats) == 1 and type(floats[0]) is float and floats[0] == float(number)
