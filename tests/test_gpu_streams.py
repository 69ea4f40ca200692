"""Append, decode and dequantization on a stream that is not the current one,
with everything that the binding allocates left to it."""
import pytest
import torch

from sub_byte_quantized_kvq_gb300 import kvq

pytestmark = pytest.mark.gpu


def test_memory_made_for_another_stream_is_that_streams_own():
    """Outputs do not come from blocks that the current stream has just given up, whose last user may be pending."""
    cache = kvq.QuantizedKVCache(kvq.KVQ_FMT_FP4_E2M1_S16, 4, 2, 64, 64, 1)
    q = torch.zeros((4, 8, 64), dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    for call in (lambda: kvq.kvq_decode_attention(cache, q, 0.1, 1024, stream=side),
                 lambda: kvq.kvq_decode_attention_noalloc(cache, q, 0.1, 1024, stream=side),
                 lambda: kvq.kvq_dequantize(cache, 0, 0, 0, 0, 32, stream=side)):
        size = 0
        for _ in range(2):   # the first call tells the output's size
            torch.cuda.synchronize()
            torch.cuda.empty_cache()
            held = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(3)] if size else []
            given_up = {t.data_ptr() for t in held}
            del held
            out = call()
            side.synchronize()
            assert out.data_ptr() not in given_up
            size = out.nbytes
            del out


def test_calls_on_another_stream_beside_pending_work():
    """The current stream is busy for some milliseconds: the other stream's calls do not wait for it to convert the
    lengths or to zero a workspace, and give the bits of calls on the current stream."""
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = [torch.randn((2, 96, 2, 64), generator=g, device="cuda") for _ in range(2)]
    q = torch.randn((2, 8, 64), generator=g, device="cuda").to(torch.bfloat16)
    lens = torch.tensor([96, 41], device="cuda")    # int64: the append converts it
    side = torch.cuda.Stream()
    results = []
    for stream in (None, side):
        cache = kvq.QuantizedKVCache(kvq.KVQ_FMT_CB2_OUTLIER, 2, 2, 64, 8, 16)
        torch.cuda.synchronize()
        if stream is not None:
            torch.cuda._sleep(20_000_000)           # about 10 ms
        kvq.kvq_quantize_append(cache, k, v, lens, stream=stream)
        out = kvq.kvq_decode_attention(cache, q, 0.125, 96, num_splits=2, stream=stream)
        vals = kvq.kvq_dequantize(cache, 1, 1, 1, 0, 41, stream=stream)
        if stream is not None:
            stream.synchronize()
        torch.cuda.synchronize()
        results.append((cache.pool, cache.seq_lens, cache.staging, out, vals))
        assert cache.status_word() == 0
    for a, b in zip(*results):
        assert torch.equal(a, b)
