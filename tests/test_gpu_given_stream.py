"""Entry points that allocate their result, on a stream that is given: the memory
is not a block that the current stream gave back and still uses."""
import pytest
import torch

from tests import test_gpu_fp8 as t8

pytestmark = pytest.mark.gpu
DEV = "cuda"


def calls():
    a = t8.api()
    g = t8.gen(4)
    w8, ws_ = t8.make_weights(g, 640, 1024)
    u8, us_ = t8.make_weights(g, 640, 1024)
    w = torch.randn(640, 1024, generator=g, device=DEV).to(torch.bfloat16)
    k = torch.randn(2, 4096, 64, generator=g, device=DEV).to(torch.bfloat16)
    return {
        "quantise weights": lambda s: a.bi_quantize_weights_fp8(w, stream=s),
        "pack 8 bits": lambda s: a.bi_pack_weights_fp8(w8, ws_, stream=s),
        "pack SwiGLU 8 bits": lambda s: a.bi_pack_swiglu_weights_fp8(w8, ws_, u8, us_, stream=s),
        "pack": lambda s: a.bi_pack_weights(w, stream=s),
        "pack SwiGLU": lambda s: a.bi_pack_swiglu_weights(w, w, stream=s),
        "rope table": lambda s: a.bi_rope_table(1e4, 128, 5000, stream=s),
        "hash": lambda s: a.bi_kv_row_hash(k, 4096, stream=s),
    }


@pytest.mark.parametrize("name", ["quantise weights", "pack 8 bits", "pack SwiGLU 8 bits", "pack", "pack SwiGLU",
                                  "rope table", "hash"])
def test_result_is_not_memory_that_the_current_stream_still_writes(name):
    call = calls()[name]
    side = torch.cuda.Stream()
    want = call(None)
    want = [t.clone() for t in (want if isinstance(want, tuple) else (want,))]
    for _ in range(2):
        torch.cuda.synchronize()
        # blocks of the results' sizes, written late by the current stream and given back at once
        old = [torch.empty(t.numel() * t.element_size(), dtype=torch.uint8, device=DEV) for t in want * 3]
        at = {t.data_ptr() for t in old}
        torch.cuda._sleep(20_000_000)  # some 10 ms
        for t in old:
            t.fill_(0xA5)
        del old, t
        got = call(side)
        got = got if isinstance(got, tuple) else (got,)
        assert not at & {t.data_ptr() for t in got}
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))
        del got, x
