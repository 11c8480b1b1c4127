"""Streams given as plain handles."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from mla_latent_kv_16_gb300 import build
    build.build()
    from mla_latent_kv_16_gb300 import capi
    capi.load()
    yield


def test_the_default_streams_handle(monkeypatch):
    """stream=0 is the default stream, not "none given" nor a stream of a pool: a call made on it from
    within another stream's block takes its missing buffers from the default stream's memory."""
    from mla_latent_kv_16_gb300 import capi
    i32 = dict(dtype=torch.int32, device="cuda")
    table, lens, refs = torch.tensor([[0, -1], [-1, -1]], **i32), torch.tensor([3, 0], **i32), torch.tensor([1, 0, 0, 0], **i32)
    q_lat, q_rope = torch.zeros(2, 1, 4, 512, device="cuda").bfloat16(), torch.zeros(2, 1, 4, 64, device="cuda").bfloat16()
    cache = torch.zeros(4, 8, 576, device="cuda").bfloat16()
    one = torch.tensor([0], **i32)
    torch.cuda.synchronize()
    made = []
    for name in ("empty", "empty_like"):
        def spy(*a, _real=getattr(torch, name), **kw):
            made.append(torch.cuda.current_stream().cuda_stream)
            return _real(*a, **kw)
        monkeypatch.setattr(torch, name, spy)
    default = torch.cuda.default_stream().cuda_stream
    assert default == 0
    with torch.cuda.stream(torch.cuda.Stream()):
        capi.mla_cache_extend(one, one, one, table, lens, refs, 8, max_new=0, stream=0)
        capi.mla_cache_compact(table, refs, stream=0)
        capi.mla_decode_window(q_lat, q_rope, cache, None, table, lens, 8, "bf16", 100, 0, num_splits=2, stream=0)
        with capi.on_stream(0):
            assert torch.cuda.current_stream() == torch.cuda.default_stream()
    assert len(made) == 6 + 4 + 2 and set(made) == {0}
    torch.cuda.synchronize()
