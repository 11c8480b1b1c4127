"""The split merge: its kernels for few and for many rows add the same partials in the same order."""
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


@pytest.mark.parametrize("cache,heads,many,few", [("bf16", 128, 40, 3), ("e4m3", 128, 30, 28), ("bf16", 5, 900, 2), ("f32", 16, 256, 7)])
@pytest.mark.parametrize("splits", [2, 3, 4, 6, 9])
def test_a_row_does_not_depend_on_how_many_there_are(cache, heads, many, few, splits):
    """A sequence's outputs are the same bits in a batch of `many` as in one of `few` (which the merge may
    do by another kernel), ones that end before the last split and empty ones among them."""
    from mla_latent_kv_16_gb300 import capi
    page, width = 64, 9
    g = torch.Generator(device="cuda").manual_seed(splits)
    t = torch.float32 if cache == "f32" else torch.bfloat16
    pool, scales = torch.randn(200, page, 576, generator=g, device="cuda"), None
    if cache == "e4m3":
        pool, scales = pool.to(torch.float8_e4m3fn).view(torch.uint8), torch.rand(200, page, 5, generator=g, device="cuda")
    else:
        pool = pool.to(t)
    table = torch.randint(0, 200, (many, width), generator=g, device="cuda", dtype=torch.int32)
    lens = torch.randint(1, page * width + 1, (many,), generator=g, device="cuda", dtype=torch.int32)
    lens[:2] = torch.tensor([page * width, 0])
    q = torch.randn(many, 1, heads, 512, generator=g, device="cuda").to(t)
    r = torch.randn(many, 1, heads, 64, generator=g, device="cuda").to(t)

    def call(n):
        return capi.mla_decode_paged(q[:n], r[:n], pool, scales, table[:n], lens[:n], page, cache, num_splits=splits)

    u, lse = call(many)
    v, lse_few = call(few)
    assert bool(torch.isfinite(u).all()) and bool((u[1] == 0).all()) and bool((lse[1] == -torch.inf).all())
    assert torch.equal(u[:few], v) and torch.equal(lse[:few], lse_few)
