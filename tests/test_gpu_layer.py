"""MLADecodeLayer as a serving loop uses it, beside test_gpu_cache_life.py: layers without a window, and
what the layer promises of its page state."""
import numpy as np
import pytest
import torch

from _util import OUT_ULP_REL, assert_close, f64
from test_gpu_cache_life import SCALE, Life

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


def make_layer(cache_dtype, heads, seqs, page, pages, width, max_pos, table=None, lens=None, **kw):
    """A bf16 layer whose workload is a page a sequence, in a wider table."""
    from mla_latent_kv_16_gb300 import workloads as W
    from mla_latent_kv_16_gb300.engine import MLADecodeLayer
    w = W.Workload("life", seqs, 1, heads, [1] * seqs, page, "bf16", cache_dtype, 0)
    g = torch.Generator(device="cuda").manual_seed(1)
    weights = [(torch.randn(heads, 128, 512, generator=g, device="cuda") / 512 ** 0.5).bfloat16() for _ in range(2)]
    table = torch.full((seqs, width), -1, dtype=torch.int32) if table is None else table
    lens = torch.zeros(seqs, dtype=torch.int32) if lens is None else lens
    return MLADecodeLayer(w, *weights, table, lens, spare_pages=pages - w.num_pages, max_pos=max_pos, **kw)


class Whole(Life):
    """A life without a window: every earlier token is visible; decode alone, and with the up-projection."""

    def check(self, what):
        layer = self.layer
        B, H = len(self.rows), layer.H
        q_lat = (0.5 * torch.randn(B, 1, H, 512, generator=self.g, device="cuda")).to(layer.act)
        q_rope = torch.randn(B, 1, H, 64, generator=self.g, device="cuda").to(layer.act)
        alone = f64(layer.decode(q_lat, q_rope)[0])
        o = f64(layer.decode_out_proj(q_lat, q_rope))
        ql, qr, w_uv, u = f64(q_lat), f64(q_rope), f64(layer.w_uv), f64(layer.u)
        for b, rows in enumerate(self.rows):
            if not rows:
                assert np.all(u[b] == 0) and np.all(alone[b] == 0) and np.all(o[b] == 0)
                continue
            r = np.array(rows)
            z = (ql[b, 0] @ r[:, :512].T + qr[b, 0] @ r[:, 512:].T) * SCALE
            e = np.exp(z - z.max(1, keepdims=True))
            want = e @ r[:, :512] / e.sum(1, keepdims=True)
            # (the output's own rounding aside: with few tokens u is as large as a row's values)
            assert_close(alone[b, 0], want, what=f"{what}, sequence {b}", ulp_rel=OUT_ULP_REL)
            assert_close(u[b, 0], want, what=f"{what}, sequence {b}, with the projection", ulp_rel=OUT_ULP_REL)
            assert_close(o[b, 0], np.einsum("hc,hdc->hd", want, w_uv), what=f"{what}, sequence {b}, o", ulp_rel=OUT_ULP_REL)


@pytest.mark.parametrize("cache,heads,page,splits", [("bf16", 128, 64, 0), ("e4m3", 128, 64, 3), ("bf16", 16, 16, 0)])
def test_a_serving_loop_without_a_window(cache, heads, page, splits):
    """A table wider than the workload's sequences, in which prompts come in, fork and grow."""
    layer = make_layer(cache, heads, 8, page, pages=-(-4000 // page), width=-(-900 // page), max_pos=900,
                       num_splits=splits)
    assert layer.splits > 1
    life = Whole(layer, seed=page + heads)
    life.extend([(0, 0, 700), (1, 1, 3 * page), (2, 2, 1)])
    life.check("prompts")
    life.extend([(0, 3, 1), (0, 4, 1), (1, 5, 2), (2, 2, 1), (0, 0, 1)])
    life.check("beams")
    for step in range(2):
        life.extend([(b, b, life.rng.choice([1, 1, page + 1])) for b, r in enumerate(life.rows) if r])
        life.check(f"step {step}")
    life.free([0, 5])
    life.extend([(3, 6, 2), (7, 7, 20)])
    n = life.held()
    stats = layer.compact()
    assert stats.tolist() == [n, n]
    life.check("compacted")
    assert layer.device_error() & ~2 == 0  # (2: the empty sequences of the batch)


def test_the_first_page_call_captured():
    """A page state that does not exist yet cannot be made inside a capture: the call is refused before
    anything is enqueued, the capture stays usable, and after prepare_pages() it is captured."""
    layer = make_layer("bf16", 16, 2, 16, pages=12, width=5, max_pos=80, window=20, sinks=1)
    every = torch.arange(2, dtype=torch.int32, device="cuda")
    grow = torch.full((2,), 17, dtype=torch.int32, device="cuda")
    pos, slots = torch.empty(34, dtype=torch.int32, device="cuda"), torch.empty(34, dtype=torch.int64, device="cuda")
    calls = [lambda: layer.extend(every, every, grow, pos, slots), lambda: layer.free(every), layer.evict, layer.compact]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for call in calls:
            with pytest.raises(RuntimeError, match="prepare_pages"):
                call()
    layer.prepare_pages()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.extend(every, every, grow, pos, slots)
    for n in (1, 2):
        graph.replay()
        torch.cuda.synchronize()
        assert layer.seq_lens.tolist() == [17 * n] * 2
        assert int((layer.ref_counts == 1).sum()) == 2 * -(-17 * n // 16) and int(layer.ref_counts.sum()) == int((layer.block_table >= 0).sum())
    assert layer.device_error() == 0


def test_pages_outside_the_pool_are_not_handed_out():
    """A table with entries past the pool: the pages that extend() hands out are the pool's."""
    table = torch.full((2, 6), -1, dtype=torch.int32)
    table[1, :3] = torch.tensor([3, 5000, 1])
    layer = make_layer("bf16", 16, 2, 16, pages=5, width=6, max_pos=96, table=table,
                       lens=torch.tensor([0, 48], dtype=torch.int32))
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    pos, slots = torch.empty(40, dtype=torch.int32, device="cuda"), torch.empty(40, dtype=torch.int64, device="cuda")
    layer.extend(one, one, one + 40, pos, slots)
    assert layer.block_table[0].tolist() == [0, 2, 4, -1, -1, -1] and layer.device_error() == 0
    layer.extend(one, one, one + 9, pos, slots)  # none is left
    assert layer.block_table[0].tolist() == [0, 2, 4, -1, -1, -1] and layer.device_error() == 64
