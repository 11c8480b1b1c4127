"""What MLADecodeLayer sets up on the host: buffer sizes, refused arguments, the page state
(no GPU needed: nothing is launched)."""
import pytest
import torch

from mla_latent_kv_16_gb300 import build


@pytest.fixture(scope="module")
def capi():
    build.build()
    from mla_latent_kv_16_gb300 import capi as C
    C.load()
    return C


def make(seqs, page, width, heads=128, cache="bf16", table=None, lens=None, pages_each=1, **kw):
    from mla_latent_kv_16_gb300 import workloads as W
    from mla_latent_kv_16_gb300.engine import MLADecodeLayer
    act = "f32" if cache == "f32" else "bf16"
    w = W.Workload("layer", seqs, 1, heads, [pages_each * page] * seqs, page, act, cache, 0)
    weights = [torch.zeros(heads, 128, 512, dtype=W.TORCH_DTYPE[act]) for _ in range(2)]
    if table is None:
        table = torch.full((seqs, width), -1, dtype=torch.int32)
    return MLADecodeLayer(w, *weights, table, torch.zeros(seqs, dtype=torch.int32) if lens is None else lens, device="cpu",
                          **kw)


@pytest.mark.parametrize("window", [0, 200])
@pytest.mark.parametrize("cache,heads,splits", [("bf16", 128, None), ("bf16", 128, 9), ("e4m3", 128, None), ("bf16", 16, None),
                                                ("f32", 16, 7)])
def test_workspace_is_sized_by_the_table(capi, cache, heads, splits, window):
    """The calls take their split count from the table's width, which may exceed what the workload's
    sequences need: the layer's count and workspace have to be those."""
    layer = make(8, 64, 11, heads, cache, num_splits=splits, window=window, sinks=3 if window else 0)
    asked = splits or 0
    if window:
        args = (8, 1, 11, 64, window, 3, asked, heads, cache)
        want, need = capi.mla_decode_window_num_splits(*args), capi.mla_decode_window_workspace_size(*args)
    else:
        args = (8, 1, 11, 64, asked, heads, cache)
        want, need = capi.mla_decode_num_splits(*args), capi.mla_decode_workspace_size(*args)
    assert want > 1
    assert layer.splits == want
    assert layer.workspace.numel() >= need


def test_page_state_counts_the_pool_only(capi):
    """Entries outside the pool are nobody's pages: the counts are as many as the pool has pages,
    or new pages would be handed out behind its end."""
    table = torch.tensor([[0, 2, -1, -1], [3, 9, 2 ** 31 - 1, -2 ** 31], [2, 10, 8, -1]], dtype=torch.int32)
    layer = make(3, 16, 4, heads=16, table=table, pages_each=3)
    assert layer.num_pages == 9
    layer.prepare_pages()
    assert layer.ref_counts.dtype == torch.int32
    assert layer.ref_counts.tolist() == [1, 0, 2, 1, 0, 0, 0, 0, 1]
    counts = layer.ref_counts
    layer.prepare_pages()  # once
    assert layer.ref_counts is counts


@pytest.mark.parametrize("kw", [dict(window=-1), dict(sinks=-1), dict(window=5, sinks=-3)])
def test_negative_window_or_sinks_are_refused(capi, kw):
    """A negative window is none of the masks there are (0 stands for every earlier token)."""
    with pytest.raises(ValueError, match="negative"):
        make(2, 16, 2, heads=16, **kw)
