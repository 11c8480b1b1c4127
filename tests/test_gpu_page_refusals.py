"""Requests of mla_cache_extend that its state cannot serve, and the largest lists: what is refused is
flagged and leaves the state as it was, and what the other requests get does not change."""
import numpy as np
import pytest
import torch

from test_gpu_pages import BAD_PAGE, BAD_SEQLEN, Device, Model, both, same

pytestmark = pytest.mark.gpu
INT_MAX = 2 ** 31 - 1


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from mla_latent_kv_16_gb300 import build
    build.build()
    from mla_latent_kv_16_gb300 import capi
    capi.load()
    yield


@pytest.mark.parametrize("width", [8, 9000])  # (one launch, two launches)
@pytest.mark.parametrize("entry", [-1, -2 ** 31, 20, INT_MAX])
def test_a_source_without_its_last_page(width, entry):
    """The partly filled last page of a source is missing from the table, or lies outside the pool: its rows
    cannot be copied and no new token can follow them, so forks and growths are refused."""
    m = Model(6, width, 20, 4)
    d = Device(m)
    both(m, d, "extend", [(0, 0, 10), (2, 2, 3)], 13)
    lost = int(m.table[0, 2])
    for x in (m.table, d.table):
        x[0, 2] = entry
    before = m.table.copy(), m.lens.copy(), m.refs.copy()
    # a fork, one that adds nothing, a growth; then a growth and a prompt that have what they need
    reqs = [(0, 1, 3), (0, 3, 0), (0, 0, 2), (2, 2, 1), (4, 4, 5)]
    cs, cd, cr, pos, slot = (t.cpu().numpy() for t in d.extend(reqs, 13))
    assert int(d.err.item()) == BAD_PAGE
    table, lens, refs = before
    free = [p for p in range(20) if refs[p] == 0]
    # the refused forks would have taken 2 pages and 1, the growths 0: the prompt gets the next ones
    new = free[3:5]
    table[4, :2] = new
    refs[new] = 1
    lens[2], lens[4] = 4, 5
    assert np.array_equal(d.table.cpu().numpy(), table)
    assert np.array_equal(d.lens.cpu().numpy(), lens)
    assert np.array_equal(d.refs.cpu().numpy(), refs) and refs[lost] == 1
    assert cs.tolist() == [-1] * 5 and cd.tolist() == [-1] * 5 and cr.tolist() == [0] * 5
    assert pos.tolist() == [0] * 5 + [3] + [0, 1, 2, 3, 4] + [-7] * 2
    assert slot.tolist() == [-1] * 5 + [int(table[2, 0]) * 4 + 3] + [new[0] * 4 + k for k in range(4)] + [new[1] * 4] + [-7] * 2
    d.err.zero_()
    d.extend([(0, 0, 0)], 0)  # asks for nothing of that page
    assert int(d.err.item()) == 0


def test_a_source_whose_last_page_is_full():
    """There is no partly filled page then: a fork shares what the row holds, none where it holds none."""
    m = Model(4, 8, 20, 4)
    d = Device(m)
    both(m, d, "extend", [(0, 0, 8), (1, 1, 12)], 20)
    for x in (m.table, d.table):
        x[0, 1] = -1
    m.refs[1] = 0
    d.refs[1] = 0
    both(m, d, "extend", [(0, 2, 3), (0, 0, 1), (1, 3, 0)], 4)
    # outside the pool: the entry is not shared and says so
    m.table[1, 0] = d.table[1, 0] = 20
    both(m, d, "free", [3])
    m.err = 0
    d.extend([(1, 3, 0)], 0)
    assert int(d.err.item()) == BAD_PAGE
    assert d.table[3].tolist() == [-1] + m.table[1, 1:3].tolist() + [-1] * 5
    assert int(d.lens[3]) == 12 and d.refs[m.table[1, 1:3].tolist()].tolist() == [2, 2]


def test_the_longest_list_of_new_tokens():
    """A refused request owns its places whatever their number: 2^31 - 1 of them, where a 32-bit signed
    count of steps of thousands would pass its end."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 26 GB")
    from mla_latent_kv_16_gb300 import capi
    m = Model(2, 4, 8, 4)
    d = Device(m)
    pos = torch.full((INT_MAX,), -7, dtype=torch.int32, device="cuda")
    slot = torch.full((INT_MAX,), -7, dtype=torch.int64, device="cuda")
    one, n = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.full((1,), INT_MAX, dtype=torch.int32, device="cuda")
    capi.mla_cache_extend(one, one, n, d.table, d.lens, d.refs, 4, positions=pos, slots=slot, dev_error=d.err)
    assert int(d.err.item()) == BAD_SEQLEN
    assert int(pos.max()) == int(pos.min()) == 0 and int(slot.max()) == int(slot.min()) == -1
    m.err = BAD_SEQLEN
    same(m, d)
