"""The paged cache where the page table is much wider than the rows (a cache that held a prompt and decodes within its
budget, a server's tables made for the longest context), and evictions to other arrays by clusters."""
import pytest
import torch

from gpuhelp import dev
from test_gpu_paged import Cache, Case, _positions

pytestmark = pytest.mark.gpu

NONE = 2 ** 31 - 1  # past the used pages the table holds no page numbers


def _widen(table, max_pages):
    wide = torch.full((table.shape[0], max_pages), NONE, dtype=torch.int32, device=table.device)
    wide[:, :table.shape[1]] = table
    return wide


@pytest.mark.parametrize("G", [1, 4, 7])
@pytest.mark.parametrize("inplace", [False, True])
def test_weights_in_a_wide_table(cuda_lib, G, inplace):
    lens = [0, 1, 40, 300, 2065]
    c = Case(lens, 2 * G, 2, 128, 16, weights=True, seed=G, poison=float("nan"))
    pages = 32768 // 16
    c.table = _widen(c.table, pages)
    wide = torch.full((len(lens), 2, pages * 16), float("nan"), device=dev())
    for r, n in enumerate(lens):
        wide[r, :, :n] = c.acc[r, :, :n]  # the slots past the rows may hold anything
    c.acc = wide
    c.acc_out = torch.full_like(wide, 7.0)
    ws = c.b.bastion_paged_attention_workspace_bytes(len(lens), 2 * G, 2, 128, pages * 16, True)
    c.ws = c.b.workspace(ws, dev())
    c.ws[-(ws // 2):] = 0xff  # the scores' place: NaN in every slot that is not written
    c.run()
    if inplace:
        torch.cuda.synchronize()
        first, acc = c.acc_out.clone(), c.acc.clone()
        c.b.bastion_paged_attention(c.q, c.k, c.v, c.table, c.seq_len, c.scale, c.out, c.ws, c.status, lse=c.lse,
                                    acc=acc, acc_out=acc)
        torch.cuda.synchronize()
        for r, n in enumerate(lens):
            assert torch.equal(acc[r, :, :n], first[r, :, :n])
            assert bool(torch.isnan(acc[r, :, n:]).all())
    c.check()


def _wide(lens, max_pages, wide_pages, **kw):
    c = Cache(lens, max_pages, **kw)
    narrow_acc, narrow = c.acc, c.cap
    c.table = _widen(c.table, wide_pages)
    c.cap = wide_pages * c.page
    c.acc = torch.full((c.B, c.Hkv, c.cap), float("nan"))
    c.acc[:, :, :narrow] = narrow_acc
    c.pos = torch.zeros(c.B, c.Hkv, c.cap, dtype=torch.int32)
    _positions(c)
    return c


@pytest.mark.parametrize("inplace", [True, False])
@pytest.mark.parametrize("B,Hkv,pages", [(2, 2, 4096), (4, 40, 1024), (40, 8, 1024)])
def test_evict_in_a_wide_table(cuda_lib, B, Hkv, pages, inplace):
    """Clusters of eight, CTAs whose segments lie past the rows, keys that fill the shared memory; rows within the
    budget beside rows past it."""
    lens = [[300, 2065, 40, 0][r % 4] for r in range(B)]
    c = _wide(lens, 260, pages, Hkv=Hkv, D=64, page=8, seed=B)
    c.evict(256, 4, 32, inplace)
    c.same()
    assert int(c.status.sum()) == 0


@pytest.mark.parametrize("Hkv,max_pages,budget", [(1, 600, 4000), (2, 1200, 3001), (4, 2500, 255), (3, 4200, 8190)])
def test_evict_to_other_arrays_by_clusters(cuda_lib, Hkv, max_pages, budget):
    """Separate outputs with the keys in the shared memory of two to eight CTAs: every slot below the budget is
    copied or moved, none past it is written."""
    n = max_pages * 8
    c = Cache([n, n - 5, min(n, budget + 1), budget // 2], max_pages, Hkv=Hkv, D=64, page=8, seed=max_pages)
    _positions(c)
    c.evict(budget, 4, 100, False)
    c.same()
    assert int(c.status.sum()) == 0


def test_append_to_a_wide_table(cuda_lib):
    c = _wide([5, 0, 61], 12, 4096, Hkv=2, D=64, page=8, seed=9)
    c.append(*c.rows(20), n_new=torch.tensor([20, 3, 0], dtype=torch.int32))
    c.same()
    assert int(c.status.sum()) == 0
