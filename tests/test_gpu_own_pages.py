"""A cache that gives its requests their pages, and what append brings: nothing reaches a page that is another request's."""
import pytest
import torch

from gpuhelp import dev

pytestmark = pytest.mark.gpu


def make(b, B=3, n_pages=12, **kw):
    c = b.PagedCache(B, 4, 2, 64, 8, 6, dev(), n_pages=n_pages, new_tokens=40, **kw)
    c.k_pool.normal_()
    c.v_pool.normal_()
    return c


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=dev())


def rows(B, n):
    return tuple(torch.randn(B, n, 2, 64, device=dev()).bfloat16() for _ in range(2))


@pytest.mark.parametrize("marshal", [True, False])
def test_a_request_that_has_ended_writes_nowhere(cuda_lib, monkeypatch, marshal):
    """Its pages have gone to another request, and its table still names them."""
    b = cuda_lib
    if not marshal:
        monkeypatch.setattr(b, "_marshal", None)
    c = make(b)
    c.reserve(20, i32([20, 5, 0]))
    c.seq_len[0] = 0
    c.reserve(30, i32([0, 27, 0]), trim=True)
    torch.cuda.synchronize()
    assert c.status.tolist() == [0, 0, 0] and c.held.tolist() == [0, 4, 0]
    theirs, table = set(c.page_table[1, :4].tolist()), c.page_table[0].tolist()
    assert theirs & set(table[:3])  # what makes it dangerous
    k, v, k0, v0 = *rows(3, 3), c.k_pool.clone(), c.v_pool.clone()
    c.append(k, v, n_new=i32([3, 0, 1]))
    torch.cuda.synchronize()
    assert c.status.tolist() == [256, 0, 256]
    assert c.seq_len.tolist() == [0, 32, 0] and c.n_seen.tolist() == [0, 0, 0]
    assert torch.equal(c.k_pool, k0) and torch.equal(c.v_pool, v0)
    # the request that holds its pages may fill them, up to their end and no further
    c.status.zero_()
    c.seq_len[1] = 30
    c.append(k, v, n_new=i32([0, 3, 0]))
    torch.cuda.synchronize()
    assert c.status.tolist() == [0, 256, 0] and torch.equal(c.k_pool, k0)
    c.status.zero_()
    c.append(k, v, n_new=i32([0, 2, 0]))
    torch.cuda.synchronize()
    page = int(c.page_table[1, 3])
    assert c.status.tolist() == [0, 0, 0] and c.seq_len.tolist() == [0, 32, 0]
    assert torch.equal(c.k_pool[page, 6:8], k[1, :2]) and torch.equal(c.v_pool[page, 6:8], v[1, :2])
    k0[page, 6:8], v0[page, 6:8] = k[1, :2], v[1, :2]
    assert torch.equal(c.k_pool, k0) and torch.equal(c.v_pool, v0)


@pytest.mark.parametrize("graph", [False, True])
def test_accepted_paths_enter_reserved_pages(cuda_lib, graph):
    """Pages for the longest path, the path itself by verify's list, and the pages that it did not need go back."""
    b = cuda_lib
    B, n_max, depth = 3, 16, 7
    c = make(b, B, 16)
    c.reserve(13, i32([13, 8, 0]))
    lens = [13, 8, 0]
    torch.cuda.synchronize()
    held = {(r, j): (c.k_pool[int(c.page_table[r, j // 8]), j % 8].clone(), c.v_pool[int(c.page_table[r, j // 8]), j % 8].clone())
            for r in range(B) for j in range(lens[r])}
    k, v = rows(B, n_max)
    path = torch.full((B, depth), -1, dtype=torch.int32, device=dev())

    def step():
        c.reserve(depth, trim=True, advance=False)
        c.append(k, v, rows=path)

    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
    gen = torch.Generator().manual_seed(5)
    for i in range(12):
        if i == 5:  # a request ends and starts anew
            c.seq_len[1] = 0
            held = {x: y for x, y in held.items() if x[0] != 1}
            lens[1] = 0
        new = [sorted(torch.randperm(n_max, generator=gen)[:int(torch.randint(0, depth + 1, (1,), generator=gen))].tolist())
               for _ in range(B)]
        if any(lens[r] + depth > 48 for r in range(B)):
            break
        path.copy_(torch.tensor([x + [-1] * (depth - len(x)) for x in new], dtype=torch.int32))
        for x in (k, v):
            x.normal_()
        g.replay() if graph else step()
        torch.cuda.synchronize()
        assert c.held.tolist() == [-(-(n + depth) // 8) for n in lens] and int(c.n_free) == 16 - sum(c.held.tolist())
        for r in range(B):
            for x in new[r]:
                held[r, lens[r]] = k[r, x].clone(), v[r, x].clone()
                lens[r] += 1
        assert c.seq_len.tolist() == lens and not bool(c.status.any())
        table = c.page_table.cpu()
        used = [p for r in range(B) for p in table[r, :int(c.held[r])].tolist()]
        assert len(set(used)) == len(used)
        for (r, j), (x, y) in held.items():
            p = int(table[r, j // 8])
            assert torch.equal(c.k_pool[p, j % 8], x) and torch.equal(c.v_pool[p, j % 8], y), (r, j)
    assert i >= 6


def test_counts_of_pages_that_cannot_be(cuda_lib):
    b = cuda_lib
    c = make(b)
    c.reserve(10)
    k, v = rows(3, 2)
    k0 = c.k_pool.clone()
    torch.cuda.synchronize()
    c.held.copy_(i32([-1, 7, 2]))
    c.append(k, v, n_new=i32([1, 2, 0]))
    torch.cuda.synchronize()
    assert c.status.tolist() == [64, 64, 0] and c.seq_len.tolist() == [10, 10, 10] and torch.equal(c.k_pool, k0)
    c.status.zero_()
    c.held.copy_(i32([2 ** 31 - 1, -2 ** 31, 0]))
    c.append(k, v, n_new=i32([0, 0, 0]))  # nothing to bring: nothing to say
    torch.cuda.synchronize()
    assert c.status.tolist() == [0, 0, 0] and c.seq_len.tolist() == [10, 10, 10]
