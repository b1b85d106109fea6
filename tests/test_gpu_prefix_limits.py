"""Shared-prefix attention where there is nothing to attend to, and at its limits of heads and groups."""
import math

import pytest
import torch

import layerref as ref
import pagedref
from gpuhelp import dev
from test_gpu_prefix import BF, HF, Prefix

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=dev())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("plens,lens", [([0, 0], [0] * 5), ([0, 0], [3, 0, 9, 1, 0]), ([40, 0], [0] * 5), ([0], [17])])
def test_empty_prefixes_and_empty_own_slots(cuda_lib, D, wide, plens, lens):
    p = Prefix(plens, [3, 2] if len(plens) == 2 else [1], lens, 8, 2, D, 8, seed=D, poison=math.nan)
    if wide:  # own slots by the one-token kernel
        t = torch.full((len(lens), 200), -1, dtype=torch.int32)
        t[:, :p.table_h.shape[1]] = p.table_h
        p.table_h, p.table = t, t.to(dev())
    p.run().check()
    nothing = [r for r, n in enumerate(lens) if n == 0 and not (r < 3 and plens[0])]
    assert bool((p.out[nothing] == 0).all()) and bool(torch.isneginf(p.lse[nothing]).all())


def test_more_groups_than_requests(cuda_lib):
    """1,024 groups of which three have a request each."""
    start = [0] * 300 + [1] * 400 + [2] * 100 + [3] * 225
    plens = [(37 * g) % 200 for g in range(1024)]
    p = Prefix([plens[299], plens[699], plens[799]], [1, 1, 1], [5, 0, 70], 8, 2, 128, 16, seed=2)
    p.run().check()
    table = torch.full((1024, p.prefix_table.shape[1]), 2 ** 31 - 1, dtype=torch.int32, device=dev())
    table[[299, 699, 799]] = p.prefix_table
    out, lse = torch.zeros_like(p.out), torch.zeros_like(p.lse)
    ws = p.b.workspace(p.b.bastion_paged_prefix_attention_workspace_bytes(3, 8, 2, 128, 1024), dev())
    p.b.bastion_paged_prefix_attention(p.q, p.k, p.v, p.table, p.seq_len, table, i32(plens), i32(start), p.scale, out, ws,
                                       p.status, lse=lse)
    torch.cuda.synchronize()
    assert not bool(p.status.any()) and torch.equal(out, p.out) and torch.equal(lse, p.lse)


def test_without_the_logarithms(cuda_lib):
    p = Prefix([300], [6], [30] * 6, 8, 2, dtype=HF, seed=6)
    p.run().check()
    out = torch.zeros_like(p.out)
    p.b.bastion_paged_prefix_attention(p.q, p.k, p.v, p.table, p.seq_len, p.prefix_table, p.prefix_len, p.group_start, p.scale,
                                       out, p.ws, p.status)
    torch.cuda.synchronize()
    assert torch.equal(out, p.out)


@pytest.mark.parametrize("B,Hkv,G", [(1023, 64, 1), (1, 65535, 1), (3, 21845, 2), (4095 // 16, 256, 16)])
def test_as_many_heads_as_there_can_be(cuda_lib, B, Hkv, G):
    """B * Hkv up to 65,535; a few of the heads in 64 bits, the rest by their being those of the same inputs."""
    b, D, page, P, own = cuda_lib, 64, 8, 21, 5
    g = torch.Generator("cuda").manual_seed(B)
    same = max(1, Hkv // 5)  # heads repeat after so many
    n = 3 + B
    k, v = (torch.randn(n, page, same, D, generator=g, device=dev()).to(BF).repeat(1, 1, -(-Hkv // same), 1)[:, :, :Hkv].contiguous()
            for _ in range(2))
    q = (2 * torch.randn(B, same, G, D, generator=g, device=dev())).to(BF).repeat(1, -(-Hkv // same), 1, 1)[:, :Hkv]
    q = q.reshape(B, Hkv * G, D).contiguous()
    table, prefix = i32([[3 + r] for r in range(B)]), i32([[2, 0, 1]])
    lens = [(r * 3) % (own + 1) for r in range(B)]
    out, lse, status = torch.full_like(q, 7.0), torch.full((B, Hkv * G), 7.0, device=dev()), i32([0] * B)
    ws = b.workspace(b.bastion_paged_prefix_attention_workspace_bytes(B, Hkv * G, Hkv, D, 1), dev())
    b.bastion_paged_prefix_attention(q, k, v, table, i32(lens), prefix, i32([P]), i32([0, B]), ref.scale_of(D), out, ws, status,
                                     lse=lse)
    torch.cuda.synchronize()
    assert not bool(status.any())
    out, lse = out.view(B, Hkv, G, D), lse.view(B, Hkv, G)
    for h in range(same, Hkv, same):
        w = min(same, Hkv - h)
        assert torch.equal(out[:, h:h + w], out[:, :w]) and torch.equal(lse[:, h:h + w], lse[:, :w])
    few = sorted({0, 1 % same, same // 2, same - 1})
    kk, vv, t, total = ref.joined(k[:, :, few], v[:, :, few], table.cpu(), lens, prefix.cpu(), [P], [0, B])
    pagedref.check_attention(out[:, few].reshape(B, -1, D).contiguous(), lse[:, few].reshape(B, -1),
                             q.view(B, Hkv, G, D)[:, few].reshape(B, -1, D), kk, vv, t, total, ref.scale_of(D))
