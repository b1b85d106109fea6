"""Shared prefixes so long that a CTA's sums are formed in several chains of products."""
import math

import pytest
import torch

import layerref as ref
import pagedref
from gpuhelp import dev
from test_gpu_prefix import BF, HF, Prefix

pytestmark = pytest.mark.gpu


def check_by_group(p):
    torch.cuda.synchronize()
    assert int(p.status.abs().sum()) == 0
    for i, n in enumerate(p.plens):
        a, b = p.start[i], p.start[i + 1]
        if a == b:
            continue
        k, v, t, lens = ref.joined(p.k, p.v, p.table_h[a:b], p.lens[a:b], p.prefix_h[i:i + 1], [n], [0, b - a])
        pagedref.check_attention(p.out[a:b].contiguous(), p.lse[a:b], p.q[a:b], k, v, t, lens, p.scale)


def raise_late(p, at, dtype):
    """Keys of every prefix along one of its queries, longer ones further on: maxima that move from chain to chain."""
    H, page = p.k.shape[2], p.k.shape[1]
    G = p.q.shape[1] // H
    for i, n in enumerate(p.plens):
        for x, (j, f) in enumerate(at):
            if j < n:
                q = p.q[p.start[i]].view(H, G, -1)[:, x % G].float()
                p.k[int(p.prefix_h[i, j // page]), j % page] = (f * q / 16).to(dtype)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_chains_of_one_m_tile(cuda_lib, dtype):
    """Two warpgroups in turn: chains of 128 key tiles, and one more, or one less."""
    plens = [16384, 16385, 16383, 16500, 16256, 33000, 129, 12800, 32768, 16512] * 10
    p = Prefix(plens, [1] * 100, [(7 * r) % 40 for r in range(100)], 4, 2, 64, 64, "head", dtype, seed=3, poison=math.nan)
    raise_late(p, [(100, 3.0), (16300, 5.0), (16383, 7.0), (16400, 9.0), (32700, 12.0)], dtype)
    p.run()
    check_by_group(p)


@pytest.mark.parametrize("dtype,D", [(BF, 128), (HF, 64)])
def test_chains_of_two_m_tiles(cuda_lib, dtype, D):
    """A warpgroup an M tile: chains of 64 key tiles; the second M tile has one request."""
    plens = [8192, 8193, 8191, 8320, 16500, 24700, 8064, 100, 16384, 8256] * 6
    p = Prefix(plens, [9] * 60, [(5 * r) % 50 for r in range(540)], 32, 2, D, 32, "slot", dtype, seed=4, poison=math.nan)
    raise_late(p, [(50, 3.0), (8150, 5.0), (8191, 7.0), (8192, 9.0), (16390, 11.0), (24600, 13.0)], dtype)
    p.run()
    check_by_group(p)


def test_long_sums_are_not_cut_short(cuda_lib):
    """The outputs' mean error in their own direction, over 800,000 tokens and 256 rows a KV head.  A chain has at most
    64 * 16 sums, each cut by at most 2^-23 of itself, half of that on average, and half of that again as a sum that grows
    evenly is on average half of what it becomes: 2^-15.  The roundings of 131,072 outputs add 2^-12 / 362, 2^-20.5, to it,
    and the other roundings to 32 bits have no direction."""
    page, P, B, Hq, Hkv, D = 128, 800_000, 16, 128, 8, 64
    b, g = cuda_lib, torch.Generator("cuda").manual_seed(1)
    n = P // page
    k, v = (torch.empty(n, page, Hkv, D, dtype=HF, device=dev()).normal_(generator=g) for _ in range(2))
    q = torch.empty(B, Hq, D, dtype=HF, device=dev()).normal_(generator=g)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev())  # noqa: E731
    table = torch.randperm(n, device=dev()).to(torch.int32)[None].contiguous()
    out, status = torch.zeros_like(q), i32([0] * B)
    ws = b.workspace(b.bastion_paged_prefix_attention_workspace_bytes(B, Hq, Hkv, D, 1), dev())
    b.bastion_paged_prefix_attention(q, k, v, i32([[0]] * B), i32([0] * B), table, i32([P]), i32([0, B]), ref.scale_of(D), out,
                                     ws, status)
    torch.cuda.synchronize()
    assert not bool(status.any())
    got = out.double().view(B, Hkv, Hq // Hkv, D)
    along = size = 0.0
    for h in range(Hkv):
        x = q.view(B, Hkv, Hq // Hkv, D)[:, h].reshape(-1, D).double()
        s = torch.softmax(x @ k[:, :, h].reshape(-1, D).double().T * ref.scale_of(D), -1)
        want = (s @ v[:, :, h].reshape(-1, D).double()).view(B, -1, D)
        along += float(((got[:, h] - want) * want).sum())
        size += float((want * want).sum())
    assert abs(along / size) <= 2.0 ** -15 + 2.0 ** -20, along / size
