"""Calls that follow one another without a pause, each reading what the one before wrote."""
import pytest
import torch

import layerref as ref
import pagedref
from gpuhelp import dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("own", [40, 300])
@pytest.mark.parametrize("graph", [False, True])
def test_prefixes_that_grow_between_calls(cuda_lib, own, graph):
    """The page plan lengthens the groups' prefixes, in place, and the attention behind it reads their new lengths and
    pages; own slots on both sides of the two kernels' border."""
    b, page, B, Hq, Hkv, D, steps = cuda_lib, 16, 9, 8, 2, 128, 24
    g = torch.Generator().manual_seed(own)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev())  # noqa: E731
    grow, wide = [37, 5, 61], 100
    n_pages = 3 * wide + B * 20
    k, v = (pagedref.make_pool(n_pages, page, Hkv, D, torch.bfloat16, "slot", g, dev()) for _ in range(2))
    ids = torch.randperm(n_pages, generator=g).to(torch.int32)
    table_h = ids[:B * 20].view(B, 20).contiguous()
    lens = [(own + 7 * r) % (own + 1) for r in range(B)]
    table, seq_len, start = table_h[:, :-(-own // page)].contiguous().to(dev()), i32(lens), i32([0, 4, 5, 8])
    prefix, plen, held, n_free = i32([[-1] * wide] * 3), i32([0, 0, 0]), i32([0, 0, 0]), i32([3 * wide])
    stack = torch.cat([ids[B * 20:], torch.zeros(B * 20, dtype=torch.int32)]).to(dev())
    new, slots = i32(grow), torch.zeros(3 * 64, dtype=torch.int64, device=dev())
    pos, status, plan_status = torch.zeros(3 * 64, dtype=torch.int32, device=dev()), i32([0] * B), i32([0] * 3)
    q = (2 * torch.randn(B, Hq, D, generator=g)).bfloat16().to(dev())
    outs = [torch.zeros_like(q) for _ in range(steps)]
    lses = [torch.zeros(B, Hq, device=dev()) for _ in range(steps)]
    ws = b.workspace(b.bastion_paged_prefix_attention_workspace_bytes(B, Hq, Hkv, D, 3), dev())
    ws_plan = b.workspace(b.bastion_paged_plan_workspace_bytes(3), dev())

    def run():
        for out, lse in zip(outs, lses):
            b.bastion_paged_plan(prefix, page, plen, 64, held, held, stack, n_free, n_free, slots, pos, ws_plan, plan_status,
                                 n_new=new, seq_len_out=plen)
            b.bastion_paged_prefix_attention(q, k, v, table, seq_len, prefix, plen, start, ref.scale_of(D), out, ws, status,
                                             lse=lse)

    torch.cuda.synchronize()
    if graph:
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg):
            run()
        cg.replay()
    else:
        run()
    torch.cuda.synchronize()
    assert not bool(status.any()) and not bool(plan_status.any()) and plen.tolist() == [steps * x for x in grow]
    prefix_h = prefix.cpu()
    for i, (out, lse) in enumerate(zip(outs, lses)):
        kk, vv, t, n = ref.joined(k, v, table_h, lens, prefix_h, [(i + 1) * x for x in grow], [0, 4, 5, 8])
        pagedref.check_attention(out, lse, q, kk, vv, t, n, ref.scale_of(D))
