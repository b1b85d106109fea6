"""GPU parity of the norm and rotation of queries and keys with float64, and of what is stored with what is returned."""
import math

import pytest
import torch

import layerref as ref
from gpuhelp import dev

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


class Rope:
    def __init__(self, T, Hq, Hkv, D=128, dtype=BF, rot=None, interleaved=False, norm=True, factor=1.0, pos=None,
                 page=16, layout="slot", store=True, rows=True, fused=True, seed=0, base=1e6, eps=1e-6):
        from draft_tree_build_gb300 import bastion
        self.b = bastion
        g = torch.Generator().manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g).to(dtype).to(dev())  # noqa: E731
        if fused:
            x = rand(T, Hq + 2 * Hkv, D)
            self.q, self.k, self.v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        else:
            self.q, self.k, self.v = rand(T, Hq, D), rand(T, Hkv, D), rand(T, Hkv, D)
        self.rot = D if rot is None else rot
        self.kw = dict(interleaved=interleaved, factor=factor, eps=eps)
        self.qw = rand(D) if norm else None
        self.kw_ = rand(D) if norm else None
        if pos is None:
            pos = torch.randint(0, 1 << 20, (T,), generator=g)
        self.pos = torch.as_tensor(pos, dtype=torch.int32).to(dev())
        self.freq = None
        if self.rot:
            self.freq = base ** (-torch.arange(0, self.rot, 2, dtype=torch.float64, device=dev()) / self.rot)
        self.q_out = torch.full((T, Hq, D), 7.0, dtype=dtype, device=dev())
        self.k_out = torch.full((T, Hkv, D), 7.0, dtype=dtype, device=dev()) if rows else None
        self.pool = {}
        if store:
            n_pages = -(-T // page) + 2
            shape = (n_pages, page, Hkv, D) if layout == "slot" else (n_pages, Hkv, page, D)
            pools = [torch.full(shape, 9.0, dtype=dtype, device=dev()) for _ in range(2)]
            if layout == "head":
                pools = [x.transpose(1, 2) for x in pools]
            slots = torch.randperm(n_pages * page, generator=g)[:T]
            self.pool = dict(v=self.v, k_pool=pools[0], v_pool=pools[1], slots=slots.to(dev()))
        self.status = torch.zeros(1, dtype=torch.int32, device=dev())
        self.q0, self.k0, self.v0 = self.q.clone(), self.k.clone(), self.v.clone()

    def run(self, stream=None):
        self.b.bastion_qk_norm_rope(self.q, self.k, self.pos, self.freq, self.q_out, self.status, k_out=self.k_out,
                                    q_weight=self.qw, k_weight=self.kw_, stream=stream, **self.kw, **self.pool)
        return self

    def check(self):
        torch.cuda.synchronize()
        assert int(self.status) == 0
        on = self.pos >= 0
        args = (self.kw["eps"], self.pos, self.freq, self.rot, self.kw["interleaved"], self.kw["factor"])
        if self.q_out is not None:
            want, size = ref.norm_rope(self.q0, self.qw, *args)
            ref.check_norm_rope(self.q_out[on], want[on], size[on])
            if self.q_out.data_ptr() != self.q.data_ptr():
                assert bool((self.q_out[~on] == 7).all())
        want, size = ref.norm_rope(self.k0, self.kw_, *args)
        if self.k_out is not None:
            ref.check_norm_rope(self.k_out[on], want[on], size[on])
            if self.k_out.data_ptr() != self.k.data_ptr():
                assert bool((self.k_out[~on] == 7).all())
        if self.pool:
            page, slots = self.pool["k_pool"].shape[1], self.pool["slots"]
            on = on & (slots >= 0)
            at, slot = slots[on] // page, slots[on] % page
            ref.check_norm_rope(self.pool["k_pool"][at, slot], want[on], size[on])
            if self.k_out is not None:
                assert torch.equal(self.pool["k_pool"][at, slot], self.k_out[on])
            assert torch.equal(self.pool["v_pool"][at, slot], self.v0[on])
            for x in (self.pool["k_pool"], self.pool["v_pool"]):  # the other slots are left as they were
                x[at, slot] = 9.0
                assert bool((x == 9).all())


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D,rot", [(64, 64), (64, 0), (64, 16), (64, 48), (128, 128), (128, 64), (128, 96), (128, 32)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_layouts(cuda_lib, dtype, D, rot, interleaved, norm):
    Rope(37, 5, 3, D, dtype, rot, interleaved, norm, 1.0 if norm else 1.2, seed=rot + D).run().check()


@pytest.mark.parametrize("T", [1, 2, 3, 7, 63, 64, 65, 1000, 4099])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (32, 8), (7, 1), (14, 2), (3, 3), (80, 5)])
def test_tokens_and_heads(cuda_lib, T, Hq, Hkv):
    D = 64 if Hq == 14 else 128
    Rope(T, Hq, Hkv, D, seed=T + Hq, page=8, layout="head").run().check()


@pytest.mark.parametrize("store,rows", [(True, False), (False, True), (True, True)])
@pytest.mark.parametrize("page,layout", [(8, "slot"), (128, "head"), (32, "head"), (64, "slot")])
def test_outputs(cuda_lib, store, rows, page, layout):
    Rope(100, 8, 2, 128, HF, page=page, layout=layout, store=store, rows=rows, fused=False, seed=page).run().check()


def test_far_positions(cuda_lib):
    """The angle is reduced before it is rounded: the last positions of 31 bits are as exact as the first."""
    pos = [0, 1, 2, 100, 4095, 65537, 1 << 20, (1 << 24) + 1, (1 << 30) + 12345, (1 << 31) - 1, (1 << 31) - 2]
    for inter in (False, True):
        r = Rope(len(pos), 4, 2, 128, HF, interleaved=inter, pos=pos, base=10000.0)
        # float64 products of position and frequency are off by 2^-22 of a radian at 2^31: exactly, instead
        r.run()
        torch.cuda.synchronize()
        r.freq = (r.freq * 2 ** 40).round() / 2 ** 40
        r.run()
        t = [[(p * int(f * 2 ** 40)) / 2 ** 40 for f in r.freq.tolist()] for p in pos]
        x = r.q0.double()
        y = x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + 1e-6) * r.qw.double()
        i = torch.arange(64, device=dev())
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + 64)
        c = torch.tensor([[math.cos(v) for v in row] for row in t], dtype=torch.float64, device=dev())[:, None]
        s = torch.tensor([[math.sin(v) for v in row] for row in t], dtype=torch.float64, device=dev())[:, None]
        want, size = torch.empty_like(y), torch.empty_like(y)
        want[..., a], want[..., b] = y[..., a] * c - y[..., b] * s, y[..., b] * c + y[..., a] * s
        size[..., a] = size[..., b] = y[..., a].abs() + y[..., b].abs()
        torch.cuda.synchronize()
        # the frequency, 2 pi away from its fraction of a turn, is held to 2^-53 of itself: 2^-21 radians at 2^31
        ref.check_norm_rope(r.q_out, want, size * 5)


def test_negative_positions_and_slots(cuda_lib):
    r = Rope(50, 8, 2, pos=[(-1) ** (i % 3 == 0) * (i + 1) for i in range(50)])
    r.pool["slots"][1::4] = -1
    r.run().check()
    r = Rope(5, 8, 2, pos=[-1] * 5)
    r.run().check()


def test_slots_past_the_pools(cuda_lib):
    r = Rope(6, 8, 2)
    n = r.pool["k_pool"].shape[0] * 16
    for bad in (n, n + 1, 1 << 40, (1 << 63) - 1):
        r.status.zero_()
        r.pool["slots"][2] = bad
        r.run()
        torch.cuda.synchronize()
        assert int(r.status) == 64
    r.status.zero_()
    r.pool["slots"][2] = -5
    r.check()


def test_in_place(cuda_lib):
    r = Rope(300, 14, 2, 64, HF, interleaved=True, fused=True)
    r.q_out, r.k_out = r.q, r.k
    r.run().check()
    assert torch.equal(r.v, r.v0)


def test_strides(cuda_lib):
    """Rows far apart, heads far apart, one token's rows for all."""
    r = Rope(20, 4, 2, fused=False)
    wide = torch.zeros(20, 9, 4, 136, dtype=BF, device=dev())
    wide[:, 3, :, :128] = r.q0
    r.q = wide[:, 3, :, :128]
    r.k = r.k0[:1].expand(20, 2, 128)
    r.k0 = r.k.clone()
    out = torch.full((20, 2, 4, 128), 7.0, dtype=BF, device=dev())
    r.q_out = out[:, 1]
    r.run().check()
    assert bool((out[:, 0] == 7).all())


def test_values_at_the_ends(cuda_lib):
    """Zeros, infinities and NaN stay in their heads; what is not turned is not mixed."""
    for norm in (False, True):
        r = Rope(4, 4, 2, 128, BF, rot=64, norm=norm, store=False)
        r.q[0, 0] = 0
        r.q[1, 1, 100] = math.inf
        r.q[2, 2, 3] = math.nan
        r.q0 = r.q.clone()
        r.run()
        torch.cuda.synchronize()
        assert bool((r.q_out[0, 0] == 0).all())
        if norm:
            assert bool(r.q_out[2, 2].isnan().all())
        else:
            assert float(r.q_out[1, 1, 100]) == math.inf and int(r.q_out[1, 1].isfinite().sum()) == 127
            assert r.q_out[2, 2].isnan().nonzero().flatten().tolist() == [3, 35]
        clean = torch.ones(4, 4, dtype=torch.bool, device=dev())
        clean[1, 1] = clean[2, 2] = False
        assert bool(r.q_out[clean].isfinite().all())


def test_many_tokens_and_32_bit_offsets(cuda_lib):
    """More than 2^31 elements between the first token and the last."""
    T, H = 40, 2
    big = torch.zeros(T, 1 << 26, dtype=BF, device=dev())
    r = Rope(T, H, 1, store=False, fused=False)
    r.q = big[:, :H * 128].view(T, H, 128)
    r.q.copy_(r.q0)
    r.q_out = big[:, 1024:1024 + H * 128].view(T, H, 128)
    r.q_out.fill_(7.0)
    r.run().check()


def test_streams_and_graphs(cuda_lib):
    a, b = Rope(500, 8, 2), Rope(3, 4, 4, 64, HF)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        a.run(s1)
        b.run(s2)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.run()
        b.run()
    a.q.normal_()
    a.pos.random_(0, 1000)
    a.q0 = a.q.clone()
    torch.cuda.synchronize()
    g.replay()
    a.check()
    b.check()


@pytest.mark.parametrize("scaling", [None, "linear", "base", "bands", "yarn"])
def test_scaled_frequencies(cuda_lib, scaling):
    from draft_tree_build_gb300 import bastion
    kw = dict(low=1.0, high=32.0) if scaling == "yarn" else {}
    r = Rope(64, 4, 2, norm=False)
    r.freq, size = bastion.rope_frequencies(128, 5e5, dev(), scaling, 8.0, **kw)
    r.kw["factor"] = size
    r.run().check()
