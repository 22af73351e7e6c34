"""smcsd_qk_norm_rope against the definition in 64 bits.

Bound on an element: its rounding u|y| (u = finfo.eps / 2) plus half the smallest subnormal,
and the fp32 steps before it: the sum of squares (at most D + 8 roundings, halved by the root),
root, division and two products (8), and the rotation's products and sum (3) on both elements of
the pair: (D / 2 + 16) 2^-24 (|a| + |b|)."""
import pytest
import torch

import smc_verification_resampling_amd as sm

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
SUB = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25}


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


class Case:
    def __init__(self, dt="bf16", S=3, R=4, Hq=6, Hkv=2, D=64, rot=64, bs=16, lens=(5, 30, 0), interleaved=False, norm=(True, True),
                 layout="token", positions=False, nodes=None, seed=0, max_pos=200, fused=True, eps=1e-6):
        g = torch.Generator().manual_seed(seed)
        self.dt, self.S, self.R, self.Hq, self.Hkv, self.D, self.rot, self.bs = dt, S, R, Hq, Hkv, D, rot, bs
        self.interleaved, self.eps = interleaved, eps
        self.lens = [lens[i % len(lens)] for i in range(S)]
        M = max(-(-(x + R) // bs) for x in self.lens)
        P = S * M + 2
        self.tables = torch.randperm(P, generator=g)[: S * M].view(S, M).int().cuda()
        qkv = torch.randn((S, R, Hq + 2 * Hkv, D), generator=g).to(DT[dt]).cuda()
        self.q, self.k, self.v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
        if not fused:
            self.q, self.k, self.v = (t.contiguous() for t in (self.q, self.k, self.v))
        self.w = [(1 + 0.3 * torch.randn(D, generator=g)).to(DT[dt]).cuda() if n else None for n in norm]
        a = torch.rand((max_pos, max(rot // 2, 1)), generator=g, dtype=torch.float64) * 6.283
        self.cs = torch.cat([a.cos(), a.sin()], 1).float().cuda() if rot else None
        self.positions = torch.randint(0, max_pos, (S, R), generator=g).int().cuda() if positions else None
        self.nodes = nodes
        self.nodes_t = None if nodes is None else torch.tensor([nodes[i % len(nodes)] for i in range(S)], dtype=torch.int32, device="cuda")
        shape = (P, bs, Hkv, D) if layout == "token" else (P, Hkv, bs, D)
        kv = [torch.full(shape, 7.0, dtype=DT[dt], device="cuda") for _ in range(2)]
        self.kc, self.vc = kv if layout == "token" else [x.transpose(1, 2) for x in kv]
        self.lens_t = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.q_out = torch.full((S, R, Hq, D), 7.0, dtype=DT[dt], device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call(self, **kw):
        a = dict(q_weight=self.w[0], k_weight=self.w[1], eps=self.eps, cos_sin=self.cs, interleaved=self.interleaved,
                 positions=self.positions, num_nodes=self.nodes_t)
        a.update(kw)
        sm.qk_norm_rope(self.q, self.k, self.v, self.lens_t, self.tables, self.kc, self.vc, self.q_out, self.status, **a)
        return self

    def want(self, x, w, pos):
        """One token's heads [H, D] and what their roundings may add."""
        x = x.double()
        if w is not None:
            x = x / (x.square().mean(-1, keepdim=True) + self.eps).sqrt() * w.double()
        y, size = x.clone(), x.abs()
        if self.rot:
            h = self.rot // 2
            c, s = self.cs[pos, :h].double(), self.cs[pos, h:].double()
            i = torch.arange(h, device="cuda")
            lo, hi = (2 * i, 2 * i + 1) if self.interleaved else (i, i + h)
            y[:, lo], y[:, hi] = x[:, lo] * c - x[:, hi] * s, x[:, hi] * c + x[:, lo] * s
            size[:, lo] = size[:, hi] = x[:, lo].abs() + x[:, hi].abs()
        u = torch.finfo(DT[self.dt]).eps / 2
        exact = w is None and not self.rot
        return y, (0 if exact else u * y.abs() + SUB[self.dt] + (self.D / 2 + 16) * 2.0 ** -24 * size)

    def check(self, skip=()):
        kc = torch.full_like(self.kc, 7.0)
        seen = torch.zeros(self.kc.shape[:2], dtype=torch.bool, device="cuda")
        for s in range(self.S):
            for j in range(self.R):
                if (s, j) in skip or (self.nodes is not None and j >= self.nodes[s % len(self.nodes)]):
                    assert (self.q_out[s, j] == 7).all()
                    continue
                p = self.lens[s] + j
                pos = int(self.positions[s, j]) if self.positions is not None else p
                at = int(self.tables[s, p // self.bs]), p % self.bs
                seen[at] = True
                for got, x, w in ((self.q_out[s, j], self.q[s, j], self.w[0]), (self.kc[at], self.k[s, j], self.w[1])):
                    y, tol = self.want(x, w, pos)
                    err = (got.double() - y).abs()
                    assert (err <= tol).all(), (s, j, float((err / tol).max()) if not isinstance(tol, int) else float(err.max()))
                assert torch.equal(self.vc[at], self.v[s, j])
        assert (self.kc[~seen] == 7).all() and (self.vc[~seen] == 7).all()
        return self


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(8, 0), (16, 16), (64, 64), (64, 32), (80, 80), (80, 32), (128, 128), (128, 64), (136, 112), (192, 64), (256, 256)])
def test_head_sizes_and_rotations(dt, interleaved, D, rot):
    c = Case(dt, D=D, rot=rot, interleaved=interleaved).call().check()
    assert int(c.status) == 0


@pytest.mark.parametrize("norm", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("rot", [0, 64])
def test_without_norms(norm, rot):
    c = Case(norm=norm, rot=rot, fused=False).call().check()
    assert int(c.status) == 0


@pytest.mark.parametrize("S,R,Hq,Hkv", [(1, 1, 1, 1), (1, 1, 32, 8), (7, 1, 3, 3), (2, 64, 5, 1), (40, 5, 8, 2)])
@pytest.mark.parametrize("layout", ["token", "head"])
@pytest.mark.parametrize("bs", [1, 5, 16])
def test_shapes(S, R, Hq, Hkv, layout, bs):
    c = Case(S=S, R=R, Hq=Hq, Hkv=Hkv, layout=layout, bs=bs, lens=(0, 3, 11, 30)).call().check()
    assert int(c.status) == 0


def test_given_positions_and_ragged_nodes():
    c = Case(S=5, R=6, positions=True, nodes=(6, 0, 2), layout="head").call().check()
    assert int(c.status) == 0


def test_small_and_large_values():
    c = Case("f16", S=2)
    c.q[0] *= 1e-4  # squares below fp16's range, not fp32's
    c.k[1] *= 200.0
    c.call().check()
    c = Case("bf16", S=2, eps=0.0)
    c.q[0] *= 1e15
    c.call().check()


def test_in_place():
    c = Case(fused=False)
    want = Case(fused=False).call()
    c.q_out = c.q
    c.call()
    assert torch.equal(c.q, want.q_out) and torch.equal(c.kc, want.kc)


def test_bad_indexes_leave_the_token_alone():
    for what in ("page", "page2", "length", "negative", "position", "position2"):
        c = Case(S=3, R=2, lens=(14, 20, 3), positions=True)
        skip = [(1, 0), (1, 1)]
        if what == "page":
            c.tables[1, 1] = c.kc.shape[0]
        elif what == "page2":
            c.tables[1, 1] = -1
        elif what == "length":
            c.lens_t[1] = 10 ** 9
        elif what == "negative":
            c.lens_t[1] = -5
        else:
            c.positions[1, 1] = 200 if what == "position" else -1
            skip = [(1, 1)]
        c.call()
        c.check(skip=skip)
        assert int(c.status) == sm.ST_BAD_INPUT, what


def test_another_stream_and_graph_replays():
    c = Case(S=6, R=5, lens=(9, 33))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    c.call(stream=st)
    st.synchronize()
    c.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call()
    for k in range(3):
        c.q.copy_(torch.randn_like(c.q))
        c.k.copy_(torch.randn_like(c.k))
        c.kc.fill_(7)
        c.vc.fill_(7)
        c.lens = [x + 1 for x in c.lens]
        c.lens_t += 1
        g.replay()
        torch.cuda.synchronize()
        c.check()
        torch.randn(1000, device="cuda").sum()


def test_pages_past_32_bits():
    page = 1 << 31
    buf = torch.empty(2 * page + (1 << 20), dtype=torch.bfloat16, device="cuda")
    c = Case(S=1, R=4, lens=(14,))
    c.kc = buf.as_strided((3, 16, 2, 64), (page, 128, 64, 1))
    c.vc = buf.as_strided((3, 16, 2, 64), (page, 128, 64, 1), 1 << 16)
    c.kc.fill_(7)
    c.vc.fill_(7)
    c.tables = torch.tensor([[1, 2]], dtype=torch.int32, device="cuda")
    c.call().check()


def test_refusals():
    c = Case()
    for kw in (dict(q_weight=c.w[0][:32]), dict(q_weight=c.w[0].float()), dict(cos_sin=c.cs.double()), dict(cos_sin=c.cs[0]),
               dict(cos_sin=c.cs[:, :24].contiguous()), dict(positions=torch.zeros(2, dtype=torch.int32, device="cuda")),
               dict(num_nodes=torch.zeros(3, dtype=torch.int64, device="cuda")), dict(eps=-1.0)):
        with pytest.raises(sm.SmcsdError):
            c.call(**kw)
    for name, val in (("q", c.q.transpose(1, 2)), ("k", c.k[..., :32]), ("v", c.v[:, :, :1]), ("kc", c.kc.float()), ("kc", c.kc[:, ::2]),
                      ("q_out", c.q_out[:1]), ("tables", c.tables[:2]), ("q", c.q.float()), ("kc", c.kc[..., :32])):
        d = Case()
        setattr(d, name, val)
        with pytest.raises(sm.SmcsdError):
            d.call()
