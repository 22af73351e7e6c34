"""smcsd_kv_append against the definition in 64 bits.

Bound on a 16-bit element, as in smcsd_qk_norm_rope's tests: its rounding u|y| (u = finfo.eps / 2)
plus half the smallest subnormal, and the fp32 steps before it, f = (D / 2 + 16) 2^-24 (|a| + |b|)
on both elements of the pair.  An 8-bit element in units of its scale 2^(x - 127), which divides
exactly: half a step 2^-4 |y| + 2^-10, and f in those units.  The scale's code is that of the
largest magnitude, which f may move too.  Values (no norm, no rotation) are exact in both kinds:
they have to be the correctly rounded bits, and their codes the definition's.  Older tokens that
follow a grown scale are the correctly rounded bits too."""
import math

import pytest
import torch

import smc_verification_resampling_amd as sm
from attention_checks import DT, E4M3, SUB, on_gpu

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def code_of(top):
    """The least code in [1, 247] whose scale holds `top` within 448."""
    m, e = math.frexp(top)
    return 1 if top == 0 else max(1, min(247, (e - 9 if m <= 0.875 else e - 8) + 127))


class Case:
    def __init__(self, dt="bf16", e4m3=True, new=(5, 30, 0, 2), ctx=(3, 0, 17), S=4, Hq=6, Hkv=2, D=64, rot=64, bs=16, interleaved=False,
                 norm=(True, True), layout="token", positions=False, seed=0, max_pos=400, before=0, behind=0, fused=True, size=1.0, queries=True,
                 no_ctx=False):
        g = torch.Generator().manual_seed(seed)
        self.dt, self.e4m3, self.S, self.Hq, self.Hkv, self.D, self.rot, self.bs = dt, e4m3, S, Hq, Hkv, D, rot, bs
        self.interleaved, self.eps = interleaved, 1e-6
        self.new = [new[i % len(new)] for i in range(S)]
        self.ctx = [0 if no_ctx else ctx[i % len(ctx)] for i in range(S)]
        M = max(-(-(c + n) // bs) for c, n in zip(self.ctx, self.new)) or 1
        P = S * M + 2
        self.tables = torch.randperm(P, generator=g)[: S * M].view(S, M).int().cuda()
        cu = [before]
        for n in self.new:
            cu.append(cu[-1] + n)
        self.cu, self.T = cu, cu[-1] + behind
        self.cu_t = torch.tensor(cu, **I32)
        self.ctx_t = None if no_ctx else torch.tensor(self.ctx, **I32)
        qkv = (size * torch.randn((self.T, Hq + 2 * Hkv, D), generator=g)).to(DT[dt]).cuda()
        self.q, self.k, self.v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        if not fused:
            self.q, self.k, self.v = (t.contiguous() for t in (self.q, self.k, self.v))
        self.w = [(1 + 0.3 * torch.randn(D, generator=g)).to(DT[dt]).cuda() if n else None for n in norm]
        a = torch.rand((max_pos, max(rot // 2, 1)), generator=g, dtype=torch.float64) * 6.283
        self.cs = torch.cat([a.cos(), a.sin()], 1).float().cuda() if rot else None
        self.positions = torch.randint(0, max_pos, (self.T,), generator=g).int().cuda() if positions else None
        shape = (P, bs, Hkv, D) if layout == "token" else (P, Hkv, bs, D)
        kv = [torch.randint(0, 127, shape, generator=g, dtype=torch.uint8).view(E4M3) if e4m3 else torch.randn(shape, generator=g).to(DT[dt]) for _ in range(2)]
        kv = [x if layout == "token" else x.transpose(1, 2) for x in kv]
        self.was = [on_gpu(x) for x in kv]
        self.kc, self.vc = (on_gpu(x) for x in kv)
        codes = [torch.randint(110, 125, (P, Hkv), generator=g, dtype=torch.uint8).cuda() for _ in range(2)] if e4m3 else [None, None]
        self.codes_were = codes
        self.sk, self.sv = [None if c is None else c.clone() for c in codes]
        self.q_out = torch.full((self.T, Hq, D), 7.0, dtype=DT[dt], device="cuda") if queries else None
        self.status = torch.zeros(1, **I32)

    def call(self, **kw):
        a = dict(k_scales=self.sk, v_scales=self.sv, q_weight=self.w[0], k_weight=self.w[1], eps=self.eps, cos_sin=self.cs, interleaved=self.interleaved,
                 positions=self.positions)
        a.update(kw)
        sm.kv_append(self.q if self.q_out is not None else None, self.k, self.v, self.cu_t, self.ctx_t, self.tables, self.kc, self.vc, self.q_out, self.status, **a)
        return self

    def want(self, x, w, pos):
        """Tokens' heads [n, H, D] in 64 bits, and what the fp32 steps may add."""
        x = x.double()
        if w is not None:
            x = x / (x.square().mean(-1, keepdim=True) + self.eps).sqrt() * w.double()
        y, size = x.clone(), x.abs()
        if self.rot:
            h = self.rot // 2
            c, s = self.cs[pos, :h].double()[:, None], self.cs[pos, h:].double()[:, None]
            i = torch.arange(h, device="cuda")
            lo, hi = (2 * i, 2 * i + 1) if self.interleaved else (i, i + h)
            y[..., lo], y[..., hi] = x[..., lo] * c - x[..., hi] * s, x[..., hi] * c + x[..., lo] * s
            size[..., lo] = size[..., hi] = x[..., lo].abs() + x[..., hi].abs()
        exact = w is None and not self.rot
        return y, size * (0 if exact else (self.D / 2 + 16) * 2.0 ** -24)

    def check(self, skip=(), skip_kv=(), status=0):
        """skip: tokens that are left alone altogether; skip_kv: those whose queries alone are written."""
        assert int(self.status) == status
        real = [(s, i) for s in range(self.S) for i in range(self.new[s]) if self.cu[s] + i not in skip]
        t = torch.tensor([self.cu[s] + i for s, i in real], device="cuda", dtype=torch.long)
        at = [(s, self.ctx[s] + i) for s, i in real]
        pos = self.positions[t].long() if self.positions is not None else torch.tensor([p for _, p in at], device="cuda", dtype=torch.long)
        if self.q_out is not None:
            rest = torch.ones(self.T, dtype=torch.bool, device="cuda")
            rest[t] = False
            assert (self.q_out[rest] == 7).all()
            if len(real):
                y, f = self.want(self.q[t], self.w[0], pos)
                tol = 0 if self.w[0] is None and not self.rot else torch.finfo(DT[self.dt]).eps / 2 * y.abs() + SUB[self.dt] + f
                assert ((self.q_out[t].double() - y).abs() <= tol).all()
        keep = [n for n, (s, i) in enumerate(real) if self.cu[s] + i not in skip_kv]
        t, pos, at = t[keep], pos[keep], [at[n] for n in keep]
        block = torch.tensor([int(self.tables[s, p // self.bs]) for s, p in at], device="cuda", dtype=torch.long)
        off = torch.tensor([p % self.bs for _, p in at], device="cuda", dtype=torch.long)
        for x, cache, was, codes, codes_were, w, turned in ((self.k, self.kc, self.was[0], self.sk, self.codes_were[0], self.w[1], True),
                                                            (self.v, self.vc, self.was[1], self.sv, self.codes_were[1], None, False)):
            y, f = (self.want(x[t], w, pos) if turned else (x[t].double(), torch.zeros((), device="cuda", dtype=torch.float64)))
            exact = not turned or (w is None and not self.rot)
            if not self.e4m3:
                got, expect = cache.clone(), was.clone()
                new = got[block, off].double()
                tol = 0 if exact else torch.finfo(DT[self.dt]).eps / 2 * y.abs() + SUB[self.dt] + f
                assert ((new - y).abs() <= tol).all()
                got[block, off] = 0
                expect[block, off] = 0
                assert torch.equal(got, expect)
                continue
            got, expect = cache.view(torch.uint8).clone(), was.view(torch.uint8).clone()
            expect_codes = codes_were.clone()
            f = f.expand(y.shape) if f.dim() else torch.zeros_like(y)
            fine = y.isfinite()
            low = torch.where(fine, (y.abs() - f).clamp_min(0), 0.0).amax(-1)
            high = torch.where(fine, y.abs() + f, 0.0).amax(-1)
            by_block = {}
            for n, (s, p) in enumerate(at):
                by_block.setdefault((s, p // self.bs), []).append(n)
            for (s, slot), ns in by_block.items():
                b = int(self.tables[s, slot])
                held = max(0, self.ctx[s] - slot * self.bs)
                for h in range(self.Hkv):
                    a, z = code_of(float(low[ns, h].max())), code_of(float(high[ns, h].max()))
                    now, old = int(codes[b, h]), int(codes_were[b, h])
                    if held:
                        a, z = max(a, old), max(z, old)
                    assert a <= now <= z, (s, slot, h, a, now, z, old)
                    expect_codes[b, h] = now
                    if held and now != old:
                        older = was.view(torch.uint8)[b, :held, h].view(E4M3).float() * 2.0 ** (old - now)
                        expect[b, :held, h] = older.to(E4M3).view(torch.uint8)
            assert torch.equal(codes, expect_codes)
            unit = 2.0 ** (codes[block].double() - 127)[..., None]
            new = got[block, off].view(E4M3).double()
            assert ((new - y / unit).abs() <= 2.0 ** -4 * (y / unit).abs() + 2.0 ** -10 + f / unit)[fine].all()
            assert new[~fine].isnan().all()
            if exact:
                bits = (y / unit).float().to(E4M3).view(torch.uint8)
                assert torch.equal(got[block, off][fine], bits[fine])
            got[block, off] = 0
            expect[block, off] = 0
            assert torch.equal(got, expect)
        return self


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(16, 0), (16, 16), (64, 64), (64, 32), (80, 80), (96, 32), (128, 128), (128, 64), (144, 112), (192, 64), (256, 256)])
def test_head_sizes_and_rotations(dt, e4m3, interleaved, D, rot):
    Case(dt, e4m3, D=D, rot=rot, interleaved=interleaved).call().check()


@pytest.mark.parametrize("D,rot", [(8, 0), (24, 16), (72, 64), (136, 112)])
def test_head_sizes_of_16_bit_pages_alone(D, rot):
    Case(e4m3=False, D=D, rot=rot).call().check()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("norm", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("rot", [0, 64])
def test_without_norms(e4m3, norm, rot):
    Case(e4m3=e4m3, norm=norm, rot=rot, fused=False).call().check()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("bs", [1, 2, 3, 16, 24, 100, 256])
@pytest.mark.parametrize("layout", ["token", "head"])
def test_page_sizes(e4m3, bs, layout):
    Case(e4m3=e4m3, bs=bs, layout=layout, new=(250, 97, 1, 33), ctx=(0, 5, 100, 15), D=128, rot=128).call().check()


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 64, 65, 129])
@pytest.mark.parametrize("ctx", [0, 1, 15, 16, 33])
def test_lengths(n, ctx):
    Case(new=(n,), ctx=(ctx,), S=2).call().check()


@pytest.mark.parametrize("S", [1, 63, 64, 65, 130, 4097, 5000])
@pytest.mark.parametrize("e4m3", [False, True])
def test_numbers_of_sequences(S, e4m3):
    new = (1, 0, 3, 0, 0, 2) if S > 1 else (2,)
    Case(e4m3=e4m3, S=S, new=new, ctx=(4, 0, 1), bs=4, Hq=1, Hkv=1, D=16, rot=16).call().check()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("new", [(0,), (0, 0, 5), (5, 0, 0, 0), (0, 9, 0)])
def test_empty_sequences_and_tokens_of_none(e4m3, new):
    Case(e4m3=e4m3, new=new, S=6, before=3, behind=5).call().check()


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (40, 8), (7, 7), (64, 1)])
def test_head_numbers(Hq, Hkv):
    Case(Hq=Hq, Hkv=Hkv).call().check()
    Case(Hq=Hq, Hkv=Hkv, D=256, rot=64, e4m3=False).call().check()


def test_positions_of_their_own():
    Case(positions=True).call().check()
    Case(positions=True, e4m3=False, interleaved=True).call().check()


@pytest.mark.parametrize("e4m3", [False, True])
def test_empty_caches_and_keys_and_values_alone(e4m3):
    Case(e4m3=e4m3, no_ctx=True).call().check()
    Case(e4m3=e4m3, queries=False).call().check()


@pytest.mark.parametrize("size", [1e-30, 1e-6, 0.03, 1.0, 300.0, 1e5, 1e30])
def test_scales_follow_the_values(size):
    Case("bf16", size=size, norm=(False, False), rot=0).call().check()
    Case("bf16", size=size, norm=(False, False), rot=64).call().check()


def test_scales_at_the_borders():
    """Largest magnitudes at 448 times a power of two, one step above and below."""
    c = Case(S=1, new=(5,), ctx=(0,), bs=1, Hq=1, Hkv=1, D=16, rot=0, norm=(False, False))
    for i, x in enumerate((448.0, 450.0, 446.0, 448.0 * 2.0 ** -40, 0.0)):
        c.k[i] = 0.0
        c.k[i, 0, 3] = -x
        c.v[i] = x / 2
    c.call().check()
    b = c.tables[0].long()
    assert c.sk[b, 0].tolist() == [127, 128, 127, 87, 1]


def test_zeros_and_small_values_keep_an_older_scale():
    c = Case(S=2, new=(3,), ctx=(5, 0), norm=(False, False), rot=0)
    c.k.zero_()
    c.v.mul_(1e-3)
    c.call().check()
    b = int(c.tables[0, 0])
    assert torch.equal(c.sk[b], c.codes_were[0][b])
    assert (c.sk[int(c.tables[1, 0])] == 1).all()


def test_growing_round_after_round():
    """A sequence of rounds into one block, each louder than the last: older tokens lose nothing but
    what falls below e4m3's normal range, half a step of the block's last scale at most."""
    S, bs = 3, 16
    c = Case(S=S, new=(2,), ctx=(0,), bs=bs, norm=(False, False), rot=0)
    told = []
    for t in range(8):
        c.k.copy_((torch.randn(c.k.shape, device="cuda") * 1.7 ** t).to(DT[c.dt]))
        c.v.copy_((torch.randn(c.v.shape, device="cuda") * 0.6 ** t).to(DT[c.dt]))
        c.ctx = [2 * t] * S
        c.ctx_t.fill_(2 * t)
        c.was = [c.kc.clone(), c.vc.clone()]
        c.codes_were = [c.sk.clone(), c.sv.clone()]
        c.call().check()
        told.append((c.k.double().clone(), c.v.double().clone()))
    for cache, codes, j in ((c.kc, c.sk, 0), (c.vc, c.sv, 1)):
        for s in range(S):
            b = int(c.tables[s, 0])
            unit = 2.0 ** (codes[b].double() - 127)[:, None]
            for t in range(8):
                y = told[t][j][2 * s: 2 * s + 2]
                err = (cache[b, 2 * t: 2 * t + 2].double() * unit - y).abs()
                # the first rounding, and one more to a fixed point of the last scale
                assert (err <= 2.0 ** -4 * y.abs() + 2 * 2.0 ** -10 * unit).all()


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("e4m3", [False, True])
def test_what_is_not_finite(bad, e4m3):
    c = Case(e4m3=e4m3, S=2, new=(20,), ctx=(7,), norm=(False, False), rot=0)
    c.k[3, 1, 5] = bad
    c.v[25, 0, 63] = bad
    if e4m3:
        c.call().check()
    else:
        c.call()
        at = int(c.tables[0, 0]), 10
        assert torch.equal(c.kc[at][1].view(torch.int16), c.k[3, 1].view(torch.int16))


def test_a_block_that_is_not_a_number_stays_so():
    c = Case(S=1, new=(2,), ctx=(3,), bs=16)
    b = int(c.tables[0, 0])
    c.sk[b, 1] = 255
    c.call()
    assert int(c.sk[b, 1]) == 255 and int(c.status) == 0


def test_queries_in_place():
    c = Case(fused=False)
    want = Case(fused=False).call().check().q_out
    c.q_out = c.q
    c.call()
    assert torch.equal(c.q, want)


@pytest.mark.parametrize("e4m3", [False, True])
def test_bad_indexes_are_flagged_and_never_followed(e4m3):
    P = Case(e4m3=e4m3).kc.shape[0]
    for bad in (P, -1, -2, 2 ** 31 - 1, -2 ** 31):
        c = Case(e4m3=e4m3)
        c.tables[1, 1] = bad
        c.call().check(skip_kv=[c.cu[1] + i for i in range(30) if 16 <= i < 32], status=sm.ST_BAD_INPUT)
    for ctx in (-1, -100, -2 ** 31):
        c = Case(e4m3=e4m3)
        c.ctx_t[1] = ctx
        c.call().check(skip=[c.cu[1] + i for i in range(30)], status=sm.ST_BAD_INPUT)
    for ctx in (1000, 2 ** 31 - 1, 2 ** 31 - 20):
        c = Case(e4m3=e4m3, positions=True)
        c.ctx_t[1] = ctx
        c.call()
        c.check(skip_kv=[c.cu[1] + i for i in range(30)], status=sm.ST_BAD_INPUT)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("value", [-1, 400, 2 ** 31 - 1, -2 ** 31])
def test_positions_outside_the_table(e4m3, value):
    c = Case(e4m3=e4m3, positions=True)
    gone = [0, 1, 2, 3, 4, 7, 20]  # all of the first sequence, some of the second
    c.positions[torch.tensor(gone, device="cuda")] = value
    c.call().check(skip=gone, status=sm.ST_BAD_INPUT)
    c = Case(e4m3=e4m3, max_pos=20)  # lengths that pass the table
    c.call().check(skip=[c.cu[s] + i for s in range(4) for i in range(c.new[s]) if c.ctx[s] + i >= 20], status=sm.ST_BAD_INPUT)


def test_lengths_out_of_order_are_flagged():
    for at, value in ((1, -1), (1, 10 ** 6), (2, 3), (0, -5), (4, 2 ** 31 - 1), (3, -2 ** 31)):
        c = Case()
        c.cu_t[at] = value
        before = [x.view(torch.uint8).clone() for x in (c.kc, c.vc)]
        c.call()
        assert int(c.status) & sm.ST_BAD_INPUT
        free = sorted(set(range(c.kc.shape[0])) - set(c.tables.view(-1).tolist()))
        for x, y in zip((c.kc, c.vc), before):  # nothing outside the tables is written
            assert torch.equal(x.view(torch.uint8)[free], y[free])


def test_on_another_stream_and_in_a_graph():
    c = Case(new=(5, 3, 1, 8), ctx=(6, 20, 0))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    c.call(stream=st)
    st.synchronize()
    c.check()
    c = Case(new=(5, 3, 1, 8), ctx=(6, 20, 0))
    c.call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call()
    for t in range(4):
        c.k.copy_((torch.randn(c.k.shape, device="cuda") * (1 + t)).to(DT[c.dt]))
        c.ctx = [6 + t, 20 - t, t, 17]
        c.ctx_t.copy_(torch.tensor(c.ctx, dtype=torch.int32))
        c.was, c.codes_were = [c.kc.clone(), c.vc.clone()], [c.sk.clone(), c.sv.clone()]
        c.q_out.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        c.check()


def test_repeats_bit_for_bit():
    a, b = Case(new=(100, 33, 2, 7), D=128, rot=128).call(), Case(new=(100, 33, 2, 7), D=128, rot=128).call()
    for x, y in ((a.kc, b.kc), (a.vc, b.vc)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert torch.equal(a.sk, b.sk) and torch.equal(a.q_out, b.q_out)


def test_pages_past_32_bits():
    page = 1 << 31  # bytes: block 2 begins 2^32 bytes in
    buf = torch.zeros(2 * page + (1 << 20), dtype=torch.uint8, device="cuda").view(E4M3)
    c = Case(S=1, new=(40,), ctx=(0,), Hkv=2, D=64)
    c.tables = torch.tensor([[2, 0, 1]], **I32)
    c.kc = buf.as_strided((3, 16, 2, 64), (page, 128, 64, 1))
    c.vc = buf.as_strided((3, 16, 2, 64), (page, 128, 64, 1), 1 << 16)
    c.was = [c.kc.clone(), c.vc.clone()]
    c.codes_were = [x[:3].clone() for x in c.codes_were]
    c.sk, c.sv = (x.clone() for x in c.codes_were)
    c.call().check()
