"""smcsd_tree_attention against the definition in 64 bits: types, head layouts, lengths from
nothing to long, page sizes that end inside a tile, shared prefixes, trees, rows that see
nothing, garbage (NaN, infinities) wherever nothing may be read, and the calls a server makes
(another stream, a captured graph, one workspace for several calls).

The bound on an output element, with u = finfo(dtype).eps / 2 (half a step) and p the exact
probabilities: the output's own rounding u|out| (+ half the smallest subnormal), the
probabilities' rounding u sum p|v| (each is off by at most u p; those below the type's normal
range by half its smallest subnormal, on at most `len` tokens), and the scores' fp32 error d:
a dot product of D terms and a scale, |dz| <= d = (D + 4) 2^-24 sum|q k| scale, moves each p
by a factor exp(+-2d), and the sum of p and of p v over at most len terms adds (len + 64) 2^-24,
so (4 d + 2 (len + 64) 2^-24) sum p|v|.  lse: 2 d + (len + 64) 2^-24 + 2^-23 |lse|."""
import math

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
    """A batch with its cache: pages in shuffled order, `shared` leading tokens common to a
    prompt's particles, everything that no node sees filled with `junk`."""

    def __init__(self, dt="bf16", B=1, N=1, R=1, Hq=4, Hkv=2, D=64, lens=(17,), bs=16, shared=0, tree=False, nodes=None,
                 layout="token", junk=math.nan, seed=0, spare=3, qpad=0, scale=None, loud=1.0):
        g = torch.Generator().manual_seed(seed)
        self.dt, self.B, self.N, self.R, self.Hq, self.Hkv, self.D, self.bs = dt, B, N, R, Hq, Hkv, D, bs
        S = self.S = B * N
        self.lens = [lens[i % len(lens)] for i in range(S)]
        self.nodes = [R if nodes is None else nodes[i % len(nodes)] for i in range(S)]
        M = max(-(-(x + R) // bs) for x in self.lens) + 1
        first = shared // bs
        P = B * first + S * (M - first) + spare
        ids = torch.randperm(P, generator=g).tolist()
        tables = torch.full((S, M), -1, dtype=torch.int32)
        pool = iter(ids)
        for b in range(B):
            head = [next(pool) for _ in range(first)]
            for n in range(N):
                s = b * N + n
                used = -(-(self.lens[s] + self.nodes[s]) // bs)
                row = (head + [next(pool) for _ in range(max(0, used - first))])[:used]
                tables[s, :used] = torch.tensor(row, dtype=torch.int32)
        self.tables = tables.cuda()
        shape = (P, bs, Hkv, D) if layout == "token" else (P, Hkv, bs, D)
        kv = [torch.randn(shape, generator=g).to(DT[dt]).cuda() for _ in range(2)]
        self.k, self.v = kv if layout == "token" else [x.transpose(1, 2) for x in kv]
        live = torch.zeros(P, bs, dtype=torch.bool)
        for s in range(S):
            for p in range(self.lens[s] + self.nodes[s]):
                live[tables[s, p // bs], p % bs] = True
        self.k[~live.cuda()] = junk
        self.v[~live.cuda()] = junk
        self.qfull = (loud * torch.randn((S, R, Hq + qpad, D), generator=g)).to(DT[dt]).cuda()
        self.q = self.qfull[:, :, :Hq]
        self.mask = None
        if tree:
            bits = torch.zeros(S, R, dtype=torch.int64)
            for s in range(S):
                for i in range(R):
                    up = int(torch.randint(0, i, (1,), generator=g)) if i else None
                    bits[s, i] = (0 if up is None else bits[s, up]) | (1 << i if i < 63 else -(1 << 63))
            self.mask = bits.cuda()
        self.scale = D ** -0.5 if scale is None else scale
        self.lens_t = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.nodes_t = None if nodes is None else torch.tensor(self.nodes, dtype=torch.int32, device="cuda")
        self.out = torch.full((S, R, Hq, D), 77.0, dtype=DT[dt], device="cuda")
        self.lse = torch.full((S, R, Hq), 77.0, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.ws = sm.alloc_workspace(sm.OP_TREE_ATTN, B, N, K=R, V=Hq * D, P=Hkv)
        self.ws.fill_(0xFF)  # no initial contents needed

    def call(self, **kw):
        a = dict(tree_mask=self.mask, num_nodes=self.nodes_t, lse=self.lse)
        a.update(kw)
        ws = a.pop("workspace", self.ws)
        sm.tree_attention(self.q, self.k, self.v, self.tables, self.lens_t, self.B, self.N, self.scale, self.out,
                          self.status, ws, **a)
        return self

    def sees(self, s, i):
        """The positions that node i of sequence s sees."""
        ctx, n = self.lens[s], self.nodes[s]
        if self.mask is None:
            js = range(min(i + 1, n))
        else:
            m = int(self.mask[s, i].item())
            js = [j for j in range(n) if (m >> j) & 1]
        return list(range(ctx)) + [ctx + j for j in js]

    def check(self, rows=None):
        S, R, G, D = self.S, self.R, self.Hq // self.Hkv, self.D
        u, sub = torch.finfo(DT[self.dt]).eps / 2, SUB[self.dt]
        assert int(self.status) == 0
        for s in range(S) if rows is None else rows:
            n, ctx = self.nodes[s], self.lens[s]
            assert (self.out[s, n:] == 77).all() and (self.lse[s, n:] == 77).all()
            if n == 0:
                continue
            L = ctx + n
            pos = torch.arange(L, device="cuda")
            at = self.tables[s].long()[pos // self.bs]
            k, v = (c[at, pos % self.bs].double().transpose(0, 1) for c in (self.k, self.v))  # [Hkv, L, D]
            vis = torch.zeros(n, L, dtype=torch.bool)
            for i in range(n):
                vis[i, self.sees(s, i)] = True
            vis = vis.cuda()
            for h in range(self.Hkv):
                hs = slice(h * G, h * G + G)
                q = self.q[s, :n, hs].double().reshape(n * G, D)
                ok = vis.repeat_interleave(G, 0)
                z = (q @ k[h].t() * self.scale).masked_fill(~ok, -math.inf)
                d = (D + 4) * 2.0 ** -24 * ((q.abs() @ k[h].abs().t()) * abs(self.scale)).masked_fill(~ok, 0).amax(1, keepdim=True)
                top = z.amax(1, keepdim=True)
                p = torch.where(ok, (z - top.masked_fill(top == -math.inf, 0)).exp(), 0.0)
                tot = p.sum(1, keepdim=True)
                want_lse = (top + tot.log()).view(n, G)
                p = p / tot.clamp_min(1e-300)
                want = p @ v[h]
                mag = p @ v[h].abs()
                lost = min(sub, 1.0) * (ok.double() @ v[h].abs()) / tot.clamp_min(1e-300)
                tol = u * want.abs() + sub + (u + 4 * d + 2 * (L + 64) * 2.0 ** -24) * mag + lost
                got = self.out[s, :n, hs].double().reshape(n * G, D)
                err = (got - want).abs()
                assert (err <= tol).all(), (s, h, float((err - tol).max()), float((err / tol.clamp_min(1e-300)).max()))
                gl = self.lse[s, :n, hs].double()
                empty = tot.view(n, G) == 0
                assert ((gl == -math.inf) == empty).all()
                ltol = 2 * d.view(n, G) + (L + 64) * 2.0 ** -24 + 2.0 ** -23 * want_lse.abs()
                assert ((gl - want_lse).abs() <= ltol)[~empty].all(), (s, h)
        return self


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("D", [8, 64, 72, 128, 200, 256])
def test_head_sizes(dt, D):
    Case(dt, N=2, R=3, D=D, lens=(37, 70), layout="head").call().check()


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 1), (3, 1), (7, 1), (16, 2), (8, 8), (32, 2)])
@pytest.mark.parametrize("R", [1, 2, 5, 16])
def test_head_groups_and_nodes(Hq, Hkv, R):
    Case(Hq=Hq, Hkv=Hkv, R=R, N=2, lens=(45, 130)).call().check()


@pytest.mark.parametrize("L", [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 300])
@pytest.mark.parametrize("R", [1, 4])
def test_lengths(L, R):
    Case(lens=(L,), R=R, B=2, N=1).call().check()


@pytest.mark.parametrize("bs", [1, 2, 3, 16, 24, 100, 256])
@pytest.mark.parametrize("layout", ["token", "head"])
def test_page_sizes(bs, layout):
    Case(bs=bs, layout=layout, N=3, R=5, lens=(250, 97, 3)).call().check()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("R", [1, 7, 33, 63, 64])
@pytest.mark.parametrize("ctx", [0, 50])
def test_trees(dt, R, ctx):
    Case(dt, N=2, R=R, tree=True, lens=(ctx, ctx + 9), Hq=8, Hkv=1).call().check()


def test_long_context_is_split_and_joined():
    c = Case(B=1, N=1, R=6, Hq=8, Hkv=2, D=128, lens=(20000,), tree=True)
    c.call(max_len=20006).check()
    first = c.out.clone(), c.lse.clone()
    for hint in (0, 1, 300, 10 ** 9):  # a hint, and no bound: whatever it says, every token is seen
        c.out.fill_(77)
        c.call(max_len=hint).check()
    c.call(max_len=20006)
    assert torch.equal(c.out, first[0]) and torch.equal(c.lse, first[1])  # and runs repeat bit for bit


@pytest.mark.parametrize("N,shared", [(2, 64), (3, 100), (16, 512), (5, 1000), (64, 160)])
@pytest.mark.parametrize("R,Hq", [(1, 2), (5, 8)])
def test_shared_prefix(N, shared, R, Hq):
    lens = tuple(shared + x for x in (0, 1, 40, 17, 133))
    Case(B=2, N=N, R=R, Hq=Hq, Hkv=2, lens=lens, shared=shared, tree=R > 1, layout="head").call().check()


@pytest.mark.parametrize("dt,D", [("f16", 80), ("bf16", 128), ("bf16", 256), ("f16", 64)])
def test_shared_prefix_types(dt, D):
    Case(dt, B=2, N=6, R=5, Hq=14, Hkv=2, D=D, lens=(700, 701, 790), shared=690, bs=24).call().check()


def test_shared_prefix_longer_than_some_contexts():
    # a particle shorter than the common tables: only what all of them hold as context is common
    Case(B=1, N=4, R=2, lens=(200, 90, 200, 64), shared=64, bs=16).call().check()
    c = Case(B=1, N=3, R=3, lens=(160, 160, 160), shared=160, bs=16, seed=4)
    c.tables[1] = c.tables[0]  # the same blocks throughout, the new tokens' too
    c.call().check()
    c.lens = [160, 33, 0]  # ... and shorter particles on them: their nodes lie in shared blocks
    c.lens_t.copy_(torch.tensor(c.lens, dtype=torch.int32))
    c.tables[2] = c.tables[0]
    c.call().check()


def test_whole_tables_shared():
    c = Case(B=2, N=4, R=1, lens=(320,), bs=16, seed=9)
    for b in range(2):
        c.tables[4 * b: 4 * b + 4] = c.tables[4 * b]
    c.call().check()


def test_ragged_nodes_leave_rows_alone():
    Case(B=2, N=3, R=6, nodes=(6, 0, 1, 4), lens=(40, 0, 129), tree=True, qpad=3).call().check()
    Case(B=1, N=5, R=4, nodes=(0, 4, 2), lens=(200, 210), shared=192).call().check()


def test_rows_that_see_nothing():
    c = Case(B=1, N=4, R=5, lens=(0, 0, 30, 0), tree=True)
    c.mask[0] = 0            # nothing at all
    c.mask[1, 2] = 0         # one row
    c.mask[3, :] = 1 << 4    # all see the last node only, the last too
    c.call().check()
    assert (c.out[0] == 0).all() and (c.lse[0] == -math.inf).all() and (c.out[1, 2] == 0).all()


def test_bits_past_the_nodes_mean_nothing():
    c = Case(B=1, N=2, R=5, nodes=(3, 5), lens=(20,), tree=True)
    c.mask |= -(1 << 5)
    c.mask[0] |= 0b11000  # nodes 3 and 4 of a sequence of three
    c.call().check()


@pytest.mark.parametrize("poison", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("R", [6, 40])
def test_a_node_that_a_row_does_not_see_cannot_reach_it(poison, R):
    c = Case(B=1, N=2, R=R, lens=(50, 0), tree=True, Hq=4, Hkv=2)
    j = R - 2
    others = [[i for i in range(R) if not (int(c.mask[s, i]) >> j) & 1] for s in range(2)]
    k, v = c.k.clone(), c.v.clone()
    for s in range(2):
        p = c.lens[s] + j
        c.k[c.tables[s, p // c.bs].long(), p % c.bs] = poison
        c.v[c.tables[s, p // c.bs].long(), p % c.bs] = poison
    c.call()
    assert int(c.status) == 0
    got = c.out.clone(), c.lse.clone()
    c.k, c.v = k, v
    c.call().check()  # without the poison
    for s in range(2):
        assert torch.equal(got[0][s, others[s]], c.out[s, others[s]]), s
        assert torch.equal(got[1][s, others[s]], c.lse[s, others[s]]), s


@pytest.mark.parametrize("bs", [1, 2])
@pytest.mark.parametrize("N,shared", [(1, 0), (3, 700)])
def test_a_context_of_many_small_pages(bs, N, shared):
    Case(N=N, R=5, D=128, lens=(1000, 777, 2077), bs=bs, shared=shared).call().check()


@pytest.mark.parametrize("D", [136, 256])
@pytest.mark.parametrize("R", [1, 9, 40])
@pytest.mark.parametrize("N,shared", [(1, 0), (4, 512)])
def test_wide_heads_over_split_contexts(D, R, N, shared):
    Case(N=N, R=R, Hq=8, Hkv=2, D=D, lens=(3000, 513), shared=shared, tree=R > 1, layout="head").call().check()


@pytest.mark.parametrize("D", [24, 64, 96, 200])
@pytest.mark.parametrize("L", [600, 1500, 9000])
def test_parts_of_several_numbers(D, L):
    Case(B=2, N=3, R=2, D=D, lens=(L, L - 99), shared=L // 2, nodes=(2, 1, 0)).call().check()


@pytest.mark.parametrize("poison", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("L", [5, 30, 3000])
def test_a_value_that_is_not_finite_is_seen_by_its_rows(poison, L):
    """Node 1's value holds one element that is not finite: node 0 does not see it, nodes 1 and
    2 do, at every head of that key/value head."""
    c = Case(R=3, Hq=4, Hkv=2, D=64, lens=(L,))
    at = c.tables[0, (L + 1) // c.bs].long()
    c.v[at, (L + 1) % c.bs, 1, 37] = poison
    c.call()
    out = c.out[0].float()
    assert torch.isfinite(out[0]).all() and torch.isfinite(out[:, :2]).all()
    hit = out[1:, 2:, 37]
    assert (torch.isnan(hit) if math.isnan(poison) else hit == poison).all()
    rest = torch.cat([out[1:, 2:, :37], out[1:, 2:, 38:]], -1)
    assert torch.isfinite(rest).all()


def test_infinite_scores():
    # A key that scores +inf against a positive query makes its rows NaN; -inf leaves them out.
    c = Case(B=1, N=1, R=1, Hq=1, Hkv=1, D=64, lens=(40,))
    c.q.fill_(1.0)
    at = c.tables[0, 0].long(), 5
    c.k[at] = -math.inf
    c.v[at] = 3.0
    c.call()
    z = (c.k[c.tables[0, :3].long()].reshape(-1, 64)[:41].double().sum(1) * c.scale)
    p = torch.softmax(z, 0)
    v = c.v[c.tables[0, :3].long()].reshape(-1, 64)[:41].double()
    assert float(p[5]) == 0 and torch.allclose(c.out.view(-1).double(), p @ v, atol=0.02)


def test_loud_scores():
    # Scores up to some hundreds: the running maximum moves by far.
    Case(B=1, N=2, R=4, Hq=8, Hkv=2, D=128, lens=(333, 150), loud=40.0).call().check()
    Case("f16", B=1, N=4, R=4, Hq=8, Hkv=2, D=128, lens=(333, 350), shared=320, loud=40.0).call().check()


@pytest.mark.parametrize("scale", [0.0, -0.3])
def test_other_scales(scale):
    Case(B=1, N=2, R=3, lens=(100, 30), scale=scale, shared=16).call().check()


def test_bad_indexes_are_flagged_and_never_followed():
    c = Case(B=1, N=4, R=2, lens=(100, 100, 100, 100), bs=16)
    c.call().check()
    good = c.out.clone()
    P = c.k.shape[0]
    for bad in (P, P + 5, -2, -1, 2 ** 31 - 1, -2 ** 31):
        d = Case(B=1, N=4, R=2, lens=(100, 100, 100, 100), bs=16)
        d.tables[1, 2] = bad
        d.call()
        assert int(d.status) == sm.ST_BAD_INPUT
        assert torch.equal(d.out[[0, 2, 3]], good[[0, 2, 3]])
        pos = [p for p in range(100) if p // 16 != 2]  # the rest of the sequence is seen
        at = d.tables[1].long()
        k = torch.stack([d.k[at[p // 16], p % 16] for p in pos + [100]]).double()[:, 0]
        v = torch.stack([d.v[at[p // 16], p % 16] for p in pos + [100]]).double()[:, 0]
        p = torch.softmax(k @ d.q[1, 0, 0].double() * d.scale, 0)
        assert torch.allclose(d.out[1, 0, 0].double(), p @ v, atol=0.02)
    for n in (-1, 10 ** 6, 2 ** 31 - 1, -2 ** 31):
        d = Case(B=1, N=4, R=2, lens=(100, 100, 100, 100), bs=16)
        d.lens_t[2] = n
        d.call()
        assert int(d.status) == sm.ST_BAD_INPUT
        assert torch.equal(d.out[[0, 1, 3]], good[[0, 1, 3]])
        assert (d.out[2] == 0).all() and (d.lse[2] == -math.inf).all()
    for n in (-3, 3, 2 ** 31 - 1):
        d = Case(B=1, N=4, R=2, nodes=(2,), lens=(100, 100, 100, 100), bs=16)
        d.nodes_t[3] = n
        d.call()
        assert int(d.status) == sm.ST_BAD_INPUT
        assert torch.equal(d.out[:3], good[:3])
        assert torch.equal(d.out[3], good[3]) if n > 0 else (d.out[3] == 77).all()


def test_without_lse_and_on_another_stream():
    c = Case(B=1, N=3, R=4, lens=(77, 300, 5), shared=0)
    c.call()
    want = c.out.clone()
    c.out.fill_(77)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    c.call(stream=st, lse=None)
    st.synchronize()
    assert torch.equal(c.out, want)
    c.check()


def test_one_workspace_for_several_calls():
    a = Case(B=1, N=4, R=5, lens=(600, 610), shared=592, seed=1)
    b = Case(B=1, N=4, R=5, lens=(900, 30), seed=2)
    for _ in range(3):
        a.call()
        b.call(workspace=a.ws)
    a.check()
    b.check()


def test_graph_replays():
    c = Case(B=2, N=4, R=5, lens=(600, 610, 640), shared=592, tree=True)
    long = Case(B=1, N=1, R=3, lens=(5000,))
    c.call()
    long.call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call()
        long.call()
    for k in range(4):
        q, x = torch.randn_like(c.q), torch.randn_like(long.q)
        c.q.copy_(q)
        long.q.copy_(x)
        if k == 2:  # lengths are device data: a replay follows them
            c.lens[1] = long_len = 599
            c.lens_t[1] = long_len
            long.lens[0] = 777
            long.lens_t[0] = 777
        c.out.fill_(77)
        long.out.fill_(77)
        g.replay()
        torch.cuda.synchronize()
        c.check()
        long.check()
        torch.randn(1000, device="cuda").sum()


def test_pages_past_32_bits():
    page = 1 << 31  # elements: block 2 begins 2^32 elements in
    buf = torch.empty(2 * page + (1 << 20), dtype=torch.bfloat16, device="cuda")
    c = Case(B=1, N=2, R=3, Hq=4, Hkv=2, D=64, lens=(30, 12), bs=16)
    k = buf.as_strided((3, 16, 2, 64), (page, 128, 64, 1))
    v = buf.as_strided((3, 16, 2, 64), (page, 128, 64, 1), 1 << 16)
    c.tables = torch.tensor([[2, 0, 1], [2, -1, -1]], dtype=torch.int32, device="cuda")
    for x in (k, v):
        x.copy_(torch.randn(3, 16, 2, 64, device="cuda"))
    c.k, c.v = k, v
    c.call().check()


def test_largest_batch_of_short_sequences():
    c = Case(B=64, N=16, R=2, Hq=4, Hkv=1, D=64, lens=(3, 17, 0, 9), bs=4)
    c.call().check(rows=range(0, 1024, 37))


@pytest.mark.parametrize("shared", [1023, 1024, 1025, 2047, 2048, 2049, 2300])
def test_more_shared_blocks_than_are_compared_at_once(shared):
    Case(N=5, R=2, lens=(2310, 2400, 2333), bs=1, shared=shared).call().check()


@pytest.mark.parametrize("differ", [
    ((2, 1024),), ((1, 2047), (3, 1024)), ((3, 1500), (1, 1900), (2, 1026), (4, 2047)), ((4, 2048), (1, 2049), (2, 2299)),
    ((1, 1023), (2, 1024)), ((4, 2299),), ((1, 1100), (1, 2100), (3, 2200))])
def test_several_particles_leave_the_shared_blocks(differ):
    """Tables alike past 2048 blocks but for single entries: (particle, slot) that names another block."""
    c = Case(N=5, R=2, lens=(2310, 2400, 2333), bs=1, shared=2300, seed=len(differ))
    for n, slot in differ:
        c.tables[n, slot] = c.tables[n, 2305].item()
    c.call().check()


@pytest.mark.parametrize("N,R,Hq", [(8, 5, 8), (14, 5, 8), (1, 33, 8), (1, 48, 6), (2, 64, 9)])
def test_row_tiles_of_three_waves(N, R, Hq):
    """129 to 192 rows of a head in two tiles, 257 to 288 in three: their fourth wave has no rows."""
    c = Case(B=2, N=N, R=R, Hq=Hq, Hkv=2 if Hq % 2 == 0 else 3, D=128, lens=(300, 311), shared=288 if N > 1 else 0, tree=True)
    c.call().check()
