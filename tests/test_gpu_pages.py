"""The pages' own operations against plain Python on the same state: smcsd_kv_fork,
smcsd_kv_free, smcsd_kv_compact and smcsd_kv_copy, each alone, on corrupt states, and in the
order a server uses them, with smcsd_kv_check recounting the state after every step."""
import random

import pytest
import torch

import smc_verification_resampling_amd as sm

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def dev(x):
    return torch.tensor(x, **I32)


class Pool:
    """Block tables, refcounts and free stack, on the device and as lists."""

    def __init__(self, S, M, P, seed=0, share=0.5, fill=1.0):
        r = random.Random(seed)
        ids = list(range(P))
        r.shuffle(ids)
        self.S, self.M, self.P = S, M, P
        self.T = [[-1] * M for _ in range(S)]
        for s in range(S):
            n = int(M * fill * (0.5 + 0.5 * r.random()))
            for i in range(n):
                if s and r.random() < share and self.T[s - 1][i] >= 0:
                    self.T[s][i] = self.T[s - 1][i]
                elif ids:
                    self.T[s][i] = ids.pop()
        self.rc = [0] * P
        for row in self.T:
            for b in row:
                if b >= 0:
                    self.rc[b] += 1
        self.stack = [b for b in range(P) if self.rc[b] == 0]
        r.shuffle(self.stack)
        self.up()

    def up(self):
        self.dT, self.drc = dev(self.T).view(self.S, self.M), dev(self.rc)
        self.dfl, self.dtop = dev(self.stack + [-9] * (self.P - len(self.stack))), dev([len(self.stack)])
        self.st = torch.zeros(1, **I32)

    def same(self, status=0):
        assert int(self.st) == status
        assert self.dT.tolist() == self.T
        assert self.drc.tolist() == self.rc
        assert int(self.dtop) == len(self.stack)
        assert self.dfl[: len(self.stack)].tolist() == self.stack

    def consistent(self):
        viol, st = torch.zeros(sm.KV_CHECK_KINDS, **I32), torch.zeros(1, **I32)
        sm.kv_check(self.dT, self.M, self.drc, self.dfl, self.dtop, viol, st, sm.alloc_workspace(sm.OP_KV_CHECK, 0, 0, P=self.P))
        assert viol.tolist() == [0] * sm.KV_CHECK_KINDS

    def free(self, which):
        ws = sm.alloc_workspace(sm.OP_KV_FREE, 0, 0, P=self.P)
        ws.fill_(0xFF)
        sm.kv_free(dev([int(s in which) for s in range(self.S)]), self.dT, self.drc, self.dfl, self.dtop, self.st, ws)
        gone = []
        for s in which:
            for i, b in enumerate(self.T[s]):
                self.T[s][i] = -1
                if 0 <= b < self.P and self.rc[b] > 0:
                    self.rc[b] -= 1
                    if self.rc[b] == 0:
                        gone.append(b)
        self.stack += sorted(gone, reverse=True)

    def fork(self, which, N):
        sm.kv_fork(dev([int(b in which) for b in range(self.S // N)]), self.S // N, N, self.dT, self.drc, self.st)
        for b in which:
            for i, x in enumerate(self.T[b * N]):
                for n in range(1, N):
                    if 0 <= x < self.P and self.T[b * N + n][i] == -1:
                        self.T[b * N + n][i] = x
                        self.rc[x] += 1

    def compact(self, bs=16):
        moves, n = torch.full((self.P // 2, 3), -5, **I32), dev([-5])
        ws = sm.alloc_workspace(sm.OP_KV_COMPACT, 0, 0, P=self.P)
        ws.fill_(0xFF)
        sm.kv_compact(self.dT, bs, self.drc, self.dfl, self.dtop, moves, n, self.st, ws)
        live = [b for b in range(self.P) if self.rc[b] > 0]
        k = len(live)
        movers, holes = [b for b in live if b >= k], [b for b in range(k) if self.rc[b] <= 0]
        to = dict(zip(movers, holes))
        for row in self.T:
            for i, b in enumerate(row):
                if 0 <= b < self.P:
                    row[i] = to.get(b, b) if self.rc[b] > 0 else -1
        self.rc = [max(r, 0) for r in self.rc]
        for a, b in to.items():
            self.rc[b], self.rc[a] = self.rc[a], 0
        self.stack = list(range(self.P - 1, k - 1, -1))
        assert int(n) == len(movers)
        assert moves[: len(movers)].tolist() == [[a, b, bs] for a, b in to.items()]
        assert (moves[len(movers):] == -5).all()
        return moves, n


SIZES = [(1, 1, 1), (1, 3, 4), (6, 5, 40), (12, 40, 500), (16, 300, 9000), (8, 1000, 70000), (40, 200, 17000)]


@pytest.mark.parametrize("S,M,P", SIZES)
def test_free(S, M, P):
    p = Pool(S, M, P, seed=P)
    p.free([])
    p.same()
    p.free(list(range(0, S, 2)))
    p.same()
    p.consistent()
    p.free(list(range(S)))
    p.same()
    p.consistent()
    assert len(p.stack) == P


@pytest.mark.parametrize("N,M,P", [(1, 7, 20), (2, 1, 4), (4, 7, 100), (16, 300, 4000), (40, 257, 2000), (1024, 3, 50)])
def test_fork(N, M, P):
    B = 3
    p = Pool(B * N, M, P, seed=N, share=0.0, fill=1.0 if N < 4 else 0.9)
    for s in range(B * N):
        if s % N:
            p.T[s] = [-1] * M
    p.rc = [0] * P
    for row in p.T:
        for b in row:
            if b >= 0:
                p.rc[b] += 1
    p.stack = [b for b in range(P) if p.rc[b] == 0]
    p.up()
    p.fork([0, 2], N)
    p.same()
    p.consistent()
    p.free([s for s in range(B * N) if s // N == 2 and s % N])  # all but particle 0 retire again
    p.same()
    p.consistent()


@pytest.mark.parametrize("S,M,P", SIZES)
@pytest.mark.parametrize("fill", [0.2, 1.0])
def test_compact(S, M, P, fill):
    p = Pool(S, M, P, seed=P + 1, fill=fill)
    p.compact()
    p.same()
    p.consistent()
    p.compact(4)  # dense already: nothing moves
    p.same()


def test_a_pool_of_millions_of_blocks():
    P = (1 << 20) + 12345
    p = Pool(4, 5000, P, seed=1, share=0.2)
    p.free([1, 3])
    p.same()
    p.compact()
    p.same()
    p.consistent()


def test_compact_full_and_empty_pools():
    p = Pool(2, 50, 100, share=0.0)
    for s in range(2):
        p.T[s] = list(range(99 - 50 * s, 49 - 50 * s, -1))
    p.rc, p.stack = [1] * 100, []
    p.up()
    p.compact()
    p.same()
    p.free([0, 1])
    p.compact()
    p.same()
    assert int(p.dtop) == 100


def test_corrupt_states_are_flagged_and_stay_in_bounds():
    B = sm.ST_BAD_INPUT
    p = Pool(6, 8, 60, seed=5)
    p.T[1][2], p.T[2][3] = 60, -7
    p.up()
    p.free([1, 2])
    p.same(B)
    p = Pool(6, 8, 60, seed=6, share=0.0)
    p.rc[p.T[0][0]] = 0  # fewer references than its tables name
    p.rc[p.T[0][1]] = -4
    p.T[1][0] = p.T[2][0]  # rc 1, two tables
    p.up()
    p.free([0, 1, 2])
    p.same(B)
    p = Pool(4, 8, 60, seed=7)
    p.dtop.fill_(59)  # more pushes than the stack holds
    p.free([0, 1, 2, 3])
    assert int(p.st) == B and int(p.dtop) == 60
    for top in (-1, 61, 2 ** 31 - 1):
        p = Pool(4, 8, 60, seed=7)
        p.dtop.fill_(top)
        p.free([0])
        assert int(p.st) == B and 0 <= int(p.dtop) <= 60
    p = Pool(4, 8, 60, seed=8, share=0.0)
    p.T[1] = [-1] * 8
    p.T[0][0], p.T[0][1], p.T[1][2] = 60, -2, 5
    p.up()
    p.fork([0], 2)
    p.same(B)
    p = Pool(4, 8, 60, seed=9, share=0.0)
    p.rc[p.T[0][0]], p.rc[p.T[1][1]] = 0, -3
    p.T[2][0], p.T[3][0] = 60, -8
    p.up()
    p.compact()
    p.same(B)


@pytest.mark.parametrize("count", [1, 2, 7])
@pytest.mark.parametrize("times", [2, 3, 64])
def test_a_block_that_loses_far_more_references_than_it_has(count, times):
    """Every block has `count` references; row 0 names it once, the others `times` times in a run."""
    n, rows = 256, 10 * times
    p = Pool(rows, n, n + 30, share=0.0, fill=0.0)
    p.T[0] = list(range(n))
    for s in range(1, rows):
        p.T[s] = [(s * (n // times) + i // times) % n for i in range(n)]
    p.rc = [count] * n + [0] * 30
    p.stack = list(range(n, n + 30))
    p.up()
    p.free(list(range(rows)))
    p.same(sm.ST_BAD_INPUT)
    p.consistent()


def caches(n, P, bs, H, D, dtype, layout, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    shape = (P, bs, H, D) if layout == "token" else (P, H, bs, D)
    c = [torch.randint(-100, 100, shape, generator=g, device="cuda").to(dtype) for _ in range(n)]
    return c if layout == "token" else [x.transpose(1, 2) for x in c]


def run_copy(cs, entries, count=None, cap=None):
    moves = dev(entries + [[0, 0, 0]] * ((cap or len(entries)) - len(entries))).view(-1, 3)
    st = torch.zeros(1, **I32)
    sm.kv_copy(cs, moves, dev([len(entries) if count is None else count]), st)
    return int(st)


@pytest.mark.parametrize("layout", ["token", "head"])
@pytest.mark.parametrize("dtype,D", [(torch.bfloat16, 64), (torch.float32, 3), (torch.float16, 5), (torch.uint8, 7), (torch.bfloat16, 128)])
@pytest.mark.parametrize("bs,H", [(1, 1), (4, 2), (16, 8), (24, 3), (16, 1)])
def test_copy(layout, dtype, D, bs, H):
    r = random.Random(bs * H)
    P = 64
    cs = caches(3, P, bs, H, D, dtype, layout)
    want = [c.clone() for c in cs]
    ids = r.sample(range(P), 40)
    entries = [[ids[i // 2], ids[20 + i], r.choice([0, 1, bs // 2, bs - 1, bs])] for i in range(20)]
    entries.append([ids[3], -1, bs])  # found no block
    entries.append([ids[4], ids[4], bs])
    for w in want:
        for a, b, t in entries:
            if b >= 0:
                w[b, :t] = w[a, :t].clone()
    assert run_copy(cs, entries) == 0
    assert all(torch.equal(c, w) for c, w in zip(cs, want))


def test_copy_counts_and_bad_entries():
    P, bs = 16, 4
    cs = caches(2, P, bs, 2, 8, torch.bfloat16, "token")
    for entries, count, done in (([[0, 1, 4], [2, 3, 4]], 1, 1), ([[0, 1, 4], [2, 3, 4]], 0, 0)):
        want = [c.clone() for c in cs]
        for w in want:
            for a, b, t in entries[:done]:
                w[b, :t] = w[a, :t].clone()
        assert run_copy(cs, entries, count) == 0
        assert all(torch.equal(c, w) for c, w in zip(cs, want))
    for bad in ([16, 1, 4], [-1, 1, 4], [0, 16, 4], [0, -2, 4], [0, 1, 5], [0, 1, -1], [2 ** 31 - 1, 1, 4]):
        want = [c.clone() for c in cs]
        for w in want:
            w[5, :3] = w[4, :3].clone()
        assert run_copy(cs, [bad, [4, 5, 3]]) == sm.ST_BAD_INPUT
        assert all(torch.equal(c, w) for c, w in zip(cs, want))
    want = [c.clone() for c in cs]
    assert run_copy(cs, [[6, 6, 4]], 3) == sm.ST_BAD_INPUT and run_copy(cs, [[6, 6, 4]], -1) == sm.ST_BAD_INPUT
    assert all(torch.equal(c, w) for c, w in zip(cs, want))


def test_copy_of_many_entries_and_caches():
    P, bs = 6000, 16
    cs = caches(6, P, bs, 2, 64, torch.bfloat16, "head")
    want = [c.clone() for c in cs]
    src, dst = torch.arange(0, 3000), torch.arange(3000, 6000)
    tok = torch.randint(0, bs + 1, (3000,), generator=torch.Generator().manual_seed(1))
    fresh = (torch.arange(bs)[None] < tok[:, None]).cuda()[:, :, None, None]
    for w in want:
        w[3000:] = torch.where(fresh, w[:3000], w[3000:])
    st = torch.zeros(1, **I32)
    moves = torch.stack([src, dst, tok], 1).int().cuda()
    sm.kv_copy(cs, moves, dev([3000]), st)
    assert int(st) == 0 and all(torch.equal(c, w) for c, w in zip(cs, want))


def test_copy_past_32_bits():
    page = 1 << 33  # bytes
    buf = torch.empty(page + (1 << 20), dtype=torch.uint8, device="cuda")
    c = buf.as_strided((2, 16, 2, 64), (page, 128, 64, 1))
    c.copy_(torch.randint(0, 255, (2, 16, 2, 64), device="cuda"))
    want = c.clone()
    want[1, :9] = want[0, :9].clone()
    assert run_copy([c], [[0, 1, 9]]) == 0
    assert torch.equal(c, want)


def test_copy_refusals():
    c = caches(1, 8, 4, 2, 8, torch.bfloat16, "token")[0]
    st = torch.zeros(1, **I32)
    m, n = dev([[0, 1, 2]]), dev([1])
    for bad in ([c, c.float()], [c, c[:4]], [c[:, ::2]], [c[..., :4]], [c.view(8, 4, 16)], [c] * 257, [c, c.transpose(1, 2).contiguous().transpose(1, 2)]):
        with pytest.raises(sm.SmcsdError):
            sm.kv_copy(bad, m, n, st)
    with pytest.raises(sm.SmcsdError):
        sm.kv_copy([c], m.view(-1), n, st)
    with pytest.raises(sm.SmcsdError):
        sm.kv_copy([c], m.long(), n, st)
    sm.kv_copy([], m, n, st)
    assert int(st) == 0


def test_graph_replays():
    p = Pool(8, 20, 400, seed=3)
    ws, wc = sm.alloc_workspace(sm.OP_KV_FREE, 0, 0, P=400), sm.alloc_workspace(sm.OP_KV_COMPACT, 0, 0, P=400)
    moves, n = torch.zeros(200, 3, **I32), torch.zeros(1, **I32)
    freed = dev([0] * 8)
    cs = caches(2, 400, 4, 2, 8, torch.bfloat16, "head")

    def work():
        sm.kv_free(freed, p.dT, p.drc, p.dfl, p.dtop, p.st, ws)
        sm.kv_compact(p.dT, 4, p.drc, p.dfl, p.dtop, moves, n, p.st, wc)
        sm.kv_copy(cs, moves, n, p.st)
    work()
    torch.cuda.synchronize()
    q = Pool(8, 20, 400, seed=3)
    q.compact(4)
    p.T, p.rc, p.stack = q.T, q.rc, q.stack
    p.same()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        work()
    for s in (3, 5, 0):
        q = Pool(8, 20, 400, seed=3)
        q.T, q.rc, q.stack = [list(r) for r in p.T], list(p.rc), list(p.stack)
        q.up()
        data = [c.clone() for c in cs]
        q.free([s])
        mv, k = q.compact(4)
        sm.kv_copy(data, mv, k, q.st)
        freed.copy_(dev([int(i == s) for i in range(8)]))
        g.replay()
        torch.cuda.synchronize()
        p.T, p.rc, p.stack = q.T, q.rc, q.stack
        p.same()
        assert all(torch.equal(a, b) for a, b in zip(cs, data))
        torch.randn(1000, device="cuda").sum()


def test_on_another_stream():
    p = Pool(8, 20, 400, seed=3)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    ws = sm.alloc_workspace(sm.OP_KV_FREE, 0, 0, P=400)
    f = dev([1] * 8)
    st.wait_stream(torch.cuda.current_stream())
    sm.kv_free(f, p.dT, p.drc, p.dfl, p.dtop, p.st, ws, stream=st)
    st.synchronize()
    assert int(p.dtop) == 400 and (p.dT == -1).all() and (p.drc == 0).all()
