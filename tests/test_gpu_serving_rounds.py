"""The serving operators together, as a server runs them: prompts are prefilled into particle 0
(qk_norm_rope), forked, reserved and copied on write (kv_fork, kv_reassign, kv_copy); each round
writes its new tokens (qk_norm_rope), attends (tree_attention), scores (token_logprobs) and
resamples (resample_kv_reassign, kv_copy); a prompt retires (kv_free), the pool is compacted
(kv_compact, kv_copy) and another is admitted in its place.  After every step the pages, read
through the tables, have to hold each particle's own history.

Bounds, u = finfo(dtype).eps / 2: keys u|k| + (D + 16) 2^-24 (|y| + |y'|) for the norm's sum over
D terms, its root and product, the two products of the rotation and their sum (y, y': the normed
pair); values as given; attention and log-probabilities as in their own tests."""
import math

import pytest
import torch

import smc_verification_resampling_amd as sm

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
B, N, R, HQ, HKV, D, V, BS, PLEN, EPS = 3, 4, 4, 4, 2, 64, 777, 16, 37, 1e-6
S, M, P = B * N, 8, 90
E = 70 * 2.0 ** -24


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


class Server:
    def __init__(self, dt, layout, seed):
        g = torch.Generator().manual_seed(seed)
        self.dt, self.g, self.u = DT[dt], g, torch.finfo(DT[dt]).eps / 2
        self.sub = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25}[dt]
        self.emb = torch.randn(V, HQ + 2 * HKV, D, generator=g).to(self.dt).cuda()
        self.kw = (1 + 0.1 * torch.randn(D, generator=g)).to(self.dt).cuda()
        self.head = (torch.randn(HQ * D, V, generator=g) / 8).cuda()
        a = torch.arange(M * BS).double()[:, None] * 10000.0 ** (-torch.arange(D // 2).double() / (D // 2))
        self.angles = a
        self.cos_sin = torch.cat([a.cos(), a.sin()], 1).float().cuda()
        shape = (P, BS, HKV, D) if layout == "token" else (P, HKV, BS, D)
        kv = [torch.full(shape, math.nan, dtype=self.dt, device="cuda") for _ in range(2)]
        self.k, self.v = kv if layout == "token" else [x.transpose(1, 2) for x in kv]
        self.tables, self.rc = torch.full((S, M), -1, **I32), torch.zeros(P, **I32)
        self.free_list, self.free_top = torch.randperm(P, generator=g).int().cuda(), torch.tensor([P], **I32)
        self.st = torch.zeros(1, **I32)
        self.cow, self.cow_n = torch.full((S, 3), -7, **I32), torch.zeros(1, **I32)
        self.ws_kv = {n: sm.alloc_workspace(sm.OP_KV, n, N, P=P).zero_() for n in (1, B)}
        self.ws_attn = sm.alloc_workspace(sm.OP_TREE_ATTN, B, N, K=R, V=HQ * D, P=HKV)
        self.ws_lp = sm.alloc_workspace(sm.OP_LOGPROBS, S * R, 1, K=5, V=V)
        self.hist = [[] for _ in range(S)]
        self.len = 0

    def rows(self, tokens, s0, ctx):
        """Writes tokens [n, r] of sequences s0.. behind ctx; their queries."""
        n, r = tokens.shape
        x = self.emb[tokens.long()]
        q = torch.empty(n, r, HQ, D, dtype=self.dt, device="cuda")
        sm.qk_norm_rope(x[:, :, :HQ], x[:, :, HQ:HQ + HKV], x[:, :, HQ + HKV:], torch.full((n,), ctx, **I32),
                        self.tables[s0:s0 + n], self.k, self.v, q, self.st, k_weight=self.kw, eps=EPS, cos_sin=self.cos_sin)
        return q

    def copy(self, moves, count):
        sm.kv_copy([self.k, self.v], moves, count, self.st)

    def admit(self, b, length):
        """The host's part: blocks for particle 0; then prefill, fork, reserve."""
        need, top = -(-length // BS), int(self.free_top)
        ids = self.free_list[top - need:top].flip(0)
        self.free_top -= need
        self.tables[b * N, :need] = ids
        self.rc[ids.long()] = 1
        prompt = torch.randint(0, V, (1, length), generator=self.g, dtype=torch.int32).cuda()
        self.rows(prompt, b * N, 0)
        sm.kv_fork((torch.arange(B, device="cuda") == b).int(), B, N, self.tables, self.rc, self.st)
        sm.kv_reassign(torch.arange(N, **I32), torch.zeros(1, **I32), 1, N, self.tables[b * N:(b + 1) * N], BS, length, R,
                       self.rc, self.free_list, self.free_top, self.cow, self.cow_n, self.st, self.ws_kv[1])
        assert int(self.cow_n) == (N - 1 if length % BS else 0)  # all but one leave the shared tail
        self.copy(self.cow, self.cow_n)
        for n in range(N):
            self.hist[b * N + n] = prompt[0].tolist()

    def round(self, t, tau):
        tokens = torch.randint(0, V, (S, R), generator=self.g, dtype=torch.int32).cuda()
        ctx = torch.full((S,), self.len, **I32)
        q = self.rows(tokens, 0, self.len)
        out = torch.full((S, R, HQ, D), 9.0, dtype=self.dt, device="cuda")
        sm.tree_attention(q, self.k, self.v, self.tables, ctx, B, N, D ** -0.5, out, self.st, self.ws_attn, max_len=M * BS)
        logits = (out.view(S * R, HQ * D).float() @ self.head).to(torch.bfloat16)
        logp, lse = torch.empty(S * R, 1, device="cuda"), torch.empty(S * R, device="cuda")
        ids, top = torch.empty(S * R, 5, **I32), torch.empty(S * R, 5, device="cuda")
        sm.token_logprobs(logits, S * R, V, 0.7, self.st, self.ws_lp, tokens=tokens.view(S * R, 1), out_logp=logp, out_lse=lse,
                          top_ids=ids, top_logp=top)
        for s in range(S):
            self.hist[s] += tokens[s].tolist()
        self.len += R
        self.check_pages()
        self.check_attention(q, out)
        z = logits.double() / float(torch.tensor(0.7, dtype=torch.float32))
        ref = torch.log_softmax(z, 1).gather(1, tokens.view(S * R, 1).long())
        tol = E + 2.0 ** -23 * ref.abs()
        assert ((logp.double() - ref).abs() <= tol).all()
        assert ((lse.double() - z.logsumexp(1)).abs() <= E + 2.0 ** -24 * z.logsumexp(1).abs()).all()
        order = torch.sort(torch.where(z == 0, 0.0, z).cpu(), dim=1, descending=True, stable=True).indices[:, :5]
        assert ids.tolist() == order.tolist()
        weights = (logp.view(B, N, R).sum(2) * 0.1).contiguous()
        anc, ess, res = torch.empty(B, N, **I32), torch.empty(B, device="cuda"), torch.empty(B, **I32)
        sm.resample_kv_reassign(weights, B, N, tau, 11, t, anc, ess, res, self.tables, BS, self.len, R, self.rc, self.free_list,
                                self.free_top, self.cow, self.cow_n, self.st, self.ws_kv[B])
        self.copy(self.cow, self.cow_n)
        for b in range(B):
            if int(res[b]):
                self.hist[b * N:(b + 1) * N] = [list(self.hist[b * N + int(a)]) for a in anc[b].tolist()]
        self.check_pages()
        return int(res.sum())

    def retire(self, b):
        sm.kv_free((torch.arange(S, device="cuda") // N == b).int(), self.tables, self.rc, self.free_list, self.free_top, self.st,
                   sm.alloc_workspace(sm.OP_KV_FREE, 0, 0, P=P))
        for n in range(N):
            self.hist[b * N + n] = []

    def compact(self):
        moves, n = torch.full((P // 2, 3), -5, **I32), torch.zeros(1, **I32)
        sm.kv_compact(self.tables, BS, self.rc, self.free_list, self.free_top, moves, n, self.st,
                      sm.alloc_workspace(sm.OP_KV_COMPACT, 0, 0, P=P))
        self.copy(moves, n)
        live = int((self.rc > 0).sum())
        assert int(self.tables.max()) == live - 1 and int(n) > 0

    def gather(self, s, n):
        pos = torch.arange(n, device="cuda")
        at = self.tables[s].long()[pos // BS]
        assert (at >= 0).all()
        return self.k[at, pos % BS].double(), self.v[at, pos % BS].double()  # [n, HKV, D]

    def check_pages(self):
        assert int(self.st) == 0
        viol, st = torch.zeros(sm.KV_CHECK_KINDS, **I32), torch.zeros(1, **I32)
        sm.kv_check(self.tables, M, self.rc, self.free_list, self.free_top, viol, st, sm.alloc_workspace(sm.OP_KV_CHECK, 0, 0, P=P))
        assert viol.tolist() == [0] * sm.KV_CHECK_KINDS
        for s in range(S):
            h = self.hist[s]
            if not h:
                assert (self.tables[s] == -1).all()
                continue
            k, v = self.gather(s, len(h))
            x = self.emb[torch.tensor(h, device="cuda")].double()
            assert torch.equal(v, x[:, HQ + HKV:]), s
            y = x[:, HQ:HQ + HKV]
            y = y / (y.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * self.kw.double()
            c, n = (f(self.angles[:len(h)]).cuda()[:, None] for f in (torch.cos, torch.sin))
            a, b = y[..., :D // 2], y[..., D // 2:]
            want = torch.cat([a * c - b * n, b * c + a * n], -1)
            mag = (a.abs() + b.abs()).repeat(1, 1, 2)
            tol = self.u * want.abs() + self.sub + (D + 16) * 2.0 ** -24 * mag
            assert ((k - want).abs() <= tol).all(), (s, float(((k - want).abs() - tol).max()))

    def check_attention(self, q, out):
        G = HQ // HKV
        for s in range(S):
            k, v = self.gather(s, self.len)
            see = torch.ones(self.len, device="cuda", dtype=torch.bool).repeat(R, 1).tril(self.len - R)
            for h in range(HKV):
                x = q[s, :, h * G:(h + 1) * G].double().reshape(R * G, D)
                ok = see.repeat_interleave(G, 0)
                z = (x @ k[:, h].t() * D ** -0.5).masked_fill(~ok, -math.inf)
                d = (D + 4) * 2.0 ** -24 * ((x.abs() @ k[:, h].abs().t()) * D ** -0.5).masked_fill(~ok, 0).amax(1, keepdim=True)
                p = (z - z.amax(1, keepdim=True)).exp()
                tot = p.sum(1, keepdim=True)
                want, mag = p @ v[:, h] / tot, p @ v[:, h].abs() / tot
                lost = min(self.sub, 1.0) * (ok.double() @ v[:, h].abs()) / tot
                tol = self.u * want.abs() + self.sub + (self.u + 4 * d + 2 * (self.len + 64) * 2.0 ** -24) * mag + lost
                got = out[s, :, h * G:(h + 1) * G].double().reshape(R * G, D)
                assert ((got - want).abs() <= tol).all(), (s, h)


@pytest.mark.parametrize("dt,layout", [("bf16", "token"), ("f16", "head")])
@pytest.mark.parametrize("side", [False, True])
@pytest.mark.parametrize("tau", [0.95, 2.0])
def test_rounds_of_a_server(dt, layout, side, tau):
    stream = torch.cuda.Stream() if side else torch.cuda.current_stream()
    with torch.cuda.stream(stream):
        sv = Server(dt, layout, seed=5)
        for b in range(B):
            sv.admit(b, PLEN)
        sv.len = PLEN
        sv.check_pages()
        resampled = sum(sv.round(t, tau) for t in range(4))
        sv.retire(1)
        sv.check_pages()
        sv.compact()
        sv.check_pages()
        sv.admit(1, sv.len)
        sv.check_pages()
        resampled += sum(sv.round(4 + t, tau) for t in range(3))
        # particles were exchanged, with tau > 1 in every round of every prompt
        assert resampled == 7 * B if tau > 1 else resampled > 0
    stream.synchronize()


class Pass:
    """One round's pass over fixed buffers: write, attend, score."""

    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        blocks = -(-(300 + R) // BS)
        self.tables = torch.randperm(S * blocks, generator=g).int().view(S, blocks).cuda()
        self.tables[:, :10] = self.tables[::N, :10].repeat_interleave(N, 0)  # prompts share 160 tokens,
        if seed % 2:
            self.tables[:, :18] = self.tables[::N, :18].repeat_interleave(N, 0)  # or 288
        self.k, self.v = (torch.randn(S * blocks, BS, HKV, D, generator=g).bfloat16().cuda() for _ in range(2))
        self.lens = torch.randint(290, 301, (S,), generator=g, dtype=torch.int32).cuda()
        self.x = torch.randn(S, R, HQ + 2 * HKV, D, generator=g).bfloat16().cuda()
        a = torch.arange(blocks * BS).double()[:, None] * 10000.0 ** (-torch.arange(D // 2).double() / (D // 2))
        self.cos_sin = torch.cat([a.cos(), a.sin()], 1).float().cuda()
        self.head = (torch.randn(HQ * D, V, generator=g) / 8).bfloat16().cuda()
        self.q, self.out = (torch.empty(S, R, HQ, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.lse, self.logits = torch.empty(S, R, HQ, device="cuda"), torch.empty(S * R, V, dtype=torch.bfloat16, device="cuda")
        self.ids, self.top = torch.empty(S * R, 5, **I32), torch.empty(S * R, 5, device="cuda")
        self.entropy, self.st = torch.empty(S * R, device="cuda"), torch.zeros(1, **I32)
        self.ws = sm.alloc_workspace(sm.OP_TREE_ATTN, B, N, K=R, V=HQ * D, P=HKV)
        self.ws_lp = sm.alloc_workspace(sm.OP_LOGPROBS, S * R, 1, K=5, V=V)

    def run(self):
        x = self.x
        sm.qk_norm_rope(x[:, :, :HQ], x[:, :, HQ:HQ + HKV], x[:, :, HQ + HKV:], self.lens, self.tables, self.k, self.v, self.q,
                        self.st, cos_sin=self.cos_sin)
        sm.tree_attention(self.q, self.k, self.v, self.tables, self.lens, B, N, D ** -0.5, self.out, self.st, self.ws, lse=self.lse)
        torch.mm(self.out.view(S * R, HQ * D), self.head, out=self.logits)
        sm.token_logprobs(self.logits, S * R, V, 1.0, self.st, self.ws_lp, out_entropy=self.entropy, top_ids=self.ids, top_logp=self.top)

    def results(self):
        assert int(self.st) == 0
        return [t.clone() for t in (self.q, self.out, self.lse, self.logits, self.ids, self.top, self.entropy)]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_two_passes_at_once():
    one, two = Pass(1), Pass(2)
    alone = []
    for p in (one, two):
        p.run()
        torch.cuda.synchronize()
        alone.append(p.results())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for p in (one, two):
            p.out.fill_(3.0)
            p.ids.fill_(-2)
        torch.cuda.synchronize()
        for p, s in zip((one, two), streams):
            with torch.cuda.stream(s):
                p.run()
                p.run()
        torch.cuda.synchronize()
        assert same(one.results(), alone[0]) and same(two.results(), alone[1])


def test_a_captured_pass():
    p = Pass(1)
    p.run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        p.run()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.run()
    inputs = [Pass(seed) for seed in (1, 2, 3, 1)]
    for other in inputs:  # other inputs in the same buffers, eager work between the replays
        for name in ("tables", "k", "v", "lens", "x", "head"):
            getattr(p, name).copy_(getattr(other, name))
        p.out.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        got = p.results()
        other.run()
        torch.cuda.synchronize()
        assert same(got, other.results())
        graph.replay()
        p.run()
        torch.cuda.synchronize()
        assert same(p.results(), got)
