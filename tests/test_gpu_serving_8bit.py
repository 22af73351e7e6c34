"""The operators together on 8-bit pages, as a server runs them: prompts come in packed chunks
(kv_append, prompt_attention), are forked, reserved and copied on write (kv_fork, kv_reassign, kv_copy
with scales); each round writes its new tokens (kv_append), attends (tree_attention) and resamples
(resample_kv_reassign, kv_copy); a prompt retires (kv_free), the pool is compacted (kv_compact, kv_copy)
and another is admitted.  After every step the pages, read through the tables and scales, have to hold
each particle's own history, and every attention's rows are held to the definition over them.

Bounds on a held element: its first rounding (2^-4 |y|, and half e4m3's smallest step, 2^-10, in units of the
scale), once more that 2^-10 for each growth of the block's scale (which roundings of what falls below e4m3's
normal range add; a value in it stays), a block growing 16 times at most here since every call of the test
writes one token or more; and the fp32 steps of norm and rotation, (D + 16) 2^-24 (|a| + |b|) as in the rounds on
16-bit pages.  Attention as in attention_checks, over what the pages hold."""
import math

import pytest
import torch

import smc_verification_resampling_amd as sm
from attention_checks import DT, E4M3, check_rows, tokens_at

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")
B, N, R, HQ, HKV, D, V, BS, EPS = 3, 4, 4, 4, 2, 64, 777, 16, 1e-6
S, M, P = B * N, 9, 100


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


class Server:
    def __init__(self, dt, layout, seed):
        g = torch.Generator().manual_seed(seed)
        self.dt, self.g = dt, g
        self.emb = (torch.randn(V, HQ + 2 * HKV, D, generator=g) * torch.exp(torch.randn(V, 1, 1, generator=g))).to(DT[dt]).cuda()
        self.kw = (1 + 0.1 * torch.randn(D, generator=g)).to(DT[dt]).cuda()
        self.angles = torch.arange(M * BS).double()[:, None] * 10000.0 ** (-torch.arange(D // 2).double() / (D // 2))
        self.cos_sin = torch.cat([self.angles.cos(), self.angles.sin()], 1).float().cuda()
        shape = (P, BS, HKV, D) if layout == "token" else (P, HKV, BS, D)
        kv = [torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2)]
        self.k, self.v = kv if layout == "token" else [x.transpose(1, 2) for x in kv]
        self.sk, self.sv = (torch.full((P, HKV), 255, dtype=torch.uint8, device="cuda") for _ in range(2))
        self.tables, self.rc = torch.full((S, M), -1, **I32), torch.zeros(P, **I32)
        self.free_list, self.free_top = torch.randperm(P, generator=g).int().cuda(), torch.tensor([P], **I32)
        self.st = torch.zeros(1, **I32)
        self.cow, self.cow_n = torch.full((S, 3), -7, **I32), torch.zeros(1, **I32)
        self.ws_kv = {n: sm.alloc_workspace(sm.OP_KV, n, N, P=P).zero_() for n in (1, B)}
        self.ws_attn = sm.alloc_workspace(sm.OP_TREE_ATTN, B, N, K=R, V=HQ * D, P=HKV)
        self.ws_prompt = sm.alloc_workspace(sm.OP_PROMPT_ATTN, B, B * 50, K=D, V=HQ * D, P=HKV)
        self.hist = [[] for _ in range(S)]
        self.len = 0

    def rows(self, tokens, lens, ctx, tables):
        """Writes packed tokens behind ctx; their queries and sums of lengths."""
        x = self.emb[tokens.long()]
        q = torch.empty(len(tokens), HQ, D, dtype=DT[self.dt], device="cuda")
        cu = torch.tensor([0] + lens, device="cuda").cumsum(0).int()
        sm.kv_append(x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:], cu, ctx, tables, self.k, self.v, q, self.st, k_scales=self.sk, v_scales=self.sv,
                     k_weight=self.kw, eps=EPS, cos_sin=self.cos_sin)
        return q, cu

    def copy(self, moves, count):
        sm.kv_copy([self.k, self.v], moves, count, self.st, scales=[self.sk, self.sv])

    def admit(self, prompts, length, chunk):
        """Prompts come in together, `chunk` tokens of each at a time; their first tokens may be fewer."""
        firsts = torch.tensor([b * N for b in prompts], device="cuda")
        need = -(-length // BS)
        for b in prompts:
            top = int(self.free_top)
            ids = self.free_list[top - need:top].flip(0)
            self.free_top -= need
            self.tables[b * N, :need] = ids
            self.rc[ids.long()] = 1
        text = torch.randint(0, V, (len(prompts), length), generator=self.g, dtype=torch.int32).cuda()
        done = [0] * len(prompts)
        while min(done) < length:
            lens = [min(chunk - 3 * j if d == 0 else chunk, length - d) for j, d in enumerate(done)]
            ctx = torch.tensor(done, **I32)
            tables = self.tables[firsts].contiguous()
            tokens = torch.cat([text[j, d:d + n] for j, (d, n) in enumerate(zip(done, lens))])
            q, cu = self.rows(tokens, lens, ctx, tables)
            out, lse = torch.full_like(q, 9.0), torch.empty(len(tokens), HQ, device="cuda")
            sm.prompt_attention(q, self.k, self.v, tables, ctx, cu, D ** -0.5, out, self.st, self.ws_prompt, k_scales=self.sk, v_scales=self.sv, lse=lse, max_len=length)
            for j, (d, n) in enumerate(zip(done, lens)):
                if n:
                    t = slice(int(cu[j]), int(cu[j + 1]))
                    self.check_rows(int(firsts[j]), d + n, n, q[t], out[t], lse[t])
            done = [d + n for d, n in zip(done, lens)]
        sm.kv_fork(torch.tensor([int(b in prompts) for b in range(B)], **I32), B, N, self.tables, self.rc, self.st)
        for j, b in enumerate(prompts):
            sm.kv_reassign(torch.arange(N, **I32), torch.zeros(1, **I32), 1, N, self.tables[b * N:(b + 1) * N], BS, length, R, self.rc, self.free_list,
                           self.free_top, self.cow, self.cow_n, self.st, self.ws_kv[1])
            assert int(self.cow_n) == (N - 1 if length % BS else 0)
            self.copy(self.cow, self.cow_n)
            for n in range(N):
                self.hist[b * N + n] = text[j].tolist()

    def round(self, t, tau):
        tokens = torch.randint(0, V, (S, R), generator=self.g, dtype=torch.int32).cuda()
        ctx = torch.full((S,), self.len, **I32)
        q, _ = self.rows(tokens.view(-1), [R] * S, ctx, self.tables)
        q = q.view(S, R, HQ, D)
        out, lse = torch.full_like(q, 9.0), torch.empty(S, R, HQ, device="cuda")
        sm.tree_attention(q, self.k, self.v, self.tables, ctx, B, N, D ** -0.5, out, self.st, self.ws_attn, max_len=M * BS, lse=lse, k_scales=self.sk,
                          v_scales=self.sv)
        for s in range(S):
            self.hist[s] += tokens[s].tolist()
        self.len += R
        self.check_pages()
        for s in range(S):
            self.check_rows(s, self.len, R, q[s], out[s], lse[s])
        weights = torch.randn(B, N, generator=self.g).cuda()
        anc, ess, res = torch.empty(B, N, **I32), torch.empty(B, device="cuda"), torch.empty(B, **I32)
        sm.resample_kv_reassign(weights, B, N, tau, 11, t, anc, ess, res, self.tables, BS, self.len, R, self.rc, self.free_list, self.free_top, self.cow,
                                self.cow_n, self.st, self.ws_kv[B])
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
        sm.kv_compact(self.tables, BS, self.rc, self.free_list, self.free_top, moves, n, self.st, sm.alloc_workspace(sm.OP_KV_COMPACT, 0, 0, P=P))
        self.copy(moves, n)
        assert int(n) > 0

    def held(self, s, n):
        pos = torch.arange(n, device="cuda")
        at = self.tables[s].long()[pos // BS]
        assert (at >= 0).all()
        return [tokens_at(c, x, at, pos % BS, torch.float64) for c, x in ((self.k, self.sk), (self.v, self.sv))] + [at]

    def check_rows(self, s, total, n, q, out, lse):
        pos = torch.arange(total, device="cuda")
        at = self.tables[s].long()[pos // BS]
        k, v = (tokens_at(c, x, at, pos % BS, DT[self.dt]) for c, x in ((self.k, self.sk), (self.v, self.sv)))
        check_rows(q, k, v, pos[None] <= (total - n + torch.arange(n, device="cuda"))[:, None], D ** -0.5, out, lse, self.dt, s)

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
            k, v, at = self.held(s, len(h))
            x = self.emb[torch.tensor(h, device="cuda")].double()
            y = x[:, HQ:HQ + HKV]
            y = y / (y.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * self.kw.double()
            c, n = (f(self.angles[:len(h)]).cuda()[:, None] for f in (torch.cos, torch.sin))
            a, b = y[..., :D // 2], y[..., D // 2:]
            y = torch.cat([a * c - b * n, b * c + a * n], -1)
            mag = (a.abs() + b.abs()).repeat(1, 1, 2)
            for got, want, codes, f in ((k, y, self.sk, (D + 16) * 2.0 ** -24 * mag), (v, x[:, HQ + HKV:], self.sv, 0.0)):
                unit = 2.0 ** (codes[at].double() - 127)[..., None]
                tol = 2.0 ** -4 * want.abs() + 17 * 2.0 ** -10 * unit + f
                assert ((got - want).abs() <= tol).all(), (s, float(((got - want).abs() - tol).max()))


@pytest.mark.parametrize("dt,layout", [("bf16", "token"), ("f16", "head")])
@pytest.mark.parametrize("side", [False, True])
@pytest.mark.parametrize("tau", [0.6, 2.0])
def test_rounds_of_a_server_on_8_bit_pages(dt, layout, side, tau):
    stream = torch.cuda.Stream() if side else torch.cuda.current_stream()
    with torch.cuda.stream(stream):
        sv = Server(dt, layout, seed=5)
        sv.admit([0, 1, 2], 45, 20)
        sv.len = 45
        sv.check_pages()
        resampled = sum(sv.round(t, tau) for t in range(4))
        sv.retire(1)
        sv.check_pages()
        sv.compact()
        sv.check_pages()
        sv.admit([1], sv.len, 50)
        sv.check_pages()
        resampled += sum(sv.round(4 + t, tau) for t in range(3))
        assert resampled > 0
    stream.synchronize()


def test_two_prefills_at_once():
    """Two streams, each with its own sequences and workspace, on one pool."""
    out = []
    for parallel in (False, True):
        sv = Server("bf16", "token", seed=8)
        sv.tables[:2, :3] = torch.arange(6, **I32).view(2, 3)
        text = torch.randint(0, V, (2, 40), generator=sv.g, dtype=torch.int32).cuda()
        ws = [sm.alloc_workspace(sm.OP_PROMPT_ATTN, 1, 40, K=D, V=HQ * D, P=HKV) for _ in range(2)]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)] if parallel else [torch.cuda.current_stream()] * 2
        got = []
        for j, st in enumerate(streams):
            with torch.cuda.stream(st):
                q, cu = sv.rows(text[j], [40], None, sv.tables[j:j + 1])
                o = torch.empty_like(q)
                sm.prompt_attention(q, sv.k, sv.v, sv.tables[j:j + 1], None, cu, D ** -0.5, o, sv.st, ws[j], k_scales=sv.sk, v_scales=sv.sv)
                got.append(o)
        torch.cuda.synchronize()
        assert int(sv.st) == 0
        out.append(torch.stack(got))
    assert torch.equal(*out)
