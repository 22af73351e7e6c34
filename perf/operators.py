"""The serving operators around an SMC-SD round, as cases to measure: query/key norms with rotation into the paged
cache, attention of drafted trees over that cache, log-probabilities with entropy and top alternatives, and the
pages' own operations (copy, fork, free, compact).  With `own` false a pass runs the operators' plain form in torch;
with `own` true it calls the library.  Sizes follow workloads/configs.py."""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # One new token for each of 4 particles on a short context: the latency of a single decode step.
        dict(name="attention, one token", op="attention", dtype="f16", B=1, N=4, R=1, Hq=8, Hkv=2, D=64, ctx=16, private=0,
             block=4, shared=False, tree=False, layout="token"),
        # The batched round: 32 prompts x 16 particles score 5 positions, prompt blocks shared, about 80 tokens of their own.
        dict(name="attention, batched round", op="attention", dtype="bf16", B=32, N=16, R=5, Hq=32, Hkv=8, D=128, ctx=2048, private=80,
             block=16, shared=True, tree=False, layout="head"),
        # The wide-particle round with unshared blocks and ragged lengths up to 4096: bound by reading every page.
        dict(name="attention, wide unshared", op="attention", dtype="bf16", B=4, N=64, R=9, Hq=32, Hkv=8, D=128, ctx=4093, private=0,
             block=16, shared=False, tree=False, layout="token"),
        # One long document and a tree of 64 drafted nodes: the work is split over the keys and joined.
        dict(name="attention, long tree", op="attention", dtype="bf16", B=1, N=1, R=64, Hq=16, Hkv=4, D=128, ctx=131071, private=0,
             block=16, shared=False, tree=True, layout="head"),
        # The tiny round's new tokens: latency.
        dict(name="norm and rotation, tiny", op="rope", dtype="f16", B=1, N=4, R=3, Hq=8, Hkv=2, D=64, rot=64, ctx=16, private=0, block=4,
             interleaved=True, norm=True, layout="token"),
        # The batched round's 2560 new tokens, read out of one fused projection.
        dict(name="norm and rotation, batched", op="rope", dtype="bf16", B=32, N=16, R=5, Hq=32, Hkv=8, D=128, rot=128, ctx=2048, private=80,
             block=16, interleaved=False, norm=True, layout="head"),
        # One sequence's five positions of a 32000-entry vocabulary: latency.
        dict(name="log probabilities, few rows", op="logprobs", dtype="bf16", n=5, V=32000, C=1, k=5, T=1.0, pad=0, masked=False),
        # The batched round's target rows, with the twenty best alternatives.
        dict(name="log probabilities, batched", op="logprobs", dtype="bf16", n=2560, V=128256, C=1, k=20, T=0.8, pad=0, masked=False),
        # 32-bit rows of odd length and stride, part of the entries masked by a grammar.
        dict(name="log probabilities, masked", op="logprobs", dtype="f32", n=576, V=152063, C=4, k=8, T=1.0, pad=2, masked=True),
        # The copy-on-write list of a batched round on four layers' pages.
        dict(name="pages, copy on write", op="copy", B=32, N=16, Hkv=8, D=128, block=16, layers=4, blocks=6144, layout="head"),
        # Two prompts retire and two are admitted: their tables are freed, then forked from particle 0.
        dict(name="pages, retire and admit", op="admit", B=32, N=16, block=16, ctx=2048, private=80, churn=2),
        # A fragmented pool made dense, with the data of two layers moved.
        dict(name="pages, compact", op="compact", S=128, slots=132, Hkv=8, D=128, block=16, layers=2, blocks=24576, share=0.4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "rope", "logprobs", "logprobs", "copy", "admit", "compact"])
    if op == "attention":
        D = rng.choice([64, 64, 80, 96, 128, 128, 128, 192, 256])
        Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 4, 7, 8])
        N, R, ctx = _log(rng, 1, 64), rng.choice([1, 1, 3, 5, 9, _log(rng, 2, 64)]), _log(rng, 1, 65536)
        B = _log(rng, 1, 32)
        while B > 1 and B * N * (ctx + R) * Hkv * D > 5e8:
            B = (B + 1) // 2
        while N > 1 and B * N * (ctx + R) * Hkv * D > 5e8:
            N = (N + 1) // 2
        while ctx > 64 and 4 * B * N * R * G * Hkv * (ctx + R) * D > 1e11:
            ctx = (ctx + 1) // 2
        shared = rng.random() < 0.5
        return dict(op=op, dtype=rng.choice(["bf16", "f16"]), B=B, N=N, R=R, Hq=Hkv * G, Hkv=Hkv, D=D, ctx=ctx,
                    private=_log(rng, 1, 300) if shared else 0, block=rng.choice([1, 8, 16, 16, 24, 64, 128]), shared=shared, tree=rng.random() < 0.5,
                    layout=rng.choice(["token", "head"]))
    if op == "rope":
        D = rng.choice([64, 80, 128, 128, 192, 256])
        Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 7, 8])
        return dict(op=op, dtype=rng.choice(["bf16", "f16"]), B=_log(rng, 1, 32), N=_log(rng, 1, 16), R=rng.choice([1, 3, 5]), Hq=min(32, Hkv * G), Hkv=Hkv,
                    D=min(D, 128) if Hkv * G > 16 else D, rot=rng.choice([32, 64, 64]), ctx=_log(rng, 1, 32768 if Hkv < 4 else 2048),
                    private=_log(rng, 1, 80), block=rng.choice([4, 16, 24, 64]), interleaved=rng.random() < 0.5, norm=rng.random() < 0.8,
                    layout=rng.choice(["token", "head"]))
    if op == "logprobs":
        V = _log(rng, 8, 200000)
        n = max(1, min(_log(rng, 1, 2560), int(8e7 / V)))
        return dict(op=op, dtype=rng.choice(["bf16", "f32"]), n=n, V=V, C=rng.choice([1, 1, 2, 8]), k=min(V, rng.choice([0, 1, 5, 20, 32, 64])),
                    T=rng.choice([0.5, 0.8, 1.0, 1.3]), pad=rng.choice([0, 0, 1, 6, 64]), masked=rng.random() < 0.4)
    if op == "copy":
        Hkv = rng.choice([1, 2, 4, 8])
        return dict(op=op, B=_log(rng, 1, 32), N=_log(rng, 1, 16), Hkv=Hkv, D=rng.choice([64, 80, 128]), block=rng.choice([1, 4, 16, 24, 32]),
                    layers=rng.randint(1, 4), blocks=_log(rng, 1200, 3000), layout=rng.choice(["token", "head"]))
    if op == "admit":
        B = _log(rng, 2, 32)
        return dict(op=op, B=B, N=_log(rng, 1, 16), block=rng.choice([4, 16, 24]), ctx=_log(rng, 1, 2048), private=_log(rng, 1, 80), churn=rng.randint(1, max(1, B // 4)))
    return dict(op=op, S=_log(rng, 1, 128), slots=_log(rng, 1, 132), Hkv=rng.choice([1, 2, 4]), D=rng.choice([64, 128]), block=rng.choice([4, 16, 24]),
                layers=rng.randint(1, 2), blocks=_log(rng, 17000, 24000), share=rng.uniform(0.0, 0.8))


# ------------------------------------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _i32(x):
    return x.to(torch.int32).contiguous()


def _cache(blocks, block, Hkv, D, dtype, layout, g):
    """Pages seen as [blocks, block, Hkv, D], laid out by token or by head."""
    if layout == "token":
        return torch.randn(blocks, block, Hkv, D, generator=g, device=DEV, dtype=torch.float32 if blocks * block * Hkv * D < 1 << 28 else dtype).to(dtype)
    return _cache(blocks, Hkv, block, D, dtype, "token", g).transpose(1, 2)


def _tables(case, g):
    """Block tables with room for each sequence's context and its new tokens, in a shuffled pool; the context lengths."""
    B, N, bs = case["B"], case["N"], case["block"]
    S, ctx = B * N, case["ctx"]
    shared = case.get("shared", case["private"] > 0)
    first = ctx // bs if shared else 0  # leading blocks that a prompt's particles share
    if shared:
        lens = ctx + torch.randint(0, case["private"] + 1, (S,), generator=g, device=DEV)
    elif S > 1:
        lens = torch.randint((ctx + 1) // 2, ctx + 1, (S,), generator=g, device=DEV)
    else:
        lens = torch.full((1,), ctx, device=DEV)
    slots = -(-(ctx + case["private"] + case["R"]) // bs)
    blocks = B * first + S * (slots - first)
    ids = torch.randperm(blocks, generator=g, device=DEV)
    tables = torch.empty(S, slots, dtype=torch.int64, device=DEV)
    tables[:, :first] = ids[: B * first].view(B, 1, first).expand(B, N, first).reshape(S, first)
    tables[:, first:] = ids[B * first:].view(S, slots - first)
    return _i32(tables), _i32(lens), blocks


def _prepare_attention(c, g):
    S, R, Hq, Hkv, D, dt = c["B"] * c["N"], c["R"], c["Hq"], c["Hkv"], c["D"], DTYPES[c["dtype"]]
    tables, lens, blocks = _tables(c, g)
    k = _cache(blocks, c["block"], Hkv, D, dt, c["layout"], g)
    v = _cache(blocks, c["block"], Hkv, D, dt, c["layout"], g)
    q = (1.5 * torch.randn(S, R, Hq, D, generator=g, device=DEV)).to(dt)
    mask = None
    if c["tree"]:  # node j's parent is an earlier node: it sees its ancestors and itself
        node = torch.arange(R, device=DEV)
        parent = (torch.rand(S, R, generator=g, device=DEV) * node).long()
        reach = torch.eye(R, device=DEV).repeat(S, 1, 1)
        step = torch.zeros(S, R, R, device=DEV).scatter_(2, parent[:, :, None], 1.0)
        step[:, 0] = 0
        for _ in range(max(1, R.bit_length())):
            reach = ((reach + step @ reach) > 0).float()
            step = ((step @ step) > 0).float()
        mask = ((reach > 0).long() << node).sum(-1)
    return dict(q=q, k=k, v=v, tables=tables, lens=lens, mask=mask, N=c["N"], scale=D ** -0.5, longest=c["ctx"] + c["private"] + R,
                out=torch.empty_like(q), lse=torch.empty(S, R, Hq, device=DEV), status=torch.zeros(1, dtype=torch.int32, device=DEV))


def _prepare_rope(c, g):
    S, R, Hq, Hkv, D, dt = c["B"] * c["N"], c["R"], c["Hq"], c["Hkv"], c["D"], DTYPES[c["dtype"]]
    tables, lens, blocks = _tables(c, g)
    qkv = torch.randn(S, R, Hq + 2 * Hkv, D, generator=g, device=DEV).to(dt)
    longest = c["ctx"] + c["private"] + R
    angle = torch.arange(longest, device=DEV, dtype=torch.float64)[:, None] * 500000.0 ** (-torch.arange(0, c["rot"], 2, device=DEV, dtype=torch.float64) / c["rot"])
    w = [(1 + 0.2 * torch.randn(D, generator=g, device=DEV)).to(dt) if c["norm"] else None for _ in range(2)]
    return dict(q=qkv[:, :, :Hq], k=qkv[:, :, Hq:Hq + Hkv], v=qkv[:, :, Hq + Hkv:], q_weight=w[0], k_weight=w[1], eps=1e-6, rot=c["rot"], interleaved=c["interleaved"],
                table=torch.cat([angle.cos(), angle.sin()], 1).float(), tables=tables, lens=lens, k_cache=_cache(blocks, c["block"], Hkv, D, dt, c["layout"], g),
                v_cache=_cache(blocks, c["block"], Hkv, D, dt, c["layout"], g), q_out=torch.empty(S, R, Hq, D, dtype=dt, device=DEV),
                status=torch.zeros(1, dtype=torch.int32, device=DEV))


def _prepare_logprobs(c, g):
    n, V, k, C = c["n"], c["V"], c["k"], c["C"]
    rank = torch.randperm(V, generator=g, device=DEV).float() + 1
    x = torch.empty(n, V + c["pad"], dtype=DTYPES[c["dtype"]], device=DEV)
    noise = torch.randn(n, V, generator=g, device=DEV)
    x[:, :V] = noise.mul_(0.3).sub_(1.1 * rank.log())
    if c["masked"]:  # a grammar leaves about a third of the vocabulary, and always the first entry
        off = torch.rand(1, V, generator=g, device=DEV) < 0.66
        off[:, 0] = False
        x[:, :V].masked_fill_(off, -math.inf)
    x[:, V:] = 7.0  # what stands in the rows' padding is no logit
    i32 = dict(dtype=torch.int32, device=DEV)
    return dict(x=x, V=V, T=c["T"], tokens=_i32(torch.randint(0, V, (n, C), generator=g, device=DEV)), logp=torch.empty(n, C, device=DEV),
                entropy=torch.empty(n, device=DEV), lse=torch.empty(n, device=DEV), top_ids=torch.empty(n, k, **i32), top_logp=torch.empty(n, k, device=DEV),
                status=torch.zeros(1, **i32))


def _prepare_copy(c, g):
    # Each particle holds at most one partial tail: about half of them diverge from it in a round.
    S, P = c["B"] * c["N"], c["blocks"]
    ids = torch.randperm(P, generator=g, device=DEV)
    at = torch.randint(0, S, (S,), generator=g, device=DEV)
    count = max(1, S // 2)
    moves = torch.stack([ids[at], ids[S:2 * S], torch.randint(0, c["block"] + 1, (S,), generator=g, device=DEV)], 1)
    return dict(caches=[_cache(P, c["block"], c["Hkv"], c["D"], torch.bfloat16, c["layout"], g) for _ in range(2 * c["layers"])], moves=_i32(moves),
                count=torch.full((1,), count, dtype=torch.int32, device=DEV), status=torch.zeros(1, dtype=torch.int32, device=DEV))


def _prepare_admit(c, g):
    # `churn` prompts are done; as many new ones have their prompt's blocks in particle 0 only.
    B, N, bs, n = c["B"], c["N"], c["block"], c["churn"]
    used, first = -(-(c["ctx"] + c["private"]) // bs), -(-c["ctx"] // bs)
    P = 2 * B * first + 2 * B * N * (used - first + 1)
    ids = torch.randperm(P, generator=g, device=DEV)
    tables = torch.full((B, N, used + 4), -1, dtype=torch.int64, device=DEV)
    tables[:, :, :first] = ids[: B * first].view(B, 1, first)
    tables[:, :, first:used] = ids[B * first: B * first + B * N * (used - first)].view(B, N, used - first)
    order = torch.randperm(B, generator=g, device=DEV)
    gone, new = order[:n], order[n:2 * n]
    tables[new, 1:] = -1
    tables[new, 0, first:] = -1
    rc = torch.zeros(P + 1, dtype=torch.int64, device=DEV).scatter_add_(0, torch.where(tables >= 0, tables, P).view(-1), torch.ones(tables.numel(), dtype=torch.int64, device=DEV))[:P]
    free = (rc == 0).nonzero().view(-1).flip(0)
    stack = torch.zeros(P, dtype=torch.int64, device=DEV)
    stack[: len(free)] = free
    freed, forked = torch.zeros(B, N, dtype=torch.int64, device=DEV), torch.zeros(B, dtype=torch.int64, device=DEV)
    freed[gone] = 1
    forked[new] = 1
    kept = [_i32(t) for t in (tables.view(B * N, -1), rc, stack, torch.tensor([len(free)], device=DEV))]
    return dict(kept=kept, work=[t.clone() for t in kept], freed=_i32(freed.view(-1)), forked=_i32(forked), B=B, N=N, status=torch.zeros(1, dtype=torch.int32, device=DEV))


def _prepare_compact(c, g):
    # Blocks of live sequences lie anywhere in the pool; a part of each sequence's blocks is its neighbour's too.
    S, M, P = c["S"], c["slots"], c["blocks"]
    tables = torch.randperm(P, generator=g, device=DEV)[: S * M].view(S, M)
    both = int(M * c["share"])
    tables[1::2, :both] = tables[: S - S % 2: 2, :both]
    rc = torch.zeros(P, dtype=torch.int64, device=DEV).scatter_add_(0, tables.reshape(-1), torch.ones(S * M, dtype=torch.int64, device=DEV))
    free = (rc == 0).nonzero().view(-1)
    stack = torch.zeros(P, dtype=torch.int64, device=DEV)
    stack[: len(free)] = free[torch.randperm(len(free), generator=g, device=DEV)]
    kept = [_i32(t) for t in (tables, rc, stack, torch.tensor([len(free)], device=DEV))]
    i32 = dict(dtype=torch.int32, device=DEV)
    return dict(kept=kept, work=[t.clone() for t in kept], block=c["block"], caches=[_cache(P, c["block"], c["Hkv"], c["D"], torch.bfloat16, "token", g) for _ in range(2 * c["layers"])],
                moves=torch.zeros(P // 2, 3, **i32), count=torch.zeros(1, **i32), status=torch.zeros(1, **i32))


def prepare(case, seed):
    makers = {"attention": _prepare_attention, "rope": _prepare_rope, "logprobs": _prepare_logprobs, "copy": _prepare_copy, "admit": _prepare_admit, "compact": _prepare_compact}
    return dict(makers[case["op"]](case, _gen(seed)), op=case["op"])


# ------------------------------------------------------------------------------------------------ the plain form
def _attention(s):
    q, tables, lens = s["q"], s["tables"].long(), s["lens"].long()
    S, R, Hq, D = q.shape
    bs, Hkv = s["k"].shape[1:3]
    L = s["longest"]
    pos = torch.arange(L, device=DEV)
    block = tables[:, pos // bs].clamp_min(0)
    node = pos[None] - lens[:, None]  # which new token a position holds; negative: context
    if s["mask"] is None:
        seen = node[:, None] <= torch.arange(R, device=DEV)[None, :, None]
    else:
        bit = (s["mask"][:, :, None] >> node.clamp(0, R - 1)[:, None]) & 1
        seen = (node < 0)[:, None] | ((node < R)[:, None] & (bit != 0))
    k = s["k"][block, pos % bs].float().permute(0, 2, 3, 1)  # [S, Hkv, D, L]
    rows = q.float().view(S, R, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(S, Hkv, -1, D)
    score = torch.matmul(rows, k).view(S, Hkv, R, Hq // Hkv, L) * s["scale"]
    del k
    score.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    v = s["v"][block, pos % bs].float().permute(0, 2, 1, 3)  # [S, Hkv, L, D]
    out = torch.matmul(p.view(S, Hkv, -1, L), v).view(S, Hkv, R, Hq // Hkv, D) / torch.where(total == 0, 1.0, total)
    lse = (total.log() + top).squeeze(-1)
    return out.permute(0, 2, 1, 3, 4).reshape(S, R, Hq, D).to(q.dtype), lse.permute(0, 2, 1, 3).reshape(S, R, Hq)


def _norm_rotate(x, weight, s, cos, sin):
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * weight.float()
    rot = s["rot"]
    a, b = (x[..., :rot:2], x[..., 1:rot:2]) if s["interleaved"] else (x[..., :rot // 2], x[..., rot // 2:rot])
    turned = [a * cos - b * sin, b * cos + a * sin]
    turned = torch.stack(turned, -1).flatten(-2) if s["interleaved"] else torch.cat(turned, -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _rope(s):
    q, bs = s["q"], s["k_cache"].shape[1]
    S, R = q.shape[:2]
    pos = s["lens"].long()[:, None] + torch.arange(R, device=DEV)
    cos, sin = s["table"][pos][:, :, None].chunk(2, -1)
    block = s["tables"].long().gather(1, pos // bs)
    s["k_cache"][block, pos % bs] = _norm_rotate(s["k"], s["k_weight"], s, cos, sin).to(q.dtype)
    s["v_cache"][block, pos % bs] = s["v"]
    return _norm_rotate(q, s["q_weight"], s, cos, sin).to(q.dtype), s["k_cache"], s["v_cache"]


def _logprobs(s):
    x = s["x"][:, :s["V"]].float() + 0.0  # one zero only
    n, V = x.shape
    z = x * (1 / s["T"])
    top = z.amax(-1, keepdim=True)
    z = z - top
    e = z.exp()
    total = e.sum(-1, keepdim=True)
    entropy = total.squeeze(-1).log() - (e * z.clamp_min(-1e30)).sum(-1) / total.squeeze(-1)
    del e
    logp = z.gather(1, s["tokens"].long()) - total.log()
    k = s["top_ids"].shape[1]
    bits = x.view(torch.int32)
    bits = bits ^ ((bits >> 31) & 0x7FFFFFFF)  # the floats' order as whole numbers
    key = (bits.long() << 32) | (0xFFFFFFFF - torch.arange(V, device=DEV))  # equal values: the lowest index first
    ids = 0xFFFFFFFF - (key.topk(k, -1, sorted=True).values & 0xFFFFFFFF)
    best = z.gather(1, ids) - total.log()
    return logp, entropy, (top + total.log()).squeeze(-1), torch.where(best == -math.inf, -1, ids).int(), best


def _copy(caches, moves, count):
    src, dst, tokens = moves.long().unbind(1)
    use = torch.arange(len(moves), device=DEV) < count
    src = torch.where(use, src, dst)
    fresh = torch.arange(caches[0].shape[1], device=DEV)[None] < tokens[:, None]
    moved = [torch.where(fresh[:, :, None, None], c[src], c[dst]) for c in caches]
    [c.__setitem__(dst, m) for c, m in zip(caches, moved)]
    return caches


def _pool(s):
    """The pool's state as it was before the pass: block tables, reference counts, free stack and its top."""
    [w.copy_(k) for w, k in zip(s["work"], s["kept"])]
    return s["work"]


def _admit(s):
    tables, rc, stack, top = _pool(s)
    P = len(rc)
    lost = torch.where((s["freed"] != 0)[:, None] & (tables >= 0), tables, P).view(-1).long()
    less = torch.zeros(P + 1, dtype=torch.int32, device=DEV).scatter_add_(0, lost, torch.ones_like(lost, dtype=torch.int32))[:P]
    free = (less > 0) & (rc == less)
    rc -= less
    tables.masked_fill_((s["freed"] != 0)[:, None], -1)
    up = free.long().cumsum(0)
    room = torch.cat([stack, stack[:1]])
    room[torch.where(free, top + up[-1] - up, P)] = torch.arange(P, dtype=torch.int32, device=DEV)  # the highest id first
    stack.copy_(room[:P])
    top += up[-1].int()
    t = tables.view(s["B"], s["N"], -1)
    ids = t[:, 0]
    new = (s["forked"] != 0)[:, None] & (ids >= 0)
    t[:, 1:] = torch.where(new[:, None], ids[:, None], t[:, 1:])
    rc += torch.zeros(P + 1, dtype=torch.int32, device=DEV).scatter_add_(0, torch.where(new, ids, P).view(-1).long(), torch.full((ids.numel(),), s["N"] - 1, dtype=torch.int32, device=DEV))[:P]
    return tables, rc, stack, top


def _compact(s):
    tables, rc, stack, top = _pool(s)
    P = len(rc)
    live = rc > 0
    at = torch.arange(P, device=DEV)
    below = live.long().cumsum(0) - live.long()
    total = below[-1] + live[-1]
    hole, mover = (at < total) & ~live, (at >= total) & live
    order = hole.long().cumsum(0) - 1
    first = torch.zeros(P + 1, dtype=torch.int64, device=DEV)
    first[torch.where(hole, order, P)] = at  # the i-th hole
    to = torch.where(mover, first[(mover.long().cumsum(0) - 1).clamp_min(0)], at)  # every block's new id
    room = torch.zeros(P // 2 + 1, 3, dtype=torch.int32, device=DEV)
    room[torch.where(mover, mover.long().cumsum(0) - 1, P // 2)] = torch.stack([at, to, torch.full_like(at, s["block"])], 1).int()
    n = mover.sum()
    s["moves"].copy_(torch.where((torch.arange(P // 2, device=DEV) < n)[:, None], room[:-1], s["moves"]))
    s["count"].copy_(n)
    tables.copy_(torch.where(tables >= 0, to[tables.long().clamp_min(0)].int(), tables))
    fresh = torch.zeros(P + 1, dtype=torch.int32, device=DEV)
    fresh[torch.where(live, to, P)] = rc
    rc.copy_(fresh[:P])
    stack.copy_(torch.where(at < P - total, (P - 1 - at).int(), stack))
    top.copy_(P - total)
    src, dst = torch.where(mover, at, 0), torch.where(mover, to, 0)
    src, dst = src[mover], dst[mover]
    [c.__setitem__(dst, c[src]) for c in s["caches"]]
    return tables, rc, stack, top, s["moves"], s["count"], s["caches"]


# ------------------------------------------------------------------------------------------------ the library's calls
def _own(s):
    import smc_verification_resampling_amd as sm

    if s["op"] == "attention":
        S, R, Hq, D = s["q"].shape
        if "ws" not in s:
            s["ws"] = sm.alloc_workspace(sm.OP_TREE_ATTN, S // s["N"], s["N"], K=R, V=Hq * D, P=s["k"].shape[2])
        sm.tree_attention(s["q"], s["k"], s["v"], s["tables"], s["lens"], S // s["N"], s["N"], s["scale"], s["out"], s["status"], s["ws"],
                          tree_mask=s["mask"], lse=s["lse"], max_len=s["longest"])
        return s["out"], s["lse"]
    if s["op"] == "rope":
        sm.qk_norm_rope(s["q"], s["k"], s["v"], s["lens"], s["tables"], s["k_cache"], s["v_cache"], s["q_out"], s["status"], q_weight=s["q_weight"],
                        k_weight=s["k_weight"], eps=s["eps"], cos_sin=s["table"], interleaved=s["interleaved"])
        return s["q_out"], s["k_cache"], s["v_cache"]
    if s["op"] == "logprobs":
        n, k = s["top_ids"].shape
        if "ws" not in s:
            s["ws"] = sm.alloc_workspace(sm.OP_LOGPROBS, n, 1, K=k, V=s["V"])
        sm.token_logprobs(s["x"], n, s["V"], s["T"], s["status"], s["ws"], tokens=s["tokens"], out_logp=s["logp"], out_entropy=s["entropy"], out_lse=s["lse"],
                          top_ids=s["top_ids"], top_logp=s["top_logp"], row_stride=s["x"].shape[1])
        return s["logp"], s["entropy"], s["lse"], s["top_ids"], s["top_logp"]
    if s["op"] == "copy":
        sm.kv_copy(s["caches"], s["moves"], s["count"], s["status"])
        return s["caches"]
    tables, rc, stack, top = _pool(s)
    P = len(rc)
    if s["op"] == "admit":
        if "ws" not in s:
            s["ws"] = sm.alloc_workspace(sm.OP_KV_FREE, 0, 0, P=P)
        sm.kv_free(s["freed"], tables, rc, stack, top, s["status"], s["ws"])
        sm.kv_fork(s["forked"], s["B"], s["N"], tables, rc, s["status"])
        return tables, rc, stack, top
    if "ws" not in s:
        s["ws"] = sm.alloc_workspace(sm.OP_KV_COMPACT, 0, 0, P=P)
    sm.kv_compact(tables, s["block"], rc, stack, top, s["moves"], s["count"], s["status"], s["ws"])
    sm.kv_copy(s["caches"], s["moves"], s["count"], s["status"])
    return tables, rc, stack, top, s["moves"], s["count"], s["caches"]


def run(state):
    if own:
        return _own(state)
    if state["op"] == "copy":
        return _copy(state["caches"], state["moves"], state["count"])
    return {"attention": _attention, "rope": _rope, "logprobs": _logprobs, "admit": _admit, "compact": _compact}[state["op"]](state)


# ------------------------------------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "attention":
        S, e = c["B"] * c["N"], 2
        mean = c["ctx"] + c["private"] / 2 if c["shared"] else c["ctx"] * (0.75 if S > 1 else 1.0)
        keys = c["B"] * (c["ctx"] // c["block"] * c["block"]) + S * (mean - c["ctx"] // c["block"] * c["block"] + c["R"]) if c["shared"] else S * (mean + c["R"])
        return {"bytes": 2 * keys * c["Hkv"] * c["D"] * e + 2 * S * c["R"] * c["Hq"] * c["D"] * e + 4 * S * c["R"] * c["Hq"],
                "flops": 4.0 * S * c["R"] * c["Hq"] * c["D"] * (mean + (c["R"] + 1) / 2)}
    if c["op"] == "rope":
        rows = c["B"] * c["N"] * c["R"]
        return {"bytes": 2 * 2 * rows * (c["Hq"] + 2 * c["Hkv"]) * c["D"] + 4 * c["rot"] * rows, "flops": 8.0 * rows * (c["Hq"] + c["Hkv"]) * c["D"]}
    if c["op"] == "logprobs":
        return {"bytes": c["n"] * (c["V"] * (2 if c["dtype"] == "bf16" else 4) + 8 * (c["C"] + c["k"] + 1)), "flops": 6.0 * c["n"] * c["V"]}
    token = 2 * c["Hkv"] * c["D"] * 2 * c["layers"] if "layers" in c else 0  # bytes of a token in all layers' k and v
    if c["op"] == "copy":
        return {"bytes": 2 * max(1, c["B"] * c["N"] // 2) * (c["block"] / 2) * token, "flops": 0}
    if c["op"] == "admit":
        used = -(-(c["ctx"] + c["private"]) // c["block"])
        return {"bytes": 4 * (2 * c["churn"] * c["N"] * 2 * used + c["B"] * c["N"] + c["B"]) + 8 * 4 * c["B"] * c["N"] * (used + 4), "flops": 0}
    blocks = c["S"] * c["slots"] - (c["S"] // 2) * int(c["slots"] * c["share"])
    moved = blocks * (1 - blocks / c["blocks"])
    return {"bytes": 2 * moved * c["block"] * token + 4 * (2 * c["S"] * c["slots"] + 3 * c["blocks"] + 3 * moved), "flops": 0}


# ------------------------------------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "attention":
        S, R, Hq, D = s["q"].shape
        bs, Hkv = s["k"].shape[1:3]
        out, lse = torch.zeros(S, R, Hq, D, dtype=torch.float64, device=DEV), torch.full((S, R, Hq), -math.inf, dtype=torch.float64, device=DEV)
        for b, ctx in enumerate(s["lens"].tolist()):
            used = s["tables"][b, : -(-(ctx + R) // bs)].long()
            k = s["k"][used].reshape(-1, Hkv, D)[: ctx + R].double()
            v = s["v"][used].reshape(-1, Hkv, D)[: ctx + R].double()
            sees = torch.ones(R, ctx + R, dtype=torch.bool, device=DEV)
            if s["mask"] is None:
                sees[:, ctx:] = torch.ones(R, R, dtype=torch.bool, device=DEV).tril()
            else:
                sees[:, ctx:] = torch.stack([(s["mask"][b] >> j) % 2 == 1 for j in range(R)], 1)
            for h in range(Hkv):
                mine = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
                z = s["q"][b, :, mine].double().reshape(-1, D) @ k[:, h].t() * s["scale"]
                z = torch.where(sees.repeat_interleave(Hq // Hkv, 0), z, -math.inf)
                lse[b, :, mine] = torch.logsumexp(z, 1).view(R, -1)
                out[b, :, mine] = (torch.softmax(z, 1) @ v[:, h]).view(R, -1, D)
        return out, lse
    if s["op"] == "rope":
        bs, R, rot = s["k_cache"].shape[1], s["q"].shape[1], s["rot"]
        pos = s["lens"].long()[:, None] + torch.arange(R, device=DEV)
        angle = torch.complex(s["table"][pos][..., : rot // 2].double(), s["table"][pos][..., rot // 2:].double())[:, :, None]
        turned = []
        for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
            x = x.double()
            if w is not None:
                x = w.double() * x / ((x * x).sum(-1, keepdim=True) / x.shape[-1] + s["eps"]).sqrt()
            pairs = x[..., :rot].unflatten(-1, (-1, 2)) if s["interleaved"] else x[..., :rot].unflatten(-1, (2, -1)).transpose(-1, -2)
            pairs = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * angle)
            x[..., :rot] = pairs.flatten(-2) if s["interleaved"] else pairs.transpose(-1, -2).flatten(-2)
            turned.append(x)
        at = s["tables"].long().gather(1, pos // bs)
        k_cache = s["k_cache"].double()
        k_cache[at, pos % bs] = turned[1]
        v_cache = s["v_cache"].double()
        v_cache[at, pos % bs] = s["v"].double()
        return turned[0], k_cache, v_cache
    if s["op"] == "logprobs":
        n, k = s["top_ids"].shape
        found = [[], [], [], []]
        for r in range(0, n, 64):
            p = torch.log_softmax(s["x"][r:r + 64, :s["V"]].double() / s["T"], -1)
            found[0].append(p.gather(1, s["tokens"][r:r + 64].long()))
            found[1].append(-torch.where(p == -math.inf, 0.0, p.exp() * p).sum(-1))
            found[2].append(torch.logsumexp(s["x"][r:r + 64, :s["V"]].double() / s["T"], -1))
            found[3].append(p.topk(k, -1).values)
        logp, entropy, lse, best = (torch.cat(f) for f in found)
        return logp, entropy, lse, None, best
    if s["op"] == "copy":
        for src, dst, tokens in s["moves"][: int(s["count"])].tolist():
            for cache in s["caches"]:
                cache[dst, :tokens] = cache[src, :tokens]
        return [cache.double() for cache in s["caches"]]
    if s["op"] == "compact":
        blocks = sorted(set(s["kept"][0].view(-1).tolist()))  # the live ones
        holes = sorted(set(range(len(blocks))) - set(blocks))
        movers = [b for b in blocks if b >= len(blocks)]
        for cache in s["caches"]:
            cache[torch.tensor(holes, device=DEV, dtype=torch.int64)] = cache[torch.tensor(movers, device=DEV, dtype=torch.int64)]
        return [None] * 6 + [[cache.double() for cache in s["caches"]]]
    return None  # whole numbers only
