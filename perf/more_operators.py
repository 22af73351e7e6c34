"""The operators that bring prompts into the paged cache and hold that cache in 8 bits, as cases to measure: attention of
whole prompts (packed, causal, behind what the pages hold already), the packed tokens' norms, rotation and append to 16- or
8-bit pages, attention of drafted trees over 8-bit pages, and copies of 8-bit pages with their scales.  An 8-bit page holds
e4m3 numbers and, for each head, the code x of a scale 2^(x - 127).  With `own` false a pass runs the operators' plain form
in torch; with `own` true it calls the library.  Sizes follow workloads/configs.py."""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # Four short questions are admitted at once: the latency of a small prefill.
        dict(name="prompts, short", op="prompt", dtype="f16", kv="16", S=4, n=45, least=0.2, ctx=0, Hq=8, Hkv=2, D=64, block=4, layout="token"),
        # A batch's 32 prompts of up to 2048 tokens, packed.
        dict(name="prompts, packed batch", op="prompt", dtype="bf16", kv="16", S=32, n=2048, least=0.25, ctx=0, Hq=32, Hkv=8, D=128, block=16, layout="head"),
        # One long document in one pass.
        dict(name="prompts, long document", op="prompt", dtype="bf16", kv="16", S=1, n=32767, least=1.0, ctx=0, Hq=16, Hkv=4, D=128, block=16, layout="token"),
        # Chunks of four prompts behind up to 30,000 tokens that an 8-bit cache already holds.
        dict(name="prompts, chunks behind 8 bits", op="prompt", dtype="bf16", kv="8", S=4, n=511, least=0.5, ctx=30000, Hq=32, Hkv=8, D=128, block=16, layout="token"),
        # A tiny round's new tokens into 8-bit pages: latency.
        dict(name="append, tiny round", op="append", dtype="f16", kv="8", S=4, n=3, least=1.0, ctx=17, Hq=8, Hkv=2, D=64, rot=64, block=4, interleaved=True,
             norm=True, layout="token"),
        # The batched round's 2560 new tokens into 8-bit pages, behind about 2100 tokens each.
        dict(name="append, batched round", op="append", dtype="bf16", kv="8", S=512, n=5, least=1.0, ctx=2128, Hq=32, Hkv=8, D=128, rot=128, block=16, interleaved=False,
             norm=True, layout="head"),
        # The packed batch of prompts into 16-bit pages.
        dict(name="append, packed prompts", op="append", dtype="bf16", kv="16", S=32, n=2048, least=0.25, ctx=0, Hq=32, Hkv=8, D=128, rot=128, block=16, interleaved=False,
             norm=True, layout="head"),
        # One new token for each of 4 particles over 8-bit pages: the latency of a single decode step.
        dict(name="8-bit attention, one token", op="tree", dtype="f16", B=1, N=4, R=1, Hq=8, Hkv=2, D=64, ctx=16, private=0, block=4, shared=False, tree=False, layout="token"),
        # The batched round over 8-bit pages, prompt blocks shared.
        dict(name="8-bit attention, batched round", op="tree", dtype="bf16", B=32, N=16, R=5, Hq=32, Hkv=8, D=128, ctx=2048, private=80, block=16, shared=True, tree=False,
             layout="head"),
        # The wide-particle round with unshared 8-bit pages, drafts as trees: bound by reading every page.
        dict(name="8-bit attention, wide", op="tree", dtype="bf16", B=4, N=64, R=9, Hq=32, Hkv=8, D=128, ctx=4093, private=0, block=16, shared=False, tree=True, layout="token"),
        # The copy-on-write list of a batched round on four layers' 8-bit pages and their scales.
        dict(name="8-bit pages, copy on write", op="copy", S=512, whole=False, Hkv=8, D=128, block=16, layers=4, blocks=6144, layout="head"),
        # Whole blocks of a compaction, moved with their scales in two layers.
        dict(name="8-bit pages, moved", op="copy", S=8192, whole=True, Hkv=8, D=128, block=16, layers=2, blocks=24576, layout="token"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "append", "append", "tree", "tree", "copy"])
    D = rng.choice([64, 64, 80, 96, 128, 128, 128, 192, 256])
    Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 4, 7, 8])
    common = dict(op=op, dtype=rng.choice(["bf16", "f16"]), Hq=Hkv * G, Hkv=Hkv, D=D, block=rng.choice([1, 8, 16, 16, 24, 64, 128]), layout=rng.choice(["token", "head"]))
    if op == "prompt":
        S, n, ctx = _log(rng, 1, 64), _log(rng, 1, 16384), rng.choice([0, 0, _log(rng, 1, 32768)])
        while n > 1 and (S * Hkv * G * n * (ctx + n) > 1e10 or S * (ctx + n) * Hkv * D > 5e8):
            n, ctx, S = (n + 1) // 2, ctx // 2, (S + 1) // 2
        return dict(common, kv=rng.choice(["16", "8"]), S=S, n=n, least=rng.choice([0.1, 0.5, 1.0]), ctx=ctx)
    if op == "append":
        S, n, ctx = _log(rng, 1, 512), rng.choice([1, 1, 3, 5, _log(rng, 2, 4096)]), _log(rng, 1, 2048)
        while n > 1 and S * n * (G + 2) * Hkv * D > 2e8:
            n = (n + 1) // 2
        while S > 1 and S * (ctx + n) * Hkv * D > 5e8:
            S = (S + 1) // 2
        return dict(common, kv=rng.choice(["16", "8", "8"]), S=S, n=n, least=rng.choice([0.3, 1.0]), ctx=ctx, rot=rng.choice([32, 64, 64]), interleaved=rng.random() < 0.5,
                    norm=rng.random() < 0.7)
    if op == "tree":
        N, R, ctx = _log(rng, 1, 64), rng.choice([1, 1, 3, 5, 9, _log(rng, 2, 64)]), _log(rng, 1, 65536)
        B = _log(rng, 1, 32)
        while B > 1 and B * N * (ctx + R) * Hkv * D > 5e8:
            B = (B + 1) // 2
        while N > 1 and B * N * (ctx + R) * Hkv * D > 5e8:
            N = (N + 1) // 2
        while ctx > 64 and 4 * B * N * R * G * Hkv * (ctx + R) * D > 1e11:
            ctx = (ctx + 1) // 2
        shared = rng.random() < 0.5
        return dict(common, B=B, N=N, R=R, ctx=ctx, private=_log(rng, 1, 300) if shared else 0, shared=shared, tree=rng.random() < 0.5)
    return dict(op=op, S=_log(rng, 1, 1000), whole=rng.random() < 0.5, Hkv=Hkv, D=rng.choice([64, 80, 128]), block=rng.choice([1, 4, 16, 24, 32]), layers=rng.randint(1, 4),
                blocks=_log(rng, 2100, 6000), layout=common["layout"])


def _lengths(case):
    """New tokens and context of each packed sequence: spread evenly between `least` and all of n (of ctx)."""
    part = [case["least"] + (1 - case["least"]) * ((s * 0.6180339887498949) % 1.0) for s in range(case["S"])]
    if case["S"] == 1:
        part = [1.0]
    return [max(1, round(case["n"] * p)) for p in part], [round(case["ctx"] * (0.5 + 0.5 * p)) for p in part[::-1]]


# ------------------------------------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _i32(x):
    return x.to(torch.int32).contiguous()


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV, dtype=dtype)


def _cache(blocks, block, Hkv, D, dtype, layout, g):
    """Pages seen as [blocks, block, Hkv, D], laid out by token or by head; 8-bit ones fill e4m3's range."""
    shape = (blocks, block, Hkv, D) if layout == "token" else (blocks, Hkv, block, D)
    if dtype is E4M3:
        pages = _randn(g, *shape, dtype=torch.bfloat16).mul_(70).clamp_(-448, 448).to(E4M3)
    else:
        pages = _randn(g, *shape, dtype=dtype)
    return pages if layout == "token" else pages.transpose(1, 2)


def _scales(blocks, Hkv, g):
    """Codes of scales between 2^-8 and 2^-5: values of some units."""
    return torch.randint(119, 123, (blocks, Hkv), generator=g, device=DEV, dtype=torch.uint8)


def _packed(case, g):
    """Lengths, their sums, contexts and block tables of packed sequences in a shuffled pool."""
    new, ctx = _lengths(case)
    slots = max(-(-(c + n) // case["block"]) for c, n in zip(ctx, new))
    blocks = case["S"] * slots + 1
    tables = torch.randperm(blocks, generator=g, device=DEV)[: case["S"] * slots].view(case["S"], slots)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return _i32(tables), _i32(torch.tensor(ctx, device=DEV)), _i32(torch.tensor(cu, device=DEV)), cu[-1], blocks, max(c + n for c, n in zip(ctx, new)), max(new)


def _prepare_prompt(c, g):
    dt = DTYPES[c["dtype"]]
    tables, lens, cu, T, blocks, longest, most = _packed(c, g)
    kind = E4M3 if c["kv"] == "8" else dt
    k, v = (_cache(blocks, c["block"], c["Hkv"], c["D"], kind, c["layout"], g) for _ in range(2))
    q = (1.5 * _randn(g, T, c["Hq"], c["D"])).to(dt)
    sc = [_scales(blocks, c["Hkv"], g) if c["kv"] == "8" else None for _ in range(2)]
    return dict(q=q, k=k, v=v, k_scales=sc[0], v_scales=sc[1], tables=tables, lens=lens, cu=cu, scale=c["D"] ** -0.5, longest=longest, most=most, out=torch.empty_like(q),
                lse=torch.empty(T, c["Hq"], device=DEV), status=torch.zeros(1, dtype=torch.int32, device=DEV))


def _prepare_append(c, g):
    Hq, Hkv, D, dt = c["Hq"], c["Hkv"], c["D"], DTYPES[c["dtype"]]
    tables, lens, cu, T, blocks, longest, _ = _packed(c, g)
    kind = E4M3 if c["kv"] == "8" else dt
    size = torch.where(torch.rand(Hq + 2 * Hkv, D, generator=g, device=DEV) < 0.03, 8.0, 1.0)  # a few channels are larger
    qkv = (_randn(g, T, Hq + 2 * Hkv, D) * size).to(dt)
    angle = torch.arange(longest, device=DEV, dtype=torch.float64)[:, None] * 500000.0 ** (-torch.arange(0, c["rot"], 2, device=DEV, dtype=torch.float64) / c["rot"])
    w = [(1 + 0.2 * _randn(g, D)).to(dt) if c["norm"] else None for _ in range(2)]
    sc = [_scales(blocks, Hkv, g) if c["kv"] == "8" else None for _ in range(2)]
    return dict(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:], q_weight=w[0], k_weight=w[1], eps=1e-6, rot=c["rot"], interleaved=c["interleaved"],
                table=torch.cat([angle.cos(), angle.sin()], 1).float(), tables=tables, lens=lens, cu=cu, k_cache=_cache(blocks, c["block"], Hkv, D, kind, c["layout"], g),
                v_cache=_cache(blocks, c["block"], Hkv, D, kind, c["layout"], g), k_scales=sc[0], v_scales=sc[1], q_out=torch.empty(T, Hq, D, dtype=dt, device=DEV),
                status=torch.zeros(1, dtype=torch.int32, device=DEV))


def _prepare_tree(c, g):
    S, R, Hq, Hkv, D, dt, bs = c["B"] * c["N"], c["R"], c["Hq"], c["Hkv"], c["D"], DTYPES[c["dtype"]], c["block"]
    ctx, B, N = c["ctx"], c["B"], c["N"]
    first = ctx // bs if c["shared"] else 0  # leading blocks that a prompt's particles share
    if c["shared"]:
        lens = ctx + torch.randint(0, c["private"] + 1, (S,), generator=g, device=DEV)
    elif S > 1:
        lens = torch.randint((ctx + 1) // 2, ctx + 1, (S,), generator=g, device=DEV)
    else:
        lens = torch.full((1,), ctx, device=DEV)
    slots = -(-(ctx + c["private"] + R) // bs)
    blocks = B * first + S * (slots - first)
    ids = torch.randperm(blocks, generator=g, device=DEV)
    tables = torch.empty(S, slots, dtype=torch.int64, device=DEV)
    tables[:, :first] = ids[: B * first].view(B, 1, first).expand(B, N, first).reshape(S, first)
    tables[:, first:] = ids[B * first:].view(S, slots - first)
    k, v = (_cache(blocks, bs, Hkv, D, E4M3, c["layout"], g) for _ in range(2))
    q = (1.5 * _randn(g, S, R, Hq, D)).to(dt)
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
    return dict(q=q, k=k, v=v, k_scales=_scales(blocks, Hkv, g), v_scales=_scales(blocks, Hkv, g), tables=_i32(tables), lens=_i32(lens), mask=mask, N=N, scale=D ** -0.5,
                longest=ctx + c["private"] + R, out=torch.empty_like(q), lse=torch.empty(S, R, Hq, device=DEV), status=torch.zeros(1, dtype=torch.int32, device=DEV))


def _prepare_copy(c, g):
    # Copy on write: each particle holds at most one partial tail, about half of them diverge.  Moves: whole blocks.
    S, P = c["S"], c["blocks"]
    ids = torch.randperm(P, generator=g, device=DEV)
    at = torch.randint(0, S, (S,), generator=g, device=DEV) if not c["whole"] else torch.arange(S, device=DEV)
    tokens = torch.full((S,), c["block"], device=DEV) if c["whole"] else torch.randint(0, c["block"] + 1, (S,), generator=g, device=DEV)
    count = S if c["whole"] else max(1, S // 2)
    moves = torch.stack([ids[at], ids[S:2 * S], tokens], 1)
    return dict(caches=[_cache(P, c["block"], c["Hkv"], c["D"], E4M3, c["layout"], g) for _ in range(2 * c["layers"])],
                scales=[_scales(P, c["Hkv"], g) for _ in range(2 * c["layers"])], moves=_i32(moves), count=torch.full((1,), count, dtype=torch.int32, device=DEV),
                status=torch.zeros(1, dtype=torch.int32, device=DEV))


def prepare(case, seed):
    makers = {"prompt": _prepare_prompt, "append": _prepare_append, "tree": _prepare_tree, "copy": _prepare_copy}
    return dict(makers[case["op"]](case, _gen(seed)), op=case["op"])


# ------------------------------------------------------------------------------------------------ the plain form
def _gathered(pages, scales, block, offset):
    """The tokens at (block, offset) as fp32 values."""
    if scales is None:
        return pages[block, offset].float()
    return torch.ldexp(pages.view(torch.uint8)[block, offset].view(E4M3).float(), scales[block].int()[..., None] - 127)


def _softmax_product(rows, k, v, seen, scale):
    """rows [S, Hkv, n, D], k, v [S, L, Hkv, D] and seen [S, n, L]: the outputs and their lse."""
    score = torch.matmul(rows, k.permute(0, 2, 3, 1).contiguous()).mul_(scale)
    score.masked_fill_(~seen[:, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v.permute(0, 2, 1, 3).contiguous()) / torch.where(total == 0, 1.0, total)
    return out, (total.log() + top).squeeze(-1)


def _prompt(s):
    q, lens, cu = s["q"], s["lens"].long(), s["cu"].long()
    T, Hq, D = q.shape
    bs, Hkv = s["k"].shape[1:3]
    S, n, L, G = len(lens), s["most"], s["longest"], Hq // Hkv
    i = torch.arange(n, device=DEV)
    real = i < (cu[1:] - cu[:-1])[:, None]
    at = torch.where(real, cu[:-1, None] + i, 0)  # [S, n]: tokens of the padded rows
    rows = q[at].float().view(S, n, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(S, Hkv, n * G, D)
    pos = torch.arange(L, device=DEV)
    block = s["tables"].long()[:, pos // bs]
    k, v = (_gathered(s[x], s[x + "_scales"], block, pos % bs) for x in "kv")
    v = torch.where((pos < (lens + cu[1:] - cu[:-1])[:, None])[:, :, None, None], v, 0.0)
    seen = (pos <= (lens[:, None] + i)[:, :, None]).repeat_interleave(G, 1)
    out, lse = _softmax_product(rows, k, v, seen, s["scale"])
    seq = torch.searchsorted(cu, torch.arange(T, device=DEV), right=True) - 1
    row = torch.arange(T, device=DEV) - cu[seq]
    out = out.view(S, Hkv, n, G, D)[seq, :, row].reshape(T, Hq, D)
    return out.to(q.dtype), lse.view(S, Hkv, n, G)[seq, :, row].reshape(T, Hq)


def _norm_rotate(x, weight, s, cos, sin):
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * weight.float()
    rot = s["rot"]
    a, b = (x[..., :rot:2], x[..., 1:rot:2]) if s["interleaved"] else (x[..., :rot // 2], x[..., rot // 2:rot])
    turned = [a * cos - b * sin, b * cos + a * sin]
    turned = torch.stack(turned, -1).flatten(-2) if s["interleaved"] else torch.cat(turned, -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _quantised(values, cache, scales, block, offset, tail, held):
    """Writes fp32 values [T, Hkv, D] to 8-bit pages at (block, offset), their scales grown as far as they need; `tail` [S]: the
    block with a sequence's last older tokens, `held` of them, which follow the scale."""
    P, Hkv = scales.shape
    top = torch.zeros(P, Hkv, device=DEV).scatter_reduce_(0, block[:, None].expand(-1, Hkv), values.abs().amax(-1), "amax")
    m, e = torch.frexp(top)  # top = m 2^e, and 448 = 0.875 2^9
    need = (e - 9 + (m > 0.875).int() + 127).clamp(1, 247)
    need = torch.where(top == 0, 1, need).to(torch.uint8)
    older = torch.zeros(P, dtype=torch.bool, device=DEV)
    older[tail] = held > 0
    fresh = torch.where(older[:, None], torch.maximum(scales, need), need)
    touched = torch.zeros(P, dtype=torch.bool, device=DEV)
    touched[block] = True
    fresh = torch.where(touched[:, None], fresh, scales)
    shrink = (scales[tail].int() - fresh[tail].int())[:, None, :, None]
    was = cache.view(torch.uint8)[tail]
    moved = torch.ldexp(was.view(E4M3).float(), shrink).to(E4M3).view(torch.uint8)
    keep = torch.arange(cache.shape[1], device=DEV)[None] < held[:, None]
    cache.view(torch.uint8)[tail] = torch.where(keep[:, :, None, None], moved, was)
    cache.view(torch.uint8)[block, offset] = torch.ldexp(values, 127 - fresh[block].int()[..., None]).to(E4M3).view(torch.uint8)
    scales.copy_(fresh)


def _append(s):
    q, bs, cu, lens, tables = s["q"], s["k_cache"].shape[1], s["cu"].long(), s["lens"].long(), s["tables"].long()
    T = q.shape[0]
    seq = torch.searchsorted(cu, torch.arange(T, device=DEV), right=True) - 1
    pos = lens[seq] + torch.arange(T, device=DEV) - cu[seq]
    cos, sin = s["table"][pos][:, None].chunk(2, -1)
    block = tables[seq, pos // bs]
    k = _norm_rotate(s["k"], s["k_weight"], s, cos, sin)
    if s["k_scales"] is None:
        s["k_cache"][block, pos % bs] = k.to(q.dtype)
        s["v_cache"][block, pos % bs] = s["v"]
    else:
        tail = tables.gather(1, (lens // bs)[:, None])[:, 0]
        _quantised(k, s["k_cache"], s["k_scales"], block, pos % bs, tail, lens % bs)
        _quantised(s["v"].float(), s["v_cache"], s["v_scales"], block, pos % bs, tail, lens % bs)
    return _norm_rotate(q, s["q_weight"], s, cos, sin).to(q.dtype), s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"]


def _tree(s):
    q, tables, lens = s["q"], s["tables"].long(), s["lens"].long()
    S, R, Hq, D = q.shape
    bs, Hkv = s["k"].shape[1:3]
    L, G = s["longest"], Hq // Hkv
    pos = torch.arange(L, device=DEV)
    block = tables[:, pos // bs]
    node = pos[None] - lens[:, None]  # which new token a position holds; negative: context
    if s["mask"] is None:
        seen = node[:, None] <= torch.arange(R, device=DEV)[None, :, None]
    else:
        bit = (s["mask"][:, :, None] >> node.clamp(0, R - 1)[:, None]) & 1
        seen = (node < 0)[:, None] | ((node < R)[:, None] & (bit != 0))
    k, v = (_gathered(s[x], s[x + "_scales"], block, pos % bs) for x in "kv")
    rows = q.float().view(S, R, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(S, Hkv, -1, D)
    out, lse = _softmax_product(rows, k, v, seen.repeat_interleave(G, 1), s["scale"])
    out = out.view(S, Hkv, R, G, D).permute(0, 2, 1, 3, 4).reshape(S, R, Hq, D)
    return out.to(q.dtype), lse.view(S, Hkv, R, G).permute(0, 2, 1, 3).reshape(S, R, Hq)


def _copy(s):
    src, dst, tokens = s["moves"].long().unbind(1)
    use = torch.arange(len(src), device=DEV) < s["count"]
    src = torch.where(use, src, dst)
    fresh = torch.arange(s["caches"][0].shape[1], device=DEV)[None] < tokens[:, None]
    pages = [c.view(torch.uint8) for c in s["caches"]]
    moved = [torch.where(fresh[:, :, None, None], c[src], c[dst]) for c in pages]
    [c.__setitem__(dst, m) for c, m in zip(pages, moved)]
    moved = [torch.where((tokens > 0)[:, None], c[src], c[dst]) for c in s["scales"]]
    [c.__setitem__(dst, m) for c, m in zip(s["scales"], moved)]
    return s["caches"], s["scales"]


# ------------------------------------------------------------------------------------------------ the library's calls
def _own(s):
    import smc_verification_resampling_amd as sm

    if s["op"] == "prompt":
        T, Hq, D = s["q"].shape
        if "ws" not in s:
            s["ws"] = sm.alloc_workspace(sm.OP_PROMPT_ATTN, len(s["lens"]), T, K=D, V=Hq * D, P=s["k"].shape[2])
        sm.prompt_attention(s["q"], s["k"], s["v"], s["tables"], s["lens"], s["cu"], s["scale"], s["out"], s["status"], s["ws"], k_scales=s["k_scales"], v_scales=s["v_scales"],
                            lse=s["lse"], max_len=s["longest"])
        return s["out"], s["lse"]
    if s["op"] == "append":
        sm.kv_append(s["q"], s["k"], s["v"], s["cu"], s["lens"], s["tables"], s["k_cache"], s["v_cache"], s["q_out"], s["status"], k_scales=s["k_scales"], v_scales=s["v_scales"],
                     q_weight=s["q_weight"], k_weight=s["k_weight"], eps=s["eps"], cos_sin=s["table"], interleaved=s["interleaved"])
        return s["q_out"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"]
    if s["op"] == "tree":
        S, R, Hq, D = s["q"].shape
        if "ws" not in s:
            s["ws"] = sm.alloc_workspace(sm.OP_TREE_ATTN, S // s["N"], s["N"], K=R, V=Hq * D, P=s["k"].shape[2])
        sm.tree_attention(s["q"], s["k"], s["v"], s["tables"], s["lens"], S // s["N"], s["N"], s["scale"], s["out"], s["status"], s["ws"], tree_mask=s["mask"], lse=s["lse"],
                          max_len=s["longest"], k_scales=s["k_scales"], v_scales=s["v_scales"])
        return s["out"], s["lse"]
    sm.kv_copy(s["caches"], s["moves"], s["count"], s["status"], scales=s["scales"])
    return s["caches"], s["scales"]


def run(state):
    if own:
        return _own(state)
    return {"prompt": _prompt, "append": _append, "tree": _tree, "copy": _copy}[state["op"]](state)


# ------------------------------------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "copy":
        count = c["S"] if c["whole"] else max(1, c["S"] // 2)
        tokens = c["block"] if c["whole"] else c["block"] / 2
        return {"bytes": 2 * count * 2 * c["layers"] * c["Hkv"] * (tokens * c["D"] + 1), "flops": 0}
    if c["op"] == "tree":
        S = c["B"] * c["N"]
        mean = c["ctx"] + c["private"] / 2 if c["shared"] else c["ctx"] * (0.75 if S > 1 else 1.0)
        common = c["ctx"] // c["block"] * c["block"] if c["shared"] else 0
        keys = c["B"] * common + S * (mean - common + c["R"])
        return {"bytes": 2 * keys * c["Hkv"] * (c["D"] + 1 / c["block"]) + S * c["R"] * c["Hq"] * (4 * c["D"] + 4),
                "flops": 4.0 * S * c["R"] * c["Hq"] * c["D"] * (mean + (c["R"] + 1) / 2)}
    new, ctx = _lengths(c)
    e = 1 if c["kv"] == "8" else 2
    if c["op"] == "prompt":
        return {"bytes": 2 * e * (sum(new) + sum(ctx)) * c["Hkv"] * c["D"] + sum(new) * c["Hq"] * (4 * c["D"] + 4),
                "flops": 4.0 * c["Hq"] * c["D"] * sum(n * x + n * (n + 1) / 2 for n, x in zip(new, ctx))}
    rows = sum(new)
    return {"bytes": rows * c["D"] * (4 * c["Hq"] + 2 * (2 + e) * c["Hkv"]) + 4 * c["rot"] * rows, "flops": 8.0 * rows * (c["Hq"] + c["Hkv"]) * c["D"]}


# ------------------------------------------------------------------------------------------------ the definition in 64 bits
def _values(pages, scales, blocks):
    """Whole blocks' values in 64 bits, [tokens, Hkv, D]."""
    x = pages[blocks].double() if scales is None else pages.view(torch.uint8)[blocks].view(E4M3).double() * 2.0 ** (scales[blocks].double() - 127)[:, None, :, None]
    return x.reshape(-1, *pages.shape[2:])


def _attend(q, k, v, sees, scale, G):
    """q [n, Hq, D], k, v [L, Hkv, D] and sees [n, L] in 64 bits, a head and 4096 rows at a time."""
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float64, device=DEV)
    for h in range(q.shape[1]):
        for r in range(0, len(q), 4096):
            z = torch.where(sees[r:r + 4096], q[r:r + 4096, h] @ k[:, h // G].t() * scale, -math.inf)
            lse[r:r + 4096, h] = torch.logsumexp(z, 1)
            out[r:r + 4096, h] = torch.softmax(z, 1) @ v[:, h // G]
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "copy":
        for src, dst, tokens in s["moves"][: int(s["count"])].tolist() if case["S"] <= 1000 else []:
            for cache, scale in zip(s["caches"], s["scales"]):
                cache.view(torch.uint8)[dst, :tokens] = cache.view(torch.uint8)[src, :tokens]
        if case["S"] > 1000:  # whole blocks, no destination a source
            src, dst, _ = s["moves"][: int(s["count"])].long().unbind(1)
            for cache in s["caches"]:
                cache.view(torch.uint8).index_copy_(0, dst, cache.view(torch.uint8).index_select(0, src))
        return [cache.double() for cache in s["caches"]], [None for _ in s["scales"]]
    bs = case["block"]
    G = case["Hq"] // case["Hkv"]
    if s["op"] == "prompt":
        if 4.0 * sum(n * (n + x) for n, x in zip(*_lengths(case))) * case["Hq"] * case["D"] > 3e13:
            return None
        q, found = s["q"].double(), []
        cu = s["cu"].tolist()
        for b, ctx in enumerate(s["lens"].tolist()):
            n = cu[b + 1] - cu[b]
            used = s["tables"][b, : -(-(ctx + n) // bs)].long()
            k, v = (_values(s[x], s[x + "_scales"], used)[: ctx + n] for x in "kv")
            sees = torch.ones(n, ctx + n, dtype=torch.bool, device=DEV).tril_(ctx)
            found.append(_attend(q[cu[b]:cu[b + 1]], k, v, sees, s["scale"], G))
        return torch.cat([f[0] for f in found]), torch.cat([f[1] for f in found])
    if s["op"] == "tree":
        S, R, Hq, D = s["q"].shape
        found = []
        for b, ctx in enumerate(s["lens"].tolist()):
            used = s["tables"][b, : -(-(ctx + R) // bs)].long()
            k, v = (_values(s[x], s[x + "_scales"], used)[: ctx + R].transpose(0, 1).contiguous() for x in "kv")
            sees = torch.ones(R, ctx + R, dtype=torch.bool, device=DEV)
            sees[:, ctx:] = torch.ones(R, R, dtype=torch.bool, device=DEV).tril() if s["mask"] is None else torch.stack([(s["mask"][b] >> j) % 2 == 1 for j in range(R)], 1)
            z = s["q"][b].double().transpose(0, 1).reshape(-1, G * R, D) @ k.transpose(1, 2).contiguous() * s["scale"]
            z = torch.where(sees.repeat(G, 1), z, -math.inf)
            found.append(((torch.softmax(z, -1) @ v).view(Hq, R, D).transpose(0, 1), torch.logsumexp(z, -1).view(Hq, R).t()))
        return torch.stack([f[0] for f in found]), torch.stack([f[1] for f in found])
    # append: positions walked sequence by sequence; 8-bit pages as quotients by their scales, not rounded
    cu, lens, rot = s["cu"].tolist(), s["lens"].tolist(), s["rot"]
    where = [(b, lens[b] + i) for b in range(len(lens)) for i in range(cu[b + 1] - cu[b])]
    seq, pos = (torch.tensor(x, device=DEV) for x in zip(*where))
    angle = torch.complex(s["table"][pos, : rot // 2].double(), s["table"][pos, rot // 2:].double())[:, None]
    turned = []
    for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        x = x.double()
        if w is not None:
            x = w.double() * x / ((x * x).sum(-1, keepdim=True) / x.shape[-1] + s["eps"]).sqrt()
        pairs = x[..., :rot].unflatten(-1, (-1, 2)) if s["interleaved"] else x[..., :rot].unflatten(-1, (2, -1)).transpose(-1, -2)
        pairs = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * angle)
        x = torch.cat([pairs.flatten(-2) if s["interleaved"] else pairs.transpose(-1, -2).flatten(-2), x[..., rot:]], -1)
        turned.append(x)
    at = s["tables"].long()[seq, pos // bs]
    pages = []
    for new, cache, codes in ((turned[1], s["k_cache"], s["k_scales"]), (s["v"].double(), s["v_cache"], s["v_scales"])):
        held = cache.double()
        if codes is not None:
            top = torch.zeros(codes.shape, dtype=torch.float64, device=DEV).index_reduce_(0, at, new.abs().amax(-1), "amax", include_self=True)
            code = torch.ceil(torch.log2(top / 448)).clamp(-126, 120) + 127
            last = s["tables"].long()[torch.arange(len(lens), device=DEV), s["lens"].long() // bs]
            part = last[s["lens"] % bs > 0]
            code[part] = torch.maximum(code[part], codes[part].double())
            for b, n in enumerate(lens):
                if n % bs:
                    held[last[b], : n % bs] *= 2.0 ** (codes[last[b]].double() - code[last[b]])[:, None]
            new = new * 2.0 ** (127 - code[at])[..., None]
        held[at, pos % bs] = new
        pages.append(held)
    return turned[0], pages[0], pages[1], None, None
