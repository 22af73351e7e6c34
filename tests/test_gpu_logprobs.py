"""smcsd_token_logprobs against the definition in 64 bits: whole numbers exactly, values to

  ln S: at most 32 additions of positive terms on a path (32 2^-24), exp2 to one unit in the
  last place (2 2^-24), an exponent t whose product and constant are each rounded (2 2^-24 |t|
  ln 2 on a term of weight e, so 2 2^-24 ln 2 times the mean |t|, which is at most the 24 bits of
  the largest vocabulary): below 70 2^-24, and the result's own rounding 2^-24 |lse|;
  entropy: the same relative error on both of its positive parts, ln S <= H and U/S <= H."""
import math

import pytest
import torch

import smc_verification_resampling_amd as sm

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
E = 70 * 2.0 ** -24


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def call(x, V, T=1.0, tokens=None, k=0, stream=None, ws=None):
    n = x.shape[0]
    o = dict(logp=None if tokens is None else torch.full(tokens.shape, 9.0, device="cuda"), entropy=torch.full((n,), 9.0, device="cuda"),
             lse=torch.full((n,), 9.0, device="cuda"), ids=torch.full((n, k), 9, dtype=torch.int32, device="cuda"),
             top=torch.full((n, k), 9.0, device="cuda"), status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    if ws is None:
        ws = sm.alloc_workspace(sm.OP_LOGPROBS, n, 1, K=k, V=V)
        ws.fill_(0xFF)
    sm.token_logprobs(x, n, V, T, o["status"], ws, tokens=tokens, out_logp=o["logp"], out_entropy=o["entropy"], out_lse=o["lse"],
                      top_ids=o["ids"], top_logp=o["top"], row_stride=x.shape[1], stream=stream)
    return o


def check(o, x, V, T=1.0, tokens=None, rows=None):
    T = float(torch.tensor(T, dtype=torch.float32))
    k = o["ids"].shape[1]
    for r in range(x.shape[0]) if rows is None else rows:
        z = x[r, :V].double().cpu() / T
        order = torch.sort(torch.where(z == 0, 0.0, z), descending=True, stable=True)  # equal values: the smaller id
        want = torch.where(order.values[:k] == -math.inf, -1, order.indices[:k])
        assert o["ids"][r].tolist() == want.tolist(), r
        m = float(z.max())
        if m == -math.inf:
            assert float(o["lse"][r]) == -math.inf and float(o["entropy"][r]) == 0
            assert tokens is None or (o["logp"][r] == -math.inf).all()
            continue
        e = torch.where(z == -math.inf, 0.0, (z - m).exp())
        ln = math.log(float(e.sum()))  # log p = (z - m) - ln: z - (m + ln) would lose ln beside a large m
        lse = m + ln
        tol = E + 2.0 ** -24 * abs(lse)
        assert abs(float(o["lse"][r]) - lse) <= tol, (r, float(o["lse"][r]), lse)
        H = ln - float((e * torch.where(e > 0, z - m, 0.0)).sum() / e.sum())
        assert abs(float(o["entropy"][r]) - H) <= E * (1 + 2 * H) and float(o["entropy"][r]) >= 0, (r, float(o["entropy"][r]), H)
        got, ref = o["top"][r].cpu().double(), (order.values[:k] - m) - ln
        if tokens is not None:
            t = tokens[r].long().cpu()
            ok = (t >= 0) & (t < V)
            assert torch.isnan(o["logp"][r].cpu()[~ok]).all()
            got, ref = torch.cat([got, o["logp"][r].cpu()[ok].double()]), torch.cat([ref, (z[t[ok]] - m) - ln])
        inf = ref == -math.inf
        assert (got[inf] == -math.inf).all() and ((got - ref).abs() <= E + 2.0 ** -23 * ref.abs())[~inf].all(), r


def logits(n, V, dt="bf16", pad=0, seed=0, sigma=2.0):
    g = torch.Generator().manual_seed(seed)
    x = (sigma * torch.randn((n, V + pad), generator=g)).to(DT[dt]).cuda()
    x[:, V:] = math.nan  # what follows a row is not part of it
    return x


def some(n, V, C, seed=1):
    return torch.randint(0, V, (n, C), generator=torch.Generator().manual_seed(seed), dtype=torch.int32).cuda()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 63, 511, 512, 513, 2047, 2048, 2049, 16384, 32000, 50257, 128256])
@pytest.mark.parametrize("pad", [0, 3])
def test_sizes(dt, V, pad):
    x, t = logits(3, V, dt, pad), some(3, V, 2)
    check(call(x, V, 0.7, t, min(V, 20)), x, V, 0.7, t)


@pytest.mark.parametrize("k", [0, 1, 2, 31, 32, 63, 64])
@pytest.mark.parametrize("n", [1, 2, 300])
def test_alternatives(k, n):
    V = 4000
    x = logits(n, V, "bf16", 1, seed=k)
    check(call(x, V, k=k), x, V, rows=range(0, n, 29))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n,V,k", [(1, 11789, 32), (3, 1502, 64), (2, 6807, 33), (9, 409, 32), (2, 16900, 64), (1, 40001, 64)])
@pytest.mark.parametrize("steps", [0, 40])
def test_more_alternatives_than_segments(dt, n, V, k, steps):
    """Rows of fewer segments than alternatives, or hardly more; with `steps`, of few distinct values."""
    x = logits(n, V, dt, 1)
    if steps:
        x[:, :V] = (x[:, :V].float() * (steps / 8)).round().clamp(-steps / 2, steps / 2).to(x.dtype)
    check(call(x, V, 0.8, k=k), x, V, 0.8)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("V,k", [(1500, 20), (32000, 64), (128256, 20), (50001, 5)])
def test_masked_with_the_lowest_value(dt, V, k):
    """0, 1, 3, k - 1, k and 700 allowed tokens of a row, the others at the type's lowest value:
    the alternatives past the allowed ones are the smallest ids."""
    x = logits(6, V, dt, 1)
    g = torch.Generator().manual_seed(3)
    for r, n in enumerate([0, 1, 3, k - 1, k, 700]):
        keep = torch.randperm(V, generator=g)[:n].cuda()
        kept = x[r, keep].clone()
        x[r, :V] = torch.finfo(DT[dt]).min
        x[r, keep] = kept
    check(call(x, V, 1.0, k=k), x, V)


@pytest.mark.parametrize("down", [False, True])
def test_a_sorted_row_of_millions(down):
    V = (1 << 21) + 5
    x = torch.linspace(-8, 8, V)
    x = torch.stack([x.flip(0) if down else x, (x * 16).round() / 16]).cuda()
    check(call(x, V, 1.0, k=64), x, V)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_many_rows(dt):
    n, V = 700, 33000
    x, t = logits(n, V, dt, 5, sigma=1.0), some(n, V, 3)
    check(call(x, V, 1.0, t, 8), x, V, 1.0, t, rows=list(range(0, n, 83)) + [n - 1])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("V", [5, 600, 40000, 128256])
def test_equal_logits_name_the_smallest_ids(dt, V):
    k = min(V, 20)
    x = torch.full((3, V), -1.25, dtype=DT[dt], device="cuda")
    x[1, V // 2:] = 0.0
    x[1, : V // 2] = -0.0  # the two zeros are equal
    x[2, V // 3:] = 3.0
    o = call(x, V, k=k)
    check(o, x, V)
    assert o["ids"][0].tolist() == list(range(k)) and o["ids"][1].tolist() == list(range(k))


def test_a_thousand_equals_below_a_few_larger():
    V = 60000
    x = torch.full((2, V), -4.0, device="cuda")
    x[:, 1000:30000] = 1.0
    x[0, [59999, 7, 30000]] = torch.tensor([2.0, 5.0, 2.0], device="cuda")
    check(call(x, V, k=33), x, V)
    check(call(x.bfloat16(), V, k=33), x.bfloat16(), V)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T", [0.25, 1.0, 3.0])
def test_masks(dt, T):
    V = 9000
    low = torch.finfo(DT[dt]).min
    x, t = logits(8, V, dt, 3), some(8, V, 4)
    x[0, :V] = torch.where(torch.arange(V, device="cuda") % 3 == 0, x[0, :V], -math.inf)
    x[1, : V - 1] = -math.inf       # one entry left, in the tail
    x[2, 1:V] = -math.inf           # the first
    x[3, :V] = torch.where(torch.arange(V, device="cuda") % 5 == 0, x[3, :V], low)
    x[4, 10:V] = -math.inf          # fewer than k
    x[5, :V] = -math.inf
    x[5, [100, 8000]] = 0.5
    o = call(x, V, T, t, 16)
    rows = [0, 1, 2, 4, 5, 6, 7]
    check(o, x, V, T, t, rows=rows)
    assert int(o["status"]) == 0
    # lowest values take no share (their own log-probability may be past fp32: -inf then)
    keep = torch.arange(0, V, 5, device="cuda")
    z = x[3, keep].double() / float(torch.tensor(T))
    lse = float(torch.logsumexp(z, 0))
    assert abs(float(o["lse"][3]) - lse) <= E + 2.0 ** -24 * abs(lse)
    best = torch.sort(z, descending=True, stable=True)
    assert o["ids"][3].tolist() == (5 * best.indices[:16]).tolist()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T", [0.5, 1.0])
def test_rows_of_lowest_values(dt, T):
    V = 3000
    x = torch.full((2, V), torch.finfo(DT[dt]).min, dtype=DT[dt], device="cuda")
    x[1, 7] = -1.0
    o = call(x, V, T, k=3)
    assert o["ids"].tolist() == [[0, 1, 2], [7, 0, 1]] and int(o["status"]) == 0
    assert abs(float(o["entropy"][0]) - math.log(V)) <= E * (1 + 2 * math.log(V)) and float(o["entropy"][1]) == 0
    assert torch.allclose(o["top"][0], torch.full((3,), -math.log(V), device="cuda"), atol=1e-5)


def test_huge_values():
    x = torch.tensor([[3e38, 3e38, -3e38, 0.0], [2.9e38, 1.0, 3.0, -math.inf]], device="cuda")
    o = call(x, 4, 0.5, k=2)
    assert o["ids"].tolist() == [[0, 1], [0, 1]] or o["ids"].tolist() == [[0, 1], [0, 2]]
    assert o["ids"][1].tolist() == [0, 2]
    assert torch.allclose(o["top"][0], torch.full((2,), -math.log(2), device="cuda"), atol=1e-6)
    assert torch.allclose(o["entropy"], torch.tensor([math.log(2), 0.0], device="cuda"), atol=1e-6) and int(o["status"]) == 0


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("size", [1e3, 1e5, 3e6, 1e12, 1e30])
@pytest.mark.parametrize("T", [0.5, 3.0])
def test_far_from_zero(dt, size, T):
    # logits around +-size, apart by what the type resolves there
    V = 5000
    step = torch.finfo(DT[dt]).eps * size
    x = torch.stack([s * size + step * (torch.arange(V, device="cuda") * 7919 % 13) for s in (1.0, -1.0)]).to(DT[dt])
    x[1, 77] = -0.5 * size
    t = some(2, V, 3)
    o = call(x, V, T, t, 16)
    assert int(o["status"]) == 0
    check(o, x, V, T, t)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("at", [0, 1, 500, 2999])
def test_nan_and_infinite_rows(dt, bad, at):
    V = 3000
    x, t = logits(3, V, dt, 1), some(3, V, 2)
    x[1, at] = bad
    o = call(x, V, 1.0, t, 4)
    assert int(o["status"]) == sm.ST_NAN_INPUT
    check(o, x, V, 1.0, t, rows=[0, 2])
    assert o["ids"][1].tolist() == [-1] * 4
    assert all(torch.isnan(o[w][1]).all() for w in ("logp", "entropy", "lse", "top"))


def test_empty_rows_and_bad_tokens():
    V = 700
    x, t = logits(3, V), some(3, V, 3)
    x[1, :] = -math.inf
    o = call(x, V, 1.0, t, 4)
    assert int(o["status"]) == sm.ST_EMPTY_ROW
    check(o, x, V, 1.0, t)
    assert (o["top"][1] == -math.inf).all()
    x = logits(3, V)
    t[0, 0], t[2, 1], t[2, 2] = -1, V, 2 ** 31 - 1
    o = call(x, V, 1.0, t, 4)
    assert int(o["status"]) == sm.ST_BAD_INPUT
    check(o, x, V, 1.0, t)


def test_a_large_vocabulary():
    V = 1 << 20
    for dt in ("bf16", "f32"):
        x = logits(2, V, dt, 1)
        check(call(x, V, k=64), x, V)
    V = 1 << 24
    x = torch.randn((1, V), device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    check(call(x, V, k=10), x, V)


def test_each_output_alone():
    V = 5000
    x, t = logits(4, V), some(4, V, 2)
    full = call(x, V, 1.0, t, 5)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = sm.alloc_workspace(sm.OP_LOGPROBS, 4, 1, K=5, V=V)
    for name, kw in (("logp", dict(tokens=t, out_logp=torch.zeros(4, 2, device="cuda"))), ("entropy", dict(out_entropy=torch.zeros(4, device="cuda"))),
                     ("lse", dict(out_lse=torch.zeros(4, device="cuda"))), ("ids", dict(top_ids=torch.zeros(4, 5, dtype=torch.int32, device="cuda"))),
                     ("top", dict(top_logp=torch.zeros(4, 5, device="cuda")))):
        sm.token_logprobs(x, 4, V, 1.0, st, ws, **kw)
        assert torch.equal(list(kw.values())[-1], full[name]), name


def test_runs_repeat_on_another_stream_and_in_graphs():
    V = 20000
    x, t = logits(6, V), some(6, V, 2)
    x[3] = 1.0  # more equal candidates than fit
    a = call(x, V, 1.0, t, 20)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    b = call(x, V, 1.0, t, 20, stream=st)
    st.synchronize()
    assert all(torch.equal(a[w], b[w]) for w in a)
    ws = sm.alloc_workspace(sm.OP_LOGPROBS, 6, 1, K=20, V=V)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o = call(x, V, 1.0, t, 20, ws=ws)
    for k in range(3):
        x.copy_(logits(6, V, seed=10 + k))
        g.replay()
        torch.cuda.synchronize()
        check(o, x, V, 1.0, t)
        torch.randn(1000, device="cuda").sum()


def test_rows_past_32_bits():
    stride = (1 << 31) + 1  # elements: row 2 begins past 2^32, off 16-byte alignment
    buf = torch.empty(2 * stride + 4096, dtype=torch.bfloat16, device="cuda")
    V = 3000
    x = buf.as_strided((3, V), (stride, 1))
    x.copy_(logits(3, V))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = sm.alloc_workspace(sm.OP_LOGPROBS, 3, 1, K=5, V=V)
    o = dict(entropy=torch.zeros(3, device="cuda"), lse=torch.zeros(3, device="cuda"), ids=torch.zeros(3, 5, dtype=torch.int32, device="cuda"),
             top=torch.zeros(3, 5, device="cuda"))
    sm.token_logprobs(buf, 3, V, 1.0, st, ws, out_entropy=o["entropy"], out_lse=o["lse"], top_ids=o["ids"], top_logp=o["top"], row_stride=stride)
    check(o, x, V)


def test_agrees_with_the_verify():
    # the same rows, tokens and temperature through smcsd_verify
    B, N, K, V, T = 2, 3, 2, 32003, 0.8
    S = B * N
    tgt, drf = logits(S * (K + 1), V).view(S, K + 1, V), logits(S * K, V, seed=5).view(S, K, V)
    x = some(S, V, K)
    i32, f32 = dict(dtype=torch.int32, device="cuda"), dict(dtype=torch.float32, device="cuda")
    logp, lse, st = torch.zeros((S, K + 1), **f32), torch.zeros((S, 2 * K + 1), **f32), torch.zeros(1, **i32)
    tok = torch.zeros((S, K + 1), **i32)
    sm.verify(tgt, drf, x, B, N, K, V, T, 1.0, sm.MODE_SMC, 1, 2, tok, st, sm.alloc_workspace(sm.OP_VERIFY_SMC, B, N, K, V),
              log_weights=torch.zeros(S, **f32), out_logp=logp, out_lse=lse)
    o = call(tgt.view(S * (K + 1), V), V, T, tok.view(-1, 1), 5)
    assert torch.allclose(o["logp"].view(S, K + 1), logp, atol=2 * E, rtol=1e-6)
    assert torch.allclose(o["lse"].view(S, K + 1), lse[:, : K + 1], atol=2 * E, rtol=1e-6)


def test_refusals():
    x = logits(2, 100)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = sm.alloc_workspace(sm.OP_LOGPROBS, 2, 1, K=5, V=100)
    t = some(2, 100, 1)
    for kw in (dict(tokens=t.long(), out_logp=torch.zeros(2, 1, device="cuda")), dict(tokens=t.view(-1), out_logp=torch.zeros(2, device="cuda")),
               dict(tokens=t, out_logp=torch.zeros(1, device="cuda")), dict(out_lse=torch.zeros(1, device="cuda")),
               dict(top_ids=torch.zeros(2, 5, dtype=torch.int32, device="cuda"), top_logp=torch.zeros(2, 4, device="cuda")),
               dict(top_ids=torch.zeros(2, 65, dtype=torch.int32, device="cuda")), dict(row_stride=99)):
        with pytest.raises(sm.SmcsdError):
            sm.token_logprobs(x, 2, 100, 1.0, st, ws, **kw)
    with pytest.raises(sm.SmcsdError):
        sm.token_logprobs(x.half(), 2, 100, 1.0, st, ws)
    with pytest.raises(sm.SmcsdError):
        sm.token_logprobs(x, 3, 100, 1.0, st, ws)
