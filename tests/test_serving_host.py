"""The serving operators' host checks (CPU only: every call here is refused, or answered, before
anything is enqueued): the C entry points' limits, the workspace sizes and the binding's
refusals of host tensors."""
import ctypes
import os

import pytest
import torch

import smc_verification_resampling_amd as sm

P0 = ctypes.c_void_p(0x1000)  # never dereferenced
ODD = ctypes.c_void_p(0x1008)  # not 16-byte aligned


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(sm.LIB_PATH):
        from smc_verification_resampling_amd import build
        build.build()
    return sm.load_library()


def caller(fn, order, base):
    def call(**kw):
        a = dict(base)
        a.update(kw)
        return fn(*[a[n] for n in order.split()])
    return call


def test_workspace_sizes(lib):
    w = sm.workspace_bytes
    assert w(sm.OP_TREE_ATTN, 32, 16, 5, 32 * 128, 8) > 0
    assert w(sm.OP_TREE_ATTN, 1, 1, 0, 64, 1) == 0 and w(sm.OP_TREE_ATTN, 1, 1, 65, 64, 1) == 0
    assert w(sm.OP_TREE_ATTN, 1, 1, 1, 64, 0) == 0 and w(sm.OP_TREE_ATTN, 1, 1, 1, 64, 3) == 0
    assert w(sm.OP_LOGPROBS, 512, 1, 20, 128256) >= 512 * 4 * 250  # a maximum for each 512 bf16 entries
    assert w(sm.OP_LOGPROBS, 4, 1, 65, 1000) == 0 and w(sm.OP_LOGPROBS, 4, 1, 5, 4) == 0
    assert w(sm.OP_LOGPROBS, 4, 1, 0, (1 << 24) + 1) == 0
    for op in (sm.OP_KV_FREE, sm.OP_KV_COMPACT):
        assert w(op, 0, 0, P=1) > 0 and w(op, 0, 0, P=0) == 0
        assert w(op, 0, 0, P=1 << 26) > 0 and w(op, 0, 0, P=(1 << 26) + 1) == 0
    assert w(sm.OP_KV_COMPACT, 0, 0, P=100000) >= 3 * 4 * 100000


@pytest.mark.parametrize("B,N,R,Hkv,G,most", [(4, 64, 9, 8, 4, 0.5e9), (1, 256, 9, 8, 4, 0.5e9), (1, 1024, 5, 8, 4, 0.5e9),
                                            (1, 64, 64, 8, 4, 0.5e9), (1, 1024, 64, 1, 8, 1e9), (1, 1, 64, 1, 32, 1.1e9)])
def test_attention_workspace_follows_the_rows_that_exist(lib, B, N, R, Hkv, G, most):
    """Heads of 128.  Splits fall as row tiles grow: the parts stay near those of 1024 tiles of 128 rows
    (67 MB, G times that where the heads of a group are not known), or one a row."""
    assert 0 < sm.workspace_bytes(sm.OP_TREE_ATTN, B, N, R, Hkv * G * 128, Hkv) < most


def test_kv_fork(lib):
    f = caller(lib.smcsd_kv_fork, "m B N T M rc P st s",
               dict(m=P0, B=2, N=4, T=P0, M=8, rc=P0, P=64, st=P0, s=None))
    assert f(N=0) == -1 and f(N=1025) == -1 and f(M=0) == -1 and f(P=0) == -1 and f(P=1 << 31) == -1
    assert f(B=-1) == -1 and f(B=1 << 20, N=1024, M=64) == -1
    for n in ("m", "T", "rc", "st"):
        assert f(**{n: None}) == -1
    assert f(B=0) == 0
    assert f(N=1, M=1) == 0  # one particle: nothing to share, nothing enqueued


def test_kv_fork_sizes_whose_product_passes_64_bits(lib):
    f = caller(lib.smcsd_kv_fork, "m B N T M rc P st s",
               dict(m=P0, B=2, N=1024, T=P0, M=8, rc=P0, P=64, st=P0, s=None))
    assert f(B=1 << 30, M=1 << 24) == -1 and f(B=1 << 29, M=1 << 25) == -1 and f(B=(1 << 31) - 1, N=1, M=1) == -1
    assert f(B=(1 << 31) - 2, N=1, M=1) == 0  # one particle each: nothing is enqueued


def test_kv_free(lib):
    f = caller(lib.smcsd_kv_free, "m S T M rc fl top P st ws wsb s",
               dict(m=P0, S=4, T=P0, M=8, rc=P0, fl=P0, top=P0, P=64, st=P0, ws=P0, wsb=1 << 20, s=None))
    assert f(S=-1) == -1 and f(M=0) == -1 and f(P=0) == -1 and f(P=(1 << 26) + 1) == -1
    assert f(S=1 << 28, M=8) == -1 and f(S=1 << 62) == -1
    for n in ("m", "T", "rc", "fl", "top", "st"):
        assert f(**{n: None}) == -1
    assert f(ws=None) == -4 and f(ws=ctypes.c_void_p(0x1010)) == -4 and f(wsb=4) == -4
    assert f(S=0) == 0


def test_kv_compact(lib):
    f = caller(lib.smcsd_kv_compact, "T S M bs rc fl top P mv n st ws wsb s",
               dict(T=P0, S=4, M=8, bs=16, rc=P0, fl=P0, top=P0, P=64, mv=P0, n=P0, st=P0, ws=P0, wsb=1 << 20,
                    s=None))
    assert f(S=-1) == -1 and f(M=0) == -1 and f(bs=0) == -1 and f(P=0) == -1 and f(P=(1 << 26) + 1) == -1
    assert f(S=1 << 28, M=8) == -1
    for n in ("T", "rc", "fl", "top", "mv", "n", "st"):
        assert f(**{n: None}) == -1
    assert f(ws=None) == -4 and f(ws=ctypes.c_void_p(0x1010)) == -4 and f(wsb=16) == -4


def test_kv_copy(lib):
    two = (ctypes.c_void_p * 2)(0x1000, 0x2000)
    f = caller(lib.smcsd_kv_copy, "c n page seg segs tok bs list count cap P st s",
               dict(c=two, n=2, page=4096, seg=8, segs=512, tok=32, bs=16, list=P0, count=P0, cap=4, P=64, st=P0,
                    s=None))
    assert f(n=-1) == -1 and f(n=257) == -1 and f(seg=0) == -1 and f(tok=0) == -1 and f(bs=0) == -1
    assert f(tok=1 << 31) == -1 and f(tok=1 << 28, bs=16) == -1 and f(page=-1) == -1 and f(segs=-1) == -1
    assert f(P=0) == -1 and f(cap=-1) == -1 and f(cap=1 << 31) == -1
    for n in ("c", "list", "count", "st"):
        assert f(**{n: None}) == -1
    assert f(c=(ctypes.c_void_p * 2)(0x1000, None)) == -1
    assert f(n=0) == 0 and f(cap=0) == 0


ROPE = dict(q=P0, k=P0, v=P0, dt=1, qs=512, ks=128, vs=128, S=2, R=3, Hq=8, Hkv=2, D=64, qw=P0, kw=P0, eps=1e-6,
            cs=P0, maxpos=100, rot=64, il=0, pos=None, ctx=P0, nn=None, T=P0, M=8, bs=16, P=64, kc=P0, vc=P0,
            page=2048, tok=128, head=64, qo=P0, st=P0, s=None)


def test_qk_norm_rope(lib):
    f = caller(lib.smcsd_qk_norm_rope, " ".join(ROPE), ROPE)
    assert f(dt=0) == -2 and f(dt=3) == -2
    for kw in (dict(S=-1), dict(R=0), dict(Hq=0), dict(Hkv=0), dict(D=0), dict(D=12), dict(D=264), dict(rot=72),
               dict(rot=24), dict(rot=-16), dict(maxpos=-1), dict(eps=-1.0), dict(eps=float("nan")),
               dict(eps=float("inf")), dict(qs=504), dict(qs=516), dict(ks=64), dict(vs=64), dict(M=0), dict(bs=0),
               dict(P=0), dict(P=1 << 31), dict(page=32), dict(tok=32), dict(head=32), dict(page=2052),
               dict(tok=132), dict(head=68), dict(M=1 << 20, bs=1 << 12), dict(S=1 << 30), dict(S=1 << 28, M=8),
               dict(qw=ODD), dict(kw=ODD), dict(cs=ODD), dict(cs=None)):
        assert f(**kw) == -1, kw
    for n in ("q", "k", "v", "qo", "kc", "vc"):
        assert f(**{n: None}) == -1 and f(**{n: ODD}) == -1, n
    for n in ("ctx", "T", "st"):
        assert f(**{n: None}) == -1, n
    assert f(S=0) == 0


ATTN = dict(q=P0, dt=1, qs=512, kc=P0, vc=P0, page=2048, tok=128, head=64, T=P0, M=8, bs=16, P=64, ctx=P0, nn=None,
            mask=None, B=2, N=2, R=3, Hq=8, Hkv=2, D=64, scale=0.125, ml=0, out=P0, lse=None, st=P0, ws=P0,
            wsb=1 << 30, s=None)


def test_tree_attention(lib):
    f = caller(lib.smcsd_tree_attention, " ".join(ATTN), ATTN)
    assert f(dt=0) == -2 and f(dt=3) == -2
    for kw in (dict(B=-1), dict(N=-1), dict(R=0), dict(R=65), dict(Hq=0), dict(Hkv=0), dict(Hq=7), dict(D=0),
               dict(D=12), dict(D=264), dict(scale=float("nan")), dict(scale=float("inf")), dict(ml=-1), dict(qs=504),
               dict(qs=516), dict(M=0), dict(bs=0), dict(P=0), dict(P=1 << 31), dict(page=32), dict(tok=32),
               dict(head=32), dict(page=2052), dict(M=1 << 20, bs=1 << 12), dict(B=1 << 28), dict(B=1 << 14, N=1 << 14),
               dict(mask=ctypes.c_void_p(0x1004))):
        assert f(**kw) == -1, kw
    for n in ("q", "out", "kc", "vc"):
        assert f(**{n: None}) == -1 and f(**{n: ODD}) == -1, n
    for n in ("ctx", "T", "st"):
        assert f(**{n: None}) == -1, n
    assert f(ws=None) == -4 and f(ws=ctypes.c_void_p(0x1010)) == -4
    assert f(wsb=sm.workspace_bytes(sm.OP_TREE_ATTN, 2, 2, 3, 512, 2) - 1) == -4
    assert f(B=0) == 0 and f(N=0) == 0


def test_tree_attention_rows(lib):
    """128 threads a query row at least, and a launch has fewer than 2^32: 2^25 rows are refused, one
    less is not (what it is refused for here is the missing workspace)."""
    f = caller(lib.smcsd_tree_attention, " ".join(ATTN), dict(ATTN, M=1, ws=None))
    one = dict(R=1, Hq=1, Hkv=1, N=1, D=8, qs=8)
    assert f(**dict(one, B=1 << 25)) == -1 and f(**dict(one, B=(1 << 25) - 1)) == -4
    assert f(**dict(one, B=1 << 15, N=1 << 10)) == -1 and f(**dict(one, B=(1 << 15) - 1, N=1 << 10)) == -4
    many = dict(R=64, Hq=16, Hkv=16, N=1, D=8, qs=128)
    assert f(**dict(many, B=1 << 15)) == -1 and f(**dict(many, B=(1 << 15) - 1)) == -4


def test_tree_attention_scales_past_a_float(lib):
    f = caller(lib.smcsd_tree_attention, " ".join(ATTN), dict(ATTN, ws=None))
    for scale in (3e38, -3e38, float("-inf")):  # scale * log2(e) is infinite
        assert f(scale=scale) == -1, scale
    for scale in (2.0 ** 127, -2.0 ** 127, 0.0, 1e-45):
        assert f(scale=scale) == -4, scale


def test_token_logprobs(lib):
    f = caller(lib.smcsd_token_logprobs, "x dt rs n V T tok C k lp en lse ti tl st ws wsb s",
               dict(x=P0, dt=1, rs=64, n=4, V=64, T=1.0, tok=P0, C=1, k=5, lp=P0, en=P0, lse=P0, ti=P0, tl=P0, st=P0,
                    ws=P0, wsb=1 << 20, s=None))
    assert f(dt=2) == -2
    for kw in (dict(n=-1), dict(V=0), dict(V=(1 << 24) + 1, rs=1 << 25), dict(rs=63), dict(C=-1), dict(C=1025),
               dict(k=-1), dict(k=65), dict(V=4, k=5), dict(T=0.0), dict(T=float("nan")), dict(T=float("inf")),
               dict(x=None), dict(x=ctypes.c_void_p(0x1001)), dict(st=None), dict(tok=None)):
        assert f(**kw) == -1, kw
    assert f(ws=None) == -4 and f(ws=ctypes.c_void_p(0x1010)) == -4 and f(wsb=16) == -4
    assert f(n=0) == 0


def test_token_logprobs_temperatures_whose_inverse_is_no_number(lib):
    f = caller(lib.smcsd_token_logprobs, "x dt rs n V T tok C k lp en lse ti tl st ws wsb s",
               dict(x=P0, dt=1, rs=64, n=4, V=64, T=1.0, tok=P0, C=1, k=5, lp=P0, en=P0, lse=P0, ti=P0, tl=P0, st=P0,
                    ws=None, wsb=0, s=None))
    for T in (2.0 ** -149, 1e-40, 4e-39):  # log2(e) / T is past the largest float
        assert f(T=T) == -1 and f(T=T, n=0) == -1, T
    for T in (2.0 ** -127, 2.0 ** -126, 3e38):  # no refusal but the missing workspace's
        assert f(T=T) == -4, T


def test_binding_refuses_host_tensors(lib):
    i = torch.zeros(8, dtype=torch.int32)
    t = torch.zeros(2, 4, dtype=torch.int32)
    c = torch.zeros(2, 4, 1, 8, dtype=torch.bfloat16)
    u8 = torch.zeros(1 << 16, dtype=torch.uint8)
    with pytest.raises(sm.SmcsdError):
        sm.kv_fork(i, 1, 2, t, i, i)
    with pytest.raises(sm.SmcsdError):
        sm.kv_free(i, t, i, i, i, i, u8)
    with pytest.raises(sm.SmcsdError):
        sm.kv_compact(t, 4, i, i, i, t, i, i, u8)
    with pytest.raises(sm.SmcsdError):
        sm.kv_copy([c], torch.zeros(2, 3, dtype=torch.int32), i, i)
    with pytest.raises(sm.SmcsdError):
        sm.qk_norm_rope(c, c, c, i, t, c, c, c, i)
    with pytest.raises(sm.SmcsdError):
        sm.tree_attention(c, c, c, t, i, 1, 2, 1.0, c, i, u8)
    with pytest.raises(sm.SmcsdError):
        sm.token_logprobs(c.view(2, -1), 2, 32, 1.0, i, u8)
