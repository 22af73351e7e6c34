"""What the tests of attention over 8-bit pages and of prompts share: pages of either kind, what
they stand for, and an attention's rows against the definition in 64 bits.

The bound on an output element, with u = finfo(dtype).eps / 2 (half a step) and p the exact
probabilities: the output's own rounding u|out| (+ half the smallest subnormal), the
probabilities' rounding u sum p|v| (each is off by at most u p; those below the type's normal
range by half its smallest subnormal, on at most `len` tokens), and the scores' fp32 error d:
a dot product of D terms and a scale, |dz| <= d = (D + 4) 2^-24 sum|q k| scale, moves each p
by a factor exp(+-2d), and the sum of p and of p v over at most len terms adds (len + 64) 2^-24,
so (4 d + 2 (len + 64) 2^-24) sum p|v|.  lse: 2 d + (len + 64) 2^-24 + 2^-23 |lse|.
8-bit pages add nothing: what they hold is widened exactly, or as widen() says."""
import math

import torch

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
SUB = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25}
E4M3 = torch.float8_e4m3fn


def pages(blocks, bs, Hkv, D, dt, e4m3, layout, g):
    """(cache seen as [blocks, bs, Hkv, D], scales or None) of random values, on the CPU."""
    shape = (blocks, bs, Hkv, D) if layout == "token" else (blocks, Hkv, bs, D)
    x = torch.randn(shape, generator=g)
    c = (x * 60).clamp(-448, 448).to(E4M3) if e4m3 else x.to(DT[dt])
    s = torch.randint(119, 123, (blocks, Hkv), generator=g, dtype=torch.uint8) if e4m3 else None
    return (c if layout == "token" else c.transpose(1, 2)), s


def on_gpu(c):
    """A copy on the GPU with the same strides between rows."""
    if c.is_contiguous():
        return c.cuda()
    return c.transpose(1, 2).contiguous().cuda().transpose(1, 2)


def widen(bits, codes, dtype):
    """e4m3 elements (uint8, [..., Hkv, D]) and codes [..., Hkv] as values of `dtype`, in 64 bits."""
    x = bits.view(E4M3).double() * torch.where(codes == 255, math.nan, 2.0 ** (codes.double() - 127))[..., None]
    y = x.to(dtype).double()
    top = torch.finfo(dtype).max
    return torch.where(y.isinf(), top * y.sign(), y)


def tokens_at(cache, scales, block, offset, dtype):
    """[n, Hkv, D] in 64 bits."""
    if scales is None:
        return cache[block, offset].double()
    return widen(cache.view(torch.uint8)[block, offset], scales[block], dtype)


def check_rows(q, k, v, sees, scale, out, lse, dt, what=""):
    """q, out [n, Hq, D], lse [n, Hq]; k, v [L, Hkv, D] in 64 bits; sees [n, L]."""
    n, Hq, D = q.shape
    L, Hkv = k.shape[:2]
    G = Hq // Hkv
    u, sub = torch.finfo(DT[dt]).eps / 2, SUB[dt]
    for h in range(Hkv):
        hs = slice(h * G, h * G + G)
        x = q[:, hs].double().reshape(n * G, D)
        ok = sees.repeat_interleave(G, 0)
        kh, vh = torch.nan_to_num(k[:, h]), torch.nan_to_num(v[:, h])  # (only for what is not seen)
        z = (x @ kh.t() * scale).masked_fill(~ok, -math.inf)
        d = (D + 4) * 2.0 ** -24 * ((x.abs() @ kh.abs().t()) * abs(scale)).masked_fill(~ok, 0).amax(1, keepdim=True)
        top = z.amax(1, keepdim=True)
        p = torch.where(ok, (z - top.masked_fill(top == -math.inf, 0)).exp(), 0.0)
        tot = p.sum(1, keepdim=True)
        want_lse = (top + tot.log()).view(n, G)
        p = p / tot.clamp_min(1e-300)
        want = p @ vh
        mag = p @ vh.abs()
        lost = min(sub, 1.0) * (ok.double() @ vh.abs()) / tot.clamp_min(1e-300)
        tol = u * want.abs() + sub + (u + 4 * d + 2 * (L + 64) * 2.0 ** -24) * mag + lost
        err = (out[:, hs].double().reshape(n * G, D) - want).abs()
        assert (err <= tol).all(), (what, h, float((err - tol).max()), float((err / tol.clamp_min(1e-300)).max()))
        gl = lse[:, hs].double()
        empty = tot.view(n, G) == 0
        assert ((gl == -math.inf) == empty).all(), (what, h)
        ltol = 2 * d.view(n, G) + (L + 64) * 2.0 ** -24 + 2.0 ** -23 * want_lse.abs()
        assert ((gl - want_lse).abs() <= ltol)[~empty].all(), (what, h)
