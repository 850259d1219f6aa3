"""A plain 64-bit restatement of the 8-bit paged cache, request by request, and the error bounds
that the tests of its kernels use. Shares no code with the library."""
import math

import torch

D, PAGE = 128, 64
F8_STEPS = 3          # mantissa bits of e4m3
EPS_BF16 = 2.0 ** -8  # half a step, relative
EPS_F16 = 2.0 ** -11


def decode_e4m3(codes):
    """uint8 codes -> float64 values (NaN for 0x7f and 0xff)."""
    c = codes.to(torch.int64)
    sign = 1.0 - 2.0 * (c >> 7).double()
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (1.0 + m / 8.0) * torch.exp2(e.double() - 7.0))
    v = torch.where((e == 15) & (m == 7), torch.full_like(v, math.nan), v)
    return sign * v


def to_e4m3(x):
    """float64 |x| <= 448 -> the nearest e4m3 value, ties to even, as float64."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -60))).clamp(min=-6.0)
    unit = torch.exp2(e - F8_STEPS)
    return torch.round(x / unit) * unit


def scale_for(amax: float) -> float:
    """The smallest power of two s >= 2^-64 with amax <= 448 s."""
    n = -64
    while amax > 448.0 * 2.0 ** n:
        n += 1
    return 2.0 ** n


def quantise(rows):
    """bf16 rows as float64 [64][128] -> (values of the codes, scale)."""
    if not torch.isfinite(rows).all():
        return torch.zeros_like(rows), math.nan
    s = scale_for(float(rows.abs().max()))
    return to_e4m3(rows / s), s


def rotate(x, pos, inv_freq, interleaved):
    """x float64 [T][H][128], pos [T] -> rotated, float64."""
    r = len(inv_freq)
    if r == 0:
        return x.clone()
    a = pos.double()[:, None] * torch.tensor(inv_freq, dtype=torch.float64)
    c, s = a.cos()[:, None], a.sin()[:, None]
    y = x.clone()
    for j in range(r):
        i0, i1 = (2 * j, 2 * j + 1) if interleaved else (j, j + r)
        y[..., i0] = x[..., i0] * c[..., j] - x[..., i1] * s[..., j]
        y[..., i1] = x[..., i0] * s[..., j] + x[..., i1] * c[..., j]
    return y


def rotate_slack(x, inv_freq, interleaved):
    """What fp32 arithmetic on the rotation may be off by: a few units of 2^-24 of the pair's size."""
    r = len(inv_freq)
    w = torch.zeros_like(x)
    for j in range(r):
        i0, i1 = (2 * j, 2 * j + 1) if interleaved else (j, j + r)
        w[..., i0] = w[..., i1] = 2.0 ** -22 * (x[..., i0].abs() + x[..., i1].abs())
    return w


def keys_and_values(pages, scales, tails, table, b, h, n, which=None):
    """Dequantised float64 keys, values and positions of request b, head h at length n; `which`: the
    pages to take (all complete ones where None), the tail always."""
    full = n // PAGE
    which = list(range(full)) if which is None else [p for p in which if 0 <= p < full]
    ks, vs, pos = [], [], []
    for p in which:
        i = int(table[b, h, p])
        if not 0 <= i < pages.shape[0]:
            continue
        x = decode_e4m3(pages[i]) * scales[i].double()[:, None, None]
        ks.append(x[0])
        vs.append(x[1])
        pos.append(torch.arange(p * PAGE, (p + 1) * PAGE))
    t = tails[b, h, :, : n % PAGE].double()
    ks.append(t[0])
    vs.append(t[1])
    pos.append(torch.arange(full * PAGE, n))
    return torch.cat(ks), torch.cat(vs), torch.cat(pos)


def attend(q, pages, scales, tails, table, past, cu, scale, sel=None):
    """All on the CPU. q bf16 [T][Hq][128] -> (out float64, bound float64): the exact result for
    this cache, and how far a kernel with fp16 operands and fp32 sums may be from it.

    The bound, per output element: one rounding to bf16; probabilities off by half an fp16 step
    (EPS_F16), by the score's error twice (in the weight and in the sum) and by the fp32 sums' over n
    tokens; a score's error is that of 128 fp32 additions of its terms' sizes and of the operands'
    own roundings (2^-24 of the largest query or tail element each: another 2 * 2^-24 of 128 terms)."""
    T, Hq = q.shape[0], q.shape[1]
    B, H = table.shape[0], table.shape[1]
    G = Hq // H
    out = torch.zeros((T, Hq, D), dtype=torch.float64)
    bound = torch.zeros_like(out)
    for b in range(B):
        r0, r1 = int(cu[b]), int(cu[b + 1])
        if r1 == r0:
            continue
        n0 = int(past[b])
        n = n0 + r1 - r0
        for h in range(H):
            which = None if sel is None else [int(p) for p in sel[b * H + h] if p >= 0]
            k, v, pos = keys_and_values(pages, scales, tails, table, b, h, n, which)
            if pos.numel() == 0:
                continue
            qq = q[r0:r1, h * G:(h + 1) * G].double()
            s = torch.einsum("igd,jd->igj", qq, k) * scale
            hid = pos[None, None] > (n0 + torch.arange(r1 - r0))[:, None, None]
            s = s.masked_fill(hid, -math.inf)
            top = s.amax(-1, keepdim=True)
            p = torch.exp(s - torch.where(torch.isinf(top), 0.0, top))
            p = torch.where(hid, 0.0, p)
            tot = p.sum(-1, keepdim=True)
            p = p / torch.where(tot == 0, 1.0, tot)
            bad = torch.isnan(p).any(-1, keepdim=True) | ((p > 0).double() @ (~torch.isfinite(v)).any(-1).double() > 0)[..., None]
            vz = torch.nan_to_num(v, nan=0.0, posinf=0.0, neginf=0.0)
            kz = torch.nan_to_num(k, nan=0.0, posinf=0.0, neginf=0.0)
            pz = torch.nan_to_num(p)
            o = torch.einsum("igj,jd->igd", pz, vz)
            out[r0:r1, h * G:(h + 1) * G] = torch.where(bad, math.nan, o)
            size = torch.einsum("igd,jd->igj", qq.abs(), kz.abs()) * abs(scale)
            big = (qq.abs().amax(-1, keepdim=True) * kz.abs().sum(-1) + qq.abs().sum(-1, keepdim=True) * kz.abs().amax()) * abs(scale)
            ds = (128 * size + 2 * big) * 2.0 ** -24
            rel = EPS_F16 + 2 * ds + (pos.numel() + 64) * 2.0 ** -24
            off = torch.einsum("igj,jd->igd", pz * rel, vz.abs()) + (pz * rel).sum(-1, keepdim=True) * o.abs()
            off = off + 2.0 ** -23 * vz.abs().amax()
            bound[r0:r1, h * G:(h + 1) * G] = off + EPS_BF16 * (o.abs() + off)
    return out, bound


class Cache:
    """The reference's own cache: every token's rotated bf16 key and value, and their pages."""

    def __init__(self, batch, kv_heads, inv_freq, interleaved):
        self.B, self.H, self.f, self.i = batch, kv_heads, inv_freq, interleaved
        self.k = [torch.zeros((0, kv_heads, D), dtype=torch.float64) for _ in range(batch)]
        self.v = [torch.zeros((0, kv_heads, D), dtype=torch.float64) for _ in range(batch)]
        self.x = [torch.zeros((0, kv_heads, D), dtype=torch.float64) for _ in range(batch)]  # keys, not rounded

    def append(self, k, v, cu, positions=None):
        for b in range(self.B):
            r0, r1 = int(cu[b]), int(cu[b + 1])
            n = self.k[b].shape[0]
            pos = torch.arange(n, n + r1 - r0) if positions is None else positions[r0:r1]
            x = rotate(k[r0:r1].double(), pos, self.f, self.i)
            self.x[b] = torch.cat([self.x[b], x])
            self.k[b] = torch.cat([self.k[b], x.to(torch.bfloat16).double()])
            self.v[b] = torch.cat([self.v[b], v[r0:r1].double()])
