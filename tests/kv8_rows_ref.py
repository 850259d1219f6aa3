"""Attention where every token lists its pages, over the 8-bit cache, restated in 64 bits, with the error bound that the
tests of its kernel use. Shares no code with the library."""
import math

import torch

from kv8_ref import D, EPS_BF16, PAGE, decode_e4m3

EPS_WEIGHT = 2.0 ** -11  # half a step of a weight, relative
FLOOR = 2.0 ** -20       # and of one that is far below its row's largest, relative to that one


def attend_rows(q, pages, scales, tails, table, past, cu, scale, sel):
    """All on the CPU. q bf16 [T][Hq][128], sel [T][H][k] -> (out float64, bound float64).

    The bound, per output element: one rounding to bf16; a weight (a probability times the power of two, or scale, that its
    token's values have) off by EPS_WEIGHT of itself and FLOOR of the row's largest weight; by its score's error twice (in the weight
    and in the sum) and by fp32 sums over n tokens; a score's error is that of 128 fp32 additions of its terms' sizes, of one
    rounding of the score itself, and of the operands' own (2^-22 of the largest query or key element each)."""
    T, Hq = q.shape[0], q.shape[1]
    B, H = table.shape[0], table.shape[1]
    G = Hq // H
    out = torch.zeros((T, Hq, D), dtype=torch.float64)
    bound = torch.zeros_like(out)
    for b in range(B):
        r0, r1 = int(cu[b]), int(cu[b + 1])
        n0, n = int(past[b]), int(past[b]) + r1 - r0
        for t in range(r0, r1):
            see = n0 + t - r0 + 1
            for h in range(H):
                which = sorted({int(p) for p in sel[t, h] if 0 <= int(p) < see // PAGE})
                last = see // PAGE
                ks, vs, us, lost = [], [], [], False
                for p in which + ([last] if last < n // PAGE else []):
                    i = int(table[b, h, p])
                    m = min(PAGE, see - p * PAGE)
                    if m <= 0 or not 0 <= i < pages.shape[0]:
                        continue
                    s = scales[i].double()
                    lost |= not bool(torch.isfinite(s).all())
                    ks.append(decode_e4m3(pages[i, 0, :m]) * s[0])
                    vs.append(decode_e4m3(pages[i, 1, :m]) * s[1])
                    us.append(s[1].expand(m))
                m = see - n // PAGE * PAGE
                if m > 0:
                    x = tails[b, h, :, :m].double()
                    lost |= not bool(torch.isfinite(x).all())
                    x = torch.nan_to_num(x, nan=0.0, posinf=0.0, neginf=0.0)
                    ks.append(x[0])
                    vs.append(x[1])
                    us.append(x[1].abs().amax(-1).clamp(min=1e-30) / 256)
                if not ks:
                    continue
                k, v, u = torch.cat(ks), torch.cat(vs), torch.cat(us)
                qq = q[t, h * G:(h + 1) * G].double()
                lost = lost | ~torch.isfinite(qq).all(-1, keepdim=True)
                qq, k, v, u = (torch.nan_to_num(x, nan=0.0, posinf=0.0, neginf=0.0) for x in (qq, k, v, u))
                w = qq @ k.T * scale
                p = torch.softmax(w, -1)
                o = p @ v
                out[t, h * G:(h + 1) * G] = torch.where(lost, math.nan, o) if torch.is_tensor(lost) else o
                size = qq.abs() @ k.abs().T * abs(scale)
                big = (qq.abs().amax(-1, keepdim=True) * k.abs().sum(-1) + qq.abs().sum(-1, keepdim=True) * k.abs().amax()) * abs(scale)
                ds = 130 * size * 2.0 ** -24 + big * 2.0 ** -22
                rel = EPS_WEIGHT + 2 * ds + (k.shape[0] + 64) * 2.0 ** -24
                floor = FLOOR * (p * u).amax(-1, keepdim=True) / u.clamp(min=1e-300)
                dp = p * rel + floor
                off = dp @ v.abs() + (p * rel).sum(-1, keepdim=True) * o.abs()
                bound[t, h * G:(h + 1) * G] = off + EPS_BF16 * (o.abs() + off)
    return out, bound
