"""The softmax steps of the 8-bit cache's attention, restated operation by operation in float32: for scores of any
size they end, their weights stay in fp16's range, and the result is the softmax of the float32 scores."""
import numpy as np
import pytest

F = np.float32
NEG = F(-np.inf)


def fma(a, b, c):
    """One rounding: the product of two float32 is exact in float64, and the sum's rounding there is 2^-29 of one here."""
    return (np.asarray(a, np.float64) * np.asarray(b, np.float64) + np.asarray(c, np.float64)).astype(F)


def ex2(x):
    with np.errstate(over="ignore"):
        y = np.exp2(np.asarray(x, np.float64)).astype(F)
    return np.where(y < F(2.0 ** -126), F(0), y)  # subnormal results are flushed


def half(x):
    return np.asarray(x, F).astype(np.float16).astype(np.float64)


class Many:
    """One row of k_kv8_prefill.cu: two pages a step, the reference (M, V) from the first step, raised where a page's
    weights sum to more than 2^15; such a page, and every one where |M| is 2^11 or more, is worked out twice."""
    UP, MOST, FAR, TOP = F(6), F(32768), F(2048), 2.0 ** 15

    def __init__(self):
        self.M, self.V, self.L, self.o, self.again = NEG, F(0), F(0), 0.0, 0

    @staticmethod
    def largest(page, tm, tv):
        s = F(page["x"].max() * page["fac"])
        return (s, page["vlog"]) if (s - tm) + (page["vlog"] - tv) > 0 else (tm, tv)

    def step(self, pages):
        first = None
        if self.M == NEG:
            for page in pages:
                self.M, self.V = self.largest(page, self.M, self.V)
        for page in pages:
            at = F(0) if self.M == NEG else self.M
            y = ex2(fma(page["x"], page["fac"], F(page["vlog"] + F(F(self.UP - self.V) - at))))
            if y.sum(dtype=np.float64) > (self.MOST if abs(at) < self.FAR else -1):
                self.again += 1
                tm, tv = self.largest(page, self.M, self.V)
                above = F(F(tm - self.M) + F(tv - self.V))
                if above > 3:
                    d = F(np.ceil(above)) if above < 64 else above
                    self.V = F(self.V + F(d - F(tm - self.M))) if above < 64 else tv
                    self.M, f = tm, ex2(-d)
                    self.L, self.o = F(self.L * f), self.o * float(f)
                    if first is not None:
                        first = (half(first[0] * float(f)), first[1])
                at = F(0) if self.M == NEG else self.M
                y = ex2((((page["x"] * page["fac"]).astype(F) - at).astype(F) + F(page["vlog"] + F(self.UP - self.V))).astype(F))
            assert np.isfinite(y).all() and y.max() <= self.TOP, (y.max(), self.M, self.V)
            self.L = F(self.L + F(y.sum(dtype=np.float64) * float(page["vinv"])))
            if first is not None:
                self.o += first[0] @ first[1]
            first = (half(y), page["codes"])
        self.o += first[0] @ first[1]

    def run(self, pages):
        for i in range(0, len(pages), 2):
            self.step(pages[i:i + 2])
        return self.o / float(self.L)


class Few:
    """One row of one warp of k_kv8_attend.cu: 16 tokens of each page, the reference raised where a weight passes it by
    more than a factor of 2."""
    SHIFT, TOP, NONE = F(14), 2.0 ** 15, F(-3e38)

    def __init__(self):
        self.M, self.w, self.L, self.o, self.again = self.NONE, self.SHIFT, F(0), 0.0, 0

    def run(self, pages):
        for page in pages:
            for at in range(0, 64, 16):  # (a warp has 16 of a page's tokens: here one has them all, one set after another)
                z = (page["x"][at:at + 16] * page["fac"]).astype(F)
                x = ((z - self.M).astype(F) + F(page["vlog"] + self.w)).astype(F)
                if x.max() > self.SHIFT + 1:
                    f = ex2(self.SHIFT - x.max())
                    self.M, self.w, self.L, self.o = z.max(), F(self.SHIFT - page["vlog"]), F(self.L * f), self.o * float(f)
                    x = ((z - self.M).astype(F) + F(page["vlog"] + self.w)).astype(F)
                y = ex2(x)
                assert np.isfinite(y).all() and y.max() <= self.TOP, (y.max(), self.M, self.w)
                self.L = F(self.L + F(y.sum(dtype=np.float64) * float(page["vinv"])))
                self.o += half(y) @ page["codes"][at:at + 16]
        return self.o / float(self.L)


def wanted(pages):
    """The softmax of the float32 scores in 64 bits: the result, the mean size of what it weighs, and what an error of one
    in every weight, relative to the largest weight and scale, would change."""
    s = np.concatenate([(p["x"] * p["fac"]).astype(F) for p in pages]).astype(np.float64)
    v = np.concatenate([p["codes"] * 2.0 ** float(p["vlog"]) for p in pages])
    l = np.concatenate([np.full(64, float(p["vlog"])) for p in pages])
    w = np.exp2(s - s.max())
    ref = ((s - s.max()) + l).max()
    c = np.concatenate([p["codes"] for p in pages])
    return (w @ v) / w.sum(), (w @ np.abs(v)) / w.sum(), np.abs(c).sum() * 2.0 ** ref / w.sum()


def page(rng, x, fac, vlog):
    return dict(x=np.asarray(x, F), fac=F(fac), vlog=F(vlog), vinv=F(2.0 ** -vlog), codes=rng.integers(-448, 449, 64).astype(np.float64))


def pages_of(kind, rng, size, count):
    """Scores of about `size`, in pages whose values' scales differ."""
    fac = F(rng.uniform(1, 2) * 2.0 ** -8)
    base = F(size / fac)
    lo = -60 if kind == "scales" else -7
    vlogs = rng.integers(lo, 60 if kind == "scales" else 0, count)
    out = []
    for i in range(count):
        if kind in ("equal", "scales"):
            x = np.full(64, base)
        elif kind == "mixed":     # both signs
            x = rng.choice([base, -base], 64)
        elif kind == "normal":
            x = rng.normal(size=64) * base
        elif kind == "near":      # a few roundings of float32 apart
            x = base * (1 + rng.integers(-4, 5, 64) * 2.0 ** -22)
        elif kind == "rising":    # from page to page by more than a rounding, and less than fp32's range
            x = np.full(64, base + abs(base) * 2.0 ** -20 * i + 30 * i / fac)
        else:                     # "jump": from small scores to large ones
            x = np.full(64, base if i >= count // 2 else F(rng.normal()) / fac)
        out.append(page(rng, x, fac, vlogs[i]))
    return out


@pytest.mark.parametrize("kind", ["equal", "scales", "mixed", "normal", "near", "rising", "jump"])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("rows", [Many, Few], ids=lambda c: c.__name__.lower())
def test_scores_of_any_size(rows, sign, kind):
    rng = np.random.default_rng(7)
    for e in (0, 4, 8, 10, 11, 12, 16, 20, 22, 23, 24, 25, 26, 27, 28, 30, 32, 36):
        for _ in range(6):
            pages = pages_of(kind, rng, sign * rng.uniform(1, 2) * 2.0 ** e, int(rng.integers(1, 9)))
            row = rows()
            got = row.run(pages)
            assert row.again <= len(pages)
            want, size, floor = wanted(pages)
            # Twice (in the weights and in their sum): half an fp16 step, an exponent's 2^-12 near the reference, and
            # what fp32 sums of 512 tokens lose. A weight below fp16's normal numbers: half of its smallest step, 2^-25,
            # where the largest weight is 2^5 or more (the reference is less than one above it).
            tol = 2 * (2.0 ** -11 + 2.0 ** -12 + 2.0 ** -15) * size + 2.0 ** -25 * floor * 2.0 ** -5
            assert abs(got - want) <= tol, (e, got, want, tol)
