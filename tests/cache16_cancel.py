"""Keys and values whose weighted sum cancels, so that what is left shows the rounding of the weights themselves.

Every 16 tokens are a period: four keys of score 0 (weight 1, the row's largest), six of a score z_a with V = 1 and six
of z_b with V = -v, where v is about 2^(z_a - z_b).  The scores are chosen among what the type can hold so that too few
16-bit terms of the weights (two of BF16, one of FP16) are off by nearly as much as they can be, with opposite signs.  Values of two of the four leading
keys take up what does not cancel, so the output is far smaller than what it is summed from, and its own
rounding with it."""
import math

import torch

SCALE = 0.125
PERIOD, SIX = 16, 6
LOG2E = 1.44269504088896340736


def terms(w, dtype, n):
    """w (64 bits) as the sum of n terms of the type, each the nearest to what the earlier ones leave."""
    held = torch.zeros_like(w)
    for _ in range(n):
        held = held + (w - held).to(dtype).double()
    return held


def weight(k):
    """Weight of keys k against one query of 1, next to the largest weight 1."""
    return torch.exp2(k.double() * (SCALE * LOG2E))


class Cancel:
    def __init__(self, dtype):
        k = torch.unique(-torch.exp2(torch.linspace(-2.0, 3.0, 40001, dtype=torch.float64)).to(dtype)).double()
        w = weight(k)
        off = (terms(w, dtype, 2 if dtype is torch.bfloat16 else 1) - w) / w
        a, b = int(off.argmax()), int(off.argmin())
        self.dtype, self.k_a, self.k_b, self.w_a, self.w_b = dtype, float(k[a]), float(k[b]), float(w[a]), float(w[b])
        self.z = max(abs(self.k_a), abs(self.k_b)) * SCALE * LOG2E
        to = lambda x: float(torch.tensor(x, dtype=torch.float64).to(dtype))  # noqa: E731
        self.v = to(self.w_a / self.w_b)
        rest = SIX * (self.w_a - self.v * self.w_b)
        self.c1 = to(-rest)
        self.c2 = to(-rest - self.c1)
        # [16] keys and values; the leading keys stand apart
        lead, a, b = [0, 5, 10, 15], [1, 3, 6, 8, 11, 13], [2, 4, 7, 9, 12, 14]
        self.keys, self.values = torch.zeros(PERIOD, dtype=torch.float64), torch.zeros(PERIOD, dtype=torch.float64)
        self.keys[a], self.keys[b] = self.k_a, self.k_b
        self.values[a], self.values[b] = 1.0, -self.v
        self.values[lead[1]], self.values[lead[2]] = self.c1, self.c2
        w = weight(self.keys)
        self.sum = float(w.sum())
        self.out = float((w * self.values).sum()) / self.sum
        self.size = float((w * self.values.abs()).sum()) / self.sum
        self.top = float((w * self.values.abs()).max()) / self.sum

    def bound(self):
        """How far out may be where the weights are FP32's, or within 2^-22 of them.

        The score is one product (exact) times a factor of 24 bits, rounded: |z| 2^-23; less the maximum, rounded again:
        |z| 2^-24; both in the exponent.  The exponential is off by 2^-22 of itself.  What the terms leave is 2^-22 at
        most (two of 11 bits; three of 8 leave less).  A product of 16 tokens adds its 16 terms and what came before in
        FP32, each addition off by 2^-23 of the largest term at most (what came before has cancelled); two or three
        products a period.  The sum of the weights, the joins and the rounding to the type are relative to out."""
        half, least = torch.finfo(self.dtype).eps / 2, torch.finfo(self.dtype).tiny * torch.finfo(self.dtype).eps
        weights = (math.log(2.0) * self.z * (2.0 ** -23 + 2.0 ** -24) + 2.0 ** -22 + 2.0 ** -22) * self.size
        products = 3 * 17 * 2.0 ** -23 * self.top
        return weights + products + abs(self.out) * (half + 2.0 ** -16) + least / 2

    def off_with(self, n):
        """The error of out that weights of n terms alone make."""
        w = weight(self.keys)
        return abs(float(((terms(w, self.dtype, n) - w) * self.values).sum())) / self.sum

    def tokens(self, n, D):
        """K and V [n, 1, D] and the factor of each dim's values (a power of two with a sign)."""
        sign = torch.tensor([(-1.0) ** (d // 3) * 2.0 ** (d % 5) for d in range(D)], dtype=torch.float64)
        i = torch.arange(n) % PERIOD
        k = torch.zeros(n, 1, D, dtype=torch.float64)
        k[:, 0, 0] = self.keys[i]
        return k.to(self.dtype), (self.values[i][:, None] * sign)[:, None].to(self.dtype), sign
