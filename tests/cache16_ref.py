"""The live 16-bit cache and the position rotation from their definitions (no code of the package): pages, the
rotation in 64 bits and operation by operation in FP32, attention in 64 bits, and how far results of the stated
arithmetic may be from it."""
import math

import torch

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def tables(positions, R, theta=1e6):
    """FP32 cosines and sines [positions, R / 2] of the angles p theta^(-2 i / R)."""
    a = torch.arange(positions, dtype=torch.float64)[:, None] * theta ** (
        -2.0 * torch.arange(R // 2, dtype=torch.float64) / R)
    return a.cos().float(), a.sin().float()


def turn(x, pos, cos, sin, neighbours):
    """Rows x [n, heads, D] turned by positions pos [n], in the precision of x (each product and sum rounded once);
    positions outside the tables turn to NaN."""
    R = 2 * cos.shape[1]
    pos = torch.as_tensor(pos)
    ok = (pos >= 0) & (pos < cos.shape[0])
    at = torch.where(ok, pos, 0)
    c, s = (torch.where(ok[:, None], t[at], math.nan).to(x.dtype)[:, None] for t in (cos, sin))
    y = x.clone()
    first = torch.arange(R // 2) * (2 if neighbours else 1)
    second = first + (1 if neighbours else R // 2)
    a, b = x[..., first], x[..., second]
    y[..., first] = a * c - b * s
    y[..., second] = b * c + a * s
    return y


class Setup:
    """Pages on the CPU [pages, T, H, D] (K and V), tables, and tensors for the device calls.  What no token holds is
    any 16 bits, NaN and infinities among them."""

    def __init__(self, *, D, H, T, lens, dtype, layout="nhd", seed=0, spare=3, spread=0.5, dev="cuda"):
        self.g = torch.Generator().manual_seed(seed)
        self.D, self.H, self.T, self.lens, self.layout, self.dev = D, H, T, list(lens), layout, dev
        self.dtype_name, self.dtype, self.spread = dtype, DTYPES[dtype], spread
        counts = [-(-n // T) for n in self.lens]
        self.pages = sum(counts) + spare
        order = torch.randperm(self.pages, generator=self.g).tolist()
        self.tables = torch.full((len(self.lens), max([1] + counts)), -1, dtype=torch.int32)
        for s, n in enumerate(counts):
            for i in range(n):
                self.tables[s, i] = order.pop()
        noise = lambda: torch.randint(-32768, 32768, (self.pages, T, H, D), generator=self.g, dtype=torch.int16)  # noqa: E731
        self.pool = [noise().view(self.dtype) for _ in range(2)]

    def values(self, n, heads=None):
        heads = heads or self.H
        x = torch.randn(n, heads, self.D, generator=self.g)
        return (x * torch.exp(self.spread * torch.randn(n, heads, 1, generator=self.g))).to(self.dtype)

    def put(self, s, start, k, v):
        """Tokens start, start + 1, ... of sequence s, as they are; those without a page or a position are left out."""
        for i in range(k.shape[0]):
            p = start + i
            if p < 0 or p // self.T >= self.tables.shape[1]:
                continue
            pid = int(self.tables[s, p // self.T])
            if 0 <= pid < self.pages:
                self.pool[0][pid, p % self.T], self.pool[1][pid, p % self.T] = k[i], v[i]

    def fill(self, lens=None):
        for s, n in enumerate(self.lens if lens is None else lens):
            if n:
                self.put(s, 0, self.values(n), self.values(n))

    def strides(self):
        T, H, D = self.T, self.H, self.D
        return {"nhd": (T * H * D, H * D, D), "hnd": (H * T * D, D, T * D), "packed": (2 * H * T * D, 2 * D, 2 * T * D)}[self.layout]

    def cache(self, cache16, HQ):
        return cache16.Cache16(dtype=self.dtype_name, head_dim=self.D, num_kv_heads=self.H, num_q_heads=HQ,
                               block_tokens=self.T, num_blocks=self.pages, strides=self.strides())

    def device_layer(self, cache16):
        if self.layout == "packed":
            both = torch.cat([x.transpose(1, 2) for x in self.pool], dim=3).contiguous().to(self.dev)
            return cache16.Layer(both[..., :self.D], both[..., self.D:])
        return cache16.Layer(*((x if self.layout == "nhd" else x.transpose(1, 2)).contiguous().to(self.dev) for x in self.pool))

    def bits_of(self, layer):
        """The device's pages [pages, T, H, D] as 16-bit whole numbers (NaN compare as what they are)."""
        return [(x if self.layout == "nhd" else x.transpose(1, 2)).cpu().contiguous().view(torch.int16)
                for x in (layer.k, layer.v)]

    def batch(self, cache8, new=None, lens=None, errors=None, hints=True):
        lens = self.lens if lens is None else lens
        cu, n_new = None, None
        if new is not None:
            cu = torch.tensor([0] + torch.tensor(new).cumsum(0).tolist(), dtype=torch.int32, device=self.dev)
            n_new = sum(new)
        kw = dict(max_new=max(new) if new else 1, max_len=max(lens)) if hints else {}
        return cache8.Batch(self.tables.to(self.dev), torch.tensor(lens, dtype=torch.int32, device=self.dev), cu, n_new=n_new,
                            errors=errors, **kw)

    def tokens(self, role, s, n):
        """Values [n, H, D] in 64 bits of a sequence's first n tokens, and which of them have a page."""
        x, ok = torch.zeros(n, self.H, self.D, dtype=torch.float64), torch.zeros(n, dtype=torch.bool)
        for a in range(0, n, self.T):
            i = a // self.T
            pid = int(self.tables[s, i]) if i < self.tables.shape[1] else -1
            if 0 <= pid < self.pages:
                b = min(n, a + self.T)
                x[a:b], ok[a:b] = self.pool[role][pid, :b - a].double(), True
        return x, ok

    def attend(self, s, n, q, causal=True, window=0, scale=None):
        """q [c, HQ, D], the last c of n tokens: (out, lse, the largest error of out, that of lse)."""
        c, HQ, D = q.shape
        G = HQ // self.H
        q = q.double().view(c, self.H, G, D)
        (k, ok), (v, _) = self.tokens(0, s, n), self.tokens(1, s, n)
        scale = 1.0 / math.sqrt(D) if scale is None else scale
        at, j = torch.arange(n - c, n)[:, None], torch.arange(n)[None, :]
        see = ok[None, :] & (at >= 0)
        if causal:
            see = see & (j <= at)
        if window:
            see = see & (j > at - window)
        out = torch.zeros(c, self.H, G, D, dtype=torch.float64)
        lse = torch.full((c, self.H, G), -math.inf, dtype=torch.float64)
        eo, el = torch.zeros_like(out), torch.zeros_like(lse)
        half = torch.finfo(self.dtype).eps / 2
        # a weight as two terms: the first is off by half a step of it, the second by half a step of that; below FP16's
        # normal range by half of its smallest step, 2^-25, where the largest weight is held as 2^11 at least
        two = half * half * 2
        for i in range(c):
            m = int(see[i].sum())
            if not m:
                continue
            kk, vv = k[see[i]], v[see[i]]
            for h in range(self.H):
                z = scale * (q[i, h] @ kk[:, h].T)                       # [G, m]
                lse[i, h] = torch.logsumexp(z, -1)
                p = torch.exp(z - lse[i, h][:, None])
                out[i, h] = p @ vv[:, h]
                # FP32 sums of D products, each step off by 2^-23 at most of what has come together, and some
                # roundings of the score (which that sum bounds)
                dz = (scale * (q[i, h].abs() @ kk[:, h].abs().T)).amax(-1) * (D + 16) * 2.0 ** -23
                # the exponential and the FP32 steps around it 2^-20; sums over m keys (and 2 m products) by FP32 steps
                rel = two + 2.0 ** -20 + 2 * dz + 3 * m * 2.0 ** -23
                size = p @ vv[:, h].abs()
                low = p.amax(-1, keepdim=True) * vv[:, h].abs().sum(0) * 2.0 ** -36
                eo[i, h] = (size * rel[:, None] + low) * (1 + half) + out[i, h].abs() * half + torch.finfo(self.dtype).tiny
                el[i, h] = dz + lse[i, h].abs() * 2.0 ** -22 + 2.0 ** -19 + m * 2.0 ** -23
        flat = lambda x: x.view(c, HQ, *x.shape[3:])  # noqa: E731
        return flat(out), flat(lse), flat(eo), flat(el)
