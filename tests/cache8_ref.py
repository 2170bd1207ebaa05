"""The live 8-bit cache in 64 bits, from its definition (no code of the package):
pages, scales, writing, reading and attention, and how far 16-bit results of the
stated arithmetic may be from it."""
import math
import random

import torch

E_MIN, E_MAX = -60, 119


def e4m3_table():
    out = []
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
        out.append(math.nan if b & 127 == 127 else (-x if b & 128 else x))
    return torch.tensor(out, dtype=torch.float64)


TABLE = e4m3_table()


def encode(x):
    """Bytes of the nearest E4M3 values of float64 x, ties to even, saturating; NaN has the code 0x7F."""
    a = x.abs()
    step = torch.exp2((torch.frexp(torch.where(torch.isfinite(a), a, 0.0))[1] - 1).clamp(min=-6).double() - 3)
    y = torch.where(torch.isinf(a), 448.0, (torch.round(a / step) * step).clamp(max=448.0))
    code = torch.searchsorted(TABLE[:127], torch.nan_to_num(y).contiguous()).to(torch.uint8)
    code = torch.where(torch.isnan(x), torch.full_like(code, 127), code)
    return code | (torch.signbit(x) & ~torch.isnan(x)).to(torch.uint8) * 128


def page_exponent(amax):
    """The smallest e with amax <= 448 * 2^e, within [E_MIN, E_MAX] (a Python float)."""
    e = E_MIN
    while e < E_MAX and amax > math.ldexp(448.0, e):
        e += 1
    return e


class Cache:
    """One layer on the CPU: codes [pages, T, H, D] (uint8), scales [pages, H] (float64)."""

    def __init__(self, pages, T, H, D):
        self.T, self.H, self.D = T, H, D
        self.codes = [torch.zeros(pages, T, H, D, dtype=torch.uint8) for _ in range(2)]
        self.scale = [torch.zeros(pages, H, dtype=torch.float64) for _ in range(2)]

    def write(self, table, start, new):
        """new: (k, v), each [n, H, D]; the tokens start, start + 1, ... of the sequence of `table`."""
        for role in range(2):
            x, n, t = new[role].double(), new[role].shape[0], 0
            if start < 0:
                t = -start
            while t < n:
                page, lead = divmod(start + t, self.T)
                here = x[t:min(n, t + self.T - lead)]
                pid = int(table[page]) if page < len(table) else -1
                if 0 <= pid < self.codes[role].shape[0]:
                    for h in range(self.H):
                        y = here[:, h]
                        f = y[torch.isfinite(y)].abs()
                        s = 2.0 ** page_exponent(float(f.max()) if f.numel() else 0.0)
                        was = float(self.scale[role][pid, h])
                        if lead:
                            if s > was:
                                old = self.codes[role][pid, :lead, h]
                                self.codes[role][pid, :lead, h] = encode(TABLE[old.long()] * was / s)
                            s = max(s, was)
                        self.codes[role][pid, lead:lead + here.shape[0], h] = encode(y / s)
                        self.scale[role][pid, h] = s
                t += here.shape[0]

    def tokens(self, role, table, n):
        """Values [n, H, D] of a sequence's first n tokens, and which of them have a page."""
        x = torch.zeros(n, self.H, self.D, dtype=torch.float64)
        ok = torch.zeros(n, dtype=torch.bool)
        for a in range(0, n, self.T):
            i = a // self.T
            pid = int(table[i]) if i < len(table) else -1
            if 0 <= pid < self.codes[role].shape[0]:
                b = min(n, a + self.T)
                x[a:b] = (TABLE[self.codes[role][pid].long()] * self.scale[role][pid][None, :, None])[:b - a]
                ok[a:b] = True
        return x, ok

    def attend(self, table, n, q, causal, window, scale=None):
        """q [c, HQ, D]: (out, lse, size, dz) of the last c of n tokens; size = (sum of p |v|, the largest p times
        the sum of |v| as codes times the largest scale): what the relative and the absolute rounding of the
        weights act on; dz = the error bound of a row's scores."""
        c, HQ, D = q.shape
        G = HQ // self.H
        q = q.double().view(c, self.H, G, D)
        (k, ok), (v, _) = self.tokens(0, table, n), self.tokens(1, table, n)
        scale = 1.0 / math.sqrt(D) if scale is None else scale
        at = torch.arange(n - c, n)[:, None]
        j = torch.arange(n)[None, :]
        see = ok[None, :] & (at >= 0)
        if causal:
            see = see & (j <= at)
        if window:
            see = see & (j > at - window)
        out = torch.zeros(c, self.H, G, D, dtype=torch.float64)
        lse = torch.full((c, self.H, G), -math.inf, dtype=torch.float64)
        size, dz = torch.zeros(2, c, self.H, G, D, dtype=torch.float64), torch.zeros_like(lse)
        for i in range(c):
            if not bool(see[i].any()):
                continue
            kk, vv = k[see[i]], v[see[i]]
            pages = [int(table[a]) for a in sorted(set((see[i].nonzero()[:, 0] // self.T).tolist()))]
            for h in range(self.H):
                z = scale * (q[i, h] @ kk[:, h].T)                       # [G, m]
                lse[i, h] = torch.logsumexp(z, -1)
                p = torch.exp(z - lse[i, h][:, None])
                out[i, h] = p @ vv[:, h]
                size[0, i, h] = p @ vv[:, h].abs()
                top = self.scale[1][pages, h].max()
                codes = TABLE[self.codes[1][pages][:, :, h].long()].abs().nan_to_num(0.0).sum((0, 1))
                size[1, i, h] = p.amax(-1, keepdim=True) * top * codes
                dz[i, h] = (scale * (q[i, h].abs() @ kk[:, h].abs().T)).amax(-1) * (D + 16) * 2.0 ** -23
        return out.view(c, HQ, D), lse.view(c, HQ), size.view(2, c, HQ, D), dz.view(c, HQ)


def bounds(out, lse, size, dz, dtype, n):
    """Largest error of out and lse.  A weight carries its rounding to FP16 (2^-11), that of the exponential and
    the FP32 steps around it (2^-20), and the score's error dz on it and on the sum (FP32 sums over n keys:
    n 2^-24); below FP16's normal range its rounding is half of the smallest step, 2^-25, where the largest weight
    is held as at least 2^11; the output is rounded once."""
    rel = 2.0 ** -11 + 2.0 ** -20 + 2 * dz[..., None] + n * 2.0 ** -24
    half = torch.finfo(dtype).eps / 2
    o = (size[0] * rel + size[1] * 2.0 ** -36) * (1 + half) + out.abs() * half + torch.finfo(dtype).tiny
    return o, dz + lse.abs().nan_to_num(0, 0, 0) * 2.0 ** -22 + 2.0 ** -19 + n * 2.0 ** -24


class Setup:
    """A cache on the CPU filled by writes, its tables, and tensors for the device calls."""

    def __init__(self, *, D, H, T, lens, dtype, by_head=False, seed=0, spare=3, spread=1.0, dev="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.rng = random.Random(seed)
        self.D, self.H, self.T, self.lens, self.by_head, self.g, self.dev = D, H, T, list(lens), by_head, g, dev
        self.dtype = torch.float16 if dtype == "fp16" else torch.bfloat16
        self.dtype_name = dtype
        counts = [-(-n // T) for n in self.lens]
        self.pages = sum(counts) + spare
        order = torch.randperm(self.pages, generator=g).tolist()
        width = max([1] + counts)
        self.tables = torch.full((len(self.lens), width), -1, dtype=torch.int32)
        for s, n in enumerate(counts):
            for i in range(n):
                self.tables[s, i] = order.pop()
        self.ref = Cache(self.pages, T, H, D)
        for role in range(2):  # what no token holds is any byte, NaN among them, under a scale of NaN
            self.ref.codes[role].copy_(torch.randint(0, 256, self.ref.codes[role].shape, generator=g, dtype=torch.uint8))
            self.ref.scale[role].fill_(math.nan)
        self.spread = spread

    def values(self, n):
        x = torch.randn(n, self.H, self.D, generator=self.g) * torch.exp(
            self.spread * torch.randn(n, self.H, 1, generator=self.g))
        return x.to(self.dtype)

    def fill(self, lens=None):
        for s, n in enumerate(self.lens if lens is None else lens):
            if n:
                self.ref.write(self.tables[s], 0, (self.values(n), self.values(n)))

    def queries(self, n, HQ):
        return (torch.randn(n, HQ, self.D, generator=self.g) * 1.5).to(self.dtype)

    def strides(self):
        T, H, D = self.T, self.H, self.D
        return (H * T * D, D, T * D) if self.by_head else (T * H * D, H * D, D)

    def device_layer(self, cache8):
        k, v = ((c.transpose(1, 2) if self.by_head else c).contiguous().to(self.dev) for c in self.ref.codes)
        ks, vs = (s.float().to(self.dev) for s in self.ref.scale)
        return cache8.Layer(k, v, ks, vs)

    def cache(self, cache8, HQ):
        return cache8.Cache8(dtype=self.dtype_name, head_dim=self.D, num_kv_heads=self.H, num_q_heads=HQ,
                             block_tokens=self.T, num_blocks=self.pages, strides=self.strides())

    def batch(self, cache8, new=None, lens=None, errors=None, hints=True):
        lens = self.lens if lens is None else lens
        dev = self.dev
        cu, n_new = None, None
        if new is not None:
            cu = torch.tensor([0] + torch.tensor(new).cumsum(0).tolist(), dtype=torch.int32, device=dev)
            n_new = sum(new)
        kw = dict(max_new=max(new) if new else 1, max_len=max(lens)) if hints else {}
        return cache8.Batch(self.tables.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev), cu, n_new=n_new,
                            errors=errors, **kw)

    def codes_of(self, layer):
        return [(c.transpose(1, 2) if self.by_head else c).cpu() for c in (layer.k, layer.v)]
