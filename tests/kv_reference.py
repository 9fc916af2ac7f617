"""Paged key/value caches for tests, and the three operators' definitions in
binary64 (torch on whatever device the tensors are on; none of the package's
code)."""

import math

import torch

LIMIT = {"int8": 127.0, "e4m3": 448.0}
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # relative error of one rounding
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}  # the smallest subnormal


def quantise(x, fmt):
    """Codes (one byte each, as int8) and scales of x[..., dim], in binary32 as documented."""
    x = x.float()
    a = x.abs().amax(-1)
    limit = torch.full_like(a, LIMIT[fmt])  # tensor by tensor: a true division
    scale = a / limit
    inv = torch.where(a > 0, torch.clamp(limit / a, max=torch.finfo(torch.float32).max), torch.zeros_like(a))
    y = torch.clamp(x * inv[..., None], -LIMIT[fmt], LIMIT[fmt])
    if fmt == "int8":
        return torch.round(y).nan_to_num(0.0).to(torch.int8), scale
    return y.to(torch.float8_e4m3fn).view(torch.int8), scale


def codes64(codes, fmt):
    return codes.contiguous().view(torch.float8_e4m3fn).float().double() if fmt == "e4m3" else codes.double()


class Case:
    """A cache with its batch: lens[b] cached tokens, new[b] of them this call's."""

    def __init__(self, lens, new, *, heads=2, group=2, dim=64, page=16, dtype=torch.bfloat16, fmt="16bit",
                 layout="thd", seed=0, spare=3, k_gain=1.0, fill=None, device="cuda", table_pages=None):
        g = torch.Generator(device=device).manual_seed(seed)
        self.lens, self.new, self.heads, self.group, self.dim, self.page = list(lens), list(new), heads, group, dim, page
        self.dtype, self.fmt, self.device = dtype, fmt, device
        need = [-(-n // page) for n in lens]
        self.pages = sum(need) + spare
        width = table_pages or max(need + [1])
        perm = torch.randperm(self.pages, generator=g, device=device).to(torch.int32)
        # entries past a sequence's last page name no page: they must not be followed
        self.table = torch.full((len(lens), width), 0x7FFFFFF0, dtype=torch.int32, device=device)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.cu = torch.tensor([0] + list(torch.tensor(new).cumsum(0)), dtype=torch.int32, device=device)
        self.len_dev = torch.tensor(lens, dtype=torch.int32, device=device)
        self.T = sum(new)

        def rand(*shape, gain=1.0):
            return torch.randn(*shape, generator=g, device=device) * gain

        shape = (self.pages, page, heads, dim)
        gain = torch.exp(torch.linspace(-1.5, 1.5, heads, device=device))[:, None]
        kf, vf = rand(*shape, gain=k_gain).to(dtype), (rand(*shape) * gain + 0.25).to(dtype)
        store = dtype if fmt == "16bit" else torch.int8

        def place(shape):
            if layout == "thd":
                return torch.empty(shape, dtype=store, device=device)
            if layout == "htd":
                return torch.empty(shape[0], shape[2], shape[1], shape[3], dtype=store, device=device).transpose(1, 2)
            # K and V side by side in one allocation, rows padded by 16 bytes
            pad = 16 // store.itemsize
            return torch.empty(shape[0], shape[1], 2, shape[2], shape[3] + pad, dtype=store,
                               device=device)[:, :, 0, :, :shape[3]]

        if layout == "kv":
            pad = 16 // store.itemsize
            both = torch.empty(self.pages, page, 2, heads, dim + pad, dtype=store, device=device)
            self.k, self.v = both[:, :, 0, :, :dim], both[:, :, 1, :, :dim]
        else:
            self.k, self.v = place(shape), place(shape)
        self.ks = self.vs = None
        if fmt == "16bit":
            self.k.copy_(kf)
            self.v.copy_(vf)
        else:
            self.ks, self.vs = (torch.empty(self.pages, heads, page, device=device).transpose(1, 2) for _ in range(2))
            for data, scales, x in ((self.k, self.ks, kf), (self.v, self.vs, vf)):
                c, s = quantise(x, fmt)
                data.copy_(c)
                scales.copy_(s)
        if fill is not None:  # what no sequence has written yet
            used = torch.zeros(self.pages, page, dtype=torch.bool, device=device)
            for b, n in enumerate(self.lens):
                for i in range(need[b]):
                    used[int(self.table[b, i]), :min(page, n - i * page)] = True
            if fmt == "16bit":
                self.k[~used], self.v[~used] = fill, fill
            else:
                self.ks[~used], self.vs[~used] = fill, fill
                if fmt == "e4m3":
                    self.k[~used], self.v[~used] = 0x7F, 0x7F
        self.q = rand(self.T, heads * group, dim).to(dtype)
        self.k_new, self.v_new = rand(self.T, heads, dim).to(dtype), (rand(self.T, heads, dim) * gain).to(dtype)

    def objects(self, cc, **over):
        fmt = {"16bit": cc.CCCL_KV_16BIT, "int8": cc.CCCL_KV_INT8, "e4m3": cc.CCCL_KV_E4M3}[self.fmt]
        cache = cc.KvCache(self.k, self.v, self.ks, self.vs, dtype=self.dtype, fmt=fmt)
        kw = dict(n_tokens=self.T, max_new=max(self.new + [1]), max_len=max(self.lens + [1]))
        kw.update(over)
        return cache, cc.KvBatch(self.table, self.cu, self.len_dev, **kw)

    def stored(self, b):
        """K and V of sequence b's positions, [len, heads, dim] in binary64."""
        n = self.lens[b]
        rows = self.table[b, :-(-n // self.page)].long()
        out = []
        for data, scales in ((self.k, self.ks), (self.v, self.vs)):
            x = data[rows].flatten(0, 1)[:n]
            x = x.double() if self.fmt == "16bit" else codes64(x, self.fmt)
            if scales is not None:
                x = x * scales[rows].flatten(0, 1)[:n].double()[..., None]
            out.append(x)
        return out

    def visible(self, b, causal, window):
        """[new, len] truth values."""
        n, t = self.new[b], self.lens[b]
        pos = torch.arange(t - n, t, device=self.device)[:, None]
        at = torch.arange(t, device=self.device)[None]
        seen = torch.ones(n, t, dtype=torch.bool, device=self.device)
        if causal:
            seen &= at <= pos
        if window:
            seen &= at > pos - window
        return seen

    def attention(self, scale=None, causal=True, window=0):
        """Result and log-sum-exp in binary64, with elementwise error bounds for
        a kernel that takes exact products of its 16-bit (8-bit) operands, sums
        in binary32, rounds each probability once to the 16-bit type and rounds
        the result once.

        A score is off by at most d = (dim + 8) 2^-23 |scale| sum |q k| (any
        order of summation, one rounding per term, and the rounding of its
        product with the scale), a probability relatively by 2 d (its score and
        the maximum it is taken against) + 2^-20 (exponential, its argument's
        rounding is in d) + one rounding u; the sums over keys add
        (tiles + 8) 2^-23 < 2^-12 relative to sum p |v| for the lengths tested."""
        u = UNIT[self.dtype]
        scale = 1.0 / math.sqrt(self.dim) if scale is None else scale
        H, G, D = self.heads, self.group, self.dim
        out = torch.zeros(self.T, H * G, D, dtype=torch.float64, device=self.device)
        lse = torch.full((self.T, H * G), -math.inf, dtype=torch.float64, device=self.device)
        tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
        row = 0
        for b, n in enumerate(self.new):
            if n == 0 or self.lens[b] == 0:
                row += n
                continue
            k, v = self.stored(b)
            seen = self.visible(b, causal, window)
            some = seen.any(1)
            clean_k, clean_v = k, v
            for h in range(H * G):
                q = self.q[row:row + n, h].double()
                kk, vv = clean_k[:, h // G], clean_v[:, h // G]
                s = torch.where(seen, (q[:, None] * kk[None]).sum(-1) if k.isnan().any() else q @ kk.T, 0.0) * scale
                s = torch.where(seen, s, -math.inf)
                m = s.amax(1, keepdim=True)
                p = torch.where(seen, torch.exp(s - m), 0.0)
                l = p.sum(1, keepdim=True)
                p = p / l
                # hidden keys take no part, whatever they hold
                if not torch.isfinite(vv).all():
                    o = torch.where(seen[..., None], p[..., None] * vv[None], 0.0).sum(1)
                    av = torch.where(seen[..., None], p[..., None] * vv[None].abs(), 0.0).sum(1)
                else:
                    o, av = p @ vv, p @ vv.abs()
                mag = torch.where(seen, q.abs() @ kk.abs().T, 0.0).amax(1, keepdim=True) * abs(scale)
                d = (D + 8) * 2.0 ** -23 * mag
                rel = 2 * (2 * d + 2.0 ** -20 + 2.0 ** -12) + u
                out[row:row + n, h] = torch.where(some[:, None], o, 0.0)
                tol[row:row + n, h] = torch.where(some[:, None], rel * av + u * (o.abs() + rel * av) + TINY[self.dtype], 0.0)
                lse[row:row + n, h] = torch.where(some, (m + torch.log(l)).squeeze(1), -math.inf)
                ltol[row:row + n, h] = (2 * d.squeeze(1) + 2.0 ** -12 + 2.0 ** -22 * lse[row:row + n, h].abs().nan_to_num(0, 0, 0))
            row += n
        return out, lse, tol, ltol
