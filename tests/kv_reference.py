"""Plain references of the cache-writing and 8-bit operators, for the tests:
paged caches of every type drawn from a seed, appending in fp32 or fp64, and
(causal) attention in fp64 with the bounds that its rounding errors obey.
Everything here runs on the CPU."""

from __future__ import annotations

import math

import torch

QMAX = {"fp8_e4m3": 448.0, "fp8_e4m3_block": 448.0, "int8_block": 127.0}
FORMATS = ["bf16", "fp8_e4m3", "fp8_e4m3_block", "int8_block"]
BLOCK_FORMATS = ["fp8_e4m3_block", "int8_block"]


def is_block(kv):
    return kv.endswith("_block")


def cache_dtype(kv):
    return {"bf16": torch.bfloat16, "int8_block": torch.int8}.get(kv, torch.float8_e4m3fn)


def encode(x, kv):
    """Nearest code (ties to even), saturating."""
    if kv == "bf16":
        return x.to(torch.bfloat16)
    x = x.clamp(-QMAX[kv], QMAX[kv])
    return x.round().to(torch.int8) if kv == "int8_block" else x.float().to(torch.float8_e4m3fn)


def scale_exponent(amax, kv):
    """The smallest e in [-100, 100] with amax <= QMAX 2^e."""
    if not amax > 0:
        return -100
    m, e = math.frexp(amax)
    m0, e0 = math.frexp(QMAX[kv])
    return max(-100, min(100, e - e0 + (m > m0)))


def poison(kv):
    return {"bf16": float("nan"), "int8_block": -128.0}.get(kv, float("nan"))


class Cache:
    """A paged cache on the CPU: k, v [num_blocks, Hk, B, D] logical pages (in
    the cache's element type), scales, block tables and lengths.  Unused slots
    and blocks hold NaN (int8: -128), unused table entries -1, the scales of
    unused blocks NaN."""

    def __init__(self, kv, lens, Hk, D, B, seed=0, spare=5, amplitude=1.0, pow2=True,
                 max_blocks=None, shared_blocks=0):
        self.kv, self.Hk, self.D, self.B = kv, Hk, D, B
        g = torch.Generator().manual_seed(seed)
        nb = [-(-t // B) for t in lens]
        width = max_blocks or max(1, max(nb, default=1))
        need = shared_blocks + sum(max(0, n - shared_blocks) for n in nb)
        self.num_blocks = need + spare
        perm = torch.randperm(self.num_blocks, generator=g)
        self.tables = torch.full((len(lens), width), -1, dtype=torch.int32)
        at = shared_blocks
        for s, n in enumerate(nb):
            k = min(n, shared_blocks)
            self.tables[s, :k] = perm[:k].int()
            self.tables[s, k:n] = perm[at:at + n - k].int()
            at += n - k
        self.lens = torch.tensor(lens, dtype=torch.int32)
        dt = cache_dtype(kv)
        shape = (self.num_blocks, Hk, B, D)
        self.k = torch.full(shape, poison(kv)).to(dt)
        self.v = torch.full(shape, poison(kv)).to(dt)
        if is_block(kv):
            self.ks = torch.full((self.num_blocks, Hk), float("nan"))
            self.vs = self.ks.clone()
        elif kv == "fp8_e4m3":
            self.ks, self.vs = torch.tensor([0.05]), torch.tensor([0.03])
        else:
            self.ks = self.vs = None
        for s, t in enumerate(lens):
            for j in range(nb[s]):
                blk, m = int(self.tables[s, j]), min(B, t - j * B)
                for pages, scale in ((self.k, self.ks), (self.v, self.vs)):
                    x = torch.randn((Hk, m, D), generator=g) * amplitude
                    x = x * torch.exp(0.5 * torch.randn((Hk, 1, 1), generator=g))
                    if is_block(kv):
                        a = x.abs().amax(dim=(1, 2))
                        if pow2:
                            sc = torch.tensor([2.0 ** scale_exponent(float(y), kv) for y in a])
                        else:
                            sc = a / QMAX[kv]
                        scale[blk] = sc
                        x = x / sc[:, None, None]
                    elif kv == "fp8_e4m3":
                        x = x / scale
                    self._set(pages, blk, slice(0, m), encode(x, kv))

    @staticmethod
    def _raw(t):
        return t if t.dtype in (torch.bfloat16, torch.int8) else t.view(torch.uint8)

    def _set(self, pages, blk, slots, x):
        self._raw(pages)[blk][:, slots] = self._raw(x)

    # ---- the library's layouts
    def packed(self, device="cpu"):
        x = 16 // self.k.element_size()
        nb, Hk, B, D = self.k.shape
        k = self._raw(self.k).view(nb, Hk, B, D // x, x).permute(0, 1, 3, 2, 4).contiguous()
        v = self._raw(self.v).permute(0, 1, 3, 2).contiguous()
        return k.view(self.k.dtype).to(device), v.view(self.v.dtype).to(device)

    def scales(self, device="cpu"):
        return (None, None) if self.ks is None else (self.ks.to(device), self.vs.to(device))

    def unpacked(self, kc, vc):
        """The logical pages of caches in the library's layouts."""
        dt = kc.dtype
        kc, vc = self._raw(kc.cpu()), self._raw(vc.cpu())
        nb, Hk, C, B, x = kc.shape
        k = kc.permute(0, 1, 3, 2, 4).reshape(nb, Hk, B, C * x).contiguous().view(dt)
        return k, vc.permute(0, 1, 3, 2).contiguous().view(dt)

    # ---- values in fp64
    def values(self, s):
        """Keys and values [T, Hk, D] of sequence s in fp64, and the V scale of
        each (token, head)."""
        t = int(self.lens[s])
        n = -(-t // self.B)
        ids = self.tables[s, :n].long()
        out = []
        for pages, scale in ((self.k, self.ks), (self.v, self.vs)):
            x = self._raw(pages)[ids].view(pages.dtype).double()  # [n, Hk, B, D]
            sc = torch.ones((n, self.Hk), dtype=torch.float64)
            if is_block(self.kv):
                sc = scale[ids].double()
            elif scale is not None:
                sc = sc * scale.double()
            x = x * sc[:, :, None, None]
            out.append(x.transpose(1, 2).reshape(-1, self.Hk, self.D)[:t])
            last = sc
        per_token = last.repeat_interleave(self.B, dim=0)[:t]
        return out[0], out[1], per_token

    # ---- appending
    def append(self, key, value, query_start, angles=None, interleaved=False, positions=None,
               query=None, dtype=torch.float64):
        """Write rows of key / value [T, Hk, D] (bf16) as pa_append_kv does, with
        the arithmetic in `dtype`; returns the rotated queries (unrounded)."""
        start = query_start.tolist()
        out = None if query is None else torch.zeros(query.shape, dtype=dtype)
        for s in range(len(start) - 1):
            a, b = start[s], start[s + 1]
            n, t = b - a, int(self.lens[s])
            if n == 0:
                continue
            pos = torch.arange(t - n, t) if positions is None else positions[a:b].long()
            k = rotate(key[a:b].to(dtype), pos, angles, interleaved)
            v = value[a:b].to(dtype)
            if query is not None:
                out[a:b] = rotate(query[a:b].to(dtype), pos, angles, interleaved)
            i = 0
            while i < n:
                j, off = divmod(t - n + i, self.B)
                m = min(n - i, self.B - off)
                blk = int(self.tables[s, j])
                for pages, scale, x in ((self.k, self.ks, k), (self.v, self.vs, v)):
                    self._append_block(pages, scale, blk, off, x[i:i + m].transpose(0, 1))
                i += m
        return out

    def _append_block(self, pages, scale, blk, off, x):  # x [Hk, m, D]
        kv, m = self.kv, x.shape[1]
        if is_block(kv):
            for h in range(self.Hk):
                a = x[h].abs()
                a = a[torch.isfinite(a)]
                want = 2.0 ** scale_exponent(float(a.max()) if a.numel() else 0.0, kv)
                old = float(scale[blk, h])
                if off and old >= want:
                    want = old
                elif off:
                    page = self._raw(pages)[blk, h]
                    codes = page.view(pages.dtype)[:off].to(x.dtype)
                    page[:off] = self._raw(encode(codes * (old / want), kv))
                scale[blk, h] = want
            x = x / scale[blk].to(x.dtype)[:, None, None]
        elif kv == "fp8_e4m3":
            x = x / scale.to(x.dtype)
        codes = encode(x, kv)
        if kv == "int8_block":  # (a NaN is stored as 0)
            codes = torch.where(torch.isnan(x), torch.zeros_like(codes), codes)
        self._set(pages, blk, slice(off, off + m), codes)


def rotate(x, pos, angles, interleaved):
    """x [n, H, D] rotated at positions pos by the table angles [P, R]."""
    if angles is None:
        return x
    R = angles.shape[1]
    c = angles[pos, :R // 2].to(x.dtype)[:, None]
    s = angles[pos, R // 2:].to(x.dtype)[:, None]
    y = x.clone()
    lo, hi = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2),
                                                                   slice(R // 2, R))
    a, b = x[..., lo], x[..., hi]
    y[..., lo], y[..., hi] = a * c - b * s, a * s + b * c
    return y


def angle_table(positions, R, base=10000.0):
    f = base ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
    a = torch.arange(positions, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], dim=1).float()


def attention(cache, query, query_start, scale, alibi=None):
    """Causal attention of the last rows of each sequence in fp64, and a bound
    on what the kernels may be off by: (out, bound), both [T, Hq, D].  Rows that
    no sequence owns are zeros.

    The bound, with u = eps / 2 of a type (bf16 2^-8, f16 2^-11):
      * the output is rounded to bf16: u_bf16 |o|;
      * each weight is rounded to the operand's type, relative to itself
        (2^-8 in bf16, 2^-11 in f16, whose weights also have an absolute error
        of 2^-25 of the largest one): u A with A = sum_t p_t |v_t|, and
        2^-25 sum_t |code_t| max_t (vs_t p_t) for the codes of an 8-bit cache;
      * a logit is off by at most D 2^-23 scale sum_d |q_d k_d| (fp32 sums in
        the tensor cores, which may truncate) plus 2^-22 of its own size, and
        that is the relative error of its weight, in the sum and in the
        denominator: 2 A times that;
      * exponentials and the fp32 sums of weights: 2^-20 A covers them."""
    start = query_start.tolist()
    T, Hq, D = query.shape
    out = torch.zeros((T, Hq, D), dtype=torch.float64)
    bound = torch.zeros_like(out)
    G = Hq // cache.Hk
    u_w = 2.0 ** -8 if cache.kv == "bf16" else 2.0 ** -11
    for s in range(len(start) - 1):
        a, b = start[s], start[s + 1]
        n, t = b - a, int(cache.lens[s])
        if n == 0 or t == 0:
            continue
        k, v, vs = cache.values(s)
        hidden = torch.arange(t)[None, :] > torch.arange(t - n, t)[:, None]  # [n, t]
        for h in range(Hq):
            q, kh, vh = query[a:b, h].double(), k[:, h // G], v[:, h // G]
            x = q @ torch.nan_to_num(kh).T * scale
            size = q.abs() @ torch.nan_to_num(kh).abs().T * abs(scale)
            nan = torch.isnan(kh).any(dim=1)
            x = torch.where(nan[None], float("nan"), x)
            if alibi is not None:
                x = x + float(alibi[h]) * (torch.arange(t) - (t - 1))
            x = x.masked_fill(hidden, -math.inf)
            p = torch.softmax(x, dim=1)
            o = torch.stack([(p[i, :t - n + i + 1, None] * vh[:t - n + i + 1]).sum(0)
                             for i in range(n)])
            va = torch.nan_to_num(vh).abs()
            A = torch.nan_to_num(p) @ va
            seen = torch.where(hidden, 0.0, size)
            dx = (D * 2.0 ** -23 + 2.0 ** -22) * seen.amax(dim=1, keepdim=True)
            err = 2.0 ** -8 * o.abs() + A * (u_w + 2 * dx + 2.0 ** -20)
            if cache.kv != "bf16":
                w = vs[:, h // G]
                code = (~hidden).double() @ (va / torch.where(w > 0, w, 1.0)[:, None])
                err = err + 2.0 ** -25 * code * (torch.nan_to_num(p) * w).amax(1, keepdim=True)
            out[a:b, h], bound[a:b, h] = o, err
    return out, bound
