"""What is measured of the operators that write a paged KV cache and read it in 8 bits.

``append``: new tokens' keys and values go into a paged cache (bf16, e4m3 with
one scale per tensor, e4m3 or int8 with one scale per block of tokens and kv
head), keys and queries rotated by their positions on the way.

``decode``: one query token per sequence attends over a cache of 8-bit codes
with a scale per block and kv head.

``prefill``: the last query tokens of each sequence (a prompt, or a chunk of
one), whose keys and values are in the cache already, attend over it causally.

``run`` computes them in plain torch where ``own`` is false, and through the
package where it is true.  A case's lengths come from its own ``lens`` number,
its values from the seed.
"""

import math
import random

import torch

own = False

DEV = "cuda"
QMAX = {"fp8_e4m3": 448.0, "fp8_e4m3_block": 448.0, "int8_block": 127.0}
MIN_EXP, MAX_EXP = -100, 100  # exponents of a block's scale


# ------------------------------------------------------------------ the cases
def _append(name, kv, seqs, hq, hk, d, b, new, past, lens, rot=None, interleaved=False, fused=True):
    c = dict(op="append", kv=kv, seqs=seqs, hq=hq, hk=hk, d=d, b=b, new_lo=new[0], new_hi=new[1],
             past_lo=past[0], past_hi=past[1], lens=lens, rot=d if rot is None else rot,
             interleaved=interleaved, fused=fused)
    return dict(c, name=name) if name else c


def _decode(name, kv, seqs, hq, hk, d, b, length, lens, prefix=0, pow2=True):
    c = dict(op="decode", kv=kv, seqs=seqs, hq=hq, hk=hk, d=d, b=b, len_lo=length[0],
             len_hi=length[1], lens=lens, prefix=prefix, pow2=pow2)
    return dict(c, name=name) if name else c


def _prefill(name, kv, seqs, hq, hk, d, b, new, past, lens):
    c = dict(op="prefill", kv=kv, seqs=seqs, hq=hq, hk=hk, d=d, b=b, new_lo=new[0], new_hi=new[1],
             past_lo=past[0], past_hi=past[1], lens=lens)
    return dict(c, name=name) if name else c


def listed():
    return [
        # A decode step's append for the tiny MHA batch: latency only.
        _append("append 4x1 bf16", "bf16", 4, 8, 8, 64, 16, (1, 1), (0, 255), 11),
        # A decode step of 256 sequences over an 8-bit cache: pages partly filled, some scales grow.
        _append("append 256x1 e4m3 block", "fp8_e4m3_block", 256, 32, 8, 128, 16, (1, 1),
                (0, 900), 13),
        # Prompts of several requests in one call, grouped heads, into a bf16 cache.
        _append("append prompts bf16 gqa", "bf16", 16, 64, 8, 128, 16, (200, 1801), (0, 0), 14),
        # Chunks of long prompts behind what is cached, odd lengths, int8 blocks of 32 tokens,
        # a partial, interleaved rotation, dense rows.
        _append("append chunks int8 block", "int8_block", 12, 32, 8, 128, 32, (300, 2501),
                (0, 3001), 15, rot=64, interleaved=True, fused=False),
        # The tiny MHA batch: latency only.
        _decode("decode 4x256 int8", "int8_block", 4, 8, 8, 64, 16, (1, 256), 21),
        # Grouped heads, lengths far apart.
        _decode("decode gqa 512-8192 e4m3", "fp8_e4m3_block", 128, 64, 8, 128, 16, (512, 8192), 22),
        # One head per kv head, scales of another quantiser (not powers of two).
        _decode("decode mha 32x4096 int8", "int8_block", 32, 32, 32, 128, 16, (4001, 4096), 24,
                pow2=False),
        # One long sequence: the tokens are split over the GPU and joined.
        _decode("decode 1x131072 e4m3 b32", "fp8_e4m3_block", 1, 32, 8, 128, 32, (131072, 131072),
                25),
        # One long prompt.
        _prefill("prefill 1x8192 bf16", "bf16", 1, 32, 8, 128, 16, (8192, 8192), (0, 0), 31),
        # Prompts of several short requests, one head per kv head.
        _prefill("prefill prompts bf16 mha", "bf16", 8, 16, 16, 128, 16, (100, 900), (0, 0), 32),
        # Chunks behind cached tokens, grouped heads, an 8-bit cache.
        _prefill("prefill chunks e4m3 block", "fp8_e4m3_block", 4, 64, 8, 128, 16, (257, 1025),
                 (0, 4001), 33),
        # A few tokens against a long cache: the tokens are split over the GPU and joined.
        _prefill("prefill 7 over 30000 int8", "int8_block", 2, 32, 8, 128, 32, (3, 7),
                 (28001, 30000), 34),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    d = rng.choice([64, 128, 128])
    b = rng.choice([16, 32])
    hk = rng.choice([1, 2, 4, 8, 8, 32])
    g = rng.choice([1, 1, 2, 4, 4, 5, 8, 16]) if hk < 32 else 1
    lens = rng.randrange(1 << 20)
    op = rng.choice(["append", "append", "decode", "prefill"])
    if op == "append":
        kv = rng.choice(["bf16", "fp8_e4m3", "fp8_e4m3_block", "int8_block"])
        seqs = _log_int(rng, 1, 256)
        one = rng.random() < 0.4
        # rows x elements of a row stay within the largest listed case's
        most = 1 if one else max(1, min(8192, 16384 * 80 * 128 // (seqs * (2 * hk + hk * g) * d)))
        hi = 1 if one else _log_int(rng, 1, most)
        lo = rng.choice([0, 1, hi]) if hi > 1 else 1
        past = rng.choice([0, 17, 1000])
        return _append(None, kv, seqs, hk * g, hk, d, b, (min(lo, hi), hi), (0, past), lens,
                       rot=rng.choice([d, d, d // 2, 16]), interleaved=rng.random() < 0.5,
                       fused=rng.random() < 0.5)
    if op == "prefill":
        kv = rng.choice(["bf16", "fp8_e4m3", "fp8_e4m3_block", "int8_block"])
        seqs = _log_int(rng, 1, 16)
        # logits (of a padded batch) and codes stay within the largest listed cases'
        logits = 8192 * 8192 * 32 // (seqs * hk * g)
        hi = _log_int(rng, 1, max(1, min(8192, math.isqrt(logits))))
        past = rng.choice([0, 0, _log_int(rng, 1, max(1, min(60000, logits // hi - hi,
                                                               (1 << 30) // (seqs * hk * d))))])
        return _prefill(None, kv, seqs, hk * g, hk, d, b, (rng.choice([0, 1, hi]), hi),
                        (rng.choice([0, past]), past), lens)
    kv = rng.choice(["fp8_e4m3_block", "int8_block"])
    seqs = _log_int(rng, 1, 128)
    # neither codes nor products are more than the largest listed case's
    most = max(1, min(131072, (1 << 29) // (seqs * hk * d),
                      128 * 4352 * 64 * 128 // (seqs * hk * g * d)))
    hi = _log_int(rng, 1, most)
    lo = rng.choice([0, 1, max(1, hi // 4), hi])
    prefix = rng.choice([0, 0, 0, lo // b // 2])
    return _decode(None, kv, seqs, hk * g, hk, d, b, (lo, hi), lens, prefix=prefix,
                   pow2=rng.random() < 0.5)


def _new_and_past(c):
    r = random.Random(c["lens"])
    new = [r.randint(c["new_lo"], c["new_hi"]) for _ in range(c["seqs"])]
    past = [r.randint(c["past_lo"], c["past_hi"]) for _ in range(c["seqs"])]
    return new, past


def _decode_lens(c):
    r = random.Random(c["lens"])
    return [r.randint(c["len_lo"], c["len_hi"]) for _ in range(c["seqs"])]


def _elem(kv):
    return 2 if kv == "bf16" else 1


def work(c):
    hq, hk, d, b = c["hq"], c["hk"], c["d"], c["b"]
    if c["op"] == "append":
        new, past = _new_and_past(c)
        t = sum(new)
        rows = {p for n, q in zip(new, past) for p in range(q, q + n)}
        n = t * (hq + 2 * hk) * d * 2 + len(rows) * c["rot"] * 4         # rows and angles
        n += t * hq * d * 2 + 2 * t * hk * d * _elem(c["kv"])            # queries, keys, values
        blocks = sum((q + m - 1) // b - q // b + 1 for m, q in zip(new, past) if m)
        n += 4 * blocks + 8 * c["seqs"]
        if c["kv"].endswith("_block"):
            n += 2 * blocks * hk * 4
        return {"bytes": n, "flops": 3 * t * (hq + hk) * c["rot"]}
    if c["op"] == "prefill":
        new, past = _new_and_past(c)
        tokens = sum(m + q for m, q in zip(new, past) if m)
        blocks = sum(-(-(m + q) // b) for m, q in zip(new, past) if m)
        n = 2 * tokens * hk * d * _elem(c["kv"]) + 2 * sum(new) * hq * d * 2 + 4 * blocks
        n += 2 * blocks * hk * 4 if c["kv"].endswith("_block") else 0
        pairs = sum(m * q + m * (m + 1) // 2 for m, q in zip(new, past))
        return {"bytes": n + 8 * c["seqs"], "flops": 4 * pairs * hq * d}
    lens = _decode_lens(c)
    own_tokens = sum(max(0, t - c["prefix"] * b) for t in lens) + c["prefix"] * b
    own_blocks = sum(max(0, -(-t // b) - c["prefix"]) for t in lens) + c["prefix"]
    n = 2 * own_tokens * hk * d + 2 * own_blocks * hk * 4  # codes and scales
    n += 2 * c["seqs"] * hq * d * 2 + 4 * sum(-(-t // b) for t in lens) + 4 * c["seqs"]
    return {"bytes": n, "flops": 4 * sum(lens) * hq * d}


# ----------------------------------------------------------------- the inputs
def _tables(blocks_of, prefix, gen):
    """Block tables of sequences of so many blocks each, all blocks distinct but
    the first `prefix`; entries behind a sequence's last block are -1."""
    width = max(1, max(blocks_of))
    need = prefix + sum(max(0, n - prefix) for n in blocks_of)
    pool = need + max(2, need // 16)
    perm = torch.randperm(pool, generator=gen, device=DEV).to(torch.int32)
    bt = torch.full((len(blocks_of), width), -1, dtype=torch.int32, device=DEV)
    at = prefix
    for s, n in enumerate(blocks_of):
        k = min(n, prefix)
        bt[s, :k] = perm[:k]
        bt[s, k:n] = perm[at:at + n - k]
        at += n - k
    return bt, pool


def _cache_type(kv):
    return {"bf16": torch.bfloat16, "int8_block": torch.int8}.get(kv, torch.float8_e4m3fn)


def _random_pages(kv, pool, hk, shape, pow2, gen):
    """[pool, hk, *shape] pages of normal values (a few channels larger, as keys
    have them) in the cache's type, and the scale of each (block, head)."""
    pages = torch.empty((pool, hk) + shape, dtype=_cache_type(kv), device=DEV)
    scale = torch.ones((pool, hk), device=DEV) if kv.endswith("_block") else None
    step = max(1, (1 << 26) // (hk * math.prod(shape)))
    for i in range(0, pool, step):
        x = torch.randn((min(step, pool - i), hk) + shape, generator=gen, device=DEV)
        x *= torch.exp(0.5 * torch.randn((x.shape[0], hk) + (1,) * len(shape), generator=gen,
                                         device=DEV))
        if kv == "bf16":
            pages[i:i + step] = x.to(torch.bfloat16)
            continue
        if kv == "fp8_e4m3":
            x /= 0.05
        else:
            s = x.abs().amax(dim=tuple(range(2, x.dim()))) / QMAX[kv]
            s = torch.exp2(torch.ceil(torch.log2(s))) if pow2 else s
            scale[i:i + step] = s
            x /= s.view(s.shape + (1,) * len(shape))
        x = x.clamp_(-QMAX[kv], QMAX[kv])
        pages[i:i + step] = x.round_().to(torch.int8) if kv == "int8_block" else x.to(
            torch.float8_e4m3fn)
    return pages, scale


def _angles(positions, rot):
    """fp32 [positions, rot]: the cosines, then the sines, of p * 10000^(-2i/rot)."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    a = torch.arange(positions, dtype=torch.float64, device=DEV)[:, None] * f
    return torch.cat([a.cos(), a.sin()], dim=1).float()


def prepare(c, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    hq, hk, d, b, kv = c["hq"], c["hk"], c["d"], c["b"], c["kv"]
    x = 8 if kv == "bf16" else 16
    st = dict(c)
    if c["op"] == "append":
        new, past = _new_and_past(c)
        total = [n + p for n, p in zip(new, past)]
        st["bt"], pool = _tables([-(-t // b) for t in total], 0, gen)
        pow2 = True
        t = sum(new)
        if c["fused"]:  # views of one projection's output
            qkv = torch.randn((t, (hq + 2 * hk) * d), generator=gen, device=DEV)
            qkv *= torch.exp(0.5 * torch.randn((t, 1), generator=gen, device=DEV))
            qkv = qkv.to(torch.bfloat16)
            st["query"] = qkv[:, :hq * d].view(t, hq, d)
            st["key"] = qkv[:, hq * d:(hq + hk) * d].view(t, hk, d)
            st["value"] = qkv[:, (hq + hk) * d:].view(t, hk, d)
        else:
            for name, h in (("query", hq), ("key", hk), ("value", hk)):
                st[name] = torch.randn((t, h, d), generator=gen, device=DEV).to(torch.bfloat16)
        st["query_out"] = torch.zeros((t, hq, d), dtype=torch.bfloat16, device=DEV)
        ends = [0]
        for n in new:
            ends.append(ends[-1] + n)
        st["start"] = None if new == [1] * len(new) else torch.tensor(ends, dtype=torch.int32,
                                                                      device=DEV)
        st["angles"] = _angles(max(1, max(total)), c["rot"])
    elif c["op"] == "prefill":
        new, past = _new_and_past(c)
        total = [n + p for n, p in zip(new, past)]
        st["bt"], pool = _tables([-(-t // b) for t in total], 0, gen)
        pow2 = True
        ends = [0]
        for n in new:
            ends.append(ends[-1] + n)
        st["start"] = torch.tensor(ends, dtype=torch.int32, device=DEV)
        st["query"] = torch.randn((ends[-1], hq, d), generator=gen, device=DEV).to(torch.bfloat16)
        st["out"] = torch.empty_like(st["query"])
        st["max_len"], st["max_new"] = max(total), max(new)
    else:
        total = _decode_lens(c)
        st["bt"], pool = _tables([-(-t // b) for t in total], c["prefix"], gen)
        pow2 = c["pow2"]
        st["query"] = torch.randn((len(total), hq, d), generator=gen, device=DEV).to(torch.bfloat16)
        st["out"] = torch.empty_like(st["query"])
        st["max_len"] = max(total)
    st["lens"] = torch.tensor(total, dtype=torch.int32, device=DEV)
    st["kc"], st["ks"] = _random_pages(kv, pool, hk, (d // x, b, x), pow2, gen)
    st["vc"], st["vs"] = _random_pages(kv, pool, hk, (d, b), pow2, gen)
    if kv == "fp8_e4m3":
        st["ks"] = torch.full((1,), 0.05, device=DEV)
        st["vs"] = torch.full((1,), 0.05, device=DEV)
    return st


# ------------------------------------------------------------ the plain forms
def _rotate(x, cos, sin, rot, interleaved):
    """x [T, H, D] in 32 bits; cos, sin [T, rot / 2]."""
    cos, sin = cos[:, None], sin[:, None]
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, a * sin + b * cos
    return y


def _encode(x, kv):
    x = x.clamp(-QMAX[kv], QMAX[kv])
    return x.round().to(torch.int8) if kv == "int8_block" else x.to(torch.float8_e4m3fn)


def _bytes(t):
    return t if t.dtype == torch.bfloat16 else t.view(torch.uint8)


def _store(pages, scale, x, kv, blk, off, first, first_off, is_value):
    """Rows x [T, H, D] (32 bits) into blocks `blk` at slots `off`.  first,
    first_off [S]: the block that each sequence's run begins in, and the slot."""
    t, h, d = x.shape
    if kv.endswith("_block"):
        amax = x.abs().amax(dim=2)  # [T, H]
        need = torch.zeros_like(scale).scatter_reduce_(0, blk[:, None].expand(t, h), amax, "amax")
        m, e = torch.frexp(need)  # the smallest e with need <= QMAX 2^e
        m_max, e_max = math.frexp(QMAX[kv])
        e = torch.where(need > 0, e - e_max + (m > m_max).int(), MIN_EXP).clamp(MIN_EXP, MAX_EXP)
        wanted = torch.ldexp(torch.ones_like(need), e)
        touched = torch.zeros(scale.shape[0], dtype=torch.bool, device=x.device)
        touched[blk] = True
        kept = torch.zeros_like(touched)
        kept[first[first_off > 0]] = True  # blocks that hold earlier tokens
        old = scale.clone()
        now = torch.where(kept[:, None], torch.maximum(old, wanted), wanted)
        scale.copy_(torch.where(touched[:, None], now, old))
        # earlier tokens of blocks whose scale grew: their codes in the new scale
        f, fo = first[first_off > 0], first_off[first_off > 0]
        page = pages[f] if pages.dtype == torch.int8 else pages.view(torch.uint8)[f].view(
            pages.dtype)
        slot = torch.arange(page.shape[3], device=x.device)
        shape = (1, 1, 1, -1) if is_value else (1, 1, 1, -1, 1)
        earlier = slot.view(shape) < fo.view((-1,) + (1,) * (page.dim() - 1))
        ratio = (old[f] / scale[f]).view(scale[f].shape + (1,) * (page.dim() - 2))
        grown = torch.where(earlier, _encode(page.float() * ratio, kv).float(),
                            page.float()).to(pages.dtype)
        _bytes(pages)[f] = _bytes(grown)
        x = x / scale[blk][:, :, None]
    elif kv == "fp8_e4m3":
        x = x / scale
    row = x.to(torch.bfloat16) if kv == "bf16" else _encode(x, kv)
    if is_value:
        _bytes(pages)[blk, :, :, off] = _bytes(row)
    else:
        _bytes(pages)[blk, :, :, off] = _bytes(row).view(t, h, d // pages.shape[4], pages.shape[4])


def _plain_append(st):
    kv, b, rot = st["kv"], st["b"], st["rot"]
    t, seqs = st["key"].shape[0], st["bt"].shape[0]
    row = torch.arange(t, device=DEV)
    start = torch.arange(seqs + 1, device=DEV) if st["start"] is None else st["start"].long()
    s = torch.searchsorted(start[1:].contiguous(), row, right=True)
    lens = st["lens"].long()
    begin = lens - (start[1:] - start[:-1])  # index of each run's first token
    pos = begin[s] + row - start[s]
    blk, off = st["bt"][s, pos // b].long(), pos % b
    some = start[1:] > start[:-1]
    width = st["bt"].shape[1]
    first = st["bt"].gather(1, (begin // b).clamp(max=width - 1)[:, None])[:, 0].long()[some]
    first_off = (begin % b)[some]
    cos, sin = st["angles"][pos, :rot // 2], st["angles"][pos, rot // 2:]
    key = _rotate(st["key"].float(), cos, sin, rot, st["interleaved"])
    _store(st["kc"], st["ks"], key, kv, blk, off, first, first_off, False)
    _store(st["vc"], st["vs"], st["value"].float(), kv, blk, off, first, first_off, True)
    st["query_out"].copy_(_rotate(st["query"].float(), cos, sin, rot, st["interleaved"]))


def _plain_attention(st, query, first):
    """query [S, N, Hq, D] in 32 bits; the token n of sequence s sees the keys
    up to index first[s] + n, and none behind the sequence's last."""
    hk, d, b = st["hk"], st["d"], st["b"]
    seqs, n, hq = query.shape[:3]
    g, nb = hq // hk, st["bt"].shape[1]
    bt = st["bt"].clamp(min=0).long()

    def values(pages, scale):
        x = pages[bt] if pages.element_size() > 1 else pages.view(torch.uint8)[bt]
        x = x.view(pages.dtype).float()
        if st["kv"].endswith("_block"):
            return x * scale[bt].view(scale[bt].shape + (1,) * (pages.dim() - 2))
        return x if scale is None else x * scale

    at = torch.arange(nb * b, device=DEV)
    inside = at < st["lens"][:, None]  # [S, T]
    seen = at <= first[:, None, None] + torch.arange(n, device=DEV)[:, None]  # [S, N, T]
    seen = (seen & inside[:, None]).repeat_interleave(g, dim=1)[:, None]  # [S, 1, N G, T]
    k = values(st["kc"], st["ks"]).permute(0, 2, 3, 5, 1, 4).reshape(seqs, hk, d, nb * b)
    q = query.view(seqs, n, hk, g, d).transpose(1, 2).reshape(seqs, hk, n * g, d)
    p = (q @ k).mul_(1.0 / math.sqrt(d)).masked_fill_(~seen, -math.inf)  # the logits
    del k
    m = p.amax(dim=3, keepdim=True)
    p = p.sub_(torch.where(m > -math.inf, m, 0.0)).exp_()
    v = values(st["vc"], st["vs"]).permute(0, 2, 1, 4, 3).reshape(seqs, hk, nb * b, d)
    v = torch.where(inside[:, None, :, None], v, 0.0)
    total = p.sum(dim=3, keepdim=True)
    o = (p @ v) / torch.where(total > 0, total, 1.0)
    return o.view(seqs, hk, n, g, d).transpose(1, 2).reshape(seqs, n, hq, d)


def _plain_decode(st):
    o = _plain_attention(st, st["query"].float()[:, None], st["lens"] - 1)
    st["out"].copy_(o[:, 0])


def _plain_prefill(st):
    t, seqs = st["query"].shape[0], st["bt"].shape[0]
    start = st["start"].long()
    s = torch.searchsorted(start[1:].contiguous(), torch.arange(t, device=DEV), right=True)
    n = torch.arange(t, device=DEV) - start[s]
    padded = torch.zeros((seqs, max(1, st["max_new"])) + st["query"].shape[1:], device=DEV)
    padded[s, n] = st["query"].float()
    o = _plain_attention(st, padded, st["lens"] - (start[1:] - start[:-1]))
    st["out"].copy_(o[s, n])


def _answer(st):
    if st["op"] != "append":
        return {"out": st["out"]}
    out = {"key_cache": st["kc"], "value_cache": st["vc"], "query": st["query_out"]}
    if st["kv"].endswith("_block"):
        out |= {"k_scale": st["ks"], "v_scale": st["vs"]}
    return out


def run(st):
    if own:
        import paged_kv_cache_471_b200 as pa
        if st["op"] == "append":
            pa.append_kv(st["kc"], st["vc"], st["key"], st["value"], st["bt"], st["lens"], st["b"],
                         st["kv"], st["ks"], st["vs"], query_start=st["start"],
                         cos_sin=st["angles"], interleaved=st["interleaved"], query=st["query"],
                         query_out=st["query_out"])
        elif st["op"] == "prefill":
            pa.prefill(st["out"], st["query"], st["kc"], st["vc"], st["hk"],
                       1.0 / math.sqrt(st["d"]), st["bt"], st["lens"], st["start"], st["b"],
                       st["max_len"], st["kv"], st["ks"], st["vs"])
        else:
            pa.decode(st["out"], st["query"], st["kc"], st["vc"], st["hk"],
                      1.0 / math.sqrt(st["d"]), st["bt"], st["lens"], st["b"], st["max_len"],
                      st["kv"], st["ks"], st["vs"], shared_prefix_blocks=st["prefix"])
    elif st["op"] == "append":
        _plain_append(st)
    elif st["op"] == "prefill":
        _plain_prefill(st)
    else:
        _plain_decode(st)
    return _answer(st)


# -------------------------------------------------------- the same in 64 bits
def _exact_rotate(x, pos, st):
    """One sequence's rows x [n, H, D] at positions pos, in 64 bits, by complex
    multiplication; the angles are the table's."""
    r = st["rot"]
    turn = torch.complex(st["angles"][pos, :r // 2].double(), st["angles"][pos, r // 2:].double())
    x = x.double()
    if st["interleaved"]:
        z = torch.view_as_complex(x[..., :r].unflatten(-1, (r // 2, 2)).contiguous())
        y = torch.view_as_real(z * turn[:, None]).flatten(-2)
    else:
        z = torch.complex(x[..., :r // 2], x[..., r // 2:r]) * turn[:, None]
        y = torch.cat([z.real, z.imag], dim=-1)
    return torch.cat([y, x[..., r:]], dim=-1)


def _exact_code(x, kv):
    """The nearest code's value, in 64 bits."""
    x = x.clamp(-QMAX[kv], QMAX[kv])
    return torch.round(x) if kv == "int8_block" else x.to(torch.float8_e4m3fn).double()


def _exact_append(c, seed):
    st = prepare(c, seed)
    kv, b, hk, d = c["kv"], c["b"], c["hk"], c["d"]
    new, past = _new_and_past(c)
    block = kv.endswith("_block")
    kc = st["kc"].permute(0, 1, 3, 2, 4).reshape(-1, hk, b, d).double()  # [pool, H, slot, D]
    vc = st["vc"].transpose(2, 3).double()
    q = torch.zeros(st["query"].shape, dtype=torch.float64, device=DEV)
    bt, row = st["bt"].tolist(), 0
    for s, (n, p0) in enumerate(zip(new, past)):
        pos = torch.arange(p0, p0 + n, device=DEV)
        rows = slice(row, row + n)
        row += n
        q[rows] = _exact_rotate(st["query"][rows], pos, st)
        k, v = _exact_rotate(st["key"][rows], pos, st), st["value"][rows].double()
        i = 0
        while i < n:  # one block at a time
            j = (p0 + i) // b
            lo = (p0 + i) % b
            m = min(n - i, b - lo)
            for pages, scale, x in ((kc, st["ks"], k), (vc, st["vs"], v)):
                tile = x[i:i + m].transpose(0, 1)  # [H, m, D]
                page = pages[bt[s][j]]
                if block:
                    a = tile.abs().amax(dim=(1, 2)) / QMAX[kv]
                    m2, e = torch.frexp(a)  # 2^(e - 1) <= a < 2^e, for a > 0
                    e = torch.where(a > 0, e - (m2 == 0.5).int(), MIN_EXP)
                    want = torch.exp2(e.double().clamp(MIN_EXP, MAX_EXP))
                    if lo:
                        old = scale[bt[s][j]].double()
                        want = torch.maximum(want, old)
                        page[:, :lo] = _exact_code(page[:, :lo] * (old / want)[:, None, None], kv)
                    scale[bt[s][j]] = want.float()
                    tile = _exact_code(tile / want[:, None, None], kv)
                elif kv == "fp8_e4m3":
                    tile = _exact_code(tile / scale.double(), kv)
                page[:, lo:lo + m] = tile
            i += m
    x = st["kc"].shape[4]
    kc = kc.view(-1, hk, b, d // x, x).transpose(2, 3).contiguous()
    vc = vc.transpose(2, 3).contiguous()
    whole = kv == "int8_block"  # whole numbers are compared with the plain form's
    out = {"key_cache": None if whole else kc, "value_cache": None if whole else vc, "query": q}
    if block:
        out |= {"k_scale": st["ks"].double(), "v_scale": st["vs"].double()}
    return out


def exact(c, seed):
    if c["op"] == "append":
        return _exact_append(c, seed)
    st = prepare(c, seed)
    hk, d, block = c["hk"], c["d"], c["kv"].endswith("_block")
    out = torch.zeros(st["query"].shape, dtype=torch.float64, device=DEV)
    if c["op"] == "prefill":
        new, past = _new_and_past(c)
    else:
        new, past = [1] * c["seqs"], [t - 1 for t in _decode_lens(c)]
    row = 0
    for s, (n, p0) in enumerate(zip(new, past)):
        rows, t = slice(row, row + n), n + p0
        row += n
        if not t or not n:
            continue
        ids = st["bt"][s, :-(-t // c["b"])].long()
        late = torch.arange(t, device=DEV)[:, None] > p0 + torch.arange(n, device=DEV)  # [t, n]
        for h in range(hk):
            k, v = st["kc"][:, h], st["vc"][:, h]
            if c["kv"] != "bf16":
                k, v = k.view(torch.uint8), v.view(torch.uint8)
            k = k[ids].view(st["kc"].dtype).double().transpose(1, 2).reshape(-1, d)[:t]
            v = v[ids].view(st["vc"].dtype).double().transpose(1, 2).reshape(-1, d)[:t]
            if block:
                k = k * st["ks"][ids, h].double().repeat_interleave(c["b"])[:t, None]
                v = v * st["vs"][ids, h].double().repeat_interleave(c["b"])[:t, None]
            elif c["kv"] != "bf16":
                k, v = k * st["ks"].double(), v * st["vs"].double()
            for j in range(h * (c["hq"] // hk), (h + 1) * (c["hq"] // hk)):
                z = k @ st["query"][rows, j].double().T / math.sqrt(d)  # [t, n]
                out[rows, j] = torch.softmax(z.masked_fill(late, -math.inf), dim=0).T @ v
    return {"out": out}
