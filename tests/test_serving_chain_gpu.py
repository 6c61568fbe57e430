"""The cache's operators as a server uses them (GPU): prompts are appended and
attended, sequences fork with copy on write, single tokens are appended and
decoded, all over block-manager tables and through one cache; every output is
compared with attention over the reference cache in fp64."""

import pytest
import torch

import paged_kv_cache_471_b200 as pa
from kv_reference import FORMATS, Cache, angle_table, attention, is_block

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("D,B", [(128, 16), (64, 32)])
@pytest.mark.parametrize("kv", FORMATS)
def test_prompts_forks_and_steps(kv, D, B):
    Hk, G, NB, MAXB = 2, 4, 90, 12
    Hq, scale = Hk * G, D ** -0.5
    bm = pa.BlockManager(NB, B, MAXB)
    ref = Cache(kv, [], Hk, D, B, spare=NB, max_blocks=MAXB)
    kc, vc = ref.packed(DEV)
    ks, vs = ref.scales(DEV)
    angles = angle_table(MAXB * B, D)
    table = angles.to(DEV)
    g = torch.Generator().manual_seed(1)
    pa.read_status(device=DEV, clear=True)

    def rows(n):
        qkv = torch.randn((n, Hq + 2 * Hk, D), generator=g).to(torch.bfloat16)
        d = qkv.to(DEV)
        return qkv, d[:, :Hq], d[:, Hq:Hq + Hk], d[:, Hq + Hk:]

    def step(seqs, new):
        """Grow seqs by new tokens each, append, attend; check every row."""
        copies = []
        for s, n in zip(seqs, new):
            cow = bm.append(s, n)
            if cow:
                copies.append(cow)
        if copies:
            src, dst = (torch.tensor(x) for x in zip(*copies))
            pa.copy_blocks(kc, vc, src.to(DEV), dst.to(DEV), kv, k_scale=ks, v_scale=vs)
            for t in (ref.k, ref.v):
                ref._raw(t)[dst] = ref._raw(t)[src]
            if is_block(kv):
                ref.ks[dst], ref.vs[dst] = ref.ks[src], ref.vs[src]
        bt, sl = (torch.from_numpy(x) for x in bm.export(seqs))
        host, q, k, v = rows(sum(new))
        start = torch.tensor([0] + list(torch.tensor(new).cumsum(0)), dtype=torch.int32)
        single = all(n == 1 for n in new)
        qr = torch.empty((sum(new), Hq, D), dtype=torch.bfloat16, device=DEV)
        bt_d, sl_d, start_d = bt.to(DEV), sl.to(DEV), start.to(DEV)
        pa.append_kv(kc, vc, k, v, bt_d, sl_d, B, kv, ks, vs,
                     query_start=None if single else start_d, cos_sin=table, query=q,
                     query_out=qr)
        out = torch.empty_like(qr)
        if single:
            pa.decode(out, qr, kc, vc, Hk, scale, bt_d, sl_d, B, MAXB * B, kv, ks, vs)
        else:
            pa.prefill(out, qr, kc, vc, Hk, scale, bt_d, sl_d, start_d, B, MAXB * B, kv, ks, vs)
        torch.cuda.synchronize()
        ref.tables, ref.lens = bt, sl
        want_q = ref.append(host[:, Hq:Hq + Hk], host[:, Hq + Hk:], start, angles,
                            query=host[:, :Hq], dtype=torch.float32).to(torch.bfloat16)
        assert torch.equal(qr.cpu(), want_q)
        o, tol = attention(ref, want_q, start, scale)
        err = (out.cpu().double() - o).abs()
        # Decode over bf16 pages also rounds the sum's weights: twice u A.
        assert (err <= 2 * tol).all(), float((err / tol).max())
        if single and not is_block(kv):
            return
        assert (err <= tol).all(), float((err / tol).max())

    prompts = [bm.add_sequence() for _ in range(3)]
    step(prompts, [70, 1, 33])               # three prompts
    step(prompts, [5, 40, 2])                # chunks behind them
    step(prompts, [1, 1, 1])                 # a decode step
    kids = [bm.fork(prompts[0]) for _ in range(2)]
    for i in range(4):                       # forks diverge: copy on write
        step(kids + prompts, [1] * 5)
    step([kids[1], prompts[2]], [20, 1])     # a chunk and a single token together
    bm.free(prompts[0])
    fresh = bm.add_sequence()                # blocks are reused without clearing
    step([fresh, kids[0]], [60, 3])
    step([fresh, kids[0]], [1, 1])
    assert pa.read_status(device=DEV) == 0
