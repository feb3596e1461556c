"""GPU parity of dspark_rope_append from one wave of blocks on, where a block takes two rows: every pair layout and item width,
odd numbers of rows. Tolerances as in test_gpu_cache.py."""
import numpy as np
import pytest
import torch

from oracle import tree
from tests.test_gpu_cache import TYPES, f64, paged

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,T,Hq,H,D,rot,page,inter,axes", [
    (611, 3, 2, 1, 64, 64, 16, False, 1),        # 1,833 rows, the last block with one
    (611, 3, 4, 2, 64, 64, 16, True, 3),         # interleaved, 16-byte items
    (1, 1825, 2, 2, 80, 40, 24, False, 2),       # 20 pairs: four at a time
    (609, 3, 2, 1, 40, 20, 16, True, 1),         # interleaved, 20 columns
    (611, 3, 3, 1, 72, 36, 5, False, 2),         # 18 pairs: one at a time
    (203, 9, 2, 1, 24, 6, 7, True, 3),           # interleaved, one at a time
    (1, 4001, 1, 1, 256, 256, 64, False, 1),     # the widest head
    (1831, 1, 2, 1, 128, 128, 16, False, 1)])    # a row a request
def test_two_rows_a_block(dtype, R, T, Hq, H, D, rot, page, inter, axes):
    import dspark_draft_selection_gb300 as ds
    assert R * T >= 12 * 152
    gen = torch.Generator().manual_seed(R + T + D)
    dt = TYPES[dtype]
    lens = torch.randint(0, 20, (R,), generator=gen).int()
    n = torch.randint(0, T + 1, (R,), generator=gen).int()
    n[0] = n[-1] = T
    table, kc, vc = paged(gen, R, 20 + T, page, H, D, dt, order="phtd" if D % 16 else "pthd")
    k0, v0 = kc.clone(), vc.clone()
    qkv = torch.randn((R, T, Hq + 2 * H, D), generator=gen).to(dt).cuda()
    q, k, v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + H], qkv[:, :, Hq + H:]
    P = 300
    ang = torch.arange(P).double()[:, None] * 50.0 ** (-torch.arange(rot // 2).double() / (rot // 2))
    cs = torch.cat([ang.cos(), ang.sin()], 1).float()
    pos = torch.randint(0, P, (R, T, axes), generator=gen).int()
    axis = torch.randint(0, axes, (rot // 2,), generator=gen).int()
    qo, st = ds.dspark_rope_append(q, k, v, pos.cuda(), cs.cuda(), kc, vc, table, lens.cuda(), axis=axis.cuda(), n_nodes=n.cuda(),
                                   interleaved=inter)
    assert ds.read_status(st) == 0
    f = torch.arange(rot // 2)
    at = pos.long()[:, :, axis.long()]
    c, s = (cs.double().numpy()[at, f + off][:, :, None] for off in (0, rot // 2))
    live = (torch.arange(T) < n[:, None]).numpy()

    def near(got, x):
        want, big = x.copy(), x.copy()
        a, b = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
        want[..., a], want[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
        big[..., a] = np.abs(x[..., a] * c) + np.abs(x[..., b] * s)
        big[..., b] = np.abs(x[..., b] * c) + np.abs(x[..., a] * s)
        tol = 3 * 2.0 ** -24 * np.abs(big) + (2.0 ** -8 if dtype == "bf16" else 0.0) * np.abs(want) * (1 + 2.0 ** -14)
        off = np.abs(got - want) <= tol
        assert off[live].all()

    near(f64(qo), f64(q))
    assert not f64(qo)[~live].any()
    one = tree.rope(f64(q)[0, 0], c[0, 0, 0], s[0, 0, 0], inter)             # the oracle's rotation is the one above
    np.testing.assert_allclose(f64(qo)[0, 0], one, rtol=2.0 ** -7, atol=1e-5)
    slot = (lens[:, None] + torch.arange(T)).long()
    pages, places = torch.gather(table.cpu().long(), 1, slot // page).cuda(), (slot % page).cuda()
    near(f64(kc[pages, places]), f64(k))
    assert torch.equal(vc[pages, places][torch.from_numpy(live).cuda()], v[torch.from_numpy(live).cuda()])
    there = torch.zeros(kc.shape[:2], dtype=torch.bool, device="cuda")
    there[pages[torch.from_numpy(live).cuda()], places[torch.from_numpy(live).cuda()]] = True
    assert torch.equal(kc[~there], k0[~there]) and torch.equal(vc[~there], v0[~there])   # nothing else was written
