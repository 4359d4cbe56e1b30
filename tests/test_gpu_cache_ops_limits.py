"""Cache operators at the limits of what they take: every group size, the largest batch,
odd and large pages, calls at once on two streams, calls one after the other without a
wait, the largest positions."""
import numpy as np
import pytest
import torch

import cache_oracle as co
import test_gpu_cache_ops as base
from compressed_sparse_kv_fp32_b200 import adamas

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("G", range(1, 9))
def test_every_group_size(G):
    base.test_chunk_attend_and_its_weights(3 * G, 3, [70, 1, 150], [200, 300, 333], 352, 32, 0, 0)


@pytest.mark.parametrize("page", [2, 4, 12, 40, 2048])
def test_pages_of_any_size(page):
    base.test_chunk_attend_and_its_weights(8, 2, [40, 130], [700, 500], 720, page, 0, 0)


def test_largest_batch():
    n = 1024
    base.test_chunk_attend_and_its_weights(4, 1, [1] * n, [1 + (i * 37) % 150 for i in range(n)], 160, 16, 0, 0)
    base.test_chunk_attend_and_its_weights(6, 2, [i % 4 for i in range(n)], [3 + (i * 53) % 130 for i in range(n)], 136, 0, 0, 1)


# chunks of up to two tiles of rows, whose units are placed by what they cost: heads of one
# unit, of many, sequences without rows or tokens between them
@pytest.mark.parametrize("Hq,Hkv,ns,lens", [
    (4, 1, [64], [9000]),
    (20, 5, [1, 0, 64, 33, 0, 17], [2000, 900, 255, 257, 0, 4000]),
    (8, 8, [256, 1, 0, 128, 129, 200], [256, 5000, 10, 1, 2500, 700]),
    (32, 4, [0, 0, 32, 0], [4000, 0, 3000, 700]),
    (3, 3, [0], [500]),
])
def test_weights_of_unequal_heads(Hq, Hkv, ns, lens):
    base.test_chunk_attend_and_its_weights(Hq, Hkv, ns, lens, max(lens), 0, 0, 0)


@pytest.mark.parametrize("Hkv", [1, 5])
@pytest.mark.parametrize("N,keep", [(5, 3), (2047, 1000), (2049, 2048), (16385, 5000), (70000, 69999)])
def test_eviction_in_place_is_the_one_to_another_cache(N, keep, Hkv):
    g = torch.Generator().manual_seed(N)
    K, V = (torch.randn(2, Hkv, N, 128, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    C = torch.randint(0, 256, (2, Hkv, N, 32), generator=g, dtype=torch.uint8).to(DEV)
    mass = torch.randint(0, 50, (2, Hkv, N), generator=g).float().to(DEV)
    lens = base.i32([N, max(1, N - 3)])
    ws = adamas.ChunkWorkspace(1, 2, Hkv, Hkv)
    to = dict(K_out=torch.zeros_like(K[:, :, :keep]), V_out=torch.zeros_like(V[:, :, :keep]),
              codes_out=torch.zeros_like(C[:, :, :keep]), mass_out=torch.ones_like(mass[:, :, :keep]))
    to = {k: v.contiguous() for k, v in to.items()}
    k1, l1 = adamas.evict(K, V, mass, lens, keep, ws, codes=C, n_sink=1, n_recent=2, **to)
    k2, l2 = adamas.evict(K, V, mass, lens, keep, ws, codes=C, n_sink=1, n_recent=2)
    assert torch.equal(k1, k2) and torch.equal(l1, l2) and l1.tolist() == [keep, min(keep, max(1, N - 3))]
    for b in range(2):
        n = int(l1[b])
        for x, y in zip((K, V, C, mass), to.values()):
            assert base.same(x[b, :, :n], y[b, :, :n])
        assert not mass[b, :, n:].any() and not to["mass_out"][b, :, n:].any()


@pytest.mark.parametrize("in_place", [False, True])
def test_evictions_one_after_the_other(in_place):
    """The second kernel of a call uses this call's selection, whatever the buffers held."""
    g = torch.Generator().manual_seed(3)
    N, keep = 20000, 700
    K = torch.randn(1, 4, N, 128, generator=g).to(torch.bfloat16).to(DEV)
    V = torch.randn(1, 4, N, 128, generator=g).to(torch.bfloat16).to(DEV)
    masses = [torch.rand(1, 4, N, generator=g).to(DEV) for _ in range(2)]
    ws, lens = adamas.ChunkWorkspace(1, 1, 4, 4), base.i32([N])
    kept = torch.full((1, 4, keep), 3, dtype=torch.int32, device=DEV)
    Ko, Vo = (torch.zeros(1, 4, keep, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    mo = torch.zeros(1, 4, keep, device=DEV)
    got = []
    for i in range(20):
        m = masses[i % 2]
        if in_place:
            Ko, Vo, mo = K.clone(), V.clone(), m.clone()
            adamas.evict(Ko, Vo, mo, lens, keep, ws, kept=kept)
        else:
            adamas.evict(K, V, m, lens, keep, ws, kept=kept, K_out=Ko, V_out=Vo, mass_out=mo)
        got.append([x[:, :, :keep].clone() for x in (Ko, Vo, mo)] + [kept.clone()])
    for i, (k, v, m, at) in enumerate(got):
        want, _ = co.evict_select(masses[i % 2].cpu().numpy(), [N], keep, 0, 0)
        assert np.array_equal(at.cpu().numpy(), want)
        j = at.long()
        assert base.same(m, masses[i % 2].gather(2, j))
        j = j[..., None].expand(-1, -1, -1, 128)
        assert base.same(k, K.gather(2, j)) and base.same(v, V.gather(2, j))


def test_two_streams_at_once():
    """Calls with workspaces of their own at the same time give the bits of calls alone."""
    lens, ns = [900, 700, 650, 300], [50, 1, 200, 3]
    calls = []
    for seed in (5, 6):
        g = torch.Generator().manual_seed(seed)
        q = torch.randn(sum(ns), 16, 128, generator=g).to(torch.bfloat16).to(DEV)
        K = base.make_cache(seed, 4, 4, 960, lens, 16, gain=2.0)
        V = base.make_cache(seed + 1, 4, 4, 960, lens, 16, table_seed=seed)
        table = base.tab(base.make_table(seed, 4, 960, 16))
        ws = adamas.ChunkWorkspace(sum(ns), 4, 16, 4)
        a = (q, K, V, base.i32(base.offsets(ns)), base.i32(lens), ws)
        calls.append((a, table, adamas.chunk_attend(*a, block_table=table)))
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(20):
        new = []
        for (a, table, (out, lse)), st in zip(calls, streams):
            o, z = torch.zeros_like(out), torch.zeros_like(lse)
            st.wait_stream(torch.cuda.current_stream())
            adamas.chunk_attend(*a, block_table=table, out=o, lse=z, stream=st)
            new.append((o, z))
        torch.cuda.synchronize()
        for (_, _, (out, lse)), (o, z) in zip(calls, new):
            assert base.same(o, out) and base.same(z, lse)


def test_largest_positions():
    k = torch.randn(4, 2, 128, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16)
    K = torch.zeros(1, 2, 8, 128, dtype=torch.bfloat16, device=DEV)
    V = torch.zeros_like(K)
    freqs, _ = adamas.rope_frequencies()
    positions = [-2**31, 2**31 - 1, -1, 0]
    ws = adamas.ChunkWorkspace(4, 1, 2, 2)
    adamas.rope_append(None, k.to(DEV), k.to(DEV), base.i32([0, 4]), base.i32([0]), K, V, freqs, ws, positions=base.i32(positions))
    turns = freqs.cpu().numpy().view(np.uint64)
    for i, p in enumerate(positions):
        want = co.rotate(k[i].float().numpy(), p, turns, 128, False, 1.0)
        assert base.same(K[0, :, i].cpu(), torch.from_numpy(want).to(torch.bfloat16))
