"""Calls of the cache operators that their documentation allows and that once went wrong:
capacities far above the lengths, sequences without tokens between others, streams."""
import numpy as np
import pytest
import torch

import cache_oracle as co
import test_gpu_cache_ops as base
from compressed_sparse_kv_fp32_b200 import adamas

pytestmark = pytest.mark.gpu
DEV = "cuda"


# ---------------------------------------------------------------- eviction: the capacity is no bound on the lengths
@pytest.mark.parametrize("to", [None, 0])
def test_evict_of_short_sequences_in_a_large_cache(to):
    """More than 8 x 40,960 slots, where the keys of a full sequence do not stay in shared
    memory and those of the short ones beside it do."""
    base.test_evict(1, [330000, 5000, 0], 330000, 700, 4, 64, 0, to, False, True)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("lens", [[5000, 300, 0], [4096, 5120, 1]])
def test_evict_behind_a_wide_block_table(lens, in_place):
    """A block table of 480,000 slots per sequence whose entries are there for the tokens
    there are."""
    B, Hkv, page, per, keep = len(lens), 2, 16, 30000, 400
    g = torch.Generator().manual_seed(81)
    used = [-(-n // page) for n in lens]
    order = torch.randperm(sum(used), generator=g).to(torch.int32)
    table = torch.full((B, per), -1, dtype=torch.int32)
    for b, n in enumerate(used):
        table[b, :n] = order[sum(used[:b]):sum(used[:b + 1])]
    K, V = (torch.randn(sum(used), Hkv, page, 128, generator=g).to(torch.bfloat16) for _ in range(2))
    m = base.masses(82, B, Hkv, per * page, True)
    dK, dV, dm = K.to(DEV), V.to(DEV), torch.from_numpy(m.copy()).to(DEV)
    dst = {}
    if not in_place:
        dst = dict(K_out=torch.zeros(B, Hkv, keep, 128, dtype=torch.bfloat16, device=DEV), mass_out=torch.ones(B, Hkv, keep, device=DEV))
        dst["V_out"] = torch.zeros_like(dst["K_out"])
    ws = adamas.ChunkWorkspace(1, B, Hkv, Hkv)
    kept, new_lens = adamas.evict(dK, dV, dm, base.i32(lens), keep, ws, n_sink=2, n_recent=8, block_table=table.to(DEV), **dst)
    assert ws.device_error() == 0
    want, wlens = co.evict_select(m, np.asarray(lens), keep, 2, 8)
    assert np.array_equal(kept.cpu().numpy(), want) and np.array_equal(new_lens.cpu().numpy(), wlens)
    t = table.long()
    for b in range(B):
        j = np.arange(wlens[b])
        for h in range(Hkv):
            src = want[b, h, j].astype(np.int64)
            for old, here, there in ((K, dK, dst.get("K_out")), (V, dV, dst.get("V_out"))):
                got = here.cpu()[t[b][j // page], h, j % page] if in_place else there.cpu()[b, h, j]
                assert base.same(got, old[t[b][src // page], h, src % page])
            mass = (dm if in_place else dst["mass_out"])[b, h].cpu().numpy()
            assert np.array_equal(mass[j].view(np.uint32), m[b, h, src].view(np.uint32)) and not mass[len(j):].any()


# ---------------------------------------------------------------- attention: tiles that end inside, one after the other
@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("lens", [
    [0],                                      # rows that see nothing: tiles without a single copied row
    [0, 5, 0, 0, 130, 0, 64, 1],
    [1, 127, 100],
    [129, 0, 255, 256, 0, 7],
])
def test_many_units_that_end_inside_a_tile(lens, page):
    """Every block goes through a dozen units whose V tiles all have rows to be zeroed, many
    of them without a row to be copied."""
    n = 500
    base.test_chunk_attend_and_its_weights(8, 4, [1 + (i * 7) % 3 for i in range(n)], [lens[i % len(lens)] for i in range(n)], 256,
                                           page, 0, 0)


def test_units_without_tokens_between_longer_ones():
    ns = [40, 200, 1, 70, 3] * 20
    lens = [0, 150, 0, 30, 512] * 20
    base.test_chunk_attend_and_its_weights(6, 2, ns, lens, 512, 16, 1, 2)
