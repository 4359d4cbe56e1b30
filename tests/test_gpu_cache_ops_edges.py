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


# ---------------------------------------------------------------- results of a call on a stream of its own
def calls():
    """name -> (call of a stream, giving the tensors it made)."""
    B, Hq, Hkv, N, keep = 2, 8, 2, 300, 40
    g = torch.Generator().manual_seed(91)
    q = torch.randn(21, Hq, 128, generator=g).to(torch.bfloat16).to(DEV)
    k = torch.randn(21, Hkv, 128, generator=g).to(torch.bfloat16).to(DEV)
    K, V = base.make_cache(92, B, Hkv, N, [N, N], 0), base.make_cache(93, B, Hkv, N, [N, N], 0)
    codes = adamas.encode_keys(K, torch.zeros(B, Hkv, N, 32, dtype=torch.uint8, device=DEV))
    mass = torch.rand(B, Hkv, N, generator=g).to(DEV)
    cu, lens, none = base.i32([0, 20, 21]), base.i32([N, 211]), base.i32([0, 0])
    freqs, _ = adamas.rope_frequencies()
    to = dict(K_out=K[:, :, :keep].clone(), V_out=V[:, :, :keep].clone(), mass_out=mass[:, :, :keep].clone())
    ws, dws, sws = adamas.ChunkWorkspace(21, B, Hq, Hkv), adamas.Workspace(B, Hq, Hkv, N, 32), adamas.Workspace(B, Hq, Hkv, N, 32, sharded=True)
    K2, V2, q1 = K.clone(), V.clone(), q[:2].contiguous()
    hist = adamas.shard_score(q1, codes, lens, 32, sws).unsqueeze(0)
    partial = adamas.shard_attend(q1, K, V, lens, 32, hist, 0, sws)[0].unsqueeze(0)
    return {
        "rope_append": lambda s: (adamas.rope_append(q, k, k, cu, none, K2, V2, freqs, ws, stream=s),),
        "chunk_attend": lambda s: adamas.chunk_attend(q, K, V, cu, lens, ws, stream=s),
        "evict": lambda s: adamas.evict(K, V, mass, lens, keep, ws, stream=s, **to),
        "decode": lambda s: adamas.decode(q1, codes, K, V, lens, 32, dws, stream=s),
        "decode_step": lambda s: adamas.decode_step(q1, codes, K, V, lens, 32, dws, stream=s),
        "score": lambda s: (adamas.score(q1, codes, lens, stream=s),),
        "shard_score": lambda s: (adamas.shard_score(q1, codes, lens, 32, sws, stream=s),),
        "shard_attend": lambda s: (adamas.shard_score(q1, codes, lens, 32, sws, stream=s), *adamas.shard_attend(q1, K, V, lens, 32, hist, 0, sws, stream=s)),
        "merge_partials": lambda s: (adamas.merge_partials(partial, stream=s),),
        "workspace": lambda s: (adamas.ChunkWorkspace(21, B, Hq, Hkv, stream=s).buffer, adamas.Workspace(B, Hq, Hkv, N, 32, stream=s).buffer),
    }


@pytest.mark.parametrize("name", ["rope_append", "chunk_attend", "evict", "decode", "decode_step", "score", "shard_score",
                                  "shard_attend", "merge_partials", "workspace"])
def test_results_belong_to_the_stream_of_the_call(name):
    """What a call makes for its results must not wait for the current stream: neither is it
    filled there behind the call, nor is it memory that work queued there still writes to."""
    call = calls()[name]
    want = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    blocks = [torch.empty_like(t) for t in want for _ in range(8)]
    torch.cuda._sleep(200000000)                     # a tenth of a second of the current stream
    for x in blocks:
        x.view(torch.uint8).fill_(0x55)
    del blocks, x                                    # given back: to the current stream's next tensors
    got = call(side)
    torch.cuda.synchronize()
    assert all(base.same(a, b) for a, b in zip(got, want, strict=True))


# ---------------------------------------------------------------- offsets that are no offsets
@pytest.mark.parametrize("T,cu", [(3, [0, 4]), (3, [-1, 2]), (3, [2, 1]), (3, [5, 3]), (3, [0, 1, 0]), (3, [0, 0, 7, 7]),
                                  (3, [2, 2, 1, 2]), (600, [600] * 200 + [599] + [600] * 300)])
def test_bad_offsets_are_flagged_by_every_call(T, cu):
    B = len(cu) - 1
    q = torch.randn(T, 2, 128, generator=torch.Generator().manual_seed(95)).to(torch.bfloat16).to(DEV)
    K = torch.zeros(B, 2, 8, 128, dtype=torch.bfloat16, device=DEV)
    ws, lens = adamas.ChunkWorkspace(T, B, 2, 2), base.i32([8] * B)
    lse, mass = torch.zeros(T, 2, device=DEV), torch.zeros(B, 2, 8, device=DEV)
    freqs, _ = adamas.rope_frequencies()
    for call in (lambda: adamas.rope_append(q, None, None, base.i32(cu), lens, K, K, freqs, ws),
                 lambda: adamas.rope_append(None, q, q, base.i32(cu), lens, K, K, freqs, ws),
                 lambda: adamas.chunk_attend(q, K, K, base.i32(cu), lens, ws),
                 lambda: adamas.accumulate_chunk(q, K, lse, base.i32(cu), lens, mass, ws)):
        call()
        assert ws.device_error() == adamas.DEVERR_OFFSETS
        ws.reset()


def test_good_offsets_are_not_flagged():
    q = torch.randn(4, 2, 128, generator=torch.Generator().manual_seed(96)).to(torch.bfloat16).to(DEV)
    K = torch.zeros(3, 2, 8, 128, dtype=torch.bfloat16, device=DEV)
    ws, freqs = adamas.ChunkWorkspace(4, 3, 2, 2), adamas.rope_frequencies()[0]
    for cu in ([0, 0, 0, 0], [4, 4, 4, 4], [1, 2, 2, 3], [0, 4, 4, 4]):
        adamas.rope_append(q, q, q, base.i32(cu), base.i32([1, 2, 3]), K, K.clone(), freqs, ws)
        assert ws.device_error() == 0


# ---------------------------------------------------------------- one token that is part of a projection's row
@pytest.mark.parametrize("rot,inter", [(128, False), (128, True), (6, False)])
def test_one_token_is_rotated_in_place_in_its_projection(rot, inter):
    Hq, Hkv = 4, 2
    row = torch.randn(1, Hq + 2 * Hkv, 128, generator=torch.Generator().manual_seed(97)).to(torch.bfloat16).to(DEV)
    q, k, v = row.split([Hq, Hkv, Hkv], 1)
    assert q.stride(0) == row.stride(0)
    K, V = (torch.zeros(1, Hkv, 9, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    ws, freqs = adamas.ChunkWorkspace(1, 1, Hq, Hkv), adamas.rope_frequencies(rot)[0]
    cu, before = base.i32([0, 1]), base.i32([5])
    want = adamas.rope_append(q, k, v, cu, before, K, V, freqs, ws, interleaved=inter)
    K2, V2, rest = torch.zeros_like(K), torch.zeros_like(V), row[:, Hq:].clone()
    assert adamas.rope_append(q, k, v, cu, before, K2, V2, freqs, ws, interleaved=inter, out=q) is q
    assert base.same(row[:, :Hq], want) and base.same(row[:, Hq:], rest)
    assert base.same(K, K2) and base.same(V, V2) and ws.device_error() == 0


# ---------------------------------------------------------------- a workspace that is somewhere else
def test_a_workspace_of_another_device_is_refused():
    class Elsewhere:
        buffer, nbytes = torch.zeros(1 << 20, dtype=torch.uint8), 1 << 20

    q = torch.zeros(1, 2, 128, dtype=torch.bfloat16, device=DEV)
    K = torch.zeros(1, 2, 8, 128, dtype=torch.bfloat16, device=DEV)
    lens, cu, mass, ws = base.i32([8]), base.i32([0, 1]), torch.zeros(1, 2, 8, device=DEV), Elsewhere()
    for call in (lambda: adamas.rope_append(q, q, q, cu, base.i32([0]), K, K, adamas.rope_frequencies()[0], ws),
                 lambda: adamas.chunk_attend(q, K, K, cu, lens, ws),
                 lambda: adamas.accumulate_chunk(q, K, torch.zeros(1, 2, device=DEV), cu, lens, mass, ws),
                 lambda: adamas.accumulate_kept(q, K, torch.zeros(1, 2, 4, dtype=torch.int32, device=DEV), lens, mass, ws),
                 lambda: adamas.evict(K, K.clone(), mass, lens, 4, ws)):
        with pytest.raises(ValueError, match="workspace"):
            call()


def test_a_captured_run_over_two_streams():
    """Part of a captured run goes to a second stream that the first one forks to and joins;
    its results are of the graph's memory like the others."""
    call = calls()["chunk_attend"]
    want = [t.clone() for t in call(None)]
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        side.wait_stream(main)
        got = call(side)
        main.wait_stream(side)
        twice = [t + t for t in got]
    for _ in range(2):
        for t in (*got, *twice):
            t.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(base.same(a, b) and base.same(a + a, c) for a, b, c in zip(want, got, twice, strict=True))
