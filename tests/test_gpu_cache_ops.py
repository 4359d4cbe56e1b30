"""Cache operators on the GPU against their 64-bit definitions (cache_oracle.py).

Rotated rows and codes are equal bit for bit; attention, its log-sum-exp and the
accumulated weights lie within bounds counted from the roundings on the way; kept
tokens and moved rows are equal.  Everything that no sequence owns -- padded rows,
other pages, slots past a length -- holds NaN or a pattern and must stay as it was."""
import numpy as np
import pytest
import torch

import cache_oracle as co
from compressed_sparse_kv_fp32_b200 import adamas
from helpers import assert_close_out

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32).to(DEV)


def f64(t):
    return t.double().cpu().numpy()


def offsets(ns, lead=0):
    return np.cumsum([lead] + list(ns)).tolist()


def make_cache(seed, B, Hkv, N, lens, page, gain=1.0, fill=float("nan"), table_seed=None):
    """bf16 rows of B sequences; rows past each length and unused pages hold `fill`."""
    g = torch.Generator().manual_seed(seed)
    x = torch.full((B, Hkv, N, 128), fill, dtype=torch.bfloat16)
    for b, L in enumerate(lens):
        L = min(max(L, 0), N)
        x[b, :, :L] = (torch.randn(Hkv, L, 128, generator=g) * gain).to(torch.bfloat16)
    return to_pages(x, make_table(seed if table_seed is None else table_seed, B, N, page), page, fill)


def make_table(seed, B, N, page, spare=2):
    if not page:
        return None
    per = -(-N // page)
    perm = torch.randperm(B * per + spare, generator=torch.Generator().manual_seed(seed + 7))[: B * per]
    return perm.to(torch.int32).view(B, per)


def to_pages(x, table, page, fill, spare=2):
    if table is None:
        return x.to(DEV)
    B, H, N, w = x.shape
    per = table.shape[1]
    pad = torch.full((B, H, per * page, w), fill).to(x.dtype)
    pad[:, :, :N] = x
    out = torch.full((B * per + spare, H, page, w), fill).to(x.dtype)
    out[table.long()] = pad.view(B, H, per, page, w).transpose(1, 2)
    return out.to(DEV)


def tab(t):
    return None if t is None else t.to(DEV)


def npt(t):
    return None if t is None else t.numpy()


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# ---------------------------------------------------------------- rotary append
ROPE = [
    # Hq, Hkv, new tokens, cached before, N, page, rot, interleaved, scaling, far, lead, tail
    (1, 1, [1], [0], 1, 0, 128, False, None, 0, 0, 0),
    (8, 8, [1, 1, 1], [5, 0, 39], 40, 0, 128, False, "yarn", 1000000, 0, 0),
    (8, 2, [3, 0, 17, 1], [5, 3, 0, 30], 40, 16, 64, True, "linear", 131072, 2, 3),
    (6, 2, [40, 7], [0, 1], 41, 1, 96, False, "ntk", 0, 0, 1),
    (15, 3, [9, 5], [11, 0], 21, 7, 6, False, None, -5, 1, 0),       # pairs that no two lanes hold alone
    (7, 1, [4, 4], [20, 0], 24, 24, 2, False, None, 2 ** 31 - 40, 0, 0),
    (8, 1, [5, 2], [0, 3], 6, 0, 0, True, None, 0, 0, 0),            # nothing rotated
    (4, 4, [6, 2], [-2, 5], 6, 0, 128, True, None, 0, 0, 0),         # slots before 0 and past Nmax are not written
    (4, 4, [300, 211], [0, 100], 320, 16, 128, False, None, 0, 0, 0),
]


@pytest.mark.parametrize("spaced", [False, True])
@pytest.mark.parametrize("Hq,Hkv,ns,before,N,page,rot,inter,scaling,far,lead,tail", ROPE)
def test_rope_append(Hq, Hkv, ns, before, N, page, rot, inter, scaling, far, lead, tail, spaced, orc):
    B, cu = len(ns), offsets(ns, lead)
    T = cu[-1] + tail
    g = torch.Generator().manual_seed(3)
    qkv = torch.randn(T, (Hq + 2 * Hkv) * 128 + (24 if spaced else 0), generator=g).to(torch.bfloat16)
    qkv[:lead], qkv[cu[-1]:] = float("nan"), float("nan")
    dq = qkv.to(DEV)
    parts = [dq[:, a * 128:(a + n) * 128].unflatten(1, (n, 128)) for a, n in ((0, Hq), (Hq, Hkv), (Hq + Hkv, Hkv))]
    if not spaced:
        parts = [x.contiguous() for x in parts]
    K, V = make_cache(1, B, Hkv, N, before, page), make_cache(2, B, Hkv, N, before, page, table_seed=1)
    table = make_table(1, B, N, page)
    codes = torch.full(K.shape[:-1] + (32,), 0x5A, dtype=torch.uint8, device=DEV)
    K0, V0, c0 = K.cpu(), V.cpu(), codes.cpu()
    freqs, mscale = adamas.rope_frequencies(rot, scaling=scaling, factor=8.0 if scaling else 1.0)
    pos = np.concatenate([np.zeros(lead, int)] + [np.arange(s, s + n) + far for s, n in zip(before, ns)] + [np.zeros(tail, int)])
    out = torch.full((T, Hq, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = adamas.ChunkWorkspace(T, B, Hq, Hkv)
    adamas.rope_append(*parts, i32(cu), i32(before), K, V, freqs, ws, positions=i32(pos), interleaved=inter,
                       mscale=mscale, codes=codes, block_table=tab(table), out=out)
    assert ws.device_error() == 0

    x = qkv[:, :(Hq + 2 * Hkv) * 128].float().numpy().reshape(T, -1, 128)
    f = freqs.cpu().numpy().view(np.uint64)
    want_q = torch.full((T, Hq, 128), 7.0, dtype=torch.bfloat16)
    wK, wV, wc = K0.clone(), V0.clone(), c0.clone()
    for b in range(B):
        for i in range(ns[b]):
            r, t = cu[b] + i, before[b] + i
            y = torch.from_numpy(co.rotate(x[r, : Hq + Hkv], int(pos[r]), f, rot, inter, mscale)).to(torch.bfloat16)
            want_q[r] = y[:Hq]
            if not 0 <= t < (N if table is None else table.shape[1] * page):
                continue
            at = (b, slice(None), t) if table is None else (int(table[b, t // page]), slice(None), t % page)
            wK[at], wV[at] = y[Hq:], torch.from_numpy(x[r, Hq + Hkv:]).to(torch.bfloat16)
            k16 = y[Hq:].view(torch.int16).numpy().view(np.uint16).reshape(1, Hkv, 1, 128)
            wc[at] = torch.from_numpy(orc.encode(k16)[0, :, 0])
    assert same(out.cpu(), want_q)
    assert same(K.cpu(), wK) and same(V.cpu(), wV) and same(codes.cpu(), wc)


def test_rope_parts_of_a_call(orc):
    g = torch.Generator().manual_seed(5)
    q = torch.randn(4, 8, 128, generator=g).to(torch.bfloat16).to(DEV)
    k, v = q[:, :2].contiguous(), q[:, 2:4].contiguous()
    K, V = torch.zeros(1, 2, 9, 128, dtype=torch.bfloat16, device=DEV), torch.zeros(1, 2, 9, 128, dtype=torch.bfloat16, device=DEV)
    freqs, _ = adamas.rope_frequencies()
    ws = adamas.ChunkWorkspace(4, 1, 8, 2)
    cu, before = i32([0, 4]), i32([3])
    full = adamas.rope_append(q, k, v, cu, before, K, V, freqs, ws)          # positions: the slots
    pos = i32([3, 4, 5, 6])
    assert same(full, adamas.rope_append(q, None, None, cu, before, K, V, freqs, ws, positions=pos))
    K2, V2 = torch.zeros_like(K), torch.zeros_like(V)
    assert adamas.rope_append(None, k, v, cu, before, K2, V2, freqs, ws, positions=pos) is None
    assert same(K, K2) and same(V, V2) and not K[:, :, :3].any() and not K[:, :, 7:].any()
    inplace = q.clone()
    assert adamas.rope_append(inplace, None, None, cu, before, K, V, freqs, ws, out=inplace) is inplace
    assert same(inplace, full)
    three, _ = adamas.rope_frequencies(6)                                     # the row is read twice: in place too
    a = adamas.rope_append(q, None, None, cu, before, K, V, three, ws)
    inplace = q.clone()
    adamas.rope_append(inplace, None, None, cu, before, K, V, three, ws, out=inplace)
    assert same(inplace, a)


def test_rope_flags_bad_pages_and_offsets():
    k = torch.ones(3, 1, 128, dtype=torch.bfloat16, device=DEV)
    K, V = torch.zeros(2, 1, 4, 128, dtype=torch.bfloat16, device=DEV), torch.zeros(2, 1, 4, 128, dtype=torch.bfloat16, device=DEV)
    freqs, _ = adamas.rope_frequencies()
    ws = adamas.ChunkWorkspace(3, 1, 1, 1)
    for entry in (-1, 2, 2 ** 31 - 1):
        adamas.rope_append(None, k, k, i32([0, 3]), i32([3]), K, V, freqs, ws, block_table=i32([[1, entry]]))
        assert ws.device_error() == adamas.DEVERR_TABLE
        assert not K[0].any() and not K[1, :, :3].any() and K[1, 0, 3].any()      # the good page's token alone
        K.zero_(), ws.reset()
    for cu in ([0, 4], [-1, 2], [2, 1]):
        out = adamas.rope_append(k, k, k, i32(cu), i32([0]), K[:1], V[:1], freqs, ws)
        assert ws.device_error() in (0, adamas.DEVERR_OFFSETS) and not K.any() and not out.any()
        ws.reset()


# ---------------------------------------------------------------- attention of a chunk
ATTEND = [
    # Hq, Hkv, new, lens, N, page, lead, tail
    (1, 1, [1], [1], 1, 0, 0, 0),
    (4, 4, [1, 1, 1], [1, 130, 77], 130, 0, 0, 0),
    (8, 1, [1, 2, 0, 1], [300, 129, 50, 0], 300, 16, 0, 0),       # an absent sequence, an empty one
    (6, 2, [17, 5, 33], [17, 100, 128], 128, 48, 1, 4),           # prompts from their first token; pages that end inside a tile
    (5, 1, [130], [131], 140, 1, 0, 0),
    (7, 1, [3, 4], [2, 3], 5, 24, 0, 0),                          # rows whose slots are negative see nothing
    (3, 3, [64, 200], [64, 333], 333, 64, 0, 3),
    (16, 2, [40], [1000], 1000, 256, 0, 0),
    (2, 2, [257], [513], 513, 0, 0, 0),
    (24, 8, [1, 9, 2], [700, 350, 512], 704, 16, 0, 0),
    (8, 2, [300, 1], [2000, 2300], 2304, 16, 0, 0),
    # many short sequences: blocks go from head to head, with one to three units of each
    (8, 8, [1 + i % 3 for i in range(60)], [1 + (i * 397) % 760 for i in range(60)], 768, 16, 0, 0),
    (16, 8, [1 + (i * 7) % 150 for i in range(24)], [150 + (i * 397) % 600 for i in range(24)], 768, 0, 0, 2),
    (8, 1, [32, 33, 1, 64, 65] * 8, [600, 70, 300, 520, 257] * 8, 640, 32, 0, 0),
]


@pytest.mark.parametrize("Hq,Hkv,ns,lens,N,page,lead,tail", ATTEND)
def test_chunk_attend_and_its_weights(Hq, Hkv, ns, lens, N, page, lead, tail):
    B, cu = len(ns), offsets(ns, lead)
    T = cu[-1] + tail
    q = torch.randn(T, Hq, 128, generator=torch.Generator().manual_seed(11)).to(torch.bfloat16)
    q[:lead], q[cu[-1]:] = float("nan"), float("nan")
    q = q.to(DEV)
    K = make_cache(12, B, Hkv, N, lens, page, gain=2.0)
    V = make_cache(13, B, Hkv, N, lens, page, table_seed=12)
    table = make_table(12, B, N, page)
    ws = adamas.ChunkWorkspace(T, B, Hq, Hkv)
    out = torch.full((T, Hq, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((T, Hq), 7.0, device=DEV)
    cud, ld = i32(cu), i32(lens)
    adamas.chunk_attend(q, K, V, cud, ld, ws, block_table=tab(table), out=out, lse=lse)
    assert ws.device_error() == 0
    want, wlse, tol, ltol = co.attend(f64(q), f64(K), f64(V), cu, lens, npt(table))
    mine = slice(cu[0], cu[-1])
    o, z = f64(out), f64(lse)
    assert (o[:lead] == 7).all() and (o[cu[-1]:] == 7).all() and (z[:lead] == 7).all() and (z[cu[-1]:] == 7).all()
    assert (np.abs(o - want)[mine] <= tol[mine]).all()
    seen = np.isfinite(wlse)
    assert np.array_equal(z[mine][~seen[mine]], wlse[mine][~seen[mine]])
    seen[:cu[0]] = seen[cu[-1]:] = False
    assert (np.abs(z[seen] - wlse[seen]) <= ltol[seen]).all()
    # the same bits again, in a workspace that was used, and without lse
    again = torch.full_like(out, 7.0)
    adamas.chunk_attend(q, K, V, cud, ld, ws, block_table=tab(table), out=again)
    assert same(out, again)

    # the weights, from the lse the kernel wrote
    cap = N if table is None else table.shape[1] * page
    mass = torch.rand(B, Hkv, cap, generator=torch.Generator().manual_seed(14)).to(DEV)
    m0 = mass.cpu().numpy()
    m1 = mass.clone()
    adamas.accumulate_chunk(q, K, lse, cud, ld, mass, ws, block_table=tab(table))
    assert ws.device_error() == 0
    wm, mtol = co.accumulate_chunk(f64(q), f64(K), z, cu, lens, m0, npt(table))
    assert (np.abs(f64(mass) - wm) <= mtol).all()
    adamas.accumulate_chunk(q, K, lse, cud, ld, m1, ws, block_table=tab(table))
    assert same(mass, m1)


def test_chunk_attend_long_context_with_far_pages():
    """Row offsets past 2^31 elements: pages at the end of a 4.3 GB array."""
    page, n_pages = 64, 270000                                # 64 * 270000 * 128 > 2^31
    K = torch.empty(n_pages, 1, page, 128, dtype=torch.bfloat16, device=DEV)
    V = torch.empty_like(K)
    table = torch.arange(n_pages - 20, n_pages, dtype=torch.int32).flip(0).view(1, 20).contiguous()
    g = torch.Generator().manual_seed(21)
    K[-20:], V[-20:] = torch.randn(20, 1, page, 128, generator=g).to(torch.bfloat16).to(DEV), torch.randn(20, 1, page, 128, generator=g).to(torch.bfloat16).to(DEV)
    q = torch.randn(3, 4, 128, generator=g).to(torch.bfloat16).to(DEV)
    ws = adamas.ChunkWorkspace(3, 1, 4, 1)
    out, lse = adamas.chunk_attend(q, K, V, i32([0, 3]), i32([1277]), ws, block_table=tab(table))
    small = torch.arange(20, dtype=torch.int32).flip(0).view(1, 20).contiguous()
    want, wlse, tol, ltol = co.attend(f64(q), f64(K[-20:]), f64(V[-20:]), [0, 3], [1277], small.numpy())
    assert (np.abs(f64(out) - want) <= tol).all() and (np.abs(f64(lse) - wlse) <= ltol).all()
    k = torch.randn(2, 1, 128, generator=g).to(torch.bfloat16).to(DEV)
    freqs, _ = adamas.rope_frequencies(0)
    adamas.rope_append(None, k, k, i32([0, 2]), i32([1278]), K, V, freqs, ws, block_table=tab(table))
    assert same(K[n_pages - 20, 0, 62:], k[:, 0]) and same(V[n_pages - 20, 0, 62:], k[:, 0])
    mass = torch.rand(1, 1, 1280, generator=g).to(DEV)
    kept, lens = adamas.evict(K, V, mass.clone(), i32([1280]), 100, ws, block_table=tab(table))
    wk, _ = co.evict_select(mass.cpu().numpy(), [1280], 100, 0, 0)
    assert np.array_equal(kept.cpu().numpy(), wk) and lens.tolist() == [100]


def test_chunk_attend_flags():
    q = torch.randn(4, 2, 128).to(torch.bfloat16).to(DEV)
    K = torch.randn(3, 2, 16, 128).to(torch.bfloat16).to(DEV)
    ws = adamas.ChunkWorkspace(4, 1, 2, 2)
    t = i32([[1, 9, 2]])
    adamas.chunk_attend(q, K, K, i32([0, 4]), i32([40]), ws, block_table=t)       # page 0 is read for entry 9
    assert ws.device_error() == adamas.DEVERR_TABLE
    ws.reset()
    a, _ = adamas.chunk_attend(q, K, K, i32([0, 4]), i32([40]), ws, block_table=i32([[1, 0, 2]]))
    assert ws.device_error() == 0
    b, _ = adamas.chunk_attend(q, K, K, i32([0, 4]), i32([40]), ws, block_table=t)
    assert same(a, b)
    ws.reset()
    adamas.chunk_attend(q, K, K, i32([0, 4]), i32([49]), ws, block_table=i32([[1, 0, 2]]))   # clamped to 48
    assert ws.device_error() == adamas.DEVERR_SEQLEN
    for cu in ([0, 5], [-1, 3], [3, 2]):
        ws.reset()
        out, _ = adamas.chunk_attend(q, K[:1], K[:1], i32(cu), i32([16]), ws)
        assert ws.device_error() in (0, adamas.DEVERR_OFFSETS) and not out.any()


def test_bindings_refuse():
    q = torch.zeros(4, 2, 128, dtype=torch.bfloat16, device=DEV)
    K = torch.zeros(1, 2, 16, 128, dtype=torch.bfloat16, device=DEV)
    ws = adamas.ChunkWorkspace(4, 1, 2, 2)
    cu, lens = i32([0, 4]), i32([16])
    mass = torch.zeros(1, 2, 16, device=DEV)
    with pytest.raises(TypeError):
        adamas.chunk_attend(q.float(), K, K, cu, lens, ws)
    with pytest.raises(ValueError):
        adamas.chunk_attend(q, K, K[:, :, :8], cu, lens, ws)
    with pytest.raises(ValueError):
        adamas.chunk_attend(q, K.cpu(), K, cu, lens, ws)
    with pytest.raises(ValueError):
        adamas.chunk_attend(q, K, K, cu[:1], lens, ws)
    with pytest.raises(ValueError):
        adamas.chunk_attend(q[:, :, :64], K, K, cu, lens, ws)
    with pytest.raises(TypeError):
        adamas.accumulate_chunk(q, K, torch.zeros(4, 2, device=DEV), cu, lens, mass.double(), ws)
    with pytest.raises(ValueError):
        adamas.accumulate_chunk(q, K, torch.zeros(4, 2, device=DEV), cu, lens, mass[:, :, :8], ws)
    with pytest.raises(ValueError):
        adamas.accumulate_kept(q[:1], K, torch.zeros(1, 1, 4, dtype=torch.int32, device=DEV), lens, mass, ws)
    with pytest.raises(ValueError):
        adamas.evict(K, K, mass, lens, 4, ws, K_out=K)
    with pytest.raises(adamas.AdamasError):
        adamas.evict(K, K, mass, lens, 4, ws, new_lens=lens)
    with pytest.raises(adamas.AdamasError):
        adamas.evict(K, K, mass, lens, -1, ws)
    with pytest.raises(ValueError):
        adamas.rope_append(q.transpose(0, 1), None, None, cu, lens, K, K, adamas.rope_frequencies()[0], ws)


# ---------------------------------------------------------------- kept tokens
@pytest.mark.parametrize("B,Hq,Hkv,N,lens,budget,page,shared", [
    (1, 1, 1, 1, [1], 1, 0, False),
    (2, 8, 2, 90, [90, 13], 20, 0, False),
    (2, 8, 2, 90, [90, 13], 20, 7, True),
    (3, 6, 2, 400, [400, 0, 77], 100, 16, False),
    (1, 8, 1, 5000, [5000], 1024, 64, False),
    (1, 4, 4, 9000, [9000], 9000, 0, False),
    (2, 5, 1, 700, [700, 500], 333, 1, False),
    (1, 8, 1, 60000, [60000], 60000, 0, False),           # longer lists than a cluster's shared memory holds
    (1, 8, 1, 60000, [60000], 60000, 0, True),
])
def test_accumulate_kept(B, Hq, Hkv, N, lens, budget, page, shared):
    rng = np.random.default_rng(31)
    rows = Hkv if shared else Hq
    idx = np.full((B, rows, budget), -1, np.int32)
    for b in range(B):
        for h in range(rows):
            k = min(budget, lens[b])
            idx[b, h, :k] = rng.permutation(lens[b])[:k]
    if lens[0] > 2 and budget > 2:
        idx[0, 0, 1] = lens[0] + 3                        # outside the sequence: skipped
        idx[0, 0, 2] = -5
    q = torch.randn(B, Hq, 128, generator=torch.Generator().manual_seed(32)).to(torch.bfloat16).to(DEV)
    K = make_cache(33, B, Hkv, N, lens, page, gain=2.0)
    table = make_table(33, B, N, page)
    cap = N if table is None else table.shape[1] * page
    mass = torch.zeros(B, Hkv, cap, device=DEV)
    mass[..., ::3] = 0.5
    m0, ws = mass.cpu().numpy(), adamas.ChunkWorkspace(B, B, Hq, Hkv)
    m1 = mass.clone()
    policy = adamas.SELECT_GROUP_SHARED if shared else adamas.SELECT_PER_HEAD
    adamas.accumulate_kept(q, K, i32(idx), i32(lens), mass, ws, policy=policy, block_table=tab(table))
    assert ws.device_error() == 0
    want, tol = co.accumulate_kept(f64(q), f64(K), idx, lens, m0, npt(table))
    assert (np.abs(f64(mass) - want) <= tol).all()
    adamas.accumulate_kept(q, K, i32(idx), i32(lens), m1, ws, policy=policy, block_table=tab(table))
    assert same(mass, m1)


# ---------------------------------------------------------------- eviction
EVICT = [
    # Hkv, lens, N, keep, sink, recent, page, to (None: in place, 0: contiguous, P: pages), codes
    (1, [1], 1, 1, 0, 0, 0, None, True),
    (2, [40, 13, 0], 40, 12, 2, 3, 0, None, True),
    (2, [40, 13, 0], 40, 12, 2, 3, 7, 5, True),
    (1, [300, 299], 300, 0, 0, 0, 16, 0, False),
    (3, [700, 350], 700, 699, 0, 700, 0, None, True),          # all forced; one evicted
    (2, [1000], 1000, 500, 4, 64, 16, None, True),
    (8, [2000, 1500], 2048, 300, 0, 32, 64, 0, True),
    (2, [5000, 4999], 5000, 4500, 16, 0, 24, None, False),
    (1, [40000], 40000, 20000, 4, 128, 0, None, True),
    (4, [9000, 130, 9000], 9000, 4096, 4, 64, 1, 16, True),
    (1, [400000], 400000, 700, 4, 64, 0, 0, True),             # a block's slice does not fit its shared memory
    (1, [330000], 330000, 329000, 0, 0, 16, None, False),
    (16, [3000, 2999, 1, 3000, 64, 500, 2000, 3000, 2048, 7], 3000, 1024, 0, 0, 0, None, True),
]


def masses(seed, B, Hkv, N, ties):
    rng = np.random.default_rng(seed)
    m = rng.exponential(1.0, (B, Hkv, N)).astype(np.float32)
    if ties:
        m = np.where(rng.random(m.shape) < 0.5, np.float32(0), np.round(m))
        m[rng.random(m.shape) < 0.1] = -0.0
        m[rng.random(m.shape) < 0.05] = np.nan
        m[rng.random(m.shape) < 0.05] = np.inf
        m[rng.random(m.shape) < 0.05] = -np.inf
        m[rng.random(m.shape) < 0.05] = np.float32(1e-45)
    return m.astype(np.float32)


@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("Hkv,lens,N,keep,sink,recent,page,to,codes", EVICT)
def test_evict(Hkv, lens, N, keep, sink, recent, page, to, codes, ties):
    B = len(lens)
    table = make_table(41, B, N, page)
    cap = N if table is None else table.shape[1] * page
    K = make_cache(41, B, Hkv, N, [N] * B, page, fill=9.0)
    V = make_cache(42, B, Hkv, N, [N] * B, page, fill=9.0, table_seed=41)
    g = torch.Generator().manual_seed(43)
    C = torch.randint(0, 256, K.shape[:-1] + (32,), generator=g, dtype=torch.uint8).to(DEV) if codes else None
    m = masses(44, B, Hkv, cap, ties)
    mass = torch.from_numpy(m.copy()).to(DEV)
    if to is None:
        dst = dict()
        K2, V2, C2, m2, table2, page2 = K, V, C, mass, table, page
    else:
        table2, page2 = make_table(45, B, max(keep, 1), to), to
        K2 = to_pages(torch.zeros(B, Hkv, max(keep, 1), 128, dtype=torch.bfloat16), table2, to, 3.0)
        V2 = K2.clone()
        C2 = torch.full(K2.shape[:-1] + (32,), 0x33, dtype=torch.uint8, device=DEV) if codes else None
        m2 = torch.full((B, Hkv, max(keep, 1) if table2 is None else table2.shape[1] * to), 5.0, device=DEV)
        dst = dict(K_out=K2, V_out=V2, codes_out=C2, mass_out=m2, table_out=tab(table2))
    old = [None if x is None else x.cpu() for x in (K, V, C)]
    before = [None if x is None else x.cpu() for x in (K2, V2, C2)]
    ws = adamas.ChunkWorkspace(1, B, Hkv, Hkv)
    kept, new_lens = adamas.evict(K, V, mass, i32(lens), keep, ws, codes=C, n_sink=sink, n_recent=recent,
                                  block_table=tab(table), **dst)
    assert ws.device_error() == 0
    want, wlens = co.evict_select(m, np.asarray(lens), keep, sink, recent)
    assert np.array_equal(new_lens.cpu().numpy(), wlens)
    assert np.array_equal(kept.cpu().numpy(), want)
    wm = np.zeros(tuple(m2.shape), np.float32)
    expect = [None if x is None else x.clone() for x in before]
    for b in range(B):
        k = int(wlens[b])
        for h in range(Hkv):
            src = want[b, h, :k].astype(np.int64)
            wm[b, h, :k] = m[b, h, src]
            j = np.arange(k)
            for o, e in zip(old, expect):
                if o is None:
                    continue
                rows = o[b, h, src] if table is None else o[table[b].long()[src // page], h, src % page]
                if table2 is None:
                    e[b, h, j] = rows
                else:
                    e[table2[b].long()[j // page2], h, j % page2] = rows
    assert np.array_equal(m2.cpu().numpy().view(np.uint32), wm.view(np.uint32))
    for x, e in zip((K2, V2, C2), expect):
        assert x is None or same(x.cpu(), e)
    if to is not None:
        assert np.array_equal(mass.cpu().numpy().view(np.uint32), m.view(np.uint32))


def test_evict_flags_bad_pages():
    K = torch.randn(4, 1, 8, 128).to(torch.bfloat16).to(DEV)
    V, mass = K.clone(), torch.rand(1, 1, 24, device=DEV)
    K2, V2 = torch.zeros(2, 1, 8, 128, dtype=torch.bfloat16, device=DEV), torch.zeros(2, 1, 8, 128, dtype=torch.bfloat16, device=DEV)
    ws = adamas.ChunkWorkspace(1, 1, 1, 1)
    adamas.evict(K, V, mass, i32([24]), 12, ws, block_table=i32([[3, 1, 0]]), K_out=K2, V_out=V2,
                 mass_out=torch.zeros(1, 1, 16, device=DEV), table_out=i32([[1, 7]]))
    assert ws.device_error() == adamas.DEVERR_TABLE
    assert not K2[0].any() and K2[1].any()                    # nothing written through the bad entry
    ws.reset()
    adamas.evict(K, V, mass, i32([25]), 12, ws, block_table=i32([[3, 1, 0]]), K_out=K2, V_out=V2,
                 mass_out=torch.zeros(1, 1, 16, device=DEV), table_out=i32([[1, 0]]))
    assert ws.device_error() == adamas.DEVERR_SEQLEN


# ---------------------------------------------------------------- a run of them, as a serving loop makes it
@pytest.mark.parametrize("page", [0, 16])
def test_prompt_evict_decode(page, orc):
    """Two prompts are appended and attended in two chunks, their weights accumulated,
    the caches cut to 64 tokens in place, then three decode steps append, select,
    attend and accumulate -- against the same steps of the definitions."""
    B, Hq, Hkv, N, keep, budget = 2, 8, 2, 160, 64, 16
    prompts, chunk = [150, 97], 80
    rng = torch.Generator().manual_seed(51)
    table = make_table(51, B, N, page)
    cap = N if table is None else table.shape[1] * page
    zeros = torch.zeros(B, Hkv, N, 128, dtype=torch.bfloat16)
    K, V = to_pages(zeros, table, page, 0.0), to_pages(zeros, table, page, 0.0)
    codes = torch.zeros(K.shape[:-1] + (32,), dtype=torch.uint8, device=DEV)
    mass, td = torch.zeros(B, Hkv, cap, device=DEV), tab(table)
    freqs, mscale = adamas.rope_frequencies(128, scaling="yarn", factor=32.0)
    ws = adamas.ChunkWorkspace(2 * chunk, B, Hq, Hkv)
    done = [0, 0]
    wmass = np.zeros((B, Hkv, cap))
    mtol = np.zeros_like(wmass)
    while done != prompts:
        ns = [min(chunk, p - d) for p, d in zip(prompts, done)]
        cu, T = i32(offsets(ns)), sum(ns)
        q, k, v = (torch.randn(T, h, 128, generator=rng).to(torch.bfloat16).to(DEV) for h in (Hq, Hkv, Hkv))
        q = adamas.rope_append(q, k, v, cu, i32(done), K, V, freqs, ws, mscale=mscale, codes=codes, block_table=td)
        done = [d + n for d, n in zip(done, ns)]
        out, lse = adamas.chunk_attend(q, K, V, cu, i32(done), ws, block_table=td)
        adamas.accumulate_chunk(q, K, lse, cu, i32(done), mass, ws, block_table=td)
        want, wlse, tol, ltol = co.attend(f64(q), f64(K), f64(V), offsets(ns), done, npt(table))
        assert (np.abs(f64(out) - want) <= tol).all() and (np.abs(f64(lse) - wlse) <= ltol).all()
        add, t = co.accumulate_chunk(f64(q), f64(K), f64(lse), offsets(ns), done, np.zeros_like(wmass), npt(table))
        wmass, mtol = wmass + add, mtol + t
    mtol += 8 * co.U32 * wmass
    assert (np.abs(f64(mass) - wmass) <= mtol).all()
    # every prompt row gives its heads' whole weight away
    assert np.allclose(f64(mass).sum((1, 2)), [p * Hq for p in prompts], rtol=1e-4)

    m0, K0 = mass.cpu().numpy(), K.cpu()
    kept, lens = adamas.evict(K, V, mass, i32(done), keep, ws, codes=codes, n_sink=4, n_recent=16, block_table=td)
    wkept, _ = co.evict_select(m0, np.asarray(done), keep, 4, 16)
    assert np.array_equal(kept.cpu().numpy(), wkept) and lens.tolist() == [keep, keep]
    for b in range(B):
        for h in range(Hkv):
            t = wkept[b, h].astype(np.int64)
            k0 = K0[b, h, t] if table is None else K0[table[b].long()[t // page], h, t % page]
            got = torch.from_numpy(co.gather(K.cpu().float().numpy(), npt(table), b, h, np.arange(keep))).to(torch.bfloat16)
            assert same(got, k0)

    dws = adamas.Workspace(B, Hq, Hkv, cap, budget)
    one = i32([0, 1, 2])
    for step in range(3):
        q, k, v = (torch.randn(B, h, 128, generator=rng).to(torch.bfloat16).to(DEV) for h in (Hq, Hkv, Hkv))
        pos = i32([p + step for p in prompts])                 # positions go on; slots start at the kept count
        q = adamas.rope_append(q, k, v, one, lens, K, V, freqs, dws, positions=pos, mscale=mscale, codes=codes,
                               block_table=td)
        lens = lens + 1
        out, idx = adamas.decode(q, codes, K, V, lens, budget, dws, block_table=td, n_sink=2, n_recent=4)
        m0 = mass.cpu().numpy()
        adamas.accumulate_kept(q, K, idx, lens, mass, dws, block_table=td)
        assert dws.device_error() == 0
        dense = np.stack([[co.gather(K.view(torch.int16).cpu().numpy().view(np.uint16), npt(table), b, h, np.arange(N))
                           for h in range(Hkv)] for b in range(B)])
        densev = np.stack([[co.gather(V.view(torch.int16).cpu().numpy().view(np.uint16), npt(table), b, h, np.arange(N))
                            for h in range(Hkv)] for b in range(B)])
        q16 = q.view(torch.int16).cpu().numpy().view(np.uint16)
        ln = lens.cpu().numpy()
        wout, widx = orc.decode_step_forced(q16, dense, densev, orc.encode(dense), ln, budget, 2, 4)
        assert np.array_equal(idx.cpu().numpy(), widx)
        assert_close_out(f64(out), wout)
        wm, t = co.accumulate_kept(f64(q), f64(K), widx, ln, m0, npt(table))
        assert (np.abs(f64(mass) - wm) <= t).all()


def test_captured_calls_and_other_streams():
    """Two captured runs share one workspace and are replayed in turn; a third runs on
    another stream with its own workspace."""
    B, Hq, Hkv, N = 3, 8, 2, 600
    ns, lens = [1, 40, 3], [600, 411, 77]
    cu = i32(offsets(ns))
    qs = [torch.randn(44, Hq, 128, generator=torch.Generator().manual_seed(s)).to(torch.bfloat16).to(DEV) for s in (1, 2)]
    K, V = make_cache(61, B, Hkv, N, lens, 16), make_cache(62, B, Hkv, N, lens, 16, table_seed=61)
    table = tab(make_table(61, B, N, 16))
    ld = i32(lens)
    ws = adamas.ChunkWorkspace(44, B, Hq, Hkv)
    mass0 = torch.rand(B, Hkv, table.shape[1] * 16, generator=torch.Generator().manual_seed(3)).to(DEV)

    def run(q, ws, mass, stream=None):
        out, lse = adamas.chunk_attend(q, K, V, cu, ld, ws, block_table=table, stream=stream)
        adamas.accumulate_chunk(q, K, lse, cu, ld, mass, ws, block_table=table, stream=stream)
        return out, lse

    masses_ = [mass0.clone() for _ in qs]
    eager = [run(q, ws, m) for q, m in zip(qs, masses_)]
    side = torch.cuda.Stream()
    graphs, outs, gm = [], [], [mass0.clone() for _ in qs]
    with torch.cuda.stream(side):
        for q, m in zip(qs, gm):
            g = torch.cuda.CUDAGraph()
            side.synchronize()
            with torch.cuda.graph(g, stream=side):
                outs.append(run(q, ws, m))
            graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(2):
        for m in gm:
            m.copy_(mass0)
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for (a, la), (b, lb), m, w in zip(eager, outs, gm, masses_):
        assert same(a, b) and same(la, lb) and same(m, w)
    ws2, m2 = adamas.ChunkWorkspace(44, B, Hq, Hkv), mass0.clone()
    torch.cuda.synchronize()
    o2, l2 = run(qs[0], ws2, m2, stream=side)
    o1, l1 = run(qs[1], ws, mass0.clone())
    torch.cuda.synchronize()
    assert same(o2, eager[0][0]) and same(l2, eager[0][1]) and same(m2, masses_[0]) and same(o1, eager[1][0])
    assert ws.device_error() == 0 and ws2.device_error() == 0


def test_empty_cache_and_empty_batch():
    q = torch.randn(3, 4, 128).to(torch.bfloat16).to(DEV)
    K = torch.zeros(2, 2, 0, 128, dtype=torch.bfloat16, device=DEV)
    ws = adamas.ChunkWorkspace(3, 2, 4, 2)
    out, lse = adamas.chunk_attend(q, K, K, i32([0, 1, 3]), i32([0, 0]), ws)
    assert not out.any() and (lse == -float("inf")).all() and ws.device_error() == 0
    adamas.accumulate_chunk(q, K, lse, i32([0, 1, 3]), i32([0, 0]), torch.zeros(2, 2, 0, device=DEV), ws)
    out, lse = adamas.chunk_attend(q[:0], K, K, i32([0, 0, 0]), i32([0, 0]), ws)
    assert out.shape == (0, 4, 128) and lse.shape == (0, 4)
    none = torch.zeros(0, 2, 16, 128, dtype=torch.bfloat16, device=DEV)
    adamas.chunk_attend(q, none, none, i32([0]), i32([]), ws)
    kept, lens = adamas.evict(none, none, torch.zeros(0, 2, 16, device=DEV), i32([]), 4, ws)
    assert kept.shape == (0, 2, 4) and lens.shape == (0,)
    assert ws.device_error() == 0


def test_captured_append_and_eviction():
    """A captured decode-side run -- append, weights of kept tokens, eviction in place --
    replayed on fresh copies of its caches gives the eager run's bits; two replays in a
    row start from the same inputs again."""
    B, Hq, Hkv, N, budget, keep = 2, 8, 2, 500, 32, 256
    lens = [499, 380]
    g = torch.Generator().manual_seed(71)
    K0, V0 = make_cache(71, B, Hkv, N, [N, N], 0), make_cache(72, B, Hkv, N, [N, N], 0)
    q, k, v = (torch.randn(B, h, 128, generator=g).to(torch.bfloat16).to(DEV) for h in (Hq, Hkv, Hkv))
    idx = torch.stack([torch.stack([torch.randperm(n, generator=g)[:budget] for _ in range(Hq)]) for n in lens]).to(torch.int32).to(DEV)
    m0 = torch.rand(B, Hkv, N, generator=g).to(DEV)
    freqs, _ = adamas.rope_frequencies()
    one, before, after = i32([0, 1, 2]), i32(lens), i32([n + 1 for n in lens])
    ws = adamas.ChunkWorkspace(B, B, Hq, Hkv)
    K, V, mass = torch.empty_like(K0), torch.empty_like(V0), torch.empty_like(m0)
    codes = torch.zeros(K.shape[:-1] + (32,), dtype=torch.uint8, device=DEV)

    def run():
        K.copy_(K0), V.copy_(V0), mass.copy_(m0), codes.zero_()
        r = adamas.rope_append(q, k, v, one, before, K, V, freqs, ws, codes=codes)
        adamas.accumulate_kept(r, K, idx, after, mass, ws)
        return (r, *adamas.evict(K, V, mass, after, keep, ws, codes=codes, n_sink=2, n_recent=8), K, V, mass, codes)

    eager = [x.clone() for x in run()]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = run()
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(eager, got))
    assert ws.device_error() == 0
