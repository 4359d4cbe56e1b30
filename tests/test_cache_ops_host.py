"""Cache operators without a GPU: the ctypes mirrors against the C compiler's layout of
include/adamas.h, refusals before any CUDA call, the frequency tables, and the
64-bit definitions the GPU tests compare with, against brute force and differences."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest
import torch

import cache_oracle as co
from compressed_sparse_kv_fp32_b200 import adamas, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    build.build()
    return adamas.load()


@pytest.mark.parametrize("cls,name", [(adamas.RopeArgs, "adamas_rope_args"), (adamas.ChunkArgs, "adamas_chunk_args"),
                                      (adamas.KeptArgs, "adamas_kept_args"), (adamas.EvictArgs, "adamas_evict_args")])
def test_argument_structs_match_the_header(cls, name, tmp_path):
    fields = [f for f, _ in cls._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "adamas.h"\nint main(void) {\n'
                   + f'  printf("%zu\\n", sizeof({name}));\n'
                   + "".join(f'  printf("%zu\\n", offsetof({name}, {f}));\n' for f in fields) + "  return 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got[0] == ctypes.sizeof(cls)
    assert got[1:] == [getattr(cls, f).offset for f in fields]


FAKE = 1 << 20                                     # never dereferenced: the checks come first


def _call(lib, name, cls, base, **kw):
    a = cls(**dict(base, **kw))
    return getattr(lib, "adamas_" + name)(ctypes.byref(a), None)


ROPE = dict(q=FAKE, k=FAKE, v=FAKE, q_stride=512, k_stride=128, v_stride=128, cu_new=FAKE, cache_lens=FAKE,
            freqs=FAKE, rot_dim=128, mscale=1.0, T=3, B=1, Hq=4, Hkv=1, Nmax=64, d=128, q_out=FAKE, K=FAKE, V=FAKE,
            workspace=FAKE, workspace_bytes=256)


@pytest.mark.parametrize("kw,rc", [
    (dict(d=64), -2), (dict(Hq=9, q_stride=1152), -2), (dict(Hq=5, Hkv=2), -1), (dict(T=-1), -1),
    (dict(rot_dim=130), -1), (dict(rot_dim=63), -1), (dict(rot_dim=-2), -1), (dict(v=None), -1),
    (dict(cu_new=None), -1), (dict(freqs=None), -1), (dict(q_out=None), -1), (dict(q_stride=511), -1),
    (dict(q_stride=500), -1), (dict(k_stride=64), -1), (dict(v_stride=132), -1),
    (dict(q_out=FAKE, q_stride=1024), -1),         # in place with spaced rows
    (dict(codes=FAKE + 16), -1), (dict(K=FAKE + 8), -1), (dict(K=None), -1), (dict(positions=FAKE + 2), -1),
    (dict(block_table=FAKE, page_size=0, max_pages=4, n_pages=8), -1),
    (dict(block_table=FAKE, page_size=1 << 20, max_pages=1 << 12, n_pages=8), -2),
    (dict(workspace=None), -3), (dict(workspace_bytes=128), -3), (dict(Nmax=1 << 31), -2),
    (dict(B=0), 0), (dict(T=0), 0), (dict(q=None, k=None, v=None), 0),
])
def test_rope_append_refuses(lib, kw, rc):
    assert _call(lib, "rope_append", adamas.RopeArgs, ROPE, **kw) == rc


CHUNK = dict(q=FAKE, K=FAKE, V=FAKE, cu_q=FAKE, seq_lens=FAKE, T=3, B=1, Hq=4, Hkv=1, Nmax=64, d=128, out=FAKE,
             lse=FAKE, mass=FAKE, workspace=FAKE, workspace_bytes=1 << 40)


@pytest.mark.parametrize("kw,rc", [
    (dict(d=64), -2), (dict(Hq=5, Hkv=2), -1), (dict(T=-1), -1), (dict(q=None), -1), (dict(V=None), -1),
    (dict(out=None), -1), (dict(out=FAKE + 2), -1), (dict(cu_q=None), -1), (dict(seq_lens=FAKE + 1), -1),
    (dict(lse=FAKE + 2), -1), (dict(K=FAKE + 8), -1), (dict(B=2000), -2),
    (dict(block_table=FAKE + 2, page_size=16, max_pages=4, n_pages=8), -1),
    (dict(workspace=None), -3), (dict(workspace_bytes=255), -3), (dict(B=0), 0), (dict(T=0), 0),
])
def test_chunk_attend_refuses(lib, kw, rc):
    assert _call(lib, "chunk_attend", adamas.ChunkArgs, CHUNK, **kw) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(d=64), -2), (dict(lse=None), -1), (dict(mass=None), -1), (dict(mass=FAKE + 2), -1), (dict(K=None), -1),
    (dict(workspace=None), -3), (dict(B=0), 0), (dict(T=0), 0), (dict(Nmax=0, K=None, mass=None), 0),
])
def test_accumulate_chunk_refuses(lib, kw, rc):
    assert _call(lib, "accumulate_chunk", adamas.ChunkArgs, dict(CHUNK, V=None, out=None), **kw) == rc


KEPT = dict(q=FAKE, K=FAKE, idx=FAKE, seq_lens=FAKE, B=1, Hq=4, Hkv=1, Nmax=64, d=128, budget=8, policy=0, mass=FAKE,
            workspace=FAKE, workspace_bytes=256)


@pytest.mark.parametrize("kw,rc", [
    (dict(d=64), -2), (dict(budget=-1), -1), (dict(policy=2), -1), (dict(idx=None), -1), (dict(mass=None), -1),
    (dict(q=FAKE + 8), -1), (dict(workspace_bytes=0), -3), (dict(budget=0), 0), (dict(B=0), 0),
])
def test_accumulate_kept_refuses(lib, kw, rc):
    assert _call(lib, "accumulate_kept", adamas.KeptArgs, KEPT, **kw) == rc


EVICT = dict(K=FAKE, V=FAKE, codes=FAKE, mass=FAKE, seq_lens=FAKE, B=1, Hkv=1, Nmax=64, d=128, keep=8, kept=FAKE,
             new_lens=2 * FAKE, workspace=FAKE, workspace_bytes=256)
OUT = dict(K_out=2 * FAKE, V_out=3 * FAKE, codes_out=2 * FAKE, mass_out=2 * FAKE, Nmax_out=8)


@pytest.mark.parametrize("kw,rc", [
    (dict(d=64), -2), (dict(keep=-1), -1), (dict(n_sink=-1), -1), (dict(n_recent=-1), -1), (dict(kept=None), -1),
    (dict(new_lens=FAKE), -1), (dict(new_lens=None), -1), (dict(mass=None), -1), (dict(workspace=None), -3),
    (dict(OUT, Nmax_out=7), -1), (dict(OUT, codes_out=None), -1), (dict(OUT, codes=None), -1),
    (dict(OUT, K_out=FAKE), -1), (dict(OUT, mass_out=None), -1), (dict(OUT, V_out=FAKE + 8), -1),
    (dict(OUT, block_table_out=FAKE, page_size_out=4, max_pages_out=1, n_pages_out=3), -1), (dict(B=0), 0),
])
def test_evict_refuses(lib, kw, rc):
    assert _call(lib, "evict", adamas.EvictArgs, EVICT, **kw) == rc


def test_null_argument_structs(lib):
    for name in ("rope_append", "chunk_attend", "accumulate_chunk", "accumulate_kept", "evict"):
        assert getattr(lib, "adamas_" + name)(None, None) == -1


def test_bindings_refuse_tensors_on_the_host():
    K = torch.zeros(1, 1, 4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        adamas.chunk_attend(K[0, :, :1], K, K, None, None, None)
    with pytest.raises(ValueError, match="CUDA"):
        adamas.evict(K, K, None, None, 1, None)
    with pytest.raises(TypeError):
        adamas.accumulate_kept(None, K, None, None, None, None)


# ---------------------------------------------------------------- frequency tables
@pytest.mark.parametrize("rot", [2, 6, 64, 128])
def test_frequencies_as_trained(rot):
    f, m = adamas.rope_frequencies(rot, 10000.0, device="cpu")
    want = 10000.0 ** (-np.arange(0, rot, 2) / rot) / (2 * math.pi)
    assert m == 1.0 and f.dtype == torch.int64
    # the table's entries are whole numbers of 2^-64 turns: half a unit is 2^-65 (the
    # slowest pairs are 2^-16 turns, where that is more than the power's own 2^-50)
    assert np.allclose(f.numpy() / 2.0 ** 64, want, rtol=2.0 ** -50, atol=2.0 ** -65)


def test_scaled_frequencies():
    plain = adamas.rope_frequencies(128, device="cpu")[0].double()
    lin, m = adamas.rope_frequencies(128, scaling="linear", factor=8.0, device="cpu")
    assert m == 1.0 and np.allclose(lin.double() * 8, plain, rtol=1e-12)
    ntk, m = adamas.rope_frequencies(128, scaling="ntk", factor=8.0, device="cpu")
    assert m == 1.0 and ntk[0] == plain[0].long()                      # the fastest pair as trained
    assert np.isclose(float(ntk[-1]) * 8, float(plain[-1]), rtol=1e-9)  # the slowest by the factor
    yarn, m = adamas.rope_frequencies(128, scaling="yarn", factor=32.0, original_len=4096, device="cpu")
    assert np.isclose(m, 0.1 * math.log(32.0) + 1.0)
    turns = plain / 2.0 ** 64 * 4096                                   # within the trained length
    ratio = (yarn.double() / plain).numpy()
    assert np.allclose(ratio[(turns > 40).numpy()], 1.0) and np.allclose(ratio[(turns < 0.8).numpy()], 1 / 32, rtol=1e-9)
    assert (np.diff(ratio) <= 1e-12).all()
    assert adamas.rope_frequencies(0, device="cpu")[0].shape == (0,)


@pytest.mark.parametrize("kw", [dict(rot_dim=3), dict(rot_dim=130), dict(base=1.0), dict(factor=0.5), dict(scaling="x"),
                                dict(rot_dim=2, scaling="ntk", factor=2.0)])
def test_frequencies_refuse(kw):
    with pytest.raises(ValueError):
        adamas.rope_frequencies(device="cpu", **kw)


# ---------------------------------------------------------------- the definitions
@pytest.mark.parametrize("inter,rot", [(False, 128), (True, 64), (False, 6)])
def test_rotation_definition(inter, rot):
    # the stepwise fp32 rotation against 64 bits: cos, sin, two products and a sum are
    # rounded to fp32, 4 half-steps of the two products' sizes at most
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 128)).astype(np.float32)
    f, _ = adamas.rope_frequencies(rot, device="cpu")
    freq = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    for pos in (0, 1, 4095, 1000000, -7):
        y = co.rotate(x, pos, f.numpy().view(np.uint64), rot, inter, 1.25)
        want = co.rotate64(x, pos, freq, rot, inter, 1.25)
        size = 1.25 * 2 * np.abs(x).max()
        assert np.abs(y - want).max() <= 4 * co.U32 * size + abs(pos) * 1e-15 * size
        assert np.array_equal(y[:, rot:], x[:, rot:])
    # relative positions: the product of two rotated rows depends on the distance alone
    a, b = x[:1], x[1:2]
    d = [float((co.rotate64(a, p + 9, freq, rot, inter, 1.0) * co.rotate64(b, p, freq, rot, inter, 1.0)).sum())
         for p in (0, 5, 70000)]
    assert np.allclose(d, d[0], atol=1e-8)


def test_attention_definition_against_differences_and_softmax():
    rng = np.random.default_rng(1)
    q, K, V = rng.standard_normal((3, 2, 128)), rng.standard_normal((1, 1, 9, 128)), rng.standard_normal((1, 1, 9, 128))
    out, lse, _, _ = co.attend(q, K, V, [0, 3], [9], None)
    s = torch.tensor(q).permute(1, 0, 2) @ torch.tensor(K[0, 0]).T / math.sqrt(128)
    s = s.masked_fill(torch.arange(9) > torch.arange(6, 9)[:, None], -math.inf)
    p = torch.softmax(s, -1)
    assert np.allclose(out, (p @ torch.tensor(V[0, 0])).permute(1, 0, 2))
    assert np.allclose(lse, torch.logsumexp(s, -1).T)
    mass, _ = co.accumulate_chunk(q, K, lse, [0, 3], [9], np.zeros((1, 1, 9), np.float32), None)
    assert np.allclose(mass[0, 0], p.sum((0, 1)))
    # the weight of a token is d lse / d score: a small step of one key along q
    e = 1e-6
    K2 = K.copy()
    K2[0, 0, 2] += e * q[1, 0] * math.sqrt(128) / (q[1, 0] @ q[1, 0])
    _, lse2, _, _ = co.attend(q, K2, V, [0, 3], [9], None)
    assert abs((lse2[1, 0] - lse[1, 0]) / e - float(p[0, 1, 2])) < 1e-5
    # rows that see nothing
    out, lse, _, _ = co.attend(q, K, V, [0, 3], [2], None)
    assert lse[0, 0] == -math.inf and not out[0].any() and np.allclose(out[1], V[0, 0, 0])


def test_eviction_definition():
    m = np.array([[[0.0, 3.0, float("nan"), -0.0, 3.0, 1.0, 9.0, 5.0]]], np.float32)
    kept, lens = co.evict_select(m, [7], 4, 0, 0)
    assert kept.tolist() == [[[1, 4, 5, 6]]] and lens.tolist() == [4]
    assert co.evict_select(m, [7], 3, 0, 1)[0].tolist() == [[[1, 4, 6]]]
    assert co.evict_select(m, [7], 6, 0, 0)[0].tolist() == [[[0, 1, 3, 4, 5, 6]]]   # NaN goes first
    assert co.evict_select(m, [7], 2, 1, 3)[0].tolist() == [[[0, 4]]]              # the lowest slots of the forced
    assert co.evict_select(m, [2], 4, 0, 0)[0].tolist() == [[[0, 1, -1, -1]]]
