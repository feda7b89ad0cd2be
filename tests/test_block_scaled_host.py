"""The block-scaled and scored restatements against closed forms, torch's E4M3
and scaled dot products, and the host refusals of the new calls (no GPU)."""

import ctypes
import math

import numpy as np
import pytest
import torch

import scored_ref as R


def test_e4m3_codes_equal_torchs():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(R.e4m3_value(codes), want, equal_nan=True)
    x = np.random.default_rng(0).standard_normal(20000).astype(np.float32) * 200
    edges = np.concatenate([want[np.isfinite(want)].astype(np.float32)] * 2)
    mid = np.unique(np.abs(edges))
    x = np.concatenate([x, x * 1e-4, edges, (mid[1:] + mid[:-1]) / 2]).astype(np.float32)
    x = np.clip(x, -448, 448)
    got = R.e4m3_code(x)
    ref = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(R.e4m3_value(got), R.e4m3_value(ref))
    assert R.e4m3_value(R.e4m3_code(np.float32([1e9, -np.inf]))).tolist() == [448.0, -448.0]


@pytest.mark.parametrize("cache", ["fp8_e4m3", "int8"])
def test_block_scale_follows_the_largest_row(cache):
    """A block filled row by row: every stored value within half a step of its
    own row at each rescale (at most one per row), and the scale is the largest
    |x| / qmax so far; starting anew forgets the old block."""
    rng = np.random.default_rng(1)
    codes, scales = np.zeros((2, 4, 1, 8), np.uint8), np.full((2, 1), 9.0, np.float32)
    rows = rng.standard_normal((4, 1, 8)).astype(np.float32) * np.float32([[[1]], [[3]], [[2]], [[9]]])
    top = 0.0
    for i in range(4):
        R.append_block_scaled(codes, scales, rows[i:i + 1], [4 + i], cache)
        top = max(top, np.abs(rows[i]).max())
        assert scales[1, 0] == np.float32(np.float32(top) / R.QMAX[cache])
        held = R.values(codes[1, :i + 1, 0], cache) * scales[1, 0]
        # int8: half a step of each scale so far; E4M3: 2^-4 relative per
        # rounding (or half its smallest step)
        rounds = i + 1
        step = rounds * 0.5 * scales[1, 0] if cache == "int8" else \
            np.abs(rows[:i + 1, 0]) * ((1 + 2.0 ** -4) ** rounds - 1) + rounds * 2.0 ** -10 * scales[1, 0]
        assert (np.abs(held - rows[:i + 1, 0]) <= step * 1.001 + 1e-7).all()
    R.append_block_scaled(codes, scales, rows[:1], [4], cache)
    assert scales[1, 0] == np.float32(np.abs(rows[0]).max() / R.QMAX[cache])
    assert scales[0, 0] == 9.0


def test_scored_reference_closed_forms():
    """No modification: torch's attention; a cap far above the scores changes
    nothing; a window of 1 gives the own value; slopes so steep that only the
    own token counts; nothing visible gives zeros; a full prefix is the
    unmasked attention."""
    rng = np.random.default_rng(2)
    L, hq, hkv, d, bs = 11, 4, 2, 16, 4
    k, v = rng.standard_normal((2, 3, bs, hkv, d))
    table, pos = np.array([2, 0, 1]), np.arange(L)
    q = rng.standard_normal((L, hq, d))
    run = lambda **kw: R.attention(q, k, v, table, L, pos, 0.25, **kw)
    kk, vv = (torch.from_numpy(x[table].reshape(-1, hkv, d)[:L].copy()).transpose(0, 1) for x in (k, v))
    sdpa = lambda **kw: torch.nn.functional.scaled_dot_product_attention(
        torch.from_numpy(q).transpose(0, 1), kk.repeat_interleave(2, 0), vv.repeat_interleave(2, 0),
        scale=0.25, **kw).transpose(0, 1).numpy()
    plain = run()
    assert np.abs(plain - sdpa(is_causal=True)).max() < 1e-12
    assert np.abs(run(prefix=L) - sdpa()).max() < 1e-12
    assert np.abs(run(softcap=1e9) - plain).max() < 1e-9
    own = vv.transpose(0, 1).numpy().repeat(2, 1)
    assert np.abs(run(window=1) - own).max() == 0
    assert np.abs(run(slopes=np.full(hq, 1e4)) - own).max() < 1e-12
    assert (run(first=pos + 1) == 0).all()
    assert np.abs(run(first=np.zeros(L)) - plain).max() == 0
    # two documents packed in one request = two requests
    doc = np.where(pos < 5, 0, 5)
    both = run(first=doc)
    assert np.abs(both[:5] - plain[:5]).max() < 1e-12
    t = torch.from_numpy(q[5:]).transpose(0, 1)
    alone = torch.nn.functional.scaled_dot_product_attention(
        t, kk[:, 5:].repeat_interleave(2, 0), vv[:, 5:].repeat_interleave(2, 0), scale=0.25,
        is_causal=True).transpose(0, 1).numpy()
    assert np.abs(both[5:] - alone).max() < 1e-12


def test_host_refusals():
    from paged_kv_cache_68_gb300 import pagedkv
    lib = pagedkv.load()
    fake, mis = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1008)
    h = ctypes.c_void_p()
    bf16, f32 = pagedkv.DTYPE_CODE[torch.bfloat16], pagedkv.DTYPE_CODE[torch.float32]

    def create(n=4, bs=16, hkv=2, d=128, cache=pagedkv.KV_INT8, dt=bf16, k=fake, v=fake, ks=fake,
               vs=fake, out=ctypes.byref(h)):
        return lib.kv_pool_create_block_scaled(n, bs, hkv, d, cache, dt, k, v, ks, vs, out)

    assert create(out=None) == pagedkv.KV_EINVAL
    assert create(cache=bf16) == create(dt=f32) == create(d=64) == create(bs=8) == \
        pagedkv.KV_EUNSUPPORTED
    for bad in (dict(n=0), dict(bs=512), dict(hkv=0), dict(k=None), dict(v=mis), dict(ks=None),
                dict(vs=mis), dict(n=1 << 28)):
        assert create(**bad) == pagedkv.KV_EINVAL, bad
    assert h.value is None
    mods = pagedkv.ScoreMods()
    size = ctypes.c_size_t()
    assert lib.paged_attention_scored_workspace_size(None, 1, 1, ctypes.byref(size)) == pagedkv.KV_EINVAL
    assert lib.paged_attention_decode_scored(None, None, None, None, 1, None, 1, 1, 1.0, 1,
                                             ctypes.byref(mods), None, 0, None) == pagedkv.KV_EINVAL
    assert lib.paged_attention_prefill_scored(None, None, None, None, 1, 1, None, 1, None, 1, 1, 1.0,
                                              1, ctypes.byref(mods), None) == pagedkv.KV_EINVAL


def test_score_mods_layout_matches_the_header(tmp_path):
    """The binding's struct has the C struct's size and offsets."""
    import os
    import shutil
    import subprocess
    from conftest import ROOT
    from paged_kv_cache_68_gb300 import pagedkv
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "s.c"
    names = [n for n, _ in pagedkv.ScoreMods._fields_]
    src.write_text('#include "pagedkv.h"\n#include <stdio.h>\nint main(void) {\n'
                   + "".join(f'  printf("%d ", (int)offsetof(kv_score_mods, {n}));\n' for n in names)
                   + '  printf("%d\\n", (int)sizeof(kv_score_mods));\n  return 0;\n}\n')
    exe = tmp_path / "s"
    subprocess.run([cc, "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    got = list(map(int, subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()))
    want = [getattr(pagedkv.ScoreMods, n).offset for n in names] + [ctypes.sizeof(pagedkv.ScoreMods)]
    assert got == want


def test_the_python_module_refuses_wrong_tensors():
    """Shapes, counts and host tensors are refused before any call."""
    from paged_kv_cache_68_gb300 import pagedkv
    m = pagedkv._fast()
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    plan = [0, i(3), i(3), i(3, 4), i(9), i(1), 5, None]
    with pytest.raises(TypeError):
        m.plan_step(*plan[:-1])
    for k, bad in ((1, 7), (1, i(3, 1)), (2, i(2)), (3, i(3)), (3, i(2, 4)), (5, i(2)), (6, -1),
                   (6, 1 << 40), (1, i(3))):
        with pytest.raises(ValueError):
            m.plan_step(*[bad if n == k else a for n, a in enumerate(plan)])
    q = torch.zeros(2, 4, 128)
    dec = [0, q, i(2, 3), i(2), 0.1, 2, 0.0, None, 0, None, None, i(1), None]
    pre = [0, q, i(3), 1, i(2, 3), i(2), 0.1, 2, 0.0, None, 0, None, None, None, None]
    for fn, good, bads in ((m.decode_scored, dec, ((1, q[0]), (2, i(3, 3)), (3, i(3)), (7, i(4)),
                                                   (9, i(3)), (8, 1 << 40))),
                           (m.prefill_scored, pre, ((1, q[0]), (2, i(2)), (4, i(2)), (9, i(4)),
                                                    (11, i(3)), (12, i(1))))):
        with pytest.raises(TypeError):
            fn(*good[1:])
        for k, bad in bads + ((1, q),):
            with pytest.raises(ValueError):
                fn(*[bad if n == k else a for n, a in enumerate(good)])


def test_append_refuses_fewer_rows_than_slots():
    """Rows that would be read past their end are refused before any call."""
    from paged_kv_cache_68_gb300 import pagedkv
    m = pagedkv._fast()
    rows, slots = torch.zeros(3, 2, 128, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int64)
    full = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    for k, v in ((rows, full), (full, rows)):
        with pytest.raises(ValueError, match="a row for each of the 4 slots"):
            m.append(0, k, v, slots, 256, None)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        m.append(0, full, full, slots, 256, None)
    with pytest.raises(TypeError):
        m.append(0, full, full, slots, 256)
