"""Calls that the documentation of the step plan, the block-scaled pools and
scored attention allows and that sit at an edge: the largest window, the largest
and smallest caps, offsets past 32 bits, two appends at once, graphs that outlive
their pool's workspace, layers of several kinds in one step."""

import numpy as np
import pytest
import torch

import scored_ref as R
from paged_kv_cache_68_gb300 import pagedkv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pagedkv.load()


def _decode_ref(s, q, **mods):
    q64 = q.double().cpu().numpy()
    return np.stack([R.attention(q64[b:b + 1], s.k, s.v, s.tables[b], int(L), [int(L) - 1], s.scale,
                                 **mods)[0] for b, L in enumerate(s.lens)])


@pytest.mark.parametrize("dtype,d,bs", [("f32", 64, 1), ("bf16", 128, 16), ("f16", 128, 8)])
def test_largest_window(dtype, d, bs):
    s = R.Setup("plain", dtype, [1, 40, 77], hq=4, hkv=2, d=d, bs=bs, seed=1)
    q = s.queries(3).cuda()
    pool = s.pool()
    try:
        out = pool.decode_scored(q, R.cuda_i32(s.tables), R.cuda_i32(s.lens), s.scale,
                                 window=2 ** 31 - 1)
        R.check(out.double().cpu().numpy(), _decode_ref(s, q), dtype)
        if d == 128:
            pre = pool.prefill_scored(q, R.cuda_i32([0, 1, 2, 3]), 1, R.cuda_i32(s.tables),
                                      R.cuda_i32(s.lens), s.scale, window=2 ** 31 - 1)
            R.check(pre.double().cpu().numpy(), _decode_ref(s, q), dtype)
        assert pool.get_error() == 0
    finally:
        pool.close()


@pytest.mark.parametrize("cap", [2.0 ** -10, 1024.0])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_smallest_and_largest_cap(dtype, cap):
    """The 16-bit forms' score error is cap 2^-22 (2.4e-4 at the largest cap): a
    weight is off by as much, the output by twice that times |v| <= 5, beside the
    bound of the other steps.  fp32 takes tanhf, whose error is relative."""
    s = R.Setup("plain", dtype, [1, 40, 300], hq=4, hkv=2, bs=16, seed=2)
    q = s.queries(3).cuda()
    ref = _decode_ref(s, q, softcap=cap)
    pool = s.pool()
    try:
        t, n = R.cuda_i32(s.tables), R.cuda_i32(s.lens)
        outs = [pool.decode_scored(q, t, n, s.scale, softcap=cap)]
        if dtype != "f32":
            outs.append(pool.prefill_scored(q, R.cuda_i32([0, 1, 2, 3]), 1, t, n, s.scale, softcap=cap))
        for out in outs:
            err = np.abs(out.double().cpu().numpy() - ref)
            eps = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[dtype]
            lim = 1e-5 if dtype == "f32" else 5e-4 + 2 * cap * 2.0 ** -22 * 5
            assert (err <= lim + eps * np.abs(ref)).all(), err.max()
    finally:
        pool.close()


def test_negative_scale_in_decode():
    """Decode takes any finite scale."""
    s = R.Setup("plain", "bf16", [30, 90], hq=4, hkv=2, bs=16, seed=3)
    s.scale = -s.scale
    q = s.queries(2).cuda()
    pool = s.pool()
    try:
        out = pool.decode_scored(q, R.cuda_i32(s.tables), R.cuda_i32(s.lens), s.scale, softcap=7.0)
        R.check(out.double().cpu().numpy(), _decode_ref(s, q, softcap=7.0), "bf16")
    finally:
        pool.close()


@pytest.mark.slow
def test_offsets_past_32_bits():
    """A block-scaled pool of more than 2^32 codes: rows appended to its last
    blocks (both ways of finding a block's rows) and attended there equal the
    same rows in a small pool."""
    bs, h, n = 16, 8, 270_000                                 # 4.4e9 codes of K, and of V
    assert n * bs * h * 128 > 2 ** 32
    L = [1500, 37]
    nb = [-(-x // bs) for x in L]
    small_n = sum(nb)
    outs = []
    g = torch.Generator(device="cuda").manual_seed(5)
    k = torch.randn((sum(L), h, 128), generator=g, device="cuda").bfloat16()
    v = torch.randn((sum(L), h, 128), generator=g, device="cuda").bfloat16()
    q = torch.randn((2, 32, 128), generator=g, device="cuda").bfloat16()
    for blocks in (small_n, n):
        codes = [torch.zeros((blocks, bs, h, 128), dtype=torch.uint8, device="cuda") for _ in range(2)]
        sc = [torch.zeros((blocks, h), device="cuda") for _ in range(2)]
        pool = pagedkv.KVPool(*codes, cache="fp8_e4m3", dtype=torch.bfloat16, k_scales=sc[0],
                              v_scales=sc[1], scale_per="block")
        try:
            ids = np.arange(blocks - small_n, blocks)
            tab = np.full((2, max(nb)), -1, np.int64)
            tab[0, :nb[0]], tab[1, :nb[1]] = ids[:nb[0]], ids[nb[0]:]
            slots = [tab[b, t // bs] * bs + t % bs for b in range(2) for t in range(L[b])]
            slots = torch.tensor(slots, device="cuda")
            pool.append(k[:L[0]], v[:L[0]], slots[:L[0]])      # noted rows
            pool.append(k[L[0]:], v[L[0]:], slots[L[0]:])      # scanned rows
            t, ln = R.cuda_i32(tab), R.cuda_i32(L)
            outs.append((pool.decode(q, t, ln, 0.09), pool.decode_scored(q, t, ln, 0.09, softcap=20.0),
                         pool.prefill_scored(q, R.cuda_i32([0, 1, 2]), 1, t, ln, 0.09, softcap=20.0),
                         codes[0][-small_n:].clone(), sc[1][-small_n:].clone()))
            torch.cuda.synchronize()
            assert pool.get_error() == 0
        finally:
            pool.close()
        del codes, sc, pool
        torch.cuda.empty_cache()
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_two_appends_at_once():
    """Large appends to disjoint blocks on two streams leave what one after the
    other leaves."""
    n, bs, h, t = 400, 16, 4, 2000
    g = torch.Generator(device="cuda").manual_seed(6)
    k = [torch.randn((t, h, 128), generator=g, device="cuda").half() for _ in range(2)]
    slots = [torch.arange(8 + i * 200 * bs, 8 + i * 200 * bs + t, device="cuda") for i in range(2)]
    res = []
    for at_once in (False, True):
        codes = [torch.zeros((n, bs, h, 128), dtype=torch.uint8, device="cuda") for _ in range(2)]
        sc = [torch.zeros((n, h), device="cuda") for _ in range(2)]
        pool = pagedkv.KVPool(*codes, cache="int8", dtype=torch.float16, k_scales=sc[0], v_scales=sc[1],
                              scale_per="block")
        try:
            torch.cuda.synchronize()
            streams = [torch.cuda.Stream(), torch.cuda.Stream()] if at_once else [None, None]
            for _ in range(3):
                for i in range(2):
                    pool.append(k[i], k[1 - i], slots[i], stream=streams[i])
            torch.cuda.synchronize()
            assert pool.get_error() == 0
        finally:
            pool.close()
        res.append(codes + sc)
    for a, b in zip(*res):
        assert torch.equal(a, b)


def test_a_graph_outlives_a_larger_batch():
    """A captured scored decode replays right after a larger batch has outgrown
    the pool's workspace."""
    lens = [3000, 2900]
    s = R.Setup("plain", "bf16", lens, hq=8, hkv=2, bs=16, seed=7)
    q = s.queries(2).cuda()
    t, n = R.cuda_i32(s.tables), R.cuda_i32(lens)
    pool = s.pool()
    try:
        out = pool.decode_scored(q, t, n, s.scale, softcap=9.0)
        want = out.clone()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pool.decode_scored(q, t, n, s.scale, softcap=9.0, out=out)
        many = 2000
        big_q = q[:1].expand(many, -1, -1).contiguous()
        pool.decode_scored(big_q, t[:1].expand(many, -1).contiguous(), n[:1].expand(many).contiguous(),
                           s.scale, softcap=9.0)
        junk = [torch.full((1 << 22,), 255, dtype=torch.uint8, device="cuda") for _ in range(16)]
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and len(junk) == 16
    finally:
        pool.close()


def test_layers_of_several_kinds_in_turn():
    """Windowed, global, plain and cascade calls in turn on one pool keep giving
    each its own result (their launch plans are kept side by side)."""
    lens = [700, 33, 16, 300]
    s = R.Setup("plain", "bf16", lens, hq=8, hkv=2, bs=16, seed=8)
    q = s.queries(4).cuda()
    t, n = R.cuda_i32(s.tables), R.cuda_i32(lens)
    gr = R.cuda_i32([[0, 2, 0]])
    pool = s.pool()
    try:
        calls = [lambda: pool.decode_scored(q, t, n, s.scale, window=40),
                 lambda: pool.decode_scored(q, t, n, s.scale, softcap=8.0),
                 lambda: pool.decode(q, t, n, s.scale),
                 lambda: pool.decode_cascade(q, t, n, s.scale, gr),
                 lambda: pool.decode_scored(q[:2].contiguous(), t[:2].contiguous(), n[:2].contiguous(), s.scale)]
        first = [c().clone() for c in calls]
        for _ in range(3):
            for c, w in zip(calls, first):
                assert torch.equal(c(), w)
        R.check(first[0].double().cpu().numpy(), _decode_ref(s, q, window=40), "bf16")
        R.check(first[1].double().cpu().numpy(), _decode_ref(s, q, softcap=8.0), "bf16")
    finally:
        pool.close()


def test_append_of_infinities_into_a_block_of_zeros():
    """FP8: a block whose finite values are all zero has scale 0, and an infinity
    in it becomes NaN, in the codes and the restatement alike."""
    x = np.zeros((2, 1, 128), np.float32)
    x[1, 0, 3] = np.inf
    codes, sc = np.zeros((1, 16, 1, 128), np.uint8), np.zeros((1, 1), np.float32)
    dev = [torch.from_numpy(codes.copy()).cuda() for _ in range(2)]
    dsc = [torch.zeros((1, 1), device="cuda") for _ in range(2)]
    pool = pagedkv.KVPool(*dev, cache="fp8_e4m3", dtype=torch.bfloat16, k_scales=dsc[0], v_scales=dsc[1],
                          scale_per="block")
    try:
        k = torch.from_numpy(x).bfloat16().cuda()
        pool.append(k, k, torch.tensor([0, 1], device="cuda"))
        R.append_block_scaled(codes, sc, x, [0, 1], "fp8_e4m3")
        got, want = R.values(dev[0].cpu().numpy(), "fp8_e4m3"), R.values(codes, "fp8_e4m3")
        assert np.array_equal(got, want, equal_nan=True) and np.isnan(got[0, 1, 0, 3])
        assert float(dsc[0]) == 0.0
    finally:
        pool.close()


def test_first_append_on_another_stream_than_the_pool_was_made_on():
    """A new pool's notes are zero for any stream, however busy the stream it was
    made on is."""
    n, bs, h, t = 2000, 16, 2, 3000
    g = torch.Generator(device="cuda").manual_seed(9)
    k, v = (torch.randn((t, h, 128), generator=g, device="cuda").bfloat16() for _ in range(2))
    slots = torch.arange(5, 5 + t, device="cuda")
    busy = torch.randn((4096, 4096), device="cuda")
    res = []
    for other in (False, True):
        codes = [torch.zeros((n, bs, h, 128), dtype=torch.uint8, device="cuda") for _ in range(2)]
        sc = [torch.zeros((n, h), device="cuda") for _ in range(2)]
        torch.cuda.synchronize()
        if other:
            for _ in range(20):
                busy = busy @ busy * 1e-3
        pool = pagedkv.KVPool(*codes, cache="fp8_e4m3", dtype=torch.bfloat16, k_scales=sc[0],
                              v_scales=sc[1], scale_per="block")
        try:
            stream = torch.cuda.Stream() if other else None
            for _ in range(2):
                pool.append(k, v, slots, stream=stream)
            torch.cuda.synchronize()
            assert pool.get_error() == 0
        finally:
            pool.close()
        res.append(codes + sc)
    for a, b in zip(*res):
        assert torch.equal(a, b)
