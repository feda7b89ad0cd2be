"""8-bit pools with a scale for each (block, KV head): the append's codes and
scales equal the restatement's, copy and swap move both, decode and prefill
attend to the values the codes and scales stand for."""

import ctypes

import numpy as np
import pytest
import torch

import scored_ref as R
from paged_kv_cache_68_gb300 import pagedkv

pytestmark = pytest.mark.gpu
CACHES = ["fp8_e4m3", "int8"]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pagedkv.load()


def _random_pool(rng, n, bs, hkv, cache):
    c = R.encode((rng.standard_normal((n, bs, hkv, 128)) * (90 if cache != "int8" else 40))
                 .astype(np.float32), cache)
    s = (np.exp(0.5 * rng.standard_normal((n, hkv))) / (90 if cache != "int8" else 40)).astype(np.float32)
    return c, s


def _append_both(cache, dtype, n, bs, hkv, calls, seed=0):
    """The same calls (k rows, v rows, slots) on the GPU and in the restatement."""
    rng = np.random.default_rng(seed)
    (kc, ks), (vc, vs) = (_random_pool(rng, n, bs, hkv, cache) for _ in range(2))
    dev = [torch.from_numpy(a.copy()).cuda() for a in (kc, vc, ks, vs)]
    pool = pagedkv.KVPool(dev[0], dev[1], cache=cache, dtype=R.TORCH[dtype], k_scales=dev[2],
                          v_scales=dev[3], scale_per="block")
    try:
        for k, v, slots in calls:
            k, v = (torch.from_numpy(a).to(R.TORCH[dtype]) for a in (k, v))
            pool.append(k.cuda(), v.cuda(), torch.from_numpy(np.asarray(slots, np.int64)).cuda())
            R.append_block_scaled(kc, ks, k.float().numpy(), slots, cache)
            R.append_block_scaled(vc, vs, v.float().numpy(), slots, cache)
        torch.cuda.synchronize()
        err = pool.get_error()
    finally:
        pool.close()
    for got, want, what in zip(dev, (kc, vc, ks, vs), ("k", "v", "k scales", "v scales")):
        got = got.cpu().numpy()
        if want.dtype == np.uint8:
            g, w = R.values(got, cache), R.values(want, cache)
            bad = ~((g == w) | (np.isnan(g) & np.isnan(w)))
            assert not bad.any(), f"{what}: {int(bad.sum())} codes differ, first at {np.argwhere(bad)[:3]}"
        else:
            assert np.array_equal(got, want, equal_nan=True), what
    return err


def _rows(rng, t, hkv, gain=1.0):
    return (rng.standard_normal((t, hkv, 128)) * gain).astype(np.float32)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hkv,bs", [(8, 16), (1, 16), (5, 48), (2, 256)])
def test_append_runs(cache, dtype, hkv, bs):
    """Runs of every length that start, continue and fill blocks, one call."""
    rng = np.random.default_rng(bs + hkv)
    slots, n = [], 0
    for start, length in ((0, 1), (0, bs), (3, 2), (bs - 1, 1), (5, bs), (0, 2 * bs + 1), (bs // 2, 1)):
        slots += list(range(n * bs + start, n * bs + start + length))
        n += -(-(start + length) // bs) + 1
    t = len(slots)
    assert _append_both(cache, dtype, n, bs, hkv, [(_rows(rng, t, hkv, 2.0), _rows(rng, t, hkv), slots)]) == 0


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("t", [1, 2, 1023, 1024, 1025, 3000])
def test_append_any_order_and_repeats(cache, t):
    """Shuffled slots, padding and repeated slots (the last row wins), at sizes
    on both sides of the two ways rows are found."""
    rng = np.random.default_rng(t)
    n, bs, hkv = t // 8 + 2, 16, 2
    slots = rng.permutation(n * bs)[:t]
    if t > 10:
        slots[rng.integers(0, t, t // 10)] = -1
        slots[rng.integers(0, t, t // 10)] = slots[t // 2]
        slots[-1] = slots[0]
    assert _append_both(cache, "bf16", n, bs, hkv, [(_rows(rng, t, hkv), _rows(rng, t, hkv), slots)]) == 0


@pytest.mark.parametrize("cache", CACHES)
def test_append_call_after_call(cache):
    """Decode steps through a block: the scale grows, holds, and starts anew;
    large calls alternate with small ones (the notes are cleared)."""
    rng = np.random.default_rng(4)
    bs, hkv, calls = 16, 3, []
    for i in range(20):
        g = float(np.exp(rng.normal(0, 1.5)))
        calls.append((_rows(rng, 2, hkv, g), _rows(rng, 2, hkv, 1 / g), [i % bs, 16 * 5 + (i + 3) % bs]))
    big = list(range(7 * bs, 7 * bs + 1500))
    calls.append((_rows(rng, 1500, hkv), _rows(rng, 1500, hkv), big))
    calls.append((_rows(rng, 1500, hkv, 4), _rows(rng, 1500, hkv, .1), [s + 5 for s in big]))
    calls.append((_rows(rng, 3, hkv), _rows(rng, 3, hkv), big[20:23]))
    assert _append_both(cache, "f16", 110, bs, hkv, calls) == 0


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("pad", [0, 1100])
def test_append_special_rows(cache, pad):
    """Zeros, tiny rows (scale below 2^-126), values near the type's largest,
    infinities and NaN, and slots outside the pool."""
    rng = np.random.default_rng(5)
    bs, hkv, n = 16, 2, 90
    k = _rows(rng, 9, hkv)
    k[0] = 0                                   # block 0: zeros, then values on top
    k[2] = 1e-38                               # block 1: flushed
    k[3] = 3e38                                # block 2
    k[4, 0, 5], k[4, 1, 7] = np.inf, -np.inf   # block 3
    k[5, 0, 3] = np.nan                        # block 4
    slots = [0, 1, 16, 32, 48, 64, 65, 49, n * bs]
    fill = list(range(6 * bs, 6 * bs + pad))
    k2 = np.concatenate([k, _rows(rng, pad, hkv)])
    first = (k2, k2[::-1].copy(), slots + fill)
    second = (_rows(rng, 5 + pad, hkv), _rows(rng, 5 + pad, hkv), [2, 17, 33, 50, 66] + fill)
    anew = (_rows(rng, 3, hkv), _rows(rng, 3, hkv), [0, 48, 64])
    err = _append_both(cache, "bf16", n, bs, hkv, [first, second, anew])
    assert err == pagedkv.KV_DEVERR_SLOT_RANGE


@pytest.mark.parametrize("hkv", [1, 3, 8])
def test_copy_and_swap_move_scales(hkv):
    rng = np.random.default_rng(hkv)
    c, s = _random_pool(rng, 9, 16, hkv, "int8")
    d = [torch.from_numpy(a.copy()).cuda() for a in (c, c[::-1].copy(), s, s[::-1].copy())]
    pool = pagedkv.KVPool(d[0], d[1], cache="int8", dtype=torch.float16, k_scales=d[2],
                          v_scales=d[3], scale_per="block")
    want = [t.cpu().clone() for t in d]
    try:
        pool.copy_blocks(R.cuda_i32([[0, 5], [3, 8], [1, 99]]))
        for w in want:
            w[5], w[8] = w[0], w[3]
        host = pool.host_pool(4)
        pool.swap_out(host, R.cuda_i32([[5, 2], [7, 0]]))
        torch.cuda.synchronize()
        for h, w in zip(host, want):
            assert torch.equal(h[2], w[5]) and torch.equal(h[0], w[7])
        pool.swap_in(host, R.cuda_i32([[1, 2], [2, 0]]))
        torch.cuda.synchronize()
        for w in want:
            w[1], w[2] = w[5].clone(), w[7].clone()
        assert all(torch.equal(t.cpu(), w) for t, w in zip(d, want))
        assert pool.get_error() == pagedkv.KV_DEVERR_PAIR_RANGE
    finally:
        pool.close()


def _decode_ref(s, q, sel=None):
    q64 = q.double().numpy()
    return np.stack([R.attention(q64[b:b + 1], s.k, s.v, s.tables[b], int(s.lens[b]),
                                 [int(s.lens[b]) - 1], s.scale)[0] for b in range(len(s.lens))])


@pytest.mark.parametrize("kind", ["fp8_e4m3_block", "int8_block"])
@pytest.mark.parametrize("hq,hkv,bs", [(32, 8, 16), (4, 4, 16), (4, 2, 32), (16, 2, 16), (8, 1, 48),
                                       (8, 2, 128)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_decode(kind, hq, hkv, bs, dtype):
    lens = [0, 1, 15, 16, 17, 31, 32, 33, bs, bs + 1, 3 * bs - 1, 700]
    s = R.Setup(kind, dtype, lens, hq=hq, hkv=hkv, bs=bs, seed=hq + bs)
    q = s.queries(len(lens))
    pool = s.pool()
    try:
        out = pool.decode(q.cuda(), R.cuda_i32(s.tables), R.cuda_i32(lens), s.scale)
        torch.cuda.synchronize()
        assert pool.get_error() == 0
        # the cascade call decodes plainly
        same = pool.decode_cascade(q.cuda(), R.cuda_i32(s.tables), R.cuda_i32(lens), s.scale,
                                   R.cuda_i32([[4, 3, 0]]))
        assert torch.equal(same.view(torch.int16), out.view(torch.int16))
    finally:
        pool.close()
    R.check(out.double().cpu().numpy(), _decode_ref(s, q), dtype, kind)


@pytest.mark.parametrize("kind", ["fp8_e4m3", "int8", "fp8_e4m3_block", "int8_block"])
def test_decode_refuses_blocks_that_do_not_fit(kind):
    """Block size 256: four stages of K and V tiles are 256 KB, more than a CTA's
    shared memory, on every 8-bit pool; the append and the copies still run."""
    s = R.Setup(kind, "bf16", [256, 700], hq=8, hkv=2, bs=256, seed=1)
    q = s.queries(2).cuda()
    pool = s.pool()
    try:
        for call in (pool.decode, pool.decode_scored):
            with pytest.raises(pagedkv.PagedKVError) as e:
                call(q, R.cuda_i32(s.tables), R.cuda_i32(s.lens), s.scale)
            assert e.value.status == pagedkv.KV_EUNSUPPORTED
    finally:
        pool.close()


@pytest.mark.parametrize("kind", ["fp8_e4m3_block", "int8_block"])
def test_decode_split_sequences_and_scale_jumps(kind):
    """Few long sequences (pieces cut across warps and merged), with V scales of
    zero in the first blocks and 100 times larger in one later block."""
    lens = [5000, 1, 3001, 2000]
    s = R.Setup(kind, "bf16", lens, hq=8, hkv=2, bs=16, seed=9)
    for b, L in enumerate(lens):
        nb = -(-L // 16)
        for j, f in ((0, 0.0), (1, 0.0), ((3 * nb) // 5, 100.0)):
            if j < nb and nb > 4:
                blk = s.tables[b, j]
                s.vs[blk] *= f
                s.v[blk] *= f
    q = s.queries(len(lens))
    pool = s.pool()
    try:
        out = pool.decode(q.cuda(), R.cuda_i32(s.tables), R.cuda_i32(lens), s.scale)
        torch.cuda.synchronize()
        assert pool.get_error() == 0
    finally:
        pool.close()
    got, ref = out.double().cpu().numpy(), _decode_ref(s, q)
    # |v| up to 100 times the check's 5: its arithmetic term grows as much
    assert (np.abs(got - ref) <= 5e-2 + 2.0 ** -8 * np.abs(ref)).all()


@pytest.mark.parametrize("kind", ["fp8_e4m3_block", "int8_block"])
@pytest.mark.parametrize("hq,hkv,bs", [(32, 8, 16), (2, 2, 32), (4, 2, 64), (8, 1, 128)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_prefill(kind, hq, hkv, bs, dtype):
    lens, c = [1, 70, 64, 200, 333, 130], [1, 70, 1, 63, 140, 129]
    s = R.Setup(kind, dtype, lens, hq=hq, hkv=hkv, bs=bs, seed=bs)
    q = s.queries(sum(c))
    cu = np.concatenate([[0], np.cumsum(c)])
    pool = s.pool()
    try:
        out = pool.prefill(q.cuda(), R.cuda_i32(cu), max(c), R.cuda_i32(s.tables), R.cuda_i32(lens),
                           s.scale)
        torch.cuda.synchronize()
        assert pool.get_error() == 0
    finally:
        pool.close()
    q64 = q.double().numpy()
    ref = np.concatenate([R.attention(q64[cu[b]:cu[b + 1]], s.k, s.v, s.tables[b], L,
                                      np.arange(L - c[b], L), s.scale) for b, L in enumerate(lens)])
    R.check(out.double().cpu().numpy(), ref, dtype, kind)


def test_ids_outside_the_pool_are_skipped():
    """Bad table entries: their tokens take no part, the error bit is set."""
    lens = [64, 40]
    s = R.Setup("fp8_e4m3_block", "bf16", lens, hq=4, hkv=1, bs=16, seed=3)
    q = s.queries(2)
    ref_k, tab = s.k.copy(), s.tables.copy()
    tab[0, 2], tab[0, 3] = -5, 1 << 20
    pool = s.pool()
    try:
        out = pool.decode(q.cuda(), R.cuda_i32(tab), R.cuda_i32(lens), s.scale)
        torch.cuda.synchronize()
        assert pool.get_error() == pagedkv.KV_DEVERR_BLOCK_RANGE
    finally:
        pool.close()
    q64 = q.double().numpy()
    ref = np.stack([R.attention(q64[:1], ref_k, s.v, s.tables[0], 32, [31], s.scale)[0],
                    R.attention(q64[1:], ref_k, s.v, s.tables[1], 40, [39], s.scale)[0]])
    R.check(out.double().cpu().numpy(), ref, "bf16")


def test_append_captured_and_replayed():
    """A captured append gives the same pool at every replay, small and large,
    whatever order the graphs run in."""
    for t in (40, 1400):
        rng = np.random.default_rng(t)
        n, bs, hkv = t // 16 + 4, 16, 4
        c, sc = _random_pool(rng, n, bs, hkv, "fp8_e4m3")
        d = [torch.from_numpy(a.copy()).cuda() for a in (c, c, sc, sc)]
        pool = pagedkv.KVPool(d[0], d[1], cache="fp8_e4m3", dtype=torch.bfloat16, k_scales=d[2],
                              v_scales=d[3], scale_per="block")
        try:
            k = torch.randn(t, hkv, 128, device="cuda").bfloat16()
            slots = torch.arange(3, 3 + t, device="cuda")
            pool.append(k, k, slots)
            torch.cuda.synchronize()
            want = [x.clone() for x in d]
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                pool.append(k, k, slots)
            for _ in range(3):
                for x, w in zip(d, (c, c, sc, sc)):
                    x.copy_(torch.from_numpy(w))
                g.replay()
                torch.cuda.synchronize()
                assert all(torch.equal(x, w) for x, w in zip(d, want))
            assert pool.get_error() == 0
        finally:
            pool.close()


def test_binding_refusals():
    z = torch.zeros((4, 16, 2, 128), dtype=torch.uint8, device="cuda")
    ok = torch.zeros((4, 2), device="cuda")
    tok = torch.zeros((4, 2, 16), device="cuda")
    for kw in (dict(k_scales=tok, v_scales=tok), dict(k_scales=ok), dict(k_scales=ok, v_scales=ok.half()),
               dict(k_scales=ok, v_scales=ok.cpu())):
        with pytest.raises(ValueError):
            pagedkv.KVPool(z, z, cache="int8", dtype=torch.bfloat16, scale_per="block", **kw)
    with pytest.raises(ValueError):
        pagedkv.KVPool(z, z, cache="int8", dtype=torch.bfloat16, scale_per="row", k_scales=ok, v_scales=ok)
    with pytest.raises(ValueError):
        pagedkv.KVPool(z.half(), z.half(), scale_per="block", k_scales=ok, v_scales=ok)
    pool = pagedkv.KVPool(z, z.clone(), cache="int8", dtype=torch.bfloat16, scale_per="block",
                          k_scales=ok, v_scales=ok.clone())
    try:
        hk, hv, hs, ht = pool.host_pool(2)
        assert hs.shape == (2, 2)
        lib = pagedkv.load()
        p = R.cuda_i32([[0, 0]])
        P = lambda t: ctypes.c_void_p(t.data_ptr())
        assert lib.kv_swap_blocks(pool.handle, P(hk), P(hv), None, None, 2, P(p), 1, 0, None) == \
            pagedkv.KV_EINVAL
    finally:
        pool.close()
