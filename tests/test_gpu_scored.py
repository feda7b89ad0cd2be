"""Scored attention (capped, biased, masked) on the GPU against the 64-bit
restatement: decode and prefill, every pool kind, head grouping and tile path."""

import ctypes

import numpy as np
import pytest
import torch

import plan_oracle
import scored_ref as R
from paged_kv_cache_68_gb300 import pagedkv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pagedkv.load()


def _slopes(hq):
    return np.exp2(-8.0 * np.arange(1, hq + 1) / hq).astype(np.float32)


def _dev_mods(m):
    d = dict(m)
    if d.get("slopes") is not None:
        d["alibi_slopes"] = torch.from_numpy(d.pop("slopes")).cuda()
    else:
        d.pop("slopes", None)
    for k in ("first_visible", "prefix_lens"):
        if d.get(k) is not None:
            d[k] = R.cuda_i32(d[k])
    return d


def _decode(s, mods, lens=None, tables=None, err=0):
    lens = s.lens if lens is None else lens
    q = s.queries(len(lens))
    pool = s.pool()
    try:
        out = pool.decode_scored(q.cuda(), R.cuda_i32(s.tables if tables is None else tables),
                                 R.cuda_i32(lens), s.scale, **_dev_mods(mods))
        torch.cuda.synchronize()
        assert pool.get_error() == err
    finally:
        pool.close()
    q64, first = q.double().numpy(), mods.get("first_visible")
    ref = np.stack([
        R.attention(q64[b:b + 1], s.k, s.v, s.tables[b], int(L), [int(L) - 1], s.scale,
                    softcap=mods.get("softcap", 0), slopes=mods.get("slopes"),
                    window=mods.get("window", 0), first=None if first is None else [first[b]])[0]
        for b, L in enumerate(lens)])
    return out.double().cpu().numpy(), ref


def _all_mods(lens, hq, bs):
    """Each modification alone, then together; first visible positions at block
    edges, inside blocks, past the end (nothing visible) and negative."""
    lens = np.asarray(lens)
    first = np.minimum(lens, np.resize([0, bs - 1, bs, bs + 1, 3, 2 * bs + 5], len(lens)))
    first[-1] = lens[-1] + 3
    first[0] = -4
    s = _slopes(hq)
    return [dict(softcap=5.0), dict(slopes=s), dict(window=1), dict(window=bs), dict(window=bs + 3),
            dict(window=10 ** 9), dict(first_visible=first),
            dict(softcap=30.0, slopes=s, window=2 * bs + 7, first_visible=first), dict()]


@pytest.mark.parametrize("kind,dtype,d,bs", [
    ("plain", "f32", 64, 4), ("plain", "f32", 128, 16), ("plain", "f16", 64, 16),
    ("plain", "bf16", 128, 8), ("plain", "bf16", 128, 16), ("plain", "f16", 128, 32),
    ("plain", "bf16", 128, 24), ("plain", "f16", 128, 1),
    ("fp8_e4m3", "bf16", 128, 16), ("fp8_e4m3", "f16", 128, 64), ("int8", "bf16", 128, 16),
    ("int8", "f16", 128, 32), ("fp8_e4m3_block", "bf16", 128, 16),
    ("fp8_e4m3_block", "f16", 128, 48), ("int8_block", "f16", 128, 16),
    ("int8_block", "bf16", 128, 32)])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (4, 2), (8, 2), (8, 1)])
def test_decode_every_pool(kind, dtype, d, bs, hq, hkv):
    lens = [1, bs - 1 or 1, bs, bs + 1, 2 * bs + 3, 5 * bs, 190, 3 * bs]
    for i, mods in enumerate(_all_mods(lens, hq, bs)):
        s = R.Setup(kind, dtype, lens, hq=hq, hkv=hkv, d=d, bs=bs, seed=i)
        got, ref = _decode(s, mods)
        R.check(got, ref, dtype, f"{kind} {sorted(mods)}")


def test_decode_zero_lengths_and_rows_that_see_nothing():
    lens = [0, 7, 0, 33, 16]
    s = R.Setup("plain", "bf16", lens, hq=4, hkv=1, bs=16, seed=1)
    got, ref = _decode(s, dict(first_visible=np.array([0, 7, 5, 100, 15])))
    assert (got[:4] == 0).all() and (ref[:4] == 0).all()
    R.check(got, ref, "bf16")


@pytest.mark.parametrize("kind,dtype", [("plain", "bf16"), ("plain", "f16"), ("int8", "bf16"),
                                        ("fp8_e4m3_block", "bf16"), ("plain", "f32")])
def test_decode_long_contexts_cut_across_warps(kind, dtype):
    """Few long sequences: pieces merged by the second kernel (few pairs) and in
    the first one (many)."""
    for lens in ([4100, 9000, 2], [700] * 40 + [3000]):
        s = R.Setup(kind, dtype, lens, hq=8, hkv=2, bs=16, seed=2)
        for mods in (dict(softcap=20.0, window=2500), dict(slopes=_slopes(8))):
            got, ref = _decode(s, mods)
            R.check(got, ref, dtype, f"{kind} {sorted(mods)}")


@pytest.mark.parametrize("kind,dtype,bs", [("plain", "bf16", 16), ("plain", "f16", 8),
                                           ("plain", "f32", 16), ("fp8_e4m3", "bf16", 16),
                                           ("fp8_e4m3_block", "f16", 16)])
def test_decode_masked_places_may_hold_nan(kind, dtype, bs):
    """NaN (all-ones codes) in every row before the first visible position,
    the visible block's own leading rows included."""
    lens, first = [100, 64, 90, 33], np.array([37, 48, 89, 17])
    s = R.Setup(kind, dtype, lens, hq=4, hkv=2, bs=bs, seed=4)
    for b in range(4):
        for t in range(first[b]):
            for x in s.dev:
                x[s.tables[b, t // bs], t % bs] = float("nan") if kind == "plain" else 0x7f
    got, ref = _decode(s, dict(first_visible=first, softcap=9.0))
    R.check(got, ref, dtype, kind)


def test_decode_without_mods_is_the_plain_decode():
    """Nothing set: the same sums as paged_attention_decode, bit for bit, on the
    same grid (the cut into pieces is the same)."""
    lens = [1, 40, 700, 16]
    for kind, dtype in (("plain", "bf16"), ("int8", "f16"), ("fp8_e4m3_block", "bf16")):
        s = R.Setup(kind, dtype, lens, hq=8, hkv=2, bs=16, seed=5)
        q = s.queries(4).cuda()
        pool = s.pool()
        try:
            a = pool.decode(q, R.cuda_i32(s.tables), R.cuda_i32(lens), s.scale)
            b = pool.decode_scored(q, R.cuda_i32(s.tables), R.cuda_i32(lens), s.scale)
            assert (a.float() - b.float()).abs().max() <= 2.0 ** -7 * a.float().abs().max()
        finally:
            pool.close()


def test_decode_table_too_short_and_bad_ids():
    lens = [64, 40]
    s = R.Setup("plain", "bf16", lens, hq=4, hkv=1, bs=16, seed=6)
    got, ref = _decode(s, dict(window=20), lens=np.array([64, 80]),
                       tables=np.ascontiguousarray(s.tables[:, :4]), err=pagedkv.KV_DEVERR_SEQ_RANGE | pagedkv.KV_DEVERR_BLOCK_RANGE)
    R.check(got[:1], ref[:1], "bf16")
    # a bad entry before the window is never read
    tab = s.tables.copy()
    tab[0, 0] = -9
    got, ref = _decode(s, dict(window=20), tables=tab)
    R.check(got, ref, "bf16")


# -- prefill -----------------------------------------------------------------------------

def _prefill(s, c, mods, max_q=None, err=0):
    cu = np.concatenate([[0], np.cumsum(c)])
    q = s.queries(int(cu[-1]) + 2)                    # rows behind the last request
    out = torch.full_like(q, 7.0).cuda()
    pool = s.pool()
    m = dict(mods)
    if m.get("first_visible") is not None:            # one per row of the stream
        m["first_visible"] = np.concatenate([m["first_visible"], [0, 0]])
    try:
        pool.prefill_scored(q.cuda(), R.cuda_i32(cu), max_q or max(c), R.cuda_i32(s.tables),
                            R.cuda_i32(s.lens), s.scale, out=out, **_dev_mods(m))
        torch.cuda.synchronize()
        assert pool.get_error() == err
    finally:
        pool.close()
    assert (out[-2:] == 7.0).all()
    q64, first, prefix = q.double().numpy(), mods.get("first_visible"), mods.get("prefix_lens")
    ref = np.concatenate([
        R.attention(q64[cu[b]:cu[b + 1]], s.k, s.v, s.tables[b], int(L),
                    np.arange(int(L) - c[b], int(L)), s.scale, softcap=mods.get("softcap", 0),
                    slopes=mods.get("slopes"), window=mods.get("window", 0),
                    first=None if first is None else first[cu[b]:cu[b + 1]],
                    prefix=0 if prefix is None else int(prefix[b])) for b, L in enumerate(s.lens)])
    return out[:-2].double().cpu().numpy(), ref


def _prefill_mods(lens, c, hq, seed):
    rng = np.random.default_rng(seed)
    lens, c = np.asarray(lens), np.asarray(c)
    first = []
    for L, n in zip(lens, c):
        cuts = np.sort(np.concatenate([[0], rng.integers(0, max(1, L), 3)]))
        p = np.arange(L - n, L)
        f = cuts[np.searchsorted(cuts, p, side="right") - 1]
        f[rng.random(n) < 0.1] = L + 5                 # sees nothing
        first.append(f)
    first = np.concatenate(first)
    prefix = rng.integers(0, lens + 9)
    s = _slopes(hq)
    return [dict(softcap=5.0), dict(slopes=s), dict(window=1), dict(window=70),
            dict(first_visible=first), dict(prefix_lens=prefix),
            dict(prefix_lens=prefix, slopes=s, window=100),
            dict(softcap=30.0, slopes=s, window=90, first_visible=first, prefix_lens=prefix), dict()]


@pytest.mark.parametrize("kind,dtype,bs", [
    ("plain", "bf16", 16), ("plain", "f16", 8), ("plain", "bf16", 128), ("fp8_e4m3", "bf16", 16),
    ("fp8_e4m3", "f16", 32), ("int8", "bf16", 64), ("int8", "f16", 16),
    ("fp8_e4m3_block", "bf16", 16), ("fp8_e4m3_block", "f16", 128), ("int8_block", "f16", 16),
    ("int8_block", "bf16", 32)])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (4, 2), (8, 2), (8, 1)])
def test_prefill_every_pool(kind, dtype, bs, hq, hkv):
    lens, c = [1, 70, 64, 200, 333, 130], [1, 70, 1, 63, 140, 129]
    for i, mods in enumerate(_prefill_mods(lens, c, hq, bs + hq)):
        s = R.Setup(kind, dtype, lens, hq=hq, hkv=hkv, bs=bs, seed=i)
        got, ref = _prefill(s, c, mods)
        R.check(got, ref, dtype, f"{kind} {sorted(mods)}")


def test_prefill_negative_positions_and_empty_requests():
    """More queries than context (their positions are negative), a request with
    no context and one with no queries."""
    lens, c = [3, 0, 90], [9, 4, 0]
    s = R.Setup("plain", "bf16", lens, hq=4, hkv=1, bs=16, seed=7)
    for mods in (dict(softcap=4.0), dict(prefix_lens=np.array([3, 5, 0])), dict(window=2)):
        got, ref = _prefill(s, c, mods)
        assert (got[:6] == 0).all() and (got[9:] == 0).all()
        R.check(got, ref, "bf16")


def test_prefill_windows_skip_whole_tiles():
    """A chunk far behind its window's start: only the window's tiles matter,
    and what lies before them may hold NaN; more requests than the launch order
    ranks."""
    lens, c = [1000, 517], [200, 3]
    s = R.Setup("plain", "f16", lens, hq=4, hkv=1, bs=16, seed=8)
    for b in range(2):
        for t in range(lens[b] - c[b] - 64):
            for x in s.dev:
                x[s.tables[b, t // 16], t % 16] = float("nan")
    got, ref = _prefill(s, c, dict(window=65))
    R.check(got, ref, "f16")
    lens = list(np.random.default_rng(1).integers(1, 40, 300))
    s = R.Setup("plain", "bf16", lens, hq=2, hkv=1, bs=16, seed=9)
    c = [max(1, int(x) // 2) for x in lens]
    got, ref = _prefill(s, c, dict(window=9, slopes=_slopes(2)))
    R.check(got, ref, "bf16")


def test_prefill_of_a_whole_prompt_is_its_chunks():
    """Scored prefill in one chunk and in two gives the same rows (same tiles,
    same order: only the first tile's start may differ with the window)."""
    s = R.Setup("plain", "bf16", [256], hq=8, hkv=2, bs=16, seed=10)
    q = s.queries(256).cuda()
    m = dict(softcap=20.0, alibi_slopes=torch.from_numpy(_slopes(8)).cuda())
    pool = s.pool()
    try:
        t = R.cuda_i32(s.tables)
        one = pool.prefill_scored(q, R.cuda_i32([0, 256]), 256, t, R.cuda_i32([256]), s.scale, **m)
        a = pool.prefill_scored(q[:128], R.cuda_i32([0, 128]), 128, t, R.cuda_i32([128]), s.scale, **m)
        b = pool.prefill_scored(q[128:].contiguous(), R.cuda_i32([0, 128]), 128, t, R.cuda_i32([256]),
                                s.scale, **m)
        d = (torch.cat([a, b]).float() - one.float()).abs()
        assert (d <= 2.0 ** -8 * one.float().abs() + 1e-3).all()
        assert pool.get_error() == 0
    finally:
        pool.close()


# -- as they are used together ---------------------------------------------------------

@pytest.mark.parametrize("cache", ["fp8_e4m3", "int8"])
def test_a_captured_serving_loop(cache):
    """plan -> append -> scored decode on a block-scaled cache, captured once and
    replayed: sequences grow through block boundaries, and every step's output
    equals the restatement's over the same codes."""
    bs, hq, hkv, b, steps = 16, 8, 2, 6, 40
    rng = np.random.default_rng(11)
    n = 80
    codes = [torch.zeros((n, bs, hkv, 128), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros((n, hkv), device="cuda") for _ in range(2)]
    pool = pagedkv.KVPool(*codes, cache=cache, dtype=torch.bfloat16, k_scales=scales[0],
                          v_scales=scales[1], scale_per="block")
    ref = [(np.zeros((n, bs, hkv, 128), np.uint8), np.zeros((n, hkv), np.float32)) for _ in range(2)]
    order = rng.permutation(n).astype(np.int32)
    slopes = _slopes(hq)
    ctx, tables, head = np.zeros(b, np.int64), np.full((b, 8), -1, np.int32), 0
    d_ctx, d_new, d_tab = R.cuda_i32(ctx), R.cuda_i32(np.ones(b)), R.cuda_i32(tables)
    d_free, d_head = R.cuda_i32(order), R.cuda_i32([0])
    q = torch.zeros((b, hq, 128), dtype=torch.bfloat16, device="cuda")
    k, v = (torch.zeros((b, hkv, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws, d_sl = pool.scored_workspace(b, hq), torch.from_numpy(slopes).cuda()
    plan = pool.plan_step(d_ctx, R.cuda_i32(np.zeros(b)), d_tab, d_free, d_head, b)
    out = torch.empty_like(q)
    mods = dict(softcap=20.0, window=19)

    def step():
        pool.plan_step(d_ctx, d_new, d_tab, d_free, d_head, b, out=plan)
        pool.append(k, v, plan.slot_mapping)
        pool.decode_scored(q, d_tab, plan.seq_lens, 0.09, alibi_slopes=d_sl, out=out, workspace=ws,
                           **mods)
        d_ctx.copy_(plan.seq_lens)
        d_head.copy_(plan.free_head)

    try:
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        for i in range(steps):
            x = [torch.from_numpy((rng.standard_normal(t.shape) * gain).astype(np.float32)).bfloat16()
                 for t, gain in ((q, 1), (k, 1 + i % 3), (v, 1))]
            for t, y in zip((q, k, v), x):
                t.copy_(y)
            g.replay()
            torch.cuda.synchronize()
            tables, _, lens, slots, _, head, err = plan_oracle.plan_step(
                ctx, np.ones(b, np.int64), tables, order, head, b, bs, n)
            assert err == 0 and plan.slot_mapping.tolist() == slots.tolist()
            for (c, s), y in zip(ref, x[1:]):
                R.append_block_scaled(c, s, y.float().numpy(), slots, cache)
            kv = [R.values(c, cache) * s[:, None, :, None].astype(np.float64) for c, s in ref]
            want = np.stack([R.attention(x[0][r:r + 1].double().numpy(), kv[0], kv[1], tables[r],
                                         int(lens[r]), [int(lens[r]) - 1], 0.09, slopes=slopes,
                                         **mods)[0] for r in range(b)])
            R.check(out.double().cpu().numpy(), want, "bf16", f"step {i}")
            ctx = lens.astype(np.int64)
        assert pool.get_error() == 0
    finally:
        pool.close()


@pytest.mark.parametrize("scored", [False, True])
def test_replayed_decode_merges_its_pieces(scored):
    """Long sequences whose pieces are merged by the warp that finishes last:
    every replay of one captured decode gives the first call's result for its
    own inputs."""
    lens = [900] * 160
    s = R.Setup("plain", "bf16", lens, hq=16, hkv=8, bs=16, seed=12)
    q = s.queries(len(lens)).cuda()
    t, n = R.cuda_i32(s.tables), R.cuda_i32(lens)
    pool = s.pool()
    try:
        assert pagedkv.paged_attention_decode_launches(pool.handle, len(lens), 16) == 1
        out = torch.empty_like(q)
        call = (lambda: pool.decode_scored(q, t, n, s.scale, softcap=30.0, out=out)) if scored else \
            (lambda: pool.decode(q, t, n, s.scale, out=out))
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        for i in range(3):
            q.copy_(torch.randn(q.shape, device="cuda"))
            out.fill_(9.0)
            g.replay()
            torch.cuda.synchronize()
            got = out.clone()
            call()
            assert torch.equal(got, out), f"replay {i}"
        assert pool.get_error() == 0
    finally:
        pool.close()


def test_another_stream():
    s = R.Setup("plain", "bf16", [100, 30], hq=4, hkv=1, bs=16, seed=13)
    q = s.queries(2).cuda()
    t, n = R.cuda_i32(s.tables), R.cuda_i32(s.lens)
    pool = s.pool()
    try:
        want = pool.decode_scored(q, t, n, s.scale, window=17)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        got = pool.decode_scored(q, t, n, s.scale, window=17, stream=st)
        pre = pool.prefill_scored(q, R.cuda_i32([0, 1, 2]), 1, t, n, s.scale, window=17, stream=st)
        st.synchronize()
        assert torch.equal(got, want)
        assert (pre.float() - want.float()).abs().max() <= 2.0 ** -7
    finally:
        pool.close()


@pytest.mark.parametrize("block", [False, True])
def test_wait_limit_reports_a_timeout(block):
    """A limit of 0 makes a wait that does not find its tile give up (tiles come
    from HBM at this size, so many do): the call returns, the bit is set, and the
    next call with the default limit is right again."""
    b, L, hkv, hq = 64, 2000, 8, 16
    n = b * (L // 16)
    shape = (n, 16, hkv, 128)
    if block:
        d = [torch.randint(0, 0x70, shape, dtype=torch.uint8, device="cuda") for _ in range(2)]
        sc = torch.full((n, hkv), 0.01, device="cuda")
        pool = pagedkv.KVPool(*d, cache="fp8_e4m3", dtype=torch.bfloat16, k_scales=sc, v_scales=sc,
                              scale_per="block")
    else:
        pool = pagedkv.KVPool(*(torch.randn(shape, device="cuda").bfloat16() for _ in range(2)))
    q = torch.randn((b, hq, 128), device="cuda").bfloat16()
    t = torch.randperm(n, device="cuda").int().view(b, -1)
    lens = torch.full((b,), L, dtype=torch.int32, device="cuda")
    cu = torch.arange(b + 1, device="cuda").int()
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    try:
        dec = lambda: pool.decode_scored(q, t, lens, 0.1, softcap=9.0)
        pre = lambda: pool.prefill_scored(q, cu, 1, t, lens, 0.1, softcap=9.0)
        for call in (dec, pre):
            want = call().clone()
            assert pool.get_error() == 0
            flush.zero_()
            pool.set_wait_limit(0)
            call()
            torch.cuda.synchronize()
            assert pool.get_error() == pagedkv.KV_DEVERR_TIMEOUT
            pool.clear_error()
            pool.set_wait_limit(2 * 10 ** 9)
            assert torch.equal(call(), want)
            assert pool.get_error() == 0
    finally:
        pool.close()


def test_refusals():
    s = R.Setup("plain", "bf16", [20, 5], hq=4, hkv=2, bs=16, seed=15)
    q = s.queries(2).cuda()
    t, n, cu = R.cuda_i32(s.tables), R.cuda_i32(s.lens), R.cuda_i32([0, 1, 2])
    ws = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")
    lib = pagedkv.load()
    pool = s.pool()
    P = lambda x: ctypes.c_void_p(x.data_ptr())
    try:
        def dec(mods, wb=1 << 24, tables=t, width=3):
            return lib.paged_attention_decode_scored(
                pool.handle, P(q), P(q.clone()), P(tables), width, P(n), 2, 4, 0.1, 2,
                None if mods is None else ctypes.byref(mods), P(ws), wb, None)

        def pre(mods):
            return lib.paged_attention_prefill_scored(
                pool.handle, P(q), P(q.clone()), P(cu), 2, 1, P(t), int(t.shape[1]), P(n), 2, 4, 0.1, 2,
                None if mods is None else ctypes.byref(mods), None)

        M = pagedkv.ScoreMods
        for call in (dec, pre):
            assert call(M()) == pagedkv.KV_OK
            for bad in (None, M(softcap=-1.0), M(softcap=float("nan")), M(softcap=float("inf")),
                        M(window=-1), M(alibi_slopes=n.data_ptr() + 2), M(first_visible=n.data_ptr() + 1),
                        M(prefix_lens=n.data_ptr() + 2)):
                assert call(bad) == pagedkv.KV_EINVAL
        assert dec(M(prefix_lens=n.data_ptr())) == pagedkv.KV_EINVAL
        assert dec(M(), wb=16) == pagedkv.KV_ENOWORKSPACE
        assert dec(M(), width=1 << 28) == pagedkv.KV_EINVAL
        torch.cuda.synchronize()
        f = torch.zeros(4, device="cuda")
        for kw in (dict(alibi_slopes=f[:3]), dict(alibi_slopes=f.half()), dict(first_visible=n[:1]),
                   dict(first_visible=n.long()), dict(alibi_slopes=f.cpu()),
                   dict(out=torch.empty(1, 4, 128, dtype=torch.bfloat16, device="cuda"))):
            with pytest.raises(ValueError):
                pool.decode_scored(q, t, n, s.scale, **kw)
        with pytest.raises(ValueError):
            pool.prefill_scored(q, cu, 1, t, n, s.scale, prefix_lens=n[:1])
        with pytest.raises(ValueError):
            pool.decode_scored(q, t[:1], n, s.scale)
        # fp32 prefill is not built, scored or not
        s32 = R.Setup("plain", "f32", [20, 5], hq=4, hkv=2, bs=16, seed=16)
        p32 = s32.pool()
        try:
            with pytest.raises(pagedkv.PagedKVError) as e:
                p32.prefill_scored(q.float(), cu, 1, t, n, s.scale, softcap=1.0)
            assert e.value.status == pagedkv.KV_EUNSUPPORTED
        finally:
            p32.close()
    finally:
        pool.close()
