"""The step plan on the GPU: every array equal to the plain restatement's."""

import ctypes

import numpy as np
import pytest
import torch

import plan_oracle
from paged_kv_cache_68_gb300 import pagedkv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pagedkv.load()


def _pool(num_blocks, bs):
    k = torch.zeros((num_blocks, bs, 1, 64), dtype=torch.float16, device="cuda")
    return pagedkv.KVPool(k, torch.zeros_like(k))


def _cuda_i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _check(ctx, new, bs, *, width=None, num_free=None, head=0, cap=None, num_blocks=None, bad=None):
    ctx, new = np.asarray(ctx, np.int64), np.asarray(new, np.int64)
    rng = np.random.default_rng(len(ctx) * 31 + bs)
    old = -(-np.maximum(ctx, 0) // bs)
    full = -(-(np.maximum(ctx, 0) + np.maximum(new, 0)) // bs)
    width = int(max(1, full.max()) + 2) if width is None else width
    need = int((full - old).sum())
    num_free = need + 5 + head if num_free is None else num_free
    n = int(np.minimum(old, width).sum()) + num_free + 1
    perm = rng.permutation(n).astype(np.int32)
    tables = np.full((len(ctx), width), -7, np.int32)
    used = 0
    for r in range(len(ctx)):
        k = min(int(old[r]), width)
        tables[r, :k] = perm[used:used + k]
        used += k
    free = perm[used:used + num_free].copy()
    if bad is not None:
        bad(tables, free)
    total = int(np.maximum(new, 0).sum())
    cap = total + 5 if cap is None else cap
    want = plan_oracle.plan_step(ctx, new, tables, free, head, cap, bs, n)
    pool = _pool(n, bs)
    try:
        t = _cuda_i32(tables)
        got = pool.plan_step(_cuda_i32(ctx), _cuda_i32(new), t, _cuda_i32(free), _cuda_i32([head]), cap)
        torch.cuda.synchronize()
        err = pool.get_error()
    finally:
        pool.close()
    assert np.array_equal(t.cpu().numpy(), want[0])
    assert np.array_equal(got.cu_seqlens.cpu().numpy(), want[1])
    assert np.array_equal(got.seq_lens.cpu().numpy(), want[2])
    assert np.array_equal(got.slot_mapping.cpu().numpy(), want[3])
    assert np.array_equal(got.positions.cpu().numpy(), want[4])
    assert int(got.free_head) == want[5]
    assert err == want[6], (hex(err), hex(want[6]))


@pytest.mark.parametrize("bs", [1, 7, 16, 128, 256])
@pytest.mark.parametrize("batch", [1, 2, 31, 257, 1025, 4096])
def test_decode_steps(batch, bs):
    rng = np.random.default_rng(batch + bs)
    ctx = rng.integers(0, 5 * bs, batch)
    ctx[0] = 0
    _check(ctx, np.ones(batch, np.int64), bs, head=2)


@pytest.mark.parametrize("bs", [1, 16, 64])
@pytest.mark.parametrize("batch,most", [(1, 1), (1, 5000), (3, 17), (100, 300), (1500, 40)])
def test_mixed_steps(batch, most, bs):
    """Prompts, single tokens and waiting requests; more tokens than one CTA places."""
    rng = np.random.default_rng(batch * 7 + bs)
    new = rng.integers(0, most + 1, batch)
    new[rng.random(batch) < 0.3] = 0
    new[-1] = most
    _check(rng.integers(0, 3 * bs + 1, batch), new, bs)


def test_large_step():
    rng = np.random.default_rng(5)
    _check(rng.integers(0, 100, 300), rng.integers(0, 3000, 300), 16)


def test_waiting_and_empty_steps():
    _check([0, 5, 16], [0, 0, 0], 16)
    _check([0, 5, 16], [0, 0, 0], 16, cap=0)
    _check([0], [1], 16, cap=1)


def test_requests_that_cannot_be_placed():
    # the free list ends inside the second request; a later one without need goes on
    _check([0, 0, 3, 0], [16, 40, 2, 1], 16, num_free=2)
    _check([0, 0], [16, 1], 16, num_free=0)
    # past the table row, past the token arrays, negative lengths, a head out of range
    _check([30, 3, 0], [10, 1, 4], 8, width=4)
    _check([0, 0, 5], [9, 9, 1], 8, cap=12)
    _check([-3, 4, 2], [5, -1, 2], 8)
    _check([4, 4], [5, 1], 8, head=-2, num_free=9)
    _check([4, 4], [5, 1], 8, head=12, num_free=9)


def test_ids_outside_the_pool():
    def bad(tables, free):
        tables[0, 0] = -1
        tables[2, 0] = 1 << 30
        free[1] = 1 << 29
    _check([3, 8, 5], [2, 9, 1], 8, bad=bad)


def test_captured_step_grows_its_sequences():
    """A captured plan, replayed with its results fed back, walks a batch of
    sequences through block boundaries like the restatement does."""
    bs, b, width = 4, 9, 12
    rng = np.random.default_rng(3)
    order = rng.permutation(100).astype(np.int32)
    ctx = np.zeros(b, np.int64)
    tables, head = np.full((b, width), -1, np.int32), 0
    pool = _pool(100, bs)
    try:
        d_ctx, d_new, d_tab = _cuda_i32(ctx), _cuda_i32(np.ones(b)), _cuda_i32(tables)
        d_free, d_head = _cuda_i32(order), _cuda_i32([0])
        out = pool.plan_step(d_ctx, d_new, d_tab, d_free, d_head, b)     # warm-up, then undone
        d_tab.fill_(-1)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pool.plan_step(d_ctx, d_new, d_tab, d_free, d_head, b, out=out)
            d_ctx.copy_(out.seq_lens)
            d_head.copy_(out.free_head)
        for _ in range(11):
            g.replay()
            tables, _, lens, slots, pos, head, err = plan_oracle.plan_step(
                ctx, np.ones(b, np.int64), tables, order, head, b, bs, 100)
            torch.cuda.synchronize()
            assert err == 0 and np.array_equal(out.slot_mapping.cpu().numpy(), slots)
            assert np.array_equal(d_tab.cpu().numpy(), tables) and int(d_head) == head
            ctx = lens.astype(np.int64)
        assert pool.get_error() == 0
    finally:
        pool.close()


def test_another_stream():
    pool = _pool(50, 8)
    try:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        t = _cuda_i32(np.full((2, 4), -1))
        args = (_cuda_i32([0, 0]), _cuda_i32([9, 3]), t, _cuda_i32(np.arange(50)), _cuda_i32([0]))
        s.wait_stream(torch.cuda.current_stream())
        out = pool.plan_step(*args, 12, stream=s)
        s.synchronize()
        assert out.slot_mapping.tolist() == list(range(9)) + [16, 17, 18]
    finally:
        pool.close()


def test_refusals():
    pool = _pool(8, 8)
    lib = pagedkv.load()
    try:
        z = torch.zeros(64, dtype=torch.int32, device="cuda")
        at = lambda k: ctypes.c_void_p(z.data_ptr() + 4 * k)
        sl = torch.zeros(8, dtype=torch.int64, device="cuda")
        good = [pool.handle, at(0), at(1), 1, at(2), 4, at(8), 8, at(16), at(17), at(20), at(24),
                ctypes.c_void_p(sl.data_ptr()), at(32), 8, None]

        def call(**kw):
            a = list(good)
            for k, v in kw.items():
                a[int(k[1:])] = v
            return lib.kv_plan_step(*a)

        for k in (0, 1, 2, 4, 6, 8, 9, 10, 11, 12):
            assert call(**{f"a{k}": None}) == pagedkv.KV_EINVAL, k
        assert call(a3=0) == pagedkv.KV_EINVAL and call(a3=4097) == pagedkv.KV_EUNSUPPORTED
        assert call(a5=0) == pagedkv.KV_EINVAL and call(a5=1 << 29) == pagedkv.KV_EINVAL
        assert call(a7=-1) == pagedkv.KV_EINVAL and call(a14=-1) == pagedkv.KV_EINVAL
        assert call(a9=at(16)) == pagedkv.KV_EINVAL                      # head in place
        assert call(a11=at(0)) == pagedkv.KV_EINVAL                      # lengths in place
        assert call(a1=ctypes.c_void_p(z.data_ptr() + 2)) == pagedkv.KV_EINVAL
        assert call(a12=ctypes.c_void_p(sl.data_ptr() + 4)) == pagedkv.KV_EINVAL
        assert call(a13=None) == pagedkv.KV_OK                           # positions are optional
        torch.cuda.synchronize()
        i = _cuda_i32
        ok = (i([0]), i([1]), i([[0, 0]]), i([1, 2]), i([0]), 1)
        for k, wrong in ((0, i([0]).long()), (1, i([1, 1])), (2, i([0, 0])), (4, i([0, 0])),
                         (3, torch.zeros(2, dtype=torch.int32))):
            with pytest.raises(ValueError):
                pool.plan_step(*[wrong if n == k else a for n, a in enumerate(ok)])
    finally:
        pool.close()
