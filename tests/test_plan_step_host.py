"""The step plan's restatement against the block manager, and its refusals (no GPU)."""

import numpy as np
import pytest

import plan_oracle
from paged_kv_cache_68_gb300.block_manager import BlockManager


@pytest.mark.parametrize("bs", [1, 4, 16])
def test_plan_oracle_equals_the_block_manager(bs):
    """Steps of mixed prompts and single tokens: tables, slots and the free
    list's order are those of the host block manager (first in, first out)."""
    rng = np.random.default_rng(bs)
    n_blocks, b, width = 400, 7, 60
    order = rng.permutation(n_blocks).astype(np.int32)
    bm = BlockManager(n_blocks, bs, free_order=order)
    tables = np.full((b, width), -1, np.int32)
    ctx, head = np.zeros(b, np.int64), 0
    for r in range(b):
        bm.allocate_prompt(r, 0)
    for step in range(6):
        new = rng.integers(0, 9, b) if step % 2 else np.ones(b, np.int64)
        want = []
        for r in range(b):
            for _ in range(int(new[r])):
                want.append(bm.append_slot(r)[0])
        t, cu, lens, slots, pos, head, err = plan_oracle.plan_step(
            ctx, new, tables, order, head, int(new.sum()) + 3, bs, n_blocks)
        assert err == 0 and head == n_blocks - bm.num_free()
        assert slots[:len(want)].tolist() == want and (slots[len(want):] == -1).all()
        for r in range(b):
            assert t[r, :len(bm.table(r))].tolist() == bm.table(r)
        assert (np.diff(cu) == new).all() and (lens == ctx + new).all()
        tables, ctx = t, lens.astype(np.int64)


def test_plan_step_refuses_a_null_pool():
    from paged_kv_cache_68_gb300 import pagedkv
    lib = pagedkv.load()
    assert lib.kv_plan_step(None, None, None, 1, None, 1, None, 0, None, None, None, None, None,
                            None, 0, None) == pagedkv.KV_EINVAL
