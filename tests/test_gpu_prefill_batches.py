"""Prefill over batches of every size that orders its requests in its own way:
within a warp (up to 32), in shared memory (up to 256), not at all (above), with
requests that have no queries, no tokens, or tie in length."""

import numpy as np
import pytest
import torch

import scored_ref as R
from paged_kv_cache_68_gb300 import pagedkv
from test_gpu_scored import _prefill

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pagedkv.load()


@pytest.mark.parametrize("kind,dtype", [("plain", "bf16"), ("plain", "f16"), ("fp8_e4m3_block", "bf16")])
@pytest.mark.parametrize("batch", [1, 2, 31, 32, 33, 255, 256, 257])
def test_every_way_of_ordering(batch, kind, dtype):
    rng = np.random.default_rng(batch)
    lens = rng.integers(1, 150, batch)
    lens[rng.random(batch) < 0.2] = 64                # ties
    c = np.minimum(lens, rng.integers(0, 40, batch))
    c[-1] = lens[-1] = max(1, lens[-1])               # a whole prompt, two tile pairs at 8 heads
    lens[c == 0] = rng.integers(0, 2, (c == 0).sum())
    first = np.concatenate([rng.integers(0, L + 1, n) for L, n in zip(lens, c)])
    for mods in (dict(), dict(window=33), dict(softcap=20.0, first_visible=first)):
        s = R.Setup(kind, dtype, lens, hq=8, hkv=1, bs=16, seed=batch)
        got, ref = _prefill(s, [int(n) for n in c], mods)
        R.check(got, ref, dtype, f"{batch} {kind} {sorted(mods)}")
