"""Cases of the step-plan, block-scaled cache and masked / capped attention operators.

Four operators of a serving step over a paged KV cache:

* ``plan``     block tables, slot mapping, positions, offsets and lengths of one
               step, built on the GPU from the requests' lengths
               (``KVPool.plan_step``);
* ``append``   new K/V rows quantised into an 8-bit pool with one scale for each
               (block, KV head) (``KVPool.append`` on such a pool);
* ``decode``   one query per sequence, scores capped by a tanh, biased by
               distance, limited to a window or to the query's document, on any
               kind of pool (``KVPool.decode`` / ``KVPool.decode_scored``);
* ``prefill``  the same for several queries per request, with a prefix mask too
               (``KVPool.prefill`` / ``KVPool.prefill_scored``).

``own`` false: each operator in elementary torch operations, in 32 bits.  ``own``
true: the library's calls.  ``exact`` gives the same outputs from the definitions
in 64 bits.
"""

import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_QMAX = {"fp8_e4m3": 448.0, "int8": 127.0}
_TINY = 2.0 ** -126          # scales below the smallest normal fp32 count as zero


# -- cases -----------------------------------------------------------------------

def _attn(op, name=None, **kw):
    c = dict(op=op, dtype="bf16", pool="plain", hq=32, hkv=8, d=128, bs=16, batch=64, lens=1,
             median=1024, most=8192, softcap=0.0, alibi=False, window=0, docs=0)
    if op == "prefill":
        c.update(chunk=256, prefix=0.0)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # a decode step's bookkeeping: every running request adds one token
        dict(name="plan decode 256", op="plan", batch=256, bs=16, kind="decode", median=1024,
             most=8192, lens=1),
        # a large mixed step: long new prompts beside running requests
        dict(name="plan prompts 1000", op="plan", batch=1000, bs=16, kind="prompt", median=300,
             most=4000, lens=2),
        # one decode step's rows into an FP8 cache
        dict(name="append fp8 decode 256", op="append", cache="fp8_e4m3", dtype="bf16", tokens=256,
             runs=256, hkv=8, bs=16, lens=3),
        # prompt chunks of 17 requests into an INT8 cache
        dict(name="append int8 chunks 8191", op="append", cache="int8", dtype="bf16", tokens=8191,
             runs=17, hkv=8, bs=16, lens=4),
        # a large serving batch on an FP8 cache with block scales
        _attn("decode", "decode fp8 blocks 256", pool="fp8_e4m3_block", batch=256, lens=5),
        # a handful of sequences, capped and windowed, INT8 cache with block scales
        _attn("decode", "decode int8 blocks cap 4", pool="int8_block", dtype="f16", hq=16, hkv=2,
              bs=32, batch=4, median=700, most=2000, softcap=30.0, window=512, lens=6),
        # multi-head model whose scores fall with distance
        _attn("decode", "decode f16 distance 33", dtype="f16", hq=40, hkv=40, batch=33, median=600,
              most=2048, alibi=True, lens=7),
        # few long contexts, capped scores, a window over the last tokens
        _attn("decode", "decode long capped 8", batch=8, median=40000, most=65536, softcap=50.0,
              window=32768, lens=8),
        # small fp32 model with packed documents
        _attn("decode", "decode f32 documents 5", dtype="f32", hq=4, hkv=4, d=64, bs=4, batch=5,
              median=50, most=200, docs=3, lens=9),
        # prompt chunks behind cached prefixes, capped scores
        _attn("prefill", "prefill capped 16x512", batch=16, chunk=512, median=1500, most=4096,
              softcap=50.0, lens=10),
        # prompts whose first part is seen by every token, scores falling with distance
        _attn("prefill", "prefill prefix distance 7", dtype="f16", hq=16, hkv=8, bs=32, batch=7,
              chunk=333, median=400, most=700, alibi=True, prefix=0.5, lens=11),
        # packed documents in a window, on the block-scaled FP8 cache
        _attn("prefill", "prefill fp8 blocks docs 9", pool="fp8_e4m3_block", batch=9, chunk=900,
              median=1500, most=3000, docs=5, window=600, lens=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "decode", "decode", "prefill", "prefill"])
    lens = rng.randrange(1, 1 << 20)
    if op == "plan":
        kind = rng.choice(["decode", "prompt", "mixed"])
        batch = _log(rng, 1, 4096 if kind == "decode" else 1000)
        most = _log(rng, 16, 8000 if kind == "decode" else 4000)
        return dict(op=op, batch=batch, bs=rng.choice([8, 16, 16, 32, 64, 128]), kind=kind,
                    median=max(1, most // rng.choice([3, 5, 8, 13])), most=most, lens=lens)
    if op == "append":
        tokens = _log(rng, 1, 8191)
        hkv = rng.choice([1, 2, 4, 5, 8])
        return dict(op=op, cache=rng.choice(["fp8_e4m3", "int8"]), dtype=rng.choice(["bf16", "f16"]),
                    tokens=tokens, runs=rng.choice([1, min(tokens, 7), max(1, tokens // 9), tokens]),
                    hkv=hkv, bs=rng.choice([16, 16, 32, 48, 64]), lens=lens)
    soft = rng.choice([0.0, 0.0, 15.0, 30.0, 50.0])
    alibi = rng.random() < 0.35
    if op == "decode":
        pool = rng.choice(["plain", "plain", "fp8_e4m3", "int8", "fp8_e4m3_block", "int8_block"])
        if pool == "plain":
            dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
            d = rng.choice([64, 128, 128])
            bs = rng.choice([4, 8, 16, 16, 32, 24])
        else:
            dtype, d, bs = rng.choice(["f16", "bf16"]), 128, rng.choice([16, 16, 32, 64])
        hkv = rng.choice([1, 2, 4, 8, 8, 10])
        hq = hkv * rng.choice([1, 2, 4, 4, 8])
        batch = _log(rng, 1, 200)
        top = min(8000, 6000 * 64 // batch)
        most = _log(rng, 16, top)
        window = rng.choice([0, 0, _log(rng, 1, most)])
        docs = rng.choice([0, 0, 1, 4])
        return _attn(op, dtype=dtype, pool=pool, hq=hq, hkv=hkv, d=d, bs=bs, batch=batch,
                     median=max(1, most // rng.choice([2, 4, 8])), most=most, softcap=soft,
                     alibi=alibi, window=window, docs=docs, lens=lens)
    pool = rng.choice(["plain", "plain", "fp8_e4m3", "int8", "fp8_e4m3_block", "int8_block"])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 8])
    hq, hkv = min(hq, 32), min(hkv, 32)
    batch = _log(rng, 1, 16)
    most = _log(rng, 16, 4000)
    chunk = min(most, _log(rng, 1, 900))
    window = rng.choice([0, 0, _log(rng, 1, most)])
    return _attn(op, dtype=rng.choice(["f16", "bf16"]), pool=pool, hq=hq, hkv=hkv,
                 bs=rng.choice([16, 16, 32, 64, 128]), batch=batch, chunk=chunk,
                 median=max(1, most // 3), most=most, softcap=soft, alibi=alibi, window=window,
                 docs=rng.choice([0, 0, 2, 6]), prefix=rng.choice([0.0, 0.0, 0.3, 0.8]), lens=lens)


# -- what a case's requests look like (from the case alone) ------------------------

def _lengths(case):
    """Context lengths including this step's tokens, and (prefill) queries per request."""
    r = np.random.RandomState(case["lens"] % (1 << 31))
    b, most, med = case["batch"], case["most"], case["median"]
    total = np.clip(np.exp(np.log(med) + 0.8 * r.randn(b)), 1, most).astype(np.int64)
    if case["op"] == "prefill":
        c = np.minimum(total, case["chunk"])
        if b > 2:                                   # ragged last chunks, one single token
            c[1::3] = np.maximum(1, c[1::3] - r.randint(0, max(1, case["chunk"] // 2), c[1::3].shape))
            c[2] = 1
        return total, c
    return total, np.ones(b, np.int64)


def _plan_lengths(case):
    r = np.random.RandomState(case["lens"] % (1 << 31))
    b, most, med = case["batch"], case["most"], case["median"]
    ln = np.clip(np.exp(np.log(med) + 0.8 * r.randn(b)), 1, most).astype(np.int64)
    if case["kind"] == "decode":
        return ln, np.ones(b, np.int64)
    new = ln.copy()
    ctx = np.where(r.rand(b) < 0.3, r.randint(0, most, b), 0).astype(np.int64)
    if case["kind"] == "mixed":
        dec = r.rand(b) < 0.6
        new = np.where(dec, 1, new)
        ctx = np.where(dec, ln, ctx)
        new[r.rand(b) < 0.05] = 0                   # a request that waits this step
    return ctx, new


def _visible(case):
    """first_visible and prefix_lens of a case's queries (numpy, or None each)."""
    total, c = _lengths(case)
    r = np.random.RandomState((case["lens"] * 7 + 3) % (1 << 31))
    if case["op"] == "decode":
        if not case["docs"]:
            return None, None
        first = np.array([0 if r.rand() < 0.3 else r.randint(0, t) for t in total], np.int64)
        if case["batch"] > 3:
            first[3] = total[3]                     # nothing is visible: the row is zero
        return first, None
    first = None
    if case["docs"]:
        rows = []
        for t, n in zip(total, c):
            starts = np.sort(np.concatenate([[0], r.randint(0, max(1, t), case["docs"])]))
            pos = np.arange(t - n, t)
            f = starts[np.searchsorted(starts, pos, side="right") - 1]
            if n > 8:
                f[n // 2] = pos[n // 2] + 1         # a padding token: it sees nothing
            rows.append(f)
        first = np.concatenate(rows)
    prefix = None
    if case["prefix"]:
        prefix = np.floor(total * case["prefix"] * r.rand(len(total))).astype(np.int64) + (total > 3)
    return first, prefix


def _spans(case):
    """Per query (flattened): request, position, first and last visible position."""
    total, c = _lengths(case)
    first, prefix = _visible(case)
    req = np.repeat(np.arange(len(c)), c)
    start = np.concatenate([[0], np.cumsum(c)])[:-1]
    pos = np.arange(int(c.sum())) - start[req] + (total - c)[req]
    lo = np.zeros_like(pos)
    if case["window"]:
        lo = np.maximum(lo, pos - case["window"] + 1)
    if first is not None:
        lo = np.maximum(lo, first)
    hi = pos.copy()
    if prefix is not None:
        hi = np.maximum(hi, np.minimum(prefix, total)[req] - 1)
    return req, pos, lo, hi


# -- inputs --------------------------------------------------------------------------

def _gen(seed, device="cuda"):
    return torch.Generator(device=device).manual_seed(int(seed))


def _tables(lens, bs, seed):
    """Block tables of contexts `lens` over a scattered pool: (tables, blocks in the pool)."""
    nb = -(-np.asarray(lens) // bs)
    used = int(nb.sum())
    n = max(2, used + used // 8 + 1)
    perm = np.random.RandomState(seed % (1 << 31)).permutation(n)[:used].astype(np.int32)
    width = max(1, int(nb.max()))
    t = np.full((len(nb), width), -1, np.int32)
    t[np.arange(width)[None, :] < nb[:, None]] = perm
    return t, n


def _fill_pool(case, n, g):
    """K and V of a pool of n blocks: (k, v, k_scales, v_scales, k_scale, v_scale)."""
    dev, bs, h, d = "cuda", case["bs"], case["hkv"], case["d"]
    shape = (n, bs, h, d)
    if case["pool"] == "plain":
        dt = _DT[case["dtype"]]
        return tuple(torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(dt)
                     for _ in range(2)) + (None, None, 1.0, 1.0)
    block = case["pool"].endswith("_block")
    codes = []
    for _ in range(2):
        if case["pool"].startswith("fp8"):
            x = torch.randn(shape, generator=g, device=dev) * (100.0 if block else 1.0)
            codes.append(x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
        else:
            codes.append(torch.randint(-127, 128, shape, generator=g, device=dev, dtype=torch.int8)
                         .view(torch.uint8))
    if case["pool"] == "fp8_e4m3":
        return codes[0], codes[1], None, None, 0.75, 1.25
    sshape = (n, h) if block else (n, h, bs)
    unit = 1.0 / 100.0 if case["pool"].startswith("fp8") else 1.0 / 64.0
    sc = [unit * torch.exp(0.4 * torch.randn(sshape, generator=g, device=dev)) for _ in range(2)]
    return codes[0], codes[1], sc[0], sc[1], 1.0, 1.0


def _handle(state, k, v, pool, dtype, ks, vs, k_scale, v_scale):
    from paged_kv_cache_68_gb300 import pagedkv
    if pool == "plain":
        return pagedkv.KVPool(k, v)
    kw = dict(cache="fp8_e4m3" if pool.startswith("fp8") else "int8", dtype=dtype)
    if pool.endswith("_block"):
        return pagedkv.KVPool(k, v, k_scales=ks, v_scales=vs, scale_per="block", **kw)
    return pagedkv.KVPool(k, v, k_scales=ks, v_scales=vs, k_scale=k_scale, v_scale=v_scale, **kw)


def _prepare_plan(case, seed):
    ctx, new = _plan_lengths(case)
    bs, b = case["bs"], case["batch"]
    old = -(-ctx // bs)
    full = -(-(ctx + new) // bs)
    width = int(max(1, full.max()) + 2)
    n = int(full.sum()) + 64
    perm = np.random.RandomState(seed % (1 << 31)).permutation(n).astype(np.int32)
    t = np.full((b, width), -1, np.int32)
    t[np.arange(width)[None, :] < old[:, None]] = perm[:int(old.sum())]
    free = perm[int(old.sum()):]
    cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    total = int(new.sum())
    cap = total + (-total) % 64 if case["kind"] != "prompt" else total   # padded for a captured step
    st = dict(case=case, ctx=cuda(ctx.astype(np.int32)), new=cuda(new.astype(np.int32)),
              tables=cuda(t), free=cuda(free), head=torch.full((1,), 3, dtype=torch.int32, device="cuda"),
              cap=max(1, cap))
    if own:
        # a pool to plan for: the plan reads its geometry only, so one head of 64 fp16 values does
        k = torch.empty((n, bs, 1, 64), dtype=torch.float16, device="cuda")
        st["pool"] = _handle(st, k, torch.empty_like(k), "plain", None, None, None, 1.0, 1.0)
    return st


def _prepare_append(case, seed):
    """`runs` requests take `tokens` rows; some start a block, some go on inside one."""
    g = _gen(seed)
    bs, h, t, runs = case["bs"], case["hkv"], case["tokens"], case["runs"]
    r = np.random.RandomState(case["lens"] % (1 << 31))
    cuts = np.sort(r.choice(np.arange(1, t), runs - 1, replace=False)) if runs > 1 else np.zeros(0, int)
    n_new = np.diff(np.concatenate([[0], cuts, [t]]))
    ctx = r.randint(0, 4 * bs, runs)
    tables, n = _tables(ctx + n_new, bs, seed)
    req = np.repeat(np.arange(runs), n_new)
    pos = np.arange(t) - np.concatenate([[0], np.cumsum(n_new)])[:-1][req] + ctx[req]
    slots = tables[req, pos // bs].astype(np.int64) * bs + pos % bs
    if t > 20:
        slots[t // 3] = -1                          # padding
    kc, vc, ks, vs, _, _ = _fill_pool(dict(bs=bs, hkv=h, d=128, pool=case["cache"] + "_block"), n, g)
    dt = _DT[case["dtype"]]
    rows = lambda: (torch.randn((t, h, 128), generator=g, device="cuda")
                    * torch.exp(0.3 * torch.randn((t, 1, 1), generator=g, device="cuda"))).to(dt)
    st = dict(case=case, kc=kc, vc=vc, ks=ks, vs=vs, k=rows(), v=rows(),
              slots=torch.from_numpy(slots).cuda())
    if own:
        st["pool"] = _handle(st, kc, vc, case["cache"] + "_block", dt, ks, vs, 1.0, 1.0)
    return st


def _prepare_attn(case, seed):
    g = _gen(seed)
    total, c = _lengths(case)
    tables, n = _tables(total, case["bs"], seed)
    k, v, ks, vs, k_scale, v_scale = _fill_pool(case, n, g)
    dt = _DT[case["dtype"]]
    t = int(c.sum())
    q = (2.0 * torch.randn((t, case["hq"], case["d"]), generator=g, device="cuda")).to(dt)
    first, prefix = _visible(case)
    i32 = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()
    cu = np.concatenate([[0], np.cumsum(c)])
    slopes = None
    if case["alibi"]:
        e = torch.arange(1, case["hq"] + 1, device="cuda", dtype=torch.float32)
        slopes = torch.exp2(-8.0 * e / case["hq"])
    st = dict(case=case, q=q, k=k, v=v, ks=ks, vs=vs, k_scale=k_scale, v_scale=v_scale,
              tables=i32(tables), lens=i32(total), cu=i32(cu), max_q=int(c.max()),
              first=i32(first), prefix=i32(prefix), slopes=slopes,
              scale=1.0 / math.sqrt(case["d"]))
    if own:
        st["pool"] = _handle(st, k, v, case["pool"], dt, ks, vs, k_scale, v_scale)
    return st


def prepare(case, seed):
    if case["op"] == "plan":
        return _prepare_plan(case, seed)
    if case["op"] == "append":
        return _prepare_append(case, seed)
    return _prepare_attn(case, seed)


# -- plain forms ---------------------------------------------------------------------

def _plain_plan(s):
    bs = s["case"]["bs"]
    ctx, new, tables, cap = s["ctx"].long(), s["new"].long(), s["tables"], s["cap"]
    lens = ctx + new
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device=ctx.device), torch.cumsum(new, 0)])
    old = (ctx + bs - 1) // bs
    need = (lens + bs - 1) // bs - old
    off = torch.cumsum(need, 0) - need + s["head"].long()
    # the new table entries, row by row
    j = torch.arange(tables.shape[1], device=ctx.device)[None, :]
    fresh = (j >= old[:, None]) & (j < (old + need)[:, None])
    idx = (off[:, None] + j - old[:, None]).clamp(0, s["free"].numel() - 1)
    tables.copy_(torch.where(fresh, s["free"][idx], tables))
    # the tokens
    i = torch.arange(cap, device=ctx.device)
    req = (torch.searchsorted(cu, i, right=True) - 1).clamp(max=new.numel() - 1)
    live = i < cu[-1]
    pos = torch.where(live, ctx[req] + i - cu[req], 0)
    slot = tables[req, torch.where(live, pos // bs, 0)].long() * bs + pos % bs
    slot = torch.where(live, slot, -1)
    head = (s["head"].long() + need.sum()).int()
    return dict(tables=tables, cu=cu.int(), lens=lens.int(), slots=slot, positions=pos.int(), head=head)


def _codes_f32(codes, cache):
    return codes.view(torch.float8_e4m3fn if cache.startswith("fp8") else torch.int8).float()


def _plain_quantise(codes, scales, rows, slots, cache):
    bs = codes.shape[1]
    qmax = _QMAX[cache]
    keep = slots >= 0
    sl, x = slots[keep], rows[keep].float()
    blk, off = sl // bs, sl % bs
    h = codes.shape[2]
    amax = torch.zeros_like(scales)
    amax.index_reduce_(0, blk, x.abs().amax(-1), "amax")
    touched = torch.zeros(codes.shape[0], dtype=torch.bool, device=codes.device)
    touched[blk] = True
    restart = torch.zeros_like(touched)
    restart[blk[off == 0]] = True
    s_old = torch.where(restart[:, None], torch.zeros_like(scales), scales)
    s_new = torch.maximum(s_old, amax / torch.full_like(amax, qmax))     # the quotient rounded once
    s_new = torch.where(s_new < _TINY, torch.zeros_like(s_new), s_new)
    s_new = torch.where(touched[:, None], s_new, scales)
    grow = touched[:, None] & ~restart[:, None] & (s_new > s_old)
    # rows that stay are rounded again where the scale grew
    b = torch.unique(blk)
    ratio = torch.where(grow[b], s_old[b] / s_new[b], torch.ones_like(s_new[b]))
    old = _codes_f32(codes[b], cache) * ratio[:, None, :, None]
    codes[b] = torch.where(grow[b][:, None, :, None], _encode(old, cache), codes[b])
    inv = torch.where(s_new > 0, 1.0 / s_new, torch.zeros_like(s_new))
    codes[blk, off] = _encode(x * inv[blk][:, :, None], cache)
    scales.copy_(s_new)


def _encode(y, cache):
    if cache.startswith("fp8"):
        return y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.round(y).clamp(-127, 127).to(torch.int8).view(torch.uint8)


def _held(codes, cache):
    return codes.view(torch.float8_e4m3fn if cache.startswith("fp8") else torch.int8)


def _plain_append(s):
    cache = s["case"]["cache"]
    _plain_quantise(s["kc"], s["ks"], s["k"], s["slots"], cache)
    _plain_quantise(s["vc"], s["vs"], s["v"], s["slots"], cache)
    return dict(k=_held(s["kc"], cache), v=_held(s["vc"], cache), k_scales=s["ks"], v_scales=s["vs"])


def _gather(s, codes, scales, one, width):
    """[batch, width, hkv, d] fp32 rows of every sequence, through its table."""
    case = s["case"]
    bs = case["bs"]
    dev = codes.device
    t = torch.arange(width, device=dev)
    blk = s["tables"].long().clamp(min=0)[:, t // bs]
    x = codes[blk, t % bs]
    if case["pool"] == "plain":
        return x.float()
    x = _codes_f32(x, case["pool"])
    if scales is None:
        return x * one
    if scales.dim() == 2:
        return x * scales[blk][..., None]
    return x * scales[blk, :, (t % bs)[None, :]][..., None]


def _plain_attn(s):
    case = s["case"]
    bs, hq, hkv, d = case["bs"], case["hq"], case["hkv"], case["d"]
    grp, b = hq // hkv, case["batch"]
    lens = s["lens"].long()
    width = s["tables"].shape[1] * bs
    k = _gather(s, s["k"], s["ks"], s["k_scale"], width).permute(0, 2, 3, 1)      # [b, hkv, d, L]
    dev = k.device
    prefill = case["op"] == "prefill"
    n = s["cu"].long().diff() if prefill else torch.ones_like(lens)
    mq = s["max_q"]
    i = torch.arange(mq, device=dev)
    qpos = (lens - n)[:, None] + i                                                # [b, mq]
    row = (s["cu"].long()[:-1] if prefill else torch.arange(b, device=dev))[:, None] + i
    row = torch.minimum(row, torch.tensor(s["q"].shape[0] - 1, device=dev))
    q = s["q"][row].float().view(b, mq, hkv, grp, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, grp * mq, d)
    sc = torch.matmul(q, k).mul_(s["scale"]).view(b, hkv, grp, mq, width)
    del k
    if case["softcap"]:
        sc = sc.div_(case["softcap"]).tanh_().mul_(case["softcap"])
    t = torch.arange(width, device=dev)
    if s["slopes"] is not None:
        dist = (t[None, None, :] - qpos[:, :, None]).abs().float()
        sc = sc.sub_(s["slopes"].view(1, hkv, grp, 1, 1) * dist[:, None, None])
    last = qpos
    if s["prefix"] is not None:
        last = torch.maximum(qpos, torch.minimum(s["prefix"].long(), lens)[:, None] - 1)
    seen = t[None, None, :] <= last[:, :, None]
    if case["window"]:
        seen &= t[None, None, :] > (qpos - case["window"])[:, :, None]
    if s["first"] is not None:
        seen &= t[None, None, :] >= s["first"].long()[row][:, :, None]
    sc = sc.masked_fill_(~seen[:, None, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    p = sc.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)).exp_()
    p = p.div_(p.sum(-1, keepdim=True).clamp(min=1e-30)).view(b, hkv, grp * mq, width)
    v = _gather(s, s["v"], s["vs"], s["v_scale"], width).permute(0, 2, 1, 3)      # [b, hkv, L, d]
    # rows past a sequence's end hold nothing
    v = torch.where((t[None, :] < lens[:, None])[:, None, :, None], v, torch.zeros((), device=dev))
    o = torch.matmul(p, v).view(b, hkv, grp, mq, d).permute(0, 3, 1, 2, 4).reshape(b, mq, hq, d)
    o = o.to(s["q"].dtype)
    if not prefill:
        return o.view(b, hq, d)
    out = torch.empty_like(s["q"])
    live = i[None, :] < n[:, None]
    out[row[live]] = o[live]
    return out


# -- the library's calls -----------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if not own:
        return {"plan": _plain_plan, "append": _plain_append}.get(op, _plain_attn)(s)
    pool, case = s["pool"], s["case"]
    if op == "plan":
        p = pool.plan_step(s["ctx"], s["new"], s["tables"], s["free"], s["head"], s["cap"])
        return dict(tables=s["tables"], cu=p.cu_seqlens, lens=p.seq_lens, slots=p.slot_mapping,
                    positions=p.positions, head=p.free_head)
    if op == "append":
        pool.append(s["k"], s["v"], s["slots"])
        return dict(k=_held(s["kc"], case["cache"]), v=_held(s["vc"], case["cache"]),
                    k_scales=s["ks"], v_scales=s["vs"])
    mods = dict(softcap=case["softcap"], alibi_slopes=s["slopes"], window=case["window"],
                first_visible=s["first"])
    plain = not (case["softcap"] or case["alibi"] or case["window"] or case["docs"])
    if op == "decode":
        if plain:
            return pool.decode(s["q"], s["tables"], s["lens"], s["scale"])
        return pool.decode_scored(s["q"], s["tables"], s["lens"], s["scale"], **mods)
    if plain and s["prefix"] is None:
        return pool.prefill(s["q"], s["cu"], s["max_q"], s["tables"], s["lens"], s["scale"])
    return pool.prefill_scored(s["q"], s["cu"], s["max_q"], s["tables"], s["lens"], s["scale"],
                               prefix_lens=s["prefix"], **mods)


# -- what a pass cannot do without -----------------------------------------------------------

def work(case):
    if case["op"] == "plan":
        ctx, new = _plan_lengths(case)
        need = -(-(ctx + new) // case["bs"]) - -(-ctx // case["bs"])
        b, t = case["batch"], int(new.sum())
        # lengths read and written, offsets; ids read and entered; the last old entry; slots and positions
        return {"bytes": 4.0 * (4 * b + 1) + 8.0 * float(need.sum()) + 12.0 * t, "flops": float(4 * t)}
    if case["op"] == "append":
        n = case["tokens"] * case["hkv"] * 128
        blocks = case["tokens"] / case["bs"] if case["runs"] < case["tokens"] else case["tokens"]
        return {"bytes": 2.0 * n * 3 + 16.0 * blocks * case["hkv"] + 8.0 * case["tokens"], "flops": 4.0 * n}
    total, c = _lengths(case)
    req, pos, lo, hi = _spans(case)
    pairs = float(np.maximum(0, hi - lo + 1).sum())
    # K and V of every position that some query of the request sees, once
    order = len(total)
    first = np.full(order, 1 << 40)
    last = np.full(order, -1)
    some = hi >= lo
    np.minimum.at(first, req[some], lo[some])
    np.maximum.at(last, req[some], hi[some])
    seen = float(np.maximum(0, last - first + 1)[last >= 0].sum())
    elt = {"plain": 4 if case["dtype"] == "f32" else 2}.get(case["pool"], 1)
    kv = 2.0 * seen * case["hkv"] * case["d"] * elt
    if case["pool"].endswith("_block"):
        kv += 8.0 * seen / case["bs"] * case["hkv"]
    elif case["pool"] == "int8":
        kv += 8.0 * seen * case["hkv"]
    qo = 2.0 * len(pos) * case["hq"] * case["d"] * (4 if case["dtype"] == "f32" else 2)
    return {"bytes": kv + qo + 4.0 * seen / case["bs"], "flops": 4.0 * pairs * case["hq"] * case["d"]}


# -- the definitions in 64 bits ----------------------------------------------------------------

def _round_e4m3(y):
    """Nearest E4M3 value (ties to even, saturating) of float64 y."""
    a = y.abs().clamp(max=448.0)
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -40))).clamp(min=-6.0)
    step = torch.exp2(e - 3.0)
    return torch.sign(y) * (torch.round(a / step) * step).clamp(max=448.0)


def _exact_append(case, seed):
    s = _prepare_append(case, seed)
    bs, cache = case["bs"], case["cache"]
    qmax = _QMAX[cache]
    slots = s["slots"].cpu().numpy()
    by_block = {}
    for i, sl in enumerate(slots):
        if sl >= 0:
            by_block.setdefault(int(sl) // bs, []).append((int(sl) % bs, i))
    f32 = lambda x: x.to(torch.float32).double()
    enc = _round_e4m3 if cache.startswith("fp8") else lambda y: torch.round(y).clamp(-127, 127)
    outs = {}
    for part, codes, scales, rows in (("k", s["kc"], s["ks"], s["k"]), ("v", s["vc"], s["vs"], s["v"])):
        val, sc = _codes_f32(codes, cache).double().cpu(), scales.double().cpu()
        x = rows.double().cpu()
        for blk, items in by_block.items():
            off = [o for o, _ in items]
            new = x[[i for _, i in items]]
            prev = torch.zeros_like(sc[blk]) if 0 in off else sc[blk].clone()
            cur = torch.maximum(prev, f32(new.abs().amax(-1).amax(0) / qmax))
            cur = torch.where(cur < _TINY, torch.zeros_like(cur), cur)
            up = (cur > prev) if 0 not in off else torch.zeros_like(cur, dtype=torch.bool)
            if up.any():
                ratio = f32(prev / cur.clamp(min=_TINY))
                val[blk] = torch.where(up[None, :, None], enc(f32(val[blk] * ratio[None, :, None])), val[blk])
            inv = torch.where(cur > 0, f32(1.0 / cur.clamp(min=_TINY)), torch.zeros_like(cur))
            val[blk, off] = enc(f32(new * inv[None, :, None]))
            sc[blk] = cur
        outs[part] = None if cache == "int8" else val
        outs[part + "_scales"] = sc
    return outs


def _exact_attn(case, seed):
    s = _prepare_attn(case, seed)
    req, pos, lo, hi = _spans(case)
    total, c = _lengths(case)
    if float(np.maximum(0, hi - lo + 1).sum()) * case["hq"] * case["d"] > 2e11:
        return None
    bs, hkv, grp, d = case["bs"], case["hkv"], case["hq"] // case["hkv"], case["d"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    start = np.concatenate([[0], np.cumsum(c)])
    tables = s["tables"].long()
    for r in range(len(total)):
        n = int(total[r])
        blocks = tables[r, :-(-n // bs)]

        def rows(codes, scales, one):
            x = codes[blocks]
            if case["pool"] == "plain":
                y = x.double()
            else:
                y = _codes_f32(x, case["pool"]).double()
                if scales is None:
                    y = y * one
                elif scales.dim() == 2:
                    y = y * scales[blocks].double()[:, None, :, None]
                else:
                    y = y * scales[blocks].double().transpose(1, 2)[..., None]
            return y.reshape(-1, hkv, d)[:n]

        k, v = rows(s["k"], s["ks"], s["k_scale"]), rows(s["v"], s["vs"], s["v_scale"])
        a, e = int(start[r]), int(start[r + 1])
        lo_r, hi_r, pos_r = (torch.from_numpy(z[a:e]).cuda() for z in (lo, hi, pos))
        t = torch.arange(n, device="cuda")
        ok = (t[None] >= lo_r[:, None]) & (t[None] <= hi_r[:, None])
        for h in range(hkv):
            q = s["q"][a:e, h * grp:(h + 1) * grp].double()
            z = torch.einsum("qgd,td->qgt", q, k[:, h]) * s["scale"]
            if case["softcap"]:
                z = case["softcap"] * torch.tanh(z / case["softcap"])
            if s["slopes"] is not None:
                far = (t[None] - pos_r[:, None]).abs().double()
                z = z - s["slopes"][h * grp:(h + 1) * grp].double()[None, :, None] * far[:, None]
            z = torch.where(ok[:, None], z, torch.full_like(z, -math.inf))
            top = z.amax(-1, keepdim=True)
            w = torch.exp(z - torch.where(top == -math.inf, torch.zeros_like(top), top))
            den = w.sum(-1, keepdim=True)
            w = torch.where(den > 0, w / torch.where(den > 0, den, torch.ones_like(den)), torch.zeros_like(w))
            out[a:e, h * grp:(h + 1) * grp] = torch.einsum("qgt,td->qgd", w, v[:, h])
    return out


def exact(case, seed):
    if case["op"] == "plan":
        return None                                  # whole numbers: equal or wrong
    if case["op"] == "append":
        return _exact_append(case, seed) if case["tokens"] <= 20000 else None
    return _exact_attn(case, seed)
