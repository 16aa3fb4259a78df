"""The step plan, the insert into the 8-bit key / value cache and the attention over it,
each against the oracle, and the three in a row as a serving step uses them."""

import numpy as np
import pytest
import torch

import compressed_sparse_long_c128a_gb300 as csa
from oracle import kv8_oracle as K
from kv8_util import Batch, dev, stored

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from compressed_sparse_long_c128a_gb300 import build as csa_build

    csa_build.build()


def _err():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ step plan


def _run_plan(cached, new, free, table, P, blocks, rows, slot=True):
    B = len(cached)
    t = dev(table)
    out = [torch.full((n,), -7, dtype=dt, device="cuda") for n, dt in
           ((B + 1, torch.int32), (rows, torch.int32), (rows, torch.int32), (rows, torch.int64), (1, torch.int32))]
    err = _err()
    csa.step_plan(dev(cached), dev(new), dev(free), t, P, blocks, out[0], out[1], out[2], out[3] if slot else None, out[4], err)
    return [x.cpu().numpy() for x in [t, *out]], csa.read_status(err)


def _plan_case(B, P, cached_hi, new_hi, seed, zeros=0.2):
    r = np.random.RandomState(seed)
    cached, new = r.randint(0, cached_hi + 1, B), r.randint(0, new_hi + 1, B)
    new[r.random_sample(B) < zeros] = 0
    held, need = -(-cached // P), -(-(cached + new) // P)
    ids = r.permutation(int(need.sum()) + 5)
    table = np.full((B, int(need.max()) + 2), 9999)  # what is past the held blocks is stale
    at = 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    return cached, new, ids[at:], table, len(ids)


@pytest.mark.parametrize("B,P,cached_hi,new_hi,pad", [
    (1, 256, 0, 1, 0), (1, 16, 100, 1000, 7), (5, 1, 40, 9, 3), (64, 256, 70000, 1, 0), (511, 64, 500, 3, 61),
    (512, 16, 90, 33, 1), (513, 32, 1000, 17, 0), (1700, 48, 3000, 40, 130), (6, 256, 5000, 9000, 1)])
def test_plan_matches_the_oracle(B, P, cached_hi, new_hi, pad):
    cached, new, free, table, blocks = _plan_case(B, P, cached_hi, new_hi, seed=B + P)
    rows = int(new.sum()) + pad
    want = K.step_plan(cached, new, free, table, P, rows)
    got, status = _run_plan(cached, new, free, table, P, blocks, rows)
    assert status == csa.OK
    for g, w in zip(got, want):
        assert np.array_equal(g.reshape(np.shape(w)), w)
    # again on the table it wrote: the same (a captured step may be replayed)
    again, status = _run_plan(cached, new, free, got[0], P, blocks, rows)
    assert status == csa.OK and all(np.array_equal(a, g) for a, g in zip(again, got))


def test_plan_without_slots_or_free_blocks():
    (table, starts, seq, pos, slot, used), status = _run_plan([3, 0], [2, 0], [], [[4], [-1]], 16, 8, 4, slot=False)
    assert status == csa.OK and used[0] == 0 and table.tolist() == [[4], [-1]]
    assert starts.tolist() == [0, 2, 2] and seq.tolist() == [0, 0, -1, -1] and pos.tolist() == [3, 4, -1, -1]
    assert (slot == -7).all()


def test_plan_of_no_requests():
    (table, starts, seq, pos, slot, used), status = _run_plan(np.zeros(0), np.zeros(0), [5], np.zeros((0, 2)), 16, 8, 3)
    assert status == csa.OK and starts.tolist() == [0] and used[0] == 0
    assert seq.tolist() == pos.tolist() == slot.tolist() == [-1] * 3


def test_plan_reports_what_does_not_fit():
    # too few free blocks: request 1 gets one of the two it needs
    (table, _, seq, pos, slot, used), status = _run_plan([0, 0], [16, 32], [5, 6], [[0, 0, 0], [0, 0, 0]], 16, 8, 48)
    assert status == csa.ERR_DEVICE_BOUNDS and used[0] == 2
    assert table.tolist() == [[5, -1, -1], [6, -1, -1]]
    assert slot.tolist() == list(range(80, 96)) + list(range(96, 112)) + [-1] * 16
    # fewer rows than tokens: the rest is dropped
    (_, starts, seq, pos, slot, _), status = _run_plan([0, 0], [3, 4], [5, 6], [[0], [0]], 16, 8, 5)
    assert status == csa.ERR_DEVICE_BOUNDS and starts.tolist() == [0, 3, 5] and seq.tolist() == [0, 0, 0, 1, 1]
    # negative lengths and positions past 2^31 - 1 count as nothing new
    (_, starts, seq, _, _, used), status = _run_plan([-1, 0, 2 ** 31 - 2], [3, -4, 5], [5], [[0], [0], [0]], 16, 8, 2)
    assert status == csa.ERR_DEVICE_BOUNDS and starts.tolist() == [0, 0, 0, 0] and seq.tolist() == [-1, -1] and used[0] == 0
    # more blocks than the table is wide, a held block that is not mapped, a free block that does not exist
    (table, _, _, pos, slot, used), status = _run_plan([15], [18], [5, 6, 7], [[3, 0]], 16, 8, 18)
    assert status == csa.ERR_DEVICE_BOUNDS and table.tolist() == [[3, 5]] and used[0] == 1
    assert slot.tolist() == [63] + list(range(80, 96)) + [-1] and pos.tolist() == list(range(15, 33))
    (_, _, _, _, slot, _), status = _run_plan([15], [2], [88], [[-1, 0]], 16, 8, 2)
    assert status == csa.ERR_DEVICE_BOUNDS and slot.tolist() == [-1, -1]


# ------------------------------------------------------------------ insert


def _run_store(b, k, v, cache, start=None, cached=None, table=None):
    err = _err()
    csa.kv8_store(k, v, dev(b.start if start is None else start), dev(b.cached if cached is None else cached), cache,
                  dev(b.table if table is None else table), err)
    torch.cuda.synchronize()
    return csa.read_status(err)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cached,new,Hk,D,P,layout", [
    ([0], [1], 1, 16, 16, "dense"), ([255, 256, 3], [1, 1, 0], 8, 128, 256, "fused"),
    ([7, 0, 130, 64], [300, 16, 1, 65], 3, 80, 32, "fused"), ([100, 5], [1000, 700], 2, 64, 64, "odd"),
    ([250], [513], 1, 256, 128, "dense"), ([0, 15, 31, 16], [2, 2, 2, 15], 5, 48, 16, "odd")])
def test_store_matches_the_oracle(cached, new, Hk, D, P, layout, dtype):
    """Codes and scales bit for bit, and everything that the call does not write as it was."""
    b = Batch(cached, new, Hk, Hk, D, P, dtype, seed=D + P)
    r = np.random.RandomState(1)
    loud = np.where(r.random_sample((b.rows, 1, 1)) < 0.05, 30.0, 1.0)
    x = [stored(loud * r.standard_normal((b.rows, Hk, D)), dtype) for _ in range(2)]
    if layout == "dense":
        k, v = (t.cuda() for t in x)
    elif layout == "fused":  # parts of one projection's rows
        both = torch.stack(x, 1).cuda()
        k, v = both[:, 0], both[:, 1]
    else:  # rows that start at odd elements
        buf = torch.zeros(b.rows, 2 * Hk * D + 3, dtype=dtype, device="cuda")
        k, v = buf[:, 1:1 + Hk * D].unflatten(1, (Hk, D)), buf[:, 2 + Hk * D:2 + 2 * Hk * D].unflatten(1, (Hk, D))
        k.copy_(x[0]), v.copy_(x[1])
    cache = b.cache()
    assert _run_store(b, k, v, cache) == csa.OK
    for codes, scale, xx, gc, gs in ((b.k, b.ks, x[0], cache.k, cache.k_scale), (b.v, b.vs, x[1], cache.v, cache.v_scale)):
        wc, wsc = K.store(xx.float().numpy(), b.start, b.cached, b.table, codes, scale)
        assert np.array_equal(gs.cpu().numpy(), wsc)
        assert np.array_equal(gc.cpu().numpy(), wc)
    # once more: the scales are there already, nothing changes
    kc = cache.k.clone()
    assert _run_store(b, k, v, cache) == csa.OK
    assert torch.equal(kc, cache.k)


def test_store_edge_values():
    """Zeros, the smallest and largest fp32 values, NaN and infinities."""
    for vals, status in (([0.0, -0.0], csa.OK), ([1e-44, 1.4e-45], csa.OK), ([3.4028235e38, -1e38], csa.OK),
                         ([np.nan, 2.0], csa.ERR_NONFINITE), ([np.inf, -3.0, -np.inf], csa.ERR_NONFINITE)):
        b = Batch([16], [4], 1, 1, 16, 16, torch.float32, seed=3)
        x = np.resize(np.array(vals, np.float32), (b.rows, 1, 16))
        cache = b.cache()
        assert _run_store(b, stored(x, torch.float32).cuda(), stored(x, torch.float32).cuda(), cache) == status
        wc, wsc = K.store(x, b.start, b.cached, b.table, b.k, b.ks)
        assert np.array_equal(cache.k.cpu().numpy(), wc) and np.array_equal(cache.k_scale.cpu().numpy(), wsc)


def test_store_skips_what_is_out_of_bounds():
    b = Batch([5, 20, 3], [4, 40, 2], 2, 2, 32, 16, seed=4)
    x = stored(np.random.RandomState(2).standard_normal((b.rows, 2, 32)), torch.bfloat16).cuda()
    for kind in ("unmapped", "past", "order", "rows", "table"):
        start, cached, table = b.start.copy(), b.cached.copy(), b.table.copy()
        if kind == "unmapped":
            table[1, 2] = -1
        elif kind == "past":
            table[1, 2] = 10 ** 6
        elif kind == "order":
            start[2] = start[1] - 1
        elif kind == "rows":
            start[3] = b.rows + 1
        else:
            cached[1] = 16 * table.shape[1] - 10
        cache = b.cache()
        assert _run_store(b, x, x, cache, start, cached, table) == csa.ERR_DEVICE_BOUNDS
        got = cache.k.cpu().numpy()
        wc, _ = K.store(x.float().cpu().numpy(), b.start[:2], b.cached[:1], b.table[:1], b.k, b.ks)
        assert np.array_equal(got[b.table[0, 0]], wc[b.table[0, 0]])  # request 0 is stored
        if kind in ("unmapped", "past"):
            assert np.array_equal(got[b.table[1, 2]], b.k[b.table[1, 2]])
            assert not np.array_equal(got[b.table[1, 1]], b.k[b.table[1, 1]])
        elif kind == "table":
            assert np.array_equal(got[b.table[1, :4]], b.k[b.table[1, :4]])


# ------------------------------------------------------------------ attention

BF, F32 = torch.bfloat16, torch.float32


def _slopes(H):
    return 2.0 ** (-8.0 * np.arange(1, H + 1) / H)


SHAPES = [
    # cached, new, heads, kv_heads, dim, block, type
    ([0], [1], 8, 1, 128, 64, BF),
    ([0, 1, 62, 63, 64, 65, 511], [1] * 7, 16, 2, 128, 64, BF),
    ([517], [1], 32, 8, 128, 256, BF),
    ([2000, 0, 900], [1, 0, 1], 5, 1, 64, 16, BF),
    ([1023, 16], [3, 2], 24, 3, 64, 32, BF),
    ([300, 4000], [1, 1], 64, 1, 128, 128, BF),
    ([77, 1500, 3], [1, 1, 1], 14, 2, 256, 64, BF),
    ([0], [130], 8, 2, 128, 64, BF),
    ([100, 0, 31], [200, 1, 65], 12, 4, 128, 16, BF),
    ([513], [257], 7, 1, 64, 256, BF),
    ([40, 300], [90, 1], 6, 6, 64, 128, BF),
    ([10], [70], 48, 1, 128, 32, BF),
    ([64], [140], 4, 2, 256, 256, BF),
    ([33, 200], [1, 40], 4, 2, 96, 32, BF),
    ([500, 40], [1, 2], 4, 2, 16, 16, BF),
    ([90], [80], 8, 2, 48, 64, BF),
    ([300, 5], [2, 90], 6, 2, 112, 32, BF),
    ([200, 77], [1, 60], 10, 2, 160, 64, BF),
    ([400], [50], 4, 4, 240, 128, BF),
    ([6000], [37], 16, 2, 128, 256, BF),
    ([300], [3], 16, 2, 128, 64, BF),
    ([3], [1], 16, 2, 64, 16, BF),
    ([100, 500, 0, 0], [1, 2, 1, 0], 40, 4, 128, 64, BF),
    ([5000, 9], [90, 1], 4, 1, 64, 64, BF),
    ([4100], [50], 8, 1, 192, 32, BF),
    ([100, 7], [1, 30], 12, 4, 80, 16, F32),
    ([1500], [1], 8, 8, 128, 64, F32),
    ([20], [33], 9, 3, 16, 16, F32),
    ([31], [5], 4, 1, 256, 32, F32),
]


@pytest.mark.parametrize("mask", ["causal", "window", "bias", "cap", "prefix", "docs", "all"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{len(s[0])}x{s[2]}x{s[3]}x{s[4]}p{s[5]}n{max(s[1])}{'f' if s[6] == F32 else 'b'}")
def test_attn_matches_the_oracle(shape, mask):
    b = Batch(*shape, seed=len(mask))
    r = np.random.RandomState(5)
    m = {}
    if mask in ("window", "all"):
        m["window"] = 37
    if mask in ("bias", "all"):
        m["slopes"] = _slopes(b.H)
    if mask in ("cap", "all"):
        m["softcap"] = 2.5  # low enough that it bends most scores
    if mask in ("prefix", "all"):
        m["prefix"] = np.minimum(r.randint(0, 100, b.B), b.cached + b.new)
    if mask in ("docs", "all"):
        pos = np.concatenate([c + np.arange(n) for c, n in zip(b.cached, b.new)])
        first = (r.random_sample(b.T) * (pos + 1)).astype(np.int64)
        first[r.random_sample(b.T) < 0.2] = 10 ** 9  # rows that see nothing
        m["first"] = np.concatenate([first, np.zeros(b.rows - b.T, np.int64)])
    out, lse, status = b.attn(**m)
    assert status == csa.OK
    b.check(out, lse, **m)


@pytest.mark.parametrize("dim,cap,docs", [(64, 0.0, True), (128, 0.0, False), (128, 5.0, True), (256, 0.0, True), (96, 0.0, False)])
def test_more_parts_than_sms(dim, cap, docs):
    """Prompts by the dozen, short and long, single tokens and nothing among them: every CTA goes through
    several parts, some of which see nothing."""
    r = np.random.RandomState(60)
    cached, new = r.randint(0, 400, 70), r.choice([0, 1, 3, 20, 64, 65, 129], 70)
    b = Batch(cached, new, 16, 4, dim, 32, BF, seed=60)
    m = {"softcap": cap, "window": 150}
    if docs:
        first = r.randint(0, 500, b.rows)
        first[r.random_sample(b.rows) < 0.3] = 10 ** 6
        first[b.start[5]:b.start[6]] = first[b.start[9]:b.start[10]] = 10 ** 6
        m["first"] = first
    out, lse, st = b.attn(**m)
    assert st == csa.OK
    b.check(out, lse, **m)


def test_attn_types_strides_and_scale():
    b = Batch([100, 9], [1, 3], 8, 2, 128, 64, BF, seed=8)
    wide = torch.zeros(b.rows, 2 * b.H * b.D, dtype=BF, device="cuda")
    q = wide[:, b.H * b.D:].unflatten(1, (b.H, b.D))
    q.copy_(b.q)
    out, lse, st = b.attn(q=q, scale=0.3)
    assert st == csa.OK
    b.check(out, lse, scale=0.3)
    out, _, st = b.attn(out_dtype=F32, lse=False)  # bf16 queries, fp32 result
    assert st == csa.OK
    b.check(out, None)
    odd = torch.zeros(b.rows, b.H * b.D + 1, dtype=BF, device="cuda")  # rows at odd elements
    q = odd[:, 1:].unflatten(1, (b.H, b.D))
    q.copy_(b.q)
    out, lse, st = b.attn(q=q)
    assert st == csa.OK
    b.check(out, lse)


@pytest.mark.parametrize("softcap", [0.3, 30.0, 1e3, 1e6])
@pytest.mark.parametrize("new", [2, 150])
def test_caps_near_and_far_above_the_scores(new, softcap):
    b = Batch([400, 3], [new, new], 8, 2, 128, 64, BF, seed=13)
    for slopes in (None, _slopes(8)):
        out, lse, st = b.attn(softcap=softcap, slopes=slopes)
        assert st == csa.OK
        b.check(out, lse, softcap=softcap, slopes=slopes)
    c = Batch([60], [7], 4, 2, 80, 32, F32, seed=13)
    out, lse, st = c.attn(softcap=softcap)
    assert st == csa.OK
    c.check(out, lse, softcap=softcap)


@pytest.mark.parametrize("factor", [1e-30, 1e4, 1e30])
def test_attn_extreme_queries_and_scales(factor):
    """Queries far from 1 (scores stay moderate through the scale), and blocks whose scales differ by 2^60."""
    b = Batch([700], [2], 8, 1, 128, 64, BF, seed=9, q_scale=1.5 * factor)
    b.vs[b.table[0, 3]] *= 2.0 ** 40
    b.vs[b.table[0, 7]] *= 2.0 ** -60
    b.ks[b.table[0, 5]] *= 2.0 ** -40
    scale = b.D ** -0.5 / factor
    out, lse, st = b.attn(scale=scale)
    assert st == csa.OK
    b.check(out, lse, scale=scale)


@pytest.mark.parametrize("new", [1, 150])
def test_attn_skips_what_is_out_of_bounds(new):
    b = Batch([70, 20, 33], [new, new, new], 8, 2, 128, 16, BF, seed=10)
    # an unmapped block: its keys are not there, and the others are
    keep = b.table.copy()
    b.table[1, 1] = -1
    out, lse, st = b.attn()
    assert st == csa.ERR_DEVICE_BOUNDS
    b.check(out, lse, skip=(1,))
    b.table = keep
    # more rows than announced, or tokens past the table: the request's rows stay as they were
    cached = b.cached.copy()
    b.cached[1] = 16 * b.table.shape[1] - new + 1
    out, lse, st = b.attn()
    assert st == csa.ERR_DEVICE_BOUNDS
    assert (out[b.start[1]:b.start[2]] == 7).all() and (lse[b.start[1]:b.start[2]] == 7).all()
    b.cached = cached
    b.check(out, lse, skip=(1,))
    if new > 1:
        out, lse, st = b.attn(max_new=new - 1)
        assert st == csa.ERR_DEVICE_BOUNDS and (out == 7).all()


@pytest.mark.parametrize("new", [1, 5, 150])
def test_one_request_in_a_padded_call(new):
    """Rows behind the request and a bound far above its rows, as a captured call of fixed shapes has."""
    for spare, max_new in ((3, 200), (300, 400)):
        b = Batch([700], [new], 8, 2, 128, 64, BF, seed=21, spare_rows=spare)
        out, lse, st = b.attn(max_new=max_new)
        assert st == csa.OK
        b.check(out, lse)
        if new > 1:
            out, lse, st = b.attn(max_new=new - 1)
            assert st == csa.ERR_DEVICE_BOUNDS and (out == 7).all() and (lse == 7).all()


def test_nan_query_stays_in_its_row():
    for new in (1, 3, 200):
        b = Batch([40], [new], 8, 2, 128, 64, BF, seed=11)
        q = b.q.clone()
        q[0, 3, 5] = float("nan")
        out, lse, st = b.attn(q=q.cuda())
        assert st == csa.OK
        bad = torch.isnan(out.float()).all(-1)
        assert bad[0, 3] and int(bad.sum()) == 1 and int(torch.isnan(out.float()).sum()) == b.D
        assert torch.isnan(lse[0, 3]) and int(torch.isnan(lse).sum()) == 1


def test_same_call_same_bits():
    for shape in (([5000, 100, 3000], [1, 1, 2], 32, 4, 128, 64, BF), ([900, 10], [150, 300], 16, 2, 128, 32, BF)):
        b = Batch(*shape, seed=12)
        cache = b.cache()
        first = b.attn(cache)
        for _ in range(3):
            again = b.attn(cache)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


# ------------------------------------------------------------------ a step, and steps in a row


def test_serving_steps():
    """Prompts in two chunks, then single tokens: plan, insert and attention on one table, each step's
    attention against the oracle on the cache that the oracle's own insert built."""
    r = np.random.RandomState(20)
    B, H, Hk, D, P, blocks = 4, 16, 2, 128, 32, 64
    cache, err = csa.Kv8Cache.empty(blocks, Hk, P, D), _err()
    ok, ov = np.zeros((blocks, Hk, P, D), np.uint8), np.zeros((blocks, Hk, P, D), np.uint8)
    oks, ovs = np.zeros((blocks, Hk), np.float32), np.zeros((blocks, Hk), np.float32)
    table, free = torch.full((B, 12), -1, dtype=torch.int32, device="cuda"), list(r.permutation(blocks))
    cached = np.zeros(B, np.int64)
    for new in ([40, 7, 0, 100], [33, 90, 64, 1], [1, 1, 1, 1], [1, 0, 2, 1], [1, 1, 1, 1]):
        T, cap = int(np.sum(new)), int(np.sum(new)) + 2
        start, seq, pos = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (B + 1, cap, cap))
        slot, used = torch.empty(cap, dtype=torch.int64, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
        cd = dev(cached)
        csa.step_plan(cd, dev(new), dev(free), table, P, blocks, start, seq, pos, slot, used, err)
        free = free[int(used):]
        qkv = stored(r.standard_normal((cap, H + 2 * Hk, D)), BF).cuda()
        q, k, v = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
        csa.kv8_store(k, v, start, cd, cache, table, err)
        out = torch.empty(cap, H, D, dtype=BF, device="cuda")
        n = csa.kv8_attn_workspace_size(cap, B, H, cache, max(new))
        csa.kv8_attn(q, start, cd, cache, table, max(new), out, torch.empty(max(n, 1), dtype=torch.uint8, device="cuda"), err,
                     window=50)
        assert csa.read_status(err) == csa.OK
        # the slot of a row is where its codes are
        t, st = table.cpu().numpy(), start.cpu().numpy()
        ok, oks = K.store(k.float().cpu().numpy(), st, cached, t, ok, oks)
        ov, ovs = K.store(v.float().cpu().numpy(), st, cached, t, ov, ovs)
        assert np.array_equal(cache.k.cpu().numpy(), ok) and np.array_equal(cache.v_scale.cpu().numpy(), ovs)
        sl = slot.cpu().numpy()[:T]
        assert np.array_equal(cache.k.transpose(1, 2).reshape(-1, Hk, D)[torch.from_numpy(sl).cuda()].cpu().numpy(),
                              ok.transpose(0, 2, 1, 3).reshape(-1, Hk, D)[sl])
        for b in range(B):
            if not new[b]:
                continue
            p = cached[b] + np.arange(new[b])
            see = K.sees(p, int(cached[b] + new[b]), np.zeros(new[b]), 0, 50)
            for h in range(Hk):
                kk, vv = K.gather(ok, oks, t[b], len(see[0]), h), K.gather(ov, ovs, t[b], len(see[0]), h)
                qq = q[st[b]:st[b + 1], h * 8:(h + 1) * 8].double().cpu().numpy()
                want, _, wabs, _ = K.attend(qq, kk, vv, p, see, D ** -0.5)
                got = out[st[b]:st[b + 1], h * 8:(h + 1) * 8].double().cpu().numpy()
                assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * wabs)
        cached = cached + np.array(new)


def test_captured_step_follows_its_inputs():
    """A step captured once, replayed on other lengths, blocks and rows: two graphs with workspaces of
    their own, on another stream than the default one."""
    B, H, Hk, D, P = 3, 16, 2, 128, 16
    for new_cap, lens in ((1, [([5, 300, 64], [1, 1, 1]), ([700, 0, 15], [1, 0, 1])]),
                          (200, [([5, 30, 64], [100, 1, 60]), ([10, 300, 15], [1, 200, 33])])):
        side, graphs = torch.cuda.Stream(), []
        for cached, new in lens:
            b = Batch(cached, new, H, Hk, D, P, seed=30)
            cap = 3 * new_cap
            s = {"cached": dev(np.zeros(B)), "start": dev(np.zeros(B + 1)), "table": dev(np.full((B, 70), -1)),
                 "q": torch.zeros(cap, H, D, dtype=BF, device="cuda"), "out": torch.zeros(cap, H, D, dtype=BF, device="cuda"),
                 "cache": csa.Kv8Cache.empty(200, Hk, P, D), "err": _err()}
            n = csa.kv8_attn_workspace_size(cap, B, H, s["cache"], new_cap)
            s["ws"] = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")

            def step():
                csa.kv8_attn(s["q"], s["start"], s["cached"], s["cache"], s["table"], new_cap, s["out"], s["ws"], s["err"])

            torch.cuda.synchronize()
            with torch.cuda.stream(side):
                step()
            side.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                step()
            graphs.append((g, s, b))
        for g, s, b in graphs:  # the lengths come after the capture
            nb = b.k.shape[0]
            s["cached"].copy_(dev(b.cached)), s["start"].copy_(dev(b.start))
            s["table"].fill_(-1)
            s["table"][:, : b.table.shape[1]].copy_(dev(b.table))
            s["q"][: b.T].copy_(b.q[: b.T])
            for n, x in (("k", b.k), ("v", b.v), ("k_scale", b.ks), ("v_scale", b.vs)):
                getattr(s["cache"], n)[:nb].copy_(torch.from_numpy(x))
        torch.cuda.synchronize()
        for g, s, b in graphs:
            g.replay()
        torch.cuda.synchronize()
        for g, s, b in graphs:
            assert csa.read_status(s["err"]) == csa.OK
            got = torch.full((b.rows, H, D), 7.0, dtype=BF)
            got[: b.T] = s["out"][: b.T].cpu()
            b.check(got, None)


def test_whole_step_captured():
    """Plan, insert and attention in one graph, replayed for steps of other lengths; rows behind a step's
    last one keep what they held."""
    B, H, Hk, D, P, blocks, cap, most = 3, 8, 2, 64, 16, 60, 130, 64
    r = np.random.RandomState(70)
    i32 = torch.int32
    cache, err = csa.Kv8Cache.empty(blocks, Hk, P, D), _err()
    cd, nd, start, used = (torch.zeros(n, dtype=i32, device="cuda") for n in (B, B, B + 1, 1))
    seq, pos = (torch.zeros(cap, dtype=i32, device="cuda") for _ in range(2))
    slot = torch.zeros(cap, dtype=torch.int64, device="cuda")
    free, table = torch.zeros(blocks, dtype=i32, device="cuda"), torch.full((B, 20), -1, dtype=i32, device="cuda")
    qkv = torch.zeros(cap, H + 2 * Hk, D, dtype=BF, device="cuda")
    out = torch.zeros(cap, H, D, dtype=BF, device="cuda")
    ws = torch.empty(csa.kv8_attn_workspace_size(cap, B, H, cache, most), dtype=torch.uint8, device="cuda")

    def step():
        csa.step_plan(cd, nd, free, table, P, blocks, start, seq, pos, slot, used, err)
        csa.kv8_store(qkv[:, H:H + Hk], qkv[:, H + Hk:], start, cd, cache, table, err)
        csa.kv8_attn(qkv[:, :H], start, cd, cache, table, most, out, ws, err, softcap=20.0)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step()
    ok = [np.zeros((blocks, Hk, P, D), np.uint8) for _ in range(2)]
    os_ = [np.zeros((blocks, Hk), np.float32) for _ in range(2)]
    ids, cached = list(r.permutation(blocks)), np.zeros(B, np.int64)
    for new in ([50, 3, 64], [1, 0, 1], [0, 40, 1], [1, 1, 1]):
        T = int(np.sum(new))
        x = stored(r.standard_normal((cap, H + 2 * Hk, D)), BF)
        qkv.copy_(x), out.fill_(7), cd.copy_(dev(cached)), nd.copy_(dev(new))
        free[: len(ids)].copy_(dev(ids))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert csa.read_status(err) == csa.OK
        ids = ids[int(used):]
        st, t = start.cpu().numpy(), table.cpu().numpy()
        assert np.array_equal(st, np.concatenate([[0], np.cumsum(new)])) and (pos[T:] == -1).all()
        for i in range(2):
            ok[i], os_[i] = K.store(x[:, H + i * Hk:H + (i + 1) * Hk].float().numpy(), st, cached, t, ok[i], os_[i])
        assert np.array_equal(cache.k.cpu().numpy(), ok[0]) and np.array_equal(cache.v.cpu().numpy(), ok[1])
        got = out.double().cpu().numpy()
        assert (got[T:] == 7).all()
        for b in range(B):
            if not new[b]:
                continue
            p, n = cached[b] + np.arange(new[b]), int(cached[b] + new[b])
            for h in range(Hk):
                kk, vv = (K.gather(ok[i], os_[i], t[b], n, h) for i in range(2))
                want, _, wabs, _ = K.attend(x[st[b]:st[b + 1], 4 * h:4 * h + 4].double().numpy(), kk, vv, p,
                                            K.sees(p, n, np.zeros(new[b]), 0, 0), D ** -0.5, 20.0)
                assert np.all(np.abs(got[st[b]:st[b + 1], 4 * h:4 * h + 4] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * wabs)
        cached = cached + np.array(new)


def test_two_streams_at_once():
    """Calls that overlap, each with a workspace of its own, give what they give alone."""
    bs = [Batch([3000, 17, 900], [1, 1, 2], 16, 2, 128, 64, BF, seed=80), Batch([400, 30], [200, 90], 16, 2, 128, 64, BF, seed=81)]
    alone = [b.attn()[:2] for b in bs]
    streams, state = [torch.cuda.Stream() for _ in bs], []
    for b in bs:
        c = b.cache()
        n = csa.kv8_attn_workspace_size(b.rows, b.B, b.H, c, b.max_new)
        state.append((b.q.cuda(), dev(b.start), dev(b.cached), c, dev(b.table), b.max_new,
                      torch.full((b.rows, b.H, b.D), 7.0, dtype=BF, device="cuda"), torch.empty(n, dtype=torch.uint8, device="cuda"), _err()))
    torch.cuda.synchronize()
    for _ in range(10):
        for s, a in zip(streams, state):
            csa.kv8_attn(*a, stream=s)
    torch.cuda.synchronize()
    for a, want in zip(state, alone):
        assert csa.read_status(a[-1]) == csa.OK and torch.equal(a[6].cpu(), want[0])


def test_offsets_past_32_bits():
    """Blocks behind 4 GiB of codes, read and written."""
    H, Hk, D, P, blocks = 8, 8, 256, 256, 8300
    cache = csa.Kv8Cache(*(torch.empty(blocks, Hk, P, D, dtype=torch.uint8, device="cuda") for _ in range(2)),
                         *(torch.zeros(blocks, Hk, device="cuda") for _ in range(2)))
    assert cache.k.numel() > 2 ** 32
    r = np.random.RandomState(40)
    table = np.array([[blocks - 1, 3], [blocks - 2, 8200]])
    T = 300
    x = stored(r.standard_normal((3, 2 * T, Hk, D)), BF)
    start, cached, err = np.array([0, T, 2 * T]), np.array([0, 0]), _err()
    csa.kv8_store(x[0].cuda(), x[1].cuda(), dev(start), dev(cached), cache, dev(table), err)
    out = torch.empty(2 * T, H, D, dtype=BF, device="cuda")
    n = csa.kv8_attn_workspace_size(2 * T, 2, H, cache, T)
    csa.kv8_attn(x[2].cuda(), dev(start), dev(cached), cache, dev(table), T, out, torch.empty(max(n, 1), dtype=torch.uint8, device="cuda"), err)
    assert csa.read_status(err) == csa.OK
    ids = table.reshape(-1)
    codes, scales = (np.zeros((4, Hk, P, D), np.uint8) for _ in range(2)), (np.zeros((4, Hk), np.float32) for _ in range(2))
    small = np.array([[0, 1], [2, 3]])
    (kc, ks), (vc, vs) = (K.store(x[i].float().numpy(), start, cached, small, c, s) for i, (c, s) in enumerate(zip(codes, scales)))
    tail = np.array([0, 2])
    assert np.array_equal(cache.k[dev(ids[tail], torch.int64)].cpu().numpy(), kc[tail])
    for b in range(2):
        p = np.arange(T)
        see = K.sees(p, T, np.zeros(T), 0, 0)
        want, _, wabs, _ = K.attend(x[2][b * T:(b + 1) * T, :1].double().numpy(), K.gather(kc, ks, small[b], T, 0),
                                    K.gather(vc, vs, small[b], T, 0), p, see, D ** -0.5)
        got = out[b * T:(b + 1) * T, :1].double().cpu().numpy()
        assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * wabs)


def test_tensors_are_checked():
    b = Batch([3], [1], 8, 2, 64, 16, BF, seed=50)
    cache = b.cache()
    good = dict(q=b.q.cuda(), row_start=dev(b.start), cached=dev(b.cached), cache=cache, bt=dev(b.table), max_new=1,
                out=torch.empty(b.rows, 8, 64, dtype=BF, device="cuda"), ws=torch.empty(1 << 22, dtype=torch.uint8, device="cuda"),
                err=_err())
    csa.kv8_attn(**good)
    for bad in (dict(q=b.q), dict(q=b.q.cuda().transpose(1, 2)), dict(row_start=dev(b.start, torch.int64)), dict(cached=dev([1, 2])),
                dict(out=torch.empty(b.rows, 8, 32, dtype=BF, device="cuda")), dict(first=dev([0])), dict(prefix=dev([0, 1])),
                dict(slopes=torch.zeros(7, device="cuda")), dict(lse=torch.zeros(3, device="cuda")), dict(q=b.q.cuda().half())):
        with pytest.raises(ValueError):
            csa.kv8_attn(**{**good, **bad})
    for bad in (dict(softcap=-1.0), dict(window=-1), dict(scale=0.0), dict(scale=float("inf"))):
        with pytest.raises(csa.CsaError):
            csa.kv8_attn(**{**good, **bad})
