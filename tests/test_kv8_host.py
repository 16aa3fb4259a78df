"""Host checks of the step plan and the 8-bit cache entries, and pins of their oracle (CPU only)."""

import ctypes

import numpy as np
import pytest
import torch

import compressed_sparse_long_c128a_gb300 as csa
from compressed_sparse_long_c128a_gb300 import build as csa_build
from oracle import kv8_oracle as K


@pytest.fixture(scope="module")
def lib():
    csa_build.build()
    return csa.lib()


def _cache(**kw):
    f = dict(k=0x1000, v=0x2000, k_scale=0x3000, v_scale=0x4000, num_blocks=8, rows_per_block=64, kv_heads=2, dim=128)
    return csa.Kv8C(**{**f, **kw})


BT = csa.BlockTableC(0x3000, 2, 4)


def test_plan_refusals(lib):
    good = dict(cached=0x10, n_new=0x10, B=2, free=0x10, n_free=3, table=0x10, stride=4, P=16, blocks=8, rows=5, starts=0x10,
                seq=0x10, pos=0x10, slot=0x10, used=0x10, err=0x10, stream=None)
    bad = [dict(cached=None), dict(n_new=None), dict(table=None), dict(starts=None), dict(used=None), dict(err=None),
           dict(free=None), dict(seq=None), dict(pos=None), dict(B=-1), dict(n_free=-1), dict(rows=-1), dict(stride=0), dict(P=0),
           dict(blocks=0)]
    for b in bad:
        assert lib.csa_step_plan(*{**good, **b}.values()) == csa.ERR_INVALID_ARG, b


def test_store_refusals(lib):
    def call(k=0x100, v=0x100, dt=csa.BF16, ks=256, vs=256, n=4, start=0x10, cached=0x10, cache=None, bt=BT, err=0x10):
        return lib.csa_kv8_store(k, v, dt, ks, vs, n, start, cached, cache or _cache(), bt, err, None)

    for b in (dict(k=None), dict(v=None), dict(start=None), dict(cached=None), dict(err=None), dict(n=-1), dict(ks=-1),
              dict(cache=_cache(k=None)), dict(cache=_cache(v_scale=None)), dict(cache=_cache(k=0x1008)), dict(cache=_cache(num_blocks=0)),
              dict(cache=_cache(dim=0)), dict(bt=csa.BlockTableC(0x10, 0, 4)), dict(bt=csa.BlockTableC(None, 2, 4)), dict(k=0x101)):
        assert call(**b) == csa.ERR_INVALID_ARG, b
    for b in (dict(dt=csa.E4M3), dict(cache=_cache(dim=24)), dict(cache=_cache(dim=272)), dict(cache=_cache(rows_per_block=8)),
              dict(cache=_cache(rows_per_block=48)), dict(cache=_cache(rows_per_block=512)), dict(cache=_cache(kv_heads=70000))):
        assert call(**b) == csa.ERR_UNSUPPORTED, b
    assert call(n=0, k=None, v=None) == csa.OK  # no rows: nothing to do


def test_attn_refusals(lib):
    def call(q=0x100, qd=csa.BF16, qs=1024, n=4, heads=8, start=0x10, cached=0x10, max_new=2, cache=None, bt=BT, mask=None, out=0x100,
             od=csa.BF16, lse=None, ws=None, ws_bytes=0, err=0x10):
        mask = mask or csa.Kv8MaskC(0.1, 0.0, 0, None, None, None)
        return lib.csa_kv8_attn(q, qd, qs, n, heads, start, cached, max_new, cache or _cache(), bt, mask, out, od, lse, ws, ws_bytes,
                                err, None)

    nan, inf = float("nan"), float("inf")
    for b in (dict(q=None), dict(out=None), dict(err=None), dict(start=None), dict(cached=None), dict(n=-1), dict(heads=0),
              dict(heads=7), dict(max_new=-1), dict(qs=-1), dict(q=0x101), dict(out=0x102, od=csa.F32), dict(cache=_cache(v=None)),
              *(dict(mask=csa.Kv8MaskC(*m, None, None, None)) for m in
                ((0.0, 0, 0), (-1.0, 0, 0), (nan, 0, 0), (inf, 0, 0), (1, -1, 0), (1, 1e-20, 0), (1, nan, 0), (1, inf, 0), (1, 0, -1)))):
        assert call(**b) == csa.ERR_INVALID_ARG, b
    for b in (dict(qd=csa.E4M3), dict(od=csa.E4M3), dict(cache=_cache(dim=40)), dict(heads=70000, cache=_cache(kv_heads=1))):
        assert call(**b) == csa.ERR_UNSUPPORTED, b
    # fewer bytes than the size that is asked for, or none, or a workspace that is not aligned
    need = lib.csa_kv8_attn_workspace_size(4, 2, 8, _cache(), 2)
    assert need > 0
    for b in (dict(ws=None, ws_bytes=need), dict(ws=0x1000, ws_bytes=need - 1), dict(ws=0x1004, ws_bytes=need)):
        assert call(**b) == csa.ERR_WORKSPACE, b
    assert call(n=0, q=None, out=None) == csa.OK and call(max_new=0) == csa.OK
    assert lib.csa_kv8_attn_workspace_size(0, 2, 8, _cache(), 2) == 0


def test_status_string(lib):
    assert "infinity" in csa.status_string(csa.ERR_NONFINITE)


def test_binding_refuses_host_tensors():
    z = torch.zeros(1, 1, 16, 16, dtype=torch.uint8)
    with pytest.raises(ValueError):
        csa.Kv8Cache(z, z, torch.zeros(1, 1), torch.zeros(1, 1))
    with pytest.raises(ValueError):
        csa.Kv8Cache(z, z, torch.zeros(1, 2), torch.zeros(1, 1))


# ------------------------------------------------------------------ the oracle itself


def test_oracle_store_keeps_values_within_half_a_step():
    """Decoded rows are within half an e4m3 step (2^-4) of the inputs, and within another one for rows
    rounded again after a louder token."""
    r = np.random.RandomState(0)
    codes, scale = np.zeros((2, 1, 16, 32), np.uint8), np.zeros((2, 1), np.float32)
    table, x = [[1, 0]], r.standard_normal((20, 1, 32)).astype(np.float32)
    x[10] *= 50
    for c, n in ((0, 10), (10, 10)):
        codes, scale = K.store(x[c:c + n], [0, n], [c], table, codes, scale)
    got = K.gather(codes, scale, table[0], 20, 0)
    assert np.allclose(scale[1, 0], np.abs(x[:16]).max() / 448, rtol=1e-6)
    assert np.all(np.abs(got[10:] - x[10:, 0]) <= 2.0 ** -4 * np.abs(x[10:, 0]) + scale[1, 0] * 2.0 ** -10)
    assert np.all(np.abs(got[:10] - x[:10, 0]) <= 2.0 ** -3 * np.abs(x[:10, 0]) + scale[1, 0] * 2.0 ** -9)


def test_oracle_attend_matches_brute_force():
    r = np.random.RandomState(1)
    q, k, v = r.standard_normal((3, 2, 8)), r.standard_normal((9, 8)), r.standard_normal((9, 8))
    p, slopes = np.array([4, 5, 6]), [0.5, 0.1]
    see = K.sees(p, 9, [0, 2, 100], 1, 3)
    assert [np.flatnonzero(s).tolist() for s in see] == [[0, 2, 3, 4], [3, 4, 5], []]
    out, lse, _, _ = K.attend(q, k, v, p, see, 0.3, 1.5, slopes)
    for i in range(3):
        for g in range(2):
            a = [1.5 * np.tanh(0.3 * q[i, g] @ k[t] / 1.5) - slopes[g] * abs(p[i] - t) for t in np.flatnonzero(see[i])]
            if not a:
                assert np.all(out[i, g] == 0) and lse[i, g] == -np.inf
                continue
            w = np.exp(a) / np.exp(a).sum()
            assert np.allclose(out[i, g], w @ v[see[i]]) and np.isclose(lse[i, g], np.log(np.exp(a).sum()))


def test_oracle_plan_slots():
    table, start, seq, pos, slot, used = K.step_plan([3, 0, 4], [2, 0, 5], [7, 8, 9], [[1, 0, 0], [0, 0, 0], [2, 0, 0]], 4, 8)
    assert table.tolist() == [[1, 7, -1], [-1, -1, -1], [2, 8, 9]]
    assert start.tolist() == [0, 2, 2, 7] and seq.tolist() == [0, 0, 2, 2, 2, 2, 2, -1] and pos.tolist() == [3, 4, 4, 5, 6, 7, 8, -1]
    assert slot[:2].tolist() == [7, 28] and used == 3 and slot[-1] == -1
