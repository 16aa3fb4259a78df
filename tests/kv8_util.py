"""A batch of the 8-bit cache's operators on the device, and its oracle."""

import numpy as np
import torch

import compressed_sparse_long_c128a_gb300 as csa
from oracle import kv8_oracle as K


def dev(x, dtype=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(x)).to(device="cuda", dtype=dtype)


def stored(x, dtype):
    """fp32 values as `dtype` holds them."""
    return torch.from_numpy(np.asarray(x, np.float32)).to(dtype)


class Batch:
    """Requests with `cached` tokens and `new` rows over a cache of `P`-row blocks in random order.

    Every row of every block holds valid codes (the rows behind a sequence's tokens too: they are read by
    nobody), and unused blocks hold the NaN code, so that a stray read shows."""

    def __init__(self, cached, new, heads, kv_heads, dim, P, dtype=torch.bfloat16, seed=0, spare_rows=3, q_scale=1.5):
        r = np.random.RandomState(seed)
        self.cached, self.new, self.H, self.Hk, self.D, self.P = np.array(cached), np.array(new), heads, kv_heads, dim, P
        self.B, self.T, self.dtype = len(cached), int(np.sum(new)), dtype
        self.start = np.concatenate([[0], np.cumsum(new)])
        need = -(-(self.cached + self.new) // P)
        blocks = int(need.sum()) + 2
        ids = r.permutation(blocks)
        self.table = np.full((self.B, int(max(need.max(initial=0), 1)) + 1), -1, np.int64)
        at = 0
        for b in range(self.B):
            self.table[b, :need[b]] = ids[at:at + need[b]]
            at += need[b]
        shape = (blocks, kv_heads, P, dim)
        self.k, self.v = (self._codes(r, shape) for _ in range(2))
        for x in (self.k, self.v):
            x[ids[at:]] = 0x7F
        self.ks, self.vs = ((0.02 * (0.2 + r.random_sample(shape[:2]))).astype(np.float32) for _ in range(2))
        self.rows = self.T + spare_rows
        self.q = stored(q_scale * r.standard_normal((self.rows, heads, dim)), dtype)
        self.max_new = int(max(np.max(new, initial=0), 1))

    @staticmethod
    def _codes(r, shape):
        x = torch.from_numpy((60 * r.standard_normal(shape)).clip(-448, 448).astype(np.float32))
        return x.to(torch.float8_e4m3fn).view(torch.uint8).numpy().copy()

    def cache(self):
        u8, f32 = torch.uint8, torch.float32
        return csa.Kv8Cache(dev(self.k, u8), dev(self.v, u8), dev(self.ks, f32), dev(self.vs, f32))

    def attn(self, cache=None, out_dtype=None, scale=None, softcap=0.0, window=0, slopes=None, first=None, prefix=None,
             lse=True, q=None, stream=None, max_new=None):
        """(out, lse, status) as torch tensors on the host; rows behind the last request keep 7."""
        cache = cache or self.cache()
        q = self.q.cuda() if q is None else q
        out = torch.full((self.rows, self.H, self.D), 7.0, dtype=out_dtype or self.dtype, device="cuda")
        ls = torch.full((self.rows, self.H), 7.0, device="cuda") if lse else None
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        mn = self.max_new if max_new is None else max_new
        n = csa.kv8_attn_workspace_size(self.rows, self.B, self.H, cache, mn)
        ws = torch.full((max(n, 1),), 0xFF, dtype=torch.uint8, device="cuda")  # scratch that starts as NaN
        csa.kv8_attn(q, dev(self.start), dev(self.cached), cache, dev(self.table), mn, out, ws, err, scale=scale,
                     softcap=softcap, window=window, slopes=None if slopes is None else dev(slopes, torch.float32),
                     first=None if first is None else dev(first), prefix=None if prefix is None else dev(prefix), lse=ls,
                     stream=stream)
        torch.cuda.synchronize()
        return out.cpu(), None if ls is None else ls.cpu(), csa.read_status(err)

    def check(self, out, lse, scale=None, softcap=0.0, window=0, slopes=None, first=None, prefix=None, skip=()):
        """Compare with the oracle; the tolerance is each rounding's half step.

        The scores: fp32 sums of D products, an error of at most (D + 8) 2^-23 of the sum of magnitudes (the
        tensor cores add with truncation, twice the half step), and 2^-21 of the capped score or of the bias from
        tanh and exp.  A score off by d changes a weight by 2 d of itself.  bf16 outputs may come from weights in
        fp16 (half a step: 2^-11) and are rounded to bf16 (2^-8); fp32 ones are sums over n keys, n 2^-24."""
        half = out.dtype == torch.bfloat16
        out, lse = out.double().numpy(), None if lse is None else lse.double().numpy()
        scale, G = self.D ** -0.5 if scale is None else scale, self.H // self.Hk
        q = self.q.double().numpy()
        worst = 0.0
        for b in range(self.B):
            if b in skip or not self.new[b]:
                continue
            n, r0, r1 = int(self.cached[b] + self.new[b]), int(self.start[b]), int(self.start[b + 1])
            p = self.cached[b] + np.arange(r1 - r0)
            f = np.zeros(r1 - r0, np.int64) if first is None else np.asarray(first)[r0:r1]
            see = K.sees(p, n, f, 0 if prefix is None else int(prefix[b]), window)
            for h in range(self.Hk):
                k, v = (K.gather(c, s, self.table[b], n, h) for c, s in ((self.k, self.ks), (self.v, self.vs)))
                hs = slice(h * G, (h + 1) * G)
                want, wl, wabs, mag = K.attend(q[r0:r1, hs], k, v, p, see, scale, softcap,
                                               None if slopes is None else np.asarray(slopes)[hs])
                capped = np.minimum(softcap, mag) if softcap else 0.0
                d = (self.D + 8) * 2.0 ** -23 * mag + 2.0 ** -21 * (capped + (mag if slopes is not None else 0) + 1)
                rel = 2 * d + (2.0 ** -11 if half else 0) + n * 2.0 ** -24
                tol = rel[..., None] * wabs + np.abs(want) * (2.0 ** -8 if half else 2.0 ** -23) + 1e-30
                got = out[r0:r1, hs]
                off = np.abs(got - want) / tol
                worst = max(worst, float(off.max()))
                assert off.max() <= 1, (b, h, float(off.max()), np.unravel_index(off.argmax(), off.shape))
                if lse is not None:
                    gl, seen = lse[r0:r1, hs], np.isfinite(wl)
                    assert np.array_equal(np.isneginf(gl), ~seen), (b, h)
                    lt = d + 2.0 ** -22 * (np.abs(wl) + 1) + n * 2.0 ** -24
                    far = np.abs(gl[seen] - wl[seen])
                    assert np.all(far <= lt[seen]), (b, h, far.max())
        assert np.all(out[self.start[-1]:] == 7.0)
        return worst
