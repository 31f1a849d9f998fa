"""Batches for the paged-cache tests: pages filled on the host, ragged metadata, and the float64
view of what the pages hold."""
import numpy as np
import torch

import oracle.paged_oracle as P

HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


class Batch:
    """lengths (new tokens included) and new-token counts of a ragged batch over random pages.

    Every page starts filled with `fill` (NaN by default: nothing behind a sequence's end may be
    used), then the cached rows of every sequence are written; `held` keeps them in float64."""

    def __init__(self, total, new, Hkv, d, page, bits, dtype, seed=0, spare=2, scale_of=None,
                 poison=True, k_std=1.0, v_std=1.0):
        rng = np.random.default_rng(seed)
        self.total, self.new, self.Hkv, self.d, self.page, self.bits = total, new, Hkv, d, page, bits
        self.dtype = dtype
        B = len(total)
        need = [-(-t // page) for t in total]
        n_pages = sum(need) + spare
        order = rng.permutation(n_pages)
        max_pages = max(1, max(need))
        table = np.full((B, max_pages), 2 ** 30, np.int32)   # entries never read name no page
        at = 0
        for b, m in enumerate(need):
            table[b, :m] = order[at:at + m]
            at += m
        nan = float("nan") if poison else 0.0
        if bits == 4:
            kp = torch.full((n_pages, Hkv, page, d // 2), 0xA5, dtype=torch.uint8)
            vp = kp.clone()
            sc = torch.full((n_pages, Hkv, page, 4), nan, dtype=torch.float16)
        else:
            kp = torch.full((n_pages, Hkv, page, d), nan, dtype=dtype)
            vp, sc = kp.clone(), None
        self.held = []                                        # (k, v) [L, Hkv, d] float64
        self.vz = []                                          # value zeros [L, Hkv]
        for b, L in enumerate(total):
            kx = rng.standard_normal((L, Hkv, d)) * k_std
            vx = rng.standard_normal((L, Hkv, d)) * v_std
            if scale_of is not None:
                vx = vx * scale_of(rng, L)[:, None, None]
            pg, sl = torch.as_tensor(table[b][np.arange(L) // page]).long(), torch.arange(L) % page
            if bits == 4:
                kc, ks, kz = P.quantise4(kx)
                vc, vs, vz = P.quantise4(vx)
                if L:
                    kp[pg, :, sl] = torch.as_tensor(P.pack4(kc))
                    vp[pg, :, sl] = torch.as_tensor(P.pack4(vc))
                    sc[pg, :, sl] = torch.as_tensor(np.stack([ks, kz, vs, vz], -1))
                self.held.append((P.dequantise4(kc, ks, kz), P.dequantise4(vc, vs, vz)))
                self.vz.append(vz.astype(np.float64))
            else:
                kt, vt = torch.as_tensor(kx).to(dtype), torch.as_tensor(vx).to(dtype)
                if L:
                    kp[pg, :, sl], vp[pg, :, sl] = kt, vt
                self.held.append((kt.double().numpy(), vt.double().numpy()))
                self.vz.append(None)
        self.k, self.v, self.scales = kp, vp, sc
        self.table = torch.as_tensor(table)
        self.lengths = torch.tensor(total, dtype=torch.int32)
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32)
        self.tokens = int(sum(new))
        self.rng = rng

    def cache(self, cls):
        c = lambda t: None if t is None else t.cuda()
        return cls.PagedCache.from_pages(c(self.k), c(self.v), c(self.table), c(self.lengths),
                                         c(self.scales), torch.zeros(1, dtype=torch.int32, device="cuda"))

    def rows(self, heads, dtype=None, std=1.0):
        x = self.rng.standard_normal((self.tokens, heads, self.d)) * std
        return torch.as_tensor(x).to(dtype or self.dtype)

    def attention(self, q, scale=None, tensor=False):
        """(o, tolerance) [tokens, H, d] in float64.

        The tolerance, in the kernel's order of rounding:
          each weight is rounded to float16 (2^-11 of it), or to two bfloat16 terms (2^-16): as
          much of sum_j p_j (|v_j| + |vz_j|), which bounds what the weights multiply (7.5 value
          steps at most, centred codes);
          weights below float16's normal range keep an absolute 2^-25 beside a largest of at
          least 1 in 2^7 (value scales are brought there): 2^-27 per key of the largest value
          range, 2^-25 of the values at 16 bits;
          a score sums products in float32 (a relative 2^-20 of the magnitudes' sum covers d <=
          128 terms and the scale's and exponential's own roundings), which moves every weight
          by as much;
          with `tensor` (4 bits, many rows a sequence) held keys and values are rounded to float16
          (2^-11 of the magnitudes behind a score, and of the values), and some exponentials come
          from a cubic (2^-13);
          the result is rounded to its type (half a step)."""
        outs, tols, t0 = [], [], 0
        sc = self.d ** -0.5 if scale is None else scale
        w = 2.0 ** -16 if self.bits == 16 and self.dtype == torch.bfloat16 else 2.0 ** -11
        s = 2.0 ** -20
        if tensor:
            w, s = 2.0 ** -10 + 2.0 ** -13, s + 2.0 ** -11
        for b, n in enumerate(self.new):
            k, v = self.held[b]
            qb = q[t0:t0 + n].double().numpy()
            o, mass, mag = P.attention(qb, k, v, sc, self.vz[b])
            top = np.abs(v).max() if v.size else 0.0
            small = len(v) * 2.0 ** -25 * 2 * top
            tols.append(mass * (w + 2.0 ** -20 + s * mag[..., None]) + small
                        + np.abs(o) * HALF_STEP[q.dtype] + 1e-7)
            outs.append(o)
            t0 += n
        return np.concatenate(outs), np.concatenate(tols)


def assert_within(got, ref, tol, what=""):
    got = got.detach().double().cpu().numpy()
    assert got.shape == ref.shape, (got.shape, ref.shape)
    err = np.abs(got - ref)
    bad = ~(err <= tol)
    if bad.any():
        i = np.unravel_index(np.nanargmax(np.where(np.isnan(err), np.inf, err / tol)), err.shape)
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} off; worst at {i}: got {got[i]}, "
                             f"ref {ref[i]}, tolerance {tol[i]}")
    print(f"{what}: worst {np.max(err / tol):.3f} of the tolerance")
