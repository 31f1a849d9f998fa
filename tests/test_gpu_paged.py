"""The paged cache on the GPU against its float64 definition: append (with the rotation), dense
read-back, attention over the pages, and the layer's prefill and decode on top of them."""
import itertools

import numpy as np
import pytest
import torch

import oracle.cca_oracle as O
import oracle.paged_oracle as P
import workloads as W
from gpu_helpers import BF16_TOL, bf16_err, f64, oracle_config, oracle_weights
from paged_helpers import HALF_STEP, Batch, assert_within

pytestmark = pytest.mark.gpu
BASE = 10000.0


def rotated(x, pos, base):
    """(rotated rows, error bound of the rotation): sine and cosine within 2^-20."""
    ref = P.rotate(x, pos, base)
    half = x.shape[-1] // 2
    mag = np.abs(x[..., :half]) + np.abs(x[..., half:])
    return ref, np.concatenate([mag, mag], -1) * 2.0 ** -20


def positions(t):
    return np.concatenate([np.arange(L - n, L) for L, n in zip(t.total, t.new)]).astype(int)


# ------------------------------------------------------------------------------- append
@pytest.mark.parametrize("bits,dtype", [(16, torch.float16), (16, torch.bfloat16),
                                        (4, torch.float16), (4, torch.bfloat16), (4, torch.float32)])
@pytest.mark.parametrize("d,page", [(16, 16), (32, 64), (64, 16), (128, 32)])
def test_append_ragged(cuda_lib, bits, dtype, d, page):
    cls = cuda_lib
    pages_dt = dtype if bits == 16 else torch.float16
    Hkv, H = 3, 6
    t = Batch([1, 37, 0, 64, 200, 17], [1, 5, 0, 64, 1, 3], Hkv, d, page, bits, pages_dt, seed=d)
    cache = t.cache(cls)
    k, v, q = t.rows(Hkv, dtype), t.rows(Hkv, dtype), t.rows(H, dtype)
    before = [x.clone() for x in (cache.k, cache.v)]
    qo = cache.append(k.cuda(), v.cuda(), q.cuda(), cu_seqlens=t.cu.cuda(), rope_base=BASE)
    torch.cuda.synchronize()
    cache.check()
    pos = positions(t)
    qr, qt = rotated(q.double().numpy(), pos, BASE)
    assert_within(qo, qr, qt + np.abs(qr) * HALF_STEP[dtype] + 1e-7, "q")
    seq = np.repeat(np.arange(len(t.new)), t.new)
    pg = torch.as_tensor(t.table.numpy()[seq, pos // page]).long()
    sl = torch.as_tensor(pos % page)
    kr, kt = rotated(k.double().numpy(), pos, BASE)
    vr = v.double().numpy()
    kc, vc = cache.k.cpu(), cache.v.cpu()
    if bits == 16:
        assert_within(kc[pg, :, sl], kr, kt + np.abs(kr) * HALF_STEP[pages_dt] + 1e-7, "k")
        assert torch.equal(vc[pg, :, sl], v.to(pages_dt))
    else:
        sc = cache.scales.cpu()[pg, :, sl].numpy()
        codes, vs, vz = P.quantise4(v.float().numpy())
        assert np.array_equal(P.unpack4(vc[pg, :, sl].numpy()), codes)
        assert np.array_equal(sc[..., 2], vs) and np.array_equal(sc[..., 3], vz)
        # keys: within half a step of the rotated value, the ends by what float16 rounds off
        held = P.dequantise4(P.unpack4(kc[pg, :, sl].numpy()), sc[..., 0], sc[..., 1])
        lo, hi = kr.min(-1, keepdims=True), kr.max(-1, keepdims=True)
        step = (hi - lo) / 15 * (1 + 2.0 ** -11)
        assert_within(torch.as_tensor(held), kr,
                      step / 2 + (hi - lo + np.abs(lo)) * 2.0 ** -11 + 2 * kt.max(-1, keepdims=True) + 1e-6, "k")
    # nothing else changed
    keep = torch.ones(kc.shape[0], page, dtype=torch.bool)
    keep[pg, sl] = False
    for was, now in zip(before, (kc, vc)):
        w8, n8 = was.cpu().transpose(1, 2)[keep], now.transpose(1, 2)[keep]
        assert torch.equal(w8.view(torch.uint8), n8.contiguous().view(torch.uint8))


@pytest.mark.parametrize("bits", [16, 4])
def test_append_uniform_strided_and_no_rotation(cuda_lib, bits):
    """Rows inside a wider projection, head-major rows, and [batch, n] layouts give the same pages."""
    cls = cuda_lib
    B, n, Hkv, H, d = 4, 6, 2, 4, 32
    t = Batch([10, 6, 33, 64], [n] * B, Hkv, d, 16, bits, torch.float16, seed=5)
    g = torch.Generator().manual_seed(3)
    qkv = torch.randn(B * n, (H + 2 * Hkv) * d + 24, generator=g).half().cuda()
    q, k, v = (qkv[:, a * d:b * d].unflatten(1, (-1, d)) for a, b in ((0, H), (H, H + Hkv), (H + Hkv, H + 2 * Hkv)))
    one, two, three = (t.cache(cls) for _ in range(3))
    qa = one.append(k, v, q, rope_base=BASE)
    hm = lambda x: x.reshape(B, n, -1, d).transpose(1, 2).contiguous().transpose(1, 2)
    out = torch.zeros(B, H, n, d, dtype=torch.half, device="cuda").transpose(1, 2)
    two.append(hm(k), hm(v), hm(q), rope_base=BASE, q_out=out)
    three.append(k, v, q, cu_seqlens=t.cu.cuda(), rope_base=BASE)
    for c in (two, three):
        for a, b in ((one.k, c.k), (one.v, c.v)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        if bits == 4:
            assert torch.equal(one.scales.view(torch.uint8), c.scales.view(torch.uint8))
    assert torch.equal(qa.view(B, n, H, d), out)
    # no rotation: q is copied, keys are stored as they are
    qc = one.append(k, v, q)
    assert torch.equal(qc, q)
    kd, _ = one.gather(80 * B, dtype=torch.float32)
    pos = [L - n for L in t.total]
    got = kd.view(B, 80, Hkv, d)[0, pos[0]:pos[0] + n].cpu()
    if bits == 16:
        assert torch.equal(got, k[:n].float().cpu())
    else:
        codes, s, z = P.quantise4(k[:n].float().cpu().numpy())
        assert np.allclose(got.numpy(), P.dequantise4(codes, s, z), rtol=2.0 ** -23, atol=1e-7)


def test_append_far_positions(cuda_lib):
    """Positions near 2^24: the table repeats one page, only the last is written."""
    cls = cuda_lib
    d, page = 64, 4096
    pos = 2 ** 24 - 3
    k = torch.randn(1, 1, d, generator=torch.Generator().manual_seed(0))
    cache = cls.PagedCache(1, 2 ** 24 // page, page, 1, d, bits=16, n_pages=2)
    cache.lengths.fill_(pos + 1)
    cache.append(k.half().cuda(), k.half().cuda(), rope_base=BASE)
    ref, tol = rotated(k.half().double().numpy(), [pos], BASE)
    # beside the sine's own error, the angle's: a few 1e-8 turns
    got = cache.k[0, 0, pos % page].view(1, 1, d)
    assert_within(got, ref, tol + 2.0 ** -20 * np.abs(k.numpy()).max() * 2 + np.abs(ref) * 2.0 ** -11 + 1e-6, "far")


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 1e6])
@pytest.mark.parametrize("bits", [16, 4])
def test_append_reports_what_float16_cannot_hold(cuda_lib, bad, bits):
    cls = cuda_lib
    t = Batch([5, 5], [1, 1], 1, 16, 16, bits, torch.float16, seed=1)
    cache = t.cache(cls)
    k, v = t.rows(1, torch.float32), t.rows(1, torch.float32)
    v[1, 0, 3] = bad
    cache.append(k.cuda(), v.cuda())
    with pytest.raises(cls.CCAError) as e:
        cache.check()
    assert e.value.code == cls.CCA_ERR_RANGE
    cache.check()                                        # cleared
    kd, vd = cache.gather(10, dtype=torch.float32)
    vd = vd.view(2, 5, 16).cpu()
    assert torch.isfinite(vd[0, 4]).all() and torch.isfinite(kd.view(2, 5, 16)[1, 4]).all()
    assert not torch.isfinite(vd[1, 4, 3])
    if bits == 4:
        assert torch.isnan(vd[1, 4]).all()


def test_append_constant_and_tiny_vectors(cuda_lib):
    """A range of zero, and one whose step float16 rounds to nothing."""
    cls = cuda_lib
    t = Batch([1, 1, 1, 1], [1] * 4, 1, 32, 16, 4, torch.float16)
    cache = t.cache(cls)
    v = torch.zeros(4, 1, 32)
    v[1] = 3.25
    v[2] = torch.linspace(0, 1e-8, 32)
    v[3, 0, 0] = 65504.0
    cache.append(v.cuda(), v.cuda())
    cache.check()
    kd, vd = cache.gather(64 * 4 // 4, dtype=torch.float32)
    codes, s, z = P.quantise4(v.numpy())
    ref = P.dequantise4(codes, s, z)
    got = vd.view(4, 16, 1, 32)[:, 0].cpu().numpy()
    assert np.array_equal(got, ref.astype(np.float32))
    assert np.array_equal(kd.view(4, 16, 1, 32)[:, 0].cpu().numpy(), got)


# ------------------------------------------------------------------------------- gather
@pytest.mark.parametrize("bits,dtype", [(16, torch.float16), (16, torch.bfloat16), (4, torch.float16)])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_gather(cuda_lib, bits, dtype, out_dtype):
    cls = cuda_lib
    Hkv, d = 3, 64
    t = Batch([0, 1, 33, 100, 16], [0] * 5, Hkv, d, 16, bits, dtype, seed=9)
    cache = t.cache(cls)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(t.total)]), dtype=torch.int32, device="cuda")
    k, v = cache.gather(sum(t.total), cu_seqlens=cu, dtype=out_dtype)
    for got, i in ((k, 0), (v, 1)):
        ref = np.concatenate([h[i] for h in t.held])
        # one rounding of the product, one of the sum (float32), one to the output's type
        tol = np.abs(ref) * HALF_STEP[out_dtype] + (np.abs(ref) + 8) * 2.0 ** -22
        assert_within(got, ref, tol, "gather")
    # dense [B, Hkv, max_seq, d] buffers, shorter and longer than the sequences; the rest stays
    for room in (40, 120):
        kd = torch.full((5, Hkv, room, d), 7.0, dtype=out_dtype, device="cuda")
        vd = kd.clone()
        cache.gather(k_out=kd.transpose(1, 2), v_out=vd.transpose(1, 2))
        for b, L in enumerate(t.total):
            n = min(L, room)
            assert torch.equal(kd[b, :, :n].transpose(0, 1), k[int(cu[b]):int(cu[b]) + n])
            assert torch.equal(vd[b, :, :n].transpose(0, 1), v[int(cu[b]):int(cu[b]) + n])
            assert (kd[b, :, n:] == 7).all() and (vd[b, :, n:] == 7).all()
    cache.check()


# ------------------------------------------------------------------------------- attention
FORMS = [(4, torch.float16), (4, torch.bfloat16), (16, torch.float16), (16, torch.bfloat16)]


@pytest.mark.parametrize("bits,dtype", FORMS)
@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("G", [1, 3, 4, 8, 13])
def test_attention_single_tokens(cuda_lib, bits, dtype, d, G):
    """One new token a sequence, lengths around the tile and page edges, empty slots among them."""
    cls = cuda_lib
    Hkv = 2
    total = [1, 0, 15, 16, 17, 63, 64, 65, 200, 513]
    t = Batch(total, [1] * len(total), Hkv, d, 16, bits, dtype, seed=10 * d + G)
    t.held[1] = (np.zeros((0, Hkv, d)),) * 2
    q = t.rows(Hkv * G)
    o = t.cache(cls).attend(q.cuda())
    ref, tol = t.attention(q)
    assert (o[1] == 0).all()
    assert_within(o, ref, tol, f"{bits} bits {dtype} d={d} G={G}")


@pytest.mark.parametrize("bits,dtype", FORMS)
@pytest.mark.parametrize("d,page", [(16, 64), (32, 32), (64, 128), (128, 16)])
@pytest.mark.parametrize("new,total", [((2, 1, 5, 0, 7), (2, 40, 129, 3, 300)),
                                       ((33, 1, 64, 90), (33, 700, 65, 401))])
def test_attention_several_tokens(cuda_lib, bits, dtype, d, page, new, total):
    """Ragged new tokens: causal among themselves, row tiles of 8, 16 and 32 rows."""
    cls = cuda_lib
    Hkv, G = 2, 3
    t = Batch(list(total), list(new), Hkv, d, page, bits, dtype, seed=d + len(new))
    q = t.rows(Hkv * G)
    cache = t.cache(cls)
    o = cache.attend(q.cuda(), cu_seqlens=t.cu.cuda())
    ref, tol = t.attention(q)
    assert_within(o, ref, tol, f"{bits} bits {dtype} d={d}")
    cache.check()


@pytest.mark.parametrize("bits,dtype", FORMS)
def test_attention_long_split(cuda_lib, bits, dtype):
    """Long sequences: every warp of the machine works on pieces of one; positions beyond 2^15."""
    cls = cuda_lib
    t = Batch([40001, 5, 9000], [1, 1, 1], 1, 64, 64, bits, dtype, seed=4)
    q = t.rows(4, std=3.0)
    o = t.cache(cls).attend(q.cuda())
    ref, tol = t.attention(q)
    assert_within(o, ref, tol, "long")


@pytest.mark.parametrize("bits,dtype", FORMS)
def test_attention_sharp_and_rising_scores(cuda_lib, bits, dtype):
    """Scores of tens, rising along the sequence (the running maximum moves many times), an
    explicit scale, and a sequence whose first keys are far below the rest."""
    cls = cuda_lib
    t = Batch([900, 700], [1, 3], 1, 32, 16, bits, dtype, seed=8, k_std=4.0)
    q = t.rows(2, std=2.0)
    for scale in (None, 0.7, -0.1, 1e-4):
        o = t.cache(cls).attend(q.cuda(), cu_seqlens=t.cu.cuda(), scale=scale)
        ref, tol = t.attention(q, scale)
        if scale is not None:
            tol = tol * (1 if abs(scale) <= 1 else abs(scale))
        assert_within(o, ref, tol, f"scale {scale}")


def test_attention_value_scales_apart(cuda_lib):
    """4 bits: value scales over nine binades within a sequence, ascending and descending, and
    all tiny; queries of very different size."""
    cls = cuda_lib
    forms = [lambda r, L: np.exp2(np.linspace(-9, 0, L)), lambda r, L: np.exp2(np.linspace(0, -9, L)),
             lambda r, L: np.full(L, 2.0 ** -9), lambda r, L: np.full(L, 2.0 ** 11)]
    for i, f in enumerate(forms):
        t = Batch([300, 70], [1, 2], 2, 64, 16, 4, torch.float16, seed=i, scale_of=f)
        q = t.rows(6)
        q[0] *= 2.0 ** -10
        q[1] *= 2.0 ** 3
        o = t.cache(cls).attend(q.cuda(), cu_seqlens=t.cu.cuda(),
                                out=torch.empty(3, 6, 64, device="cuda"))
        ref, tol = t.attention(q)
        assert_within(o, ref, tol, f"form {i}")


def test_attention_bfloat16_queries_beyond_float16(cuda_lib):
    """4-bit keys, bfloat16 queries of 1e-6 and 1e6: the products' power of two follows them."""
    cls = cuda_lib
    for size in (1e-6, 1e6):
        t = Batch([150], [1], 1, 64, 16, 4, torch.bfloat16, seed=2)
        q = t.rows(4, std=size)
        o = t.cache(cls).attend(q.cuda(), scale=0.125 / size)
        ref, tol = t.attention(q, 0.125 / size)
        assert_within(o, ref, tol, f"queries of {size}")


def test_attention_strides_types_and_untouched_rows(cuda_lib):
    cls = cuda_lib
    Hkv, G, d, n, B = 2, 2, 32, 3, 3
    t = Batch([40, 3, 129], [n] * B, Hkv, d, 16, 4, torch.float16, seed=3)
    q = t.rows(Hkv * G).cuda()
    cache = t.cache(cls)
    ref, tol = t.attention(q.cpu())
    # head-major strided queries, float32 strided output inside a larger buffer
    qs = q.view(B, n, Hkv * G, d).transpose(1, 2).contiguous().transpose(1, 2)
    big = torch.full((B, n + 2, Hkv * G + 1, d + 4), 9.0, device="cuda")
    cache.attend(qs, out=big[:, :n, :Hkv * G, :d])
    assert_within(big[:, :n, :Hkv * G, :d].reshape(B * n, Hkv * G, d), ref, tol, "strided")
    assert (big[:, n:] == 9).all() and (big[:, :, Hkv * G] == 9).all() and (big[..., d:] == 9).all()
    # packed with rows behind the last sequence
    wide = torch.cat([q, torch.full((5, Hkv * G, d), float("nan"), dtype=q.dtype, device="cuda")])
    out = torch.full_like(wide, 5.0)
    cache.attend(wide, cu_seqlens=t.cu.cuda(), out=out)
    assert_within(out[:B * n], ref, tol, "packed")
    assert (out[B * n:] == 5).all()
    for dt in (torch.bfloat16, torch.float32):
        o = cache.attend(q, out=torch.empty(q.shape, dtype=dt, device="cuda"))
        assert_within(o, ref, tol + np.abs(ref) * HALF_STEP[dt], str(dt))
    # one query broadcast to all heads and tokens (stride 0)
    qb = q[:1, :1].expand(B * n, Hkv * G, d)
    o = cache.attend(qb)
    ref, tol = t.attention(qb.cpu())
    assert_within(o, ref, tol, "broadcast")


def test_attention_positions_below_zero(cuda_lib):
    """More new tokens than the length counts: the first see nothing and get zeros."""
    cls = cuda_lib
    t = Batch([5, 0, 2], [3, 3, 3], 1, 16, 16, 16, torch.float16, seed=6)
    q = t.rows(2)
    o = t.cache(cls).attend(q.cuda())
    t.held[1] = (np.zeros((0, 1, 16)),) * 2
    ref, tol = t.attention(q)
    assert (o[3:6] == 0).all() and (o[6] == 0).all()
    assert_within(o, ref, tol, "below zero")


@pytest.mark.parametrize("bits", [4, 16])
def test_attention_nonfinite_rows_stay_with_those_who_see_them(cuda_lib, bits):
    """A NaN key or value in one sequence leaves the others alone, and tokens before it at 4 bits."""
    cls = cuda_lib
    t = Batch([70, 70], [4, 4], 1, 32, 16, bits, torch.float16, seed=7)
    cache = t.cache(cls)
    q = t.rows(2)
    clean = cache.attend(q.cuda()).clone()
    pg, sl = int(t.table[1, 68 // 16]), 68 % 16           # seen by the last two new tokens
    for which in (0, 1):
        c = t.cache(cls)
        if bits == 4:
            c.scales[pg, 0, sl, 2 * which] = float("nan")
        else:
            (c.v if which else c.k)[pg, 0, sl, 3] = float("nan")
        o = c.attend(q.cuda())
        assert torch.equal(o[:4], clean[:4])
        if bits == 4 or which == 0:
            assert torch.equal(o[4:6], clean[4:6])
        assert torch.isnan(o[6:]).any(-1).all()


@pytest.mark.parametrize("bits,dtype", [(4, torch.float16), (16, torch.float16)])
@pytest.mark.parametrize("B,Hkv,longest,page", [(300, 8, 400, 16), (200, 4, 200, 16), (129, 3, 700, 32), (4096, 1, 40, 64)])
def test_attention_many_sequences(cuda_lib, bits, dtype, B, Hkv, longest, page):
    """More items than warps, batches beyond one scan of a warp, the largest batch, tables so short
    that no item is split; empty slots in between."""
    cls = cuda_lib
    rng = np.random.default_rng(B)
    total = [int(x) for x in rng.integers(0, longest + 1, B)]
    total[0], total[-1] = longest, 0
    t = Batch(total, [1] * B, Hkv, 32, page, bits, dtype, seed=B)
    q = t.rows(2 * Hkv)
    cache = t.cache(cls)
    o = cache.attend(q.cuda())
    ref, tol = t.attention(q)
    assert_within(o, ref, tol, f"{B} sequences")
    cache.check()


def test_attention_infinite_scale_behind_the_row(cuda_lib):
    """A value scale of infinity in a later token's vector changes nothing for the tokens before it."""
    cls = cuda_lib
    t = Batch([70], [4], 1, 32, 16, 4, torch.float16, seed=7)
    q = t.rows(2)
    cache = t.cache(cls)
    ref, tol = t.attention(q)
    cache.scales[int(t.table[0, 68 // 16]), 0, 68 % 16, 2] = float("inf")
    o = cache.attend(q.cuda())
    assert_within(o[:2], ref[:2], tol[:2], "before it")
    assert not torch.isfinite(o[2:]).any()


def test_attention_rows_do_not_disturb_each_other(cuda_lib):
    """An infinite, a NaN and a huge query head beside ordinary ones (4 bits: the queries' power of
    two is each row's own)."""
    cls = cuda_lib
    for n, d in ((1, 32), (5, 64), (60, 64)):
        t = Batch([300], [n], 1, d, 16, 4, torch.bfloat16, seed=9)
        q = t.rows(8)
        clean = t.cache(cls).attend(q.cuda())
        q[:, 1, 3], q[:, 2, 5], q[:, 3] = float("inf"), float("nan"), q[:, 3] * 1e30
        o = t.cache(cls).attend(q.cuda())
        keep = [0, 4, 5, 6, 7]
        assert torch.equal(o[:, keep], clean[:, keep])
        assert torch.isnan(o[:, 1]).all() and torch.isnan(o[:, 2]).all()


def test_refusals_of_the_binding(cuda_lib):
    cls = cuda_lib
    t = Batch([20, 5], [1, 1], 2, 32, 16, 4, torch.float16)
    c = t.cache(cls)
    q, k = t.rows(4).cuda(), t.rows(2).cuda()
    bad = [lambda: c.attend(q.cpu()), lambda: c.attend(q[..., :16]), lambda: c.attend(q.double()),
           lambda: c.attend(q.view(1, 2, 4, 32)), lambda: c.attend(q, scale=0.0),
           lambda: c.attend(q, cu_seqlens=torch.zeros(3, dtype=torch.int64, device="cuda")),
           lambda: c.attend(q, cu_seqlens=torch.zeros(2, dtype=torch.int32, device="cuda")),
           lambda: c.attend(q, out=q[:1]), lambda: c.append(k, k[:, :1]), lambda: c.append(k, k, q[:1]),
           lambda: c.append(q, q), lambda: c.gather(), lambda: c.attend(q.transpose(-1, -2).contiguous().transpose(-1, -2)),
           lambda: cls.PagedCache.from_pages(c.k, c.v, c.page_table, c.lengths),
           lambda: cls.PagedCache.from_pages(c.k, c.v[:1], c.page_table, c.lengths, c.scales),
           lambda: cls.PagedCache.from_pages(c.k, c.v, c.page_table.long(), c.lengths, c.scales),
           lambda: cls.PagedCache.from_pages(c.k, c.v, c.page_table, c.lengths[:1], c.scales),
           lambda: cls.PagedCache.from_pages(c.k, c.v, c.page_table, c.lengths, c.scales[..., :2])]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            print(i)
    for f in (lambda: c.attend(t.rows(3).cuda()), lambda: c.attend(q, out=q), lambda: c.append(k, k, rope_base=0.5),
              lambda: c.attend(q, out=torch.empty(2, 1, 32, device="cuda").half().expand(2, 4, 32))):
        with pytest.raises(cls.CCAError):
            f()
    c.check()


def test_append_in_place_and_on_another_stream(cuda_lib):
    cls = cuda_lib
    t = Batch([20, 5], [1, 1], 2, 32, 16, 4, torch.float16)
    a, b = t.cache(cls), t.cache(cls)
    k, q = t.rows(2).cuda(), t.rows(4).cuda()
    want = a.append(k, k, q, rope_base=BASE)
    q2 = q.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = b.append(k, k, q2, rope_base=BASE, q_out=q2, stream=side)
    side.synchronize()
    assert got is q2 and torch.equal(q2, want) and torch.equal(a.k, b.k)


# many rows a sequence: the tensor-core kernel (4 bits, d~ >= 32)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d,page,G", [(32, 16, 4), (64, 64, 4), (64, 16, 3), (128, 32, 8), (64, 32, 1)])
@pytest.mark.parametrize("new,past", [((70, 300, 0, 1, 129), (0, 500, 9, 700, 33)), ((640, 3, 257), (1000, 0, 2)),
                                      ((40, 60, 200) * 30, (10, 0, 150) * 30)])
def test_attention_prompt_pieces(cuda_lib, dtype, d, page, G, new, past):
    """Ragged pieces beside single tokens and empty slots: row tiles and key tiles that end inside
    each other, runs that hold the end of one item and the start of the next."""
    cls = cuda_lib
    Hkv = 2
    if G == 1:
        new = tuple(2 * n for n in new)
    t = Batch([n + p for n, p in zip(new, past)], list(new), Hkv, d, page, 4, dtype, seed=d + G)
    q = t.rows(Hkv * G)
    cache = t.cache(cls)
    o = cache.attend(q.cuda(), cu_seqlens=t.cu.cuda())
    ref, tol = t.attention(q, tensor=True)
    assert_within(o, ref, tol, f"{dtype} d={d} G={G}")
    cache.check()
    again = cache.attend(q.cuda(), cu_seqlens=t.cu.cuda())
    assert torch.equal(o, again)


def test_attention_prompt_piece_long_and_split(cuda_lib):
    """One sequence: every CTA works on a piece of it; an explicit scale, of either sign; float32 out."""
    cls = cuda_lib
    t = Batch([6000], [130], 1, 64, 64, 4, torch.float16, seed=3, k_std=2.0)
    q = t.rows(4)
    for scale in (None, 0.3, -0.05):
        o = t.cache(cls).attend(q.cuda(), scale=scale, out=torch.empty(130, 4, 64, device="cuda"))
        ref, tol = t.attention(q, scale, tensor=True)
        assert_within(o, ref, tol, f"scale {scale}")


def test_attention_prompt_piece_positions_below_zero_and_extremes(cuda_lib):
    """Lengths below the new tokens; values at float16's end; tiny and huge bfloat16 queries."""
    cls = cuda_lib
    t = Batch([100, 0, 300], [200, 200, 200], 1, 64, 16, 4, torch.bfloat16, seed=5, v_std=15000.0)
    assert all(np.isfinite(v).all() for _, v in t.held)
    q = t.rows(2)
    q[:200] *= 1e-6
    q[400:] *= 1e5
    o = t.cache(cls).attend(q.cuda(), scale=1e-5, out=torch.empty(600, 2, 64, device="cuda"))
    t.held[1] = (np.zeros((0, 1, 64)),) * 2
    ref, tol = t.attention(q, 1e-5, tensor=True)
    assert (o[:100] == 0).all() and (o[200:400] == 0).all()
    assert_within(o, ref, tol + np.abs(ref) * 2.0 ** -24, "extremes")


@pytest.mark.parametrize("which", [0, 1, 2, 3])
def test_attention_prompt_piece_nonfinite_row(cuda_lib, which):
    """A NaN in a cached vector's scale or zero reaches the rows that see it and no others."""
    cls = cuda_lib
    t = Batch([300, 300], [200, 200], 1, 64, 16, 4, torch.float16, seed=7)
    cache = t.cache(cls)
    q = t.rows(2)
    clean = cache.attend(q.cuda()).clone()
    pos = 250                                              # new token 150 of the second sequence
    cache.scales[int(t.table[1, pos // 16]), 0, pos % 16, which] = float("nan")
    o = cache.attend(q.cuda())
    assert torch.equal(o[:350], clean[:350])
    assert torch.isnan(o[350:]).all()


# ------------------------------------------------------------------------------- kernel-side errors
def test_bad_pages_are_reported_and_read_as_zeros(cuda_lib):
    cls = cuda_lib
    for bits in (4, 16):
        t = Batch([40, 40], [1, 1], 1, 32, 16, bits, torch.float16, seed=11)
        for bad in (-1, int(t.k.shape[0]), 2 ** 31 - 1):
            cache = t.cache(cls)
            cache.page_table[1, 1] = bad
            q, k = t.rows(2).cuda(), t.rows(1).cuda()
            o = cache.attend(q)
            with pytest.raises(cls.CCAError) as e:
                cache.check()
            assert e.value.code == cls.CCA_ERR_PAGE
            t2 = Batch([40, 40], [1, 1], 1, 32, 16, bits, torch.float16, seed=11)
            for x in t2.held[1]:
                x[16:32] = 0
            if bits == 4:
                t2.vz[1][16:32] = 0
            ref, tol = t2.attention(q.cpu())
            assert_within(o, ref, tol, "bad page")
            cache.page_table[1, 1], cache.page_table[1, 2] = t.table[1, 1].item(), bad
            was = cache.k.clone()
            cache.append(k, k)
            with pytest.raises(cls.CCAError):
                cache.check()
            pg = int(t.table[0, 2])
            changed = (was.view(torch.uint8) != cache.k.view(torch.uint8)).flatten(1).any(1)
            assert changed.nonzero().flatten().tolist() == [pg]


def test_full_and_invalid_sequences(cuda_lib):
    cls = cuda_lib
    t = Batch([40, 33], [1, 1], 1, 32, 16, 4, torch.float16, seed=12)
    q, k = t.rows(2).cuda(), t.rows(1).cuda()
    ref, tol = t.attention(q.cpu())
    for length, code in ((49, cls.CCA_ERR_CACHE_FULL), (2 ** 31 - 1, cls.CCA_ERR_CACHE_FULL),
                         (-1, cls.CCA_ERR_PAGE), (-2 ** 31, cls.CCA_ERR_PAGE)):
        cache = t.cache(cls)
        cache.lengths[1] = length
        o = cache.attend(q)
        assert (o[1] == 0).all()
        assert_within(o[:1], ref[:1], tol[:1], "beside a bad length")
        with pytest.raises(cls.CCAError) as e:
            cache.check()
        assert e.value.code == code
        was = cache.k.clone()
        cache.append(k, k)
        with pytest.raises(cls.CCAError):
            cache.check()
        changed = (was != cache.k).flatten(1).any(1).nonzero().flatten().tolist()
        assert changed == [int(t.table[0, 2])]
    for cu in ([0, 1, 3], [0, 5, 2], [-1, 1, 2], [0, 1, -5]):
        cache = t.cache(cls)
        out = torch.full_like(q, 3.0)
        cache.attend(q, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"), out=out)
        with pytest.raises(cls.CCAError) as e:
            cache.check()
        assert e.value.code == cls.CCA_ERR_PAGE
        if cu[:2] == [0, 1]:
            assert_within(out[:1], ref[:1], tol[:1], "the valid sequence")
            assert (out[1] == 3).all()


@pytest.mark.parametrize("bits,d", [(4, 16), (4, 64), (16, 32)])
def test_overlapping_sequences_compute_nothing(cuda_lib, bits, d):
    """Row ranges of which one runs backwards and the others have more rows than the call: few
    rows, many, and units (rows x keys) beyond 32 bits between them."""
    cls = cuda_lib
    for B, pages, n, length in ((4, 8, 3, 40), (4, 8, 200, 512), (256, 2 ** 14, 2 ** 17, 2 ** 20)):
        cache = cls.PagedCache(B, pages, 64, 2, d, bits, n_pages=1)
        cache.lengths.fill_(length)
        q = torch.ones(n, 8, d, dtype=torch.float16, device="cuda")
        cu = torch.tensor([0, n] * (B // 2) + [0], dtype=torch.int32, device="cuda")
        out = torch.full_like(q, 3.0)
        cache.attend(q, cu_seqlens=cu, out=out)
        with pytest.raises(cls.CCAError) as e:
            cache.check()
        assert e.value.code == cls.CCA_ERR_PAGE
        assert (out == 3).all()
    # two sequences on the same rows, one row short of too many: computed
    cache = cls.PagedCache(3, 8, 64, 2, d, bits, n_pages=1)
    cache.lengths.fill_(40)
    q = torch.ones(4, 8, d, dtype=torch.float16, device="cuda")
    cu = torch.tensor([0, 2, 0, 2], dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 3.0)
    cache.attend(q, cu_seqlens=cu, out=out)
    assert (out[:2] == 0).all() and (out[2:] == 3).all()


# ------------------------------------------------------------------------------- together
def test_a_run_of_steps_streams_and_graphs(cuda_lib):
    """Prompt, then steps of one token: append + attend on a side stream, captured once and
    replayed with the lengths advanced on the device; two graphs in flight at once."""
    cls = cuda_lib
    B, Hkv, G, d, page = 3, 2, 4, 32, 16
    lens = [20, 1, 50]
    g = torch.Generator().manual_seed(0)
    mk = lambda: cls.PagedCache(B, 8, page, Hkv, d, bits=4)
    prompt = torch.randn(sum(lens), Hkv, d, generator=g).half().cuda()
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    steps = 5
    ks = torch.randn(steps, B, Hkv, d, generator=g).half().cuda()
    qs = torch.randn(steps, B, Hkv * G, d, generator=g).half().cuda()

    def start():
        c = mk()
        c.lengths.copy_(torch.tensor(lens, dtype=torch.int32))
        c.append(prompt, prompt * 0.5, cu_seqlens=cu, rope_base=BASE)
        return c

    eager, outs = start(), []
    for i in range(steps):
        eager.lengths += 1
        q = eager.append(ks[i], ks[i] * 0.5, qs[i], rope_base=BASE)
        outs.append(eager.attend(q))
    # float64, from the pages' own content
    tot = int(eager.lengths.sum())
    kcu = torch.tensor(np.concatenate([[0], np.cumsum(eager.lengths.cpu())]), dtype=torch.int32, device="cuda")
    kd, vd = eager.gather(tot, cu_seqlens=kcu, dtype=torch.float32)
    for b in range(B):
        a, e = int(kcu[b]), int(kcu[b + 1])
        pos = [e - a - 1]
        qr = P.rotate(qs[-1][b:b + 1].double().cpu().numpy(), pos, BASE)
        ref, mass, mag = P.attention(qr, kd[a:e].double().cpu().numpy(), vd[a:e].double().cpu().numpy(), d ** -0.5)
        # the queries' own rounding to float16 moves a score by 2^-11 of its magnitudes' sum
        tol = mass * 2 * (2.0 ** -11 * (1 + 2 * mag[..., None])) + np.abs(ref) * 2.0 ** -11 + 1e-4
        assert_within(outs[-1][b:b + 1], ref, tol, "the last step")
    # captured: two caches, each its own graph, replayed on two streams at once
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    caches = [start(), start()]
    kin = [torch.empty_like(ks[0]) for _ in side]
    qin = [torch.empty_like(qs[0]) for _ in side]
    graphs, gout = [], []
    torch.cuda.synchronize()
    for i, c in enumerate(caches):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=side[i]):
            c.lengths.add_(1)
            q = c.append(kin[i], kin[i] * 0.5, qin[i], rope_base=BASE)
            gout.append(c.attend(q))
        graphs.append(gr)
    for s in range(steps):
        for i in range(2):
            with torch.cuda.stream(side[i]):
                kin[i].copy_(ks[s])
                qin[i].copy_(qs[s])
                graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(gout[i], outs[s]), (s, i)
    for c in caches:
        assert torch.equal(c.k, eager.k) and torch.equal(c.scales, eager.scales)
        c.check()


def test_results_do_not_depend_on_timing(cuda_lib):
    cls = cuda_lib
    t = Batch([5000, 77, 1, 3000], [1, 1, 1, 1], 2, 64, 16, 4, torch.bfloat16, seed=13)
    cache, q = t.cache(cls), t.rows(8).cuda()
    first = cache.attend(q)
    other = torch.cuda.Stream()
    for i in range(20):
        o = cache.attend(q, stream=other if i % 2 else None)
        torch.cuda.synchronize()
        assert torch.equal(o, first)


# ------------------------------------------------------------------------------- the layer
@pytest.mark.parametrize("dl,kv,bits", [(16, 2, 4), (32, 4, 4), (64, 2, 4), (16, 4, 16), (32, 1, 16), (64, 2, 16)])
def test_layer_prefill_and_decode_over_pages(cuda_lib, dl, kv, bits):
    """CCALayer over a paged cache: y of every step against the oracle, attending over exactly
    what the pages hold; at 16 bits also against the dense cache."""
    cls = cuda_lib
    H = 8 if kv == 1 else 4
    w = W.Workload("paged", 3, 45, H * dl * 2, H, kv, 2)
    inp = W.make_inputs(w, seed=dl, conv_std=0.4)
    layer = cls.CCALayer.from_workload(w, inp)
    S0 = 40
    x = inp.x.cuda()
    paged = layer.new_paged_cache(w.batch, 4, 16, bits)
    dense = layer.new_cache(w.batch, 64)
    y0 = layer.prefill(x[:, :S0].contiguous(), cache=paged)
    y1 = layer.prefill(x[:, :S0].contiguous(), cache=dense)
    assert torch.equal(y0, y1)
    assert torch.equal(paged.conv_state, dense.conv_state) and torch.equal(paged.vshift_state, dense.vshift_state)
    cfg, ow = oracle_config(w), oracle_weights(oracle_config(w), inp)
    for i in range(S0, w.seq):
        xt = x[:, i].contiguous()
        cs, vs = f64(paged.conv_state), f64(paged.vshift_state)
        y = layer.decode(xt, paged)
        assert paged.lengths.tolist() == [i + 1] * w.batch
        kd, vd = paged.gather(w.batch * (i + 1), dtype=torch.float32)
        kd, vd = (f64(t).reshape(w.batch, i + 1, -1) for t in (kd, vd))
        ref = []
        for b in range(w.batch):
            pq, pk, pv = O.down_project(f64(xt[b:b + 1]), ow)
            q, k, v, _ = O.latent_qkv(cfg, ow, pq, pk, pv, np.array([i]), conv_history=cs[b],
                                      chan_history=np.zeros((0, cfg.n_q + cfg.n_kv)), vshift_prev=vs[b])
            if bits == 16:
                assert np.allclose(kd[b, i], k[0], atol=4e-3, rtol=2e-3)
                assert np.allclose(vd[b, i], v[0], atol=4e-3, rtol=2e-3)
            o = O.causal_attention(q, kd[b], vd[b], cfg, q_positions=np.array([i]))
            ref.append(O.up_project(o, ow)[0])
        assert bf16_err(f64(y), np.stack(ref)) <= BF16_TOL
        if bits == 16:
            yd = layer.decode(xt, dense)
            assert bf16_err(f64(y), f64(yd)) <= BF16_TOL
            assert torch.equal(paged.lengths, dense.lengths)
    paged.check()


def test_tp_shares_over_pages(cuda_lib):
    """Ranks of a tensor-parallel layer over their own pages: the shares add up to the layer's y."""
    cls = cuda_lib
    from compressed_latent_space_b200.tp import TPLayer
    w = W.Workload("paged", 2, 30, 256, 4, 2, 2)
    inp = W.make_inputs(w, seed=3, conv_std=0.4)
    x = inp.x.cuda()
    one = cls.CCALayer.from_workload(w, inp)
    c1 = one.new_paged_cache(2, 2, 16, 16)
    one.prefill(x[:, :29].contiguous(), cache=c1)
    y = one.decode(x[:, 29].contiguous(), c1)
    total = 0
    for rank in range(2):
        tp = TPLayer.from_workload(w, inp, 2, rank)
        c = tp.new_paged_cache(2, 2, 16, 16)
        tp.prefill_share(x[:, :29].contiguous(), cache=c)
        total = total + tp.decode_share(x[:, 29].contiguous(), c).float()
    assert bf16_err(f64(total), f64(y)) <= BF16_TOL


def test_layer_refuses_another_layers_pages(cuda_lib):
    cls = cuda_lib
    w = W.Workload("paged", 2, 32, 256, 4, 2, 2)
    layer = cls.CCALayer.from_workload(w, W.make_inputs(w))
    w2 = W.Workload("paged", 2, 32, 512, 8, 2, 2)
    other = cls.CCALayer.from_workload(w2, W.make_inputs(w2)).new_paged_cache(2, 2, 16)
    x = torch.zeros(2, 256, dtype=torch.bfloat16, device="cuda")
    mine = layer.new_paged_cache(2, 2, 16)
    for f in (lambda: layer.decode(x, other), lambda: layer.prefill(x[:, None], cache=other),
              lambda: layer.decode(x[:1], mine), lambda: layer.decode(x, cls.PagedCache(2, 2, 16, 2, 32)),
              lambda: layer.prefill(x[:, None].expand(2, 40, 256).contiguous(), cache=mine)):
        with pytest.raises(ValueError):
            f()


def test_layer_refuses_misplaced_states_and_rows(cuda_lib):
    cls = cuda_lib
    w = W.Workload("paged", 2, 32, 256, 4, 2, 2)
    layer = cls.CCALayer.from_workload(w, W.make_inputs(w))
    x = torch.zeros(2, 256, dtype=torch.bfloat16, device="cuda")
    for name in ("conv_state", "vshift_state"):
        for spoil in (lambda t: t[:1], lambda t: t.cpu(), lambda t: t.half(), lambda t: None,
                      lambda t: t.repeat_interleave(2, -1)[..., ::2]):
            c = layer.new_paged_cache(2, 2, 16)
            setattr(c, name, spoil(getattr(c, name)))
            for f in (lambda: layer.decode(x, c), lambda: layer.prefill(x[:, None], cache=c)):
                with pytest.raises(ValueError):
                    f()
    c = layer.new_paged_cache(2, 2, 16)
    wide = torch.zeros(2, 512, dtype=torch.bfloat16, device="cuda")
    for bad in (x.float(), x.cpu(), wide[:, ::2], wide):
        for f in (lambda: layer.decode(bad, c), lambda: layer.prefill(bad[:, None], cache=c),
                  lambda: layer.decode(x, c, out=bad),
                  lambda: layer.prefill(x[:, None], cache=c, out=bad[:, None])):
            with pytest.raises(ValueError):
                f()
    assert c.lengths.tolist() == [0, 0]


def test_replaced_lengths_and_table_are_used(cuda_lib):
    cls = cuda_lib
    g = torch.Generator().manual_seed(5)
    c = cls.PagedCache(2, 2, 16, 2, 32, 16)
    k, v = (torch.randn(2, 9, 2, 32, generator=g).half().cuda() for _ in range(2))
    c.lengths = torch.full((2,), 9, dtype=torch.int32, device="cuda")
    c.page_table = torch.tensor([[3, 0], [1, 2]], dtype=torch.int32, device="cuda")
    c.append(k, v)
    assert torch.equal(c.k[3, :, :9], k[0].transpose(0, 1))
    assert torch.equal(c.v[1, :, :9], v[1].transpose(0, 1))
    kd, vd = c.gather(18)
    assert torch.equal(kd.view(2, 9, 2, 32), k) and torch.equal(vd.view(2, 9, 2, 32), v)
    c.check()


def test_layer_paged_full_sequence_is_left_alone(cuda_lib):
    cls = cuda_lib
    w = W.Workload("paged", 2, 32, 256, 4, 2, 2)
    inp = W.make_inputs(w, seed=1, conv_std=0.4)
    layer = cls.CCALayer.from_workload(w, inp)
    x = inp.x.cuda()
    cache = layer.new_paged_cache(2, 2, 16, 4)
    layer.prefill(x[:, :31].contiguous(), cache=cache)
    cache.lengths[0] = 32                                  # sequence 0 is full
    k0, s0 = cache.k[:2].clone(), cache.conv_state[0].clone()
    y = layer.decode(x[:, 31].contiguous(), cache)
    assert (y[0] == 0).all() and (y[1] != 0).any()
    assert cache.lengths.tolist() == [32, 32]
    assert torch.equal(cache.k[:2], k0) and torch.equal(cache.conv_state[0], s0)
    with pytest.raises(cls.CCAError) as e:
        cache.check()
    assert e.value.code == cls.CCA_ERR_CACHE_FULL
