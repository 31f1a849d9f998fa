"""Host-side checks of the paged-cache calls that need no GPU: refusals before any launch, sizes,
the 4-bit form's own properties, and the oracle's pins."""
import ctypes
import os

import numpy as np
import pytest

import oracle.cca_oracle as O
import oracle.paged_oracle as P


@pytest.fixture(scope="module")
def cls():
    from compressed_latent_space_b200 import build
    build.build()
    import compressed_latent_space_b200 as c
    c.load()
    return c


def pages(c, **kw):
    base = dict(k=1 << 20, v=2 << 20, scales=3 << 20, page_table=4 << 20, lengths=5 << 20, status=None,
                batch=2, max_pages=4, n_pages=8, page_size=16, n_kv_heads=2, head_dim=32, bits=4,
                dtype=c.CCA_F16)
    base.update(kw)
    return c.cca_paged_cache_t(*[base[f] for f, _ in c.cca_paged_cache_t._fields_])


def rows(c, **kw):
    base = dict(ptr=6 << 20, dtype=c.CCA_F16, seq_stride=64, token_stride=64, head_stride=32)
    base.update(kw)
    return c.cca_rows_t(*[base[f] for f, _ in c.cca_rows_t._fields_])


def call(c, name, *args):
    conv = [ctypes.byref(a) if isinstance(a, ctypes.Structure) else a for a in args]
    rc = getattr(c.load(), name)(*conv)
    return rc


BAD_PAGES = [
    (dict(batch=0), -1), (dict(max_pages=-1), -1), (dict(n_pages=0), -1), (dict(page_size=0), -1),
    (dict(n_kv_heads=0), -1), (dict(bits=8), -1), (dict(bits=16, dtype=0), -1),
    (dict(head_dim=48), -2), (dict(head_dim=256), -2), (dict(page_size=8), -2), (dict(page_size=24), -2),
    (dict(page_size=8192), -2), (dict(max_pages=2 ** 21), -2), (dict(batch=4097), -2), (dict(n_kv_heads=4097), -2),
    (dict(n_pages=2 ** 27), -2), (dict(n_pages=2 ** 26, n_kv_heads=2), -2), (dict(k=None), -1), (dict(scales=None), -1),
    (dict(page_table=None), -1), (dict(lengths=None), -1), (dict(k=(1 << 20) + 8), -5),
    (dict(scales=(1 << 20) + 2), -5),
]


@pytest.mark.parametrize("kw,code", BAD_PAGES)
def test_invalid_caches_are_refused(cls, kw, code):
    p, r = pages(cls, **kw), rows(cls)
    assert call(cls, "cca_paged_append", p, None, r, r, None, 0, None, 2, 0.0, None) == code
    assert cls.cca_last_error_string() != ""
    assert call(cls, "cca_paged_gather", p, r, r, None, 2, None) == code
    assert call(cls, "cca_paged_attention", p, r, r, 2, None, 2, 0.0, 1 << 20, 1 << 30, None) == code
    assert cls.cca_paged_attention_workspace_size(p, 2, 2) == 0
    cfg = cls.make_config(256, 4, 2, 2)
    assert cls.cca_decode_step_paged_workspace_size(cfg, p) == 0


def test_invalid_rows_are_refused(cls):
    p, r = pages(cls), rows(cls)
    app = lambda q=None, k=r, v=r, qo=None, H=0, cu=None, n=2, base=0.0: call(
        cls, "cca_paged_append", p, q, k, v, qo, H, cu, n, base, None)
    assert app(k=None) == -1 and app(v=None) == -1
    assert app(q=r, H=4) == -1 and app(qo=r, H=4) == -1       # q without q_out, and the reverse
    assert app(q=r, qo=rows(cls, head_stride=32), H=3) == -1   # 3 heads over 2
    assert app(n=3) == -1 and app(n=-2) == -1                  # 3 tokens over 2 sequences
    assert app(base=1.0) == -1 and app(base=-1.0) == -1 and app(base=float("nan")) == -1
    assert app(base=float("inf")) == -1
    assert app(k=rows(cls, dtype=5)) == -1 and app(k=rows(cls, ptr=None)) == -1
    assert app(k=rows(cls, ptr=(6 << 20) + 2)) == -5 and app(k=rows(cls, token_stride=60)) == -5
    assert app(k=rows(cls, head_stride=-32)) == -1
    assert app(k=rows(cls, seq_stride=68)) == -5
    assert app(n=2 ** 26) == -2 and app(k=rows(cls, head_stride=2 ** 31)) == -2
    # rows of an output that overlap
    over = rows(cls, token_stride=16)
    assert app(q=r, qo=over, H=4, cu=1 << 20) == -1
    assert app(q=r, qo=rows(cls, head_stride=0), H=4) == -1
    assert app(q=r, qo=rows(cls, seq_stride=0), H=4) == -1
    assert call(cls, "cca_paged_gather", p, rows(cls, head_stride=16), r, None, 2, None) == -1
    out = rows(cls, ptr=7 << 20)
    assert call(cls, "cca_paged_attention", p, r, r, 4, None, 2, 0.0, 1 << 20, 1 << 30, None) == -1   # q is o
    att = lambda q=r, o=out, H=4, n=2, scale=0.0, ws=1 << 20, nb=1 << 30, pg=p: call(
        cls, "cca_paged_attention", pg, q, o, H, None, n, scale, ws, nb, None)
    assert att(H=3) == -1 and att(H=0) == -1 and att(q=None) == -1 and att(o=None) == -1
    assert att(scale=float("inf")) == -1 and att(scale=float("nan")) == -1
    assert att(q=rows(cls, dtype=cls.CCA_F32)) == -2
    assert att(q=rows(cls, dtype=cls.CCA_BF16), pg=pages(cls, bits=16, scales=None)) == -1
    assert att(ws=None) == -3 and att(nb=16) == -3 and att(ws=(1 << 20) + 4) == -5
    assert att(n=0) == 0 and app(n=0) == 0                     # nothing to do


def test_launch_failure_is_reported(cls, monkeypatch):
    monkeypatch.setenv("CCA_FAULT_INJECT", "launch")
    p, r = pages(cls), rows(cls)
    assert call(cls, "cca_paged_append", p, None, r, r, None, 0, None, 2, 0.0, None) == -6
    assert call(cls, "cca_paged_gather", p, r, r, None, 2, None) == -6
    assert call(cls, "cca_paged_attention", p, rows(cls, seq_stride=128, token_stride=128),
                rows(cls, ptr=7 << 20, seq_stride=128, token_stride=128), 4, None, 2, 0.0, 1 << 20, 1 << 30, None) == -6
    cfg, w = cls.make_config(256, 4, 2, 2), cls.cca_weights_t(1 << 20, 1 << 20, 1 << 20, 1 << 20)
    n = cls.cca_decode_step_paged_workspace_size(cfg, p)
    assert n > 0
    step = lambda pg=p, cf=cfg, nb=n, cs=1 << 20: call(
        cls, "cca_decode_step_paged", cf, w, 1 << 20, 1 << 20, pg, cs, 1 << 20, 1 << 20, nb, None)
    assert step() == -6
    assert step(nb=n - 1) == -3 and step(cs=None) == -1
    assert step(pg=pages(cls, n_kv_heads=4)) == -1 and step(pg=pages(cls, head_dim=64)) == -1
    assert step(pg=pages(cls, bits=16, scales=None, dtype=cls.CCA_BF16)) == -1
    assert step(cf=cls.make_config(256, 4, 2, 2, dtype=cls.CCA_F32)) == -2
    many = pages(cls, n_kv_heads=1, head_dim=16)
    assert step(pg=many, cf=cls.make_config(256, 16, 1, 1)) == -2        # 16 query heads on one


def test_workspace_grows_with_the_machine_not_the_capacity(cls):
    a = cls.cca_paged_attention_workspace_size(pages(cls, max_pages=2 ** 12), 2, 2)
    b = cls.cca_paged_attention_workspace_size(pages(cls, max_pages=2 ** 20), 2, 2)
    assert 0 < a <= b < 64 << 20


def test_quantise_properties():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((500, 64)).astype(np.float32)
    n, s, z = P.quantise4(x)
    assert n.min() == 0 and n.max() == 15
    held = P.dequantise4(n, s, z)
    rng_ = (x.max(-1) - x.min(-1))[:, None]
    assert (np.abs(held - x) <= rng_ / 30 * (1 + 2 ** -10) + (rng_ + np.abs(x.min(-1))[:, None]) * 2 ** -11).all()
    assert np.array_equal(P.unpack4(P.pack4(n)), n)
    again = P.quantise4(held)
    assert np.abs(P.dequantise4(*again) - held).max() <= 2 * np.abs(s).max()
    n, s, z = P.quantise4(np.full((1, 16), 2.5, np.float32))
    assert (n == 0).all() and s[0] == 0 and z[0] == 2.5
    for bad in (np.nan, np.inf, 1e6):
        y = np.zeros((1, 16), np.float32)
        y[0, 3] = bad
        assert np.isnan(P.dequantise4(*P.quantise4(y))).all()


def test_oracle_agrees_with_the_layer_oracle():
    rng = np.random.default_rng(1)
    n, H, Hkv, d = 5, 4, 2, 32
    cfg = O.OracleConfig(d_model=H * d, n_heads=H, n_kv_heads=Hkv, compression=1)
    x = rng.standard_normal((n, H, d))
    pos = np.array([0, 3, 7, 100, 4001])
    assert np.allclose(P.rotate(x, pos, 1e4).reshape(n, -1), O.rope_heads(x.reshape(n, -1), pos, H, d, 1e4))
    L = 9
    k, v = rng.standard_normal((L, Hkv, d)), rng.standard_normal((L, Hkv, d))
    o, mass, mag = P.attention(x, k, v, d ** -0.5)
    ref = O.causal_attention(x.reshape(n, -1), k.reshape(L, -1), v.reshape(L, -1), cfg,
                             q_positions=np.arange(L - n, L))
    assert np.allclose(o.reshape(n, -1), ref)
    assert (np.abs(o) <= mass + 1e-12).all()
    # a query before the first key
    o, _, _ = P.attention(x, k[:3], v[:3], 1.0)
    assert (o[:2] == 0).all() and (o[2] != 0).any()


def test_replaced_tensors_reach_the_calls(cls):
    import torch
    c = cls.PagedCache(2, 3, 16, 2, 16, 4, device="cpu")
    for name in ("k", "v", "page_table", "lengths", "scales", "status"):
        t = getattr(c, name).clone()
        setattr(c, name, t)
        assert getattr(c, name) is t
        assert getattr(c.struct, name) == t.data_ptr()
    c.lengths += 1
    assert c.lengths.tolist() == [1, 1] and c.struct.lengths == c.lengths.data_ptr()
    before, desc = c.lengths, bytes(c.struct)
    for bad in (torch.zeros(3, dtype=torch.int32), torch.zeros(2), None,
                torch.zeros(4, dtype=torch.int32)[::2]):
        with pytest.raises(ValueError):
            c.lengths = bad
        assert c.lengths is before and bytes(c.struct) == desc
    c.status = None
    assert not c.struct.status
    c.page_table = torch.zeros(2, 5, dtype=torch.int32)
    assert c.max_pages == 5 and c.struct.max_pages == 5
