"""Host-side checks of the latent cache's operators: RoPE table scalings, refused arguments, and the
float64 definitions the GPU tests compare with.  Nothing here launches a kernel."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

import dsa_indexer_cross_gb300 as D
from dsa_indexer_cross_gb300 import _lib
from oracle import latent_oracle as LO


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dsa_indexer_cross_gb300.build import build
    build()


@pytest.mark.parametrize("kind,kw", [
    ("none", {}), ("linear", dict(factor=4.0)), ("linear", dict(factor=1.0)),
    ("yarn", dict(factor=40.0, orig_len=4096, beta_fast=32.0, beta_slow=1.0)),
    ("yarn", dict(factor=8.0, orig_len=32768, beta_fast=16.0, beta_slow=2.0)),
    ("yarn", dict(factor=2.0, orig_len=7, beta_fast=1.0, beta_slow=1.0)),
])
@pytest.mark.parametrize("theta,dim,mscale", [(1e4, 64, 1.0), (8e6, 64, 1.1386294), (1e4, 6, 0.5)])
def test_scaled_rope_table(kind, kw, theta, dim, mscale):
    f = LO.rope_frequencies(theta, dim, kind, **kw)
    sc = {"none": lambda: D.RopeScaling(D.DSA_ROPE_SCALE_NONE, 0, 0.0, 0.0, 0.0, mscale),
          "linear": lambda: D.rope_scaling_linear(mscale=mscale, **kw),
          "yarn": lambda: D.rope_scaling_yarn(mscale=mscale, **kw)}[kind]()
    n = 70000
    tab = D.dsa_rope_table_scaled(theta, dim, n, sc).double().numpy()
    for p in (0, 1, 77, 65536, n - 1):
        # float64 angles differ by a few units of their last place; the table is rounded to 32 bits
        tol = 2.0 ** -24 * mscale + 8 * 2.0 ** -52 * max(1.0, p)
        assert np.all(np.abs(tab[p, :, 0] - mscale * np.cos(p * f)) <= tol)
        assert np.all(np.abs(tab[p, :, 1] - mscale * np.sin(p * f)) <= tol)


def test_unscaled_table_is_the_plain_table():
    assert torch.equal(D.dsa_rope_table_scaled(8e6, 64, 1000), D.dsa_rope_table(8e6, 64, 1000))
    none = D.RopeScaling(D.DSA_ROPE_SCALE_NONE, 0, 0.0, 0.0, 0.0, 1.0)
    assert torch.equal(D.dsa_rope_table_scaled(8e6, 64, 1000, none), D.dsa_rope_table(8e6, 64, 1000))


def test_yarn_keeps_fast_dims_and_interpolates_slow_ones():
    f0, f = LO.rope_frequencies(1e4, 64), LO.rope_frequencies(1e4, 64, "yarn", 16.0, 4096)
    assert f[0] == f0[0] and f[-1] == pytest.approx(f0[-1] / 16.0, rel=1e-12)
    assert np.all(np.diff(f / f0) <= 1e-15)


@pytest.mark.parametrize("bad", [dict(kind=3), dict(kind=-1), dict(mscale=0.0), dict(mscale=math.nan),
                                 dict(factor=0.5), dict(orig_len=0), dict(beta_slow=0.0), dict(beta_fast=0.5)])
def test_bad_scalings_are_refused(bad):
    a = dict(kind=2, orig_len=4096, factor=4.0, beta_fast=32.0, beta_slow=1.0, mscale=1.0)
    a.update(bad)
    with pytest.raises(D.DsaError) as e:
        D.dsa_rope_table_scaled(1e4, 64, 16, D.RopeScaling(*a.values()))
    assert e.value.name == "DSA_ERR_ARG"


def test_yarn_needs_a_base_above_one():
    with pytest.raises(D.DsaError):
        D.dsa_rope_table_scaled(1.0, 64, 16, D.rope_scaling_yarn(4.0, 4096))


# ------------------------------------------------------------------ the definitions themselves

def test_fp8_definition_matches_torch_and_rounds_within_half_a_step():
    v = LO.e4m3_values()
    t = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(v[~np.isnan(v)], t[~np.isnan(v)]) and np.array_equal(np.isnan(v), np.isnan(t))
    g = torch.Generator().manual_seed(3)
    x = (torch.randn((6, 512), generator=g) * torch.tensor([1e-30, 1e-3, 1.0, 30.0, 5e4, 3e38])[:, None]).to(torch.bfloat16)
    x64 = x.double().numpy()
    codes, scale = LO.fp8_encode(x64)
    y = LO.fp8_decode(codes, scale)
    e = scale.astype(np.float64).repeat(128, axis=1) - 127
    # a group in which a draw passed bf16's range holds an infinity and is stored as NaN
    finite = np.isfinite(x64).reshape(6, 4, 128).all(axis=2)
    assert np.array_equal(scale == 255, ~finite) and np.all(np.isnan(y[~finite.repeat(128, axis=1)]))
    ok = finite.repeat(128, axis=1)
    inside = (np.abs(x64) <= 448.0 * 2.0 ** 7) & ok
    err = np.abs(y - x64)
    assert np.all(err[inside] <= np.maximum(np.abs(x64) * 2.0 ** -4, 2.0 ** -10 * 2.0 ** e)[inside])
    assert np.all(np.abs(y[~inside & ok]) == 448.0 * 2.0 ** 7) and (~inside & ok).any()


def test_rope_definition_inverse_and_adjoint():
    rng = np.random.default_rng(0)
    x, y = rng.standard_normal((5, 8)), rng.standard_normal((5, 8))
    a = rng.standard_normal((5, 4))
    for inter in (False, True):
        fwd = LO.rope(x, np.cos(a), np.sin(a), inter, False)
        assert np.allclose(LO.rope(fwd, np.cos(a), np.sin(a), inter, True), x, atol=1e-14)
        # the inverse is the transpose, so it is the rotation's gradient
        assert np.sum(fwd * y) == pytest.approx(np.sum(x * LO.rope(y, np.cos(a), np.sin(a), inter, True)), abs=1e-12)


# ------------------------------------------------------------------ refused arguments

def _status(fn, *args):
    st = fn(*args)
    return _lib.STATUS_NAMES[st], D.lib().dsa_last_error().decode()


WS = 0x100000


def _rope(**kw):
    a = dict(n_tokens=4, n_heads=2, rope_dim=64, dtype=0, x_token_stride=128, x_head_stride=64, out_token_stride=128,
             out_head_stride=64, flags=0)
    a.update(kw)
    return _lib.RopeDesc(*a.values())


@pytest.mark.parametrize("kw,name", [
    (dict(n_tokens=-1), "DSA_ERR_ARG"), (dict(n_heads=0), "DSA_ERR_ARG"), (dict(rope_dim=3), "DSA_ERR_ARG"),
    (dict(rope_dim=0), "DSA_ERR_ARG"), (dict(rope_dim=514), "DSA_ERR_ARG"), (dict(dtype=2), "DSA_ERR_ARG"),
    (dict(flags=4), "DSA_ERR_ARG"), (dict(x_token_stride=-1), "DSA_ERR_ARG"), (dict(out_head_stride=32), "DSA_ERR_ARG"),
    (dict(out_token_stride=0), "DSA_ERR_ARG"), (dict(n_tokens=1 << 30, n_heads=4), "DSA_ERR_SHAPE"),
])
def test_rope_descriptors_refused(kw, name):
    d = _rope(**kw)
    assert _status(D.lib().dsa_rope_apply, C.byref(d), 0x1000, 0x2000, 0x3000, 8, 0x4000, WS, 256, None)[0] == name


@pytest.mark.parametrize("x,pos,cs,n_pos,out,ws,ws_bytes,name", [
    (None, 0x2000, 0x3000, 8, 0x4000, WS, 256, "DSA_ERR_ARG"), (0x1000, None, 0x3000, 8, 0x4000, WS, 256, "DSA_ERR_ARG"),
    (0x1000, 0x2000, None, 8, 0x4000, WS, 256, "DSA_ERR_ARG"), (0x1000, 0x2000, 0x3000, 0, 0x4000, WS, 256, "DSA_ERR_ARG"),
    (0x1000, 0x2000, 0x3000, 8, None, WS, 256, "DSA_ERR_ARG"), (0x1001, 0x2000, 0x3000, 8, 0x4000, WS, 256, "DSA_ERR_ARG"),
    (0x1000, 0x2000, 0x3004, 8, 0x4000, WS, 256, "DSA_ERR_ARG"), (0x1000, 0x2000, 0x3000, 8, 0x4000, None, 256, "DSA_ERR_ARG"),
    (0x1000, 0x2000, 0x3000, 8, 0x4000, WS + 16, 256, "DSA_ERR_ARG"), (0x1000, 0x2000, 0x3000, 8, 0x4000, WS, 255, "DSA_ERR_WORKSPACE"),
])
def test_rope_pointers_refused(x, pos, cs, n_pos, out, ws, ws_bytes, name):
    d = _rope()
    assert _status(D.lib().dsa_rope_apply, C.byref(d), x, pos, cs, n_pos, out, ws, ws_bytes, None)[0] == name


def test_rope_in_place_needs_equal_strides():
    d = _rope(out_token_stride=192)
    assert _status(D.lib().dsa_rope_apply, C.byref(d), 0x1000, 0x2000, 0x3000, 8, 0x1000, WS, 256, None)[0] == "DSA_ERR_ARG"


@pytest.mark.parametrize("kw", [dict(out_token_stride=64), dict(out_head_stride=65, out_token_stride=128),
                                dict(n_heads=3), dict(out_head_stride=255, out_token_stride=64)])
def test_rope_refuses_an_out_whose_heads_overlap(kw):
    d = _rope(**kw)
    st, msg = _status(D.lib().dsa_rope_apply, C.byref(d), 0x1000, 0x2000, 0x3000, 8, 0x4000, WS, 256, None)
    assert st == "DSA_ERR_ARG" and "out's heads" in msg


@pytest.mark.parametrize("kw", [dict(), dict(out_head_stride=256, out_token_stride=64), dict(n_heads=1, out_head_stride=0),
                                dict(n_tokens=1, out_token_stride=0), dict(out_token_stride=1 << 62, n_heads=1 << 20)])
def test_rope_accepts_token_and_head_major_outs(kw):
    """(refused for the missing workspace, which is looked at after the strides)"""
    d = _rope(**kw)
    st, msg = _status(D.lib().dsa_rope_apply, C.byref(d), 0x1000, 0x2000, 0x3000, 8, 0x4000, None, 256, None)
    assert st == "DSA_ERR_ARG" and "workspace" in msg


def test_rope_refuses_more_pairs_of_a_token_than_a_launch_turns():
    d = _rope(n_tokens=1, n_heads=1 << 27, rope_dim=64)
    assert _status(D.lib().dsa_rope_apply, C.byref(d), 0x1000, 0x2000, 0x3000, 8, 0x4000, WS, 256, None)[0] == "DSA_ERR_SHAPE"


def test_latent_attention_refuses_a_selection_beyond_int32_tiles():
    d = _lib.AttnDesc(2, 256, 16, 576, 512, (1 << 30) + 1, 0.04, 0)
    c, p = _cache(), _lib.PagedCache(0x4000, 0x5000, 2, 2, 128)
    got = _status(D.lib().dsa_latent_attn_paged, C.byref(d), 0x1000, C.byref(c), 0x6000, C.byref(p), 0x2000, None, WS, 1 << 40, None)
    assert got[0] == "DSA_ERR_SHAPE"


def _cache(**kw):
    a = dict(latent=0x10000, scale=0x20000, rope=0x30000, n_rows=256, format=1)
    a.update(kw)
    return _lib.LatentCache(*a.values())


BAD_CACHES = [
    (dict(format=2), "DSA_ERR_ARG"), (dict(latent=None), "DSA_ERR_ARG"), (dict(scale=None), "DSA_ERR_ARG"),
    (dict(rope=None), "DSA_ERR_ARG"), (dict(latent=0x10008), "DSA_ERR_ARG"), (dict(scale=0x20004), "DSA_ERR_ARG"),
    (dict(n_rows=0), "DSA_ERR_SHAPE"), (dict(n_rows=200), "DSA_ERR_SHAPE"),
]


@pytest.mark.parametrize("kw,name", BAD_CACHES)
def test_bad_caches_refused_everywhere(kw, name):
    c = _cache(**kw)
    w = _lib.CacheWriteDesc(4, 0, 576)
    p = _lib.PagedCache(0x40000, 0x50000, 2, max(1, c.n_rows // 128), 128)
    a = D.attn_desc(2, c.n_rows, 16, 0, 0.04)
    L = D.lib()
    assert _status(L.dsa_latent_cache_write, C.byref(w), 0x1000, 0x2000, None, None, 0, C.byref(c), WS, 256, None)[0] == name
    assert _status(L.dsa_latent_cache_read, C.byref(c), C.byref(p), 2, 0x2000, 0x3000, 10, WS, 256, None)[0] == name
    assert _status(L.dsa_latent_attn_paged, C.byref(a), 0x1000, C.byref(c), None, C.byref(p), 0x2000, None, WS, 1 << 40,
                   None)[0] == name


@pytest.mark.parametrize("desc,kv,slot,pos,cs,n_pos,name", [
    ((-1, 0, 576), 0x1000, 0x2000, None, None, 0, "DSA_ERR_ARG"), ((4, 0, 575), 0x1000, 0x2000, None, None, 0, "DSA_ERR_ARG"),
    ((4, 0, 580), 0x1000, 0x2000, None, None, 0, "DSA_ERR_ARG"), ((4, 2, 576), 0x1000, 0x2000, None, None, 0, "DSA_ERR_ARG"),
    ((4, 0, 576), None, 0x2000, None, None, 0, "DSA_ERR_ARG"), ((4, 0, 576), 0x1000, None, None, None, 0, "DSA_ERR_ARG"),
    ((4, 0, 576), 0x1008, 0x2000, None, None, 0, "DSA_ERR_ARG"), ((4, 256, 576), 0x1000, 0x2000, None, 0x4000, 8, "DSA_ERR_ARG"),
    ((4, 256, 576), 0x1000, 0x2000, 0x3000, None, 8, "DSA_ERR_ARG"), ((4, 256, 576), 0x1000, 0x2000, 0x3000, 0x4000, 0, "DSA_ERR_ARG"),
])
def test_cache_write_refused(desc, kv, slot, pos, cs, n_pos, name):
    d, c = _lib.CacheWriteDesc(*desc), _cache()
    assert _status(D.lib().dsa_latent_cache_write, C.byref(d), kv, slot, pos, cs, n_pos, C.byref(c), WS, 256, None)[0] == name


@pytest.mark.parametrize("pages,n_seq,start,out,n_out,name", [
    ((0x4000, 0x5000, 2, 2, 64), 1, 0x2000, 0x3000, 9, "DSA_ERR_UNSUPPORTED"),
    ((0x4000, 0x5000, 2, 3, 128), 1, 0x2000, 0x3000, 9, "DSA_ERR_SHAPE"),
    ((None, 0x5000, 2, 2, 128), 1, 0x2000, 0x3000, 9, "DSA_ERR_ARG"),
    ((0x4000, 0x5000, 0, 2, 128), 1, 0x2000, 0x3000, 9, "DSA_ERR_ARG"),
    ((0x4000, 0x5000, 1 << 20, 2, 128), 1 << 20, 0x2000, 0x3000, 9, "DSA_ERR_SHAPE"),
    ((0x4000, 0x5000, 1 << 25, 2, 128), 1, 0x2000, 0x3000, 9, "DSA_ERR_SHAPE"),
    ((0x4000, 0x5000, 2, 2, 128), -1, 0x2000, 0x3000, 9, "DSA_ERR_ARG"),
    ((0x4000, 0x5000, 2, 2, 128), 1, None, 0x3000, 9, "DSA_ERR_ARG"),
    ((0x4000, 0x5000, 2, 2, 128), 1, 0x2000, 0x3008, 9, "DSA_ERR_ARG"),
])
def test_cache_read_refused(pages, n_seq, start, out, n_out, name):
    c, p = _cache(), _lib.PagedCache(*pages)
    assert _status(D.lib().dsa_latent_cache_read, C.byref(c), C.byref(p), n_seq, start, out, n_out, WS, 256, None)[0] == name


@pytest.mark.parametrize("kw,idx,name", [
    (dict(n_heads=129), None, "DSA_ERR_UNSUPPORTED"), (dict(d_qk=192), None, "DSA_ERR_UNSUPPORTED"),
    (dict(n_kv=128), None, "DSA_ERR_SHAPE"), (dict(softmax_scale=0.0), None, "DSA_ERR_ARG"),
    (dict(topk=0), 0x6000, "DSA_ERR_ARG"), (dict(flags=1), None, "DSA_ERR_ARG"), (dict(n_q=-1), None, "DSA_ERR_ARG"),
    (dict(n_q=1 << 25, n_heads=128), None, "DSA_ERR_SHAPE"),
])
def test_latent_attention_refused(kw, idx, name):
    a = dict(n_q=2, n_kv=256, n_heads=16, d_qk=576, d_v=512, topk=8, softmax_scale=0.04, flags=0)
    a.update(kw)
    d, c, p = _lib.AttnDesc(*a.values()), _cache(), _lib.PagedCache(0x4000, 0x5000, 2, 2, 128)
    got = _status(D.lib().dsa_latent_attn_paged, C.byref(d), 0x1000, C.byref(c), idx, C.byref(p), 0x2000, None, WS, 1 << 40, None)
    assert got[0] == name


def test_latent_attention_workspace():
    a = D.attn_desc(64, 1 << 20, 128, 0, 0.04)
    n = D.dsa_latent_attn_workspace_size(a)
    assert n % 256 == 0 and n > 152 * 128 * 2048       # the partial outputs of a fully split call
    assert n < 128 << 20
    with pytest.raises(D.DsaError):
        D.dsa_latent_attn_workspace_size(D.attn_desc(64, 1 << 20, 0, 0, 0.04))


def test_binding_checks_views():
    x = torch.zeros((3, 2, 192), dtype=torch.bfloat16)
    o = torch.zeros((3, 2, 576), dtype=torch.bfloat16)
    d = D.rope_desc(x[..., 128:], o[..., 512:])
    assert (d.x_token_stride, d.x_head_stride, d.out_token_stride, d.out_head_stride) == (384, 192, 1152, 576)
    with pytest.raises(ValueError):
        D.rope_desc(x, o)
    with pytest.raises(ValueError):
        D.rope_desc(x.half(), x.half())
    with pytest.raises(ValueError):
        D.rope_desc(x.transpose(1, 2)[:, :2], x.transpose(1, 2)[:, :2])
    with pytest.raises(ValueError):      # host tensors are refused before their address is used
        D.dsa_rope_apply(d, x[..., 128:], torch.zeros(3, dtype=torch.int32), D.dsa_rope_table(1e4, 64, 4), o[..., 512:])
    with pytest.raises(ValueError):
        D.cache_write_desc(torch.zeros((4, 640), dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        D.latent_cache(torch.zeros((128, 512), dtype=torch.bfloat16))


@pytest.mark.parametrize("name", ["latent_cache.cu", "latent_attn.cu", "latent_attn.cuh", "latent_pair.cu", "fp8.cuh"])
def test_overlapped_kernels_read_memory_with_ordinary_loads(name):
    """Every kernel of these files is resident while the one before it still writes, so none of what it
    reads is read-only for its lifetime: no non-coherent load, and no const pointer that the compiler may
    read with one."""
    import os
    import re
    with open(os.path.join(os.path.dirname(_lib.__file__), "csrc", name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert not re.search(r"__ldg\b|\.nc\b|__restrict__|ld\.global\.nc", code)


def test_an_empty_batch_needs_no_tables():
    """(the address of an empty tensor is NULL)"""
    L, c = D.lib(), _cache()
    p = _lib.PagedCache(None, None, 2, 2, 128)
    d = D.attn_desc(0, 256, 16, 8, 0.04)
    for idx in (None, 0x6000):
        assert _status(L.dsa_latent_attn_paged, C.byref(d), None, C.byref(c), idx, C.byref(p), None, None, None, 0, None)[0] == "DSA_OK"
    assert _status(L.dsa_sparse_attn_paged, C.byref(d), None, None, None, C.byref(p), None, None, None, 0, None)[0] == "DSA_OK"
    n = D.indexer_desc(0, 256, 64, 128, 64, 8, 256, D.DSA_IDX_ROPE_Q | D.DSA_IDX_INDEPENDENT_ROWS)
    assert _status(L.dsa_indexer_topk_paged, C.byref(n), None, None, None, None, C.byref(p), None, 0, None, None, None, 0, None)[0] == "DSA_OK"
    d = D.attn_desc(2, 256, 16, 8, 0.04)
    assert _status(L.dsa_latent_attn_paged, C.byref(d), 0x1000, C.byref(c), None, C.byref(p), 0x2000, None, WS, 1 << 40, None)[0] == "DSA_ERR_ARG"
    with pytest.raises(ValueError, match="must be set"):
        _lib._paged_args(p, 1)
    _lib._paged_args(p, 0)


class _Placed:
    """As much of a tensor as the binding looks at, on a device of choice."""

    def __init__(self, t, dev):
        self.t, self.dev, self.is_cuda, self.dtype, self.device = t, dev, True, t.dtype, f"cuda:{dev}"

    def get_device(self):
        return self.dev

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_page_tables_are_checked_before_a_kernel_reads_them():
    z = lambda dt, *s: _Placed(torch.zeros(s, dtype=dt), 0)  # noqa: E731
    i32 = torch.int32
    for bt, ln in ((z(torch.int64, 3, 4), z(i32, 3)), (z(i32, 3, 4), z(torch.int64, 3)), (z(i32, 12), z(i32, 3))):
        with pytest.raises(ValueError, match="block_table|seq_len"):
            D.paged_cache(bt, ln, 9)
    with pytest.raises(ValueError, match="CUDA"):
        D.paged_cache(torch.zeros((3, 4), dtype=i32), torch.zeros(3, dtype=i32), 9)
    with pytest.raises(ValueError, match="one device"):
        D.paged_cache(z(i32, 3, 4), _Placed(torch.zeros(3, dtype=i32), 1), 9)
    for n_table, n_len in ((3, 5), (5, 3)):
        pages = D.paged_cache(z(i32, n_table, 4), z(i32, n_len), 9)
        assert (pages.rows, pages.device, pages.max_pages) == (3, 0, 4)
        _lib._paged_args(pages, 3)
        with pytest.raises(ValueError, match="a call of 4 rows"):
            _lib._paged_args(pages, 4)
    # a handle made by hand says nothing of its rows
    _lib._paged_args(_lib.PagedCache(0x4000, 0x5000, 2, 2, 128), 1 << 20)


def test_every_tensor_of_a_call_is_on_the_current_device(monkeypatch):
    bf, i32, u8, f32 = torch.bfloat16, torch.int32, torch.uint8, torch.float32
    monkeypatch.setattr(_lib, "_device", lambda: 0)
    at = lambda t, here: _Placed(t, 0 if here else 1)  # noqa: E731
    tab, ws = torch.zeros((4, 32, 2)), torch.zeros(256, dtype=u8)
    attn = dict(q=torch.zeros((2, 16, 576), dtype=bf), rows=torch.zeros((256, 576), dtype=bf), idx=torch.zeros((2, 8), dtype=i32),
                bt=torch.zeros((2, 2), dtype=i32), ln=torch.zeros(2, dtype=i32), out=torch.zeros((2, 16, 512), dtype=bf),
                lse=torch.zeros((2, 16)), ws=ws)
    read = dict(rows=attn["rows"], bt=attn["bt"], ln=attn["ln"], start=torch.zeros(2, dtype=i32), out=torch.zeros((9, 576), dtype=bf), ws=ws)
    write = dict(kv=torch.zeros((2, 576), dtype=bf), slot=torch.zeros(2, dtype=i32), pos=torch.zeros(2, dtype=i32), tab=tab,
                 codes=torch.zeros((256, 512), dtype=u8), scale=torch.zeros((256, 4), dtype=u8), rope=torch.zeros((256, 64), dtype=bf), ws=ws)
    rope = dict(x=torch.zeros((2, 3, 64)), pos=write["pos"], tab=tab, out=torch.zeros((2, 3, 64)), ws=ws)

    def call_attn(q, rows, idx, bt, ln, out, lse, ws):
        D.dsa_latent_attn_paged(D.attn_desc(2, 256, 16, 8, 0.04), q, D.latent_cache(rows), idx, D.paged_cache(bt, ln, 2), out, lse, ws=ws)

    def call_read(rows, bt, ln, start, out, ws):
        D.dsa_latent_cache_read(D.latent_cache(rows), D.paged_cache(bt, ln, 2), 2, start, out, ws=ws)

    def call_write(kv, slot, pos, tab, codes, scale, rope, ws):
        D.dsa_latent_cache_write(D.cache_write_desc(kv, D.DSA_CACHE_ROPE), kv, slot, pos, tab, D.latent_cache(codes, scale, rope), ws=ws)

    def call_rope(x, pos, tab, out, ws):
        D.dsa_rope_apply(D.rope_desc(x, out), x, pos, tab, out, ws=ws)
    reached = []
    monkeypatch.setattr(_lib, "_stream", lambda s: reached.append(1) or (_ for _ in ()).throw(StopIteration))
    for call, tensors in ((call_attn, attn), (call_read, read), (call_write, write), (call_rope, rope)):
        with pytest.raises((StopIteration, RuntimeError)):       # all in place: as far as the launch
            call(**{k: at(t, True) for k, t in tensors.items()})
        assert reached.pop()
        for other in tensors:
            with pytest.raises(ValueError, match="cuda:1"):
                call(**{k: at(t, k != other) for k, t in tensors.items()})
            assert not reached


def test_strides_of_a_single_token_or_head_are_not_looked_at():
    """Views of one row carry whatever stride they were cut with."""
    one = torch.zeros((5, 1001), dtype=torch.bfloat16)[2:3, :576]
    for kv, stride in ((one, 576), (one[:0], 576), (torch.zeros((1, 2000), dtype=torch.bfloat16)[:, :576], 576),
                       (torch.zeros((2, 640), dtype=torch.bfloat16)[:, :576], 640)):
        assert D.cache_write_desc(kv).kv_stride == stride
    d = _rope(n_tokens=1, x_token_stride=7, out_token_stride=192)            # in place: the missing workspace is met
    st, msg = _status(D.lib().dsa_rope_apply, C.byref(d), 0x1000, 0x2000, 0x3000, 8, 0x1000, None, 256, None)
    assert st == "DSA_ERR_ARG" and "workspace" in msg
    d = _rope(n_heads=1, x_head_stride=-3, out_head_stride=1)
    st, msg = _status(D.lib().dsa_rope_apply, C.byref(d), 0x1000, 0x2000, 0x3000, 8, 0x1000, None, 256, None)
    assert st == "DSA_ERR_ARG" and "workspace" in msg
    bf, x = torch.bfloat16, torch.zeros((4, 3, 64))
    for t, ok in ((x, True), (torch.zeros((4, 9, 64))[:, ::3], False), (torch.zeros((4, 3, 70))[..., :64], False)):
        try:
            _lib._rope_view(_Placed(t, 0), torch.float32, (4, 3, 64), 192, 64, "x", 0)
            assert ok
        except ValueError as e:
            assert not ok and "strides" in str(e)
    head = torch.zeros((4, 9, 64), dtype=bf)[:, 4:5]
    _lib._rope_view(_Placed(head, 0), bf, (4, 1, 64), 576, 1234, "x", 0)
    _lib._rope_view(_Placed(head[1:2], 0), bf, (1, 1, 64), 1, 1234, "x", 0)
    with pytest.raises(ValueError, match="strides"):
        _lib._rope_view(_Placed(head, 0), bf, (4, 1, 64), 64, 64, "x", 0)
