"""GPU tests of rotary positions and of the latent cache's writing and reading back, against the
float64 definitions in oracle/latent_oracle.py.

Tolerances.  A rotation is two fp32 products and a sum: |error| <= 2^-23 (|a c| + |b s|) + half a step
of the output type (2^-8 of the value for bf16, 2^-24 for fp32).  Codes, scale bytes and rows read
back are exact."""
import numpy as np
import pytest
import torch

import dsa_indexer_cross_gb300 as D
from latent_cases import DEV, P, Paged, encode, gen, i32, randn
from oracle import latent_oracle as LO

pytestmark = pytest.mark.gpu
THETA = 8e6


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dsa_indexer_cross_gb300.build import build
    build()
    assert torch.cuda.is_available()


def _check_turned(got, x, cs, inter, inverse, eps_half):
    c, s = cs[..., 0], cs[..., 1]
    want = LO.rope(x, c, s, inter, inverse)
    mag = LO.rope(np.abs(x), np.abs(c), np.abs(s), inter, False)      # upper pair: |a||c| - |b||s|; use the sum
    half = x.shape[-1] // 2
    both = np.empty_like(mag)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + half)
        both[..., a] = np.abs(x[..., a] * c[..., i]) + np.abs(x[..., b] * s[..., i])
        both[..., b] = np.abs(x[..., a] * s[..., i]) + np.abs(x[..., b] * c[..., i])
    tol = 2.0 ** -23 * both + eps_half * np.abs(want) * (1 + 2.0 ** -7) + 1e-38
    assert np.all(np.abs(got - want) <= tol), float(np.max(np.abs(got - want) / tol))


# (tokens, heads, width in, offset in, width out, offset out, rope): vector paths, and every reason
# to leave them (odd widths, unaligned offsets, rope not a multiple of the vector)
ROPE_SHAPES = [(1, 1, 64, 0, 64, 0, 64), (3, 128, 192, 128, 576, 512, 64), (257, 5, 576, 512, 192, 128, 64),
               (70, 4, 128, 64, 64, 0, 64), (9, 3, 66, 2, 70, 6, 64), (5, 2, 21, 1, 33, 3, 18), (4, 7, 2, 0, 2, 0, 2),
               (33, 1, 40, 8, 24, 8, 16), (2, 3, 512, 0, 512, 0, 512), (6, 2, 104, 0, 104, 0, 100)]


@pytest.mark.parametrize("dtype,eps_half", [(torch.bfloat16, 2.0 ** -8), (torch.float32, 2.0 ** -24)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("shape", ROPE_SHAPES)
def test_rope_apply(shape, inter, inverse, dtype, eps_half):
    n, h, wi, oi, wo, oo, r = shape
    g = gen(n * 31 + h)
    x = torch.randn((n, h, wi), generator=g, device=DEV).to(dtype)
    out = torch.randn((n, h, wo), generator=g, device=DEV).to(dtype)
    before = out.clone()
    tab = D.dsa_rope_table(THETA, r, 3000).to(DEV)
    pos = torch.randint(0, 3000, (n,), generator=g, device=DEV, dtype=torch.int32)
    pos[0] = 2999
    xv, ov = x[..., oi:oi + r], out[..., oo:oo + r]
    flags = (D.DSA_ROPE_INTERLEAVED if inter else 0) | (D.DSA_ROPE_INVERSE if inverse else 0)
    ws = D.dsa_rope_apply(D.rope_desc(xv, ov, flags), xv, pos, tab, ov)
    assert D.dsa_workspace_status(ws) == 0
    cs = tab.double().cpu().numpy()[pos.cpu().numpy()][:, None]
    _check_turned(ov.double().cpu().numpy(), xv.double().cpu().numpy(), cs, inter, inverse, eps_half)
    before[..., oo:oo + r] = ov
    assert torch.equal(before, out)                  # the other dims stay as they were
    # in place gives the same bits
    y = x.clone()
    yv = y[..., oi:oi + r]
    D.dsa_rope_apply(D.rope_desc(yv, yv, flags), yv, pos, tab, yv)
    assert torch.equal(yv, ov)


def test_rope_is_undone_by_its_inverse_and_is_its_own_gradient():
    g = gen(5)
    n, h = 40, 6
    x, y = (torch.randn((n, h, 64), generator=g, device=DEV) for _ in range(2))
    tab = D.dsa_rope_table_scaled(1e4, 64, 5000, D.rope_scaling_yarn(40.0, 4096)).to(DEV)
    pos = torch.randint(0, 5000, (n,), generator=g, device=DEV, dtype=torch.int32)
    for flag in (0, D.DSA_ROPE_INTERLEAVED):
        fx, back, gy = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
        D.dsa_rope_apply(D.rope_desc(x, fx, flag), x, pos, tab, fx)
        inv = D.rope_desc(x, fx, flag | D.DSA_ROPE_INVERSE)
        D.dsa_rope_apply(inv, fx, pos, tab, back)
        # two rotations, each off by 2^-23 (|a| + |b|) + 2^-24, of values of at most |x| sqrt 2; the
        # table's c^2 + s^2 is within 2^-22 of one
        assert float((back - x).abs().max()) <= 2.0 ** -20 * float(x.abs().max())
        D.dsa_rope_apply(inv, y, pos, tab, gy)
        # the gradient of sum(y * rope(x)): central differences of a linear map are exact up to rounding
        lhs, rhs = (fx.double() * y.double()).sum(), (x.double() * gy.double()).sum()
        assert abs(float(lhs - rhs)) <= 2.0 ** -22 * float((fx.double().abs() * y.double().abs()).sum() * 4)
        e = torch.zeros_like(x)
        e[3, 2, 10] = 0.5
        up, dn = torch.empty_like(x), torch.empty_like(x)
        D.dsa_rope_apply(D.rope_desc(x, fx, flag), x + e, pos, tab, up)
        D.dsa_rope_apply(D.rope_desc(x, fx, flag), x - e, pos, tab, dn)
        slope = float(((up.double() - dn.double()) * y.double()).sum())
        # two pairs' differences of values rounded to 2^-24 of at most 8
        assert abs(slope - float(gy[3, 2, 10])) <= 2.0 ** -18 * (1 + float(y[3, 2].abs().max()))


def test_rope_skips_and_flags_positions_outside_the_table():
    x = torch.ones((4, 2, 64), device=DEV)
    out = torch.full_like(x, 9.0)
    tab = D.dsa_rope_table(THETA, 64, 10).to(DEV)
    ws = D.dsa_rope_apply(D.rope_desc(x, out), x, i32([0, 10, -1, 3]), tab, out)
    assert D.dsa_workspace_status(ws, raise_on_fault=False) == 2
    assert torch.all(out[1:3] == 9.0) and torch.equal(out[0], x[0]) and not torch.any(out[3] == 9.0)
    ws = D.dsa_rope_apply(D.rope_desc(x, out), x, i32([0, 9, 1, 3]), tab, out, ws=ws)
    assert D.dsa_workspace_status(ws) == 0
    e = torch.empty((0, 2, 64), device=DEV)
    D.dsa_rope_apply(D.rope_desc(e, e), e, i32([]), tab, e)


@pytest.mark.parametrize("rope,offset", [(512, 0), (510, 1)])
def test_rope_of_more_pairs_than_one_launch_turns(rope, offset):
    """2^31 pairs and more of few tokens (odd widths: one a thread): several launches, one status.  x is
    one token's heads for all (a stride of zero); a token outside the table lies in the last launch."""
    n, h = 260, 32768 + 700
    g = gen(77)
    x = torch.randn((h, 512), generator=g, device=DEV).to(torch.bfloat16)[:, offset:offset + rope].expand(n, h, rope)
    out = torch.full((n, h, 512), 3.0, dtype=torch.bfloat16, device=DEV)
    ov = out[..., offset:offset + rope]
    tab = D.dsa_rope_table(THETA, rope, 50).to(DEV)
    pos = torch.randint(0, 50, (n,), generator=g, device=DEV, dtype=torch.int32)
    pos[258] = 50
    ws = D.dsa_rope_apply(D.rope_desc(x, ov), x, pos, tab, ov)
    assert D.dsa_workspace_status(ws, raise_on_fault=False) == 2
    for t in (0, 100, 255, 256, 257, 259):
        hs = torch.tensor([0, 1, h // 2, h - 1], device=DEV)
        cs = tab.double().cpu().numpy()[int(pos[t])][None]
        _check_turned(ov[t, hs].double().cpu().numpy(), x[t, hs].double().cpu().numpy(), cs, False, False, 2.0 ** -8)
    assert torch.all(out[258] == 3.0)
    assert torch.all(out[..., :offset] == 3.0) and torch.all(out[..., offset + rope:] == 3.0)


def _write(kv, slot, fmt, n_pages, pos=None, tab=None, flags=0):
    n_rows = n_pages * P
    if fmt == "bf16":
        bufs = [torch.full((n_rows, 576), 5.0, dtype=torch.bfloat16, device=DEV)]
    else:
        bufs = [torch.full((n_rows, 512), 0x31, dtype=torch.uint8, device=DEV),
                torch.full((n_rows, 4), 99, dtype=torch.uint8, device=DEV),
                torch.full((n_rows, 64), 5.0, dtype=torch.bfloat16, device=DEV)]
    ws = D.dsa_latent_cache_write(D.cache_write_desc(kv, flags), kv, slot, pos, tab, D.latent_cache(*bufs))
    return bufs, D.dsa_workspace_status(ws, raise_on_fault=False)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("n,stride,rot", [(1, 576, None), (7, 576, False), (129, 640, True), (300, 576, None), (64, 1152, False)])
def test_cache_write(fmt, n, stride, rot):
    """rot: None = stored as given, else turned in the half (False) or interleaved (True) layout."""
    g = gen(n)
    kv = randn((n, stride), g)[:, :576]
    kv = kv * (10.0 ** torch.randint(-6, 5, (n, 1), generator=g, device=DEV)).to(torch.bfloat16)
    kv = torch.nn.functional.pad(kv, (0, stride - 576))[:, :576]
    assert n == 1 or kv.stride(0) == stride
    n_pages = (n + P - 1) // P + 2
    slot = torch.randperm(n_pages * P, generator=g, device=DEV)[:n].to(torch.int32)
    if n > 5:
        slot[2], slot[n - 1] = -1, -5
    tab = D.dsa_rope_table(THETA, 64, 4000).to(DEV)
    pos = torch.randint(0, 4000, (n,), generator=g, device=DEV, dtype=torch.int32)
    flags = 0 if rot is None else D.DSA_CACHE_ROPE | (D.DSA_ROPE_INTERLEAVED if rot else 0)
    bufs, bits = _write(kv, slot, fmt, n_pages, pos if flags else None, tab if flags else None, flags)
    assert bits == 0
    keep = (slot >= 0).cpu().numpy()
    at = slot.cpu().numpy()[keep].astype(np.int64)
    x = kv.double().cpu().numpy()[keep]
    rope = (bufs[0][:, 512:] if fmt == "bf16" else bufs[2]).double().cpu().numpy()
    if rot is None:
        assert np.array_equal(rope[at], x[:, 512:])
    else:
        _check_turned(rope[at], x[:, 512:], tab.double().cpu().numpy()[pos.cpu().numpy()[keep]], rot, False, 2.0 ** -8)
    if fmt == "bf16":
        assert np.array_equal(bufs[0][:, :512].double().cpu().numpy()[at], x[:, :512])
    else:
        codes, scale = LO.fp8_encode(x[:, :512])
        assert np.array_equal(bufs[1].cpu().numpy()[at], scale)
        assert np.array_equal(bufs[0].cpu().numpy()[at], codes)
        c2, s2 = encode(kv[torch.as_tensor(keep, device=DEV)][:, :512])      # the helper the other tests use
        assert np.array_equal(c2.cpu().numpy(), codes) and np.array_equal(s2.cpu().numpy(), scale)
    other = np.ones(n_pages * P, dtype=bool)
    other[at] = False
    for b, v in zip(bufs, (5.0,) if fmt == "bf16" else (0x31, 99, 5.0)):
        assert np.all(b.double().cpu().numpy()[other] == v)


def test_cache_write_special_values():
    kv = torch.zeros((8, 576), dtype=torch.bfloat16, device=DEV)
    kv[0, 5] = float("inf")               # group 0 of token 0 becomes NaN, the others are zero
    kv[1, 200] = float("nan")
    kv[2, :] = 3.0e38                     # saturates
    kv[3, :] = 2.0 ** -133                # the smallest bf16
    kv[4, 0], kv[4, 1] = 448.0, 449.0     # scale borders
    kv[5, 0] = 450.0
    kv[6, 0], kv[6, 1], kv[6, 2] = 1.0, 2.0 ** -17, -(2.0 ** -19)      # subnormal codes and ties
    kv[7, 512] = float("nan")             # the rotary dims are stored as they are
    bufs, bits = _write(kv, i32(np.arange(8)), "fp8", 1)
    assert bits == 0
    x = kv.double().cpu().numpy()[:, :512]
    codes, scale = LO.fp8_encode(x)
    assert np.array_equal(bufs[1].cpu().numpy()[:8], scale)
    assert np.array_equal(bufs[0].cpu().numpy()[:8], codes)
    assert torch.isnan(bufs[2][7, 0])
    out = torch.zeros((8, 576), dtype=torch.bfloat16, device=DEV)
    bt, ln = i32([[0]]), i32([8])
    D.dsa_latent_cache_read(D.latent_cache(*bufs), D.paged_cache(bt, ln, 1), 1, i32([0]), out)
    y = out.double().cpu().numpy()[:, :512]
    assert np.all(np.isnan(y[0, :128])) and np.all(y[0, 128:] == 0) and np.all(np.isnan(y[1, 128:256]))
    assert np.all(y[2] == 57344.0) and np.all(y[3] == 0.0)


def test_cache_write_skips_and_flags_bad_slots_and_positions():
    g = gen(1)
    kv = randn((4, 576), g)
    tab = D.dsa_rope_table(THETA, 64, 10).to(DEV)
    bufs, bits = _write(kv, i32([0, 128, 2, 3]), "bf16", 1, i32([0, 1, 10, -1]), tab, D.DSA_CACHE_ROPE)
    assert bits == 2
    assert torch.all(bufs[0][1:] == 5.0) and torch.equal(bufs[0][0, :512], kv[0, :512])


def test_every_code_and_scale_reads_back_exactly():
    """All 256 codes under every scale byte; the stored value is exact in bf16 wherever it is within
    bf16's range."""
    codes = torch.arange(512, device=DEV).remainder(256).to(torch.uint8).expand(256, 512).contiguous()
    scale = torch.arange(256, device=DEV).to(torch.uint8)[:, None].expand(256, 4).contiguous()
    rope = randn((256, 64), gen(2))
    out = torch.zeros((256, 576), dtype=torch.bfloat16, device=DEV)
    bt, ln = i32([[1, 0]]), i32([256])
    D.dsa_latent_cache_read(D.latent_cache(codes, scale, rope), D.paged_cache(bt, ln, 2), 1, i32([0]), out)
    back = torch.cat([out[128:], out[:128]])
    assert torch.equal(back[:, 512:], rope)
    got = back[:, :512].double().cpu().numpy()
    for b in range(256):
        if b > 134:
            assert np.all(np.isnan(got[b]))
            continue
        want = LO.e4m3_values()[codes[b].cpu().numpy()] * 2.0 ** (b - 127)
        fin = np.isfinite(want)                       # the writer never stores the NaN codes under these bytes
        big = np.abs(want) >= 2.0 ** -126             # below, bf16's own subnormals
        assert np.array_equal(got[b][fin & big], want[fin & big])
        assert np.all(np.abs(got[b][fin] - want[fin]) <= 2.0 ** -134)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("lens", [[1], [0, 128, 129, 0, 1], [300, 1000, 127, 64], [0]])
def test_cache_read(fmt, lens):
    pc = Paged(lens, fmt, seed=sum(lens))
    start = np.concatenate([[0], np.cumsum(lens)[:-1]]) + 3            # rows before and behind stay
    start[-1] += 2
    total = sum(lens) + 9
    out = torch.full((total, 576), 4.0, dtype=torch.bfloat16, device=DEV)
    ws = D.dsa_latent_cache_read(pc.cache, pc.pages, len(lens), i32(start), out)
    assert D.dsa_workspace_status(ws) == 0
    want = np.full((total, 576), 4.0)
    for t, L in enumerate(lens):
        want[start[t]:start[t] + L] = pc.stored(t)
    assert np.array_equal(out.double().cpu().numpy(), want)


def test_cache_read_skips_and_flags():
    pc = Paged([200, 130, 5], "fp8", seed=8)
    bt = pc.bt.copy()
    bt[0, 1] = pc.n_pages                       # a page outside the cache: its rows are skipped
    out = torch.full((400, 576), 4.0, dtype=torch.bfloat16, device=DEV)
    bt_d = i32(bt)
    start = i32([0, 272, 399])                  # sequence 1's second page and sequence 2 do not fit
    ws = D.dsa_latent_cache_read(pc.cache, D.paged_cache(bt_d, pc.len_d, pc.n_pages), 3, start, out)
    assert D.dsa_workspace_status(ws, raise_on_fault=False) == 2
    o = out.double().cpu().numpy()
    assert np.array_equal(o[:128], pc.stored(0)[:128]) and np.all(o[128:272] == 4.0)
    assert np.array_equal(o[272:400], pc.stored(1)[:128])
    # lengths outside the table are cut and flagged
    ln = i32([-3, 100000, 5])
    ws = D.dsa_latent_cache_read(pc.cache, D.paged_cache(pc.bt_d, ln, pc.n_pages), 1, i32([0]), out, ws=ws)
    assert D.dsa_workspace_status(ws, raise_on_fault=False) == 8


def _dirty():
    """A workspace as an earlier call may have left it."""
    return torch.full((256,), 0xFF, dtype=torch.uint8, device=DEV)


def test_large_rotations_equal_small_ones_and_flag():
    """Calls whose status words are cleared before the kernel, against calls of a few thousand tokens."""
    n, g = 40000, gen(91)
    x = torch.randn((n, 2, 64), generator=g, device=DEV)
    tab = D.dsa_rope_table(THETA, 64, 3000).to(DEV)
    pos = torch.randint(0, 3000, (n,), generator=g, device=DEV, dtype=torch.int32)
    out, ref = torch.full_like(x, 9.0), torch.full_like(x, 9.0)
    ws = _dirty()
    for bad in (None, 0, n - 1, 17001):
        p = pos.clone()
        if bad is not None:
            p[bad] = 3000
        D.dsa_rope_apply(D.rope_desc(x, out), x, p, tab, out, ws=ws)
        assert D.dsa_workspace_status(ws, raise_on_fault=False) == (0 if bad is None else 2)
    out.fill_(9.0)
    pos[17001] = -1
    D.dsa_rope_apply(D.rope_desc(x, out), x, pos, tab, out, ws=ws)
    for i in range(0, n, 4000):
        D.dsa_rope_apply(D.rope_desc(x[i:i + 4000], ref[i:i + 4000]), x[i:i + 4000], pos[i:i + 4000], tab, ref[i:i + 4000])
    assert torch.equal(out, ref) and torch.all(out[17001] == 9.0)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_large_writes_equal_small_ones_and_flag(fmt):
    n, g = 9001, gen(92)
    kv = randn((n, 576), g)
    n_pages = n // P + 3
    slot = torch.randperm(n_pages * P, generator=g, device=DEV)[:n].to(torch.int32)
    slot[5], slot[8000], slot[n - 1], slot[7777] = n_pages * P, -1, 1 << 30, -9
    tab = D.dsa_rope_table(THETA, 64, 500).to(DEV)
    pos = torch.randint(0, 500, (n,), generator=g, device=DEV, dtype=torch.int32)
    pos[8000], pos[4000] = 500, -1                     # the first is a token without a slot
    got, bits = _write(kv, slot, fmt, n_pages, pos, tab, D.DSA_CACHE_ROPE)
    assert bits == 2
    ref, _ = _write(kv[:1], slot[:1], fmt, n_pages, pos[:1], tab, D.DSA_CACHE_ROPE)
    cache = D.latent_cache(*ref)
    for i in range(0, n, 1000):
        k = kv[i:i + 1000]
        D.dsa_latent_cache_write(D.cache_write_desc(k, D.DSA_CACHE_ROPE), k, slot[i:i + 1000], pos[i:i + 1000], tab, cache)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    ws = _dirty()
    slot[5] = slot[n - 1] = slot[4000] = -1
    D.dsa_latent_cache_write(D.cache_write_desc(kv, D.DSA_CACHE_ROPE), kv, slot, pos, tab, D.latent_cache(*got), ws=ws)
    assert D.dsa_workspace_status(ws) == 0
    assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_large_reads_flag_and_skip():
    """More pages than one block checks: two sequences of 2300, of two pages each, share the cache's."""
    pc = Paged([200, 256], "fp8", seed=93)
    m = 2300
    bt, ln = np.repeat(pc.bt[:, :2], m // 2, axis=0), np.repeat([200, 256], m // 2)
    start = np.concatenate([[0], np.cumsum(ln)[:-1]])
    out = torch.full((int(ln.sum()), 576), 4.0, dtype=torch.bfloat16, device=DEV)
    ws = _dirty()
    bt_d, ln_d = i32(bt), i32(ln)
    D.dsa_latent_cache_read(pc.cache, D.paged_cache(bt_d, ln_d, pc.n_pages), m, i32(start), out, ws=ws)
    assert D.dsa_workspace_status(ws) == 0
    a, b = (torch.as_tensor(pc.stored(t), device=DEV).to(torch.bfloat16) for t in (0, 1))
    want = torch.cat([a.repeat(m // 2, 1), b.repeat(m // 2, 1)])
    assert torch.equal(out, want)
    bt[m - 1, 1] = pc.n_pages
    out.fill_(4.0)
    bt_d = i32(bt)
    D.dsa_latent_cache_read(pc.cache, D.paged_cache(bt_d, ln_d, pc.n_pages), m, i32(start), out, ws=ws)
    assert D.dsa_workspace_status(ws, raise_on_fault=False) == 2
    want[-128:] = 4.0
    assert torch.equal(out, want)


@pytest.mark.parametrize("n", [50, 9000])
def test_captured_cache_calls_follow_new_data(n):
    """Rotate, write and read back in a CUDA graph, small and large (with a clearing kernel), replayed on new
    positions, slots and lengths."""
    g = gen(94)
    src = randn((n, 576), g)
    kv = torch.zeros_like(src)
    n_pages = (n + P - 1) // P
    cols = 45
    n_seq = n_pages * (100 if n > 4096 else 1)          # many rows of the same few sequences, mostly empty
    rows = torch.zeros((n_pages * P, 576), dtype=torch.bfloat16, device=DEV)
    back = torch.zeros((n_pages * P, 576), dtype=torch.bfloat16, device=DEV)
    tab = D.dsa_rope_table(THETA, 64, 100).to(DEV)
    pos = torch.zeros(n, dtype=torch.int32, device=DEV)
    slot = torch.full((n,), -1, dtype=torch.int32, device=DEV)
    bt = torch.zeros((n_seq, cols), dtype=torch.int32, device=DEV)
    bt[:n_pages, 0] = torch.arange(n_pages, device=DEV)
    ln = torch.zeros(n_seq, dtype=torch.int32, device=DEV)
    start = torch.zeros(n_seq, dtype=torch.int32, device=DEV)
    start[:n_pages] = torch.arange(n_pages, device=DEV) * P
    cache, pages = D.latent_cache(rows), D.paged_cache(bt, ln, n_pages)
    ws = [torch.zeros(256, dtype=torch.uint8, device=DEV) for _ in range(3)]
    xv, ov = src[:, None, 512:], kv[:, None, 512:]

    def step():
        D.dsa_rope_apply(D.rope_desc(xv, ov), xv, pos, tab, ov, ws=ws[0])
        D.dsa_latent_cache_write(D.cache_write_desc(kv), kv, slot, None, None, cache, ws=ws[1])
        D.dsa_latent_cache_read(cache, pages, n_seq, start, back, ws=ws[2])
    kv[:, :512] = src[:, :512]
    step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            step()
    torch.cuda.synchronize()
    for it in range(3):
        pos.copy_(torch.randint(0, 100, (n,), generator=g, device=DEV))
        if it == 1:
            pos[n - 1] = 100
        slot.copy_(torch.randperm(n_pages * P, generator=g, device=DEV)[:n])
        ln[:n_pages] = P
        back.zero_()
        graph.replay()
        bits = [D.dsa_workspace_status(w, raise_on_fault=False) for w in ws]
        assert bits == [2 if it == 1 else 0, 0, 0]
        assert torch.equal(back, rows)
        assert torch.equal(rows[slot.long()], kv)
        ref = torch.zeros_like(kv)
        m = n - 1 if it == 1 else n
        for i in range(0, m, 1000):
            j = min(m, i + 1000)
            D.dsa_rope_apply(D.rope_desc(xv[i:j], ref[i:j, None, 512:]), xv[i:j], pos[i:j], tab, ref[i:j, None, 512:])
        assert torch.equal(kv[:m, 512:], ref[:m, 512:])


@pytest.mark.parametrize("n", [1, 200, 4000, 20000])
def test_calls_in_a_row_see_what_the_one_before_wrote(n):
    """No call starts on its data before the call (or the torch operation) ahead of it on the stream has
    ended, although its blocks may be scheduled earlier: torch copies, rotates, writes, reads back and turns
    back, many times over the same buffers without a synchronisation."""
    g, turns = gen(95), 40
    src = randn((turns, n, 576), g) if n < 10000 else None
    n_pages = (n + P - 1) // P
    tab = D.dsa_rope_table(THETA, 64, 64).to(DEV)
    pos = torch.randint(0, 64, (n,), generator=g, device=DEV, dtype=torch.int32)
    rows = torch.zeros((n_pages * P, 576), dtype=torch.bfloat16, device=DEV)
    kv, back = torch.zeros((n, 576), dtype=torch.bfloat16, device=DEV), torch.zeros((n, 576), dtype=torch.bfloat16, device=DEV)
    slot = i32(np.random.default_rng(1).permutation(n_pages)[np.arange(n) // P] * P + np.arange(n) % P)
    bt = (slot[::P] // P)[None].contiguous()
    cache, pages = D.latent_cache(rows), D.paged_cache(bt, i32([n]), n_pages)
    ln, start = i32([n]), i32([0])
    pages = D.paged_cache(bt, ln, n_pages)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    kr, br = kv[:, None, 512:], back[:, None, 512:]
    want, sums = [], []
    for it in range(turns):
        x = src[it] if src is not None else randn((n, 576), g)
        want.append(x.float().abs().sum(dim=1)[:: max(1, n // 100)])
        kv.copy_(x)
        D.dsa_rope_apply(D.rope_desc(kr, kr), kr, pos, tab, kr, ws=ws)
        D.dsa_latent_cache_write(D.cache_write_desc(kv), kv, slot, None, None, cache, ws=ws)
        D.dsa_latent_cache_read(cache, pages, 1, start, back, ws=ws)
        D.dsa_rope_apply(D.rope_desc(br, br, D.DSA_ROPE_INVERSE), br, pos, tab, br, ws=ws)
        sums.append(back.float().abs().sum(dim=1)[:: max(1, n // 100)])
    assert D.dsa_workspace_status(ws) == 0
    for a, b in zip(want, sums):
        # the 64 rotary dims are rounded twice, by at most 2^-8 of a pair's length each (1.5 of the value's
        # sum over a pair at most); sums of 576 terms in fp32
        assert torch.all((a - b).abs() <= a * (2 * 2.0 ** -8 * 1.5 + 576 * 2.0 ** -23))


def test_rope_of_as_many_tokens_as_an_int_holds():
    """2^31 - 1 tokens of one head and one pair: two launches, the second of 255 tokens, and no third."""
    n, g = (1 << 31) - 1, gen(78)
    x = randn((1, 1, 2), g).expand(n, 1, 2)
    out = torch.full((n + 64, 1, 2), 3.0, dtype=torch.bfloat16, device=DEV)
    ov = out[:n]
    tab = D.dsa_rope_table(THETA, 2, 50).to(DEV)
    pos = torch.zeros(n, dtype=torch.int32, device=DEV)
    at = [0, 1, 12345, (1 << 30) + 7, n - 256, n - 255, n - 254, n - 2, n - 1]
    pos[at] = i32([3, 49, 7, 11, 5, 6, 8, 50, 9])
    ws = D.dsa_rope_apply(D.rope_desc(x, ov), x, pos, tab, ov)
    assert D.dsa_workspace_status(ws, raise_on_fault=False) == 2
    p64 = pos[at].cpu().numpy()
    keep = p64 < 50
    cs = tab.double().cpu().numpy()[p64[keep]][:, None]
    got = ov[at].double().cpu().numpy()[keep]
    _check_turned(got, np.broadcast_to(x[0].double().cpu().numpy(), got.shape), cs, False, False, 2.0 ** -8)
    assert torch.all(out[n - 2] == 3.0) and torch.all(out[n:] == 3.0)
    out[at] = x[at]                           # everywhere else: a turn by nothing
    flat = out[:n].view(torch.int32).view(-1)
    step = 1 << 28
    assert all(torch.all(flat[i:i + step] == flat[0]) for i in range(0, n, step))


def _empty_calls():
    """(name, call with a workspace) of every call that takes rows, without any."""
    bf, f32, i32_ = torch.bfloat16, torch.float32, torch.int32
    some = lambda dt, *s: torch.zeros(s, dtype=dt, device=DEV)  # noqa: E731
    rows, codes = some(bf, P, 576), some(torch.uint8, P, 512)
    bt, ln = some(i32_, 1, 1), some(i32_, 1)
    pages = D.paged_cache(bt, ln, 1)
    c16, c8 = D.latent_cache(rows), D.latent_cache(codes, some(torch.uint8, P, 4), some(bf, P, 64))
    tab, x = some(f32, 4, 32, 2), some(bf, 0, 2, 64)
    q, out, idx, pos = some(bf, 0, 16, 576), some(bf, 0, 16, 512), some(i32_, 0, 8), some(i32_, 0)
    kv = some(bf, 0, 576)
    ad, ad0 = D.attn_desc(0, P, 16, 8, 0.04), D.attn_desc(0, P, 16, 0, 0.04)
    nd = D.indexer_desc(0, P, 64, 128, 64, 8, P, D.DSA_IDX_ROPE_Q | D.DSA_IDX_ROPE_K)
    npd = D.indexer_desc(0, P, 64, 128, 64, 8, P, D.DSA_IDX_ROPE_Q | D.DSA_IDX_INDEPENDENT_ROWS)
    pd = D.ProjDesc(0, 64, 64, 64, 128, 1e-6)
    one = some(bf, 64 * 128 * 64)
    of = some(f32, 64 * 64)
    qi, ki, w = some(bf, 0, 64, 128), some(bf, P, 128), some(f32, 0, 64)
    keep = (rows, codes, bt, ln, c16, c8)
    return keep, [
        ("rope", lambda ws: D.dsa_rope_apply(D.rope_desc(x, x), x, pos, tab, x, ws=ws)),
        ("write", lambda ws: D.dsa_latent_cache_write(D.cache_write_desc(kv), kv, pos, None, None, c8, ws=ws)),
        ("read", lambda ws: D.dsa_latent_cache_read(c8, pages, 0, pos, rows, ws=ws)),
        ("every key", lambda ws: D.dsa_latent_attn_paged(ad0, q, c8, None, pages, out, ws=ws)),
        ("selected, fp8", lambda ws: D.dsa_latent_attn_paged(ad, q, c8, idx, pages, out, ws=ws)),
        ("selected, bf16", lambda ws: D.dsa_latent_attn_paged(ad, q, c16, idx, pages, out, ws=ws)),
        ("sparse", lambda ws: D.dsa_sparse_attn(ad, q, rows, idx, pos, out, ws=ws)),
        ("sparse, paged", lambda ws: D.dsa_sparse_attn_paged(ad, q, rows, idx, pages, out, ws=ws)),
        ("indexer", lambda ws: D.dsa_indexer_topk(nd, qi, ki, w, pos, some(i32_, P), pos, pos, tab, idx, ws=ws)),
        ("indexer, paged", lambda ws: D.dsa_indexer_topk_paged(npd, qi, ki, w, pos, pages, tab, idx, ws=ws)),
        ("projections", lambda ws: D.dsa_indexer_projections(pd, one, one, one, one, of, of, one, one, one, of, ws=ws)),
    ]


def test_calls_without_rows_clear_the_status():
    """A reused workspace holds the faults of the call before, a new one whatever its memory held."""
    keep, calls = _empty_calls()
    for name, call in calls:
        ws = torch.full((64 << 20,), 0xFF, dtype=torch.uint8, device=DEV)
        call(ws)
        assert D.dsa_workspace_status(ws) == 0, name
        assert torch.all(ws[256:] == 0xFF), name


def test_empty_batches_and_outputs_made_of_empty_tensors():
    c = D.latent_cache(torch.zeros((2 * P, 576), dtype=torch.bfloat16, device=DEV))
    e = lambda dt, *s: torch.empty(s, dtype=dt, device=DEV)  # noqa: E731
    none = D.paged_cache(e(torch.int32, 0, 5), e(torch.int32, 0), 2)
    q, out = e(torch.bfloat16, 0, 16, 576), e(torch.bfloat16, 0, 16, 512)
    ws = D.dsa_latent_attn_paged(D.attn_desc(0, 2 * P, 16, 0, 0.04), q, c, None, none, out)
    assert D.dsa_workspace_status(ws) == 0
    ws = D.dsa_sparse_attn_paged(D.attn_desc(0, 2 * P, 16, 4, 0.04), q, torch.zeros((2 * P, 576), dtype=torch.bfloat16, device=DEV),
                                 e(torch.int32, 0, 4), none, out)
    assert D.dsa_workspace_status(ws) == 0
    back = e(torch.bfloat16, 0, 576)
    ws = D.dsa_latent_cache_read(c, none, 0, e(torch.int32, 0), back)
    assert D.dsa_workspace_status(ws) == 0
    # sequences that are all empty have no output rows; a row without room is flagged
    bt, ln = i32([[0], [1]]), i32([0, 0])
    pages = D.paged_cache(bt, ln, 2)
    ws = D.dsa_latent_cache_read(c, pages, 2, i32([0, 0]), back)
    assert D.dsa_workspace_status(ws) == 0
    ln[1] = 1
    ws = D.dsa_latent_cache_read(c, pages, 2, i32([0, 0]), back, ws=ws)
    assert D.dsa_workspace_status(ws, raise_on_fault=False) == 2


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_a_single_row_cut_from_odd_rows(fmt):
    """One token of a tensor whose rows are not a multiple of eight elements apart, and one head of it turned
    in place through views of different strides: what the same values in plain tensors give."""
    buf = randn((7, 1001), gen(81))
    kv = torch.as_strided(buf, (1, 576), (1001, 1), 8)      # 16-byte aligned
    tab, slot, pos = D.dsa_rope_table(THETA, 64, 50).to(DEV), i32([3]), i32([17])
    got, bits = _write(kv, slot, fmt, 1, pos, tab, D.DSA_CACHE_ROPE)
    want, _ = _write(kv.clone(), slot, fmt, 1, pos, tab, D.DSA_CACHE_ROPE)
    assert bits == 0 and all(torch.equal(a, b) for a, b in zip(got, want))
    x = torch.as_strided(buf, (1, 1, 64), (1001, 3, 1), 16)
    y = torch.as_strided(buf, (1, 1, 64), (5, 77, 1), 16)
    ref = torch.empty((1, 1, 64), dtype=torch.bfloat16, device=DEV)
    plain = x.clone()
    D.dsa_rope_apply(D.rope_desc(plain, ref), plain, pos, tab, ref)
    ws = D.dsa_rope_apply(D.rope_desc(x, y), y, pos, tab, x)
    assert D.dsa_workspace_status(ws) == 0 and torch.equal(x, ref)


@pytest.mark.parametrize("how", ["stream", "handle", "default"])
def test_a_workspace_made_for_a_call_on_another_stream(how):
    """It comes from that stream's memory: what is freed on the current stream, whose work may still use it, is
    not taken, and the workspace, freed before its call has run, is not given to the current stream."""
    s = torch.cuda.Stream()
    given = {"stream": s, "handle": s.cuda_stream, "default": 0}[how]
    here = torch.cuda.Stream()                # the current stream
    g = gen(83)
    x, out = torch.randn((4, 2, 64), generator=g, device=DEV), torch.zeros((4, 2, 64), device=DEV)
    tab, pos = D.dsa_rope_table(THETA, 64, 10).to(DEV), i32([0, 1, 2, 3])
    cache = D.latent_cache(torch.zeros((P, 576), dtype=torch.bfloat16, device=DEV))
    kv, slot = randn((4, 576), g), i32([5, 6, 7, 8])
    back = torch.zeros((P, 576), dtype=torch.bfloat16, device=DEV)
    bt, ln, start = i32([[0]]), i32([9]), i32([0])
    pages = D.paged_cache(bt, ln, 1)
    q, o = randn((1, 16, 576), g), torch.zeros((1, 16, 512), dtype=torch.bfloat16, device=DEV)
    calls = [lambda: D.dsa_rope_apply(D.rope_desc(x, out), x, pos, tab, out, stream=given),
             lambda: D.dsa_latent_cache_write(D.cache_write_desc(kv), kv, slot, None, None, cache, stream=given),
             lambda: D.dsa_latent_cache_read(cache, pages, 1, start, back, stream=given),
             lambda: D.dsa_latent_attn_paged(D.attn_desc(1, P, 16, 0, 0.04), q, cache, None, pages, o, stream=given)]
    torch.cuda.synchronize()
    with torch.cuda.stream(here):
        for call in calls:
            freed = [torch.empty(256, dtype=torch.uint8, device=DEV) for _ in range(4)]
            taken = {t.data_ptr() for t in freed}
            del freed
            ws = call()
            assert ws.data_ptr() not in taken
            size, at = ws.numel(), ws.data_ptr()
            del ws
            new = [torch.empty(size, dtype=torch.uint8, device=DEV) for _ in range(8)]
            assert at not in {t.data_ptr() for t in new}
            del new
    torch.cuda.synchronize()
    assert torch.equal(back[5:9], kv)
