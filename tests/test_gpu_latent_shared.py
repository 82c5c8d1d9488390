"""GPU tests of latent attention over shared prefixes (dsa_latent_attn_shared) against float64: every row is
its own attention over all of its keys, whatever is shared.  Every unused cache row is NaN."""
import numpy as np
import pytest
import torch

import dsa_indexer_cross_gb300 as D
from latent_cases import DEV, P, TAU, check_exceptional, check_rows, gen, i32, randn
from shared_cases import SharedPaged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dsa_indexer_cross_gb300.build import build
    build()
    assert torch.cuda.is_available()


def _check(groups, H, fmt, seed=1, check=None, bits=0, wide=True, **kw):
    sp = SharedPaged(groups, fmt, seed=seed, wide=wide)
    q = randn((len(sp.lens), H, 576), gen(seed + 50))
    out, lse, ws = sp.attend(q, **kw)
    assert D.dsa_workspace_status(ws, raise_on_fault=False) == bits
    check_rows(out, lse, q, [sp.stored(t) if check is None or t in check else None for t in range(len(sp.lens))])
    return sp, q, out, lse


MIXED = [
    (0, [70], False), (300, [300, 301, 450, 0, 1, 299, 600], False), (128, [128, 128], False), (63, [64, 65, 90], False),
    (1000, [1200], False), (640, [650, 640, 1000], False), (500, [501, 502, 503, 504], True), (0, [5, 0, 200], False),
    (129, [0, 0, 0], False), (2000, [100, 200, 300, 2100], False), (64, [64, 64, 64], True), (256, [], False), (192, [193, 250], False)]


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("H", [1, 3, 8, 16, 17, 32, 33, 64, 65, 100, 128])
def test_groups_of_every_kind(H, fmt):
    _check(MIXED, H, fmt, seed=H)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("H", [8, 40, 100, 128])
def test_small_calls_share_nothing(H, fmt):
    sp, q, out, lse = _check(MIXED, H, fmt, seed=H, wide=False)
    # the unshared call's results, bit for bit
    desc = D.attn_desc(q.shape[0], sp.n_pages * P, H, 0, TAU)
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    D.dsa_latent_attn_paged(desc, q, sp.cache, None, sp.pages, o2, l2)
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    # and its groups are checked all the same
    pre = list(sp.prefix)
    pre[3] = -1
    for kw in (dict(start=i32([0, 5, 4] + sp.start[3:])), dict(prefix=i32(pre))):
        o3, l3, ws = sp.attend(q, **kw)
        assert D.dsa_workspace_status(ws, raise_on_fault=False) == 8
        assert torch.equal(out, o3) and torch.equal(lse, l3)
    sp = SharedPaged([(5, [7], False)], fmt, seed=2, wide=False)       # one row, one CTA
    q = randn((1, H, 576), gen(3))
    out, lse, ws = sp.attend(q)
    assert D.dsa_workspace_status(ws) == 0
    check_rows(out, lse, q, [sp.stored(0)])


@pytest.mark.parametrize("max_rows", [1, 2, 4, 1000])
@pytest.mark.parametrize("H", [5, 16, 64, 100])
def test_the_hint_only_chooses_kernels(H, max_rows):
    _check(MIXED, H, "fp8", seed=3, max_rows=max_rows)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("rows,H,prefix", [(4, 16, 5000), (48, 16, 8000), (2, 1, 700), (8, 64, 20000), (16, 100, 6000),
                                           (3, 128, 3000), (9, 128, 5000), (70, 3, 12345), (130, 8, 1000), (2, 16, 129)])
def test_one_group(rows, H, prefix, fmt):
    rng = np.random.default_rng(rows)
    lens = (prefix + rng.integers(0, 700, rows)).tolist()
    _check([(prefix, lens, False)], H, fmt, seed=rows, check=set(range(0, rows, max(1, rows // 6))))
    _check([(prefix, [prefix + 1 + i for i in range(rows)], True)], H, fmt, seed=rows + 1,
           check=set(range(0, rows, max(1, rows // 6))))


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_many_groups_and_rows(fmt):
    rng = np.random.default_rng(7)
    groups = []
    for _ in range(1200):
        p = int(rng.integers(0, 400))
        groups.append((p, (p + rng.integers(0, 90, int(rng.integers(0, 4)))).tolist(), bool(rng.random() < 0.3)))
    n = sum(len(g[1]) for g in groups)
    for H in (4, 40):
        _check(groups, H, fmt, seed=H, check=set(range(0, n, 97)) | {0, n - 1})


def test_rows_outside_the_groups():
    sp = SharedPaged(MIXED, "bf16", seed=5)
    q = randn((len(sp.lens), 16, 576), gen(9))
    out, lse, ws = sp.attend(q, start=sp.start_d[3:8].contiguous(), prefix=sp.prefix_d[3:7].contiguous())
    assert D.dsa_workspace_status(ws) == 0
    check_rows(out, lse, q, [sp.stored(t) for t in range(len(sp.lens))])
    e = torch.empty(0, dtype=torch.int32, device=DEV)
    out, lse, ws = sp.attend(q, start=torch.zeros(1, dtype=torch.int32, device=DEV), prefix=e, max_rows=1)
    assert D.dsa_workspace_status(ws) == 0
    check_rows(out, lse, q, [sp.stored(t) for t in range(len(sp.lens))])


@pytest.mark.parametrize("H", [16, 64, 128])
def test_equals_the_unshared_call(H):
    """Same inputs, same roundings of the weights, other sums: within both calls' bounds of float64; and with no
    group at all each row is walked as there."""
    sp = SharedPaged([(900, [900 + 37 * i for i in range(9)], False)], "fp8", seed=2)
    q = randn((9, H, 576), gen(3))
    out, lse, _ = sp.attend(q)
    desc = D.attn_desc(9, sp.n_pages * P, H, 0, TAU)
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    D.dsa_latent_attn_paged(desc, q, sp.cache, None, sp.pages, o2, l2)
    check_rows(out, lse, q, [sp.stored(t) for t in range(9)])
    assert torch.all((lse - l2).abs() <= 2.0 ** -12)
    assert torch.all((out.float() - o2.float()).abs() <= 2.0 ** -6)


@pytest.mark.parametrize("H", [8, 40, 100])
def test_bad_groups_pages_and_lengths(H):
    sp = SharedPaged(MIXED, "bf16", seed=6)
    n = len(sp.lens)
    q = randn((n, H, 576), gen(8))
    want = [sp.stored(t) for t in range(n)]
    for bad in ([0, 5, 4] + sp.start[3:], [-1] + sp.start[1:], sp.start[:-1] + [n + 1], [n] + sp.start[1:]):
        out, lse, ws = sp.attend(q, start=i32(bad))
        assert D.dsa_workspace_status(ws, raise_on_fault=False) == 8
        check_rows(out, lse, q, want)
    pre = list(sp.prefix)
    pre[1] = -3
    out, lse, ws = sp.attend(q, prefix=i32(pre))
    assert D.dsa_workspace_status(ws, raise_on_fault=False) == 8
    check_rows(out, lse, q, want)
    # lengths beyond the table are cut to it, negative ones are empty
    lens = sp.len_d.clone()
    t0 = sp.start[4]
    sp.len_d[t0] = -1
    out, lse, ws = sp.attend(q)
    assert D.dsa_workspace_status(ws, raise_on_fault=False) == 8
    check_rows(out, lse, q, [w if t != t0 else w[:0] for t, w in enumerate(want)])
    sp.len_d.copy_(lens)
    # a page outside the cache, in a prefix that several rows walk: its keys are left out of all of them
    g = 5                                     # prefix 640, lengths 650, 640, 1000
    rows = list(range(sp.start[g], sp.start[g + 1]))
    keep = sp.bt_d.clone()
    for r in rows:
        sp.bt_d[r, 1] = sp.n_pages
    out, lse, ws = sp.attend(q)
    assert D.dsa_workspace_status(ws, raise_on_fault=False) == 2
    check_rows(out, lse, q, [np.concatenate([w[:P], w[2 * P:]]) if t in rows else w for t, w in enumerate(want)])
    sp.bt_d.copy_(keep)
    out, lse, ws = sp.attend(q)
    assert D.dsa_workspace_status(ws) == 0
    check_rows(out, lse, q, want)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("H", [16, 100])
def test_infinities_and_nan_stay_with_their_rows(H, fmt):
    groups = [(400, [400, 520, 70, 0, 410], False), (200, [201, 202, 203], True)]
    sp = SharedPaged(groups, fmt, seed=4)
    q = randn((len(sp.lens), H, 576), gen(5))
    # an own key of row 1, and one of the last draft, are NaN or infinite; row 4's own key is -inf in a rotary dim
    def row(t, j):
        return int(sp.bt[t, j // P]) * P + j % P
    store = sp.rows if fmt == "bf16" else sp.rope
    off = 512 if fmt == "bf16" else 0
    store[row(1, 500), off + 3] = float("nan")
    store[row(7, 202), off + 5] = float("inf")
    store[row(4, 405), off + 1] = -float("inf")
    out, lse, ws = sp.attend(q)
    assert D.dsa_workspace_status(ws) == 0
    check_exceptional(out, lse, q, [sp.stored(t) for t in range(len(sp.lens))])
    assert torch.all(torch.isnan(out[1])) and torch.all(torch.isfinite(out[0])) and torch.all(torch.isfinite(out[5:7]))


def test_two_streams_graphs_and_a_shared_workspace():
    sps = [SharedPaged([(700, [700 + 11 * i for i in range(6)], False)], "fp8", seed=s) for s in (1, 2)]
    H = 24
    qs = [randn((6, H, 576), gen(s + 20)) for s in (1, 2)]
    want = [tuple(x.clone() for x in sp.attend(q)[:2]) for sp, q in zip(sps, qs)]
    streams = [torch.cuda.Stream() for _ in sps]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                got.append((k, sps[k].attend(qs[k])))
    torch.cuda.synchronize()
    for k, (out, lse, _) in got:
        assert torch.equal(out, want[k][0]) and torch.equal(lse, want[k][1])
    # captured, two calls on one workspace, then other queries and lengths in place
    sp, q = sps[0], qs[0].clone()
    ws = sp.attend(q)[2]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a = sp.attend(q, ws=ws)
        b = sp.attend(q, ws=ws)
    q.copy_(qs[1])
    sp.len_d[2] = 300                       # shorter than the prefix now
    g.replay()
    torch.cuda.synchronize()
    assert D.dsa_workspace_status(ws) == 0
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    kv = [sp.stored(t)[:300] if t == 2 else sp.stored(t) for t in range(6)]
    check_rows(a[0], a[1], q, kv)


def _staged_groups():
    """Enough columns and tiles that an fp8 cache's prefixes are brought to bf16 first: several groups, odd numbers of
    tiles and of pages, rows shorter than their prefix, a group and rows that share nothing."""
    rng = np.random.default_rng(3)
    lens = lambda p, n: (p + rng.integers(0, 300, n)).tolist()  # noqa: E731
    return [(0, [100, 0], False), (2100, lens(2100, 9), False), (4000, lens(4000, 12) + [0, 50, 3900], False),
            (1, [300], False), (1290, [1291 + i for i in range(8)], True), (60, lens(60, 3), False)]


@pytest.mark.parametrize("H", [64, 100, 128])
def test_staged_prefixes(H):
    groups = _staged_groups()
    n = sum(len(g[1]) for g in groups)
    sp, q, out, lse = _check(groups, H, "fp8", seed=H, check=set(range(0, n, 4)) | {12, 23, 24, 25})
    again, l2, _ = sp.attend(q)
    assert torch.equal(out, again) and torch.equal(lse, l2)
    # a page outside the cache: its keys are left out of the rows that walk it
    rows = list(range(2, 11))
    keep = sp.bt_d.clone()
    sp.bt_d[rows, 3] = -1
    o3, l3, ws = sp.attend(q)
    assert D.dsa_workspace_status(ws, raise_on_fault=False) == 2
    kv = [None] * n
    for t in (2, 7, 12):
        w = sp.stored(t)
        kv[t] = np.concatenate([w[:3 * P], w[4 * P:]]) if t in rows else w
    check_rows(o3, l3, q, kv)
    sp.bt_d.copy_(keep)
    # captured, with other lengths in place: now too short to be shared by most
    ws = torch.empty_like(ws)
    g = torch.cuda.CUDAGraph()
    sp.attend(q, ws=ws)
    with torch.cuda.graph(g):
        o4, l4, _ = sp.attend(q, ws=ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o4, out) and torch.equal(l4, lse)
    sp.len_d.clamp_(max=700)
    g.replay()
    torch.cuda.synchronize()
    assert D.dsa_workspace_status(ws) == 0
    check_rows(o4, l4, q, [sp.stored(t)[:700] if t in (0, 2, 12, 25, 30) else None for t in range(n)])


def test_prefixes_of_more_pages_than_are_staged():
    """1100 pages in two groups: they are walked from the cache."""
    groups = [(70000, [70000 + 10 * i for i in range(14)], True), (70700, [70700 + 5 * i for i in range(13)], True)]
    _check(groups, 64, "fp8", seed=2, check={0, 26})


def test_without_lse_and_empty_calls():
    sp = SharedPaged([(300, [310, 400], False)], "bf16", seed=1)
    q = randn((2, 16, 576), gen(2))
    out, lse, ws = sp.attend(q)
    o2, none, _ = sp.attend(q, lse=False)
    assert none is None and torch.equal(out, o2)
    e = torch.empty((0, 16, 576), dtype=torch.bfloat16, device=DEV)
    desc = D.attn_desc(0, sp.n_pages * P, 16, 0, TAU)
    groups = D.shared_rows(torch.zeros(1, dtype=torch.int32, device=DEV), torch.empty(0, dtype=torch.int32, device=DEV), 1)
    ws.fill_(255)
    D.dsa_latent_attn_shared(desc, e, sp.cache, groups, sp.pages, torch.empty((0, 16, 512), dtype=torch.bfloat16, device=DEV), ws=ws)
    assert D.dsa_workspace_status(ws) == 0
    sp = SharedPaged([(300, [0, 0, 0], False)], "bf16", seed=1)
    out, lse, ws = sp.attend(randn((3, 16, 576), gen(2)))
    assert torch.all(out == 0) and torch.all(lse == -float("inf"))


def test_results_repeat():
    sp = SharedPaged([(3000, [3000 + 100 * i for i in range(20)], False), (500, [600] * 5, False)], "fp8", seed=1)
    for H in (16, 64, 128):
        q = randn((25, H, 576), gen(H))
        out, lse, _ = sp.attend(q)
        for _ in range(4):
            o2, l2, _ = sp.attend(q)
            assert torch.equal(out, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("H", [8, 40, 100])
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_a_wait_that_runs_out_is_reported(H, fmt):
    """The rows' producers stop at the start (a test hook; a share may hold no more than two tiles); the waits behind
    them run out after a millisecond."""
    sp = SharedPaged([(9000, [9000 + 50 * i for i in range(6)], False)], fmt, seed=3)
    q = randn((6, H, 576), gen(4))
    ref = sp.attend(q)
    D.dsa_debug_pipeline(0, 1_000_000)
    try:
        _, _, ws = sp.attend(q, ws=ref[2])
        assert D.dsa_workspace_status(ws, raise_on_fault=False) & 1
    finally:
        D.dsa_debug_pipeline(-1, 0)
    out, lse, ws = sp.attend(q, ws=ref[2])
    assert D.dsa_workspace_status(ws) == 0
    assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])


@pytest.mark.parametrize("fill", [0x7F, 0x00, 0xFF])
@pytest.mark.parametrize("H,rows", [(8, 6), (40, 6), (100, 6), (100, 9)])
def test_a_wait_that_runs_out_in_a_workspace_of_anything(H, rows, fill):
    """The join finds no pieces noted where the walks gave up, whatever the workspace held."""
    sp = SharedPaged([(9000, [9000 + 50 * i for i in range(rows)], False)], "fp8", seed=3)
    q = randn((rows, H, 576), gen(4))
    ref = sp.attend(q)
    ws = torch.full_like(ref[2], fill)
    D.dsa_debug_pipeline(0, 1_000_000)
    try:
        sp.attend(q, ws=ws)
        assert D.dsa_workspace_status(ws, raise_on_fault=False) & 1
    finally:
        D.dsa_debug_pipeline(-1, 0)
    ws.fill_(fill)
    out, lse, ws = sp.attend(q, ws=ws)
    assert D.dsa_workspace_status(ws) == 0
    assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("H", [1, 16, 64, 100, 128])
@pytest.mark.parametrize("lens", [[100], [0], [70, 300], [128] * 40])
def test_no_groups_need_no_arrays(lens, H, fmt):
    """n_groups = 0 with NULL arrays, from one row of one page (one CTA, no join) on: the unshared call's results.  What
    an array of no groups holds is not looked at."""
    sp = SharedPaged([(0, lens, False)], fmt, seed=H, wide=False)
    bt = sp.bt_d[:, :max(1, -(-max(lens) // P))].contiguous()
    pages = D.paged_cache(bt, sp.len_d, sp.n_pages)
    n = len(lens)
    q = randn((n, H, 576), gen(5))
    desc = D.attn_desc(n, sp.n_pages * P, H, 0, TAU)
    want = torch.empty((n, H, 512), dtype=torch.bfloat16, device=DEV), torch.empty((n, H), device=DEV)
    D.dsa_latent_attn_paged(desc, q, sp.cache, None, pages, *want)
    start = i32([-1])
    for groups in (D.SharedRows(None, None, 0, 1), D.SharedRows(None, None, 0, 1000), D.SharedRows(start.data_ptr(), None, 0, 1)):
        out, lse = torch.full_like(want[0], 7.0), torch.full_like(want[1], 7.0)
        ws = D.dsa_latent_attn_shared(desc, q, sp.cache, groups, pages, out, lse)
        assert D.dsa_workspace_status(ws) == 0
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("H,rows,fmt,lists", [(128, 5, "fp8", False), (128, 1, "fp8", False), (128, 9, "bf16", False), (100, 4, "fp8", False),
                                              (100, 4, "bf16", False), (65, 2, "bf16", False), (65, 3, "bf16", True), (126, 63, "bf16", False), (128, 6, "fp8", True),
                                              (100, 5, "fp8", True), (100, 5, "bf16", True), (64, 2, "fp8", True)])
def test_calls_that_cannot_share_run_the_unshared_kernels(H, rows, fmt, lists):
    """Where a group's rows fill as many blocks of columns as there are rows (2 x 65 columns: two of 128; 3 x 65: two), no
    list is made (the launch log shows it), the results are the unshared call's and the groups are checked all the same."""
    sp = SharedPaged([(700, [701 + i for i in range(rows)], True)] * 4 + [(0, [900], False)], fmt, seed=H + rows)
    n = len(sp.lens)
    q = randn((n, H, 576), gen(3))
    ref = sp.attend(q)
    assert D.dsa_workspace_status(ref[2]) == 0
    D.dsa_profile_enable(True)
    try:
        out, lse, ws = sp.attend(q)
        kinds = [k for k, _ in D.dsa_profile_read()]
    finally:
        D.dsa_profile_enable(False)
    assert kinds == ["attn_prep"] * lists + ["attn"]
    assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])
    check_rows(out, lse, q, [sp.stored(t) if t % 5 == 0 or t == n - 1 else None for t in range(n)])
    if not lists:
        o2, l2 = torch.empty_like(out), torch.empty_like(lse)
        D.dsa_latent_attn_paged(D.attn_desc(n, sp.n_pages * P, H, 0, TAU), q, sp.cache, None, sp.pages, o2, l2)
        assert torch.equal(out, o2) and torch.equal(lse, l2)
    for kw in (dict(start=i32(sp.start[:-1] + [n + 1])), dict(prefix=i32(sp.prefix[:-1] + [-1]))):
        o3, l3, ws = sp.attend(q, **kw)
        assert D.dsa_workspace_status(ws, raise_on_fault=False) == 8
        check_rows(o3, l3, q, [sp.stored(t) if t == 0 else None for t in range(n)])


@pytest.mark.parametrize("at", [0, 1, 31, 32, 255, 256, 1023, 1024, 2999, 3000])
@pytest.mark.parametrize("H,fmt", [(128, "bf16"), (8, "bf16")])
def test_every_one_of_many_groups_is_checked(H, fmt, at):
    """3000 groups, most of them empty, of a call that shares nothing (and of one that lists them): a fault in any."""
    sp = SharedPaged([(200, [210, 220], False), (0, [5], False)], fmt, seed=4)
    n = 3
    q = randn((n, H, 576), gen(3))
    start = np.full(3001, 2, dtype=np.int32)
    start[0], start[3000] = 0, 3
    prefix = np.full(3000, 100, dtype=np.int32)
    out, lse, ws = sp.attend(q, start=i32(start), prefix=i32(prefix))
    assert D.dsa_workspace_status(ws) == 0
    check_rows(out, lse, q, [sp.stored(t) for t in range(n)])
    bad = start.copy()
    bad[at] = 4 if at else -1          # past the rows, or before them
    o2, l2, ws = sp.attend(q, start=i32(bad), prefix=i32(prefix))
    assert D.dsa_workspace_status(ws, raise_on_fault=False) == 8
    check_rows(o2, l2, q, [sp.stored(t) for t in range(n)])
    if at < 3000:
        bad = prefix.copy()
        bad[at] = -1
        o2, l2, ws = sp.attend(q, start=i32(start), prefix=i32(bad))
        assert D.dsa_workspace_status(ws, raise_on_fault=False) == 8
        check_rows(o2, l2, q, [sp.stored(t) for t in range(n)])
