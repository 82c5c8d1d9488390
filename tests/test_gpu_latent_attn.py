"""GPU tests of latent attention over a paged cache (dsa_latent_attn_paged) against float64, at the
lengths, head counts and masks where it can go wrong.  Every unused cache row is NaN."""
import numpy as np
import pytest
import torch

import dsa_indexer_cross_gb300 as D
from latent_cases import DEV, P, TAU, Paged, attend, check_exceptional, check_rows, gen, i32, randn
from oracle import latent_oracle as LO

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dsa_indexer_cross_gb300.build import build
    build()
    assert torch.cuda.is_available()


def _dense(lens, H, fmt, seed=1, std=1.0, check=None):
    pc = Paged(lens, fmt, seed=seed)
    q = randn((len(lens), H, 576), gen(seed + 50), std)
    out, lse, ws = attend(pc, q)
    assert D.dsa_workspace_status(ws) == 0
    check_rows(out, lse, q, [pc.stored(t) if check is None or t in check else None for t in range(len(lens))])
    return pc, q, out, lse


EDGES = [0, 1, 2, 63, 64, 65, 127, 128, 129, 0, 191, 192, 193, 1000, 0]


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("H", [1, 3, 16, 17, 32, 33, 64, 65, 128])
def test_every_key_at_edge_lengths(H, fmt):
    _dense(EDGES, H, fmt)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("H,L", [(16, 1), (128, 64), (1, 700), (64, 9000), (128, 33333), (40, 20001)])
def test_one_row_split_over_all_ctas(H, L, fmt):
    _dense([L], H, fmt, seed=L)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_many_rows_and_uneven_lengths(fmt):
    rng = np.random.default_rng(4)
    lens = rng.integers(0, 400, size=700).tolist()
    lens[13], lens[500] = 12000, 7001
    _dense(lens, 16, fmt, seed=9, check={0, 1, 12, 13, 14, 350, 499, 500, 501, 698, 699})


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("lens", [[500] * 20 + [510, 0, 450], [64] * 70, [40] * 76, [65] * 77, [1000, 1000, 1001],
                                  [0, 0, 3000, 2900, 0, 3100] * 6])
def test_rows_of_nearly_equal_length(lens, fmt):
    """The pair kernel takes whole rows where the longest is near the even share."""
    _dense(lens, 100, fmt, seed=len(lens))


@pytest.mark.parametrize("n,topk", [(9, 512), (64, 512), (30, 1000), (77, 130)])
def test_selections_of_equal_size(n, topk):
    lens = [topk + 300 * (t % 5) for t in range(n)]
    pc = Paged(lens, "fp8", seed=n)
    q = randn((n, 128, 576), gen(n))
    idx = _selection(lens, topk, n)
    out, lse, ws = attend(pc, q, i32(idx))
    assert D.dsa_workspace_status(ws) == 0
    check_rows(out, lse, q, [pc.stored(t)[idx[t]] if t % 7 in (0, 3) else None for t in range(n)])


def test_no_keys_at_all():
    pc, q, out, lse = _dense([0, 0, 0], 24, "fp8")
    assert torch.all(out == 0) and torch.all(lse == -float("inf"))
    desc = D.attn_desc(0, pc.n_pages * P, 16, 0, TAU)
    e = torch.empty((0, 16, 576), dtype=torch.bfloat16, device=DEV)
    D.dsa_latent_attn_paged(desc, e, pc.cache, None, pc.pages, torch.empty((0, 16, 512), dtype=torch.bfloat16, device=DEV))


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_scores_that_keep_rising(fmt):
    """Keys whose scores grow along the sequence: the running maximum moves in many tiles, in both
    orders of the lengths, and weights underflow behind it."""
    pc = Paged([2000, 900], fmt, seed=2)
    q = randn((2, 33, 576), gen(3))
    for t in range(2):
        L = pc.lens[t]
        ramp = torch.linspace(0.0, 30.0, L, device=DEV)[:, None]
        if fmt == "bf16":
            pc.kv[t] = (pc.kv[t].float() * 0.3 + ramp * q[t, 0].float() * (24.0 / 576)).to(torch.bfloat16)
            pc.rows[pc.phys[t]] = pc.kv[t]
        else:
            from latent_cases import encode
            kv = (pc.kv[t].float() * 0.3 + ramp * q[t, 0].float() * (24.0 / 576)).to(torch.bfloat16)
            pc.codes[pc.phys[t]], pc.scale[pc.phys[t]] = encode(kv[:, :512])
            pc.rope[pc.phys[t]] = kv[:, 512:]
    out, lse, ws = attend(pc, q)
    assert D.dsa_workspace_status(ws) == 0
    check_rows(out, lse, q, [pc.stored(0), pc.stored(1)])


def test_fp8_equals_the_rows_read_back():
    """Attention over the fp8 cache and over its rows read back into a bf16 cache: the same bits."""
    lens = [5, 700, 0, 3000, 129]
    pc = Paged(lens, "fp8", seed=6)
    bf = Paged(lens, "bf16", seed=6)
    start = np.concatenate([[0], np.cumsum(lens)[:-1]])
    rows = torch.empty((sum(lens), 576), dtype=torch.bfloat16, device=DEV)
    D.dsa_latent_cache_read(pc.cache, pc.pages, len(lens), i32(start), rows)
    for t, L in enumerate(lens):
        bf.rows[bf.phys[t]] = rows[start[t]:start[t] + L]
    for H in (16, 128):
        q = randn((len(lens), H, 576), gen(7))
        a, b = attend(pc, q), attend(bf, q)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def _selection(lens, topk, seed, holes=False):
    rng = np.random.default_rng(seed)
    idx = np.full((len(lens), topk), -1, dtype=np.int32)
    for t, L in enumerate(lens):
        m = min(topk, L)
        if holes:
            m = m // 2
        j = np.sort(rng.choice(L, size=m, replace=False)) if m else np.zeros(0, int)
        if holes:      # unused slots anywhere, order arbitrary
            at = rng.choice(topk, size=m, replace=False)
            idx[t, at] = rng.permutation(j)
        else:
            idx[t, :m] = j
    return idx


@pytest.mark.parametrize("H", [1, 16, 33, 128])
@pytest.mark.parametrize("topk,holes", [(1, False), (64, False), (100, True), (777, False), (2048, True)])
def test_selected_keys_of_an_fp8_cache(H, topk, holes):
    lens = [0, 1, 50, 64, 3000, 129, 0, 2048, 5000, 777]
    pc = Paged(lens, "fp8", seed=topk)
    q = randn((len(lens), H, 576), gen(topk + H))
    idx = _selection(lens, topk, topk, holes)
    out, lse, ws = attend(pc, q, i32(idx))
    assert D.dsa_workspace_status(ws) == 0
    check_rows(out, lse, q, [pc.stored(t)[idx[t][idx[t] >= 0]] for t in range(len(lens))])


def test_selected_keys_of_a_bf16_cache_are_the_sparse_call():
    lens = [900, 64, 3000]
    pc = Paged(lens, "bf16", seed=3)
    q = randn((3, 64, 576), gen(4))
    idx = i32(_selection(lens, 256, 5))
    out, lse, ws = attend(pc, q, idx)
    assert D.dsa_workspace_status(ws) == 0
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    D.dsa_sparse_attn_paged(D.attn_desc(3, pc.n_pages * P, 64, 256, TAU), q, pc.rows, idx, pc.pages, o2, l2)
    assert torch.equal(out, o2) and torch.equal(lse, l2)


def test_whole_selection_is_every_key():
    """An index row listing every key gives what the call without an index gives."""
    lens = [300, 1024, 7]
    pc = Paged(lens, "fp8", seed=12)
    q = randn((3, 16, 576), gen(13))
    idx = np.full((3, 1024), -1, dtype=np.int32)
    for t, L in enumerate(lens):
        idx[t, :L] = np.arange(L)
    a, b = attend(pc, q), attend(pc, q, i32(idx))
    kv = [pc.stored(t) for t in range(3)]
    check_rows(a[0], a[1], q, kv)
    check_rows(b[0], b[1], q, kv)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_pages_outside_the_cache_are_skipped_and_flagged(fmt):
    pc = Paged([500, 128, 70], fmt, seed=5)
    q = randn((3, 20, 576), gen(6))
    bt = pc.bt.copy()
    bt[0, 1], bt[1, 0] = pc.n_pages, -1
    bt_d = i32(bt)
    good = pc.pages
    pc.pages = D.paged_cache(bt_d, pc.len_d, pc.n_pages)
    out, lse, ws = attend(pc, q)
    assert D.dsa_workspace_status(ws, raise_on_fault=False) == 2
    k0 = pc.stored(0)
    check_rows(out, lse, q, [np.concatenate([k0[:128], k0[256:]]), np.zeros((0, 576)), pc.stored(2)])
    if fmt == "fp8":
        idx = i32(np.array([[0, 130, 300, -1], [0, 1, 2, 3], [69, 70, 5, 100000]]))
        out, lse, ws = attend(pc, q, idx, ws=ws)
        assert D.dsa_workspace_status(ws, raise_on_fault=False) == 2
        check_rows(out, lse, q, [k0[[0, 300]], np.zeros((0, 576)), pc.stored(2)[[69, 5]]])
    # lengths outside the table are cut to it and flagged
    pc.pages = good
    full = Paged([256], fmt, seed=5, extra_cols=0)
    ln = i32([300])
    full.pages = D.paged_cache(full.bt_d, ln, full.n_pages)
    out, lse, ws = attend(full, q[:1])
    assert D.dsa_workspace_status(ws, raise_on_fault=False) == 8
    check_rows(out, lse, q[:1], [full.stored(0)])
    ln[0] = -1
    out, lse, ws = attend(full, q[:1], ws=ws)
    assert D.dsa_workspace_status(ws, raise_on_fault=False) == 8 and torch.all(out == 0)


def test_nan_and_infinity_in_a_used_row_reach_the_output():
    pc = Paged([100, 100, 5000], "bf16", seed=1)
    q = randn((3, 16, 576), gen(2))
    pc.rows[pc.phys[1][50], 3] = float("nan")
    pc.rows[pc.phys[2][4000], 3] = float("nan")
    out, lse, _ = attend(pc, q)
    check_rows(out, lse, q, [pc.stored(0), None, None])
    assert torch.all(torch.isnan(out[1:])) and torch.all(torch.isnan(lse[1:]))


def test_same_bits_every_time_without_lse_and_on_other_streams():
    pc = Paged([3000, 77, 9000, 0, 640], "fp8", seed=21)
    q = randn((5, 128, 576), gen(22))
    ref, lse, _ = attend(pc, q)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for s in streams:                    # at the same time, a workspace each
        with torch.cuda.stream(s):
            got.append(attend(pc, q, lse=len(got) != 1))
    torch.cuda.synchronize()
    for o, l, _ in got:
        assert torch.equal(o, ref) and (l is None or torch.equal(l, lse))


def test_captured_call_follows_new_lengths_and_pages():
    """Decode in a CUDA graph: the captured call reads lengths, pages and rows as they are at replay."""
    pc = Paged([1, 500, 2000, 300], "fp8", seed=31, extra_cols=2)
    q = randn((4, 64, 576), gen(32))
    desc = D.attn_desc(4, pc.n_pages * P, 64, 0, TAU)
    ws = torch.empty(D.dsa_latent_attn_workspace_size(desc), dtype=torch.uint8, device=DEV)
    out, lse, _ = attend(pc, q, ws=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            D.dsa_latent_attn_paged(desc, q, pc.cache, None, pc.pages, out, lse, ws=ws)
    torch.cuda.synchronize()
    for lens in ([1, 500, 2000, 300], [0, 1, 64, 2], [1, 130, 1999, 0], [1, 500, 1, 300]):
        pc.len_d.copy_(i32(lens))
        out.fill_(3.0)
        graph.replay()
        assert D.dsa_workspace_status(ws) == 0
        check_rows(out, lse, q, [pc.stored(t)[:L] for t, L in enumerate(lens)])


@pytest.mark.parametrize("H,fmt", [(16, "fp8"), (64, "fp8"), (128, "fp8"), (128, "bf16")])
def test_two_captured_graphs_share_a_workspace(H, fmt):
    """Graphs of two shapes, one over every key and one over selected ones, replayed in turn on one
    stream with one workspace, and between eager calls on it."""
    pa, pb = Paged([700, 3, 2100], fmt, seed=33), Paged([90, 1500, 0, 64, 800], fmt, seed=34)
    qa, qb = randn((3, H, 576), gen(35)), randn((5, H, 576), gen(36))
    sel = i32(_selection(pb.lens, 150, 3))
    need = max(D.dsa_latent_attn_workspace_size(D.attn_desc(n, pc.n_pages * P, H, k, TAU))
               for n, pc, k in ((3, pa, 0), (5, pb, 150)))
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    calls = [(pa, qa, None), (pb, qb, sel)]
    want = [attend(*c, ws=ws) for c in calls]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs, outs = [], []
    with torch.cuda.stream(s):
        for pc, q, idx in calls:
            graphs.append(torch.cuda.CUDAGraph())
            desc = D.attn_desc(q.shape[0], pc.n_pages * P, H, 0 if idx is None else idx.shape[1], TAU)
            out, lse = torch.empty_like(want[len(outs)][0]), torch.empty_like(want[len(outs)][1])
            outs.append((out, lse))
            with torch.cuda.graph(graphs[-1], stream=s):
                D.dsa_latent_attn_paged(desc, q, pc.cache, idx, pc.pages, out, lse, ws=ws)
        for turn in range(6):
            for gr, (o, l), w, c in zip(graphs, outs, want, calls):
                o.fill_(3.0)
                l.fill_(3.0)
                gr.replay()
                if turn & 1:
                    again = attend(*c, ws=ws)
                    assert torch.equal(again[0], w[0])
                assert torch.equal(o, w[0]) and torch.equal(l, w[1])
        assert D.dsa_workspace_status(ws) == 0
    torch.cuda.synchronize()


@pytest.mark.parametrize("H,fmt,sel", [(16, "bf16", False), (128, "bf16", False), (16, "fp8", True), (128, "fp8", True),
                                       (128, "fp8", False)])
@pytest.mark.parametrize("stop", [1, 3])
def test_waits_that_run_out_in_mid_sequence(H, fmt, sel, stop):
    """The feed stops after a tile or three of each CTA: reported, and the next call is clean."""
    pc = Paged([30000, 20000], fmt, seed=63)
    q = randn((2, H, 576), gen(64))
    idx = i32(_selection(pc.lens, 12000, 5)) if sel else None
    ref, lse, ws = attend(pc, q, idx)
    try:
        D.dsa_debug_pipeline(stop_after_tiles=stop, wait_ns=1_000_000)
        attend(pc, q, idx, ws=ws)
        assert D.dsa_workspace_status(ws, raise_on_fault=False) & 1
    finally:
        D.dsa_debug_pipeline(-1, 0)
    out, l2, _ = attend(pc, q, idx, ws=ws)
    assert D.dsa_workspace_status(ws) == 0
    assert torch.equal(out, ref) and torch.equal(l2, lse)


def test_rows_of_drafts_share_their_sequence():
    """Verifying drafts: rows with the same pages and growing lengths, each causal."""
    pc = Paged([1003], "bf16", seed=41)
    bt = i32(np.repeat(pc.bt, 4, axis=0))
    ln = i32([1000, 1001, 1002, 1003])
    pc.pages = D.paged_cache(bt, ln, pc.n_pages)
    q = randn((4, 16, 576), gen(42))
    out, lse, ws = attend(pc, q)
    assert D.dsa_workspace_status(ws) == 0
    check_rows(out, lse, q, [pc.stored(0)[:1000 + t] for t in range(4)])


def test_long_cache_offsets_pass_32_bits():
    """Rows whose byte and element offsets pass 2^31: the last pages of a 5 GB bf16 cache."""
    n_pages = (1 << 31) // (P * 576) + 600           # 2^31 elements and more
    rows = torch.full((n_pages * P, 576), float("nan"), dtype=torch.bfloat16, device=DEV)
    kv = randn((300, 576), gen(51))
    bt = np.array([[n_pages - 1, 0, n_pages - 3]], dtype=np.int32)
    for j, p in enumerate(bt[0]):
        part = kv[j * P:(j + 1) * P]
        rows[int(p) * P:int(p) * P + part.shape[0]] = part
    bt_d, ln = i32(bt), i32([300])
    q = randn((1, 128, 576), gen(52))
    out = torch.empty((1, 128, 512), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((1, 128), device=DEV)
    cache, pages = D.latent_cache(rows), D.paged_cache(bt_d, ln, n_pages)
    ws = D.dsa_latent_attn_paged(D.attn_desc(1, n_pages * P, 128, 0, TAU), q, cache, None, pages, out, lse)
    assert D.dsa_workspace_status(ws) == 0
    check_rows(out, lse, q, [kv.double().cpu().numpy()])
    back = torch.empty_like(kv)
    D.dsa_latent_cache_read(cache, pages, 1, i32([0]), back)
    assert torch.equal(back, kv)
    slot = i32([(n_pages - 2) * P + 5])
    D.dsa_latent_cache_write(D.cache_write_desc(kv[:1]), kv[:1], slot, None, None, cache)
    assert torch.equal(rows[(n_pages - 2) * P + 5], kv[0])


def test_wait_that_runs_out_is_reported_and_the_next_call_is_clean():
    for fmt in ("bf16", "fp8"):
        pc = Paged([3000, 2000], fmt, seed=61)
        q = randn((2, 64, 576), gen(62))
        ref, lse, ws = attend(pc, q)
        try:
            D.dsa_debug_pipeline(stop_after_tiles=0, wait_ns=1_000_000)
            attend(pc, q, ws=ws)
            assert D.dsa_workspace_status(ws, raise_on_fault=False) & 1
        finally:
            D.dsa_debug_pipeline(-1, 0)
        out, l2, _ = attend(pc, q, ws=ws)
        assert D.dsa_workspace_status(ws) == 0
        assert torch.equal(out, ref) and torch.equal(l2, lse)


def test_a_decode_step_through_every_operator():
    """Three decode steps as a server runs them: rotate the queries into the absorbed layout, write the
    new rows rotated into their pages, attend over every key and over selected ones, and read the
    sequences back for a prefill chunk."""
    B, H, g = 6, 32, gen(71)
    lens = np.array([0, 5, 127, 128, 600, 1500])
    steps, cap = 3, 1500 + 3
    cols = (cap + P - 1) // P
    n_pages = B * cols + 1
    bt = np.random.default_rng(7).permutation(n_pages)[:B * cols].reshape(B, cols).astype(np.int32)
    bt_d, len_d = i32(bt), i32(lens)
    codes = torch.full((n_pages * P, 512), 0x7F, dtype=torch.uint8, device=DEV)
    scale = torch.full((n_pages * P, 4), 255, dtype=torch.uint8, device=DEV)
    rope = torch.full((n_pages * P, 64), float("nan"), dtype=torch.bfloat16, device=DEV)
    cache, pages = D.latent_cache(codes, scale, rope), D.paged_cache(bt_d, len_d, n_pages)
    tab = D.dsa_rope_table_scaled(1e4, 64, 2048, D.rope_scaling_yarn(4.0, 512)).to(DEV)
    tab64 = tab.double().cpu().numpy()
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    hist = [[] for _ in range(B)]           # the rows each sequence was given, float64, unrotated

    def slots(seqs, pos):
        return i32(bt[seqs, pos // P].astype(np.int64) * P + pos % P)

    def store(kv, seqs, pos):
        D.dsa_latent_cache_write(D.cache_write_desc(kv, D.DSA_CACHE_ROPE | D.DSA_ROPE_INTERLEAVED), kv, slots(seqs, pos),
                                 i32(pos), tab, cache, ws=ws)
        assert D.dsa_workspace_status(ws) == 0
        for r, t in zip(kv.double().cpu().numpy(), seqs):
            hist[t].append(r)

    for t in range(B):                       # the prompts
        if lens[t]:
            store(randn((int(lens[t]), 576), g), np.full(lens[t], t), np.arange(lens[t]))
    for _ in range(steps):
        store(randn((B, 576), g), np.arange(B), lens.copy())
        lens += 1
        len_d.copy_(i32(lens))
        q = torch.empty((B, H, 576), dtype=torch.bfloat16, device=DEV)
        q[..., :512] = randn((B, H, 512), g)
        proj = randn((B, H, 192), g)
        x, o = proj[..., 128:], q[..., 512:]
        D.dsa_rope_apply(D.rope_desc(x, o, D.DSA_ROPE_INTERLEAVED), x, i32(lens - 1), tab, o, ws=ws)
        turned = LO.rope(x.double().cpu().numpy(), tab64[lens - 1][:, None, :, 0], tab64[lens - 1][:, None, :, 1], True, False)
        assert np.all(np.abs(o.double().cpu().numpy() - turned) <= 2.0 ** -7 * np.abs(turned) + 1e-5)
        kv = []
        for t in range(B):
            h = np.stack(hist[t])
            at = tab64[np.arange(lens[t])]
            r = LO.rope(h[:, 512:], at[..., 0], at[..., 1], True, False)
            c, s = LO.fp8_encode(h[:, :512])
            ph = bt[t, np.arange(lens[t]) // P].astype(np.int64) * P + np.arange(lens[t]) % P
            stored = rope[torch.as_tensor(ph, device=DEV)].double().cpu().numpy()
            assert np.all(np.abs(stored - r) <= 2.0 ** -8 * np.abs(r) * (1 + 2.0 ** -7) + 2.0 ** -20)
            kv.append(np.concatenate([LO.fp8_decode(c, s), stored], axis=1))
        desc = D.attn_desc(B, n_pages * P, H, 100, TAU)
        out = torch.empty((B, H, 512), dtype=torch.bfloat16, device=DEV)
        lse = torch.empty((B, H), device=DEV)
        aws = D.dsa_latent_attn_paged(desc, q, cache, None, pages, out, lse)
        assert D.dsa_workspace_status(aws) == 0
        check_rows(out, lse, q, kv)
        idx = _selection(lens, 100, int(lens[0]))
        D.dsa_latent_attn_paged(desc, q, cache, i32(idx), pages, out, lse, ws=aws)
        assert D.dsa_workspace_status(aws) == 0
        check_rows(out, lse, q, [k[i[i >= 0]] for k, i in zip(kv, idx)])
    start = np.concatenate([[0], np.cumsum(lens)[:-1]])
    back = torch.empty((int(lens.sum()), 576), dtype=torch.bfloat16, device=DEV)
    D.dsa_latent_cache_read(cache, pages, B, i32(start), back, ws=ws)
    assert D.dsa_workspace_status(ws) == 0
    assert np.array_equal(back.double().cpu().numpy(), np.concatenate(kv))


@pytest.mark.parametrize("H,fmt,sel", [(16, "bf16", False), (16, "fp8", True), (64, "fp8", False), (128, "bf16", False),
                                       (128, "fp8", False), (128, "fp8", True)])
def test_calls_in_a_row_see_what_the_one_before_wrote(H, fmt, sel):
    """Attention right behind the writing of its rows, queries, lengths and selection, without a
    synchronisation, gives what it gives alone; so does a torch operation right behind it."""
    lens, g = [130, 700, 64, 1500, 1], gen(97)
    pc = Paged(lens, fmt, seed=98)
    slot = torch.cat([p.to(torch.int32) for p in pc.phys])
    n, turns = slot.numel(), 12
    kvs, qs = [randn((n, 576), g) for _ in range(turns)], [randn((5, H, 576), g) for _ in range(turns)]
    ids = [i32(_selection(lens, 200, it)) for it in range(turns)]
    kv, q, idx = torch.zeros_like(kvs[0]), torch.zeros_like(qs[0]), torch.zeros_like(ids[0])
    ln = pc.len_d.clone()
    desc = D.attn_desc(5, pc.n_pages * P, H, 200 if sel else 0, TAU)
    ws, w1 = torch.empty(D.dsa_latent_attn_workspace_size(desc), dtype=torch.uint8, device=DEV), torch.zeros(256, dtype=torch.uint8, device=DEV)
    out, lse = torch.zeros((5, H, 512), dtype=torch.bfloat16, device=DEV), torch.zeros((5, H), device=DEV)

    def run(it, wait):
        sync = torch.cuda.synchronize if wait else (lambda: None)
        kv.copy_(kvs[it])
        sync()
        D.dsa_latent_cache_write(D.cache_write_desc(kv), kv, slot, None, None, pc.cache, ws=w1)
        sync()
        q.copy_(qs[it])
        idx.copy_(ids[it])
        pc.len_d.copy_(ln - (it % 3) * (ln > 2))
        sync()
        D.dsa_latent_attn_paged(desc, q, pc.cache, idx if sel else None, pc.pages, out, lse, ws=ws)
        sync()
        return out.clone(), lse.clone()
    want = [run(it, True) for it in range(turns)]
    for _ in range(4):
        for (o, l), (a, b) in zip(want, [run(it, False) for it in range(turns)]):
            assert torch.equal(o, a) and torch.equal(l, b)


@pytest.mark.parametrize("H,fmt,sel", [(16, "bf16", False), (64, "fp8", True), (128, "fp8", False)])
def test_captured_with_copies_and_a_second_stream(H, fmt, sel):
    """A graph of memory copies, the operators and two branches: writing and attention on one stream, the
    rotation of another tensor on a second one, joined by events."""
    lens, g = [130, 700, 64, 1500, 1], gen(99)
    pc = Paged(lens, fmt, seed=100)
    slot = torch.cat([p.to(torch.int32) for p in pc.phys])
    n = slot.numel()
    kv_in, q_in = torch.zeros((n, 576), dtype=torch.bfloat16, device=DEV), torch.zeros((5, H, 576), dtype=torch.bfloat16, device=DEV)
    kv, q = torch.zeros_like(kv_in), torch.zeros_like(q_in)
    idx = i32(_selection(lens, 200, 6)) if sel else None
    desc = D.attn_desc(5, pc.n_pages * P, H, 200 if sel else 0, TAU)
    ws, w1, w2 = (torch.zeros(k, dtype=torch.uint8, device=DEV) for k in (D.dsa_latent_attn_workspace_size(desc), 256, 256))
    out, lse = torch.zeros((5, H, 512), dtype=torch.bfloat16, device=DEV), torch.zeros((5, H), device=DEV)
    got, turned = torch.zeros_like(out), torch.zeros((5, H, 64), dtype=torch.bfloat16, device=DEV)
    tab, pos = D.dsa_rope_table(1e4, 64, 100).to(DEV), i32([0, 7, 99, 31, 5])
    qv = q[..., 512:]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()

    def step(sync):
        kv.copy_(kv_in)
        q.copy_(q_in)
        sync()
        e = torch.cuda.Event()
        e.record()
        with torch.cuda.stream(s2):
            s2.wait_event(e)
            D.dsa_rope_apply(D.rope_desc(qv, turned), qv, pos, tab, turned, ws=w2)
            done = torch.cuda.Event()
            done.record()
        D.dsa_latent_cache_write(D.cache_write_desc(kv), kv, slot, None, None, pc.cache, ws=w1)
        sync()
        D.dsa_latent_attn_paged(desc, q, pc.cache, idx, pc.pages, out, lse, ws=ws)
        sync()
        torch.cuda.current_stream().wait_event(done)
        got.copy_(out)
    with torch.cuda.stream(s1):
        step(torch.cuda.synchronize)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s1):
            step(lambda: None)
        for it in range(6):
            kv_in.copy_(randn((n, 576), g))
            q_in.copy_(randn((5, H, 576), g))
            graph.replay()
            a = got.clone(), lse.clone(), turned.clone()
            step(torch.cuda.synchronize)
            torch.cuda.synchronize()
            assert torch.equal(a[0], got) and torch.equal(a[1], lse) and torch.equal(a[2], turned)
    assert D.dsa_workspace_status(ws) == 0


def test_random_shapes_one_after_another():
    """Calls of ever new shapes, each kernel's code cold now and then: no wait runs out, whatever the order
    in which the warps get going."""
    rng = np.random.default_rng(77)
    for it in range(90):
        H = int(rng.choice([1, 16, 24, 40, 64, 100, 128]))
        fmt = "fp8" if it % 3 else "bf16"
        lens = rng.integers(0, 1200, size=int(rng.integers(1, 9))).tolist()
        pc = Paged(lens, fmt, seed=it)
        q = randn((len(lens), H, 576), gen(it))
        idx = None
        if fmt == "fp8" and it % 2:
            idx = i32(_selection(lens, 200, it))
        out, lse, ws = attend(pc, q, idx)
        assert D.dsa_workspace_status(ws) == 0, (it, H, fmt, lens)
        if it % 10 == 0:
            rows = [pc.stored(t) for t in range(len(lens))]
            if idx is not None:
                sel = idx.cpu().numpy()
                rows = [r[s[s >= 0]] for r, s in zip(rows, sel)]
            check_rows(out, lse, q, rows)


class _Calls:
    """Attention calls of different shapes and data on one workspace, to be issued directly behind one
    another: every tensor is made beforehand."""

    def __init__(self, H, fmt, sel, seed):
        rng = np.random.default_rng(seed)
        shapes = [rng.integers(0, 300, size=200).tolist(), [64] * 310, [5000, 3], rng.integers(0, 2000, size=31).tolist(),
                  [1], [130] * 77, [0, 9000, 0, 700, 64, 1]]
        self.calls, need = [], 0
        for i, lens in enumerate(shapes):
            pc = Paged(lens, fmt, seed=seed + i)
            n, k = len(lens), 150 if sel else 0
            desc = D.attn_desc(n, pc.n_pages * P, H, k, TAU)
            q = randn((n, H, 576), gen(seed + 20 + i))
            idx = i32(_selection(lens, k, seed + i)) if sel else None
            out = torch.empty((n, H, 512), dtype=torch.bfloat16, device=DEV)
            lse = torch.empty((n, H), device=DEV)
            need = max(need, D.dsa_latent_attn_workspace_size(desc))
            self.calls.append((desc, q, pc, idx, out, lse))
        self.ws = torch.empty(need, dtype=torch.uint8, device=DEV)

    def run(self, after=lambda: None):
        for desc, q, pc, idx, out, lse in self.calls:
            D.dsa_latent_attn_paged(desc, q, pc.cache, idx, pc.pages, out, lse, ws=self.ws)
            after()

    def results(self):
        return [(out.clone(), lse.clone()) for *_, out, lse in self.calls]

    def forget(self):
        for *_, out, lse in self.calls:
            out.fill_(7.0)
            lse.fill_(7.0)

    def check(self, want):
        for (o, l), (a, b) in zip(want, self.results()):
            assert torch.equal(o, a) and torch.equal(l, b)


def _alone_and_in_a_row(c):
    """The results of synchronised calls, of calls without a synchronisation, and of a captured graph."""
    def check_status():
        assert D.dsa_workspace_status(c.ws) == 0
    c.run(check_status)                       # (dsa_workspace_status synchronises)
    want = c.results()
    for desc, q, pc, idx, out, lse in c.calls:
        at = [0, len(pc.lens) - 1]
        kv = [None] * len(pc.lens)
        for t in at:
            kv[t] = pc.stored(t) if idx is None else pc.stored(t)[[j for j in idx[t].tolist() if j >= 0]]
        check_rows(out, lse, q, kv)
    for _ in range(10):
        c.forget()
        for _ in range(3):
            c.run()
        c.check(want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            c.run()
            c.run()
        for _ in range(10):
            c.forget()
            graph.replay()
            graph.replay()
            c.check(want)
    torch.cuda.synchronize()
    check_status()


@pytest.mark.parametrize("H,fmt,sel", [(100, "bf16", False), (128, "bf16", False), (100, "fp8", True), (128, "fp8", False)])
def test_pairs_take_over_the_shared_memory_of_the_call_before(H, fmt, sel):
    """Calls of the pair kernel directly behind one another, a pair walking from no row to many: nothing of
    the call before (copies, commits to the peer's barriers) may reach the shared memory of the next one."""
    _alone_and_in_a_row(_Calls(H, fmt, sel, 500 + H))


@pytest.mark.parametrize("H,fmt,sel", [(16, "bf16", False), (16, "fp8", True), (64, "fp8", False), (64, "fp8", True),
                                       (128, "fp8", False), (128, "fp8", True), (128, "bf16", False)])
def test_attention_calls_right_behind_one_another(H, fmt, sel):
    """Split calls with different queries, lengths and selections on one workspace, no other operation
    between them: partials, starts, tile counts and the ring are the call's own, never the one's before."""
    _alone_and_in_a_row(_Calls(H, fmt, sel, 700 + H))


@pytest.mark.parametrize("H,fmt,sel", [(16, "bf16", False), (16, "fp8", False), (64, "fp8", True), (128, "bf16", False),
                                       (128, "fp8", False), (128, "fp8", True)])
def test_attention_right_behind_the_writing_of_its_rows(H, fmt, sel):
    """Turns of rotation into q, writing every cached row and attention, with nothing between them and ever
    other data: the bits of synchronised turns, eagerly and captured."""
    lens, g, turns = [130, 700, 64, 1500, 1, 4000], gen(197), 5
    pc = Paged(lens, fmt, seed=198)
    slot = torch.cat([p.to(torch.int32) for p in pc.phys])
    n, B = slot.numel(), len(lens)
    kvs = [randn((n, 576), g) for _ in range(turns)]
    src = [randn((B, H, 576), g) for _ in range(turns)]
    ids = [i32(_selection(lens, 200, it)) if sel else None for it in range(turns)]
    q = src[0].clone()
    tab, pos = D.dsa_rope_table(1e4, 64, 100).to(DEV), i32([0, 7, 99, 31, 5, 60])
    desc = D.attn_desc(B, pc.n_pages * P, H, 200 if sel else 0, TAU)
    ws, w1, w2 = (torch.zeros(k, dtype=torch.uint8, device=DEV) for k in (D.dsa_latent_attn_workspace_size(desc), 256, 256))
    outs = [(torch.zeros((B, H, 512), dtype=torch.bfloat16, device=DEV), torch.zeros((B, H), device=DEV)) for _ in range(turns)]

    def run(sync):
        for it in range(turns):
            x, y = src[it][..., 512:], q[..., 512:]
            D.dsa_rope_apply(D.rope_desc(x, y), x, pos, tab, y, ws=w2)
            sync()
            D.dsa_latent_cache_write(D.cache_write_desc(kvs[it]), kvs[it], slot, None, None, pc.cache, ws=w1)
            sync()
            D.dsa_latent_attn_paged(desc, q, pc.cache, ids[it], pc.pages, *outs[it], ws=ws)
            sync()

    run(torch.cuda.synchronize)
    want = [(o.clone(), l.clone()) for o, l in outs]
    assert not torch.equal(want[0][0], want[1][0])

    def check():
        for (o, l), (a, b) in zip(want, outs):
            assert torch.equal(o, a) and torch.equal(l, b)
            a.fill_(7.0)
            b.fill_(7.0)
    for _ in range(10):
        run(lambda: None)
        check()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            run(lambda: None)
        for _ in range(10):
            graph.replay()
            check()
    torch.cuda.synchronize()
    assert all(D.dsa_workspace_status(w) == 0 for w in (ws, w1, w2))


@pytest.mark.parametrize("H,fmt,sel", [(1, "bf16", False), (16, "bf16", False), (64, "bf16", False), (128, "bf16", False),
                                       (16, "fp8", False), (64, "fp8", False), (100, "fp8", False), (16, "fp8", True),
                                       (40, "fp8", True), (128, "fp8", True)])
def test_infinities_and_nan_in_used_rows(H, fmt, sel):
    """Scores of plus and minus infinity (an infinite rotary dim: the query's sign decides), a NaN in the
    rotary and in the latent dims, infinite values (fp8: a group stored as NaN), in the first tile, in the last
    and in the middle of a split row, as the only key, and (selected) in a row that is not selected."""
    lens = [100, 700, 5000, 300, 1, 1, 9000, 64, 65, 2000]
    pc = Paged(lens, fmt, seed=H)
    q = randn((len(lens), H, 576), gen(H + 1))
    inf, nan = float("inf"), float("nan")

    def poke(t, j, dim, value):
        if fmt == "bf16":
            pc.rows[pc.phys[t][j], dim] = value
            pc.kv[t][j, dim] = value
        elif dim >= 512:
            pc.rope[pc.phys[t][j], dim - 512] = value
        else:
            pc.codes[pc.phys[t][j], dim // 128 * 128:dim // 128 * 128 + 128] = 0x7F
            pc.scale[pc.phys[t][j], dim // 128] = 255
    pokes = [(0, 5, 520, inf), (1, 300, 575, -inf), (1, 699, 512, inf), (2, 4000, 530, nan), (3, 299, 17, inf),
             (4, 0, 540, inf), (5, 0, 100, nan), (6, 8999, 515, inf), (8, 64, 513, -inf), (9, 1000, 300, nan)]
    for p in pokes:
        poke(*p)
    idx = None
    rows = [pc.stored(t) for t in range(len(lens))]
    if sel:
        idx = _selection(lens, 200, H)
        for t, j, _, _ in pokes:
            if t == 9:
                idx[t, idx[t] == j] = 999                      # not selected: its NaN stays out
            elif not np.any(idx[t] == j):
                idx[t, 7] = j
        rows = [r[i[i >= 0]] for r, i in zip(rows, idx)]
        assert np.all(np.isfinite(rows[9]))
        idx = i32(idx)
    out, lse, ws = attend(pc, q, idx)
    assert D.dsa_workspace_status(ws) == 0
    check_exceptional(out, lse, q, rows)


@pytest.mark.parametrize("H,fmt", [(16, "bf16"), (33, "fp8"), (64, "bf16"), (100, "bf16"), (128, "fp8")])
def test_nothing_of_an_unused_row_shows(H, fmt):
    """Every cache row past a sequence's end, and every row of a page outside the cache's used ones, is NaN:
    all results are finite."""
    pc = Paged(EDGES + [4000, 20000], fmt, seed=H + 3)
    q = randn((len(pc.lens), H, 576), gen(H + 4))
    cases = [None] + ([i32(_selection(pc.lens, 300, H, holes=True))] if fmt == "fp8" else [])
    for idx in cases:
        out, lse, ws = attend(pc, q, idx)
        assert D.dsa_workspace_status(ws) == 0
        assert torch.all(torch.isfinite(out)) and not torch.any(torch.isnan(lse))
        rows = [pc.stored(t) for t in range(len(pc.lens))]
        if idx is not None:
            rows = [r[i[i >= 0]] for r, i in zip(rows, idx.cpu().numpy())]
        check_exceptional(out, lse, q, rows)


@pytest.mark.parametrize("H,fmt", [(16, "bf16"), (16, "fp8"), (128, "bf16"), (128, "fp8")])
def test_nothing_shows_in_place_of_a_page_outside_the_cache(H, fmt):
    """The skipped keys count as absent even where the page that is read in their place holds NaN."""
    pc = Paged([500, 130], fmt, seed=71)
    spare = sorted(set(range(pc.n_pages)) - set(pc.bt[pc.bt >= 0].tolist()))
    bt = pc.bt.copy()
    if 0 not in spare:                            # page 0, unused, becomes one of NaN
        bt[pc.bt == 0] = spare[0]
        old, new = slice(0, P), slice(spare[0] * P, spare[0] * P + P)
        for b in ((pc.rows,) if fmt == "bf16" else (pc.codes, pc.scale, pc.rope)):
            kept = b[new].clone()
            b[new] = b[old]
            b[old] = kept
        for t, L in enumerate(pc.lens):
            j = np.arange(L)
            pc.phys[t] = torch.as_tensor(bt[t, j // P].astype(np.int64) * P + j % P, device=DEV)
    rows = [pc.stored(t) for t in range(2)]
    bt[0, 2], bt[1, 1] = pc.n_pages + 3, -9
    bt_d = i32(bt)
    pc.pages = D.paged_cache(bt_d, pc.len_d, pc.n_pages)
    q = randn((2, H, 576), gen(72))
    out, lse, ws = attend(pc, q)
    assert D.dsa_workspace_status(ws, raise_on_fault=False) == 2
    check_exceptional(out, lse, q, [np.concatenate([rows[0][:256], rows[0][384:]]), rows[1][:128]])


def test_long_fp8_cache_offsets_pass_32_bits():
    """Codes whose offsets pass 2^31, at the end of a 2.2 GB array, through every fp8 path."""
    n_pages = (1 << 31) // (P * 512) + 40
    codes = torch.full((n_pages * P, 512), 0x7F, dtype=torch.uint8, device=DEV)
    scale = torch.full((n_pages * P, 4), 255, dtype=torch.uint8, device=DEV)
    rope = torch.full((n_pages * P, 64), float("nan"), dtype=torch.bfloat16, device=DEV)
    cache = D.latent_cache(codes, scale, rope)
    kv, L = randn((300, 576), gen(151)), 300
    bt = np.array([[n_pages - 1, 0, n_pages - 3]], dtype=np.int32)
    j = np.arange(L)
    slot = i32(bt[0, j // P].astype(np.int64) * P + j % P)
    ws = D.dsa_latent_cache_write(D.cache_write_desc(kv), kv, slot, None, None, cache)
    assert D.dsa_workspace_status(ws) == 0
    at = slot.long()
    x = kv.double().cpu().numpy()
    c, s = LO.fp8_encode(x[:, :512])
    assert np.array_equal(codes[at].cpu().numpy(), c) and np.array_equal(scale[at].cpu().numpy(), s)
    stored = np.concatenate([LO.fp8_decode(c, s), x[:, 512:]], axis=1)
    bt_d, ln = i32(bt), i32([L])
    pages = D.paged_cache(bt_d, ln, n_pages)
    back = torch.empty_like(kv)
    D.dsa_latent_cache_read(cache, pages, 1, i32([0]), back)
    assert np.array_equal(back.double().cpu().numpy(), stored)
    for H in (16, 128):
        q = randn((1, H, 576), gen(152))
        for pick in (None, [299, 0, 130, 257, 256, 127, 128]):
            idx = None if pick is None else i32([pick])
            out = torch.empty((1, H, 512), dtype=torch.bfloat16, device=DEV)
            lse = torch.empty((1, H), device=DEV)
            desc = D.attn_desc(1, n_pages * P, H, 0 if pick is None else len(pick), TAU)
            ws = D.dsa_latent_attn_paged(desc, q, cache, idx, pages, out, lse)
            assert D.dsa_workspace_status(ws) == 0
            check_exceptional(out, lse, q, [stored if pick is None else stored[pick]])


@pytest.mark.parametrize("H", [16, 64, 128])
def test_a_key_listed_twice_counts_twice(H):
    pc = Paged([400, 90], "fp8", seed=161)
    q = randn((2, H, 576), gen(162))
    idx = np.full((2, 130), -1, dtype=np.int32)
    idx[0, :129] = np.repeat(np.arange(43) * 9, 3)
    idx[1, 5:] = 77
    out, lse, ws = attend(pc, q, i32(idx))
    assert D.dsa_workspace_status(ws) == 0
    check_exceptional(out, lse, q, [pc.stored(t)[idx[t][idx[t] >= 0]] for t in range(2)])
