"""GPU tests of the attention weight that cached keys receive (dsa_latent_key_weights) against float64."""
import numpy as np
import pytest
import torch

import dsa_indexer_cross_gb300 as D
from latent_cases import DEV, P, TAU, Paged, attend, gen, randn
from oracle import serving_oracle as SO

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dsa_indexer_cross_gb300.build import build
    build()
    assert torch.cuda.is_available()


MARK = -7.25        # elements that the call leaves alone


def _weigh(pc, q, lse, w_in=None, out=None, ws=None, pad=0, stream=None, tau=TAU):
    n, H = q.shape[0], q.shape[1]
    desc = D.attn_desc(n, pc.n_pages * P, H, 0, tau)
    width = pc.bt.shape[1] * P
    if out is None:
        out = torch.full((n, width + pad), MARK, device=DEV)[:, :width]
    ws = D.dsa_latent_key_weights(desc, q, pc.cache, pc.pages, lse, w_in, out, ws=ws, stream=stream)
    return out, ws


def _compare(pc, q, lse, out, w_in=None, rows=None, tau=TAU):
    """A score is a sum of 576 products in fp32, each addition off by at most 2^-23 of the terms' sum B (the tensor
    core may truncate); scaling it, the log-sum-exp in log2 and their difference add 2^-22 of their sizes, the
    exponential 2^-21: each weight is off by the factor e, 576 * 2^-23 B + 2^-21 (|s| + |lse| + 2).  The sum over
    heads and the addition of what was there add (H + 1) 2^-24 of the result's terms."""
    q64, l64, o64 = q.double().cpu().numpy(), lse.double().cpu().numpy(), out.double().cpu().numpy()
    i64 = None if w_in is None else w_in.double().cpu().numpy()
    for t, L in enumerate(pc.lens):
        if rows is not None and t not in rows:
            continue
        kv = pc.stored(t)
        want, w, B = SO.key_weights(q64[t], kv, l64[t], tau)
        before = 0.0 if i64 is None else i64[t, :L]
        with np.errstate(invalid="ignore"):
            s = tau * np.abs(q64[t] @ kv.T) + np.where(np.isfinite(l64[t]), np.abs(l64[t]), 0.0)[:, None]
        e = 576 * 2.0 ** -23 * B + 2.0 ** -21 * (s + 2.0)
        tol = (w * e * (1 + e)).sum(axis=0) + (q.shape[1] + 1) * 2.0 ** -24 * (want + np.abs(before)) + 2.0 ** -120
        bad = np.abs(o64[t, :L] - (want + before)) > tol
        assert not bad.any(), (t, int(bad.sum()), float(np.nanmax(np.abs(o64[t, :L] - (want + before)) / tol)))
        assert np.all(o64[t, L:] == MARK)


EDGES = [0, 1, 2, 63, 64, 65, 127, 128, 129, 0, 191, 192, 193, 1000, 0]


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("H", [1, 3, 16, 17, 32, 33, 64, 65, 100, 128])
def test_edge_lengths(H, fmt):
    pc = Paged(EDGES, fmt, seed=H)
    q = randn((len(EDGES), H, 576), gen(H + 1))
    _, lse, _ = attend(pc, q)
    out, ws = _weigh(pc, q, lse)
    assert D.dsa_workspace_status(ws) == 0
    _compare(pc, q, lse, out)
    # a row's weights are those of its heads: each head's add up to one
    for t, L in enumerate(EDGES):
        if L:
            assert abs(float(out[t, :L].double().sum()) - H) <= H * 2.0 ** -9
    # on top of what the keys have, in other rows' stride, and in place
    w_in = torch.rand((len(EDGES), pc.bt.shape[1] * P + 3), generator=gen(2), device=DEV)[:, :-3]
    out2, ws = _weigh(pc, q, lse, w_in, pad=3)
    _compare(pc, q, lse, out2, w_in)
    w = w_in.clone()
    w3 = torch.empty((len(EDGES), pc.bt.shape[1] * P), device=DEV)
    w3.copy_(w)
    _weigh(pc, q, lse, w3, out=w3)
    for t, L in enumerate(EDGES):
        assert torch.equal(w3[t, :L], out2[t, :L]) and torch.equal(w3[t, L:], w[t, L:])


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("H,lens", [(16, [20000]), (64, [9000, 17, 300]), (128, [33333]), (8, list(range(1, 400, 7))),
                                    (70, [700] * 40), (24, [5000] * 3 + [0] * 70 + [100])])
def test_long_and_many_rows(H, lens, fmt):
    pc = Paged(lens, fmt, seed=len(lens))
    q = randn((len(lens), H, 576), gen(3))
    _, lse, _ = attend(pc, q)
    out, ws = _weigh(pc, q, lse)
    assert D.dsa_workspace_status(ws) == 0
    _compare(pc, q, lse, out, rows=set(range(0, len(lens), max(1, len(lens) // 8))))
    out2, _ = _weigh(pc, q, lse)
    assert torch.equal(out, out2)


@pytest.mark.parametrize("H", [5, 70])
def test_heads_without_keys_infinities_and_nan(H):
    pc = Paged([200, 130, 64], "bf16", seed=1)
    q = randn((3, H, 576), gen(2))
    lse = torch.zeros((3, H), device=DEV)
    _, lse, _ = attend(pc, q)
    lse = lse.clone()
    lse[0, 1] = -float("inf")             # weighs nothing
    lse[1, H - 1] = float("inf")          # weighs nothing either: exp(s - inf)
    lse[2, 0] = float("nan")
    out, ws = _weigh(pc, q, lse)
    assert D.dsa_workspace_status(ws) == 0
    assert torch.all(torch.isnan(out[2, :64])) and torch.all(out[2, 64:] == MARK)
    _compare(pc, q, lse, out, rows={0, 1})
    # a key that is NaN, one that is infinite: only their own weights show it
    _, lse, _ = attend(pc, q)
    pc.rows[pc.phys[0][77], 3] = float("nan")
    out, _ = _weigh(pc, q, lse)
    assert bool(torch.isnan(out[0, 77])) and int(torch.isnan(out[:, :].float()).sum()) == 1


@pytest.mark.parametrize("H", [5, 40, 100])
def test_other_rows_columns_do_not_count(H):
    """A key that is -inf in a dim where this row's heads are positive, and the next row's, which lie behind them in
    q, negative: its scores are -inf, its weight is zero."""
    pc = Paged([300, 300], "bf16", seed=1)
    q = randn((2, H, 576), gen(2))
    q[0, :, 9], q[1, :, 9] = 1.0, -1.0
    pc.rows[pc.phys[0][77], 9] = -float("inf")
    _, lse, _ = attend(pc, q)
    out, ws = _weigh(pc, q, lse)
    assert D.dsa_workspace_status(ws) == 0
    assert float(out[0, 77]) == 0.0 and bool(torch.isfinite(out[0, :300]).all())
    assert abs(float(out[0, :300].double().sum()) - H) <= H * 2.0 ** -9


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("H", [16, 100])
def test_bad_pages_and_lengths(H, fmt):
    pc = Paged([300, 500, 100], fmt, seed=1)
    q = randn((3, H, 576), gen(2))
    _, lse, _ = attend(pc, q)
    good, ws = _weigh(pc, q, lse)
    pc.bt_d[1, 2] = pc.n_pages
    out, ws = _weigh(pc, q, lse)
    assert D.dsa_workspace_status(ws, raise_on_fault=False) == 2
    assert torch.all(out[1, 256:384] == MARK)
    out[1, 256:384] = good[1, 256:384]
    assert torch.equal(out, good)
    pc.bt_d[1, 2] = int(pc.bt[1, 2])
    pc.len_d[2] = -5
    out, ws = _weigh(pc, q, lse)
    assert D.dsa_workspace_status(ws, raise_on_fault=False) == 8
    assert torch.all(out[2] == MARK) and torch.equal(out[:2], good[:2])
    pc.len_d[2] = 100
    out, ws = _weigh(pc, q, lse)
    assert D.dsa_workspace_status(ws) == 0 and torch.equal(out, good)


def test_two_streams_a_graph_and_an_empty_call():
    pcs = [Paged([900, 40, 2000], "fp8", seed=s) for s in (1, 2)]
    for H in (16, 90):
        qs = [randn((3, H, 576), gen(s)) for s in (1, 2)]
        ls = [attend(pc, q)[1] for pc, q in zip(pcs, qs)]
        want = [_weigh(pc, q, l)[0].clone() for pc, q, l in zip(pcs, qs, ls)]
        streams = [torch.cuda.Stream() for _ in pcs]
        torch.cuda.synchronize()
        got = []
        for _ in range(4):
            for k in range(2):
                with torch.cuda.stream(streams[k]):
                    got.append((k, _weigh(pcs[k], qs[k], ls[k])[0]))
        torch.cuda.synchronize()
        assert all(torch.equal(x[t, :L], want[k][t, :L]) for k, x in got for t, L in enumerate(pcs[k].lens))
        q, lse = qs[0].clone(), ls[0].clone()
        ws = _weigh(pcs[0], q, lse)[1]
        acc = torch.zeros_like(want[0])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _weigh(pcs[0], q, lse, acc, out=acc, ws=ws)
            _weigh(pcs[0], q, lse, acc, out=acc, ws=ws)
        acc.zero_()
        g.replay()
        for t, L in enumerate(pcs[0].lens):
            assert torch.equal(acc[t, :L], want[0][t, :L] + want[0][t, :L])
            assert torch.all(acc[t, L:] == 0)
    desc = D.attn_desc(0, pcs[0].n_pages * P, 16, 0, TAU)
    e = torch.empty((0, 16, 576), dtype=torch.bfloat16, device=DEV)
    ws.fill_(255)
    D.dsa_latent_key_weights(desc, e, pcs[0].cache, pcs[0].pages, torch.empty((0, 16), device=DEV), None,
                             torch.empty((0, pcs[0].bt.shape[1] * P), device=DEV), ws=ws)
    assert D.dsa_workspace_status(ws) == 0


@pytest.mark.parametrize("H", [16, 100])
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_a_wait_that_runs_out_is_reported(H, fmt):
    pc = Paged([9000, 5000], fmt, seed=3)
    q = randn((2, H, 576), gen(4))
    _, lse, _ = attend(pc, q)
    want, ws = _weigh(pc, q, lse)
    D.dsa_debug_pipeline(0, 1_000_000)
    try:
        _weigh(pc, q, lse, ws=ws)
        assert D.dsa_workspace_status(ws, raise_on_fault=False) & 1
    finally:
        D.dsa_debug_pipeline(-1, 0)
    out, ws = _weigh(pc, q, lse, ws=ws)
    assert D.dsa_workspace_status(ws) == 0 and torch.equal(out, want)
