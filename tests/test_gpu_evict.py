"""GPU tests of eviction from the paged latent cache (dsa_latent_cache_evict): whole numbers, copied bytes and
copied weights, all of which have to be equal to the definition's."""
import numpy as np
import pytest
import torch

import dsa_indexer_cross_gb300 as D
from latent_cases import DEV, P, Paged, attend, gen, i32, randn
from oracle import serving_oracle as SO

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dsa_indexer_cross_gb300.build import build
    build()
    assert torch.cuda.is_available()


def _weights(pc, seed, kind="spread"):
    g = gen(seed)
    shape = (len(pc.lens), pc.bt.shape[1] * P)
    if kind == "spread":
        return torch.exp(2 * torch.randn(shape, generator=g, device=DEV))
    if kind == "ties":
        return torch.randint(0, 5, shape, generator=g, device=DEV).float()
    if kind == "equal":
        return torch.full(shape, 0.75, device=DEV)
    if kind == "close":       # neighbours in the last places
        return (torch.randint(0, 40, shape, generator=g, device=DEV) + 0x3F800000).to(torch.int32).view(torch.float32).clone()
    x = torch.randn(shape, generator=g, device=DEV)
    pick = torch.randint(0, 12, shape, generator=g, device=DEV)
    for k, v in enumerate((float("nan"), float("inf"), -float("inf"), 0.0, -0.0, 1e-42, -1e-42)):
        x[pick == k] = v
    return x


class Target:
    """Pages for what stays, in an order of their own, in a cache of their own."""

    def __init__(self, pc, keep, seed=0, spare=2):
        need = [(min(L, keep) + P - 1) // P for L in pc.lens]
        self.n_pages = sum(need) + spare
        cols = max(1, -(-min(keep, pc.bt.shape[1] * P) // P))
        perm = np.random.default_rng(seed + 1).permutation(self.n_pages)
        self.bt = np.full((len(need), cols), -7, dtype=np.int32)
        k = 0
        for t, n in enumerate(need):
            self.bt[t, :n] = perm[k:k + n]
            k += n
        rows = self.n_pages * P
        if pc.fmt == "bf16":
            self.arrays = [torch.full((rows, 576), 3.0, dtype=torch.bfloat16, device=DEV)]
        else:
            self.arrays = [torch.full((rows, 512), 17, dtype=torch.uint8, device=DEV),
                           torch.full((rows, 4), 99, dtype=torch.uint8, device=DEV),
                           torch.full((rows, 64), 3.0, dtype=torch.bfloat16, device=DEV)]
        self.cache = D.latent_cache(*self.arrays)
        self.len_d = torch.full((len(need),), -9, dtype=torch.int32, device=DEV)
        self.bt_d = i32(self.bt)
        self.pages = D.paged_cache(self.bt_d, self.len_d, self.n_pages)


def _source(pc):
    return [pc.rows] if pc.fmt == "bf16" else [pc.codes, pc.scale, pc.rope]


def _bytes(x):
    return x.contiguous().view(torch.uint8)


def _evict(pc, w, keep, first, last, to=None, ws=None, pad=0, stream=None, seed=0):
    n = len(pc.lens)
    to = to or Target(pc, keep, seed)
    kept = torch.full((n, keep), -9, dtype=torch.int32, device=DEV)
    w_out = torch.full((n, to.bt.shape[1] * P + pad), -5.0, device=DEV)[:, :to.bt.shape[1] * P]
    desc = D.evict_desc(n, keep, first, last)
    ws = D.dsa_latent_cache_evict(desc, pc.cache, pc.pages, w, to.cache, to.pages, kept, w_out, to.len_d, ws=ws, stream=stream)
    return to, kept, w_out, ws


def _verify(pc, w, keep, first, last, to, kept, w_out, rows=None):
    wh = w.cpu().numpy()
    fresh = Target(pc, keep)
    expect = [a.clone() for a in fresh.arrays]
    kept_h, out_h, len_h = kept.cpu().numpy(), w_out.cpu(), to.len_d.tolist()
    for t, L in enumerate(pc.lens):
        j = SO.evict(wh[t], L, keep, first, last)
        assert len_h[t] == len(j)
        assert np.array_equal(kept_h[t, :len(j)], j) and np.all(kept_h[t, len(j):] == -1), t
        assert torch.equal(_bytes(out_h[t, :len(j)]), _bytes(w[t].cpu()[torch.as_tensor(j)]))
        assert torch.all(out_h[t, len(j):] == -5.0)
        i = np.arange(len(j))
        dst = torch.as_tensor(to.bt[t, i // P].astype(np.int64) * P + i % P, device=DEV)
        src = torch.as_tensor(pc.bt[t, j // P].astype(np.int64) * P + j % P, device=DEV)
        for e, s in zip(expect, _source(pc)):
            e[dst] = s[src]
    for e, a in zip(expect, to.arrays):
        assert torch.equal(_bytes(e), _bytes(a))          # (rows that nothing is copied to: as they were)


EDGES = [0, 1, 2, 31, 32, 33, 127, 128, 129, 255, 256, 257, 1000, 5003]


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("keep,first,last", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (2, 1, 1), (32, 0, 0), (128, 4, 60), (129, 0, 1),
                                             (200, 100, 100), (256, 1, 7), (1000, 4, 64), (6000, 0, 0), (5002, 1, 1)])
@pytest.mark.parametrize("kind", ["spread", "ties", "odd"])
def test_edges(keep, first, last, kind, fmt):
    pc = Paged(EDGES, fmt, seed=keep)
    w = _weights(pc, keep + first, kind)
    to, kept, w_out, ws = _evict(pc, w, keep, first, last)
    assert D.dsa_workspace_status(ws) == 0
    _verify(pc, w, keep, first, last, to, kept, w_out)


@pytest.mark.parametrize("kind", ["spread", "ties", "equal", "close", "odd"])
@pytest.mark.parametrize("lens,keep", [([70000], 30000), ([40001, 3], 1), ([9000] * 50, 2048), (list(range(0, 800, 2)), 100),
                                       ([20000, 100, 15000], 14999), ([250000, 5], 9000), ([14000] * 170, 3000)])
def test_long_and_many_sequences(lens, keep, kind):
    pc = Paged(lens, "fp8", seed=len(lens))
    w = _weights(pc, 5, kind)
    first, last = min(4, keep // 2), keep // 8
    to, kept, w_out, ws = _evict(pc, w, keep, first, last)
    assert D.dsa_workspace_status(ws) == 0
    _verify(pc, w, keep, first, last, to, kept, w_out)


@pytest.mark.parametrize("kind", ["spread", "ties", "odd"])
@pytest.mark.parametrize("lens,keep", [([65000, 48000, 30000, 6145, 6144] + list(range(500, 543)), 2048),       # clusters of six
                                       ([24576, 24575, 5] + [3000] * 149, 1000), ([49152, 49000] + [700] * 98, 4000)])    # of two, of three
def test_keys_held_in_shared_memory(lens, keep, kind):
    """Tables so wide, and so many sequences, that a CTA holds its keys in shared memory (up to the most it can)."""
    pc = Paged(lens, "fp8", seed=len(lens))
    w = _weights(pc, 6, kind)
    to, kept, w_out, ws = _evict(pc, w, keep, 4, 64)
    assert D.dsa_workspace_status(ws) == 0
    _verify(pc, w, keep, 4, 64, to, kept, w_out)
    again = _evict(pc, w, keep, 4, 64)
    assert torch.equal(kept, again[1])


def test_strided_weights_and_no_weights_out():
    pc = Paged([900, 300], "bf16", seed=1)
    wide = torch.full((2, pc.bt.shape[1] * P + 5), float("inf"), device=DEV)
    w = wide[:, :pc.bt.shape[1] * P]
    w.copy_(_weights(pc, 3))
    to, kept, w_out, ws = _evict(pc, w, 200, 3, 10, pad=7)
    _verify(pc, w, 200, 3, 10, to, kept, w_out)
    to2 = Target(pc, 200)
    kept2 = torch.empty_like(kept)
    D.dsa_latent_cache_evict(D.evict_desc(2, 200, 3, 10), pc.cache, pc.pages, w, to2.cache, to2.pages, kept2, None, to2.len_d)
    assert torch.equal(kept, kept2) and torch.equal(to.arrays[0], to2.arrays[0])


def test_within_one_cache_and_shared_source_pages():
    """Two sequences that share a page, copied to other pages of the same arrays."""
    pc = Paged([512, 512], "fp8", seed=2, spare=8)
    pc.bt[1, 0] = pc.bt[0, 0]
    pc.bt_d.copy_(i32(pc.bt))
    free = sorted(set(range(pc.n_pages)) - set(pc.bt[:, :4].ravel().tolist()))
    w = _weights(pc, 9)
    table = i32(np.array([[free[0], free[1]], [free[2], free[3]]]))
    new_len = torch.zeros(2, dtype=torch.int32, device=DEV)
    kept = torch.empty((2, 200), dtype=torch.int32, device=DEV)
    before = [a.clone() for a in _source(pc)]
    D.dsa_latent_cache_evict(D.evict_desc(2, 200, 16, 16), pc.cache, pc.pages, w, pc.cache,
                             D.paged_cache(table, new_len, pc.n_pages), kept, None, new_len)
    assert new_len.tolist() == [200, 200]
    for t in range(2):
        j = SO.evict(w[t].cpu().numpy(), 512, 200, 16, 16)
        assert np.array_equal(kept[t].cpu().numpy(), j)
        i = np.arange(200)
        for a, b in zip(_source(pc), before):
            dst = torch.as_tensor(table[t].cpu().numpy()[i // P].astype(np.int64) * P + i % P, device=DEV)
            src = torch.as_tensor(pc.bt[t, j // P].astype(np.int64) * P + j % P, device=DEV)
            assert torch.equal(_bytes(a[dst]), _bytes(b[src]))
    used = torch.as_tensor(np.unique(pc.bt[:, :4]).astype(np.int64), device=DEV)
    for a, b in zip(_source(pc), before):
        assert torch.equal(_bytes(a.view(pc.n_pages, -1)[used]), _bytes(b.view(pc.n_pages, -1)[used]))


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_bad_pages_and_lengths(fmt):
    pc = Paged([600, 700, 50], fmt, seed=3)
    w = _weights(pc, 4)
    want = SO.evict(w[0].cpu().numpy(), 600, 300, 4, 200)
    pc.bt_d[0, 4] = pc.n_pages                     # keys 512 ..: the last 88 of them stay
    to, kept, w_out, ws = _evict(pc, w, 300, 4, 200)
    assert D.dsa_workspace_status(ws, raise_on_fault=False) == 2
    assert np.array_equal(kept[0].cpu().numpy(), want)
    i = np.nonzero(want >= 512)[0]
    rows = torch.as_tensor(to.bt[0, i // P].astype(np.int64) * P + i % P, device=DEV)
    fresh = Target(pc, 300)
    for a, b in zip(to.arrays, fresh.arrays):
        assert torch.equal(a[rows], b[rows])       # left as they were
    pc.bt_d[0, 4] = int(pc.bt[0, 4])
    to = Target(pc, 300)
    to.bt_d[1, 1] = -1
    _, _, _, ws = _evict(pc, w, 300, 4, 200, to=to)
    assert D.dsa_workspace_status(ws, raise_on_fault=False) == 2
    pc.len_d[2], pc.len_d[1] = -4, 1 << 30
    to, kept, w_out, ws = _evict(pc, w, 50, 4, 0, to=Target(pc, 300))
    assert D.dsa_workspace_status(ws, raise_on_fault=False) & 8
    assert to.len_d.tolist() == [50, 50, 0] and torch.all(kept[2] == -1)
    pc.len_d.copy_(i32(pc.lens))
    to, kept, w_out, ws = _evict(pc, w, 300, 4, 200)
    assert D.dsa_workspace_status(ws) == 0
    _verify(pc, w, 300, 4, 200, to, kept, w_out)


def test_two_streams_a_graph_and_an_empty_call():
    pcs = [Paged([3000, 200, 5000], "fp8", seed=s) for s in (1, 2)]
    ws_in = [_weights(pc, 7) for pc in pcs]
    streams = [torch.cuda.Stream() for _ in pcs]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                got.append((k, _evict(pcs[k], ws_in[k], 1000, 4, 100)))
    torch.cuda.synchronize()
    for k, (to, kept, w_out, _) in got:
        _verify(pcs[k], ws_in[k], 1000, 4, 100, to, kept, w_out)
    w = ws_in[0].clone()
    to = Target(pcs[0], 1000)
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    kept = torch.empty((3, 1000), dtype=torch.int32, device=DEV)
    w_out = torch.full((3, to.bt.shape[1] * P), -5.0, device=DEV)
    call = lambda: D.dsa_latent_cache_evict(D.evict_desc(3, 1000, 4, 100), pcs[0].cache, pcs[0].pages, w, to.cache,  # noqa: E731
                                            to.pages, kept, w_out, to.len_d, ws=ws)
    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
        call()
    w.copy_(_weights(pcs[0], 77))
    for a, b in zip(to.arrays, Target(pcs[0], 1000).arrays):
        a.copy_(b)
    g.replay()
    _verify(pcs[0], w, 1000, 4, 100, to, kept, w_out)
    e = torch.empty((0, 1000), dtype=torch.int32, device=DEV)
    ws.fill_(255)
    D.dsa_latent_cache_evict(D.evict_desc(0, 1000), pcs[0].cache, pcs[0].pages, w, to.cache, to.pages, e, None,
                             torch.empty(0, dtype=torch.int32, device=DEV), ws=ws)
    assert D.dsa_workspace_status(ws) == 0


def test_a_decode_step_then_eviction_then_attention():
    """The operators as they are used: rows decode, their keys' weights add up, the cache is cut, and attention over
    what stays equals attention over these rows."""
    from latent_cases import check_rows
    pc = Paged([700, 2000, 90], "fp8", seed=4)
    H, keep = 16, 512
    acc = torch.zeros((3, pc.bt.shape[1] * P), device=DEV)
    desc = D.attn_desc(3, pc.n_pages * P, H, 0, 1 / 24)
    for step in range(3):
        q = randn((3, H, 576), gen(step))
        _, lse, _ = attend(pc, q)
        D.dsa_latent_key_weights(desc, q, pc.cache, pc.pages, lse, acc, acc)
    to, kept, w_out, ws = _evict(pc, acc, keep, 4, 64)
    _verify(pc, acc, keep, 4, 64, to, kept, w_out)
    q = randn((3, H, 576), gen(9))
    out = torch.empty((3, H, 512), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((3, H), device=DEV)
    D.dsa_latent_attn_paged(D.attn_desc(3, to.n_pages * P, H, 0, 1 / 24), q, to.cache, None, to.pages, out, lse)
    k = kept.cpu().numpy()
    check_rows(out, lse, q, [pc.stored(t)[k[t][k[t] >= 0]] for t in range(3)])
