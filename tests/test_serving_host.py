"""Host-side checks of the operators around a decode step: refused arguments and the float64 definitions
that the GPU tests compare with.  Nothing here launches a kernel."""
import ctypes as C

import numpy as np
import pytest
import torch

import dsa_indexer_cross_gb300 as D
from dsa_indexer_cross_gb300 import _lib
from oracle import serving_oracle as SO


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dsa_indexer_cross_gb300.build import build
    build()


A16 = 1 << 20         # an aligned address that is never read: every call here is refused first


def _verify(desc, target=A16, draft=A16, tokens=A16, lens=None, u=A16, us=A16, out=A16, acc=A16, ws=A16, n=256):
    return _lib.lib().dsa_mtp_verify(desc, target, draft, tokens, lens, u, us, out, acc, ws, n, None)


def test_verify_refusals():
    mk = lambda **k: D.VerifyDesc(**{**dict(n_seq=2, n_draft=3, vocab=100, dtype=D.DSA_F32, target_stride=100,  # noqa: E731
                                           draft_stride=100), **k})
    ok = mk()
    assert _lib.lib().dsa_mtp_verify(None, *[A16] * 8, A16, 256, None) == 1
    for bad in (dict(n_seq=-1), dict(n_draft=-1), dict(vocab=0), dict(dtype=2), dict(target_stride=99), dict(draft_stride=99)):
        assert _verify(mk(**bad)) == 1, bad
    assert _verify(mk(vocab=(1 << 30) + 1, target_stride=1 << 31, draft_stride=1 << 31)) == 2
    assert _verify(mk(n_seq=1 << 30, n_draft=1)) == 2
    for k in ("target", "tokens", "u", "us", "out", "acc", "ws"):
        assert _verify(ok, **{k: None}) == 1, k
    assert _verify(ok, ws=A16 + 128) == 1 and _verify(ok, n=255) == 6
    assert _verify(ok, target=A16 + 2) == 1 and _verify(ok, draft=A16 + 2) == 1
    assert _verify(mk(dtype=D.DSA_BF16), target=A16 + 1) == 1
    # everything in order: only the device is missing here
    if not torch.cuda.is_available():
        assert _verify(ok) == 4 and _verify(mk(n_draft=0), tokens=None, u=None, draft=None) == 4
        assert _verify(mk(draft_stride=0), draft=None) == 4


def test_verify_desc_of_views():
    t = torch.zeros((4, 3, 100))
    d = D.verify_desc(t, torch.zeros((4, 2, 100)))
    assert (d.n_seq, d.n_draft, d.vocab, d.dtype, d.target_stride, d.draft_stride) == (4, 2, 100, D.DSA_F32, 100, 100)
    assert D.verify_desc(torch.zeros((4, 3, 128))[..., :100]).target_stride == 128
    assert D.verify_desc(torch.zeros((4, 1, 100))).n_draft == 0
    assert D.verify_desc(torch.zeros((4, 2, 100), dtype=torch.bfloat16)[:, :1]).target_stride == 200
    for bad in (lambda: D.verify_desc(t[0]), lambda: D.verify_desc(t.half()), lambda: D.verify_desc(t, torch.zeros((4, 3, 100))),
                lambda: D.verify_desc(t, torch.zeros((4, 2, 100), dtype=torch.bfloat16)), lambda: D.verify_desc(t[..., ::2]),
                lambda: D.verify_desc(torch.zeros((4, 5, 100))[:, :3]), lambda: D.verify_desc(t[:, :0])):
        with pytest.raises(ValueError):
            bad()


def test_verify_definition_by_hand():
    p = np.array([[0.5, 0.25, 0.25, 0.0], [0.1, 0.2, 0.3, 0.4], [0.0, 0.0, 1.0, 0.0]])
    q = np.array([[0.25, 0.5, 0.25, 0.0], [0.4, 0.3, 0.2, 0.1]])
    # both taken, the last row's token drawn
    out, a = SO.verify(p, q, [0, 3], 2, [0.9, 0.9], 0.5)
    assert out.tolist() == [0, 3, 2] and a == 2
    # the first refused (0.9 * 0.5 >= 0.25): the rest of row 0 is [.25, 0, 0, 0]
    out, a = SO.verify(p, q, [1, 3], 2, [0.9, 0.0], 0.99)
    assert out.tolist() == [0, -1, -1] and a == 0
    # the second refused: row 1 leaves [0, 0, .1, .3]
    for u, want in ((0.2, 2), (0.26, 3), (0.0, 2)):
        out, a = SO.verify(p, q, [0, 0], 2, [0.0, 0.5], u)
        assert out.tolist() == [0, want, -1] and a == 1
    # one draft only: drawn from row 1 itself
    out, a = SO.verify(p, q, [0, 0], 1, [0.0, 0.0], 0.35)
    assert out.tolist() == [0, 2, -1] and a == 1
    # without draft probabilities: u < p, and the refused token takes no part
    out, a = SO.verify(p, None, [0, 3], 2, [0.5, 0.0], 0.4)
    assert out.tolist() == [1, -1, -1] and a == 0


def test_verify_definition_follows_the_target():
    """Summed over every draft and a fine grid of numbers, the first token's distribution is the target's."""
    rng = np.random.default_rng(0)
    p, q = rng.dirichlet(np.ones(4)), rng.dirichlet(np.ones(4))
    n, got = 2000, np.zeros(4)
    grid = (np.arange(n) + 0.5) / n
    for x in range(4):
        taken = np.mean(grid * q[x] < p[x])
        got[x] += q[x] * taken
        if taken < 1:
            drawn = [SO.verify(np.stack([p, p]), q[None], [x], 1, [1.0], u)[0][0] for u in grid]
            got += q[x] * (1 - taken) * np.bincount(drawn, minlength=4) / n
    assert np.all(np.abs(got - p) <= 4.0 / n)


# ------------------------------------------------------------------------------- the latent cache's calls

def _cache(n_rows=1024, fmt=0, latent=A16, scale=None, rope=None):
    return D.LatentCache(latent, scale, rope, n_rows, fmt)


def _pages(max_pages=8, n_pages=8, page_rows=128, table=A16, lens=A16):
    return _lib.PagedCache(table, lens, max_pages, n_pages, page_rows)


def _desc(n=4, H=16, n_kv=1024, tau=0.1, **k):
    return D.attn_desc(n, n_kv, H, 0, tau, **k)


def _attend_shared(desc=None, q=A16, cache=None, groups=None, pages=None, out=A16, ws=A16, n=1 << 40):
    groups = D.SharedRows(A16, A16, 2, 3) if groups is None else groups
    return _lib.lib().dsa_latent_attn_shared(desc or _desc(), q, cache or _cache(), groups, pages or _pages(), out, None, ws, n,
                                             None)


LATENT_REFUSALS = [(dict(desc=_desc(H=0)), 4), (dict(desc=_desc(H=129)), 4), (dict(desc=_desc(n=-1)), 1),
                   (dict(desc=_desc(d_qk=512)), 4), (dict(desc=_desc(n_kv=2048)), 2), (dict(cache=_cache(n_rows=1000)), 2),
                   (dict(cache=_cache(latent=None)), 1), (dict(cache=_cache(fmt=2)), 1), (dict(cache=_cache(fmt=1)), 1),
                   (dict(cache=_cache(latent=A16 + 8)), 1), (dict(pages=_pages(page_rows=64)), 4),
                   (dict(pages=_pages(table=None)), 1), (dict(pages=_pages(lens=None)), 1), (dict(pages=_pages(max_pages=0)), 1),
                   (dict(pages=_pages(n_pages=9)), 2), (dict(pages=_pages(max_pages=1 << 25)), 2),
                   (dict(desc=_desc(n=1 << 28, H=128)), 2), (dict(q=None), 1), (dict(out=None), 1), (dict(ws=None), 1),
                   (dict(q=A16 + 2), 1), (dict(ws=A16 + 128), 1)]


@pytest.mark.parametrize("bad,status", LATENT_REFUSALS + [
    (dict(groups=D.SharedRows(A16, A16, -1, 3)), 1), (dict(groups=D.SharedRows(A16, A16, 2, 0)), 1),
    (dict(groups=D.SharedRows(None, A16, 2, 3)), 1), (dict(groups=D.SharedRows(A16, None, 2, 3)), 1),
    (dict(groups=D.SharedRows(A16, A16, (1 << 24) + 1, 3)), 2), (dict(out=A16 + 2), 1)])
def test_shared_attention_refusals(bad, status):
    assert _attend_shared(**bad) == status


def test_shared_attention_in_order_wants_only_a_device():
    if torch.cuda.is_available():
        pytest.skip("a device is there: the call would run on addresses that are none")
    assert _attend_shared() == 4 and _attend_shared(groups=D.SharedRows(None, None, 0, 1)) == 4
    assert _attend_shared(desc=_desc(n=0), q=None, out=None, ws=None, pages=_pages(table=None, lens=None)) == 0
    assert _lib.lib().dsa_latent_attn_shared(None, A16, _cache(), D.SharedRows(A16, A16, 2, 3), _pages(), A16, None, A16, 1 << 40,
                                             None) == 1


def test_shared_attention_workspace():
    size = lambda n, H, g, r: D.dsa_latent_attn_shared_workspace_size(_desc(n, H), D.SharedRows(None, None, g, r))  # noqa: E731
    assert size(4, 16, 1, 4) >= D.dsa_latent_attn_workspace_size(_desc(4, 16)) - (1 << 20)
    assert size(64, 16, 1, 64) > size(64, 16, 1, 4)
    # what the header says: 4 KB a row and head, and up to 40, 130, 320 MB
    for n, H, g, r, most in ((4, 16, 1, 4, 40), (64, 1, 64, 1, 40), (40, 16, 4, 40, 130), (200, 128, 20, 10, 320), (2000, 64, 1, 2000, 320)):
        assert size(n, H, g, r) <= 4096 * n * H + 200 * (n + g) + (most << 20), (n, H)
    for bad in (lambda: size(-1, 16, 1, 1), lambda: size(4, 16, -1, 1), lambda: size(4, 16, 1, 0), lambda: size(1 << 28, 128, 1, 1)):
        with pytest.raises(D.DsaError):
            bad()


def test_shared_rows_of_tensors():
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32)  # noqa: E731
    for bad in (lambda: D.shared_rows(i32(0, 2).long(), i32(5), 2), lambda: D.shared_rows(i32(0), i32(5), 2),
                lambda: D.shared_rows(i32(0, 2), i32(5).float(), 2), lambda: D.shared_rows(i32(0, 2), i32(5), 2)):
        with pytest.raises(ValueError):      # (the last: not on a device)
            bad()


def _weigh(desc=None, q=A16, cache=None, pages=None, lse=A16, out=A16, stride=1024, ws=A16, n=256):
    return _lib.lib().dsa_latent_key_weights(desc or _desc(), q, cache or _cache(), pages or _pages(), lse, None, out, stride, ws, n,
                                             None)


@pytest.mark.parametrize("bad,status", LATENT_REFUSALS + [(dict(lse=None), 1), (dict(stride=1023), 1), (dict(stride=0), 1)])
def test_key_weights_refusals(bad, status):
    assert _weigh(**bad) == status


def test_key_weights_in_order_wants_only_a_device():
    if not torch.cuda.is_available():
        assert _weigh() == 4 and _weigh(stride=5000) == 4
        assert _weigh(desc=_desc(n=0), q=None, lse=None, out=None, ws=None) == 0
    size = C.c_size_t(0)
    assert _lib.lib().dsa_latent_key_weights_workspace_size(_desc(H=128), _pages(), C.byref(size)) == 0 and size.value == 256
    assert _lib.lib().dsa_latent_key_weights_workspace_size(_desc(H=200), _pages(), C.byref(size)) == 4
    assert _lib.lib().dsa_latent_key_weights_workspace_size(_desc(), _pages(max_pages=0), C.byref(size)) == 1
    assert _lib.lib().dsa_latent_key_weights_workspace_size(_desc(), _pages(), None) == 1


def _evict(desc=None, cache=None, pages=None, w=A16, stride=1024, to=None, to_pages=None, kept=A16, wo=None, wo_stride=0,
           new_len=A16 + 4096, ws=A16, n=256):
    return _lib.lib().dsa_latent_cache_evict(desc or D.evict_desc(2, 500, 4, 16), cache or _cache(), pages or _pages(), w, stride,
                                             to or _cache(), to_pages or _pages(max_pages=4), kept, wo, wo_stride, new_len, ws, n, None)


@pytest.mark.parametrize("bad,status", [
    (dict(desc=D.evict_desc(-1, 5)), 1), (dict(desc=D.evict_desc(2, 0)), 1), (dict(desc=D.evict_desc(2, 5, -1, 0)), 1),
    (dict(desc=D.evict_desc(2, 5, 0, -1)), 1), (dict(desc=D.evict_desc(2, 5, 3, 3)), 1),
    (dict(desc=D.evict_desc(2, 1 << 30, 1 << 30, 1 << 30)), 1), (dict(desc=D.evict_desc(2, 600)), 2),
    (dict(desc=D.evict_desc(2, (1 << 30) + 1)), 2), (dict(cache=_cache(n_rows=1000)), 2), (dict(cache=_cache(latent=None)), 1),
    (dict(to=_cache(fmt=1, scale=A16, rope=A16)), 1), (dict(to=_cache(latent=A16 + 8)), 1), (dict(pages=_pages(table=None)), 1),
    (dict(pages=_pages(lens=None)), 1), (dict(to_pages=_pages(table=None, max_pages=4)), 1), (dict(to_pages=_pages(max_pages=3)), 2),
    (dict(pages=_pages(page_rows=64)), 4), (dict(to_pages=_pages(page_rows=256, max_pages=4)), 4), (dict(to_pages=_pages(n_pages=7)), 2),
    (dict(pages=_pages(max_pages=(1 << 23) + 1), stride=1 << 31), 2), (dict(stride=1023), 1), (dict(wo=A16 + 64, wo_stride=499), 1),
    (dict(w=None), 1), (dict(kept=None), 1), (dict(new_len=None), 1), (dict(ws=None), 1), (dict(ws=A16 + 128), 1), (dict(n=255), 6),
    (dict(wo=A16, wo_stride=500), 1), (dict(new_len=A16), 1)])
def test_evict_refusals(bad, status):
    assert _evict(**bad) == status


def test_evict_in_order_wants_only_a_device():
    if not torch.cuda.is_available():
        assert _evict() == 4 and _evict(wo=A16 + 64, wo_stride=500) == 4
        # the lengths of to_pages are not read, so they may be missing, or be where the new ones go
        assert _evict(to_pages=_pages(max_pages=4, lens=None)) == 4 and _evict(to_pages=_pages(max_pages=4, lens=A16 + 4096)) == 4
        # a budget beyond what the table holds needs no more room than that
        assert _evict(desc=D.evict_desc(2, 5000), pages=_pages(max_pages=4), stride=512) == 4


def test_evict_definition_by_hand():
    w = np.array([5.0, 1.0, 3.0, 3.0, np.nan, 3.0, 9.0, 0.0])
    assert SO.evict(w, 8, 8, 0, 0).tolist() == list(range(8))
    assert SO.evict(w, 8, 4, 0, 0).tolist() == [0, 2, 3, 6]            # of three threes, the first two
    assert SO.evict(w, 8, 4, 1, 1).tolist() == [0, 2, 6, 7]
    assert SO.evict(w, 8, 7, 0, 0).tolist() == [0, 1, 2, 3, 5, 6, 7]   # NaN goes first
    assert SO.evict(w, 8, 3, 2, 1).tolist() == [0, 1, 7]
    assert SO.evict(w, 6, 3, 0, 2).tolist() == [0, 4, 5]


def test_key_weights_definition():
    """The weights of a row are its heads' softmax, summed: one for each head in all."""
    rng = np.random.default_rng(1)
    q, kv = rng.standard_normal((3, 576)), rng.standard_normal((50, 576))
    s = 0.05 * (q @ kv.T)
    lse = np.log(np.exp(s).sum(axis=1))
    w, each, _ = SO.key_weights(q, kv, lse, 0.05)
    assert w.sum() == pytest.approx(3.0, rel=1e-12) and np.allclose(each.sum(axis=1), 1.0)
    w, _, _ = SO.key_weights(q, kv, np.array([lse[0], -np.inf, lse[2]]), 0.05)
    assert w.sum() == pytest.approx(2.0, rel=1e-12)
