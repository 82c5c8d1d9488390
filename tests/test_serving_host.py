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
