"""GPU tests of draft verification (dsa_mtp_verify) against float64: every result is a whole number and has
to be equal."""
import numpy as np
import pytest
import torch

import dsa_indexer_cross_gb300 as D
from oracle import serving_oracle as SO

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dsa_indexer_cross_gb300.build import build
    build()
    assert torch.cuda.is_available()


def _case(n, d, V, dtype, probs=True, seed=0, sharp=4.0, pad=0, offset=0):
    """Seeded distributions that mostly agree, as views of rows V + pad elements apart that begin `offset`
    elements behind a 16-byte boundary."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rand = lambda *s: torch.rand(s, generator=g, device=DEV)  # noqa: E731
    logits = sharp * torch.randn((n, d + 1, V), generator=g, device=DEV)
    p = torch.softmax(logits + torch.randn((n, d + 1, V), generator=g, device=DEV), -1).to(dtype)
    q = torch.softmax(logits[:, :d], -1).to(dtype)

    def view(x):
        rows = x.shape[0] * x.shape[1]
        buf = torch.full((rows * (V + pad) + offset + 8,), float("nan"), dtype=dtype, device=DEV)
        v = buf[offset:offset + rows * (V + pad)].view(x.shape[0], x.shape[1], V + pad)[..., :V]
        v.copy_(x)
        return v

    src = q if probs else p[:, :d]
    tokens = torch.multinomial(src.float().reshape(n * d, V), 1, generator=g).reshape(n, d).to(torch.int32) \
        if d else torch.empty((n, 0), dtype=torch.int32, device=DEV)
    lens = torch.randint(0, d + 1, (n,), generator=g, device=DEV)
    lens = torch.where(rand(n) < 0.5, lens, d).to(torch.int32)
    return dict(target=view(p), draft=view(q) if probs else None, tokens=tokens, draft_len=lens, u_accept=rand(n, d),
                u_sample=rand(n))


def _run(c, ws=None, stream=None):
    n, m, _ = c["target"].shape
    out = torch.full((n, m), -9, dtype=torch.int32, device=DEV)
    acc = torch.full((n,), -9, dtype=torch.int32, device=DEV)
    desc = D.verify_desc(c["target"], c["draft"])
    ws = D.dsa_mtp_verify(desc, c["target"], c["draft"], c["tokens"], c["draft_len"], c["u_accept"], c["u_sample"], out,
                          acc, ws=ws, stream=stream)
    return out, acc, ws


def _want(c):
    h = {k: None if v is None else v.double().cpu().numpy() if v.is_floating_point() else v.cpu().numpy() for k, v in c.items()}
    rows = [SO.verify(h["target"][t], None if h["draft"] is None else h["draft"][t], h["tokens"][t],
                      None if h["draft_len"] is None else h["draft_len"][t], h["u_accept"][t], h["u_sample"][t])
            for t in range(h["target"].shape[0])]
    return np.stack([r[0] for r in rows]), np.array([r[1] for r in rows])


def _check(c, bits=0):
    out, acc, ws = _run(c)
    want, taken = _want(c)
    assert D.dsa_workspace_status(ws, raise_on_fault=False) == bits
    assert np.array_equal(acc.cpu().numpy(), taken)
    assert np.array_equal(out.cpu().numpy(), want)
    return out, acc


@pytest.mark.parametrize("probs", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1, 2, 3, 7, 8, 31, 33, 127, 1000, 1024, 4097, 8191, 32000, 50257, 100003])
def test_vocabularies(V, dtype, probs):
    _check(_case(5, 4, V, dtype, probs, seed=V))


@pytest.mark.parametrize("n,d", [(1, 1), (1, 0), (3, 0), (1, 31), (2, 32), (2, 33), (3, 70), (200, 2), (700, 7), (2000, 3)])
def test_sequences_and_drafts(n, d):
    _check(_case(n, d, 1500, torch.float32, d > 0, seed=n + d))


@pytest.mark.parametrize("n", [36, 37, 39, 43, 47, 58, 59, 75, 97, 98, 152, 153, 305])
def test_every_size_of_cluster(n):
    """Numbers of sequences around those that leave room for another CTA each."""
    _check(_case(n, 2, 33001, torch.float32, n % 2 == 0, seed=n))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pad,offset", [(0, 1), (1, 0), (3, 3), (8, 2), (16, 0), (5, 7)])
def test_strides_and_alignment(pad, offset, dtype):
    """NaN lies between the rows: nothing outside them is used."""
    for probs in (True, False):
        _check(_case(6, 3, 5003, dtype, probs, seed=pad + offset, pad=pad, offset=offset))


def test_no_lengths_given_and_no_drafts():
    c = _case(4, 3, 2000, torch.float32)
    c["draft_len"] = None
    _check(c)
    c = _case(4, 3, 2000, torch.float32)
    c["draft_len"] = torch.zeros(4, dtype=torch.int32, device=DEV)
    c["tokens"].fill_(-1)          # not read
    _check(c)


def test_exact_borders():
    """Probabilities that are multiples of 2^-12: every sum is exact, and u times it falls on a border."""
    V = 4096
    p = torch.full((1, 2, V), 2.0 ** -12, device=DEV)
    q = torch.zeros((1, 1, V), device=DEV)
    q[0, 0, 5] = 1.0
    for u in (0, 1, 2047, 2048, 4095):
        c = dict(target=p, draft=q, tokens=torch.full((1, 1), 5, dtype=torch.int32, device=DEV), draft_len=None,
                 u_accept=torch.full((1, 1), 2.0 ** -12, device=DEV),       # u q = p: not taken
                 u_sample=torch.full((1,), u / 4096.0, device=DEV))
        out, acc = _check(c)
        assert int(acc) == 0
        c["u_accept"].fill_(2.0 ** -12 * (1 - 2.0 ** -24))                  # u q < p by one step: taken
        out, acc = _check(c)
        assert out.tolist() == [[5, u]]
    # the drawn token has weight, even at u = 0 and u just below 1
    p = torch.zeros((2, 1, V), device=DEV)
    p[:, 0, 100], p[:, 0, 3000] = 0.25, 0.75
    c = dict(target=p, draft=None, tokens=torch.empty((2, 0), dtype=torch.int32, device=DEV), draft_len=None,
             u_accept=torch.empty((2, 0), device=DEV), u_sample=torch.tensor([0.0, 1 - 2.0 ** -24], device=DEV))
    out, _ = _check(c)
    assert out.tolist() == [[100], [3000]]


def test_numbers_outside_the_unit_interval():
    c = _case(6, 1, 3000, torch.float32, seed=3)
    c["u_sample"] = torch.tensor([1.0, 1.5, -0.5, float("nan"), float("inf"), 0.0], device=DEV)
    c["u_accept"] = torch.tensor([[float("nan")], [2.0], [-1.0], [float("inf")], [0.0], [1.0]], device=DEV)
    _check(c)


def test_no_weight_left():
    """A draft distribution that covers the target's: the token comes from the target; no target, no token."""
    V = 5000
    c = _case(4, 2, V, torch.float32, seed=5)
    c["draft_len"].fill_(2)
    c["draft"].copy_(c["target"][:, :2])
    c["u_accept"].fill_(1.0)               # u q = p: refused
    c["target"][2].zero_()
    c["draft"][3, 0] = 2.0
    out, acc = _check(c)
    assert acc.tolist() == [0, 0, 0, 0] and out[2].tolist() == [-1, -1, -1]
    # a drafted token that holds all of the target's weight, without draft probabilities
    c = _case(1, 1, V, torch.float32, False, seed=6)
    c["target"].zero_()
    c["target"][:, :, 77] = 0.5
    c["tokens"].fill_(77)
    c["u_accept"].fill_(0.75)
    c["draft_len"].fill_(1)
    out, acc = _check(c)
    assert out.tolist() == [[77, -1]] and acc.tolist() == [0]


def test_infinities_nan_and_negative_probabilities():
    V = 20000
    c = _case(5, 1, V, torch.float32, seed=8)
    c["draft_len"].fill_(1)
    c["u_accept"].fill_(1.0)
    c["tokens"].fill_(3)
    c["draft"][:, 0, 3], c["target"][:, 0, 3] = 1.0, 0.0
    c["target"][0, 0, 9000:9100] = float("nan")
    c["draft"][1, 0, 100] = float("nan")
    c["target"][2, 0, 15000] = float("inf")
    c["target"][3, 0, :9000] = -1.0
    c["draft"][4, 0, 50] = float("inf")
    out, acc = _check(c)
    assert out[2, 0] == -1


@pytest.mark.parametrize("n", [3, 3000])       # one block writes the status, or every sequence adds to it
def test_bad_tokens_and_lengths_are_flagged(n):
    c = _case(n, 4, 600, torch.float32, seed=11)
    c["draft_len"].fill_(4)
    _check(c)
    c["tokens"][1, 0] = 600
    _check(c, bits=2)
    c["tokens"][1, 0] = 5
    c["tokens"][n - 1, 3] = -1
    _check(c, bits=2)
    c["draft_len"][0], c["draft_len"][2] = 5, -2
    _check(c, bits=8 if n == 3 else 2 | 8)      # (of three, the last has no draft left: its token is not read)
    c["tokens"][n - 1, 3] = 0
    _check(c, bits=8)
    c["draft_len"].fill_(4)
    _check(c)                                   # the words are cleared
    c = _case(n, 2, 600, torch.float32, False, seed=12)
    c["draft_len"].fill_(2)
    c["tokens"][1, 1] = 1 << 30
    c["u_accept"][1].zero_()
    _check(c, bits=2)


def test_tokens_follow_the_targets_distribution():
    """20000 sequences of one draft: the frequencies of the first token lie within five deviations."""
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    N, V = 20000, 16
    p = torch.softmax(torch.randn(V, generator=g, device=DEV), 0)
    q = torch.softmax(torch.randn(V, generator=g, device=DEV), 0)
    x = torch.multinomial(q, N, replacement=True, generator=g).to(torch.int32)[:, None]
    out = torch.empty((N, 2), dtype=torch.int32, device=DEV)
    acc = torch.empty(N, dtype=torch.int32, device=DEV)
    P, Q = p.expand(N, 2, V).contiguous(), q.expand(N, 1, V).contiguous()
    D.dsa_mtp_verify(D.verify_desc(P, Q), P, Q, x, None, torch.rand((N, 1), generator=g, device=DEV),
                     torch.rand(N, generator=g, device=DEV), out, acc)
    f = torch.bincount(out[:, 0].long(), minlength=V).double() / N
    assert torch.all((f - p.double()).abs() <= 5 * (p.double() * (1 - p.double()) / N).sqrt())


def test_two_streams_a_graph_and_an_empty_call():
    cs = [_case(40, 3, 9001, torch.float32, seed=s) for s in (1, 2)]
    want = [_run(c)[0].clone() for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        for c, s in zip(cs, streams):
            with torch.cuda.stream(s):
                outs.append(_run(c))
    torch.cuda.synchronize()
    for i, (out, _, _) in enumerate(outs):
        assert torch.equal(out, want[i % 2])
    c = {k: v.clone() if v is not None else None for k, v in cs[0].items()}
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    _run(c, ws=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, acc, _ = _run(c, ws=ws)
        out2, _, _ = _run(c, ws=ws)
    for k in ("target", "draft", "tokens", "draft_len", "u_accept", "u_sample"):
        c[k].copy_(cs[1][k])
    g.replay()
    assert torch.equal(out, want[1]) and torch.equal(out2, want[1])
    e = torch.empty((0, 3, 50), device=DEV)
    i = torch.empty((0, 3), dtype=torch.int32, device=DEV)
    D.dsa_mtp_verify(D.verify_desc(e, None), e, None, i, None, torch.empty((0, 2), device=DEV), torch.empty(0, device=DEV), i,
                     torch.empty(0, dtype=torch.int32, device=DEV), ws=ws)
    assert D.dsa_workspace_status(ws) == 0


def test_repeated_calls_are_equal():
    c = _case(64, 4, 131072, torch.float32, seed=4, sharp=6.0)
    first = _run(c)
    for _ in range(3):
        again = _run(c)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    _check(c)


def test_results_over_the_inputs_are_refused():
    """A sequence's lengths and drafts are read by several CTAs, so the results cannot take their place."""
    c = _case(3, 4, 9000, torch.float32, seed=2)
    out, acc, ws = _run(c)
    n, d = 3, 4
    buf = torch.zeros(64, dtype=torch.int32, device=DEV)
    f = torch.zeros(64, device=DEV)
    base = dict(tokens=c["tokens"], draft_len=c["draft_len"], u_accept=c["u_accept"], u_sample=c["u_sample"],
                out=torch.empty((n, d + 1), dtype=torch.int32, device=DEV), acc=torch.empty(n, dtype=torch.int32, device=DEV))
    desc = D.verify_desc(c["target"], c["draft"])

    def call(**kw):
        a = {**base, **kw}
        D.dsa_mtp_verify(desc, c["target"], c["draft"], a["tokens"], a["draft_len"], a["u_accept"], a["u_sample"], a["out"], a["acc"],
                         ws=ws)
        return a
    for bad in (dict(acc=c["draft_len"]), dict(tokens=buf[:12], out=buf[:15]), dict(tokens=buf[14:26], out=buf[:15]),
                dict(draft_len=buf[:3], out=buf[2:17]), dict(out=buf[:15], acc=buf[14:17]), dict(tokens=buf[:12], acc=buf[11:14]),
                dict(u_accept=f[:12], out=f[11:26].view(torch.int32)), dict(u_sample=f[:3], acc=f[:3].view(torch.int32))):
        with pytest.raises(D.DsaError, match="overlap"):
            call(**bad)
    # one behind the other in one buffer: no overlap
    buf[:12] = c["tokens"].reshape(-1)
    buf[12:15] = c["draft_len"]
    a = call(tokens=buf[:12], draft_len=buf[12:15], out=buf[15:30], acc=buf[30:33])
    assert D.dsa_workspace_status(ws) == 0
    assert torch.equal(a["out"].view(n, d + 1), out) and torch.equal(a["acc"], acc)
