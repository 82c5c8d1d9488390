"""GPU tests of the operators around a decode step together: offsets beyond 32 bits, and steps of drafting as a
serving program runs them, eagerly and captured."""
import numpy as np
import pytest
import torch

import dsa_indexer_cross_gb300 as D
from latent_cases import DEV, P, TAU, check_rows, encode, gen, i32, randn
from oracle import latent_oracle as LO
from oracle import serving_oracle as SO

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dsa_indexer_cross_gb300.build import build
    build()
    assert torch.cuda.is_available()


def _store(arrays, at, kv):
    if len(arrays) == 1:
        arrays[0][at] = kv
    else:
        arrays[0][at], arrays[1][at] = encode(kv[:, :512])
        arrays[2][at] = kv[:, 512:]


def _stored(arrays, at):
    if len(arrays) == 1:
        return arrays[0][at].double().cpu().numpy()
    y = LO.fp8_decode(arrays[0][at].cpu().numpy(), arrays[1][at].cpu().numpy())
    return np.concatenate([y, arrays[2][at].double().cpu().numpy()], axis=1)


def _poisoned(n_pages, fmt):
    n = n_pages * P
    if fmt == "bf16":
        return [torch.full((n, 576), float("nan"), dtype=torch.bfloat16, device=DEV)]
    return [torch.full((n, 512), 0x7F, dtype=torch.uint8, device=DEV), torch.full((n, 4), 255, dtype=torch.uint8, device=DEV),
            torch.full((n, 64), float("nan"), dtype=torch.bfloat16, device=DEV)]


@pytest.mark.parametrize("fmt,H", [("bf16", 16), ("fp8", 16), ("fp8", 64), ("fp8", 128)])
def test_offsets_pass_32_bits(fmt, H):
    """Rows whose byte and element offsets pass 2^31, at the end of caches of 5 and 2.2 GB."""
    n_pages = (1 << 31) // (P * (576 if fmt == "bf16" else 512)) + 400
    arrays = _poisoned(n_pages, fmt)
    cache = D.latent_cache(*arrays)
    # 12 rows of 5000 and more keys, their first 4992 (39 pages) shared (enough columns to be staged from 64 heads on)
    n, shared = 12, 39
    lens = [5000 + 3 * t for t in range(n)]
    bt = np.full((n, 90), -1, dtype=np.int32)
    bt[:, :shared] = n_pages - 1 - np.arange(shared)
    bt[:, shared] = n_pages - 1 - shared - np.arange(n)
    bt[:, 0] = 0                                   # and one at its beginning
    phys = [torch.as_tensor(bt[t, np.arange(L) // P].astype(np.int64) * P + np.arange(L) % P, device=DEV)
            for t, L in enumerate(lens)]
    common = randn((shared * P, 576), gen(1))
    for t, L in enumerate(lens):
        _store(arrays, phys[t], torch.cat([common, randn((L - shared * P, 576), gen(2 + t))]))
    bt_d, len_d = i32(bt), i32(lens)
    pages = D.paged_cache(bt_d, len_d, n_pages)
    q = randn((n, H, 576), gen(30))
    out = torch.empty((n, H, 512), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((n, H), device=DEV)
    desc = D.attn_desc(n, n_pages * P, H, 0, TAU)
    start, prefix = i32([0, n]), i32([shared * P])
    ws = D.dsa_latent_attn_shared(desc, q, cache, D.shared_rows(start, prefix, n), pages, out, lse)
    assert D.dsa_workspace_status(ws) == 0
    kv = [_stored(arrays, phys[t]) if t in (0, 7) else None for t in range(n)]
    check_rows(out, lse, q, kv)
    weight = torch.zeros((n, 90 * P), device=DEV)
    D.dsa_latent_key_weights(desc, q, cache, pages, lse, None, weight)
    want, _, _ = SO.key_weights(q[7].double().cpu().numpy(), kv[7], lse[7].double().cpu().numpy(), TAU)
    assert np.all(np.abs(weight[7, :lens[7]].double().cpu().numpy() - want) <= 2.0 ** -10 * want + 1e-30)
    to = np.full((n, 8), -1, dtype=np.int32)
    to[:, :] = n_pages - 60 - np.arange(n * 8).reshape(n, 8)
    to_d, new_len = i32(to), torch.zeros(n, dtype=torch.int32, device=DEV)
    kept = torch.empty((n, 1000), dtype=torch.int32, device=DEV)
    ws = D.dsa_latent_cache_evict(D.evict_desc(n, 1000, 4, 64), cache, pages, weight, cache, D.paged_cache(to_d, new_len, n_pages),
                                  kept, None, new_len)
    assert D.dsa_workspace_status(ws) == 0
    j = SO.evict(weight[7].cpu().numpy(), lens[7], 1000, 4, 64)
    assert np.array_equal(kept[7].cpu().numpy(), j)
    i = np.arange(1000)
    dst = torch.as_tensor(to[7, i // P].astype(np.int64) * P + i % P, device=DEV)
    for a in arrays:
        assert torch.equal(a[dst].view(torch.uint8), a[phys[7][torch.as_tensor(j, device=DEV)]].view(torch.uint8))


class Steps:
    """Sequences that draft `d` tokens a step: the drafts' rows (and the last token's) go into the cache, are attended
    as rows of their own over the shared sequence, and are verified; what was refused is taken off the lengths."""

    def __init__(self, lens, d, H, V, fmt, seed):
        self.n, self.d, self.H, self.V = len(lens), d, H, V
        self.cols = 60                  # (so wide that the calls share)
        n, rows = self.n, self.n * (d + 1)
        self.n_pages = n * self.cols + 1
        self.arrays = _poisoned(self.n_pages, fmt)
        self.cache = D.latent_cache(*self.arrays)
        self.bt = np.random.default_rng(seed).permutation(self.n_pages)[:n * self.cols].reshape(n, self.cols).astype(np.int32)
        g = gen(seed)
        for t, L in enumerate(lens):
            _store(self.arrays, self.rows_of(t, np.arange(L)), randn((L, 576), g))
        self.len = i32(lens)
        self.seq = torch.arange(n, device=DEV).repeat_interleave(d + 1)
        self.place = torch.arange(d + 1, device=DEV).repeat(n)
        self.bt_d = i32(self.bt)
        self.bt_rows = self.bt_d[self.seq].contiguous()
        self.row_len = torch.zeros(rows, dtype=torch.int32, device=DEV)
        self.slot = torch.zeros(rows, dtype=torch.int32, device=DEV)
        self.start = i32(np.arange(n + 1) * (d + 1))
        self.kv = torch.zeros((rows, 576), dtype=torch.bfloat16, device=DEV)
        self.q = torch.zeros((rows, H, 576), dtype=torch.bfloat16, device=DEV)
        self.target = torch.zeros((n, d + 1, V), device=DEV)
        self.draft = torch.zeros((n, d, V), device=DEV)
        self.tokens = torch.zeros((n, d), dtype=torch.int32, device=DEV)
        self.u, self.us = torch.zeros((n, d), device=DEV), torch.zeros(n, device=DEV)
        self.out = torch.zeros((rows, H, 512), dtype=torch.bfloat16, device=DEV)
        self.lse = torch.zeros((rows, H), device=DEV)
        self.weight = torch.zeros((rows, self.cols * P), device=DEV)
        self.tokens_out = torch.zeros((n, d + 1), dtype=torch.int32, device=DEV)
        self.accepted = torch.zeros(n, dtype=torch.int32, device=DEV)
        self.pages = D.paged_cache(self.bt_rows, self.row_len, self.n_pages)
        self.desc = D.attn_desc(rows, self.n_pages * P, H, 0, TAU)
        self.groups = D.shared_rows(self.start, self.len, d + 1)
        size = max(D.dsa_latent_attn_shared_workspace_size(self.desc, self.groups), 256)
        self.ws = torch.empty(size, dtype=torch.uint8, device=DEV)

    def rows_of(self, t, j):
        return torch.as_tensor(self.bt[t, j // P].astype(np.int64) * P + j % P, device=DEV)

    def feed(self, seed):
        g = gen(seed)
        rand = lambda *s: torch.rand(s, generator=g, device=DEV)  # noqa: E731
        self.kv.copy_(randn(self.kv.shape, g))
        self.q.copy_(randn(self.q.shape, g))
        logits = 4.0 * torch.randn(self.target.shape, generator=g, device=DEV)
        self.target.copy_(torch.softmax(logits + 0.5 * torch.randn(logits.shape, generator=g, device=DEV), -1))
        self.draft.copy_(torch.softmax(logits[:, :self.d], -1))
        self.tokens.copy_(torch.multinomial(self.draft.reshape(-1, self.V), 1, generator=g).reshape(self.n, self.d))
        self.u.copy_(rand(self.n, self.d))
        self.us.copy_(rand(self.n))

    def step(self):
        j = self.len[self.seq] + self.place                      # the row's own key
        self.slot.copy_(torch.gather(self.bt_rows.long(), 1, (j // P).long()[:, None])[:, 0] * P + j % P)
        self.row_len.copy_(j + 1)
        D.dsa_latent_cache_write(D.cache_write_desc(self.kv), self.kv, self.slot, None, None, self.cache, ws=self.ws)
        D.dsa_latent_attn_shared(self.desc, self.q, self.cache, self.groups, self.pages, self.out, self.lse, ws=self.ws)
        D.dsa_latent_key_weights(self.desc, self.q, self.cache, self.pages, self.lse, self.weight, self.weight, ws=self.ws)
        D.dsa_mtp_verify(D.verify_desc(self.target, self.draft), self.target, self.draft, self.tokens, None, self.u, self.us,
                         self.tokens_out, self.accepted, ws=self.ws)
        self.len.add_(self.accepted + 1)

    def state(self):
        return [x.clone() for x in (self.len, self.out, self.lse, self.weight, self.tokens_out, self.accepted)]


@pytest.mark.parametrize("fmt,H", [("fp8", 16), ("bf16", 64), ("fp8", 100)])
def test_steps_of_drafting(fmt, H):
    lens, d, V = [2000, 130, 900, 1], 4, 5000
    a, b = Steps(lens, d, H, V, fmt, 1), Steps(lens, d, H, V, fmt, 1)
    graph = None
    moved = 0
    for step in range(4):
        before = a.len.clone()
        a.feed(100 + step)
        a.step()
        rows = [t for t in range(a.n * (d + 1)) if t % 7 == step % 7]
        kv = [_stored(a.arrays, a.rows_of(t // (d + 1), np.arange(int(a.row_len[t])))) if t in rows else None
              for t in range(a.n * (d + 1))]
        check_rows(a.out, a.lse, a.q, kv)
        for t in range(a.n):
            want, taken = SO.verify(a.target[t].cpu().numpy(), a.draft[t].cpu().numpy(), a.tokens[t].cpu().numpy(), None,
                                    a.u[t].cpu().numpy(), float(a.us[t]))
            assert int(a.accepted[t]) == taken and np.array_equal(a.tokens_out[t].cpu().numpy(), want)
            moved += taken
        assert torch.equal(a.len, before + a.accepted + 1)
        # the same steps captured once and replayed
        b.feed(100 + step)
        if graph is None:
            saved = [x.clone() for x in (b.len, b.weight, *b.arrays)]
            b.step()                               # (whatever the first call sets up)
            for x, y in zip((b.len, b.weight, *b.arrays), saved):
                x.copy_(y)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                b.step()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(a.state(), b.state()):
            assert torch.equal(x, y)
    assert moved > 0


@pytest.mark.parametrize("lens,shares", [([700, 300], False), ([700, 300, 5, 60, 900], True)])
def test_the_launch_log_names_the_calls(lens, shares):
    s = Steps(lens, 3, 16, 1000, "fp8", 3)
    s.feed(1)
    s.step()
    want = s.state()
    s.len.copy_(i32(lens))
    s.weight.zero_()
    D.dsa_profile_enable(True)
    try:
        s.step()
        kinds = [k for k, _ in D.dsa_profile_read()]
    finally:
        D.dsa_profile_enable(False)
    # (a small call shares nothing, and lists nothing)
    assert kinds == ["cache"] + ["attn_prep"] * shares + ["attn", "attn", "verify"]
    assert all(torch.equal(a, b) for a, b in zip(s.state(), want))


FIRST = """
import threading, torch
import dsa_indexer_cross_gb300 as D
dev = "cuda"
torch.manual_seed(0)
n, V, L, keep = 40, 40000, 40000, 300
t, q = torch.softmax(torch.randn(n, 3, V, device=dev), -1), torch.softmax(torch.randn(n, 2, V, device=dev), -1)
x = torch.randint(0, V, (n, 2), dtype=torch.int32, device=dev)
u, us = torch.rand(n, 2, device=dev), torch.rand(n, device=dev)
pages = (L + 127) // 128
rows = torch.randn(64 * 128, 576, device=dev).bfloat16()
bt = torch.randint(0, 8, (n, pages), dtype=torch.int32, device=dev)
lens = torch.randint(1000, L, (n,), dtype=torch.int32, device=dev)
w = torch.rand(n, pages * 128, device=dev)
def outs():
    dst = torch.zeros(n * 3 * 128, 576, device=dev).bfloat16()
    return dict(out=torch.zeros(n, 3, dtype=torch.int32, device=dev), acc=torch.zeros(n, dtype=torch.int32, device=dev),
                kept=torch.zeros(n, keep, dtype=torch.int32, device=dev), new=torch.zeros(n, dtype=torch.int32, device=dev), dst=dst,
                to=torch.arange(n * 3, dtype=torch.int32, device=dev).view(n, 3), ws=torch.zeros(512, dtype=torch.uint8, device=dev))
def run(o, stream=None):
    D.dsa_mtp_verify(D.verify_desc(t, q), t, q, x, None, u, us, o["out"], o["acc"], ws=o["ws"][:256], stream=stream)
    D.dsa_latent_cache_evict(D.evict_desc(n, keep, 4, 16), D.latent_cache(rows), D.paged_cache(bt, lens, 64), w, D.latent_cache(o["dst"]),
                             D.paged_cache(o["to"], o["new"], n * 3), o["kept"], None, o["new"], ws=o["ws"][256:], stream=stream)
def same(a, b):
    return all(torch.equal(a[k], b[k]) for k in ("out", "acc", "kept", "new", "dst"))
first, many = outs(), [outs() for _ in range(4)]
torch.cuda.synchronize()
"""


@pytest.mark.parametrize("how", [
    "g = torch.cuda.CUDAGraph()\nwith torch.cuda.graph(g):\n    run(first)\ng.replay()\n",
    "ts = [threading.Thread(target=lambda o=o: [run(o, torch.cuda.Stream()) for _ in range(20)]) for o in many]\n"
    "[x.start() for x in ts]\n[x.join() for x in ts]\ntorch.cuda.synchronize()\nrun(first)\nassert all(same(first, o) for o in many)\n"])
def test_a_process_first_calls(how):
    """What a call finds out about the device at its first use: while a graph is captured, and by four threads at once."""
    import subprocess
    import sys
    from pathlib import Path
    check = "torch.cuda.synchronize()\nagain = outs()\nrun(again)\nassert same(first, again) and int(again['new'].min()) == 300\nprint('same')\n"
    r = subprocess.run([sys.executable, "-c", FIRST + how + check], capture_output=True, text=True, timeout=300,
                       cwd=Path(__file__).resolve().parent.parent)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stderr[-2000:]
