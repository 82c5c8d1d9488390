"""Shared helpers of the latent-cache GPU tests: paged caches with poisoned unused rows, and the
error bounds of the attention."""
from __future__ import annotations

import numpy as np
import torch

import dsa_indexer_cross_gb300 as D
from oracle import latent_oracle as LO

DEV = "cuda"
P = D.DSA_PAGE_ROWS
TAU = 1.0 / 24.0


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(shape, g, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(torch.bfloat16)


def i32(a):
    return torch.as_tensor(np.ascontiguousarray(a), dtype=torch.int32, device=DEV)


class Paged:
    """Sequences of the given lengths in shuffled pages.  Every cache row that no sequence uses --
    spare pages and the tails of last pages -- is NaN."""

    def __init__(self, lens, fmt, seed=0, std=1.0, spare=2, extra_cols=1, share=None):
        g = gen(seed)
        self.lens, self.fmt = list(lens), fmt
        need = [(L + P - 1) // P for L in lens]
        self.n_pages = max(1, sum(need)) + spare
        perm = np.random.default_rng(seed).permutation(self.n_pages)
        cols = max(1, max(need, default=1)) + extra_cols
        self.bt = np.full((len(lens), cols), -7, dtype=np.int32)      # never read past a sequence's pages
        k = 0
        for t, n in enumerate(need):
            self.bt[t, :n] = perm[k:k + n]
            k += n
        n_rows = self.n_pages * P
        self.kv = [randn((L, 576), g, std) for L in lens]             # what was stored, bf16
        used = torch.zeros(n_rows, dtype=torch.bool, device=DEV)
        self.phys = []
        for t, L in enumerate(lens):
            j = np.arange(L)
            ph = torch.as_tensor(self.bt[t, j // P].astype(np.int64) * P + j % P, device=DEV)
            self.phys.append(ph)
            used[ph] = True
        if fmt == "bf16":
            self.rows = torch.full((n_rows, 576), float("nan"), dtype=torch.bfloat16, device=DEV)
            for t in range(len(lens)):
                self.rows[self.phys[t]] = self.kv[t]
            self.cache = D.latent_cache(self.rows)
        else:
            self.codes = torch.full((n_rows, 512), 0x7F, dtype=torch.uint8, device=DEV)
            self.scale = torch.full((n_rows, 4), 255, dtype=torch.uint8, device=DEV)
            self.rope = torch.full((n_rows, 64), float("nan"), dtype=torch.bfloat16, device=DEV)
            for t in range(len(lens)):
                if lens[t] == 0:
                    continue
                c, s = encode(self.kv[t][:, :512])
                self.codes[self.phys[t]], self.scale[self.phys[t]] = c, s
                self.rope[self.phys[t]] = self.kv[t][:, 512:]
            self.cache = D.latent_cache(self.codes, self.scale, self.rope)
        self.bt_d, self.len_d = i32(self.bt), i32(self.lens)
        self.pages = D.paged_cache(self.bt_d, self.len_d, self.n_pages)

    def stored(self, t) -> np.ndarray:
        """Sequence t's rows as the cache holds them, float64."""
        if self.fmt == "bf16":
            return self.kv[t].double().cpu().numpy()
        ph = self.phys[t]
        y = LO.fp8_decode(self.codes[ph].cpu().numpy(), self.scale[ph].cpu().numpy())
        return np.concatenate([y, self.rope[ph].double().cpu().numpy()], axis=1)


def encode(x):
    """Codes and scale bytes of latent dims in torch (checked against the float64 definition in the
    cache-writing tests; used where a test needs a filled fp8 cache)."""
    v = x.float().reshape(-1, 4, 128)
    m, k = torch.frexp(v.abs().amax(dim=-1))
    e = (k - 9 + (m > 0.875).to(torch.int32)).clamp(-100, 7)
    inv = ((127 - e) << 23).view(torch.float32)
    c = (v * inv.unsqueeze(-1)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return c.view(torch.uint8).reshape(-1, 512), (e + 127).to(torch.uint8)


def attend(pc: Paged, q, idx=None, lse=True, ws=None, tau=TAU):
    n, H = q.shape[0], q.shape[1]
    desc = D.attn_desc(n, pc.n_pages * P, H, idx.shape[1] if idx is not None else 0, tau)
    out = torch.full((n, H, 512), 7.0, dtype=torch.bfloat16, device=DEV)
    ls = torch.full((n, H), 7.0, dtype=torch.float32, device=DEV) if lse else None
    ws = D.dsa_latent_attn_paged(desc, q, pc.cache, idx, pc.pages, out, ls, ws=ws)
    return out, ls, ws


def check_rows(out, lse, q, rows_kv, tau=TAU, heads=None):
    """Every element within the bound of its roundings.

    Half a bf16 step is u = 2^-8 of the value.  The weights are rounded once (u each) and divided by
    the sum of the rounded ones: an output moves by at most u (A + |o|) (1 + 2u), A = sum w |v|; its own
    rounding adds u |o|.  Scores are fp32 sums of 576 products: off by at most eps = 576 * 2^-23 * B,
    B = max_j tau sum |q kv| (the tensor core may truncate), plus 2^-21 of the score for the scaling and
    the exponential; each weight then moves by 2 eps, lse by eps.  2^-13 A covers fp32 sums over many
    tiles (an O of N / 64 products' sums, each off by 2^-23 of its terms)."""
    u = 2.0 ** -8
    q64 = q.double().cpu().numpy()
    o64 = out.double().cpu().numpy()
    l64 = lse.double().cpu().numpy() if lse is not None else None
    for t, kv in enumerate(rows_kv):
        if kv is None:
            continue
        o, l, A, B = LO.latent_attn_row(q64[t], kv, tau)
        if kv.shape[0] == 0:
            assert np.all(o64[t] == 0.0)
            if l64 is not None:
                assert np.all(l64[t] == -np.inf)
            continue
        eps = (576 * 2.0 ** -23 + 2.0 ** -20) * np.maximum(B, 1.0)[:, None]
        tol = u * np.abs(o) + (u * (1 + 2 * u) + 2 * eps + 2.0 ** -13) * (A + np.abs(o))
        bad = np.abs(o64[t] - o) > tol
        assert not bad.any(), (t, int(bad.sum()), float(np.nanmax(np.abs(o64[t] - o) / tol)))
        if l64 is not None:
            lt = eps[:, 0] + 2.0 ** -20 * np.maximum(1.0, np.abs(l))
            assert np.all(np.abs(l64[t] - l) <= lt), (t, float(np.max(np.abs(l64[t] - l) / lt)))


def check_exceptional(out, lse, q, rows_kv, tau=TAU):
    """As check_rows, where rows may hold infinities and NaN, and never passing a NaN that the formula does
    not give.  A head with a NaN or +inf score is NaN throughout.  A score of -inf weighs zero, so its row only
    shows in the dims where zero times its value is NaN; everywhere else the result is finite and within
    check_rows' bound over the other keys (without any: zeros, and a log-sum-exp of -inf)."""
    u = 2.0 ** -8
    q64, o64, l64 = q.double().cpu().numpy(), out.double().cpu().numpy(), lse.double().cpu().numpy()
    for t, kv in enumerate(rows_kv):
        with np.errstate(invalid="ignore"):
            s = tau * (q64[t] @ kv.T)
            nan_dims = np.isnan(kv[:, :512] * 0.0)
        for h in range(q.shape[1]):
            got, l = o64[t, h], l64[t, h]
            if np.any(np.isnan(s[h]) | (s[h] == np.inf)):
                assert np.all(np.isnan(got)) and np.isnan(l), (t, h)
                continue
            used = s[h] > -np.inf
            shown = nan_dims[~used].any(axis=0)
            assert np.array_equal(np.isnan(got), shown), (t, h)
            o, ref, A, B = (x[0] for x in LO.latent_attn_row(q64[t, h:h + 1], kv[used], tau))
            eps = (576 * 2.0 ** -23 + 2.0 ** -20) * max(B, 1.0)
            tol = u * np.abs(o) + (u * (1 + 2 * u) + 2 * eps + 2.0 ** -13) * (A + np.abs(o))
            assert np.all(np.abs(got - o)[~shown] <= tol[~shown]), (t, h)
            assert l == ref if not used.any() else abs(l - ref) <= eps + 2.0 ** -20 * max(1.0, abs(ref)), (t, h)
