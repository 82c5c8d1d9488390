"""Paged caches whose rows share prefixes, for the tests of shared-prefix attention."""
from __future__ import annotations

import numpy as np
import torch

import dsa_indexer_cross_gb300 as D
from latent_cases import DEV, P, TAU, encode, gen, i32, randn
from oracle import latent_oracle as LO


class SharedPaged:
    """groups: [(prefix, [length of each row], drafts)].  The rows of a group hold the same first prefix keys
    (as far as each is long): in common pages where a page lies whole in the prefix (drafts: in every page), in
    copies where it does not.  Every cache row that nobody uses is NaN, every table entry that nobody uses -7.
    wide: a table so wide that the call cannot know it for one of the small ones that share nothing."""

    def __init__(self, groups, fmt, seed=0, std=1.0, wide=True):
        g = gen(seed)
        self.fmt, self.lens, self.kv = fmt, [], []
        tables, pages = [], []              # pages: [contents [<= 128, 576]]
        self.start, self.prefix = [0], []
        for prefix, lens, drafts in groups:
            most = max(lens) if lens else 0
            common = randn((max(most if drafts else prefix, 0), 576), g, std)
            shared = {}
            for L in lens:
                if drafts or L <= prefix:
                    kv = common[:L]
                else:
                    kv = torch.cat([common, randn((L - prefix, 576), g, std)])
                self.kv.append(kv)
                self.lens.append(L)
                row = []
                for p in range((L + P - 1) // P):
                    whole = drafts or (p + 1) * P <= prefix
                    if whole and p in shared:
                        row.append(shared[p])
                        if len(kv[p * P:(p + 1) * P]) > len(pages[shared[p]]):
                            pages[shared[p]] = kv[p * P:(p + 1) * P]
                        continue
                    pages.append(kv[p * P:(p + 1) * P])
                    row.append(len(pages) - 1)
                    if whole:
                        shared[p] = len(pages) - 1
                tables.append(row)
            self.start.append(len(self.lens))
            self.prefix.append(prefix)
        self.n_pages = len(pages) + 3
        perm = np.random.default_rng(seed).permutation(self.n_pages)
        cols = max([1] + [len(r) for r in tables]) + 1
        if wide:
            cols = max(cols, 1001 // max(1, len(tables)) + 1)
        self.bt = np.full((len(tables), cols), -7, dtype=np.int32)
        for t, r in enumerate(tables):
            self.bt[t, :len(r)] = perm[r] if r else []
        n = self.n_pages * P
        if fmt == "bf16":
            self.rows = torch.full((n, 576), float("nan"), dtype=torch.bfloat16, device=DEV)
        else:
            self.codes = torch.full((n, 512), 0x7F, dtype=torch.uint8, device=DEV)
            self.scale = torch.full((n, 4), 255, dtype=torch.uint8, device=DEV)
            self.rope = torch.full((n, 64), float("nan"), dtype=torch.bfloat16, device=DEV)
        for k, x in enumerate(pages):
            a, b = int(perm[k]) * P, int(perm[k]) * P + len(x)
            if fmt == "bf16":
                self.rows[a:b] = x
            else:
                self.codes[a:b], self.scale[a:b] = encode(x[:, :512])
                self.rope[a:b] = x[:, 512:]
        self.cache = D.latent_cache(self.rows) if fmt == "bf16" else D.latent_cache(self.codes, self.scale, self.rope)
        self.bt_d, self.len_d = i32(self.bt), i32(self.lens)
        self.pages = D.paged_cache(self.bt_d, self.len_d, self.n_pages)
        self.start_d, self.prefix_d = i32(self.start), i32(self.prefix)
        self.max_rows = max(1, max((b - a for a, b in zip(self.start, self.start[1:])), default=1))

    def stored(self, t):
        """Row t's keys as the cache holds them, float64."""
        L = self.lens[t]
        j = np.arange(L)
        ph = torch.as_tensor(self.bt[t, j // P].astype(np.int64) * P + j % P, device=DEV)
        if self.fmt == "bf16":
            return self.rows[ph].double().cpu().numpy()
        y = LO.fp8_decode(self.codes[ph].cpu().numpy(), self.scale[ph].cpu().numpy())
        return np.concatenate([y, self.rope[ph].double().cpu().numpy()], axis=1)

    def attend(self, q, ws=None, tau=TAU, max_rows=None, start=None, prefix=None, lse=True, stream=None):
        n, H = q.shape[0], q.shape[1]
        desc = D.attn_desc(n, self.n_pages * P, H, 0, tau)
        groups = D.shared_rows(self.start_d if start is None else start, self.prefix_d if prefix is None else prefix,
                               max_rows or self.max_rows)
        out = torch.full((n, H, 512), 7.0, dtype=torch.bfloat16, device=DEV)
        ls = torch.full((n, H), 7.0, dtype=torch.float32, device=DEV) if lse else None
        ws = D.dsa_latent_attn_shared(desc, q, self.cache, groups, self.pages, out, ls, ws=ws, stream=stream)
        return out, ls, ws
