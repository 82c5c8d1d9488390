"""More operators of decoding over the paged latent cache as workloads: latent attention of rows that
share a prefix, verification of drafted tokens, the attention weight that cached keys receive, and
eviction of the keys that received least.

Each case is one call of one operator on seeded inputs.  `run` computes it in elementary torch
operations where `own` is false and through this package's entry points where it is true.

Formats.  A latent row is 512 latent dims and 64 rotary dims.  A bf16 cache holds [rows][576]
bf16.  An fp8 cache holds e4m3 codes [rows][512], one scale byte b per 128 latent dims
[rows][4] (a code c stands for c * 2^(b - 127)) and the rotary dims as bf16 [rows][64].  Pages
hold 128 rows; logical key j of sequence t is cache row
block_table[t][j // 128] * 128 + j % 128.
"""
import math
import random

import torch

own = False

DEV = "cuda"
LAT, ROPE, ROW, PAGE = 512, 64, 576, 128
TAU = 1.0 / math.sqrt(576.0)


def _libdsa():
    import dsa_indexer_cross_gb300 as D
    return D


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # one conversation's drafted tokens, verified as rows of their own over the same cache: latency
        _shared("shared_drafts", 1, 4, 5000, 5000, 0, 0, 16, "bf16", True),
        # a batch of chats behind one system prompt, one GPU's share of the heads
        _shared("shared_prompt", 1, 48, 8000, 8000, 50, 1500, 16, "bf16", False),
        # a few documents, each asked several questions, all heads over an fp8 cache
        _shared("shared_documents", 4, 16, 16384, 32768, 100, 4000, 128, "fp8", False),
        # one long document, many short answers
        _shared("shared_long", 1, 32, 100000, 100000, 200, 2000, 64, "fp8", False),
        # one conversation's drafts against the target's probabilities: latency
        _verify("verify_one", 1, 3, 32000, "f32", True),
        # a batch of conversations, a large vocabulary
        _verify("verify_batch", 64, 4, 131072, "f32", True),
        # drafts without probabilities (looked up, or a greedy draft), bf16 probabilities, an odd vocabulary
        _verify("verify_lookup", 200, 7, 50257, "bf16", False),
        # the weights that a few short sequences' keys receive in one step: latency
        _weights("weights_short", 4, 1, 700, 16, "bf16"),
        # a batch of decodes over an fp8 cache
        _weights("weights_batch", 32, 1000, 33000, 64, "fp8"),
        # all heads, long sequences
        _weights("weights_all_heads", 16, 8192, 65536, 128, "fp8"),
        # two sequences cut to a small budget
        _evict("evict_few", 2, 3000, 5000, 1024, 4, 128, "bf16"),
        # a batch of long sequences, a quarter of the longest kept
        _evict("evict_long", 24, 8192, 65536, 16384, 64, 2048, "fp8"),
    ]


def _shared(name, groups, rows, lo, hi, tail_lo, tail_hi, heads, fmt, drafts):
    """groups of up to `rows` rows over prefixes of lo .. hi keys; drafts: a group's rows are positions of one
    sequence, else sequences of their own behind whole shared pages, with tails of tail_lo .. tail_hi keys."""
    return {"name": name, "op": "shared", "groups": groups, "rows": rows, "lo": lo, "hi": hi, "tail_lo": tail_lo,
            "tail_hi": tail_hi, "heads": heads, "fmt": fmt, "drafts": drafts}


def _verify(name, seqs, drafts, vocab, dtype, draft_probs):
    return {"name": name, "op": "verify", "seqs": seqs, "drafts": drafts, "vocab": vocab, "dtype": dtype,
            "draft_probs": draft_probs}


def _weights(name, seqs, lo, hi, heads, fmt):
    return {"name": name, "op": "weights", "seqs": seqs, "lo": lo, "hi": hi, "heads": heads, "fmt": fmt}


def _evict(name, seqs, lo, hi, keep, first, last, fmt):
    return {"name": name, "op": "evict", "seqs": seqs, "lo": lo, "hi": hi, "keep": keep, "first": first, "last": last,
            "fmt": fmt}


def draw(rng):
    log = lambda a, b: int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))  # noqa: E731
    kind = rng.choice(["shared", "shared", "verify", "weights", "evict"])
    fmt = rng.choice(["bf16", "fp8"])
    if kind == "shared":
        heads = rng.choice([1, 3, 8, 16, 24, 32, 64, 100, 128])
        groups = rng.choice([1, 1, 2, 5])
        drafts = rng.random() < 0.4
        rows = rng.randint(2, 8) if drafts else log(2, 48 // groups)
        hi = log(130, min(100000, 200000000 // (groups * rows * heads)))
        lo = max(1, hi // rng.choice([1, 2, 8]))
        tail = log(1, 4000)
        c = _shared("", groups, rows, lo, hi, max(0, tail // rng.choice([1, 4, 5000])), tail, heads, fmt, drafts)
    elif kind == "verify":
        vocab, drafts = log(1000, 131072), rng.randint(1, 8)
        c = _verify("", log(1, 256 if vocab < 50000 else 64), drafts, vocab, rng.choice(["f32", "f32", "bf16"]),
                    rng.random() < 0.75)
    elif kind == "weights":
        n = log(1, 48)
        hi = log(2, min(65536, 700000 // n))
        c = _weights("", n, max(1, hi // rng.choice([1, 2, 8, 64])), hi, rng.choice([1, 3, 8, 16, 32, 40, 64, 100, 128]), fmt)
    else:
        n = log(1, 48)
        hi = log(2, min(65536, 700000 // n))
        keep = max(1, int(hi * rng.choice([0.1, 0.25, 0.5, 0.9])))
        first = min(keep, rng.choice([0, 1, 4, 64]))
        c = _evict("", n, max(1, hi // rng.choice([1, 2, 8])), hi, keep, first, (keep - first) // rng.choice([1, 4, 16]), fmt)
    del c["name"]
    return c


def _lengths(case):
    """The sequences' lengths: part of the case, not of its data."""
    n = case["seqs"]
    r = random.Random(n * 1000003 + case["lo"] * 7919 + case["hi"])
    return [r.randint(case["lo"], case["hi"]) for _ in range(n)]


def _groups(case):
    """[(prefix, [length of each row])] of a shared case."""
    r = random.Random(case["groups"] * 1000003 + case["rows"] * 7919 + case["hi"])
    out = []
    for _ in range(case["groups"]):
        n = case["rows"] if case["groups"] == 1 else r.randint(max(1, case["rows"] // 2), case["rows"])
        p = r.randint(case["lo"], case["hi"])
        if case["drafts"]:
            out.append((p, [p + 1 + i for i in range(n)]))
        else:
            p = max(1, p // PAGE) * PAGE
            out.append((p, [p + r.randint(case["tail_lo"], case["tail_hi"]) for _ in range(n)]))
    return out


def _row_bytes(case):
    return ROW * 2 if case["fmt"] == "bf16" else LAT + 4 + ROPE * 2


def work(case):
    if case["op"] == "shared":
        groups = _groups(case)
        rows = sum(len(ls) for _, ls in groups)
        once = sum(max(ls) if case["drafts"] else p + sum(L - p for L in ls) for p, ls in groups)
        keys = sum(sum(ls) for _, ls in groups)
        return {"bytes": once * _row_bytes(case) + 4 * once // PAGE + rows * case["heads"] * (ROW * 2 + LAT * 2 + 4),
                "flops": 2 * keys * case["heads"] * (ROW + LAT)}
    if case["op"] == "verify":
        # the row a token is drawn from, and (after a rejection, in some two of three sequences) the draft's
        el = 4 if case["dtype"] == "f32" else 2
        rows = 1.0 + (0.65 if case["draft_probs"] else 0.0)
        return {"bytes": int(case["seqs"] * (rows * case["vocab"] * el + case["drafts"] * (2 * el + 12) + 12)),
                "flops": int(case["seqs"] * (rows + 1) * case["vocab"])}
    lens = _lengths(case)
    keys = sum(lens)
    if case["op"] == "weights":
        return {"bytes": keys * (_row_bytes(case) + 8) + 4 * keys // PAGE + case["seqs"] * case["heads"] * (ROW * 2 + 4),
                "flops": keys * case["heads"] * (2 * ROW + 3)}
    kept = sum(min(L, case["keep"]) for L in lens)
    return {"bytes": 4 * keys + kept * (2 * _row_bytes(case) + 8) + 4 * kept // PAGE, "flops": keys}


# ------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _pow2(e):
    """2^e in fp32 for integers e in [-126, 127], by its bits."""
    return ((e + 127) << 23).view(torch.float32)


def _encode(x):
    """Latent dims [n][512] (fp32) -> e4m3 codes as bytes, scale bytes."""
    g = x.reshape(-1, 4, 128)
    m, k = torch.frexp(g.abs().amax(dim=-1))
    e = (k - 9 + (m > 0.875).to(torch.int32)).clamp(-100, 7)
    c = (g * _pow2(-e).unsqueeze(-1)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return c.view(torch.uint8).reshape(-1, LAT), (e + 127).to(torch.uint8)


def _cache(n_rows, fmt, g):
    """A cache whose rows hold latents like a trained model's: per-row magnitudes that vary."""
    if fmt == "bf16":
        rows = torch.empty((n_rows, ROW), dtype=torch.bfloat16, device=DEV)
    else:
        codes = torch.empty((n_rows, LAT), dtype=torch.uint8, device=DEV)
        scale = torch.empty((n_rows, 4), dtype=torch.uint8, device=DEV)
        rope = torch.empty((n_rows, ROPE), dtype=torch.bfloat16, device=DEV)
    step = 1 << 19
    for a in range(0, n_rows, step):
        b = min(n_rows, a + step)
        x = torch.randn((b - a, ROW), generator=g, device=DEV)
        x *= torch.rand((b - a, 1), generator=g, device=DEV) + 0.5
        x = x.to(torch.bfloat16)
        if fmt == "bf16":
            rows[a:b] = x
        else:
            codes[a:b], scale[a:b] = _encode(x[:, :LAT].float())
            rope[a:b] = x[:, LAT:]
    return {"rows": rows} if fmt == "bf16" else {"codes": codes, "scale": scale, "rope": rope}


def _empty_cache(n_rows, fmt):
    z = lambda w, dt: torch.zeros((n_rows, w), dtype=dt, device=DEV)  # noqa: E731
    if fmt == "bf16":
        return {"rows": z(ROW, torch.bfloat16)}
    return {"codes": z(LAT, torch.uint8), "scale": z(4, torch.uint8), "rope": z(ROPE, torch.bfloat16)}


def _pages(lens, g, spare=3):
    """A shuffled block table over the lengths' pages; -1 past a sequence's last page."""
    need = torch.tensor([(L + PAGE - 1) // PAGE for L in lens], device=DEV)
    total, most = int(need.sum()), max(1, int(need.max()))
    perm = torch.randperm(total + spare, generator=g, device=DEV).to(torch.int32)
    col = torch.arange(most, device=DEV)
    used = col < need[:, None]
    table = torch.full((len(lens), most), -1, dtype=torch.int32, device=DEV)
    table[used] = perm[:total]
    return table.contiguous(), total + spare


def _shared_pages(case, groups, g):
    """Block table of rows whose groups share the prefixes' whole pages (drafts: every page)."""
    owner, cols = [], 0
    for p, lens in groups:
        most = max((L + PAGE - 1) // PAGE for L in lens)
        cols = max(cols, most)
        owner.append((most if case["drafts"] else p // PAGE, [(L + PAGE - 1) // PAGE for L in lens]))
    table, at = [], 0
    for share, need in owner:
        common = list(range(at, at + share))
        at += share
        for n in need:
            mine = common[:n] + list(range(at, at + max(0, n - share)))
            at += max(0, n - share)
            table.append(mine + [-1] * (cols - n))
    perm = torch.randperm(at + 3, generator=g, device=DEV).to(torch.int32)
    t = torch.tensor(table, dtype=torch.int64, device=DEV)
    return torch.where(t >= 0, perm[t.clamp(min=0)], -1).to(torch.int32).contiguous(), at + 3


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    if case["op"] == "verify":
        _prepare_verify(s, g)
    elif case["op"] == "shared":
        groups = _groups(case)
        s["bt"], s["n_pages"] = _shared_pages(case, groups, g)
        lens = [L for _, ls in groups for L in ls]
        starts = [0]
        for _, ls in groups:
            starts.append(starts[-1] + len(ls))
        s["plan_groups"] = groups
        s["len"], s["start"], s["prefix"] = i32(lens), i32(starts), i32([p for p, _ in groups])
        s.update(_cache(s["n_pages"] * PAGE, case["fmt"], g))
        n, h = len(lens), case["heads"]
        s["seqs"] = n
        s["q"] = torch.randn((n, h, ROW), generator=g, device=DEV).to(torch.bfloat16)
        s["out"] = torch.empty((n, h, LAT), dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty((n, h), dtype=torch.float32, device=DEV)
    else:
        lens = _lengths(case)
        n = len(lens)
        s["lens"] = lens
        s["bt"], s["n_pages"] = _pages(lens, g)
        s["len"] = i32(lens)
        s.update(_cache(s["n_pages"] * PAGE, case["fmt"], g))
        width = s["bt"].shape[1] * PAGE
        # what the keys have received so far: a few receive most; one in ten has received nothing
        s["w_in"] = torch.exp(2.0 * torch.randn((n, width), generator=g, device=DEV)) \
            * (torch.rand((n, width), generator=g, device=DEV) > 0.1)
        if case["op"] == "weights":
            s["q"] = torch.randn((n, case["heads"], ROW), generator=g, device=DEV).to(torch.bfloat16)
            s["w_out"] = torch.zeros((n, width), device=DEV)
            # the log-sum-exp that the attention of the same rows returned
            s["lse"] = torch.stack([_lse(torch.matmul(s["q"][t].float(), _rows_of(s, _phys(s, t, L)).T) * TAU)
                                    for t, L in enumerate(lens)])
        else:
            kept = [min(L, case["keep"]) for L in lens]
            s["kept_n"] = kept
            table, n_to = _pages(kept, g)
            s["to_bt"], s["to_pages"] = table, n_to
            s["to"] = _empty_cache(n_to * PAGE, case["fmt"])
            s["kept"] = torch.zeros((n, case["keep"]), dtype=torch.int32, device=DEV)
            s["to_len"] = torch.zeros(n, dtype=torch.int32, device=DEV)
            s["w_out"] = torch.zeros((n, table.shape[1] * PAGE), device=DEV)
    if own:
        s["plan"] = _plan(s)
    return s


def _prepare_verify(s, g):
    """Draft and target distributions that mostly agree, tokens drawn from the draft's, uniform numbers."""
    n, d, v = s["seqs"], s["drafts"], s["vocab"]
    dt = torch.float32 if s["dtype"] == "f32" else torch.bfloat16
    logits = 6.0 * torch.randn((n, d + 1, v), generator=g, device=DEV)
    q = torch.softmax(logits, dim=-1)
    s["target"] = torch.softmax(logits + 0.5 * torch.randn((n, d + 1, v), generator=g, device=DEV), dim=-1).to(dt)
    del logits
    q = q[:, :d].to(dt).contiguous()
    if s["draft_probs"]:
        s["draft"] = q
        s["tokens"] = torch.multinomial(q.float().reshape(n * d, v), 1, generator=g).reshape(n, d).to(torch.int32)
    else:
        s["draft"] = None
        s["tokens"] = torch.multinomial(s["target"][:, :d].float().reshape(n * d, v).pow(1.5), 1,
                                        generator=g).reshape(n, d).to(torch.int32)
    # a sequence in four drafted fewer tokens than the others
    short = torch.rand(n, generator=g, device=DEV) < 0.25
    s["draft_len"] = torch.where(short, torch.randint(0, d + 1, (n,), generator=g, device=DEV), d).to(torch.int32)
    s["u_accept"] = torch.rand((n, d), generator=g, device=DEV)
    s["u_sample"] = torch.rand(n, generator=g, device=DEV)
    s["out_tokens"] = torch.zeros((n, d + 1), dtype=torch.int32, device=DEV)
    s["accepted"] = torch.zeros(n, dtype=torch.int32, device=DEV)


def _handle(D, c):
    return D.latent_cache(c["codes"], c["scale"], c["rope"]) if "codes" in c else D.latent_cache(c["rows"])


def _plan(s):
    """What a program keeps between its calls: descriptors, cache handles, a workspace."""
    D = _libdsa()
    if s["op"] == "verify":
        return D.verify_desc(s["target"], s["draft"]), torch.empty(256, dtype=torch.uint8, device=DEV)
    cache = _handle(D, s)
    pages = D.paged_cache(s["bt"], s["len"], s["n_pages"])
    if s["op"] == "evict":
        desc = D.evict_desc(s["seqs"], s["keep"], s["first"], s["last"])
        ws = torch.empty(D.dsa_latent_cache_evict_workspace_size(desc), dtype=torch.uint8, device=DEV)
        return desc, cache, pages, _handle(D, s["to"]), D.paged_cache(s["to_bt"], s["to_len"], s["to_pages"]), ws
    desc = D.attn_desc(s["seqs"], s["n_pages"] * PAGE, s["heads"], 0, TAU)
    if s["op"] == "shared":
        groups = D.shared_rows(s["start"], s["prefix"], max(len(lens) for _, lens in s["plan_groups"]))
        ws = torch.empty(D.dsa_latent_attn_shared_workspace_size(desc, groups), dtype=torch.uint8, device=DEV)
        return desc, cache, groups, pages, ws
    ws = torch.empty(D.dsa_latent_key_weights_workspace_size(desc, pages), dtype=torch.uint8, device=DEV)
    return desc, cache, pages, ws


# ------------------------------------------------------------------------------- one pass

def run(state):
    return {"shared": _run_shared, "verify": _run_verify, "weights": _run_weights, "evict": _run_evict}[state["op"]](state)


def _phys(s, t, n, a=0):
    """Cache rows of keys a .. n - 1 of sequence t."""
    j = torch.arange(a, n, device=DEV)
    return s["bt"][t].long()[j // PAGE] * PAGE + j % PAGE


def _rows_of(s, phys):
    """Cache rows `phys` as fp32 [..., 576]."""
    if s["fmt"] == "bf16":
        return s["rows"][phys].float()
    c = s["codes"].view(torch.float8_e4m3fn)[phys].float().reshape(*phys.shape, 4, 128)
    c = c * _pow2(s["scale"][phys].to(torch.int32) - 127).unsqueeze(-1)
    return torch.cat([c.reshape(*phys.shape, LAT), s["rope"][phys].float()], dim=-1)


def _lse(x):
    m = x.amax(dim=-1)
    return m + torch.log(torch.exp(x - m[..., None]).sum(dim=-1))


def _run_shared(s):
    if own:
        desc, cache, groups, pages, ws = s["plan"]
        _libdsa().dsa_latent_attn_shared(desc, s["q"], cache, groups, pages, s["out"], s["lse"], ws=ws)
        return s["out"], s["lse"]
    h, at = s["heads"], 0
    for prefix, lens in s["plan_groups"]:
        n = len(lens)
        q = s["q"][at:at + n].float().reshape(n * h, ROW)
        # the prefix once for all rows, then the rows' own keys, padded to the longest tail
        kv = _rows_of(s, _phys(s, at, prefix))
        x = torch.matmul(q, kv.T) * TAU
        tail = max(lens) - prefix
        if tail:
            j = prefix + torch.arange(tail, device=DEV).expand(n, -1)
            valid = j < s["len"][at:at + n, None]
            page = torch.gather(s["bt"][at:at + n].long(), 1, j // PAGE)
            kt = _rows_of(s, torch.where(valid, page * PAGE + j % PAGE, 0))
            y = torch.matmul(q.reshape(n, h, ROW), kt.transpose(1, 2)) * TAU
            y = y.masked_fill(~valid[:, None], -math.inf).reshape(n * h, tail)
            m = torch.maximum(x.amax(dim=1), y.amax(dim=1))
        else:
            m = x.amax(dim=1)
        p = torch.exp(x - m[:, None])
        total, o = p.sum(dim=1), torch.matmul(p, kv[:, :LAT])
        if tail:
            r = torch.exp(y - m[:, None])
            total = total + r.sum(dim=1)
            o = o + torch.matmul(r.reshape(n, h, tail), kt[..., :LAT]).reshape(n * h, LAT)
        s["out"][at:at + n] = (o / total[:, None]).reshape(n, h, LAT).to(torch.bfloat16)
        s["lse"][at:at + n] = (m + torch.log(total)).reshape(n, h)
        at += n
    return s["out"], s["lse"]


def _run_verify(s):
    if own:
        desc, ws = s["plan"]
        _libdsa().dsa_mtp_verify(desc, s["target"], s["draft"], s["tokens"], s["draft_len"], s["u_accept"],
                                 s["u_sample"], s["out_tokens"], s["accepted"], ws=ws)
        return s["out_tokens"], s["accepted"]
    n, d, v = s["seqs"], s["drafts"], s["vocab"]
    tok = s["tokens"].long()
    row, col = torch.arange(n, device=DEV), torch.arange(d, device=DEV)
    p_tok = s["target"][:, :d].gather(2, tok[..., None])[..., 0].double()
    q_tok = s["draft"].gather(2, tok[..., None])[..., 0].double() if s["draft"] is not None else torch.ones_like(p_tok)
    # the first draft that is not taken ends the run
    taken = (s["u_accept"].double() * q_tok < p_tok) & (col < s["draft_len"][:, None])
    a = taken.long().cumprod(dim=1).sum(dim=1)
    rejected = a < s["draft_len"]
    r = s["target"][row, a].double()
    ai = a.clamp(max=d - 1)
    if s["draft"] is not None:
        less = r - s["draft"][row, ai].double()
    else:
        less = torch.where(torch.arange(v, device=DEV) == tok[row, ai][:, None], 0.0, r)
    r = torch.where(rejected[:, None], less.clamp(min=0.0), r)
    c = torch.cumsum(r, dim=1)
    drawn = (c <= s["u_sample"].double()[:, None] * c[:, -1:]).sum(dim=1)
    out = torch.full_like(s["out_tokens"], -1)
    out[:, :d] = torch.where(col < a[:, None], s["tokens"], -1)
    out[row, a] = drawn.to(torch.int32)
    return out, a.to(torch.int32)


def _run_weights(s):
    if own:
        desc, cache, pages, ws = s["plan"]
        _libdsa().dsa_latent_key_weights(desc, s["q"], cache, pages, s["lse"], s["w_in"], s["w_out"], ws=ws)
        return s["w_out"]
    for t, L in enumerate(s["lens"]):
        x = torch.matmul(s["q"][t].float(), _rows_of(s, _phys(s, t, L)).T) * TAU
        s["w_out"][t, :L] = s["w_in"][t, :L] + torch.exp(x - s["lse"][t][:, None]).sum(dim=0)
    return s["w_out"]


def _evict_out(s):
    to = s["to"]
    arrays = (to["rows"],) if "rows" in to else (to["codes"].view(torch.float8_e4m3fn), to["scale"], to["rope"])
    return (*arrays, s["w_out"], s["kept"], s["to_len"])


def _run_evict(s):
    if own:
        desc, cache, pages, to, to_pages, ws = s["plan"]
        _libdsa().dsa_latent_cache_evict(desc, cache, pages, s["w_in"], to, to_pages, s["kept"], s["w_out"], s["to_len"],
                                         ws=ws)
        return _evict_out(s)
    keep, first, last = s["keep"], s["first"], s["last"]
    for t, L in enumerate(s["lens"]):
        n = min(L, keep)
        j = torch.arange(L, device=DEV)
        if L > keep:
            order = torch.sort(s["w_in"][t, first:L - last], descending=True, stable=True).indices
            middle = torch.sort(order[:keep - first - last]).values + first
            j = torch.cat([j[:first], middle, j[L - last:]])
        src = s["bt"][t].long()[j // PAGE] * PAGE + j % PAGE
        i = torch.arange(n, device=DEV)
        dst = s["to_bt"][t].long()[i // PAGE] * PAGE + i % PAGE
        for k, a in s["to"].items():
            a[dst] = s[k][src]
        s["w_out"][t, :n] = s["w_in"][t][j]
        s["kept"][t] = -1
        s["kept"][t, :n] = j.to(torch.int32)
        s["to_len"][t] = n
    return _evict_out(s)


# ------------------------------------------------------------------------------- in 64 bits

def _two64(e):
    """2^e in 64 bits for integers e, by its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _row64(s, phys):
    if s["fmt"] == "bf16":
        return s["rows"][phys].double()
    c = s["codes"][phys].view(torch.float8_e4m3fn).double()
    f = _two64(s["scale"][phys].long() - 127)
    return torch.cat([c * f.repeat_interleave(128, dim=-1), s["rope"][phys].double()], dim=-1)


def _all_rows(s, t, L):
    pages = s["bt"][t, :(L + PAGE - 1) // PAGE].long()
    return (pages[:, None] * PAGE + torch.arange(PAGE, device=DEV)).flatten()[:L]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "verify":
        return _exact_verify(s)
    if case["op"] == "shared":
        # every row by itself, over all of its keys
        outs, sums = [], []
        for t, L in enumerate(L for _, ls in s["plan_groups"] for L in ls):
            kv = _row64(s, _all_rows(s, t, L))
            score = (kv @ s["q"][t].double().T) * TAU
            top = score.amax(0)
            weight = torch.exp(score - top)
            total = weight.sum(0)
            outs.append((weight / total).T @ kv[:, :LAT])
            sums.append(top + torch.log(total))
        return torch.stack(outs), torch.stack(sums)
    if case["op"] == "weights":
        out = s["w_out"].double()
        for t, L in enumerate(s["lens"]):
            score = (_row64(s, _all_rows(s, t, L)) @ s["q"][t].double().T) * TAU
            out[t, :L] = s["w_in"][t, :L].double() + torch.exp(score - s["lse"][t].double()).sum(1)
        return out
    return _exact_evict(s)


def _exact_verify(s):
    """One sequence after the other, as the method is told."""
    n, d, v = s["seqs"], s["drafts"], s["vocab"]
    out = torch.full((n, d + 1), -1, dtype=torch.int32)
    accepted = torch.zeros(n, dtype=torch.int32)
    tokens, u, last, own_u = s["tokens"].tolist(), s["u_accept"].tolist(), s["draft_len"].tolist(), s["u_sample"].tolist()
    at = s["tokens"].long()[..., None]
    pt = s["target"][:, :d].gather(2, at)[..., 0].tolist()
    qt = s["draft"].gather(2, at)[..., 0].tolist() if s["draft"] is not None else None
    for t in range(n):
        i = 0
        while i < last[t] and u[t][i] * (qt[t][i] if qt else 1.0) < pt[t][i]:
            out[t, i] = tokens[t][i]
            i += 1
        accepted[t] = i
        r = s["target"][t, i].double()
        if i < last[t]:
            if s["draft"] is not None:
                r = torch.relu(r - s["draft"][t, i].double())
            else:
                r[tokens[t][i]] = 0.0
        c = torch.cumsum(r, 0)
        out[t, i] = int(torch.searchsorted(c, torch.tensor([own_u[t]], dtype=torch.float64, device=DEV) * c[-1],
                                           right=True))
    return out.to(DEV), accepted.to(DEV)


def _exact_evict(s):
    """Which keys stay, by rank: a key's rank is the number of keys that weigh more, or as much at a lower place."""
    arrays = {k: a.view(torch.float8_e4m3fn).double() if k == "codes" else a.long() if k == "scale" else a.double()
              for k, a in s["to"].items()}
    source = {k: s[k].view(torch.float8_e4m3fn) if k == "codes" else s[k] for k in arrays}
    w_out, kept, size = s["w_out"].double(), torch.full_like(s["kept"], -1), torch.zeros_like(s["to_len"])
    for t, L in enumerate(s["lens"]):
        stays = torch.ones(L, dtype=torch.bool, device=DEV)
        a, b, room = s["first"], L - s["last"], s["keep"] - s["first"] - s["last"]
        if L > s["keep"]:
            w = s["w_in"][t, a:b]
            values = torch.unique(w)                      # ascending
            more = w.numel() - torch.searchsorted(torch.sort(w).values, values, right=True)
            limit = values[more <= room].min() if bool((more <= room).any()) and room > 0 else math.inf
            inside = w > limit
            ties = w == limit
            inside |= ties & (torch.cumsum(ties.long(), 0) <= room - int(inside.sum()))
            stays[a:b] = inside
        j = torch.nonzero(stays).flatten()
        n = j.numel()
        src = _all_rows(s, t, L)[j]
        dst = (s["to_bt"][t].long()[:, None] * PAGE + torch.arange(PAGE, device=DEV)).flatten()[:n]
        for k in arrays:
            arrays[k][dst] = source[k][src].to(arrays[k].dtype)
        w_out[t, :n] = s["w_in"][t][j].double()
        kept[t, :n] = j.to(torch.int32)
        size[t] = n
    return (*arrays.values(), w_out, kept, size)
