"""The latent cache's operators as workloads: rotary positions, writing the paged latent cache
(bf16 or fp8), reading it back, and latent attention over it (every key, or selected keys).

Each case is one call of one operator on seeded inputs.  `run` computes it in elementary torch
operations where `own` is false and through this package's entry points where it is true.

Formats.  A latent row is 512 latent dims and 64 rotary dims.  A bf16 cache holds [rows][576]
bf16.  An fp8 cache holds e4m3 codes [rows][512], one scale byte b per 128 latent dims
[rows][4] (a code c stands for c * 2^(b - 127)) and the rotary dims as bf16 [rows][64].  The
scale exponent is the smallest integer e with amax <= 448 * 2^e, kept within [-100, 7].  Pages
hold 128 rows; logical key j of sequence t is cache row
block_table[t][j // 128] * 128 + j % 128.
"""
import math
import random

import torch

own = False

DEV = "cuda"
LAT, ROPE, ROW, PAGE = 512, 64, 576, 128
THETA = 8e6
TAU = 1.0 / math.sqrt(576.0)


def _libdsa():
    import dsa_indexer_cross_gb300 as D
    return D


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step: the rotary part of 64 tokens' queries moves from the projection's output
        # (128 + 64 dims a head) into the absorbed query (512 + 64 dims a head)
        _rope("rope_decode", 64, 128, 192, 576, "bf16", True, False),
        # the same for a prefill chunk, in the rotate-half layout
        _rope("rope_prefill", 8000, 64, 192, 576, "bf16", False, False),
        # training: the gradient of the rotation, fp32 gradients of the absorbed query
        _rope("rope_backward", 4096, 16, 576, 192, "f32", False, True),
        # one decode step's new rows, rotated and quantised into their pages
        _write("write_decode", 64, "fp8", True),
        # a long prefill's rows
        _write("write_prefill", 32768, "fp8", False),
        # the cached prefixes of a few conversations, brought back for their next prefill chunk
        _read("read_prefixes", 7, 100, 4000, "fp8"),
        # long contexts read back
        _read("read_long", 16, 8192, 131072, "fp8"),
        # one short chat on one GPU's share of the heads: latency
        _attn("attn_short", 1, 300, 300, 16, "bf16", 0),
        # a batch of decodes over a bf16 cache, 16 heads
        _attn("attn_batch16", 48, 1000, 33000, 16, "bf16", 0),
        # long decodes with all heads over an fp8 cache
        _attn("attn_long128", 64, 8192, 131072, 128, "fp8", 0),
        # selected keys of long decodes over an fp8 cache
        _attn("select_long", 64, 8192, 131072, 128, "fp8", 2048),
        # a small batch, few selected keys
        _attn("select_small", 5, 700, 5000, 64, "fp8", 256),
    ]


def _rope(name, tokens, heads, width_in, width_out, dtype, interleaved, inverse):
    return {"name": name, "op": "rope", "tokens": tokens, "heads": heads, "width_in": width_in,
            "width_out": width_out, "dtype": dtype, "interleaved": interleaved, "inverse": inverse}


def _write(name, tokens, fmt, interleaved):
    return {"name": name, "op": "write", "tokens": tokens, "fmt": fmt, "interleaved": interleaved}


def _read(name, seqs, lo, hi, fmt):
    return {"name": name, "op": "read", "seqs": seqs, "lo": lo, "hi": hi, "fmt": fmt}


def _attn(name, seqs, lo, hi, heads, fmt, topk):
    return {"name": name, "op": "attn", "seqs": seqs, "lo": lo, "hi": hi, "heads": heads, "fmt": fmt, "topk": topk}


def draw(rng):
    log = lambda a, b: int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))  # noqa: E731
    kind = rng.choice(["rope", "write", "read", "attn", "attn", "select"])
    if kind == "rope":
        heads = rng.choice([1, 2, 4, 16, 40, 64, 128])
        w = rng.choice([(192, 576), (576, 192), (64, 64)])
        c = _rope("", log(1, 500000 // heads), heads, w[0], w[1], rng.choice(["bf16", "bf16", "f32"]),
                  rng.random() < 0.5, rng.random() < 0.4)
    elif kind == "write":
        c = _write("", log(1, 60000), rng.choice(["fp8", "fp8", "bf16"]), rng.random() < 0.5)
    elif kind == "read":
        n = log(1, 48)
        hi = log(2, min(131072, 1000000 // n))
        c = _read("", n, max(1, hi // rng.choice([1, 2, 8])), hi, rng.choice(["fp8", "fp8", "bf16"]))
    else:
        heads = rng.choice([1, 3, 8, 16, 24, 32, 64, 100, 128])
        n = log(1, 64)
        hi = log(2, min(131072, 2500000 // n))
        lo = max(1, hi // rng.choice([1, 2, 8, 64]))
        if kind == "attn":
            c = _attn("", n, lo, hi, heads, rng.choice(["fp8", "bf16"]), 0)
        else:
            c = _attn("", n, lo, hi, heads, "fp8", rng.choice([1, 33, 256, 777, 1024, 2048]))
    del c["name"]
    return c


def _lengths(case):
    """The sequences' lengths: part of the case, not of its data."""
    n = case["seqs"]
    r = random.Random(n * 1000003 + case["lo"] * 7919 + case["hi"])
    return [r.randint(case["lo"], case["hi"]) for _ in range(n)]


def work(case):
    if case["op"] == "rope":
        el = 2 if case["dtype"] == "bf16" else 4
        n = case["tokens"] * case["heads"] * ROPE
        return {"bytes": 2 * n * el + case["tokens"] * (4 + ROPE * 4), "flops": 3 * n}
    if case["op"] == "write":
        out = ROW * 2 if case["fmt"] == "bf16" else LAT + 4 + ROPE * 2
        return {"bytes": case["tokens"] * (ROW * 2 + out + 8 + ROPE * 4), "flops": case["tokens"] * (2 * LAT + 3 * ROPE)}
    row = ROW * 2 if case["fmt"] == "bf16" else LAT + 4 + ROPE * 2
    lens = _lengths(case)
    if case["op"] == "read":
        n = sum(lens)
        return {"bytes": n * (row + ROW * 2) + 4 * n // PAGE, "flops": n * LAT}
    keys = sum(min(case["topk"], L) if case["topk"] else L for L in lens)
    q = case["seqs"] * case["heads"]
    index = 4 * keys if case["topk"] else 4 * keys // PAGE
    return {"bytes": keys * row + index + q * (ROW * 2 + LAT * 2 + 4), "flops": 2 * keys * case["heads"] * (ROW + LAT)}


# ------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _table(n_pos):
    """(cos, sin) of every position, evaluated in 64 bits and kept in 32."""
    f = THETA ** (-torch.arange(0, ROPE, 2, device=DEV, dtype=torch.float64) / ROPE)
    a = torch.arange(n_pos, device=DEV, dtype=torch.float64)[:, None] * f
    return torch.stack([a.cos(), a.sin()], dim=-1).float().contiguous()


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


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "rope":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        n, h = case["tokens"], case["heads"]
        n_pos = 131072
        s["table"] = _table(n_pos)
        if n <= 256:      # decoding: every token is another sequence's
            pos = torch.randint(0, n_pos, (n,), generator=g, device=DEV)
        else:             # a run of one sequence
            pos = (torch.arange(n, device=DEV) + torch.randint(0, n_pos, (1,), generator=g, device=DEV)) % n_pos
        s["pos"] = pos.to(torch.int32)
        s["src"] = torch.randn((n, h, case["width_in"]), generator=g, device=DEV).to(dt)
        s["dst"] = torch.randn((n, h, case["width_out"]), generator=g, device=DEV).to(dt)
    elif case["op"] == "write":
        n = case["tokens"]
        n_pages = (n + PAGE - 1) // PAGE + 2
        s["table"] = _table(131072)
        s["pos"] = torch.randint(0, 131072, (n,), generator=g, device=DEV).to(torch.int32)
        s["kv"] = (torch.randn((n, ROW), generator=g, device=DEV)
                   * (torch.rand((n, 1), generator=g, device=DEV) + 0.5)).to(torch.bfloat16)
        s["slot"] = torch.randperm(n_pages * PAGE, generator=g, device=DEV)[:n].to(torch.int32)
        if n > 3:
            s["slot"][n // 3] = -1      # a padded token: not stored
        s.update(_cache(n_pages * PAGE, case["fmt"], g))
        s["n_pages"] = n_pages
    else:
        lens = _lengths(case)
        s["bt"], s["n_pages"] = _pages(lens, g)
        s["len"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s.update(_cache(s["n_pages"] * PAGE, case["fmt"], g))
        n = len(lens)
        if case["op"] == "read":
            starts = [0]
            for L in lens[:-1]:
                starts.append(starts[-1] + L)
            s["start"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
            s["total"] = sum(lens)
            s["out"] = torch.zeros((s["total"], ROW), dtype=torch.bfloat16, device=DEV)
        else:
            s["q"] = torch.randn((n, case["heads"], ROW), generator=g, device=DEV).to(torch.bfloat16)
            s["out"] = torch.empty((n, case["heads"], LAT), dtype=torch.bfloat16, device=DEV)
            s["lse"] = torch.empty((n, case["heads"]), dtype=torch.float32, device=DEV)
            s["idx"] = None
            if case["topk"]:
                k = case["topk"]
                idx = torch.full((n, k), -1, dtype=torch.int32, device=DEV)
                for t, L in enumerate(lens):
                    m = min(k, L)
                    idx[t, :m] = torch.randperm(L, generator=g, device=DEV)[:m].sort().values.to(torch.int32)
                s["idx"] = idx
    if own:
        s["plan"] = _plan(s)
    return s


def _plan(s):
    """What a program keeps between its calls: descriptors, cache handles, a workspace."""
    D = _libdsa()
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    flags = D.DSA_ROPE_INTERLEAVED if s.get("interleaved") else 0
    if s["op"] == "rope":
        x, out = s["src"][..., -ROPE:], s["dst"][..., -ROPE:]
        return D.rope_desc(x, out, flags | (D.DSA_ROPE_INVERSE if s["inverse"] else 0)), x, out, ws
    cache = D.latent_cache(s["rows"]) if s["fmt"] == "bf16" else D.latent_cache(s["codes"], s["scale"], s["rope"])
    if s["op"] == "write":
        return D.cache_write_desc(s["kv"], flags | D.DSA_CACHE_ROPE), cache, ws
    pages = D.paged_cache(s["bt"], s["len"], s["n_pages"])
    if s["op"] == "read":
        return cache, pages, ws
    desc = D.attn_desc(s["seqs"], s["n_pages"] * PAGE, s["heads"], s["topk"], TAU)
    ws = torch.empty(D.dsa_latent_attn_workspace_size(desc), dtype=torch.uint8, device=DEV)
    return desc, cache, pages, ws


# ------------------------------------------------------------------------------- one pass

def run(state):
    return {"rope": _run_rope, "write": _run_write, "read": _run_read, "attn": _run_attn}[state["op"]](state)


def _rotate(x, cs, interleaved, inverse):
    """x [..., 64] rotated by cs [..., 32, 2], in the type of x."""
    c, s = cs[..., 0], cs[..., 1]
    if inverse:
        s = -s
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :ROPE // 2], x[..., ROPE // 2:])
    u, v = a * c - b * s, a * s + b * c
    return torch.stack([u, v], dim=-1).flatten(-2) if interleaved else torch.cat([u, v], dim=-1)


def _run_rope(s):
    if own:
        desc, x, out, ws = s["plan"]
        _libdsa().dsa_rope_apply(desc, x, s["pos"], s["table"], out, ws=ws)
        return s["dst"]
    y = _rotate(s["src"][..., -ROPE:].float(), s["table"][s["pos"].long()][:, None], s["interleaved"], s["inverse"])
    s["dst"][..., -ROPE:] = y.to(s["dst"].dtype)
    return s["dst"]


def _cache_out(s):
    """The cache as numbers: e4m3 codes, their scale bytes, the rotary dims."""
    return s["rows"] if s["fmt"] == "bf16" else (s["codes"].view(torch.float8_e4m3fn), s["scale"], s["rope"])


def _run_write(s):
    if own:
        desc, cache, ws = s["plan"]
        _libdsa().dsa_latent_cache_write(desc, s["kv"], s["slot"], s["pos"], s["table"], cache, ws=ws)
        return _cache_out(s)
    # a token without a slot stores token 0's row once more (token 0 always has a slot here)
    src = torch.where(s["slot"] >= 0, torch.arange(s["slot"].shape[0], device=DEV), 0)
    slot = s["slot"][src].long()
    x = s["kv"][src].float()
    r = _rotate(x[:, LAT:], s["table"][s["pos"][src].long()], s["interleaved"], False).to(torch.bfloat16)
    if s["fmt"] == "bf16":
        s["rows"][slot] = torch.cat([x[:, :LAT].to(torch.bfloat16), r], dim=1)
    else:
        s["codes"][slot], s["scale"][slot] = _encode(x[:, :LAT])
        s["rope"][slot] = r
    return _cache_out(s)


def _rows_of(s, phys):
    """Cache rows `phys` (any shape) as fp32 [..., 576]."""
    if s["fmt"] == "bf16":
        return s["rows"][phys].float()
    c = s["codes"].view(torch.float8_e4m3fn)[phys].float().reshape(*phys.shape, 4, 128)
    c = c * _pow2(s["scale"][phys].to(torch.int32) - 127).unsqueeze(-1)
    return torch.cat([c.reshape(*phys.shape, LAT), s["rope"][phys].float()], dim=-1)


def _run_read(s):
    if own:
        cache, pages, ws = s["plan"]
        _libdsa().dsa_latent_cache_read(cache, pages, s["len"].shape[0], s["start"], s["out"], ws=ws)
        return s["out"]
    seq = torch.repeat_interleave(torch.arange(s["len"].shape[0], device=DEV), s["len"], output_size=s["total"])
    j = torch.arange(s["total"], device=DEV) - s["start"].long()[seq]
    s["out"][:] = _rows_of(s, s["bt"].long()[seq, j // PAGE] * PAGE + j % PAGE).to(torch.bfloat16)
    return s["out"]


def _run_attn(s):
    if own:
        desc, cache, pages, ws = s["plan"]
        _libdsa().dsa_latent_attn_paged(desc, s["q"], cache, s["idx"], pages, s["out"], s["lse"], ws=ws)
        return s["out"], s["lse"]
    n = s["len"].shape[0]
    if s["idx"] is None:
        j = torch.arange(s["bt"].shape[1] * PAGE, device=DEV).expand(n, -1)
    else:
        j = s["idx"].long()
    valid = (j >= 0) & (j < s["len"][:, None])
    j = torch.where(valid, j, 0)
    kv = _rows_of(s, torch.gather(s["bt"].long(), 1, j // PAGE) * PAGE + j % PAGE)
    x = torch.matmul(s["q"].float(), kv.transpose(1, 2)) * TAU
    x = x.masked_fill(~valid[:, None], -math.inf)
    lse = torch.logsumexp(x, dim=-1)
    p = torch.exp(x - lse[..., None])
    return torch.matmul(p, kv[..., :LAT]).to(torch.bfloat16), lse


# ------------------------------------------------------------------------------- in 64 bits

def _turn64(x, table, pos, interleaved, inverse):
    """The rotation as a product of complex numbers."""
    cs = table.double()[pos.long()]
    w = torch.complex(cs[..., 0], -cs[..., 1] if inverse else cs[..., 1])
    x = x.double()
    z = torch.view_as_complex(x.unflatten(-1, (-1, 2)).contiguous()) if interleaved else torch.complex(*x.chunk(2, -1))
    z = z * (w[:, None] if x.dim() == 3 else w)
    return torch.view_as_real(z).flatten(-2) if interleaved else torch.cat([z.real, z.imag], -1)


def _two64(e):
    """2^e in 64 bits for integers e, by its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _codes64(x):
    """Nearest e4m3 values (ties to even) and scale bytes of latent dims, by the format's steps."""
    x = x.double().reshape(-1, 4, 128)
    top = x.abs().amax(-1)
    e = torch.full(top.shape, -100, dtype=torch.int64, device=DEV)
    for k in range(-100, 7):
        e += (top > 448.0 * 2.0 ** k).long()
    y = x / _two64(e).unsqueeze(-1)
    step = _two64(torch.frexp(y.abs().clamp(min=2.0 ** -6)).exponent - 4)      # 2^-3 of the power of two below
    return (torch.round(y / step) * step).clamp(-448.0, 448.0).reshape(-1, LAT), e + 127


def _row64(s, phys):
    if s["fmt"] == "bf16":
        return s["rows"][phys].double()
    c = s["codes"][phys].view(torch.float8_e4m3fn).double()
    f = _two64(s["scale"][phys].long() - 127)
    return torch.cat([c * f.repeat_interleave(128, dim=-1), s["rope"][phys].double()], dim=-1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        y = s["dst"].double()
        y[..., -ROPE:] = _turn64(s["src"][..., -ROPE:], s["table"], s["pos"], case["interleaved"], case["inverse"])
        return y
    if case["op"] == "write":
        at = torch.nonzero(s["slot"] >= 0).flatten()
        slot = s["slot"][at].long()
        turned = _turn64(s["kv"][at][:, LAT:], s["table"], s["pos"][at], case["interleaved"], False)
        if case["fmt"] == "bf16":
            y = s["rows"].double()
            y[slot] = torch.cat([s["kv"][at][:, :LAT].double(), turned], 1)
            return y
        y, b, r = s["codes"].view(torch.float8_e4m3fn).double(), s["scale"].long(), s["rope"].double()
        y[slot], b[slot] = _codes64(s["kv"][at][:, :LAT])
        r[slot] = turned
        return y, b, r
    lens = _lengths(case)
    parts, sums = [], []
    for t, L in enumerate(lens):
        pages = s["bt"][t, :(L + PAGE - 1) // PAGE].long()
        phys = (pages[:, None] * PAGE + torch.arange(PAGE, device=DEV)).flatten()[:L]
        if case["op"] == "read":
            parts.append(_row64(s, phys))
            continue
        if case["topk"]:
            chosen = s["idx"][t]
            phys = phys[chosen[chosen >= 0].long()]
        kv = _row64(s, phys)
        score = (kv @ s["q"][t].double().T) * TAU
        top = score.amax(0)
        weight = torch.exp(score - top)
        total = weight.sum(0)
        parts.append((weight / total).T @ kv[:, :LAT])
        sums.append(top + torch.log(total))
    if case["op"] == "read":
        return torch.cat(parts)
    return torch.stack(parts), torch.stack(sums)
