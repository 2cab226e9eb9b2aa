"""The serving operators around the paged compressed cache, as measured cases.

Each case is one call that a serving loop makes: rotary positions on a step's
queries and keys, storing a chunk of coded keys in the pages, attention of a
chunk over the paged codes, accumulating attention weights per cached key, and
evicting the keys that gathered the least.  ``run`` computes them with
elementary torch operations where ``own`` is false, and with the library's
entry points where it is true; ``exact`` states them once more in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


def listed():
    return [
        # positions of one decode step of the 8-sequence GQA batch: pure latency
        dict(name="rotary decode step", op="rotary", n=8, Hq=32, Hkv=8, d=128, rot=128,
             dtype="bf16", interleaved=False, scaling="", inverse=False, far=32768),
        # a long prompt with interleaved pairs on half of each head and
        # frequencies stretched for a context beyond the trained one
        dict(name="rotary long prompt", op="rotary", n=16384, Hq=32, Hkv=8, d=128, rot=64,
             dtype="bf16", interleaved=True, scaling="banded", inverse=False, far=1048576),
        # the gradient of the rotation (its inverse) at an odd token count
        dict(name="rotary gradient fp32", op="rotary", n=1025, Hq=12, Hkv=3, d=64, rot=64,
             dtype="f32", interleaved=False, scaling="linear", inverse=True, far=131072),
        # a few drafted tokens of each of 8 sequences entering the cache
        dict(name="store drafted tokens", op="store", B=8, n=8, Hkv=8, d=128, W=8, c=1, P=64,
             T=32768, ragged=True),
        # a 16384-token prompt of TurboQuant-prod codes (2-bit cells) entering the cache
        dict(name="store long prompt", op="store", B=1, n=16384, Hkv=8, d=128, W=12, c=2, P=64,
             T=16384, ragged=False),
        # drafted tokens verified against the GQA batch's caches (2 to 8 tokens each)
        dict(name="chunk verify", op="chunk", B=8, n=8, Hq=32, Hkv=8, d=128, m=256, P=64,
             T=32768, dtype="bf16", ragged=True),
        # a prompt's next 2048 tokens over a 32768-token cache
        dict(name="chunk prefill", op="chunk", B=1, n=2048, Hq=32, Hkv=8, d=128, m=256, P=64,
             T=32768, dtype="bf16", ragged=False),
        # ragged chunks of odd lengths, one head per KV head, d = 64, fp32 queries
        dict(name="chunk ragged d64", op="chunk", B=5, n=333, Hq=6, Hkv=6, d=64, m=128, P=32,
             T=4099, dtype="f32", ragged=True),
        # weights of one decode step of the GQA batch
        dict(name="weights gqa", op="mass", B=8, Hq=32, Hkv=8, T=32768, decay=1.0, ragged=True),
        # weights of one long sequence with a head per KV head, older weight fading
        dict(name="weights long", op="mass", B=1, Hq=32, Hkv=32, T=131072, decay=0.97,
             ragged=False),
        # halving the GQA batch's caches
        dict(name="evict gqa", op="evict", B=8, Hkv=8, d=128, W=8, c=1, P=64, T=32768,
             keep=16384, recent=256, sink=4, ragged=True),
        # a small cache kept at 256 keys
        dict(name="evict small", op="evict", B=2, Hkv=4, d=64, W=4, c=1, P=32, T=1000,
             keep=256, recent=32, sink=4, ragged=True),
    ]


def _log(rng, lo, hi):
    """A whole number spread evenly over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "store", "chunk", "chunk", "mass", "evict"])
    if op == "rotary":
        d = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 3, 8])
        Hq = Hkv * rng.choice([1, 2, 4])
        return dict(op=op, n=_log(rng, 1, 16384), Hq=Hq, Hkv=Hkv, d=d,
                    rot=rng.choice([d, d // 2, d // 4, 20]), dtype=rng.choice(["bf16", "f32"]),
                    interleaved=rng.random() < 0.5,
                    scaling=rng.choice(["", "linear", "ntk", "banded"]),
                    inverse=rng.random() < 0.3, far=_log(rng, 64, 1048576))
    if op == "store":
        B, Hkv = _log(rng, 1, 16), rng.choice([1, 2, 5, 8])
        n = _log(rng, 1, max(1, 16384 // B))
        return dict(op=op, B=B, n=n, Hkv=Hkv, d=rng.choice([64, 128]),
                    W=rng.choice([2, 4, 6, 8, 12, 16]), c=rng.choice([1, 2]),
                    P=rng.choice([32, 64, 96, 128]), T=n + _log(rng, 1, 16384), ragged=rng.random() < 0.7)
    if op == "chunk":
        B, Hkv, G = _log(rng, 1, 8), rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 8])
        T = _log(rng, 1, 32768)
        most = 2048 * 32768 * 32 // (B * Hkv * G * T)
        return dict(op=op, B=B, n=_log(rng, 1, max(1, min(2048, T, most))), Hq=Hkv * G, Hkv=Hkv,
                    d=rng.choice([64, 128]), m=rng.choice([64, 128, 256, 512]),
                    P=rng.choice([32, 64, 96, 128]), T=T, dtype=rng.choice(["bf16", "f32"]),
                    ragged=rng.random() < 0.7)
    if op == "mass":
        Hkv, G = rng.choice([1, 4, 8]), rng.choice([1, 2, 3, 4, 8])
        B = _log(rng, 1, 8)
        return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv,
                    T=_log(rng, 1, 131072 * 32 // max(32, B * Hkv * G)),
                    decay=rng.choice([1.0, 0.9, 0.0]), ragged=rng.random() < 0.7)
    B, Hkv = _log(rng, 1, 8), rng.choice([1, 2, 5, 8])
    T = _log(rng, 2, 32768)
    keep = _log(rng, 1, max(1, T // 2))
    recent = rng.randint(0, keep // 2)
    return dict(op="evict", B=B, Hkv=Hkv, d=rng.choice([64, 128]), W=rng.choice([2, 4, 8, 12]),
                c=rng.choice([1, 2]), P=rng.choice([32, 64, 96, 128]), T=T, keep=keep,
                recent=recent, sink=rng.randint(0, min(8, keep - recent)),
                ragged=rng.random() < 0.7)


# ---------------------------------------------------------------------------
# inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _sequences(c, rng=None):
    """Cached keys and new tokens of each sequence: all T and all n, or spread
    over [T/2, T] and [n/4, n] with one of them the most.  A case has the same
    ones whatever the seed, which (`rng`) only puts them in another order."""
    fixed = np.random.default_rng(c["T"])
    B, T, n = c["B"], c["T"], c.get("n", 1)
    L, k = np.full(B, T), np.full(B, n)
    if c["ragged"]:
        L = fixed.integers(max(1, T // 2), T + 1, size=B)
        k = fixed.integers(max(1, n // 4), n + 1, size=B)
        L[0], k[-1] = T, n
    k = np.minimum(k, L)
    order = np.arange(B) if rng is None else rng.permutation(B)
    return L[order], k[order]


def _table(rng, lens, P, width, first, total):
    """Block table of sequences of `lens` keys in a shuffled pool of `total`
    pages, from place `first` of the pool's order on; -1 where unused."""
    perm = np.random.default_rng(total).permutation(total)
    tab = np.full((len(lens), width), -1, dtype=np.int32)
    k = first
    for b, L in enumerate(lens):
        p = -(-int(L) // P)
        tab[b, :p] = perm[k:k + p]
        k += p
    return tab


def _dev(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(device=DEV, dtype=dtype)


def _pack(bits):
    """[..., m] 0/1 -> [..., m/32] int32 words, least significant bit first."""
    w = bits.view(*bits.shape[:-1], -1, 32).to(torch.int64)
    w = (w << torch.arange(32, device=bits.device)).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


def _words(g, *shape):
    return torch.randint(-2 ** 31, 2 ** 31, shape, generator=g, device=DEV).to(torch.int32)


def frequencies(rot, scaling, base=10000.0, factor=8.0, original_len=8192, low=1.0, high=4.0):
    """Rotary frequencies base^(-2j/rot), plain or scaled for long contexts:
    "linear" divides all by `factor`; "ntk" raises the base so that the lowest
    one is divided by it; "banded" leaves the ones that turn more than `high`
    times in `original_len` positions, divides those that turn less than `low`
    times, and blends the ones between."""
    j = np.arange(rot // 2, dtype=np.float64)
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2.0))
    f = base ** (-2.0 * j / rot)
    if scaling == "linear":
        f = f / factor
    elif scaling == "banded":
        turns = original_len * f / (2 * math.pi)
        keep = np.clip((turns - low) / (high - low), 0.0, 1.0)
        f = f * (keep + (1 - keep) / factor)
    return f.astype(np.float32)


def _prepare_rotary(c, g, rng):
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    # one projection's output holds a token's queries, keys and values, so
    # queries and keys are strided views of it
    qkv = _randn(g, c["n"], c["Hq"] + 2 * c["Hkv"], c["d"]).to(dt)
    start = int(rng.integers(0, c["far"]))
    pos = start + np.arange(c["n"]) if c["n"] > 64 else rng.integers(0, c["far"], size=c["n"])
    return dict(Q=qkv[:, :c["Hq"]], K=qkv[:, c["Hq"]:c["Hq"] + c["Hkv"]], positions=_dev(pos),
                inv_freq=_dev(frequencies(c["rot"], c["scaling"]), torch.float32),
                scale=1.2 if c["scaling"] == "banded" else 1.0)


def _prepare_store(c, g, rng):
    Hkv, P = c["Hkv"], c["P"]
    total, k = _sequences(c, rng)                          # total: lengths after the call
    width = -(-c["T"] // P)
    pages = int(sum(-(-int(x) // P) for x in total)) + 3
    N = int(k.sum()) + (3 if c["ragged"] else 0)           # a padded batch: 3 rows of no sequence
    lead = (pages, Hkv, P)
    one = () if c["c"] == 1 else (2,)
    qkv = _randn(g, N, 2 * Hkv, c["d"]).to(torch.bfloat16)
    return dict(codes=_words(g, N, Hkv, c["W"]), norms=_randn(g, N, Hkv, *one).abs().half(),
                V=qkv[:, Hkv:], cu=_dev(np.concatenate([[0], np.cumsum(k)])),
                code_pages=_words(g, *lead, c["W"]),
                norm_pages=_randn(g, *lead, *one).abs().half(),
                value_pages=_randn(g, *lead, c["d"]).to(torch.bfloat16),
                table=_dev(_table(rng, total, P, width, 0, pages)), lens=_dev(total - k))


def _prepare_chunk(c, g, rng):
    Hkv, P, d, m = c["Hkv"], c["P"], c["d"], c["m"]
    L, k = _sequences(c, rng)
    pages = int(sum(-(-int(x) // P) for x in L)) + 2
    S = _randn(g, m, d).to(torch.bfloat16)
    # keys with four outlier channels, coded page by page as the quantizer does
    keys = _randn(g, pages * Hkv * P, d)
    keys[:, torch.randperm(d, generator=g, device=DEV)[:4]] *= 10.0
    keys = keys.to(torch.bfloat16).float()
    signs = torch.cat([_pack(x @ S.float().T >= 0) for x in keys.split(1 << 19)])
    N = int(k.sum()) + (3 if c["ragged"] else 0)           # a padded batch: 3 rows of no sequence
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    return dict(Q=_randn(g, N, c["Hq"], d).to(dt), S=S,
                sign_pages=signs.view(pages, Hkv, P, m // 32),
                norm_pages=keys.norm(dim=-1).half().view(pages, Hkv, P),
                value_pages=_randn(g, pages, Hkv, P, d).to(torch.bfloat16),
                table=_dev(_table(rng, L, P, -(-c["T"] // P), 0, pages)), lens=_dev(L),
                cu=_dev(np.concatenate([[0], np.cumsum(k)])), max_len=c["T"], longest=int(k.max()),
                out=torch.zeros((N, c["Hq"], d), device=DEV, dtype=torch.bfloat16))


def _prepare_mass(c, g, rng):
    L, _ = _sequences(c, rng)
    # estimator scores of N(0, 1) queries against keys with outlier channels
    scores = _randn(g, c["B"], c["Hq"], c["T"]) * 30.0
    mass = _randn(g, c["B"], c["Hkv"], c["T"]).square() * 1e-3
    return dict(scores=scores, mass=mass, lens=_dev(L), softmax_scale=128 ** -0.5,
                out=torch.zeros_like(mass))


def _prepare_evict(c, g, rng):
    B, Hkv, P = c["B"], c["Hkv"], c["P"]
    L, _ = _sequences(c, rng)
    new = np.minimum(L, c["keep"])
    src = int(sum(-(-int(x) // P) for x in L))
    pages = src + int(sum(-(-int(x) // P) for x in new)) + 1
    mass = torch.exp(_randn(g, B, Hkv, c["T"]) * 3.0 - 6.0)
    mass[mass < 5e-4] = 0.0                                # weights that underflowed: many ties
    lead = (pages, Hkv, P)
    one = () if c["c"] == 1 else (2,)
    return dict(mass=mass, lens=_dev(L), keep=c["keep"], recent=c["recent"], sink=c["sink"],
                code_pages=_words(g, *lead, c["W"]),
                norm_pages=_randn(g, *lead, *one).abs().half(),
                value_pages=_randn(g, *lead, c["d"]).to(torch.bfloat16),
                src=_dev(_table(rng, L, P, -(-c["T"] // P), 0, pages)),
                dst=_dev(_table(rng, new, P, -(-c["keep"] // P), src, pages)))


def prepare(case, seed):
    made = {"rotary": _prepare_rotary, "store": _prepare_store, "chunk": _prepare_chunk,
            "mass": _prepare_mass, "evict": _prepare_evict}[case["op"]]
    return dict(made(case, _gen(seed), np.random.default_rng(int(seed))), case=dict(case))


# ---------------------------------------------------------------------------
# plain forms

def _rotate(x, cos, sin, interleaved, out):
    """The first 2 * cos.shape[-1] entries of each head turned by their angles."""
    r = 2 * cos.shape[-1]
    y = x.float()
    if interleaved:
        a, b = y[..., 0:r:2], y[..., 1:r:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = y[..., :r // 2], y[..., r // 2:r]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([turned.to(out), x[..., r:].to(out)], -1)


def _plain_rotary(s):
    c = s["case"]
    angle = s["positions"].double()[:, None, None] * s["inv_freq"].double()
    cos = (angle.cos() * s["scale"]).float()
    sin = (angle.sin() * (-s["scale"] if c["inverse"] else s["scale"])).float()
    return (_rotate(s["Q"], cos, sin, c["interleaved"], s["Q"].dtype),
            _rotate(s["K"], cos, sin, c["interleaved"], s["K"].dtype))


def _token_slots(cu, lens, table, N, P):
    """(page, slot) of each live token row of a chunk, and those rows."""
    rows = torch.arange(N, device=cu.device)
    b = torch.searchsorted(cu[1:].contiguous(), rows, right=True)
    rows = rows[b < lens.numel()]
    b = b[b < lens.numel()]
    pos = lens[b].long() + rows - cu[b].long()
    return table[b, pos // P].long(), pos % P, rows


def _plain_store(s):
    page, slot, rows = _token_slots(s["cu"].long(), s["lens"], s["table"], s["codes"].shape[0],
                                    s["case"]["P"])
    s["code_pages"][page, :, slot] = s["codes"][rows]
    s["norm_pages"][page, :, slot] = s["norms"][rows]
    s["value_pages"][page, :, slot] = s["V"][rows]


def _signs(words, dtype):
    """[..., W] words -> [..., 32 W] entries +1 / -1."""
    bits = (words[..., None] >> torch.arange(32, device=words.device)) & 1
    return (bits.flatten(-2) * 2 - 1).to(dtype)


def _plain_chunk(s):
    c = s["case"]
    B, Hq, Hkv, d, m, P = c["B"], c["Hq"], c["Hkv"], c["d"], c["m"], c["P"]
    T, n, G = s["max_len"], s["longest"], c["Hq"] // c["Hkv"]
    cu, lens = s["cu"].long(), s["lens"].long()
    count = cu[1:] - cu[:-1]
    # the cache in order: [B, Hkv, T, ...]
    t = torch.arange(T, device=DEV)
    page = s["table"][:, t // P].long().clamp(min=0)
    z = _signs(s["sign_pages"][page, :, t % P], torch.float32).transpose(1, 2)
    norm = s["norm_pages"][page, :, t % P].float().transpose(1, 2)
    V = s["value_pages"][page, :, t % P].float().transpose(1, 2)
    # the chunk's queries in order: [B, Hkv, n * G, d]
    i = torch.arange(n, device=DEV)
    row = (cu[:-1, None] + i).clamp(max=s["Q"].shape[0] - 1)
    Q = s["Q"][row].float().view(B, n, Hkv, G, d).transpose(1, 2).reshape(B, Hkv, n * G, d)
    U = Q @ s["S"].float().T
    logit = U @ z.transpose(-1, -2)
    logit = logit * (norm * (math.sqrt(math.pi / 2) / m * d ** -0.5))[:, :, None]
    seen = (lens - count)[:, None] + i + 1                 # keys that token i sees
    dark = (t >= seen[..., None]) | (t >= lens[:, None, None])
    dark = dark[:, None, :, None].expand(B, 1, n, G, T).reshape(B, 1, n * G, T)
    logit = logit.masked_fill(dark, -math.inf)
    top = logit.amax(-1, keepdim=True)
    w = torch.exp(logit - top.masked_fill(top == -math.inf, 0.0))
    total = w.sum(-1, keepdim=True)
    o = (w @ V) / total.masked_fill(total == 0, 1.0)
    o = o.view(B, Hkv, n, G, d).transpose(1, 2).reshape(B, n, Hq, d).to(torch.bfloat16)
    live = i < count[:, None]
    s["out"][row[live]] = o[live]
    return s["out"]


def _plain_mass(s):
    c = s["case"]
    B, Hkv, T = s["mass"].shape
    live = torch.arange(T, device=DEV) < s["lens"].long()[:, None, None]
    x = (s["scores"] * s["softmax_scale"]).masked_fill(~live, -math.inf)
    w = torch.exp(x - x.amax(-1, keepdim=True))
    w = w / w.sum(-1, keepdim=True)
    new = s["mass"] * c["decay"] + w.view(B, Hkv, -1, T).sum(2)
    s["out"].copy_(torch.where(live, new, s["out"]))
    return s["out"]


def _plain_evict(s):
    c = s["case"]
    P, keep = c["P"], s["keep"]
    B, Hkv, T = s["mass"].shape
    lens = s["lens"].long()
    t = torch.arange(T, device=DEV)
    live = t < lens[:, None]
    held = live & ((t < s["sink"]) | (t >= lens[:, None] - s["recent"]))
    rank = torch.where(held[:, None], math.inf, s["mass"]).masked_fill(~live[:, None], -math.inf)
    order = torch.sort(rank, dim=-1, descending=True, stable=True)[1][..., :keep]
    order = torch.where(order < lens[:, None, None], order, T).sort(dim=-1)[0]
    if order.shape[-1] < keep:
        order = torch.nn.functional.pad(order, (0, keep - order.shape[-1]), value=T)
    there = order < T
    at = order.clamp(max=T - 1)
    mass = torch.where(there, s["mass"].gather(-1, at), 0.0)
    b, h, j = there.nonzero(as_tuple=True)
    old = order[b, h, j]
    src, dst = s["src"][b, old // P].long(), s["dst"][b, j // P].long()
    for pool in (s["code_pages"], s["norm_pages"], s["value_pages"]):
        pool[dst, h, j % P] = pool[src, h, old % P]
    return torch.where(there, order, -1).to(torch.int32), mass, lens.clamp(max=keep).to(torch.int32)


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        import bit_jl_key_b200 as jl
    if op == "rotary":
        if own:
            return jl.jl_rotary(s["Q"], s["positions"], s["inv_freq"], K=s["K"],
                                interleaved=c["interleaved"], inverse=c["inverse"],
                                scale=s["scale"])
        return _plain_rotary(s)
    if op == "store":
        if own:
            jl.jl_store_paged(s["codes"], s["norms"], s["V"], s["cu"], s["code_pages"],
                              s["norm_pages"], s["value_pages"], s["table"], s["lens"])
        else:
            _plain_store(s)
        return s["code_pages"], s["norm_pages"], s["value_pages"]
    if op == "chunk":
        if own:
            return jl.jl_chunk_attention_paged(
                s["Q"], s["S"], s["sign_pages"], s["norm_pages"], s["value_pages"], s["table"],
                s["lens"], s["cu"], s["max_len"], out=s["out"])
        return _plain_chunk(s)
    if op == "mass":
        if own:
            return jl.jl_accumulate_attention(s["scores"], s["mass"], s["lens"],
                                              s["softmax_scale"], decay=c["decay"], out=s["out"])
        return _plain_mass(s)
    if own:
        kept = jl.jl_evict_paged(s["mass"], s["lens"], s["keep"], s["code_pages"],
                                 s["norm_pages"], s["value_pages"], s["src"], s["dst"],
                                 recent=s["recent"], sink=s["sink"])
    else:
        kept = _plain_evict(s)
    return (*kept, s["code_pages"], s["norm_pages"], s["value_pages"])


# ---------------------------------------------------------------------------
# what a pass cannot do without

def work(c):
    op = c["op"]
    if op == "rotary":
        each = 2 if c["dtype"] == "bf16" else 4
        x = c["n"] * (c["Hq"] + c["Hkv"])
        return dict(bytes=2.0 * x * c["d"] * each + 4 * c["n"], flops=3.0 * x * c["rot"])
    L, k = _sequences(c)
    if op == "mass":
        L = float(L.sum())
        read = 1 if c["decay"] == 0 else 2
        return dict(bytes=4.0 * L * (c["Hq"] + read * c["Hkv"]), flops=5.0 * L * c["Hq"])
    if op == "evict":
        row = 4 * c["W"] + 2 * c["c"] + 2 * c["d"]
        kept = float(np.minimum(L, c["keep"]).sum()) * c["Hkv"]
        return dict(bytes=4.0 * float(L.sum()) * c["Hkv"] + kept * (2 * row + 8), flops=0.0)
    if op == "store":
        row = 4 * c["W"] + 2 * c["c"] + 2 * c["d"]
        return dict(bytes=2.0 * row * float(k.sum()) * c["Hkv"], flops=0.0)
    pairs = float((k * (L - k) + k * (k + 1) / 2).sum())
    each = 2 if c["dtype"] == "bf16" else 4
    moved = float(L.sum()) * c["Hkv"] * (c["m"] / 8 + 2 + 2 * c["d"])
    moved += float(k.sum()) * c["Hq"] * c["d"] * (each + 2)
    return dict(bytes=moved, flops=2.0 * pairs * c["Hq"] * (min(c["m"], c["d"]) + c["d"]))


# ---------------------------------------------------------------------------
# the definitions in 64 bits

def _exact_rotary(s):
    c = s["case"]
    pos = s["positions"].cpu().numpy().astype(np.float64)
    f = s["inv_freq"].cpu().numpy().astype(np.float64)
    turn = np.exp(1j * (-1 if c["inverse"] else 1) * np.outer(pos, f))[:, None] * s["scale"]
    done = []
    for x in (s["Q"], s["K"]):
        y = x.double().cpu().numpy()
        h = c["rot"] // 2
        even = slice(0, 2 * h, 2) if c["interleaved"] else slice(0, h)
        odd = slice(1, 2 * h, 2) if c["interleaved"] else slice(h, 2 * h)
        v = (y[..., even] + 1j * y[..., odd]) * turn
        y[..., even], y[..., odd] = v.real, v.imag
        done.append(torch.from_numpy(y))
    return tuple(done)


def _exact_chunk(s):
    c = s["case"]
    G, P, m, d = c["Hq"] // c["Hkv"], c["P"], c["m"], c["d"]
    cu, lens, table = (s[k].cpu().numpy() for k in ("cu", "lens", "table"))
    S = s["S"].double()
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    for b in range(c["B"]):
        first, last, L = int(cu[b]), int(cu[b + 1]), int(lens[b])
        t = np.arange(L)
        page = torch.from_numpy(table[b, t // P].astype(np.int64)).to(DEV)
        slot = torch.from_numpy(t % P).to(DEV)
        tt = torch.arange(L, device=DEV)
        for h in range(c["Hkv"]):
            khat = _signs(s["sign_pages"][page, h, slot], torch.float64) @ S
            khat *= s["norm_pages"][page, h, slot].double()[:, None] * math.sqrt(math.pi / 2) / m
            v = s["value_pages"][page, h, slot].double()
            step = max(1, (1 << 27) // (G * max(L, 1)))
            for i in range(first, last, step):
                j = min(last, i + step)
                q = s["Q"][i:j, h * G:(h + 1) * G].double()
                x = (q @ khat.T) / math.sqrt(d)
                sees = L - (last - first) + torch.arange(i - first, j - first, device=DEV) + 1
                x = x.masked_fill(tt[None, None] >= sees[:, None, None], -math.inf)
                out[i:j, h * G:(h + 1) * G] = torch.softmax(x, -1) @ v
    return out


def _exact_mass(s):
    c = s["case"]
    G = c["Hq"] // c["Hkv"]
    out = torch.zeros(s["mass"].shape, dtype=torch.float64, device=DEV)
    for b, L in enumerate(s["lens"].tolist()):
        p = torch.softmax(s["scores"][b, :, :L].double() * s["softmax_scale"], -1)
        out[b, :, :L] = s["mass"][b, :, :L].double() * c["decay"] + p.view(c["Hkv"], G, L).sum(1)
    return out


def exact(case, seed):
    if case["op"] in ("store", "evict"):
        return None  # copies and whole numbers: nothing is computed
    s = prepare(case, seed)
    return {"rotary": _exact_rotary, "chunk": _exact_chunk, "mass": _exact_mass}[case["op"]](s)
