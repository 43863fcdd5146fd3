"""Cases of the rotated appends and of latent attention, with their plain forms.

Four operators of a serving step on paged caches:

* ``rope``          write_rope: rotate this step's K rows by their positions on
                    the way into bf16 pages (V is copied), and the queries too;
* ``rope_fp8``      write_rope_fp8: the same into E4M3 pages with one
                    power-of-two scale per row;
* ``latent_write``  write_latent: append one latent vector and one rotated
                    shared key part a token to latent pages, and put the
                    rotated query part into its place in the absorbed query;
* ``latent``        attend_latent: attention over those pages in the absorbed
                    form, decode rows and query chunks alike.

``run`` computes each in plain torch where ``own`` is false and calls the
library where it is true, on the state that ``prepare`` makes.
"""

import math

import numpy as np
import torch

own = False

PAGE = 16        # tokens a page
HEAD = 128       # head dimension of the K/V pages
LATENT = 512     # latent part of a latent row (keys and values)
ROPE = 64        # rotated part of a latent row (keys only)
ROW = LATENT + ROPE

# The most that a drawn case may cost, set by the largest listed cases.
MOST_TOKENS = 8191
MOST_PAIR_FLOPS = 4e11
MOST_ATTEND_BYTES = 1.5e9


def listed():
    return [
        # one token of one sequence: an interactive request alone on the card
        {"name": "rope_1", "op": "rope", "tokens": 1, "hq": 32, "hkv": 8, "rot": 128,
         "interleaved": False, "padded": 0, "max_pos": 32768},
        # several prompts' chunks in one step, half of each head rotated in pairs
        {"name": "rope_8191", "op": "rope", "tokens": 8191, "hq": 32, "hkv": 8, "rot": 64,
         "interleaved": True, "padded": 0, "max_pos": 32768},
        # decode rows beside two 512-token chunks, on 8-bit pages
        {"name": "rope_fp8_1120", "op": "rope_fp8", "tokens": 1120, "hq": 32, "hkv": 8, "rot": 128,
         "interleaved": False, "padded": 0, "max_pos": 32768},
        # a decode batch on 8-bit pages padded to a captured size, its last slots unused
        {"name": "rope_fp8_64", "op": "rope_fp8", "tokens": 64, "hq": 32, "hkv": 8, "rot": 128,
         "interleaved": False, "padded": 3, "max_pos": 32768},
        # a decode batch of a model with latent attention
        {"name": "latent_write_64", "op": "latent_write", "tokens": 64, "heads": 128,
         "interleaved": True, "padded": 0, "max_pos": 32768},
        # a prompt's chunk, an odd number of tokens, few heads (one rank's share)
        {"name": "latent_write_4097", "op": "latent_write", "tokens": 4097, "heads": 16,
         "interleaved": False, "padded": 0, "max_pos": 32768},
        # four short sequences: latency
        {"name": "latent_tiny", "op": "latent", "seqs": 4, "lo": 17, "hi": 255, "n_lo": 1, "n_hi": 1,
         "heads": 16, "chunks": 0, "chunk": 0, "ctx_lo": 0, "ctx_hi": 0},
        # an ordinary decode batch, all heads on this card
        {"name": "latent_decode", "op": "latent", "seqs": 64, "lo": 512, "hi": 4096, "n_lo": 1, "n_hi": 1,
         "heads": 128, "chunks": 0, "chunk": 0, "ctx_lo": 0, "ctx_hi": 0},
        # one long sequence: the work has to be split along the cache
        {"name": "latent_one_long", "op": "latent", "seqs": 1, "lo": 131072, "hi": 131072, "n_lo": 1, "n_hi": 1,
         "heads": 64, "chunks": 0, "chunk": 0, "ctx_lo": 0, "ctx_hi": 0},
        # a long-tailed decode batch, few heads: bound by the cache's bytes
        {"name": "latent_long_tail", "op": "latent", "seqs": 256, "lo": 16, "hi": 32768, "n_lo": 1, "n_hi": 1,
         "heads": 16, "chunks": 0, "chunk": 0, "ctx_lo": 0, "ctx_hi": 0},
        # speculative rows, two to five tokens each, an uneven number of heads
        {"name": "latent_draft", "op": "latent", "seqs": 32, "lo": 256, "hi": 8192, "n_lo": 2, "n_hi": 5,
         "heads": 20, "chunks": 0, "chunk": 0, "ctx_lo": 0, "ctx_hi": 0},
        # decode rows beside a long prompt chunk over a cached context
        {"name": "latent_mixed", "op": "latent", "seqs": 33, "lo": 256, "hi": 8192, "n_lo": 1, "n_hi": 1,
         "heads": 64, "chunks": 2, "chunk": 1023, "ctx_lo": 1536, "ctx_hi": 3584},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the ranges the listed ones stand for."""
    op = rng.choice(["rope", "rope_fp8", "latent_write", "latent", "latent"])
    if op in ("rope", "rope_fp8"):
        tokens = _log(rng, 1, MOST_TOKENS if op == "rope" else 4096)
        hq, hkv = rng.choice([(32, 8), (8, 2), (16, 16), (16, 4), (32, 2), (16, 1), (8, 8)])
        return {"op": op, "tokens": tokens, "hq": hq, "hkv": hkv, "rot": rng.choice([128, 128, 96, 64, 32]),
                "interleaved": rng.random() < 0.4, "padded": rng.choice([0, 0, 1, tokens // 8]),
                "max_pos": rng.choice([4096, 32768])}
    if op == "latent_write":
        heads = rng.choice([1, 8, 12, 16, 20, 32, 64, 128])
        tokens = _log(rng, 1, min(MOST_TOKENS, 4097 * 16 // heads))
        return {"op": op, "tokens": tokens, "heads": heads, "interleaved": rng.random() < 0.5,
                "padded": rng.choice([0, 0, 1, tokens // 8]), "max_pos": rng.choice([4096, 32768])}
    while True:
        lo = _log(rng, 1, 2048)
        n_lo = rng.choice([1, 1, 1, 2])
        seqs = _log(rng, 1, 256)
        case = {"op": op, "seqs": seqs, "lo": lo, "hi": _log(rng, max(lo, 16), 131072 if seqs < 9 else 32768),
                "n_lo": n_lo, "n_hi": rng.choice([n_lo, n_lo, 4, 6]), "heads": rng.choice([1, 8, 12, 16, 20, 32, 64, 96, 128]),
                "chunks": rng.choice([0, 0, 1, 2, 3]), "chunk": _log(rng, 9, 1023), "ctx_lo": 0, "ctx_hi": _log(rng, 1, 4096)}
        if not case["chunks"]:
            case.update(chunk=0, ctx_hi=0)
        if case["lo"] < case["n_hi"]:
            continue
        rows = case["seqs"] * case["n_hi"] * case["heads"]
        most = case["hi"] + case["ctx_hi"] + case["chunk"]
        w = work(case)
        if rows * case["hi"] <= 2 ** 29 and case["chunk"] * case["heads"] * most <= 2 ** 29 \
                and w["flops"] <= MOST_PAIR_FLOPS and w["bytes"] <= MOST_ATTEND_BYTES:
            return case


# ---- inputs -------------------------------------------------------------------


def _lengths(case):
    """(L, n) of every sequence: cached tokens with this step's, query tokens.
    They go by the case alone, so that every seed has the same shapes and work."""
    rng = np.random.Generator(np.random.PCG64([case["seqs"], case["lo"], case["hi"], case["heads"]]))
    B = case["seqs"]
    if case["hi"] > 32 * case["lo"]:  # a long tail
        L = np.round(np.exp(rng.uniform(np.log(case["lo"]), np.log(case["hi"]), B)))
    else:
        L = rng.integers(case["lo"], case["hi"], size=B, endpoint=True)
    L = np.clip(L, case["lo"], case["hi"]).astype(np.int64)
    n = rng.integers(case["n_lo"], case["n_hi"], size=B, endpoint=True)
    if case["chunks"]:
        ctx = rng.integers(case["ctx_lo"], case["ctx_hi"], size=case["chunks"], endpoint=True)
        L = np.concatenate([L, ctx + case["chunk"]])
        n = np.concatenate([n, np.full(case["chunks"], case["chunk"])])
    return L, n


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _cos_sin(max_pos, dim):
    """The rotation's table, fp32 [max_pos, dim]: cosines, then sines; angles in 64 bits."""
    freq = 10000.0 ** (-torch.arange(0, dim, 2, device="cuda", dtype=torch.float64) / dim)
    angle = torch.arange(max_pos, device="cuda", dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], dim=1).float()


def _slots(rng, tokens, padded):
    """(pages of the pool, slot of every token): distinct, shuffled; -1 for the padded last ones."""
    pages = -(-tokens // PAGE) + 3
    slots = rng.permutation(pages * PAGE)[:tokens].astype(np.int64)
    if padded:
        slots[tokens - min(padded, tokens):] = -1
    return pages, torch.from_numpy(slots).cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    if case["op"] == "latent":
        return _prepare_latent(case, seed, gen)
    rng = np.random.Generator(np.random.PCG64(seed))
    T = case["tokens"]
    pages, slots = _slots(rng, T, case["padded"])
    s = {"op": case["op"], "interleaved": case["interleaved"], "slots": slots, "pages": pages,
         "positions": torch.from_numpy(rng.integers(0, case["max_pos"], size=T)).cuda()}
    # The pools carry one page more than the library is told of: the plain form parks padded tokens there.
    if case["op"] == "latent_write":
        H = case["heads"]
        s["cos_sin"] = _cos_sin(case["max_pos"], ROPE)
        s["c_new"] = _normal(gen, T, LATENT)                      # the normalised latents
        s["k_pe"] = _normal(gen, T, ROW)[:, LATENT:]              # a slice of the down projection
        s["q_pe"] = _normal(gen, T, H, HEAD + ROPE)[..., HEAD:]   # a slice of the query projection
        s["q_out"] = _normal(gen, T, H, ROW)                      # absorbed queries, rotated part to come
        s["pool"] = _normal(gen, pages + 1, PAGE, ROW)
        return s
    hq, hkv = case["hq"], case["hkv"]
    s["cos_sin"] = _cos_sin(case["max_pos"], case["rot"])
    qkv = _normal(gen, T, hq + 2 * hkv, HEAD)                     # one fused projection's output
    s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    s["q_out"] = torch.empty(T, hq, HEAD, device="cuda", dtype=torch.bfloat16)
    shape = (pages + 1, hkv, PAGE, HEAD)
    if case["op"] == "rope":
        s["kc"], s["vc"] = _normal(gen, *shape), _normal(gen, *shape)
    else:
        for name in ("kc", "vc"):
            x = torch.randn(shape, generator=gen, device="cuda") * 64.0
            s[name] = x.clamp_(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
            s[name + "_scale"] = torch.full(shape[:3], 121, dtype=torch.uint8, device="cuda")
    return s


def _prepare_latent(case, seed, gen):
    L, n = _lengths(case)
    rng = np.random.Generator(np.random.PCG64(seed))
    H, B, T = case["heads"], len(L), int(n.sum())
    need = -(-L // PAGE)
    NB = int(need.sum())
    perm = rng.permutation(NB)
    tables = np.full((B, int(need.max())), NB, dtype=np.int32)  # unused entries name no page
    at = 0
    for b in range(B):
        tables[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
    qsl = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    s = {"op": "latent", "scale": 1.0 / math.sqrt(HEAD + ROPE), "most": int(n.max()),
         "q": _normal(gen, T, H, ROW), "pool": _normal(gen, NB, PAGE, ROW),
         "out": torch.empty(T, H, LATENT, device="cuda", dtype=torch.bfloat16),
         "tables": torch.from_numpy(tables).cuda(), "lens": torch.from_numpy(L.astype(np.int32)).cuda(),
         "qsl": torch.from_numpy(qsl).cuda()}
    # Sequences with the same number of query tokens, for the plain form.
    s["groups"] = []
    for k in sorted(set(n.tolist())):
        who = np.flatnonzero(n == k)
        s["groups"].append((k, int(L[who].max()), torch.from_numpy(who).cuda(),
                            torch.from_numpy(qsl[who].astype(np.int64)[:, None] + np.arange(k)).cuda()))
    return s


# ---- one pass -----------------------------------------------------------------


def run(s):
    if own:
        return _own(s)
    if s["op"] == "latent":
        return _plain_latent(s)
    if s["op"] == "latent_write":
        return _plain_latent_write(s)
    return _plain_rope(s)


def _own(s):
    import paged_kv_cache_pkv_gb300 as pkv
    if s["op"] == "latent":
        if "workspace" not in s:  # made once, kept beside the pool
            desc = pkv.make_latent_desc(s["pool"], s["q"].shape[1], s["tables"].shape[1])
            size = pkv.workspace_size_latent(desc, s["lens"].shape[0], s["q"].shape[0])
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        return pkv.attend_latent(s["q"], s["pool"], s["tables"], s["lens"], s["qsl"], s["scale"], out=s["out"],
                                 workspace=s["workspace"], max_query_len=s["most"])
    NB = s["pages"]
    if s["op"] == "latent_write":
        q = pkv.write_latent(s["c_new"], s["k_pe"], s["positions"], s["cos_sin"], s["slots"], s["pool"][:NB],
                             q_pe=s["q_pe"], q_out=s["q_out"], interleaved=s["interleaved"])
        return q, s["pool"][:NB]
    if s["op"] == "rope":
        q = pkv.write_rope(s["k"], s["v"], s["positions"], s["cos_sin"], s["slots"], s["kc"][:NB], s["vc"][:NB],
                           q=s["q"], q_out=s["q_out"], interleaved=s["interleaved"])
        return q, s["kc"][:NB], s["vc"][:NB]
    q = pkv.write_rope_fp8(s["k"], s["v"], s["positions"], s["cos_sin"], s["slots"], s["kc"][:NB], s["vc"][:NB],
                           s["kc_scale"][:NB], s["vc_scale"][:NB], q=s["q"], q_out=s["q_out"],
                           interleaved=s["interleaved"])
    return _fp8_outputs(s, q)


def _fp8_outputs(s, q):
    NB = s["pages"]
    e4m3 = torch.float8_e4m3fn
    return q, s["kc"][:NB].view(e4m3), s["vc"][:NB].view(e4m3), s["kc_scale"][:NB], s["vc_scale"][:NB]


def _rotate(x, positions, cos_sin, interleaved):
    """x [T, heads, D] with its first cos_sin.shape[1] dims rotated, fp32."""
    x = x.float()
    half = cos_sin.shape[1] // 2
    cs = cos_sin[positions][:, None]
    cos, sin = cs[..., :half], cs[..., half:]
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([turned, x[..., 2 * half:]], dim=-1)


def _place(s):
    """(page, row) of every token; padded ones go to the spare page."""
    slot = torch.where(s["slots"] < 0, s["pages"] * PAGE, s["slots"])
    return slot // PAGE, slot % PAGE


def _encode(x):
    """(E4M3 codes as bytes, scale bytes) of fp32 rows x [..., D]: the smallest power of two under which |x| <= 448."""
    top = x.abs().amax(dim=-1)
    mant, exp = torch.frexp(top)  # top = mant * 2^exp, mant in [0.5, 1)
    e = exp - 9 + (mant > 0.875)
    e = torch.where(top == 0, -126, e).clamp(-126, 127).int()
    inverse = ((127 - e) << 23).view(torch.float32)  # 2^-e by its bits
    codes = (x * inverse[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, (e + 127).to(torch.uint8)


def _plain_rope(s):
    page, row = _place(s)
    s["q_out"].copy_(_rotate(s["q"], s["positions"], s["cos_sin"], s["interleaved"]))
    k, v = _rotate(s["k"], s["positions"], s["cos_sin"], s["interleaved"]), s["v"]
    NB = s["pages"]
    if s["op"] == "rope":
        s["kc"][page, :, row] = k.to(torch.bfloat16)
        s["vc"][page, :, row] = v
        return s["q_out"], s["kc"][:NB], s["vc"][:NB]
    for name, x in (("kc", k), ("vc", v.float())):
        codes, scale = _encode(x)
        s[name][page, :, row] = codes
        s[name + "_scale"][page, :, row] = scale
    return _fp8_outputs(s, s["q_out"])


def _plain_latent_write(s):
    page, row = _place(s)
    s["q_out"][..., LATENT:] = _rotate(s["q_pe"], s["positions"], s["cos_sin"], s["interleaved"]).to(torch.bfloat16)
    k = _rotate(s["k_pe"][:, None], s["positions"], s["cos_sin"], s["interleaved"])[:, 0]
    s["pool"][page, row] = torch.cat([s["c_new"], k.to(torch.bfloat16)], dim=-1)
    return s["q_out"], s["pool"][:s["pages"]]


def _plain_latent(s):
    flat = s["pool"].view(-1, ROW)
    H = s["q"].shape[1]
    for n, most, who, rows in s["groups"]:
        pos = torch.arange(most, device="cuda")
        page = s["tables"][who][:, pos // PAGE].long().clamp(max=s["pool"].shape[0] - 1)
        kv = flat[page * PAGE + pos % PAGE].float()                              # [b, most, 576]
        q = s["q"][rows].float().view(len(who), n * H, ROW)
        score = torch.bmm(q, kv.transpose(1, 2)).mul_(s["scale"]).view(len(who), n, H, most)
        last = s["lens"][who].long()[:, None] - n + torch.arange(n, device="cuda")  # last key a row sees
        score.masked_fill_((pos > last[..., None])[:, :, None], -math.inf)
        p = score.sub_(score.amax(dim=-1, keepdim=True)).exp_()
        o = torch.bmm(p.view(len(who), n * H, most), kv[..., :LATENT])
        o = o.view(len(who), n, H, LATENT) / p.sum(dim=-1, keepdim=True)
        s["out"][rows] = o.to(torch.bfloat16)
    return s["out"]


# ---- cost and definition ------------------------------------------------------


def work(case):
    if case["op"] == "latent":
        H = case["heads"]
        L, n = _lengths(case)
        pairs = int((n * L - n * (n - 1) // 2).sum())
        T = int(n.sum())
        return {"bytes": int(L.sum()) * ROW * 2 + T * H * (ROW + LATENT) * 2 + int((-(-L // PAGE)).sum()) * 4,
                "flops": pairs * H * 2 * (ROW + LATENT)}
    T = case["tokens"]
    live = T - min(T, case["padded"])
    table = min(T, case["max_pos"])
    if case["op"] == "latent_write":
        H = case["heads"]
        return {"bytes": T * (16 + H * ROPE * 4) + live * ROW * 4 + table * ROPE * 4, "flops": 3 * ROPE * (T * H + live)}
    hq, hkv, rot = case["hq"], case["hkv"], case["rot"]
    kv = 2 * hkv * (HEAD * 4 if case["op"] == "rope" else HEAD * 3 + 1)
    return {"bytes": T * (16 + hq * HEAD * 4) + live * kv + table * rot * 4,
            "flops": 3 * rot * (T * hq + live * hkv)}


def exact(case, seed):
    """What run() returns, from the definition in 64 bits."""
    s = prepare(case, seed)
    if case["op"] == "latent":
        return _exact_latent(s)
    live = torch.nonzero(s["slots"] >= 0)[:, 0]
    page, row = torch.div(s["slots"][live], PAGE, rounding_mode="floor"), s["slots"][live] % PAGE
    NB = s["pages"]
    if case["op"] == "latent_write":
        q = s["q_out"].double()
        q[..., LATENT:] = _turn(s, s["q_pe"])
        pool = s["pool"][:NB].double()
        pool[page, row, :LATENT] = s["c_new"][live].double()
        pool[page, row, LATENT:] = _turn(s, s["k_pe"][:, None])[live, 0]
        return q, pool
    q, k, v = _turn(s, s["q"]), _turn(s, s["k"])[live], s["v"][live].double()
    if case["op"] == "rope":
        kc, vc = s["kc"][:NB].double(), s["vc"][:NB].double()
        kc[page, :, row], vc[page, :, row] = k, v
        return q, kc, vc
    # The codes stand for the nearest E4M3 value to the fp32 rotation: each product and each sum rounded to fp32.
    k = _turn(s, s["k"], lambda x: x.float().double())[live]
    kc, vc = (s[name][:NB].view(torch.float8_e4m3fn).double() for name in ("kc", "vc"))
    ks, vs = s["kc_scale"][:NB].clone(), s["vc_scale"][:NB].clone()
    for x, codes, scales in ((k, kc, ks), (v, vc, vs)):
        e = torch.ceil(torch.log2(x.abs().amax(dim=-1) / 448.0)).clamp(-126, 127)
        y = x * torch.exp2(-e)[..., None]
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)  # 2^-9 below the normal values
        codes[page, :, row] = torch.round(y / step) * step  # round() takes ties to even
        scales[page, :, row] = (e + 127).to(torch.uint8)
    return q, kc, vc, ks, vs


def _turn(s, x, rounded=lambda x: x):
    """x [T, heads, D] as complex numbers times the table's, in 64 bits."""
    x = x.double()
    table = s["cos_sin"].double()[s["positions"]]
    half = table.shape[1] // 2
    w = torch.complex(table[:, :half], table[:, half:])[:, None]
    first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if s["interleaved"] \
        else (slice(0, half), slice(half, 2 * half))
    out = x.clone()
    out[..., first] = rounded(rounded(x[..., first] * w.real) - rounded(x[..., second] * w.imag))
    out[..., second] = rounded(rounded(x[..., second] * w.real) + rounded(x[..., first] * w.imag))
    return out


def _exact_latent(s):
    lens, qsl = s["lens"].tolist(), s["qsl"].tolist()
    out = torch.empty(s["out"].shape, device="cuda", dtype=torch.float64)
    for b, L in enumerate(lens):
        pages = s["tables"][b, :-(-L // PAGE)].long()
        kv = s["pool"][pages].reshape(-1, ROW)[:L].double()
        n = qsl[b + 1] - qsl[b]
        for j in range(0, n, 64):  # few rows at a time bound the scores' memory
            rows = slice(qsl[b] + j, qsl[b] + min(n, j + 64))
            q = s["q"][rows].double()
            hidden = torch.arange(L, device="cuda") > L - n + torch.arange(j, min(n, j + 64), device="cuda")[:, None]
            logits = torch.einsum("thd,kd->thk", q, kv) * s["scale"]
            weights = torch.softmax(logits.masked_fill(hidden[:, None], -math.inf), dim=-1)
            out[rows] = torch.einsum("thk,kd->thd", weights, kv[:, :LATENT])
    return out
