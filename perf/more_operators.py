"""Cases of the multi-axis rotated appends, of accumulated attention weights
and of eviction by them, with their plain forms.

Three operators of a serving step on K/V pages, each on bf16 and on E4M3 pages:

* ``axes``   write_rope_axes: rotate this step's K rows and queries, each pair
             of elements by one of several positions a token has (time, height
             and width of an image's or a video's patch), on the way into the
             pages;
* ``weigh``  weigh: add up the attention weight that every cached token gets
             from this step's queries, for each kv head, into paged scores;
* ``evict``  evict: keep the tokens of the largest scores of each sequence and
             kv head beside the first and the most recent ones, and move them
             together in their pages.

``run`` computes each in plain torch where ``own`` is false and calls the
library where it is true, on the state that ``prepare`` makes.
"""

import math

import numpy as np
import torch

own = False

PAGE = 16    # tokens a page
HEAD = 128   # head dimension

# The most that a drawn case may cost, set by the largest listed cases.
MOST_TOKENS = 4099
MOST_WEIGH_FLOPS = 6.8e10
MOST_WEIGH_BYTES = 2.4e9
MOST_EVICT_BYTES = 6e8


def listed():
    return [
        # one token of one sequence behind an image prompt: all its positions are alike
        {"name": "axes_1", "op": "axes", "fp8": False, "tokens": 1, "hq": 32, "hkv": 8, "rot": 128, "axes": 3,
         "cycled": False, "interleaved": False, "padded": 0, "max_pos": 32768},
        # a chunk of video patches, the axes taking turns from pair to pair
        {"name": "axes_4099", "op": "axes", "fp8": False, "tokens": 4099, "hq": 32, "hkv": 8, "rot": 128, "axes": 3,
         "cycled": True, "interleaved": False, "padded": 0, "max_pos": 32768},
        # an image beside decode rows on 8-bit pages, the axes in blocks, the last slots unused
        {"name": "axes_fp8_1120", "op": "axes", "fp8": True, "tokens": 1120, "hq": 32, "hkv": 8, "rot": 128, "axes": 3,
         "cycled": False, "interleaved": False, "padded": 32, "max_pos": 32768},
        # four short sequences: latency
        {"name": "weigh_tiny", "op": "weigh", "fp8": False, "seqs": 4, "lo": 17, "hi": 255, "n_lo": 1, "n_hi": 1,
         "whole": False, "hq": 32, "hkv": 8, "decay": 1.0, "first": 0},
        # an ordinary decode batch that weighs its cache at every step
        {"name": "weigh_decode", "op": "weigh", "fp8": False, "seqs": 64, "lo": 512, "hi": 4096, "n_lo": 1, "n_hi": 1,
         "whole": False, "hq": 32, "hkv": 8, "decay": 1.0, "first": 4},
        # a long-tailed decode batch on 8-bit pages, older weights fading: bound by the cache's bytes
        {"name": "weigh_fp8_tail", "op": "weigh", "fp8": True, "seqs": 256, "lo": 16, "hi": 32768, "n_lo": 1, "n_hi": 1,
         "whole": False, "hq": 32, "hkv": 8, "decay": 0.9375, "first": 0},
        # speculative rows, two to five tokens each
        {"name": "weigh_draft", "op": "weigh", "fp8": False, "seqs": 32, "lo": 256, "hi": 8192, "n_lo": 2, "n_hi": 5,
         "whole": False, "hq": 32, "hkv": 8, "decay": 1.0, "first": 0},
        # the last 32 tokens of eight prompts judge all of each, before the prompts are cut down
        {"name": "weigh_window", "op": "weigh", "fp8": False, "seqs": 8, "lo": 4096, "hi": 8192, "n_lo": 32, "n_hi": 32,
         "whole": False, "hq": 32, "hkv": 8, "decay": 0.0, "first": 0},
        # every row of a prompt, an odd number of tokens
        {"name": "weigh_prompt", "op": "weigh", "fp8": False, "seqs": 1, "lo": 4095, "hi": 4095, "n_lo": 1, "n_hi": 1,
         "whole": True, "hq": 32, "hkv": 8, "decay": 0.0, "first": 0},
        # four short sequences: latency
        {"name": "evict_tiny", "op": "evict", "fp8": False, "seqs": 4, "lo": 129, "hi": 255, "hkv": 8, "keep": 128,
         "first": 4, "recent": 16},
        # a decode batch cut down to a budget, on 8-bit pages; the shortest sequences are below it already
        {"name": "evict_fp8_decode", "op": "evict", "fp8": True, "seqs": 64, "lo": 512, "hi": 4096, "hkv": 8, "keep": 1023,
         "first": 4, "recent": 64},
        # one long context cut down to a quarter
        {"name": "evict_one_long", "op": "evict", "fp8": False, "seqs": 1, "lo": 131072, "hi": 131072, "hkv": 8,
         "keep": 32768, "first": 16, "recent": 512},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the ranges the listed ones stand for."""
    op = rng.choice(["axes", "weigh", "weigh", "evict"])
    fp8 = rng.random() < 0.4
    if op == "axes":
        tokens = _log(rng, 1, MOST_TOKENS)
        hq, hkv = rng.choice([(32, 8), (8, 2), (16, 16), (16, 4), (32, 2), (16, 1), (8, 8)])
        return {"op": op, "fp8": fp8, "tokens": tokens, "hq": hq, "hkv": hkv, "rot": rng.choice([128, 128, 96, 64, 32]),
                "axes": rng.choice([2, 3, 3, 4]), "cycled": rng.random() < 0.5, "interleaved": rng.random() < 0.3,
                "padded": rng.choice([0, 0, 1, tokens // 8]), "max_pos": rng.choice([4096, 32768])}
    while True:
        hq, hkv = rng.choice([(32, 8), (32, 8), (8, 2), (16, 16), (16, 4), (32, 2), (16, 1), (8, 8)])
        seqs = _log(rng, 1, 256)
        lo = _log(rng, 1, 2048)
        hi = _log(rng, max(lo, 16), 131072 if seqs < 9 else 32768)
        if op == "evict":
            keep = _log(rng, 1, hi)
            case = {"op": op, "fp8": fp8, "seqs": seqs, "lo": lo, "hi": hi, "hkv": hkv, "keep": keep,
                    "first": rng.choice([0, 4, 16, keep // 3]), "recent": rng.choice([0, 1, 16, 64, keep // 2, keep])}
            if _most(case) * hkv * seqs <= 2 ** 26 and work(case)["bytes"] <= MOST_EVICT_BYTES:
                return case
            continue
        kind = rng.choice(["decode", "decode", "draft", "window", "whole"])
        n_lo, n_hi = {"decode": (1, 1), "draft": (rng.choice([1, 2]), rng.choice([4, 6, 9])), "whole": (1, 1),
                      "window": (rng.choice([8, 17]), rng.choice([32, 64, 100]))}[kind]
        case = {"op": op, "fp8": fp8, "seqs": seqs, "lo": lo, "hi": hi, "n_lo": n_lo, "n_hi": n_hi,
                "whole": kind == "whole", "hq": hq, "hkv": hkv, "decay": rng.choice([0.0, 0.9375, 1.0, 1.0]),
                "first": rng.choice([0, 0, 4, 100])}
        if lo < n_hi:
            continue
        w = work(case)
        if w["flops"] <= MOST_WEIGH_FLOPS and w["bytes"] <= MOST_WEIGH_BYTES:
            return case


# ---- inputs -------------------------------------------------------------------


def _lengths(case):
    """(L, n) of every sequence: cached tokens with this step's, query tokens.
    They go by the case alone, so that every seed has the same shapes and work."""
    rng = np.random.Generator(np.random.PCG64([case["seqs"], case["lo"], case["hi"], case["hkv"]]))
    B = case["seqs"]
    if case["hi"] > 32 * case["lo"]:  # a long tail
        L = np.round(np.exp(rng.uniform(np.log(case["lo"]), np.log(case["hi"]), B)))
    else:
        L = rng.integers(case["lo"], case["hi"], size=B, endpoint=True)
    L = np.clip(L, case["lo"], case["hi"]).astype(np.int64)
    if case["op"] == "evict":
        return L, np.zeros(B, dtype=np.int64)
    n = L.copy() if case["whole"] else rng.integers(case["n_lo"], case["n_hi"], size=B, endpoint=True)
    return L, n


def _most(case):
    return int(_lengths(case)[0].max())


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _codes(gen, *shape):
    """(E4M3 codes as bytes, scale bytes of the rows): values of about unit size."""
    x = torch.randn(shape, generator=gen, device="cuda").mul_(64.0).clamp_(-448.0, 448.0)
    scale = torch.randint(120, 123, shape[:-1], generator=gen, device="cuda").to(torch.uint8)
    return x.to(torch.float8_e4m3fn).view(torch.uint8), scale


def _cos_sin(max_pos, dim):
    """The rotation's table, fp32 [max_pos, dim]: cosines, then sines; angles in 64 bits."""
    freq = 10000.0 ** (-torch.arange(0, dim, 2, device="cuda", dtype=torch.float64) / dim)
    angle = torch.arange(max_pos, device="cuda", dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], dim=1).float()


def _axis_of_pairs(case):
    """The axis that each pair of elements turns by."""
    half, A = case["rot"] // 2, case["axes"]
    if case["cycled"]:
        return [i % A for i in range(half)]
    first = half // (A + 1)  # the first axis has a smaller block than the others
    return [0] * first + [1 + (i * (A - 1)) // (half - first) for i in range(half - first)]


def _tables(rng, L):
    """(pages in the pool, block tables): every sequence's pages shuffled; unused entries name no page."""
    need = -(-L // PAGE)
    NB = int(need.sum())
    perm = rng.permutation(NB)
    tables = np.full((len(L), int(need.max())), NB, dtype=np.int32)
    at = 0
    for b in range(len(L)):
        tables[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
    return NB, tables


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = np.random.Generator(np.random.PCG64(seed))
    s = {"op": case["op"], "fp8": case["fp8"]}
    # The pools carry one page more than the library is told of: the plain form parks there what has no place.
    return {"axes": _prepare_axes, "weigh": _prepare_weigh, "evict": _prepare_evict}[case["op"]](s, case, rng, gen)


def _pool(s, names, gen, *shape):
    for name in names:
        if s["fp8"]:
            s[name], s[name + "_scale"] = _codes(gen, *shape)
        else:
            s[name] = _normal(gen, *shape)


def _prepare_axes(s, case, rng, gen):
    T, hq, hkv = case["tokens"], case["hq"], case["hkv"]
    s["pages"] = -(-T // PAGE) + 3
    slots = rng.permutation(s["pages"] * PAGE)[:T].astype(np.int64)
    if case["padded"]:
        slots[T - min(case["padded"], T):] = -1
    s["slots"] = torch.from_numpy(slots).cuda()
    # patches of a frame after frame: time moves on slowly, height and width run through a grid
    t0 = int(rng.integers(0, case["max_pos"] - T)) if T < case["max_pos"] else 0
    grid = np.arange(T)
    pos = np.stack([t0 + grid // 256, t0 + grid // 16 % 16, t0 + grid % 16, t0 + grid][:case["axes"]])
    if T == 1:
        pos[:] = t0
    s["positions"] = torch.from_numpy(np.minimum(pos, case["max_pos"] - 1)).cuda()
    s["axes"] = bytes(_axis_of_pairs(case))
    s["axis_of"] = torch.tensor(list(s["axes"]), device="cuda")
    s["interleaved"] = case["interleaved"]
    s["cos_sin"] = _cos_sin(case["max_pos"], case["rot"])
    qkv = _normal(gen, T, hq + 2 * hkv, HEAD)  # one fused projection's output
    s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    s["q_out"] = torch.empty(T, hq, HEAD, device="cuda", dtype=torch.bfloat16)
    _pool(s, ("kc", "vc"), gen, s["pages"] + 1, hkv, PAGE, HEAD)
    return s


def _prepare_weigh(s, case, rng, gen):
    L, n = _lengths(case)
    hq, hkv, T = case["hq"], case["hkv"], int(n.sum())
    s["pages"], tables = _tables(rng, L)
    qsl = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    s.update(scale=1.0 / math.sqrt(HEAD), decay=case["decay"], most=int(n.max()), keys=int((-(-L // PAGE)).sum()) * PAGE,
             q=_normal(gen, T, hq, HEAD), tables=torch.from_numpy(tables).cuda(),
             lens=torch.from_numpy(L.astype(np.int32)).cuda(), qsl=torch.from_numpy(qsl).cuda(),
             first=torch.full((len(L),), case["first"], dtype=torch.int32, device="cuda"))
    _pool(s, ("kc",), gen, s["pages"] + 1, hkv, PAGE, HEAD)
    # what earlier steps have added up
    s["scores"] = torch.rand(s["pages"] + 1, hkv, PAGE, generator=gen, device="cuda").pow_(8.0)
    # For the plain form: sequences with the same number of query tokens, of like lengths, a bounded number of keys at once.
    s["groups"] = []
    for k in sorted(set(n.tolist())):
        who = np.flatnonzero(n == k)
        who = who[np.argsort(L[who], kind="stable")[::-1]]
        while len(who):
            take = max(1, (1 << 18) // int(L[who[0]]))
            part, who = who[:take], who[take:]
            s["groups"].append((k, int(L[part[0]]), torch.from_numpy(part.copy()).cuda(),
                                torch.from_numpy(qsl[part].astype(np.int64)[:, None] + np.arange(k)).cuda()))
    return s


def _prepare_evict(s, case, rng, gen):
    L, _ = _lengths(case)
    hkv = case["hkv"]
    s["pages"], tables = _tables(rng, L)
    s.update(most=int(L.max()), most_kept=int(min(case["keep"], L.max())), recent=case["recent"],
             tables=torch.from_numpy(tables).cuda(), lens=torch.from_numpy(L.astype(np.int32)).cuda(),
             keep=torch.full((len(L),), case["keep"], dtype=torch.int32, device="cuda"),
             first=torch.full((len(L),), case["first"], dtype=torch.int32, device="cuda"),
             new_lens=torch.empty(len(L), dtype=torch.int32, device="cuda"))
    _pool(s, ("kc", "vc"), gen, s["pages"] + 1, hkv, PAGE, HEAD)
    # heavy-tailed weights; some tokens were never looked at
    shape = (s["pages"] + 1, hkv, PAGE)
    s["scores"] = torch.randn(shape, generator=gen, device="cuda").mul_(2.0).exp_().mul_(1e-3)
    s["scores"].mul_((torch.rand(shape, generator=gen, device="cuda") > 0.1).float())
    return s


# ---- one pass -----------------------------------------------------------------


def run(s):
    if own:
        return {"axes": _own_axes, "weigh": _own_weigh, "evict": _own_evict}[s["op"]](s)
    return {"axes": _plain_axes, "weigh": _plain_weigh, "evict": _plain_evict}[s["op"]](s)


def _outputs(s, names):
    """The pools as values, 8-bit ones with their scale bytes."""
    NB = s["pages"]
    if not s["fp8"]:
        return tuple(s[name][:NB] for name in names)
    return tuple(s[name][:NB].view(torch.float8_e4m3fn) for name in names) + tuple(s[name + "_scale"][:NB] for name in names)


def _own_axes(s):
    import paged_kv_cache_pkv_gb300 as pkv
    NB = s["pages"]
    if s["fp8"]:
        q = pkv.write_rope_axes_fp8(s["k"], s["v"], s["positions"], s["axes"], s["cos_sin"], s["slots"], s["kc"][:NB],
                                    s["vc"][:NB], s["kc_scale"][:NB], s["vc_scale"][:NB], q=s["q"], q_out=s["q_out"],
                                    interleaved=s["interleaved"])
    else:
        q = pkv.write_rope_axes(s["k"], s["v"], s["positions"], s["axes"], s["cos_sin"], s["slots"], s["kc"][:NB],
                                s["vc"][:NB], q=s["q"], q_out=s["q_out"], interleaved=s["interleaved"])
    return (q,) + _outputs(s, ("kc", "vc"))


def _own_weigh(s):
    import paged_kv_cache_pkv_gb300 as pkv
    NB = s["pages"]
    if "workspace" not in s:  # made once, kept beside the pool
        desc = pkv.make_desc(s["kc"][:NB], s["q"].shape[1], s["tables"].shape[1])
        size = pkv.workspace_size_weigh(desc, s["lens"].shape[0], s["q"].shape[0], max_query_len=s["most"], num_keys=s["keys"])
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    more = dict(decay=s["decay"], first=s["first"], workspace=s["workspace"], max_query_len=s["most"], num_keys=s["keys"])
    if s["fp8"]:
        pkv.weigh_fp8(s["q"], s["kc"][:NB], s["kc_scale"][:NB], s["scores"][:NB], s["tables"], s["lens"], s["qsl"],
                      s["scale"], **more)
    else:
        pkv.weigh(s["q"], s["kc"][:NB], s["scores"][:NB], s["tables"], s["lens"], s["qsl"], s["scale"], **more)
    return s["scores"][:NB]


def _own_evict(s):
    import paged_kv_cache_pkv_gb300 as pkv
    NB = s["pages"]
    if "workspace" not in s:
        desc = pkv.make_desc(s["kc"][:NB], s["kc"].shape[1], s["tables"].shape[1])
        size = pkv.workspace_size_evict(desc, s["lens"].shape[0])
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    more = dict(first=s["first"], recent=s["recent"], new_lens=s["new_lens"], workspace=s["workspace"])
    if s["fp8"]:
        new = pkv.evict_fp8(s["kc"][:NB], s["vc"][:NB], s["kc_scale"][:NB], s["vc_scale"][:NB], s["scores"][:NB],
                            s["tables"], s["lens"], s["keep"], **more)
    else:
        new = pkv.evict(s["kc"][:NB], s["vc"][:NB], s["scores"][:NB], s["tables"], s["lens"], s["keep"], **more)
    return (new, s["scores"][:NB]) + _outputs(s, ("kc", "vc"))


def _rotate(s, x):
    """x [T, heads, D] with its first cos_sin.shape[1] elements rotated, pair i by the position of its axis, fp32."""
    x = x.float()
    half = s["cos_sin"].shape[1] // 2
    pos = s["positions"][s["axis_of"]].t()                       # [T, half]
    pair = torch.arange(half, device="cuda")
    cos, sin = s["cos_sin"][pos, pair][:, None], s["cos_sin"][pos, half + pair][:, None]
    if s["interleaved"]:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([turned, x[..., 2 * half:]], dim=-1)


def _encode(x):
    """(E4M3 codes as bytes, scale bytes) of fp32 rows x [..., D]: the smallest power of two under which |x| <= 448."""
    top = x.abs().amax(dim=-1)
    mant, exp = torch.frexp(top)  # top = mant * 2^exp, mant in [0.5, 1)
    e = exp - 9 + (mant > 0.875)
    e = torch.where(top == 0, -126, e).clamp(-126, 127).int()
    inverse = ((127 - e) << 23).view(torch.float32)  # 2^-e by its bits
    return (x * inverse[..., None]).to(torch.float8_e4m3fn).view(torch.uint8), (e + 127).to(torch.uint8)


def _plain_axes(s):
    slot = torch.where(s["slots"] < 0, s["pages"] * PAGE, s["slots"])
    page, row = slot // PAGE, slot % PAGE
    s["q_out"].copy_(_rotate(s, s["q"]))
    k, v = _rotate(s, s["k"]), s["v"]
    for name, x in (("kc", k), ("vc", v)):
        if s["fp8"]:
            s[name][page, :, row], s[name + "_scale"][page, :, row] = _encode(x.float())
        else:
            s[name][page, :, row] = x.to(torch.bfloat16)
    return (s["q_out"],) + _outputs(s, ("kc", "vc"))


def _keys(s, who, pos):
    """K of positions pos of sequences `who`, fp32 [b, Hkv, keys, D]; pages of unused table entries are the spare one."""
    page, row = s["tables"][who][:, pos // PAGE].long(), (pos % PAGE).expand(len(who), -1)
    k = s["kc"][page, :, row].permute(0, 2, 1, 3)
    if not s["fp8"]:
        return k.float()
    scale = s["kc_scale"][page, :, row].permute(0, 2, 1).float()
    return k.contiguous().view(torch.float8_e4m3fn).float() * torch.exp2(scale - 127.0)[..., None]


def _plain_weigh(s):
    hkv, hq = s["kc"].shape[1], s["q"].shape[1]
    G = hq // hkv
    for n, most, who, rows in s["groups"]:
        b = len(who)
        pos = torch.arange(most, device="cuda")
        k = _keys(s, who, pos)
        w = torch.zeros(b, hkv, most, device="cuda")
        step = max(1, (1 << 28) // (b * hq * most))
        for j in range(0, n, step):  # few rows at a time bound the scores' memory
            m = min(n, j + step) - j
            q = s["q"][rows[:, j:j + m]].float().view(b, m, hkv, G, HEAD).permute(0, 2, 1, 3, 4).reshape(b, hkv, m * G, HEAD)
            score = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"]).view(b, hkv, m, G, most)
            last = s["lens"][who].long()[:, None] - n + torch.arange(j, j + m, device="cuda")  # last key a row sees
            score.masked_fill_((pos > last[..., None])[:, None, :, None], -math.inf)
            p = score.sub_(score.amax(dim=-1, keepdim=True)).exp_()
            p.div_(p.sum(dim=-1, keepdim=True))
            w += p.sum(dim=(2, 3))
        L = s["lens"][who].long()[:, None]
        counted = (pos < L) & (pos >= s["first"][who].long()[:, None])
        page = torch.where(counted, s["tables"][who][:, pos // PAGE].long(), s["pages"])
        row = (pos % PAGE).expand(b, -1)
        old = s["scores"][page, :, row].permute(0, 2, 1) * s["decay"]
        if s["decay"] != 0.0:  # this step's own tokens have none
            w += torch.where((pos < L - n)[:, None], old, 0.0)
        s["scores"][page, :, row] = w.permute(0, 2, 1)
    return s["scores"][:s["pages"]]


def _plain_evict(s):
    hkv, most, kept = s["kc"].shape[1], s["most"], s["most_kept"]
    B = len(s["lens"])
    L, keep = s["lens"].long()[:, None], s["keep"].long()[:, None]
    first = torch.minimum(s["first"].long()[:, None], keep)
    recent = (keep - first).clamp(max=s["recent"])
    pos = torch.arange(most, device="cuda")
    page = s["tables"][:, pos // PAGE].long()
    row = (pos % PAGE).expand(B, -1)
    score = s["scores"][page, :, row].permute(0, 2, 1)                          # [B, Hkv, most]
    score = score.masked_fill(((pos < first) | (pos >= L - recent))[:, None], math.inf)
    score = score.masked_fill((pos >= L)[:, None], -math.inf)
    rank = torch.sort(score, dim=-1, descending=True, stable=True).indices     # ties: the lowest token first
    chosen = torch.zeros(B, hkv, most, dtype=torch.bool, device="cuda")
    chosen.scatter_(2, rank, (pos < torch.minimum(keep, L))[:, None].expand(B, hkv, most))
    src = torch.sort((~chosen).to(torch.uint8), dim=-1, stable=True).indices[..., :kept]  # kept tokens in their order
    dst = torch.arange(kept, device="cuda").expand(B, hkv, kept)
    live = dst < torch.minimum(keep, L)[:, None]
    head = torch.arange(hkv, device="cuda")[:, None]

    def place(token):  # row of the pools [pages * Hkv * 16, ...]; what is not kept goes to the spare page
        p = torch.gather(s["tables"].long()[:, None].expand(B, hkv, -1), 2, token // PAGE)
        p = torch.where(live, p, s["pages"])
        return ((p * hkv + head) * PAGE + token % PAGE).flatten()

    src, dst = place(src), place(dst)
    for name in ("kc", "vc", "scores") + (("kc_scale", "vc_scale") if s["fp8"] else ()):
        x = s[name].view(-1, HEAD) if s[name].dim() == 4 else s[name].view(-1)
        x[dst] = x[src]
    s["new_lens"].copy_(torch.minimum(keep, L)[:, 0])
    return (s["new_lens"], s["scores"][:s["pages"]]) + _outputs(s, ("kc", "vc"))


# ---- cost and definition ------------------------------------------------------


def work(case):
    row = HEAD + 1 if case["fp8"] else 2 * HEAD  # a cached row of K or of V
    hkv = case["hkv"]
    if case["op"] == "axes":
        T = case["tokens"]
        live = T - min(T, case["padded"])
        return {"bytes": T * (8 * case["axes"] + 8 + case["hq"] * HEAD * 4) + live * 2 * hkv * (2 * HEAD + row)
                + min(T, case["max_pos"]) * case["rot"] * 4,
                "flops": 3 * case["rot"] * (T * case["hq"] + live * hkv)}
    L, n = _lengths(case)
    pages = int((-(-L // PAGE)).sum())
    if case["op"] == "weigh":
        pairs = int((n * L - n * (n - 1) // 2).sum())
        scored = np.maximum(L - case["first"], 0)
        read = np.maximum(L - n - case["first"], 0) if case["decay"] else 0 * L
        return {"bytes": int(L.sum()) * hkv * row + int(n.sum()) * case["hq"] * HEAD * 2
                + int((scored + read).sum()) * hkv * 4 + pages * 4,
                "flops": pairs * case["hq"] * 2 * HEAD}
    cut = L > case["keep"]
    moved = int(cut.sum()) * (case["keep"] - min(case["first"], case["keep"]))
    return {"bytes": int(L[cut].sum()) * hkv * 4 + moved * hkv * (4 * row + 8) + pages * 4, "flops": 0}


def exact(case, seed):
    """What run() returns, from the definition in 64 bits."""
    s = prepare(case, seed)
    return {"axes": _exact_axes, "weigh": _exact_weigh, "evict": _exact_evict}[case["op"]](s)


def _turn(s, x, rounded=lambda x: x):
    """x [T, heads, D] with each pair turned by its axis's position, pair by pair, in 64 bits."""
    x = x.double()
    out = x.clone()
    half = s["cos_sin"].shape[1] // 2
    for i, axis in enumerate(s["axes"]):
        c = s["cos_sin"][s["positions"][axis], i].double()[:, None]
        d = s["cos_sin"][s["positions"][axis], half + i].double()[:, None]
        j, k = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + half)
        out[..., j] = rounded(rounded(x[..., j] * c) - rounded(x[..., k] * d))
        out[..., k] = rounded(rounded(x[..., k] * c) + rounded(x[..., j] * d))
    return out


def _exact_axes(s):
    live = torch.nonzero(s["slots"] >= 0)[:, 0]
    page, row = torch.div(s["slots"][live], PAGE, rounding_mode="floor"), s["slots"][live] % PAGE
    NB, q, v = s["pages"], _turn(s, s["q"]), s["v"][live].double()
    if not s["fp8"]:
        kc, vc = s["kc"][:NB].double(), s["vc"][:NB].double()
        kc[page, :, row], vc[page, :, row] = _turn(s, s["k"])[live], v
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


def _exact_weigh(s):
    lens, qsl, first = s["lens"].tolist(), s["qsl"].tolist(), s["first"].tolist()
    hkv, hq = s["kc"].shape[1], s["q"].shape[1]
    scores = s["scores"][:s["pages"]].double()
    for b, L in enumerate(lens):
        pages = s["tables"][b, :-(-L // PAGE)].long()
        n = qsl[b + 1] - qsl[b]
        if s["fp8"]:
            kv = s["kc"][pages].view(torch.float8_e4m3fn).double() * torch.exp2(s["kc_scale"][pages].double() - 127)[..., None]
        else:
            kv = s["kc"][pages].double()
        kv = kv.transpose(0, 1).reshape(hkv, -1, HEAD)[:, :L].repeat_interleave(hq // hkv, dim=0)  # a copy a query head
        total = torch.zeros(hq, L, device="cuda", dtype=torch.float64)
        for j in range(0, n, 256):  # few rows at a time bound the scores' memory
            m = min(n, j + 256) - j
            q = s["q"][qsl[b] + j:qsl[b] + j + m].double().transpose(0, 1)
            hidden = torch.arange(L, device="cuda") > L - n + torch.arange(j, j + m, device="cuda")[:, None]
            logits = torch.einsum("hqd,hkd->hqk", q, kv) * s["scale"]
            total += torch.softmax(logits.masked_fill(hidden, -math.inf), dim=-1).sum(dim=1)
        total = total.view(hkv, hq // hkv, L).sum(dim=1)
        token = torch.arange(L, device="cuda")
        page, row = pages[token // PAGE], token % PAGE
        if s["decay"]:
            earlier = (token < L - n).double()[:, None]
            total += (scores[page, :, row] * earlier * s["decay"]).t()
        on = token >= first[b]
        scores[page[on], :, row[on]] = total.t()[on]
    return scores


def _exact_evict(s):
    names = ("kc", "vc") + (("kc_scale", "vc_scale") if s["fp8"] else ())
    old = {name: s[name][:s["pages"]] for name in names + ("scores",)}
    new = {name: x.clone() for name, x in old.items()}
    lens = s["lens"].clone()
    for b, L in enumerate(s["lens"].tolist()):
        m = int(s["keep"][b])
        if L <= m:
            continue
        lens[b] = m
        f = min(int(s["first"][b]), m)
        r = min(s["recent"], m - f)
        token = torch.arange(L, device="cuda")
        page, row = s["tables"][b].long()[token // PAGE], token % PAGE
        for h in range(old["kc"].shape[1]):
            middle = old["scores"][page, h, row].double()[f:L - r]
            best = torch.argsort(-middle, stable=True)[:m - f - r] + f
            src = torch.cat([token[:f], torch.sort(best).values, token[L - r:]])
            for name, x in old.items():
                new[name][page[:m], h, row[:m]] = x[page[src], h, row[src]]
    values = lambda x: x.view(torch.float8_e4m3fn) if s["fp8"] else x
    return (lens, new["scores"].double(), values(new["kc"]).double(), values(new["vc"]).double()) \
        + tuple(new[name] for name in names[2:])
