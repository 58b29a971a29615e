"""The serving and position operators beside the attention kernels, in plain form and as the library's calls.

Four kinds of case:

* ``rotary``  rotary positions with several axes on q and k; a training case also takes the gradients.
* ``write``   new keys and values quantised into the pages of an 8-bit cache, and read back dequantised.
* ``attend``  attention of the newest tokens of many sequences over such a cache.
* ``pages``   what a server does with the pages: fork sequences, free and admit them, compact the pool.

An 8-bit cache holds codes (e4m3 or int8) in pages of ``page`` tokens, [layers, pages, Hkv, page, D], with one scale
for each page and head, always a power of two: the smallest 2^e whose largest code reaches the page's largest
magnitude. ``page_table`` [slots, pages of a slot] names a sequence's pages, ``seq_lens`` its tokens, ``ref_counts``
how many sequences hold a page (0: free). Pages are handed out lowest first.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
MOST_CODE = {"e4m3": 448.0, "int8": 127.0}
CODE_TYPE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
MIN_EXP = -120  # the smallest scale is 2^-120: a page of zeros has it


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one short chat being answered, token by token: nothing but latency
        dict(name="attend one short", kind="attend", n=1, lo=777, hi=777, q_len=1, Hq=16, Hkv=4, D=128, page=64,
             code="e4m3", mask="causal", sink=0, window=0, cap=0.0, alibi=False, shape_seed=1),
        # an ordinary server batch, ragged lengths
        dict(name="attend ragged batch", kind="attend", n=64, lo=1, hi=16384, q_len=1, Hq=32, Hkv=8, D=128, page=64,
             code="e4m3", mask="causal", sink=0, window=0, cap=0.0, alibi=False, shape_seed=2),
        # endless streams: 4 first tokens and the last 1024 of 32k stay visible
        dict(name="attend sinks and window", kind="attend", n=64, lo=900, hi=32768, q_len=1, Hq=32, Hkv=8, D=128,
             page=16, code="int8", mask="stream", sink=4, window=1024, cap=0.0, alibi=False, shape_seed=3),
        # long contexts, four drafted tokens a sequence to be verified at once, capped scores
        dict(name="attend long drafted", kind="attend", n=24, lo=8192, hi=65536, q_len=4, Hq=32, Hkv=8, D=128, page=128,
             code="e4m3", mask="causal", sink=0, window=0, cap=30.0, alibi=False, shape_seed=4),
        # one new token of each of 200 sequences
        dict(name="write one token each", kind="write", n=200, lo=1, hi=2048, new_lo=1, new_hi=1, Hkv=8, D=128, page=64,
             code="e4m3", layers=1, shape_seed=5),
        # prompts of many lengths that arrive together, behind what their sequences hold already
        dict(name="write prompts", kind="write", n=24, lo=0, hi=300, new_lo=1, new_hi=4000, Hkv=8, D=128, page=64,
             code="int8", layers=1, shape_seed=6),
        # decoding: a token of each sequence, text positions on three axes
        dict(name="rotate one token each", kind="rotary", train=False, B=0, T=48, Hq=32, Hkv=8, D=128, axes=3,
             interleaved=False, far=200000, shape_seed=7),
        # packed prompts with images and video among the text
        dict(name="rotate packed prompts", kind="rotary", train=False, B=0, T=30011, Hq=32, Hkv=8, D=128, axes=3,
             interleaved=False, far=32768, shape_seed=8),
        # a training step's rotation and its gradient, heads before tokens
        dict(name="rotate and gradients", kind="rotary", train=True, B=4, T=8192, Hq=16, Hkv=4, D=128, axes=3,
             interleaved=False, far=8192, shape_seed=9),
        # eight continuations of each of eight prompts: the old ones go, new ones fork
        dict(name="fork 64", kind="pages", what="fork", n=8, each=8, lo=300, hi=4000, Hkv=8, D=128, page=64,
             code="e4m3", layers=4, spare=64, shape_seed=10),
        # finished sequences leave, new ones are admitted
        dict(name="free and admit", kind="pages", what="turn", n=256, each=4, lo=1, hi=4096, Hkv=2, D=64, page=16,
             code="e4m3", layers=1, spare=500, shape_seed=11),
        # half of a pool was freed: the rest moves to its front
        dict(name="compact half", kind="pages", what="compact", n=96, each=2, lo=100, hi=4096, Hkv=8, D=128, page=64,
             code="e4m3", layers=8, spare=100, shape_seed=12),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    kind = rng.choice(["attend", "attend", "write", "rotary", "pages"])
    seed = rng.randrange(1 << 30)
    code, D = rng.choice(["e4m3", "int8"]), rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128])
    if kind == "attend":
        Hkv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 3, 4, 7, 8, 16])
        n, hi = log_int(1, 200), log_int(1, 40000)
        n = max(1, min(n, 1_000_000 // hi))
        mask = rng.choice(["causal", "stream"])
        return dict(kind=kind, n=n, lo=rng.choice([0, 1, hi // 2]), hi=hi, q_len=rng.choice([1, 1, 2, 5, 9]),
                    Hq=Hkv * group, Hkv=Hkv, D=D, page=page, code=code, mask=mask,
                    sink=rng.randrange(0, 40) if mask == "stream" else 0,
                    window=log_int(1, 4096) if mask == "stream" else 0, cap=rng.choice([0.0, 30.0]),
                    alibi=rng.random() < 0.3, shape_seed=seed)
    if kind == "write":
        new_hi = log_int(1, 5000)
        n = max(1, min(log_int(1, 300), 60000 // new_hi))
        return dict(kind=kind, n=n, lo=0, hi=log_int(1, 3000), new_lo=rng.choice([0, 1, new_hi]), new_hi=new_hi,
                    Hkv=rng.choice([1, 2, 5, 8]), D=D, page=page, code=code, layers=rng.choice([1, 2]),
                    shape_seed=seed)
    if kind == "rotary":
        B = rng.choice([0, 0, 1, 3])
        T = log_int(1, 30000 // max(1, B))
        Hkv = rng.choice([1, 4, 8])
        return dict(kind=kind, train=rng.random() < 0.5, B=B, T=T, Hq=Hkv * rng.choice([1, 4]), Hkv=Hkv, D=D,
                    axes=rng.choice([1, 2, 3]), interleaved=rng.random() < 0.5, far=log_int(10, 1000000),
                    shape_seed=seed)
    what = rng.choice(["fork", "turn", "compact"])
    return dict(kind=kind, what=what, n=log_int(5, 60), each=rng.randrange(2 if what == "turn" else 1, 5),
                lo=rng.choice([0, 1, 50]), hi=log_int(60, 3000), Hkv=rng.choice([1, 2, 8]), D=D, page=page, code=code,
                layers=rng.choice([1, 3]), spare=rng.randrange(70, 300), shape_seed=seed)


def spread(case, lo, hi, n, salt=0):
    """n lengths between lo and hi, the largest among them: the case's own, whatever the inputs' seed."""
    r = random.Random(case["shape_seed"] * 8 + salt)
    got = [r.randint(lo, hi) for _ in range(n)]
    got[r.randrange(n)] = hi
    return got


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def running(counts):
    return [0] + list(np.cumsum(counts).tolist())


# ------------------------------------------------------------------ inputs
def codes_like(shape, code, gen):
    """Codes of normal values whose page scale lets them use the code's range."""
    out = torch.empty(shape, dtype=CODE_TYPE[code], device=DEV)
    flat = out.view(-1)
    for at in range(0, flat.numel(), 1 << 27):
        some = torch.randn(min(1 << 27, flat.numel() - at), device=DEV, generator=gen)
        some = (some * (MOST_CODE[code] / 5)).clamp_(-MOST_CODE[code], MOST_CODE[code])
        flat[at:at + some.numel()] = (some.round_() if code == "int8" else some).to(out.dtype)
    return out


def make_cache(case, lens, slots, spare, gen, room=0):
    """A cache that holds `lens` tokens in slots 0.., its pages in random places of the pool. `room`: more slots' pages."""
    P, Hkv, D, code, layers = case["page"], case["Hkv"], case["D"], case["code"], case.get("layers", 1)
    held = [-(-x // P) for x in lens]
    pages = sum(held) + spare
    wide = max(1, max(held) + room)
    order = torch.randperm(pages, device=DEV, generator=gen).to(torch.int32)
    table = torch.full((slots, wide), -1, dtype=torch.int32, device=DEV)
    row = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(held)).to(DEV)
    first = torch.tensor(running(held)[:-1], dtype=torch.int64)
    col = (torch.arange(sum(held)) - torch.repeat_interleave(first, torch.tensor(held))).to(DEV)
    table[row, col] = order[:sum(held)]
    refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
    refs[order[:sum(held)].long()] = 1
    seq_lens = torch.zeros(slots, dtype=torch.int32, device=DEV)
    seq_lens[:len(lens)] = ints(lens)
    shape = (layers, pages, Hkv, P, D)
    s = dict(k=codes_like(shape, code, gen), v=codes_like(shape, code, gen), page_table=table, seq_lens=seq_lens,
             ref_counts=refs)
    base = -7 if code == "e4m3" else -5
    for name in ("k_scale", "v_scale"):
        e = torch.randint(base - 1, base + 2, shape[:3], device=DEV, generator=gen)
        s[name] = torch.ldexp(torch.ones(shape[:3], device=DEV), e)
    return s


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return {"attend": prepare_attend, "write": prepare_write, "rotary": prepare_rotary,
            "pages": prepare_pages}[case["kind"]](case, gen)


def bf16(shape, gen):
    return torch.randn(shape, device=DEV, generator=gen, dtype=torch.bfloat16)


def query_lens(case, lens):
    """A sequence's newest tokens that are queries: all of q_len, or what it has."""
    return [min(case["q_len"], max(x, 1)) for x in lens]


def prepare_attend(case, gen):
    lens = spread(case, case["lo"], case["hi"], case["n"])
    s = dict(case=case, cache=make_cache(case, lens, case["n"], 3, gen))
    s["seqs"] = torch.randperm(case["n"], device=DEV, generator=gen).to(torch.int32)  # the batch's order is not the slots'
    got = np.array(query_lens(case, lens))[s["seqs"].cpu().numpy()]
    s["cu"] = ints(running(got)) if case["q_len"] > 1 else None
    s["q"] = bf16((int(got.sum()), case["Hq"], case["D"]), gen)
    return s


def prepare_write(case, gen):
    lens = spread(case, case["lo"], case["hi"], case["n"])
    new = spread(case, case["new_lo"], case["new_hi"], case["n"], 1)
    total = [a + b for a, b in zip(lens, new)]  # extended already: the new tokens' places are there, not their values
    s = dict(case=case, cache=make_cache(case, total, case["n"], 3, gen), seqs=ints(list(range(case["n"]))),
             starts=ints(lens))
    s["cu"] = None if case["new_hi"] == 1 and case["new_lo"] == 1 else ints(running(new))
    both = bf16((sum(new), 2, case["Hkv"], case["D"]), gen)  # as one projection gives them
    s["k"], s["v"] = both[:, 0], both[:, 1]
    s["layer"] = case["layers"] - 1
    return s


def sections_of(case):
    pairs, axes = case["D"] // 2, case["axes"]
    some = [pairs * 3 // 8] * (axes - 1)
    return [pairs - sum(some)] + some


def prepare_rotary(case, gen):
    B, T, D = case["B"], case["T"], case["D"]
    shape = (lambda H: (B, H, T, D)) if B else (lambda H: (T, H, D))
    s = dict(case=case, sections=sections_of(case), positions=torch.randint(
        0, case["far"], (case["axes"], B, T) if B else (case["axes"], T), device=DEV, generator=gen, dtype=torch.int32))
    s["q"], s["k"] = bf16(shape(case["Hq"]), gen), bf16(shape(case["Hkv"]), gen)
    if case["train"]:
        s["q"].requires_grad_()
        s["k"].requires_grad_()
        s["dq"], s["dk"] = bf16(shape(case["Hq"]), gen), bf16(shape(case["Hkv"]), gen)
    return s


def prepare_pages(case, gen):
    n, each = case["n"], case["each"]
    if case["what"] == "fork":
        lens = spread(case, case["lo"], case["hi"], n)
        s = dict(case=case, cache=make_cache(case, lens, n + n * each, case["spare"] + n * each, gen))
        s["src"] = ints([i for i in range(n) for _ in range(each)])
        s["dst"] = ints([n + i for i in range(n * each)])
        return s
    if case["what"] == "turn":
        lens, new = spread(case, case["lo"], case["hi"], n), spread(case, case["lo"], case["hi"], n, 1)
        most = max(max(lens), max(new))
        gone = list(range(0, n, each))
        need = sum(-(-new[i] // case["page"]) for i in gone)
        s = dict(case=case, cache=make_cache(case, lens, n, case["spare"] + need, gen, room=-(-most // case["page"])))
        s["seqs"], s["counts"] = ints(gone), ints([new[i] for i in gone])
        return s
    lens = spread(case, case["lo"], case["hi"], n)
    s = dict(case=case, cache=make_cache(case, lens, n, case["spare"], gen))
    c = s["cache"]
    if each > 1:  # every each-th sequence left, so that its pages are holes
        refs = torch.zeros_like(c["ref_counts"])
        c["page_table"][::each] = -1
        c["seq_lens"][::each] = 0
        refs[c["page_table"][c["page_table"] >= 0].long()] = 1
        c["ref_counts"] = refs
    s["table_before"], s["refs_before"] = c["page_table"].clone(), c["ref_counts"].clone()
    return s


# ------------------------------------------------------------------ a pass
def run(s):
    return {"attend": run_attend, "write": run_write, "rotary": run_rotary, "pages": run_pages}[s["case"]["kind"]](s)


def cache_of(s):
    import block_sparse_masked_tile_b200 as bsmt
    return bsmt.PagedCache(**s["cache"])


def run_attend(s):
    case = s["case"]
    if own:
        import block_sparse_masked_tile_b200 as bsmt
        mask = bsmt.causal()
        if case["mask"] == "stream":
            mask = bsmt.and_masks(mask, bsmt.or_masks(bsmt.sink(case["sink"]), bsmt.sliding_window(case["window"])))
        mods = [bsmt.softcap(case["cap"])] * (case["cap"] > 0) + [bsmt.alibi()] * case["alibi"]
        return bsmt.paged_attention(s["q"], cache_of(s), s["seqs"], cu_seqlens_q=s["cu"], mask_mod=mask,
                                    score_mod=mods, enable_gqa=True)
    return plain_attend(case, s["cache"], s["q"], s["seqs"].long(), s["cu"])


def run_write(s):
    if own:
        import block_sparse_masked_tile_b200 as bsmt
        cache = cache_of(s)
        bsmt.cache_write(cache, s["seqs"], s["starts"], s["k"], s["v"], cu_seqlens=s["cu"], layer=s["layer"])
        k, v = bsmt.cache_gather(cache, s["seqs"], s["starts"], s["k"].shape[0], cu_seqlens=s["cu"], layer=s["layer"])
    else:
        k, v = plain_write(s)
    return k, v, s["cache"]["k_scale"], s["cache"]["v_scale"]


def run_rotary(s):
    case = s["case"]
    if own:
        import block_sparse_masked_tile_b200 as bsmt
        spec = bsmt.rotary_spec(case["D"], s["sections"], interleaved=case["interleaved"])
        q, k = bsmt.rotary(s["q"], s["k"], s["positions"], spec)
        if not case["train"]:
            return q, k
        return q.detach(), k.detach(), *torch.autograd.grad((q, k), (s["q"], s["k"]), (s["dq"], s["dk"]))
    cos, sin = plain_turns(case, s["sections"], s["positions"])
    got = [plain_rotate(s[x].detach(), cos, sin, case["interleaved"]) for x in ("q", "k")]
    if case["train"]:
        got += [plain_rotate(s[x], cos, -sin, case["interleaved"]) for x in ("dq", "dk")]
    return tuple(got)


def run_pages(s):
    case, c = s["case"], s["cache"]
    if own:
        import block_sparse_masked_tile_b200 as bsmt
        cache = cache_of(s)
        if case["what"] == "fork":
            bsmt.cache_free(cache, s["dst"])
            bsmt.cache_fork(cache, s["src"], s["dst"])
        elif case["what"] == "turn":
            bsmt.cache_free(cache, s["seqs"])
            return bsmt.cache_extend(cache, s["seqs"], s["counts"]), c["page_table"], c["seq_lens"], c["ref_counts"]
        else:
            c["page_table"].copy_(s["table_before"])
            c["ref_counts"].copy_(s["refs_before"])
            bsmt.cache_compact(cache)
    elif case["what"] == "fork":
        plain_free(c, s["dst"].long(), case["page"])
        plain_fork(c, s["src"].long(), s["dst"].long(), case["page"])
    elif case["what"] == "turn":
        plain_free(c, s["seqs"].long(), case["page"])
        return plain_extend(c, s["seqs"].long(), s["counts"], case["page"]), c["page_table"], c["seq_lens"], c["ref_counts"]
    else:
        c["page_table"].copy_(s["table_before"])
        c["ref_counts"].copy_(s["refs_before"])
        plain_compact(c, case["page"])
    return c["page_table"], c["seq_lens"], c["ref_counts"], c["k"], c["v"], c["k_scale"], c["v_scale"]


# ------------------------------------------------------------------ plain forms
def plain_turns(case, sections, positions):
    """cos and sin [..., T, D / 2] of position (of the pair's axis) times frequency, the angle in 64 bits."""
    half = case["D"] // 2
    freq = 10000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)
    axis = torch.repeat_interleave(torch.arange(len(sections), device=DEV), torch.tensor(sections, device=DEV))
    angle = positions.double()[axis].movedim(0, -1) * freq
    return angle.cos().float(), angle.sin().float()


def plain_rotate(x, cos, sin, interleaved):
    """(a, b) -> (a cos - b sin, a sin + b cos) for each pair of x, [T, H, D] or [B, H, T, D]."""
    at = -2 if x.dim() == 3 else -3  # the heads
    cos, sin, y = cos.unsqueeze(at), sin.unsqueeze(at), x.float()
    if interleaved:
        a, b = y[..., 0::2], y[..., 1::2]
        return torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2).to(x.dtype)
    a, b = y.chunk(2, -1)
    return torch.cat((a * cos - b * sin, a * sin + b * cos), -1).to(x.dtype)


def plain_scale(largest, code):
    """The smallest power of two whose largest code reaches `largest`."""
    m, e = torch.frexp(largest)
    top_m, top_e = math.frexp(MOST_CODE[code])
    e = torch.where(m <= top_m, e - top_e, e - top_e + 1)
    e = torch.where(largest > 0, e, MIN_EXP).clamp_min(MIN_EXP)
    return torch.ldexp(torch.ones_like(largest), e)


def plain_encode(x, code):
    x = x.clamp(-MOST_CODE[code], MOST_CODE[code])
    return (x.round() if code == "int8" else x).to(CODE_TYPE[code])


def places(s, P):
    """Page [T] and row [T] of each token of a ragged batch, and its sequence."""
    n = s["seqs"].numel()
    T = s["k"].shape[0]
    token = torch.arange(T, device=DEV)
    if s["cu"] is None:
        seg, at = token, s["starts"].long()
    else:
        seg = torch.searchsorted(s["cu"][1:].long(), token, right=True).clamp_max(n - 1)
        at = s["starts"].long()[seg] + token - s["cu"].long()[seg]
    return s["cache"]["page_table"].long()[s["seqs"].long()[seg], at // P], at % P


def plain_write(s):
    case, c, P, layer, code = s["case"], s["cache"], s["case"]["page"], s["layer"], s["case"]["code"]
    page, row = places(s, P)
    pages, Hkv = c["k_scale"].shape[1:]
    # the pages that hold tokens already: the first of a sequence that starts inside one and gets tokens
    starts = s["starts"].long()
    count = torch.ones_like(starts) if s["cu"] is None else s["cu"].long().diff()
    kept_row = starts % P
    kept = (kept_row > 0) & (count > 0)
    kept_page = c["page_table"].long()[s["seqs"].long(), (starts // P).clamp_max(c["page_table"].shape[1] - 1)]
    dummy = torch.where(kept, kept_page, pages)
    written = torch.zeros(pages, dtype=torch.bool, device=DEV).index_fill_(0, page, True)
    found = []
    for name, x in (("k", s["k"].float()), ("v", s["v"].float())):
        codes, scale = c[name][layer], c[name + "_scale"][layer]
        largest = torch.zeros(pages, Hkv, device=DEV).scatter_reduce_(
            0, page[:, None].expand(-1, Hkv), x.abs().amax(-1), "amax")
        held = torch.zeros(pages + 1, Hkv, device=DEV).index_copy_(0, dummy, torch.cat(
            (scale, scale[:1]))[dummy])[:pages]
        new = torch.maximum(plain_scale(largest, code), held)
        # the kept rows under the page's new scale
        safe = kept_page.clamp(0, pages - 1)
        old = codes[safe].float()
        again = plain_encode(old * (scale[safe] / new[safe])[..., None, None], code)
        keep = kept[:, None] & (torch.arange(P, device=DEV) < kept_row[:, None])
        at_seq, at_row = keep.nonzero(as_tuple=True)
        bits = codes.view(torch.int8)
        bits[safe[at_seq], :, at_row] = again.view(torch.int8)[at_seq, :, at_row]
        bits[page, :, row] = plain_encode(x / new[page][..., None], code).view(torch.int8)
        scale.copy_(torch.where(written[:, None], new, scale))
        found.append((codes[page, :, row].float() * scale[page][..., None]).bfloat16())
    return found


def plain_seen(case, at, keys):
    """Which keys (positions) the queries (positions `at`) see."""
    seen = keys <= at
    if case["mask"] == "stream":
        seen = seen & ((keys < case["sink"]) | (at - keys < case["window"]))
    return seen


def plain_attend(case, c, q, seqs, cu):
    n, P, Hkv, D = seqs.numel(), case["page"], case["Hkv"], case["D"]
    G = case["Hq"] // Hkv
    lens = c["seq_lens"].long()[seqs]
    count = torch.ones_like(lens) if cu is None else cu.long().diff()
    first = torch.arange(n, device=DEV) if cu is None else cu.long()[:-1]
    wide = case["q_len"]
    slot = torch.arange(wide, device=DEV)
    there = slot < count[:, None]
    rows = q[(first[:, None] + slot).clamp_max(q.shape[0] - 1)].float().view(n, wide, Hkv, G, D)
    pages = c["page_table"].long()[seqs].clamp_min(0)
    k = (c["k"][0][pages].float() * c["k_scale"][0][pages][..., None, None]).transpose(1, 2).reshape(n, Hkv, -1, D)
    z = torch.einsum("nwhgd,nhkd->nhgwk", rows, k) * D ** -0.5
    del k
    keys = torch.arange(z.shape[-1], device=DEV)
    at = (lens - count)[:, None] + slot
    if case["cap"] > 0:
        z = case["cap"] * torch.tanh(z / case["cap"])
    if case["alibi"]:
        slope = (2.0 ** (-8.0 * torch.arange(1, case["Hq"] + 1, device=DEV) / case["Hq"])).view(Hkv, G, 1, 1)
        z = z + slope * (keys - at[..., None])[:, None, None].float()
    seen = plain_seen(case, at[..., None], keys) & (keys < lens[:, None, None])
    z = z.masked_fill(~seen[:, None, None], -math.inf)
    top = z.amax(-1, keepdim=True).clamp_min(-1e30)
    p = (z - top).exp()
    total = p.sum(-1, keepdim=True)
    lse = (total.log() + top).squeeze(-1)
    v = (c["v"][0][pages].float() * c["v_scale"][0][pages][..., None, None]).transpose(1, 2).reshape(n, Hkv, -1, D)
    out = torch.einsum("nhgwk,nhkd->nwhgd", p / total.clamp_min(1e-30), v)
    at_seq, at_slot = there.nonzero(as_tuple=True)
    out = out.reshape(n, wide, -1, D)[at_seq, at_slot].to(q.dtype)
    return out, lse.reshape(n, -1, wide)[at_seq, :, at_slot].t().contiguous()


def held_pages(c, seqs, P):
    """(row, column) of each page that the sequences hold in the table."""
    held = (c["seq_lens"].long()[seqs] + P - 1) // P
    return (torch.arange(c["page_table"].shape[1], device=DEV) < held[:, None]).nonzero(as_tuple=True)


def plain_free(c, seqs, P):
    row, col = held_pages(c, seqs, P)
    page = c["page_table"][seqs[row], col].long()
    c["ref_counts"].index_add_(0, page, torch.full_like(page, -1, dtype=torch.int32))
    c["page_table"][seqs[row], col] = -1
    c["seq_lens"][seqs] = 0


def plain_extend(c, seqs, counts, P):
    start = c["seq_lens"][seqs]
    have, want = (start + P - 1) // P, (start + counts + P - 1) // P
    col = torch.arange(c["page_table"].shape[1], device=DEV)
    row, at = ((col >= have[:, None]) & (col < want[:, None])).nonzero(as_tuple=True)
    page = (c["ref_counts"] == 0).nonzero().squeeze(1)[:row.numel()]
    c["page_table"][seqs[row], at] = page.int()
    c["ref_counts"][page] = 1
    c["seq_lens"][seqs] = start + counts
    return start


def plain_fork(c, src, dst, P):
    row, col = held_pages(c, src, P)
    lens = c["seq_lens"].long()[src]
    part = lens % P
    own_copy = part[row] > 0
    own_copy &= col == lens[row] // P
    old = c["page_table"][src[row], col].long()
    shared = old[~own_copy]
    c["ref_counts"].index_add_(0, shared, torch.ones_like(shared, dtype=torch.int32))
    page = (c["ref_counts"] == 0).nonzero().squeeze(1)[:int(own_copy.sum())]
    c["ref_counts"][page] = 1
    name = old.clone()
    name[own_copy] = page
    c["page_table"][dst[row], col] = name.int()
    c["seq_lens"][dst] = c["seq_lens"][src]
    was = old[own_copy]
    keep = torch.arange(P, device=DEV) < part[row[own_copy]][:, None]
    k, v = c["k"].view(torch.int8), c["v"].view(torch.int8)
    k[:, page] = torch.where(keep[:, None, :, None], k[:, was], k[:, page])
    v[:, page] = torch.where(keep[:, None, :, None], v[:, was], v[:, page])
    c["k_scale"][:, page] = c["k_scale"][:, was]
    c["v_scale"][:, page] = c["v_scale"][:, was]


def plain_compact(c, P):
    refs = c["ref_counts"]
    live = refs > 0
    count = int(live.sum())
    hole = (~live[:count]).nonzero().squeeze(1)
    mover = live[count:].nonzero().squeeze(1) + count
    to = torch.arange(refs.numel(), device=DEV)
    to[mover] = hole
    row, col = held_pages(c, torch.arange(c["seq_lens"].numel(), device=DEV), P)
    c["page_table"][row, col] = to[c["page_table"][row, col].long()].int()
    k, v = c["k"].view(torch.int8), c["v"].view(torch.int8)
    k[:, hole] = k[:, mover]
    v[:, hole] = v[:, mover]
    c["k_scale"][:, hole] = c["k_scale"][:, mover]
    c["v_scale"][:, hole] = c["v_scale"][:, mover]
    refs[hole] = refs[mover]
    refs[mover] = 0


# ------------------------------------------------------------------ what a pass cannot do without
def seen_keys(case, length, count):
    """Keys that some of the `count` newest tokens of a sequence see, and the (query, key) pairs seen."""
    keys, pairs = 0, 0
    first = max(length - count, 0)
    if case["mask"] == "stream":
        lo = max(first - case["window"] + 1, 0)
        sinks = min(case["sink"], length)
        keys = min(length, sinks + length - max(lo, sinks)) if length else 0
        for at in range(first, length):
            lo = max(at - case["window"] + 1, 0)
            pairs += at + 1 - lo + min(case["sink"], lo)
    else:
        keys = length
        pairs = sum(range(first + 1, length + 1))
    return keys, pairs


def work(case):
    kind, D = case["kind"], case["D"]
    if kind == "attend":
        lens = spread(case, case["lo"], case["hi"], case["n"])
        got = query_lens(case, lens)
        seen = [seen_keys(case, a, b) for a, b in zip(lens, got)]
        rows = sum(got) * case["Hq"]
        keys, pairs = sum(x[0] for x in seen), sum(x[1] for x in seen) * case["Hq"]
        pages = sum(-(-x[0] // case["page"]) for x in seen)
        return {"bytes": keys * case["Hkv"] * D * 2 + pages * (8 * case["Hkv"] + 4) + rows * (4 * D + 4) + case["n"] * 8,
                "flops": pairs * D * 4}
    if kind == "write":
        new = spread(case, case["new_lo"], case["new_hi"], case["n"], 1)
        one = case["Hkv"] * D * 2
        pages = sum(-(-x // case["page"]) + 1 for x in new)
        # k and v: read in bf16, written in 8 bits, read again and given out in bf16
        return {"bytes": sum(new) * one * (2 + 1 + 1 + 2) + pages * (case["Hkv"] * 8 * 2 + 4), "flops": sum(new) * one * 4}
    if kind == "rotary":
        n = max(1, case["B"]) * case["T"]
        one = n * (case["Hq"] + case["Hkv"]) * D
        return {"bytes": (one * 4 + n * case["axes"] * 4) * (2 if case["train"] else 1),
                "flops": one * 3 * (2 if case["train"] else 1)}
    P, n, each = case["page"], case["n"], case["each"]
    one = case["layers"] * case["Hkv"] * D * 2
    lens = spread(case, case["lo"], case["hi"], n)
    if case["what"] == "fork":
        rows = sum(x % P for x in lens) * each
        entries = sum(-(-x // P) for x in lens) * each
        return {"bytes": rows * one * 2 + entries * (4 + 4 + 8 + 4 + 8), "flops": 0}
    if case["what"] == "turn":
        new = spread(case, case["lo"], case["hi"], n, 1)
        entries = sum(-(-lens[i] // P) + -(-new[i] // P) for i in range(0, n, each))
        return {"bytes": entries * 16 + (n // each) * 20, "flops": 0}
    held = [-(-x // P) for x in lens]
    pool = sum(held) + case["spare"]
    live = sum(h for i, h in enumerate(held) if each == 1 or i % each)
    moved = live * (pool - live) / pool  # the live pages behind the first `live` places, on average
    # the bookkeeping: the table and the counts put back, read and written; the pages that move
    return {"bytes": moved * (P * one + case["layers"] * case["Hkv"] * 8) * 2 + live * 16 + pool * 12, "flops": 0}


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    if case["kind"] == "pages":  # moved codes and whole numbers
        return None
    s = prepare(case, seed)
    return {"attend": exact_attend, "write": exact_write, "rotary": exact_rotary}[case["kind"]](case, s)


def exact_rotary(case, s):
    half = case["D"] // 2
    freq = torch.tensor([10000.0 ** (-i / half) for i in range(half)], dtype=torch.float64, device=DEV)
    axis = sum(([a] * m for a, m in enumerate(s["sections"])), [])
    pos = torch.stack([s["positions"][a] for a in axis], -1).double()
    turn = torch.polar(torch.ones_like(pos), pos * freq).unsqueeze(1 if case["B"] else -2)

    def rotate(x, turn):
        x = x.detach().double()
        pair = x.unflatten(-1, (half, 2)) if case["interleaved"] else x.unflatten(-1, (2, half)).transpose(-1, -2)
        y = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
        return (y if case["interleaved"] else y.transpose(-1, -2)).flatten(-2)

    got = [rotate(s["q"], turn), rotate(s["k"], turn)]
    if case["train"]:
        got += [rotate(s["dq"], turn.conj()), rotate(s["dk"], turn.conj())]
    return got


def exact_write(case, s):
    P, code, layer = case["page"], case["code"], s["layer"]
    top = MOST_CODE[code]
    c = {k: v.cpu() for k, v in s["cache"].items() if k in ("page_table", "k_scale", "v_scale")}
    table, starts = c["page_table"].numpy(), s["starts"].cpu().numpy()
    n, T = case["n"], s["k"].shape[0]
    cu = list(range(n + 1)) if s["cu"] is None else s["cu"].cpu().tolist()
    got = []
    for name in ("k", "v"):
        x = s[name].double().cpu().numpy()
        scale = c[name + "_scale"].double().numpy().copy()
        out = np.zeros_like(x)
        for i in range(n):
            t, pos = cu[i], int(starts[i])
            while t < cu[i + 1]:
                m = min(P - pos % P, cu[i + 1] - t)
                page = table[i, pos // P]
                most = np.abs(x[t:t + m]).max((0, 2))
                e = np.ceil(np.log2(np.maximum(most, 2.0 ** -200) / top) - 1e-12)
                e += most > top * 2.0 ** e  # the logarithm's own rounding
                e -= most <= top * 2.0 ** (e - 1)
                new = 2.0 ** np.maximum(e, MIN_EXP)
                if pos % P:
                    new = np.maximum(new, scale[layer, page])
                scale[layer, page] = new
                y = x[t:t + m] / new[None, :, None]
                step = 1.0 if code == "int8" else 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(np.abs(y), 1e-300))), -6) - 3)
                out[t:t + m] = np.clip(np.rint(y / step) * step, -top, top) * new[None, :, None]
                t, pos = t + m, pos + m
        got.append((out, scale))
    return got[0][0], got[1][0], got[0][1], got[1][1]


def exact_attend(case, s):
    c, P, D, Hq = s["cache"], case["page"], case["D"], case["Hq"]
    G = Hq // case["Hkv"]
    seqs, lens = s["seqs"].cpu().tolist(), c["seq_lens"].cpu().tolist()
    cu = list(range(len(seqs) + 1)) if s["cu"] is None else s["cu"].cpu().tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full((Hq, s["q"].shape[0]), -math.inf, dtype=torch.float64, device=DEV)
    slope = torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)], dtype=torch.float64, device=DEV)
    for i, slot in enumerate(seqs):
        L, m = lens[slot], cu[i + 1] - cu[i]
        if L == 0 or m == 0:
            continue
        pages = c["page_table"][slot, :-(-L // P)].long()
        k, v = ((c[x][0][pages].double() * c[x + "_scale"][0][pages].double()[:, :, None, None]).transpose(0, 1)
                .flatten(1, 2)[:, :L] for x in ("k", "v"))
        q = s["q"][cu[i]:cu[i + 1]].double().transpose(0, 1).unflatten(0, (-1, G))  # [Hkv, G, m, D]
        z = (q.flatten(1, 2) @ k.transpose(1, 2)).unflatten(1, (G, m)).flatten(0, 1) / math.sqrt(D)
        at = torch.arange(L - m, L, device=DEV)[:, None]
        key = torch.arange(L, device=DEV)[None]
        if case["cap"] > 0:
            z = case["cap"] * torch.tanh(z / case["cap"])
        if case["alibi"]:
            z = z + slope[:, None, None] * (key - at)
        hidden = key > at
        if case["mask"] == "stream":
            hidden = hidden | ((key >= case["sink"]) & (key <= at - case["window"]))
        z = z.masked_fill(hidden, -math.inf)
        total = torch.logsumexp(z, -1)
        p = torch.exp(z - torch.where(total.isinf(), 0.0, total)[..., None])
        out[cu[i]:cu[i + 1]] = (p.unflatten(0, (-1, G)).flatten(1, 2) @ v).unflatten(1, (G, m)).flatten(0, 1).transpose(0, 1)
        lse[:, cu[i]:cu[i + 1]] = total
    return out, lse
