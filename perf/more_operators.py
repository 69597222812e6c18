"""Workloads of the operators for image, video and document prompts: the rotation by several
position axes (forward and backward, and with the append to a paged cache), attention whose
scores are capped, biased by distance or open over a prefix (packed, with its backward, and
over a paged cache), and the page tables and slots of a serving step, made on the device.

``run`` has two forms of each.  The plain one is elementary torch arithmetic in binary32,
rounded once to bf16 at the end; the other calls the library.  ``exact`` evaluates the
definitions in binary64 (the tables in Python integers).
"""
import math
import random

import numpy as np
import torch

own = False

MAX_ELEMS = 1 << 28      # values drawn at a time, so that a large buffer needs no binary32 copy of itself


# ---------------------------------------------------------------------------- the cases

def listed():
    return [
        # one decoding step of a batch whose prompts held images: rotate by three axes, append; latency counts
        {"name": "axes-append-8", "op": "append", "n": 8, "new_lo": 1, "new_hi": 1, "ctx_lo": 100, "ctx_hi": 4000,
         "hq": 32, "hkv": 8, "d": 128, "page": 64, "theta": 1.0e6, "sections": "16,24,24", "interleaved": False,
         "own_w": False, "wide": False, "lens": 21},
        # a prefill chunk of text and images from several prompts, a large model's heads, axes taking turns
        {"name": "axes-append-16k", "op": "append", "n": 12, "new_lo": 900, "new_hi": 1900, "ctx_lo": 0, "ctx_hi": 8000,
         "hq": 64, "hkv": 8, "d": 128, "page": 64, "theta": 1.0e6, "sections": "24,20,20", "interleaved": True,
         "own_w": False, "wide": True, "lens": 22},
        # patches of a few images in an image encoder: two axes with frequencies of their own, heads of 80, odd count
        {"name": "axes-patches-odd", "op": "axes", "pack": "1036,2520,187,777", "hq": 16, "hkv": 16, "d": 80,
         "theta": 1.0e4, "sections": "20,20", "interleaved": False, "own_w": True, "wide": True, "train": False, "lens": 23},
        # a training step's rotations of a packed batch with images among the text
        {"name": "axes-train-16k", "op": "axes", "pack": "16384:0.8:32:512:2048:8192", "hq": 32, "hkv": 8, "d": 128,
         "theta": 1.0e6, "sections": "16,24,24", "interleaved": False, "own_w": False, "wide": False, "train": True,
         "lens": 24},
        # a decoding step of 64 conversations: most need no new page, a few have ended
        {"name": "tables-decode-64", "op": "tables", "n": 64, "new_lo": 1, "new_hi": 1, "ctx_lo": 500, "ctx_hi": 16000,
         "page": 64, "ended": 0.05, "spare": 64, "lens": 25},
        # a large server's step: chunks of many prompts at once
        {"name": "tables-chunks-4096", "op": "tables", "n": 4096, "new_lo": 0, "new_hi": 512, "ctx_lo": 0, "ctx_hi": 8000,
         "page": 16, "ended": 0.1, "spare": 4096, "lens": 26},
        # four samples of 5 to 33 tokens, capped scores: the smallest pack
        {"name": "fwd-cap-tiny", "op": "fwd", "pack": "5,17,33,9", "hq": 4, "hkv": 2, "d": 64, "cap": 50.0,
         "slopes": False, "prefix": False, "causal": True, "used": False, "lens": 27},
        # the packed fine-tuning batch, 16,384 tokens, scores biased by distance, as evaluation runs it
        {"name": "fwd-slopes-16k", "op": "fwd", "pack": "16384:0.8:32:512:2048:8192", "hq": 32, "hkv": 32, "d": 64,
         "cap": 0.0, "slopes": True, "prefix": False, "causal": True, "used": False, "lens": 28},
        # an attention layer of a training step on the packed fine-tuning batch, capped scores
        {"name": "train-cap-16k", "op": "train", "pack": "16384:0.8:32:512:2048:8192", "hq": 32, "hkv": 8, "d": 128,
         "cap": 50.0, "slopes": False, "prefix": False, "causal": True, "used": False, "lens": 29},
        # odd shapes in training: prefixes that all rows see, distance bias and cap, padded rows, heads of 80
        {"name": "train-prefix-odd", "op": "train", "pack": "1,777,130,0,2051,63,500", "hq": 10, "hkv": 2, "d": 80,
         "cap": 30.0, "slopes": True, "prefix": True, "causal": True, "used": True, "lens": 30},
        # a serving batch: one token each of 64 conversations of uneven length, capped scores
        {"name": "paged-cap-64", "op": "paged", "n": 64, "new_lo": 1, "new_hi": 1, "ctx_lo": 500, "ctx_hi": 16000,
         "hq": 32, "hkv": 8, "d": 128, "page": 64, "cap": 50.0, "slopes": False, "prefix": False, "lens": 31},
        # chunked prefill of long prompts that open with an image or a document which all rows see
        {"name": "paged-prefix-4x2k", "op": "paged", "n": 4, "new_lo": 1500, "new_hi": 2048, "ctx_lo": 0, "ctx_hi": 8000,
         "hq": 16, "hkv": 4, "d": 128, "page": 128, "cap": 0.0, "slopes": False, "prefix": True, "lens": 32},
    ]


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw_lengths(rng, case, decode_most):
    """New and cached tokens of a serving step: one token each, a few, or chunks of prompts."""
    kind = rng.choice(["decode", "draft", "chunk"])
    if kind == "decode":
        case.update(n=log_int(rng, 1, decode_most), new_lo=1, new_hi=1)
    elif kind == "draft":
        case.update(n=log_int(rng, 1, 32), new_lo=1, new_hi=rng.randrange(2, 17))
    else:
        hi = log_int(rng, 17, 2048)
        case.update(n=rng.randrange(1, 5), new_lo=max(1, hi // 2), new_hi=hi)
    ctx = log_int(rng, 1, 12000)
    case.update(ctx_lo=ctx // 4, ctx_hi=ctx)


def draw(rng):
    op = rng.choice(["append", "axes", "tables", "fwd", "train", "paged", "paged"])
    case = {"op": op, "lens": rng.randrange(1 << 30)}
    if op == "tables":
        most = log_int(rng, 1, 300)
        ctx = log_int(rng, 1, 8000)
        case.update(n=log_int(rng, 1, 4096), new_lo=rng.randrange(2), new_hi=most, ctx_lo=0, ctx_hi=ctx,
                    page=rng.choice([8, 16, 24, 32, 64, 128]), ended=rng.choice([0.0, 0.05, 0.3]),
                    spare=rng.randrange(1000))
        return case
    hkv = rng.choice([1, 2, 4, 8])
    case.update(hkv=hkv, hq=hkv * rng.choice([1, 2, 3, 4, 5, 7, 8]), d=rng.choice([64, 64, 80, 96, 128, 128]))
    if op in ("append", "axes"):
        half = case["d"] // 2
        n = rng.choice([2, 3, 3, 4])
        cuts = sorted(rng.sample(range(1, half), n - 1))
        case.update(theta=rng.choice([1.0e4, 5.0e5, 1.0e6]), interleaved=rng.random() < 0.5, wide=rng.random() < 0.3,
                    own_w=rng.random() < 0.3, sections=",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [half])))
    else:
        rules = [0.0, False, False]
        while rules == [0.0, False, False]:
            rules = [rng.choice([0.0, 20.0, 30.0, 50.0]), rng.random() < 0.4, rng.random() < 0.4]
        case.update(cap=rules[0], slopes=rules[1], prefix=rules[2])
    if op in ("append", "paged"):
        case["page"] = rng.choice([16, 24, 32, 64, 128, 256])
        draw_lengths(rng, case, 96)
        return case
    tokens = log_int(rng, 40, 16384)
    n = log_int(rng, 1, max(2, tokens // 100))
    cuts = sorted(rng.randrange(tokens + 1) for _ in range(n - 1))
    case["pack"] = ",".join(str(min(b - a, 8192)) for a, b in zip([0] + cuts, cuts + [tokens]))
    if op == "axes":
        case["train"] = rng.random() < 0.5
    else:
        case.update(causal=case["prefix"] or rng.random() < 0.75, used=rng.random() < 0.2)
    return case


# ----------------------------------------------------------------- lengths of a case (host)

def pack_lengths(case):
    """Tokens of every sample: given one by one, or drawn as tokens:share:lo:hi:lo:hi."""
    text = case["pack"]
    if ":" not in text:
        return [int(x) for x in text.split(",")]
    total, share, a, b, c, e = text.split(":")
    rng = random.Random("pack %d" % case["lens"])
    lengths = []
    while sum(lengths) < int(total):
        lo, hi = (int(a), int(b)) if rng.random() < float(share) else (int(c), int(e))
        lengths.append(min(rng.randint(lo, hi), int(total) - sum(lengths)))
    return lengths


def used_lengths(case):
    """Rows of every sample that hold tokens (all of them unless the case is a padded batch)."""
    lengths = pack_lengths(case)
    if not case["used"]:
        return lengths
    rng = random.Random("used %d" % case["lens"])
    return [rng.randint(min(64, n), n) for n in lengths]


def cache_lengths(case):
    """(new tokens, tokens in the cache with them) of every sequence."""
    rng = random.Random("cache %d" % case["lens"])
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["n"])]
    return new, [n + rng.randint(case["ctx_lo"], case["ctx_hi"]) for n in new]


def prefix_lengths(case, lengths):
    """Keys of every sequence that all its rows see: none of some, all of a few."""
    rng = random.Random("prefix %d" % case["lens"])
    return [rng.choice([0, rng.randint(0, n), rng.randint(0, n // 2), n]) for n in lengths]


def ended(case):
    """Sequences that are over: their pages go back, and they take no new tokens."""
    rng = random.Random("ended %d" % case["lens"])
    return [rng.random() < case["ended"] for _ in range(case["n"])]


def offsets(lengths):
    return [0] + [int(x) for x in np.cumsum(lengths)]


def sections_of(case):
    return tuple(int(x) for x in case["sections"].split(","))


# ------------------------------------------------------------------------------- inputs

def normal(shape, gen, scale=1.0):
    x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    flat = x.view(-1)
    for at in range(0, flat.numel(), MAX_ELEMS):
        end = min(at + MAX_ELEMS, flat.numel())
        flat[at:end] = torch.randn(end - at, generator=gen, device="cuda") * scale
    return x


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def axis_positions(case, n_axes, lengths, starts, seed):
    """Positions [axes, tokens] of prompts that mix text (all axes alike) with images and clips
    (time, height and width of a grid); the text after a grid goes on past its largest side."""
    rng = np.random.Generator(np.random.PCG64([case["lens"], seed]))
    columns = []
    for n, start in zip(lengths, starts):
        at, p = 0, start
        while at < n:
            run = min(int(rng.integers(1, 400)), n - at)
            columns.append(np.repeat(np.arange(p, p + run)[None], n_axes, axis=0))
            at, p = at + run, p + run
            side = rng.integers(2, 40, size=n_axes)
            side[0] = rng.integers(1, 4) if n_axes > 2 else side[0]
            if n_axes > 3:
                side[-1] = 2
            grid = np.stack([g.ravel() for g in np.meshgrid(*[np.arange(s) for s in side], indexing="ij")])[:, :n - at] + p
            columns.append(grid)
            at, p = at + grid.shape[1], p + int(side.max())
    return np.concatenate(columns, axis=1)


def page_tables(case, kv, gen, spare=8):
    """(pages of every sequence, order of the pool's pages, table [n, width])."""
    page = case["page"]
    pages = [-(-x // page) for x in kv]
    width = max(1, max(pages))
    n_pages = sum(pages) + spare
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    slot = torch.arange(width, device="cuda")[None, :]
    first = ints(offsets(pages)[:-1], torch.int64)[:, None]
    held = ints(pages, torch.int64)[:, None]
    table = torch.where(slot < held, order[(first + slot).clamp(max=n_pages - 1)], torch.full_like(order[:1], -1))
    return pages, order, table


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"op": case["op"]}
    if case["op"] == "tables":
        return prepare_tables(case, gen, s)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    s.update(hq=hq, hkv=hkv, d=d, scale=1.0 / math.sqrt(d))
    if case["op"] in ("append", "axes"):
        s.update(theta=case["theta"], sections=sections_of(case), interleaved=case["interleaved"], own_w=case["own_w"])
        w, axis = frequencies(case)
        s.update(w=torch.from_numpy(w).cuda(), axis=torch.from_numpy(axis).cuda())
    else:
        # slopes of a geometric series over the heads, 1/2 down to 2^-8
        steps = [2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)]
        s.update(cap=case["cap"], slopes=ints(steps, torch.float32) if case["slopes"] else None)
    if case["op"] in ("fwd", "train", "axes"):
        lengths = pack_lengths(case)
        T = sum(lengths)
        qkv = normal((T, hq + 2 * hkv, d), gen)          # one projection's output; q, k and v are views of it
        s.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:])
        if case["op"] == "axes":
            pos = axis_positions(case, len(s["sections"]), lengths, [0] * len(lengths), seed)
            s.update(pos=ints(pos, torch.int64 if case["wide"] else torch.int32), train=case["train"])
            for name in ("q", "k") + (("dq", "dk") if case["train"] else ()):
                s[name + "_out"] = torch.empty((T, hq if name[-1] == "q" else hkv, d), dtype=torch.bfloat16, device="cuda")
            if case["train"]:
                s.update(dq=normal((T, hq, d), gen), dk=normal((T, hkv, d), gen))
            return s
        used = used_lengths(case)
        prefix = prefix_lengths(case, lengths) if case["prefix"] else None
        s.update(causal=case["causal"], cu=ints(offsets(lengths)), starts=offsets(lengths), used=used,
                 seq_used=ints(used) if case["used"] else None, prefixes=prefix,
                 prefix=ints(prefix) if case["prefix"] else None)
        s["q"].mul_(1.5 if not case["cap"] else 6.0)      # sharper scores than chance; far enough to be capped
        if case["op"] == "train":
            s["dout"] = normal((T, hq, d), gen)
        return s
    new, kv = cache_lengths(case)
    pages, order, table = page_tables(case, kv, gen)
    T, page = sum(new), case["page"]
    s.update(cu=ints(offsets(new)), new=new, kv=kv, table=table, page=page, kv_lens=ints(kv),
             k_pages=normal((order.numel(), page, hkv, d), gen), v_pages=normal((order.numel(), page, hkv, d), gen))
    if case["op"] == "append":
        qkv = normal((T, hq + 2 * hkv, d), gen)
        pos = axis_positions(case, len(s["sections"]), new, [k - n for n, k in zip(new, kv)], seed)
        s.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:],
                 pos=ints(pos, torch.int64 if case["wide"] else torch.int32),
                 q_out=torch.empty((T, hq, d), dtype=torch.bfloat16, device="cuda"))
    else:
        prefix = prefix_lengths(case, kv) if case["prefix"] else None
        s.update(q=normal((T, hq, d), gen, 1.5 if not case["cap"] else 6.0), prefixes=prefix,
                 prefix=ints(prefix) if case["prefix"] else None)
    return s


def prepare_tables(case, gen, s):
    new, kv = cache_lengths(case)
    over = ended(case)
    new = [0 if e else n for n, e in zip(new, over)]
    past = [k - n for n, k in zip(cache_lengths(case)[0], kv)]
    pages, order, table = page_tables(case, past, gen, case["spare"] + sum(-(-x // case["page"]) for x in new) + len(new))
    width = max(1, max(-(-(p + n) // case["page"]) for p, n in zip(past, new)))
    wide = torch.full((len(new), width), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table[:, :width]
    held, n_pages = sum(pages), order.numel()
    free = torch.cat([order[held:], torch.zeros(held, dtype=torch.int32, device="cuda")])   # a stack: its top is at the count
    s.update(page=case["page"], past=ints(past), new=ints(new), ended=ints(over, torch.int32), table=wide, free=free,
             count=ints([n_pages - held]), count_out=ints([0]), tokens=max(1, sum(new)))
    return s


def frequencies(case):
    """(w_j rounded once to binary32, the axis of frequency j).  Sections are consecutive, or the
    axes take turns until each has its section; the exponent counts all frequencies, or those of
    the axis alone."""
    sections, half = sections_of(case), case["d"] // 2
    axis, left, turn = [], list(sections), 0
    while len(axis) < half:
        if case["interleaved"]:
            while left[turn % len(left)] == 0:
                turn += 1
            axis.append(turn % len(left))
            left[axis[-1]] -= 1
            turn += 1
        else:
            a = next(i for i, x in enumerate(left) if x)
            axis.append(a)
            left[a] -= 1
    share = [axis[:j].count(a) / sections[a] if case["own_w"] else j / half for j, a in enumerate(axis)]
    return (float(case["theta"]) ** (-np.array(share))).astype(np.float32), np.array(axis, dtype=np.int64)


# ----------------------------------------------------------------------- one pass (run)

def run(s):
    return run_own(s) if own else run_plain(s)


def run_own(s):
    import packed_varlen_rope_gb300 as pr

    if s["op"] == "tables":
        cu, kv_lens, slots = pr.paged_kv_step(s["free"], s["count"], s["table"], s["past"], s["new"], s["page"],
                                              s["tokens"], finished=s["ended"], count_out=s["count_out"])
        return {"cu": cu, "kv_lens": kv_lens, "slots": slots, "table": s["table"], "free": s["free"],
                "count": s["count_out"]}
    if s["op"] == "axes":
        axes = dict(interleaved=s["interleaved"], own_frequencies=s["own_w"])
        out = dict(zip(("q", "k"), pr.rope_axes_apply(s["q"], s["k"], s["theta"], s["sections"], s["pos"],
                                                      q_out=s["q_out"], k_out=s["k_out"], **axes)))
        if s["train"]:
            out["dq"], out["dk"] = pr.rope_axes_apply(s["dq"], s["dk"], s["theta"], s["sections"], s["pos"], backward=True,
                                                      q_out=s["dq_out"], k_out=s["dk_out"], **axes)
        return out
    if s["op"] in ("fwd", "train"):
        rule = dict(causal=s["causal"], scale=s["scale"], seq_used=s["seq_used"], score_cap=s["cap"],
                    distance_slopes=s["slopes"], prefix_lens=s["prefix"])
        if s["op"] == "fwd":
            return pr.attn_varlen_fwd(s["q"], s["k"], s["v"], s["cu"], **rule)
        o, lse = pr.attn_varlen_fwd(s["q"], s["k"], s["v"], s["cu"], return_lse=True, **rule)
        dq, dk, dv = pr.attn_varlen_bwd(s["dout"], s["q"], s["k"], s["v"], o, lse, s["cu"], **rule)
        return {"o": o, "dq": dq, "dk": dk, "dv": dv}
    cache = pr.PagedKVCache(s["k_pages"], s["v_pages"])
    if s["op"] == "append":
        pr.rope_kv_append(s["q"], s["k"], s["v"], cache, s["table"], s["kv_lens"], s["cu"], s["theta"], q_out=s["q_out"],
                          position_ids=s["pos"], sections=s["sections"], interleaved=s["interleaved"],
                          own_frequencies=s["own_w"])
        return {"q": s["q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    return pr.attn_paged(s["q"], cache, s["table"], s["kv_lens"], s["cu"], scale=s["scale"], score_cap=s["cap"],
                         distance_slopes=s["slopes"], prefix_lens=s["prefix"])


def heads_first(x, group=1):
    """[tokens, heads, d] to binary32 [heads * group, tokens, d], every head `group` times."""
    return x.float().transpose(0, 1).repeat_interleave(group, dim=0)


def turned(s, x, back=False):
    """Rows [tokens, heads, d] rotated by their positions (backward: by the opposite angles)."""
    phi = (s["pos"].float()[s["axis"]] * s["w"][:, None]).t()[:, None, :].double()   # the angle is a binary32 product
    c, sn = phi.cos().float(), phi.sin().float()
    if back:
        sn = -sn
    lo, hi = x.float().split(s["d"] // 2, dim=2)
    return torch.cat([lo * c - hi * sn, hi * c + lo * sn], dim=2).to(torch.bfloat16)


def plain_sample(s, i, n):
    """(p, t, q, k, v) of the first n rows of sample i: p the softmax of the visible scores, t the
    tanh of the capped ones."""
    a, g = s["starts"][i], s["hq"] // s["hkv"]
    q, k, v = heads_first(s["q"][a:a + n]), heads_first(s["k"][a:a + n], g), heads_first(s["v"][a:a + n], g)
    x, t = (q @ k.transpose(1, 2)).mul_(s["scale"]), None
    if s["cap"]:
        t = x.div_(s["cap"]).tanh_()
        x = t * s["cap"]
    at = torch.arange(n, device="cuda")
    if s["slopes"] is not None:
        x = x - s["slopes"][:, None, None] * (at[:, None] - at[None, :]).abs()
    if s["causal"]:
        hidden = at[:, None] < at[None, :]
        if s["prefixes"] is not None:
            hidden &= at[None, :] >= s["prefixes"][i]
        x.masked_fill_(hidden, float("-inf"))
    x = x.sub_(x.amax(dim=2, keepdim=True)).exp_()
    return x.div_(x.sum(dim=2, keepdim=True)), t, q, k, v


def run_plain(s):
    if s["op"] == "tables":
        return plain_tables(s)
    if s["op"] == "axes":
        out = {n: s[n + "_out"].copy_(turned(s, s[n])) for n in ("q", "k")}
        if s["train"]:
            out.update({n: s[n + "_out"].copy_(turned(s, s[n], back=True)) for n in ("dq", "dk")})
        return out
    if s["op"] == "fwd":
        o = torch.zeros(s["q"].shape, dtype=torch.bfloat16, device="cuda")
        for i, n in enumerate(s["used"]):
            if n:
                p, _, _, _, v = plain_sample(s, i, n)
                o[s["starts"][i]:s["starts"][i] + n] = (p @ v).transpose(0, 1)
        return o
    if s["op"] == "train":
        out = {"o": torch.zeros(s["q"].shape, dtype=torch.bfloat16, device="cuda")}
        for name, x in (("dq", s["q"]), ("dk", s["k"]), ("dv", s["v"])):
            out[name] = torch.zeros(x.shape, dtype=torch.bfloat16, device="cuda")
        g = s["hq"] // s["hkv"]
        for i, n in enumerate(s["used"]):
            if n == 0:
                continue
            a = s["starts"][i]
            p, t, q, k, v = plain_sample(s, i, n)
            do = heads_first(s["dout"][a:a + n])
            out["o"][a:a + n] = (p @ v).transpose(0, 1)
            dv = p.transpose(1, 2) @ do
            dp = do @ v.transpose(1, 2)
            ds = dp.sub_((dp * p).sum(dim=2, keepdim=True)).mul_(p).mul_(s["scale"])
            if t is not None:
                ds = ds.mul_(1.0 - t * t)
            dq, dk = ds @ k, ds.transpose(1, 2) @ q
            out["dq"][a:a + n] = dq.transpose(0, 1)
            out["dk"][a:a + n] = dk.view(s["hkv"], g, n, -1).sum(dim=1).transpose(0, 1)
            out["dv"][a:a + n] = dv.view(s["hkv"], g, n, -1).sum(dim=1).transpose(0, 1)
        return out
    T, d, page = s["q"].shape[0], s["d"], s["page"]
    cu, kv = s["cu"].long(), s["kv_lens"].long()
    t = torch.arange(T, device="cuda")
    seq = torch.searchsorted(cu, t, right=True) - 1          # every sequence has a new token
    pos = t - cu[seq + 1] + kv[seq]
    if s["op"] == "append":
        s["q_out"].copy_(turned(s, s["q"]))
        at = s["table"][seq, pos // page].long()
        s["k_pages"][at, pos % page] = turned(s, s["k"])
        s["v_pages"][at, pos % page] = s["v"]
        return {"q": s["q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    # one sequence at a time where prompts are long, else all padded to the longest: queries
    # [n, hkv, g, new, d] over keys [n, hkv, 1, kv, d]
    out = torch.empty(s["q"].shape, dtype=torch.bfloat16, device="cuda")
    together = len(s["new"]) if max(s["new"]) <= 16 else 1
    for lo in range(0, len(s["new"]), together):
        part = slice(lo, lo + together)
        n, g = len(s["new"][part]), s["hq"] // s["hkv"]
        rows, keys = max(s["new"][part]), max(s["kv"][part])
        own_rows = (seq >= lo) & (seq < lo + together) if together == 1 else slice(None)
        sq, sp = seq[own_rows] - lo, pos[own_rows]
        i = (t[own_rows] - cu[lo + sq])
        q = torch.zeros((n, rows, s["hkv"], g, d), device="cuda")
        q[sq, i] = s["q"][own_rows].float().view(-1, s["hkv"], g, d)
        q = q.permute(0, 2, 3, 1, 4)
        j = torch.arange(keys, device="cuda")
        at = s["table"][part][:, j // page].clamp(min=0).long()
        k, v = (x[at, j % page].float().permute(0, 2, 1, 3)[:, :, None] for x in (s["k_pages"], s["v_pages"]))
        x = (q.reshape(n, s["hkv"], 1, g * rows, d) @ k.transpose(3, 4)).mul_(s["scale"]).view(n, s["hkv"], g, rows, keys)
        if s["cap"]:
            x = x.div_(s["cap"]).tanh_().mul_(s["cap"])
        # rows that pad a sequence see the gap between its keys and the longest's: they are dropped below
        last = torch.full((n, rows), keys, device="cuda")
        last[sq, i] = sp
        if s["slopes"] is not None:
            x = x - s["slopes"].view(1, s["hkv"], g, 1, 1) * (last[:, None, None, :, None] - j).abs()
        seen = j <= last[:, :, None]
        if s["prefix"] is not None:
            seen |= (j < torch.minimum(s["prefix"], s["kv_lens"])[part, None])[:, None, :]
        x.masked_fill_(~seen[:, None, None], float("-inf"))
        x = x.sub_(x.amax(dim=4, keepdim=True)).exp_()
        x.div_(x.sum(dim=4, keepdim=True))
        o = (x.view(n, s["hkv"], 1, g * rows, keys) @ v).view(n, s["hkv"], g, rows, d).permute(0, 3, 1, 2, 4)
        out[own_rows] = o[sq, i].reshape(-1, s["hq"], d).to(torch.bfloat16)
    return out


def plain_tables(s):
    """The pages of ended sequences go to the top of the free stack, in the order of sequences and
    of their tables; the growing ones then take theirs from the top in the same order."""
    page, table, free = s["page"], s["table"], s["free"]
    n, width = table.shape
    over = s["ended"] != 0
    index = torch.arange(width, device="cuda")[None, :]
    back = over[:, None] & (index * page < s["past"][:, None]) & (table >= 0)
    rank = back.flatten().cumsum(0) - 1 + s["count"]
    # entries that do not go back are written over one spare place past the end
    place = torch.where(back.flatten() & (rank < free.numel()), rank, free.numel())
    grown = torch.cat([free, free[:1]]).scatter_(0, place, table.flatten())
    free.copy_(grown[:-1])
    count = s["count"] + back.sum()
    past = torch.where(over, 0, s["past"])
    kv = past + s["new"]
    held, want = (past + page - 1) // page, (kv + page - 1) // page
    need = want - held
    first = need.cumsum(0) - need
    takes = (index >= held[:, None]) & (index < want[:, None])
    top = count - 1 - (first[:, None] + index - held[:, None])
    taken = torch.where(takes & (top >= 0), free[top.clamp(0, free.numel() - 1).long()], -1)
    table.copy_(torch.where(takes, taken, table))
    s["count_out"].copy_((count - need.sum()).clamp(min=0))
    cu = torch.cat([torch.zeros_like(s["new"][:1]), s["new"].cumsum(0)]).to(torch.int32)
    t = torch.arange(s["tokens"], device="cuda")
    seq = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=n - 1)
    pos = (past[seq] + t - cu[seq]).clamp(0, width * page - 1)
    got = table[seq, pos // page].long()
    slots = torch.where((got >= 0) & (t < cu[n]), got * page + pos % page, -1)
    return {"cu": cu, "kv_lens": kv.to(torch.int32), "slots": slots, "table": table, "free": free, "count": s["count_out"]}


# ------------------------------------------------------------------------- what it needs

def visible(case):
    """Pairs of a query row and a key that it sees, over all sequences (per query head)."""
    pairs = 0
    if case["op"] in ("fwd", "train"):
        lengths = pack_lengths(case)
        prefix = prefix_lengths(case, lengths) if case["prefix"] else [0] * len(lengths)
        for n, p in zip(used_lengths(case), prefix):
            p = min(p, n)
            pairs += n * (n + 1) // 2 + p * (p - 1) // 2 if case["causal"] else n * n
        return pairs
    new, kv = cache_lengths(case)
    prefix = prefix_lengths(case, kv) if case["prefix"] else [0] * len(kv)
    for n, k, p in zip(new, kv, prefix):
        more = max(0, p - (k - n) - 1)                       # rows whose own position is before the prefix's last key
        pairs += n * k - n * (n - 1) // 2 + more * (more + 1) // 2
    return pairs


def work(case):
    if case["op"] == "tables":
        new, kv = cache_lengths(case)
        over, page = ended(case), case["page"]
        taken = sum(-(-k // page) - -(-(k - n) // page) for n, k, e in zip(new, kv, over) if not e)
        back = sum(-(-(k - n) // page) for n, k, e in zip(new, kv, over) if e)
        tokens = sum(n for n, e in zip(new, over) if not e)
        # lengths and marks read, offsets and lengths written; a page's id read and written; the
        # slots.  Operations: a division and a product a token, sums over sequences and pages
        return {"bytes": 20 * case["n"] + 8 * (taken + back) + 8 * tokens, "flops": 3 * tokens + 4 * case["n"]}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] in ("append", "axes"):
        T = sum(cache_lengths(case)[0] if case["op"] == "append" else pack_lengths(case))
        passes = 2 if case["op"] == "axes" and case["train"] else 1
        heads = hq + hkv + (hkv if case["op"] == "append" else 0)
        ids = T * len(sections_of(case)) * (8 if case["wide"] else 4)
        return {"bytes": passes * (4 * T * heads * d + ids), "flops": passes * 3 * T * (hq + hkv) * d}
    pairs = visible(case)
    if case["op"] == "paged":
        new, kv = cache_lengths(case)
        return {"bytes": 4 * sum(new) * hq * d + 4 * sum(kv) * hkv * d, "flops": 4 * d * hq * pairs}
    read = sum(used_lengths(case))
    T = sum(pack_lengths(case))
    fwd = 2 * d * (read * (hq + 2 * hkv) + T * hq)
    if case["op"] == "fwd":
        return {"bytes": fwd, "flops": 4 * d * hq * pairs}
    # q, k, v and dout read; o, dq, dk and dv written.  Seven products: two forward, five
    # backward, the scores among them again, as they are too many to keep (tokens^2 a head)
    return {"bytes": fwd + 2 * d * (read * hq + T * (hq + 2 * hkv)), "flops": 14 * d * hq * pairs}


# ----------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    """Attention one head at a time, its gradient from autograd's chain rule through the
    definition; rotations as products of complex numbers; tables sequence by sequence."""
    attention = case["op"] in ("fwd", "train", "paged")
    if attention and visible(case) * case["hq"] * case["d"] * (14 if case["op"] == "train" else 4) > 3e12:
        return None
    s = prepare(case, seed)
    if case["op"] == "tables":
        return exact_tables(s)
    if case["op"] in ("axes", "append"):
        return exact_rotation(s)
    g = s["hq"] // s["hkv"]

    def scores(q, k, row, key, h, prefix, causal):
        """Scores of one head, -infinity where the key is hidden: rows and keys at these positions."""
        x = torch.einsum("id,jd->ij", q, k) * s["scale"]
        if s["cap"]:
            e = torch.exp(2.0 * x / s["cap"])
            x = s["cap"] * (e - 1.0) / (e + 1.0)
        far = (row[:, None] - key[None, :]).double()
        if s["slopes"] is not None:
            x = x - s["slopes"][h].double() * far.abs()
        seen = (far >= 0) | (key[None, :] < prefix) if causal else torch.ones_like(far, dtype=torch.bool)
        return torch.where(seen, x, torch.full((), -math.inf, dtype=torch.float64, device="cuda"))

    if case["op"] in ("fwd", "train"):
        want = {"o": torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")}
        if case["op"] == "train":
            want.update({"d" + n: torch.zeros(s[n].shape, dtype=torch.float64, device="cuda") for n in "qkv"})
        for i, n in enumerate(s["used"]):
            a, at = s["starts"][i], torch.arange(n, device="cuda")
            for h in range(s["hq"] if n else 0):
                q, k, v = (x[a:a + n, e].double().requires_grad_() for x, e in
                           ((s["q"], h), (s["k"], h // g), (s["v"], h // g)))
                sc = scores(q, k, at, at, h, s["prefixes"][i] if s["prefixes"] else 0, s["causal"])
                o = torch.exp(sc - torch.logsumexp(sc, dim=1)[:, None]) @ v
                want["o"][a:a + n, h] = o.detach()
                if case["op"] == "train":
                    dq, dk, dv = torch.autograd.grad(o, (q, k, v), s["dout"][a:a + n, h].double())
                    want["dq"][a:a + n, h] = dq
                    want["dk"][a:a + n, h // g] += dk
                    want["dv"][a:a + n, h // g] += dv
        return want if case["op"] == "train" else want["o"]
    o = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for i, (n, m) in enumerate(zip(s["new"], s["kv"])):
        ids = s["table"][i, :-(-m // s["page"])].long()
        k, v = (x[ids].flatten(0, 1)[:m].double() for x in (s["k_pages"], s["v_pages"]))
        key = torch.arange(m, device="cuda")
        for h in range(s["hq"]):
            sc = scores(s["q"][at:at + n, h].double(), k[:, h // g], key[m - n:], key, h,
                        s["prefixes"][i] if s["prefixes"] else 0, True)
            w = torch.exp(sc - sc.amax(dim=1, keepdim=True))
            o[at:at + n, h] = (w @ v[:, h // g]) / w.sum(dim=1, keepdim=True)
        at += n
    return o


def exact_rotation(s):
    pos, half = s["pos"].cpu().numpy(), s["d"] // 2
    axis, w = s["axis"].cpu().numpy(), s["w"].cpu().numpy()
    phi = pos[axis].T.astype(np.float32) * w[None, :]                   # binary32 product
    z = torch.from_numpy(np.exp(1j * phi.astype(np.float64))).cuda()[:, None, :]

    def turn(x, by):
        y = torch.complex(x[..., :half].double(), x[..., half:].double()) * by
        return torch.cat([y.real, y.imag], dim=-1)

    if s["op"] == "axes":
        out = {"q": turn(s["q"], z), "k": turn(s["k"], z)}
        if s["train"]:
            out.update(dq=turn(s["dq"], z.conj()), dk=turn(s["dk"], z.conj()))
        return out
    kp, vp, kr, at = s["k_pages"].double(), s["v_pages"].double(), turn(s["k"], z), 0
    for i, (n, k) in enumerate(zip(s["new"], s["kv"])):
        p = torch.arange(k - n, k, device="cuda")
        page = s["table"][i][p // s["page"]].long()
        kp[page, p % s["page"]] = kr[at:at + n]
        vp[page, p % s["page"]] = s["v"][at:at + n].double()
        at += n
    return {"q": turn(s["q"], z), "k_pages": kp, "v_pages": vp}


def exact_tables(s):
    past, new, over = (s[n].tolist() for n in ("past", "new", "ended"))
    table, free, page = s["table"].cpu().numpy().copy(), s["free"].cpu().numpy().copy(), s["page"]
    count = int(s["count"].item())
    for i, p in enumerate(past):
        if over[i]:
            for x in table[i, :-(-p // page)]:
                if x >= 0 and count < len(free):
                    free[count] = x
                    count += 1
            past[i] = 0
    slots = np.full(s["tokens"], -1, dtype=np.int64)
    at, kv = 0, []
    for i, (p, n) in enumerate(zip(past, new)):
        for j in range(-(-p // page), -(-(p + n) // page)):
            table[i, j] = free[count - 1] if count > 0 else -1
            count = max(0, count - 1)
        q = np.arange(p, p + n)
        ids = table[i, q // page].astype(np.int64)
        slots[at:at + n] = np.where(ids >= 0, ids * page + q % page, -1)
        at += n
        kv.append(p + n)
    return {"cu": ints(offsets(new)), "kv_lens": ints(kv), "slots": ints(slots, torch.int64), "table": ints(table),
            "free": ints(free), "count": ints([count])}
