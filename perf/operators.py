"""Workloads of the attention operators: packed variable-length attention (forward, and
forward with backward), attention of new tokens over a paged key/value cache, and the
append that rotates new keys into that cache.

``run`` has two forms of each.  The plain one is elementary torch arithmetic in binary32,
rounded once to bf16 at the end; the other calls the library.  ``exact`` evaluates the
definitions in binary64.
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
        # one decoding step of a small batch: the rotation and the append alone, latency counts
        {"name": "append-decode-8", "op": "append", "n": 8, "new_lo": 1, "new_hi": 1, "ctx_lo": 100, "ctx_hi": 4000,
         "hq": 32, "hkv": 8, "d": 128, "page": 64, "theta": 1.0e6, "lens": 1},
        # a prefill chunk of a large model's heads from several prompts at once
        {"name": "append-prefill-16k", "op": "append", "n": 12, "new_lo": 900, "new_hi": 1900, "ctx_lo": 0, "ctx_hi": 8000,
         "hq": 64, "hkv": 8, "d": 128, "page": 64, "theta": 1.0e6, "lens": 2},
        # one token of one conversation over its cache: the shortest serving step
        {"name": "paged-decode-1", "op": "paged", "n": 1, "new_lo": 1, "new_hi": 1, "ctx_lo": 4097, "ctx_hi": 4097,
         "hq": 32, "hkv": 8, "d": 128, "page": 64, "lens": 3},
        # a serving batch: one token each of 64 conversations of uneven length
        {"name": "paged-decode-64", "op": "paged", "n": 64, "new_lo": 1, "new_hi": 1, "ctx_lo": 500, "ctx_hi": 16000,
         "hq": 32, "hkv": 8, "d": 128, "page": 64, "lens": 4},
        # drafted tokens checked together: a few new tokens each, small heads, a page size that is no power of two
        {"name": "paged-draft-16x5", "op": "paged", "n": 16, "new_lo": 3, "new_hi": 7, "ctx_lo": 0, "ctx_hi": 3000,
         "hq": 12, "hkv": 4, "d": 64, "page": 24, "lens": 5},
        # chunked prefill: a chunk of each of four long prompts over what is already cached
        {"name": "paged-chunk-4x2k", "op": "paged", "n": 4, "new_lo": 1500, "new_hi": 2048, "ctx_lo": 2000, "ctx_hi": 16000,
         "hq": 32, "hkv": 8, "d": 128, "page": 128, "lens": 6},
        # four samples of 5 to 33 tokens: the smallest pack
        {"name": "fwd-tiny-64", "op": "fwd", "pack": "5,17,33,9", "hq": 4, "hkv": 2, "d": 64, "causal": True,
         "used": False, "lens": 7},
        # the packed fine-tuning batch, 16,384 tokens, as evaluation runs it
        {"name": "fwd-pack-16k", "op": "fwd", "pack": "16384:0.8:32:512:2048:8192", "hq": 32, "hkv": 8, "d": 128,
         "causal": True, "used": False, "lens": 8},
        # a padded batch of 8 x 2048 rows whose pad rows are left out
        {"name": "fwd-padded-8x2048", "op": "fwd", "pack": "2048,2048,2048,2048,2048,2048,2048,2048", "hq": 32,
         "hkv": 8, "d": 128, "causal": True, "used": True, "lens": 9},
        # an attention layer of a training step on the packed fine-tuning batch
        {"name": "train-pack-16k", "op": "train", "pack": "16384:0.8:32:512:2048:8192", "hq": 32, "hkv": 8, "d": 128,
         "causal": True, "used": False, "lens": 10},
        # the same at a large model's head count and 65,536 tokens
        {"name": "train-pack-64k", "op": "train", "pack": "65536:0.5:16:256:1024:4096", "hq": 64, "hkv": 8, "d": 128,
         "causal": True, "used": False, "lens": 11},
        # an encoder's odd shape: both directions, five heads to a key head, head_dim 80, uneven lengths
        {"name": "train-bidir-odd", "op": "train", "pack": "1,777,130,0,2051,63,500", "hq": 10, "hkv": 2, "d": 80,
         "causal": False, "used": False, "lens": 12},
    ]


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "paged", "paged", "fwd", "train"])
    case = {"op": op, "lens": rng.randrange(1 << 30)}
    if op in ("append", "paged"):
        hkv = rng.choice([1, 2, 4, 8])
        case.update(hkv=hkv, hq=hkv * rng.choice([1, 2, 3, 4, 5, 7, 8]), d=rng.choice([64, 64, 80, 96, 128, 128]),
                    page=rng.choice([16, 24, 32, 64, 128, 256]))
        kind = rng.choice(["decode", "draft", "chunk"])
        if kind == "decode":
            case.update(n=log_int(rng, 1, 96), new_lo=1, new_hi=1)
        elif kind == "draft":
            case.update(n=log_int(rng, 1, 32), new_lo=1, new_hi=rng.randrange(2, 17))
        else:
            hi = log_int(rng, 17, 2048)
            case.update(n=rng.randrange(1, 5), new_lo=max(1, hi // 2), new_hi=hi)
        ctx = log_int(rng, 1, 12000)
        case.update(ctx_lo=ctx // 4, ctx_hi=ctx)
        if op == "append":
            case["theta"] = rng.choice([1.0e4, 5.0e5, 1.0e6])
        return case
    hkv = rng.choice([1, 2, 4, 8])
    case.update(hkv=hkv, hq=hkv * rng.choice([1, 2, 3, 4, 5, 8]), d=rng.choice([64, 64, 80, 96, 128, 128]),
                causal=rng.random() < 0.75, used=rng.random() < 0.2)
    tokens = log_int(rng, 40, 16384)
    n = log_int(rng, 1, max(2, tokens // 100))
    cuts = sorted(rng.randrange(tokens + 1) for _ in range(n - 1))
    lengths = [b - a for a, b in zip([0] + cuts, cuts + [tokens])]
    case["pack"] = ",".join(str(min(x, 8192)) for x in lengths)
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


def offsets(lengths):
    return [0] + [int(x) for x in np.cumsum(lengths)]


# ------------------------------------------------------------------------------- inputs

def normal(shape, gen, scale=1.0):
    x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    flat = x.view(-1)
    for at in range(0, flat.numel(), MAX_ELEMS):
        end = min(at + MAX_ELEMS, flat.numel())
        flat[at:end] = torch.randn(end - at, generator=gen, device="cuda") * scale
    return x


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    s = {"op": case["op"], "hq": hq, "hkv": hkv, "d": d, "scale": 1.0 / math.sqrt(d)}
    if case["op"] in ("fwd", "train"):
        lengths, used = pack_lengths(case), used_lengths(case)
        T = sum(lengths)
        qkv = normal((T, hq + 2 * hkv, d), gen)          # one projection's output; q, k and v are views of it
        s.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], causal=case["causal"],
                 cu=torch.tensor(offsets(lengths), dtype=torch.int32, device="cuda"), starts=offsets(lengths),
                 used=used, seq_used=torch.tensor(used, dtype=torch.int32, device="cuda") if case["used"] else None)
        s["q"].mul_(1.5)                                  # sharper scores than chance
        if case["op"] == "train":
            s["dout"] = normal((T, hq, d), gen)
        return s
    new, kv = cache_lengths(case)
    page = case["page"]
    width = max(-(-x // page) for x in kv)
    pages = [-(-x // page) for x in kv]
    n_pages = sum(pages) + 8
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros((len(kv), width), dtype=torch.int32, device="cuda")
    slot = torch.arange(width, device="cuda")[None, :]
    held = torch.tensor(pages, device="cuda")[:, None]
    first = torch.tensor(offsets(pages)[:-1], device="cuda")[:, None]
    table.copy_(torch.where(slot < held, order[(first + slot).clamp(max=n_pages - 1)], table))
    T = sum(new)
    s.update(cu=torch.tensor(offsets(new), dtype=torch.int32, device="cuda"), new=new, kv=kv, table=table, page=page,
             kv_lens=torch.tensor(kv, dtype=torch.int32, device="cuda"),
             k_pages=normal((n_pages, page, hkv, d), gen), v_pages=normal((n_pages, page, hkv, d), gen))
    if case["op"] == "append":
        qkv = normal((T, hq + 2 * hkv, d), gen)
        s.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], theta=case["theta"],
                 q_out=torch.empty((T, hq, d), dtype=torch.bfloat16, device="cuda"),
                 w=torch.from_numpy(frequencies(case["theta"], d)).cuda())
    else:
        s["q"] = normal((T, hq, d), gen, 1.5)
    return s


def frequencies(theta, d):
    """w_j = theta^(-2j/d), rounded once to binary32 (the rotation's definition)."""
    return (float(theta) ** (-2.0 * np.arange(d // 2, dtype=np.float64) / d)).astype(np.float32)


# ----------------------------------------------------------------------- one pass (run)

def run(s):
    return run_own(s) if own else run_plain(s)


def run_own(s):
    import packed_varlen_rope_gb300 as pr

    if s["op"] == "fwd":
        return pr.attn_varlen_fwd(s["q"], s["k"], s["v"], s["cu"], causal=s["causal"], scale=s["scale"],
                                  seq_used=s["seq_used"])
    if s["op"] == "train":
        o, lse = pr.attn_varlen_fwd(s["q"], s["k"], s["v"], s["cu"], causal=s["causal"], scale=s["scale"],
                                    seq_used=s["seq_used"], return_lse=True)
        dq, dk, dv = pr.attn_varlen_bwd(s["dout"], s["q"], s["k"], s["v"], o, lse, s["cu"], causal=s["causal"],
                                        scale=s["scale"], seq_used=s["seq_used"])
        return {"o": o, "dq": dq, "dk": dk, "dv": dv}
    cache = pr.PagedKVCache(s["k_pages"], s["v_pages"])
    if s["op"] == "append":
        pr.rope_kv_append(s["q"], s["k"], s["v"], cache, s["table"], s["kv_lens"], s["cu"], s["theta"],
                          q_out=s["q_out"])
        return {"q": s["q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    return pr.attn_paged(s["q"], cache, s["table"], s["kv_lens"], s["cu"], scale=s["scale"])


def heads_first(x, group=1):
    """[tokens, heads, d] to binary32 [heads * group, tokens, d], every head `group` times."""
    return x.float().transpose(0, 1).repeat_interleave(group, dim=0)


def plain_sample(s, a, b):
    """(p, q, k, v) of the sample of rows a..b: p the softmax of the visible scores."""
    g = s["hq"] // s["hkv"]
    q, k, v = heads_first(s["q"][a:b]), heads_first(s["k"][a:b], g), heads_first(s["v"][a:b], g)
    x = (q @ k.transpose(1, 2)).mul_(s["scale"])
    if s["causal"]:
        i = torch.arange(b - a, device="cuda")
        x.masked_fill_(i[:, None] < i[None, :], float("-inf"))
    x = x.sub_(x.amax(dim=2, keepdim=True)).exp_()
    return x.div_(x.sum(dim=2, keepdim=True)), q, k, v


def run_plain(s):
    if s["op"] == "fwd":
        o = torch.zeros(s["q"].shape, dtype=torch.bfloat16, device="cuda")
        for a, n in zip(s["starts"], s["used"]):
            if n:
                p, _, _, v = plain_sample(s, a, a + n)
                o[a:a + n] = (p @ v).transpose(0, 1)
        return o
    if s["op"] == "train":
        out = {"o": torch.zeros(s["q"].shape, dtype=torch.bfloat16, device="cuda")}
        for name, x in (("dq", s["q"]), ("dk", s["k"]), ("dv", s["v"])):
            out[name] = torch.zeros(x.shape, dtype=torch.bfloat16, device="cuda")
        g = s["hq"] // s["hkv"]
        for a, n in zip(s["starts"], s["used"]):
            if n == 0:
                continue
            p, q, k, v = plain_sample(s, a, a + n)
            do = heads_first(s["dout"][a:a + n])
            out["o"][a:a + n] = (p @ v).transpose(0, 1)
            dv = p.transpose(1, 2) @ do
            dp = do @ v.transpose(1, 2)
            ds = dp.sub_((dp * p).sum(dim=2, keepdim=True)).mul_(p).mul_(s["scale"])
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
        phi = pos.float()[:, None, None] * s["w"]
        c, sn = phi.cos(), phi.sin()

        def rotate(x):
            lo, hi = x.float().split(d // 2, dim=2)
            return torch.cat([lo * c - hi * sn, hi * c + lo * sn], dim=2).to(torch.bfloat16)

        s["q_out"].copy_(rotate(s["q"]))
        at = s["table"][seq, pos // page].long()
        s["k_pages"][at, pos % page] = rotate(s["k"])
        s["v_pages"][at, pos % page] = s["v"]
        return {"q": s["q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    # every sequence padded to the longest: queries [n, hkv, g, new, d] over keys [n, hkv, 1, kv, d]
    n, g = len(s["new"]), s["hq"] // s["hkv"]
    rows, keys = max(s["new"]), max(s["kv"])
    i = t - cu[seq]
    q = torch.zeros((n, rows, s["hkv"], g, d), device="cuda")
    q[seq, i] = s["q"].float().view(T, s["hkv"], g, d)
    q = q.permute(0, 2, 3, 1, 4)
    j = torch.arange(keys, device="cuda")
    at = s["table"][:, j // page].long()
    k, v = (x[at, j % page].float().permute(0, 2, 1, 3)[:, :, None] for x in (s["k_pages"], s["v_pages"]))
    x = (q.reshape(n, s["hkv"], 1, g * rows, d) @ k.transpose(3, 4)).mul_(s["scale"]).view(n, s["hkv"], g, rows, keys)
    last = torch.full((n, rows), keys, device="cuda")
    last[seq, i] = pos
    x.masked_fill_(j > last[:, None, None, :, None], float("-inf"))
    # rows that pad a sequence see the gap between its keys and the longest's: they are dropped below
    x = x.sub_(x.amax(dim=4, keepdim=True)).exp_()
    x.div_(x.sum(dim=4, keepdim=True))
    o = (x.view(n, s["hkv"], 1, g * rows, keys) @ v).view(n, s["hkv"], g, rows, d).permute(0, 3, 1, 2, 4)
    return o[seq, i].reshape(T, s["hq"], d).to(torch.bfloat16)


# ------------------------------------------------------------------------- what it needs

def visible(case):
    """Pairs of a query row and a key that it sees, over all sequences (per query head)."""
    if case["op"] in ("fwd", "train"):
        return sum(n * (n + 1) // 2 if case["causal"] else n * n for n in used_lengths(case))
    return sum(n * k - n * (n - 1) // 2 for n, k in zip(*cache_lengths(case)))


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "append":
        T = sum(cache_lengths(case)[0])
        return {"bytes": 4 * T * (hq + 2 * hkv) * d, "flops": 3 * T * (hq + hkv) * d}
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
    """One head at a time; the gradient from autograd's chain rule through the definition."""
    if case["op"] != "append" and visible(case) * case["hq"] * case["d"] * (14 if case["op"] == "train" else 4) > 3e12:
        return None
    s = prepare(case, seed)
    g = s["hq"] // s["hkv"]
    if case["op"] in ("fwd", "train"):
        want = {"o": torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")}
        if case["op"] == "train":
            want.update({"d" + n: torch.zeros(s[n].shape, dtype=torch.float64, device="cuda") for n in "qkv"})
        for a, n in zip(s["starts"], s["used"]):
            for h in range(s["hq"] if n else 0):
                q, k, v = (x[a:a + n, e].double().requires_grad_() for x, e in
                           ((s["q"], h), (s["k"], h // g), (s["v"], h // g)))
                sc = torch.einsum("id,jd->ij", q, k) * s["scale"]
                if s["causal"]:
                    sc = sc + torch.full_like(sc, float("-inf")).triu(1)
                o = torch.exp(sc - torch.logsumexp(sc, dim=1)[:, None]) @ v
                want["o"][a:a + n, h] = o.detach()
                if case["op"] == "train":
                    dq, dk, dv = torch.autograd.grad(o, (q, k, v), s["dout"][a:a + n, h].double())
                    want["dq"][a:a + n, h] = dq
                    want["dk"][a:a + n, h // g] += dk
                    want["dv"][a:a + n, h // g] += dv
        return want if case["op"] == "train" else want["o"]
    if case["op"] == "append":
        cos_sin = []
        for n, k in zip(s["new"], s["kv"]):
            pos = np.arange(k - n, k, dtype=np.float32)
            phi = (pos[:, None] * frequencies(s["theta"], s["d"])).astype(np.float64)     # binary32 product
            cos_sin.append(np.exp(1j * phi))
        z = torch.from_numpy(np.concatenate(cos_sin)).cuda()[:, None, :]
        half = s["d"] // 2

        def turn(x):
            y = torch.complex(x[..., :half].double(), x[..., half:].double()) * z
            return torch.cat([y.real, y.imag], dim=-1)

        kp, vp = s["k_pages"].double(), s["v_pages"].double()
        kr, at = turn(s["k"]), 0
        for i, (n, k) in enumerate(zip(s["new"], s["kv"])):
            p = torch.arange(k - n, k, device="cuda")
            page = s["table"][i][p // s["page"]].long()
            kp[page, p % s["page"]] = kr[at:at + n]
            vp[page, p % s["page"]] = s["v"][at:at + n].double()
            at += n
        return {"q": turn(s["q"]), "k_pages": kp, "v_pages": vp}
    o = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for i, (n, m) in enumerate(zip(s["new"], s["kv"])):
        ids = s["table"][i, :-(-m // s["page"])].long()
        k, v = (x[ids].flatten(0, 1)[:m].double() for x in (s["k_pages"], s["v_pages"]))
        seen = torch.ones((n, m), dtype=torch.bool, device="cuda").tril(m - n)
        for h in range(s["hq"]):
            sc = torch.einsum("id,jd->ij", s["q"][at:at + n, h].double(), k[:, h // g]) * s["scale"]
            w = torch.where(seen, torch.exp(sc - sc.max()), torch.zeros((), dtype=torch.float64, device="cuda"))
            o[at:at + n, h] = (w @ v[:, h // g]) / w.sum(dim=1, keepdim=True)
        at += n
    return o
