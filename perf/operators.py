"""The paged-cache operators and the verification of drafted tokens: cases, their plain forms, and the library's calls.

A serving loop over a pool of cache pages goes: append a chunk's keys and values to each sequence's pages
("append"; the pages hold bf16, or e4m3 codes with one scale for each token and kv head), attend the chunk's
queries over each sequence's pages ("attend"), and, where the chunk was drafted, verify it against the target's
logits ("verify").  "read" copies pages back into dense bf16 rows, as the dense-cache calls take them.
"""
import math

import torch

own = False

E4M3_MAX = 448.0

# Head layouts of the repository's workloads: SmolLM2-135M, the 125M-class block, the SmolLM3 block.
SMOLLM2 = dict(H=9, KV=3, hd=64)
SLM125M = dict(H=12, KV=4, hd=64)
SMOLLM3 = dict(H=16, KV=4, hd=128)


def listed():
    return [
        # one decode step's keys and values of 30 layers into the pages of 64 sequences, 8-bit pages
        dict(name="append_step_e4m3", op="append", kind="e4m3", **SMOLLM2, L=30, B=64, T=1, lo=1024, hi=4096, page=64, ragged=False),
        # the keys and values of a prefill of 8 prompts, 1 to 2048 tokens, packed one behind the other, quantised
        dict(name="append_prompts_e4m3", op="append", kind="e4m3", **SMOLLM2, L=30, B=8, T=2048, lo=0, hi=0, page=16, ragged=True),
        # one sequence's pages back into a dense cache row (it leaves the pool)
        dict(name="read_one_bf16", op="read", kind="bf16", **SMOLLM2, L=30, B=1, T=700, lo=0, hi=0, page=32, ragged=False),
        # a batch's 8-bit pages back into the dense decode cache of four SmolLM3 blocks
        dict(name="read_batch_e4m3", op="read", kind="e4m3", **SMOLLM3, L=4, B=16, T=4096, lo=0, hi=0, page=64, ragged=True),
        # a single user's next token: latency
        dict(name="attend_b1_t1", op="attend", kind="bf16", **SMOLLM2, B=1, T=1, lo=700, hi=700, page=16, window=0, ragged=False),
        # a decode step of 64 sequences of 1024 to 4096 tokens
        dict(name="attend_b64_t1", op="attend", kind="bf16", **SMOLLM2, B=64, T=1, lo=1024, hi=4096, page=64, window=0, ragged=False),
        # five drafted tokens for each of 32 sequences over 8-bit pages
        dict(name="attend_draft_e4m3", op="attend", kind="e4m3", **SMOLLM3, B=32, T=5, lo=2000, hi=8191, page=32, window=0, ragged=False),
        # prompts' chunks of 1 to 1024 tokens over caches of other lengths, in one packed batch, with a window
        dict(name="attend_mixed_window", op="attend", kind="e4m3", **SLM125M, B=24, T=1024, lo=0, hi=6000, page=16, window=2048, ragged=True),
        # a long prompt's later chunk: the largest call
        dict(name="attend_long_chunk", op="attend", kind="bf16", **SMOLLM3, B=1, T=2048, lo=32000, hi=32000, page=64, window=0, ragged=False),
        # greedy verification of four tokens for one user: latency
        dict(name="verify_greedy_b1", op="verify", B=1, T=4, V=49152, temperature=0.0, top_k=0, top_p=1.0, probs=False, ragged=False),
        # a serving batch with the usual filters, drafts drawn from a smaller model's probabilities
        dict(name="verify_filtered_b64", op="verify", B=64, T=5, V=49152, temperature=0.75, top_k=50, top_p=0.9375, probs=True, ragged=True),
        # plain sampling over a larger vocabulary of an odd size
        dict(name="verify_plain_b32", op="verify", B=32, T=7, V=128257, temperature=1.0, top_k=0, top_p=1.0, probs=True, ragged=False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["append", "read", "attend", "attend", "attend", "verify", "verify"])
    if op == "verify":
        V = rng.choice([49152, rng.randrange(1000, 60000), rng.randrange(60000, 152000)])
        T = rng.randint(1, 8)
        B = _log(rng, 1, max(1, min(96, 24_000_000 // ((T + 1) * V))))
        return dict(op=op, B=B, T=T, V=V, temperature=rng.choice([0.0, 0.5, 0.75, 1.0, 1.25]), top_k=rng.choice([0, 0, 1, 40, rng.randint(2, 500)]),
                    top_p=rng.choice([1.0, 1.0, 0.9375, 0.5 + rng.randrange(1, 60) / 128]), probs=rng.random() < 0.7, ragged=rng.random() < 0.5)
    heads = rng.choice([SMOLLM2, SLM125M, SMOLLM3, dict(H=rng.choice([4, 8, 14, 20, 32]), KV=rng.choice([1, 2, 4]), hd=rng.choice([64, 128]))])
    if heads["H"] % heads["KV"] or heads["H"] // heads["KV"] > 8:
        heads = dict(heads, KV=heads["H"] // 2)
    row = dict(op=op, kind=rng.choice(["bf16", "e4m3"]), **heads, page=rng.choice([16, 32, 64, 128]), ragged=rng.random() < 0.5)
    if op in ("append", "read"):
        L = rng.choice([1, 4, rng.randint(2, 30)])
        T = _log(rng, 1, 4096)
        per = L * heads["KV"] * heads["hd"]
        B = _log(rng, 1, max(1, min(64, 24_000_000 // (per * T))))
        lo = 0 if op == "read" else rng.choice([0, _log(rng, 1, 2000)])
        return dict(row, L=L, B=B, T=T, lo=lo, hi=lo if op == "read" else max(lo, _log(rng, 1, 4000)))
    T = rng.choice([1, 1, rng.randint(2, 9), _log(rng, 10, 2048)])
    hi = _log(rng, 8, 32000)
    B = _log(rng, 1, max(1, min(64, int(2e8 / (T * (hi + T)) / heads["H"] * 16), 6_000_000 // ((hi + T) * heads["KV"]))))
    return dict(row, B=B, T=T, lo=rng.randint(0, hi), hi=hi, window=rng.choice([0, 0, _log(rng, 1, 4096)]))


def _spread(lo, hi, n):
    """n whole numbers spread evenly over [lo, hi]: the work of a case does not depend on the seed."""
    return [lo + ((hi - lo) * i) // max(1, n - 1) if n > 1 else hi for i in range(n)]


def _news(case):
    return _spread(1, case["T"], case["B"]) if case["ragged"] else [case["T"]] * case["B"]


def _mixed(values, g):
    t = torch.tensor(values, dtype=torch.int32, device="cuda")
    return t[torch.randperm(len(values), generator=g, device="cuda")]


def _quantise(x):
    """Codes and scales of rows of floats: one scale for each row, its largest magnitude on the largest code."""
    scale = x.abs().amax(-1) / E4M3_MAX
    return (x / scale.clamp_min(1e-30)[..., None]).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)

    def randn(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)

    if case["op"] == "verify":
        return _prepare_verify(case, g, randn)
    B, T, H, KV, hd, page = (case[k] for k in ("B", "T", "H", "KV", "hd", "page"))
    L = case.get("L", 1)
    pos, n = _mixed(_spread(case["lo"], case["hi"], B), g), _mixed(_news(case), g)
    start = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    start[1:] = n.cumsum(0)
    cols = -(-(case["hi"] + T) // page)
    P = B * cols + 3
    s = dict(case=case, pos=pos, n=n, start=start, rows=sum(_news(case)), cols=cols,
             table=torch.randperm(P, generator=g, device="cuda")[: B * cols].to(torch.int32).view(B, cols))
    pool = (L, P, KV, page, hd)
    for x in ("k", "v"):
        if case["kind"] == "bf16":
            s[x + "_pages"], s[x + "_scale"] = randn(*pool) if case["op"] != "append" else torch.zeros(pool, dtype=torch.bfloat16, device="cuda"), None
        elif case["op"] == "append":
            s[x + "_pages"], s[x + "_scale"] = torch.zeros(pool, dtype=torch.float8_e4m3fn, device="cuda"), torch.zeros(pool[:-1], device="cuda")
        else:
            s[x + "_pages"], s[x + "_scale"] = _quantise(randn(*pool, dtype=torch.float32))
    if case["op"] == "attend":
        # queries that single out some keys, as trained heads do: scores of a standard deviation of 2
        shape = (s["rows"], H, hd) if case["ragged"] else (B, T, H, hd)
        s["q"] = (2 * randn(*shape, dtype=torch.float32)).to(torch.bfloat16)
        s["out"] = torch.empty_like(s["q"])
    elif case["op"] == "append":
        # as the prefill and the decode step return them, [L, B, KV, T, hd], or packed [L, rows, KV, hd]
        for x in ("k", "v"):
            s[x + "_new"] = randn(L, s["rows"], KV, hd) if case["ragged"] else randn(L, B, KV, T, hd)
    else:
        for x in ("k", "v"):   # the dense cache, [L, B, KV, T, hd]
            s[x + "_out"] = torch.zeros(L, B, KV, T, hd, dtype=torch.bfloat16, device="cuda")
    if own:   # what a program keeps beside its pages: their descriptor, the chunk's, and a workspace
        from llama_decoder_forward_gb300 import smol as S
        s["cache"] = S.PagedCache(s["k_pages"], s["v_pages"], s["table"], s["k_scale"], s["v_scale"])
        if case["op"] == "read":
            s["chunk"] = S.Chunk(B, T, pos, n_new=n)
        else:
            s["chunk"] = S.Chunk(B, T, pos, row_start=start) if case["ragged"] else S.Chunk(B, T, pos)
        if case["op"] == "attend":
            s["ws"] = S.alloc_paged_workspace(s["cache"], H, B, T)
    return s


def _prepare_verify(case, g, randn):
    B, T, V = case["B"], case["T"], case["V"]
    # logits with a long tail and a few likely tokens, as a trained model's; the drafter's are those, disturbed
    base = 2.0 * randn(B, T + 1, V, dtype=torch.float32)
    likely = torch.randint(0, V, (B, T + 1, 24), generator=g, device="cuda")
    base.scatter_add_(2, likely, 5.0 + 4.0 * torch.rand(B, T + 1, 24, generator=g, device="cuda"))
    draft = torch.softmax(base[:, :T] + 0.5 * randn(B, T, V, dtype=torch.float32), -1)
    if not case["probs"]:   # a drafter that names its likeliest token
        drafts = (base[:, :T] + 0.1 * randn(B, T, V, dtype=torch.float32)).argmax(-1)
    else:
        u = torch.rand(B, T, 1, generator=g, device="cuda")
        drafts = torch.searchsorted(draft.cumsum(-1), u).squeeze(-1).clamp_max(V - 1)
    n = _mixed([min(T, v) for v in _spread(0, T, B)] if case["ragged"] else [T] * B, g)
    s = dict(case=case, logits=base.to(torch.bfloat16), drafts=drafts.to(torch.int32), n=n, probs=draft if case["probs"] else None,
             u=torch.rand(B, T + 1, generator=g, device="cuda"), accepted=torch.zeros(B, dtype=torch.int32, device="cuda"),
             next=torch.zeros(B, dtype=torch.int32, device="cuda"), p=torch.zeros(B, T, device="cuda"))
    if own:
        from llama_decoder_forward_gb300 import smol as S
        s["ws"] = S.alloc_verify_workspace(B, T)
    return s


def run(s):
    return {"append": _append, "read": _read, "attend": _attend, "verify": _verify}[s["case"]["op"]](s)


def _places(s):
    """Page and slot of row t of each sequence, [B, T], and whether there is such a row."""
    c = s["case"]
    t = torch.arange(c["T"], device="cuda")
    at = s["pos"][:, None].long() + t
    page = s["table"].long().gather(1, (at // c["page"]).clamp_max(s["cols"] - 1))
    return page, at % c["page"], t < s["n"][:, None]


def _append(s):
    if own:
        from llama_decoder_forward_gb300 import smol as S
        k, v = s["k_new"], s["v_new"]
        if not s["case"]["ragged"]:
            k, v = k.transpose(2, 3), v.transpose(2, 3)
        S.paged_append(s["cache"], s["chunk"], k, v)
    else:
        page, slot, there = _places(s)
        page, slot = page[there], slot[there]
        for x in ("k", "v"):
            new = s[x + "_new"]
            rows = new if s["case"]["ragged"] else new.transpose(2, 3).flatten(1, 2)[:, there.flatten()]
            if s["case"]["kind"] == "bf16":
                s[x + "_pages"][:, page, :, slot] = rows.transpose(0, 1)
            else:
                codes, scale = _quantise(rows.float())
                s[x + "_pages"].view(torch.uint8)[:, page, :, slot] = codes.view(torch.uint8).transpose(0, 1)
                s[x + "_scale"][:, page, :, slot] = scale.transpose(0, 1)
    return {x: s[x] for x in ("k_pages", "v_pages", "k_scale", "v_scale") if s[x] is not None}


def _values(s, x, page, slot):
    """The pages' values in 32 bits at [..., B, T] places: [L, B, T, KV, hd]."""
    pages = s[x + "_pages"]
    if s["case"]["kind"] == "bf16":
        return pages[:, page, :, slot].float().permute(2, 0, 1, 3, 4)
    codes = pages.view(torch.uint8)[:, page, :, slot].view(torch.float8_e4m3fn).float()
    return (codes * s[x + "_scale"][:, page, :, slot][..., None]).permute(2, 0, 1, 3, 4)


def _read(s):
    if own:
        from llama_decoder_forward_gb300 import smol as S
        S.paged_read(s["cache"], s["chunk"], s["k_out"].transpose(2, 3), s["v_out"].transpose(2, 3))
    else:
        page, slot, there = _places(s)
        for x in ("k", "v"):
            out = s[x + "_out"].transpose(2, 3)
            out.copy_(torch.where(there[..., None, None], _values(s, x, page, slot).to(torch.bfloat16), out))
    return {"k": s["k_out"], "v": s["v_out"]}


def _attend(s):
    c = s["case"]
    if own:
        from llama_decoder_forward_gb300 import smol as S
        S.paged_attention(s["cache"], 0, s["chunk"], s["q"], s["out"], s["ws"], window=c["window"])
        return s["out"]
    B, T, H, KV, hd = (c[k] for k in ("B", "T", "H", "KV", "hd"))
    G, keys = H // KV, c["hi"] + T
    j = torch.arange(keys, device="cuda")
    page = s["table"].long()[:, j // c["page"]]
    slot = (j % c["page"]).expand(B, keys)
    k, v = (_values(s, x, page, slot)[0].permute(0, 2, 1, 3) for x in ("k", "v"))   # [B, KV, keys, hd]
    t = torch.arange(T, device="cuda")
    there = t < s["n"][:, None]
    q = s["q"]
    if c["ragged"]:
        q = q[(s["start"][:-1, None].long() + t).clamp_max(s["rows"] - 1)]          # [B, T, H, hd]
    q = q.float().view(B, T, KV, G, hd).permute(0, 2, 3, 1, 4).reshape(B, KV, G * T, hd)
    scores = (q @ k.transpose(2, 3)).view(B, KV, G, T, keys).div_(math.sqrt(hd))
    at = s["pos"][:, None].long() + t                                               # [B, T]
    seen = j <= at[..., None]
    if c["window"]:
        seen &= j > at[..., None] - c["window"]
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    scores.sub_(scores.amax(-1, keepdim=True)).exp_()
    total = scores.sum(-1, keepdim=True)
    out = ((scores.view(B, KV, G * T, keys) @ v).view(B, KV, G, T, hd) / total).permute(0, 3, 1, 2, 4).reshape(B, T, H, hd)
    return (out[there] if c["ragged"] else out).to(torch.bfloat16)


def _verify(s):
    c = s["case"]
    if own:
        from llama_decoder_forward_gb300 import smol as S
        S.verify_drafts(s["logits"], s["drafts"], s["accepted"], s["next"], s["ws"], uniform=s["u"], draft_probs=s["probs"], n_draft=s["n"],
                        p_draft=s["p"], temperature=c["temperature"], top_k=c["top_k"], top_p=c["top_p"], do_sample=c["temperature"] > 0)
        return {"accepted": s["accepted"], "next": s["next"], "p": s["p"]}
    # in 64 bits: a draw falls next to a border of the cumulative sums too often in 32
    B, T, V = c["B"], c["T"], c["V"]
    z = s["logits"].double()
    if c["temperature"] > 0:
        # the temperature and top_p that a 32-bit call takes: 0.75, 0.9375 and the like are the same in both
        z = z / c["temperature"]
        if 0 < c["top_k"] < V:
            z = z.masked_fill(z < z.topk(c["top_k"], -1).values[..., -1:], -math.inf)
        w = (z - z.amax(-1, keepdim=True)).exp()
        p = w / w.sum(-1, keepdim=True)
        if c["top_p"] < 1:
            order = z.sort(dim=-1, descending=True, stable=True).indices
            ranked = p.gather(-1, order)
            cut = torch.zeros_like(ranked, dtype=torch.bool)
            cut[..., 1:] = ranked.cumsum(-1)[..., :-1] > c["top_p"]
            p = p.masked_fill(torch.zeros_like(cut).scatter(-1, order, cut), 0.0)
            p = p / p.sum(-1, keepdim=True)
    else:
        p = torch.zeros_like(z).scatter(-1, z.argmax(-1, keepdim=True), 1.0)
    x = s["drafts"].long()[..., None]
    px = p[:, :T].gather(-1, x).squeeze(-1)
    there = torch.arange(T, device="cuda") < s["n"][:, None]
    if c["temperature"] > 0:
        qx = s["probs"].double().gather(-1, x).squeeze(-1) if c["probs"] else torch.ones_like(px)
        kept = there & (s["u"][:, :T].double() * qx < px)
    else:
        kept = there & (px > 0)
    accepted = kept.int().cumprod(-1).sum(-1)
    p = p.gather(1, accepted[:, None, None].expand(B, 1, V)).squeeze(1)              # [B, V]
    refused = accepted < s["n"]
    if c["temperature"] > 0:
        i = accepted.clamp_max(T - 1)[:, None, None]
        if c["probs"]:
            q = s["probs"].gather(1, i.expand(B, 1, V)).squeeze(1).double()
        else:
            q = torch.zeros_like(p).scatter(-1, x.gather(1, i).squeeze(1), 2.0)
        rest = (p - q).clamp_min(0)
        p = torch.where(refused[:, None] & (rest.sum(-1, keepdim=True) > 0), rest, p)
        run_sum = p.cumsum(-1)
        # the first index at which the running sum exceeds u times the whole
        chosen = (run_sum > s["u"][:, T:].double() * run_sum[:, -1:]).int().argmax(-1)
    else:
        chosen = p.argmax(-1)
    return {"accepted": accepted.int(), "next": chosen.int(), "p": torch.where(there, px, 0.0).float()}


def work(case):
    c = case
    if c["op"] == "verify":
        n = [min(c["T"], v) for v in _spread(0, c["T"], c["B"])] if c["ragged"] else [c["T"]] * c["B"]
        rows = sum(n) + c["B"]
        # every target row; of the drafter's probabilities the row of a refusal, and one number for each draft
        return {"bytes": rows * c["V"] * 2 + (c["B"] * c["V"] * 4 if c["probs"] and c["temperature"] > 0 else 0), "flops": 10.0 * rows * c["V"]}
    KV, hd = c["KV"], c["hd"]
    held = hd * 2 if c["kind"] == "bf16" else hd + 4
    news = _news(c)
    if c["op"] in ("append", "read"):
        rows = 2 * c["L"] * KV * sum(news)
        return {"bytes": rows * (hd * 2 + held), "flops": 2.0 * rows * hd}
    keys = pairs = 0
    for i, at in enumerate(_spread(c["lo"], c["hi"], c["B"])):
        n, w = news[i], c["window"] or 1 << 30
        keys += min(at + n, w + n - 1)
        full = max(0, min(n, w - 1 - at))          # rows that see all before them
        pairs += full * at + full * (full + 1) // 2 + (n - full) * min(w, 1 << 30) if c["window"] else n * at + n * (n + 1) // 2
    return {"bytes": keys * KV * held * 2 + 2 * sum(news) * c["H"] * hd * 2, "flops": 4.0 * hd * c["H"] * pairs}


def exact(case, seed):
    """From the definitions, sequence by sequence, in 64 bits."""
    s = prepare(case, seed)
    c = case
    if c["op"] == "verify":
        z = s["logits"].double()
        keep = torch.ones_like(z, dtype=torch.bool)
        if c["temperature"] <= 0:
            best = z.argmax(-1)
            px = (best[:, : c["T"]] == s["drafts"]).double()
        else:
            z = z / c["temperature"]
            if 0 < c["top_k"] < c["V"]:
                keep = z >= z.kthvalue(c["V"] - c["top_k"] + 1, dim=-1, keepdim=True).values
            pr = torch.softmax(z.masked_fill(~keep, -math.inf), -1)
            if c["top_p"] < 1:
                for b in range(c["B"]):
                    for i in range(c["T"] + 1):
                        val, at = pr[b, i].sort(descending=True, stable=True)
                        many = int((val.cumsum(0) <= c["top_p"]).sum()) + 1
                        pr[b, i, at[many:]] = 0
                pr = pr / pr.sum(-1, keepdim=True)
            px = torch.stack([pr[:, i].gather(1, s["drafts"][:, i : i + 1].long())[:, 0] for i in range(c["T"])], 1)
        px[torch.arange(c["T"], device="cuda") >= s["n"][:, None]] = 0
        return {"accepted": None, "next": None, "p": px}
    lens, news, page = s["pos"].tolist(), s["n"].tolist(), c["page"]

    def held(x, b, lo, hi):
        """Sequence b's values at positions lo .. hi - 1: [L, KV, hi - lo, hd] in 64 bits."""
        ids = s["table"][b, lo // page : -(-hi // page)].long()
        v = s[x + "_pages"][:, ids] if c["kind"] == "bf16" else s[x + "_pages"].view(torch.uint8)[:, ids].view(torch.float8_e4m3fn)
        v = v.double().transpose(1, 2).flatten(2, 3)
        if c["kind"] != "bf16":
            v = v * s[x + "_scale"][:, ids].double().transpose(1, 2).flatten(2, 3)[..., None]
        return v[:, :, lo % page : lo % page + hi - lo]

    if c["op"] == "read":
        for b, n in enumerate(news):
            for x in ("k", "v"):
                s[x + "_out"] = s[x + "_out"].double()
                s[x + "_out"][:, b, :, :n] = held(x, b, lens[b], lens[b] + n)
        return {"k": s["k_out"], "v": s["v_out"]}
    if c["op"] == "append":
        first = 0
        got = {}
        for x in ("k", "v"):
            got[x + "_pages"] = torch.zeros(s[x + "_pages"].shape, dtype=torch.float64 if c["kind"] == "bf16" else torch.float32, device="cuda")
            if c["kind"] != "bf16":
                got[x + "_scale"] = torch.zeros(s[x + "_scale"].shape, dtype=torch.float64, device="cuda")
        for b, n in enumerate(news):
            at = torch.arange(lens[b], lens[b] + n, device="cuda")
            ids, slot = s["table"][b][at // page].long(), at % page
            for x in ("k", "v"):
                new = s[x + "_new"][:, first : first + n].transpose(1, 2) if c["ragged"] else s[x + "_new"][:, b]
                new = new.double()                                                    # [L, KV, n, hd]
                if c["kind"] != "bf16":
                    unit = new.abs().amax(-1, keepdim=True) / E4M3_MAX
                    got[x + "_scale"][:, ids, :, slot] = unit[..., 0].permute(2, 0, 1)
                    new = (new / unit).float().to(torch.float8_e4m3fn).float()
                got[x + "_pages"][:, ids, :, slot] = new.permute(2, 0, 1, 3).to(got[x + "_pages"].dtype)
            first += n
        return got
    G, outs = c["H"] // c["KV"], []
    for b, n in enumerate(news):
        first = sum(news[:b])
        q = (s["q"][first : first + n] if c["ragged"] else s["q"][b]).double()        # [n, H, hd]
        lo = max(0, lens[b] - c["window"] + 1) if c["window"] else 0
        k, v = held("k", b, lo, lens[b] + n)[0], held("v", b, lo, lens[b] + n)[0]     # [KV, keys, hd]
        rows, cols = lens[b] + torch.arange(n, device="cuda")[:, None], lo + torch.arange(k.shape[1], device="cuda")
        dark = (cols > rows) | (cols <= rows - c["window"] if c["window"] else cols < 0)
        heads = [torch.softmax((q[:, h] @ k[h // G].T / math.sqrt(c["hd"])).masked_fill(dark, -math.inf), -1) @ v[h // G] for h in range(c["H"])]
        outs.append(torch.stack(heads, 1))
    return torch.cat(outs) if c["ragged"] else torch.stack(outs)
