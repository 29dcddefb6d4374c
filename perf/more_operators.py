"""Cases, plain forms and calls of the paged cache's operators for prompts and shared pages.

    attn      several new tokens per sequence against their pages, causal (mcs_paged_attn)
    shared    one new token per sequence, groups of sequences with a common beginning
              (mcs_paged_decode_shared)
    fork      new sequences from old ones: pages shared, copied and freed (mcs_paged_fork,
              mcs_paged_copy)
    compact   pages moved to the front of the cache (mcs_paged_compact, mcs_paged_copy)

With `own` false run() computes an operator in elementary torch operations, in
32 bits or more, rounded once; with `own` true it calls the library.  exact()
is a separate 64-bit statement of each definition.
"""

import math
import random

import torch

own = False

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
K_SCALE, V_SCALE = 3 / 256, 45 / 4096  # E4M3 caches: about the largest magnitude / 448
MAX_SCORES = 3_200_000_000  # of the plain form, which holds them all


def listed():
    return [
        # one short prompt of a conversation that begins: latency
        dict(name="attn_one", op="attn", B=1, page=16, before=0, new=77, ragged=False, Hq=16, Hkv=16, D=64, e4m3=False, fused=True),
        # a few proposed tokens per sequence, checked in one step of a server's ragged batch
        dict(name="attn_few", op="attn", B=32, page=32, before=8000, new=5, ragged=True, Hq=32, Hkv=8, D=128, e4m3=False, fused=True),
        # prompts admitted together, some of them behind earlier turns
        dict(name="attn_prompts", op="attn", B=6, page=64, before=4096, new=4001, ragged=True, Hq=32, Hkv=8, D=128, e4m3=False, fused=True),
        # a piece of a context as long as the large video workload, E4M3 cache, its 40 heads
        dict(name="attn_long", op="attn", B=1, page=64, before=73552, new=1024, ragged=False, Hq=40, Hkv=8, D=128, e4m3=True, fused=False),
        # four beams of a conversation: latency
        dict(name="shared_beams", op="shared", R=1, W=4, page=16, prompt=1023, after=40, ragged=False, Hq=32, Hkv=8, D=128, e4m3=False, fused=True),
        # requests of one application, all behind the same long instructions
        dict(name="shared_prompt", op="shared", R=1, W=96, page=64, prompt=16384, after=700, ragged=True, Hq=32, Hkv=8, D=128, e4m3=False, fused=True),
        # documents asked about several times each, E4M3 cache, the large workload's 40 heads
        dict(name="shared_documents", op="shared", R=6, W=8, page=64, prompt=40000, after=1500, ragged=True, Hq=40, Hkv=8, D=128, e4m3=True, fused=False),
        # a step of beam search: 16 requests with 8 beams, every beam goes on from one of its request's
        dict(name="fork_beams", op="fork", kind="reorder", R=16, W=8, page=16, prompt=2000, after=200, Hkv=8, D=128, e4m3=False),
        # one long prompt answered 64 times, others of the batch go on or end
        dict(name="fork_prompt", op="fork", kind="branch", R=120, W=1, more=64, page=128, prompt=20001, after=700, Hkv=8, D=128, e4m3=False),
        # every page in front after most of a day's sequences ended
        dict(name="compact_all", op="compact", R=40, W=2, page=64, prompt=4000, after=900, most=0, spare=1500, Hkv=8, D=128, e4m3=False),
        # a few pages between two steps, E4M3 cache
        dict(name="compact_some", op="compact", R=64, W=1, page=32, prompt=3000, after=300, most=24, spare=3001, Hkv=8, D=128, e4m3=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "shared", "shared", "fork", "compact"])
    D, page, e4m3, fused = rng.choice([64, 128]), rng.choice([16, 32, 64, 128]), rng.random() < 0.5, rng.random() < 0.5
    Hkv, group = rng.choice([1, 2, 4, 5, 8, 10, 16]), rng.choice([1, 2, 4, 5, 8, 16, 20])
    if op == "attn":
        Hq = Hkv * group
        while Hq > 64:
            Hq -= Hkv
        B, new = _log(rng, 1, 48), _log(rng, 1, 4096)
        B = max(1, min(B, 24000 // new))
        room = min(MAX_SCORES // (B * new * Hq), 300_000_000 // (B * Hkv * D), 75600)
        if room <= 2 * new:
            B, new = 1, max(1, min(new, int(math.sqrt(MAX_SCORES / Hq / 2))))
            room = min(MAX_SCORES // (new * Hq), 300_000_000 // (Hkv * D), 75600)
        before = _log(rng, 1, max(1, room - new)) - 1
        return dict(op=op, B=B, page=page, before=before, new=new, ragged=rng.random() < 0.6, Hq=Hq, Hkv=Hkv, D=D, e4m3=e4m3, fused=fused)
    if op == "shared":
        R, W = _log(rng, 1, 12), _log(rng, 1, 96)
        R = max(1, min(R, 128 // W))
        after = _log(rng, 1, 1500)
        prompt = _log(rng, 1, max(1, min(40000, 900_000_000 // (R * W * Hkv * D) - after)))
        return dict(op=op, R=R, W=W, page=page, prompt=prompt, after=after, ragged=rng.random() < 0.6, Hq=Hkv * group, Hkv=Hkv, D=D, e4m3=e4m3, fused=fused)
    Hkv = min(Hkv, 8)
    case = dict(op=op, R=_log(rng, 1, 100), W=rng.choice([1, 1, 2, 4, 8]), page=page, prompt=_log(rng, 1, 4000), after=_log(rng, 1, 900), Hkv=Hkv, D=D, e4m3=e4m3)
    case["R"] = max(1, min(case["R"], 250_000 // (case["prompt"] + case["W"] * case["after"])))
    if op == "fork":
        case["kind"] = rng.choice(["reorder", "branch"])
        case["more"] = _log(rng, 1, 64)
    else:
        case["spare"] = _log(rng, 1, 2000)
        case["most"] = rng.choice([0, 0, _log(rng, 1, 500)])
    return case


# ------------------------------------------------------------------ inputs

def _sizes(c):
    """Token counts: a fixed choice for the case's sizes.

    attn: (tokens before, new tokens) of each sequence; others: (shared tokens of each
    request, own tokens of each of its sequences)."""
    if c["op"] == "attn":
        r = random.Random(1_000_003 * c["B"] + 97 * c["new"] + c["before"])
        before, new = [c["before"]] * c["B"], [c["new"]] * c["B"]
        if c["ragged"]:
            before = [int(c["before"] * r.random()) for _ in before]
            new = [max(1, int(c["new"] * r.uniform(0.3, 1.0))) for _ in new]
            before[-1], new[0] = c["before"], c["new"]
            if c["B"] >= 4:
                before[1], new[2] = 0, 0  # a fresh one, and one that has nothing new
        return before, new
    r = random.Random(1_000_003 * c["R"] + 97 * c["prompt"] + c["after"])
    ragged = c.get("ragged", True)
    prompt = [max(1, int(c["prompt"] * r.uniform(0.3, 1.0))) if ragged else c["prompt"] for _ in range(c["R"])]
    prompt[0] = c["prompt"]
    after = [[max(1, int(c["after"] * r.random())) if ragged else c["after"] for _ in range(c["W"])] for _ in prompt]
    after[-1][0] = c["after"]
    return prompt, after


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=F32)


def _ints(v):
    return torch.tensor(v, dtype=I32, device="cuda")


def _cache(g, total, Hkv, page, D, e4m3, scale, fill, level, empty):
    """A cache whose pages are alike inside (a vector of their own plus noise); rows that hold no token are `empty`."""
    out = torch.empty(total, Hkv, page, D, dtype=torch.uint8 if e4m3 else BF16, device="cuda")
    step = max(1, (1 << 26) // (Hkv * page * D))
    hole = torch.arange(page, device="cuda")[None] >= fill[:, None]
    for a in range(0, total, step):
        z = min(total, a + step)
        x = level * _randn(g, z - a, Hkv, 1, D) + 0.7 * _randn(g, z - a, Hkv, page, D)
        x = (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) if e4m3 else x.to(BF16)
        out[a:z] = x.masked_fill(hole[a:z, None, :, None], empty)
    return out


def _caches_of(s, g, total, fill, empty):
    c = s["c"]
    s["scales"] = (K_SCALE, V_SCALE) if c["e4m3"] else (1.0, 1.0)
    for name, f, level in (("k_cache", s["scales"][0], 0.8), ("v_cache", s["scales"][1], 0.3)):
        s[name] = _cache(g, total, c["Hkv"], c["page"], c["D"], c["e4m3"], f, fill, level, empty)


def _rows(g, T, H, D, fused, behind):
    """[T, H, D] bf16 rows: of their own, or a view into rows of a fused projection."""
    x = _randn(g, T, (H + behind) * D if fused else H * D).to(BF16)
    return x[:, : H * D].view(T, H, D)


def _families(c, g, spare):
    """Sequences of R requests, W of each, which hold the full pages of their request's prompt together:
    (lens, first sequence of each request, shared pages of each, table, holders of each page beyond the
    first, tokens in each page)."""
    page = c["page"]
    prompt, after = _sizes(c)
    lens, starts, shared, total = [], [0], [], 0
    for p, own_tokens in zip(prompt, after):
        lens += [p + x for x in own_tokens]
        starts.append(len(lens))
        shared.append(p // page)
        total += p // page + sum(-(-(p + x) // page) - p // page for x in own_tokens)
    P = max(-(-x // page) for x in lens) + 2  # room to go on
    # (numbers in the order in which they are handed out, then shuffled)
    table = torch.full((len(lens), P), -1, dtype=I32)
    extra, fill, at = torch.zeros(total + spare, dtype=I32), torch.zeros(total + spare, dtype=torch.int64), 0
    for r, n in enumerate(shared):
        rows = range(starts[r], starts[r + 1])
        table[rows.start: rows.stop, :n] = torch.arange(at, at + n, dtype=I32)
        extra[at: at + n], fill[at: at + n] = len(rows) - 1, page
        at += n
        for b in rows:
            m = -(-lens[b] // page) - n
            table[b, n: n + m] = torch.arange(at, at + m, dtype=I32)
            fill[at: at + m] = page
            if lens[b] % page:
                fill[at + m - 1] = lens[b] % page
            at += m
    order = torch.randperm(total + spare, generator=g, device="cuda")
    table = table.cuda()
    table = torch.where(table >= 0, order[table.long().clamp(min=0)].to(I32), -1)
    back = torch.argsort(order)
    return lens, starts, shared, table, extra.cuda()[back], fill.cuda()[back]


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"c": c}
    page, Hkv, D = c["page"], c["Hkv"], c["D"]
    nan = 0x7F if c["e4m3"] else float("nan")
    if c["op"] == "attn":
        before, new = _sizes(c)
        lens = [a + n for a, n in zip(before, new)]
        pages = [-(-x // page) for x in lens]
        total, P, B = sum(pages) + 3, max(1, max(pages)), c["B"]
        s["table"] = torch.full((B, P), -1, dtype=I32, device="cuda")
        live = torch.arange(P, device="cuda")[None] < _ints(pages)[:, None]
        s["table"][live] = torch.randperm(total, generator=g, device="cuda").to(I32)[: sum(pages)]
        held = (_ints(lens)[:, None] - torch.arange(P, device="cuda")[None] * page).clamp(0, page)
        fill = torch.zeros(total, dtype=torch.int64, device="cuda")
        fill[s["table"][live].long()] = held[live].long()
        s["lens"], s["longest"], s["most"] = _ints(lens), max(lens), max(new)
        s["cu"] = torch.cat([_ints([0]), _ints(new).cumsum(0).to(I32)])
        s["T"] = sum(new) + 5  # a step's buffers are a little longer than its tokens
        _caches_of(s, g, total, fill, nan)
        s["q"] = _rows(g, s["T"], c["Hq"], D, c["fused"], 2 * Hkv)
        if own:
            from token_sparse_attention_gb300 import mcs
            s["p"] = mcs.paged(B, c["Hq"], Hkv, D, page, total, P, kv=mcs.KV_E4M3 if c["e4m3"] else mcs.KV_BF16, k_scale=s["scales"][0],
                               v_scale=s["scales"][1], q_stride=(c["Hq"] + 2 * Hkv) * D if c["fused"] else 0)
            # rows behind the last token stay as they are
            s["out"] = [torch.zeros(s["T"], c["Hq"], D, dtype=BF16, device="cuda"), torch.zeros(s["T"], c["Hq"], device="cuda")]
            s["ws"] = mcs.empty_workspace(mcs.mcs_paged_attn_workspace(s["p"]))
        return s
    spare = c.get("spare", 3 if c["op"] == "shared" else 200)
    lens, starts, shared, s["table"], s["extra"], fill = _families(c, g, spare)
    B, total, P = len(lens), fill.numel(), s["table"].shape[1]
    s["lens"] = _ints(lens)
    if c["op"] == "shared":
        s["starts"], s["shared"] = _ints(starts), _ints(shared)
        _caches_of(s, g, total, fill, nan)
        s["q"] = _rows(g, B, c["Hq"], D, c["fused"], 2 * Hkv)
        if own:
            from token_sparse_attention_gb300 import mcs
            s["p"] = mcs.paged(B, c["Hq"], Hkv, D, page, total, P, kv=mcs.KV_E4M3 if c["e4m3"] else mcs.KV_BF16, k_scale=s["scales"][0],
                               v_scale=s["scales"][1], q_stride=(c["Hq"] + 2 * Hkv) * D if c["fused"] else 0)
            s["out"] = [torch.empty(B, c["Hq"], D, dtype=BF16, device="cuda"), torch.empty(B, c["Hq"], device="cuda")]
            s["ws"] = mcs.empty_workspace(mcs.mcs_paged_decode_shared_workspace(s["p"]))
        return s
    _caches_of(s, g, total, fill, 0)  # comparable: nothing undefined stays in what comes back
    s["k_mean"] = _randn(g, total, Hkv, D).to(BF16)
    free = torch.nonzero(fill == 0)[:, 0].to(I32)
    s["head"] = _ints([total - free.numel()])
    s["free"] = torch.cat([torch.full((total - free.numel(),), -1, dtype=I32, device="cuda"), free[torch.randperm(free.numel(), generator=g, device="cuda")]])
    if c["op"] == "fork":
        s["parents"] = _ints(_parents(c, starts, seed))
        n = s["n"] = s["parents"].numel()
    if own:
        from token_sparse_attention_gb300 import mcs
        s["p"] = mcs.paged(B, Hkv, Hkv, D, page, total, P, kv=mcs.KV_E4M3 if c["e4m3"] else mcs.KV_BF16, k_scale=s["scales"][0], v_scale=s["scales"][1])
        rows, moves = (n, n) if c["op"] == "fork" else (B, c["most"] or total // 2)
        s["out"] = dict(lens=_ints([0] * rows), table=torch.empty(rows, P, dtype=I32, device="cuda"), extra=torch.empty_like(s["extra"]),
                        free=s["free"].clone(), head=_ints([0]), moves=torch.empty(moves, 3, dtype=I32, device="cuda"))
        s["ws"] = mcs.empty_workspace(mcs.mcs_paged_fork_workspace(s["p"]) if c["op"] == "fork" else mcs.mcs_paged_compact_workspace(s["p"]))
    return s


def _parents(c, starts, seed):
    """Which sequence each new one goes on from (-1: an empty row)."""
    r = random.Random(seed)
    if c["kind"] == "reorder":  # every request's beams from its own, some of them twice, some not at all
        return [r.randrange(a, z) for a, z in zip(starts, starts[1:]) for _ in range(a, z)]
    on = [b for b in range(starts[-1]) if b % 9 != 5]  # every ninth ends
    return on + [-1] + [0] * c["more"]


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        return _call(s)
    op = s["c"]["op"]
    if op == "attn":
        return _attn(s)
    if op == "shared":
        return _decode(s)
    return _fork(s) if op == "fork" else _compact(s)


def _call(s):
    from token_sparse_attention_gb300 import mcs
    c = s["c"]
    if c["op"] in ("attn", "shared"):
        out, lse = s["out"]
        if c["op"] == "attn":
            mcs.mcs_paged_attn(s["p"], s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["cu"], out, s["ws"], lse=lse)
        else:
            mcs.mcs_paged_decode_shared(s["p"], s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["starts"], s["shared"], out, s["ws"], lse=lse)
        return {"out": out, "lse": lse}
    o = s["out"]
    if c["op"] == "fork":
        mcs.mcs_paged_fork(s["p"], s["parents"], s["lens"], s["table"], s["extra"], s["free"], s["head"], o["lens"], o["table"], o["extra"], o["free"], o["head"], o["moves"], s["ws"])
    else:
        mcs.mcs_paged_compact(s["p"], s["lens"], s["table"], s["extra"], o["table"], o["extra"], o["free"], o["head"], o["moves"], s["ws"])
    mcs.mcs_paged_copy(s["p"], o["moves"], s["k_cache"], s["v_cache"], s["k_mean"])
    kept = {"table": o["table"], "extra": o["extra"], "free": o["free"], "head": o["head"], "moves": o["moves"], **_held(s)}
    return {"lens": o["lens"], **kept} if c["op"] == "fork" else kept


def _held(s):
    values = (lambda x: x.view(torch.float8_e4m3fn)) if s["c"]["e4m3"] else (lambda x: x)
    return {"k_cache": values(s["k_cache"]), "v_cache": values(s["v_cache"]), "k_mean": s["k_mean"]}


def _values(codes):
    return (codes.view(torch.float8_e4m3fn) if codes.dtype == torch.uint8 else codes).float()


def _keys(s, cache):
    """A cache in the order of the sequences' tokens [B, Hkv, longest, D], fp32."""
    x = _values(cache[s["table"].long().clamp(min=0)])  # [B, P, Hkv, page, D]
    return x.transpose(1, 2).flatten(2, 3)


def _softmax(s, score, v):
    """(sum of the weights' products with v, natural-log sum of exponentials), zeros and -inf for rows of nothing.  Writes over score."""
    top = score.amax(-1, keepdim=True)
    score.sub_(torch.where(top > -math.inf, top, 0.0)).exp_()
    total = score.sum(-1, keepdim=True)
    out = torch.matmul(score, v) * s["scales"][1] / torch.where(total > 0, total, 1.0)
    return out, (torch.log(total) + top)[..., 0]


def _attn(s):
    c = s["c"]
    B, Hq, Hkv, D = (c[k] for k in ("B", "Hq", "Hkv", "D"))
    lens, cu, most = s["lens"].long(), s["cu"].long(), s["most"]
    i = torch.arange(most, device="cuda")
    new = cu[1:] - cu[:-1]
    row = torch.where(i[None] < new[:, None], cu[:-1, None] + i[None], s["T"] - 1)  # [B, most]; the last row is no token's
    q = s["q"].float()[row].view(B, most, Hkv, -1, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    k, v = _keys(s, s["k_cache"]), _keys(s, s["v_cache"])
    key = torch.arange(k.shape[2], device="cuda")
    seen = key[None, None] <= (lens - new)[:, None, None] + i[None, :, None]  # [B, most, keys]
    seen &= i[None, :, None] < new[:, None, None]
    score = torch.matmul(q, k.transpose(2, 3)).mul_(s["scales"][0] / math.sqrt(D)).view(B, Hkv, -1, most, k.shape[2])
    score.masked_fill_(~seen[:, None, None], -math.inf)
    v = torch.where((key[None] < lens[:, None])[:, None, :, None], v, 0.0)
    out, lse = _softmax(s, score.view(B, Hkv, -1, k.shape[2]), v)
    outs, lses = torch.zeros(s["T"], Hq, D, dtype=BF16, device="cuda"), torch.zeros(s["T"], Hq, device="cuda")
    live = row < cu[-1]
    outs[row[live]] = out.view(B, Hkv, -1, most, D).permute(0, 3, 1, 2, 4).reshape(B, most, Hq, D)[live].to(BF16)
    lses[row[live]] = lse.view(B, Hkv, -1, most).permute(0, 3, 1, 2).reshape(B, most, Hq)[live]
    return {"out": outs, "lse": lses}


def _decode(s):
    """Each sequence over all of its pages."""
    c = s["c"]
    B, Hq, Hkv, D = s["lens"].numel(), c["Hq"], c["Hkv"], c["D"]
    k, v = _keys(s, s["k_cache"]), _keys(s, s["v_cache"])
    live = (torch.arange(k.shape[2], device="cuda")[None] < s["lens"].long()[:, None])[:, None, None]
    score = torch.matmul(s["q"].float().view(B, Hkv, -1, D), k.transpose(2, 3)).mul_(s["scales"][0] / math.sqrt(D))
    score.masked_fill_(~live, -math.inf)
    out, lse = _softmax(s, score, torch.where(live.transpose(2, 3), v, 0.0))
    return {"out": out.to(BF16).view(B, Hq, D), "lse": lse.view(B, Hq)}


def _fork(s):
    page, n, total = s["c"]["page"], s["n"], s["extra"].numel()
    parents, lens, table = s["parents"].long(), s["lens"].long(), s["table"].long()
    extra, free, head = s["extra"].long(), s["free"].long().clone(), s["head"].long()
    B, P = table.shape
    j, i = torch.arange(P, device="cuda"), torch.arange(n, device="cuda")
    at = parents.clamp(min=0)
    lens_out = torch.where(parents >= 0, lens[at], 0)
    pages = (lens_out + page - 1) // page
    last = (lens_out - 1).clamp(min=0) // page  # the page that is not full, where there is one
    open_page = table[at, last]
    first = torch.full((B,), n, device="cuda").scatter_reduce(0, at, torch.where(parents >= 0, i, n), "amin")
    keeps = (first[at] == i) & (extra[open_page.clamp(min=0)] == 0)
    copies = (lens_out % page > 0) & ~keeps
    rank = copies.long().cumsum(0) - 1
    fresh = free[(head + rank).clamp(0, total - 1)]
    table_out = torch.where(j[None] < pages[:, None], table[at], -1)
    table_out = torch.where(copies[:, None] & (j[None] == last[:, None]), fresh[:, None], table_out)
    moves = torch.where(copies[:, None], torch.stack([open_page, fresh, lens_out % page], 1), torch.tensor([-1, -1, 0], device="cuda"))
    held = (j[None] < ((lens + page - 1) // page)[:, None])
    change = torch.zeros(total + 1, dtype=torch.int64, device="cuda")  # (the last for entries that are no page)
    change.scatter_add_(0, torch.where(held, table, total).flatten(), torch.full((B * P,), -1, device="cuda"))
    change.scatter_add_(0, torch.where(table_out >= 0, table_out, total).flatten(), torch.ones(n * P, dtype=torch.int64, device="cuda"))
    change = change[:total]
    handed = torch.zeros(total + 1, dtype=torch.bool, device="cuda").scatter(0, torch.where(copies, fresh, total), True)[:total]
    holders = torch.where(handed, 1, extra + 1 + change)
    gone = (holders == 0) & (change < 0)
    extra_out = torch.where(gone, 0, holders - 1)
    count = gone.sum()
    head_out = head + copies.sum() - count
    slot = head_out + gone.long().cumsum(0) - 1  # the freed pages, ascending, from head_out on
    free = torch.cat([free, free[:1]]).scatter(0, torch.where(gone, slot, total), torch.arange(total, device="cuda"))[:total]
    _copy(s, moves)
    out = {"lens": lens_out, "table": table_out, "extra": extra_out, "free": free, "head": head_out, "moves": moves}
    return {**{k: v.to(I32) for k, v in out.items()}, **_held(s)}


def _compact(s):
    c, page, total = s["c"], s["c"]["page"], s["extra"].numel()
    lens, table, extra = s["lens"].long(), s["table"].long(), s["extra"].long()
    j, number = torch.arange(table.shape[1], device="cuda"), torch.arange(total, device="cuda")
    rows = (lens[:, None] - j[None] * page).clamp(0, page)  # tokens of each entry's page
    fill = torch.zeros(total + 1, dtype=torch.int64, device="cuda")
    fill = fill.scatter_reduce(0, torch.where(rows > 0, table, total).flatten(), rows.flatten(), "amax")[:total]
    used = fill > 0
    above = used.long().flip(0).cumsum(0).flip(0) - 1  # used pages behind each
    below = (~used).long().cumsum(0) - 1               # free pages in front of each
    most = c["most"] or total // 2
    # the i-th used page from the back goes to the i-th free one from the front, while that lies in front of it
    source = torch.full((total + 1,), -1, device="cuda").scatter(0, torch.where(used, above, total), number)[:most]
    target = torch.full((total + 1,), total, device="cuda").scatter(0, torch.where(used, total, below), number)[:most]
    go = source > target
    source, target = torch.where(go, source, total), torch.where(go, target, total)
    pad = lambda x: torch.cat([x, x[:1]])  # one more place, for what moves nowhere
    to = pad(number).scatter(0, source, target)[:total]
    moves = torch.where(go[:, None], torch.stack([source, target, pad(fill)[source]], 1), torch.tensor([-1, -1, 0], device="cuda"))
    table_out = torch.where(rows > 0, to[table.clamp(min=0)], table)
    now = pad(used).scatter(0, source, False).scatter(0, target, True)[:total]
    extra_out = pad(torch.where(used, extra, 0)).scatter(0, target, pad(extra)[source]).scatter(0, source, 0)[:total]
    count = (~now).sum()
    head_out = total - count
    slot = head_out + (~now).long().cumsum(0) - 1
    free = pad(s["free"].long()).scatter(0, torch.where(now, total, slot), number)[:total]
    _copy(s, moves)
    out = {"table": table_out, "extra": extra_out, "free": free, "head": head_out.view(1), "moves": moves}
    return {**{k: v.to(I32) for k, v in out.items()}, **_held(s)}


def _copy(s, moves):
    """The first rows of pages to other pages."""
    page = s["c"]["page"]
    src, dst, rows = moves[moves[:, 0] >= 0].unbind(1)
    live = (torch.arange(page, device="cuda")[None] < rows[:, None])[:, None, :, None]
    for cache in (s["k_cache"], s["v_cache"]):
        cache[dst] = torch.where(live, cache[src], cache[dst])
    s["k_mean"][dst] = s["k_mean"][src]


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c, page, size = case, case["page"], 1 if case["e4m3"] else 2
    row = c["Hkv"] * c["D"] * size
    if c["op"] == "attn":
        before, new = _sizes(c)
        seen = sum(n * a + n * (n + 1) // 2 for a, n in zip(before, new))
        keys = sum(a + n for a, n in zip(before, new) if n)
        return {"bytes": 2 * keys * row + sum(new) * c["Hq"] * (4 * c["D"] + 4), "flops": 4 * seen * c["Hq"] * c["D"]}
    prompt, after = _sizes(c)
    lens = [[p + x for x in a] for p, a in zip(prompt, after)]
    flat = [x for a in lens for x in a]
    if c["op"] == "shared":
        common = [p // page * page for p in prompt]
        keys = sum(common) + sum(x - m for a, m in zip(lens, common) for x in a)
        return {"bytes": 2 * keys * row + len(flat) * c["Hq"] * (4 * c["D"] + 4), "flops": 4 * sum(flat) * c["Hq"] * c["D"]}
    pages = [-(-x // page) for x in flat]
    P, distinct = max(pages) + 2, sum(p // page + sum(-(-x // page) - p // page for x in a) for p, a in zip(prompt, lens))
    total = distinct + c.get("spare", 200)
    if c["op"] == "fork":
        starts = [k * c["W"] for k in range(c["R"] + 1)]
        parents = _parents(c, starts, 0)
        seen, tokens = set(), 0
        for p in parents:
            tokens += flat[p] % page if p in seen else 0
            seen.add(p)
        return {"bytes": 4 * tokens * row + 4 * sum(pages) + 4 * len(parents) * (P + 5) + 8 * total, "flops": 0}
    # pages behind the first `distinct` numbers, which any numbering has to empty
    moved = min(c["most"] or total // 2, distinct * c.get("spare", 200) // total)
    held = sum(flat) * distinct // max(1, sum(pages)) * moved // max(1, distinct)
    return {"bytes": 4 * held * row + 8 * sum(pages) + 12 * total, "flops": 0}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] in ("fork", "compact"):
        return _exact_pages(c, s)
    Hq, Hkv, D, page = (c[k] for k in ("Hq", "Hkv", "D", "page"))
    group, rows = Hq // Hkv, s["q"].shape[0]
    out = torch.zeros(rows, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(rows, Hq, dtype=torch.float64, device="cuda")
    at = 0
    for b, n in enumerate(s["lens"].tolist()):
        new = _sizes(c)[1][b] if c["op"] == "attn" else 1
        pages = s["table"][b, : -(-n // page)].long()
        for h in range(Hkv):
            k, v = (x[pages, h].reshape(-1, D)[:n] for x in (s["k_cache"], s["v_cache"]))
            k, v = ((x.view(torch.float8_e4m3fn) if c["e4m3"] else x).double() * f for x, f in zip((k, v), s["scales"]))
            heads = slice(h * group, (h + 1) * group)
            for a in range(0, new, 512):
                m = min(512, new - a)
                last = n - new + a + m  # keys that the piece's last token sees
                z = torch.einsum("thd,kd->htk", s["q"][at + a: at + a + m, heads].double(), k[:last]) / math.sqrt(D)
                hidden = torch.ones(m, last, dtype=torch.bool, device="cuda").triu(last - m + 1)
                z = z.masked_fill(hidden, -math.inf)
                lse[at + a: at + a + m, heads] = torch.logsumexp(z, -1).T
                out[at + a: at + a + m, heads] = torch.einsum("htk,kd->thd", torch.softmax(z, -1), v[:last])
        at += new
    return {"out": out, "lse": lse}


def _exact_pages(c, s):
    """The copied pages, from a walk over the sequences; whole numbers have no value in 64 bits of their own."""
    page, lens, table = c["page"], s["lens"].tolist(), s["table"].tolist()
    moves = []
    if c["op"] == "fork":
        free, extra, taken, kept = s["free"].tolist(), s["extra"].tolist(), int(s["head"]), set()
        for p in s["parents"].tolist():
            if p < 0 or lens[p] % page == 0:
                continue
            pid = table[p][lens[p] // page]
            if p in kept or extra[pid]:
                moves.append((pid, free[taken], lens[p] % page))
                taken += 1
            kept.add(p)
    else:
        held = {}
        for b, n in enumerate(lens):
            for t in range(0, n, page):
                held[table[b][t // page]] = min(page, n - t)
        total = s["extra"].numel()
        holes = [x for x in range(total) if x not in held]
        for src, dst in list(zip(sorted(held, reverse=True), holes))[: c["most"] or total // 2]:
            if src > dst:
                moves.append((src, dst, held[src]))
    got = {}
    for name in ("k_cache", "v_cache"):
        x = (s[name].view(torch.float8_e4m3fn) if c["e4m3"] else s[name]).double()
        for src, dst, rows in moves:
            x[dst, :, :rows] = x[src, :, :rows]
        got[name] = x
    mean = s["k_mean"].double()
    for src, dst, _ in moves:
        mean[dst] = mean[src]
    names = ["table", "extra", "free", "head", "moves"]
    return {**{k: None for k in (["lens"] if c["op"] == "fork" else []) + names}, **got, "k_mean": mean}
