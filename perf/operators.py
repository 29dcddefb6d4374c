"""Cases, plain forms and calls of the paged-decode and norm-and-rotate operators.

    plan      new tokens' pages and slots from the requests' lengths (mcs_paged_plan)
    write     new key and value rows into the pages, page means along (mcs_paged_write)
    decode    one new token per sequence against its pages (mcs_paged_decode)
    sparse    the same over the pages a cheap score keeps (mcs_paged_select, mcs_paged_decode_sparse)
    norm      RMS norm per head of queries and keys, and their rotation (mcs_qk_norm_rope)
    norm_grad its gradients (mcs_qk_norm_rope_backward)

With `own` false run() computes an operator in elementary torch operations, in
32 bits or more, rounded once; with `own` true it calls the library.  exact()
is a separate 64-bit statement of each definition.
"""

import math
import random

import numpy as np
import torch

own = False

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
K_SCALE, V_SCALE = 3 / 256, 45 / 4096  # E4M3 caches: about the largest magnitude / 448
EPS = 1e-6


def listed():
    return [
        # one denoising step's projections at the large video workload (75600 tokens, 40 heads),
        # read in place from the fused projection
        dict(name="norm_video", op="norm", B=1, N=75600, Hq=40, Hkv=40, D=128, rot=128, interleaved=True, bhnd=True, fused=True, given=False, rows=75600),
        # one decoding step of 64 requests at far positions, rotated in part
        dict(name="norm_step", op="norm", B=64, N=1, Hq=32, Hkv=8, D=128, rot=64, interleaved=False, bhnd=False, fused=True, given=True, rows=75600),
        # tuning at the small video workload (32760 tokens, 12 heads): both gradients and the weights'
        dict(name="norm_grad_video", op="norm_grad", B=1, N=32760, Hq=12, Hkv=12, D=128, rot=128, interleaved=True, bhnd=True, fused=False, given=False, rows=32760),
        # a decoding step of a busy server: one token for each of 256 requests
        dict(name="plan_step", op="plan", B=256, page=16, longest=8192, new=1, spare=40),
        # long prompts admitted together, in pieces of uneven length
        dict(name="plan_prompts", op="plan", B=9, page=64, longest=40000, new=16000, spare=1000),
        # a prompt chunk's keys and values into a bf16 cache, page means along
        dict(name="write_prompts", op="write", B=5, page=64, longest=20000, new=7001, Hkv=8, D=128, e4m3=False, fused=True),
        # a decoding step's keys and values into an E4M3 cache
        dict(name="write_step", op="write", B=128, page=32, longest=4096, new=1, Hkv=8, D=128, e4m3=True, fused=True),
        # a single conversation, a short cache: latency
        dict(name="decode_one", op="decode", B=1, page=16, longest=1023, ragged=False, Hq=32, Hkv=8, D=128, e4m3=False, fused=True),
        # a server's ragged batch, an empty and a one-token sequence among it
        dict(name="decode_ragged", op="decode", B=48, page=32, longest=16001, ragged=True, Hq=32, Hkv=8, D=128, e4m3=False, fused=True),
        # contexts as long as the large video workload, E4M3 cache
        dict(name="decode_long", op="decode", B=12, page=64, longest=75600, ragged=False, Hq=40, Hkv=8, D=128, e4m3=True, fused=False),
        # one long sequence of the large workload's 40 heads, a fifth of its pages kept
        dict(name="sparse_one", op="sparse", B=1, page=16, longest=75600, ragged=False, Hq=40, Hkv=40, D=128, e4m3=False, fused=True, select=945, sink=1, recent=1),
        # a ragged batch at D = 64 (the 3D workload's 16 heads), E4M3 cache, 64 pages kept
        dict(name="sparse_batch", op="sparse", B=32, page=64, longest=32768, ragged=True, Hq=16, Hkv=16, D=64, e4m3=True, fused=False, select=64, sink=1, recent=2),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "plan", "write", "decode", "decode", "sparse", "sparse"])
    D, page = rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    Hkv, group = rng.choice([1, 2, 4, 5, 8, 10, 16]), rng.choice([1, 2, 4, 5, 8, 16, 20])
    if op in ("norm", "norm_grad"):
        B = rng.randint(1, 4)
        Hq = min(40, Hkv * group) // Hkv * Hkv
        N = _log(rng, 1, min(75600, 380_000_000 // (B * (Hq + Hkv) * D * (1 if op == "norm" else 4))))
        return dict(op=op, B=B, N=N, Hq=Hq, Hkv=Hkv, D=D, rot=rng.choice([D // 4, D // 2, D, D]), interleaved=rng.random() < 0.5,
                    bhnd=rng.random() < 0.5, fused=rng.random() < 0.5, given=rng.random() < 0.5, rows=N + rng.randint(0, 999))
    if op == "plan":
        new = _log(rng, 1, 16000)
        return dict(op=op, B=_log(rng, 1, max(1, min(1024, 100_000 // new))), page=page, longest=_log(rng, 1, 40000), new=new, spare=rng.randint(0, 999))
    e4m3, fused = rng.random() < 0.5, rng.random() < 0.5
    if op == "write":
        new = _log(rng, 1, 7000)
        return dict(op=op, B=_log(rng, 1, max(1, min(256, 28_000 // new))), page=page, longest=_log(rng, 1, 20000), new=new, Hkv=min(Hkv, 8), D=D, e4m3=e4m3, fused=fused)
    B = _log(rng, 1, 64)
    longest = _log(rng, 1, min(75600, 380_000_000 // (B * Hkv * D)))
    case = dict(op=op, B=B, page=page, longest=longest, ragged=rng.random() < 0.5, Hq=Hkv * group, Hkv=Hkv, D=D, e4m3=e4m3, fused=fused)
    if op == "sparse":
        sink, recent = rng.randint(0, 2), rng.randint(0, 2)
        case.update(select=max(_log(rng, 1, max(1, -(-longest // page) // 3)), sink + recent), sink=sink, recent=recent)
    return case


# ------------------------------------------------------------------ inputs

def _lengths(c, least=0):
    """Tokens in the cache of each sequence: a fixed choice for the case's sizes."""
    r = random.Random(1_000_003 * c["B"] + c["longest"])
    if not c.get("ragged", True):
        return [c["longest"]] * c["B"]
    lens = [max(least, int(c["longest"] ** r.uniform(0.6, 1.0))) for _ in range(c["B"])]
    lens[-1] = c["longest"]
    if c["B"] >= 4:
        lens[1], lens[2] = least, 1
    return lens


def _added(c):
    """New tokens of each sequence."""
    if c["new"] == 1:
        return [1] * c["B"]
    r = random.Random(7919 * c["B"] + c["new"])
    new = [int(c["new"] * r.uniform(0.3, 1.0)) for _ in range(c["B"])]
    new[-1] = c["new"]
    return new


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=F32)


def _ints(v):
    return torch.tensor(v, dtype=I32, device="cuda")


def _pages(lens, page, g, spare):
    """(block table [B, P], number of pages): the sequences' pages in random order, -1 behind them."""
    n = [-(-x // page) for x in lens]
    total, P = sum(n) + spare, max(1, max(n))
    table = torch.full((len(lens), P), -1, dtype=I32, device="cuda")
    live = torch.arange(P, device="cuda")[None] < _ints(n)[:, None]
    table[live] = torch.randperm(total, generator=g, device="cuda").to(I32)[: sum(n)]
    return table, total


def _fills(table, lens, page, total):
    """Tokens held by each page [total]."""
    pos = torch.arange(table.shape[1], device="cuda")[None] * page
    held = (_ints(lens)[:, None] - pos).clamp(0, page)
    fill = torch.zeros(total, dtype=torch.int64, device="cuda")
    fill[table[table >= 0].long()] = held[table >= 0].long()
    return fill


def _cache(g, total, Hkv, page, D, e4m3, scale, fill, level):
    """A cache whose pages are alike inside (a vector of their own plus noise); rows that hold no token are NaN."""
    out = torch.empty(total, Hkv, page, D, dtype=torch.uint8 if e4m3 else BF16, device="cuda")
    step = max(1, (1 << 26) // (Hkv * page * D))
    empty = torch.arange(page, device="cuda")[None] >= fill[:, None]
    for a in range(0, total, step):
        z = min(total, a + step)
        x = level * _randn(g, z - a, Hkv, 1, D) + 0.7 * _randn(g, z - a, Hkv, page, D)
        x = (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) if e4m3 else x.to(BF16)
        out[a:z] = x.masked_fill(empty[a:z, None, :, None], 0x7F if e4m3 else float("nan"))
    return out


def _values(codes):
    return (codes.view(torch.float8_e4m3fn) if codes.dtype == torch.uint8 else codes).float()


def _means(cache, fill, scale):
    """bf16 mean key of each page [pages, Hkv, D]; NaN where a page holds nothing."""
    total, Hkv, page, D = cache.shape
    out = torch.empty(total, Hkv, D, dtype=BF16, device="cuda")
    step = max(1, (1 << 26) // (Hkv * page * D))
    live = torch.arange(page, device="cuda")[None] < fill[:, None]
    for a in range(0, total, step):
        x = torch.where(live[a:a + step, None, :, None], _values(cache[a:a + step]) * scale, 0.0)
        out[a:a + step] = (x.sum(2) / fill[a:a + step, None, None]).to(BF16)
    return out


def _rows(g, T, H, D, fused, behind):
    """[T, H, D] bf16 rows: of their own, or a view into rows of a fused projection."""
    x = _randn(g, T, (H + behind) * D if fused else H * D).to(BF16)
    return x[:, : H * D].view(T, H, D)


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"c": c}
    if c["op"] in ("norm", "norm_grad"):
        B, N, Hq, Hkv, D, rot = (c[k] for k in ("B", "N", "Hq", "Hkv", "D", "rot"))
        if c["fused"]:
            x = torch.empty(B, N, (Hq + 2 * Hkv) * D, dtype=BF16, device="cuda")
            for b in range(B):
                x[b] = _randn(g, N, (Hq + 2 * Hkv) * D).to(BF16)
            s["q"] = x[..., : Hq * D].view(B, N, Hq, D)
            s["k"] = x[..., Hq * D: (Hq + Hkv) * D].view(B, N, Hkv, D)
        else:
            s["q"], s["k"] = (_randn(g, B, N, h, D).to(BF16) for h in (Hq, Hkv))
        s["wq"], s["wk"] = (1 + 0.2 * _randn(g, D) for _ in range(2))
        angle = torch.arange(c["rows"], device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        s["positions"] = torch.randint(0, c["rows"], (B, N), generator=g, device="cuda", dtype=I32) if c["given"] else None
        out = [(B, h, N, D) if c["bhnd"] else (B, N, h, D) for h in (Hq, Hkv)]
        if c["op"] == "norm_grad":
            s["dq_out"], s["dk_out"] = (_randn(g, *o).to(BF16) for o in out)
        if own:
            from token_sparse_attention_gb300 import mcs
            s["p"] = mcs.rope_params(B, N, Hq, Hkv, D, rot, c["rows"], interleaved=c["interleaved"], layout=mcs.LAYOUT_BHND if c["bhnd"] else mcs.LAYOUT_BNHD,
                                     eps=EPS, q_stride=(Hq + 2 * Hkv) * D if c["fused"] else 0, k_stride=(Hq + 2 * Hkv) * D if c["fused"] else 0)
            if c["op"] == "norm":
                s["out"] = [torch.empty(o, dtype=BF16, device="cuda") for o in out]
            else:
                # the gradients lie as the inputs do: in one buffer where q and k are views of one
                x = torch.empty(B, N, (Hq + 2 * Hkv) * D, dtype=BF16, device="cuda") if c["fused"] else None
                s["out"] = [x[..., : Hq * D].view(B, N, Hq, D), x[..., Hq * D: (Hq + Hkv) * D].view(B, N, Hkv, D)] if c["fused"] else \
                    [torch.empty(B, N, h, D, dtype=BF16, device="cuda") for h in (Hq, Hkv)]
                s["out"] += [torch.empty(D, device="cuda") for _ in range(2)]
                s["ws"] = mcs.empty_workspace(mcs.mcs_qk_norm_rope_backward_workspace(s["p"]))
        return s
    B, page = c["B"], c["page"]
    if c["op"] in ("plan", "write"):
        old, new = _lengths(c), _added(c)
        after = [a + n for a, n in zip(old, new)]
        table, total = _pages(after, page, g, c.get("spare", 7))
        have = _ints([-(-x // page) for x in old])[:, None]
        j = torch.arange(table.shape[1], device="cuda")[None]
        taken = table[(j >= have) & (table >= 0)]  # handed out by the plan, in this order
        head = 3  # free pages that earlier steps took
        s["free"] = torch.cat([torch.zeros(head, dtype=I32, device="cuda"), taken, torch.zeros(c.get("spare", 7), dtype=I32, device="cuda")])
        s["head"] = _ints([head])
        s["old"], s["new"], s["T"] = _ints(old), _ints(new), sum(new) + 5  # a step's buffers are a little longer than its tokens
        s["table"] = torch.where(j < have, table, -1)
        if c["op"] == "write":
            Hkv, D = c["Hkv"], c["D"]
            planned = _plan(s, page)
            s["slots"] = planned["slots"]
            s["scales"] = (K_SCALE, V_SCALE) if c["e4m3"] else (1.0, 1.0)
            fill = _fills(table, old, page, total)
            s["k_cache"] = _cache(g, total, Hkv, page, D, c["e4m3"], s["scales"][0], fill, 0.8)
            s["v_cache"] = _cache(g, total, Hkv, page, D, c["e4m3"], s["scales"][1], fill, 0.3)
            s["k_mean"] = _means(s["k_cache"], fill, s["scales"][0])
            for x in (s["k_cache"], s["v_cache"], s["k_mean"]):  # comparable: nothing undefined stays in what comes back
                x.nan_to_num_(0) if x.dtype == BF16 else x.masked_fill_(x == 0x7F, 0)
            s["k"], s["v"] = (_rows(g, s["T"], Hkv, D, c["fused"], 5 * Hkv) for _ in range(2))
            # the pages that get tokens and what they hold afterwards, as the plan's user knows them
            fresh = (j >= (_ints(old) // page)[:, None]) & (table >= 0) & (_ints(new) > 0)[:, None]
            s["touched"], s["held"] = table[fresh].long(), _fills(table, after, page, total)[table[fresh].long()]
        if own:
            from token_sparse_attention_gb300 import mcs
            if c["op"] == "plan":
                s["p"] = mcs.paged(B, 1, 1, 128, page, total, s["table"].shape[1])
                s["out"] = [torch.empty(n, dtype=I32, device="cuda") for n in (B, 1, B + 1, s["T"], s["T"])]
            else:
                s["p"] = mcs.paged(B, Hkv, Hkv, D, page, total, s["table"].shape[1], kv=mcs.KV_E4M3 if c["e4m3"] else mcs.KV_BF16,
                                   k_scale=s["scales"][0], v_scale=s["scales"][1], kv_stride=6 * Hkv * D if c["fused"] else 0)
        return s
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    lens = _lengths(c)
    s["table"], total = _pages(lens, page, g, 3)
    s["lens"] = _ints(lens)
    fill = _fills(s["table"], lens, page, total)
    s["scales"] = (K_SCALE, V_SCALE) if c["e4m3"] else (1.0, 1.0)
    s["k_cache"] = _cache(g, total, Hkv, page, D, c["e4m3"], s["scales"][0], fill, 0.8)
    s["v_cache"] = _cache(g, total, Hkv, page, D, c["e4m3"], s["scales"][1], fill, 0.3)
    s["q"] = _rows(g, B, Hq, D, c["fused"], 2 * Hkv)
    if c["op"] == "sparse":
        s["k_mean"] = _means(s["k_cache"], fill, s["scales"][0])
    if own:
        from token_sparse_attention_gb300 import mcs
        s["p"] = mcs.paged(B, Hq, Hkv, D, page, total, s["table"].shape[1], kv=mcs.KV_E4M3 if c["e4m3"] else mcs.KV_BF16,
                           k_scale=s["scales"][0], v_scale=s["scales"][1], q_stride=(Hq + 2 * Hkv) * D if c["fused"] else 0)
        s["out"] = [torch.empty(B, Hq, D, dtype=BF16, device="cuda"), torch.empty(B, Hq, device="cuda")]
        s["ws"] = mcs.empty_workspace(mcs.mcs_paged_decode_workspace(s["p"]))
        if c["op"] == "sparse":
            s["sel"] = torch.empty(B, Hkv, c["select"], dtype=I32, device="cuda")
            s["ws_select"] = mcs.empty_workspace(mcs.mcs_paged_select_workspace(s["p"]))
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    c = s["c"]
    if own:
        return _call(s)
    if c["op"] == "norm":
        at = _at(s)
        return [_laid(_rotate(_normed(s[x], s["w" + x])[0], at, c), c) for x in "qk"]
    if c["op"] == "norm_grad":
        at, grads, weights = _at(s), [], []
        for x in "qk":
            y = s["d%s_out" % x].float()
            got = _rotate(y.transpose(1, 2) if c["bhnd"] else y, at, c, back=True)
            hat, r = _normed(s[x], None)
            scaled = got * s["w" + x]
            grads.append((r * (scaled - hat * (scaled * hat).mean(-1, keepdim=True))).to(BF16))
            weights.append((got * hat).sum((0, 1, 2), dtype=torch.float64).float())
        return grads + weights
    if c["op"] == "plan":
        return _plan(s, c["page"])
    if c["op"] == "write":
        return _write(s)
    if c["op"] == "decode":
        out, lse = _attend(s, torch.arange(s["table"].shape[1], device="cuda", dtype=I32).expand(c["B"], c["Hkv"], -1))
        return {"out": out, "lse": lse}
    sel = _select(s)
    out, lse = _attend(s, sel)
    return {"sel": sel, "out": out, "lse": lse}


def _call(s):
    from token_sparse_attention_gb300 import mcs
    c = s["c"]
    if c["op"] == "norm":
        mcs.mcs_qk_norm_rope(s["p"], s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"], s["positions"], *s["out"])
        return s["out"]
    if c["op"] == "norm_grad":
        mcs.mcs_qk_norm_rope_backward(s["p"], s["dq_out"], s["dk_out"], s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"], s["positions"], *s["out"], s["ws"])
        return s["out"]
    if c["op"] == "plan":
        lens, head, cu, slots, positions = s["out"]
        mcs.mcs_paged_plan(s["p"], s["new"], s["old"], s["free"], s["head"], s["table"], lens, head, cu, slots, positions)
        return {"lens": lens, "head": head, "cu": cu, "slots": slots, "positions": positions, "table": s["table"]}
    if c["op"] == "write":
        mcs.mcs_paged_write(s["p"], s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], s["k_mean"])
        return _caches(s)
    out, lse = s["out"]
    if c["op"] == "decode":
        mcs.mcs_paged_decode(s["p"], s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], out, s["ws"], lse=lse)
        return {"out": out, "lse": lse}
    mcs.mcs_paged_select(s["p"], s["q"], s["k_mean"], s["table"], s["lens"], s["sel"], s["ws_select"], sink=c["sink"], recent=c["recent"])
    mcs.mcs_paged_decode_sparse(s["p"], s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["sel"], out, s["ws"], lse=lse)
    return {"sel": s["sel"], "out": out, "lse": lse}


def _caches(s):
    values = (lambda x: x.view(torch.float8_e4m3fn)) if s["c"]["e4m3"] else (lambda x: x)
    return {"k_cache": values(s["k_cache"]), "v_cache": values(s["v_cache"]), "k_mean": s["k_mean"]}


def _normed(x, w):
    """x / rms(x) (times w), and 1 / rms(x)."""
    x = x.float()
    r = 1 / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
    return (x * r if w is None else x * r * w), r


def _at(s):
    """Cosines and sines of every token [B or 1, N, 1, rot / 2]."""
    if s["positions"] is None:
        n = s["c"]["N"]
        return s["cos"][None, :n, None], s["sin"][None, :n, None]
    i = s["positions"].long()
    return s["cos"][i][:, :, None], s["sin"][i][:, :, None]


def _rotate(x, at, c, back=False):
    """The first `rot` values of each head rotated by their angles (back: by minus the angles)."""
    rot, (cos, sin) = c["rot"], at
    sin = -sin if back else sin
    if c["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([a, b], -1).flatten(-2) if c["interleaved"] else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _laid(x, c):
    x = x.to(BF16)
    return x.transpose(1, 2).contiguous() if c["bhnd"] else x


def _plan(s, page):
    old, new, table, free, head = (s[k].long() for k in ("old", "new", "table", "free", "head"))
    B, zero = len(old), torch.zeros(1, dtype=torch.int64, device="cuda")
    lens, cu = old + new, torch.cat([zero, new.cumsum(0)])
    have = (old + page - 1) // page
    need = (lens + page - 1) // page - have
    base = need.cumsum(0) - need
    j = torch.arange(table.shape[1], device="cuda")[None]
    fresh = (j >= have[:, None]) & (j < (have + need)[:, None])
    table = torch.where(fresh, free[(head + base[:, None] + j - have[:, None]).clamp(0, len(free) - 1)], table)
    t = torch.arange(s["T"], device="cuda")
    b = torch.searchsorted(cu[1:], t, right=True).clamp(max=B - 1)
    live = t < cu[-1]
    pos = torch.where(live, old[b] + t - cu[b], 0)
    slots = torch.where(live, table[b, pos // page] * page + pos % page, -1)
    got = {"lens": lens, "head": head + need.sum(), "cu": cu, "slots": slots, "positions": torch.where(live, pos, -1), "table": table}
    return {k: v.to(I32) for k, v in got.items()}


def _write(s):
    c, page = s["c"], s["c"]["page"]
    live = s["slots"] >= 0
    first = torch.argmax(live.int())  # a padding token repeats the first live one, which changes nothing
    slot = torch.where(live, s["slots"], s["slots"][first]).long()
    for x, cache, scale in ((s["k"], s["k_cache"], s["scales"][0]), (s["v"], s["v_cache"], s["scales"][1])):
        # (a tensor divides; a number would multiply by its rounded reciprocal)
        y = (x.float() / torch.full((1,), scale, device="cuda")).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) if c["e4m3"] else x
        cache[slot // page, :, slot % page] = torch.where(live[:, None, None], y, y[first])
    rows = _values(s["k_cache"][s["touched"]]) * s["scales"][0]
    held = torch.arange(page, device="cuda")[None] < s["held"][:, None]
    mean = torch.where(held[:, None, :, None], rows, 0.0).sum(2) / s["held"][:, None, None]
    s["k_mean"][s["touched"]] = mean.to(BF16)
    return _caches(s)


def _select(s):
    """The kept pages of each sequence and KV head, ascending, -1 behind them [B, Hkv, select]."""
    c, page = s["c"], s["c"]["page"]
    B, Hkv, P = c["B"], c["Hkv"], s["table"].shape[1]
    n = (s["lens"].long() + page - 1) // page
    q = s["q"].double().view(B, Hkv, -1, c["D"]).sum(2)
    mean = s["k_mean"][s["table"].long().clamp(min=0)].double()
    score = torch.einsum("bhd,bphd->bhp", q, mean).float()
    j = torch.arange(P, device="cuda")
    forced = (j[None] < c["sink"]) | (j[None] >= (n - c["recent"])[:, None])
    score = torch.where(forced[:, None], math.inf, score)
    score = torch.where((j[None] < n[:, None])[:, None], score, -math.inf)
    keep = min(c["select"], P)
    best = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :keep]
    best = torch.where(best < n[:, None, None], best, P).sort(-1).values  # pages past the end go last
    sel = torch.full((B, Hkv, c["select"]), -1, dtype=I32, device="cuda")
    sel[..., :keep] = torch.where(best < P, best, -1)
    return sel


def _attend(s, logical):
    """Attention of one token per sequence over the pages `logical` [B, Hkv, S] of its table."""
    c, page = s["c"], s["c"]["page"]
    B, Hkv, D, S = c["B"], c["Hkv"], c["D"], logical.shape[-1]
    at = logical.long()
    phys = s["table"].long()[:, None].expand(B, Hkv, -1).gather(2, at.clamp(min=0)).clamp(min=0)
    h = torch.arange(Hkv, device="cuda")[None, :, None]
    token = at[..., None] * page + torch.arange(page, device="cuda")
    live = ((at >= 0)[..., None] & (token < s["lens"].long()[:, None, None, None])).view(B, Hkv, 1, S * page)
    k = _values(s["k_cache"][phys, h]).view(B, Hkv, S * page, D)
    score = torch.matmul(s["q"].float().view(B, Hkv, -1, D), k.transpose(2, 3)) * (s["scales"][0] / math.sqrt(D))
    score = torch.where(live, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    e = torch.exp(score - torch.where(top > -math.inf, top, 0.0))
    total = e.sum(-1, keepdim=True)
    v = torch.where(live.transpose(2, 3), _values(s["v_cache"][phys, h]).view(B, Hkv, S * page, D), 0.0)
    out = torch.matmul(e, v) * s["scales"][1] / torch.where(total > 0, total, 1.0)
    return out.to(BF16).view(B, -1, D), (torch.log(total) + top).view(B, -1)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    if c["op"] in ("norm", "norm_grad"):
        n, tokens = c["B"] * c["N"] * (c["Hq"] + c["Hkv"]) * c["D"], c["B"] * c["N"]
        table = min(c["rows"], tokens) * c["rot"] * 4 + (4 * tokens if c["given"] else 0)
        return {"bytes": (4 if c["op"] == "norm" else 6) * n + table, "flops": (8 if c["op"] == "norm" else 16) * n}
    page = c["page"]
    if c["op"] in ("plan", "write"):
        old, new = _lengths(c), _added(c)
        fresh = sum(-(-(a + n) // page) - -(-a // page) for a, n in zip(old, new))
        if c["op"] == "plan":  # lengths in and out, free pages in, table entries out, slots and positions out
            return {"bytes": 16 * c["B"] + 8 * fresh + 8 * sum(new), "flops": 0}
        row, size = c["Hkv"] * c["D"], 1 if c["e4m3"] else 2
        started = sum(a % page for a, n in zip(old, new) if n)
        touched = sum(-(-(a + n) // page) - a // page for a, n in zip(old, new) if n)
        return {"bytes": sum(new) * (4 + 2 * row * (2 + size)) + started * row * size + touched * row * 2, "flops": 4 * row * sum(new)}
    Hq, Hkv, D, size = c["Hq"], c["Hkv"], c["D"], 1 if c["e4m3"] else 2
    lens = _lengths(c)
    pages = [-(-x // page) for x in lens]
    extra = flops = 0
    if c["op"] == "sparse":
        extra = sum(pages) * Hkv * D * 2 + sum(min(c["select"], n) for n in pages) * Hkv * 4
        flops = 2 * sum(pages) * Hkv * D
        lens = [min(x, c["select"] * page) for x in lens]
    moved = sum(lens) * Hkv * D * 2 * size + c["B"] * Hq * (4 * D + 4) + 4 * sum(pages)
    return {"bytes": moved + extra, "flops": 4 * sum(lens) * Hq * D + flops}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] == "plan":
        return None
    if c["op"] in ("norm", "norm_grad"):
        return _exact_norm(c, s)
    if c["op"] == "write":
        return _exact_write(c, s)
    B, Hq, Hkv, D, page = (c[k] for k in ("B", "Hq", "Hkv", "D", "page"))
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
    group = Hq // Hkv
    for b, n in enumerate(_lengths(c)):
        if n == 0:
            continue
        pages = s["table"][b, : -(-n // page)].long()
        for h in range(Hkv):
            q = s["q"][b, h * group: (h + 1) * group].double()
            kept = np.arange(len(pages))
            if c["op"] == "sparse":
                score = (q.sum(0) @ s["k_mean"][pages, h].double().T).cpu().numpy().astype(np.float32)
                score[: c["sink"]] = np.inf
                score[max(0, len(pages) - c["recent"]):] = np.inf
                kept = np.sort(np.lexsort((kept, -score))[: c["select"]])
            kept = torch.from_numpy(kept).cuda()
            count = len(kept) * page - ((len(pages) * page - n) if int(kept[-1]) == len(pages) - 1 else 0)
            k, v = (x[pages[kept], h].reshape(-1, D)[:count] for x in (s["k_cache"], s["v_cache"]))
            k, v = ((x.view(torch.float8_e4m3fn) if c["e4m3"] else x).double() * f for x, f in zip((k, v), s["scales"]))
            z = q @ k.T / math.sqrt(D)
            lse[b, h * group: (h + 1) * group] = torch.logsumexp(z, -1)
            out[b, h * group: (h + 1) * group] = torch.softmax(z, -1) @ v
    got = {"out": out, "lse": lse}
    return {"sel": None, **got} if c["op"] == "sparse" else got


def _exact_norm(c, s):
    B, N, D, rot, half = c["B"], c["N"], c["D"], c["rot"], c["rot"] // 2
    place = s["positions"].long() if c["given"] else torch.arange(N, device="cuda").expand(B, N)
    # the rotation as a complex factor per pair of values
    one = np.arange(0, rot, 2) if c["interleaved"] else np.arange(half)
    other = one + 1 if c["interleaved"] else one + half
    turn = torch.complex(s["cos"].double(), s["sin"].double())
    outs, weights = [], []
    for x in "qk":
        H = s[x].shape[2]
        forward = c["op"] == "norm"
        got = torch.empty((B, H, N, D) if c["bhnd"] and forward else (B, N, H, D), dtype=torch.float64, device="cuda")
        w, dw = s["w" + x].double(), torch.zeros(D, dtype=torch.float64, device="cuda")
        step = max(1, (1 << 25) // (H * D))
        for b in range(B):
            for a in range(0, N, step):
                v = s[x][b, a:a + step].double()
                size = torch.sqrt((v * v).sum(-1, keepdim=True) / D + EPS)
                unit = v / size
                t = turn[place[b, a:a + step]][:, None]
                if forward:
                    y = unit * w
                    z = torch.complex(y[..., one], y[..., other]) * t
                    y[..., one], y[..., other] = z.real, z.imag
                    if c["bhnd"]:
                        got[b, :, a:a + step] = y.transpose(0, 1)
                    else:
                        got[b, a:a + step] = y
                else:
                    y = s["d%s_out" % x]
                    y = (y[b, :, a:a + step].transpose(0, 1) if c["bhnd"] else y[b, a:a + step]).double()
                    z = torch.complex(y[..., one], y[..., other]) * t.conj()
                    y[..., one], y[..., other] = z.real, z.imag
                    dw += (y * unit).sum((0, 1))
                    y = y * w
                    got[b, a:a + step] = (y - unit * (y * unit).sum(-1, keepdim=True) / D) / size
        outs.append(got)
        weights.append(dw)
    return outs if c["op"] == "norm" else outs + weights


def _exact_write(c, s):
    page, total = c["page"], s["k_cache"].shape[0]
    slots = s["slots"].long()
    t = torch.nonzero(slots >= 0)[:, 0]
    got = {}
    for x, f in (("k", s["scales"][0]), ("v", s["scales"][1])):
        cache = s[x + "_cache"]
        held = (cache.view(torch.float8_e4m3fn) if c["e4m3"] else cache).double()
        new = s[x][t].double()
        if c["e4m3"]:
            new = (new / f).clamp(-448, 448).float().to(torch.float8_e4m3fn).double()
        held = held.transpose(1, 2).reshape(total * page, c["Hkv"], c["D"])
        held[slots[t]] = new
        got[x + "_cache"] = held.view(total, page, c["Hkv"], c["D"]).transpose(1, 2)
    mean = s["k_mean"].double()
    for p, n in zip(s["touched"].tolist(), s["held"].tolist()):
        mean[p] = (got["k_cache"][p, :, :n] * s["scales"][0]).sum(1) / n
    return {**got, "k_mean": mean}
