"""Operators over the paged key-value cache: their cases, plain forms and 64-bit definitions.

- ``prompt_attention``: causal attention of packed prompt rows over the cache.
- ``prompt_weights``: the attention weight that those rows give each cached token.
- ``attention_weights``: attention of one new token per sequence, adding its weights.
- ``evict``: keeps the recent and the heaviest tokens of each sequence and head.

The cache is ``[blocks, kv heads, 16, head_dim]`` fp16 for K and for V, the
accumulated weights ``[blocks, kv heads, 16]`` fp32; a block table maps each
sequence's tokens to blocks.
"""
import math
import random

import torch

own = False

BLOCK = 16
MAX_CTX = 16384
DEVICE = "cuda" if torch.cuda.is_available() else "cpu"

# (query heads, kv heads, head_dim) of the repository's shapes and tests
HEADS = {"tiny": (4, 2, 64), "1b": (32, 8, 64), "8b": (32, 8, 128), "34b": (64, 8, 128),
         "mha": (16, 16, 64), "pair": (8, 4, 128)}


def _prompt(name, op, heads, seqs, new, past=(0, 0), lens_seed=1):
    return {"name": name, "op": op, "heads": heads, "seqs": seqs, "new_min": new[0], "new_max": new[1],
            "past_min": past[0], "past_max": past[1], "lens_seed": lens_seed}


def _decode(name, heads, seqs, ctx, lens_seed=1):
    return {"name": name, "op": "attention_weights", "heads": heads, "seqs": seqs, "ctx_min": ctx[0], "ctx_max": ctx[1],
            "lens_seed": lens_seed}


def _evict(name, heads, seqs, ctx, keep, recent, lens_seed=1):
    return {"name": name, "op": "evict", "heads": heads, "seqs": seqs, "ctx_min": ctx[0], "ctx_max": ctx[1], "keep": keep,
            "recent": recent, "lens_seed": lens_seed}


def listed():
    return [
        # one short prompt of a small model: latency counts
        _prompt("prompt 1b 512", "prompt_attention", "1b", 1, (512, 512)),
        # a batch of prompts of different lengths, packed
        _prompt("prompt 8b pack of 32", "prompt_attention", "8b", 32, (256, 2048), lens_seed=1237),
        # the longest prompt the library takes
        _prompt("prompt 8b 16384", "prompt_attention", "8b", 1, (16384, 16384)),
        # chunks of a few rows behind long cached prefixes
        _prompt("chunk 34b behind 4096", "prompt_attention", "34b", 8, (3, 61), (3001, 4096), 34),
        # what a short prompt's tokens weigh
        _prompt("weights 1b 512", "prompt_weights", "1b", 1, (512, 512)),
        # what the tokens of eight long prompts of a large model weigh
        _prompt("weights 34b 8 x 4096", "prompt_weights", "34b", 8, (4096, 4096)),
        # the smallest decode step: a few dozen tokens
        _decode("decode tiny", "tiny", 1, (33, 33)),
        # one sequence behind its prompt
        _decode("decode 8b one", "8b", 1, (2113, 2113)),
        # a batch of sequences of different lengths
        _decode("decode 8b batch of 32", "8b", 32, (257, 2176), 1237),
        # a short history cut to a small budget
        _evict("evict 1b 513 to 256", "1b", 1, (513, 513), 256, 32),
        # one very long history cut to a quarter
        _evict("evict 8b 16384 to 4096", "8b", 1, (16384, 16384), 4096, 256),
        # a batch of which some sequences are within the budget already
        _evict("evict 8b batch of 32", "8b", 32, (256, 2304), 1024, 64, 1237),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo..hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(("prompt_attention", "prompt_attention", "prompt_weights", "attention_weights", "attention_weights",
                     "evict"))
    heads = rng.choice(sorted(HEADS))
    n_heads = HEADS[heads][0]
    case = {"op": op, "heads": heads, "lens_seed": rng.randrange(1 << 20)}
    if op in ("prompt_attention", "prompt_weights"):
        # the padded scores of the plain form: at most half of the largest listed case's
        most = 8 * 64 * 4096 * 4096 // 2
        hi = _spread(rng, 16, 8192)
        past = rng.choice((0, 0, _spread(rng, 1, 6000)))
        fits = max(1, most // (n_heads * hi * (hi + past)))
        case["seqs"] = min(_spread(rng, 1, 32), fits)
        while case["seqs"] * n_heads * hi * (hi + past) > most:
            hi //= 2
        case.update(new_min=_spread(rng, 1, hi), new_max=hi, past_min=rng.randint(0, past), past_max=past)
    else:
        hi = _spread(rng, 2, MAX_CTX)
        case["seqs"] = max(1, min(_spread(rng, 1, 64), 64 * 2048 * 8 // (hi * HEADS[heads][1])))
        case.update(ctx_min=_spread(rng, 1, hi), ctx_max=hi)
        if op == "evict":
            case["keep"] = _spread(rng, 1, hi)
            case["recent"] = rng.randint(0, case["keep"])
    return case


def _lengths(case):
    """(new rows, cached tokens with them) of each sequence."""
    r = random.Random(case["lens_seed"])
    if case["op"] in ("prompt_attention", "prompt_weights"):
        new = [r.randint(case["new_min"], case["new_max"]) for _ in range(case["seqs"])]
        return new, [n + r.randint(case["past_min"], case["past_max"]) for n in new]
    return None, [r.randint(case["ctx_min"], case["ctx_max"]) for _ in range(case["seqs"])]


def _pairs(new, ctx):
    """(query row, key) pairs under the causal mask."""
    return sum(n * (c - n) + n * (n + 1) // 2 for n, c in zip(new, ctx))


def work(case):
    n_heads, n_kv, hd = HEADS[case["heads"]]
    new, ctx = _lengths(case)
    tokens, kv = sum(ctx), n_kv * hd * 2
    if case["op"] == "prompt_attention":
        rows = sum(new)
        return {"bytes": rows * n_heads * (2 * hd * 2 + 4) + 2 * tokens * kv, "flops": 4 * hd * n_heads * _pairs(new, ctx)}
    if case["op"] == "prompt_weights":
        rows = sum(new)
        return {"bytes": rows * n_heads * (hd * 2 + 4) + tokens * (kv + 8 * n_kv), "flops": 2 * hd * n_heads * _pairs(new, ctx)}
    if case["op"] == "attention_weights":
        return {"bytes": 2 * tokens * kv + case["seqs"] * n_heads * hd * 8 + tokens * n_kv * 8,
                "flops": 4 * hd * n_heads * tokens}
    kept = sum(min(c, case["keep"]) for c in ctx)
    return {"bytes": tokens * n_kv * 4 + kept * (2 * 2 * kv + n_kv * 4) + case["seqs"] * case["keep"] * n_kv * 4, "flops": 0}


def prepare(case, seed):
    n_heads, n_kv, hd = HEADS[case["heads"]]
    new, ctx = _lengths(case)
    g = torch.Generator(device=DEVICE).manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=DEVICE)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=DEVICE)

    per_seq = -(-max(ctx) // BLOCK)
    n_src = case["seqs"] * per_seq
    keep_blocks = -(-case["keep"] // BLOCK) if case["op"] == "evict" else 0
    n_blocks = n_src + case["seqs"] * keep_blocks
    # keys of real models differ in size, and the first token draws weight
    table = torch.randperm(n_src, generator=g, device=DEVICE).to(torch.int32).view(case["seqs"], per_seq)
    bias = randn(n_kv, 1, hd)
    size = 0.6 + 0.8 * torch.rand((n_blocks, n_kv, BLOCK, 1), generator=g, device=DEVICE)
    keys = randn(n_blocks, n_kv, BLOCK, hd) * size
    keys[table[:, 0].long(), :, 0] += bias[:, 0]
    s = {"op": case["op"], "n_heads": n_heads, "n_kv": n_kv, "hd": hd, "max_ctx": max(ctx), "table": table,
         "k": keys.half(), "ctx": ints(ctx)}
    del keys, size
    if case["op"] in ("attention_weights", "evict"):
        # accumulated so far: most tokens weigh little, some nothing at all
        w = randn(n_blocks, n_kv, BLOCK).square() * 0.5
        s["w"] = torch.where(w < 0.01, torch.zeros_like(w), w)
    if case["op"] != "prompt_weights":
        s["v"] = randn(n_blocks, n_kv, BLOCK, hd).half()
    if case["op"] == "evict":
        s["dst"] = n_src + torch.arange(case["seqs"] * keep_blocks, device=DEVICE, dtype=torch.int32).view(-1, keep_blocks)
        s["k"][n_src:], s["v"][n_src:], s["w"][n_src:] = 0, 0, 0
        s.update(keep=case["keep"], recent=case["recent"], n_src=n_src)
    elif case["op"] == "attention_weights":
        s["q"] = randn(case["seqs"], n_heads * hd) + bias.repeat_interleave(n_heads // n_kv, 0).view(1, -1) * 0.5
        s["pos"] = s["ctx"] - 1
    else:
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        s["q"] = (randn(cu[-1], n_heads * hd) + bias.repeat_interleave(n_heads // n_kv, 0).view(1, -1) * 0.5).half()
        s.update(cu=ints(cu), max_new=max(new))
        if case["op"] == "prompt_weights":
            s["w"] = torch.zeros(n_blocks, n_kv, BLOCK, device=DEVICE)
            # the rows' log-sum-exp, as the attention before leaves it
            sc = _scores(s, *_padded(s))
            s["lse"] = _rows(s, torch.logsumexp(sc, -1).view(*sc.shape[:3], -1)).permute(1, 0).contiguous()
    return s


# ------------------------------------------------------------ plain forms

def _history(cache, table, n):
    """The first n tokens of each sequence: [sequences, kv heads, n, ...] in 32 bits."""
    t = torch.arange(n, device=cache.device)
    x = cache[table[:, t // BLOCK].long(), :, t % BLOCK].float()
    return x.transpose(1, 2)


def _padded(s):
    """Queries [sequences, kv heads, group, rows, hd] and their positions [sequences, rows], padded to the longest."""
    i = torch.arange(s["max_new"], device=s["q"].device)
    n = s["cu"][1:] - s["cu"][:-1]
    rows = (s["cu"][:-1, None] + i).clamp(max=s["q"].shape[0] - 1).long()
    q = s["q"][rows].float().view(len(n), len(i), s["n_kv"], -1, s["hd"]).permute(0, 2, 3, 1, 4)
    pos = torch.where(i < n[:, None], s["ctx"][:, None] - n[:, None] + i, -1)
    return q, pos


def _scores(s, q, pos):
    """Masked scores [sequences, kv heads, group, rows, tokens]."""
    k = _history(s["k"], s["table"], s["max_ctx"])
    b, h, g, r, d = q.shape
    sc = torch.matmul((q * d ** -0.5).reshape(b, h, g * r, d), k.transpose(2, 3)).view(b, h, g, r, -1)
    t = torch.arange(s["max_ctx"], device=q.device)
    return sc.masked_fill_((t > pos[:, :, None])[:, None, None], -math.inf)


def _rows(s, x):
    """Padded rows [sequences, kv heads, group, rows, ...] packed again: [rows, heads, ...]."""
    n = s["cu"][1:] - s["cu"][:-1]
    b, h, g, r = x.shape[:4]
    live = torch.arange(r, device=x.device) < n[:, None]
    return x.permute(0, 3, 1, 2, *range(4, x.dim())).reshape(b, r, h * g, *x.shape[4:])[live]


def _add_weights(s, p):
    """Adds p [sequences, kv heads, tokens] to the tokens' accumulated weights."""
    t = torch.arange(s["max_ctx"], device=p.device)
    live = t < s["ctx"][:, None]
    blocks = s["table"][:, t // BLOCK].long()
    s["w"][blocks[live], :, (t % BLOCK).expand_as(blocks)[live]] += p.transpose(1, 2)[live]


def _plain_prompt_attention(s):
    sc = _scores(s, *_padded(s))
    m = sc.amax(-1, keepdim=True).clamp(min=-3e38)
    p = sc.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    v = _history(s["v"], s["table"], s["max_ctx"])
    b, h, g, r, t = p.shape
    o = torch.matmul(p.view(b, h, g * r, t), v).view(b, h, g, r, -1) / total
    lse = m + total.log()
    return _rows(s, o).reshape(s["q"].shape).half(), _rows(s, lse[..., 0]).permute(1, 0).contiguous()


def _plain_prompt_weights(s):
    q, pos = _padded(s)
    rows = s["lse"].view(s["n_kv"], -1, s["lse"].shape[1])
    at = (s["cu"][:-1, None] + torch.arange(s["max_new"], device=q.device)).clamp(max=rows.shape[2] - 1).long()
    lse = rows[:, :, at].permute(2, 0, 1, 3)
    p = _scores(s, q, pos).sub_(lse[..., None]).exp_()
    _add_weights(s, p.sum((2, 3)))
    return s["w"]


def _plain_attention_weights(s):
    k, v = (_history(s[x], s["table"], s["max_ctx"]) for x in "kv")
    q = s["q"].view(len(s["ctx"]), s["n_kv"], -1, s["hd"]) * s["hd"] ** -0.5
    sc = torch.matmul(q, k.transpose(2, 3))
    t = torch.arange(s["max_ctx"], device=q.device)
    sc.masked_fill_((t >= s["ctx"][:, None])[:, None, None], -math.inf)
    p = (sc - sc.amax(-1, keepdim=True)).exp()
    p = p / p.sum(-1, keepdim=True)
    _add_weights(s, p.sum(2))
    return torch.matmul(p, v).reshape(s["q"].shape), s["w"]


def _plain_evict(s):
    keep, recent, ctx = s["keep"], s["recent"], s["ctx"][:, None, None]
    t = torch.arange(s["max_ctx"], device=ctx.device)
    blocks = s["table"][:, t // BLOCK].long()
    w = s["w"][blocks, :, t % BLOCK].transpose(1, 2)
    # recent tokens before all others, tokens beyond the end after all others; equal weights by index
    w = torch.where(t >= ctx - recent, math.inf, w)
    w = torch.where(t >= ctx, -math.inf, w)
    best = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :keep]
    if best.shape[-1] < keep:
        best = torch.nn.functional.pad(best, (0, keep - best.shape[-1]), value=s["max_ctx"])
    kept = best.masked_fill(best >= ctx, 1 << 30).sort(-1).values
    live = kept < (1 << 30)
    seq, head, slot = live.nonzero(as_tuple=True)
    tok = kept[live]
    src = s["table"][seq, tok // BLOCK].long(), head, tok % BLOCK
    dst = s["dst"][seq, slot // BLOCK].long(), head, slot % BLOCK
    for x in "kvw":
        s[x][dst] = s[x][src]
    return kept.masked_fill(~live, -1).int(), s["ctx"].clamp(max=keep), s["k"], s["v"], s["w"]


# ------------------------------------------------------------ one pass

def run(s):
    op = s["op"]
    if own:
        import early_exit_decoding_layer_gb300 as ee
        shape = (s["n_heads"], s["n_kv"], s["hd"], s["max_ctx"])
        if op == "prompt_attention":
            out = ee.prompt_attention(s["q"], s["k"], s["v"], s["table"], s["cu"], s["ctx"], *shape)
        elif op == "prompt_weights":
            out = ee.prompt_weights(s["q"], s["k"], s["table"], s["cu"], s["ctx"], s["lse"], s["w"], *shape)
        elif op == "attention_weights":
            out = ee.attention_weights(s["q"], s["k"], s["v"], s["table"], s["pos"], s["w"], *shape), s["w"]
        else:
            out = ee.evict(s["k"], s["v"], s["w"], s["table"], s["ctx"], s["keep"], s["recent"], s["max_ctx"],
                           dst_table=s["dst"]) + (s["k"], s["v"], s["w"])
    elif op == "prompt_attention":
        out = _plain_prompt_attention(s)
    elif op == "prompt_weights":
        out = _plain_prompt_weights(s)
    elif op == "attention_weights":
        out = _plain_attention_weights(s)
    else:
        out = _plain_evict(s)
    if op == "evict":
        kept, length, k, v, w = out
        return {"kept": kept, "length": length, "k": k[s["n_src"]:], "v": v[s["n_src"]:], "w": w[s["n_src"]:]}
    if op == "prompt_weights":
        return {"w": out}
    return dict(zip(("o", "lse") if op == "prompt_attention" else ("o", "w"), out))


# ------------------------------------------------------------ from the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    n_heads, n_kv, hd = HEADS[case["heads"]]
    new, ctx = _lengths(case)
    if case["op"] == "evict":
        return None  # whole numbers, and values that are moved as they are
    group = n_heads // n_kv
    q = s["q"].view(-1, n_heads, hd)
    o = torch.zeros(q.shape, dtype=torch.float64, device=DEVICE)
    lse = torch.zeros((n_heads, q.shape[0]), dtype=torch.float64, device=DEVICE)
    w = s["w"].double() if "w" in s else None
    first = 0
    for b, c in enumerate(ctx):
        n = new[b] if new else 1
        for h in range(n_heads):
            blocks = s["table"][b, :-(-c // BLOCK)].long()
            keys = s["k"][blocks, h // group].reshape(-1, hd)[:c].double()
            vals = s["v"][blocks, h // group].reshape(-1, hd)[:c].double() if "v" in s else None
            weight = torch.zeros(c, dtype=torch.float64, device=DEVICE)
            for i in range(0, n, 2048):
                m = min(n, i + 2048)
                end = c - n + m  # no later key is seen by these rows
                z = q[first + i:first + m, h].double() @ keys[:end].T / math.sqrt(hd)
                row = torch.arange(c - n + i, end, device=DEVICE)
                z = z.masked_fill(torch.arange(end, device=DEVICE) > row[:, None], -math.inf)
                total = torch.logsumexp(z, 1)
                lse[h, first + i:first + m] = total
                if case["op"] == "prompt_weights":
                    total = s["lse"][h, first + i:first + m].double()
                p = torch.exp(z - total[:, None])
                if vals is not None:
                    o[first + i:first + m, h] = p @ vals[:end]
                weight[:end] += p.sum(0)
            if w is not None:
                full = torch.nn.functional.pad(weight, (0, len(blocks) * BLOCK - c))
                w[blocks, h // group] += full.view(-1, BLOCK)
        first += n
    o = o.view(s["q"].shape)
    if case["op"] == "prompt_attention":
        return {"o": o, "lse": lse}
    return {"w": w} if case["op"] == "prompt_weights" else {"o": o, "w": w}
