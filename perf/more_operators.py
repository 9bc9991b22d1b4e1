"""Operators of batches that share a prefix and of caches held in eight bits: their
cases, plain forms and 64-bit definitions.

- ``quantize_cache``: K and V rows of new tokens written into an eight-bit cache.
- ``dequantize_cache``: sequences of it read back into the fp16 cache.
- ``quantized_attention``: decode attention that reads the eight-bit cache.
- ``shared_attention``: decode attention of a batch whose sequences begin with the
  same tokens, over the fp16 cache.

The fp16 cache is ``[blocks, kv heads, 16, head_dim]`` for K and for V.  The eight-bit
cache holds both side by side, ``codes [blocks, kv heads, 2, 16, head_dim]`` in e4m3 and
``exponents [blocks, kv heads, 2, 16]`` in int8: a value is its code times 2 to the
exponent of its token's row.  A block table maps each sequence's tokens to blocks.
"""
import math
import random

import torch

own = False

BLOCK = 16
MAX_CTX = 16384
DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
E4M3_MAX = 448.0
E_MIN, HALF_END = -15, 65520.0  # the smallest exponent; what fp16 no longer holds

# (query heads, kv heads, head_dim) of the repository's shapes and tests
HEADS = {"tiny": (4, 2, 64), "1b": (32, 8, 64), "8b": (32, 8, 128), "34b": (64, 8, 128),
         "mha": (16, 16, 64), "pair": (8, 4, 128)}


def _write(name, heads, seqs, new, past=(0, 0), rows="fp16", lens_seed=1):
    return {"name": name, "op": "quantize_cache", "heads": heads, "seqs": seqs, "new_min": new[0], "new_max": new[1],
            "past_min": past[0], "past_max": past[1], "rows": rows, "lens_seed": lens_seed}


def _tokens(name, op, heads, seqs, ctx, lens_seed=1):
    return {"name": name, "op": op, "heads": heads, "seqs": seqs, "ctx_min": ctx[0], "ctx_max": ctx[1], "lens_seed": lens_seed}


def _shared(name, heads, seqs, prefix, tail, lens_seed=1):
    return {"name": name, "op": "shared_attention", "heads": heads, "seqs": seqs, "prefix": prefix, "tail_min": tail[0],
            "tail_max": tail[1], "lens_seed": lens_seed}


def listed():
    return [
        # one new token of one sequence, as a projection's fp32 output: latency counts
        _write("write 1b one token", "1b", 1, (1, 1), (512, 512), "fp32"),
        # a batch of prompts of different lengths, packed
        _write("write 8b pack of 32", "8b", 32, (256, 2048), lens_seed=1237),
        # a short history brought back for a chunk of its prompt
        _tokens("read 1b 513", "dequantize_cache", "1b", 1, (513, 513)),
        # a batch of histories brought back
        _tokens("read 8b batch of 32", "dequantize_cache", "8b", 32, (257, 2176), 1237),
        # the smallest decode step: a few dozen tokens
        _tokens("decode tiny", "quantized_attention", "tiny", 1, (33, 33)),
        # one sequence behind its prompt
        _tokens("decode 8b one", "quantized_attention", "8b", 1, (2113, 2113)),
        # a batch of sequences of different lengths
        _tokens("decode 8b batch of 32", "quantized_attention", "8b", 32, (257, 2176), 1237),
        # long histories, the reason to hold them in eight bits
        _tokens("decode 34b 16 of 16384", "quantized_attention", "34b", 16, (15001, 16384), 34),
        # a few answers to one short prompt
        _shared("shared 1b 4 behind 512", "1b", 4, 512, (1, 33)),
        # a batch behind a system prompt
        _shared("shared 8b 32 behind 2048", "8b", 32, 2048, (17, 300), 1237),
        # the largest batch behind a long document
        _shared("shared 34b 64 behind 15000", "34b", 64, 15000, (1, 1300), 34),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo..hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(("quantize_cache", "dequantize_cache", "quantized_attention", "quantized_attention", "shared_attention",
                     "shared_attention"))
    heads = rng.choice(sorted(HEADS))
    n_kv = HEADS[heads][1]
    case = {"op": op, "heads": heads, "lens_seed": rng.randrange(1 << 20)}
    if op == "shared_attention":
        case["seqs"] = _spread(rng, 1, 64)
        case["prefix"] = _spread(rng, 8, 15000)
        hi = min(_spread(rng, 1, 4000), MAX_CTX - case["prefix"], max(1, 64 * 1300 * 8 // (case["seqs"] * n_kv)))
        case.update(tail_min=_spread(rng, 1, hi), tail_max=hi)
        return case
    hi = _spread(rng, 2, MAX_CTX)
    case["seqs"] = max(1, min(_spread(rng, 1, 64), 64 * 2048 * 8 // (hi * n_kv)))
    lo = _spread(rng, 1, hi)
    if op != "quantize_cache":
        case.update(ctx_min=lo, ctx_max=hi)
        return case
    # whole prompts, chunks or single tokens, behind what is there already
    new = rng.choice((1, hi, _spread(rng, 1, hi)))
    past = rng.choice((0, MAX_CTX - new, rng.randint(0, MAX_CTX - new))) if case["seqs"] * n_kv <= 128 else 0
    case.update(new_min=min(lo, new), new_max=new, past_min=rng.randint(0, past), past_max=past, rows=rng.choice(("fp16", "fp32")))
    return case


def _lengths(case):
    """(new rows, cached tokens with them) of each sequence."""
    r = random.Random(case["lens_seed"])
    if case["op"] == "quantize_cache":
        new = [r.randint(case["new_min"], case["new_max"]) for _ in range(case["seqs"])]
        return new, [n + r.randint(case["past_min"], case["past_max"]) for n in new]
    if case["op"] == "shared_attention":
        return None, [case["prefix"] + r.randint(case["tail_min"], case["tail_max"]) for _ in range(case["seqs"])]
    return None, [r.randint(case["ctx_min"], case["ctx_max"]) for _ in range(case["seqs"])]


def work(case):
    n_heads, n_kv, hd = HEADS[case["heads"]]
    new, ctx = _lengths(case)
    tokens, held = sum(ctx), n_kv * (2 * hd + 2)  # bytes of a token in the eight-bit cache
    if case["op"] == "quantize_cache":
        return {"bytes": sum(new) * (2 * n_kv * hd * (4 if case["rows"] == "fp32" else 2) + held), "flops": 0}
    if case["op"] == "dequantize_cache":
        return {"bytes": tokens * (held + 4 * n_kv * hd), "flops": 0}
    rows = case["seqs"] * n_heads * hd * 4
    if case["op"] == "quantized_attention":
        return {"bytes": tokens * held + rows, "flops": 4 * hd * n_heads * tokens}
    once = case["prefix"] // BLOCK * BLOCK  # whole blocks are shared
    return {"bytes": (tokens - (case["seqs"] - 1) * once) * 4 * n_kv * hd + rows, "flops": 4 * hd * n_heads * tokens}


def prepare(case, seed):
    n_heads, n_kv, hd = HEADS[case["heads"]]
    new, ctx = _lengths(case)
    op, seqs = case["op"], case["seqs"]
    g = torch.Generator(device=DEVICE).manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=DEVICE)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=DEVICE)

    def keys_and_values(n):
        """n tokens' K and V [n, kv heads, hd]: tokens differ in size, and some channels of K are large."""
        k = randn(n, n_kv, hd) * (0.6 + 0.8 * torch.rand((n, n_kv, 1), generator=g, device=DEVICE))
        k[..., :: hd // 4] *= 4
        return k, randn(n, n_kv, hd) * (0.3 + torch.rand((n, n_kv, 1), generator=g, device=DEVICE))

    per_seq = -(-max(ctx) // BLOCK)
    s = {"op": op, "n_heads": n_heads, "n_kv": n_kv, "hd": hd, "max_ctx": max(ctx), "ctx": ints(ctx)}
    if op == "shared_attention":
        first = case["prefix"] // BLOCK
        own_blocks = per_seq - first
        order = torch.randperm(first + seqs * own_blocks, generator=g, device=DEVICE).to(torch.int32)
        s["table"] = torch.cat([order[:first].expand(seqs, first), order[first:].view(seqs, own_blocks)], 1).contiguous()
        s["prefix"] = case["prefix"]
        n_blocks = len(order)
    else:
        n_blocks = seqs * per_seq
        s["table"] = torch.randperm(n_blocks, generator=g, device=DEVICE).to(torch.int32).view(seqs, per_seq)
    if op == "quantize_cache":
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        k, v = keys_and_values(cu[-1])
        t = torch.float32 if case["rows"] == "fp32" else torch.float16
        s.update(k=k.to(t).view(cu[-1], -1), v=v.to(t).view(cu[-1], -1), cu=ints(cu))
        s["codes"] = torch.zeros(n_blocks, n_kv, 2, BLOCK, hd, dtype=torch.uint8, device=DEVICE)
        s["exps"] = torch.zeros(n_blocks, n_kv, 2, BLOCK, dtype=torch.int8, device=DEVICE)
        return s
    k, v = (x.view(n_blocks, BLOCK, n_kv, hd).transpose(1, 2).half().contiguous() for x in keys_and_values(n_blocks * BLOCK))
    if op != "shared_attention":
        codes, s["exps"] = _quantized(torch.stack((k, v), 2).float())
        s["codes"] = codes.view(torch.uint8)
    if op == "dequantize_cache":
        s["k"], s["v"] = torch.zeros_like(k), torch.zeros_like(v)
        s["dst"] = torch.randperm(n_blocks, generator=g, device=DEVICE).to(torch.int32).view(seqs, per_seq)
        return s
    if op == "shared_attention":
        s["k"], s["v"] = k, v
    # the first token draws weight
    at = k[s["table"][0, 0].long(), :, 0].float().repeat_interleave(n_heads // n_kv, 0)
    s["q"] = (randn(seqs, n_heads, hd) + 2 * at / at.norm(dim=-1, keepdim=True)).half().view(seqs, -1)
    s["pos"] = s["ctx"] - 1
    return s


# ------------------------------------------------------------ plain forms

def _quantized(x):
    """Rows of x as (codes in e4m3, exponents): the least exponent, -15 or more, with which a row's
    largest finite value is at most 448 codes; what fp16 does not hold is NaN."""
    x = torch.where(x.abs() < HALF_END, x, math.nan)
    big = torch.nan_to_num(x.abs(), nan=0.0).amax(-1)
    part, exponent = torch.frexp(big)  # big = part * 2^exponent, 448 = 0.875 * 2^9
    e = (exponent - 9 + (part > 0.875).int()).clamp(min=E_MIN)
    e = torch.where(big > 0, e, E_MIN)
    return torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn), e.to(torch.int8)


def _values(codes, exps):
    return torch.ldexp(codes.view(torch.float8_e4m3fn).float(), exps.int()[..., None])


def _plain_quantize_cache(s):
    n = s["cu"][1:] - s["cu"][:-1]
    row = torch.arange(s["k"].shape[0], device=n.device)
    seq = torch.searchsorted(s["cu"], row, right=True) - 1
    pos = s["ctx"][seq] - s["cu"][seq + 1] + row
    x = torch.stack((s["k"], s["v"]), 1).float().view(len(row), 2, s["n_kv"], s["hd"]).transpose(1, 2)
    codes, exps = _quantized(x)
    block, slot = s["table"][seq, pos // BLOCK].long(), pos % BLOCK
    s["codes"][block, :, :, slot] = codes.view(torch.uint8)
    s["exps"][block, :, :, slot] = exps
    return s["codes"], s["exps"]


def _plain_dequantize_cache(s):
    t = torch.arange(s["max_ctx"], device=s["ctx"].device)
    seq, tok = (t < s["ctx"][:, None]).nonzero(as_tuple=True)
    src, dst, slot = s["table"][seq, tok // BLOCK].long(), s["dst"][seq, tok // BLOCK].long(), tok % BLOCK
    x = _values(s["codes"][src, :, :, slot], s["exps"][src, :, :, slot]).clamp(-65504, 65504).half()
    s["k"][dst, :, slot], s["v"][dst, :, slot] = x[:, :, 0], x[:, :, 1]
    return s["k"], s["v"]


def _softmax(z):
    p = (z - z.amax(-1, keepdim=True)).exp()
    return p / p.sum(-1, keepdim=True)


def _plain_quantized_attention(s):
    t = torch.arange(s["max_ctx"], device=s["ctx"].device)
    at = s["table"][:, t // BLOCK].long(), slice(None), slice(None), t % BLOCK
    k, v = _values(s["codes"][at], s["exps"][at]).permute(3, 0, 2, 1, 4)  # [sequences, kv heads, tokens, hd]
    q = s["q"].float().view(len(s["ctx"]), s["n_kv"], -1, s["hd"]) * s["hd"] ** -0.5
    z = torch.matmul(q, k.transpose(2, 3)).masked_fill_((t >= s["ctx"][:, None])[:, None, None], -math.inf)
    return torch.matmul(_softmax(z), v).reshape(s["q"].shape).half()


def _plain_shared_attention(s):
    # the shared blocks once for all rows, the rest of each sequence by itself
    b, h, d, once = len(s["ctx"]), s["n_kv"], s["hd"], s["prefix"] // BLOCK
    q = s["q"].float().view(b, h, -1, d) * d ** -0.5
    shared = [s[x][s["table"][0, :once].long()].transpose(0, 1).reshape(h, -1, d).float() for x in "kv"]
    tails = [s[x][s["table"][:, once:].long()].transpose(1, 2).reshape(b, h, -1, d).float() for x in "kv"]
    rows = q.transpose(0, 1).reshape(h, -1, d)
    zs = torch.matmul(rows, shared[0].transpose(1, 2)).view(h, b, q.shape[2], once * BLOCK).transpose(0, 1)
    t = once * BLOCK + torch.arange(tails[0].shape[2], device=q.device)
    zt = torch.matmul(q, tails[0].transpose(2, 3)).masked_fill_((t >= s["ctx"][:, None])[:, None, None], -math.inf)
    p = _softmax(torch.cat((zs, zt), -1))
    ps = p[..., : once * BLOCK].transpose(0, 1).reshape(*rows.shape[:2], once * BLOCK)
    o = torch.matmul(ps, shared[1]).view(h, b, q.shape[2], d).transpose(0, 1) + torch.matmul(p[..., once * BLOCK:], tails[1])
    return o.reshape(s["q"].shape).half()


# ------------------------------------------------------------ one pass

def run(s):
    op = s["op"]
    if own:
        import early_exit_decoding_layer_gb300 as ee
        shape = (s["n_heads"], s["n_kv"], s["hd"], s["max_ctx"])
        if op == "quantize_cache":
            out = ee.quantize_cache(s["k"], s["v"], s["codes"], s["exps"], s["table"], s["cu"], s["ctx"], s["max_ctx"])
        elif op == "dequantize_cache":
            out = ee.dequantize_cache(s["codes"], s["exps"], s["table"], s["ctx"], s["k"], s["v"], s["max_ctx"], dst_table=s["dst"])
        elif op == "quantized_attention":
            out = ee.quantized_attention(s["q"], s["codes"], s["exps"], s["table"], s["pos"], *shape)
        else:
            out = ee.shared_attention(s["q"], s["k"], s["v"], s["table"], s["pos"], s["prefix"], *shape)
    elif op == "quantize_cache":
        out = _plain_quantize_cache(s)
    elif op == "dequantize_cache":
        out = _plain_dequantize_cache(s)
    elif op == "quantized_attention":
        out = _plain_quantized_attention(s)
    else:
        out = _plain_shared_attention(s)
    if op == "quantize_cache":
        return {"codes": out[0].view(torch.float8_e4m3fn), "exponents": out[1]}
    return dict(zip("kv", out)) if op == "dequantize_cache" else {"o": out}


# ------------------------------------------------------------ from the definitions, in 64 bits

def _grid(y):
    """y (64 bits) rounded to e4m3's values: eight steps to each power of two, 2^-9 below 2^-6; ties to the even one."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step


def _decoded(codes, exps):
    """The stored values in 64 bits, from the bits of a code: sign, four of exponent (bias 7), three of fraction."""
    c = codes.int()
    e, f = (c >> 3) & 15, (c & 7).double()
    x = torch.where(e > 0, (1 + f / 8) * torch.exp2(e.double() - 7), f * 2.0 ** -9)
    return torch.where(c > 127, -x, x) * torch.exp2(exps.double())[..., None]


def exact(case, seed):
    s = prepare(case, seed)
    n_heads, n_kv, hd = HEADS[case["heads"]]
    new, ctx = _lengths(case)
    if case["op"] == "quantize_cache":
        codes, exps, first = s["codes"].double(), s["exps"].double(), 0
        for b, (n, c) in enumerate(zip(new, ctx)):
            t = torch.arange(c - n, c, device=DEVICE)
            block, slot = s["table"][b, t // BLOCK].long(), t % BLOCK
            for i, x in enumerate((s["k"], s["v"])):
                y = x[first:first + n].view(n, n_kv, hd).double()
                # 2^e is the power of two at or above a 448th of the largest (values of 24 bits
                # are 8e-8 apart in log2, and that of a power of two may come out inexact)
                e = torch.ceil(torch.log2(y.abs().amax(-1) / E4M3_MAX) - 1e-9).clamp(min=E_MIN)
                codes[block, :, i, slot] = _grid(y * torch.exp2(-e)[..., None])
                exps[block, :, i, slot] = e
            first += n
        return {"codes": codes, "exponents": exps.to(torch.int8)}
    if case["op"] == "dequantize_cache":
        x = _decoded(s["codes"], s["exps"])
        k, v = s["k"].double(), s["v"].double()
        for b, c in enumerate(ctx):
            t = torch.arange(c, device=DEVICE)
            src, dst, slot = s["table"][b, t // BLOCK].long(), s["dst"][b, t // BLOCK].long(), t % BLOCK
            k[dst, :, slot], v[dst, :, slot] = x[src, :, 0, slot], x[src, :, 1, slot]
        return {"k": k, "v": v}
    q = s["q"].view(-1, n_heads, hd).double()
    o = torch.zeros_like(q)
    for b, c in enumerate(ctx):
        blocks = s["table"][b, :-(-c // BLOCK)].long()
        for g in range(n_kv):
            if case["op"] == "shared_attention":
                kv = torch.stack((s["k"][blocks, g], s["v"][blocks, g])).double()
            else:
                kv = _decoded(s["codes"][blocks, g], s["exps"][blocks, g]).transpose(0, 1)
            keys, vals = kv.reshape(2, -1, hd)[:, :c]
            heads = slice(g * n_heads // n_kv, (g + 1) * n_heads // n_kv)
            z = q[b, heads] @ keys.T / math.sqrt(hd)
            o[b, heads] = torch.exp(z - torch.logsumexp(z, 1, keepdim=True)) @ vals
    return {"o": o.view(s["q"].shape)}
