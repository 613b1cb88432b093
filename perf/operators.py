"""Measured cases of the paged TQ3 cache: append, read back, and attention of new tokens over it.

Each case is one call on a cache whose K and V records (48 bytes of 3-bit indices, an fp32 norm, an
fp32 scale) live in pools [pages, kv_heads, page_size, 56] reached through one page table per
sequence:

* ``append``: quantise the K and V of new tokens and write them to their slots;
* ``read``: decode ragged sequences back to dense K and V;
* ``attend``: causal attention of ragged chunks of new tokens over the cache, optionally with a
  sliding window and a few first tokens that stay visible.

``run`` computes a case in elementary torch operations, or through the framework where ``own`` is set.
"""
import math

import numpy as np
import torch

own = False

D = 128
CENTROIDS = (-0.9816, -0.6168, -0.3479, -0.1129, 0.1129, 0.3479, 0.6168, 0.9816)
BOUNDARIES = (-0.7992, -0.4824, -0.2304, 0.0, 0.2304, 0.4824, 0.7992)
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------
def _append(name, tokens, kv_heads, page, dtype, q_heads):
    return {"name": name, "op": "append", "tokens": tokens, "kv_heads": kv_heads, "page": page, "dtype": dtype,
            "q_heads": q_heads}


def _read(name, batch, kv, kv_heads, page, dtype):
    return {"name": name, "op": "read", "batch": batch, "kv": kv, "kv_heads": kv_heads, "page": page, "dtype": dtype}


def _attend(name, batch, new, kv, q_heads, kv_heads, page, dtype, window=0, sinks=0, ragged=True):
    return {"name": name, "op": "attend", "batch": batch, "new": new, "kv": kv, "q_heads": q_heads,
            "kv_heads": kv_heads, "page": page, "dtype": dtype, "window": window, "sinks": sinks, "ragged": ragged}


def listed():
    return [
        # one decoding step of 64 sequences: every step of a server writes this
        _append("append_step", 64, 8, 16, "bf16", 32),
        # the whole prompt of 8 sequences of 4096 tokens, out of a fused projection
        _append("append_prompt", 32768, 8, 16, "bf16", 32),
        # an odd number of fp32 tokens, heads that are no power of two
        _append("append_fp32", 4099, 5, 32, "fp32", 5),
        # a short prefix handed back to a dense kernel
        _read("read_prefix", 3, 77, 2, 16, "fp32"),
        # ragged sequences moved out of the cache
        _read("read_ragged", 16, 4096, 8, 16, "bf16"),
        # a lone user's token on a short conversation: latency
        _attend("decode_lone", 1, 1, 515, 32, 8, 16, "bf16"),
        # decoding at a long context: 64 (sequence, KV head) pairs of 32768 keys
        _attend("decode_long", 8, 1, 32768, 32, 8, 16, "bf16", ragged=False),
        # a continuous batch: most sequences decode, some bring a chunk of their prompt
        _attend("mixed_batch", 12, 256, 4096, 32, 8, 16, "bf16"),
        # a 2048-token piece of a long prompt
        _attend("chunk_long", 1, 2048, 16384, 32, 8, 64, "bf16"),
        # fp32 queries, odd sizes, one query head per KV head
        _attend("chunk_fp32", 3, 37, 1531, 4, 4, 32, "fp32"),
        # streaming decode: a window and four sinks on long contexts
        _attend("window_decode", 32, 1, 16384, 32, 8, 16, "bf16", window=4096, sinks=4),
        # a windowed layer's piece of a prompt
        _attend("window_chunk", 2, 1024, 8192, 16, 4, 32, "bf16", window=1024, sinks=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "read", "decode", "chunk", "window"))
    page, kv_heads = rng.choice((8, 16, 32, 64, 128)), rng.choice((1, 2, 3, 4, 5, 8))
    dtype = rng.choice(("bf16", "bf16", "fp32"))
    if op == "append":
        return {k: v for k, v in _append("", _log(rng, 1, 16384), kv_heads, page, dtype, kv_heads * rng.choice((1, 2, 4))).items()
                if k != "name"}
    if op == "read":
        batch = _log(rng, 1, 32)
        return {k: v for k, v in _read("", batch, _log(rng, 1, 65536 // batch), kv_heads, page, dtype).items()
                if k != "name"}
    group = rng.choice((1, 2, 4, 7, 8))
    window = _log(rng, 16, 4096) if op == "window" else 0
    sinks = rng.choice((0, 1, 4, 16, 64)) if op == "window" else 0
    if op == "decode" or (op == "window" and rng.random() < 0.5):
        batch, new = _log(rng, 1, 64), 1
        kv = _log(rng, 1, 200000 // batch)
    else:
        batch, new = _log(rng, 1, 8), _log(rng, 2, 1024)
        # at most half of the largest listed chunk's (row, key) pairs
        most = 4.5e8 / (batch * new * kv_heads * group)
        kv = new + _log(rng, 1, max(2, min(16384, int(most) - new)))
    return {k: v for k, v in _attend("", batch, new, kv, kv_heads * group, kv_heads, page, dtype, window, sinks).items()
            if k != "name"}


def _lengths(case):
    """(new tokens, keys) of each sequence; both belong to the case, not to the seed."""
    b, kv, new = case["batch"], case["kv"], case.get("new", 0)
    if not case.get("ragged", True):
        return [new] * b, [kv] * b
    keys = [max(1, kv - (kv * ((37 * i) % 64)) // 96) for i in range(b)]  # the whole of it down to a third
    # in a batch of chunks every third sequence brings one, the others decode
    fresh = [max(1, new - (new * ((11 * i) % 32)) // 64) if i % 3 == 0 else 1 for i in range(b)]
    return [min(n, k) for n, k in zip(fresh, keys)], keys


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------
def _tables(device):
    """The sign flips, the signed transform and the printed tables."""
    g = torch.Generator(device="cpu")
    g.manual_seed(42)
    signs = torch.randint(0, 2, (D,), generator=g, dtype=torch.float32) * 2 - 1
    h = torch.ones(1, 1, dtype=torch.float64)
    for _ in range(7):
        h = torch.cat((torch.cat((h, h), 1), torch.cat((h, -h), 1)), 0)
    bits = (signs > 0).to(torch.int64)
    words = [int((bits[32 * w:32 * w + 32] << torch.arange(32)).sum()) for w in range(4)]
    return {"signs": signs.to(device), "hadamard": h.to(device),
            "centroids": torch.tensor(CENTROIDS, dtype=torch.float32, device=device),
            "boundaries": torch.tensor(BOUNDARIES, dtype=torch.float32, device=device),
            "group": torch.arange(8, dtype=torch.int32, device=device) * 3,
            "mask": np.array(words, dtype=np.uint32)}


def _vectors(shape, g, device):
    """Keys or values: Gaussian, with a per-token offset and a few outlier channels."""
    x = torch.randn(shape, generator=g, device=device)
    x[..., :2] *= 8
    return x + torch.randn(shape[:-1] + (1,), generator=g, device=device)


def _fill(pool, g, t):
    """Records of random vectors in every place of the pool (fp32: these are only inputs)."""
    flat, rot = pool.view(-1, 56), (t["hadamard"] * t["signs"]).float().T
    for at in range(0, flat.shape[0], 1 << 18):
        z = _vectors((min(1 << 18, flat.shape[0] - at), D), g, pool.device) @ rot
        norm, top = (z * z).sum(1, keepdim=True).sqrt() / math.sqrt(D), z.abs().amax(1, keepdim=True)
        flat[at:at + (1 << 18)] = _pack(torch.bucketize(z / top, t["boundaries"]), norm,
                                        top / norm / math.sqrt(D), t)


def prepare(case, seed):
    device = torch.device("cuda")
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    t = _tables(device)
    s = {"case": case, "t": t, "mask": t["mask"]}
    heads, page, dtype = case["kv_heads"], case["page"], DTYPES[case["dtype"]]
    if case["op"] == "append":
        n = case["tokens"]
        fused = torch.empty((n, case["q_heads"] + 2 * heads, D), dtype=dtype, device=device)
        fused[:, :case["q_heads"]] = 0
        s["k"], s["v"] = fused[:, -2 * heads:-heads], fused[:, -heads:]
        s["k"].copy_(_vectors((n, heads, D), g, device))
        s["v"].copy_(_vectors((n, heads, D), g, device))
        pages = -(-n // page) + 3
        order = torch.randperm(pages, generator=g, device=device)
        at = torch.arange(n, device=device) + 5 % page  # the sequences' last pages are partly filled
        s["slots"] = order[at // page] * page + at % page
        s["pools"] = [torch.zeros((pages, heads, page, 56), dtype=torch.uint8, device=device) for _ in range(2)]
    else:
        new, keys = _lengths(case)
        need = [-(-k // page) for k in keys]
        pages, width = sum(need) + 3, max(need) + 1
        order = torch.randperm(pages, generator=g, device=device, dtype=torch.int32)
        table = torch.full((len(keys), width), -1, dtype=torch.int32, device=device)
        at = 0
        for b, m in enumerate(need):
            table[b, :m] = order[at:at + m]
            at += m
        s["table"] = table
        s["pools"] = [torch.empty((pages, heads, page, 56), dtype=torch.uint8, device=device) for _ in range(2)]
        for pool in s["pools"]:
            _fill(pool, g, t)
        starts = keys if case["op"] == "read" else new
        s["start"] = torch.tensor([0] + torch.tensor(starts).cumsum(0).tolist(), dtype=torch.int32, device=device)
        s["tokens"], s["kv"], s["new"] = sum(starts), max(keys), max(new)
        if case["op"] == "attend":
            s["q"] = (torch.randn((s["tokens"], case["q_heads"], D), generator=g, device=device) * 1.5).to(dtype)
            s["kv_len"] = torch.tensor(keys, dtype=torch.int32, device=device)
    floats = [p.view(torch.float32) for p in s["pools"]]
    s["records"] = [(p[..., :48], f[..., 12], f[..., 13]) for p, f in zip(s["pools"], floats)]
    return s


# ------------------------------------------------------------------------------------------------
# plain forms
# ------------------------------------------------------------------------------------------------
def _pack(index, norm, scale, t):
    """Records of indices [n, 128] with norms and scales [n, 1]."""
    word = (index.to(torch.int32).view(-1, 16, 8) << t["group"]).sum(2, dtype=torch.int32)
    low = torch.stack((word & 255, (word >> 8) & 255, word >> 16), 2).view(-1, 48).to(torch.uint8)
    tail = torch.cat((norm.float(), scale.float()), 1).view(torch.uint8)
    return torch.cat((low, tail), 1)


def _quantise(x, t):
    """Records of the rows of x, the decisions in 64 bits."""
    x = x.reshape(-1, D).double()
    z = (x * t["signs"]) @ t["hadamard"] / math.sqrt(D)
    norm = (x * x).sum(1, keepdim=True).sqrt().clamp(min=1e-8)
    y = z / norm
    scale = y.abs().amax(1, keepdim=True).clamp(min=1e-8)
    return _pack(torch.bucketize(y / scale, t["boundaries"].double()), norm, scale, t)


def _values(records, t):
    """Decoded vectors (fp32) of records [..., 56]."""
    b = records[..., :48].reshape(-1, 16, 3).to(torch.int32)
    word = b[..., 0] | (b[..., 1] << 8) | (b[..., 2] << 16)
    index = ((word.unsqueeze(2) >> t["group"]) & 7).view(-1, D)
    f = records.reshape(-1, 56)[:, 48:].contiguous().view(torch.float32)
    y = t["centroids"][index] * f[:, 1:]
    y = (y @ t["hadamard"].float()) * (1 / math.sqrt(D)) * t["signs"] * f[:, :1]
    return y.view(records.shape[:-1] + (D,))


def _gather(pool, table, sequence, position, page):
    at = table[sequence, position // page].long().clamp(min=0)
    return pool[at, :, position % page]


def run(s):
    case, t = s["case"], s["t"]
    if own:
        from weight_quantization_b200 import ops
    if case["op"] == "append":
        if own:
            ops.tq3_cache_append(s["k"], s["v"], s["mask"], s["slots"], *s["pools"])
        else:
            page = case["page"]
            for x, pool in ((s["k"], s["pools"][0]), (s["v"], s["pools"][1])):
                rec = _quantise(x, t).view(x.shape[0], x.shape[1], 56)
                pool[s["slots"] // page, :, s["slots"] % page] = rec
        return s["records"]
    if case["op"] == "read":
        if own:
            return ops.tq3_cache_read(*s["pools"], s["table"], s["start"], s["mask"], s["tokens"],
                                      out_dtype=DTYPES[case["dtype"]])
        token = torch.arange(s["tokens"], device=s["start"].device, dtype=torch.int32)
        seq = torch.bucketize(token, s["start"][1:], right=True)
        at = (token - s["start"][seq]).long()
        return [_values(_gather(p, s["table"], seq, at, case["page"]), t).to(DTYPES[case["dtype"]])
                for p in s["pools"]]
    if own:
        return ops.tq3_attention_chunk(s["q"], *s["pools"], s["table"], s["start"], s["kv_len"], s["mask"],
                                       max_q=s["new"], window=case["window"], sinks=case["sinks"])
    return _attention(s, case, t)


def _attention(s, case, t):
    q, start, kv_len, page = s["q"], s["start"].long(), s["kv_len"].long(), case["page"]
    batch, heads, group = case["batch"], case["kv_heads"], case["q_heads"] // case["kv_heads"]
    j = torch.arange(s["kv"], device=q.device)
    seq = torch.arange(batch, device=q.device)[:, None].expand(batch, s["kv"])
    j2 = j.expand(batch, s["kv"])
    k, v = (_values(_gather(p, s["table"], seq, torch.minimum(j2, kv_len[:, None] - 1), page), t).permute(0, 2, 1, 3)
            for p in s["pools"])
    i = torch.arange(s["new"], device=q.device)
    count = start[1:] - start[:-1]
    rows = (start[:-1, None] + i).clamp(max=q.shape[0] - 1)
    x = q[rows].float().view(batch, s["new"], heads, group, D).permute(0, 2, 3, 1, 4)
    x = x.reshape(batch, heads, group * s["new"], D) * D ** -0.5
    logits = (x @ k.transpose(2, 3)).view(batch, heads, group, s["new"], s["kv"])
    p = (kv_len - count)[:, None, None] + i[:, None]
    seen = j <= p
    if case["window"]:
        seen &= (j > p - case["window"]) | (j < case["sinks"])
    logits.masked_fill_(~seen[:, None, None], -math.inf)
    top = logits.amax(-1, keepdim=True)
    weight = (logits - top.masked_fill(top == -math.inf, 0.0)).exp_()
    total = weight.sum(-1, keepdim=True)
    out = (weight.view(batch, heads, group * s["new"], s["kv"]) @ v).view(batch, heads, group, s["new"], D)
    out = out / total.masked_fill(total == 0, 1.0)
    token = torch.arange(q.shape[0], device=q.device)
    seq = torch.bucketize(token, start[1:], right=True)
    out = out.permute(0, 3, 1, 2, 4).reshape(batch, s["new"], heads * group, D)
    return out[seq, token - start[seq]].to(q.dtype)


# ------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------------
def _transform64(x):
    """The 128-point Walsh-Hadamard transform by its seven butterfly stages."""
    h = 1
    while h < D:
        a = x.reshape(-1, D // (2 * h), 2, h)
        x = torch.stack((a[:, :, 0] + a[:, :, 1], a[:, :, 0] - a[:, :, 1]), 2)
        h *= 2
    return x.reshape(-1, D)


def _encode64(x, t):
    x = x.double()
    norm = x.square().sum(1).sqrt().clamp(min=1e-8)
    z = _transform64(x * t["signs"].double()) / math.sqrt(D) / norm[:, None]
    scale = z.abs().amax(1).clamp(min=1e-8)
    bound = t["boundaries"].double() * scale[:, None]
    index = torch.zeros(z.shape, dtype=torch.int64, device=z.device)
    for k in range(7):
        index += z > bound[:, k:k + 1]
    bits = (index[:, :, None] >> torch.arange(3, device=z.device)) & 1
    packed = (bits.view(-1, 48, 8) << torch.arange(8, device=z.device)).sum(2)
    return packed.to(torch.uint8), norm, scale


def _decode64(rec, t):
    bits = (rec[:, :48, None].long() >> torch.arange(8, device=rec.device)) & 1
    index = (bits.view(-1, D, 3) << torch.arange(3, device=rec.device)).sum(2)
    f = rec[:, 48:].contiguous().view(torch.float32).double()
    z = _transform64(t["centroids"].double()[index] * f[:, 1:]) / math.sqrt(D)
    return z * t["signs"].double() * f[:, :1]


def exact(case, seed):
    s = prepare(case, seed)
    t, page = s["t"], case["page"]
    if case["op"] == "append":
        outputs = []
        for x, pool in zip((s["k"], s["v"]), s["pools"]):
            shape = pool.shape[:3]
            codes = torch.zeros(shape + (48,), dtype=torch.uint8, device=pool.device)
            norms, scales = (torch.zeros(shape, dtype=torch.float64, device=pool.device) for _ in range(2))
            for h in range(case["kv_heads"]):
                c, n, a = _encode64(x[:, h], t)
                place = (s["slots"] // page, torch.full_like(s["slots"], h), s["slots"] % page)
                codes[place], norms[place], scales[place] = c, n, a
            outputs.append((codes, norms, scales))
        return outputs
    starts, table = s["start"].tolist(), s["table"].long()

    def dense(pool, b, h, n):
        pages = table[b, :-(-n // page)]
        return _decode64(pool[pages, h].reshape(-1, 56)[:n], t)

    heads = case["kv_heads"]
    if case["op"] == "read":
        return [torch.cat([torch.stack([dense(p, b, h, starts[b + 1] - starts[b]) for h in range(heads)], 1)
                           for b in range(case["batch"])]) for p in s["pools"]]
    new, keys = _lengths(case)
    group = case["q_heads"] // heads
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    for b in range(case["batch"]):
        p = torch.arange(keys[b] - new[b], keys[b], device=out.device)[:, None]
        j = torch.arange(keys[b], device=out.device)
        seen = j <= p
        if case["window"]:
            seen = seen & ((j > p - case["window"]) | (j < case["sinks"]))
        for h in range(heads):
            k, v = (dense(pool, b, h, keys[b]) for pool in s["pools"])
            for g in range(group):
                x = s["q"][starts[b]:starts[b + 1], h * group + g].double()
                w = torch.softmax((x @ k.T / math.sqrt(D)).masked_fill(~seen, -math.inf), -1)
                out[starts[b]:starts[b + 1], h * group + g] = w @ v
    return out


def work(case):
    heads, width = case["kv_heads"], DTYPES[case["dtype"]].itemsize
    if case["op"] == "append":
        vectors = 2 * case["tokens"] * heads
        return {"bytes": vectors * (D * width + 56) + 8 * case["tokens"], "flops": vectors * (7 * D + 2 * D + 2 * D)}
    new, keys = _lengths(case)
    entries = sum(-(-k // case["page"]) for k in keys)
    if case["op"] == "read":
        vectors = 2 * sum(keys) * heads
        return {"bytes": vectors * (D * width + 56) + 4 * entries, "flops": vectors * (7 * D + 3 * D)}
    pairs = read = 0
    for n, k in zip(new, keys):
        w, sinks = case["window"] or k, case["sinks"] if case["window"] else 0
        first = max(0, k - n + 1 - w)  # the first key that the first row's window holds
        read += k - first + min(sinks, first)
        for p in range(k - n, k):
            low = max(0, p + 1 - w)
            pairs += p + 1 - low + min(sinks, low)
    rows = sum(new) * case["q_heads"]
    return {"bytes": 2 * 56 * read * heads + 2 * rows * D * width + 4 * entries, "flops": 4 * D * pairs * case["q_heads"]}
