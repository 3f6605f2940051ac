"""The masked and tree-shaped attention over the packed cache, as measured work.

Three operators over the q8_0-K / TBQ-V tile records:

* ``attn_scored``: attention of the last ``n_q`` positions of each sequence (one
  token, a verify batch or a whole prompt) with a tanh cap on the scores, a
  distance bias, a sliding window, a document mask and a prefix mask;
* ``attn_tree``: attention of a tree of drafted tokens (the last ``n_q`` cached
  positions, each seeing the committed cache and its own ancestors);
* ``tree_accept``: the accepted path of such a tree moved, bit for bit, to the
  front of the drafted positions.

``run`` computes them in elementary torch operations in 32 bits; with ``own``
set it makes the library's calls on the same tensors. A case holds the sizes:
``D`` head dim, ``Hkv`` / ``Hq`` heads, ``B`` sequences of at most ``T`` cached
positions (ragged: shorter by ``_lens``), ``n_q`` query tokens or tree nodes,
``bits`` per V code, ``rot`` (the block-diagonal rotation), and the score's
``cap``, ``window``, ``alibi``, ``docs`` and ``prefix``.
"""
import math

import numpy as np
import torch

own = False

TABLES = {2: (0.4528, 1.5104), 3: (0.2451, 0.7560, 1.3439, 2.1520),
          4: (0.1284, 0.3880, 0.6568, 0.9423, 1.2562, 1.6180, 2.0690, 2.7326)}


def _case(name, op, D, Hkv, Hq, B, T, n_q, bits=3, rot=False, cap=0.0, window=0, alibi=False, docs=0, prefix=0,
          ragged=False, bf16=False):
    c = dict(name=name, op=op, D=D, Hkv=Hkv, Hq=Hq, B=B, T=T, n_q=n_q, bits=bits, rot=rot, cap=cap, window=window,
             alibi=alibi, docs=docs, prefix=prefix, ragged=ragged, bf16=bf16)
    return c if name else {k: v for k, v in c.items() if k != "name"}


def listed():
    return [
        # One chat's next token over a short cache, capped scores: nothing but latency.
        _case("scored token 256", "scored", 128, 1, 4, 1, 256, 1, cap=30.0),
        # One next token over a long cache of wide heads, capped and with a distance bias: bandwidth.
        _case("scored token 32k", "scored", 512, 2, 16, 1, 32768, 1, cap=50.0, alibi=True),
        # A served batch of a sliding-window layer, ragged lengths, the 4-bit tier: a quarter of the cache is read.
        _case("scored window batch", "scored", 256, 4, 16, 16, 16384, 1, bits=4, cap=50.0, window=4096, ragged=True),
        # A batch verifying a chain of drafted tokens with a distance bias, ragged and odd lengths.
        _case("scored verify batch", "scored", 128, 8, 32, 8, 4093, 5, alibi=True, ragged=True),
        # Several prompts packed into one sequence, no attention across documents.
        _case("scored packed prompts", "scored", 128, 2, 16, 1, 4096, 4096, docs=7, bf16=True),
        # The last chunk of a prompt after a bidirectional prefix, capped scores, wide heads, odd lengths.
        _case("scored prefix chunk", "scored", 512, 2, 16, 1, 8191, 1000, cap=50.0, prefix=7600, bf16=True),
        # One chat's small draft tree over a short cache: latency.
        _case("tree small", "tree", 128, 1, 4, 1, 333, 7),
        # A draft tree of eight nodes over a long cache of wide heads.
        _case("tree 8 at 32k", "tree", 512, 2, 16, 1, 32768, 8),
        # A served batch of ragged trees, ragged lengths, capped scores.
        _case("tree batch", "tree", 128, 8, 32, 16, 4096, 32, cap=30.0, ragged=True),
        # Two requests with the widest trees, block-diagonal 4-bit values, a sliding window and a distance bias.
        _case("tree 64 window", "tree", 512, 2, 16, 2, 16384, 64, bits=4, rot=True, window=8192, alibi=True),
        # The accepted path of one chat's small tree: latency.
        _case("accept small", "accept", 128, 1, 4, 1, 333, 7),
        # The accepted paths of a served batch of wide trees.
        _case("accept batch", "accept", 512, 2, 16, 32, 1000, 64, ragged=True),
    ]


def _cost(c):
    w = work(c)
    plain = c["B"] * c["Hkv"] * _cap(c) * c["D"] + c["B"] * c["Hq"] * c["n_q"] * c["T"]
    return w["bytes"] * 250.0 + w["flops"] + 100.0 * plain


def draw(rng):
    """One more case: any head dim, tier, rotation and head ratio, lengths and batches over their logarithm."""
    log = lambda a, b: int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))  # noqa: E731
    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["scored", "scored", "scored", "tree", "tree", "accept"])
        D = rng.choice([64, 128, 256, 512])
        Hkv = rng.choice([1, 2, 3, 4, 8])
        c = dict(op=op, D=D, Hkv=Hkv, Hq=Hkv * rng.choice([1, 2, 3, 4, 6, 8, 16]), B=log(1, 32), T=log(70, 32768),
                 n_q=log(1, 64), bits=rng.choice([2, 3, 3, 4]), rot=D >= 128 and rng.random() < 0.3,
                 cap=rng.choice([0.0, 0.0, 20.0, 30.0, 50.0]), window=0, alibi=rng.random() < 0.4, docs=0, prefix=0,
                 ragged=rng.random() < 0.6, bf16=rng.random() < 0.3)
        if rng.random() < 0.35:
            c["window"] = log(16, c["T"])
        if op == "accept":
            c.update(cap=0.0, window=0, alibi=False, bf16=False, T=min(c["T"], 2048))
        if op == "scored" and rng.random() < 0.4:  # a prompt, whole or its last chunk
            c.update(n_q=log(65, 4096), bf16=True, B=log(1, 4))
            c["T"] = c["n_q"] + (0 if rng.random() < 0.4 else log(1, 8192))
            c["docs"] = rng.choice([0, 0, 2, 3, 9])
            c["prefix"] = rng.choice([0, 0, c["T"] // 3, c["T"] - c["n_q"] // 2])
        if op != "accept" and c["n_q"] > c["T"]:
            continue
        if _cost(c) <= most:
            return c


def _cap(c):
    """Positions allocated per sequence: whole records, a few spare."""
    return (c["T"] + 15) // 16 * 16 + 32


def _lens(c):
    """Cached positions of each sequence, the n_q newest among them."""
    if not c["ragged"]:
        return [c["T"]] * c["B"]
    spare = c["T"] - min(c["T"], c["n_q"])
    return [c["T"] - (b * 3571) % (spare * 3 // 4 + 1) for b in range(c["B"])]


def _nodes(c):
    """Query tokens (or tree nodes) of each sequence; the rows after them are padding."""
    if not c["ragged"] or c["op"] == "scored":
        return [c["n_q"]] * c["B"]
    return [c["n_q"] - (b * 5) % (c["n_q"] * 3 // 4 + 1) for b in range(c["B"])]


def _doc_starts(c):
    return sorted({j * c["T"] // c["docs"] + (7 * j) % 13 for j in range(c["docs"])}) if c["docs"] else []


def _row_ranges(c, b):
    """[lo, hi) of the positions that each query token of sequence b sees, apart from a tree's mask."""
    T, n = _lens(c)[b], _nodes(c)[b]
    pos = np.arange(T - n, T)
    lo, hi = np.zeros(n, np.int64), pos + 1
    if c["op"] == "tree":
        return np.maximum(lo, pos - c["window"] + 1) if c["window"] else lo, hi
    if c["docs"]:
        s = np.array(_doc_starts(c))
        lo = s[np.searchsorted(s, pos, side="right") - 1]
    if c["window"]:
        lo = np.maximum(lo, pos - c["window"] + 1)
    return lo, np.maximum(hi, min(c["prefix"], T))


def work(c):
    D, groups = c["D"], c["D"] // 128 if c["rot"] else 1
    per_token = D + D // 16 + c["bits"] * D // 8 + 2 * groups
    if c["op"] == "accept":
        moved = sum(min(8, n) for n in _nodes(c)) * c["Hkv"]
        return {"bytes": float(2 * moved * per_token + 4 * c["B"] * (c["n_q"] + 3)), "flops": 0.0}
    keys = pairs = 0
    for b in range(c["B"]):
        lo, hi = _row_ranges(c, b)
        keys += int(hi.max() - lo.min())
        pairs += int((hi - lo).sum())
    rows = c["B"] * c["n_q"] * c["Hq"]
    return {"bytes": float(keys * c["Hkv"] * per_token + rows * (4 * D + 4)), "flops": 4.0 * D * pairs * c["Hq"]}


# ------------------------------------------------------------------ inputs --

def _signs(D, seed, dev):
    g = torch.Generator(device="cpu").manual_seed(seed)
    return (torch.randint(0, 2, (D,), generator=g) * 2 - 1).to(torch.int8).to(dev)


def _table(bits, dev, dtype):
    t = TABLES[bits]
    return torch.tensor([-x for x in reversed(t)] + list(t), device=dev, dtype=dtype)


def _fields(c, seed):
    """What the cache holds: K codes and block scales, V codes and norms, of normal keys with a few channels ten
    times larger and of normal values (whose rotated coordinates are normal too)."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed) * 7919 + 17)
    D, n = c["D"], _cap(c)
    groups = D // 128 if c["rot"] else 1
    k = torch.randn((c["B"], c["Hkv"], n, D), generator=g, device=dev)
    wide = torch.randperm(D, generator=g, device=dev)[:max(1, D // 100)]
    k[..., wide] *= 10.0
    k = k.view(c["B"], c["Hkv"], n, D // 32, 32)
    d16 = (k.abs().amax(-1) / 127.0).half()
    qs = (k / d16.float().unsqueeze(-1)).round().clamp_(-127, 127).to(torch.int8).view(c["B"], c["Hkv"], n, D)
    table = _table(c["bits"], dev, torch.float32)
    codes = torch.bucketize(torch.randn((c["B"], c["Hkv"], n, D), generator=g, device=dev),
                            (table[1:] + table[:-1]) / 2).to(torch.uint8)
    width = D // groups
    n16 = (math.sqrt(width) * (1 + torch.randn((c["B"], c["Hkv"], n, groups), generator=g, device=dev)
                               / math.sqrt(2 * width))).half()
    q = torch.randn((c["B"], c["n_q"], c["Hq"], D), generator=g, device=dev)
    q[..., wide] *= 10.0 / math.sqrt(10.0)
    return g, qs, d16, codes, n16, q.to(torch.bfloat16 if c["bf16"] else torch.float16)


def _places(D, bits, groups):
    """Where a record of 16 positions holds its parts: bytes of the K codes [16, D] and bits of the V codes [16, D, bits]."""
    p, i = np.arange(16)[:, None], np.arange(D)[None, :]
    kbyte = ((i // 32) * 32 + 4 * (p % 8) + (i % 32) // 8) * 16 + (p // 8) * 8 + i % 8
    G, stream = D // 8, bits * D // 16
    gr = next(x for x in (16, 8, 4) if stream % x == 0)
    lane, pair = 4 * (i // G) + (p % 8) // 2, 4 * ((i % G) // 2) + (i % G) % 2 + 2 * (p // 8)
    bit = (2 * bits * pair + bits * (p % 2))[..., None] + np.arange(bits)
    vbit = 8 * (17 * D + ((bit // 8 // gr) * 32 + lane[..., None]) * gr + bit // 8 % gr) + bit % 8
    return torch.from_numpy(kbyte), torch.from_numpy(vbit), 17 * D + 2 * bits * D + 32 * groups


def _records(c, qs, d16, codes, n16):
    """The fields laid out as tile records, uint8 [B, Hkv, records, bytes]."""
    D, bits = c["D"], c["bits"]
    groups = n16.shape[-1]
    kbyte, vbit, size = _places(D, bits, groups)
    B, H, n = qs.shape[:3]
    rec = torch.zeros((B, H, n // 16, size), dtype=torch.uint8, device=qs.device)
    tiles = lambda x: x.reshape(B, H, n // 16, -1)  # noqa: E731
    rec[..., kbyte.reshape(-1).to(qs.device)] = tiles(qs.view(torch.uint8) ^ 0x80)
    rec[..., 16 * D:17 * D] = tiles(d16.contiguous()).view(torch.uint8)
    rec[..., 17 * D + 2 * bits * D:] = n16.reshape(B, H, n // 16, 16, groups).transpose(-1, -2).reshape(
        B, H, n // 16, -1).contiguous().view(torch.uint8)
    # The V region: every bit of it belongs to one code.
    order = torch.argsort(vbit.reshape(-1)).to(qs.device)
    b = (codes.unsqueeze(-1) >> torch.arange(bits, dtype=torch.uint8, device=qs.device)) & 1
    b = tiles(b)[..., order].view(B, H, n // 16, 2 * bits * D, 8)
    b <<= torch.arange(8, dtype=torch.uint8, device=qs.device)
    rec[..., 17 * D:17 * D + 2 * bits * D] = b.sum(-1, dtype=torch.uint8)
    return rec


def _trees(c, rng):
    """One random tree for each sequence: node i's mask has its ancestors' bits and its own."""
    m = np.zeros((c["B"], c["n_q"]), np.uint64)
    for b, n in enumerate(_nodes(c)):
        for i in range(n):
            parent = 0 if i < 4 else int(rng.integers(max(0, i // 3 - 2), i // 2 + 1))
            m[b, i] = (m[b, parent] if i else np.uint64(0)) | np.uint64(1 << i)
    return m.view(np.int64)


def _paths(c, rng):
    """The accepted nodes of each sequence, at most 8, ascending; what a second pass would move is where it belongs already."""
    path, count = np.full((c["B"], 8), -1, np.int32), np.zeros(c["B"], np.int32)
    for b, n in enumerate(_nodes(c)):
        L = int(rng.integers(1, min(8, n) + 1))
        far = min(int(rng.integers(0, L)), n - L)
        path[b, :L - far] = np.arange(L - far)
        path[b, L - far:L] = np.sort(rng.choice(np.arange(L, n), far, replace=False)) if far else []
        count[b] = L
    return path, count


def prepare(case, seed):
    c = dict(case)
    g, qs, d16, codes, n16, q = _fields(c, seed)
    dev, rng = qs.device, np.random.default_rng(int(seed) + 99)
    ints = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32).to(dev)  # noqa: E731
    s = {"c": c, "cache": _records(c, qs, d16, codes, n16), "seq_len": ints(_lens(c)),
         "signs": _signs(c["D"], 42, dev), "signs2": _signs(c["D"], 43, dev) if c["rot"] else None,
         "scale": 1.0 / math.sqrt(c["D"]), "n_node": ints(_nodes(c)) if c["ragged"] and c["op"] != "scored" else None}
    if c["op"] == "accept":
        path, count = _paths(c, rng)
        s.update(path=ints(path), path_len=ints(count), new_len=torch.empty(c["B"], dtype=torch.int32, device=dev))
    else:
        s["q"] = q
        s["slopes"] = (2.0 ** (-8.0 * torch.arange(1, c["Hq"] + 1, device=dev) / c["Hq"])).float() if c["alibi"] else None
    if c["op"] == "tree":
        s["mask"] = torch.from_numpy(_trees(c, rng)).to(dev)
    if c["op"] == "scored":
        starts = np.array(_doc_starts(c) or [0])
        pos = np.array([np.arange(t - c["n_q"], t) for t in _lens(c)])
        s["doc_start"] = ints(starts[np.searchsorted(starts, pos, side="right") - 1]) if c["docs"] else None
        s["prefix_len"] = ints([min(c["prefix"], t) for t in _lens(c)]) if c["prefix"] else None
    if own:  # the handle and the buffers that a program keeps
        import compressed_kv_attention_gb300 as ckv
        s["packed"] = ckv.PackedCache(c["D"], c["Hkv"], c["B"], _cap(c), s["signs"], device=dev, data=s["cache"],
                                      v_bits=c["bits"], signs2=s["signs2"])
        if c["op"] != "accept":
            size = ckv.attn_tree_workspace if c["op"] == "tree" else ckv.attn_scored_workspace
            s["out"] = torch.empty_like(q)
            s["lse"] = torch.empty(q.shape[:3], dtype=torch.float32, device=dev)
            s["ws"] = torch.zeros(size(s["packed"], c["T"], c["n_q"], c["Hq"]), dtype=torch.uint8, device=dev)
    return s


# --------------------------------------------------------- the plain forms --

_kept = {}


def _static(D, bits, groups, dev):
    """Index maps and the Hadamard matrix: constants of a layout, made once."""
    key = (D, bits, groups, str(dev))
    if key not in _kept:
        kbyte, vbit, size = _places(D, bits, groups)
        w = D // groups
        i = np.arange(w)
        had = 1.0 - 2.0 * (np.array([bin(int(x)).count("1") for x in (i[:, None] & i[None, :]).reshape(-1)]).reshape(w, w) % 2)
        _kept[key] = (kbyte.to(dev), vbit.to(dev), torch.from_numpy(had).float().to(dev), _table(bits, dev, torch.float32))
    return _kept[key]


def _unpack(s):
    """K and V of every cached position in 32 bits, [B, Hkv, positions, D]."""
    c, rec = s["c"], s["cache"]
    D, bits = c["D"], c["bits"]
    groups = D // 128 if c["rot"] else 1
    kbyte, vbit, had, table = _static(D, bits, groups, rec.device)
    B, H, nt = rec.shape[:3]
    scale = rec[..., 16 * D:17 * D].contiguous().view(torch.float16).float().view(B, H, nt * 16, D // 32, 1)
    k = (rec[..., kbyte.view(-1)].view(B, H, nt * 16, D // 32, 32).float() - 128.0) * scale
    b = (rec[..., (vbit // 8).view(-1)].view(B, H, nt, 16 * D, bits) >> (vbit % 8).view(16 * D, bits).to(torch.uint8)) & 1
    codes = (b << torch.arange(bits, dtype=torch.uint8, device=rec.device)).sum(-1)
    norm = rec[..., 17 * D + 2 * bits * D:].contiguous().view(torch.float16).float()
    norm = norm.view(B, H, nt, groups, 16).transpose(-1, -2).reshape(B, H, nt * 16, groups, 1)
    u = table[codes].view(B, H, nt * 16, groups, D // groups)
    if s["signs2"] is not None:
        u = u * s["signs2"].float().view(groups, D // groups)
    v = (torch.matmul(u, had) * (norm * (groups / D))).reshape(B, H, nt * 16, D) * s["signs"].float()
    return k.view(B, H, nt * 16, D), v


def _attention(s):
    c = s["c"]
    k, v = _unpack(s)
    dev, n_q, cap = k.device, c["n_q"], k.shape[2]
    B, H, G, D = c["B"], c["Hkv"], c["Hq"] // c["Hkv"], c["D"]
    n = s["n_node"] if s["n_node"] is not None else torch.full_like(s["seq_len"], n_q)
    t = torch.arange(cap, device=dev)
    i = torch.arange(n_q, device=dev)
    base = (s["seq_len"] - n).view(B, 1, 1)
    real = i.view(1, n_q, 1) < n.view(B, 1, 1)
    if c["op"] == "tree":
        mask = s["mask"].view(B, n_q, 1)
        on = (mask >> torch.arange(64, device=dev)) & 1  # [B, n_q, 64]
        depth = on.sum(-1) - 1
        node = (t - base).clamp(0, n_q - 1)  # [B, 1, cap]
        drafted = (t >= base) & (t < base + n.view(B, 1, 1))
        seen = (t < base) | (drafted & (((mask >> node) & 1) == 1))
        at = base + depth.view(B, n_q, 1)
        key_at = torch.where(drafted, base + depth.gather(1, node.view(B, cap)).view(B, 1, cap), t)
    else:
        at, key_at = base + i.view(1, n_q, 1), t.view(1, 1, cap)
        end = at + 1
        if s["prefix_len"] is not None:
            end = torch.maximum(end, s["prefix_len"].view(B, 1, 1))
        seen = (t < end) & (t < s["seq_len"].view(B, 1, 1)) & (at >= 0)
        if s["doc_start"] is not None:
            seen = seen & (t >= s["doc_start"].view(B, n_q, 1))
    if c["window"]:
        seen = seen & (at - key_at < c["window"])
    seen = (seen & real).view(B, 1, 1, n_q, cap)
    q = s["q"].float().view(B, n_q, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * n_q, D)
    x = (torch.matmul(q, k.transpose(-1, -2)) * s["scale"]).view(B, H, G, n_q, cap)
    if c["cap"]:
        x = c["cap"] * torch.tanh(x / c["cap"])
    if s["slopes"] is not None:
        x = x - s["slopes"].view(1, H, G, 1, 1) * (at - key_at).abs().float().view(B, 1, 1, n_q, cap)
    x = x.masked_fill(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isinf(top), 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, H, G * n_q, cap), v).view(B, H, G, n_q, D) / torch.where(total > 0, total, 1.0)
    lse = torch.where(total > 0, top + torch.log(total), -math.inf)
    return {"out": o.permute(0, 3, 1, 2, 4).reshape(B, n_q, H * G, D).to(s["q"].dtype),
            "lse": lse.permute(0, 3, 1, 2, 4).reshape(B, n_q, H * G)}


def _accept(s):
    """The drafted records as bits, the accepted positions' bits moved, the records written back."""
    c, rec = s["c"], s["cache"]
    D, bits, groups = c["D"], c["bits"], c["D"] // 128 if c["rot"] else 1
    kbyte, vbit, _, _ = _static(D, bits, groups, rec.device)
    dev, (B, H, nt, size) = rec.device, rec.shape
    eight, p = torch.arange(8, device=dev), torch.arange(16, device=dev).view(16, 1)
    scale_byte = 16 * D + p * (D // 16) + torch.arange(D // 16, device=dev)
    norm_byte = 17 * D + 2 * bits * D + (32 * torch.arange(groups, device=dev).view(groups, 1) + torch.arange(2, device=dev)).view(1, -1) + 2 * p
    whole = torch.cat([kbyte, scale_byte, norm_byte], 1)
    mine = torch.cat([(whole.unsqueeze(-1) * 8 + eight).view(16, -1), vbit.view(16, -1)], 1)  # bits of each position
    n = s["n_node"] if s["n_node"] is not None else torch.full_like(s["seq_len"], c["n_q"])
    base = (s["seq_len"] - n).long()
    at = (base // 16).view(B, 1) + torch.arange((c["n_q"] + 15) // 16 + 1, device=dev)  # records of the drafted tokens
    head = torch.arange(H, device=dev).view(1, H, 1)
    seq = torch.arange(B, device=dev).view(B, 1, 1)
    some = rec[seq, head, at.view(B, 1, -1)]  # [B, H, records, size]
    b = ((some.unsqueeze(-1) >> eight.to(torch.uint8)) & 1).view(B, H, -1, size * 8)
    rows = b[..., mine.view(-1)].view(B, H, at.shape[1] * 16, -1)
    first = (base % 16).view(B, 1)
    j = torch.arange(s["path"].shape[1], device=dev)
    on = j.view(1, -1) < s["path_len"].view(B, 1)
    src = torch.where(on, first + s["path"].clamp(min=0), first + j)
    index = torch.arange(rows.shape[2], device=dev).repeat(B, 1).scatter(1, first + j, src)
    rows = rows[seq, head, index.view(B, 1, -1)]
    b = torch.empty_like(b).index_copy_(3, mine.view(-1), rows.reshape(B, H, at.shape[1], -1))
    rec[seq, head, at.view(B, 1, -1)] = (b.view(B, H, -1, size, 8) << eight.to(torch.uint8)).sum(-1, dtype=torch.uint8)
    s["new_len"].copy_(s["seq_len"] - n + s["path_len"])
    return {"cache": rec, "new_len": s["new_len"]}


def run(s):
    c = s["c"]
    if not own:
        return _accept(s) if c["op"] == "accept" else _attention(s)
    import compressed_kv_attention_gb300 as ckv
    if c["op"] == "accept":
        ckv.tree_accept(s["packed"], s["seq_len"], c["n_q"], s["path"], s["path_len"], s["new_len"], q_len=s["n_node"])
        return {"cache": s["cache"], "new_len": s["new_len"]}
    if c["op"] == "tree":
        ckv.attn_tree(s["packed"], s["seq_len"], c["T"], s["mask"], s["q"], s["scale"], s["out"], s["lse"], s["ws"],
                      softcap=c["cap"], window=c["window"], slopes=s["slopes"], q_len=s["n_node"])
    else:
        ckv.attn_scored(s["packed"], s["seq_len"], c["T"], s["q"], s["scale"], s["out"], s["lse"], s["ws"],
                        softcap=c["cap"], window=c["window"], slopes=s["slopes"], prefix_len=s["prefix_len"],
                        doc_start=s["doc_start"])
    return {"out": s["out"], "lse": s["lse"]}


# -------------------------------------------------- from the definition --

def exact(case, seed):
    """Softmax over each row's visible keys, one sequence and KV head at a time, in 64 bits and from the fields themselves."""
    c = dict(case)
    if c["op"] == "accept":
        return None  # bytes moved: nothing is computed
    g, qs, d16, codes, n16, q = _fields(c, seed)
    dev, rng = qs.device, np.random.default_rng(int(seed) + 99)
    D, G, width = c["D"], c["Hq"] // c["Hkv"], 128 if c["rot"] else c["D"]
    table = _table(c["bits"], dev, torch.float64)
    s1 = _signs(D, 42, dev).double()
    trees = _trees(c, rng).view(np.uint64) if c["op"] == "tree" else None
    out = torch.zeros((c["B"], c["n_q"], c["Hq"], D), dtype=torch.float64, device=dev)
    lse = torch.full((c["B"], c["n_q"], c["Hq"]), -math.inf, dtype=torch.float64, device=dev)
    for b in range(c["B"]):
        T, n = _lens(c)[b], _nodes(c)[b]
        lo, hi = _row_ranges(c, b)
        key_at, q_at = np.arange(T), np.arange(T - n, T)
        see = (key_at[None, :] >= lo[:, None]) & (key_at[None, :] < hi[:, None])
        if c["op"] == "tree":
            at = np.array([[int(m) >> j & 1 for j in range(n)] for m in trees[b, :n]], dtype=bool)
            level = at.sum(1) - 1
            key_at[T - n:], q_at = T - n + level, T - n + level
            see = np.ones((n, T), bool)
            see[:, T - n:] = at
            if c["window"]:
                see &= q_at[:, None] - key_at[None, :] < c["window"]
        see = torch.from_numpy(see).to(dev)
        far = torch.from_numpy(np.abs(q_at[:, None] - key_at[None, :])).to(dev).double() if c["alibi"] else None
        for h in range(c["Hkv"]):
            k = qs[b, h, :T].double() * d16[b, h, :T].double().repeat_interleave(32, 1)
            v = table[codes[b, h, :T].long()]
            if c["rot"]:
                v = v * _signs(D, 43, dev).double()
            step = 1
            while step < width:  # the Walsh-Hadamard butterflies of each group
                w = v.view(T, D // (2 * step), 2, step)
                v = torch.stack([w[:, :, 0] + w[:, :, 1], w[:, :, 0] - w[:, :, 1]], 2).reshape(T, D)
                step *= 2
            v = v * n16[b, h, :T].double().repeat_interleave(width, 1) / width * s1
            for r in range(G):
                x = q[b, :n, h * G + r].double() @ k.T / math.sqrt(D)
                if c["cap"]:
                    x = torch.tanh(x / c["cap"]) * c["cap"]
                if c["alibi"]:
                    x = x - far * float(np.float32(2.0 ** (-8.0 * (h * G + r + 1) / c["Hq"])))
                x = torch.where(see, x, -math.inf)
                some = see.any(1)
                l = torch.logsumexp(x, 1)
                p = torch.where(see, torch.exp(x - torch.where(some, l, 0.0)[:, None]), 0.0)
                out[b, :n, h * G + r] = p @ v
                lse[b, :n, h * G + r] = torch.where(some, l, -math.inf)
    return {"out": out, "lse": lse}
