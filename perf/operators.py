"""The paged low-bit KV cache and the attention that reads it, as measured cases.

A case is one call on a ragged batch: `append` normalises, rotates and quantizes the new tokens' heads
into pages and reads them back; `attend` is causal attention of the new tokens over their sequences'
pages; `prefix` is the same with a run of pages that all sequences share in front of their own.

Pages are head-major: codes [pages][kv heads][page size][64 or 128 bytes], scales (float32) and zero
points (uint8) [pages][kv heads][page size].  Token t of sequence b sits at position
cached[b] + t - cu_seqlens[b]; position p is row p % page size of page block_table[b][p // page size].
"""
import math
import random

import torch

own = False

D = 128
NORM = 1.0 / math.sqrt(D)
THETA = 1.0e6
EPS = 1.0e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of a small server: latency is all there is
        dict(name="append_step", op="append", bits=4, batch=24, hq=32, hkv=8, page=64, new_lo=1, new_hi=1,
             cached_lo=100, cached_hi=6000, pad=3, norm=True, rot=128, interleaved=False, shape=1),
        # whole prompts of four sequences, written as one batch
        dict(name="append_prompts", op="append", bits=4, batch=4, hq=32, hkv=8, page=64, new_lo=4096, new_hi=4096,
             cached_lo=0, cached_hi=0, pad=0, norm=True, rot=128, interleaved=False, shape=2),
        # chunks of prompts beside single tokens: 8-bit cache, half of each head rotated in interleaved pairs
        dict(name="append_chunks8", op="append", bits=8, batch=7, hq=16, hkv=2, page=16, new_lo=1, new_hi=901,
             cached_lo=0, cached_hi=2500, pad=9, norm=False, rot=64, interleaved=True, shape=3),
        # one user, a short chat
        dict(name="decode_one", op="attend", bits=4, batch=1, hq=32, hkv=8, page=64, new_lo=1, new_hi=1,
             cached_lo=576, cached_hi=576, pad=0, window=0, softcap=0.0, slopes=False, shape=4),
        # the decode step of the KV configuration: 16 sequences of 4096
        dict(name="decode_batch", op="attend", bits=4, batch=16, hq=32, hkv=8, page=64, new_lo=1, new_hi=1,
             cached_lo=4095, cached_hi=4095, pad=0, window=0, softcap=0.0, slopes=False, shape=5),
        # a busy server: lengths from a few tokens to thousands, 8-bit cache, capped scores
        dict(name="decode_ragged8_cap", op="attend", bits=8, batch=48, hq=32, hkv=8, page=16, new_lo=1, new_hi=1,
             cached_lo=3, cached_hi=5000, pad=5, window=0, softcap=30.0, slopes=False, shape=6),
        # two long documents
        dict(name="decode_long", op="attend", bits=4, batch=2, hq=32, hkv=8, page=128, new_lo=1, new_hi=1,
             cached_lo=118000, cached_hi=131071, pad=0, window=0, softcap=0.0, slopes=False, shape=7),
        # two whole prompts
        dict(name="prompt", op="attend", bits=4, batch=2, hq=32, hkv=8, page=64, new_lo=4096, new_hi=4096,
             cached_lo=0, cached_hi=0, pad=0, window=0, softcap=0.0, slopes=False, shape=8),
        # chunked prefill of ragged sequences: 8-bit cache, sliding window, distance bias
        dict(name="chunks8_window", op="attend", bits=8, batch=5, hq=16, hkv=2, page=32, new_lo=37, new_hi=700,
             cached_lo=0, cached_hi=4000, pad=11, window=1000, softcap=0.0, slopes=True, shape=9),
        # a few drafts of up to five tokens behind a short system prompt
        dict(name="prefix_drafts8", op="prefix", bits=8, batch=6, hq=32, hkv=8, page=32, new_lo=1, new_hi=5,
             cached_lo=0, cached_hi=40, pad=2, window=0, softcap=0.0, slopes=False, prefix=700, shape=10),
        # a chat service: 32 users behind one system prompt
        dict(name="prefix_chat", op="prefix", bits=4, batch=32, hq=32, hkv=8, page=64, new_lo=1, new_hi=1,
             cached_lo=16, cached_hi=500, pad=0, window=0, softcap=0.0, slopes=False, prefix=4096, shape=11),
        # many samples of one long document
        dict(name="prefix_large", op="prefix", bits=4, batch=192, hq=32, hkv=8, page=64, new_lo=1, new_hi=1,
             cached_lo=100, cached_hi=900, pad=0, window=0, softcap=0.0, slopes=False, prefix=12001, shape=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "prefix"])
    hq, hkv = rng.choice([(32, 8), (32, 8), (32, 32), (16, 2), (14, 2), (28, 4), (40, 8), (64, 4), (48, 1), (4, 2)])
    case = dict(op=op, bits=rng.choice([4, 8]), hq=hq, hkv=hkv, page=rng.choice([16, 32, 64, 128, 256]),
                pad=rng.choice([0, 0, 1, 7]), shape=rng.randrange(1 << 30))
    if op == "append":
        new = _log_int(rng, 1, 4096)
        case.update(batch=_log_int(rng, 1, max(1, min(64, 16384 * 40 // (hq + 2 * hkv) // new))), new_lo=rng.choice([1, new]), new_hi=new,
                    cached_lo=0, cached_hi=rng.choice([0, _log_int(rng, 1, 8000)]), norm=rng.random() < 0.6,
                    rot=rng.choice([0, 32, 64, 96, 128, 128]), interleaved=rng.random() < 0.4)
        return case
    case.update(window=0, softcap=rng.choice([0.0, 0.0, 20.0, 50.0]), slopes=rng.random() < 0.25)
    kind = rng.choice(["step", "step", "few", "chunk"]) if op == "attend" else rng.choice(["step", "step", "few"])
    if kind == "chunk":
        new = _log_int(rng, 16, 1024)
        batch = _log_int(rng, 1, max(1, min(8, 1024 // new)))
        longest = 3000
    else:
        new = 1 if kind == "step" else rng.randint(2, 8)
        batch = _log_int(rng, 1, 64 if op == "attend" else 128 if new == 1 else 32)
        longest = 60000 if op == "attend" else 700
    longest = min(longest, 1200000 // (hkv * batch))             # rows of all heads: at most the largest listed step's
    hi = _log_int(rng, 2, max(3, longest))
    case.update(batch=batch, new_lo=rng.choice([1, new]), new_hi=new, cached_lo=rng.choice([0, hi // 2, hi]), cached_hi=hi)
    if rng.random() < 0.25:
        case["window"] = _log_int(rng, 1, 4000)
    if op == "prefix":
        case["prefix"] = _log_int(rng, 40, 12000)
    return case


def _lengths(case):
    """(new, cached) of each sequence: a part of the case, whatever the seed."""
    rng = random.Random(case["shape"])
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["batch"])]
    cached = [rng.randint(case["cached_lo"], case["cached_hi"]) for _ in range(case["batch"])]
    return new, cached


# ----------------------------------------------------------------- inputs

def _quantize(x, bits):
    """Asymmetric codes of rows of 128 float32 values: (codes, scale, zero)."""
    top = float(2 ** bits - 1)
    lo, hi = x.amin(-1).clamp(max=0.0), x.amax(-1).clamp(min=0.0)
    scale = (hi - lo) / torch.full_like(hi, top)      # a tensor: by a number, torch multiplies by its reciprocal
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    zero = torch.round(-lo / scale).clamp(0.0, top)
    codes = (torch.round(x / scale[..., None]) + zero[..., None]).clamp(0.0, top)
    return codes.to(torch.uint8), scale, zero.to(torch.uint8)


def _pack(codes, bits):
    return codes if bits == 8 else codes[..., 0::2] | (codes[..., 1::2] << 4)


def _unpack(rows, bits):
    return rows if bits == 8 else torch.stack((rows & 15, rows >> 4), -1).flatten(-2)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, generator=g, device=dev)  # noqa: E731
    uniform = lambda *shape: torch.rand(shape, generator=g, device=dev)  # noqa: E731
    new, cached = _lengths(case)
    B, hq, hkv, ps, bits = case["batch"], case["hq"], case["hkv"], case["page"], case["bits"]
    total = [n + c for n, c in zip(new, cached)]
    T, used = sum(new) + case["pad"], sum(new)
    per = [-(-t // ps) for t in total]
    prefix = case.get("prefix", 0)
    ppages = -(-prefix // ps)
    pages = sum(per) + ppages + 5
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    width = max(per) + 1
    table, at = torch.zeros((B, width), dtype=torch.int64), ppages
    for b, n in enumerate(per):
        table[b, :n] = torch.arange(at, at + n)
        at += n
    s = dict(case=case, T=T, used=used, max_q=max(new), max_len=max(total),
             block_table=order[table.to(dev)].contiguous(),
             cu_seqlens=torch.tensor([0] + new).cumsum(0).to(torch.int32).to(dev),
             cached=torch.tensor(cached, dtype=torch.int32, device=dev),
             lengths=torch.tensor(total, dtype=torch.int32, device=dev),
             # which sequence a packed token belongs to, and which of its new tokens it is
             seq=torch.repeat_interleave(torch.arange(B), torch.tensor(new)).to(dev),
             nth=torch.cat([torch.arange(n) for n in new]).to(dev))
    rb = D * bits // 8
    # what earlier calls left in the pages: unit-variance heads whose size differs by head, values by token
    s["pool"] = {}
    for key, size in (("k", 0.5 + uniform(pages, hkv, 1, 1)), ("v", torch.exp(0.5 * normal(pages, hkv, ps, 1)))):
        if case["op"] == "append":
            codes = torch.zeros((pages, hkv, ps, rb), dtype=torch.uint8, device=dev)
            scale = torch.ones((pages, hkv, ps), device=dev)
            zero = torch.zeros((pages, hkv, ps), dtype=torch.uint8, device=dev)
        else:
            codes, scale, zero = _quantize(normal(pages, hkv, ps, D) * size, bits)
            codes = _pack(codes, bits).contiguous()
        s["pool"].update({key + "_codes": codes, key + "_scale": scale, key + "_zero": zero})
    if case["op"] == "append":
        # one fused projection's output: q, k and v are slices of its rows; a few key channels stand out
        qkv = normal(T, hq + 2 * hkv, D)
        qkv[:, hq:hq + hkv, :: 37] *= 8.0
        qkv = qkv.to(torch.bfloat16)
        s.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], cos=None, sin=None, q_norm=None, k_norm=None)
        if case["rot"]:
            r = case["rot"]
            freq = THETA ** (-torch.arange(0, r, 2, dtype=torch.float64, device=dev) / r)
            angle = torch.arange(max(total), dtype=torch.float64, device=dev)[:, None] * freq
            s.update(cos=angle.cos().float(), sin=angle.sin().float())
        if case["norm"]:
            s.update(q_norm=1 + 0.1 * normal(D), k_norm=1 + 0.1 * normal(D))
        s.update(q_out=torch.zeros((T, hq, D), dtype=torch.bfloat16, device=dev),
                 k_back=torch.zeros((T, hkv, D), dtype=torch.bfloat16, device=dev),
                 v_back=torch.zeros((T, hkv, D), dtype=torch.bfloat16, device=dev))
        return s
    s["q"] = (1.5 * normal(T, hq, D)).to(torch.bfloat16)
    s["slopes"] = torch.exp2(-8.0 * (torch.arange(hq, device=dev) + 1) / hq) if case["slopes"] else None
    s["out"] = torch.zeros((T, hq, D), dtype=torch.bfloat16, device=dev)
    s["lse"] = torch.zeros((T, hq), device=dev)
    if case["op"] == "prefix":
        s["prefix_table"] = order[:ppages].contiguous()
    return s


# ------------------------------------------------------------- plain forms

def _hadamard(n):
    i = torch.arange(n, device="cuda")
    x = i[:, None] & i[None, :]
    odd = torch.zeros_like(x)
    for bit in range(7):
        odd ^= (x >> bit) & 1
    return 1.0 - 2.0 * odd.double()


def _head_forward(x, weight, cos, sin, interleaved):
    """Norm over the head, rotation of its first channels, H128 / sqrt(128): float64 in and out."""
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.double()
    if cos is not None:
        r = 2 * cos.shape[-1]
        c, s, y = cos.double()[:, None], sin.double()[:, None], x[..., :r]
        a, b = (y[..., 0::2], y[..., 1::2]) if interleaved else (y[..., :r // 2], y[..., r // 2:])
        u, w = a * c - b * s, b * c + a * s
        y = torch.stack((u, w), -1).flatten(-2) if interleaved else torch.cat((u, w), -1)
        x = torch.cat((y, x[..., r:]), -1)
    return x @ _hadamard(D) * NORM


def _rows(pool, key, page, row, bits):
    """Rows of the pages as float32: codes less their zero point, times their scale."""
    codes = _unpack(pool[key + "_codes"][page, :, row], bits).float()
    return (codes - pool[key + "_zero"][page, :, row].float()[..., None]) * pool[key + "_scale"][page, :, row][..., None]


def _append(s):
    case, n, pool, bits = s["case"], s["used"], s["pool"], s["case"]["bits"]
    pos = s["cached"].long()[s["seq"]] + s["nth"]
    page = s["block_table"].long()[s["seq"], pos // case["page"]]
    row = pos % case["page"]
    cos, sin = (None, None) if s["cos"] is None else (s["cos"][pos], s["sin"][pos])
    s["q_out"][:n] = _head_forward(s["q"][:n].double(), s["q_norm"], cos, sin, case["interleaved"]).to(torch.bfloat16)
    k = _head_forward(s["k"][:n].double(), s["k_norm"], cos, sin, case["interleaved"]).float()
    for key, x in (("k", k), ("v", s["v"][:n].float())):
        codes, scale, zero = _quantize(x, bits)
        pool[key + "_codes"][page, :, row] = _pack(codes, bits)
        pool[key + "_scale"][page, :, row] = scale
        pool[key + "_zero"][page, :, row] = zero
        s[key + "_back"][:n] = _rows(pool, key, page, row, bits).to(torch.bfloat16)
    return {"q": s["q_out"], "k": s["k_back"], "v": s["v_back"]}


def _attend(s):
    case, pool, bits, ps = s["case"], s["pool"], s["case"]["bits"], s["case"]["page"]
    B, hq, hkv, Q, S, P = case["batch"], case["hq"], case["hkv"], s["max_q"], s["max_len"], case.get("prefix", 0)
    grp, dev = hq // hkv, s["q"].device
    cu, length = s["cu_seqlens"].long(), s["lengths"].long()
    i = torch.arange(Q, device=dev)
    q = s["q"][(cu[:-1, None] + i).clamp(max=s["T"] - 1)].float()                # [B, Q, hq, D]
    q = q.view(B, Q, hkv, grp, D).permute(0, 2, 3, 1, 4)                         # [B, hkv, grp, Q, D]
    j = torch.arange(S, device=dev)
    page, row = s["block_table"].long()[:, j // ps], (j % ps).expand(B, S)
    K, V = (_rows(pool, key, page, row, bits).permute(0, 2, 1, 3) for key in ("k", "v"))   # [B, hkv, S, D]
    x = q.reshape(B, hkv, grp * Q, D) @ K.transpose(-1, -2)                      # [B, hkv, grp Q, S]
    kpos = P + j
    if P:
        jp = torch.arange(P, device=dev)
        pk, pv = (_rows(pool, key, s["prefix_table"].long()[jp // ps], jp % ps, bits).permute(1, 0, 2) for key in ("k", "v"))
        flat = q.permute(1, 0, 2, 3, 4).reshape(hkv, B * grp * Q, D)
        xp = (flat @ pk.transpose(-1, -2)).view(hkv, B, grp * Q, P).transpose(0, 1)
        x, kpos = torch.cat((xp, x), -1), torch.cat((jp, kpos))
    x = x.view(B, hkv, grp, Q, P + S) * NORM
    if case["softcap"]:
        x = case["softcap"] * torch.tanh(x / case["softcap"])
    qpos = P + (length - (cu[1:] - cu[:-1]))[:, None] + i                        # [B, Q]
    dist = qpos[:, None, None, :, None] - kpos
    if s["slopes"] is not None:
        x = x - s["slopes"].view(hkv, grp, 1, 1) * dist
    hidden = dist < 0
    if case["window"]:
        hidden = hidden | (dist >= case["window"])
    x = x.masked_fill(hidden, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    y = p[..., P:].reshape(B, hkv, grp * Q, S) @ V.masked_fill((j >= length[:, None])[:, None, :, None], 0.0)
    if P:
        pp = p[..., :P].transpose(0, 1).reshape(hkv, B * grp * Q, P) @ pv
        y = y + pp.view(hkv, B, grp * Q, D).transpose(0, 1)
    y = y.view(B, hkv, grp, Q, D) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (m + torch.log(total)).squeeze(-1)
    n = s["used"]
    s["out"][:n] = y.permute(0, 3, 1, 2, 4).reshape(B, Q, hq, D)[s["seq"], s["nth"]].to(torch.bfloat16)
    s["lse"][:n] = lse.permute(0, 3, 1, 2).reshape(B, Q, hq)[s["seq"], s["nth"]]
    return {"out": s["out"], "lse": s["lse"]}


def run(s):
    case = s["case"]
    if own:
        import rotation_ptq_b200 as sq
        pages = s.get("pages")
        if pages is None:
            pages = s["pages"] = sq.KVPages(**s["pool"])
        if case["op"] == "append":
            sq.kv_paged_append(s["q"], s["k"], s["v"], pages, s["block_table"], s["cu_seqlens"], s["cached"],
                               s["cos"], s["sin"], interleaved=case["interleaved"], q_norm=s["q_norm"],
                               k_norm=s["k_norm"], eps=EPS, q_out=s["q_out"])
            sq.kv_paged_dequant(pages, s["block_table"], s["cu_seqlens"], s["cached"], s["T"],
                                k_out=s["k_back"], v_out=s["v_back"])
            return {"q": s["q_out"], "k": s["k_back"], "v": s["v_back"]}
        args = dict(softcap=case["softcap"], window=case["window"], slopes=s["slopes"], out=s["out"], lse=s["lse"])
        if case["op"] == "attend":
            sq.kv_paged_attention(s["q"], pages, s["block_table"], s["cu_seqlens"], s["lengths"], s["max_q"], **args)
        else:
            sq.kv_prefix_attention(s["q"], pages, s["prefix_table"], case["prefix"], s["block_table"],
                                   s["cu_seqlens"], s["lengths"], s["max_q"], **args)
        return {"out": s["out"], "lse": s["lse"]}
    return _append(s) if case["op"] == "append" else _attend(s)


# ------------------------------------------------------------------- work

def work(case):
    new, cached = _lengths(case)
    hq, hkv, T = case["hq"], case["hkv"], sum(new)
    row = 2 * hkv * (D * case["bits"] // 8 + 5)                  # K and V codes, scale and zero point of a token
    if case["op"] == "append":
        tables = 4 * case["rot"] * min(T, max(n + c for n, c in zip(new, cached)))
        nbytes = T * (2 * D * (hq + 2 * hkv) + 2 * D * hq + row) + tables        # append
        nbytes += T * (row + 2 * D * 2 * hkv)                                    # read-back
        flops = T * ((hq + hkv) * (7 * D + 3 * case["rot"] + 4 * D * case["norm"]) + 2 * hkv * 6 * D + 2 * hkv * 2 * D)
        return {"bytes": nbytes, "flops": flops}
    P, W = case.get("prefix", 0), case["window"]
    pairs, rows, first = 0, 0, P
    for n, c in zip(new, cached):
        a = P + c                                                # position of the first new token
        if W:
            full = min(n, max(0, W - 1 - a))                     # new tokens that see all that is before them
            pairs += full * (a + 1) + full * (full - 1) // 2 + (n - full) * W
        else:
            pairs += n * (a + 1) + n * (n - 1) // 2
        low = max(0, a - W + 1) if W else 0
        rows += P + c + n - max(P, low)                          # its own rows that some new token sees
        first = min(first, low)
    rows += P - first                                            # and the shared ones once
    return {"bytes": T * hq * (4 * D + 4) + rows * row, "flops": 4 * D * hq * pairs}


# -------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    new, cached = _lengths(case)
    hq, hkv, ps, top = case["hq"], case["hkv"], case["page"], 2 ** case["bits"] - 1
    if case["op"] == "append":
        n = sum(new)
        h = torch.ones((1, 1), dtype=torch.float64, device="cuda")
        while h.shape[0] < D:
            h = torch.cat((torch.cat((h, h), 1), torch.cat((h, -h), 1)), 0)
        pos = torch.tensor([c + i for m, c in zip(new, cached) for i in range(m)], device="cuda")

        def turn(x, w):
            x = x.double()
            if w is not None:
                x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / D + EPS) * w.double()
            y = x.clone()
            for e in range(case["rot"] // 2):
                c, d = s["cos"][pos, e].double()[:, None], s["sin"][pos, e].double()[:, None]
                a, b = (2 * e, 2 * e + 1) if case["interleaved"] else (e, e + case["rot"] // 2)
                y[..., a], y[..., b] = x[..., a] * c - x[..., b] * d, x[..., b] * c + x[..., a] * d
            return torch.einsum("thd,de->the", y, h) / math.sqrt(D)

        def f32(x):
            return x.float().double()

        def grid(x):
            # the cache's rule rounds the value, the step and every quotient to float32: bf16 values
            # lie on borders between two codes often enough for that to decide
            x = f32(x)
            lo, hi = torch.minimum(x.min(-1, keepdim=True)[0], x.new_zeros(1)), torch.maximum(x.max(-1, keepdim=True)[0], x.new_zeros(1))
            step = f32(f32(hi - lo) / torch.full_like(hi, top))
            step[step == 0] = 1
            zero = torch.round(f32(-lo / step)).clamp(0, top)
            return ((torch.round(f32(x / step)) + zero).clamp(0, top) - zero) * step

        behind = lambda x: torch.cat((x, x.new_zeros((case["pad"],) + x.shape[1:])))  # noqa: E731
        return {"q": behind(turn(s["q"][:n], s["q_norm"])), "k": behind(grid(turn(s["k"][:n], s["k_norm"]))),
                "v": behind(grid(s["v"][:n].double()))}

    def cache(key, numbers, count):
        numbers = numbers[: -(-count // ps)].long()
        c = s["pool"][key + "_codes"][numbers].long()                            # [pages, hkv, ps, bytes]
        if case["bits"] == 4:
            c = torch.stack((c % 16, c // 16), -1).reshape(c.shape[:-1] + (D,))
        x = (c - s["pool"][key + "_zero"][numbers].long()[..., None]).double() * s["pool"][key + "_scale"][numbers].double()[..., None]
        return x.permute(1, 0, 2, 3).reshape(hkv, -1, D)[:, :count]

    P, grp, at = case.get("prefix", 0), hq // hkv, 0
    out = torch.zeros((s["T"], hq, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((s["T"], hq), dtype=torch.float64, device="cuda")
    shared = [cache(key, s["prefix_table"], P) for key in ("k", "v")] if P else None
    for b, (n, c) in enumerate(zip(new, cached)):
        K, V = cache("k", s["block_table"][b], c + n), cache("v", s["block_table"][b], c + n)
        if P:
            K, V = torch.cat((shared[0], K), 1), torch.cat((shared[1], V), 1)
        where = torch.arange(P + c, P + c + n, device="cuda")[:, None] - torch.arange(P + c + n, device="cuda")[None]
        seen = (where >= 0) if not case["window"] else (where >= 0) & (where < case["window"])
        for h in range(hq):
            x = s["q"][at:at + n, h].double() @ K[h // grp].T / math.sqrt(D)
            if case["softcap"]:
                x = case["softcap"] * torch.tanh(x / case["softcap"])
            if s["slopes"] is not None:
                x = x - s["slopes"][h].double() * where
            x = torch.where(seen, x, torch.full_like(x, -math.inf))
            lse[at:at + n, h] = torch.logsumexp(x, -1)
            out[at:at + n, h] = torch.softmax(x, -1) @ V[h // grp]
        at += n
    return {"out": out, "lse": lse}
