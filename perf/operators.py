"""The paged-cache operators as they are measured: appending keys and values to a paged latent
cache (with the rotary embedding applied on the way, held in 16 or in 4 bits), reading cached
rows back, and attention over the pages.

With ``own`` false, ``run`` computes them in elementary torch operations; with ``own`` true it
calls the library.  Shapes: sequence b holds L_b tokens after the call, the last n_b of them new,
so new token i sits at position L_b - n_b + i.  Pages are [n_pages, kv heads, page size, row]; a
4-bit row packs channel 2j in the low and 2j + 1 in the high half of byte j, and ``scales`` holds
(key scale, key zero, value scale, value zero) in float16 for each (page, kv head, slot).
"""
import math

import numpy as np
import torch

own = False

ROPE_BASE = 10000.0
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------- cases
def _case(name, op, bits, dtype, batch, heads, kv_heads, dim, page, new, past):
    """new, past: (lowest, highest) over the batch; the sequences are spread between them."""
    c = dict(op=op, bits=bits, dtype=dtype, batch=batch, heads=heads, kv_heads=kv_heads, dim=dim,
             page=page, new_lo=new[0], new_hi=new[1], past_lo=past[0], past_hi=past[1])
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one new token of one short sequence: the smallest call, launch latency only
        _case("append_one_16bit_d16", "append", 16, "f16", 1, 4, 4, 16, 16, (1, 1), (100, 100)),
        # a serving step: one new token for each of 64 sequences of different lengths
        _case("append_step_16bit_d64", "append", 16, "f16", 64, 16, 4, 64, 64, (1, 1), (90, 1100)),
        # two 16k prompts written whole after their prefill
        _case("append_prompt_16bit_d64", "append", 16, "bf16", 2, 16, 4, 64, 64, (16384, 16384), (0, 0)),
        # a few tokens a sequence (a draft) into 4-bit pages, and the sequences read back dense
        _case("append_draft_4bit_d128", "append", 4, "bf16", 7, 6, 2, 128, 16, (1, 5), (0, 301)),
        # four 4k prompts of the ungrouped layer into 4-bit pages, and read back dense
        _case("append_prompt_4bit_d32", "append", 4, "f16", 4, 16, 16, 32, 32, (4096, 4096), (0, 0)),
        # one token over one short sequence: launch latency only
        _case("attend_one_4bit_d16", "attend", 4, "f16", 1, 4, 4, 16, 16, (1, 1), (100, 100)),
        # the decode workload: 64 sequences of 8k tokens
        _case("attend_8k_4bit_d32", "attend", 4, "f16", 64, 16, 4, 32, 64, (1, 1), (8191, 8191)),
        # a ragged batch, from one token to 16k, in small pages
        _case("attend_ragged_4bit_d64", "attend", 4, "bf16", 40, 16, 4, 64, 16, (1, 1), (0, 16383)),
        # one user with a long context: little else to fill the machine with
        _case("attend_long_4bit_d32", "attend", 4, "f16", 1, 32, 8, 32, 64, (1, 1), (32700, 32700)),
        # drafts of up to eight tokens verified in one pass
        _case("attend_draft_4bit_d64", "attend", 4, "bf16", 16, 32, 4, 64, 32, (1, 8), (900, 4001)),
        # a 512-token piece of each of two prompts over what is cached of them
        _case("attend_chunk_4bit_d64", "attend", 4, "f16", 2, 16, 4, 64, 64, (500, 512), (7000, 7681)),
        # the same serving step over 16-bit pages
        _case("attend_8k_16bit_d64", "attend", 16, "f16", 32, 16, 4, 64, 64, (1, 1), (8000, 8191)),
    ]


def draw(rng):
    def logint(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    while True:
        op = rng.choice(["append", "attend", "attend"])
        bits = rng.choice([4, 4, 16])
        kv = rng.choice([1, 2, 3, 4, 5, 8, 16])
        heads = kv * rng.choice([1, 1, 2, 3, 4, 4, 7, 8])
        dim = rng.choice([16, 32, 64, 128])
        page = rng.choice([16, 32, 64, 128])
        batch = logint(1, 64)
        if op == "append":
            new_hi = rng.choice([1, 1, 3, logint(2, 16384)])
            past_hi = logint(1, 2048)
        else:
            new_hi = rng.choice([1, 1, 1, rng.randint(2, 8), logint(9, 512)])
            past_hi = logint(1, 32768)
        new_lo = rng.choice([new_hi, max(1, new_hi // 2), 1])
        past_lo = rng.choice([past_hi, past_hi // 2, 0])
        c = _case(None, op, bits, rng.choice(["f16", "bf16"]), batch, heads, kv, dim, page,
                  (new_lo, new_hi), (past_lo, past_hi))
        new, past = _lengths(c)
        most = max(new) + max(past)
        held = batch * most * kv * dim                       # padded rows of the plain form
        scores = batch * heads * max(new) * most if op == "attend" else 0
        rows = sum(new) * (heads + 2 * kv) * dim
        w = work(c)
        # no more than the largest listed case of its kind: memory of the plain form, bytes, flops
        if op == "append":
            if max(rows, held) <= 2 ** 25 and w["bytes"] <= 160e6:
                return c
        elif held <= 2 ** 26 and scores <= 2 ** 27 and w["flops"] <= 30e9 and w["bytes"] <= 250e6:
            return c


def _lengths(c):
    """(new, past) of each sequence: spread over the case's ranges by multiples of two
    irrational steps, the ends taken where the batch has two or more."""
    def spread(lo, hi, step):
        out = [lo + int((hi - lo + 1) * ((b * step) % 1.0)) for b in range(c["batch"])]
        if c["batch"] > 1:
            out[1] = hi
        return out
    return spread(c["new_lo"], c["new_hi"], 0.6180339887), spread(c["past_lo"], c["past_hi"], 0.4142135624)


def work(case):
    new, past = _lengths(case)
    H, kv, d = case["heads"], case["kv_heads"], case["dim"]
    total = [n + p for n, p in zip(new, past)]
    pages = sum(-(-t // case["page"]) for t in total)
    held = 2 * (d // 2) + 8 if case["bits"] == 4 else 4 * d  # bytes of one (token, kv head)
    meta = 4 * (pages + 2 * case["batch"])
    if case["op"] == "append":
        rows = sum(new) * (H + 2 * kv) * d * 2
        byt = rows + sum(new) * (H * d * 2 + kv * held) + meta
        if case["bits"] == 4:                                # read back dense
            byt += sum(total) * kv * (held + 4 * d)
        return {"bytes": byt, "flops": 3 * sum(new) * (H + kv) * d}
    seen = sum(n * p + n * (n + 1) // 2 for n, p in zip(new, past))
    return {"bytes": sum(total) * kv * held + 2 * sum(new) * H * d * 2 + meta,
            "flops": 4 * d * H * seen}


# ------------------------------------------------------------------------------- inputs
def _quantise(x):
    """x [..., d] float32 -> (bytes [..., d / 2], scale, zero [...] float16)."""
    lo, hi = x.amin(-1), x.amax(-1)
    zero, scale = lo.half(), ((hi - lo) / 15).half()
    s = scale.float().unsqueeze(-1)
    n = torch.round((x - zero.float().unsqueeze(-1)) / torch.where(s == 0, torch.ones_like(s), s))
    n = torch.where(s == 0, torch.zeros_like(n), n.clamp(0, 15)).to(torch.uint8)
    return n[..., 0::2] | (n[..., 1::2] << 4), scale, zero


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(dev).manual_seed(1000003 * seed + 17)
    dt = DTYPES[case["dtype"]]
    B, H, kv, d, ps = (case[k] for k in ("batch", "heads", "kv_heads", "dim", "page"))
    new, past = _lengths(case)
    total = [n + p for n, p in zip(new, past)]
    need = [-(-t // ps) for t in total]
    n_pages = sum(need) + 3                                  # a pool with a few pages unused
    order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    table = torch.zeros(B, max(need), dtype=torch.int32, device=dev)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    k, v = randn(n_pages, kv, ps, d), randn(n_pages, kv, ps, d)
    scales = None
    if case["bits"] == 4:
        k, ks, kz = _quantise(k)
        v, vs, vz = _quantise(v)
        scales = torch.stack([ks, kz, vs, vz], -1).contiguous()
    else:
        k, v = k.to(dt), v.to(dt)
    T = sum(new)

    def starts(n):
        return torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device=dev)

    s = dict(case=case, k=k, v=v, scales=scales, table=table, tokens=T, kept=sum(total),
             lengths=torch.tensor(total, dtype=torch.int32, device=dev),
             cu=starts(new) if len(set(new)) > 1 else None, kv_cu=starts(total),
             q=randn(T, H, d).to(dt), max_new=max(new), max_total=max(total))
    if case["op"] == "append":
        s["k_new"], s["v_new"] = randn(T, kv, d).to(dt), randn(T, kv, d).to(dt)
    # sequence and index within it of every new token, as a scheduler has them
    s["tok_seq"] = torch.repeat_interleave(torch.arange(B, device=dev), torch.tensor(new, device=dev))
    first = torch.tensor(np.cumsum([0] + new[:-1]), device=dev)
    s["tok_idx"] = torch.arange(T, device=dev) - first[s["tok_seq"]]
    s["past"] = torch.tensor(past, device=dev)
    return s


# ------------------------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    if own:
        import compressed_latent_space_b200 as cls

        cache = cls.PagedCache.from_pages(s["k"], s["v"], s["table"], s["lengths"], s["scales"])
        if case["op"] == "attend":
            return cache.attend(s["q"], cu_seqlens=s["cu"])
        q = cache.append(s["k_new"], s["v_new"], s["q"], cu_seqlens=s["cu"], rope_base=ROPE_BASE)
        if case["bits"] == 16:
            return {"q": q, "k": s["k"], "v": s["v"]}
        k, v = cache.gather(s["kept"], cu_seqlens=s["kv_cu"], dtype=s["q"].dtype)
        return {"q": q, "k": k, "v": v}
    return _plain_attend(s) if case["op"] == "attend" else _plain_append(s)


def _rotate(x, pos):
    """x [T, heads, d] rotated at positions pos [T]; angles in 64 bits, the rest in 32."""
    half = x.shape[-1] // 2
    theta = ROPE_BASE ** (-torch.arange(half, device=x.device, dtype=torch.float64) / half)
    ang = pos.double()[:, None] * theta
    c, sn = ang.cos().float()[:, None], ang.sin().float()[:, None]
    a, b = x[..., :half].float(), x[..., half:].float()
    return torch.cat([a * c - b * sn, a * sn + b * c], -1)


def _plain_append(s):
    case, dt = s["case"], s["q"].dtype
    pos = s["past"][s["tok_seq"]] + s["tok_idx"]
    page = s["table"][s["tok_seq"], pos // case["page"]].long()
    slot = pos % case["page"]
    q, k = _rotate(s["q"], pos).to(dt), _rotate(s["k_new"], pos)
    if case["bits"] == 16:
        s["k"][page, :, slot] = k.to(dt)
        s["v"][page, :, slot] = s["v_new"]
        return {"q": q, "k": s["k"], "v": s["v"]}
    kq, ks, kz = _quantise(k)
    vq, vs, vz = _quantise(s["v_new"].float())
    s["k"][page, :, slot] = kq
    s["v"][page, :, slot] = vq
    s["scales"][page, :, slot] = torch.stack([ks, kz, vs, vz], -1)
    # every cached token in order, as one dense [tokens, kv heads, d]
    t = torch.arange(s["kept"], device=q.device)
    seq = torch.searchsorted(s["kv_cu"].long(), t, right=True) - 1
    at = t - s["kv_cu"].long()[seq]
    page, slot = s["table"][seq, at // case["page"]].long(), at % case["page"]
    sc = s["scales"][page, :, slot].float()
    return {"q": q, "k": _unpack(s["k"][page, :, slot], sc[..., 0], sc[..., 1]).to(dt),
            "v": _unpack(s["v"][page, :, slot], sc[..., 2], sc[..., 3]).to(dt)}


def _unpack(codes, scale, zero):
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()
    return n * scale[..., None] + zero[..., None]


def _plain_attend(s):
    case, dt = s["case"], s["q"].dtype
    B, H, kv, d, ps = (case[k] for k in ("batch", "heads", "kv_heads", "dim", "page"))
    N, L, G = s["max_new"], s["max_total"], H // kv
    # padded dense keys and values [B, kv heads, L, d]
    pages = s["table"].long()
    k, v = s["k"][pages], s["v"][pages]                      # [B, pages, kv, ps, row]
    if case["bits"] == 4:
        sc = s["scales"][pages].float()
        k, v = _unpack(k, sc[..., 0], sc[..., 1]), _unpack(v, sc[..., 2], sc[..., 3])
    k, v = (x.float().transpose(1, 2).reshape(B, kv, -1, d)[:, :, :L] for x in (k, v))
    key = torch.arange(L, device=k.device)
    live = key[None] < s["lengths"][:, None]
    v = torch.where(live[:, None, :, None], v, torch.zeros((), device=v.device))
    q = torch.zeros(B, N, H, d, device=k.device)
    q[s["tok_seq"], s["tok_idx"]] = s["q"].float()
    q = q.view(B, N, kv, G, d).permute(0, 2, 1, 3, 4).reshape(B, kv, N * G, d)
    x = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(d)
    pos = s["past"][:, None] + torch.arange(N, device=k.device)
    seen = (key[None, None] <= pos[..., None]) & live[:, None]
    seen = seen.repeat_interleave(G, 1)[:, None]             # [B, 1, N G, L]
    x = x.masked_fill(~seen, float("-inf"))
    x = torch.exp(x - x.amax(-1, keepdim=True))
    o = torch.matmul(x, v) / x.sum(-1, keepdim=True)
    o = o.view(B, kv, N, G, d).permute(0, 2, 1, 3, 4).reshape(B, N, H, d)
    return o[s["tok_seq"], s["tok_idx"]].to(dt)


# ------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    """The definition, sequence by sequence, in 64 bits."""
    s = prepare(case, seed)
    new, past = _lengths(case)
    H, kv, d, ps = (case[k] for k in ("heads", "kv_heads", "dim", "page"))
    four = case["bits"] == 4

    def rows(b, n):
        """The first n cached keys and values of sequence b, [n, kv, d] each."""
        at = np.arange(n)
        pg = s["table"][b].cpu().numpy()[at // ps]
        pg, sl = torch.as_tensor(pg, device="cuda").long(), torch.as_tensor(at % ps, device="cuda")
        out = []
        for i, name in enumerate("kv"):
            r = s[name][pg, :, sl]
            if four:
                sc = s["scales"][pg, :, sl].double()
                low, high = (r & 15).double(), (r >> 4).double()
                r = torch.empty(n, kv, d, dtype=torch.float64, device="cuda")
                r[..., 0::2], r[..., 1::2] = low, high
                r = r * sc[..., 2 * i, None] + sc[..., 2 * i + 1, None]
            out.append(r.double())
        return out

    def turned(x, p0):
        j = torch.arange(d // 2, dtype=torch.float64, device="cuda")
        ang = (p0 + torch.arange(len(x), dtype=torch.float64, device="cuda"))[:, None] * ROPE_BASE ** (-2 * j / d)
        w = torch.polar(torch.ones_like(ang), ang)[:, None]
        z = torch.complex(x[..., :d // 2], x[..., d // 2:]) * w
        return torch.cat([z.real, z.imag], -1)

    def in_four_bits(x):
        lo, hi = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
        zero, scale = lo.half().double(), ((hi - lo) / 15).half().double()
        n = torch.where(scale > 0, ((x - zero) / scale.clamp_min(1e-30)).round().clamp(0, 15), 0.0)
        return n * scale + zero

    T0, outs = 0, []
    if case["op"] == "attend":
        for b, (n, p) in enumerate(zip(new, past)):
            K, V = rows(b, n + p)
            q = s["q"][T0:T0 + n].double().view(n, kv, H // kv, d)
            x = torch.einsum("ngrd,lgd->ngrl", q, K) * d ** -0.5
            later = torch.arange(n + p, device="cuda")[None] > p + torch.arange(n, device="cuda")[:, None]
            x.masked_fill_(later[:, None, None], -math.inf)
            outs.append(torch.einsum("ngrl,lgd->ngrd", torch.softmax(x, -1), V).reshape(n, H, d))
            T0 += n
        return torch.cat(outs)
    q64, ks, vs = [], [], []
    if not four:
        ks, vs = s["k"].double(), s["v"].double()
    for b, (n, p) in enumerate(zip(new, past)):
        q64.append(turned(s["q"][T0:T0 + n].double(), p))
        kn, vn = turned(s["k_new"][T0:T0 + n].double(), p), s["v_new"][T0:T0 + n].double()
        if four:
            old = rows(b, p) if p else (kn[:0], vn[:0])
            ks.append(torch.cat([old[0], in_four_bits(kn)]))
            vs.append(torch.cat([old[1], in_four_bits(vn)]))
        else:
            at = np.arange(p, p + n)
            pg = torch.as_tensor(s["table"][b].cpu().numpy()[at // ps], device="cuda").long()
            sl = torch.as_tensor(at % ps, device="cuda")
            ks[pg, :, sl], vs[pg, :, sl] = kn, vn
        T0 += n
    if four:
        ks, vs = torch.cat(ks), torch.cat(vs)
    return {"q": torch.cat(q64), "k": ks, "v": vs}
