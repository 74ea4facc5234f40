"""Cases, plain forms and library calls of the paged-cache operators.

Four operators that a speculative decoding loop runs one after the other:

* ``append``  -- q | k | v rows of new tokens: optional RMS norm of each query
  and key head, rotation, K and V quantised to INT16 into the pages of their
  sequences, q returned (kv_append_paged);
* ``attend``  -- causal attention of each sequence's new tokens over its pages
  (attn_paged);
* ``softmax`` -- probabilities of logits rows (softmax_rows);
* ``verify``  -- drafted tokens accepted or rejected against the target's
  probabilities, and the token that follows them (spec_verify).

``run`` computes the plain form with elementary torch operations, or, where
``own`` is true, makes the library's calls.
"""
import math

import torch

own = False

EPS = 1e-6
SCALE = float(torch.tensor(1.0 / math.sqrt(128.0), dtype=torch.float32))
MAX_POS = 8192


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # one verification step of 64 conversations with up to 5 drafted tokens each, head norms on
        {"name": "append_draft_64x5", "op": "append", "seqs": 64, "new": 5, "ragged": True, "ctx": 512, "hq": 32,
         "hkv": 8, "page": 16, "norm": True},
        # a prompt of 8192 tokens prefilled in one call
        {"name": "append_prefill_8192", "op": "append", "seqs": 1, "new": 8192, "ragged": False, "ctx": 8192, "hq": 32,
         "hkv": 8, "page": 64, "norm": False},
        # a single conversation, one token, short context: latency
        {"name": "attend_one_300", "op": "attend", "seqs": 1, "new": 1, "ragged": False, "ctx": 300, "hq": 32, "hkv": 8,
         "page": 16},
        # the decode step of a full batch
        {"name": "attend_decode_128x2048", "op": "attend", "seqs": 128, "new": 1, "ragged": False, "ctx": 2048, "hq": 32,
         "hkv": 8, "page": 64},
        # the decode step of a batch of unequal lengths
        {"name": "attend_decode_64x8192", "op": "attend", "seqs": 64, "new": 1, "ragged": True, "ctx": 8192, "hq": 32,
         "hkv": 8, "page": 64},
        # verification of up to 5 drafted tokens a conversation, small pages
        {"name": "attend_draft_32x5", "op": "attend", "seqs": 32, "new": 5, "ragged": True, "ctx": 4099, "hq": 32,
         "hkv": 8, "page": 16},
        # chunks of prompts of unequal lengths in one call
        {"name": "attend_chunks_12x700", "op": "attend", "seqs": 12, "new": 700, "ragged": True, "ctx": 4001, "hq": 16,
         "hkv": 4, "page": 32},
        # a prompt of 8192 tokens prefilled in one call
        {"name": "attend_prefill_8192", "op": "attend", "seqs": 1, "new": 8192, "ragged": False, "ctx": 8192, "hq": 32,
         "hkv": 8, "page": 128},
        # probabilities of one conversation's draft, odd vocabulary
        {"name": "softmax_3x32003", "op": "softmax", "rows": 3, "n": 32003, "temp": 0.7},
        # probabilities of a whole verification step: 64 conversations, 4 drafted tokens and one more
        {"name": "softmax_320x32000", "op": "softmax", "rows": 320, "n": 32000, "temp": 1.0},
        # one conversation whose draft comes from a lookup (no draft probabilities)
        {"name": "verify_1x7_lookup", "op": "verify", "seqs": 1, "draft": 7, "n": 32003, "probs": False},
        # a whole verification step
        {"name": "verify_64x4", "op": "verify", "seqs": 64, "draft": 4, "n": 32000, "probs": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append", "attend", "attend", "attend", "softmax", "verify"])
    if op in ("append", "attend"):
        hq, hkv = rng.choice([(32, 8), (16, 4), (8, 2), (8, 8), (16, 8), (24, 8), (32, 4)])
        page = rng.choice([16, 32, 64, 128])
        if op == "append":
            seqs = _log(rng, 1, 128)
            new = _log(rng, 1, max(1, 8192 // seqs))
            ctx = min(MAX_POS, new + _log(rng, 1, 200))
            return {"op": op, "seqs": seqs, "new": new, "ragged": rng.random() < 0.5, "ctx": ctx, "hq": hq, "hkv": hkv,
                    "page": page, "norm": rng.random() < 0.5}
        kind = rng.choice(["decode", "draft", "chunk"])
        if kind == "decode":
            seqs, new = _log(rng, 1, 128), 1
            ctx = _log(rng, 17, min(MAX_POS, 262144 // seqs))
        elif kind == "draft":
            seqs, new = _log(rng, 1, 64), rng.randint(2, 9)
            ctx = _log(rng, 32, min(MAX_POS, 131072 // seqs))
        else:
            seqs, new = _log(rng, 1, 12), _log(rng, 16, 1024)
            ctx = max(new, _log(rng, 64, 4096))
        return {"op": op, "seqs": seqs, "new": new, "ragged": rng.random() < 0.5, "ctx": ctx, "hq": hq, "hkv": hkv,
                "page": page}
    if op == "softmax":
        n = _log(rng, 1000, 131072)
        return {"op": op, "rows": _log(rng, 1, max(1, min(512, 16777216 // n))), "n": n,
                "temp": round(rng.uniform(0.3, 2.0), 3)}
    n = _log(rng, 1000, 131072)
    return {"op": op, "seqs": _log(rng, 1, max(1, min(128, 2097152 // n))), "draft": rng.randint(1, 8), "n": n,
            "probs": rng.random() < 0.7}


# ----------------------------------------------------------------- inputs ---

def _lens(case):
    """Context lengths (the new tokens included) and new tokens of each sequence: plain numbers that go by the case
    alone, so that work() knows them without a state."""
    n, new, ctx = case["seqs"], case["new"], case["ctx"]
    if not case["ragged"]:
        return [ctx] * n, [new] * n
    news = [1 + (i * 7919 + 3) % new for i in range(n)]
    low = min(ctx, max(1, ctx // 8))
    lens = [max(k, low + (i * 104729 + 17) % (ctx - low + 1)) for i, k in enumerate(news)]
    lens[-1] = ctx
    return lens, news


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _paged(case, g):
    """Sequence descriptors and a page table over a pool of pages in random order."""
    lens, news = _lens(case)
    page, n = case["page"], case["seqs"]
    per = -(-max(lens) // page)
    pages = n * per
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).view(n, per)
    start = [0]
    for k in news:
        start.append(start[-1] + k)
    return {"table": table, "q_start": torch.tensor(start, dtype=torch.int32, device="cuda"),
            "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"), "rows": start[-1], "max_new": max(news),
            "max_len": max(lens), "pages": pages}


def _codes(x):
    """INT16 codes and scales of rows of 128 values."""
    s = x.abs().amax(-1) / 32767.0
    q = torch.round(x / s.clamp_min(1e-30).unsqueeze(-1)).clamp(-32767, 32767)
    return q.to(torch.int16), s


def _pool(case, pages, g):
    """K or V pages whose channels differ in size (a log-uniform factor from 0.1 to 10)."""
    shape = (pages, case["hkv"], case["page"], 128)
    c = torch.exp((torch.rand(case["hkv"], 1, 128, generator=g, device="cuda") * 2 - 1) * math.log(10.0))
    codes = torch.empty(shape, dtype=torch.int16, device="cuda")
    scale = torch.empty(shape[:3], dtype=torch.float32, device="cuda")
    step = max(1, (1 << 26) // (case["hkv"] * case["page"] * 128))
    for a in range(0, pages, step):
        b = min(pages, a + step)
        codes[a:b], scale[a:b] = _codes(torch.randn((b - a,) + shape[1:], generator=g, device="cuda") * c)
    return codes, scale


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op in ("append", "attend"):
        s.update(_paged(case, g))
        hq, hkv, rows = case["hq"], case["hkv"], s["rows"]
        s["k"], s["k_scale"] = _pool(case, s["pages"], g)
        s["v"], s["v_scale"] = _pool(case, s["pages"], g)
        if op == "append":
            x = torch.randn(rows, (hq + 2 * hkv) * 128, generator=g, device="cuda")
            x *= torch.exp((torch.rand(x.shape[1], generator=g, device="cuda") * 2 - 1) * math.log(10.0))
            s["qkv"] = x
            theta = torch.pow(10000.0, -torch.arange(64, dtype=torch.float64, device="cuda") / 64)
            a = torch.arange(MAX_POS, dtype=torch.float64, device="cuda")[:, None] * theta
            s["cos"], s["sin"] = a.cos().float(), a.sin().float()
            s["q_gain"], s["k_gain"] = (torch.rand(2, 128, generator=g, device="cuda") + 0.5).unbind() if case["norm"] else (None, None)
        else:
            s["q"] = torch.randn(rows, hq, 128, generator=g, device="cuda")
        return s
    if op == "softmax":
        s["logits"] = torch.randn(case["rows"], case["n"], generator=g, device="cuda") * 3.0
        s["logits"][:, 5::97] = -math.inf  # tokens that are not allowed here
        return s
    n, d, v = case["seqs"], case["draft"], case["n"]
    logits = torch.randn(n, d + 1, v, generator=g, device="cuda") * 3.0
    s["target"] = torch.softmax(logits, -1)
    draft = torch.softmax(logits[:, :d] + torch.randn(n, d, v, generator=g, device="cuda") * 0.7, -1)
    u = torch.rand(n, d, v, generator=g, device="cuda").clamp_min(1e-20)
    s["tokens"] = torch.argmax(draft / -torch.log(u), -1).to(torch.int32)
    s["draft"] = draft if case["probs"] else None
    s["u_accept"] = torch.rand(n, d, generator=g, device="cuda")
    s["u_sample"] = torch.rand(n, generator=g, device="cuda")
    return s


# ------------------------------------------------------------ plain forms ---

def _rows(s):
    """Sequence and position of each row of new tokens."""
    r = torch.arange(s["rows"], device="cuda")
    seq = torch.searchsorted(s["q_start"].long(), r, right=True) - 1
    pos = s["lens"].long()[seq] - (s["q_start"].long()[seq + 1] - r)
    return seq, pos


def _append(s):
    case = s["case"]
    hq, hkv, page = case["hq"], case["hkv"], case["page"]
    seq, pos = _rows(s)
    x = s["qkv"].view(s["rows"], hq + 2 * hkv, 128)
    qk, v = x[:, :hq + hkv], x[:, hq + hkv:]
    if case["norm"]:
        # the mean square in 64 bits: a code next to a rounding border must not depend on the order of a sum
        r = torch.rsqrt(qk.double().square().mean(-1, keepdim=True) + EPS).float()
        gain = torch.cat([s["q_gain"].expand(hq, 128), s["k_gain"].expand(hkv, 128)])
        qk = qk * r * gain
    c, sn = s["cos"][pos].unsqueeze(1), s["sin"][pos].unsqueeze(1)
    a, b = qk[..., :64], qk[..., 64:]
    qk = torch.cat([a * c - b * sn, b * c + a * sn], -1)
    where = s["table"].long()[seq, pos // page]
    most = torch.tensor(32767.0, device="cuda")  # on the device: a quotient, not a product by its reciprocal
    for w, codes, scale in ((qk[:, hq:], s["k"], s["k_scale"]), (v, s["v"], s["v_scale"])):
        t = w.abs().amax(-1) / most
        z = torch.where(t[..., None] == 0, torch.zeros_like(w), w / t[..., None])
        codes[where, :, pos % page] = torch.round(z).clamp(-32767, 32767).to(torch.int16)
        scale[where, :, pos % page] = t
    return {"q": qk[:, :hq].contiguous(), "k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _attend(s):
    case = s["case"]
    n, hq, hkv, page = case["seqs"], case["hq"], case["hkv"], case["page"]
    L, m, G = s["max_len"], s["max_new"], hq // hkv
    seq, pos = _rows(s)
    at = torch.arange(s["rows"], device="cuda") - s["q_start"].long()[seq]
    q = torch.zeros(n, m, hq, 128, device="cuda")
    q[seq, at] = s["q"]
    p = torch.full((n, m), -1, dtype=torch.long, device="cuda")
    p[seq, at] = pos
    table = s["table"].long()
    k, v = ((c[table].float() * z[table][..., None]).transpose(1, 2).reshape(n, hkv, -1, 128)[:, :, :L]
            for c, z in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])))
    q = q.view(n, m, hkv, G, 128).transpose(1, 2).reshape(n, hkv, m * G, 128)
    t = torch.matmul(q, k.transpose(2, 3)).mul_(SCALE)
    hidden = (torch.arange(L, device="cuda") > p[:, :, None]).repeat_interleave(G, 1)
    t.masked_fill_(hidden[:, None], -math.inf)
    t.sub_(t.amax(-1, keepdim=True).clamp_min(-3e38)).exp_()
    o = torch.matmul(t, v) / t.sum(-1, keepdim=True).clamp_min(1e-30)
    return o.view(n, hkv, m, G, 128).transpose(1, 2).reshape(n, m, hq, 128)[seq, at]


def _softmax(x, temp):
    t = x * (1.0 / temp)
    e = torch.exp(t - t.amax(-1, keepdim=True))
    return e / e.sum(-1, keepdim=True)


def _verify(s):
    case = s["case"]
    n, d = case["seqs"], case["draft"]
    p, x = s["target"], s["tokens"].long()
    rows = torch.arange(n, device="cuda")
    px = p[:, :d].gather(2, x[..., None])[..., 0].double()
    qx = s["draft"].gather(2, x[..., None])[..., 0].double() if case["probs"] else torch.ones_like(px)
    ok = s["u_accept"].double() * qx < px
    k = ok.long().cumprod(1).sum(1)
    w = p[rows, k].double()  # the weights and their running sums in 64 bits: a draw may fall next to a border
    if case["probs"]:
        low = torch.where((k < d)[:, None], s["draft"][rows, k.clamp_max(d - 1)].double(), torch.zeros_like(w))
        w = (w - low).clamp_min(0)
    else:
        i = x.gather(1, k.clamp_max(d - 1)[:, None])
        w.scatter_(1, i, torch.where((k < d)[:, None], torch.zeros_like(px[:, :1]), w.gather(1, i)))
    c = w.cumsum(1)
    hit = (c > s["u_sample"].double()[:, None] * c[:, -1:]) & (w > 0)
    new = hit.to(torch.uint8).argmax(1)
    place = torch.arange(d + 1, device="cuda")[None]
    tokens = torch.cat([x, x[:, :1]], 1)
    tokens = torch.where(place < k[:, None], tokens, torch.where(place == k[:, None], new[:, None], torch.full_like(tokens, -1)))
    return {"tokens": tokens.to(torch.int32), "accepted": k.to(torch.int32)}


def _own(s):
    from invariant_numerics_b200 import invnum as inv
    case = s["case"]
    op = case["op"]
    if op == "append":
        cache = inv.PagedKVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        q = inv.kv_append_paged(s["qkv"], cache, s["table"], s["q_start"], s["lens"], s["cos"], s["sin"],
                                q_gain=s["q_gain"], k_gain=s["k_gain"], eps=EPS)
        return {"q": q, "k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    if op == "attend":
        cache = inv.PagedKVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        return inv.attn_paged(s["q"], cache, s["table"], s["q_start"], s["lens"], SCALE, max_q_bound=s["max_new"],
                              max_len_bound=s["max_len"])
    if op == "softmax":
        return inv.softmax_rows(s["logits"], 1.0 / case["temp"])
    tokens, accepted = inv.spec_verify(s["target"], s["draft"], s["tokens"], s["u_accept"], s["u_sample"])
    return {"tokens": tokens, "accepted": accepted}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "append":
        return _append(state)
    if op == "attend":
        return _attend(state)
    if op == "softmax":
        return _softmax(state["logits"], state["case"]["temp"])
    return _verify(state)


# -------------------------------------------------------------------- work ---

def work(case):
    op = case["op"]
    if op in ("append", "attend"):
        lens, news = _lens(case)
        hq, hkv, rows = case["hq"], case["hkv"], sum(news)
        table = 4 * sum(-(-l // case["page"]) for l in lens) + 8 * case["seqs"]
        if op == "append":
            new = rows * ((hq + 2 * hkv) * 512 + hq * 512 + 2 * hkv * 260 + 512)
            return {"bytes": new + 4 * rows + 8 * case["seqs"], "flops": rows * (hq + 2 * hkv) * 128 * 6}
        seen = sum(l * k - k * (k - 1) // 2 for l, k in zip(lens, news))
        return {"bytes": sum(lens) * hkv * 520 + rows * hq * 1024 + table, "flops": 4 * 128 * hq * seen}
    if op == "softmax":
        return {"bytes": 8 * case["rows"] * case["n"], "flops": 5 * case["rows"] * case["n"]}
    read = 8 if case["probs"] else 4
    return {"bytes": case["seqs"] * (case["n"] * read + case["draft"] * 20 + 16), "flops": 4 * case["seqs"] * case["n"]}


# ------------------------------------------------------------------- exact ---

def _exact_append(s):
    case = s["case"]
    hq, hkv, page = case["hq"], case["hkv"], case["page"]
    q_out = torch.empty(s["rows"], hq, 128, dtype=torch.float64, device="cuda")
    k_scale, v_scale = s["k_scale"].double(), s["v_scale"].double()
    start, lens = s["q_start"].tolist(), s["lens"].tolist()
    for i, length in enumerate(lens):
        x = s["qkv"][start[i]:start[i + 1]].double().view(-1, hq + 2 * hkv, 128)
        m = x.shape[0]
        p = torch.arange(length - m, length, device="cuda")
        c, sn = s["cos"][p].double()[:, None], s["sin"][p].double()[:, None]

        def turned(y, gain):
            if gain is not None:
                y = y / (y.pow(2).sum(-1, keepdim=True) / 128 + EPS).sqrt() * gain.double()
            lo, hi = y.chunk(2, -1)
            return torch.cat((lo * c - hi * sn, hi * c + lo * sn), -1)

        q_out[start[i]:start[i + 1]] = turned(x[:, :hq], s["q_gain"])
        where, off = s["table"][i].long()[p // page], p % page
        k_scale[where, :, off] = turned(x[:, hq:hq + hkv], s["k_gain"]).abs().amax(-1) / 32767
        v_scale[where, :, off] = x[:, hq + hkv:].abs().amax(-1) / 32767
    return {"q": q_out, "k": None, "v": None, "k_scale": k_scale, "v_scale": v_scale}


def _exact_attend(s):
    case = s["case"]
    hq, hkv = case["hq"], case["hkv"]
    G = hq // hkv
    out = torch.empty(s["rows"], hq, 128, dtype=torch.float64, device="cuda")
    start, lens = s["q_start"].tolist(), s["lens"].tolist()
    for i, length in enumerate(lens):
        pages = s["table"][i, :-(-length // case["page"])].long()
        m = start[i + 1] - start[i]
        first = length - m
        for h in range(hkv):
            k = (s["k"][pages, h].double() * s["k_scale"][pages, h].double()[..., None]).flatten(0, 1)[:length]
            v = (s["v"][pages, h].double() * s["v_scale"][pages, h].double()[..., None]).flatten(0, 1)[:length]
            for a in range(0, m, 1024):
                b = min(m, a + 1024)
                e = first + b  # no row of this part sees a later key
                q = s["q"][start[i] + a:start[i] + b, h * G:(h + 1) * G].double()
                t = torch.einsum("rgd,kd->rgk", q, k[:e]) * SCALE
                late = torch.arange(e, device="cuda")[None] > first + torch.arange(a, b, device="cuda")[:, None]
                w = torch.softmax(t.masked_fill(late[:, None], -math.inf), -1)
                out[start[i] + a:start[i] + b, h * G:(h + 1) * G] = torch.einsum("rgk,kd->rgd", w, v[:e])
    return out


def _exact_verify(s):
    case = s["case"]
    d = case["draft"]
    tokens = torch.full((case["seqs"], d + 1), -1, dtype=torch.int32)
    accepted = torch.zeros(case["seqs"], dtype=torch.int32)
    drafted, u = s["tokens"].tolist(), s["u_accept"].tolist()
    for i in range(case["seqs"]):
        k = 0
        while k < d:
            x = drafted[i][k]
            if not u[i][k] * (float(s["draft"][i, k, x]) if case["probs"] else 1.0) < float(s["target"][i, k, x]):
                break
            tokens[i, k] = x
            k += 1
        left = s["target"][i, k].double().cpu()
        if k < d and case["probs"]:
            left = torch.relu(left - s["draft"][i, k].double().cpu())
        elif k < d:
            left[drafted[i][k]] = 0.0
        sums = left.cumsum(0)
        tokens[i, k] = torch.searchsorted(sums, float(s["u_sample"][i]) * sums[-1], right=True)
        accepted[i] = k
    return {"tokens": tokens, "accepted": accepted}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    if case["op"] == "attend":
        return _exact_attend(s)
    if case["op"] == "softmax":
        return torch.softmax(s["logits"].double() / case["temp"], -1)
    return _exact_verify(s)
