"""Cases and plain forms of the paged key-value cache operators.

Three operators keep the keys and values of sequences that grow and attend them
from one new token at a time:

    append  sa_cache_append: QK-norm + rotation of new tokens, written into the
            pages of the cache, with the per-page key sums the router reads
    decode  sa_attn_decode: attention of one new token over the cached pages,
            every page or the pages of a route
    route   sa_route_pages: the pages one new token attends
    step    the three together, as one layer of one decoding step (its queries
            come rotated from elsewhere)

``run`` computes them in their plain form (elementary torch operations), or
through the framework where ``own`` is true. Sizes are those of the framework's
workloads (56 heads of 128, 38,247 / 112,640 / 8,192 tokens, prefix 951) and
common serving shapes (32 query heads on 8 key-value heads).
"""

import math

import torch

own = False

PAGE = 64
E4M3_MAX = 448.0


def listed():
    return [
        # one user, one new token: the latency of a call
        dict(name="append step, one", op="append", B=1, S=1, H=32, Hkv=8, D=128, fmt="bf16",
             rope="interleaved", norm=False, past=1023, ragged=False),
        # one decoding step of a full batch, 8-bit cache
        dict(name="append step, batch", op="append", B=128, S=1, H=56, Hkv=8, D=128, fmt="fp8",
             rope="half", norm=True, past=8191, ragged=True),
        # the packed release sequence goes into an empty cache
        dict(name="append prompt", op="append", B=1, S=38247, H=56, Hkv=8, D=128, fmt="bf16",
             rope="interleaved", norm=True, past=0, ragged=False),
        # chunks of prompts of unequal length behind cached tokens
        dict(name="append chunks", op="append", B=5, S=2047, H=16, Hkv=16, D=64, fmt="fp8",
             rope="half", norm=False, past=1000, ragged=True),
        # one user, a short context: the latency of a call
        dict(name="decode one", op="decode", B=1, H=32, Hkv=8, D=128, fmt="bf16", past=777,
             ragged=False, budget=0, prefix=0),
        # a serving batch of unequal lengths
        dict(name="decode batch", op="decode", B=64, H=56, Hkv=8, D=128, fmt="bf16", past=8192,
             ragged=True, budget=0, prefix=0),
        # a few very long contexts in 8 bits
        dict(name="decode long", op="decode", B=3, H=56, Hkv=8, D=128, fmt="fp8", past=112640,
             ragged=False, budget=0, prefix=0),
        # one key-value head for all query heads
        dict(name="decode one kv head", op="decode", B=16, H=56, Hkv=1, D=64, fmt="bf16",
             past=38247, ragged=True, budget=0, prefix=0),
        # the routed form: 96 of 598 pages
        dict(name="decode routed", op="decode", B=24, H=56, Hkv=8, D=128, fmt="bf16", past=38247,
             ragged=False, budget=96, prefix=951),
        # the router for one user
        dict(name="route one", op="route", B=1, H=56, Hkv=8, D=128, past=38247, ragged=False,
             budget=96, prefix=951),
        # the router for a batch of long contexts
        dict(name="route batch", op="route", B=32, H=32, Hkv=8, D=128, past=112640, ragged=True,
             budget=256, prefix=951),
        # one layer of a decoding step: append, route, attend
        dict(name="step", op="step", B=48, S=1, H=16, Hkv=16, D=128, fmt="bf16",
             rope="interleaved", norm=True, past=8192, ragged=True, budget=48, prefix=256),
    ]


HEADS = [(32, 8), (56, 8), (16, 16), (56, 1), (40, 10), (24, 4), (8, 2), (5, 5)]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "decode", "decode", "route", "step"])
    H, Hkv = rng.choice(HEADS)
    case = dict(op=op, H=H, Hkv=Hkv, D=rng.choice([64, 128, 128]), ragged=rng.random() < 0.6,
                empty=rng.random() < 0.3)
    if op in ("append", "step"):
        case.update(rope=rng.choice(["interleaved", "half", "none"]), norm=rng.random() < 0.5)
    if op != "route":
        case.update(fmt=rng.choice(["bf16", "fp8"]))
    if op == "append":
        case["S"] = 1 if rng.random() < 0.4 else _log(rng, 2, 32768)
        case["B"] = _log(rng, 1, max(1, min(256, 32768 // case["S"])))
        case["past"] = _log(rng, 1, 8192) - 1
    else:
        if op == "step":
            case["S"] = 1
        case["past"] = _log(rng, 1, 112640)
        # the keys and values of all sequences stay within 1 GB in bf16
        most = (1 << 30) // (case["past"] * Hkv * case["D"] * 4)
        case["B"] = _log(rng, 1, max(1, min(128, most)))
        case["prefix"] = rng.choice([0, 64, 256, 951])
        sparse = op != "decode" or rng.random() < 0.4
        case["budget"] = _log(rng, 1, 512) if sparse else 0
    return case


# ------------------------------------------------------------------ inputs --

def _lengths(case, gen):
    B, past = case["B"], case["past"]
    lens = torch.full((B,), past, dtype=torch.int32)
    if case["ragged"]:
        lens = (past * (0.25 + 0.75 * torch.rand((B,), generator=gen))).ceil().to(torch.int32)
        lens[int(torch.randint(0, B, (1,), generator=gen))] = past
    if case.get("empty") and B > 1:            # a sequence that has cached nothing yet
        lens[int(torch.randint(0, B, (1,), generator=gen))] = 0
    return lens


def _tables(rows, D, device):
    inv = 1e4 ** (-torch.arange(0, D // 2, dtype=torch.float64, device=device) / (D // 2))
    ang = torch.arange(rows, dtype=torch.float64, device=device)[:, None] * inv
    return ang.cos().float(), ang.sin().float()


def prepare(case, seed):
    dev = torch.device("cuda")
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=dev).manual_seed(seed)
    op, B, H, Hkv, D = case["op"], case["B"], case["H"], case["Hkv"], case["D"]

    def randn(*shape, scale=1.0, dtype=torch.bfloat16):
        t = torch.empty(shape, dtype=torch.bfloat16, device=dev)
        return t.normal_(0.0, scale, generator=gen).to(dtype)

    s = {"case": dict(case)}
    lens = _lengths(case, host)
    S = case.get("S", 0)
    new = None
    if S > 1 and case["ragged"]:             # a padded batch: each sequence brings its own part
        new = torch.randint(1, S + 1, (B,), generator=host, dtype=torch.int32)
        new[int(torch.randint(0, B, (1,), generator=host))] = S
    # a pool that every sequence could fill, its pages in no order; entries behind a
    # sequence's last page hold no page
    need = (lens + (S if new is None else new) + PAGE - 1) // PAGE
    max_pages = (case["past"] + S + PAGE - 1) // PAGE
    n_pages = B * max_pages + 3
    perm = torch.randperm(n_pages, generator=host, dtype=torch.int64).to(torch.int32)
    table = torch.full((B, max_pages), -1, dtype=torch.int32)
    used = torch.arange(max_pages)[None, :] < need[:, None]
    table[used] = perm[: int(need.sum())]
    s.update(lens=lens.to(dev), new_lens=None if new is None else new.to(dev), table=table.to(dev))

    if op != "route":
        fp8 = case["fmt"] == "fp8"
        dt = torch.float8_e4m3fn if fp8 else torch.bfloat16
        s["kc"] = randn(n_pages, Hkv, PAGE, D, dtype=dt)
        s["vc"] = randn(n_pages, Hkv, PAGE, D, dtype=dt)
        s["ks"] = s["vs"] = None
        if fp8:                                # calibrated scales of the heads
            s["ks"] = (0.02 + 0.02 * torch.rand((Hkv,), generator=gen, device=dev))
            s["vs"] = (0.02 + 0.02 * torch.rand((Hkv,), generator=gen, device=dev))
            # the codes of unit-variance keys at those scales
            for name, sc in (("kc", "ks"), ("vc", "vs")):
                x = randn(n_pages, Hkv, PAGE, D).float() / s[sc][None, :, None, None]
                s[name] = x.clamp_(-E4M3_MAX, E4M3_MAX).to(dt)
    if op in ("route", "step", "append"):
        s["ksum"] = randn(n_pages, Hkv, D, dtype=torch.float32) * 8.0
        s["ksum"] += randn(n_pages, Hkv, D, scale=0.01, dtype=torch.float32)
    if op in ("append", "step"):
        s["k"], s["v"] = randn(B, S, Hkv, D), randn(B, S, Hkv, D)
        s["q_in"] = s["q_out"] = None
        if op == "append":
            s["q_in"] = randn(B, S, H, D)
            s["q_out"] = torch.empty_like(s["q_in"])
            if new is not None:                # rows behind a sequence's last new token stay
                s["q_out"].zero_()
        s["gq"] = s["gk"] = s["cos"] = s["sin"] = None
        if case["norm"]:
            s["gq"] = 1 + 0.1 * randn(D, dtype=torch.float32)
            s["gk"] = 1 + 0.1 * randn(D, dtype=torch.float32)
        if case["rope"] != "none":
            s["cos"], s["sin"] = _tables(max_pages * PAGE, D, dev)
        s["lens_out"] = torch.zeros_like(s["lens"])
    if op != "append":
        s["q"] = randn(B, 1, H, D, scale=2.0)
        if case["budget"]:
            per_row = min(max_pages, max(case["budget"], -(-case["prefix"] // PAGE) + 1))
            s["row_ptr"] = torch.zeros(B * Hkv + 1, dtype=torch.int32, device=dev)
            s["col_idx"] = torch.full((B * Hkv * per_row,), -1, dtype=torch.int32, device=dev)
            s["per_row"] = per_row
        if op == "decode" and case["budget"]:  # a route as the router leaves it
            _some_route(s, gen)
        if op != "route":
            s["o"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty((B, H, 1), dtype=torch.float32, device=dev)
    return s


def _some_route(s, gen):
    """Random pages, the forced ones among them, ascending."""
    c, dev = s["case"], s["lens"].device
    B, Hkv, n = c["B"], c["Hkv"], s["table"].shape[1]
    score = torch.rand((B, Hkv, n), generator=gen, device=dev, dtype=torch.float64)
    _emit_route(s, score, s["lens"])


# -------------------------------------------------------------- plain forms --

def _rotate(x, cos, sin, layout):
    """x [..., D] with the tables [..., D/2] of its positions."""
    if layout == "interleaved":
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
    a, b = x.chunk(2, dim=-1)
    return torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)


def _norm_rotate(x, gamma, s, pos):
    c = s["case"]
    x = x.float()
    if c["norm"]:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * gamma
    if c["rope"] != "none":
        x = _rotate(x, s["cos"][pos][:, :, None], s["sin"][pos][:, :, None], c["rope"])
    return x


def _store(cache, page, slot, x, scale):
    if cache.dtype == torch.bfloat16:
        x = x.to(torch.bfloat16)
    else:                                      # moved as bytes: torch indexes those everywhere
        x = (x / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(cache.dtype).view(torch.uint8)
        cache = cache.view(torch.uint8)
    cache.permute(0, 2, 1, 3)[page, slot] = x


def _append_plain(s):
    c = s["case"]
    B, S = s["k"].shape[:2]
    step = torch.arange(S, device=s["k"].device)[None, :]
    n = torch.full_like(s["lens"], S) if s["new_lens"] is None else s["new_lens"]
    valid = step < n[:, None]
    pos = s["lens"][:, None] + step
    pos = torch.where(valid, pos, torch.zeros_like(pos)).long()
    page = s["table"].gather(1, pos // PAGE).long()[valid]
    slot = (pos % PAGE)[valid]
    k = _norm_rotate(s["k"], s["gk"], s, pos)[valid]          # [tokens, Hkv, D]
    _store(s["kc"], page, slot, k, s["ks"])
    _store(s["vc"], page, slot, s["v"].float()[valid], s["vs"])
    s["ksum"][page[slot == 0]] = 0.0
    s["ksum"].index_put_((page,), k, accumulate=True)
    if s["q_in"] is not None:
        s["q_out"][valid] = _norm_rotate(s["q_in"], s["gq"], s, pos)[valid].to(torch.bfloat16)
    s["lens_out"].copy_(s["lens"] + n)


def _emit_route(s, score, lens):
    """Keeps the forced pages and those of largest score, and writes the CSR."""
    c = s["case"]
    n = s["table"].shape[1]
    nb = ((lens + PAGE - 1) // PAGE).long()[:, None, None]
    sink = ((lens.clamp(max=c["prefix"]) + PAGE - 1) // PAGE).long()[:, None, None]
    j = torch.arange(n, device=lens.device)[None, None, :]
    inside = j < nb
    forced = inside & ((j < sink) | (j == nb - 1))
    free = (inside & ~forced).expand_as(score)
    want = nb.clamp(max=c["budget"]) - forced.sum(-1, keepdim=True)
    # rank of every free page: largest score first, equal scores by index
    by_score = torch.argsort(score.masked_fill(score.isnan(), -math.inf), dim=-1, descending=True,
                             stable=True)
    behind = torch.argsort((~free).gather(-1, by_score).int(), dim=-1, stable=True)
    order = by_score.gather(-1, behind)
    rank = torch.empty_like(order).scatter_(-1, order, j.expand_as(order).contiguous())
    keep = forced | (free & (rank < want))
    flat = keep.reshape(-1, n)
    s["row_ptr"][1:] = flat.sum(-1).cumsum(0)
    row, col = flat.nonzero(as_tuple=True)
    s["col_idx"][: row.numel()] = col.to(torch.int32)


def _route_plain(s, q, lens):
    c = s["case"]
    B, G = c["B"], c["H"] // c["Hkv"]
    sums = s["ksum"][s["table"].clamp(min=0).long()].double()         # [B, pages, Hkv, D]
    qg = q.reshape(B, c["Hkv"], G, c["D"]).double()
    score = torch.matmul(qg, sums.permute(0, 2, 3, 1)).amax(2)        # [B, Hkv, pages]
    _emit_route(s, score, lens)


def _decode_plain(s, q, lens):
    c = s["case"]
    B, H, Hkv, D = c["B"], c["H"], c["Hkv"], c["D"]
    dev = q.device
    n = s["table"].shape[1]
    if c["budget"]:                            # the routed pages of every row, padded
        beg, end = s["row_ptr"][:-1].long(), s["row_ptr"][1:].long()
        at = beg[:, None] + torch.arange(s["per_row"], device=dev)[None, :]
        there = at < end[:, None]
        j = s["col_idx"][at.clamp(max=s["col_idx"].numel() - 1)].long()
        j = torch.where(there, j, torch.zeros_like(j)).view(B, Hkv, -1)
        there = there.view(B, Hkv, -1)
    else:
        j = torch.arange(n, device=dev).expand(B, Hkv, n)
        there = torch.ones_like(j, dtype=torch.bool)
    page = s["table"].long()[:, None, :].expand(B, Hkv, n).gather(2, j).clamp(min=0)
    head = torch.arange(Hkv, device=dev)[None, :, None]
    tok = j[..., None] * PAGE + torch.arange(PAGE, device=dev)
    seen = (there[..., None] & (tok < lens.long()[:, None, None, None])).flatten(2)[:, :, None]

    def pages_of(cache, scale):
        if cache.dtype == torch.bfloat16:
            return cache[page, head].flatten(2, 3).float()            # [B, Hkv, keys, D]
        x = cache.view(torch.uint8)[page, head].view(cache.dtype).flatten(2, 3).float()
        return x.mul_(scale[None, :, None, None])

    qg = q.reshape(B, Hkv, H // Hkv, D).float()
    logit = torch.matmul(qg, pages_of(s["kc"], s["ks"]).transpose(-1, -2)) * (D ** -0.5)
    logit = logit.masked_fill_(~seen, -math.inf)
    top = logit.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(logit - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, pages_of(s["vc"], s["vs"])) / total.clamp(min=1e-30)
    s["o"].copy_(o.reshape(B, 1, H, D))
    s["lse"].copy_((top + total.log()).reshape(B, H, 1))


# --------------------------------------------------------------------- run --

def _append_own(sa, s):
    c = s["case"]
    sa.sa_cache_append(s["k"], s["v"], s["kc"], s["vc"], s["table"], s["lens"], q=s["q_in"],
                       q_out=s["q_out"], new_lens=s["new_lens"], qk_norm=c["norm"],
                       gamma_q=s["gq"], gamma_k=s["gk"], eps=1e-6, cos=s["cos"], sin=s["sin"],
                       rope="interleaved" if c["rope"] == "none" else c["rope"],
                       k_scale=s["ks"], v_scale=s["vs"], k_sum=s["ksum"], lens_out=s["lens_out"])


def _route_own(sa, s, q, lens):
    c = s["case"]
    if "route_ws" not in s:                    # a program keeps its workspaces
        s["route_ws"] = torch.empty(
            sa.sa_route_pages_workspace_bytes(sa.make_cache_params(
                s["table"], q=q, k_sum=s["ksum"], prefix_len=c["prefix"], budget=c["budget"])),
            dtype=torch.uint8, device=q.device)
    sa.sa_route_pages(q, s["ksum"], s["table"], lens, c["prefix"], c["budget"],
                      row_ptr=s["row_ptr"], col_idx=s["col_idx"], workspace=s["route_ws"])


def _decode_own(sa, s, q, lens):
    if "decode_ws" not in s:
        s["decode_ws"] = torch.empty(
            sa.sa_attn_decode_workspace_bytes(sa.make_cache_params(
                s["table"], q=q, k_cache=s["kc"], v_cache=s["vc"])),
            dtype=torch.uint8, device=q.device)
    sa.sa_attn_decode(q, s["kc"], s["vc"], s["table"], lens, row_ptr=s.get("row_ptr"),
                      col_idx=s.get("col_idx"), k_scale=s["ks"], v_scale=s["vs"], o=s["o"],
                      lse=s["lse"], workspace=s["decode_ws"])


def run(state):
    s, op = state, state["case"]["op"]
    q, lens = s.get("q"), s["lens"]
    if own:
        import block_sparse_attention_sa_gb300 as sa
    if op in ("append", "step"):
        if own:
            _append_own(sa, s)
        else:
            _append_plain(s)
        lens = s["lens_out"]
    if op in ("route", "step"):
        if own:
            _route_own(sa, s, q, lens)
        else:
            _route_plain(s, q, lens)
    if op in ("decode", "step"):
        if own:
            _decode_own(sa, s, q, lens)
        else:
            _decode_plain(s, q, lens)
    names = {"append": ("kc", "vc", "ksum", "q_out", "lens_out"), "route": ("row_ptr", "col_idx"),
             "decode": ("o", "lse"),
             "step": ("kc", "vc", "ksum", "lens_out", "row_ptr", "col_idx", "o", "lse")}
    return {name: s[name] for name in names[op]}


# -------------------------------------------------------------------- work --

def work(case):
    op, B, H, Hkv, D = case["op"], case["B"], case["H"], case["Hkv"], case["D"]
    mean = case["past"] * (0.625 if case["ragged"] else 1.0)        # tokens of a sequence
    kv = 1 if case.get("fmt") == "fp8" else 2
    pages = mean / PAGE
    by = fl = 0.0
    if op in ("append", "step"):
        S = case["S"]
        tokens = B * S * (0.5 if S > 1 and case["ragged"] else 1.0)
        by += tokens * Hkv * D * (4 + 2 * kv)                         # k, v in; caches out
        by += tokens * H * D * 4 * (op == "append")                   # q in and out
        by += tokens * D * 4 * (case["rope"] != "none")
        by += max(B, tokens / PAGE) * Hkv * D * 8
        fl += tokens * (H + Hkv) * D * 8
    if op in ("route", "step"):
        by += B * pages * Hkv * D * 4 + B * H * D * 2
        fl += B * pages * H * D * 2
    if op in ("decode", "step"):
        keys = mean
        if case["budget"]:
            keys = min(mean, PAGE * max(case["budget"], -(-case["prefix"] // PAGE) + 1))
        by += B * keys * Hkv * D * 2 * kv + B * H * D * 4
        fl += B * keys * H * D * 4
    return {"bytes": by, "flops": fl}


# ------------------------------------------------------------------- exact --

def _exact_turn(x, gamma, cos, sin, case):
    x = x.double()
    if case["norm"]:
        x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + 1e-6).sqrt() * gamma.double()
    if case["rope"] == "none":
        return x
    D = x.shape[-1]
    i = torch.arange(D // 2, device=x.device)
    lo, hi = (2 * i, 2 * i + 1) if case["rope"] == "interleaved" else (i, i + D // 2)
    c, s = cos.double()[:, None], sin.double()[:, None]
    y = torch.empty_like(x)
    y[..., lo] = x[..., lo] * c - x[..., hi] * s
    y[..., hi] = x[..., lo] * s + x[..., hi] * c
    return y


def _exact_append(s):
    """Sequence by sequence, page by page."""
    c = s["case"]
    kc, vc, ksum = s["kc"].double(), s["vc"].double(), s["ksum"].double()
    q_out, lens_out = s["q_out"], s["lens"].clone()
    q_out = None if q_out is None else q_out.double()
    lens, new = s["lens"].tolist(), None if s["new_lens"] is None else s["new_lens"].tolist()
    table = s["table"].tolist()
    one = torch.ones(c["Hkv"], dtype=torch.float64, device=kc.device)
    ks, vs = (one if t is None else t.double() for t in (s["ks"], s["vs"]))
    turn = c["rope"] != "none"
    for b in range(c["B"]):
        n, t0 = (c["S"] if new is None else new[b]), lens[b]
        lens_out[b] = t0 + n
        rows = slice(t0, t0 + n)
        cos, sin = (s["cos"][rows], s["sin"][rows]) if turn else (None, None)
        if q_out is not None:
            q_out[b, :n] = _exact_turn(s["q_in"][b, :n], s["gq"], cos, sin, c)
        k, v = _exact_turn(s["k"][b, :n], s["gk"], cos, sin, c), s["v"][b, :n].double()
        t = 0
        while t < n:
            j, slot = divmod(t0 + t, PAGE)
            m = min(PAGE - slot, n - t)
            p = table[b][j]
            for cache, x, sc in ((kc, k, ks), (vc, v, vs)):
                x = x[t:t + m].transpose(0, 1) / sc[:, None, None]
                cache[p, :, slot:slot + m] = x if c["fmt"] == "bf16" else x.clamp(-448, 448)
            ksum[p] = k[t:t + m].sum(0) + (ksum[p] if slot else 0)
            t += m
    got = {"kc": kc, "vc": vc, "ksum": ksum, "lens_out": lens_out}
    return got if q_out is None else dict(got, q_out=q_out)


def _exact_decode(s):
    c = s["case"]
    B, H, Hkv, D, G = c["B"], c["H"], c["Hkv"], c["D"], c["H"] // c["Hkv"]
    dev = s["q"].device
    o = torch.zeros((B, 1, H, D), dtype=torch.float64, device=dev)
    lse = torch.full((B, H, 1), -math.inf, dtype=torch.float64, device=dev)
    rp = s["row_ptr"].tolist() if c["budget"] else None
    for b in range(B):
        n = int(s["lens"][b])
        for g in range(Hkv):
            pages = torch.arange((n + PAGE - 1) // PAGE, device=dev)
            if rp:
                pages = s["col_idx"][rp[b * Hkv + g]:rp[b * Hkv + g + 1]].long()
            if not len(pages):
                continue
            ids = s["table"][b][pages].long()
            live = (pages[:, None] * PAGE + torch.arange(PAGE, device=dev)).flatten() < n
            k, v = (x[:, g][ids] if x.dtype == torch.bfloat16 else
                    x.view(torch.uint8)[:, g][ids].view(x.dtype) for x in (s["kc"], s["vc"]))
            k, v = k.reshape(-1, D).double()[live], v.reshape(-1, D).double()[live]
            if s["ks"] is not None:
                k, v = k * s["ks"][g].double(), v * s["vs"][g].double()
            x = s["q"][b, 0, g * G:(g + 1) * G].double() @ k.T / math.sqrt(D)
            lse[b, g * G:(g + 1) * G, 0] = torch.logsumexp(x, -1)
            o[b, 0, g * G:(g + 1) * G] = torch.softmax(x, -1) @ v
    return {"o": o, "lse": lse}


def exact(case, seed):
    """The operators' definitions in 64 bits. A route is whole numbers, which
    have no nearer value, and a step attends what its own route and its own
    rounded cache say, so those give nothing here; a step's appended state does."""
    if case["op"] == "route":
        return None
    s = prepare(case, seed)
    if case["op"] == "decode":
        return _exact_decode(s)
    got = _exact_append(s)
    if case["op"] == "step":
        got.update(row_ptr=None, col_idx=None, o=None, lse=None)
    return got
