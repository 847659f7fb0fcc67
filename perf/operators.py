"""Cases of the steps around the attention layer: RMS norm (with the residual's addition and FP8 output) and its
gradient, grouped expert routing and its gradient, the attention weight each cached key has received, and the
eviction of cache rows by that weight.

`run` computes one step, in its plain form (elementary torch operations) or, where `own` is true, with the library's
kernels.  `exact` states each operator's definition in 64 bits, sequence by sequence or token by token."""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 128  # columns that share one FP8 scale
D, ROPE = 192, 64  # Q/K head dim, rotated dims


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # a decode step's norm: 64 running requests, one token each; latency counts
        dict(name="norm_T64_H4096", op="norm", T=64, H=4096, residual=True, fp8=False),
        # a prefill's norm before FP8 experts
        dict(name="norm_fp8_T16384_H4096", op="norm", T=16384, H=4096, residual=True, fp8=True),
        # training: a short ragged batch, then a full one
        dict(name="norm_bwd_T509_H2048", op="norm_bwd", T=509, H=2048, dh=True),
        dict(name="norm_bwd_T16384_H4096", op="norm_bwd", T=16384, H=4096, dh=True),
        # a speculative step's routing (64 requests x 8 draft tokens, one short), softmax scores without groups
        dict(name="route_T511_E256_softmax", op="route", T=511, E=256, groups=1, top_groups=1, k=8, softmax=True, normalize=True, bias=False),
        # the long-context batch of the router benchmark, sigmoid scores with a balance bias, 4 of 8 groups
        dict(name="route_T262144_E256_g8", op="route", T=262144, E=256, groups=8, top_groups=4, k=8, softmax=False, normalize=True, bias=True),
        # the router's gradient: weights that were not renormalised (dense in the experts), and the usual ones
        dict(name="route_bwd_T4099_E128_softmax", op="route_bwd", T=4099, E=128, k=6, softmax=True, normalize=False),
        dict(name="route_bwd_T65536_E256", op="route_bwd", T=65536, E=256, k=8, softmax=False, normalize=True),
        # KV-cache step of the global layer: 64 requests, 8 new tokens each, contexts of 1024 to 8192
        dict(name="weights_B64_q8_kv8192", op="weights", B=64, q_len=8, kv_lo=1024, kv_hi=8192, hq=64, hkv=4, window=-1, base=1e7, prev=True),
        # a chunk of a prompt against what the cache holds of it
        dict(name="weights_B1_q300_kv5000", op="weights", B=1, q_len=300, kv_lo=5000, kv_hi=5000, hq=64, hkv=4, window=-1, base=1e7, prev=False),
        # eviction down to a budget: the serving batch, and one long request
        dict(name="evict_B64_kv8192", op="evict", B=64, kv_lo=1024, kv_hi=8192, budget=2048, first=4, recent=256),
        dict(name="evict_B1_kv131072", op="evict", B=1, kv_lo=131072, kv_hi=131072, budget=16384, first=4, recent=1024),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "route", "route_bwd", "weights", "evict"])
    if op in ("norm", "norm_bwd"):
        H = 16 * _log(rng, 8, 512)
        T = _log(rng, 1, 16384 * 4096 // H)
        if op == "norm":
            return dict(op=op, T=T, H=H, residual=rng.random() < 0.7, fp8=rng.random() < 0.5)
        return dict(op=op, T=T, H=H, dh=rng.random() < 0.5)
    if op == "route":
        E = rng.choice([16, 32, 60, 64, 72, 128, 160, 192, 256])
        groups = rng.choice([g for g in (1, 1, 2, 4, 8) if E % g == 0])
        top_groups = rng.randint(1, groups)
        k = min(rng.choice([1, 2, 4, 6, 8, 8, 12]), top_groups * (E // groups))
        return dict(op=op, T=_log(rng, 1, 262144), E=E, groups=groups, top_groups=top_groups, k=k, softmax=rng.random() < 0.5, normalize=rng.random() < 0.7, bias=rng.random() < 0.6)
    if op == "route_bwd":
        E = rng.choice([16, 32, 60, 64, 72, 128, 160, 192, 256])
        return dict(op=op, T=_log(rng, 1, 65536), E=E, k=min(E, rng.choice([1, 2, 4, 6, 8, 8, 12])), softmax=rng.random() < 0.5, normalize=rng.random() < 0.6)
    if op == "weights":
        q_len = rng.choice([1, 1, 1, 2, 5, 8, _log(rng, 9, 256)])
        kv_hi = _log(rng, max(16, q_len), 8192)
        most = max(1, min(64, 64 * 8 * 8192 // (max(q_len, 8) * kv_hi)))
        B = _log(rng, 1, most)
        hq, hkv, window, base = rng.choice([(64, 4, -1, 1e7), (64, 4, -1, 1e7), (64, 8, 128, 1e4), (4, 1, -1, 1e4), (6, 2, -1, 1e7)])
        return dict(op=op, B=B, q_len=q_len, kv_lo=min(kv_hi, max(q_len, kv_hi // 8)), kv_hi=kv_hi, hq=hq, hkv=hkv, window=window, base=base, prev=rng.random() < 0.5)
    kv_hi = _log(rng, 16, 131072)
    B = _log(rng, 1, max(1, min(64, 64 * 8192 // kv_hi)))
    budget = _log(rng, 2, kv_hi)
    first = rng.randint(0, min(4, budget // 2))
    return dict(op="evict", B=B, kv_lo=max(1, kv_hi // 8), kv_hi=kv_hi, budget=budget, first=first, recent=rng.randint(0, budget // 2))


# ---------------------------------------------------------------- their inputs
def _lens(case):
    """The contexts' lengths: spread evenly over the case's range."""
    lo, hi, B = case["kv_lo"], case["kv_hi"], case["B"]
    return [hi - (hi - lo) * i // max(1, B - 1) for i in range(B)]


def _lengths(case, gen):
    n = _lens(case)
    return [n[i] for i in torch.randperm(len(n), generator=gen).tolist()]


def _indptr(lens):
    return torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).to(DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(1000 + seed)
    host = torch.Generator().manual_seed(2000 + seed)
    op = case["op"]
    s = dict(case)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=DEV).to(dtype)

    if op in ("norm", "norm_bwd"):
        T, H = case["T"], case["H"]
        s["w"] = (1 + 0.2 * normal(H)).bfloat16()
        s["x"] = normal(T, H, dtype=torch.bfloat16)
        s["r"] = (3 * normal(T, H)).bfloat16() if case.get("residual") else None
        if op == "norm_bwd":
            s["dy"] = normal(T, H, dtype=torch.bfloat16)
            s["dh"] = normal(T, H, dtype=torch.bfloat16) if case["dh"] else None
    elif op in ("route", "route_bwd"):
        T, E = case["T"], case["E"]
        s["logits"] = normal(T, E)
        if op == "route":
            s["bias"] = 0.1 * normal(E) if case["bias"] else None
        else:
            s["ids"] = torch.rand(T, E, generator=g, device=DEV).add_(s["logits"]).argsort(-1, descending=True)[:, : case["k"]].to(torch.int32).contiguous()
            s["dw"] = normal(T, case["k"])
    elif op == "weights":
        lens = _lengths(case, host)
        q = [min(case["q_len"], n) for n in lens]
        total, rows = sum(lens), sum(lens) + 64
        s.update(kv_lens=lens, q_lens=q, max_q=max(q), max_kv=max(lens))
        s["q"] = normal(sum(q), case["hq"], D, dtype=torch.bfloat16)
        s["cache"] = normal(rows, case["hkv"], D, dtype=torch.bfloat16)
        s["indices"] = torch.randperm(rows, generator=g, device=DEV)[:total].to(torch.int32)
        s["indptr"], s["cu_q"] = _indptr(lens), _indptr(q)
        s["prev_w"] = normal(total).abs_() if case["prev"] else None
        scores, _ = _scores(s)  # the layer's normaliser, with a sink on the sliding-window layers
        lse = torch.logsumexp(scores, -1)  # [B, Hq, max_q]
        if case["window"] >= 0:
            lse = torch.logaddexp(lse, normal(case["hq"])[None, :, None])
        b, i = _flat(s["cu_q"], sum(q))
        s["lse"] = lse[b, :, i].t().contiguous()
    else:
        lens = _lengths(case, host)
        total = sum(lens)
        s.update(kv_lens=lens, max_kv=max(lens), kept=sum(min(n, case["budget"]) for n in lens), total=total)
        s["indptr"] = _indptr(lens)
        s["indices"] = torch.randperm(total + 64, generator=g, device=DEV)[:total].to(torch.int32)
        # accumulated weights: heavy-tailed, a tenth of the keys never attended
        s["weights"] = torch.exp(2 * normal(total)) * (torch.rand(total, generator=g, device=DEV) > 0.1)
    return s


# ---------------------------------------------------------------- the plain forms
def _flat(indptr, total):
    """(sequence, position in it) of each entry of a packed list."""
    at = torch.arange(total, device=indptr.device)
    b = torch.searchsorted(indptr[1:].long(), at, right=True)
    return b, at - indptr.long()[b]


def _padded(indptr, most):
    """Entries of each sequence as [B, most] indices into the packed list, and which of them exist."""
    at = torch.arange(most, device=indptr.device)
    n = (indptr[1:] - indptr[:-1]).long()
    return indptr[:-1].long()[:, None] + torch.minimum(at, (n - 1).clamp(min=0)[:, None]), at < n[:, None]


def _rope(x, pos, base):
    """Rotates the first 64 dims of x [B, L, heads, 192] at pos [B, L] or [1, L]: pairs (i, i + 32)."""
    theta = base ** (-2.0 * torch.arange(ROPE // 2, device=x.device, dtype=torch.float64) / ROPE)
    a = pos.double()[..., None, None] * theta
    c, n = torch.cos(a).float(), torch.sin(a).float()
    u, v = x[..., : ROPE // 2], x[..., ROPE // 2 : ROPE]
    return torch.cat([u * c - v * n, v * c + u * n, x[..., ROPE:]], -1)


def _scores(s):
    """Scores [B, Hq, max_q, max_kv], -inf where a query may not look."""
    hq, hkv = s["hq"], s["hkv"]
    rows, has = _padded(s["indptr"], s["max_kv"])
    B, L = rows.shape
    k = _rope(s["cache"][s["indices"].long()[rows].long()].float(), torch.arange(L, device=DEV)[None], s["base"])
    qrows, qhas = _padded(s["cu_q"], s["max_q"])
    kv_len, q_len = has.sum(-1), qhas.sum(-1)
    at = (kv_len - q_len)[:, None] + torch.arange(s["max_q"], device=DEV)
    q = _rope(s["q"][qrows].float(), at, s["base"])
    q = q.view(B, s["max_q"], hkv, hq // hkv, D).permute(0, 2, 3, 1, 4).reshape(B, hkv, -1, D)
    sc = (q @ k.permute(0, 2, 3, 1)).view(B, hq, s["max_q"], L) * (D ** -0.5)
    pos = torch.arange(L, device=DEV)
    may = (pos <= at[..., None]) & has[:, None, :] & qhas[..., None]
    if s["window"] >= 0:
        may = may & (pos >= at[..., None] - s["window"])
    return sc.masked_fill_(~may[:, None], -math.inf), may


def _norm(s):
    h = s["x"] if s["r"] is None else (s["x"].float() + s["r"].float()).bfloat16()
    f = h.float()
    y = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6) * s["w"].float()
    if not s["fp8"]:
        return y.bfloat16(), h
    T, H = y.shape
    blocks = torch.nn.functional.pad(y, (0, -H % BLOCK)).view(T, -1, BLOCK)
    scale = (blocks.abs().amax(-1) / 448.0).clamp_(min=2.0 ** -126)
    codes = (blocks / scale[..., None]).clamp_(-448.0, 448.0).view(T, -1)[:, :H]
    return codes.to(torch.float8_e4m3fn), scale, h


def _norm_bwd(s):
    f, dy = s["x"].float(), s["dy"].float()
    rstd = torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6)
    n = f * rstd
    gy = dy * s["w"].float()
    dx = rstd * (gy - n * (gy * n).mean(-1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return dx.bfloat16(), (dy * n).sum(0, dtype=torch.float64).float()


def _probs(logits, softmax):
    """The experts' scores, in 64 bits: the choice compares values next to one another."""
    x = logits.double()
    if not softmax:
        return torch.where(x >= 0, 1 / (1 + torch.exp(-x.abs())), torch.exp(-x.abs()) / (1 + torch.exp(-x.abs())))
    e = torch.exp(x - x.amax(-1, keepdim=True))
    return e / e.sum(-1, keepdim=True)


def _route(s):
    p = _probs(s["logits"], s["softmax"])
    key = p.float()
    if s["bias"] is not None:
        key = key + s["bias"]
    if s["groups"] > 1:
        by = key.view(key.shape[0], s["groups"], -1)
        two = by.sort(-1, descending=True).values[..., :2]
        order = two.sum(-1).sort(dim=-1, descending=True, stable=True).indices[:, : s["top_groups"]]
        out = torch.ones(by.shape[:2], dtype=torch.bool, device=by.device).scatter_(1, order, False)
        key = by.masked_fill(out[..., None], -math.inf).view_as(key)
    ids = key.sort(dim=-1, descending=True, stable=True).indices[:, : s["k"]]
    w = p.gather(1, ids)
    if s["normalize"]:
        w = w / w.sum(-1, keepdim=True)
    return ids.to(torch.int32), (w * 2.5).float()


def _route_bwd(s):
    p = _probs(s["logits"], s["softmax"])
    ids, dw = s["ids"].long(), s["dw"].double() * 2.5
    c = p.gather(1, ids)
    if s["normalize"]:
        S = c.sum(-1, keepdim=True)
        dc = (dw - (dw * c / S).sum(-1, keepdim=True)) / S
    else:
        dc = dw
    d = torch.zeros_like(p).scatter_(1, ids, dc)
    d = p * (d - (d * p).sum(-1, keepdim=True)) if s["softmax"] else d * p * (1 - p)
    return d.float()


def _weights(s):
    sc, may = _scores(s)
    b, i = _padded(s["cu_q"], s["max_q"])
    lse = s["lse"].t()[b].permute(0, 2, 1)  # [B, Hq, max_q]
    w = torch.exp(sc - lse[..., None]).sum((1, 2))
    b, i = _flat(s["indptr"], s["indices"].numel())
    w = w[b, i]
    return w if s["prev_w"] is None else w + s["prev_w"]


def _evict(s):
    rows, has = _padded(s["indptr"], s["max_kv"])
    n = has.sum(-1, keepdim=True)
    pos = torch.arange(rows.shape[1], device=rows.device)
    always = (pos < s["first"]) | (pos >= n - s["recent"])
    key = s["weights"][rows].masked_fill(always, math.inf).masked_fill(~has, -math.inf)
    order = key.sort(dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(1, order, pos.expand_as(order).contiguous())
    b, i = _flat(s["indptr"], s["total"])
    keep = rank[b, i] < s["budget"]
    kept, freed = s["kept"], s["total"] - s["kept"]
    to = torch.where(keep, keep.cumsum(0) - 1, kept)
    away = torch.where(keep, freed, (~keep).cumsum(0) - 1)
    idx = s["indices"].new_empty(kept + 1).scatter_(0, to, s["indices"])[:kept]
    w = s["weights"].new_empty(kept + 1).scatter_(0, to, s["weights"])[:kept]
    gone = s["indices"].new_empty(freed + 1).scatter_(0, away, s["indices"])[:freed]
    new = torch.nn.functional.pad(n[:, 0].clamp(max=s["budget"]).cumsum(0), (1, 0)).to(torch.int32)
    return idx, w, new, gone


_PLAIN = dict(norm=_norm, norm_bwd=_norm_bwd, route=_route, route_bwd=_route_bwd, weights=_weights, evict=_evict)


def run(s):
    op = s["op"]
    if not own:
        return _PLAIN[op](s)
    from global_attention_moe_b200 import mimo_attn as M
    if op == "norm":
        if s["fp8"]:
            codes, scale, h = M.rms_norm_fp8(s["x"], s["w"], s["r"], eps=1e-6)
            return codes.view(torch.float8_e4m3fn), scale, h
        return M.rms_norm(s["x"], s["w"], s["r"], eps=1e-6)
    if op == "norm_bwd":
        return M.rms_norm_bwd(s["x"], s["w"], s["dy"], s["dh"], eps=1e-6)
    if op in ("route", "route_bwd"):
        score = M.ROUTE_SOFTMAX if s["softmax"] else M.ROUTE_SIGMOID
        if op == "route":
            return M.moe_route_grouped(s["logits"], s["bias"], s["k"], s["groups"], s["top_groups"], score, s["normalize"], 2.5)
        return M.moe_route_bwd(s["logits"], s["ids"], s["dw"], score, s["normalize"], 2.5)
    if op == "weights":
        layer = M.LAYER_SWA if s["window"] >= 0 else M.LAYER_GLOBAL
        return M.decode_key_weights(s["q"], s["cache"], s["indices"], s["indptr"], s["cu_q"], s["lse"], s["max_q"], s["max_kv"], layer, s["window"], s["base"], prev=s["prev_w"])
    idx, w, new, gone = M.kv_evict(s["weights"], s["indices"], s["indptr"], s["max_kv"], s["budget"], keep_first=s["first"], keep_recent=s["recent"])
    return idx[: s["kept"]], w[: s["kept"]], new, gone[: s["total"] - s["kept"]]


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "norm":
        n = case["T"] * case["H"]
        return dict(bytes=n * (2 + (4 if case["residual"] else 0) + (1 + 4 / BLOCK if case["fp8"] else 2)), flops=5 * n)
    if op == "norm_bwd":
        n = case["T"] * case["H"]
        return dict(bytes=n * (8 if case["dh"] else 6), flops=10 * n)
    if op == "route":
        return dict(bytes=case["T"] * (4 * case["E"] + 8 * case["k"]), flops=10 * case["T"] * case["E"])
    if op == "route_bwd":
        dense = case["softmax"] and not case["normalize"]
        return dict(bytes=case["T"] * (4 * case["E"] * (2 if dense else 1) + (8 if dense else 12) * case["k"]), flops=5 * case["T"] * (case["E"] if dense else case["k"]))
    lens = _lens(case)
    total = sum(lens)
    if op == "weights":
        q = [min(case["q_len"], n) for n in lens]
        reach = case["window"] if case["window"] >= 0 else case["kv_hi"]
        seen = sum(min(n, m + reach) for n, m in zip(lens, q))  # keys that some query sees
        pairs = sum(min(n - m + i, reach) + 1 for n, m in zip(lens, q) for i in range(m)) * case["hq"]
        return dict(bytes=seen * (case["hkv"] * D * 2 + 4) + total * (8 if case["prev"] else 4) + sum(q) * case["hq"] * (D * 2 + 4), flops=2 * D * pairs)
    kept = sum(min(n, case["budget"]) for n in lens)
    return dict(bytes=8 * total + 8 * kept + 4 * (total - kept), flops=total)


# ---------------------------------------------------------------- the definitions, in 64 bits
def _exact_norm(s):
    h = s["x"].double() if s["r"] is None else s["x"].double() + s["r"].double()
    f = h.to(torch.bfloat16).double()  # the norm is of the residual stream as it is stored
    y = f / torch.sqrt((f * f).sum(-1, keepdim=True) / f.shape[1] + 1e-6) * s["w"].double()
    if not s["fp8"]:
        return y, h
    parts = y.split(BLOCK, dim=-1)
    scale = torch.stack([(p.abs().max(-1).values / 448.0).clamp(min=2.0 ** -126) for p in parts], -1)
    return torch.cat([p / scale[:, j : j + 1] for j, p in enumerate(parts)], -1), scale, h


def _exact_norm_bwd(s):
    f, dy, w = s["x"].double(), s["dy"].double(), s["w"].double()
    r = 1 / torch.sqrt((f * f).sum(-1, keepdim=True) / f.shape[1] + 1e-6)
    dot = (dy * w * f).sum(-1, keepdim=True)
    dx = r * w * dy - r ** 3 * dot / f.shape[1] * f
    return dx if s["dh"] is None else dx + s["dh"].double(), torch.einsum("th,th,t->h", dy, f, r[:, 0])


def _exact_route(s):
    x = s["logits"].double()
    p = torch.softmax(x, -1) if s["softmax"] else torch.sigmoid(x)
    key = p.float() + (0 if s["bias"] is None else s["bias"])
    T, E = key.shape
    if s["groups"] > 1:
        by = key.view(T, s["groups"], -1)
        top = by.topk(min(2, by.shape[-1]), -1).values
        score = top[..., 0] + top[..., 1] if top.shape[-1] == 2 else top[..., 0]
        ahead = (score[:, :, None] < score[:, None, :]) | ((score[:, :, None] == score[:, None, :]) & torch.ones(s["groups"], s["groups"], dtype=torch.bool, device=DEV).tril(-1))
        key = torch.where((ahead.sum(-1) < s["top_groups"])[..., None], by, torch.full_like(by, -math.inf)).view(T, E)
    w, ids, left = [], [], key.clone()
    for _ in range(s["k"]):  # the largest that is left, the lowest of those that tie
        best = (left == left.max(-1, keepdim=True).values).int().argmax(-1, keepdim=True)
        ids.append(best)
        w.append(p.gather(1, best))
        left.scatter_(1, best, -math.inf)
    ids, w = torch.cat(ids, 1), torch.cat(w, 1)
    return ids.to(torch.int32), 2.5 * (w / w.sum(-1, keepdim=True) if s["normalize"] else w)


def _exact_route_bwd(s):
    x = s["logits"].double().requires_grad_(True)
    with torch.enable_grad():
        p = torch.softmax(x, -1) if s["softmax"] else torch.sigmoid(x)
        c = torch.take_along_dim(p, s["ids"].long(), 1)
        w = 2.5 * (c / c.sum(-1, keepdim=True) if s["normalize"] else c)
        return torch.autograd.grad((w * s["dw"].double()).sum(), x)[0]


def _turn(x, pos, base):
    """The rotation as a product of complex numbers."""
    a = pos.double()[:, None, None] * base ** (-torch.arange(0, ROPE, 2, device=DEV, dtype=torch.float64) / ROPE)
    z = torch.complex(x[..., : ROPE // 2], x[..., ROPE // 2 : ROPE]) * torch.polar(torch.ones_like(a), a)
    return torch.cat([z.real, z.imag, x[..., ROPE:]], -1)


def _exact_weights(s):
    out, k0, q0, group = [], 0, 0, s["hq"] // s["hkv"]
    for n, m in zip(s["kv_lens"], s["q_lens"]):
        pos = torch.arange(n, device=DEV)
        k = _turn(s["cache"][s["indices"][k0 : k0 + n].long()].double(), pos, s["base"])
        q = _turn(s["q"][q0 : q0 + m].double(), pos[n - m :], s["base"])
        w = torch.zeros(n, dtype=torch.float64, device=DEV)
        off = pos[n - m :, None] - pos[None]
        may = (off >= 0) if s["window"] < 0 else (off >= 0) & (off <= s["window"])
        for h in range(s["hq"]):
            p = torch.exp(q[:, h] @ k[:, h // group].t() / math.sqrt(D) - s["lse"][h, q0 : q0 + m].double()[:, None])
            w += (p * may).sum(0)
        out.append(w)
        k0, q0 = k0 + n, q0 + m
    w = torch.cat(out)
    return w if s["prev_w"] is None else w + s["prev_w"].double()


def _exact_evict(s):
    idx, w, gone, new, at = [], [], [], [0], 0
    for n in s["kv_lens"]:
        x, i = s["weights"][at : at + n].double(), s["indices"][at : at + n]
        must = torch.zeros(n, dtype=torch.bool, device=DEV)
        must[: s["first"]] = True
        must[max(0, n - s["recent"]) :] = True
        keep = must.clone()
        rest = (~must).nonzero()[:, 0]
        order = torch.sort(-x[rest], stable=True).indices
        keep[rest[order[: max(0, s["budget"] - int(must.sum()))]]] = True
        idx.append(i[keep])
        w.append(x[keep])
        gone.append(i[~keep])
        new.append(new[-1] + int(keep.sum()))
        at += n
    return torch.cat(idx), torch.cat(w), torch.tensor(new, dtype=torch.int32), torch.cat(gone)


_EXACT = dict(norm=_exact_norm, norm_bwd=_exact_norm_bwd, route=_exact_route, route_bwd=_exact_route_bwd, weights=_exact_weights, evict=_exact_evict)


def exact(case, seed):
    return _EXACT[case["op"]](prepare(case, seed))
