"""The serving and norm operators as measured workloads: their cases, their inputs, a plain form of each in
elementary torch operations, and their values in 64 bits from the definitions.

Five operators around the low-bit linear layers: the plan of a paged cache (`hbl_kv_plan`), the write into the
8-bit cache (`hbl_kv_append`), the attention that reads it (`hbl_kv_attention`), and the residual addition with
RMSNorm and the per-token quantizer (`hbl_add_rms_quant`) with its straight-through gradient.

Cached values: a block of tokens and a head share one absmax gamma; a code q of `bits` bits, L = 2^bits - 1, stands
for (2 q - L) gamma / L.  Codes (of the cache and of the quantized activations) are integers by contract, every
rounding on the way to them being fixed, so they are compared as whole numbers, with the scales beside them.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-5
SQRT7 = float(np.float32(math.sqrt(7.0)))


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step's bookkeeping for a batch of running requests
        dict(name="plan_decode", op="plan", B=192, longest=8192, new=1, block=64, width=160),
        # a batch of prompts admitted at once, some continuing a cached prefix
        dict(name="plan_prompts", op="plan", B=37, longest=4096, new=1500, block=16, width=384),
        # one decode step: one new token for each request, blocks partly filled
        dict(name="append_decode", op="append", B=64, longest=4096, new=1, Hkv=8, D=128, block=64, bits=8, dtype="bf16"),
        # prompts of ragged lengths written at once, multi-head layout (32 heads of 128)
        dict(name="append_prompts", op="append", B=6, longest=512, new=2731, Hkv=32, D=128, block=64, bits=8, dtype="bf16"),
        # an ordinary decode batch, ragged lengths, four query heads to a cached one
        dict(name="attend_batch", op="attend", B=64, longest=8192, new=1, Hq=32, Hkv=8, D=128, block=64, bits=8, dtype="bf16"),
        # a few draft tokens to verify for two short requests, in float, every head with a cache of its own: latency
        dict(name="attend_draft_f32", op="attend", B=2, longest=777, new=5, Hq=32, Hkv=32, D=64, block=16, bits=8, dtype="f32"),
        # two long documents being read token by token
        dict(name="attend_long", op="attend", B=2, longest=131072, new=1, Hq=32, Hkv=8, D=128, block=128, bits=8, dtype="bf16"),
        # chunks of prompts over what is cached of them
        dict(name="attend_chunk", op="attend", B=3, longest=8192, new=2048, Hq=32, Hkv=8, D=128, block=64, bits=8, dtype="bf16"),
        # one token's residual join and quantization: latency
        dict(name="norm_token", op="norm", M=1, K=2560, bits=8, dtype="bf16"),
        # a training or prompt batch
        dict(name="norm_batch", op="norm", M=8192, K=4096, bits=8, dtype="bf16"),
        # their gradient: a training batch, and an odd one in float
        dict(name="norm_grad_batch", op="norm_grad", M=8192, K=4096, dtype="bf16"),
        dict(name="norm_grad_odd_f32", op="norm_grad", M=1001, K=2560, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "attend", "attend", "norm", "norm_grad"])
    if op == "plan":
        block, B = rng.choice([16, 32, 64, 128]), _log(rng, 1, 256)
        longest, new = _log(rng, 16, 8192), rng.choice([1, 1, rng.randint(2, 8), _log(rng, 16, 1500)])
        return dict(op=op, B=B, longest=longest, new=new, block=block, width=-(-(longest + new) // block) + rng.randint(0, 40))
    if op == "append":
        heads, D, new = rng.choice([1, 4, 5, 8, 32]), rng.choice([32, 64, 128, 256]), rng.choice([1, rng.randint(2, 9), _log(rng, 16, 2700)])
        most = 60_000_000 // (heads * D * (new + 1))
        return dict(op=op, B=max(1, min(_log(rng, 1, 128), most)), longest=_log(rng, 1, 2048), new=new, Hkv=heads, D=D,
                    block=rng.choice([16, 32, 64, 128]), bits=rng.choice([8, 8, 4, 3]), dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "attend":
        D, (hq, hkv) = rng.choice([64, 128]), rng.choice([(32, 32), (32, 8), (16, 2), (20, 5), (8, 1)])
        new = rng.choice([1, 1, rng.randint(2, 9), _log(rng, 16, 2000)])
        longest = max(new + 1, _log(rng, 64, 32768 if new == 1 else 8192))
        most = min(250_000_000 // (longest * hkv * D), 1_500_000_000 // (new * longest * hq))
        return dict(op=op, B=max(1, min(_log(rng, 1, 64), most)), longest=longest, new=new, Hq=hq, Hkv=hkv, D=D,
                    block=rng.choice([16, 32, 64, 128]), bits=rng.choice([8, 8, 4, 3]), dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]))
    K = 16 * _log(rng, 16, 1024)
    case = dict(op=op, M=max(1, min(_log(rng, 1, 8192), 33_000_000 // K)), K=K, dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "norm":
        case["bits"] = rng.choice([8, 8, 4])
    return case


def _requests(case):
    """Cached and new token counts of each request: fixed by the case, ragged, the first as long as any."""
    B, longest, new = case["B"], case["longest"], case["new"]
    r = np.random.RandomState([B, longest, new, 11])
    added = np.maximum(1, np.rint(new * r.uniform(0.55, 1.0, B))).astype(np.int64) if new > 1 else np.ones(B, np.int64)
    added[0] = new
    total = np.rint(longest * r.uniform(0.02, 1.0, B)).astype(np.int64)
    total[0] = longest
    if case["op"] == "attend":
        cached = np.maximum(0, total - added)
    else:
        cached = total if case["op"] == "plan" and new == 1 else total // 2
    return cached, added


# ------------------------------------------------------------------ inputs

def _dtype(case):
    return torch.float32 if case.get("dtype") == "f32" else torch.bfloat16


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(1_000_003 * (seed % 1_000_000) + 17)


def _normal(shape, g, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _i32(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()


def _paged(case, g):
    """Pages for the requests of a case in a shuffled order, a few pages to spare: table, row offsets, lengths."""
    cached, added = _requests(case)
    total, block = cached + added, case["block"]
    pages = -(-total // block)
    num = int(pages.sum()) + 5
    order = torch.randperm(num, generator=g, device="cuda").to(torch.int32)
    width = int(pages.max()) + 2
    start = np.concatenate([[0], np.cumsum(pages)])
    j = np.arange(width)
    at = torch.as_tensor(np.where(j[None] < pages[:, None], start[:-1, None] + j[None], 0)).cuda()
    used = torch.as_tensor(j[None] < pages[:, None]).cuda()
    table = torch.where(used, order[at], torch.full_like(at, -1, dtype=torch.int32))
    rows = np.concatenate([[0], np.cumsum(added)])
    return dict(table=table.contiguous(), row_start=_i32(rows), total=_i32(total), num_blocks=num, T=int(rows[-1]),
                cached=cached, added=added)


def _levels(bits):
    return float(2 ** bits - 1)


def _code(x, gamma, bits):
    """Codes of float32 values under an absmax, each operation rounded once to float32, ties to even."""
    L = _levels(bits)
    r = torch.full_like(gamma, L) / (2.0 * (gamma + EPS))
    return torch.clamp(torch.round(x * r + 0.5 * L), 0, L)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    if op == "plan":
        cached, added = _requests(case)
        block, width = case["block"], case["width"]
        had, want = -(-cached // block), -(-(cached + added) // block)
        num = int(want.sum()) + 64
        order = torch.randperm(num, generator=g, device="cuda").to(torch.int32)
        owned = int(had.sum())
        start = np.concatenate([[0], np.cumsum(had)])
        j = np.arange(width)
        at = torch.as_tensor(np.where(j[None] < had[:, None], start[:-1, None] + j[None], 0)).cuda()
        table = torch.where(torch.as_tensor(j[None] < had[:, None]).cuda(), order[at], torch.full_like(at, -1, dtype=torch.int32))
        T = int(added.sum()) + 8            # a batch padded to a fixed number of rows
        new = lambda n: torch.empty((n,), dtype=torch.int32, device="cuda")  # noqa: E731
        return dict(case=case, cached=_i32(cached), added=_i32(added), free=order[owned:].contiguous(), taken=_i32([3]),
                    table=table.contiguous(), T=T,
                    outs=dict(total=new(case["B"]), row_start=new(case["B"] + 1), slots=new(T), positions=new(T), taken_out=new(1)))
    if op in ("append", "attend"):
        p = _paged(case, g)
        H, D, block, n, bits = case["Hkv"], case["D"], case["block"], p["num_blocks"], case["bits"]
        # cached values: heads of different size, a few large channels in K
        chan = 1.0 + 6.0 * (torch.rand((H, 1, D), generator=g, device="cuda") < 0.03)
        k_codes = torch.empty((n, H, block, D), dtype=torch.uint8, device="cuda")
        v_codes = torch.empty_like(k_codes)
        k_scales = torch.empty((n, H), device="cuda")
        v_scales = torch.empty((n, H), device="cuda")
        for codes, scales, ch in ((k_codes, k_scales, chan), (v_codes, v_scales, 0.5)):
            for i in range(0, n, 512):
                x = _normal((min(512, n - i), H, block, D), g) * ch
                gamma = x.abs().amax(dim=(2, 3), keepdim=True)
                codes[i:i + 512] = _code(x, gamma, bits).to(torch.uint8)
                scales[i:i + 512] = gamma[:, :, 0, 0]
        st = dict(case=case, k_codes=k_codes, k_scales=k_scales, v_codes=v_codes, v_scales=v_scales, **p)
        T = p["T"]
        if op == "attend":
            # q as the first columns of a fused projection's rows
            hq = case["Hq"]
            fused = _normal((T, (hq + 2 * H) * D), g, _dtype(case))
            st["q"] = fused[:, :hq * D].unflatten(1, (hq, D))
            st["o"] = torch.empty((T, hq, D), dtype=_dtype(case), device="cuda")
            return st
        fused = _normal((T, 2 * H * D), g, _dtype(case))
        st["k"], st["v"] = fused[:, :H * D].unflatten(1, (H, D)), fused[:, H * D:].unflatten(1, (H, D))
        req = np.repeat(np.arange(case["B"]), p["added"])
        pos = np.concatenate([c + np.arange(a) for c, a in zip(p["cached"], p["added"])])
        req, pos = torch.as_tensor(req).cuda(), torch.as_tensor(pos).cuda()
        st["slots"] = (p["table"][req, pos // block] * block + (pos % block).to(torch.int32)).to(torch.int32)
        return st
    M, K, dt = case["M"], case["K"], _dtype(case)
    loud = 1.0 + 20.0 * (torch.rand((K,), generator=g, device="cuda") < 0.005)
    x, r = _normal((M, K), g).mul_(loud).to(dt), _normal((M, K), g).mul_(2.0).to(dt)
    gain = 1.0 + 0.2 * _normal((K,), g)
    if op == "norm":
        return dict(case=case, x=x, residual=r, gain=gain, h=torch.empty_like(x), codes=torch.empty((M, K), dtype=torch.int8, device="cuda"),
                    scales=torch.empty((M,), device="cuda"))
    return dict(case=case, h=x, g_t=r.mul_(0.01), gain=gain, g_h=_normal((M, K), g).mul_(0.01).to(dt), g_x=torch.empty_like(x),
                g_gain=torch.empty((K,), device="cuda"))


# ------------------------------------------------------------------ the framework's calls

def _own(s):
    import ternary_gemm_b200 as hbl
    c = s["case"]
    if c["op"] == "plan":
        o = s["outs"]
        hbl.hbl_kv_plan(s["cached"], s["added"], s["free"], s["taken"], s["table"], c["block"], s["T"], **o)
        return s["table"], o["total"], o["row_start"], o["slots"], o["positions"], o["taken_out"]
    if c["op"] == "append":
        hbl.hbl_kv_append(s["k"], s["v"], s["slots"], s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], c["bits"])
        return s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"]
    if c["op"] == "attend":
        if "workspace" not in s:
            n = hbl.hbl_kv_attention_workspace_bytes(s["T"], c["Hq"], c["Hkv"], c["D"], c["B"])
            s["workspace"] = torch.empty((n,), dtype=torch.uint8, device="cuda")
        return hbl.hbl_kv_attention(s["q"], s["row_start"], s["total"], s["table"], s["k_codes"], s["k_scales"], s["v_codes"],
                                    s["v_scales"], c["bits"], o=s["o"], workspace=s["workspace"])
    if c["op"] == "norm":
        return hbl.hbl_add_rms_quant(s["x"], c["bits"], residual=s["residual"], gain=s["gain"], h=s["h"], codes=s["codes"], scales=s["scales"])
    if "workspace" not in s:
        n = hbl.hbl_add_rms_quant_backward_workspace_bytes(c["M"], c["K"])
        s["workspace"] = torch.empty((n,), dtype=torch.uint8, device="cuda")
    return hbl.hbl_add_rms_quant_backward(s["h"], s["g_t"], gain=s["gain"], g_h=s["g_h"], g_x=s["g_x"], g_gain=s["g_gain"],
                                          workspace=s["workspace"])


# ------------------------------------------------------------------ the plain forms

def _plain_plan(s):
    c = s["case"]
    block, width, T = c["block"], c["width"], s["T"]
    cached, added, free, table = s["cached"].long(), s["added"].long(), s["free"], s["table"]
    total = cached + added
    rows = torch.cat([torch.zeros_like(added[:1]), torch.cumsum(added, 0)]).clamp(max=T)
    had = ((cached + block - 1) // block).clamp(max=width)
    need = ((total + block - 1) // block).clamp(max=width) - had
    ends = torch.cumsum(need, 0)
    first = s["taken"].long() + ends - need
    j = torch.arange(width, device="cuda")[None]
    fresh = (j >= had[:, None]) & (j < (had + need)[:, None])
    at = first[:, None] + j - had[:, None]
    page = torch.where(at < free.numel(), free[at.clamp(0, free.numel() - 1)], torch.full_like(at, -1, dtype=torch.int32))
    table.copy_(torch.where(fresh, page, table))
    t = torch.arange(T, device="cuda")
    live = t < rows[-1]
    req = torch.searchsorted(rows[1:], t, right=True).clamp(max=c["B"] - 1)
    pos = cached[req] + t - rows[req]
    col = pos // block
    page = table[req, col.clamp(max=width - 1)].long()
    good = live & (col < width) & (page >= 0)
    slots = torch.where(good, page * block + pos % block, torch.full_like(pos, -1))
    pos = torch.where(live, pos, torch.full_like(pos, -1))
    i = torch.int32
    return table, total.to(i), rows.to(i), slots.to(i), pos.to(i), (s["taken"].long() + ends[-1]).to(i)


def _plain_append_one(x, slots, codes, scales, bits):
    n, H, block, D = codes.shape
    L = _levels(bits)
    slots = slots.long()
    page, off = slots // block, slots % block
    x = x.float()
    # the first of the rows written to a page, and how many of its tokens came before
    before = torch.full((n,), block, dtype=torch.long, device="cuda").scatter_reduce(0, page, off, "amin")
    old = torch.where((before > 0)[:, None], scales, torch.zeros_like(scales))
    top = torch.zeros_like(scales).index_reduce(0, page, x.abs().amax(-1), "amax")
    touched = (before < block)[:, None]
    gamma = torch.where(touched, torch.maximum(old, top), scales)
    grown = (touched & (before > 0)[:, None] & (gamma > scales)).nonzero()
    held = codes[grown[:, 0], grown[:, 1]].float()
    # gamma / L rounded once: torch divides a CUDA tensor by a number as a product with the rounded reciprocal
    gone = scales[grown[:, 0], grown[:, 1]]
    value = (2.0 * held - L) * (gone / torch.full_like(gone, L))[:, None, None]
    again = _code(value, gamma[grown[:, 0], grown[:, 1]][:, None, None], bits).to(torch.uint8)
    early = (torch.arange(block, device="cuda")[None] < before[grown[:, 0]][:, None])[:, :, None]
    codes[grown[:, 0], grown[:, 1]] = torch.where(early, again, codes[grown[:, 0], grown[:, 1]])
    codes[page, :, off] = _code(x, gamma[page][:, :, None], bits).to(torch.uint8)
    scales.copy_(gamma)


def _plain_attend(s):
    c = s["case"]
    B, Hq, H, D, block = c["B"], c["Hq"], c["Hkv"], c["D"], c["block"]
    L = _levels(c["bits"])
    T, width = s["T"], s["table"].shape[1]
    rows, total = s["row_start"].long(), s["total"].long()
    added = rows[1:] - rows[:-1]
    most = int(s["added"].max())
    pages = s["table"].clamp(min=0).long()
    # [B, H, keys, D] in float32, and the queries padded to the longest chunk
    k = ((2.0 * s["k_codes"][pages].float() - L) * (s["k_scales"][pages] / L)[..., None, None]).transpose(1, 2).reshape(B, H, width * block, D)
    i = torch.arange(most, device="cuda")[None]
    live = i < added[:, None]
    at = (rows[:-1, None] + i).clamp(max=T - 1)
    q = s["q"][at].float().view(B, most, H, Hq // H, D).permute(0, 2, 3, 1, 4).reshape(B, H, (Hq // H) * most, D)
    w = torch.matmul(q, k.transpose(-1, -2)).mul_(1.0 / math.sqrt(D))
    del k
    pos = total[:, None] - added[:, None] + i
    seen = torch.arange(width * block, device="cuda")[None, None] <= pos[:, :, None]
    w = w.view(B, H, Hq // H, most, width * block).masked_fill_(~seen[:, None, None], -math.inf)
    w = w.sub_(w.amax(-1, keepdim=True)).exp_()
    w = w.div_(w.sum(-1, keepdim=True)).view(B, H, (Hq // H) * most, width * block)
    v = ((2.0 * s["v_codes"][pages].float() - L) * (s["v_scales"][pages] / L)[..., None, None]).transpose(1, 2).reshape(B, H, width * block, D)
    o = torch.matmul(w, v).view(B, H, Hq // H, most, D).permute(0, 3, 1, 2, 4).reshape(B, most, Hq, D)
    out = torch.zeros((T, Hq, D), device="cuda")
    out[at[live]] = o[live]
    return out.to(_dtype(c))


def _plain_norm(s):
    c = s["case"]
    h = (s["x"].float() + s["residual"].float()).to(_dtype(c))
    # the statistics decide codes: sums in 64 bits, rounded once
    ms = (h.double().square().sum(-1, keepdim=True) / c["K"]).float()
    t = (h.float() * (1.0 / torch.sqrt(ms + EPS))) * s["gain"]
    if c["bits"] == 8:
        stat, k, lo, hi = t.abs().amax(-1, keepdim=True), 127.0, -128, 127
    else:
        stat, k, lo, hi = (t.double().abs().sum(-1, keepdim=True) / c["K"]).float(), SQRT7, -8, 7
    r = torch.full_like(stat, k) / (stat + EPS)
    q = torch.clamp(torch.round(t.double() * r.double()), lo, hi).to(torch.int8)
    return h, q, (stat / torch.full_like(stat, k))[:, 0]


def _plain_norm_grad(s):
    K = s["case"]["K"]
    h, g_t = s["h"].float(), s["g_t"].float()
    rstd = torch.rsqrt(h.square().sum(-1, keepdim=True) / K + EPS)
    n, g_u = h * rstd, g_t * s["gain"]
    g_x = s["g_h"].float() + rstd * (g_u - n * ((g_u * n).sum(-1, keepdim=True) / K))
    return g_x.to(s["h"].dtype), (g_t * n).double().sum(0).float()


def run(s):
    if own:
        return _own(s)
    c = s["case"]
    if c["op"] == "plan":
        return _plain_plan(s)
    if c["op"] == "append":
        _plain_append_one(s["k"], s["slots"], s["k_codes"], s["k_scales"], c["bits"])
        _plain_append_one(s["v"], s["slots"], s["v_codes"], s["v_scales"], c["bits"])
        return s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"]
    if c["op"] == "attend":
        return _plain_attend(s)
    return _plain_norm(s) if c["op"] == "norm" else _plain_norm_grad(s)


# ------------------------------------------------------------------ work and exact values

def work(case):
    size = 4 if case.get("dtype") == "f32" else 2
    if case["op"] in ("plan", "append", "attend"):
        cached, added = (a.tolist() for a in _requests(case))
        B, T, block = case["B"], sum(added), case["block"]
        total = [c + a for c, a in zip(cached, added)]
        fresh = sum(-(-t // block) + (-c // block) for t, c in zip(total, cached))
        if case["op"] == "plan":
            return {"bytes": 4.0 * (2 * B + fresh + 2 * B + 1 + fresh + 2 * (T + 8)), "flops": 8.0 * (B + T)}
        one = T * case["Hkv"] * case["D"]
        if case["op"] == "append":
            pages = sum(-(-t // block) - c // block for t, c in zip(total, cached))
            return {"bytes": 2.0 * one * (size + 1) + 4.0 * T + 16.0 * pages * case["Hkv"], "flops": 6.0 * one}
        pages = sum(-(-t // block) for t in total)
        keys = sum(a * t - a * (a - 1) // 2 for a, t in zip(added, total))
        q = T * case["Hq"] * case["D"]
        return {"bytes": 2.0 * sum(total) * case["Hkv"] * case["D"] + 8.0 * pages * case["Hkv"] + 4.0 * pages + 2.0 * q * size,
                "flops": 4.0 * keys * case["Hq"] * case["D"]}
    n = float(case["M"] * case["K"])
    if case["op"] == "norm":
        return {"bytes": n * (3 * size + 1) + 4 * case["K"] + 4 * case["M"], "flops": 10 * n}
    return {"bytes": n * 4 * size + 8 * case["K"], "flops": 12 * n}


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "plan":
        return None                      # whole numbers
    if op == "append":
        slots, block = s["slots"].cpu().numpy(), case["block"]
        first = np.flatnonzero(np.r_[True, (np.diff(slots) != 1) | (slots[1:] % block == 0)])
        if len(first) > 4000:
            return None
        scales = []
        for x, old in ((s["k"], s["k_scales"]), (s["v"], s["v_scales"])):
            new = old.double()
            for i, j in zip(first, np.r_[first[1:], len(slots)]):
                page, before = divmod(int(slots[i]), block)
                top = x[i:j].double().abs().amax((0, 2))
                new[page] = torch.maximum(top, new[page]) if before else top
            scales.append(new)
        return (None, scales[0], None, scales[1])
    if op == "attend":
        L, block, scale = 2.0 ** case["bits"] - 1.0, case["block"], case["D"] ** -0.5
        group = case["Hq"] // case["Hkv"]
        out = torch.empty((s["T"], case["Hq"], case["D"]), dtype=torch.float64, device="cuda")
        row = 0
        for b in range(case["B"]):
            n, m = int(s["cached"][b] + s["added"][b]), int(s["added"][b])
            ids = s["table"][b, :-(-n // block)].long()
            for h in range(case["Hkv"]):
                key, val = (((c[ids, h].double() * 2 - L) / L * sc[ids, h].double()[:, None, None]).reshape(-1, case["D"])[:n]
                            for c, sc in ((s["k_codes"], s["k_scales"]), (s["v_codes"], s["v_scales"])))
                q = s["q"][row:row + m, h * group:(h + 1) * group].double()
                score = torch.einsum("mgd,nd->gmn", q, key) * scale
                late = torch.ones((m, n), dtype=torch.bool, device="cuda").triu(n - m + 1)
                score = torch.softmax(score.masked_fill_(late, -math.inf), -1)
                out[row:row + m, h * group:(h + 1) * group] = torch.einsum("gmn,nd->mgd", score, val)
            row += m
        return out
    if op == "norm":
        total = s["x"].double() + s["residual"].double()
        h = total.to(_dtype(case)).double()          # the statistics are those of the h that is handed on
        t = h / (h.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * s["gain"].double()
        return (total, None, t.abs().amax(-1) / 127 if case["bits"] == 8 else t.abs().mean(-1) / math.sqrt(7))
    h, g_t, gain = s["h"].double(), s["g_t"].double(), s["gain"].double()
    sigma = (h.pow(2).mean(-1, keepdim=True) + EPS).sqrt()
    n = h / sigma
    along = (g_t * gain * n).mean(-1, keepdim=True)
    return s["g_h"].double() + (g_t * gain - along * n) / sigma, (g_t * n).sum(0)
