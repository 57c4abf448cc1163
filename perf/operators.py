"""What is measured of the serving operators around the state pool: prompts
and single tokens of a ragged batch (linear attention with a decay per head,
its state held in a pool slot), the selection of beams over beams and
vocabulary, and the reordering of the beams' states in the pool.

``own`` false: the operators in elementary torch operations.  ``own`` true:
the calls of quantized_recurrent_state_mamba_b200.
"""
import math

import torch

own = False

# Byte layout of a pool (include/ssq.h, ssq_layout), as a user's program that
# maps the pool itself would write it: header, then per slot the codes, meta
# and fp regions of every layer, each block rounded up to 256 bytes.
HEADER = 256


def _up(v):
    return (v + 255) // 256 * 256


def _layout(fmt, layers, H, P, N):
    codes = _up(H * P * N) if fmt in ("i8a", "i8s") else 0
    meta = _up(H * P * {"i8a": 8, "i8s": 4}[fmt]) if codes else 0
    elem = {"f32": 4, "bf16": 2}.get(fmt, 0)
    fp = _up(H * P * N * elem)
    meta_off = _up(layers * codes)
    fp_off = _up(meta_off + layers * meta)
    return {"codes": codes, "meta": meta, "fp": fp, "meta_off": meta_off, "fp_off": fp_off,
            "slot": _up(fp_off + layers * fp), "elem": elem}


def _slot_view(pool, L, off, shape, dtype):
    """Layer 0's block of a region of every slot, [slots, *shape], a view of the pool."""
    size = torch.empty((), dtype=dtype).element_size()
    flat = pool.view(dtype)
    strides = [L["slot"] // size]
    for k in range(len(shape)):
        strides.append(math.prod(shape[k + 1:]))
    return flat.as_strided([(pool.numel() - HEADER) // L["slot"], *shape], strides, (HEADER + off) // size)


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _prefill(name, lens, H, P, N, G, fmt, fresh, dtype="bf16"):
    c = {"op": "prefill", "lens": lens, "H": H, "P": P, "N": N, "G": G, "fmt": fmt, "fresh": fresh, "dtype": dtype}
    return dict(c, name=name) if name else c


def _beam(name, batch, beams, vocab, dtype, done):
    c = {"op": "beam", "batch": batch, "beams": beams, "vocab": vocab, "dtype": dtype, "done": done}
    return dict(c, name=name) if name else c


def _reorder(name, batch, beams, layers, H, P, N, fmt):
    c = {"op": "reorder", "batch": batch, "beams": beams, "layers": layers, "H": H, "P": P, "N": N, "fmt": fmt}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one short prompt on the 130M head shape: a user waits for the first token
        _prefill("prompt 384", "384", 24, 64, 128, 1, "bf16", True),
        # the 370M scan workload's shape as prompts: 8 requests of 2048 tokens
        _prefill("prompts 8x2048", "8*2048", 32, 64, 128, 1, "i8a", True),
        # ragged prompts on the 8B head shape (8 groups), a single token and an empty run among them
        _prefill("prompts ragged", "4096,1,777,2049,130,0,3001", 128, 64, 128, 8, "f32", True),
        # one long document
        _prefill("prompt 65536", "65536", 24, 64, 128, 1, "i8a", True),
        # a serving step that decodes most requests and takes pieces of a few prompts
        _prefill("mixed step", "252*1,512,384,512,77", 32, 128, 128, 1, "i8a", False),
        # a pure decode step in 16-bit activations
        _prefill("tokens 256", "256*1", 24, 64, 128, 1, "f32", False, "f16"),
        # one request's beams: latency
        _beam("beams 1x4", 1, 4, 32000, "bf16", False),
        # an odd vocabulary, fp32 logits, some beams finished
        _beam("beams 16x5 odd", 16, 5, 50001, "f32", True),
        # a large batch over a large vocabulary
        _beam("beams 64x8", 64, 8, 131072, "bf16", False),
        # one request's beams follow their parents (130M state, 24 layers)
        _reorder("reorder 1x4", 1, 4, 24, 24, 64, 128, "i8a"),
        # the same for a full batch of 256 slots
        _reorder("reorder 32x8", 32, 8, 24, 24, 64, 128, "i8a"),
        # the serving-scale state in fp32
        _reorder("reorder 8x4 f32", 8, 4, 30, 32, 128, 128, "f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "beam", "reorder"])
    if op == "prefill":
        H, P, N, G = rng.choice([(24, 64, 128, 1), (32, 64, 128, 1), (128, 64, 128, 8), (32, 128, 128, 1),
                                 (6, 40, 64, 2), (10, 64, 64, 2), (5, 24, 128, 5)])
        fmt = rng.choice(["f32", "bf16", "i8a", "i8s"])
        # tokens so that a drawn case costs no more than the largest listed one
        budget = _log_int(rng, 16, 1500000 // H if P <= 64 else 700000 // H)
        lens, left = [], min(budget, 60000)
        many = rng.random() < 0.3
        while left > 0 and len(lens) < (200 if many else 5):
            n = 1 if many and rng.random() < 0.9 else min(left, _log_int(rng, 1, max(2, min(left, 512 if many else 16384))))
            lens.append(n)
            left -= n
        if rng.random() < 0.3:
            lens.insert(rng.randrange(len(lens) + 1), 0)
        return _prefill(None, ",".join(map(str, lens)), H, P, N, G, fmt, rng.random() < 0.5,
                        rng.choice(["bf16", "bf16", "bf16", "f16", "f32"]))
    if op == "beam":
        beams = rng.choice([1, 2, 3, 4, 5, 6, 8, 10, 12, 16])
        vocab = _log_int(rng, 300, 150000)
        batch = _log_int(rng, 1, max(1, min(128, 60000000 // (beams * vocab))))
        return _beam(None, batch, beams, vocab, rng.choice(["bf16", "f16", "f32"]), rng.random() < 0.5)
    layers, H, P, N = rng.choice([(24, 24, 64, 128), (48, 32, 64, 128), (30, 32, 128, 128), (3, 5, 24, 64)])
    fmt = rng.choice(["f32", "bf16", "i8a", "i8s"])
    beams = rng.choice([2, 3, 4, 5, 8, 12, 16])
    slot = _layout(fmt, layers, H, P, N)["slot"]
    return _reorder(None, _log_int(rng, 1, max(1, min(128, 1800000000 // (slot * beams)))), beams, layers, H, P, N, fmt)


def _lens(case):
    out = []
    for part in case["lens"].split(","):
        n, _, v = part.rpartition("*")
        out += [int(v)] * (int(n) if n else 1)
    return out


DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if case["op"] == "prefill":
        H, P, N, G, fmt = (case[k] for k in ("H", "P", "N", "G", "fmt"))
        lens = _lens(case)
        batch, total = len(lens), sum(lens)
        t = DT[case["dtype"]]
        # x, B and C as slices of one fused activation, the way a block's
        # convolution leaves them; distributions of the library's workloads
        w = H * P + 2 * G * N
        xbc = torch.empty(total, w, dtype=t, device="cuda")
        xbc[:, :H * P] = normal(total, H * P)
        xbc[:, H * P:] = 0.25 * normal(total, 2 * G * N)
        s = {"case": case, "lens": lens, "max_len": max(lens),
             "x": xbc[:, :H * P].unflatten(1, (H, P)), "B": xbc[:, H * P:H * P + G * N].unflatten(1, (G, N)),
             "C": xbc[:, H * P + G * N:].unflatten(1, (G, N)),
             "dt": torch.log1p(torch.exp(normal(total, H) - 2.0)),
             "A": -torch.exp(torch.empty(H, device="cuda").uniform_(math.log(0.5), math.log(16.0), generator=g)),
             "D": normal(H), "y": torch.empty(total, H, P, dtype=t, device="cuda"),
             "slots": torch.randperm(batch, generator=g, device="cuda").to(torch.int32),
             "cu": torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)}
        L = _layout(fmt, 1, H, P, N)
        pool = torch.zeros(HEADER + batch * L["slot"], dtype=torch.uint8, device="cuda")
        if not case["fresh"]:
            # stored states: values of order one, in the pool's format
            if L["elem"]:
                _slot_view(pool, L, L["fp_off"], (H, P, N), DT[fmt]).copy_(normal(batch, H, P, N))
            else:
                sym = fmt == "i8s"
                q = (normal(batch, H, P, N) * 40).round().clamp(-127, 127)
                codes = q.to(torch.int8) if sym else (q + 128).to(torch.uint8)
                _slot_view(pool, L, 0, (H, P, N), codes.dtype).copy_(codes)
                m = _slot_view(pool, L, L["meta_off"], (H, P, 1 if sym else 2), torch.float32)
                m[..., 0] = 0.02 + 0.01 * normal(batch, H, P).abs()
                if not sym:
                    m[..., 1] = 128.0
        s["pool"], s["layout"] = pool, L
        s["fresh"] = torch.ones(batch, dtype=torch.uint8, device="cuda") if case["fresh"] else None
        return s
    if case["op"] == "beam":
        b, k, v = case["batch"], case["beams"], case["vocab"]
        s = {"case": case, "logits": (3.0 * normal(b, k, v)).to(DT[case["dtype"]]),
             "scores": -10.0 + normal(b, k), "done": None}
        if case["done"]:
            s["done"] = (torch.rand(b, k, generator=g, device="cuda") < 0.3).to(torch.uint8)
        return s
    b, k = case["batch"], case["beams"]
    slot = _layout(case["fmt"], case["layers"], case["H"], case["P"], case["N"])["slot"]
    pool = torch.zeros(HEADER + b * k * slot, dtype=torch.uint8, device="cuda")
    pool[HEADER:].view(torch.int64).random_(generator=g)
    return {"case": case, "pool": pool, "slot_bytes": slot,
            "slots": torch.randperm(b * k, generator=g, device="cuda").to(torch.int32),
            "parent": torch.randint(0, k, (b, k), generator=g, device="cuda", dtype=torch.int32)}


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

CHUNK = 128


def _stored(s):
    """The pool's states of layer 0 as fp32 [slots, H, P, N]."""
    c, L, pool = s["case"], s["layout"], s["pool"]
    shape = (c["H"], c["P"], c["N"])
    if L["elem"]:
        return _slot_view(pool, L, L["fp_off"], shape, DT[c["fmt"]]).float()
    sym = c["fmt"] == "i8s"
    q = _slot_view(pool, L, 0, shape, torch.int8 if sym else torch.uint8).float()
    m = _slot_view(pool, L, L["meta_off"], (*shape[:2], 1 if sym else 2), torch.float32)
    return (q if sym else q - m[..., 1:]) * m[..., :1]


def _store(s, S, kept):
    """Writes fp32 states [slots, H, P, N] into the pool in its format, but for the slots of `kept`; what the pool then
    stands for."""
    c, L, pool = s["case"], s["layout"], s["pool"]
    shape = (c["H"], c["P"], c["N"])
    if L["elem"]:
        v = _slot_view(pool, L, L["fp_off"], shape, DT[c["fmt"]])
        v.copy_(S)
        return v
    sym = c["fmt"] == "i8s"
    m = _slot_view(pool, L, L["meta_off"], (*shape[:2], 1 if sym else 2), torch.float32)
    lo, hi = S.amin(-1, keepdim=True), S.amax(-1, keepdim=True)
    if sym:
        delta = torch.maximum(-lo, hi) / 127.0
    else:
        delta = (hi - lo) / 255.0
        delta = torch.where(delta == 0, lo.abs(), delta)
    inv = torch.where(delta == 0, 0.0, 1.0 / delta)
    if sym:
        z = torch.zeros_like(lo)
        q = (S * inv).round().clamp(-127, 127)
    else:
        z = (-lo * inv).round() + 0.0
        q = ((S * inv).round() + z).clamp(max=255.0)
    codes = _slot_view(pool, L, 0, shape, torch.int8 if sym else torch.uint8)
    codes.copy_(torch.where(kept, codes, q.to(codes.dtype)))
    m.copy_(torch.where(kept, m, delta if sym else torch.cat([delta, z], -1)))
    # 8-bit codes stand for (q - z)*delta: 16 bits hold them
    return torch.where(kept, S, (q - z) * delta).to(torch.float16)


def _plain_prefill(s):
    c, lens = s["case"], s["cu"][1:] - s["cu"][:-1]
    H, P, N, G = c["H"], c["P"], c["N"], c["G"]
    L = min(CHUNK, s["max_len"])
    batch, nc = lens.numel(), -(-s["max_len"] // L)
    # the runs padded to whole chunks; what is past a run's end is zero
    pos = torch.arange(nc * L, device="cuda")
    live = pos < lens[:, None]
    tok = (s["cu"][:-1, None] + pos).where(live, 0)

    def padded(v):
        v = v[tok].float()
        return torch.where(live.reshape(*live.shape, *[1] * (v.dim() - 2)), v, 0.0).unflatten(1, (nc, L))

    x, B, C, dt = padded(s["x"]), padded(s["B"]), padded(s["C"]), padded(s["dt"])
    cs = (dt * s["A"]).double().cumsum(2)                                # [b, c, l, H]
    last = cs[:, :, -1:]
    B, C = (v.permute(0, 1, 3, 2, 4) for v in (B, C))                    # [b, c, G, l, n]
    x = x.permute(0, 1, 3, 2, 4)                                         # [b, c, H, l, p]
    cs_h = cs.permute(0, 1, 3, 2)                                        # [b, c, H, l]
    lower = torch.ones(L, L, dtype=torch.bool, device="cuda").tril()
    seg = (cs_h[..., :, None] - cs_h[..., None, :]).where(lower, -math.inf).exp().float()
    M = (C @ B.transpose(-1, -2)).repeat_interleave(H // G, 2) * seg * dt.permute(0, 1, 3, 2)[..., None, :]
    del seg
    y = M @ x
    del M
    Bh, Ch = (v.repeat_interleave(H // G, 2) for v in (B, C))
    w = ((last - cs).exp().float() * dt).permute(0, 1, 3, 2)             # [b, c, H, l]
    states = (x * w[..., None]).transpose(-1, -2) @ Bh                   # [b, c, H, p, n]
    # state at the start of each chunk: a product with the decays between chunks
    tot = last[:, :, 0].permute(0, 2, 1)                                 # [b, H, c]
    cum = torch.cat([torch.zeros_like(tot[..., :1]), tot.cumsum(-1)], -1)  # [b, H, c+1]
    E = (cum[..., :, None] - cum[..., None, :]).where(
        torch.ones(nc + 1, nc + 1, dtype=torch.bool, device="cuda").tril(), -math.inf).exp().float()
    stored = _stored(s)
    S0 = torch.zeros_like(stored) if s["fresh"] is not None else stored[s["slots"].long()]
    allS = torch.cat([S0[:, None], states], 1).permute(0, 2, 1, 3, 4).flatten(3)  # [b, H, c+1, p*n]
    inits = (E @ allS).unflatten(3, (P, N))                              # [b, H, c+1, p, n]
    y = y + (Ch @ inits[:, :, :-1].permute(0, 2, 1, 4, 3)) * cs_h.exp().float()[..., None]
    y = y + x * s["D"][:, None, None]
    out = y.permute(0, 1, 3, 2, 4).flatten(1, 2)[live].to(s["y"].dtype)
    # a request without tokens keeps its slot, unless it is fresh
    kept = torch.zeros(batch, 1, 1, 1, dtype=torch.bool, device="cuda")
    kept[s["slots"].long(), 0, 0, 0] = (lens == 0) if s["fresh"] is None else False
    after = torch.empty_like(stored)
    after[s["slots"].long()] = inits[:, :, -1]
    return {"y": out, "state": _store(s, torch.where(kept, stored, after), kept)}


def _plain_beam(s):
    c, logits, scores = s["case"], s["logits"].double(), s["scores"].double()
    b, k, v = logits.shape
    top = logits.amax(-1, keepdim=True)
    val = scores[..., None] + (logits - top - (logits - top).exp().sum(-1, keepdim=True).log())
    if s["done"] is not None:
        # a finished beam has one candidate: token 0 at its own score
        fin = torch.full((v,), -math.inf, dtype=torch.float64, device="cuda")
        fin[0] = 0.0
        val = torch.where(s["done"].bool()[..., None], scores[..., None] + fin, val)
    flat, at = val.flatten(1).sort(dim=1, descending=True, stable=True)
    flat, at = flat[:, :k], at[:, :k]
    none = flat == -math.inf
    return {"score": flat.float(), "parent": torch.where(none, -1, at // v).int(),
            "token": torch.where(none, -1, at % v).int()}


def _plain_reorder(s):
    b, k = s["case"]["batch"], s["case"]["beams"]
    bits = s["pool"][HEADER:].view(torch.int64).view(b * k, -1)
    dst = s["slots"].long().view(b, k)
    bits[dst.flatten()] = bits[dst.gather(1, s["parent"].long()).flatten()]
    # the states' bits: a reordering moves them as they are
    return bits


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def _own(s):
    from quantized_recurrent_state_mamba_b200 import ssq
    c = s["case"]
    if c["op"] == "prefill":
        H, P, N, batch = c["H"], c["P"], c["N"], len(s["lens"])
        if "cfg" not in s:  # the handle and buffers that a user's program keeps
            s["cfg"] = ssq.Config(1, batch, H, P, N, c["G"], c["fmt"])
            s["work"] = ssq.alloc_prefill_workspace(s["cfg"], batch, s["max_len"])
            s["S"] = torch.empty(batch, H, P, N, device="cuda") if c["fmt"] in ("i8a", "i8s") else None
        ssq.ssq_prefill_ragged(s["cfg"], s["pool"], s["slots"], batch, 0, s["cu"], s["max_len"], s["x"], s["B"],
                               s["C"], s["dt"], s["A"], s["D"], s["y"], fresh=s["fresh"], workspace=s["work"])
        if s["S"] is None:
            return {"y": s["y"], "state": _slot_view(s["pool"], s["layout"], s["layout"]["fp_off"], (H, P, N),
                                                     DT[c["fmt"]])}
        ssq.ssq_dequantize_rows(s["cfg"], s["pool"], None, batch, 0, 1, s["S"])
        return {"y": s["y"], "state": s["S"].to(torch.float16)}
    if c["op"] == "beam":
        score, parent, token = ssq.ssq_beam_select(s["logits"], s["scores"], done=s["done"], done_token=0)
        return {"score": score, "parent": parent, "token": token}
    if "cfg" not in s:
        s["cfg"] = ssq.Config(c["layers"], c["batch"] * c["beams"], c["H"], c["P"], c["N"], 1, c["fmt"])
    ssq.ssq_pool_reorder(s["cfg"], s["pool"], s["slots"], s["parent"], 0, c["layers"])
    return s["pool"][HEADER:].view(torch.int64).view(c["batch"] * c["beams"], -1)


def run(s):
    if own:
        return _own(s)
    return {"prefill": _plain_prefill, "beam": _plain_beam, "reorder": _plain_reorder}[s["case"]["op"]](s)


def work(case):
    if case["op"] == "prefill":
        H, P, N, G, fmt = (case[k] for k in ("H", "P", "N", "G", "fmt"))
        lens = _lens(case)
        total, batch = sum(lens), len(lens)
        e = 4 if case["dtype"] == "f32" else 2
        L = _layout(fmt, 1, H, P, N)
        state = H * P * N * (L["elem"] or 1) + L["meta"]
        # inputs and y once; a state is written once, and read once unless the request is fresh
        moved = total * (2 * H * P * e + 2 * G * N * e + 4 * H) + batch * state * (1 if case["fresh"] else 2)
        if fmt in ("i8a", "i8s"):
            moved += batch * H * P * N * 2  # the returned values
        # the recurrence: update and readout, 2 multiply-adds per state entry and token
        return {"bytes": moved, "flops": 4.0 * total * H * P * N}
    if case["op"] == "beam":
        n = case["batch"] * case["beams"] * case["vocab"]
        live = 0.7 if case["done"] else 1.0  # finished beams' logits need not be read
        return {"bytes": live * n * (4 if case["dtype"] == "f32" else 2) + 24 * case["batch"] * case["beams"],
                "flops": 4.0 * live * n}
    b, k = case["batch"], case["beams"]
    slot = _layout(case["fmt"], case["layers"], case["H"], case["P"], case["N"])["slot"]
    # expected over random parents: slots that change, and parents that some other slot takes
    written = k * (1 - 1 / k)
    read = k * (1 - (1 - 1 / k) ** (k - 1))
    return {"bytes": b * slot * (written + read), "flops": 0.0}


# ---------------------------------------------------------------------------
# From the definitions, in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "reorder":
        return None
    s = prepare(case, seed)
    if case["op"] == "beam":
        out = []
        for b in range(case["batch"]):  # one request at a time: log-probabilities, then the largest
            row = s["logits"][b].to(torch.float64)
            lp = s["scores"][b].to(torch.float64)[:, None] + torch.log(torch.exp(row) / torch.exp(row).sum(1, True))
            if s["done"] is not None:
                d = s["done"][b] != 0
                lp[d] = -math.inf
                lp[d, 0] = s["scores"][b][d].to(torch.float64)
            out.append(lp.reshape(-1).topk(case["beams"]).values)
        return {"score": torch.stack(out), "parent": None, "token": None}
    H, P, N, G, fmt = (case[k] for k in ("H", "P", "N", "G", "fmt"))
    lens, f = _lens(case), torch.float64
    sizes = torch.tensor(lens)
    order = torch.argsort(sizes, descending=True)
    start = torch.tensor([0] + lens).cumsum(0)[:-1][order].cuda()
    slots = s["slots"].long()[order.cuda()]
    shape, L, pool = (H, P, N), s["layout"], s["pool"]
    batch = len(lens)
    if case["fresh"]:
        S = torch.zeros(batch, *shape, dtype=f, device="cuda")
    elif L["elem"]:
        S = _slot_view(pool, L, L["fp_off"], shape, DT[fmt])[slots].to(f)
    else:
        q = _slot_view(pool, L, 0, shape, torch.int8 if fmt == "i8s" else torch.uint8)[slots].to(f)
        m = _slot_view(pool, L, L["meta_off"], (H, P, 1 if fmt == "i8s" else 2), torch.float32)[slots].to(f)
        S = (q - (m[..., 1:] if fmt == "i8a" else 0.0)) * m[..., :1]
    old = S.clone() if not case["fresh"] else None
    y = torch.empty(sum(lens), H, P, dtype=f, device="cuda")
    A, D = s["A"], s["D"].to(f)
    group = torch.arange(H, device="cuda") // (H // G)
    counts = [int((sizes > t).sum()) for t in range(max(lens))]
    for t, n in enumerate(counts):  # token by token over the runs that are still going
        i = start[:n] + t
        xt, dt = s["x"][i].to(f), s["dt"][i]
        lam = torch.exp((dt * A).to(f))
        Bt, Ct = s["B"][i].to(f)[:, group], s["C"][i].to(f)[:, group]
        run_ = S[:n]
        run_.mul_(lam[..., None, None]).addcmul_((dt.to(f)[..., None] * xt)[..., None], Bt[:, :, None, :])
        y[i] = torch.matmul(run_, Ct[..., None])[..., 0] + D[:, None] * xt
    if not L["elem"]:
        lo, hi = S.amin(-1, keepdim=True), S.amax(-1, keepdim=True)
        if fmt == "i8s":
            d = torch.maximum(hi, -lo) / 127
            S = torch.where(d == 0, 0.0, torch.round(S / torch.where(d == 0, 1.0, d)).clamp(-127, 127) * d)
        else:
            d = (hi - lo) / 255
            d = torch.where(d == 0, lo.abs(), d)
            safe = torch.where(d == 0, 1.0, d)
            z = torch.round(-lo / safe)
            S = torch.where(d == 0, 0.0, (torch.clamp(torch.round(S / safe) + z, max=255) - z) * d)
        if old is not None:
            idle = (sizes[order] == 0).cuda()
            S[idle] = old[idle]
    out = torch.empty_like(S)
    out[slots] = S
    return {"y": y, "state": out}
