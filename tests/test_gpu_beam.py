"""GPU tests of ssq_beam_select, ssq_pool_reorder and ssq_damp_pool_reorder
(include/ssq_serve.h), and of a beam search that uses them with the prompt and
decode calls.

ssq_beam_select is compared with the definition in 64 bits: tokens and parents
are equal (within a beam the order is that of the logits, exactly; values of
different beams carry the error of their sums of exponentials, about 1e-7, and
lie further apart than that in these inputs), and a score is off by at most
half a step of fp32, 2^-24 of itself, plus the error of the sum of
exponentials: terms rounded 2^-22 (the exponential)
and summed per lane in fp32, n * 2^-24 for n terms of a lane at the worst,
which is 2^-24 * 4096 = 2.5e-4 for the largest row here; the bound is used as
it is, the rounding errors being independent typically leave 1e-7.

A reordering moves bytes: pools are equal bit for bit.
"""
import math

import pytest
import torch

from gpu_harness import require_gpu

pytestmark = pytest.mark.gpu

LANE_TERMS = 4096


def reference(logits, scores, done, done_token, nsel):
    """(values float64, parent, token) from the definition."""
    l = logits.double()
    l = torch.where(l.isnan(), -math.inf, l)
    b, k, v = l.shape
    top = l.amax(-1, keepdim=True)
    ok = top.isfinite()
    shifted = torch.where(ok, l - torch.where(ok, top, 0.0), -math.inf)
    lse = torch.where(ok, top, 0.0) + shifted.exp().sum(-1, keepdim=True).log()
    val = torch.where(ok, scores.double()[..., None] + (l - lse), -math.inf)
    if done is not None:
        fin = torch.full((v,), -math.inf, dtype=torch.float64, device="cuda")
        fin[done_token] = 0.0
        val = torch.where(done.bool()[..., None], scores.double()[..., None] + fin, val)
    val = torch.where(val.isnan(), -math.inf, val).flatten(1)
    val, at = val.sort(dim=1, descending=True, stable=True)
    if val.shape[1] < nsel:
        pad = nsel - val.shape[1]
        val = torch.cat([val, torch.full((b, pad), -math.inf, device="cuda", dtype=val.dtype)], 1)
        at = torch.cat([at, torch.zeros(b, pad, device="cuda", dtype=at.dtype)], 1)
    val, at = val[:, :nsel], at[:, :nsel]
    none = val == -math.inf
    return val, torch.where(none, -1, at // v).int(), torch.where(none, -1, at % v).int()


def check(got, want):
    score, parent, token = got
    val, p, t = want
    assert torch.equal(parent, p) and torch.equal(token, t)
    none = val == -math.inf
    assert torch.equal(score == -math.inf, none)
    err = (score.double() - val)[~none].abs()
    assert torch.all(err <= 2.0 ** -24 * val[~none].abs() + LANE_TERMS * 2.0 ** -24 + 2.0 ** -22)


def draw(b, k, v, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = (3 * torch.randn(b, k, v, generator=g, device="cuda")).to(dtype)
    return logits, torch.randn(b, k, generator=g, device="cuda") - 5


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("shape", [(1, 1, 1, 1), (2, 1, 5, 8), (1, 4, 1000, 4), (3, 5, 4099, 10),
                                   (40, 3, 777, 3), (2, 16, 2048, 32), (1, 17, 3001, 33),
                                   (2, 64, 300, 64), (300, 2, 65, 2), (1, 2, 100003, 4)])
def test_selection(shape, dtype):
    ssq = require_gpu()
    b, k, v, nsel = shape
    logits, scores = draw(b, k, v, dtype, 1)
    check(ssq.ssq_beam_select(logits, scores, nsel=nsel),
          reference(logits, scores, None, 0, nsel))
    done = torch.arange(b * k, device="cuda").view(b, k) % 3 == 1
    done = done.to(torch.uint8)
    check(ssq.ssq_beam_select(logits, scores, done=done, done_token=v // 2, nsel=nsel),
          reference(logits, scores, done, v // 2, nsel))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_ties_go_to_the_lowest_index(dtype):
    """Equal logits within a row, across vectors, warps and blocks, and equal
    rows of equal score."""
    ssq = require_gpu()
    for v in (64, 1000, 50000):
        logits = torch.zeros(2, 4, v, dtype=dtype, device="cuda")
        logits[1, :, ::7] = 1.0
        scores = torch.zeros(2, 4, device="cuda")
        for nsel in (1, 5, 40):
            check(ssq.ssq_beam_select(logits, scores, nsel=nsel),
                  reference(logits, scores, None, 0, nsel))


def test_rising_and_falling_rows():
    """The order of the logits that costs the lists most, and least."""
    ssq = require_gpu()
    up = torch.arange(20000, device="cuda", dtype=torch.float32) / 1000
    logits = torch.stack([up, up.flip(0)])[None].contiguous()
    scores = torch.zeros(1, 2, device="cuda")
    scores[0, 1] = 0.25
    for nsel in (4, 64):
        check(ssq.ssq_beam_select(logits, scores, nsel=nsel),
              reference(logits, scores, None, 0, nsel))


def test_masked_rows():
    """Rows with nothing but -inf or NaN, a row of the type's lowest value, a
    row with +inf, scores that are -inf or NaN, fewer candidates than places."""
    ssq = require_gpu()
    logits, scores = draw(6, 3, 300, torch.float32, 2)
    logits[0] = -math.inf                                 # no candidate at all
    logits[1, 0] = math.nan
    logits[1, 1, 5:] = -math.inf
    logits[2, 1] = torch.finfo(torch.float32).min         # uniform over the row
    logits[2, 2, 7] = math.inf                            # no candidate in this beam
    scores[3, :2] = -math.inf                             # only the last beam is alive
    scores[4, 1] = math.nan
    logits[5, :, 3:] = -math.inf                          # nine candidates
    for nsel in (3, 20):
        got = ssq.ssq_beam_select(logits, scores, nsel=nsel)
        check(got, reference(logits, scores, None, 0, nsel))
    assert (got[1][0] == -1).all() and (got[2][0] == -1).all()
    assert (got[1][5, 9:] == -1).all() and (got[1][5, :9] >= 0).all()
    # the same masks in bf16, in a row that starts off a 16-byte boundary
    wide = torch.full((6, 3, 307), -7.0, dtype=torch.bfloat16, device="cuda")
    wide[..., 3:303] = logits.to(torch.bfloat16)
    view = wide[..., 3:303]
    check(ssq.ssq_beam_select(view, scores, nsel=20), reference(view, scores, None, 0, 20))


def test_all_finished_and_empty_batch():
    ssq = require_gpu()
    logits, scores = draw(2, 4, 100, torch.float16, 3)
    done = torch.ones(2, 4, dtype=torch.uint8, device="cuda")
    check(ssq.ssq_beam_select(logits, scores, done=done, done_token=99, nsel=6),
          reference(logits, scores, done, 99, 6))
    s, p, t = ssq.ssq_beam_select(logits[:0], scores[:0])
    assert s.shape == (0, 4) and p.shape == (0, 4)


def test_selection_graph_stream_and_out():
    ssq = require_gpu()
    logits, scores = draw(3, 4, 5000, torch.bfloat16, 4)
    out = tuple(torch.zeros(3, 4, dtype=d, device="cuda")
                for d in (torch.float32, torch.int32, torch.int32))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = ssq.ssq_beam_select(logits, scores, out=out, stream=st)
    st.synchronize()
    assert got[0].data_ptr() == out[0].data_ptr()
    check(out, reference(logits, scores, None, 0, 4))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ssq.ssq_beam_select(logits, scores, out=out)
    for seed in (5, 6):
        l2, s2 = draw(3, 4, 5000, torch.bfloat16, seed)
        logits.copy_(l2)
        scores.copy_(s2)
        g.replay()
        torch.cuda.synchronize()
        check(out, reference(logits, scores, None, 0, 4))
    del g


# ---------------------------------------------------------------------------
# Reordering
# ---------------------------------------------------------------------------

def random_pool(nbytes, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    pool = torch.randint(0, 256, (nbytes,), generator=g, device="cuda", dtype=torch.uint8)
    pool[:256] = 0
    return pool


def moved(pool, slot_bytes, ranges, slots, parent):
    """The pool after the reordering, by plain indexing."""
    want = pool.clone()
    src, dst = pool[256:].view(-1, slot_bytes), want[256:].view(-1, slot_bytes)
    b, k = parent.shape
    for r in range(b):
        for j in range(k):
            p = int(parent[r, j])
            if p >= 0:
                for a, n in ranges:
                    dst[int(slots[r, j]), a:a + n] = src[int(slots[r, p]), a:a + n]
    return want


PARENTS = {
    "identity": lambda b, k: torch.arange(k).repeat(b, 1),
    "all from the first": lambda b, k: torch.zeros(b, k),
    "cycle": lambda b, k: ((torch.arange(k) + 1) % k).repeat(b, 1),
    "reversed": lambda b, k: torch.arange(k).flip(0).repeat(b, 1),
    "random": lambda b, k: torch.randint(0, k, (b, k), generator=torch.Generator().manual_seed(k)),
    "some stay": lambda b, k: torch.randint(-1, k, (b, k), generator=torch.Generator().manual_seed(k)),
    "nothing": lambda b, k: torch.full((b, k), -1),
}


@pytest.mark.parametrize("kind", list(PARENTS))
@pytest.mark.parametrize("fmt", ["f32", "bf16", "i8s", "i8a", "i4s", "i4a"])
def test_reorder(fmt, kind):
    """Every format, a mask (both regions), a range of layers, permuted slots;
    what is not named stays."""
    ssq = require_gpu()
    mask = [1, 0, 1] if fmt.startswith("i") else None
    for b, k in ((1, 1), (3, 4), (2, 33), (1, 64)):
        cfg = ssq.Config(4, b * k + 3, 3, 24, 64, 1, fmt, mask)
        L = ssq.ssq_pool_layout(cfg)[0]
        pool = random_pool(L["pool_bytes"], 7)
        slots = torch.randperm(b * k + 3, generator=torch.Generator().manual_seed(b))[:b * k]
        slots = slots.view(b, k).to(torch.int32)
        parent = PARENTS[kind](b, k).to(torch.int32)
        ranges = [(L[o] + L[n], 2 * L[n]) for o, n in
                  (("codes_off", "codes_layer_bytes"), ("meta_off", "meta_layer_bytes"),
                   ("fp_off", "fp_layer_bytes"))]
        want = moved(pool, L["slot_bytes"], ranges, slots, parent)
        ssq.ssq_pool_reorder(cfg, pool, slots.cuda(), parent.cuda(), 1, 2)
        assert torch.equal(pool, want), (b, k)


@pytest.mark.parametrize("kind", ["random", "cycle"])
def test_reorder_damp(kind):
    ssq = require_gpu()
    cfg = ssq.DampConfig(3, 9, 2, 32, 48, 1, 5)
    L = ssq.ssq_damp_pool_layout(cfg)
    pool = random_pool(L["pool_bytes"], 8)
    parent = PARENTS[kind](2, 4).to(torch.int32)
    slots = torch.arange(8).view(2, 4).to(torch.int32)
    want = moved(pool, L["slot_bytes"], [(L["layer_bytes"], 2 * L["layer_bytes"])], slots, parent)
    ssq.ssq_damp_pool_reorder(cfg, pool, None, parent.cuda(), 1, 2)
    assert torch.equal(pool, want)


def test_reorder_large():
    """Slots of several megabytes (many chunks per range, several requests a
    block), all layers."""
    ssq = require_gpu()
    cfg = ssq.Config(24, 32, 24, 64, 128, 1, "i8a")
    L = ssq.ssq_pool_layout(cfg)[0]
    pool = random_pool(L["pool_bytes"], 9)
    parent = PARENTS["random"](8, 4).to(torch.int32)
    slots = torch.randperm(32, generator=torch.Generator().manual_seed(3)).view(8, 4).to(torch.int32)
    want = moved(pool, L["slot_bytes"], [(0, L["slot_bytes"])], slots, parent)
    ssq.ssq_pool_reorder(cfg, pool, slots.cuda(), parent.cuda(), 0, 24)
    assert torch.equal(pool, want)


def test_reorder_bad_requests_are_skipped():
    ssq = require_gpu()
    cfg = ssq.Config(1, 12, 2, 16, 32, 1, "i8a")
    L = ssq.ssq_pool_layout(cfg)[0]
    base = torch.arange(12).view(3, 4).to(torch.int32)
    cyc = PARENTS["cycle"](3, 4).to(torch.int32)
    for change, bit in ((("s", 1, 2, 12), "SSQ_DEVERR_SLOT"), (("s", 1, 0, -1), "SSQ_DEVERR_SLOT"),
                        (("p", 1, 3, 4), "SSQ_DEVERR_PARENT"), (("p", 1, 3, -2), "SSQ_DEVERR_PARENT"),
                        (("s", 1, 2, 5), "SSQ_DEVERR_PARENT")):         # slot 5 twice
        slots, parent = base.clone(), cyc.clone()
        which, r, j, val = change
        (slots if which == "s" else parent)[r, j] = val
        pool = random_pool(L["pool_bytes"], 10)
        ok = cyc.clone()
        ok[1] = -1
        want = moved(pool, L["slot_bytes"], [(0, L["slot_bytes"])], base, ok)
        ssq.ssq_pool_reorder(cfg, pool, slots.cuda(), parent.cuda(), 0, 1)
        assert ssq.ssq_pool_error(cfg, pool) == getattr(ssq, bit)
        assert torch.equal(pool, want)


# ---------------------------------------------------------------------------
# A run of them together
# ---------------------------------------------------------------------------

def test_beam_search():
    """Prompts of two requests into one slot each, the slots forked into beams,
    then decode step, selection and reordering in turn, against the same search
    with the states in 64 bits.  A small random model of one layer: token t has
    fixed x, B, C, dt; the logits are a product with the layer's output."""
    ssq = require_gpu()
    H, Pd, N, V, K, R, steps, eos = 4, 16, 64, 211, 3, 2, 8, 0
    g = torch.Generator(device="cuda").manual_seed(11)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    ex, eB, eC = rn(V, H, Pd), 0.25 * rn(V, 1, N), 0.25 * rn(V, 1, N)
    edt = torch.log1p(torch.exp(rn(V, H) - 2.0))
    A, D, W = -torch.exp(rn(H)), rn(H), rn(H * Pd, V) / 4
    ex, eB, eC = (t.to(torch.bfloat16).float() for t in (ex, eB, eC))
    prompts = [torch.randint(1, V, (n,), generator=g, device="cuda") for n in (75, 4)]

    def step64(S, tok):
        lam = torch.exp((edt[tok] * A).double())[..., None, None]
        S = lam * S + (edt[tok].double()[..., None] * ex[tok].double())[..., None] \
            * eB[tok].double()[:, :, None, :]
        y = (S * eC[tok].double()[:, :, None, :]).sum(-1) + D.double()[:, None] * ex[tok].double()
        return S, y

    cfg = ssq.Config(1, R * K, H, Pd, N, 1, "f32")
    pool = ssq.alloc_pool(cfg)
    slots = torch.tensor([[5, 0, 3], [1, 4, 2]], dtype=torch.int32, device="cuda")
    toks = torch.cat(prompts)
    cu = torch.tensor([0, 75, 79], dtype=torch.int32, device="cuda")
    ws = ssq.alloc_prefill_workspace(cfg, R, 75)
    y = torch.empty(79, H, Pd, dtype=torch.bfloat16, device="cuda")
    ssq.ssq_prefill_ragged(cfg, pool, slots[:, 0].contiguous(), R, 0, cu, 75,
                           ex[toks].to(torch.bfloat16), eB[toks].to(torch.bfloat16),
                           eC[toks].to(torch.bfloat16), edt[toks], A, D, y,
                           fresh=torch.ones(R, dtype=torch.uint8, device="cuda"), workspace=ws)
    # every beam starts from its request's prompt
    ssq.ssq_pool_reorder(cfg, pool, slots, torch.zeros(R, K, dtype=torch.int32, device="cuda"), 0, 1)
    S = torch.zeros(R, H, Pd, N, dtype=torch.float64, device="cuda")
    for r, p in enumerate(prompts):
        for t in p:
            S[r:r + 1], _ = step64(S[r:r + 1], t[None])
    S = S[:, None].repeat(1, K, 1, 1, 1)
    score = torch.full((R, K), -math.inf, device="cuda")
    score[:, 0] = 0.0                                      # one live beam at first
    score64, done = score.double(), torch.zeros(R, K, dtype=torch.uint8, device="cuda")
    last = torch.stack([p[-1] for p in prompts])[:, None].repeat(1, K)
    for n in range(steps):
        # the library's side
        x = ex[last].reshape(1, R * K, H, Pd).contiguous()
        yd = torch.empty_like(x)
        ssq.ssq_decode_step(cfg, pool, slots, R * K, 0, 1, x,
                            eB[last].reshape(1, R * K, 1, N).contiguous(),
                            eC[last].reshape(1, R * K, 1, N).contiguous(),
                            edt[last].reshape(1, R * K, H).contiguous(), A[None], D[None], yd)
        logits = (yd.view(R, K, -1) @ W)
        score, parent, token = ssq.ssq_beam_select(logits, score, done=done, done_token=eos)
        ssq.ssq_pool_reorder(cfg, pool, slots, parent, 0, 1)
        # 64 bits
        S2, y64 = step64(S.flatten(0, 1), last.flatten())
        l64 = y64.reshape(R, K, -1) @ W.double()
        val, p64, t64 = reference(l64, score64, done, eos, K)
        assert torch.equal(parent, p64) and torch.equal(token, t64), n
        # y is off by 2^-16 of its absolute recurrence (below 64 here) from
        # the prompt's chunk, a logit by the sum of 64 such errors times |W|
        # (about 0.2), a score by two logits' errors at each of 8 steps
        assert (score.double() - val).abs().max() < 16 * 64 * 0.2 * 64 * 2.0 ** -16
        score64 = val
        # (every place has a candidate here)
        assert (p64 >= 0).all()
        S = S2.view(R, K, H, Pd, N).gather(
            1, p64.long()[..., None, None, None].expand(R, K, H, Pd, N))
        done = (done.gather(1, p64.long()) | (t64 == eos)).to(torch.uint8)
        last = t64.long()
    got = torch.empty(R * K, H, Pd, N, device="cuda")
    ssq.ssq_dequantize_rows(cfg, pool, slots, R * K, 0, 1, got)
    # the prompt's chunk leaves 2^-16 of the absolute recurrence (see
    # test_gpu_ragged.py; that is below 8 times the largest entry), fp32 steps
    # far less
    err = (got.double().view_as(S) - S).abs().max()
    assert err <= 2.0 ** -13 * S.abs().max(), err
    assert ssq.ssq_pool_error(cfg, pool) == 0
