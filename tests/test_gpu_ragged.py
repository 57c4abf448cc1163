"""GPU tests of ssq_prefill_ragged (include/ssq_serve.h) against the recurrence
in 64 bits.

Tolerances, from the arithmetic (u = eps/2 of a type, half a step relative to
the value):
  y       normwise: |y - y_ref| <= tol * scale, scale = sum_n |C_n| |s_n| + |D x|
          with |s| the recurrence of the absolute values.
          Token by token, fp32: each step rounds s twice, and an error made k
          steps ago has decayed with its term, so the error of s stays below
          (2 + 3 T) u32 |s| (decay, product, sum: three roundings a step);
          the readout of N terms in fp32 adds N u32 |C||s|, and y is rounded
          to its type.  For T, N <= 600 and u32 = 2^-24 that is under
          2500 * 2^-24 = 1.5e-4, typically 1e-6; the bound is used as it is.
          In chunks: C B^T sums N products of bf16 (exact in fp32) and the
          result, times the decay, is rounded to bf16 (2^-8); the state is
          rounded to bf16 for its product (2^-8); both act on disjoint parts
          of the sum, so together at most 2^-8 of the scale, plus the fp32
          part above, plus the rounding of y (2^-8 of |y| <= scale).
  state   token by token as above: (2 + 3 T) u32 |s|.
          In chunks the input of the state's product is a sum of two bf16
          parts: what is left out is at most 2^-9 * 2^-9 of it (half a step of
          the second part, which is itself at most half a step, 2^-9 relative
          to the power of two below the value ... 2^-8 of the value each), so
          2^-16 of |s|, plus fp32 sums and the exponentials of running sums
          of up to 128 fp32 terms, (2 + 3*128) u32.
  Quantized pools: the stored row may differ by half a step of its grid
  besides, plus one more step where the state's error crosses a boundary.
"""
import math

import pytest
import torch

from gpu_harness import require_gpu

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
QMAX = {"i8s": 127, "i8a": 255, "i4s": 7, "i4a": 15}


def inputs(lens, H, P, N, G, dtype, seed, fused=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    total = sum(lens)
    w = H * P + 2 * G * N
    if fused:
        xbc = torch.cat([rn(total, H * P), 0.25 * rn(total, 2 * G * N)], 1).to(dtype)
        x, B, C = xbc.split([H * P, G * N, G * N], 1)
        x, B, C = x.unflatten(1, (H, P)), B.unflatten(1, (G, N)), C.unflatten(1, (G, N))
    else:
        x, B, C = rn(total, H, P).to(dtype), (0.25 * rn(total, G, N)).to(dtype), \
            (0.25 * rn(total, G, N)).to(dtype)
    dt = torch.log1p(torch.exp(rn(total, H) - 2.0))
    A = -torch.exp(torch.empty(H, device="cuda").uniform_(math.log(0.5), math.log(16.0),
                                                          generator=g))
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    return dict(x=x, B=B, C=C, dt=dt, A=A, D=rn(H), cu=cu, S0=rn(len(lens), H, P, N))


def reference(i, lens, S0):
    """y, |scale|, final states and |states| in 64 bits, token by token."""
    f = torch.float64
    total, H, P = i["x"].shape
    G, N = i["B"].shape[1:]
    grp = torch.arange(H, device="cuda") // (H // G)
    y = torch.zeros(total, H, P, dtype=f, device="cuda")
    sc = torch.zeros_like(y)
    S, M = S0.to(f).clone(), S0.to(f).abs().clone()
    off = 0
    for b, n in enumerate(lens):
        for t in range(off, off + n):
            lam = torch.exp((i["dt"][t] * i["A"]).to(f))[:, None, None]
            x, Bt, Ct = i["x"][t].to(f), i["B"][t].to(f)[grp], i["C"][t].to(f)[grp]
            dx = (i["dt"][t].to(f)[:, None] * x)
            S[b] = lam * S[b] + dx[..., None] * Bt[:, None, :]
            M[b] = lam * M[b] + (dx.abs())[..., None] * Bt.abs()[:, None, :]
            Dx = i["D"].to(f)[:, None] * x
            y[t] = (S[b] * Ct[:, None, :]).sum(-1) + Dx
            sc[t] = (M[b] * Ct.abs()[:, None, :]).sum(-1) + Dx.abs()
        off += n
    return y, sc, S, M


def chunked(i, n):
    """Whether a run of n tokens goes through chunks (include/ssq_serve.h)."""
    P, N = i["x"].shape[2], i["B"].shape[2]
    ok16 = all(i[k].data_ptr() % 16 == 0 and i[k].stride(0) % 8 == 0 for k in "xBC")
    return i["x"].dtype == torch.bfloat16 and P % 8 == 0 and N <= 128 and ok16 and n >= 32


def run(ssq, i, lens, fmt, fresh=None, layers=1, layer=0, mask=None, slots=None, y=None):
    """The call on a pool whose slots hold S0; returns y, the stored states
    before and after, the pool and its config."""
    total, H, P = i["x"].shape
    G, N = i["B"].shape[1:]
    batch = len(lens)
    n_slots = batch + 2
    cfg = ssq.Config(layers, n_slots, H, P, N, G, fmt, mask)
    pool = ssq.alloc_pool(cfg)
    if slots is None:
        slots = torch.arange(batch, 0, -1, device="cuda", dtype=torch.int32)
    ssq.ssq_quantize_rows(cfg, pool, slots, batch, layer, 1, i["S0"].contiguous())
    before = torch.empty(batch, H, P, N, device="cuda")
    ssq.ssq_dequantize_rows(cfg, pool, slots, batch, layer, 1, before)
    if y is None:
        y = torch.full((total, H, P), float("nan"), dtype=i["x"].dtype, device="cuda")
    max_len = max(lens, default=0)
    ws = ssq.alloc_prefill_workspace(cfg, batch, max_len)
    ssq.ssq_prefill_ragged(cfg, pool, slots, batch, layer, i["cu"], max_len, i["x"], i["B"],
                           i["C"], i["dt"], i["A"], i["D"], y, fresh=fresh, workspace=ws)
    after = torch.empty(batch, H, P, N, device="cuda")
    ssq.ssq_dequantize_rows(cfg, pool, slots, batch, layer, 1, after)
    return y, before, after, pool, cfg


def check(i, lens, fmt, y, before, after, fresh=None, mask=None):
    batch, (total, H, P) = len(lens), i["x"].shape
    S0 = before.clone()
    if fresh is not None:
        S0[fresh.bool()] = 0
    yr, sc, S, M = reference(i, lens, S0)
    N = S.shape[-1]
    off = 0
    for b, n in enumerate(lens):
        steps = (2 + 3 * max(n, 1)) * U32
        ys = slice(off, off + n)
        off += n
        if chunked(i, n):
            ytol = 2.0 ** -8 + steps + N * U32 + U[y.dtype]
            stol = 2.0 ** -16 + steps
        else:
            ytol, stol = steps + N * U32 + U[y.dtype], steps
        if n:
            err = (y[ys].double() - yr[ys]).abs()
            worst = (err / (sc[ys] + 1e-30)).max().item()
            assert torch.all(err <= ytol * sc[ys] + 1e-30), (b, n, "y", worst, ytol)
        err = (after[b].double() - S[b]).abs()
        bound = stol * M[b] + 1e-30
        if fmt == "bf16":
            bound = bound + 2.0 ** -8 * (S[b].abs() + bound)
        if fmt in QMAX:
            q = torch.tensor([True] * H if mask is None else [bool(m) for m in mask],
                             device="cuda")[:, None, None]
            lo, hi = S[b].amin(-1, keepdim=True), S[b].amax(-1, keepdim=True)
            step = (torch.maximum(hi, -lo) if fmt in ("i8s", "i4s") else hi - lo) / QMAX[fmt]
            # half a step, a rounding of the zero point at the ends of an
            # asymmetric grid, and the error carried through the refit
            half = 0.5 if fmt in ("i8s", "i4s") else 1.0
            grid = half * step * (1 + 2.0 ** -10) + 4 * bound.amax(-1, keepdim=True)
            bound = torch.where(q, bound + grid, bound)
        if n == 0 and (fresh is None or not fresh[b]):
            assert torch.equal(after[b], before[b])      # an idle slot stays
        else:
            worst = (err / bound).max().item()
            assert torch.all(err <= bound), (b, n, "state", worst)


FMTS = ["f32", "bf16", "i8s", "i8a", "i4s", "i4a"]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_short_runs(fmt, dtype):
    """Runs below the chunk limit: single tokens, an empty run, odd headdim."""
    ssq = require_gpu()
    lens = [1, 7, 0, 1, 31, 8]
    i = inputs(lens, 6, 12, 64, 3, dtype, 1)
    y, b, a, pool, cfg = run(ssq, i, lens, fmt)
    check(i, lens, fmt, y, b, a)
    assert ssq.ssq_pool_error(cfg, pool) == 0


@pytest.mark.parametrize("shape", [(1, 1, 16, 1), (3, 5, 32, 1), (2, 8, 256, 2), (4, 130, 128, 2),
                                   (2, 300, 16, 1)])
def test_shapes_token_by_token(shape):
    """Odd heads and rows, the smallest and largest d_state, long runs in a
    type without chunks."""
    ssq = require_gpu()
    H, P, N, G = shape
    lens = [3, 50, 1]
    i = inputs(lens, H, P, N, G, torch.float32, 2, fused=False)
    y, b, a, pool, cfg = run(ssq, i, lens, "i8a")
    check(i, lens, "i8a", y, b, a)


@pytest.mark.parametrize("fmt", FMTS)
def test_chunks_formats(fmt):
    """One and several chunks, a ragged tail, mixed with short runs, from
    stored and from fresh states."""
    ssq = require_gpu()
    lens = [128, 40, 1, 300, 0, 129, 32]
    fresh = torch.tensor([0, 1, 0, 0, 1, 1, 0], dtype=torch.uint8, device="cuda")
    i = inputs(lens, 4, 64, 128, 2, torch.bfloat16, 3)
    y, b, a, pool, cfg = run(ssq, i, lens, fmt, fresh=fresh)
    check(i, lens, fmt, y, b, a, fresh=fresh)
    assert ssq.ssq_pool_error(cfg, pool) == 0


@pytest.mark.parametrize("shape", [(1, 64, 128, 1), (3, 64, 128, 1), (2, 8, 16, 1), (3, 40, 64, 3),
                                   (2, 72, 32, 1), (2, 128, 128, 1), (5, 24, 128, 1),
                                   (1, 200, 64, 1)])
def test_chunks_shapes(shape):
    """Odd numbers of units, rows that do not fill a unit, every d_state."""
    ssq = require_gpu()
    H, P, N, G = shape
    lens = [200, 33, 256]
    i = inputs(lens, H, P, N, G, torch.bfloat16, 4)
    y, b, a, pool, cfg = run(ssq, i, lens, "f32")
    check(i, lens, "f32", y, b, a)
    assert ssq.ssq_pool_error(cfg, pool) == 0


@pytest.mark.parametrize("fmt,fresh", [("f32", True), ("i8a", False)])
def test_chunks_segments(fmt, fresh):
    """A run long enough to be cut into segments, beside one that is not."""
    ssq = require_gpu()
    lens = [1700, 150]
    i = inputs(lens, 2, 64, 128, 1, torch.bfloat16, 5)
    fr = torch.ones(2, dtype=torch.uint8, device="cuda") if fresh else None
    cfg = ssq.Config(1, 4, 2, 64, 128, 1, fmt)
    assert ssq.ssq_prefill_ragged_workspace(cfg, 2, 1700) > 0
    y, b, a, pool, cfg = run(ssq, i, lens, fmt, fresh=fr)
    check(i, lens, fmt, y, b, a, fresh=fr)
    assert ssq.ssq_pool_error(cfg, pool) == 0


@pytest.mark.parametrize("fmt,H,P,N,mask", [("bf16", 3, 64, 128, None), ("i8s", 1, 64, 64, None),
                                            ("i4a", 3, 40, 128, [1, 0, 1]),
                                            ("i8a", 2, 72, 16, None)])
def test_chunks_segments_shapes(fmt, H, P, N, mask):
    """Segments with an odd number of units, rows that do not fill one, masked
    heads, and runs that end in every segment."""
    ssq = require_gpu()
    lens = [2100, 600, 1030, 0]
    i = inputs(lens, H, P, N, 1, torch.bfloat16, 21)
    fresh = torch.tensor([0, 1, 0, 0], dtype=torch.uint8, device="cuda")
    y, b, a, pool, cfg = run(ssq, i, lens, fmt, fresh=fresh, mask=mask)
    check(i, lens, fmt, y, b, a, fresh=fresh, mask=mask)
    assert ssq.ssq_pool_error(cfg, pool) == 0


@pytest.mark.parametrize("fmt", ["f32", "bf16"])
@pytest.mark.parametrize("at", [5, 700, 1990])
def test_non_finite_in_segments(fmt, at):
    """A NaN in one row of x makes y and the state of that row NaN from there
    on, over the segments behind, and nothing else."""
    ssq = require_gpu()
    i = inputs([2000], 2, 64, 128, 1, torch.bfloat16, 22)
    y0, _, a0, _, _ = run(ssq, i, [2000], fmt)
    i["x"][at, 1, 7] = math.nan
    y, _, a, _, _ = run(ssq, i, [2000], fmt)
    hit = torch.zeros_like(y0, dtype=torch.bool)
    hit[at:, 1, 7] = True
    assert torch.equal(y[~hit], y0[~hit]) and y[hit].isnan().all()
    assert a[0, 1, 7].isnan().all()
    a[0, 1, 7] = a0[0, 1, 7]
    assert torch.equal(a, a0)


@pytest.mark.parametrize("fmt,dtype,N,mask", [("f32", torch.float16, 128, None),
                                              ("bf16", torch.float32, 256, None),
                                              ("i8a", torch.float16, 16, None),
                                              ("i4s", torch.float32, 64, [1, 0]),
                                              ("i8s", torch.float16, 128, [0, 1])])
def test_token_segments(fmt, dtype, N, mask):
    """Types without chunks: a long run cut into segments of tokens (two
    passes), beside one that ends in the second segment, one of a segment, a
    single token and none, from stored and from fresh states."""
    ssq = require_gpu()
    lens = [1200, 290, 256, 1, 0, 0]
    fresh = torch.tensor([0, 1, 0, 0, 0, 1], dtype=torch.uint8, device="cuda")
    i = inputs(lens, 2, 20, N, 1, dtype, 19)
    cfg = ssq.Config(1, 8, 2, 20, N, 1, fmt, mask)
    assert ssq.ssq_prefill_ragged_workspace(cfg, 6, 1200) >= 6 * 4 * 2 * 20 * N * 4
    y, b, a, pool, cfg = run(ssq, i, lens, fmt, fresh=fresh, mask=mask)
    check(i, lens, fmt, y, b, a, fresh=fresh, mask=mask)
    assert ssq.ssq_pool_error(cfg, pool) == 0
    again, _, a2, _, _ = run(ssq, i, lens, fmt, fresh=fresh, mask=mask)
    assert torch.equal(y, again) and torch.equal(a, a2)


# ---------------------------------------------------------------------------
# What a call may not touch, and what must not spread
# ---------------------------------------------------------------------------

def test_strides_and_alignment():
    """Slices of one fused activation, separate tensors and a base that is not
    16-byte aligned give the same values: bit for bit where the path is the
    same, within the path's tolerance where the last takes the other one."""
    ssq = require_gpu()
    lens = [150, 3, 40]
    i = inputs(lens, 4, 64, 128, 2, torch.bfloat16, 6)
    y1, b1, a1, _, _ = run(ssq, i, lens, "f32")
    j = dict(i, x=i["x"].contiguous(), B=i["B"].contiguous(), C=i["C"].contiguous(),
             dt=torch.cat([i["dt"], i["dt"]], 1)[:, :4])
    y2, _, a2, _, _ = run(ssq, j, lens, "f32")
    assert torch.equal(y1, y2) and torch.equal(a1, a2)
    total, w = sum(lens), 4 * 64 + 2 * 2 * 128
    odd = torch.empty(total * w + 1, dtype=torch.bfloat16, device="cuda")[1:].view(total, w)
    odd.copy_(torch.cat([i["x"].flatten(1), i["B"].flatten(1), i["C"].flatten(1)], 1))
    k = dict(i, x=odd[:, :256].unflatten(1, (4, 64)), B=odd[:, 256:512].unflatten(1, (2, 128)),
             C=odd[:, 512:].unflatten(1, (2, 128)))
    y3, b3, a3, _, _ = run(ssq, k, lens, "f32")
    check(k, lens, "f32", y3, b3, a3)
    # y with its own stride
    wide = torch.zeros(total, 4 * 64 + 8, dtype=torch.bfloat16, device="cuda")
    y4, _, a4, _, _ = run(ssq, i, lens, "f32", y=wide[:, :256].unflatten(1, (4, 64)))
    assert torch.equal(y4, y1) and torch.equal(a4, a1) and not wide[:, 256:].any()


@pytest.mark.parametrize("n", [1, 20, 200])
def test_leaves_the_rest_alone(n):
    """Tokens outside every request, slots that are not named and other layers
    keep what they hold."""
    ssq = require_gpu()
    H, Pd, N = 3, 64, 128
    lens = [n, n]
    i = inputs([5] + lens + [7], H, Pd, N, 1, torch.bfloat16, 7)
    i["cu"] = i["cu"][1:4].contiguous()
    i["S0"] = i["S0"][:2].contiguous()
    total = i["x"].shape[0]
    y = torch.full((total, H, Pd), 7.0, dtype=torch.bfloat16, device="cuda")
    cfg = ssq.Config(3, 5, H, Pd, N, 1, "i8a")
    pool = torch.randint(0, 255, (ssq.ssq_pool_layout(cfg)[0]["pool_bytes"],), dtype=torch.uint8,
                         device="cuda")
    pool[:256] = 0
    before = pool.clone()
    slots = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    fresh = torch.ones(2, dtype=torch.uint8, device="cuda")
    ws = ssq.alloc_prefill_workspace(cfg, 2, n)
    ssq.ssq_prefill_ragged(cfg, pool, slots, 2, 1, i["cu"], n, i["x"], i["B"], i["C"], i["dt"],
                           i["A"], i["D"], y, fresh=fresh, workspace=ws)
    assert (y[:5] == 7).all() and (y[5 + 2 * n:] == 7).all() and not (y[5:5 + 2 * n] == 7).all()
    L = ssq.ssq_pool_layout(cfg)[0]
    changed = (pool != before)
    assert not changed[:256].any()
    body = changed[256:].view(5, L["slot_bytes"])
    assert not body[[0, 2, 4]].any() and body[1].any() and body[3].any()
    for off, lay in (("codes_off", "codes_layer_bytes"), ("meta_off", "meta_layer_bytes")):
        for l in (0, 2):
            a = L[off] + l * L[lay]
            assert not body[:, a:a + L[lay]].any()


@pytest.mark.parametrize("n", [6, 150])
def test_bad_requests_are_skipped(n):
    """A range that falls, leaves the batch or is longer than max_len, and a
    slot outside the pool: the request is skipped and reported, the others
    are done."""
    ssq = require_gpu()
    lens = [n, n, n, n]
    i = inputs(lens, 2, 64, 128, 1, torch.bfloat16, 8)
    good_y, _, good_a, _, _ = run(ssq, i, lens, "f32")
    cfg = ssq.Config(1, 6, 2, 64, 128, 1, "f32")

    def call(cu, slots, max_len):
        pool = ssq.alloc_pool(cfg)
        base = torch.tensor([4, 3, 2, 1], dtype=torch.int32, device="cuda")
        ssq.ssq_quantize_rows(cfg, pool, base, 4, 0, 1, i["S0"])
        y = torch.full_like(good_y, 7.0)
        ws = ssq.alloc_prefill_workspace(cfg, 4, max_len)
        ssq.ssq_prefill_ragged(cfg, pool, torch.tensor(slots, dtype=torch.int32, device="cuda"), 4,
                               0, torch.tensor(cu, dtype=torch.int32, device="cuda"), max_len,
                               i["x"], i["B"], i["C"], i["dt"], i["A"], i["D"], y, workspace=ws)
        S = torch.empty(4, 2, 64, 128, device="cuda")
        ssq.ssq_dequantize_rows(cfg, pool, base, 4, 0, 1, S)
        return y, S, ssq.ssq_pool_error(cfg, pool)

    cu = [0, n, 2 * n, 3 * n, 4 * n]
    for slots in ([4, 99, 2, 1], [4, -1, 2, 1]):
        y, S, err = call(cu, slots, n)
        assert err == ssq.SSQ_DEVERR_SLOT
        assert (y[n:2 * n] == 7).all() and torch.equal(S[1], i["S0"][1])
        assert torch.equal(y[2 * n:], good_y[2 * n:]) and torch.equal(S[2:], good_a[2:])
    for bad, skipped in (([0, n, 2 * n, 3 * n, 4 * n + 1], [3]),          # past the batch
                         ([-1, n, 2 * n, 3 * n, 4 * n], [0]),
                         ([0, n, n - 1, 3 * n, 4 * n], [1, 2])):          # falls, then too long
        y, S, err = call(bad, [4, 3, 2, 1], n)
        assert err == ssq.SSQ_DEVERR_TOKENS
        for b in range(4):
            if b in skipped:
                assert torch.equal(S[b], i["S0"][b])
            else:
                assert torch.equal(S[b], good_a[b])
    y, S, err = call(cu, [4, 3, 2, 1], n - 1)                             # all longer than max_len
    assert err == ssq.SSQ_DEVERR_TOKENS and (y == 7).all() and torch.equal(S, i["S0"])


@pytest.mark.parametrize("dtype,n", [(torch.bfloat16, 200), (torch.float16, 30)])
@pytest.mark.parametrize("what,value", [("x", math.nan), ("x", math.inf), ("B", math.nan),
                                        ("C", math.inf), ("dt", math.nan)])
def test_non_finite_stays_where_it_is(dtype, n, what, value):
    """A non-finite value at one token of one request reaches its own and later
    tokens of that request only (x: of its row only; C: of its token only),
    not its earlier tokens in the same chunk and not the neighbours in the
    packed batch."""
    ssq = require_gpu()
    H, Pd, N = 2, 64, 128
    lens = [n, n, n]
    at = n + n // 2                                   # a token of the middle request
    i = inputs(lens, H, Pd, N, 1, dtype, 9)
    y0, _, a0, _, _ = run(ssq, i, lens, "f32")
    if what == "x":
        i["x"][at, 1, 5] = value
    elif what == "dt":
        i["dt"][at, 1] = value
    else:
        i[what][at, 0, 3] = value
    y, _, a, pool, cfg = run(ssq, i, lens, "f32")
    hit = torch.zeros_like(y0, dtype=torch.bool)      # what may change
    if what == "x":
        hit[at:2 * n, 1, 5] = True
    elif what == "dt":
        hit[at:2 * n, 1] = True
    elif what == "B":
        hit[at:2 * n] = True
    else:
        hit[at] = True
    assert torch.equal(y[~hit], y0[~hit])
    assert not y[hit].isfinite().any()
    same = torch.ones_like(a0, dtype=torch.bool)
    if what == "x":
        same[1, 1, 5] = False
    elif what == "dt":
        same[1, 1] = False
    elif what == "B":
        same[1] = False
    assert torch.equal(a[same], a0[same])
    if what in ("x", "dt"):
        assert not a[~same].isfinite().any()


@pytest.mark.parametrize("n", [5, 140])
def test_non_finite_row_is_reported(n):
    """A quantized row that is not finite at the end sets the pool's bit."""
    ssq = require_gpu()
    i = inputs([n], 2, 64, 128, 1, torch.bfloat16, 10)
    i["x"][n - 1, 0, 3] = math.nan
    y, _, a, pool, cfg = run(ssq, i, [n], "i8a")
    assert ssq.ssq_pool_error(cfg, pool) == ssq.SSQ_DEVERR_NONFINITE
    assert a[0, 0, 3].isnan().all()
    a[0, 0, 3] = 0
    assert a.isfinite().all()


def test_decay_extremes():
    """Steps that forget everything (A = -inf, large dt), steps of zero (the
    state unchanged), and growth (A > 0) in one chunked run."""
    ssq = require_gpu()
    lens = [160]
    i = inputs(lens, 4, 64, 128, 1, torch.bfloat16, 11)
    i["A"] = torch.tensor([-math.inf, -1e6, 1e-3, -2.0], device="cuda")
    i["dt"][:, 3] = 0.0
    i["dt"][7, 3] = 30.0
    y, b, a, pool, cfg = run(ssq, i, lens, "f32")
    check(i, lens, "f32", y, b, a)


def test_masked_heads():
    """Heads whose mask is 0 keep fp32 rows beside quantized ones."""
    ssq = require_gpu()
    for n, mask in ((3, [1, 0, 1, 0]), (100, [0, 1, 1, 0])):
        lens = [n, n + 1]
        i = inputs(lens, 4, 40, 64, 2, torch.bfloat16, 12)
        y, b, a, pool, cfg = run(ssq, i, lens, "i4a", mask=mask)
        check(i, lens, "i4a", y, b, a, mask=mask)


def test_equals_ssq_prefill_bit_for_bit():
    """fp32 activations: the stored codes and metadata are those of ssq_prefill
    (the same operations in the same order)."""
    ssq = require_gpu()
    H, Pd, N, T = 3, 12, 64, 70
    i = inputs([T, T], H, Pd, N, 1, torch.float32, 13, fused=False)
    for fmt in FMTS:
        _, _, _, pool, cfg = run(ssq, i, [T, T], fmt)
        slots = torch.tensor([2, 1], dtype=torch.int32, device="cuda")
        other = ssq.alloc_pool(cfg)
        ssq.ssq_quantize_rows(cfg, other, slots, 2, 0, 1, i["S0"])
        y = torch.empty(2, T, H, Pd, device="cuda")
        ssq.ssq_prefill(cfg, other, slots, 2, 0, T, i["x"], i["B"], i["C"], i["dt"], i["A"],
                        i["D"], y)
        assert torch.equal(pool, other), fmt


def test_pieces_equal_the_whole():
    """A prompt in pieces (an fp32 pool carries the state exactly) against the
    same prompt in one call: both within the chunk path's tolerance of the
    recurrence, whichever path each piece takes."""
    ssq = require_gpu()
    H, Pd, N, T = 2, 64, 128, 389
    i = inputs([T], H, Pd, N, 1, torch.bfloat16, 14)
    cfg = ssq.Config(1, 1, H, Pd, N, 1, "f32")
    pool = ssq.alloc_pool(cfg)
    ssq.ssq_quantize_rows(cfg, pool, None, 1, 0, 1, i["S0"])
    y = torch.empty(T, H, Pd, dtype=torch.bfloat16, device="cuda")
    ws = ssq.alloc_prefill_workspace(cfg, 1, T)
    at = 0
    for n in (128, 1, 31, 130, 64, 1, 34):
        cu = torch.tensor([at, at + n], dtype=torch.int32, device="cuda")
        ssq.ssq_prefill_ragged(cfg, pool, None, 1, 0, cu, n, i["x"], i["B"], i["C"], i["dt"],
                               i["A"], i["D"], y, workspace=ws)
        at += n
    assert at == T
    a = torch.empty(1, H, Pd, N, device="cuda")
    ssq.ssq_dequantize_rows(cfg, pool, None, 1, 0, 1, a)
    check(i, [T], "f32", y, i["S0"], a)


# ---------------------------------------------------------------------------
# Streams, graphs, repetition
# ---------------------------------------------------------------------------

def test_streams_and_repetition():
    """Two calls at once on two streams, each with its slots and workspace, and
    the same call again: the same bits every time."""
    ssq = require_gpu()
    lens = [1500, 9, 1, 77]
    i = inputs(lens, 2, 64, 128, 1, torch.bfloat16, 15)
    cfg = ssq.Config(1, 8, 2, 64, 128, 1, "i8a")
    want = None
    for _ in range(3):
        pool = ssq.alloc_pool(cfg)
        halves = []
        torch.cuda.synchronize()
        for k in range(2):
            st = torch.cuda.Stream()
            slots = torch.arange(4, dtype=torch.int32, device="cuda") + 4 * k
            ws = ssq.alloc_prefill_workspace(cfg, 4, 1500)
            y = torch.empty_like(i["x"], memory_format=torch.contiguous_format)
            halves.append((st, slots, ws, y))
        torch.cuda.synchronize()
        for st, slots, ws, y in halves:
            with torch.cuda.stream(st):
                ssq.ssq_prefill_ragged(cfg, pool, slots, 4, 0, i["cu"], 1500, i["x"], i["B"],
                                       i["C"], i["dt"], i["A"], i["D"], y, workspace=ws)
        torch.cuda.synchronize()
        assert torch.equal(halves[0][3], halves[1][3])
        body = pool[256:].view(8, -1)
        assert torch.equal(body[:4], body[4:])
        if want is None:
            want = (halves[0][3].clone(), pool.clone())
        assert torch.equal(halves[0][3], want[0]) and torch.equal(pool, want[1])


def test_captured_call_follows_its_inputs():
    """A captured call replayed with other tokens, lengths and slots (within
    max_len) does what an eager call on them does."""
    ssq = require_gpu()
    H, Pd, N = 3, 64, 128
    first, second = [700, 1, 20, 300], [1, 640, 100, 280]
    i, j = (inputs(l, H, Pd, N, 1, torch.bfloat16, s) for l, s in ((first, 16), (second, 17)))
    cfg = ssq.Config(1, 4, H, Pd, N, 1, "bf16")
    buf = {k: torch.empty_like(i[k], memory_format=torch.contiguous_format) for k in
           ("x", "B", "C", "dt", "A", "D", "cu")}
    slots = torch.arange(4, dtype=torch.int32, device="cuda")
    ws = ssq.alloc_prefill_workspace(cfg, 4, 700)
    fresh = torch.zeros(4, dtype=torch.uint8, device="cuda")
    pool = ssq.alloc_pool(cfg)
    y = torch.empty(sum(first), H, Pd, dtype=torch.bfloat16, device="cuda")

    def call():
        ssq.ssq_prefill_ragged(cfg, pool, slots, 4, 0, buf["cu"], 700, buf["x"], buf["B"],
                               buf["C"], buf["dt"], buf["A"], buf["D"], y, fresh=fresh, workspace=ws)

    for k in buf:
        buf[k].copy_(i[k])
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for data, order in ((i, [0, 1, 2, 3]), (j, [2, 0, 3, 1]), (i, [3, 2, 1, 0])):
        for k in buf:
            buf[k].copy_(data[k])
        slots.copy_(torch.tensor(order, dtype=torch.int32))
        fresh.copy_(torch.tensor([1, 0, 1, 0], dtype=torch.uint8))
        start = pool.clone()
        call()
        want_y, want = y.clone(), pool.clone()
        pool.copy_(start)
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want_y) and torch.equal(pool, want)
    del g


def test_many_requests():
    """More requests than a block has threads, of every kind, in one call."""
    ssq = require_gpu()
    lens = [1, 0, 3, 40] * 150
    i = inputs(lens, 1, 16, 16, 1, torch.bfloat16, 18)
    fresh = (torch.arange(600, device="cuda") % 5 == 1).to(torch.uint8)
    y, b, a, pool, cfg = run(ssq, i, lens, "f32", fresh=fresh)
    check(i, lens, "f32", y, b, a, fresh=fresh)
    assert ssq.ssq_pool_error(cfg, pool) == 0


def test_many_runs_in_chunks():
    """Runs of every length up to max_len, more than blocks and threads, in an
    order that is not theirs by length."""
    ssq = require_gpu()
    lens = [40, 1, 256, 100] + [0] * 250 + [200, 33, 129, 64, 1, 256, 180, 90, 31]
    i = inputs(lens, 64, 8, 16, 1, torch.bfloat16, 20)
    y, b, a, pool, cfg = run(ssq, i, lens, "i8s")
    check(i, lens, "i8s", y, b, a)
    again, _, a2, _, _ = run(ssq, i, lens, "i8s")
    assert torch.equal(y, again) and torch.equal(a, a2)
    assert ssq.ssq_pool_error(cfg, pool) == 0
