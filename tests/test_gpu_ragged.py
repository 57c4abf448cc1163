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
