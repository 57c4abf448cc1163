"""Host-only checks of include/ssq_serve.h: exported symbols, constants of the
binding, workspace sizes, and arguments refused before anything is launched
(no GPU here)."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ssq_serve.h")
GOOD = 0x10000000
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def ssq():
    from quantized_recurrent_state_mamba_b200 import build
    build.build()
    from quantized_recurrent_state_mamba_b200 import ssq as m
    return m


def test_exports_every_declared_symbol(ssq):
    syms = sorted(set(re.findall(r"SSQ_API\s+[\w\s\*]+?\b(ssq_\w+)\s*\(", open(HEADER).read())))
    assert syms == ["ssq_beam_select", "ssq_damp_pool_reorder", "ssq_pool_reorder",
                    "ssq_prefill_ragged", "ssq_prefill_ragged_workspace"]
    lib = ctypes.CDLL(ssq.LIB_PATH)
    for s in syms:
        assert hasattr(lib, s), s


def test_binding_constants_match_header(ssq):
    src = open(HEADER).read()
    defs = dict(re.findall(r"#define\s+(SSQ_\w+)\s+(0x[0-9a-fA-F]+|\d+)u?\b", src))
    assert {"SSQ_DEVERR_TOKENS", "SSQ_DEVERR_PARENT", "SSQ_MAX_BEAMS"} == set(defs)
    defs.update(re.findall(r"\b(SSQ_T_\w+)\s*=\s*(\d+)", src))
    for name, val in defs.items():
        assert getattr(ssq, name) == int(val, 0), name
    # the new error bits are apart from those of ssq.h
    old = ssq.SSQ_DEVERR_SLOT | ssq.SSQ_DEVERR_NONFINITE | ssq.SSQ_DEVERR_TIMEOUT | \
        ssq.SSQ_DEVERR_CHANNEL
    assert not old & (ssq.SSQ_DEVERR_TOKENS | ssq.SSQ_DEVERR_PARENT)
    assert not ssq.SSQ_DEVERR_TOKENS & ssq.SSQ_DEVERR_PARENT


def config(ssq, **over):
    kw = dict(n_layers=2, n_slots=8, nheads=4, headdim=16, d_state=64, ngroups=2, fmt="i8a")
    kw.update(over)
    return ssq.Config(**kw)


def test_workspace_sizes(ssq):
    cfg = config(ssq)
    need = lambda batch, n, c=cfg: ssq.ssq_prefill_ragged_workspace(c, batch, n)
    assert need(0, 1000) == 0 and need(4, 0) == 0 and need(4, 31) == 0
    assert need(4, 32) > 0                      # runs of 32 tokens may go through chunks
    assert need(4, 32) % 256 == 0
    # token by token: nothing, until a run is worth cutting into segments
    for odd in (config(ssq, headdim=12), config(ssq, d_state=256)):
        assert need(4, 600, odd) == 0
        assert need(4, 4096, odd) % (4 * 4 * (odd.c.headdim * odd.c.d_state + 1) * 4) == 0
        assert need(4, 4096, odd) > 0
    # a long run on few heads is cut into segments: a state per request,
    # segment and head
    states = need(1, 65536) - need(1, 129)
    assert states > 2 * 4 * 16 * 64 * 4
    # many blocks already: no segments, only the work list
    big = ssq.Config(1, 256, 128, 64, 128, 8, "i8a")
    assert need(64, 65536, big) < 4096
    for batch, n in ((-1, 4), (4, -1)):
        with pytest.raises(ssq.SsqError) as e:
            need(batch, n)
        assert e.value.status == ssq.SSQ_ERR_INVALID_ARG
    assert ssq.raw().ssq_prefill_ragged_workspace(cfg.ref, 1, 1, None) == ssq.SSQ_ERR_INVALID_ARG


def test_prefill_ragged_refusals(ssq):
    cfg = config(ssq)
    HP, GN, H = 64, 128, 4

    def call(tok_over=(), **over):
        tok = ssq.ssq_tokens()
        tok.type, tok.total = ssq.SSQ_T_BF16, 100
        for n in "x B C dt y".split():
            setattr(tok, n, GOOD)
        tok.x_stride = tok.y_stride = HP
        tok.B_stride = tok.C_stride = GN
        tok.dt_stride = H
        for k, v in dict(tok_over).items():
            setattr(tok, k, v)
        a = dict(pool=GOOD, slots=None, batch=2, layer=0, cu=GOOD, max_len=64, fresh=None, A=GOOD,
                 D=GOOD, ws=GOOD, bytes=1 << 20, tok=ctypes.byref(tok))
        a.update(over)
        return ssq.raw().ssq_prefill_ragged(
            cfg.ref, P(a["pool"]), P(a["slots"]), a["batch"], a["layer"], P(a["cu"]), a["max_len"],
            P(a["fresh"]), a["tok"], P(a["A"]), P(a["D"]), P(a["ws"]), a["bytes"], None)

    bad, align = ssq.SSQ_ERR_INVALID_ARG, ssq.SSQ_ERR_ALIGNMENT
    assert call(batch=0) == ssq.SSQ_OK          # an empty batch is a no-op
    assert call(pool=0) == bad and call(pool=GOOD + 16) == align
    assert call(batch=-1) == bad and call(batch=9) == bad       # > n_slots, identity slots
    assert call(layer=2) == bad and call(layer=-1) == bad
    assert call(slots=GOOD + 2) == align
    assert call(cu=0) == bad and call(cu=GOOD + 2) == align
    assert call(max_len=-1) == bad
    assert call(tok=None) == bad
    assert call(A=0) == bad and call(D=GOOD + 1) == align
    assert call(ws=0) == bad and call(ws=GOOD + 16) == align and call(bytes=16) == bad
    assert "workspace" in ssq.ssq_last_error_detail()
    assert call({"type": 3}) == bad and call({"type": -1}) == bad
    assert call({"total": -1}) == bad and call({"total": 1 << 31}) == bad
    for n in "x B C dt y".split():
        assert call({n: 0}) == bad, n
        assert call({n: GOOD + 1}) == align, n
    for n, least in (("x", HP), ("B", GN), ("C", GN), ("dt", H), ("y", HP)):
        assert call({n + "_stride": least - 1}) == bad, n
        assert call({n + "_stride": 1 << 40}) == bad, n
    # fp32 activations need 4-byte alignment
    assert call({"type": ssq.SSQ_T_F32, "x": GOOD + 2}) == align


def test_beam_select_refusals(ssq):
    def call(**over):
        a = dict(batch=2, beams=4, vocab=100, type=ssq.SSQ_T_F32, logits=GOOD, stride=100,
                 scores=GOOD, done=None, done_token=0, nsel=4, s=GOOD, p=GOOD, t=GOOD)
        a.update(over)
        return ssq.raw().ssq_beam_select(a["batch"], a["beams"], a["vocab"], a["type"],
                                         P(a["logits"]), a["stride"], P(a["scores"]), P(a["done"]),
                                         a["done_token"], a["nsel"], P(a["s"]), P(a["p"]), P(a["t"]),
                                         None)

    bad, align, unsup = ssq.SSQ_ERR_INVALID_ARG, ssq.SSQ_ERR_ALIGNMENT, ssq.SSQ_ERR_UNSUPPORTED
    assert call(batch=0) == ssq.SSQ_OK
    assert call(batch=-1) == bad and call(batch=1 << 30) == unsup
    assert call(beams=0) == bad and call(beams=65) == unsup
    assert call(vocab=0) == bad and call(vocab=1 << 30, stride=1 << 30) == unsup
    assert call(nsel=0) == bad and call(nsel=65) == unsup
    assert call(stride=99) == bad
    assert call(type=7) == bad
    for n in ("logits", "scores", "s", "p", "t"):
        assert call(**{n: 0}) == bad, n
        assert call(**{n: GOOD + 2}) == align, n
    assert call(logits=GOOD + 1, type=ssq.SSQ_T_BF16) == align
    assert call(done=GOOD, done_token=100) == bad and call(done=GOOD, done_token=-1) == bad


@pytest.mark.parametrize("damp", [False, True])
def test_reorder_refusals(ssq, damp):
    cfg = ssq.DampConfig(2, 8, 4, 16, 64, 1, 16) if damp else config(ssq)
    f = ssq.raw().ssq_damp_pool_reorder if damp else ssq.raw().ssq_pool_reorder

    def call(pool=GOOD, slots=None, batch=2, beams=4, parent=GOOD, layer0=0, nl=2):
        return f(cfg.ref, P(pool), P(slots), batch, beams, P(parent), layer0, nl, None)

    bad, align = ssq.SSQ_ERR_INVALID_ARG, ssq.SSQ_ERR_ALIGNMENT
    assert call(batch=0, parent=0) == ssq.SSQ_OK
    assert call(pool=0) == bad and call(pool=GOOD + 16) == align
    assert call(batch=-1) == bad
    assert call(beams=0) == bad and call(beams=65, batch=0) == ssq.SSQ_ERR_UNSUPPORTED
    assert call(batch=3) == bad                 # 12 beams, 8 slots
    assert call(parent=0) == bad and call(parent=GOOD + 2) == align
    assert call(slots=GOOD + 1) == align
    assert call(layer0=1) == bad and call(layer0=-1, nl=1) == bad and call(nl=0) == bad


def test_binding_refuses_before_the_library(ssq):
    """Types, devices and shapes that the C ABI cannot see."""
    import torch
    cfg = config(ssq)
    t = torch.zeros(4)
    with pytest.raises(TypeError):
        ssq.ssq_beam_select(t.int(), t)
    with pytest.raises(ValueError):
        ssq.ssq_beam_select(torch.zeros(1, 2, 3), torch.zeros(1, 2))        # not CUDA
    with pytest.raises(ValueError):
        ssq.ssq_pool_reorder(cfg, t, None, torch.zeros(2, 2), 0, 1)          # pool not CUDA
    with pytest.raises(ValueError):
        ssq.ssq_pool_reorder(cfg, t, None, t, 0, 1)                          # parent not 2-d
    assert ssq.alloc_prefill_workspace(cfg, 2, 16) is None
