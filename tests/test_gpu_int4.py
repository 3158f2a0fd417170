"""GPU parity of the INT4 KV cache, the read-back of quantised caches and
prefill on them.

Bit-exact: the codes and scales that an append, a decode or a prefill writes,
and the rows read back. Outputs: ``helpers.check_bf16_output`` against the
oracle's attention over the rows the cache stands for, lse within
``helpers.check_lse``.
"""

import math

import numpy as np
import pytest
import torch

import sink_augmented_gqa_b200 as sa
from oracle import attention as oatt
from oracle import fp8 as ofp8
from oracle import int4 as oint4
from oracle import kvcache as okv
from oracle import rope as orope
from oracle.bf16 import round_bf16
from sink_augmented_gqa_b200 import workloads as wl

from helpers import OracleOut, check_bf16_output, check_lse, oracle_tables, to64

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _tables(cfg, max_pos):
    y = cfg.yarn
    return sa.yarn_rope_tables(max_pos, cfg.d, y["theta"], y["scaling"], y["orig_ctx"], y["alpha"], y["beta"],
                               device=DEV)


def _special_rows(shape, seed, shift=0, nonfinite=False):
    """bf16 rows [B, T, n_kv, d]: zero rows, rows at 1e30, 1e-30 and 1e-37,
    rows of one element, of negative zeros, of equal magnitudes (ties of m and
    -m) and, with ``nonfinite``, infinities and NaNs among normal ones."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g, dtype=torch.float32)
    for t in range(shape[1]):
        kind = (t + shift) % 16
        if kind == 0:
            x[:, t] = 0.0
        elif kind == 1:
            x[:, t] *= 1e30
        elif kind == 2:
            x[:, t] *= 1e-30
        elif kind == 3:
            x[:, t] = 0.0
            x[:, t, :, 5] = -3.0
        elif kind == 4:
            x[:, t] = -0.0
            x[:, t, :, 0] = 1.0
        elif kind == 5:
            x[:, t] = torch.sign(x[:, t]) * 2.5
        elif kind == 6:
            x[:, t] *= 1e-37
        elif kind == 7 and nonfinite:
            x[:, t, :, 33] = math.inf
            x[:, t, 0, 7] = math.nan
    return x.to(torch.bfloat16)


def _check_codes(cache, start, stop, k_rows, v_rows, what):
    """Codes and scales of positions [start, stop) against the oracle's, of
    bf16 rows [B, T, n_kv, d] (fp64)."""
    for name, codes, scales, rows in (("K", cache.k_rows, cache.k_scales, k_rows), ("V", cache.v_rows, cache.v_scales, v_rows)):
        u, s = oint4.quantize_rows(rows)
        assert np.array_equal(oint4.unpack(codes(start, stop).cpu().numpy()), u), f"{what}: {name} codes differ"
        assert np.array_equal(to64(scales(start, stop)), s, equal_nan=True), f"{what}: {name} scales differ"


def _stands_for(fmt, rows):
    """fp64 rows that rows [.., d] read back as (bf16 values)."""
    if fmt == "int4":
        return oint4.stored_rows(rows)
    if fmt == "fp8":
        return round_bf16(ofp8.dequantize_rows(*ofp8.quantize_rows(rows)))
    return rows


def _cache(fmt, B, cap, n_kv, d, ring=0):
    """A cache with never-written rows that hold anything a buffer can (a ring
    cache must be zeroed first)."""
    c = sa.KVCache(B, cap, n_kv, d, device=DEV, ring=ring, fp8=fmt == "fp8", int4=fmt == "int4")
    if not ring and fmt != "bf16":
        c.k.fill_(0x7F)
        c.v.fill_(0xFF)
        c.k_scale.fill_(math.nan)
        c.v_scale.fill_(math.inf)
    return c


def _append(cache, k, v):
    step = cache.raw.cap if cache.raw.ring else max(1, k.shape[1])
    for s in range(0, k.shape[1], step):
        cache.append(k[:, s:s + step].to(DEV), v[:, s:s + step].to(DEV))


# --------------------------------------------------------------------------- write

@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("ring", [0, 128], ids=["linear", "ring"])
def test_append_bit_exact(cuda_device, d, ring):
    B, n_kv, T = 2, 3, 61
    cap = 384 if ring else 112
    k, v = _special_rows((B, T, n_kv, d), 1, nonfinite=True), _special_rows((B, T, n_kv, d), 2, 5, nonfinite=True)
    cache = _cache("int4", B, cap, n_kv, d, ring)
    cache.append(k.to(DEV), v.to(DEV))
    # a strided source: rows of a bf16 cache viewed as [B, T, n_kv, d]
    src = sa.KVCache(B, 64, n_kv, d, device=DEV)
    k2, v2 = _special_rows((B, 20, n_kv, d), 3), _special_rows((B, 20, n_kv, d), 4)
    src.append(k2.to(DEV), v2.to(DEV))
    cache.append(src.k_rows(0, 20), src.v_rows(0, 20))
    torch.cuda.synchronize()
    assert cache.offset == T + 20
    _check_codes(cache, 0, T, to64(k), to64(v), "append")
    _check_codes(cache, T, T + 20, to64(k2), to64(v2), "strided append")
    if not ring:   # rows behind the last: as they were
        assert (cache.k[:, :, T + 20:] == 0x7F).all() and (cache.v[:, :, T + 20:] == 0xFF).all()
        assert cache.k_scale[:, :, T + 20:].isnan().all() and cache.v_scale[:, :, T + 20:].isinf().all()


@pytest.mark.parametrize("T", [0, 1, 31, 32, 33, 257])
def test_append_lengths_and_fused_source(cuda_device, T):
    cfg = wl.scaled(wl.CONFIGS["tiny"], B=3, n_q=8, n_kv=2, d=64, fused_qkv=True)
    _, k, v = wl.qkv(cfg, T)
    cache = _cache("int4", 3, 272, 2, 64)
    x = torch.empty((3, T, 64 * 12), dtype=torch.bfloat16, device=DEV)   # the fused layout, on the device
    kd, vd = x[:, :, 512:640].unflatten(2, (2, 64)), x[:, :, 640:].unflatten(2, (2, 64))
    kd.copy_(k)
    vd.copy_(v)
    cache.append(kd, vd)
    assert cache.offset == T
    _check_codes(cache, 0, T, to64(k), to64(v), f"T={T}")


def test_append_every_significand(cuda_device):
    # every pair of significands of m and x, x of either sign in 6 binades, one row per m and binade
    rows = []
    for M in range(128, 256):
        for sign in (1, -1):
            for e in range(6):
                r = torch.zeros(128, 2)
                r[:, 0] = torch.arange(128, 256) * 2.0 ** -e
                r[:, 1] = -r[:, 0]
                r = r.flatten()[r.flatten().abs() <= M] * sign
                r = torch.cat([r, torch.zeros(-len(r) % 31)]).view(-1, 31)
                rows.append(torch.cat([torch.full((len(r), 1), float(M * sign)), r], 1))
    x = torch.cat(rows)
    x = torch.cat([x, torch.zeros(-len(x) % 2, 32)]).view(1, -1, 1, 64).to(torch.bfloat16)
    cache = sa.KVCache(1, (x.shape[1] + 15) // 16 * 16, 1, 64, device=DEV, int4=True)
    cache.append(x.to(DEV), -x.to(DEV))
    _check_codes(cache, 0, x.shape[1], to64(x), -to64(x), "significands")


# --------------------------------------------------------------------------- read

@pytest.mark.parametrize("fmt", ["int4", "fp8", "bf16"])
@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("ring", [0, 100], ids=["linear", "ring"])
def test_read_back(cuda_device, fmt, d, ring):
    B, n_kv, n = 2, 3, 500
    cap = 384 if ring else 512
    k, v = _special_rows((B, n, n_kv, d), 6), _special_rows((B, n, n_kv, d), 7, 5)
    cache = _cache(fmt, B, cap, n_kv, d, ring)
    _append(cache, k, v)
    wk, wv = _stands_for(fmt, to64(k)), _stands_for(fmt, to64(v))
    first = n - cap if ring else 0
    for start, stop in ((first, n), (n - 1, n), (first + 3, first + 40), (380, 390), (n, n)):
        gk, gv = cache.read(start, stop)
        assert gk.shape == (B, stop - start, n_kv, d)
        assert np.array_equal(to64(gk), wk[:, start:stop]) and np.array_equal(to64(gv), wv[:, start:stop])
    if ring:
        with pytest.raises(sa.SinkAttnError) as e:
            cache.read(first - 1, n)
        assert e.value.name == "SA_ERR_CAPACITY"
    # into views of a larger buffer, whose other elements stay as they were
    buf = torch.full((B, 50, 2 * n_kv + 1, d), 7.0, dtype=torch.bfloat16, device=DEV)
    cache.read(first + 9, first + 49, k_out=buf[:, 5:45, :n_kv], v_out=buf[:, 5:45, n_kv:2 * n_kv])
    assert np.array_equal(to64(buf[:, 5:45, :n_kv]), wk[:, first + 9:first + 49])
    assert np.array_equal(to64(buf[:, 5:45, n_kv:2 * n_kv]), wv[:, first + 9:first + 49])
    assert (buf[:, :5] == 7).all() and (buf[:, 45:] == 7).all() and (buf[:, :, 2 * n_kv:] == 7).all()


def test_read_back_nonfinite_and_requantise(cuda_device):
    k, v = _special_rows((1, 64, 2, 64), 8, nonfinite=True), _special_rows((1, 64, 2, 64), 9)
    cache = _cache("int4", 1, 64, 2, 64)
    _append(cache, k, v)
    gk, gv = cache.read()
    assert np.array_equal(to64(gk), oint4.stored_rows(to64(k)), equal_nan=True)
    other = _cache("int4", 1, 64, 2, 64)
    other.append(gk, gv)                       # what was read back quantises to the same codes
    assert torch.equal(other.k, cache.k) and torch.equal(other.v, cache.v)
    assert np.array_equal(to64(other.k_scale), to64(cache.k_scale), equal_nan=True)
    assert torch.equal(other.v_scale, cache.v_scale)


# --------------------------------------------------------------------------- attention

def _abs_values(fmt, V):
    """A bound on what the rounding of a key's weight does to each output
    element, for ``OracleOut``: |v|, and for INT4 2^-6 of the block's scale
    (the tensor core's truncated sums of 136 times a weight times its scale,
    136 2^-22 of it at most over the two products of 16 keys)."""
    a = np.abs(V)
    if fmt == "int4":
        s = np.nan_to_num(np.abs(oint4.quantize_rows(V)[1]))
        a = a + 2.0 ** -6 * np.repeat(s, oint4.BLOCK, axis=-1)
    return a


class _Oracle:
    """The fp64 model of a quantised cache and of calls on it."""

    def __init__(self, cfg, fmt, rows, tables):
        self.cfg, self.fmt, self.tables = cfg, fmt, tables
        self.cache = okv.KVCache(cfg.B, rows, cfg.n_kv, cfg.d)

    def append(self, k, v, read):
        """``read``: the rows as they read back (prefill, INT4), else what an FP8 decode attends."""
        if self.fmt == "fp8" and not read:
            st = lambda x: ofp8.dequantize_rows(*ofp8.quantize_rows(x))   # noqa: E731
        else:
            st = lambda x: _stands_for(self.fmt, x)                       # noqa: E731
        self.cache.append(st(k), st(v))

    def call(self, q, k, v, sinks, window, rope=True, read=True):
        off, (rc, rs) = self.cache.offset, self.tables
        q, k, v = to64(q), to64(k), to64(v)
        q_rot = orope.rotate_bsh(q, off, rc, rs) if rope else q
        k_rot = orope.rotate_bsh(k, off, rc, rs) if rope else k
        self.append(k_rot, v, read)
        s = None if sinks is None else to64(sinks)
        out, lse = oatt.sink_attention(q_rot, self.cache.K, self.cache.V, s, off, window, self.cfg.sm_scale)
        vabs, _ = oatt.sink_attention(q_rot, self.cache.K, _abs_values(self.fmt, self.cache.V), s, off, window,
                                      self.cfg.sm_scale)
        return OracleOut(out, vabs), lse, k_rot


def _setup(over, fmt, off, extra, ring_window=0, special=False, seed=0):
    cfg = wl.scaled(wl.CONFIGS["tiny"], sm_scale=1 / math.sqrt(over["d"]), seed=seed, **over)
    total = off + extra
    cos, sin = _tables(cfg, total + 1)
    cap = 768 if ring_window else (total + 15) // 16 * 16
    cache = _cache(fmt, cfg.B, cap, cfg.n_kv, cfg.d, ring_window)
    oracle = _Oracle(cfg, fmt, total + 1, oracle_tables(cfg, total + 1))
    if off:
        if special:
            kp, vp = (_special_rows((cfg.B, off, cfg.n_kv, cfg.d), i, sh) for i, sh in ((11, 0), (12, 3)))
        else:
            kp, vp = wl.prefilled_cache_rows(cfg, rows=off)
        _append(cache, kp, vp)
        oracle.append(to64(kp), to64(vp), True)
    return cfg, cache, oracle, cos, sin


def _decode(cfg, cache, oracle, cos, sin, window, sinks, step, ws, what, rope=True, check=check_bf16_output):
    q, k, v = wl.qkv(cfg, 1, step=step)
    pos = cache.offset
    out, lse = sa.attn_decode(cache, q.to(DEV), k.to(DEV), v.to(DEV), None if sinks is None else sinks.to(DEV),
                              window, cfg.sm_scale, cos, sin, rope_fused=rope, workspace=ws, return_lse=True)
    torch.cuda.synchronize()
    ref, ref_lse, k_rot = oracle.call(q, k, v, sinks, window, rope)
    check(out, ref, what)
    check_lse(lse, ref_lse, what)
    assert cache.offset == pos + 1
    _check_codes(cache, pos, pos + 1, k_rot, to64(v), what)


SHAPES = [dict(B=2, n_q=8, n_kv=2, d=64), dict(B=2, n_q=8, n_kv=4, d=96), dict(B=1, n_q=16, n_kv=2, d=128),
          dict(B=1, n_q=64, n_kv=8, d=64), dict(B=3, n_q=3, n_kv=3, d=64), dict(B=2, n_q=14, n_kv=2, d=96)]
IDS = ["d64", "d96", "d128", "gptoss", "mha", "seven"]


@pytest.mark.parametrize("over", SHAPES, ids=IDS)
@pytest.mark.parametrize("window", [0, 128], ids=["full", "band"])
@pytest.mark.parametrize("off", [0, 1, 37, 255, 256, 5000])
def test_decode_matches_oracle(cuda_device, over, window, off):
    cfg, cache, oracle, cos, sin = _setup(over, "int4", off, 4)
    ws = sa.decode_workspace(cfg.B, cfg.n_q, cfg.n_kv, cfg.d, device=DEV)
    sinks = wl.sinks(cfg)
    for step in range(2):
        _decode(cfg, cache, oracle, cos, sin, window, sinks, step + 1, ws, f"int4 decode {step}")
    _decode(cfg, cache, oracle, cos, sin, window, None, 3, ws, "int4 decode without sinks, rotated inputs", rope=False)
    assert torch.count_nonzero(ws[: 8 * cfg.B * cfg.n_kv]) == 0   # tickets and stage counters


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("window", [1, 128, 300])
def test_ring_decode_matches_oracle(cuda_device, d, window):
    cfg, cache, oracle, cos, sin = _setup(dict(B=2, n_q=8, n_kv=2, d=d), "int4", 1700, 12, ring_window=window)
    sinks = wl.sinks(cfg)
    ws = sa.decode_workspace(cfg.B, cfg.n_q, cfg.n_kv, cfg.d, device=DEV)
    for step in range(3):
        _decode(cfg, cache, oracle, cos, sin, window, sinks, step, ws, f"ring decode {step}")
    snap, osnap = cache.snapshot(), oracle.cache.snapshot()
    _decode(cfg, cache, oracle, cos, sin, window, sinks, 50, ws, "ring decode, to be undone")
    cache.restore(snap)
    oracle.cache.restore(osnap)
    _decode(cfg, cache, oracle, cos, sin, window, sinks, 51, ws, "ring decode after restore")


def _check_scaled(gpu, ref, what):
    """The bf16 bar (max 1e-2, mean 1e-3) in units of each output row's
    magnitude max(1, max_d |ref|): rows scaled by up to 1e30 make absolute
    bounds meaningless."""
    g, r = to64(gpu), np.asarray(ref, dtype=np.float64)
    assert np.all(np.isfinite(g)), f"{what}: non-finite output"
    err = np.abs(g - r) / np.maximum(1.0, np.abs(r).max(axis=-1, keepdims=True))
    assert err.max() <= 1e-2 and err.mean() <= 1e-3, f"{what}: max {err.max()} mean {err.mean()}"


@pytest.mark.parametrize("over", [dict(B=40, n_q=16, n_kv=8, d=64), dict(B=37, n_q=35, n_kv=5, d=96),
                                  dict(B=75, n_q=8, n_kv=4, d=128), dict(B=10, n_q=64, n_kv=8, d=64)],
                         ids=["d64", "d96", "d128", "gptoss"])
@pytest.mark.parametrize("window", [0, 200], ids=["full", "band"])
@pytest.mark.parametrize("off", [0, 130, 777, 2048, 6001])
def test_decode_of_many_pairs(cuda_device, over, window, off):
    # more (sequence, KV head) pairs than SMs, or long ones that do not divide
    # into them: CTAs end one pair, span some and begin another
    if off == 6001 and over["B"] != 10:
        off = 1200
    cfg, cache, oracle, cos, sin = _setup(over, "int4", off, 2)
    ws = sa.decode_workspace(cfg.B, cfg.n_q, cfg.n_kv, cfg.d, device=DEV)
    sinks = wl.sinks(cfg)
    for step in range(2):
        _decode(cfg, cache, oracle, cos, sin, window, sinks, step + 1, ws, f"int4 decode {step}")
    assert torch.count_nonzero(ws[: 8 * cfg.B * cfg.n_kv]) == 0


def test_decode_of_many_pairs_on_a_ring(cuda_device):
    cfg, cache, oracle, cos, sin = _setup(dict(B=40, n_q=16, n_kv=8, d=64), "int4", 1200, 4, ring_window=300)
    sinks = wl.sinks(cfg)
    for step in range(3):
        _decode(cfg, cache, oracle, cos, sin, 300, sinks, step + 1, None, f"ring decode {step}")


def test_decode_graphs_that_share_a_workspace(cuda_device):
    # two layers' calls captured into two graphs over one workspace, replayed in turn
    over = dict(B=2, n_q=16, n_kv=2, d=64)
    ws = sa.decode_workspace(2, 16, 2, 64, device=DEV)
    made = []
    stream = torch.cuda.Stream()
    for window in (0, 128):
        cfg, cache, oracle, cos, sin = _setup(over, "int4", 2500, 1, seed=window)
        q, k, v = wl.qkv(cfg, 1, step=1)
        ref, ref_lse, _ = oracle.call(q, k, v, None, window)
        q, k, v = (t.to(DEV) for t in (q, k, v))
        out = torch.empty_like(q)
        stream.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            sa.attn_decode(cache, q, k, v, None, window, cfg.sm_scale, cos, sin, workspace=ws, out=out)
        made.append((graph, out, ref, cache, q, k, v, cos, sin))
    for _ in range(3):
        for graph, out, *_ in made:
            out.zero_()
            graph.replay()
        torch.cuda.synchronize()
        for _, out, ref, *_ in made:
            check_bf16_output(out, ref, "replayed in turn")


def test_decode_static_refuses_what_its_scratch_cannot_hold(cuda_device):
    # 240 pairs in equal shares: a record of 4 KB for each of the CTAs and borders, over a MiB
    cfg, cache, oracle, cos, sin = _setup(dict(B=30, n_q=64, n_kv=8, d=128), "int4", 600, 2)
    q, k, v = (t.to(DEV) for t in wl.qkv(cfg, 1, step=1))
    with pytest.raises(sa.SinkAttnError) as e:
        sa.attn_decode_static(cache, q, k, v, None, 0, cfg.sm_scale, cos, sin)
    assert e.value.name == "SA_ERR_WORKSPACE" and cache.offset == 600
    ws = sa.decode_workspace(cfg.B, cfg.n_q, cfg.n_kv, cfg.d, device=DEV)
    with pytest.raises(sa.SinkAttnError) as e:
        sa.attn_decode(cache, q, k, v, None, 0, cfg.sm_scale, cos, sin, workspace=ws[:1 << 20])
    assert e.value.name == "SA_ERR_WORKSPACE" and cache.offset == 600
    _decode(cfg, cache, oracle, cos, sin, 0, None, 1, ws, "with a workspace")


@pytest.mark.parametrize("over,off", [(dict(B=2, n_q=8, n_kv=2, d=64), 3000), (dict(B=40, n_q=16, n_kv=8, d=64), 700),
                                      (dict(B=1, n_q=8, n_kv=1, d=64), 40000)])
def test_zero_wait_limit_is_right_or_reported(cuda_device, over, off):
    cfg, cache, oracle, cos, sin = _setup(over, "int4", off, 40)
    ws = sa.decode_workspace(cfg.B, cfg.n_q, cfg.n_kv, cfg.d, device=DEV)
    q, k, v = (t.to(DEV) for t in wl.qkv(cfg, 1, step=1))
    q2, k2, v2 = (t.to(DEV) for t in wl.qkv(cfg, 20, step=2))
    snap, osnap = cache.snapshot(), oracle.cache.snapshot()
    ref = oracle.call(q, k, v, None, 0)[0]
    oracle.cache.restore(osnap)
    torch.cuda.synchronize()
    assert sa.device_status() == "SA_OK"
    sa.set_wait_limit(0)
    try:
        out = sa.attn_decode(cache, q, k, v, None, 0, cfg.sm_scale, cos, sin, workspace=ws)
        torch.cuda.synchronize()
        decode_status = sa.device_status()
        sa.attn_prefill_quant(cache, q2, k2, v2, None, 0, cfg.sm_scale, cos, sin)
        torch.cuda.synchronize()
        prefill_status = sa.device_status()
        print("zero wait limit:", decode_status, prefill_status)
    finally:
        sa.set_wait_limit(2_000_000_000)
    # A wait asks at least once, and the hardware holds that for a moment: what
    # arrives meanwhile is no timeout, and the answer is then right.
    assert {decode_status, prefill_status} <= {"SA_OK", "SA_ERR_TIMEOUT"}
    if decode_status == "SA_OK":
        check_bf16_output(out, ref, "without a limit")
    # the tickets are where they were, and the calls after it are right
    assert torch.count_nonzero(ws[: 8 * cfg.B * cfg.n_kv]) == 0
    cache.restore(snap)
    for step in range(2):
        _decode(cfg, cache, oracle, cos, sin, 0, None, step + 1, ws, "after timeout")
    out = sa.attn_prefill_quant(cache, q2, k2, v2, None, 0, cfg.sm_scale, cos, sin)
    check_bf16_output(out, oracle.call(q2, k2, v2, None, 0)[0], "prefill after timeout")
    assert sa.device_status() == "SA_OK"


@pytest.mark.parametrize("window", [0, 128], ids=["full", "band"])
def test_decode_mixed_magnitude_rows(cuda_device, window):
    # K of normal size, V rows from 1e-37 to 1e30 next to one another
    cfg, cache, oracle, cos, sin = _setup(dict(B=1, n_q=8, n_kv=2, d=64), "int4", 0, 306)
    kp, _ = wl.prefilled_cache_rows(cfg, rows=300)
    vp = _special_rows((1, 300, 2, 64), 12, 3)
    _append(cache, kp, vp)
    oracle.append(to64(kp), to64(vp), True)
    for step in range(2):
        _decode(cfg, cache, oracle, cos, sin, window, wl.sinks(cfg), step, None, "mixed magnitudes", check=_check_scaled)


def test_decode_nonfinite_rows_outside_the_band_do_not_matter(cuda_device):
    over = dict(B=1, n_q=8, n_kv=2, d=64)
    cfg, cache, oracle, cos, sin = _setup(over, "int4", 0, 306)
    kp, vp = wl.prefilled_cache_rows(cfg, rows=300)
    bad_k, bad_v = kp.clone(), vp.clone()
    bad_k[:, :172], bad_v[:, :172] = math.nan, math.inf      # row 172 is outside of 300's band of 128
    _append(cache, bad_k, bad_v)
    oracle.append(to64(kp), to64(vp), True)
    _decode(cfg, cache, oracle, cos, sin, 128, wl.sinks(cfg), 1, None, "NaN rows outside the band")
    # inside it they reach the output, as they do in a bf16 cache
    q, k, v = (t.to(DEV) for t in wl.qkv(cfg, 1, step=2))
    out = sa.attn_decode(cache, q, k, v, wl.sinks(cfg).to(DEV), 0, cfg.sm_scale, cos, sin)
    assert out.isnan().all()


def test_decode_zero_queries_and_extreme_sinks(cuda_device):
    cfg, cache, oracle, cos, sin = _setup(dict(B=1, n_q=8, n_kv=2, d=64), "int4", 600, 4)
    sinks = torch.tensor([-math.inf, -100.0, 0.0, 100.0, 1.0, 2.0, 3.0, 4.0])
    q, k, v = wl.qkv(cfg, 1, step=1)
    q[:, :, 5] = 0
    out, lse = sa.attn_decode(cache, q.to(DEV), k.to(DEV), v.to(DEV), sinks.to(DEV), 0, cfg.sm_scale, cos, sin,
                              return_lse=True)
    ref, ref_lse, _ = oracle.call(q, k, v, sinks, 0)
    check_bf16_output(out, ref, "extreme sinks")
    check_lse(lse, ref_lse, "extreme sinks")


def test_decode_static_graph_and_streams(cuda_device):
    over = dict(B=2, n_q=16, n_kv=2, d=64)
    cfg, cache, oracle, cos, sin = _setup(over, "int4", 3000, 40)
    sinks = wl.sinks(cfg).to(DEV)
    q, k, v = (t.to(DEV) for t in wl.qkv(cfg, 1, step=1))
    snap = cache.snapshot()
    ws = sa.decode_workspace(cfg.B, cfg.n_q, cfg.n_kv, cfg.d, device=DEV)
    call = lambda f, w: f(cache, q, k, v, sinks, 0, cfg.sm_scale, cos, sin, return_lse=True, **w)   # noqa: E731
    ref, ref_lse, _ = oracle.call(q, k, v, sinks, 0)
    out, lse = call(sa.attn_decode_static, {})
    check_bf16_output(out, ref, "static scratch")
    check_lse(lse, ref_lse, "static scratch")
    # captured, and replayed with other inputs in the same buffers
    cache.restore(snap)
    stream = torch.cuda.Stream()
    out2, lse2 = torch.empty_like(out), torch.empty_like(lse)
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        call(sa.attn_decode, dict(workspace=ws, out=out2, lse=lse2))
    graph.replay()
    torch.cuda.synchronize()
    check_bf16_output(out2, ref, "replayed")
    check_lse(lse2, ref_lse, "replayed")
    q2, k2, v2 = wl.qkv(cfg, 1, step=2)
    for t, n in ((q, q2), (k, k2), (v, v2)):
        t.copy_(n)
    graph.replay()
    torch.cuda.synchronize()
    oracle2 = _Oracle(cfg, "int4", 3004, oracle.tables)
    kp, vp = wl.prefilled_cache_rows(cfg, rows=3000)
    oracle2.append(to64(kp), to64(vp), True)
    ref2, ref_lse2, _ = oracle2.call(q2, k2, v2, sinks, 0)
    check_bf16_output(out2, ref2, "replayed with other inputs")
    check_lse(lse2, ref_lse2, "replayed with other inputs")
    # two caches on two streams at a time, a workspace each
    outs = []
    caches = [_cache("int4", 2, 3008, 2, 64) for _ in range(2)]
    for c in caches:
        _append(c, kp, vp)
    torch.cuda.synchronize()
    for c in caches:
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            w = sa.decode_workspace(cfg.B, cfg.n_q, cfg.n_kv, cfg.d, device=DEV)
            outs.append(sa.attn_decode(c, q, k, v, sinks, 0, cfg.sm_scale, cos, sin, workspace=w))
    torch.cuda.synchronize()
    for o in outs:
        check_bf16_output(o, ref2, "two streams")


@pytest.mark.parametrize("window", [0, 128], ids=["full", "band"])
def test_decode_full_size_long_context(cuda_device, window):
    # 131,071 cached positions, 64 query heads over 8 KV heads: sampled heads
    cfg = wl.CONFIGS["long_decode"]
    off = cfg.offset
    cos, sin = _tables(cfg, off + 2)
    rc, rs = oracle_tables(cfg, off + 2)
    sinks = wl.sinks(cfg)
    kp, vp = wl.prefilled_cache_rows(cfg, device=DEV)
    cache = _cache("int4", cfg.B, off + 17, cfg.n_kv, cfg.d)
    cache.append(kp, vp)
    q, k, v = wl.qkv(cfg, 1, step=1, device=DEV)
    out, lse = sa.attn_decode(cache, q, k, v, sinks.to(DEV), window, cfg.sm_scale, cos, sin, return_lse=True)
    torch.cuda.synchronize()
    lo = max(0, off + 1 - window) if window else 0
    for h in (0, 9, 63):
        g = h // cfg.q_mult
        k_new = orope.rotate_bsh(to64(k[:, :, g:g + 1]), off, rc, rs)[0, 0]
        K = oint4.stored_rows(np.concatenate([to64(kp[0, lo:, g]), k_new]))
        V = oint4.stored_rows(np.concatenate([to64(vp[0, lo:, g]), to64(v[0, 0, g:g + 1])]))
        qr = orope.rotate_bsh(to64(q[:, :, h:h + 1]), off, rc, rs)
        args = (to64(sinks[h:h + 1]), off - lo, window, cfg.sm_scale)
        o, ref_lse = oatt.sink_attention(qr, K[None, :, None], V[None, :, None], *args)
        a, _ = oatt.sink_attention(qr, K[None, :, None], _abs_values("int4", V)[None, :, None], *args)
        check_bf16_output(out[:, :, h:h + 1], OracleOut(o, a), f"long decode h{h}")
        check_lse(lse[0, h, 0], np.array(ref_lse[0, 0, 0]), f"long decode h{h}")


# --------------------------------------------------------------------------- prefill on quantised caches

@pytest.mark.parametrize("fmt", ["int4", "fp8"])
@pytest.mark.parametrize("over", [SHAPES[i] for i in (0, 1, 2, 4)], ids=[IDS[i] for i in (0, 1, 2, 4)])
@pytest.mark.parametrize("window", [0, 128], ids=["full", "band"])
@pytest.mark.parametrize("off,T", [(0, 1), (0, 129), (300, 77), (301, 1)])
def test_prefill_quant_matches_oracle(cuda_device, fmt, over, window, off, T):
    cfg, cache, oracle, cos, sin = _setup(over, fmt, off, 2 * T)
    sinks = wl.sinks(cfg)
    for step, rope in ((1, True), (2, False)):
        q, k, v = wl.qkv(cfg, T, step=step)
        s = sinks if rope else None
        pos = cache.offset
        out, lse = sa.attn_prefill_quant(cache, q.to(DEV), k.to(DEV), v.to(DEV), None if s is None else s.to(DEV),
                                         window, cfg.sm_scale, cos, sin, rope_fused=rope, return_lse=True)
        torch.cuda.synchronize()
        ref, ref_lse, k_rot = oracle.call(q, k, v, s, window, rope)
        what = f"{fmt} prefill {step}"
        check_bf16_output(out, ref, what)
        check_lse(lse, ref_lse, what)
        assert cache.offset == pos + T
        gk, gv = cache.read(pos, pos + T)
        assert np.array_equal(to64(gk), _stands_for(fmt, k_rot)) and np.array_equal(to64(gv), _stands_for(fmt, to64(v)))


@pytest.mark.parametrize("over", [dict(B=1, n_q=8, n_kv=1, d=64), dict(B=2, n_q=6, n_kv=2, d=96),
                                  dict(B=1, n_q=14, n_kv=2, d=128), dict(B=1, n_q=16, n_kv=1, d=64),
                                  dict(B=2, n_q=20, n_kv=1, d=64), dict(B=3, n_q=5, n_kv=1, d=128)],
                         ids=["8x", "3x", "7x", "16x", "20x", "5x"])
@pytest.mark.parametrize("off,T,window", [(4000, 1, 0), (4000, 2, 0), (1500, 17, 0), (5003, 77, 0), (900, 300, 0),
                                          (4000, 40, 1500), (3000, 513, 700), (0, 1025, 0)])
def test_prefill_quant_of_few_rows_behind_many(cuda_device, over, off, T, window):
    # heads of a KV group side by side in a tile, key tiles cut into parts: rows
    # whose part holds no key, parts without tiles, ends inside a tile
    cfg, cache, oracle, cos, sin = _setup(over, "int4", off, T)
    sinks = wl.sinks(cfg) if T % 2 else None
    q, k, v = wl.qkv(cfg, T, step=1)
    nb = sa.prefill_quant_workspace(cache, T, window).numel()
    ws = torch.full((nb + 256,), 0xFF, dtype=torch.uint8, device=DEV)   # NaNs, whatever is read unwritten
    out, lse = sa.attn_prefill_quant(cache, q.to(DEV), k.to(DEV), v.to(DEV), None if sinks is None else sinks.to(DEV),
                                     window, cfg.sm_scale, cos, sin, workspace=ws, return_lse=True)
    torch.cuda.synchronize()
    ref, ref_lse, _ = oracle.call(q, k, v, sinks, window)
    check_bf16_output(out, ref, "prefill in parts")
    check_lse(lse, ref_lse, "prefill in parts")
    assert (ws[nb:] == 0xFF).all()


@pytest.mark.parametrize("fmt", ["int4", "fp8"])
def test_prefill_quant_in_parts_in_graphs_and_streams(cuda_device, fmt):
    # two layers' calls captured over one workspace and replayed in turn, `out`
    # being `q` in the second; then both at a time on streams of their own
    over, off, T = dict(B=1, n_q=16, n_kv=2, d=64), 4000, 20
    stream, made, ws = torch.cuda.Stream(), [], None
    for i, window in enumerate((0, 1000)):
        cfg, cache, oracle, cos, sin = _setup(over, fmt, off, T, seed=i)
        q, k, v = wl.qkv(cfg, T, step=1)
        ref, ref_lse, _ = oracle.call(q, k, v, None, window)
        q, k, v = (t.to(DEV) for t in (q, k, v))
        q0, out, lse = q.clone(), q if i else torch.empty_like(q), torch.empty(1, 16, T, device=DEV)
        if ws is None:
            ws = sa.prefill_quant_workspace(cache, T)
        snap = cache.snapshot()

        def call(w, cache=cache, snap=snap, q=q, k=k, v=v, window=window, cos=cos, sin=sin, out=out, lse=lse):
            cache.restore(snap)
            sa.attn_prefill_quant(cache, q, k, v, None, window, cfg.sm_scale, cos, sin, workspace=w, out=out,
                                  return_lse=True, lse=lse)

        stream.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            call(ws)
        made.append((graph, call, q, q0, out, lse, ref, ref_lse, cache))

    def check(what):
        torch.cuda.synchronize()
        for _, _, _, _, out, lse, ref, ref_lse, _ in made:
            check_bf16_output(out, ref, what)
            check_lse(lse, ref_lse, what)

    for _ in range(2):
        for graph, _, q, q0, *_ in made:
            q.copy_(q0)
            graph.replay()
        check("replayed in turn")
    for _, call, q, q0, *_ in made:
        q.copy_(q0)
    torch.cuda.synchronize()
    for (_, call, *_), st in zip(made, (torch.cuda.Stream(), torch.cuda.Stream())):
        with torch.cuda.stream(st):
            call(torch.empty_like(ws))
    check("two streams")


@pytest.mark.parametrize("fmt", ["int4", "fp8"])
def test_prefill_quant_on_a_ring(cuda_device, fmt):
    cfg, cache, oracle, cos, sin = _setup(dict(B=2, n_q=8, n_kv=2, d=64), fmt, 1000, 700, ring_window=128)
    sinks = wl.sinks(cfg)
    for step, T in ((1, 333), (2, 40)):           # the first wraps the ring
        q, k, v = wl.qkv(cfg, T, step=step)
        out, lse = sa.attn_prefill_quant(cache, q.to(DEV), k.to(DEV), v.to(DEV), sinks.to(DEV), 128, cfg.sm_scale,
                                         cos, sin, return_lse=True)
        ref, ref_lse, _ = oracle.call(q, k, v, sinks, 128)
        check_bf16_output(out, ref, f"{fmt} ring prefill")
        check_lse(lse, ref_lse, f"{fmt} ring prefill")
    with pytest.raises(sa.SinkAttnError) as e:    # more rows than the ring can hold beside the band
        q, k, v = (t.to(DEV) for t in wl.qkv(cfg, 700, step=3))
        sa.attn_prefill_quant(cache, q, k, v, None, 128, cfg.sm_scale, cos, sin)
    assert e.value.name in ("SA_ERR_CAPACITY",) and cache.offset == 1373


def test_prefill_quant_in_place_workspace_and_graph(cuda_device):
    cfg, cache, oracle, cos, sin = _setup(dict(B=2, n_q=8, n_kv=2, d=64), "int4", 200, 200)
    sinks = wl.sinks(cfg).to(DEV)
    q, k, v = (t.to(DEV) for t in wl.qkv(cfg, 70, step=1))
    q0 = q.clone()
    snap = cache.snapshot()
    ref, ref_lse, _ = oracle.call(q, k, v, sinks, 0)
    nb = sa.prefill_quant_workspace(cache, 70).numel()
    ws = torch.full((nb + 256,), 0xAB, dtype=torch.uint8, device=DEV)
    out, lse = sa.attn_prefill_quant(cache, q, k, v, sinks, 0, cfg.sm_scale, cos, sin, workspace=ws, out=q,
                                     return_lse=True)   # `out` is `q` itself
    torch.cuda.synchronize()
    check_bf16_output(out, ref, "in place")
    assert (ws[nb:] == 0xAB).all()
    cache.restore(snap)
    q.copy_(q0)
    out2 = torch.empty_like(q)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        sa.attn_prefill_quant(cache, q, k, v, sinks, 0, cfg.sm_scale, cos, sin, workspace=ws, out=out2)
    for _ in range(2):
        out2.zero_()
        graph.replay()
        torch.cuda.synchronize()
        check_bf16_output(out2, ref, "replayed")


def test_a_conversation_on_quantised_caches(cuda_device):
    """Prefill, decode, roll back, decode on another branch, the next turn's
    prefill, then the rows read back and gone on with in bf16: a band layer's
    ring and a full layer, as they alternate in a model."""
    over = dict(B=2, n_q=16, n_kv=2, d=64)
    for fmt, window, ring in (("int4", 128, 128), ("int4", 0, 0), ("fp8", 0, 0)):
        cfg, cache, oracle, cos, sin = _setup(over, fmt, 0, 400, ring_window=ring)
        sinks = wl.sinks(cfg)
        ws = sa.decode_workspace(cfg.B, cfg.n_q, cfg.n_kv, cfg.d, device=DEV)

        def turn(T, step):
            q, k, v = wl.qkv(cfg, T, step=step)
            if T > 1:
                out, lse = sa.attn_prefill_quant(cache, q.to(DEV), k.to(DEV), v.to(DEV), sinks.to(DEV), window,
                                                 cfg.sm_scale, cos, sin, return_lse=True)
            else:
                out, lse = sa.attn_decode(cache, q.to(DEV), k.to(DEV), v.to(DEV), sinks.to(DEV), window,
                                          cfg.sm_scale, cos, sin, workspace=ws, return_lse=True)
            ref, ref_lse, _ = oracle.call(q, k, v, sinks, window, read=True)
            check_bf16_output(out, ref, f"{fmt} turn of {T}")
            # an FP8 decode attends code * scale, the model here the rows as they read back: 2^-9 of
            # each key apart, which moves a score by up to 2^-9 sum |q k| / 8
            check_lse(lse, ref_lse, f"{fmt} turn of {T}", **({"atol": 2e-2} if fmt == "fp8" else {}))

        turn(150, 1)
        for i in range(3):
            turn(1, 10 + i)
        snap, osnap = cache.snapshot(), oracle.cache.snapshot()
        for i in range(2):
            turn(1, 20 + i)
        cache.restore(snap)
        oracle.cache.restore(osnap)
        turn(1, 30)
        turn(45, 2)
        n = cache.offset
        kb, vb = cache.read(0, n)
        plain = sa.KVCache(cfg.B, n + 16, cfg.n_kv, cfg.d, device=DEV)
        plain.append(kb, vb)
        assert np.array_equal(to64(kb), oracle.cache.K[:, :n]) and np.array_equal(to64(vb), oracle.cache.V[:, :n])
        q, k, v = wl.qkv(cfg, 1, step=40)
        out = sa.attn_decode(plain, q.to(DEV), k.to(DEV), v.to(DEV), sinks.to(DEV), window, cfg.sm_scale, cos, sin)
        if fmt == "int4":
            # the bf16 cache's new row is not quantised: the same call on a model of that
            oracle.fmt = "bf16"
            ref, _, _ = oracle.call(q, k, v, sinks, window)
            check_bf16_output(out, ref, "gone on with in bf16")
