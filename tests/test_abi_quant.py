"""CPU-only checks of the quantised-cache entry points: the INT4 cache, the
read-back and prefill on quantised caches reject bad arguments on the host
before any launch, and leave the cache's state alone."""

import ctypes
from types import SimpleNamespace

import pytest
import torch

from sink_augmented_gqa_b200 import build as sbuild
from sink_augmented_gqa_b200 import sinkattn as S

CODE = {v: k for k, v in S.STATUS.items()}
OK, INVALID, SHAPE, CAPACITY = (CODE["SA_" + n] for n in ("OK", "ERR_INVALID_ARG", "ERR_SHAPE", "ERR_CAPACITY"))
# 16-byte aligned addresses that no host check dereferences
K, V, KS, VS, OUT = 0x10000, 0x20000, 0x30000, 0x40000, 0x50000
STR = S._I64x3(4096, 256, 64)


@pytest.fixture(scope="module")
def L():
    sbuild.build()
    return S.lib()


def _init(L, name="int4", k=K, v=V, ks=KS, vs=VS, B=1, cap=96, n_kv=2, d=64, window=0):
    c = S._KVCache()
    st = getattr(L, "sa_kv_cache_init_" + name)(ctypes.byref(c), ctypes.c_void_p(k), ctypes.c_void_p(v),
                                                ctypes.c_void_p(ks), ctypes.c_void_p(vs), B, cap, n_kv, d, window)
    return c, st


def test_int4_cache_host_rules(L):
    c, st = _init(L)
    assert st == OK and c.kv_dtype == S.KV_INT4 and (c.k_scale, c.v_scale) == (KS, VS) and c.ring == 0
    assert L.sa_kv_cache_init_int4(None, K, V, KS, VS, 1, 96, 2, 64, 0) == INVALID
    for over, want in ((dict(ks=0), INVALID), (dict(vs=VS + 8), INVALID), (dict(k=0), INVALID), (dict(v=V + 4), INVALID),
                       (dict(window=-1), INVALID), (dict(B=0), INVALID), (dict(n_kv=0), INVALID),
                       (dict(cap=100), SHAPE), (dict(d=32), SHAPE), (dict(d=80), SHAPE),
                       (dict(cap=400, window=128), SHAPE), (dict(cap=384, window=385), SHAPE),
                       (dict(cap=768, window=128), OK), (dict(d=96), OK), (dict(d=128), OK)):
        assert _init(L, **over)[1] == want, over


def _read(L, c, start, T, k=OUT, v=OUT + 0x10000, ks=STR, vs=STR):
    return L.sa_kv_read(ctypes.byref(c), start, T, ctypes.c_void_p(k), ks, ctypes.c_void_p(v), vs, None)


@pytest.mark.parametrize("name", ["int4", "fp8"])
def test_read_refusals(L, name):
    c, _ = _init(L, name)
    c.offset = c.high_water = 40
    assert _read(L, c, 41, 0) == CAPACITY and _read(L, c, 40, 0) == OK and _read(L, c, 0, 0) == OK
    assert _read(L, c, 0, 41) == CAPACITY and _read(L, c, 39, 2) == CAPACITY
    assert _read(L, c, 2 ** 62, 1) == CAPACITY
    assert _read(L, c, -1, 4) == INVALID and _read(L, c, 0, -1) == INVALID
    assert _read(L, c, 0, 4, k=0) == INVALID and _read(L, c, 0, 4, v=OUT + 2) == INVALID
    assert _read(L, c, 0, 4, ks=S._I64x3(4096, 256, 60)) == INVALID
    assert _read(L, c, 0, 4, vs=S._I64x3(-8, 256, 64)) == INVALID
    assert c.offset == 40
    c.kv_dtype = 7
    assert _read(L, c, 0, 4) == INVALID


def test_ring_read_range(L):
    c, _ = _init(L, cap=384, window=128)
    c.offset = c.high_water = 1000
    assert _read(L, c, 615, 0) == CAPACITY and _read(L, c, 616, 0) == OK     # the last 384 positions
    c.offset = 900                                                             # restored: rows up to 1000 were written
    assert _read(L, c, 615, 1) == CAPACITY and _read(L, c, 616, 285) == CAPACITY
    assert _read(L, c, 616, 0) == OK


def _args(offset=0, T=4, n_q=4, B=1, window=0):
    a = S._AttnArgs()
    for f in ("q", "k", "v", "out"):
        setattr(a, f, OUT)
    for f in ("q_strides", "k_strides", "v_strides", "out_strides"):
        setattr(a, f, S._I64x3(4096, 256, 64))
    a.B, a.T, a.n_q, a.offset, a.window, a.sm_scale = B, T, n_q, offset, window, 0.125
    a.rope_fused = 0
    return a


@pytest.mark.parametrize("name", ["int4", "fp8"])
def test_prefill_quant_refusals(L, name):
    c, _ = _init(L, name)
    need = L.sa_attn_prefill_quant_workspace_size(ctypes.byref(c), 4, 0)
    ws = ctypes.c_void_p(0x100000)

    def call(a, cache=c, ws=ws, nb=need):
        return L.sa_attn_prefill_quant(ctypes.byref(cache), ctypes.byref(a), ws, nb, None)

    assert call(_args(T=0)) == OK                                   # no-op
    assert call(_args(), ws=None) == CODE["SA_ERR_WORKSPACE"]
    assert call(_args(), nb=need - 1) == CODE["SA_ERR_WORKSPACE"]
    assert call(_args(), ws=ctypes.c_void_p(0x100008)) == CODE["SA_ERR_WORKSPACE"]
    assert call(_args(offset=3)) == CODE["SA_ERR_OFFSET_MISMATCH"]
    assert call(_args(T=97)) == CAPACITY
    assert call(_args(n_q=5)) == SHAPE
    assert call(_args(B=2)) == INVALID
    a = _args()
    a.rope_fused = 1                                                # no tables
    assert call(a) == INVALID
    a = _args()
    a.sm_scale = float("inf")
    assert call(a) == INVALID
    # the plain prefill still refuses quantised caches, this one bf16 ones
    assert L.sa_attn_prefill(ctypes.byref(c), ctypes.byref(_args()), None) == CODE["SA_ERR_UNSUPPORTED"]
    b = S._KVCache()
    assert L.sa_kv_cache_init(ctypes.byref(b), ctypes.c_void_p(K), ctypes.c_void_p(V), 1, 96, 2, 64) == OK
    assert call(_args(), cache=b) == CODE["SA_ERR_UNSUPPORTED"]
    assert c.offset == 0 and b.offset == 0


def test_prefill_quant_workspace_size(L):
    c, _ = _init(L, B=3, cap=4800, n_kv=2, d=96)

    def size(T, window=0):
        return L.sa_attn_prefill_quant_workspace_size(ctypes.byref(c), T, window)

    assert size(0) == 0 and size(-1) == 0 and L.sa_attn_prefill_quant_workspace_size(None, 4, 0) == 0
    row = 2 * 3 * 2 * 96 * 2
    assert size(5) == 5 * row
    c.offset = c.high_water = 1000
    parts = 320 * 256 * (96 + 2) * 4       # 4 key tiles of 96 and more may be cut into parts
    assert size(5) == 1005 * row + parts and size(5, 128) == 132 * row + parts and size(5, 1) == 5 * row
    assert size(5, 5000) == 1005 * row + parts
    assert size(5, 33) == 37 * row and size(5, 34) == 38 * row + parts    # 288 and 289 keys


def test_int4_decode_refusals(L):
    c, _ = _init(L)
    call = lambda a: L.sa_attn_decode(ctypes.byref(c), ctypes.byref(a), None, 0, None)   # noqa: E731
    assert call(_args(T=2)) == INVALID
    assert call(_args(T=1, n_q=18)) == SHAPE                        # more than 8 query heads per KV head
    assert call(_args(T=1, offset=1)) == CODE["SA_ERR_OFFSET_MISMATCH"]
    assert c.offset == 0


def test_binding_checks():
    with pytest.raises(ValueError):
        S.KVCache(1, 96, 2, 64, device="cpu", fp8=True, int4=True)
    c = S.KVCache(1, 96, 2, 64, device="cpu", int4=True)            # host rules only: nothing is launched
    assert c.k.shape == (1, 2, 96, 32) and c.k_scale.shape == (1, 2, 96, 2)
    with pytest.raises(ValueError):
        c.read(5, 4)
    with pytest.raises(AssertionError):
        S.KVCache(1, 96, 2, 64, device="cpu", int4=True, k_scale=c.k_scale.float())


def test_binding_refuses_other_shapes_and_devices(monkeypatch):
    """What the C side cannot see from pointers and strides: shapes that do
    not fit the cache, and tensors of a device that is not the current one."""
    monkeypatch.setattr(S, "_view4", lambda name, t: t.stride())    # CPU tensors stand in: nothing is launched
    c = S.KVCache(2, 96, 2, 64, device="cpu", int4=True)
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)             # noqa: E731
    for k, v in ((z(2, 3, 2, 64), z(2, 4, 2, 64)), (z(1, 3, 2, 64), z(1, 3, 2, 64)), (z(2, 3, 4, 64), z(2, 3, 4, 64)),
                 (z(2, 3, 2, 96), z(2, 3, 2, 96))):
        with pytest.raises(ValueError):
            c.append(k, v)
    q, kv = z(2, 3, 8, 64), z(2, 3, 2, 64)
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    for args in ((q, kv, z(2, 4, 2, 64)), (q, z(2, 2, 2, 64), z(2, 2, 2, 64)), (q, z(2, 3, 4, 64), z(2, 3, 4, 64)),
                 (z(2, 3, 8, 96), z(2, 3, 2, 96), z(2, 3, 2, 96))):
        with pytest.raises(ValueError):
            S.attn_prefill_quant(c, *args, None, 0, 0.125, rope_fused=False)
        with pytest.raises(ValueError):
            S.attn_decode(c, *args, None, 0, 0.125, rope_fused=False, workspace=ws)
    with pytest.raises(ValueError):
        S.attn_prefill_quant(c, q, kv, kv, None, 0, 0.125, rope_fused=False, out=z(2, 2, 8, 64))
    with pytest.raises(TypeError):                                   # a workspace in host memory
        S.attn_prefill_quant(c, q, kv, kv, None, 0, 0.125, rope_fused=False, workspace=ws)
    assert c.offset == 0
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 7, raising=False)
    at = lambda i: SimpleNamespace(device=SimpleNamespace(index=i))  # noqa: E731
    assert S._raw_stream(at(0)) == 7
    with pytest.raises(ValueError):
        S._raw_stream(at(1))
