"""What the bindings refuse before the library is called: tensors beside q, k, v
whose length, type, layout or device the C side cannot see from a pointer. CPU
tensors stand in for device ones, and the library is replaced by one that fails
the test where it is reached."""

import pytest
import torch

from sink_augmented_gqa_b200 import build as sbuild
from sink_augmented_gqa_b200 import sinkattn as S

B, T, NQ, NKV, D = 2, 1, 8, 2, 64


class Elsewhere(torch.Tensor):
    """A tensor on another device."""

    def get_device(self):
        return 3


def elsewhere(t):
    return t.as_subclass(Elsewhere)


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def f(*shape):
    return z(*shape, dtype=torch.float32)


class NotReached:
    def __getattr__(self, name):
        raise AssertionError(f"{name} was called")


@pytest.fixture
def caches(monkeypatch):
    sbuild.build()
    made = {n: S.KVCache(B, 96, NKV, D, device="cpu", int4=n == "int4", fp8=n == "fp8") for n in ("bf16", "fp8", "int4")}
    monkeypatch.setattr(S, "_view4", lambda name, t: t.stride())
    monkeypatch.setattr(S, "_device_stream", lambda index: 0)
    monkeypatch.setattr(S, "lib", NotReached)
    return made


def _calls(caches):
    ws = z(1 << 16, dtype=torch.uint8)
    yield "attn_prefill", lambda *a, **k: S.attn_prefill(caches["bf16"], *a, **k)
    yield "attn_decode_static", lambda *a, **k: S.attn_decode_static(caches["int4"], *a, **k)
    for fmt in ("bf16", "fp8", "int4"):
        yield "attn_decode", lambda *a, fmt=fmt, **k: S.attn_decode(caches[fmt], *a, **{"workspace": ws, **k})
        if fmt != "bf16":
            yield "attn_prefill_quant", lambda *a, fmt=fmt, **k: S.attn_prefill_quant(caches[fmt], *a, **{"workspace": ws, **k})


BAD = [("sinks", dict(sinks=f(NQ - 1)), ValueError), ("sinks", dict(sinks=f(NQ + 1)), ValueError),
       ("sinks", dict(sinks=f(1, NQ)), ValueError), ("sinks", dict(sinks=z(NQ)), TypeError),
       ("sinks", dict(sinks=f(2 * NQ)[::2]), TypeError), ("sinks", dict(sinks=elsewhere(f(NQ))), TypeError),
       ("lse", dict(lse=f(B, NQ)), ValueError), ("lse", dict(lse=f(B, T, NQ)), ValueError),
       ("lse", dict(lse=f(B - 1, NQ, T)), ValueError), ("lse", dict(lse=z(B, NQ, T)), TypeError),
       ("lse", dict(lse=f(B, 2 * NQ, T)[:, ::2]), TypeError), ("lse", dict(lse=elsewhere(f(B, NQ, T))), TypeError),
       ("cos", dict(cos=z(96, D // 2)), TypeError), ("cos", dict(cos=elsewhere(f(96, D // 2))), TypeError),
       ("cos", dict(cos=f(96, D)), ValueError), ("cos", dict(cos=f(96, D)[:, ::2]), TypeError),
       ("sin", dict(sin=z(96, D // 2)), TypeError), ("sin", dict(sin=elsewhere(f(96, D // 2))), TypeError),
       ("sin", dict(sin=f(95, D // 2)), ValueError), ("sin", dict(sin=f(96, D // 4)), ValueError)]


@pytest.mark.parametrize("name,over,error", BAD, ids=[f"{b[0]}{i}" for i, b in enumerate(BAD)])
def test_attention_refuses(caches, name, over, error):
    for call, fn in _calls(caches):
        a = dict(sinks=f(NQ), cos=f(96, D // 2), sin=f(96, D // 2), lse=f(B, NQ, T))
        a.update(over)
        with pytest.raises(error, match=f"^{name} must be"):
            fn(z(B, T, NQ, D), z(B, T, NKV, D), z(B, T, NKV, D), a["sinks"], 0, 0.125, a["cos"], a["sin"],
               lse=a["lse"], return_lse=True)
    assert all(c.offset == 0 for c in caches.values())


def test_attention_refuses_other_devices(caches):
    q, k, v = z(B, T, NQ, D), z(B, T, NKV, D), z(B, T, NKV, D)
    for call, fn in _calls(caches):
        for args, out in (((elsewhere(q), k, v), None), ((q, elsewhere(k), v), None), ((q, k, elsewhere(v)), None),
                          ((q, k, v), elsewhere(q)), ((elsewhere(q), elsewhere(k), elsewhere(v)), elsewhere(q))):
            with pytest.raises(ValueError, match="on one device"):
                fn(*args, None, 0, 0.125, rope_fused=False, out=out)


def test_attention_refuses_host_and_strided_workspaces(caches):
    q, k, v = z(B, T, NQ, D), z(B, T, NKV, D), z(B, T, NKV, D)
    for call, fn in _calls(caches):
        if call in ("attn_decode", "attn_prefill_quant"):
            for ws in (z(1 << 16, dtype=torch.uint8), z(1 << 16, 2, dtype=torch.uint8)[:, 0]):
                with pytest.raises(TypeError, match="workspace"):
                    fn(q, k, v, None, 0, 0.125, rope_fused=False, workspace=ws)


def test_append_and_read_refuse_other_devices(caches):
    rows = z(B, 3, NKV, D)
    for c in caches.values():
        for k, v in ((elsewhere(rows), rows), (rows, elsewhere(rows))):
            with pytest.raises(ValueError, match="device"):
                c.append(k, v)
            with pytest.raises(ValueError, match="device"):
                c.read(0, 3, k_out=k, v_out=v)


def test_cache_buffers_on_two_devices():
    for over in (dict(v=elsewhere(z(B, NKV, 96, D // 2, dtype=torch.uint8))), dict(k_scale=elsewhere(z(B, NKV, 96, D // 32)))):
        with pytest.raises(AssertionError):
            S.KVCache(B, 96, NKV, D, device="cpu", int4=True, **over)


def test_backward_refuses(monkeypatch):
    monkeypatch.setattr(S, "_require_bf16_cuda", lambda name, t: None)
    monkeypatch.setattr(S, "lib", NotReached)
    q, kv = z(B, 5, NQ, D), z(B, 5, NKV, D)
    ok = dict(q=q, k=kv, v=kv, out=q, d_out=q, lse=f(B, NQ, 5), sinks=f(NQ))
    for over, error, what in ((dict(lse=f(B, NQ, 4)), ValueError, "lse"), (dict(lse=z(B, NQ, 5)), TypeError, "lse"),
                              (dict(sinks=f(NQ - 1)), ValueError, "sinks"), (dict(sinks=elsewhere(f(NQ))), TypeError, "sinks"),
                              (dict(d_out=z(B, 4, NQ, D)), ValueError, "d_out"), (dict(v=z(B, 5, NKV, 32)), ValueError, "v"),
                              (dict(v=elsewhere(kv)), ValueError, "one device")):
        a = {**ok, **over}
        with pytest.raises(error, match=what):
            S.attn_backward(a["q"], a["k"], a["v"], a["out"], a["d_out"], a["lse"], a["sinks"], 0, 0.125,
                            workspace=z(16, dtype=torch.uint8))
    with pytest.raises(TypeError, match="workspace"):
        S.attn_backward(*ok.values(), 0, 0.125, workspace=z(16, dtype=torch.uint8))


def test_rope_refuses(monkeypatch):
    monkeypatch.setattr(S, "lib", NotReached)
    q, kv = z(B, 5, NQ, D), z(B, 5, NKV, D)
    for cos, sin, error in ((z(9, D // 2), f(9, D // 2), TypeError), (f(9, D), f(9, D), ValueError),
                            (f(9, D // 2), f(8, D // 2), ValueError), (f(9, D // 2), elsewhere(f(9, D // 2)), TypeError)):
        with pytest.raises(error, match="cos|sin"):
            S.rope_apply_qk(q, kv, 0, cos, sin)
