"""Decodes of different shapes and cache formats that share a workspace, or the
library's own scratch, one after another: what one leaves there is no other
one's counters."""

import pytest
import torch

import sink_augmented_gqa_b200 as sa
from sink_augmented_gqa_b200 import workloads as wl

from helpers import check_bf16_output, check_lse
from test_gpu_int4 import _setup

pytestmark = pytest.mark.gpu
DEV = "cuda"
# from few (sequence, KV head) pairs, whose records lie low in the workspace, to many
SHAPES = [(dict(B=1, n_q=16, n_kv=2, d=64), 3000), (dict(B=1, n_q=64, n_kv=8, d=64), 2000),
          (dict(B=16, n_q=16, n_kv=8, d=64), 600), (dict(B=30, n_q=16, n_kv=8, d=64), 500)]


@pytest.mark.parametrize("static", [False, True], ids=["workspace", "static"])
@pytest.mark.parametrize("formats", [("int4",), ("fp8",), ("bf16",), ("int4", "bf16", "fp8")], ids="-".join)
def test_shapes_in_turn(cuda_device, formats, static):
    made = [_setup(over, formats[i % len(formats)], off, 4) for i, (over, off) in enumerate(SHAPES)]
    ws = torch.zeros(max(sa.decode_workspace_bytes(c[0].B, c[0].n_q, c[0].n_kv, c[0].d) for c in made),
                     dtype=torch.uint8, device=DEV)
    for step in range(3):
        for cfg, cache, oracle, cos, sin in made if step != 1 else made[::-1]:
            q, k, v = wl.qkv(cfg, 1, step=step)
            args = (cache, q.to(DEV), k.to(DEV), v.to(DEV), None, 0, cfg.sm_scale, cos, sin)
            out = torch.full_like(args[1], float("nan"))
            if static:
                out, lse = sa.attn_decode_static(*args, out=out, return_lse=True)
            else:
                out, lse = sa.attn_decode(*args, workspace=ws, out=out, return_lse=True)
            torch.cuda.synchronize()
            ref, ref_lse, _ = oracle.call(q, k, v, None, 0, read=oracle.fmt != "fp8")
            what = f"{oracle.fmt} {cfg.B} x {cfg.n_kv}, step {step}"
            check_bf16_output(out, ref, what)
            if oracle.fmt != "fp8":
                check_lse(lse, ref_lse, what)
