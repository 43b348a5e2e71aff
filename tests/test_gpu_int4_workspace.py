"""What the 4-bit decode leaves in its workspace: the error word, the plan and the
partial results, nothing in between (the merge flags are the other caches')."""
import numpy as np
import pytest

import mla_workloads as W
import oracle
from test_gpu_int4 import C, M, dev, floats, plain_decode, random_cache, torch_bits  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cfg", [C("ws_h16", 16, [1, 700, 64], seed=95), C("ws_h128", 128, [2000] * 9, s=2, seed=96)],
                         ids=lambda c: c.name)
def test_only_what_the_call_needs_is_written(M, cfg):  # noqa: F811
    import torch
    d = W.make_decode_inputs(cfg, with_cache_pages=False)
    codes, scales = random_cache(d, cfg.seed)
    q, dims = W.make_q_abs(cfg), M.dims(cfg.H)
    size = M.mla_decode_workspace_size(dims, cfg.B, cfg.s, d["block_table"].shape[1] * 64)
    lat = torch.empty(cfg.T, cfg.H, 512, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((size,), 0xA5, dtype=torch.uint8, device="cuda")
    M.mla_decode_int4(dims, torch_bits(q), dev(codes), dev(scales), dev(d["block_table"]), dev(d["seq_lens"]), cfg.s,
                      lat, None, ws)
    torch.cuda.synchronize()
    assert M.mla_decode_error(ws) == 0
    ref, _, tol, _ = plain_decode(codes, scales, d, cfg.s, oracle.bf16_to_f64(q))
    assert np.all(np.abs(floats(lat.cpu().view(torch.int16).numpy().view(np.uint16)) - ref) <= tol)
    got = ws.cpu().numpy()
    plan = 256 + 4 * (((cfg.B + 9) & ~3) + 4 * cfg.B)            # after the error word's 256 bytes
    flags = 4 * (2 * cfg.B * ((cfg.s * cfg.H + 63) // 64) * 4 + 1)
    assert np.all(got[4:256] == 0xA5) and np.all(got[plan:plan + flags] == 0xA5)
