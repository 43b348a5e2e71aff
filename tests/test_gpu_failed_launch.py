"""A call that fails leaves no error behind for the next call to report."""
import numpy as np
import pytest

import oracle
from _gpu_setup import host_bits, i32
from mla_workloads import bf16_bits_to_f32

pytestmark = pytest.mark.gpu


def gather(M):
    """A small call that checks its launch through the runtime's last error."""
    import torch
    rng = np.random.default_rng(1)
    codes, scales = rng.integers(0, 256, (1, 64, 288), dtype=np.uint8), rng.integers(0, 256, (1, 64, 36), dtype=np.uint8)
    rows = torch.empty(2, 576, dtype=torch.bfloat16, device="cuda")
    M.mla_gather_latent_int4(M.dims(16), torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), i32([0, 0]),
                             i32([3, 9]), i32([[0]]), rows)
    assert np.array_equal(bf16_bits_to_f32(host_bits(rows)), oracle.int4_values(codes, scales)[0, [3, 9]])


def test_a_grid_that_the_launch_refuses(M):
    """65,536 tiles of 128 tokens are one more than a grid's second dimension holds: the
    projection's launch fails.  (Every buffer is as large as the call says.)"""
    import torch
    T = 128 * 65536
    h = torch.zeros(T, 64, dtype=torch.bfloat16, device="cuda")
    w_dkv, w_kr = torch.zeros(512, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(64, 64, dtype=torch.bfloat16, device="cuda")
    seq = torch.zeros(T, dtype=torch.int32, device="cuda")
    cache = torch.zeros(1, 64, 576, dtype=torch.bfloat16, device="cuda")
    for _ in range(2):
        with pytest.raises(M.MLAError) as e:
            M.mla_append_cache(M.dims(16), h, w_dkv, w_kr, seq, seq, i32([[0]]), cache)
        assert e.value.status == M.MLA_ERR_CUDA
        gather(M)


@pytest.fixture(scope="module")
def M():
    import head_latent_attention_10_b200 as M
    M.load_library()
    return M
