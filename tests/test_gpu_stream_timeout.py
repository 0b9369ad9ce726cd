"""Bounded waits of the cache attention kernels that run out on purpose, on
small launches: each reports CALIBATT_ERR_TIMEOUT, drains what it has in
flight and returns, and the next launch is correct. No GPU fault is involved:
the waits end by their own limit."""
import math

import pytest
import torch

from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,kv_heads,new,kv", [(2, 2, 1, 1500), (8, 1, 1, 1500), (8, 1, 2, 700), (1, 1, 40, 900),
                                                   (1, 1, 100, 300), (2, 2, 300, 800), (1, 1, 140, 140)])
def test_cache_attention_wait_runs_out_then_context_is_usable(heads, kv_heads, new, kv):
    binding = require_gpu()
    pages = -(-kv // 128)
    k8 = torch.zeros((pages, kv_heads, 128, 128), dtype=torch.uint8, device="cuda")
    v8 = torch.full_like(k8, 0x38)  # 1.0
    scale = torch.ones((pages, kv_heads), device="cuda")
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None].contiguous()
    start, length = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, new], [kv]))
    q = torch.ones((heads, new, 128), dtype=torch.bfloat16, device="cuda")

    def call():
        return binding.cache_attn_fwd(q, k8, v8, scale, scale, start, length, table)

    assert binding.get_status() == 0
    try:
        binding.set_wait_limit(1e-9)
        # a wait that begins and ends within one tick of the GPU's timer is not
        # seen to take time, so a call may get through
        status = 0
        for _ in range(200):
            call()
            status = binding.get_status()
            if status != 0:
                break
        assert status == -6
    finally:
        binding.set_wait_limit(0.0)
    o, lse = call()
    assert binding.get_status() == 0
    assert torch.all(o == 1.0) and torch.all((lse - math.log(kv)).abs() < 1e-5)
