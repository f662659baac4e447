"""Weights of more 16-byte pieces than a launch has threads: 64 GiB of them in
one matrix."""
import pytest
import torch

from tests.gpu_util import log, require_gpu

pytestmark = pytest.mark.gpu


def test_last_expert_of_64_gib_of_weights():
    require_gpu()
    import w4a16_int4_grouped_amd as m
    E, H, I = 4096, 4096, 4128
    torch.cuda.empty_cache()
    need = 2 * E * 3 * I * H // 32 * 18 + (2 << 30)          # given and prepared, 16 bytes of codes and 2 of scale per 32
    if torch.cuda.mem_get_info()[0] < need:
        pytest.skip(f"{need >> 30} GiB of GPU memory are not free")
    log(f"case prepare E={E} H={H} I={I}")
    dev = "cuda"
    w13_q = torch.empty(E, 2 * I, H // 8, dtype=torch.int32, device=dev)
    w2_q = torch.empty(E, H, I // 8, dtype=torch.int32, device=dev)
    w13_s = torch.ones(E, 2 * I, H // 32, dtype=torch.bfloat16, device=dev)
    w2_s = torch.ones(E, H, I // 32, dtype=torch.bfloat16, device=dev)
    g = torch.Generator(device=dev).manual_seed(1)
    look = (0, E // 2, E - 1)
    for e in look:
        for q, s in ((w13_q, w13_s), (w2_q, w2_s)):
            q[e] = torch.randint(-(2 ** 31), 2 ** 31 - 1, q[e].shape, generator=g, device=dev, dtype=torch.int64).int()
            s[e] = torch.randint(1, 9, s[e].shape, generator=g, device=dev).bfloat16()
    h = m.PreparedWeights(w13_q, w13_s, w2_q, w2_s)
    for e in look:
        for which, q, s in ((13, w13_q[e], w13_s[e]), (2, w2_q[e], w2_s[e])):
            code = torch.stack([(q >> (4 * k)) & 15 for k in range(8)], -1).flatten(1)
            want = (code - 8).float() * s.float().repeat_interleave(32, 1)
            assert torch.equal(h.dequant(which, e).float(), want), (which, e)
    del h, w13_q, w2_q, w13_s, w2_s
    torch.cuda.empty_cache()
