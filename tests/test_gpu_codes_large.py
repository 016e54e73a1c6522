"""Attention over a cache of 8-bit codes that is larger than 2^32 bytes, in the kernels that prompts, heads over 256 and shared
prefixes take."""
import pytest
import torch

import transformer_rope_positional_gb300 as R
from codes_ref import bytes_of, coded_case
from scales_ref import reference
from serving_ref import assert_close, widened

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,D,new,own,P,wide", [
    (torch.bfloat16, 128, [200, 30], [300, 64], 0, True), (torch.float16, 96, [150], [260], 40, True),
    (torch.bfloat16, 256, [140], [200], 0, True), (torch.float32, 128, [40], [200], 0, False),
    (torch.bfloat16, 512, [3, 1], [70, 40], 10, False), (torch.bfloat16, 128, [1] * 20, [30] * 20, 300, False)], ids=str)
def test_cache_past_32_bit_offsets(rope_gpu, dtype, D, new, own, P, wide):
    hk, bs = 8, 64
    NB = (1 << 32) // (hk * bs * D) + 40
    if torch.cuda.mem_get_info()[0] < 3 * NB * hk * bs * D:
        pytest.skip("needs 13 GB")
    c = coded_case(61, dtype, new, own, P=P, hq=2 * hk, hk=hk, D=D, bs=bs, S=4)
    n = c["k"].shape[0]
    pages = torch.tensor([NB - 1 - i for i in range(n)])
    pages[::2] = torch.arange(len(pages[::2]))
    big = []
    for name in ("k_codes", "v_codes", "k_scale", "v_scale"):
        x = torch.empty((NB,) + tuple(c[name].shape[1:]), dtype=torch.uint8, device="cuda")
        x[pages.cuda()] = bytes_of(c[name]).cuda()
        big.append(x.view(c[name].dtype))
    ro, rl, to, tl = reference(c)
    table = torch.where(c["table"] < n, pages[c["table"].clamp(max=n - 1)], c["table"])
    if wide:
        table = widened(dict(c, table=table))["table"]
    out, lse = torch.empty(c["T"], 2 * hk * D, device="cuda", dtype=dtype), torch.empty(c["T"], 2 * hk, device="cuda")
    R.paged_attention_8bit(c["q"].cuda(), *big, table.cuda(), c["lens"].cuda(), c["starts"].cuda(), out, scale=c["scale"],
                           prefix_blocks=pages[c["prefix"]].cuda() if P else None, prefix_len=P, lse=lse)
    assert_close(out, ro, to, "out")
    assert_close(lse, rl, tl, "lse")
    assert R.get_device_error() == 0
