"""Tensors that share their memory until one of them is written (copy on write): what the serving operators write is
separated from its source first, as by any other write."""
import pytest
import torch

import transformer_rope_positional_gb300 as R

pytestmark = pytest.mark.gpu

CASES = ["cache", "cos and sin", "append", "append in place", "attention", "prepared", "workspace"]


@pytest.mark.skipif(not hasattr(torch, "_lazy_clone"), reason="this torch makes no such tensors")
@pytest.mark.parametrize("what", CASES)
def test_the_source_of_a_lazy_clone_keeps_its_values(rope_gpu, what):
    D, hq, hk, bs, T = 64, 4, 2, 16, 5
    g = torch.Generator(device="cuda").manual_seed(1)
    made = []

    def written(*shape, dtype=torch.float32):
        base = torch.randn(shape, generator=g, device="cuda").to(dtype)
        made.append((base, base.clone(), torch._lazy_clone(base)))
        return made[-1][2]

    inv, _ = R.rope_frequencies(D)
    table = torch.empty(32, D, device="cuda")
    R.scaled_cos_sin_cache(table, inv)
    q, k, v = (torch.randn(T, h * D, generator=g, device="cuda") for h in (hq, hk, hk))
    pos = torch.arange(T, device="cuda")
    if what == "cache":
        R.scaled_cos_sin_cache(written(7, D), inv)
    elif what == "cos and sin":
        R.scaled_cos_sin(written(1, 7, 1, D), written(1, 7, 1, D), inv)
    elif what.startswith("append"):
        query_out = written(T, hq * D)
        query = query_out if what == "append in place" else q
        R.append_paged_kv(pos, query, k, v, table, pos, written(2, hk, bs, D), written(2, hk, bs, D), D,
                          query_out=None if what == "append in place" else query_out)
    else:
        kc, vc = (torch.randn(2, hk, bs, D, generator=g, device="cuda") for _ in range(2))
        rest = (kc, vc, torch.zeros(1, 64, dtype=torch.int64, device="cuda"), torch.tensor([T], device="cuda"),
                torch.tensor([0, T], device="cuda"), written(T, hq * D))
        ws = None
        if what == "workspace":
            n = R.paged_attention_workspace(q, kc)
            ws = written(-(-n // 4))
        if what == "prepared":
            R.prepare_paged_attention(q, *rest, lse=written(T, hq))()
        else:
            R.paged_attention(q, *rest, lse=written(T, hq), workspace=ws)
    torch.cuda.synchronize()
    for base, before, clone in made:
        assert torch.equal(base, before)
        assert not torch.equal(clone, before)
