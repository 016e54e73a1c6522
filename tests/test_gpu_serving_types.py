"""Tensors of types that the serving operators do not take: ValueError from those on a cache of the data's type, whatever
types the ones on codes and pages know, and nothing is enqueued."""
import pytest
import torch

import transformer_rope_positional_gb300 as R

pytestmark = pytest.mark.gpu

OTHERS = [torch.int32, torch.uint8, torch.int16, torch.float64, torch.float8_e4m3fn, torch.float8_e8m0fnu]
T, D, NB, BS = 3, 64, 4, 16


def as_type(t, dtype):
    if dtype in (torch.float8_e4m3fn, torch.float8_e8m0fnu):
        return torch.zeros(t.shape, dtype=torch.uint8, device="cuda").view(dtype)
    return t.to(dtype)


def refused(call, args, names, dtypes=OTHERS):
    n = R.launch_count()
    for name in names:
        for dtype in dtypes:
            with pytest.raises(ValueError):
                call(**dict(args, **{name: as_type(args[name], dtype)}))
    assert R.launch_count() == n
    call(**args)
    assert R.launch_count() > n and R.get_device_error() == 0


def x(*shape):
    return torch.zeros(*shape, dtype=torch.float16, device="cuda")


def i64(*values):
    return torch.tensor(values, dtype=torch.int64, device="cuda")


def test_append_paged_kv(rope_gpu):
    args = {"positions": i64(0, 1, 2), "query": x(T, 2 * D), "key": x(T, D), "value": x(T, D), "cos_sin_cache": x(8, D),
            "slot_mapping": i64(0, 1, 2), "k_cache": x(NB, 1, BS, D), "v_cache": x(NB, 1, BS, D), "head_size": D,
            "query_out": x(T, 2 * D)}
    refused(R.append_paged_kv, args, [n for n in args if n != "head_size"])


def test_paged_attention(rope_gpu):
    args = {"query": x(T, 2 * D), "k_cache": x(NB, 1, BS, D), "v_cache": x(NB, 1, BS, D), "block_table": i64(0).view(1, 1),
            "seq_lens": i64(3), "query_start_loc": i64(0, 3), "out": x(T, 2 * D), "lse": torch.zeros(T, 2, device="cuda"),
            "prefix_blocks": i64(1), "prefix_len": 0}
    refused(R.paged_attention, args, [n for n in args if n != "prefix_len"])
    for dtype in OTHERS:
        with pytest.raises(ValueError):
            R.paged_attention_workspace(as_type(args["query"], dtype), args["k_cache"])


def test_scaled_tables(rope_gpu):
    inv, scale = R.rope_frequencies(D)
    refused(R.scaled_cos_sin_cache, {"inv_freq": inv, "scale": scale, "cache": x(8, D), "positions": i64(*range(8))},
            ["cache", "positions"])
