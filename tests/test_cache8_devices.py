"""8-bit cache calls refuse tensors of another device than the current one, and
caches that are not what they have to be, before anything is launched (CPU
only: tensors that say they are CUDA tensors of some device)."""
import pytest
import torch

import weight_only_int4_group_gb300 as q4
from test_devices import BF16, I32, I64, Tensor, device_zero, made, tensor  # noqa: F401

ATTENTION = dict(q=((2, 4, 64), BF16), table=((1, 2), I32), q_start=((2,), I32), kv_len=((1,), I32),
                 out=((2, 4, 64), BF16), lse=((2, 4), torch.float32), ws=((1 << 20,), torch.uint8))
ROPE = dict(qkv=((2, 8 * 64), BF16), position=((2,), I32), slot=((2,), I64), freq=((32,), torch.float64),
            out=((2, 4, 64), BF16))
READ = dict(table=((1, 2), I32), q_start=((2,), I32), kv_len=((1,), I32), k=((2, 2, 64), BF16), v=((2, 2, 64), BF16))


def cache(elsewhere="", **change):
    on = int(elsewhere == "cache")
    a = dict(k=tensor((4, 2, 16, 64), torch.int8, on), v=tensor((4, 2, 16, 64), torch.int8, on),
             k_exp=tensor((4, 2), torch.uint8, on), v_exp=tensor((4, 2), torch.uint8, on), dtype=BF16)
    return q4.KVCache8(**dict(a, **change))


@pytest.mark.parametrize("elsewhere", [*ATTENTION, "cache"])
def test_attention(elsewhere):
    a = made(ATTENTION, elsewhere)
    with pytest.raises(ValueError, match="device"):
        q4.attention(a["q"], cache(elsewhere), a["table"], a["q_start"], a["kv_len"], 2, out=a["out"], lse=a["lse"],
                     return_lse=True, ws=a["ws"], stream=1)


@pytest.mark.parametrize("elsewhere", [*ROPE, "cache"])
def test_append(elsewhere):
    a = made(ROPE, elsewhere)
    with pytest.raises(ValueError, match="device"):
        q4.rope_append(a["qkv"], cache(elsewhere), a["position"], a["slot"], a["freq"], 4, out=a["out"], stream=1)


@pytest.mark.parametrize("elsewhere", [*READ, "cache"])
def test_read(elsewhere):
    a = made(READ, elsewhere)
    with pytest.raises(ValueError, match="device"):
        q4.cache_read(cache(elsewhere), a["table"], a["q_start"], a["kv_len"], 2, out=(a["k"], a["v"]), stream=1)


@pytest.mark.parametrize("change", [
    dict(k=tensor((4, 2, 16, 64), torch.uint8, 0)), dict(k=tensor((4, 2, 64), torch.int8, 0)),
    dict(v=tensor((4, 2, 16, 64), torch.float8_e4m3fn, 0)), dict(v=tensor((4, 2, 32, 64), torch.int8, 0)),
    dict(v=tensor((4, 2, 16, 64), torch.int8, 1)), dict(k_exp=tensor((4, 3), torch.uint8, 0)),
    dict(v_exp=tensor((4, 2), torch.int8, 0)), dict(v_exp=tensor((2, 4), torch.uint8, 0).t()),
    dict(k_exp=tensor((4, 2), torch.uint8, 1)), dict(dtype=torch.float32), dict(dtype=torch.int8),
], ids=lambda c: ",".join(c))
def test_bad_caches(change):
    with pytest.raises(ValueError):
        cache(**change)


def test_read_takes_no_16_bit_cache():
    k = tensor((4, 2, 16, 64), BF16, 0)
    a = made(READ, "")
    with pytest.raises(TypeError):
        q4.cache_read(q4.KVCache(k, tensor((4, 2, 16, 64), BF16, 0)), a["table"], a["q_start"], a["kv_len"], 2, stream=1)


def test_outputs_of_the_wrong_shape():
    a = made(READ, "")
    bad = tensor((2, 2, 32), BF16, 0)
    for out in ((a["k"], bad), (bad, a["v"]), (a["k"], tensor((3, 2, 64), BF16, 0)), (a["k"], tensor((2, 2, 64), torch.float16, 0))):
        with pytest.raises(ValueError):
            q4.cache_read(cache(), a["table"], a["q_start"], a["kv_len"], 2, out=out, stream=1)
