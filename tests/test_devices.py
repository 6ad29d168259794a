"""Tensors of another device than the current one are refused before anything
is launched, for each tensor of each call (CPU only: tensors that say they are
CUDA tensors of some device, over host memory that no check reads)."""
import pytest
import torch

import weight_only_int4_group_gb300 as q4


class Tensor(torch.Tensor):
    on = 0
    is_cuda = True

    def get_device(self):
        return self.on

    @property
    def device(self):
        return torch.device("cuda", self.on)

    @classmethod
    def __torch_function__(cls, func, types, args=(), kwargs=None):
        out = super().__torch_function__(func, types, args, kwargs or {})
        if isinstance(out, Tensor) and args and isinstance(args[0], Tensor):
            out.on = args[0].on  # views stay where their base is
        return out


def tensor(shape, dtype, on):
    t = torch.zeros(shape, dtype=dtype).as_subclass(Tensor)
    t.on = on
    return t


I32, I64, BF16 = torch.int32, torch.int64, torch.bfloat16
ATTENTION = dict(q=((2, 4, 64), BF16), table=((1, 2), I32), q_start=((2,), I32), kv_len=((1,), I32),
                 out=((2, 4, 64), BF16), lse=((2, 4), torch.float32), ws=((1 << 20,), torch.uint8))
ROPE = dict(qkv=((2, 8 * 64), BF16), position=((2,), I32), slot=((2,), I64), freq=((32,), torch.float64),
            out=((2, 4, 64), BF16))
PLAN = dict(cached=((3,), I32), fresh=((3,), I32), table=((3, 4), I32), free_blocks=((5,), I32), free_count=((1,), I32))
OUT = dict(q_start=((4,), I32), kv_len=((3,), I32), position=((6,), I32), slot=((6,), I64), counts=((4,), I32))


@pytest.fixture(autouse=True)
def device_zero(monkeypatch):
    monkeypatch.setattr(q4, "_current_device", lambda: 0, raising=False)


def made(spec, elsewhere):
    return {n: tensor(*s, on=int(n == elsewhere)) for n, s in spec.items()}


def cache(elsewhere):
    on = int(elsewhere == "cache")
    return q4.KVCache(tensor((4, 2, 16, 64), BF16, on), tensor((4, 2, 16, 64), BF16, on))


@pytest.mark.parametrize("elsewhere", [*ATTENTION, "cache"])
def test_attention(elsewhere):
    with pytest.raises(ValueError, match="device"):
        q4.attention(cache=cache(elsewhere), max_fresh=2, stream=0, **made(ATTENTION, elsewhere))


@pytest.mark.parametrize("elsewhere", [*ROPE, "cache"])
def test_rope_append(elsewhere):
    with pytest.raises(ValueError, match="device"):
        q4.rope_append(cache=cache(elsewhere), heads=4, stream=0, **made(ROPE, elsewhere))


@pytest.mark.parametrize("elsewhere", [*PLAN, *OUT])
def test_cache_plan(elsewhere):
    with pytest.raises(ValueError, match="device"):
        q4.cache_plan(block_size=16, T=6, stream=0, out=q4.CachePlan(**made(OUT, elsewhere)), **made(PLAN, elsewhere))


@pytest.mark.parametrize("elsewhere", ["x", "weight", "out", "ws"])
@pytest.mark.parametrize("call", [q4.gemv, q4.gemm, q4.gemv_noalloc], ids=lambda f: f.__name__)
def test_products(call, elsewhere):
    t = made(dict(x=((4, 128), BF16), weight=((q4.weight_bytes(64, 128),), torch.uint8), out=((4, 64), BF16),
                  ws=((1 << 20,), torch.uint8)), elsewhere)
    kw = dict(out=t["out"], stream=0)
    if call is not q4.gemv_noalloc:
        kw["ws"] = t["ws"]
    elif elsewhere == "ws":
        return
    with pytest.raises(ValueError, match="device"):
        call(t["x"], q4.QWeight(t["weight"], 64, 128), **kw)


def test_packing():
    N, K = 16, 128
    w = tensor((N, K), torch.float32, 1)
    arrays = [tensor((N, K // 2), torch.uint8, 0), tensor((N, 1), torch.float32, 0), tensor((N, 1), torch.uint8, 1)]
    buf = tensor((q4.weight_bytes(N, K),), torch.uint8, 1)
    for call in (lambda: q4.quantize(w), lambda: q4.quantize_sym(w), lambda: q4.xsum(w),
                 lambda: q4.repack(*arrays, N, K, out=buf), lambda: q4.repack_compact(*arrays, N, K, out=buf),
                 lambda: q4.unpack(buf, N, K), lambda: q4.unpack_compact(buf, N, K)):
        with pytest.raises(ValueError, match="device"):
            call()
