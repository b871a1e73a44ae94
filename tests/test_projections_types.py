"""What the Python calls of the operators around the attention refuse by themselves, tried on the CPU with the library and the device
check out of the way: a call that fits reaches the library, each of the others does not."""
import pytest
import torch

from compressed_sparse_attention_c4a_gb300 import dsa

U8, E4M3 = torch.uint8, torch.float8_e4m3fn
OTHER_BYTES = [torch.float8_e5m2, torch.int8, torch.bool]


class Reached(Exception):
    pass


@pytest.fixture(autouse=True)
def no_library(monkeypatch):
    class Lib:
        dsa_status_string = dsa._lib.dsa_status_string

        def __getattr__(self, name):
            def call(*args):
                raise Reached(name)
            return call
    monkeypatch.setattr(dsa, "_lib", Lib())
    monkeypatch.setattr(dsa, "_handle", lambda fn, dev, stream: None)


def gemm(fn=dsa.dsa_gemm_q8, **over):
    args = dict(a=torch.zeros((4, 2, 256), dtype=U8), a_scale=torch.ones((4, 2, 2)), w=torch.zeros((2, 130, 256), dtype=U8),
                w_scale=torch.ones((2, 2, 2)), out=torch.zeros((4, 2, 130)))
    args.update(over)
    return lambda: fn(**args)


def stalled(**over):
    return gemm(dsa.dsa_debug_gemm_q8_stalled, wait_limit_ns=5, **over)


def norm(**over):
    args = dict(x=torch.zeros((4, 256), dtype=torch.bfloat16), gamma=torch.ones(256), eps=1e-6, out=torch.zeros((4, 256), dtype=U8),
                out_scale=torch.zeros((4, 2)))
    args.update(over)
    return lambda: dsa.dsa_norm_q8(**args)


def codes(dtype, *shape):
    return torch.zeros(shape, dtype=U8).view(dtype)


@pytest.mark.parametrize("call", [
    gemm(), stalled(), norm(), gemm(a=codes(E4M3, 4, 2, 256)), gemm(w=codes(E4M3, 2, 130, 256)), norm(out=codes(E4M3, 4, 256)),
    gemm(out=codes(U8, 4, 2, 130), out_scale=torch.ones((4, 2, 2))), gemm(out=codes(E4M3, 4, 2, 130), out_scale=torch.ones((4, 2, 2))),
    norm(gamma=None), norm(residual=torch.zeros((4, 256), dtype=torch.bfloat16), sum_out=torch.zeros((4, 256), dtype=torch.bfloat16))])
def test_calls_that_fit_reach_the_library(call):
    with pytest.raises(Reached):
        call()


WHERE = {"a": lambda t: gemm(a=t(4, 2, 256)), "w": lambda t: gemm(w=t(2, 130, 256)), "stalled a": lambda t: stalled(a=t(4, 2, 256)),
         "norm out": lambda t: norm(out=t(4, 256)), "out": lambda t: gemm(out=t(4, 2, 130), out_scale=torch.ones((4, 2, 2)))}


@pytest.mark.parametrize("dtype", OTHER_BYTES + [torch.float16, torch.int32])
@pytest.mark.parametrize("where", WHERE)
def test_codes_of_another_type_are_refused(where, dtype):
    """Bytes that are not e4m3 codes would be read, or taken later, as such."""
    t = (lambda *shape: codes(dtype, *shape)) if dtype in OTHER_BYTES else (lambda *shape: torch.zeros(shape, dtype=dtype))
    with pytest.raises(dsa.DsaError) as e:
        WHERE[where](t)()
    assert e.value.code == dsa.DSA_ERR_INVALID_ARG
