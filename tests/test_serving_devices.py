"""The binding's check that every tensor of the norm's, the cache's and the attention's calls is on one GPU:
a host address that reaches a kernel is a memory fault. On a machine without a GPU: tensors that call
themselves device tensors pass all checks and stop at the missing device, before any launch."""
import pytest
import torch

import fp8_group_quant_amd as fq

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not on any GPU")


class OnGpu(torch.Tensor):
    """A host tensor that calls itself one of GPU `index`."""
    __torch_function__ = torch._C._disabled_torch_function_impl
    index = 0
    is_cuda = True

    def get_device(self):
        return self.index


def on_gpu(t, index=0):
    t = torch.Tensor._make_subclass(OnGpu, t)
    t.index = index
    return t


def zeros(*shape, dtype=torch.bfloat16):
    return on_gpu(torch.zeros(shape, dtype=dtype))


def norm():
    x, s = zeros(4, 256), zeros(4, 2, dtype=torch.uint8)
    return fq.fp8q_rms_norm_group_quant, dict(x=x, weight=zeros(256), q=zeros(4, 256, dtype=torch.uint8), s=s,
                                              residual=zeros(4, 256), residual_out=zeros(4, 256))


def cache():
    return dict(zip(("c_k", "c_ks", "c_v", "c_vs"), (zeros(3, 16, 2, w, dtype=torch.uint8) for w in (32, 2, 32, 2))))


def with_cache(fn, c_k, c_ks, c_v, c_vs, **kw):
    return fn(cache=fq.Kv4Cache(c_k, c_ks, c_v, c_vs), **kw)


def write():
    return (lambda **kw: with_cache(fq.fp8q_kv4_write, **kw)), dict(
        k=zeros(5, 2, 64), v=zeros(5, 2, 64), slots=zeros(5, dtype=torch.int32), **cache())


def read():
    return (lambda **kw: with_cache(fq.fp8q_kv4_read, **kw)), write()[1]


def attention():
    return (lambda **kw: with_cache(fq.fp8q_kv4_attention, sm_scale=0.1, **kw)), dict(
        q=zeros(5, 4, 64), block_table=zeros(3, 2, dtype=torch.int32), kv_lens=zeros(3, dtype=torch.int32),
        out=zeros(5, 4, 64), q_indptr=zeros(4, dtype=torch.int32), lse=zeros(5, 4, dtype=torch.float32),
        workspace=zeros(256, dtype=torch.uint8), **cache())


CALLS = dict(norm=norm, write=write, read=read, attention=attention)


@pytest.mark.parametrize("name", CALLS)
def test_device_tensors_pass(name):
    fn, kw = CALLS[name]()
    with pytest.raises(fq.Fp8qError) as e:
        fn(**kw, stream=0)
    assert e.value.status == fq.EDEVICE


@pytest.mark.parametrize("name,operand", [(n, o) for n, c in CALLS.items() for o in c()[1]])
def test_a_tensor_elsewhere_is_refused(name, operand):
    fn, kw = CALLS[name]()
    host = kw[operand].as_subclass(torch.Tensor)
    for other in (host, on_gpu(host, 1)):
        with pytest.raises(ValueError):
            fn(**{**kw, operand: other}, stream=0)
