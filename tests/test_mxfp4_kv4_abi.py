"""Host-side checks of the 4-bit quantizer's and product's, the page plan's and the masked attentions' entry points:
every refusal of the C ABI with its status, and the binding's checks of tensors and of where they are. No compute
call runs: validation returns before the library touches a pointer or the device."""
import math

import pytest
import torch

import fp8_group_quant_amd as fq
from test_serving_abi import ATTN, CACHE_CASES, EALIGN, EDEVICE, EINVAL, EUNSUPPORTED, OK, no_gpu
from test_serving_devices import on_gpu, with_cache, zeros

ROWS = dict(x=0x10000, in_dtype=0, M=8, K=512, x_sm=512, q=0x20000, q_sm=256, s=0x30000, scale_fmt=1, s_sm=1, s_sg=8, stream=None)


def rows(entry, kw):
    a = {**ROWS, **kw}
    if entry == "fp8q_mxfp4_dequant":
        a = {k: a[k] for k in ("q", "q_sm", "s", "scale_fmt", "s_sm", "s_sg", "x", "in_dtype", "M", "K", "x_sm", "stream")}
    return getattr(fq.load_library(), entry)(*a.values())


@no_gpu
@pytest.mark.parametrize("entry", ["fp8q_mxfp4_quant", "fp8q_silu_mul_mxfp4_quant", "fp8q_mxfp4_dequant"])
@pytest.mark.parametrize("kw,status", [
    ({}, EDEVICE), (dict(s_sm=16, s_sg=1), EDEVICE), (dict(scale_fmt=2), EDEVICE), (dict(scale_fmt=2, s_sm=4, s_sg=1), EDEVICE),
    (dict(M=0, x=None), OK), (dict(K=0, q=None), OK), (dict(K=32, s_sg=0, x_sm=32, q_sm=16), EDEVICE),
    (dict(in_dtype=3), EUNSUPPORTED), (dict(scale_fmt=0), EUNSUPPORTED), (dict(scale_fmt=3), EUNSUPPORTED),
    (dict(M=-1), EINVAL), (dict(K=-32), EINVAL), (dict(K=500), EINVAL), (dict(K=544, scale_fmt=2), EINVAL),
    (dict(K=(1 << 30) + 128), EUNSUPPORTED),
    (dict(x_sm=-8), EINVAL), (dict(q_sm=-16), EINVAL), (dict(s_sm=-1), EINVAL), (dict(s_sg=-1), EINVAL),
    (dict(x=None), EINVAL), (dict(q=None), EINVAL), (dict(s=None), EINVAL),
    (dict(s_sm=2, s_sg=16), EINVAL), (dict(s_sg=4), EINVAL), (dict(s_sm=8, s_sg=1), EINVAL),
    (dict(x=0x10008), EALIGN), (dict(x_sm=516), EALIGN), (dict(q=0x20008), EALIGN), (dict(q_sm=264), EALIGN),
    (dict(scale_fmt=2, s=0x30002), EALIGN), (dict(s=0x30001), EDEVICE),
])
def test_rows_validation(entry, kw, status):
    assert rows(entry, kw) == status, fq.fp8q_last_error()


@no_gpu
def test_rows_that_overlap():
    assert rows("fp8q_mxfp4_quant", dict(q_sm=240)) == EINVAL and rows("fp8q_mxfp4_quant", dict(x_sm=0)) == EDEVICE
    assert rows("fp8q_mxfp4_dequant", dict(x_sm=504)) == EINVAL and rows("fp8q_mxfp4_dequant", dict(q_sm=0)) == EDEVICE


GEMM = dict(a=0x10000, lda=256, sa=0x20000, sa_fmt=2, sa_sm=1, sa_sk=8, b=0x30000, ldb=256, sb=0x40000, sb_fmt=2, sb_sn=1,
            sb_sk=100, y=0x50000, ldy=100, M=8, N=100, K=512, workspace=None, workspace_bytes=0, stream=None)


@no_gpu
@pytest.mark.parametrize("kw,status", [
    ({}, EDEVICE), (dict(sa_fmt=1, sa_sm=16, sa_sk=1), EDEVICE), (dict(sb_fmt=1, sb_sn=20, sb_sk=1), EDEVICE),
    (dict(sa_sm=4, sa_sk=1), EDEVICE), (dict(sa_sm=0, sa_sk=0), EDEVICE),
    (dict(M=0, a=None), OK), (dict(N=0, b=None), OK), (dict(K=0, y=None), OK),
    (dict(sa_fmt=0), EUNSUPPORTED), (dict(sb_fmt=0), EUNSUPPORTED), (dict(sa_fmt=3), EUNSUPPORTED),
    (dict(sa_fmt=1, sa_sm=1, sa_sk=8), EUNSUPPORTED), (dict(sb_fmt=1, sb_sn=1, sb_sk=100), EUNSUPPORTED),
    (dict(sa_fmt=1, sa_sm=18, sa_sk=1), EALIGN), (dict(sa_fmt=1, sa_sm=16, sa_sk=1, sa=0x20002), EALIGN), (dict(sb=0x40001), EALIGN),
    (dict(M=-1), EINVAL), (dict(N=-1), EINVAL), (dict(K=-128), EINVAL), (dict(K=192), EINVAL),
    (dict(M=1 << 31), EUNSUPPORTED), (dict(N=1 << 31), EUNSUPPORTED), (dict(K=1 << 31), EUNSUPPORTED),
    (dict(M=1 << 26), EDEVICE), (dict(M=(1 << 26) + 1), EUNSUPPORTED), (dict(M=1 << 20, N=1 << 20, ldy=1 << 20), EDEVICE),
    (dict(M=1 << 21, N=1 << 20, ldy=1 << 20), EUNSUPPORTED), (dict(K=1 << 25, lda=1 << 24, ldb=1 << 24), EUNSUPPORTED),
    (dict(lda=(1 << 24) - 16), EDEVICE), (dict(lda=1 << 24), EUNSUPPORTED), (dict(M=1, lda=1 << 24), EDEVICE),
    (dict(ldb=1 << 24), EUNSUPPORTED), (dict(sa_sm=1 << 22, sa_sk=1), EUNSUPPORTED), (dict(sa_sm=(1 << 22) - 1, sa_sk=1), EDEVICE),
    (dict(sb_fmt=1, sb_sn=1 << 24, sb_sk=1), EUNSUPPORTED), (dict(sa_sk=1 << 40), EDEVICE),
    (dict(lda=-16), EINVAL), (dict(sb_sk=-1), EINVAL), (dict(ldy=-1), EINVAL),
    (dict(a=None), EINVAL), (dict(b=None), EINVAL), (dict(y=None), EINVAL), (dict(sa=None), EINVAL), (dict(sb=None), EINVAL),
    (dict(lda=240), EINVAL), (dict(ldb=128), EINVAL), (dict(ldy=99), EINVAL), (dict(M=1, lda=0, ldy=0), EDEVICE),
    (dict(lda=264), EALIGN), (dict(a=0x10008), EALIGN), (dict(b=0x30004), EALIGN), (dict(y=0x50001), EALIGN),
    (dict(y=0x50002, ldy=101), EDEVICE), (dict(workspace=0x60008), EALIGN), (dict(workspace_bytes=-1), EINVAL),
])
def test_product_validation(kw, status):
    assert fq.load_library().fp8q_gemm_mxfp4(*{**GEMM, **kw}.values()) == status, fq.fp8q_last_error()


@no_gpu
def test_workspace_sizes_without_a_device_or_with_refused_sizes():
    size = fq.load_library().fp8q_gemm_mxfp4_workspace_size
    assert size(64, 4096, 7168) == 0 and size(-1, 4096, 7168) == 0 and size(64, 4096, 100) == 0 and size(0, 0, 0) == 0
    size = fq.load_library().fp8q_kv4_window_attention_workspace_size
    assert size(0, 1, 1, 32, 8, 128, 100000, 50000, 4) == 0 and size(0, 1, 1, 32, 8, 128, 100000, 0, 4) == 0
    assert size(0, 1, 1, 32, 8, 96, 100000, 50000, -4) == 0
    size = fq.load_library().fp8q_kv4_tree_attention_workspace_size
    assert size(0, 1, 1, 32, 8, 128, 100000) == 0 and size(2, 1, 1, 32, 8, 128, 100000) == 0


SHARED = CACHE_CASES + [
    (dict(lse=None), EDEVICE), (dict(q_indptr=None, T=3), EDEVICE), (dict(q_indptr=None), EINVAL), (dict(B=0, kv_lens=None), OK),
    (dict(T=0, q=None), OK), (dict(dtype=2), EUNSUPPORTED), (dict(Hkv=3), EINVAL), (dict(B=4097), EUNSUPPORTED),
    (dict(T=1 << 28), EUNSUPPORTED), (dict(max_pages=1 << 27), EUNSUPPORTED), (dict(max_pages=-1), EINVAL), (dict(table=None), EINVAL),
    (dict(sm_scale=math.inf), EINVAL), (dict(q_st=-8), EINVAL), (dict(o_sh=64), EINVAL), (dict(l_st=4), EINVAL),
    (dict(q=0x10008), EALIGN), (dict(table=0x20002), EALIGN), (dict(workspace=0x70008), EALIGN), (dict(workspace_bytes=-1), EINVAL),
]


def masked_args(kw, **own):
    a = {**ATTN}
    del a["causal"]
    tail = {k: a.pop(k) for k in ("workspace", "workspace_bytes", "stream")}
    return {**a, **own, **tail, **kw}.values()


@no_gpu
@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(window=0), EINVAL), (dict(window=-5), EINVAL), (dict(sinks=-1), EINVAL), (dict(window=1 << 62, sinks=1 << 62), EDEVICE),
    (dict(window=1, sinks=0), EDEVICE),
])
def test_window_validation(kw, status):
    rc = fq.load_library().fp8q_kv4_window_attention(*masked_args(kw, window=100, sinks=4))
    assert rc == status, fq.fp8q_last_error()


@no_gpu
@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(tree_mask=None), EINVAL), (dict(tree_mask=None, tree_words=0), EDEVICE), (dict(tree_st=-1), EINVAL),
    (dict(tree_words=-1), EINVAL), (dict(tree_words=(1 << 26) + 1), EUNSUPPORTED), (dict(tree_mask=0x80002), EALIGN),
    (dict(tree_st=0), EDEVICE),
])
def test_tree_validation(kw, status):
    rc = fq.load_library().fp8q_kv4_tree_attention(*masked_args(kw, tree_mask=0x80000, tree_st=2, tree_words=2))
    assert rc == status, fq.fp8q_last_error()


PLAN = dict(kv_lens=0x10000, q_lens=0x20000, B=8, free_pages=0x30000, F=50, table=0x40000, table_sb=10, max_pages=10, pages=100,
            page_size=16, new_lens=0x50000, q_indptr=0x60000, slots=0x70000, positions=0x80000, T=64, pages_taken=0x90000, stream=None)


@no_gpu
@pytest.mark.parametrize("kw,status", [
    ({}, EDEVICE), (dict(positions=None), EDEVICE), (dict(F=0, free_pages=None), EDEVICE), (dict(T=0, slots=None, positions=None), EDEVICE),
    (dict(B=0, kv_lens=None, q_lens=None, new_lens=None, table=None), EDEVICE), (dict(max_pages=0, table=None), EDEVICE),
    (dict(pages=0), EDEVICE), (dict(B=4096, table=1 << 30, slots=1 << 31, new_lens=1 << 32, q_indptr=1 << 33, positions=1 << 34, pages_taken=1 << 35), EDEVICE),
    (dict(B=-1), EINVAL), (dict(F=-1), EINVAL), (dict(T=-1), EINVAL), (dict(pages=-1), EINVAL), (dict(max_pages=-1), EINVAL),
    (dict(table_sb=-1), EINVAL), (dict(table_sb=9), EINVAL), (dict(table_sb=(1 << 40) + 1), EUNSUPPORTED), (dict(B=1, table_sb=0), EDEVICE),
    (dict(B=4097), EUNSUPPORTED), (dict(page_size=24), EUNSUPPORTED), (dict(page_size=0), EUNSUPPORTED), (dict(pages=1 << 28), EUNSUPPORTED),
    (dict(T=1 << 30), EUNSUPPORTED), (dict(max_pages=1 << 27, table_sb=1 << 27), EUNSUPPORTED), (dict(F=1 << 31), EUNSUPPORTED),
    (dict(kv_lens=None), EINVAL), (dict(q_lens=None), EINVAL), (dict(free_pages=None), EINVAL), (dict(table=None), EINVAL),
    (dict(new_lens=None), EINVAL), (dict(q_indptr=None), EINVAL), (dict(slots=None), EINVAL), (dict(pages_taken=None), EINVAL),
    (dict(kv_lens=0x10002), EALIGN), (dict(slots=0x70001), EALIGN), (dict(pages_taken=0x90002), EALIGN),
    # what is written shares memory with nothing
    (dict(new_lens=0x10000), EINVAL), (dict(new_lens=0x10000 + 28), EINVAL), (dict(new_lens=0x10000 + 32), EDEVICE),
    (dict(q_indptr=0x20000), EINVAL), (dict(slots=0x30000 + 196), EINVAL), (dict(positions=0x70000), EINVAL),
    (dict(pages_taken=0x60000 + 32), EINVAL), (dict(pages_taken=0x60000 + 36), EDEVICE), (dict(slots=0x40000 + 300), EINVAL),
    (dict(kv_lens=0x20000), EDEVICE),  # two inputs may
])
def test_plan_validation(kw, status):
    assert fq.load_library().fp8q_kv4_plan(*{**PLAN, **kw}.values()) == status, fq.fp8q_last_error()


# ------------------------------------------------------------------ the binding
U8, I32 = torch.uint8, torch.int32


def quant():
    return fq.fp8q_mxfp4_quant, dict(x=zeros(4, 256), q=zeros(4, 128, dtype=U8), s=zeros(4, 8, dtype=U8))


def silu():
    return fq.fp8q_silu_mul_mxfp4_quant, dict(x=zeros(4, 512), q=zeros(4, 128, dtype=U8), s=zeros(4, 2, dtype=I32))


def dequant():
    return fq.fp8q_mxfp4_dequant, dict(x=zeros(4, 256), q=zeros(4, 128, dtype=U8), s=zeros(4, 8, dtype=U8))


def product():
    return fq.fp8q_gemm_mxfp4, dict(a=zeros(4, 128, dtype=U8), sa=zeros(4, 2, dtype=I32), b=zeros(6, 128, dtype=U8),
                                    sb=zeros(6, 8, dtype=U8), y=zeros(4, 6), workspace=zeros(256, dtype=U8))


def attend(name, **own):
    cache = dict(zip(("c_k", "c_ks", "c_v", "c_vs"), (zeros(3, 16, 2, w, dtype=U8) for w in (32, 2, 32, 2))))
    return (lambda **kw: with_cache(getattr(fq, name), sm_scale=0.1, **kw)), dict(
        q=zeros(5, 4, 64), block_table=zeros(3, 2, dtype=I32), kv_lens=zeros(3, dtype=I32), out=zeros(5, 4, 64),
        q_indptr=zeros(4, dtype=I32), lse=zeros(5, 4, dtype=torch.float32), workspace=zeros(256, dtype=U8), **cache, **own)


def window():
    fn, kw = attend("fp8q_kv4_window_attention")
    return (lambda **k: fn(window=9, sinks=2, **k)), kw


def tree():
    return attend("fp8q_kv4_tree_attention", tree_mask=zeros(5, 1, dtype=I32))


def plan():
    return (lambda **kw: fq.fp8q_kv4_plan(pages=10, page_size=16, **kw)), dict(
        kv_lens=zeros(3, dtype=I32), q_lens=zeros(3, dtype=I32), free_pages=zeros(5, dtype=I32), block_table=zeros(3, 4, dtype=I32),
        new_lens=zeros(3, dtype=I32), q_indptr=zeros(4, dtype=I32), slots=zeros(7, dtype=I32), pages_taken=zeros(1, dtype=I32),
        positions=zeros(7, dtype=I32))


CALLS = dict(quant=quant, silu=silu, dequant=dequant, product=product, window=window, tree=tree, plan=plan)


@no_gpu
@pytest.mark.parametrize("name", CALLS)
def test_device_tensors_pass(name):
    fn, kw = CALLS[name]()
    with pytest.raises(fq.Fp8qError) as e:
        fn(**kw, stream=0)
    assert e.value.status == EDEVICE


@no_gpu
@pytest.mark.parametrize("name,operand", [(n, o) for n, c in CALLS.items() for o in c()[1]])
def test_a_tensor_elsewhere_is_refused(name, operand):
    fn, kw = CALLS[name]()
    for other in (kw[operand].as_subclass(torch.Tensor), on_gpu(kw[operand].as_subclass(torch.Tensor), 1)):
        with pytest.raises(ValueError):
            fn(**{**kw, operand: other}, stream=0)


@no_gpu
@pytest.mark.parametrize("name,operand", [(n, o) for n, c in CALLS.items() for o in c()[1]])
def test_another_type_or_shape_is_refused(name, operand):
    """Every tensor with a type that no operand has, one row more, and its elements apart."""
    fn, kw = CALLS[name]()
    t = kw[operand]
    if operand == "workspace":
        return
    with pytest.raises(ValueError):
        fn(**{**kw, operand: on_gpu(torch.zeros(t.shape, dtype=torch.float64))}, stream=0)
    if operand != "free_pages" and not operand.startswith("c_"):
        shape = (t.shape[0] + 1,) + tuple(t.shape[1:])
        with pytest.raises(ValueError):
            fn(**{**kw, operand: on_gpu(torch.zeros(shape, dtype=t.dtype))}, stream=0)
    if not (name in ("quant", "silu", "dequant", "product") and operand.startswith("s")) and t.shape[-1] > 1:
        apart = on_gpu(torch.zeros(tuple(t.shape) + (2,), dtype=t.dtype)[..., 0])
        with pytest.raises(ValueError):
            fn(**{**kw, operand: apart}, stream=0)


@no_gpu
def test_widths_that_are_refused():
    with pytest.raises(ValueError):
        fq.fp8q_silu_mul_mxfp4_quant(zeros(4, 255), zeros(4, 64, dtype=U8), zeros(4, 4, dtype=U8), stream=0)
    with pytest.raises(fq.Fp8qError) as e:
        fq.fp8q_mxfp4_quant(zeros(4, 48), zeros(4, 24, dtype=U8), zeros(4, 1, dtype=U8), stream=0)
    assert e.value.status == EINVAL
    with pytest.raises(ValueError):
        fq.mxfp4_quant(torch.zeros(4, 64, dtype=torch.bfloat16), "f32")
