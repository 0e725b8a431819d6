"""Host-side checks of the quantizing norm's and the 4-bit cache's entry points: every refusal of
the C ABI with its status, and the binding's checks of tensors. No compute call runs: validation
returns before the library touches a pointer or the device, so the addresses are never used."""
import ctypes
import math

import pytest
import torch

import fp8_group_quant_amd as fq

OK, EINVAL, EUNSUPPORTED, EALIGN, EDEVICE = 0, 1, 2, 3, 4
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="checks host validation on a machine without a GPU")

NORM = dict(x=0x10000, in_dtype=0, M=8, K=512, x_sm=512, residual=0x20000, r_sm=512, residual_out=0x30000, ro_sm=512,
            weight=0x40000, eps=1e-6, q=0x50000, q_sm=512, s=0x60000, scale_fmt=1, s_sm=1, s_sg=8, group_size=128,
            stream=None)


def norm(**kw):
    return fq.load_library().fp8q_rms_norm_group_quant(*{**NORM, **kw}.values())


@no_gpu
@pytest.mark.parametrize("kw,status", [
    ({}, EDEVICE),  # valid: stopped by the missing device only
    (dict(residual=None, residual_out=None), EDEVICE),
    (dict(residual_out=None), EDEVICE),
    (dict(residual=None), EINVAL),                      # residual_out without a residual
    (dict(M=0, x=None), OK), (dict(K=0, group_size=128, x=None), OK),
    (dict(in_dtype=3), EUNSUPPORTED), (dict(scale_fmt=3), EUNSUPPORTED), (dict(group_size=256), EUNSUPPORTED),
    (dict(group_size=0), EUNSUPPORTED), (dict(group_size=-128), EUNSUPPORTED),
    (dict(M=-1), EINVAL), (dict(K=500), EINVAL), (dict(K=520, group_size=520, s_sm=1, s_sg=1), EINVAL),
    (dict(K=65536 + 128, x_sm=1 << 17, r_sm=1 << 17, ro_sm=1 << 17, q_sm=1 << 17), EUNSUPPORTED),
    (dict(K=65536, x_sm=1 << 17, r_sm=1 << 17, ro_sm=1 << 17, q_sm=1 << 17), EDEVICE),
    (dict(eps=-1.0), EINVAL), (dict(eps=math.inf), EINVAL), (dict(eps=math.nan), EINVAL), (dict(eps=0.0), EDEVICE),
    (dict(x=None), EINVAL), (dict(weight=None), EINVAL), (dict(q=None), EINVAL), (dict(s=None), EINVAL),
    (dict(x_sm=-512), EINVAL), (dict(x_sm=0), EDEVICE),  # one input row for all is fine
    (dict(q_sm=256), EINVAL), (dict(ro_sm=256), EINVAL), (dict(s_sm=2, s_sg=3), EINVAL), (dict(s_sg=4), EINVAL),
    (dict(s_sm=4, s_sg=1), EDEVICE),
    (dict(scale_fmt=2, s_sm=1, s_sg=8), EDEVICE), (dict(scale_fmt=2, group_size=512), EINVAL),
    (dict(scale_fmt=2, s=0x60002), EALIGN), (dict(scale_fmt=0, s=0x60002), EALIGN), (dict(s=0x60001), EDEVICE),
    (dict(x=0x10008), EALIGN), (dict(x_sm=516), EALIGN), (dict(weight=0x40004), EALIGN), (dict(residual=0x20008), EALIGN),
    (dict(r_sm=513), EALIGN), (dict(residual_out=0x30008), EALIGN), (dict(q=0x50008), EALIGN), (dict(q_sm=520), EALIGN),
])
def test_norm_validation(kw, status):
    assert norm(**kw) == status, fq.fp8q_last_error()


CACHE = dict(kc=0x100000, ks=0x200000, vc=0x300000, vs=0x400000, pages=10, page_size=16, c_sp=2 * 16 * 64, c_st=64,
             c_sh=16 * 64, s_sp=2 * 16 * 4, s_st=4, s_sh=16 * 4)
ROWS = dict(k=0x10000, k_st=256, k_sh=128, v=0x20000, v_st=256, v_sh=128, dtype=0, T=5, H=2, D=128, slots=0x30000, **CACHE,
            stream=None)

CACHE_CASES = [
    ({}, EDEVICE),
    (dict(c_st=128, c_sh=64, c_sp=16 * 128, s_st=8, s_sh=4, s_sp=16 * 8), EDEVICE),  # a token's heads adjacent
    (dict(D=96), EUNSUPPORTED), (dict(D=0), EUNSUPPORTED), (dict(page_size=24), EUNSUPPORTED),
    (dict(page_size=0), EUNSUPPORTED), (dict(page_size=-16), EUNSUPPORTED),
    (dict(pages=1 << 28), EUNSUPPORTED), (dict(pages=(1 << 62)), EUNSUPPORTED), (dict(pages=-1), EINVAL),
    (dict(c_sp=-64), EINVAL), (dict(s_sh=-4), EINVAL),
    (dict(kc=None), EINVAL), (dict(vs=None), EINVAL),
    (dict(kc=0x100008), EALIGN), (dict(vc=0x300004), EALIGN), (dict(c_st=72), EALIGN), (dict(ks=0x200002), EALIGN),
    (dict(s_st=6), EALIGN),
]


@no_gpu
@pytest.mark.parametrize("entry", ["fp8q_kv4_write", "fp8q_kv4_read"])
@pytest.mark.parametrize("kw,status", CACHE_CASES + [
    (dict(T=0, k=None), OK), (dict(H=0, slots=None), OK),
    (dict(dtype=3), EUNSUPPORTED), (dict(T=-1), EINVAL), (dict(T=1 << 31), EUNSUPPORTED), (dict(H=-1), EINVAL),
    (dict(H=(1 << 20) + 1), EUNSUPPORTED), (dict(k=None), EINVAL), (dict(slots=None), EINVAL),
    (dict(k_st=-1), EINVAL), (dict(k=0x10008), EALIGN), (dict(v_sh=132, v_st=512), EALIGN), (dict(slots=0x30002), EALIGN),
    (dict(dtype=2, k_st=252), EDEVICE),  # fp32: 4 elements are 16 bytes; for reads the rows overlap
])
def test_rows_validation(entry, kw, status):
    if entry == "fp8q_kv4_read" and kw.get("k_st") == 252:
        status = EINVAL
    rc = getattr(fq.load_library(), entry)(*{**ROWS, **kw}.values())
    assert rc == status, fq.fp8q_last_error()


@no_gpu
def test_overlapping_rows():
    lib = fq.load_library()
    over = dict(c_st=48)  # a token's row is 64 bytes
    assert lib.fp8q_kv4_write(*{**ROWS, **over}.values()) == EINVAL
    assert lib.fp8q_kv4_read(*{**ROWS, **over}.values()) == EDEVICE  # reading them is allowed
    assert lib.fp8q_kv4_write(*{**ROWS, "s_sp": 4}.values()) == EINVAL
    same = dict(k_sh=0)  # one head's rows for all: fine as input, not as output
    assert lib.fp8q_kv4_write(*{**ROWS, **same}.values()) == EDEVICE
    assert lib.fp8q_kv4_read(*{**ROWS, **same}.values()) == EINVAL


ATTN = dict(q=0x10000, dtype=0, q_st=8 * 128, q_sh=128, **CACHE, table=0x20000, table_sb=4, max_pages=4,
            kv_lens=0x30000, q_indptr=0x40000, out=0x50000, o_st=8 * 128, o_sh=128, lse=0x60000, l_st=8, B=3, T=7, Hq=8,
            Hkv=2, D=128, sm_scale=0.1, causal=1, workspace=None, workspace_bytes=0, stream=None)


@no_gpu
@pytest.mark.parametrize("kw,status", CACHE_CASES + [
    (dict(lse=None), EDEVICE), (dict(q_indptr=None, T=3), EDEVICE), (dict(q_indptr=None), EINVAL),
    (dict(B=0, kv_lens=None), OK), (dict(T=0, q=None), OK), (dict(Hq=0, Hkv=0), OK),
    (dict(dtype=2), EUNSUPPORTED), (dict(Hkv=0), EINVAL), (dict(Hkv=3), EINVAL), (dict(Hq=-8), EINVAL),
    (dict(B=4097), EUNSUPPORTED), (dict(B=4096), EDEVICE), (dict(T=1 << 28), EUNSUPPORTED), (dict(T=1 << 31), EUNSUPPORTED),
    (dict(max_pages=1 << 27), EUNSUPPORTED), (dict(max_pages=-1), EINVAL), (dict(max_pages=1 << 40), EINVAL),
    (dict(max_pages=0, table=None), EDEVICE), (dict(table=None), EINVAL), (dict(kv_lens=None), EINVAL),
    (dict(q=None), EINVAL), (dict(out=None), EINVAL), (dict(sm_scale=math.inf), EINVAL), (dict(sm_scale=math.nan), EINVAL),
    (dict(q_st=-8), EINVAL), (dict(table_sb=-1), EINVAL), (dict(table_sb=0), EDEVICE),
    (dict(o_sh=64), EINVAL), (dict(o_st=128), EINVAL), (dict(o_st=128, o_sh=7 * 128), EDEVICE), (dict(l_st=4), EINVAL),
    (dict(q=0x10008), EALIGN), (dict(q_sh=132), EALIGN), (dict(out=0x50008), EALIGN), (dict(o_sh=129, o_st=2048), EALIGN),
    (dict(lse=0x60001), EALIGN), (dict(table=0x20002), EALIGN), (dict(workspace=0x70008), EALIGN),
    (dict(workspace_bytes=-1), EINVAL), (dict(pages=0, kc=None, ks=None, vc=None, vs=None), EDEVICE),
])
def test_attention_validation(kw, status):
    assert fq.load_library().fp8q_kv4_attention(*{**ATTN, **kw}.values()) == status, fq.fp8q_last_error()


@no_gpu
def test_workspace_size_without_a_device_or_with_refused_sizes():
    size = fq.load_library().fp8q_kv4_attention_workspace_size
    assert size(0, 1, 1, 32, 8, 128, 100000) == 0
    assert size(0, 1, 1, 32, 8, 96, 100000) == 0 and size(0, -1, 1, 32, 8, 128, 100) == 0
    assert size(2, 1, 1, 32, 8, 128, 100000) == 0


def test_binding_refuses_tensors_that_do_not_fit():
    bf = torch.bfloat16
    x, w = torch.zeros(4, 256, dtype=bf), torch.zeros(256, dtype=bf)
    q, s = torch.zeros(4, 256, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    for args, kw in [((x[0], w, q, s), {}), ((x, w.float(), q, s), {}), ((x, w[:128], q, s), {}),
                     ((x, w, q[:, :128], s), {}), ((x, w, q, s.t()), {}), ((x, w, q, s.to(torch.int16)), {}),
                     ((x, w, q.to(torch.int16), s), {}), ((x.to(torch.float64), w, q, s), {}),
                     ((x, w, q, s), dict(residual=x.float())), ((x, w, q, s), dict(residual=x[:2])),
                     ((torch.zeros(256, 4, dtype=bf).t(), w, q, s), {}), ((x, w, q, s, 0), {})]:
        with pytest.raises(ValueError):
            fq.fp8q_rms_norm_group_quant(*args, **kw)
    for layout in ("head", "token"):
        c = fq.alloc_kv4_cache(3, 16, 2, 64, layout, device="cpu")
        assert c.k.shape == (3, 16, 2, 32) and c.k_scales.shape == (3, 16, 2, 2)
        assert (c.k.stride(1) == 32) == (layout == "head")
    with pytest.raises(ValueError):
        fq.alloc_kv4_cache(3, 16, 2, 64, "page", device="cpu")
    kv = torch.zeros(5, 2, 64, dtype=bf)
    slots = torch.zeros(5, dtype=torch.int32)
    for k, v, sl in [(kv, kv[:, :1], slots), (kv, kv.float(), slots), (kv[0], kv[0], slots), (kv, kv, slots.long()),
                     (kv, kv, slots)]:  # the last: slots on the host
        with pytest.raises(ValueError):
            fq.fp8q_kv4_write(k, v, sl, c)
    for bad in [c._replace(v=c.v[:2]), c._replace(k=c.k.int()), c._replace(k_scales=c.k_scales[..., :1]),
                c._replace(v=c.v.transpose(1, 2).contiguous().transpose(1, 2))]:
        with pytest.raises(ValueError):
            fq._kv4_args(bad, 2, 64)
    with pytest.raises(ValueError):
        fq._kv4_args(c, 2, 128)
    with pytest.raises(ValueError):  # fp32 queries
        fq.fp8q_kv4_attention(torch.zeros(3, 2, 64), c, slots, slots, torch.zeros(3, 2, 64), 0.1)
