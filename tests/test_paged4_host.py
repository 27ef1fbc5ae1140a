"""CPU-only checks of the cache in 4 bits and of the bookkeeping of shared pages: host-side
validation rejects bad requests before any CUDA call, and the plain implementations that the GPU
tests compare with do what their definitions say."""
import math
import re

import numpy as np
import pytest
import torch

import attention_forward_11_gb300 as fa
from attention_forward_11_gb300 import build as fa_build
from paged4_ref import E2M1, E4M3, decode, encode, plain_fork, plain_free


@pytest.fixture(scope="module", autouse=True)
def lib():
    fa_build.build()
    return fa.load_library()


A = [0x10000000 * (i + 1) for i in range(16)]  # fake, aligned, far apart; never dereferenced
BIG = 1 << 40

FORK = dict(parents=A[0], lens=A[1], kv=A[2], n_seqs=4, page=16, free=A[3], n_free=100, head=A[4], table=A[5], max_pages=50,
            table_stride=50, shares=A[6], n_pages=300, copies=A[7], counts=A[8], stream=0)
FREE = dict(kv=A[0], keep=A[1], n_seqs=4, page=16, table=A[2], max_pages=50, table_stride=50, shares=A[3], n_pages=300,
            free=A[4], n_free=100, head=A[5], counts=A[6], stream=0)
APPEND = dict(k=A[0], v=A[1], slots=A[2], kc=A[3], ks=A[4], vc=A[5], vs=A[6], T=7, Hkv=2, D=128, n_pages=9, page=16, k_stride=256,
              v_stride=256, cps=16 * 128, cts=128, chs=64, sps=16 * 16, sts=16, shs=8, ku=1.0, vu=1.0, dtype=0, stream=0)
FWD = dict(q=A[0], kc=A[1], ks=A[2], vc=A[3], vs=A[4], o=A[5], lse=A[6], table=A[7], cu=A[8], kv=A[9], n_seqs=4, T=40, max_q=10,
           Hq=4, Hkv=2, D=128, n_pages=9, page=16, max_pages=5, qs=512, table_stride=5, cps=16 * 128, cts=128, chs=64, sps=16 * 16,
           sts=16, shs=8, causal=1, scale=0.088, ku=1.0, vu=1.0, dtype=0, ws=A[10], ws_bytes=BIG, stream=0)


def ids(d):
    return ",".join(f"{k}={v}" for k, v in d.items())


@pytest.mark.parametrize("over", [
    dict(parents=0), dict(kv=0), dict(table=0), dict(shares=0), dict(copies=0), dict(counts=0), dict(free=0), dict(n_seqs=0),
    dict(page=0), dict(n_free=-1), dict(max_pages=0), dict(n_pages=0), dict(table_stride=49), dict(table_stride=1 << 62),
    dict(parents=A[0] + 2), dict(lens=A[1] + 1), dict(copies=A[7] + 2), dict(kv=A[0]), dict(kv=A[1] + 12), dict(table=A[2] - 4),
    dict(table=A[6] + 4), dict(shares=A[3] + 396), dict(copies=A[2]), dict(counts=A[4]), dict(counts=A[7] + 44),
    dict(free=A[5] + 4 * 199),
], ids=ids)
def test_fork_refusals(over):
    assert fa.attn_paged_fork_ptr(*{**FORK, **over}.values()) == fa.ATTN_ERR_INVALID_ARG


@pytest.mark.parametrize("over", [
    dict(kv=0), dict(keep=0), dict(table=0), dict(shares=0), dict(free=0), dict(head=0), dict(counts=0), dict(n_seqs=0),
    dict(page=0), dict(max_pages=0), dict(n_pages=0), dict(n_free=0), dict(table_stride=49), dict(kv=A[0] + 1),
    dict(head=A[5] + 2), dict(shares=A[2]), dict(free=A[0]), dict(free=A[3] + 4 * 299), dict(counts=A[1]), dict(counts=A[5]),
    dict(head=A[4] + 40), dict(counts=A[4] + 396),
], ids=ids)
def test_free_refusals(over):
    assert fa.attn_paged_free_ptr(*{**FREE, **over}.values()) == fa.ATTN_ERR_INVALID_ARG


def copy_args(ptrs=(A[1], A[2]), **over):
    import ctypes
    d = dict(copies=A[0], n=5, caches=(ctypes.c_void_p * max(len(ptrs), 1))(*ptrs), m=len(ptrs), n_pages=9, page=16, Hkv=2,
             row=256, ps=16 * 512, ts=512, hs=256, stream=0)
    return {**d, **over}.values()


@pytest.mark.parametrize("over", [
    dict(copies=0), dict(n=0), dict(caches=None), dict(m=0), dict(n_pages=0), dict(page=0), dict(Hkv=0), dict(row=0), dict(row=254),
    dict(row=2), dict(ps=0), dict(ts=256), dict(hs=128), dict(hs=258), dict(ps=16 * 512 - 4), dict(copies=A[0] + 2),
    dict(ptrs=(A[1], 0)), dict(ptrs=(A[1] + 2,)), dict(ptrs=(A[1], A[0] - 64)), dict(ps=1 << 61),
], ids=ids)
def test_copy_refusals(over):
    assert fa.attn_paged_copy_ptr(*copy_args(**over)) == fa.ATTN_ERR_INVALID_ARG


def test_copy_of_enormous_pages_is_unsupported():
    args = copy_args(page=1 << 22, Hkv=2, row=256, ps=1 << 40, ts=512, hs=256)
    assert fa.attn_paged_copy_ptr(*args) == fa.ATTN_ERR_UNSUPPORTED


@pytest.mark.parametrize("over", [
    dict(k=0), dict(v=0), dict(slots=0), dict(kc=0), dict(ks=0), dict(vc=0), dict(vs=0), dict(T=0), dict(Hkv=0), dict(D=0),
    dict(n_pages=0), dict(page=0), dict(k_stride=248), dict(v_stride=260), dict(k_stride=-256), dict(cps=0), dict(cts=64),
    dict(chs=32), dict(chs=72), dict(cps=16 * 128 - 16), dict(sps=0), dict(sts=8), dict(shs=4), dict(shs=12), dict(k=A[0] + 8),
    dict(kc=A[3] + 8), dict(ks=A[4] + 4), dict(slots=A[2] + 4), dict(vc=A[3]), dict(vs=A[4]), dict(ks=A[3]), dict(k=A[3] + 2048),
    dict(v=A[6] - 16), dict(slots=A[5] + 8), dict(ku=0.0), dict(ku=-1.0), dict(vu=math.nan), dict(vu=math.inf), dict(ku=1e-45),
    dict(dtype=2), dict(cps=1 << 61),
], ids=ids)
def test_append_refusals(over):
    assert fa.attn_paged_coded_append_ptr(*{**APPEND, **over}.values()) == fa.ATTN_ERR_INVALID_ARG


@pytest.mark.parametrize("over", [
    dict(q=0), dict(kc=0), dict(ks=0), dict(vc=0), dict(vs=0), dict(o=0), dict(table=0), dict(cu=0), dict(kv=0), dict(n_seqs=0),
    dict(T=0), dict(max_q=0), dict(Hq=0), dict(Hkv=0), dict(Hq=3), dict(D=0), dict(n_pages=0), dict(page=0), dict(max_pages=0),
    dict(qs=504), dict(qs=516), dict(table_stride=4), dict(cps=16), dict(cts=8), dict(chs=0), dict(sps=8), dict(sts=4), dict(shs=0),
    dict(causal=2), dict(causal=-1), dict(scale=0.0), dict(scale=math.nan), dict(scale=math.inf), dict(scale=-1.0), dict(dtype=2),
    dict(ku=0.0), dict(vu=-2.0), dict(ku=math.inf), dict(scale=1e-30, ku=1e-30), dict(scale=1e30, ku=1e30), dict(q=A[0] + 8),
    dict(kc=A[1] + 8), dict(vs=A[4] + 4), dict(o=A[5] + 2), dict(lse=A[6] + 2), dict(table=A[7] + 2), dict(cu=A[8] + 1),
    dict(o=A[0]), dict(o=A[1] + 64), dict(o=A[2]), dict(o=A[3]), dict(o=A[4]), dict(lse=A[5] + 16), dict(lse=A[7]),
    dict(o=A[8] - 4096), dict(ws=A[10] + 16),
], ids=ids)
def test_fwd_refusals(over):
    assert fa.attn_paged_coded_fwd_ptr(*{**FWD, **over}.values()) == fa.ATTN_ERR_INVALID_ARG


@pytest.mark.parametrize("D", [32, 96, 192, 320])
def test_other_head_sizes_unsupported(D):
    assert fa.attn_paged_coded_append_ptr(*{**APPEND, "D": D}.values()) == fa.ATTN_ERR_UNSUPPORTED
    assert fa.attn_paged_coded_fwd_ptr(*{**FWD, "D": D}.values()) == fa.ATTN_ERR_UNSUPPORTED
    with pytest.raises(fa.AttnError) as e:
        fa.attn_paged_coded_fwd_workspace_size(40, 10, 4, 2, D, 16)
    assert e.value.status == fa.ATTN_ERR_UNSUPPORTED


@pytest.mark.parametrize("args", [(0, 1, 4, 2, 128, 16), (4, 0, 4, 2, 128, 16), (4, 1, 3, 2, 128, 16),
                                  (4, 1, 4, 0, 128, 16), (4, 1, 4, 2, 128, 0), (4, 1, 4, 2, 0, 16)])
def test_workspace_size_refusals(args):
    with pytest.raises(fa.AttnError) as e:
        fa.attn_paged_coded_fwd_workspace_size(*args)
    assert e.value.status == fa.ATTN_ERR_INVALID_ARG


def test_binding_refuses_host_tensors():
    i = torch.zeros(2, dtype=torch.int32)
    t = torch.zeros(2, 3, dtype=torch.int32)
    c, s = torch.zeros(2, 16, 2, 32, dtype=torch.uint8), torch.zeros(2, 16, 2, 4, dtype=torch.uint8)
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    for call in (lambda: fa.attn_paged_fork(i, i, i, t, 16, i), lambda: fa.attn_paged_free(i, i, t, 16, i, i, i[:1]),
                 lambda: fa.attn_paged_copy(torch.zeros(2, 3, dtype=torch.int32), [c]), lambda: fa.attn_paged_copy(t, []),
                 lambda: fa.attn_paged_coded_append(k, k, torch.zeros(3, dtype=torch.int64), c, s, c, s),
                 lambda: fa.attn_paged_coded_fwd(k, c, s, c, s, t, torch.zeros(3, dtype=torch.int32), i)):
        with pytest.raises(fa.AttnError) as e:
            call()
        assert e.value.status == fa.ATTN_ERR_INVALID_ARG


def recorded(monkeypatch, name):
    """Argument tuples that the binding hands to a C entry point, which is not called."""
    calls = []
    monkeypatch.setattr(fa._binding, name, lambda *args: calls.append(args) or fa.ATTN_OK)
    return calls


def test_binding_passes_what_the_header_names(monkeypatch):
    """The number of arguments, and the strides of codes and scales in bytes."""
    header = re.sub(r"/\*.*?\*/", "", open(fa_build.ROOT + "/include/attn.h").read(), flags=re.S)

    def declared(name):
        return len(re.search(r"\b%s\(([^)]*)\)" % name, header).group(1).split(","))

    codes = torch.zeros(3, 2, 16, 64, dtype=torch.uint8).transpose(1, 2)  # head by head
    scales = torch.zeros(3, 2, 16, 8, dtype=torch.float8_e4m3fn).transpose(1, 2)
    i = torch.zeros(2, dtype=torch.int32)
    table = torch.zeros(2, 5, dtype=torch.int32)
    q = torch.zeros(4, 6, 128, dtype=torch.float16)
    calls = recorded(monkeypatch, "attn_paged_coded_fwd_ptr")
    ws = torch.zeros(64, dtype=torch.uint8)
    fa._binding._paged4_fwd(torch, 0, q, codes, scales, codes, scales, table, torch.zeros(3, dtype=torch.int32), i, 2, 1, None,
                            0.5, 2.0, None, None, ws, True)
    assert len(calls[0]) == declared("attn_paged_coded_fwd")
    assert calls[0][19:27] == (768, 5, 2048, 64, 1024, 256, 8, 128) and calls[0][27:33] == (1, 128 ** -0.5, 0.5, 2.0, 1, ws.data_ptr())
    calls = recorded(monkeypatch, "attn_paged_fork_ptr")
    fa._binding._paged_fork(torch, 0, i, i, i, table, 16, i, None, None, None, None)
    assert len(calls[0]) == declared("attn_paged_fork")
    calls = recorded(monkeypatch, "attn_paged_free_ptr")
    fa._binding._paged_free(torch, 0, i, i, table, 16, i, i, i[:1], None)
    assert len(calls[0]) == declared("attn_paged_free")
    monkeypatch.setattr(fa._binding, "_on_one_gpu", lambda *t: 0)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    calls = recorded(monkeypatch, "attn_paged_copy_ptr")
    fa.attn_paged_copy(torch.zeros(2, 3, dtype=torch.int32), [codes, scales, codes.clone(), scales])
    assert len(calls) == 2 and len(calls[0]) == declared("attn_paged_copy")
    assert calls[0][3:11] == (2, 3, 16, 2, 64, 2048, 64, 1024) and calls[1][3:11] == (2, 3, 16, 2, 8, 256, 8, 128)
    calls = recorded(monkeypatch, "attn_paged_coded_append_ptr")
    k = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    fa.attn_paged_coded_append(k, k, torch.zeros(4, dtype=torch.int64), codes, scales, codes, scales, k_unit=0.5)
    assert len(calls[0]) == declared("attn_paged_coded_append") and calls[0][12:23] == (256, 256, 2048, 64, 1024, 256, 8, 128, 0.5, 1.0, 0)


@pytest.mark.parametrize("over", [dict(codes=torch.zeros(3, 16, 2, 64)), dict(scales=torch.zeros(3, 16, 2, 4, dtype=torch.uint8)),
                                  dict(scales=torch.zeros(3, 16, 1, 8, dtype=torch.uint8)), dict(other=torch.zeros(3, 2, 16, 64, dtype=torch.uint8).transpose(1, 2)),
                                  dict(codes=torch.zeros(3, 16, 64, 2, dtype=torch.uint8).transpose(2, 3))], ids=range(5))
def test_caches_of_other_shapes_and_strides_are_refused(over):
    codes = over.get("codes", torch.zeros(3, 16, 2, 64, dtype=torch.uint8))
    scales = over.get("scales", torch.zeros(3, 16, 2, 8, dtype=torch.uint8))
    with pytest.raises(fa.AttnError):
        fa._binding._cache4_shape(torch, codes, scales, over.get("other", codes), scales)


# ------------------------------------------------------------------ the plain implementations
def test_e4m3_is_torchs():
    ours = E4M3
    theirs = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ours, theirs, equal_nan=True)


def test_every_product_of_a_code_and_a_scale_is_exact_in_16_bits():
    products = np.multiply.outer(E2M1, E4M3[:127]).ravel()
    assert (products.astype(np.float16).astype(np.float64) == products).all()
    assert (torch.tensor(products).bfloat16().double().numpy() == products).all()


def test_plain_encode_by_hand():
    x = np.array([6.0, -3.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.0, 0.0, 0.2, 0.3, -5.1, 4.9, 1.0], dtype=np.float32)
    c, s = encode(x, 1.0)
    assert s.tolist() == [0x38]  # 1.0
    v = decode(c, s, 1.0)
    assert v.tolist() == [6, -3, 0, 1, 1, 2, 2, 4, 4, 0, 0, 0, .5, -6, 4, 1]
    assert np.signbit(v[9]) and not np.signbit(v[10])
    c, s = encode(2 * x, 0.25)  # half of it: a scale of 0.5
    assert s.tolist() == [0x30] and np.array_equal(decode(c, s, 4.0), 2 * v)
    assert encode(np.zeros(16, np.float32), 1.0)[1].tolist() == [0]
    assert encode(np.full(16, 1e-20, np.float32), 1.0)[1].tolist() == [1]
    c, s = encode(np.array([np.nan, np.inf, -np.inf] + [1.0] * 13, dtype=np.float32), 1.0)
    assert s.tolist() == [0x7e] and decode(c, s, 1.0)[:3].tolist() == [2688, 2688, -2688]


def test_plain_encode_is_the_nearest():
    """No other code of a block's scale is nearer, and the scale is the nearest to a sixth of the largest."""
    x = torch.randn(200, 128, generator=torch.Generator().manual_seed(1)).numpy()
    c, s = encode(x, 1.0)
    by = np.repeat(E4M3[s], 16, axis=-1)
    v = decode(c, s, 1.0)
    best = np.abs(E2M1[None, None] * by[..., None] - x[..., None]).min(-1)
    assert np.allclose(np.abs(v - x), best, rtol=0, atol=1e-12)
    sixth = np.abs(x.reshape(200, 8, 16)).max(-1) / 6
    assert (np.abs(E4M3[s] - sixth) <= np.abs(E4M3[:127] - sixth[..., None]).min(-1) + 1e-12).all()


def test_plain_fork_and_free_by_hand():
    table = [[5, 6, 7], [-9, -9, -9], [-9, -9, -9], [1, -9, -9]]
    kv, t, shares, copies, counts = plain_fork([-1, 0, 0, -1], [0, 99, 32, 0], [40, 0, 0, 3], [8, 9], 1, table, 16, [0] * 10)
    assert kv == [40, 40, 32, 3] and t == [[5, 6, 7], [5, 6, 9], [5, 6, -9], [1, -9, -9]]
    assert shares == [0, 0, 0, 0, 0, 2, 2, 0, 0, 0] and copies == [[-1, -1, 0], [7, 9, 8], [-1, -1, 0], [-1, -1, 0]]
    assert counts == [2, 2, 0, 0]
    shares, free, counts = plain_free(kv, [0, 20, 32, 0], t, 16, shares, [-1] * 9 + [8], 9)
    assert shares == [0, 0, 0, 0, 0, 1, 1, 0, 0, 0] and free == [-1] * 6 + [1, 7, 9, 8] and counts == [3, 6, 0, 1]
