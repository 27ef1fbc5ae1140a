"""CPU-only checks of the paged cache's entry points: host-side validation rejects
bad requests before any CUDA call, and the plain implementation that the GPU tests
compare with agrees with attention over dense tensors."""
import math

import numpy as np
import pytest
import torch

import attention_forward_11_gb300 as fa
import oracle
from attention_forward_11_gb300 import build as fa_build
from paged_ref import Batch, plain_tables


@pytest.fixture(scope="module", autouse=True)
def lib():
    fa_build.build()
    oracle.build()
    return fa.load_library()


A = [0x10000000 * (i + 1) for i in range(16)]  # fake, aligned, far apart; never dereferenced
BIG = 1 << 40

TABLES = dict(ctx=A[0], new=A[1], n_seqs=4, page=16, free=A[2], n_free=100, head=A[3], table=A[4], max_pages=50,
              table_stride=50, cu=A[5], kv=A[6], slots=A[7], max_tokens=300, counts=A[8], stream=0)
APPEND = dict(k=A[0], v=A[1], slots=A[2], kc=A[3], vc=A[4], T=7, Hkv=2, D=128, n_pages=9, page=16, ks=256, vs=256,
              ps=16 * 256, ts=256, hs=128, stream=0)
FWD = dict(q=A[0], kc=A[1], vc=A[2], o=A[3], lse=A[4], table=A[5], cu=A[6], kv=A[7], n_seqs=4, T=40, max_q=10, Hq=4,
           Hkv=2, D=128, n_pages=9, page=16, max_pages=5, qs=512, table_stride=5, ps=16 * 256, ts=256, hs=128, causal=1,
           scale=0.088, dtype=0, ws=A[8], ws_bytes=BIG, stream=0)


def ids(d):
    return ",".join(f"{k}={v}" for k, v in d.items())


@pytest.mark.parametrize("over", [
    dict(ctx=0), dict(new=0), dict(table=0), dict(cu=0), dict(kv=0), dict(slots=0), dict(counts=0), dict(free=0),
    dict(n_seqs=0), dict(page=0), dict(n_free=-1), dict(max_pages=0), dict(max_tokens=0), dict(max_tokens=-5),
    dict(table_stride=49), dict(table_stride=1 << 62), dict(ctx=A[0] + 2), dict(slots=A[7] + 4), dict(head=A[3] + 1),
    dict(table=A[0]), dict(cu=A[1] + 4), dict(kv=A[4] + 8), dict(slots=A[2] + 8), dict(counts=A[3]),
    dict(counts=A[7] + 8 * 299), dict(free=A[4] + 4 * 199),
], ids=ids)
def test_tables_refusals(over):
    assert fa.attn_paged_tables_ptr(*{**TABLES, **over}.values()) == fa.ATTN_ERR_INVALID_ARG


@pytest.mark.parametrize("over", [
    dict(k=0), dict(v=0), dict(slots=0), dict(kc=0), dict(vc=0), dict(T=0), dict(Hkv=0), dict(D=0), dict(n_pages=0),
    dict(page=0), dict(ks=248), dict(vs=260), dict(ks=-256), dict(ps=0), dict(ts=128), dict(hs=64), dict(hs=132),
    dict(ps=16 * 256 - 8), dict(k=A[0] + 8), dict(kc=A[3] + 2), dict(slots=A[2] + 4), dict(vc=A[3]),
    dict(k=A[3] + 16 * 256), dict(slots=A[4] + 8), dict(ps=1 << 61),
], ids=ids)
def test_append_refusals(over):
    assert fa.attn_paged_append_ptr(*{**APPEND, **over}.values()) == fa.ATTN_ERR_INVALID_ARG


@pytest.mark.parametrize("over", [
    dict(q=0), dict(kc=0), dict(vc=0), dict(o=0), dict(table=0), dict(cu=0), dict(kv=0), dict(n_seqs=0), dict(T=0),
    dict(max_q=0), dict(Hq=0), dict(Hkv=0), dict(Hq=3), dict(D=0), dict(n_pages=0), dict(page=0), dict(max_pages=0),
    dict(qs=504), dict(qs=516), dict(table_stride=4), dict(ps=8), dict(ts=8), dict(hs=0), dict(causal=2),
    dict(causal=-1), dict(scale=0.0), dict(scale=math.nan), dict(scale=math.inf), dict(scale=-1.0), dict(dtype=2),
    dict(q=A[0] + 8), dict(kc=A[1] + 4), dict(o=A[3] + 2), dict(lse=A[4] + 2), dict(table=A[5] + 2), dict(cu=A[6] + 1),
    dict(o=A[0]), dict(o=A[1] + 64), dict(o=A[2]), dict(lse=A[3] + 16), dict(lse=A[5]), dict(o=A[6] - 4096),
    dict(ws=A[8] + 16),
], ids=ids)
def test_fwd_refusals(over):
    assert fa.attn_paged_fwd_ptr(*{**FWD, **over}.values()) == fa.ATTN_ERR_INVALID_ARG


@pytest.mark.parametrize("D", [32, 96, 192, 320])
def test_other_head_sizes_unsupported(D):
    assert fa.attn_paged_append_ptr(*{**APPEND, "D": D}.values()) == fa.ATTN_ERR_UNSUPPORTED
    assert fa.attn_paged_fwd_ptr(*{**FWD, "D": D}.values()) == fa.ATTN_ERR_UNSUPPORTED
    with pytest.raises(fa.AttnError) as e:
        fa.attn_paged_fwd_workspace_size(40, 10, 4, 2, D, 16)
    assert e.value.status == fa.ATTN_ERR_UNSUPPORTED


@pytest.mark.parametrize("args", [(0, 1, 4, 2, 128, 16), (4, 0, 4, 2, 128, 16), (4, 1, 3, 2, 128, 16),
                                  (4, 1, 4, 0, 128, 16), (4, 1, 4, 2, 128, 0), (4, 1, 4, 2, 0, 16)])
def test_workspace_size_refusals(args):
    with pytest.raises(fa.AttnError) as e:
        fa.attn_paged_fwd_workspace_size(*args)
    assert e.value.status == fa.ATTN_ERR_INVALID_ARG


def test_binding_refuses_host_tensors():
    b = Batch([(20, 3)], 4, 2, 64, 16, device="cpu")
    with pytest.raises(fa.AttnError) as e:
        fa.attn_paged_fwd(**b.on_gpu())
    assert e.value.status == fa.ATTN_ERR_INVALID_ARG
    with pytest.raises(fa.AttnError):
        fa.attn_paged_append(b.q[:, :2], b.q[:, :2], torch.zeros(3, dtype=torch.int64), b.k_cache, b.v_cache)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(fa.AttnError):
        fa.attn_paged_tables(i, i, i, b.table, 16, 4)


@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("layout", ["tokens", "heads", "turns"])
def test_plain_attention_is_the_dense_one(causal, layout):
    """The paged reference against the framework's 64-bit oracle, sequence by sequence."""
    lens = [(70, 5), (16, 16), (33, 1), (4, 9)]
    b = Batch(lens, 4, 2, 64, 16, causal=causal, layout=layout, device="cpu", seed=3)
    o, lse, _, _ = b.reference()
    for s, (kv, n) in enumerate(lens):
        pages = b.table[s, :-(-kv // 16)].long()
        k, v = (c[pages].reshape(-1, 2, 64)[:kv] for c in (b.k_cache, b.v_cache))
        assert torch.equal(k, b.dense[s][0]) and torch.equal(v, b.dense[s][1])
        a = b.cu[s]
        bits = [np.ascontiguousarray(x[None].contiguous().view(torch.int16).numpy()).view(np.uint16)
                for x in (b.q[a:a + n], k, v)]
        ro, rl = oracle.attn_full(*bits, causal, b.scale)
        assert np.abs(o[a:a + n] - ro[0]).max() < 1e-6
        assert np.array_equal(np.isneginf(lse[:, a:a + n]), np.isneginf(rl[0]))
        fin = ~np.isneginf(rl[0])
        assert np.abs(lse[:, a:a + n][fin] - rl[0][fin]).max() < 1e-6


def test_plain_tables_by_hand():
    table, cu, kv, slots, counts = plain_tables([3, 0, 4], [3, 0, 1], [7, 8, 9], 1, [[5, -1], [-1, -1], [6, -1]], 4, 6)
    assert table == [[5, 8], [-1, -1], [6, 9]]
    assert cu == [0, 3, 3, 4] and kv == [6, 0, 5] and counts == [4, 3, 0, 0]
    assert slots == [5 * 4 + 3, 8 * 4, 8 * 4 + 1, 9 * 4, -1, -1]


def recorded(monkeypatch, name):
    """Argument tuples that the binding hands to a C entry point, which is not called."""
    calls = []
    monkeypatch.setattr(fa._binding, name, lambda *args: calls.append(args) or fa.ATTN_OK)
    return calls


@pytest.mark.parametrize("kind", ["strided", "expanded", "reversed axes", "column"])
def test_a_workspace_with_gaps_is_refused(kind, monkeypatch):
    """The kernels write `nbytes` from the first byte on: a view that has fewer of its own there would
    have its neighbours' bytes, or bytes past its storage, written."""
    calls = recorded(monkeypatch, "attn_paged_fwd_ptr")
    u8 = torch.uint8
    ws = {"strided": torch.zeros(8192, dtype=u8)[::2], "expanded": torch.zeros(1, dtype=u8).expand(1 << 20),
          "reversed axes": torch.zeros(64, 128, dtype=u8).t(), "column": torch.zeros(4096, 2, dtype=u8)[:, 0]}[kind]
    b = Batch([(20, 3)], 4, 2, 64, 16, device="cpu")
    a = b.on_gpu()
    args = [torch, 0, *a.values(), 3, 1, None, None, None]
    with pytest.raises(fa.AttnError, match="workspace") as e:
        fa._binding._paged_fwd(*args, ws, True)
    assert e.value.status == fa.ATTN_ERR_INVALID_ARG and not calls
    whole = torch.zeros(64, 128, dtype=torch.float32)
    fa._binding._paged_fwd(*args, whole, True)
    assert len(calls) == 1 and calls[0][-3:] == (whole.data_ptr(), 64 * 128 * 4, 0)


def test_a_stream_of_another_device_is_refused(monkeypatch):
    """A launch goes to the stream's device, where the tensors' addresses mean nothing."""
    from types import SimpleNamespace
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    entered = []
    monkeypatch.setattr(torch.cuda, "stream", lambda s: entered.append(s))
    mine = SimpleNamespace(device=torch.device("cuda", 0), cuda_stream=5)
    other = SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=5)
    assert fa._binding._on(0, mine).handle == 5
    with pytest.raises(fa.AttnError, match="stream") as e:
        fa._binding._on(0, other)
    assert e.value.status == fa.ATTN_ERR_INVALID_ARG and entered == [mine]


@pytest.mark.parametrize("axis", [0, 1, 2])
def test_caches_whose_strides_differ_on_an_axis_of_one(axis):
    """Such a stride has no meaning, so K and V of unlike origin are still one layout."""
    shape = [3, 16, 2, 64]
    shape[axis] = 1
    k = torch.zeros(shape, dtype=torch.bfloat16)
    wide = list(k.stride())
    wide[axis] += 8
    v = k.as_strided(shape, wide)
    got, strides = fa._binding._cache_shape(torch, k, v, "q", torch.bfloat16)
    assert tuple(got) == tuple(shape) and strides == k.stride()
    other = (axis + 1) % 3  # an axis that has more than one
    room = torch.zeros(10 * k.numel(), dtype=torch.bfloat16)
    wide = [2 * x if i == other else x for i, x in enumerate(k.stride())]
    with pytest.raises(fa.AttnError, match="strides"):
        fa._binding._cache_shape(torch, k, room.as_strided(shape, wide), "q", torch.bfloat16)
