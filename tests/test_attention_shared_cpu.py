"""qkv_attend_shared without a GPU: the refusal of bad arguments by status before
any CUDA call, its workspace's size, and the binding's own checks."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import ggml_block_quantized_gb300 as qg  # noqa: E402
from ggml_block_quantized_gb300 import attention as at  # noqa: E402

OK, ERR_TYPE, ERR_SHAPE, ERR_ALIGN, ERR_NULL, ERR_WS = 0, -1, -2, -3, -4, -7
A, B, C, MIS = 0x10000, 0x20000, 0x30000, 0x10008


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__.build()
    return at._lib()


def cache(data=A, n_pages=4, heads=2, d=128, page=16):
    return at._Cache(data, n_pages, heads, d, page)


SHARED = dict(type=0, q=A, q_stride=1024, out=B, prefix_table=C, prefix_pages=9, prefix_len=C, table=C, table_stride=4,
              lengths=C, q_offsets=None, n_seq=2, n_tok=2, n_heads=8, max_q_len=1, scale=0.1, workspace=A,
              workspace_bytes=1 << 40)


@pytest.mark.parametrize("want,kw", [
    (ERR_TYPE, dict(type=2)), (ERR_SHAPE, dict(n_heads=7)), (ERR_SHAPE, dict(n_heads=0)), (ERR_SHAPE, dict(n_seq=-1)),
    (ERR_SHAPE, dict(n_tok=-1)), (ERR_SHAPE, dict(max_q_len=0)), (ERR_SHAPE, dict(max_q_len=1 << 30)),
    (ERR_SHAPE, dict(table_stride=-1)), (ERR_SHAPE, dict(prefix_pages=-1)), (ERR_SHAPE, dict(prefix_pages=1 << 31)),
    (ERR_SHAPE, dict(n_tok=1)), (ERR_SHAPE, dict(n_tok=(1 << 23) + 1)), (ERR_SHAPE, dict(scale=float("nan"))),
    (ERR_SHAPE, dict(q_stride=1020)), (ERR_NULL, dict(q=None)), (ERR_NULL, dict(out=None)), (ERR_NULL, dict(lengths=None)),
    (ERR_NULL, dict(table=None)), (ERR_NULL, dict(prefix_table=None)), (ERR_NULL, dict(prefix_len=None)),
    (ERR_ALIGN, dict(q=MIS)), (ERR_ALIGN, dict(workspace=MIS)), (ERR_ALIGN, dict(prefix_table=C + 2)),
    (ERR_ALIGN, dict(prefix_len=C + 1)), (ERR_WS, dict(workspace=None)), (ERR_WS, dict(workspace_bytes=4096)),
    (OK, dict(n_seq=0, n_tok=0)),
])
def test_refusals(L, want, kw):
    assert L.qkv_attend_shared(ctypes.byref(cache()), *{**SHARED, **kw}.values(), None) == want


def test_no_cache(L):
    assert L.qkv_attend_shared(None, *SHARED.values(), None) == ERR_NULL
    assert L.qkv_attend_shared(ctypes.byref(cache(d=80)), *SHARED.values(), None) == ERR_SHAPE


def test_workspace(L):
    ws = L.qkv_attend_shared_workspace_bytes
    own = L.qkv_attend_workspace_bytes(128, 8, 32, 1)
    assert ws(128, 8, 32, 1, 1) > own and ws(128, 8, 32, 500, 1) > ws(128, 8, 32, 1, 1)
    assert ws(128, 1, 1, 1 << 26, 1) > 1 << 36  # past 32 bits
    for bad in ((96, 8, 32, 1, 1), (128, 0, 32, 1, 1), (128, 8, 31, 1, 1), (128, 8, 32, 1, 0), (128, 8, 32, -1, 1),
                (128, 8, 32, (1 << 21) + 1, 1)):
        assert ws(*bad) == 0


def test_binding_wants_cuda_tensors(L):
    x, i = torch.zeros(2, 8, 128), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError):
        qg.kv_attend_shared(None, x, i, i, i, i)
