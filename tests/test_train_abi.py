"""Host-side refusals of the training operators: answered without a GPU, before
any launch."""
import copy
import ctypes
import pickle

import pytest
import torch

from combine_warp_top_gb300 import build as libbuild
from combine_warp_top_gb300 import moe

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
OK16 = ctypes.c_void_p(0x10000)  # never dereferenced on the host
ODD = ctypes.c_void_p(0x10002)


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return moe.load()


def args(**kw):
    shape = moe.Shape(**dict(dict(N=64, H=64, E=8, k=2, W=2, I=64), **kw))
    lay = moe.MoeLayout(*([0x20000] * len(moe.LAYOUT_FIELDS)))
    return ctypes.byref(shape.c()), ctypes.byref(lay), \
        ctypes.c_size_t(moe.moe_workspace_bytes(shape))


def test_grouped_refusals(lib):
    c, L, n = args()
    f = lib.moe_grouped_gemm
    assert f(OK16, L, c, 64, 64, None, OK16, 0, OK16, n, None) == INVALID
    assert f(ODD, L, c, 64, 64, OK16, OK16, 0, OK16, n, None) == INVALID
    assert f(OK16, None, c, 64, 64, OK16, OK16, 0, OK16, n, None) == INVALID
    assert f(OK16, L, c, 64, 64, OK16, OK16, 7, OK16, n, None) == INVALID
    assert f(OK16, L, c, 0, 64, OK16, OK16, 0, OK16, n, None) == INVALID
    assert f(OK16, L, c, 60, 64, OK16, OK16, 0, OK16, n, None) == UNSUPPORTED
    assert f(OK16, L, c, 64, 64, OK16, OK16, 0, OK16, 16, None) == WORKSPACE
    assert f(OK16, L, c, 64, 64, OK16, OK16, 0, None, n, None) == WORKSPACE
    g = lib.moe_grouped_gemm_weight_grad
    assert g(OK16, OK16, L, c, 64, 64, OK16, 0, 1, OK16, n, None) == UNSUPPORTED  # bf16 +=
    assert g(None, OK16, L, c, 64, 64, OK16, 1, 1, OK16, n, None) == INVALID
    assert g(OK16, OK16, L, c, 64, 64, ODD, 1, 0, OK16, n, None) == INVALID
    assert lib.moe_grouped_gemm_input_grad(OK16, L, c, 64, 64, ODD, OK16, 0, OK16, n, None) == INVALID
    bad, L, n = args(E=9)  # E % W
    assert f(OK16, L, bad, 64, 64, OK16, OK16, 0, OK16, n, None) == INVALID
    none, L, n = args(N=0)
    assert f(None, L, none, 64, 64, None, None, 0, OK16, n, None) == 0


def test_swiglu_and_route_refusals(lib):
    c, L, _ = args()
    assert lib.moe_swiglu(None, None, L, c, OK16, None) == INVALID
    assert lib.moe_swiglu(OK16, None, L, c, ODD, None) == INVALID
    assert lib.moe_swiglu(OK16, None, None, c, OK16, None) == INVALID
    assert lib.moe_swiglu_grad(OK16, ODD, None, L, c, OK16, None, None) == INVALID
    assert lib.moe_swiglu_grad(OK16, OK16, None, L, c, None, None, None) == INVALID
    assert lib.moe_route_grad(OK16, None, OK16, c, OK16, None) == INVALID
    assert lib.moe_route_full_softmax_grad(None, OK16, OK16, c, OK16, None) == INVALID
    assert lib.moe_route_sigmoid_bias_grad(OK16, OK16, OK16, c, None, None) == INVALID


def norm(**kw):
    return ctypes.byref(moe.NormShape(**dict(dict(N=4, H=64), **kw)).c())


def test_norm_refusals(lib):
    def fwd(shape, y=OK16, residual=OK16, gate=None, s=OK16, x=OK16):
        return lib.moe_block_norm(y, residual, None, gate, None, shape, s, x, None, None, None)

    def grad(shape, ds=OK16, dx=OK16, y=OK16, gate=None, rp=OK16, rn=OK16, dy=OK16, dw_post=None,
             dgate=None, dw_pre=None, ws=OK16, n=1 << 30):
        return lib.moe_block_norm_grad(ds, dx, y, OK16, None, gate, None, rp, rn, shape, dy, OK16,
                                       dw_post, dgate, dw_pre, 0, ws, n, None)

    assert fwd(norm(H=60)) == UNSUPPORTED
    assert fwd(norm(H=16392)) == UNSUPPORTED
    assert fwd(norm(eps=-1.0)) == INVALID
    assert fwd(norm(eps=float("nan"))) == INVALID
    assert fwd(norm(), residual=None) == INVALID
    assert fwd(norm(), x=None) == INVALID                  # a norm before the next block
    assert fwd(norm(pre=False), s=None, x=None) == INVALID  # nothing wanted
    assert fwd(norm(), y=None) == INVALID                  # a norm after no block
    assert fwd(norm(gate="channel")) == INVALID
    assert fwd(norm(gate="channel"), gate=ODD) == INVALID
    assert fwd(norm(), y=ODD) == INVALID
    assert grad(norm(), ws=None) == WORKSPACE
    assert grad(norm(), n=8) == WORKSPACE
    assert grad(norm(), dx=None) == INVALID
    assert grad(norm(pre=False), ds=None) == INVALID
    assert grad(norm(), rp=None) == INVALID
    assert grad(norm(), rn=None) == INVALID
    assert grad(norm(), dy=None) == INVALID
    assert grad(norm(), dgate=OK16) == INVALID             # of a gate that is not there
    assert grad(norm(post=False), dw_post=OK16) == INVALID
    assert grad(norm(pre=False), dw_pre=OK16) == INVALID
    assert moe.moe_norm_workspace_bytes(moe.NormShape(4, 60)) == 0
    with pytest.raises(ValueError, match="gate must be"):
        moe.NormShape(4, 64, gate="row").c()
    with pytest.raises(ValueError, match="stream must be"):
        moe.NormShape(4, 64, stream="fp16").c()


def test_binding_checks_types_and_shapes(lib):
    bf = torch.bfloat16
    ns = moe.NormShape(4, 64)
    y, v = torch.empty(4, 64, dtype=bf), torch.empty(64)
    with pytest.raises(ValueError, match="y: expected torch.bfloat16"):
        moe.moe_block_norm(y.float(), y, v, None, v, ns, y, y)
    with pytest.raises(ValueError, match=r"y: expected shape \(4, 64\)"):
        moe.moe_block_norm(y[:3], y, v, None, v, ns, y, y)
    with pytest.raises(ValueError, match="device tensors"):
        moe.moe_block_norm(y, y, v, None, v, ns, y, y)
    shape = moe.Shape(4, 64, 8, 2, 1, 64)
    lay = moe.Layout.__new__(moe.Layout)
    lay.shape, lay.c = shape, moe.MoeLayout()
    with pytest.raises(ValueError, match=r"w: expected \[E = 8"):
        moe.moe_grouped_gemm(y, lay, shape, torch.empty(4, 64, 64, dtype=bf), y, y)
    with pytest.raises(ValueError, match="gu: expected shape"):
        moe.moe_swiglu(y, None, lay, shape, y)
    with pytest.raises(ValueError, match="topk_ids: expected torch.int32"):
        moe.moe_route_grad(torch.empty(4, 2, dtype=torch.int64), v, v, shape, v)


def test_shapes_copy_and_pickle_after_use():
    for shape in (moe.Shape(4, 64, 8, 2, 1, 64, gemm="pair"),
                  moe.NormShape(4, 64, gate="token", stream="fp32")):
        before = moe.load() and shape.ref  # a call keeps the C struct
        assert before is shape.ref
        for other in (copy.copy(shape), copy.deepcopy(shape), pickle.loads(pickle.dumps(shape))):
            assert other == shape and other.ref is not before
