"""Host-side refusals of the gated block, Muon and the 4-bit products: answered without a GPU,
before any launch."""
import copy
import ctypes
import pickle

import pytest
import torch

from combine_warp_top_gb300 import build as libbuild
from combine_warp_top_gb300 import moe, train

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
OK16 = ctypes.c_void_p(0x10000)  # never dereferenced on the host
ODD = ctypes.c_void_p(0x10002)
BIG = ctypes.c_size_t(1 << 40)
bf = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return moe.load()


def args(**kw):
    shape = moe.Shape(**dict(dict(N=64, H=64, E=8, k=2, W=2, I=64), **kw))
    lay = moe.MoeLayout(*([0x20000] * len(moe.LAYOUT_FIELDS)))
    return ctypes.byref(shape.c()), ctypes.byref(lay), shape


def test_gated_refusals(lib):
    c, L, s = args()
    base, full = moe.moe_workspace_bytes(s), moe.moe_gated_workspace_bytes(s)
    assert full >= base + s.R * 4

    def fwd(rows=OK16, lay=L, shape=c, ci=64, w=OK16, h=OK16, ws=OK16, n=base, gu=None):
        return lib.moe_gated_gemm(rows, lay, shape, ci, w, None, gu, h, ws, n, None)

    def grad(dout=OK16, lay=L, shape=c, co=64, w=OK16, gu=OK16, dgu=OK16, ws=OK16, n=full):
        return lib.moe_gated_gemm_grad(dout, lay, shape, co, w, None, gu, dgu, None, ws, n, None)

    for f in (fwd, grad):
        assert f(lay=None) == INVALID and f(shape=None) == INVALID and f(w=None) == INVALID
        assert f(w=ODD) == INVALID and f(ws=ODD) == INVALID
        assert f(ws=None) == WORKSPACE and f(n=16) == WORKSPACE
    assert fwd(rows=None) == INVALID and fwd(h=None) == INVALID and fwd(gu=ODD) == INVALID
    assert fwd(ci=0) == INVALID and fwd(ci=60) == UNSUPPORTED and fwd(ci=32776) == UNSUPPORTED
    assert grad(dout=None) == INVALID and grad(gu=None) == INVALID and grad(dgu=ODD) == INVALID
    assert grad(co=-8) == INVALID and grad(co=12) == UNSUPPORTED and grad(co=40000) == UNSUPPORTED
    assert grad(n=base) == WORKSPACE
    wide, Lw, sw = args(I=(1 << 28) + 8)
    more = moe.moe_gated_workspace_bytes(sw)
    assert fwd(lay=Lw, shape=wide, n=more) == UNSUPPORTED
    assert grad(lay=Lw, shape=wide, n=more) == UNSUPPORTED
    none, L0, _ = args(N=0)
    assert fwd(rows=None, lay=L0, shape=none, w=None, h=None) == 0
    assert grad(dout=None, lay=L0, shape=none, w=None, gu=None, dgu=None) == 0
    assert moe.moe_gated_workspace_bytes(moe.Shape(4, 64, 8, 9, 1, 64)) == 0


def test_muon_refusals(lib):
    def call(grad=OK16, mom=OK16, update=OK16, new=OK16, ws=OK16, n=BIG, **kw):
        shape = ctypes.byref(moe.MuonShape(**dict(dict(E=2, M=64, N=72), **kw)).c())
        return lib.moe_muon_update(grad, mom, shape, update, new, ws, n, None)

    for bad in (dict(E=0), dict(M=-8), dict(N=0), dict(steps=0), dict(steps=65),
                dict(momentum=1.0), dict(momentum=-0.1), dict(momentum=float("nan")),
                dict(eps=0.0), dict(eps=float("nan")), dict(eps=2.0)):
        assert call(**bad) == INVALID, bad
        assert moe.moe_muon_workspace_bytes(moe.MuonShape(**dict(dict(E=2, M=64, N=72), **bad))) == 0
    for bad in (dict(M=60), dict(N=4), dict(M=65544), dict(E=1025)):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(grad=None) == INVALID and call(update=None) == INVALID
    assert call(mom=None) == INVALID and call(new=None) == INVALID
    assert call(grad=ODD) == INVALID and call(new=ODD) == INVALID and call(ws=ODD) == INVALID
    assert call(ws=None) == WORKSPACE and call(n=4096) == WORKSPACE
    s = moe.MuonShape(2, 64, 72)
    assert lib.moe_muon_update(OK16, OK16, None, OK16, OK16, OK16, BIG, None) == INVALID
    for other in (copy.copy(s), copy.deepcopy(s), pickle.loads(pickle.dumps(s))):
        assert other == s
    g = torch.empty(2, 64, 72)
    with pytest.raises(ValueError, match="grad: expected bf16 or fp32"):
        moe.moe_muon_update(g.double(), g, s, g, g)
    with pytest.raises(ValueError, match="grad: expected shape"):
        moe.moe_muon_update(g[0], g, s, g, g)
    with pytest.raises(ValueError, match="device tensors"):
        moe.moe_muon_update(g, g, s, g, g)


def test_w4_refusals(lib):
    c, L, s = args()
    n = moe.moe_w4_workspace_bytes(s)
    assert n > moe.moe_workspace_bytes(s)

    def matrix(**kw):
        m = dict(dict(C_out=64, C_in=128, group=64, gated=0), **kw)
        return ctypes.byref(moe.MoeW4Matrix(m["C_out"], m["C_in"], m["group"], m["gated"]))

    def gemm(m=matrix(), rows=OK16, lay=L, shape=c, packed=OK16, out=OK16, ot=0, ws=OK16, n=n):
        return lib.moe_w4_gemm(rows, lay, shape, m, packed, out, ot, ws, n, None)

    def gated(m=matrix(gated=1), rows=OK16, packed=OK16, h=OK16, ws=OK16, n=n):
        return lib.moe_w4_gated_gemm(rows, L, c, m, packed, None, h, ws, n, None)

    assert gemm(matrix(gated=1)) == INVALID and gated(matrix()) == INVALID
    for f, kw in ((gemm, {}), (gated, dict(gated=1))):
        assert f(None) == INVALID
        assert f(matrix(group=16, **kw)) == INVALID and f(matrix(C_out=0, **kw)) == INVALID
        assert f(matrix(C_out=60, **kw)) == UNSUPPORTED
        assert f(matrix(C_in=96, **kw)) == UNSUPPORTED
        assert f(rows=None) == INVALID and f(packed=ODD) == INVALID and f(ws=ODD) == INVALID
        assert f(ws=None) == WORKSPACE and f(n=n - 1) == WORKSPACE
    assert gemm(ot=5) == INVALID and gemm(out=None) == INVALID and gated(h=ODD) == INVALID
    assert gemm(lay=None) == INVALID and gemm(shape=None) == INVALID
    none, L0, _ = args(N=0)
    assert gemm(shape=none, lay=L0, rows=None, packed=None, out=None) == 0
    quant = lib.moe_w4_quantize
    assert quant(OK16, 4, 100, 64, OK16, OK16, None) == UNSUPPORTED
    assert quant(OK16, 4, 128, 48, OK16, OK16, None) == INVALID
    assert quant(None, 4, 128, 64, OK16, OK16, None) == INVALID
    assert quant(OK16, 4, 128, 64, ODD, OK16, None) == INVALID
    assert quant(OK16, -1, 128, 64, OK16, OK16, None) == INVALID
    assert quant(None, 0, 128, 64, None, None, None) == 0
    pack = lib.moe_w4_pack
    assert pack(OK16, None, matrix(), 4, OK16, None) == INVALID
    assert pack(OK16, OK16, matrix(), 0, OK16, None) == INVALID
    assert pack(OK16, OK16, matrix(), 2000, OK16, None) == UNSUPPORTED
    # 8 warps' slabs of 32 rows, chunks of 128: 4 bits a weight and a scale for 64
    assert lib.moe_w4_packed_bytes(matrix(), 3) == 3 * 2 * (32 * 64 + 32 * 2 * 2)
    assert lib.moe_w4_packed_bytes(matrix(C_in=96), 3) == 0
    with pytest.raises(moe.MoeError):
        moe.W4Matrices(2, 64, 100, 64, False, device="cpu")


def test_w4_binding_and_layer(lib):
    s = moe.Shape(4, 128, 8, 2, 1, 64)
    lay = moe.Layout.__new__(moe.Layout)
    lay.shape, lay.c = s, moe.MoeLayout()
    plain = moe.W4Matrices(8, 128, 64, 64, False, device="cpu")
    gated = moe.W4Matrices(8, 64, 128, 64, True, device="cpu")
    y = torch.empty(8, 128, dtype=bf)
    with pytest.raises(TypeError, match="W4Matrices"):
        moe.moe_w4_gemm(y, lay, s, y, y, y)
    with pytest.raises(ValueError, match="plain matrices of E = 8"):
        moe.moe_w4_gemm(y, lay, s, gated, y, y)
    with pytest.raises(ValueError, match="rows: expected shape"):
        moe.moe_w4_gemm(y, lay, s, plain, y, y)
    with pytest.raises(ValueError, match="do not share"):
        moe.moe_w4_quantize(torch.empty(4, 128, dtype=bf), None, torch.empty(4, 3, dtype=bf))
    with pytest.raises(ValueError, match=r"w_gate_up: expected 2\*I"):
        moe.moe_gated_gemm(y, lay, s, torch.empty(8, 64, 128, dtype=bf), None, None, y, y)
    with pytest.raises(ValueError, match="w_down: expected I"):
        moe.moe_gated_gemm_grad(y, lay, s, torch.empty(8, 128, 72, dtype=bf), None, y, y, None, y)

    def layer(shape=s, w4=(gated, plain), **kw):
        return moe.MoELayer(shape, None, None, None, device="cpu", w4=w4, **kw)

    for other in (copy.copy(plain), copy.deepcopy(plain), pickle.loads(pickle.dumps(plain))):
        assert (other.C_out, other.gated) == (128, False) and other.data.shape == plain.data.shape
        assert other.ref is not plain.ref
    one = layer()
    assert one.stage_names() == ["route", "layout", "dispatch", "gate_up", "down", "combine"]
    assert one.kernel_launches_per_step() == 1 + 1 + 1 + 2 + 1
    dedup = layer(moe.Shape(4, 128, 8, 2, 2, 64, dedup=True))
    assert dedup.xe.shape == (8, 128)
    assert dedup.kernel_launches_per_step() == one.kernel_launches_per_step() + 1
    with pytest.raises(ValueError, match="own two products"):
        layer(fuse_combine=True)
    with pytest.raises(ValueError, match="own two products"):
        layer(moe.Shape(4, 128, 8, 2, 1, 64, weights="packed"))
    with pytest.raises(ValueError, match="gated matrices"):
        layer(w4=(plain, plain))
    with pytest.raises(ValueError, match="expected matrices of"):
        layer(moe.Shape(4, 256, 8, 2, 1, 64))


def test_train_block_with_the_fused_gate_is_on_its_device(lib):
    block = train.MoETrainBlock(6, 16, 4, 2, 8, device="cpu", fuse_gate=True)
    assert block.dh is None and block.ws.numel() == moe.moe_gated_workspace_bytes(block.shape)
    assert block.ws.device.type == "cpu"
