"""The projection with adapters without a GPU: every refusal comes back before
any HIP call, for the C entry points (with addresses that are never read) and
for the torch calls."""

import os

import pytest

import tiled_gemm_tgemm_amd as tg
from tiled_gemm_tgemm_amd import _lib

OK, INVALID, UNSUPPORTED = tg.TGEMM_SUCCESS, tg.TGEMM_ERROR_INVALID_VALUE, tg.TGEMM_ERROR_NOT_SUPPORTED
X_, W_, A_, B_, IDS, SC, Y_, H_, WS, DY, DX, DW, DA, DB = (i << 40 for i in range(1, 15))
BIG = 1 << 39
SHAPE = dict(dtype=1, T=70, N=96, D=64, X=X_, ldx=64, W=W_, ldw=64, count=3, rank=8, A=A_, lda=64, sa=512, B=B_, ldb=8, sb=768, ids=IDS,
             scales=SC)


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(_lib.LIBRARY):
        from tiled_gemm_tgemm_amd import build

        build.build()
    return tg.library()


def forward(Y=Y_, ldy=96, hidden=H_, ws=WS, room=BIG, **k):
    return tg.tgemm_linear_adapters_forward(*{**SHAPE, **k}.values(), Y, ldy, hidden, ws, room)


def backward(hidden=H_, dY=DY, lddy=96, dX=DX, lddx=64, dW=DW, lddw=64, dA=DA, ldda=64, sda=512, dB=DB, lddb=8, sdb=768, ws=WS, room=BIG, **k):
    return tg.tgemm_linear_adapters_backward(*{**SHAPE, **k}.values(), hidden, dY, lddy, dX, lddx, dW, lddw, dA, ldda, sda, dB, lddb, sdb,
                                             ws, room)


SHARED = [
    (dict(T=-1), INVALID), (dict(N=0), INVALID), (dict(D=0, ldx=0, ldw=0, lda=0), INVALID), (dict(count=0), INVALID), (dict(rank=0), INVALID),
    (dict(ldx=63), INVALID), (dict(ldw=63), INVALID), (dict(lda=63), INVALID), (dict(ldb=7), INVALID), (dict(sa=-1), INVALID),
    (dict(sb=-1), INVALID), (dict(X=0), INVALID), (dict(W=0), INVALID), (dict(A=0), INVALID), (dict(B=0), INVALID), (dict(ids=0), INVALID),
    (dict(X=X_ + 1), INVALID), (dict(dtype=0, B=B_ + 2), INVALID), (dict(ids=IDS + 4), INVALID), (dict(scales=SC + 2), INVALID),
    (dict(A=(1 << 64) - 1024), INVALID), (dict(ws=0), INVALID), (dict(ws=WS + 8), INVALID), (dict(room=16), INVALID), (dict(ws=X_), INVALID),
    (dict(ws=IDS), INVALID),
    (dict(dtype=3), UNSUPPORTED), (dict(T=1 << 24), UNSUPPORTED), (dict(N=(1 << 22) + 1), UNSUPPORTED),
    (dict(D=(1 << 22) + 1, ldx=1 << 23, ldw=1 << 23, lda=1 << 23), UNSUPPORTED), (dict(count=1 << 15), UNSUPPORTED),
    (dict(rank=1025, ldb=1025), UNSUPPORTED), (dict(ldx=(1 << 40) + 1), UNSUPPORTED), (dict(lda=(1 << 26) + 1), UNSUPPORTED),
    (dict(sa=(1 << 40) + 1), UNSUPPORTED),
]


@pytest.mark.parametrize("change,status", SHARED + [
    (dict(ldy=95), INVALID), (dict(N=(1 << 22) + 1, ldy=1 << 23), UNSUPPORTED), (dict(ldy=(1 << 40) + 1), UNSUPPORTED), (dict(Y=0), INVALID),
    (dict(Y=X_), INVALID), (dict(Y=B_ + 2 * 2303), INVALID), (dict(hidden=Y_), INVALID), (dict(hidden=H_ + 2), INVALID), (dict(hidden=WS), INVALID),
    (dict(T=0, X=0, ids=0, Y=0, hidden=0, ws=0, room=0), OK),
])
def test_forward_refusals(change, status):
    if "N" in change and "ldy" not in change and change["N"] > 96:
        change = dict(change, ldy=1 << 23)
    assert forward(**change) == status


@pytest.mark.parametrize("change,status", SHARED + [
    (dict(lddy=95), INVALID), (dict(lddx=63), INVALID), (dict(lddw=63), INVALID), (dict(ldda=63), INVALID), (dict(lddb=7), INVALID),
    (dict(sda=511), INVALID), (dict(sdb=767), INVALID), (dict(sda=-1), INVALID), (dict(lddy=(1 << 40) + 1), UNSUPPORTED),
    (dict(sdb=(1 << 40) + 1), UNSUPPORTED), (dict(dY=0), INVALID), (dict(dX=DY), INVALID), (dict(dA=DX), INVALID), (dict(dB=B_), INVALID),
    (dict(dW=W_ + 128), INVALID), (dict(dW=DX + 2 * 4479), INVALID), (dict(dX=WS), INVALID), (dict(hidden=DX), INVALID),
    (dict(dX=0, dW=0, dA=0, dB=0, ws=0, room=0), OK), (dict(T=0, X=0, ids=0, dY=0, hidden=0, dW=0, dA=0, dB=0, ws=0, room=0), OK),
])
def test_backward_refusals(change, status):
    if "N" in change and change["N"] > 96:
        change = dict(change, lddy=1 << 23)
    assert backward(**change) == status


def test_workspace_sizes():
    def size(T=2000, N=960, D=640, dtype=1, need=0, X=X_, W=W_, dY=DY, L=3, r=16, lddy=None):
        return tg.tgemm_linear_adapters_workspace_size(dtype, T, N, D, X, D, W, D, L, r, dY, lddy or N, need)

    assert size(T=0) == size(need=-1) == size(need=16) == size(dtype=5) == size(need=1, lddy=5) == size(L=0) == 0
    assert 0 < size(T=1) < 1 << 16
    # operands that cannot be read as they are stored are copied
    assert size(W=W_ + 2) >= size() + 2 * 960 * 640 and size(X=X_ + 2) >= size() + 2 * 2000 * 640
    assert size(dtype=0, T=8000, N=8000, D=4096) > 6 * (8000 + 8000) * 4096
    assert size(need=15) >= max(size(need=n) for n in (1, 2, 4, 8))
    # an empty batch writes zeros, for which the adapters' gradients take little
    assert 0 < size(T=0, need=12) < 1 << 16


def test_the_torch_calls_refuse():
    torch = pytest.importorskip("torch")
    z = torch.zeros
    args = dict(X=z(4, 8), W=z(6, 8), A=z(2, 3, 8), B=z(2, 6, 3), ids=z(4, dtype=torch.int64))
    with pytest.raises(TypeError):
        tg.linear_adapters(*args.values())  # the host's
    with pytest.raises(TypeError):
        tg.linear_adapters(*dict(args, X=z(4, 8, dtype=torch.float64)).values())
    with pytest.raises(TypeError):
        tg.linear_adapters_backward(z(4, 6), *args.values())
