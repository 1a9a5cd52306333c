"""The loss operators without a GPU: every refusal comes back before any HIP
call, for the C entry points (with addresses that are never read) and for the
torch calls."""

import os

import pytest

import tiled_gemm_tgemm_amd as tg
from tiled_gemm_tgemm_amd import _lib

OK, INVALID, UNSUPPORTED = tg.TGEMM_SUCCESS, tg.TGEMM_ERROR_INVALID_VALUE, tg.TGEMM_ERROR_NOT_SUPPORTED
X_, W_, Y_, LOSS, LSE, SUM, WS = (i << 36 for i in range(1, 8))
IDS, LOGITS, STUDENT, GRAD, DX, DW = (i << 36 for i in range(8, 14))
BIG = 1 << 35


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(_lib.LIBRARY):
        from tiled_gemm_tgemm_amd import build

        build.build()
    return tg.library()


def ce_forward(dtype=1, T=4, V=10, D=64, X=X_, ldx=64, W=W_, ldw=64, y=Y_, loss=LOSS, lse=LSE, summary=SUM, ws=WS, room=BIG):
    return tg.tgemm_linear_ce_forward(dtype, T, V, D, X, ldx, W, ldw, y, -100, loss, lse, summary, ws, room)


def ce_backward(dtype=1, T=4, V=10, D=64, X=X_, ldx=64, W=W_, ldw=64, y=Y_, lse=LSE, grad=GRAD, step=1, weight=0, dX=DX,
                lddx=64, dW=DW, lddw=64, ws=WS, room=BIG):
    return tg.tgemm_linear_ce_backward(dtype, T, V, D, X, ldx, W, ldw, y, -100, lse, grad, step, weight, dX, lddx, dW, lddw,
                                       ws, room)


def kd_forward(dtype=1, T=4, V=10, D=64, X=X_, ldx=64, W=W_, ldw=64, K=3, ids=IDS, ld_ids=3, kind=1, logits=LOGITS,
               ld_logits=3, temperature=1.0, loss=LOSS, lse=LSE, student=STUDENT, summary=SUM, ws=WS, room=BIG):
    return tg.tgemm_linear_kd_forward(dtype, T, V, D, X, ldx, W, ldw, K, ids, ld_ids, kind, logits, ld_logits, temperature,
                                      loss, lse, student, summary, ws, room)


def kd_backward(dtype=1, T=4, V=10, D=64, X=X_, ldx=64, W=W_, ldw=64, K=3, ids=IDS, ld_ids=3, kind=1, logits=LOGITS,
                ld_logits=3, temperature=1.0, lse=LSE, student=STUDENT, grad=GRAD, step=1, weight=0, dX=DX, lddx=64, dW=DW,
                lddw=64, ws=WS, room=BIG):
    return tg.tgemm_linear_kd_backward(dtype, T, V, D, X, ldx, W, ldw, K, ids, ld_ids, kind, logits, ld_logits, temperature,
                                       lse, student, grad, step, weight, dX, lddx, dW, lddw, ws, room)


EVERY = {"ce_forward": ce_forward, "ce_backward": ce_backward, "kd_forward": kd_forward, "kd_backward": kd_backward}

REFUSED = [
    (dict(T=-1), INVALID), (dict(V=0), INVALID), (dict(D=0, ldx=1, ldw=1), INVALID), (dict(V=-5), INVALID),
    (dict(ldx=63), INVALID), (dict(ldw=63), INVALID),
    (dict(dtype=3), UNSUPPORTED), (dict(dtype=-1), UNSUPPORTED),
    (dict(T=1 << 24), UNSUPPORTED), (dict(V=(1 << 24) + 1), UNSUPPORTED),
    (dict(D=(1 << 22) + 1, ldx=1 << 23, ldw=1 << 23), UNSUPPORTED), (dict(ldx=(1 << 40) + 1), UNSUPPORTED),
    (dict(X=0), INVALID), (dict(W=0), INVALID), (dict(X=X_ + 1), INVALID), (dict(W=W_ + 1), INVALID),
    (dict(dtype=0, X=X_ + 2), INVALID), (dict(lse=0), INVALID), (dict(lse=LSE + 2), INVALID),
    (dict(lse=X_ + 64), "overlap in forward"),
    (dict(ws=0), INVALID), (dict(ws=WS + 8), INVALID), (dict(room=64), INVALID), (dict(ws=X_ + 256), INVALID),
    (dict(ws=(1 << 64) - 4096, room=8192), INVALID),
    (dict(X=(1 << 64) - 256), INVALID), (dict(T=1 << 20, ldx=1 << 40), INVALID + 10),
]


@pytest.mark.parametrize("entry", EVERY)
@pytest.mark.parametrize("change,status", REFUSED)
def test_refusals(entry, change, status):
    if status == "overlap in forward":
        status = INVALID
        if "backward" in entry:  # two inputs may overlap; the call would be queued
            return
    if status > 10:  # rows past the end of the address space
        status -= 10
        change = dict(change, X=(1 << 64) - (1 << 60))
    assert EVERY[entry](**change) == status


@pytest.mark.parametrize("entry,change,status", [
    ("ce_forward", dict(y=0), INVALID), ("ce_forward", dict(y=Y_ + 4), INVALID), ("ce_forward", dict(loss=0), INVALID),
    ("ce_forward", dict(loss=LSE + 4), INVALID), ("ce_forward", dict(summary=SUM + 1), INVALID),
    ("ce_forward", dict(summary=LOSS + 4), INVALID), ("ce_forward", dict(loss=Y_ + 8), INVALID),
    ("ce_forward", dict(T=(1 << 24) - 1, V=1 << 24), UNSUPPORTED),  # more tiles than a launch holds
    ("kd_forward", dict(T=(1 << 24) - 1, V=1 << 24), UNSUPPORTED),
    ("ce_backward", dict(y=0), INVALID), ("ce_backward", dict(grad=0), INVALID), ("ce_backward", dict(step=-1), INVALID),
    ("ce_backward", dict(weight=GRAD + 2), INVALID), ("ce_backward", dict(dX=DX + 1), INVALID),
    ("ce_backward", dict(dX=X_), INVALID), ("ce_backward", dict(dW=W_ + 128), INVALID), ("ce_backward", dict(dX=DW + 64), INVALID),
    ("ce_backward", dict(lddx=63), INVALID), ("ce_backward", dict(lddw=10), INVALID),
    ("ce_backward", dict(lddw=(1 << 40) + 1), UNSUPPORTED), ("ce_backward", dict(dX=WS), INVALID),
    ("ce_backward", dict(dX=0, dW=0), OK),  # nothing to do
    ("kd_forward", dict(K=0), INVALID), ("kd_forward", dict(K=1025, ld_ids=2000, ld_logits=2000), UNSUPPORTED),
    ("kd_forward", dict(ld_ids=2), INVALID), ("kd_forward", dict(ld_logits=2), INVALID), ("kd_forward", dict(kind=9), UNSUPPORTED),
    ("kd_forward", dict(temperature=0.0), INVALID), ("kd_forward", dict(temperature=-1.0), INVALID),
    ("kd_forward", dict(temperature=float("nan")), INVALID), ("kd_forward", dict(temperature=float("inf")), INVALID),
    ("kd_forward", dict(temperature=1e-45), INVALID),
    ("kd_forward", dict(ids=IDS + 4), INVALID), ("kd_forward", dict(logits=LOGITS + 1), INVALID),
    ("kd_forward", dict(kind=0, logits=LOGITS + 2), INVALID), ("kd_forward", dict(student=0), INVALID),
    ("kd_forward", dict(student=LOGITS), INVALID), ("kd_forward", dict(loss=STUDENT + 4), INVALID),
    ("kd_backward", dict(student=0), INVALID), ("kd_backward", dict(ids=0), INVALID), ("kd_backward", dict(temperature=0.0), INVALID),
    ("kd_backward", dict(dX=STUDENT), INVALID), ("kd_backward", dict(dW=IDS), INVALID), ("kd_backward", dict(K=1025), INVALID),
    ("kd_backward", dict(dX=0, dW=0), OK),
])
def test_refusals_of_one_entry(entry, change, status):
    assert EVERY[entry](**change) == status


def test_no_rows():
    assert ce_forward(T=0, summary=0, X=0, y=0, loss=0, lse=0, ws=0, room=0) == OK
    assert kd_forward(T=0, summary=0, X=0, ids=0, logits=0, loss=0, lse=0, student=0, ws=0, room=0) == OK
    assert ce_backward(T=0, dW=0, dX=0) == OK and ce_backward(T=0, dW=0) == OK
    assert ce_forward(T=0, summary=SUM + 2) == INVALID and ce_backward(T=0, dW=DW + 1) == INVALID


def size(dtype=1, T=4, V=10, D=64, X=X_, ldx=64, W=W_, ldw=64, K=0, backward=0):
    return tg.tgemm_linear_loss_workspace_size(dtype, T, V, D, X, ldx, W, ldw, K, backward)


def test_workspace_sizes():
    assert size() > 0 and size(backward=1) > 0 and size(K=8) > 0
    for refused in (dict(T=0), dict(T=-1), dict(V=0), dict(dtype=7), dict(ldx=3), dict(V=1 << 25)):
        assert size(**refused) == 0 and size(**refused, backward=1) == 0
    # a copy of W is laid out only where the matrix cores cannot read it as it is stored
    stored = size(T=64, V=100000)
    for copied in (dict(W=W_ + 2), dict(ldw=68), dict(dtype=0)):
        assert size(T=64, V=100000, **copied) >= stored + 100000 * 64 * 2
    assert size(T=64, V=100000, D=60) >= stored + 100000 * 64 * 2
    # a few rows take W as it is, in float32 too
    assert size(T=32, V=100000, dtype=0) < 100000 * 64
    # the pieces of the logits' gradient are far smaller than the logits
    T, V = 16384, 131072
    assert size(T=T, V=V, backward=1) < T * V * 2 // 8


def test_a_large_workspace_is_taken_and_a_short_one_is_not():
    need = size(backward=1)
    assert ce_backward(room=need - 1) == INVALID


def test_torch_calls_refuse():
    torch = pytest.importorskip("torch")
    X, W, y = torch.zeros(4, 8), torch.zeros(10, 8), torch.zeros(4, dtype=torch.int64)
    for call in (lambda: tg.linear_cross_entropy_forward(X, W, y), lambda: tg.linear_cross_entropy(X, W, y),
                 lambda: tg.linear_cross_entropy(X.double(), W.double(), y), lambda: tg.linear_cross_entropy([1.0], W, y),
                 lambda: tg.linear_cross_entropy_backward(torch.ones(4), X, W, y, torch.zeros(4)),
                 lambda: tg.linear_distillation(X, W, y[:, None], X[:, :1])):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError):
        tg.linear_cross_entropy(X, W, y, reduction="average")
    with pytest.raises(ValueError):
        tg.linear_distillation(X, W, y[:, None], X[:, :1], reduction=None)
    with pytest.raises(ValueError):
        tg.linear_cross_entropy(X, W, y, keep_logits="yes")


KEPT = 1 << 40


@pytest.mark.parametrize("entry", EVERY)
@pytest.mark.parametrize("logits,ldz,status", [(KEPT, 9, INVALID), (KEPT, 0, INVALID), (KEPT, (1 << 40) + 1, UNSUPPORTED),
                                               (KEPT + 2, 10, INVALID), ((1 << 64) - 64, 10, INVALID), (WS + 256, 10, INVALID)])
def test_refusals_of_kept_logits(entry, logits, ldz, status, monkeypatch):
    import functools

    name = f"tgemm_linear_{entry}"
    monkeypatch.setattr(tg, name, functools.partial(getattr(tg, name), logits=logits, ldz=ldz))
    assert EVERY[entry]() == status


@pytest.mark.parametrize("entry,overlaps", [("ce_forward", (X_, W_, Y_, LOSS, LSE, SUM)), ("ce_backward", (DX, DW)),
                                            ("kd_forward", (X_, W_, IDS, LOGITS, STUDENT, LOSS, LSE, SUM)),
                                            ("kd_backward", (DX, DW))])
def test_kept_logits_overlap_nothing(entry, overlaps, monkeypatch):
    import functools

    name = f"tgemm_linear_{entry}"
    call = getattr(tg, name)
    for at in overlaps:
        monkeypatch.setattr(tg, name, functools.partial(call, logits=at, ldz=10))
        assert EVERY[entry]() == INVALID
