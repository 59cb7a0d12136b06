"""The feed-forward operators' binding on the CPU: what it does before a call
reaches the library."""
from __future__ import annotations

import pytest
import torch

import hyper_connection_rank_amd as hc


def test_a_workspace_of_the_call_s_own_has_only_its_counters_cleared(monkeypatch):
    """The counters have to be zero; clearing the rest would write up to hundreds of megabytes a call."""
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: empty(*a, **k).fill_(0xA5))
    ws = hc.ffn._scratch(None, 1 << 20, torch.device("cpu"))
    assert ws.numel() == 1 << 20 and ws.dtype == torch.uint8
    assert not ws[:4096].any()
    assert (ws[4096:] == 0xA5).all()


ROWS = sorted(set(range(1, 80)) | {2 ** i + d for i in range(6, 14) for d in (-1, 0, 1)} | set(range(100, 4200, 300)))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("k,n", [(2560, 10240), (10240, 2560), (2056, 136), (777, 4105)])
def test_a_workspace_for_the_most_rows_serves_fewer(k, n, dtype):
    for size in (hc.linear_workspace_size, hc.glu_workspace_size):
        for backward in (False, True):
            need = [size(r, k, n, dtype, backward=backward) for r in ROWS]
            assert need == sorted(need), (size.__name__, backward)
    need = [hc.residual_norm_workspace_size(r, k, dtype) for r in ROWS]
    assert need == sorted(need)


def _calls():
    """Every function's positional tensors and a call with them (CPU tensors: a call that is not refused before it
    reaches the library is refused there, with another message)."""
    t = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    y = lambda: t(4, 8)  # noqa: E731
    return {"residual_norm": ([y(), y(), t(4), t(8), t(8)],
                              lambda a, b, g, p, q: hc.residual_norm(a, b, gate=g, post_scale=p, pre_scale=q)),
            "residual_norm_backward": ([y(), y(), y(), y(), t(4), t(8), t(8)],
                                       lambda a, b, c, d, g, p, q: hc.residual_norm_backward(a, b, c, d, gate=g, post_scale=p,
                                                                                             pre_scale=q)),
            "linear": ([t(4, 8), t(8, 16), t(16), t(4, 16)], hc.linear),
            "linear_backward": ([t(4, 8), t(8, 16), t(4, 16), t(4, 16)],
                                lambda *a: hc.linear_backward(*a, activation="silu")),
            "glu": ([t(4, 8), t(8, 16), t(8, 16), t(16), t(16)], hc.glu),
            "glu_backward": ([t(4, 8), t(8, 16), t(8, 16), t(4, 16), t(4, 16), t(4, 16)], hc.glu_backward)}


@pytest.mark.parametrize("name", list(_calls()))
def test_tensors_that_require_gradients_are_refused_while_autograd_records(name):
    tensors, call = _calls()[name]
    for i, t in enumerate(tensors):
        given = list(tensors)
        given[i] = t.clone().requires_grad_()
        with pytest.raises(hc.HclrmixError, match="autograd"):
            call(*given)
        with torch.no_grad(), pytest.raises(hc.HclrmixError, match="GPU"):
            call(*given)
    with pytest.raises(hc.HclrmixError, match="GPU"):
        call(*tensors)


def _refused(f, *args, part="", **kw):
    with pytest.raises(hc.HclrmixError) as e:
        f(*args, **kw)
    assert part in str(e.value), str(e.value)


@pytest.mark.parametrize("shape", [(), (8,), (2, 8, 16)])
def test_weights_that_are_no_matrices_are_refused(shape):
    t = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    x, g, w = t(4, 8), t(4, 16), torch.zeros(shape, dtype=torch.bfloat16)
    _refused(hc.linear, x, w, part="weight must be [in, out]")
    _refused(hc.linear_backward, x, w, g, part="weight must be [in, out]")
    for gate, up, name in ((w, t(8, 16), "gate_weight"), (t(8, 16), w, "up_weight")):
        _refused(hc.glu, x, gate, up, part=name + " must be [in, out]")
        _refused(hc.glu_backward, x, gate, up, g, g, g, part=name + " must be [in, out]")


@pytest.mark.parametrize("dtype", [torch.float64, torch.int8, None])
def test_workspace_sizes_of_other_types_are_refused(dtype):
    _refused(hc.residual_norm_workspace_size, 4, 64, dtype, part="dtype")
    for size in (hc.linear_workspace_size, hc.glu_workspace_size):
        for backward in (False, True):
            _refused(size, 4, 64, 64, dtype, backward=backward, part="dtype")
