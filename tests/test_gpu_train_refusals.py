"""What dropout and the layer norm refuse in Python: valid GPU tensors, and one bad argument a
call. Only the good calls run."""
import math

import pytest

from gpu_util import device_ready

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not device_ready():
        pytest.skip("no GPU")


def refused(call, good, bad, exc=ValueError):
    """call takes the arguments of `good`, and none of `bad` in their place."""
    call(**good)
    for name, values in bad.items():
        for v in values:
            with pytest.raises(exc):
                call(**{**good, name: v})
                pytest.fail(f"{name} = {v!r} was taken")


def tensors():
    import torch
    x = torch.zeros(4, 16, device="cuda")
    # another shape, another dtype, not on the GPU, columns apart
    mats = [x[:, :8], x[:3], x.bfloat16(), x.cpu(), x.t().contiguous().t(), x[0]]
    v = torch.ones(16, device="cuda")
    vecs = [v[:8], v.bfloat16(), v.double(), v.cpu(), torch.ones(32, device="cuda")[::2], v[None]]
    r = torch.ones(4, device="cuda")
    rows = [r[:3], r.double(), r.cpu(), torch.ones(8, device="cuda")[::2], r[:, None]]
    return x, mats, v, vecs, r, rows


def rules():
    import torch
    s = torch.ones(1, dtype=torch.int64, device="cuda")
    return dict(p=[-0.1, 1.5, math.nan, math.inf], site=[-1, 2 ** 32],
                seed=[-1, 2 ** 64, s.cpu(), s.int(), s.double(), s.repeat(2), s[:0]])


def test_dropout():
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    x, mats, *_ = tensors()
    good = dict(X=x, p=0.3, seed=1, site=2, residual=x.clone(), out=x.clone())
    refused(oec.dropout, good, dict(rules(), residual=mats, out=mats, X=[x.half(), x.double(), x.cpu(), x[0]]))
    refused(oec.dropout_backward, dict(G_Y=x, p=0.3, seed=1, site=2, out=x.clone()), dict(rules(), out=mats, G_Y=[x.half(), x.cpu()]))
    y = torch.zeros(80, device="cuda")
    with pytest.raises(oec.poetx.PoetxError):   # half over its own input
        oec.dropout(y[:64].view(4, 16), 0.3, 1, out=y[8:72].view(4, 16))


def test_add_layer_norm():
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    x, mats, v, vecs, _, _ = tensors()
    good = dict(X=x, weight=v, bias=v.clone(), residual=x.clone(), p=0.3, seed=1, site=2, H=x.clone())
    refused(oec.add_layer_norm, good, dict(rules(), weight=vecs, bias=vecs, residual=mats, H=mats,
                                           X=[x.half(), x.double(), x.cpu(), x[0]]))
    refused(oec.add_layer_norm, good, dict(eps=[-1e-5, math.nan, math.inf]), oec.poetx.PoetxError)
    y = torch.zeros(80, device="cuda")
    with pytest.raises(oec.poetx.PoetxError):
        oec.add_layer_norm(y[:64].view(4, 16), v, residual=x, H=y[8:72].view(4, 16))


def test_add_layer_norm_backward():
    import torch
    import orthogonal_equivalence_cayley_amd as oec
    x, mats, v, vecs, r, rows = tensors()
    good = dict(G_Y=x, H=x.clone(), weight=v, mean=r, rstd=r.clone(), G_H=x.clone(), p=0.3, seed=1, site=2, G_X=x.clone(),
                G_R=x.clone())
    refused(oec.add_layer_norm_backward, good, dict(rules(), H=mats, weight=vecs, mean=rows, rstd=rows, G_H=mats, G_X=mats,
                                                    G_R=mats, G_Y=[x.half(), x.double(), x.cpu(), x[0]]))
    # a second gradient goes with dropout alone
    for p in (0.0, 2.0 ** -18):
        with pytest.raises(ValueError):
            oec.add_layer_norm_backward(**{**good, "p": p})
    for bad in (dict(G_X=good["H"]), dict(G_X=good["G_R"]), dict(G_R=good["H"])):
        with pytest.raises(oec.poetx.PoetxError):
            oec.add_layer_norm_backward(**{**good, **bad})
    with pytest.raises(oec.poetx.PoetxError):
        oec.add_layer_norm_backward(**{**good, "G_X": torch.as_strided(good["H"], (4, 16), (16, 1), 0)})
