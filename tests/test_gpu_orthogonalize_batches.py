"""sgemm_orthogonalize gives a matrix the same bits whatever batch it is in, and whatever tiles the
batch's size calls for."""
import numpy as np
import pytest

import dense_fp32_matrix_03_amd as sg
import orthogonalize_model as om

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    sg.sgemm_create()
    yield
    sg.sgemm_destroy()


def _run(X, steps=5):
    import torch
    B, M, N = X.shape
    Y = torch.empty_like(X)
    need = sg.sgemm_orthogonalize_workspace_size(B, M, N)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    kind = "f32" if X.dtype == torch.float32 else "bf16"
    sg.sgemm_orthogonalize(B, M, N, steps, om.STEP, 1e-7, 1.0, kind, X, N, M * N, kind, Y, N, M * N,
                           ws, need)
    return Y


# Some are on 64 x 64 tiles alone and on larger ones in a batch, some always on one or the other.
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,batch", [
    (512, 512, 16), (1024, 1024, 4), (1024, 1024, 9), (700, 515, 24), (300, 1100, 40), (129, 130, 200),
    (1500, 1001, 5), (40, 600, 50), (257, 4000, 7)])
def test_bits_do_not_depend_on_the_batch(M, N, batch, kind):
    import torch
    g = torch.Generator(device="cuda").manual_seed(M + N)
    X = torch.randn(batch, M, N, generator=g, device="cuda")
    X += 3 * torch.randn(batch, M, 1, generator=g, device="cuda")
    X = X.to(torch.float32 if kind == "f32" else torch.bfloat16)
    all_ = _run(X)
    for i in (0, 1, batch - 1):
        assert torch.equal(_run(X[i:i + 1].contiguous())[0], all_[i])
    half = max(2, batch // 2)
    assert torch.equal(_run(X[:half].contiguous()), all_[:half])
    assert torch.equal(_run(X), all_)  # and every call gives them
