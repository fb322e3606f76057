"""From how many rows per expert the weight gradients take the kernel for many
rows, seen from the workspace: only that kernel has copies of the rows there.
Where f is narrow or the experts' weights are few the copies pay from 512 rows in
the mean on, otherwise from 256."""
import os

import pytest

import expert_grouped_gemm_amd as moe


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not os.path.exists(moe.LIB_PATH):
        from expert_grouped_gemm_amd import build
        build.build()


# experts, top-k, d, f, rows per expert in the mean, whether the rows are copied
CASES = [(1, 1, 512, 512, 264, False), (8, 2, 2048, 1024, 264, False), (8, 2, 2048, 1024, 512, False),
         (8, 2, 2048, 1024, 516, True), (16, 2, 2048, 1024, 400, False), (32, 4, 1024, 512, 384, False),
         (64, 4, 4096, 512, 512, False), (64, 4, 4096, 512, 528, True), (64, 4, 4096, 640, 272, True),
         (12, 2, 2048, 2048, 252, False), (12, 2, 2048, 2048, 264, True), (11, 1, 2048, 2048, 264, False),
         (8, 2, 4096, 14336, 256, False), (8, 2, 4096, 14336, 260, True), (1, 1, 128, 128, 512, False),
         (1, 1, 128, 128, 513, True)]


@pytest.mark.parametrize("E,k,d,f,rows,copied", CASES)
def test_copies_in_the_workspace(E, k, d, f, rows, copied):
    T = rows * E // k
    assert T * k == rows * E
    p = moe.make_problem(T, d, f, E, k)
    cap = moe.row_capacity(p)
    inner = moe.backward_workspace_size(p) - moe.workspace_size(p)
    base = cap * (4 * 2 * f + 2 * f + 2 * 2 * f)  # gate and up in fp32, a, dh
    assert 0 <= inner - base - (2 * cap * d * 2 if copied else 0) <= 5 * 256
    from_checkpoint = moe.checkpoint_workspace_size(p) - moe.workspace_size(p)
    assert 0 <= from_checkpoint - cap * (2 * f + 4 * f + 2 * d) - (cap * d * 2 if copied else 0) <= 5 * 256
