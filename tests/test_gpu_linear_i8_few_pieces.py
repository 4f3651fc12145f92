"""int8 product of few tokens over K of every count of 128-byte pieces around
its waves' turns and their rings' depth, whole and cut pieces, against exact
integer sums."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from orthogonal_equivalence_amd import model  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible AMD GPU"
    torch.cuda.init()


# n on both sides of the change to 64 outputs a workgroup; T on both sides of
# one and two sets of 32 tokens
@pytest.mark.parametrize("T,n", [(1, 48), (32, 272), (33, 272), (64, 80), (1, 8208), (32, 8208)])
def test_pieces_of_k(T, n):
    g = torch.Generator(device="cuda").manual_seed(T + n)
    one = torch.ones(max(T, n), device="cuda")
    for pieces in list(range(1, 18)) + [27, 32, 33]:
        for cut in (0, 16, 112):
            m = 128 * pieces - cut
            print(f"\n[gpu] linear_i8 T={T} n={n} m={m}", end="", flush=True)
            xq = torch.randint(-128, 128, (T, m), generator=g, device="cuda", dtype=torch.int8)
            wt = torch.randint(-128, 128, (n, m), generator=g, device="cuda", dtype=torch.int8)
            z = model.linear_i8(xq, one[:T], wt, one[:n], out_dtype=torch.float32)
            # sums below 2^27, products of at most 2^14: exact in float64, rounded once to float32
            want = (xq.double() @ wt.double().t()).float()
            assert torch.equal(z, want), (T, n, m)
