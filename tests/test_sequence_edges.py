"""The sequence operators where values, sizes or streams are out of the ordinary:
sums of very different size, infinities, memory of another stream, sizes near
2^31, outputs that overlap what a call reads."""
import pytest

torch = pytest.importorskip("torch")

import sequence_reference as ref  # noqa: E402
import sparse_weight_direct_gb300 as swd  # noqa: E402
from test_sequence import BF16, F16, F32, TYPE_IDS, TYPES, Draw  # noqa: E402

# ------------------------------------------------------------------ adapters: sums of very different size


def adapter_bound(y, x, a, b, index):
    """ref.adapter with the inner sums held in 32 bits for every type: sums of C
    and R terms within n 2^-24 of their absolute terms, products within E."""
    want, _ = ref.adapter(y, x, a, b, index, None)
    bound = 2.0 ** -23 * ref.f64(y).abs()
    K, R, C = a.shape
    for n, i in enumerate(index.tolist()):
        terms = ref.f64(b[i]).abs() @ (ref.f64(a[i]).abs() @ ref.f64(x[n]).abs())
        bound[n] += ((C + R) * 2.0 ** -24 + ref.E) * terms
    return want, bound


@pytest.mark.gpu
@pytest.mark.parametrize("P", [1, 2, 40, 64])
@pytest.mark.parametrize("R", [8, 32, 63])
@pytest.mark.parametrize("apart", [10, 15, 20])
@pytest.mark.parametrize("dtype", TYPES, ids=TYPE_IDS)
def test_adapter_small_sums_beside_large_ones(dtype, apart, R, P):
    """Adapters joined along the rank: half of a's rows are 2^apart larger, and
    half of the outputs read the other half only.  Those outputs are as good as
    without the large rows."""
    d = Draw(31)
    N, C, M = 2, 48, 40
    x = d(N, C, P, dtype=dtype)
    a, b = d(1, R, C, scale=C ** -0.5), d(1, M, R)
    a[:, : R // 2] *= 2.0 ** (apart / 2)
    a[:, R // 2:] *= 2.0 ** (-apart / 2)
    b[:, M // 2:, : R // 2] = 0
    b[:, : M // 2, R // 2:] = 0
    a, b, y = a.to(dtype), b.to(dtype), torch.zeros(N, M, P, dtype=dtype, device="cuda")
    index = torch.zeros(N, dtype=torch.int32)
    out = swd.adapter_add(y, x, a, b, index.cuda())
    ref.check(out, *adapter_bound(y, x, a, b, index), "out")


@pytest.mark.gpu
@pytest.mark.parametrize("P", [1, 2, 40, 64])
@pytest.mark.parametrize("R", [16, 30, 64])
@pytest.mark.parametrize("dtype", TYPES, ids=TYPE_IDS)
def test_adapter_differences_of_large_whole_sums(dtype, R, P):
    """b takes the difference of two rows of v, whole numbers of up to 20 bits
    that are nearly alike: every product and sum is exact in 32 bits, so v has
    to keep all of its bits between the products."""
    g = torch.Generator().manual_seed(32)
    ints = lambda most, *s: torch.randint(-most, most + 1, s, generator=g).to(dtype).cuda()  # noqa: E731
    N, C, M = 2, 32, 24
    x, a = ints(200, N, C, P), ints(200, 1, R, C)
    x[:, 0], a[:, :, 0] = ints(9, N, P), ints(9, 1, R)
    a[:, R // 2:] = a[:, : R // 2]
    a[:, R // 2:, 0] += ints(9, 1, R // 2)
    b = torch.zeros(1, M, R, dtype=dtype, device="cuda")
    for m in range(M):
        b[0, m, m % (R // 2)], b[0, m, R // 2 + m % (R // 2)] = 1, -1
    y = ints(20, N, M, P)
    index = torch.zeros(N, dtype=torch.int32)
    want, _ = ref.adapter(y, x, a, b, index, None)
    v = ref.f64(a[0]) @ ref.f64(x[0])
    assert float(v.abs().max()) >= 1 << 16 and float(want.abs().max()) <= 256
    out = swd.adapter_add(y, x, a, b, index.cuda())
    assert torch.equal(out.cpu().double(), want)
