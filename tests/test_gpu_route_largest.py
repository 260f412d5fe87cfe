"""The sort by expert next to its limit, T * k just below 2^31."""
import os

import pytest

import gemv_fp16_amd as gf

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("T,E,k", [(2 ** 28 - 1, 4, 8), (2 ** 30 - 1, 1, 2), (2 ** 24 - 1, 1024, 128), (2 ** 25 - 1, 64, 64),
                                   (2 ** 31 - 1, 2, 1), (2147483647 // 3, 7, 3), (1, 8, 2 ** 31 - 1), (2 ** 20, 16, 2047)])
def test_workspace(T, E, k):
    if not os.path.exists(gf.LIB_PATH):
        from gemv_fp16_amd import build
        build.build()
    n = T * k
    assert 2 ** 31 - 2 ** 21 <= n < 2 ** 31
    chunks = -(-n // 65535)                # of entries, their counts held in 16 bits
    assert 2 * E * chunks <= gf.route_workspace_bytes(T, E, k) <= 4 * E * (chunks + 4096)


@pytest.mark.gpu
def test_rows_of_the_most_entries():
    """T * k = 2^31 - 8 choices, in a pattern whose places are known."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    T, E, k = 2 ** 28 - 1, 4, 8
    n, part = T * k, 1 << 26
    ids = torch.empty((T, k), dtype=torch.int32, device="cuda")
    flat = ids.view(-1)
    for i in range(0, n, part):            # 3 2 1 0, or 0 1 2 3 where bit 20 is set
        at = torch.arange(i, min(i + part, n), device="cuda")
        flat[i:i + part] = (3 - at) % 4 ^ torch.where(at >> 20 & 1 == 1, 3, 0)
    print("sort", T, k, E, flush=True)
    offsets, place = gf.route_rows(ids, E)
    assert offsets.tolist() == [e * (n // 4) for e in range(5)]
    place = place.view(-1)
    for i in range(0, n, part):            # every four choices name each expert once
        at = torch.arange(i, min(i + part, n), device="cuda")
        assert torch.equal(place[i:i + part].long(), flat[i:i + part].long() * (n // 4) + at // 4), i
