"""Long lists of expert ids, whose chunks' counts a kernel of its own adds up, against the stable sort."""
import numpy as np
import pytest

from test_gpu_route import S, make_ids, plain_sort  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,topk,E,kind", [
    (65536, 2, 300, "dropped"),        # 64 chunks: the most that blocks add up themselves
    (131073, 1, 33, "random"),         # one more
    (500000, 6, 64, "popular"), (1000003, 3, 2048, "dropped"), (400000, 8, 1, "one"), (3000000, 1, 31, "none"),
])
def test_sort_equals_the_stable_sort(S, T, topk, E, kind):
    import torch
    ids = make_ids(kind, T, topk, E)
    want = plain_sort(ids, E)
    for _ in range(2):
        got = S.route_sort(torch.from_numpy(ids).cuda(), E)
        for a, b in zip(got, want):
            assert np.array_equal(a.cpu().numpy(), b)
