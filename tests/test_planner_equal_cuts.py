"""Equal cuts of rows whose parts are shorter than a page: every part of a split row exists, so
that the merge that counts them runs."""
import numpy as np
import pytest
import torch

import workloads as W
from test_host import _check_partition


@pytest.fixture(scope="module", autouse=True)
def pkd():
    from paged_kv_decode_23_gb300 import build
    build.build()


@pytest.mark.parametrize("page", [128, 256])
@pytest.mark.parametrize("window", [-1, 200, 300])
def test_split_rows_have_all_their_parts(page, window):
    from paged_kv_decode_23_gb300 import plan_host
    for lens in [[n] for n in range(page, 4 * page, 7)] + [[300, 2 * page + 1], [page + 1, page + 44, 600, 5]]:
        w = W.custom(lens, 8, 8, 128, page, window_left=window)
        plan = plan_host(w.indptr, w.last_page_len, 8, 8, 128, page, window_left=window)
        _check_partition(w, plan, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("page,lens", [(256, [300]), (256, [514]), (128, [129, 200])])
def test_decode_of_rows_a_little_longer_than_a_page(page, lens):
    from helpers import assert_close, run_gpu, run_oracle
    w = W.custom(lens, 8, 8, 128, page, q_dtype="bf16", seed=3)
    q, pool = W.make_q(w), W.make_pool(w)
    assert_close(w, run_gpu(w, q, pool), run_oracle(w, q, pool))
