"""GPU tests of differential attention over a paged cache on the paths that a call's size or
layout chooses, against float64: scores of any size, many short sequences, long chunks,
queries and outputs that the wide copies do not take."""
import pytest
import torch

import differential_attention_fwd_gb300 as da
from differential_attention_fwd_gb300 import build as build_mod
from tests import paged_reference as ref
from tests.test_gpu_paged import HEADS, LAM, Problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build_mod.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.fixture(autouse=True)
def _clean():
    da.get_device_error()
    yield
    assert da.get_device_error() == 0


def put_keys(pb):
    """Writes pb.k1 and pb.k2 into the caches again."""
    for b in range(len(pb.lens)):
        for cache, rows in ((0, pb.k1[b]), (1, pb.k2[b])):
            for t in range(0, rows.shape[1], pb.page):
                part = rows[:, t:t + pb.page]
                pb.caches[cache][int(pb.table[b, t // pb.page]), :, :part.shape[1]] = part.cuda()


@pytest.mark.parametrize("head", HEADS)
@pytest.mark.parametrize("Tq,tree", [(1, False), (6, True), (20, False), (40, True)])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("size", [12, 15, 16, 17, 53])
@pytest.mark.parametrize("qf,kf", [(1.0, 1.0), (1 + 45 / 128, 1 + 91 / 128)])
def test_scores_of_any_size(head, Tq, tree, sign, size, qf, kf):
    """Queries of qf 2^size and keys of sign kf 2^size or twice that: of the two scores, 2^(2 size) and
    more apart and both exact, the higher one's keys share a weight of 1 and the others have none,
    exactly (from 2^24 on, where an exponential is 0).  A score times the scale is a float32 for the
    first pair of factors and not for the second."""
    pb = Problem(*head, 2, 1, Tq, [300, 33, 900], 16, tree=tree)
    g = torch.Generator().manual_seed(size)
    pb.q1.fill_(qf * 2.0 ** size)
    pb.q2.fill_(qf * 2.0 ** size)
    for ks in (pb.k1,) if pb.shared else (pb.k1, pb.k2):
        for k in ks:
            level = 1 + torch.randint(0, 2, (k.shape[0], k.shape[1], 1), generator=g)
            k.copy_((sign * kf * 2.0 ** size * level).expand(k.shape))
    put_keys(pb)
    out = pb.run().cpu().double()
    h = ref.half_step(pb.dtype)
    for b, head_, o, _ in pb.want():
        # weights of 0 and 1: what is left is the sums (n terms), a division and a few roundings of
        # the means of |v|, at most max|v|, and the result's
        n = pb.lens[b] + Tq
        top = (1 + LAM) * pb.v[b][0].double().abs().amax(0)
        got = out[b, head_, :o.shape[0]]
        assert torch.isfinite(got).all(), (b, head_)
        over = (got - o).abs() - (h * o.abs() + (1 + h) * ref.U * (n + 8) * top)
        assert over.max() <= 0, (b, head_)
