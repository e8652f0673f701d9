"""Phases of the attention over drafted trees of many rows: an issuer of scores that has
no tile in a segment still waits for its queries, and nothing may get a phase ahead of it."""
import os
import re

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "block_sparse_masked_mask_gb300", "csrc")


def issuer_ends(places, frees_behind, ring, segments, late):
    """Segments of one tile and up to 128 rows, in steps: the softmax brings the queries of a segment as soon as
    it is handed out, which the issuer's freeing of the one `ring` before allows; the issuer, `late` steps behind
    each, sees a phase by its parity alone.  Whether it gets through all of them; none is passed early."""
    ended = [0] * places  # phases of each barrier
    brought = copied = seen = ready = 0
    for step in range((segments + 1) * (late + 4)):
        if brought < segments and (brought < ring or (seen if frees_behind else copied) > brought - ring):
            ended[brought % places] += 1
            brought += 1
        if copied == seen and copied < min(segments, brought + ring):
            copied, ready = copied + 1, step + late
        elif copied > seen and step >= ready and ended[seen % places] % 2 != seen // places % 2:
            assert ended[seen % places] > seen // places
            seen += 1
    return seen == segments


def test_what_goes_wrong_without_places_of_their_own():
    assert issuer_ends(1, False, 4, 1, 0)
    assert not issuer_ends(1, False, 4, 2, 0) and not issuer_ends(1, False, 4, 12, 9)
    assert not issuer_ends(1, True, 4, 3, 2)


def test_no_phase_gets_ahead_of_an_idle_issuer():
    """The model above with the numbers of the kernel's source."""
    code = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "cache_tree_many.cu")).read())
    ring = int(re.search(r"\bNSEG = (\d+)", code).group(1))
    places = ring if re.search(r"\bB_KFULL = B_Q \+ 2 \* NSEG\b", code) else 1
    issuer = code[code.index("warp < C::ISSUE_O"):code.index("warp == C::ISSUE_O)", code.index("warp < C::ISSUE_O"))]
    waits = [m.start() for m in re.finditer(r"tree_wait\(bar\(C::(B_Q|queries)\b", issuer)]
    frees = [m.start() for m in re.finditer(r"mbar_arrive\(bar\(C::B_SEGFREE", issuer)]
    assert len(waits) == 2
    behind = len(frees) == 1 and frees[0] > max(waits)
    for segments in range(1, 14):
        for late in (0, 1, 2, 3, 9):
            assert issuer_ends(places, behind, ring, segments, late), (segments, late)


@pytest.mark.gpu
@pytest.mark.parametrize("most", [100, 700])
def test_a_late_issuer_of_the_second_tile(most):
    """A build whose second issuer is 30 us late in every segment: no wait runs out, and results are
    the ordinary build's."""
    import torch

    from block_sparse_masked_mask_gb300 import _native, api
    from block_sparse_masked_mask_gb300 import build as B
    from test_cache_gpu import cu_of, dev, filled, randn
    from test_tree_gpu import check_tree, device_bits, trees
    from oracle import tree as R
    batch, heads, group = 152, 8, 4  # eight segments for each SM
    n = [17 + 5 * b % 17 for b in range(batch)]
    lens = [x + 37 * b % most for b, x in enumerate(n)]
    p = filled(lens, heads, 64, 32, seed=1)
    cu, q, masks = cu_of(n), randn(sum(n), heads * group, 64, seed=2), trees(n)
    want = [x.clone() for x in check_tree(p, q, cu, lens, masks)]
    args = (q.cuda(), p.dev, device_bits(R.to_bits(masks, 2)), dev(cu), dev(lens), max(n), max(lens))
    torch.cuda.synchronize()
    with _native.use_library(B.build_variant("late", {"ATTN_TREE_LATE_NS": "30000ull"})):
        for _ in range(3):
            got = api.attn_cache_tree_fwd(*args)
            assert api.attn_cache_get_status(p.dev) == api.ATTN_OK
            assert all(torch.equal(a, b) for a, b in zip(want, got))
