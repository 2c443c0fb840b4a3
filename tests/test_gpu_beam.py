"""Beam search's selection against the oracle (oracle/paged.py)."""
import numpy as np
import pytest
import torch

import oracle.paged as P
import speculative_decode_verify_gb300 as va

pytestmark = pytest.mark.gpu


def _select(logits, scores, beams, k, finished=None, end=0, ws=None):
    groups = logits.shape[0] // beams
    pa, tk = (torch.full((groups, k), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    sc = torch.full((groups, k), float("nan"), device="cuda")
    if ws is None:
        ws = torch.zeros(va.va_beam_workspace_bytes(groups, beams, logits.shape[1], k), dtype=torch.uint8, device="cuda")
    fin = None if finished is None else torch.tensor(finished, dtype=torch.int32, device="cuda")
    va.va_beam_select(logits, torch.tensor(scores, dtype=torch.float32, device="cuda"), beams, pa, tk, sc, ws,
                      finished=fin, end_token=end)
    return pa, tk, sc


def _check(logits, scores, beams, k, finished=None, end=0, ws=None):
    got = _select(logits, scores, beams, k, finished, end, ws)
    s32 = np.asarray(scores, np.float32).astype(np.float64)
    pa, tk, sc, gap = P.beam_select(logits.double().cpu().numpy(), s32, beams, k, finished, end)
    # a row's sum of exponentials is right to 2^-18 (fp32 sums of at most 8,192 terms of 2^-22 accuracy each, in
    # trees of 32 + 5 + 8 additions), so candidates of different hypotheses that far apart keep their order
    assert gap > 2.0 ** -17
    assert got[0].tolist() == pa.tolist() and got[1].tolist() == tk.tolist()
    have = got[2].double().cpu().numpy()
    some = np.isfinite(sc)
    assert np.array_equal(some, np.isfinite(have)) and np.array_equal(have[~some], sc[~some])
    assert np.all(np.abs(have[some] - sc[some]) <= 2.0 ** -18 + 2.0 ** -24 * np.abs(sc[some]))
    return got


def _rows(seed, rows, vocab, dtype, spread=2.5, pad=8):
    g = torch.Generator(device="cuda").manual_seed(seed)
    wide = -(-vocab // 8) * 8 + pad
    x = torch.full((rows, wide), float("nan"), device="cuda", dtype=dtype)    # what lies between rows is not used
    x[:, :vocab] = (torch.randn(rows, vocab, generator=g, device="cuda") * spread).to(dtype)
    return x[:, :vocab]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("groups,beams,vocab,k", [(1, 1, 1, 1), (1, 1, 7, 7), (2, 3, 5, 32), (3, 4, 1000, 4), (1, 2, 8192, 5),
                                                  (2, 4, 8193, 8), (2, 8, 50001, 16), (1, 32, 3001, 32), (40, 2, 300, 3),
                                                  (1, 3, 262144, 32)])
def test_selection(dtype, groups, beams, vocab, k):
    rng = np.random.default_rng(vocab)
    _check(_rows(vocab + k, groups * beams, vocab, dtype), -5 + rng.standard_normal(groups * beams), beams, k)


def test_finished_and_missing_hypotheses():
    x = _rows(3, 12, 4000, torch.float32)
    scores = [-1.0, -2.0, -np.inf, -0.5] + [0.0, -np.inf, -np.inf, -np.inf] + [-3.0, -3.5, -3.25, -np.inf]
    _check(x, scores, 4, 6, finished=[0, 1, 0, 0] + [0, 0, 0, 0] + [1, 1, 1, 1], end=7)
    _check(x, [-np.inf] * 12, 4, 6)
    _check(x, [np.nan, -1, -2, -3] * 3, 4, 6, finished=[0, 0, 1, 0] * 3, end=3999)


def test_masked_infinite_and_nan_logits():
    x = _rows(4, 6, 9000, torch.float32, pad=0).clone()
    x = torch.nn.functional.pad(x, (0, 8 - 9000 % 8 if 9000 % 8 else 0)).contiguous()[:, :9000]
    x[0, 5:] = -np.inf                                     # five candidates
    x[1] = -np.inf                                         # none
    x[2, ::2] = float("nan")
    x[3, 100] = x[3, 8500] = np.inf                        # share the probability
    x[4, :8192] = -np.inf
    x[5] = torch.finfo(torch.float32).min                  # the type's lowest value is a value like another
    for row in range(6):
        _check(x[row:row + 1], [-1.0], 1, 8)
    _check(x, [-1.0, -2.0, -1.5, -40.0, -0.25, -30.0], 6, 20)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab,stride", [(5, 5), (50257, 50257), (9001, 1), (8193, 0)])
def test_a_single_rows_stride_does_not_matter(dtype, vocab, stride):
    x = _rows(vocab, 1, vocab, dtype).clone()
    _check(x.as_strided((1, vocab), (stride, 1)), [-1.0], 1, 4)
    with pytest.raises(va.VerifyAttnError):
        _select(_rows(vocab, 2, vocab, dtype).contiguous().as_strided((2, vocab - 1), (vocab, 1)), [-1.0, -2.0], 2, 2)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", ["one", "constant", "peaked"])
@pytest.mark.parametrize("top", [-720, 24, 96, 360, 720, 1016, 2032])
def test_a_rows_offset_does_not_move_its_scores(dtype, shape, top):
    """Two hypotheses of the same distribution, one with logits near 0 and one far from it; their scores are 1e-5 apart.
    The largest terms of a sum are 2^0 (exact) and the others e^-8 and less, so a sum is right to 2^-22 (the
    exponential's accuracy) times 2^-11, and the constant row's is a whole number; the log's 64 bits and the one rounding
    of the score (2^-24) add to that.  2^-21 holds them all."""
    vocab = 20000
    x = torch.full((4, vocab + 96), float("nan"), device="cuda", dtype=dtype)[:, :vocab]
    for row, far in ((0, top), (1, 8), (2, 8), (3, top)):
        x[row] = far if shape == "constant" else far - 40
        x[row, 9000 + row] = far
        if shape == "peaked":
            x[row, 50], x[row, 19999] = far, far - 8
    scores = [-1.0, -1.00001, -2.0, -1.99999]
    got = _check(x, scores, 2, 2)
    want = P.beam_select(x.double().cpu().numpy(), np.asarray(scores, np.float32).astype(np.float64), 2, 2)[2]
    assert np.all(np.abs(got[2].double().cpu().numpy() - want) <= 2.0 ** -21 + 2.0 ** -24 * np.abs(want))


def test_equal_logits_go_to_the_lowest_token_and_hypothesis():
    x = torch.zeros(4, 20000, device="cuda")
    pa, tk, _ = _select(x, [-1.0, -1.0, -1.0, -2.0], 4, 32)
    assert pa.tolist() == [[0] * 32] and tk.tolist() == [list(range(32))]
    x[:, 17777] = 1.0
    x[2, 3] = 1.0
    pa, tk, _ = _select(x[:2].contiguous(), [-1.0, -1.0], 2, 4)
    assert pa.tolist() == [[0, 1, 0, 0]] and tk.tolist() == [[17777, 17777, 0, 1]]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("finished", [None, "some", "all"])
def test_runs_of_many_tiles(dtype, finished):
    """2,080 tiles: several a CTA, over the ends of rows.  Rows whose every tile beats the one before (more candidates
    than are kept), fall, are constant, have few values or only their last ones; finished rows among them."""
    rows, vocab, beams, k = 160, 100001, 5, 12
    rng = np.random.default_rng(8)
    x = _rows(9, rows, vocab, dtype)
    for i, row in enumerate(rng.permutation(rows)[:40].tolist()):
        line = torch.linspace(-6, 6, vocab, device="cuda")
        x[row] = (line, -line, 0 * line + 1.5, (line * 0.5).round(), torch.where(line > 5.9999, line, -np.inf))[i % 5].to(dtype)
    fin = None
    if finished:
        fin = (rng.random(rows) < 0.4).astype(np.int32) if finished == "some" else np.ones(rows, np.int32)
        fin[35:40], fin[40:45] = 1, fin[40:45] if finished == "all" else 0
        fin = fin.tolist()
    _check(x, -5 + rng.standard_normal(rows), beams, k, finished=fin, end=4)


@pytest.mark.parametrize("finished", [[0, 0, 1, 0], [1, 0, 0, 0], [1, 1, 0, 1], [0, 1, 0, 1]])
def test_fewer_tiles_than_ctas_once_rows_are_finished(finished):
    rng = np.random.default_rng(5)
    ws = torch.zeros(va.va_beam_workspace_bytes(2, 4, 160000, 8), dtype=torch.uint8, device="cuda")
    for groups, vocab in ((1, 160000), (2, 40000), (1, 160000)):
        _check(_rows(vocab + groups, 4 * groups, vocab, torch.bfloat16), -5 + rng.standard_normal(4 * groups), 4, 8,
               finished=finished * groups, end=2, ws=ws)


def test_more_rows_than_ctas():
    rng = np.random.default_rng(2)
    fin = (rng.random(3000) < 0.5).astype(np.int32).tolist()
    _check(_rows(11, 3000, 50, torch.float32), -5 + 0.5 * rng.permutation(3000), 3, 4, finished=fin, end=49)


def test_one_workspace_for_every_shape_and_a_captured_call():
    ws = torch.zeros(va.va_beam_workspace_bytes(6, 8, 60000, 32), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(1)
    for groups, beams, vocab, k in ((6, 8, 60000, 32), (1, 2, 30, 3), (5, 3, 20000, 9), (6, 8, 60000, 4)):
        _check(_rows(vocab, groups * beams, vocab, torch.bfloat16), -4 + rng.standard_normal(groups * beams), beams, k, ws=ws)
    x = _rows(5, 8, 16000, torch.float32)
    scores = torch.linspace(-3, -1, 8, device="cuda")
    pa, tk = (torch.zeros(2, 4, dtype=torch.int32, device="cuda") for _ in range(2))
    sc = torch.zeros(2, 4, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        va.va_beam_select(x, scores, 4, pa, tk, sc, ws)
    for seed in range(3):
        x.copy_(_rows(50 + seed, 8, 16000, torch.float32))
        graph.replay()
        want = P.beam_select(x.double().cpu().numpy(), scores.double().tolist(), 4, 4)
        assert want[3] < 2.0 ** -17 or (pa.tolist() == want[0].tolist() and tk.tolist() == want[1].tolist())
