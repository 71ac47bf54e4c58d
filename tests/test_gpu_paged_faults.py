"""What goes wrong in the paged calls is reported and ends: negative pages in what a plan is given, waits that
run out in every way that decode brings its tiles."""
import pytest
import torch

import exact_headdim_attention_gb300 as pkg
from tests.gpu_util import device_ok
from tests.test_gpu_paged import check_decode, decode_case

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def plan(table, old, new, free, count, page, tokens):
    word = torch.zeros(1, dtype=torch.int32, device=DEV)
    t = torch.tensor(table, dtype=torch.int32, device=DEV)
    got = pkg.ffpa_page_plan(t, ints(*old), ints(*new), ints(*free), ints(count), page, tokens, status=word)
    return word.item(), t.tolist(), [x.tolist() for x in got]


@pytest.mark.parametrize("bad", [-1, -7, -2 ** 31])
def test_negative_page_of_the_free_list(bad):
    """Pages come off the end: request 0 takes 9, the bad one and 8, request 1 takes 6."""
    word, table, (slots, pos, cu, lens, left) = plan([[-1] * 4, [5, -1, -1, -1]], [0, 3], [9, 3], [7, 6, 8, bad, 9], 5, 4, 13)
    assert word == pkg.FFPA_ERR_INVALID
    assert table == [[9, bad, 8, -1], [5, 6, -1, -1]]
    assert slots == [36, 37, 38, 39, -1, -1, -1, -1, 32, 23, 24, 25, -1]
    assert pos == [0, 1, 2, 3, 4, 5, 6, 7, 8, 3, 4, 5, 0] and cu == [0, 9, 12] and lens == [9, 6] and left == [1]
    device_ok()


def test_negative_page_that_the_table_holds():
    """In the page that the request goes on filling it is reported; where no new token falls it is not looked at."""
    word, table, (slots, _, _, lens, left) = plan([[3, -1, -1, -1], [-1, 5, -1, -1]], [6, 6], [3, 1], [7, 8], 2, 4, 4)
    assert word == pkg.FFPA_ERR_INVALID
    assert table == [[3, -1, 8, -1], [-1, 5, -1, -1]] and slots == [-1, -1, 32, 22] and lens == [9, 7] and left == [1]
    word, _, (slots, _, _, _, _) = plan([[3, -1, -1, -1], [-1, 5, -1, -1]], [6, 6], [0, 1], [7, 8], 2, 4, 1)
    assert word == pkg.FFPA_OK and slots == [22]
    device_ok()


def test_negative_pages_are_not_reported_where_none_is_taken():
    """Entries of the list behind free_count, and free pages that the step does not need, may be anything."""
    word, _, (slots, _, _, _, left) = plan([[-1] * 2], [0], [4], [-1, -1, 2, -1], 3, 4, 4)
    assert word == pkg.FFPA_OK and slots == [8, 9, 10, 11] and left == [2]
    device_ok()


MOST = 2 ** 31 - 1


@pytest.mark.parametrize("new", [(MOST, 3), (MOST, MOST), (9, MOST)])
def test_plan_of_lengths_beyond_any_table_is_short(new):
    """The work goes by the step's rows and the table's pages, not by what the lengths name (a loop over
    2^31 tokens would take seconds)."""
    start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    plan([[7, -1, -1], [-1] * 3], [2, 0], [1, 1], [1, 2, 3, 4, 5], 5, 4, 6)          # (the kernel is loaded)
    start.record()
    word, table, (slots, pos, cu, lens, left) = plan([[7, -1, -1], [-1] * 3], [2, 0], new, [1, 2, 3, 4, 5], 5, 4, 6)
    stop.record()
    torch.cuda.synchronize()
    assert start.elapsed_time(stop) < 100
    assert word == pkg.FFPA_ERR_INVALID
    assert slots == [30, 31, 20, 21, 22, 23] and pos == [2, 3, 4, 5, 6, 7] and cu == [0, 6, 6]
    pages = {3: 1, MOST: 3}[new[1]]                       # of request 1, from what request 0 left
    assert table == [[7, 5, 4], [3, 2, 1][:pages] + [-1] * (3 - pages)]
    assert lens == [12 if new[0] == MOST else 11, min(new[1], 4 * pages)] and left == [3 - pages]
    device_ok()


def test_plan_with_fewer_rows_than_tokens_still_enters_every_page():
    """Pages that begin behind the last row, of requests in and behind it, each once."""
    word, table, (slots, _, cu, lens, left) = plan([[-1] * 40, [6] + [-1] * 39, [-1] * 40], [0, 3, 0], [70, 50, 9],
                                                   list(range(100, 200)), 100, 2, 21)
    assert word == pkg.FFPA_ERR_INVALID and cu == [0, 21, 21, 21] and lens == [70, 53, 9]
    free = list(range(199, 99, -1))
    want = [free[:35], [6, -1] + free[35:60], free[60:65]]
    for row, pages in zip(table, want):
        assert row == pages + [-1] * (40 - len(pages))
    assert slots == [free[t // 2] * 2 + t % 2 for t in range(21)] and left == [35]
    device_ok()


@pytest.mark.parametrize("Hq,Hkv", [(4, 2), (16, 1), (20, 1)])
@pytest.mark.parametrize("D,page", [(64, 3), (512, 3), (512, 100), (1000, 20), (200, 16), (72, 100), (256, 16)])
def test_decode_ends_when_a_wait_runs_out(D, page, Hq, Hkv):
    """A copy that never starts, in pieces (pages of 3), in boxes that end with their page (100, 20), in boxes of
    one chunk (D = 200, 72) and in whole ones: the timeout status after the call's limit, and a whole next call."""
    args, ref = decode_case([300, 20, 0, 900], Hq, Hkv, D, page, torch.bfloat16, seed=D + page)
    word = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkg.ffpa_decode_paged(*args, enable_gqa=True, status=word, wait_timeout_ns=3_000_000, test_drop_first_copy=True)
    torch.cuda.synchronize()
    assert word.item() == pkg.FFPA_ERR_DEVICE_TIMEOUT
    check_decode(args, ref)
    device_ok()
