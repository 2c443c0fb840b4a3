"""The calls for prompts at the ends of their ranges: sequences without rows."""
import pytest

from paged_cases import Cache
from test_gpu_prompts import Prompt, Rope, _room

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------------------ sequences without rows
def test_first_rows_of_sequences_without_rows_are_not_looked_at():
    lens, live = [40, 50, 20, 60, 0], [4, 0, 3, 0, 0]
    c = Cache(101, [36, 50, 17, 60, 0], 2, "e4m3", spare=20)
    _room(c, lens)
    r = Rope(c, live, 2, 128, False, gap=1)
    for b, x in ((1, -1), (3, r.tokens + 1), (4, 2 ** 31 - 1)):
        r.args[0][b] = x
    assert r.call() == 0
    r.check()
    p = Prompt(c, live, 2, gap=1)
    for b, x in ((1, -2 ** 31), (3, p.tokens + 1), (4, 2 ** 31 - 1)):
        p.ints[0][b] = x
    p.call()
    p.check()
