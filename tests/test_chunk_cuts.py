"""The cases of cut items are what they stand for on a GPU of 152 SMs, worked out without one."""
import pytest

from chunk_cuts import CASES, pieces


def cut(name, blocks=152):
    reqs, hq, hkv, causal, window = CASES[name]
    return pieces(reqs, hkv, hq // hkv, blocks, causal, window)


@pytest.mark.parametrize("name", list(CASES))
def test_every_tile_once(name):
    for a, b, of in cut(name):
        assert [t for _, t0, t1 in of for t in range(t0, t1)] == list(range(a[0], max(a[1], b[1])))
        assert [c for c, _, _ in of] == list(range(of[0][0], of[-1][0] + 1))
    # no block begins two cut items, or ends two
    begun = [of[0][0] for _, _, of in cut(name) if len(of) > 1]
    ended = [of[-1][0] for _, _, of in cut(name) if len(of) > 1]
    assert len(set(begun)) == len(begun) and len(set(ended)) == len(ended)


def words(of):
    return len({c // 16 for c, _, _ in of})


def test_the_cases():
    assert words(cut("five words")[0][2]) == 5
    assert all(words(of) >= 2 for _, _, of in cut("several items"))
    assert any(words(of) == 2 for _, _, of in cut("not causal")) and any(words(of) == 2 for _, _, of in cut("beside others"))
    for name in ("both halves", "eight heads", "window", "window of eight heads", "not causal"):
        a, b, of = cut(name)[0]
        assert len(of) > 6 and a[0] < a[1] and b[0] < b[1]
    a, b, of = cut("a half alone")[0]
    assert of[0][1:] == [a[0], a[0] + 1] and b[0] > a[0]  # the first piece is one of A's tiles
    items = cut("beside others")
    assert all(len(of) > 1 for _, _, of in items[:31]) and len(items[-1][2]) == 1
