"""Pages that leave every window of forked sequences: the room they make is
room for the step that gives them up (attn_engine.JetAttnEngine, on the CPU
with stand-ins for the library's calls)."""
import pytest

from test_attn_engine_cpu import Texts, consistent, make  # noqa: F401


def forked(make, n_pages, at, children=("b",)):  # noqa: F811
    e = make(n_pages=n_pages, windows=[16, 16])
    t = Texts(e)
    e.admit("a")
    for i in range(0, at, 16):                   # in pieces, so that no step needs more than a page beside its window
        t.step({"a": min(16, at - i)})
    t.fork("a", list(children))
    return e, t


def test_forks_that_leave_a_page_together_make_room_for_their_step(make):  # noqa: F811
    e, t = forked(make, 3, 32)                   # both hold pages 0 and 1 of the text, one page is free
    assert e.free_pages == 1
    t.step({"a": 1, "b": 1})                     # two new pages: the free one, and page 0, which both give up
    consistent(e)
    assert e.free_pages == 0


def test_forks_of_a_prompt_taken_at_once(make):  # noqa: F811
    e = make(n_pages=8, windows=[16, 16])
    t = Texts(e)
    e.admit("a")
    t.step({"a": 96})
    t.fork("a", ["b"])                           # six pages that both hold, two free
    t.step({"a": 32, "b": 32})                   # four new ones; five are given up
    consistent(e)
    assert e.free_pages == 3


def test_a_refused_step_still_gives_up_what_nobody_will_see(make):  # noqa: F811
    e, t = forked(make, 2, 32)                   # pages 0 and 1 shared, none free
    with pytest.raises(RuntimeError):            # page 0 is still the other's
        e.begin({"a": 1})
    consistent(e)
    assert e.len["a"] == 32
    t.step({"b": 1})                             # now the last holder gives it up, and takes it
    consistent(e)
    t.release("b")
    t.step({"a": 1})
    consistent(e)


def test_a_step_that_is_too_long_changes_nothing(make):  # noqa: F811
    e, t = forked(make, 4, 48)
    held = e._ref.copy()
    with pytest.raises(ValueError):
        e.begin({"a": 1, "b": 10000})
    with pytest.raises(ValueError):
        e.begin({"a": 1, "b": 0})
    assert (e._ref == held).all()
    consistent(e)


def test_three_beams_to_the_end_of_their_room(make):  # noqa: F811
    """Beams that advance together need one page more each than a window's span, whatever they shared before."""
    e, t = forked(make, 6, 32, ("b", "c"))
    for _ in range(100):
        t.step({"a": 1, "b": 1, "c": 1})
        consistent(e)
